"""Buffer accesses in the kernels' sources.  A raw buffer's bounds check covers
the vector offset and the instruction's immediate, not the scalar offset: an
access with a scalar offset can reach past the buffer's end by that much."""
import glob
import os
import re

import pytest

from logit_source_projection_amd import build

# index of the scalar offset among the arguments
SOFFSET = {"raw_buffer_load": 2, "raw_buffer_store": 3, "raw_ptr_buffer_load_lds": 4}
CALL = re.compile(r"__builtin_amdgcn_(raw_buffer_load|raw_buffer_store|raw_ptr_buffer_load_lds)(?:_b\d+)?\s*\(")


def accesses(text):
    """(builtin, its arguments, line) of every buffer access."""
    for m in CALL.finditer(text):
        depth, args, start, at = 1, [], m.end(), m.end()
        while depth:
            c = text[at]
            depth += (c in "([{") - (c in ")]}")
            if (c == "," and depth == 1) or depth == 0:
                args.append(text[start:at].strip())
                start = at + 1
            at += 1
        yield m.group(1), args, text.count("\n", 0, m.start()) + 1


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(build.CSRC, "*.hip")) +
                                        glob.glob(os.path.join(build.CSRC, "*.h"))))
def test_no_access_has_a_scalar_offset(path):
    for name, args, line in accesses(open(path).read()):
        assert args[SOFFSET[name]] == "0", f"{os.path.basename(path)}:{line}: {args}"


def test_the_parser_sees_the_accesses():
    text = "x = __builtin_amdgcn_raw_buffer_load_b128(r, f(a, b)[2], 64 * i, 0);"
    assert list(accesses(text)) == [("raw_buffer_load", ["r", "f(a, b)[2]", "64 * i", "0"], 1)]
    found = [n for p in glob.glob(os.path.join(build.CSRC, "*.h*")) for n, _, _ in accesses(open(p).read())]
    assert set(found) == set(SOFFSET)
