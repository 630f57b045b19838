"""Calls with a barrier inside, in the kernels' sources.  C++ leaves open in which
order the operands of an expression are evaluated, so what a barrier has to come
before (a read of shared memory, by an index) is a statement of its own."""
import glob
import os
import re

import pytest

from logit_source_projection_amd import build

HEAD = re.compile(r"(?:__device__[^;{}()]*?|\bauto\s+)\b(\w+)\s*(?:=\s*\[&\]\s*)?\(")
WORDS = ("__launch_bounds__", "if", "for", "while")


def closing(text, at, pair):
    """The place of the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i
    raise ValueError("no closing bracket")


def plain(text):
    """The source without comments, lines kept."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", lambda m: "\n" * m.group().count("\n"), text, flags=re.S)


def with_barrier(text):
    """Names of the functions and lambdas that wait for a barrier themselves."""
    for m in HEAD.finditer(text):
        end = closing(text, m.end() - 1, "()")
        body = re.match(r"\s*(?:const\s*)?\{", text[end + 1:])
        if body and m.group(1) not in WORDS:
            start = end + body.end()
            if "__syncthreads" in text[start:closing(text, start, "{}")]:
                yield m.group(1)


def unordered(text):
    """(line, statement) of calls with a barrier that share theirs with a read by an index."""
    text = plain(text)
    for name in sorted(set(with_barrier(text))):
        for m in re.finditer(rf"\b{name}\s*(?:<[^;(]*>)?\s*\(", text):
            end = closing(text, m.end() - 1, "()")
            if text[end + 1:].lstrip().startswith(("{", "const {")):
                continue  # the definition
            first = max(text.rfind(c, 0, m.start()) for c in ";{}") + 1
            last = min(text.find(c, end) for c in ";{" if text.find(c, end) >= 0)
            # declarations of one statement are evaluated in their order: this call's alone
            before, after = text[first:m.start()], text[end + 1:last]
            rest = before.rsplit(",", 1)[-1] + " " + after.split(",", 1)[0]
            if "=" in rest:
                rest = rest.split("=", 1)[1]  # (what is assigned to, behind its value)
            if re.search(r"\w\s*\[", rest):
                yield text.count("\n", 0, m.start()) + 1, text[first:last].strip()


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(build.CSRC, "*.hip")) +
                                        glob.glob(os.path.join(build.CSRC, "*.h"))))
def test_no_read_beside_a_barrier(path):
    assert not list(unordered(open(path).read()))


def test_the_parser_sees_the_calls():
    text = """
    __device__ __forceinline__ float total(float v, float *s) { s[0] = v; __syncthreads(); return s[0]; }
    __device__ float other(float v) { return v; }
    template <int N> __global__ __launch_bounds__(256) void k(const A a) {
        auto places = [&](int mine, int &all) { __syncthreads(); return mine; };  // p + next[0]
        float m = total(v[0], s[1]) / H, n = total(w, s[2]) / H;
        out[3] = total(v[0], s[1]) / H;
        float x = other(v[0]) + next[one];
        int p = places(mine, all) + next[one];
        int q = next[one] + places(mine, all);
        place = places(mine, all), p += next[one];
    }"""
    assert sorted(set(with_barrier(text))) == ["places", "total"]  # (a kernel is not called)
    assert [statement for _, statement in unordered(text)] == ["int p = places(mine, all) + next[one]",
                                                              "int q = next[one] + places(mine, all)"]
    found = [n for p in glob.glob(os.path.join(build.CSRC, "*.hip")) for n in with_barrier(plain(open(p).read()))]
    assert {"places", "group_sum", "sum"} <= set(found)
