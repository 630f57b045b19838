"""Validation of sb_verify_drafts on the host: every bad argument is refused with
the documented status before any GPU work, and offsets, which the kernels read on
the device, never lead out of the matrices."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

from logit_source_projection_amd import sb
from tests.test_abi_cpu import FAKE

BIG = 1 << 40
CSRC = os.path.join(os.path.dirname(sb.__file__), "csrc")


def desc(N=3, K=4, V=4096, drafts=9, offsets=FAKE, tokens=FAKE, target=FAKE, ldt=4096, draft=FAKE, ldd=4096,
         type=sb.SB_FP32, temperature=FAKE):
    return sb.sb_drafts_desc(N=N, K=K, V=V, drafts=drafts, offsets=offsets, tokens=tokens, target=target, ldt=ldt,
                             draft=draft, ldd=ldd, type=type, temperature=temperature)


def verify(d, u=FAKE, u_next=FAKE, out=FAKE, ldo=5, accepted=FAKE, ws=FAKE, n=BIG):
    return sb.lib().sb_verify_drafts(ctypes.byref(d), u, u_next, out, ldo, accepted, ws, n, None)


def ws_status(d):
    st = ctypes.c_int(0)
    n = sb.lib().sb_verify_workspace_bytes(ctypes.byref(d), ctypes.byref(st))
    assert n == 0 or st.value == sb.SB_OK
    return st.value


@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), sb.SB_ERR_SHAPE), (dict(K=-1), sb.SB_ERR_SHAPE), (dict(V=0), sb.SB_ERR_SHAPE),
    (dict(drafts=-1), sb.SB_ERR_SHAPE), (dict(type=2), sb.SB_ERR_SHAPE), (dict(type=-1), sb.SB_ERR_SHAPE),
    (dict(ldt=4092), sb.SB_ERR_SHAPE), (dict(ldd=4092), sb.SB_ERR_SHAPE), (dict(ldt=-4096), sb.SB_ERR_SHAPE),
    (dict(offsets=0), sb.SB_ERR_NULL), (dict(tokens=0), sb.SB_ERR_NULL), (dict(target=0), sb.SB_ERR_NULL),
    (dict(target=FAKE + 8), sb.SB_ERR_ALIGN), (dict(draft=FAKE + 4), sb.SB_ERR_ALIGN),
    (dict(ldt=4098), sb.SB_ERR_ALIGN), (dict(ldd=4098), sb.SB_ERR_ALIGN),
    (dict(ldt=4100, type=sb.SB_BF16), sb.SB_ERR_ALIGN), (dict(offsets=FAKE + 2), sb.SB_ERR_ALIGN),
    (dict(tokens=FAKE + 1), sb.SB_ERR_ALIGN), (dict(temperature=FAKE + 2), sb.SB_ERR_ALIGN),
    (dict(V=(1 << 30) + 8, ldt=1 << 31, ldd=1 << 31), sb.SB_ERR_UNSUPPORTED),
    (dict(ldt=1 << 45), sb.SB_ERR_UNSUPPORTED), (dict(ldd=1 << 62), sb.SB_ERR_UNSUPPORTED),
    (dict(N=1 << 24), sb.SB_ERR_UNSUPPORTED), (dict(K=1 << 30), sb.SB_ERR_UNSUPPORTED),
    (dict(N=2 ** 31 - 1, K=2 ** 31 - 1, drafts=2 ** 31 - 1), sb.SB_ERR_UNSUPPORTED),
    (dict(N=1 << 20, K=8), sb.SB_ERR_UNSUPPORTED), (dict(N=1 << 24, K=0), sb.SB_ERR_UNSUPPORTED),
    (dict(N=(1 << 22) + 5, K=1), sb.SB_OK), (dict(N=1 << 23, K=0, V=4097, ldt=8192, ldd=8192), sb.SB_ERR_UNSUPPORTED), (dict(N=1 << 19, K=8), sb.SB_OK)])
def test_descriptor(kw, want):
    assert ws_status(desc(**kw)) == want
    if want != sb.SB_OK:
        assert verify(desc(**kw), ldo=1 << 33) == want


def test_arguments():
    for kw, want in ((dict(u=0), sb.SB_ERR_NULL), (dict(u_next=0), sb.SB_ERR_NULL), (dict(out=0), sb.SB_ERR_NULL),
                     (dict(accepted=0), sb.SB_ERR_NULL), (dict(ldo=4), sb.SB_ERR_SHAPE), (dict(ldo=-5), sb.SB_ERR_SHAPE),
                     (dict(u=FAKE + 2), sb.SB_ERR_ALIGN), (dict(u_next=FAKE + 2), sb.SB_ERR_ALIGN),
                     (dict(out=FAKE + 2), sb.SB_ERR_ALIGN), (dict(accepted=FAKE + 1), sb.SB_ERR_ALIGN),
                     (dict(ldo=1 << 60), sb.SB_ERR_UNSUPPORTED), (dict(ws=0), sb.SB_ERR_NULL),
                     (dict(ws=FAKE + 8), sb.SB_ERR_ALIGN), (dict(n=100), sb.SB_ERR_WORKSPACE)):
        assert verify(desc(), **kw) == want, kw
    assert sb.lib().sb_verify_drafts(None, FAKE, FAKE, FAKE, 5, FAKE, FAKE, BIG, None) == sb.SB_ERR_NULL


def test_no_sequences():
    d = desc(N=0, drafts=0, offsets=0, tokens=0, target=0, draft=0)
    assert ws_status(d) == sb.SB_OK
    assert verify(d, u=0, u_next=0, out=0, accepted=0, ws=0, n=0) == sb.SB_OK


def test_host_tensors_are_refused():
    off = torch.zeros(2, dtype=torch.int32)
    d = sb.Drafts(torch.zeros(1, 8), off[:0], off, 0)
    with pytest.raises(ValueError, match="target must be a device tensor"):
        sb.sb_verify_drafts(d, None, torch.zeros(1), off.view(2, 1), off[:1])


def test_offsets_stay_inside(tmp_path):
    """place_of, which the kernels call, on any pair of offsets."""
    src, lib = tmp_path / "place.cpp", tmp_path / "place.so"
    src.write_text('#include "verify_place.h"\n'
                   'extern "C" void place(int32_t a, int32_t b, int32_t n, int32_t k, int32_t *out)\n'
                   '{ const sbk::Place p = sbk::place_of(a, b, n, k); out[0] = p.first; out[1] = p.count; }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror",
                    "-I", CSRC, str(src), "-o", str(lib)], check=True)
    place = ctypes.CDLL(str(lib)).place
    out = (ctypes.c_int32 * 2)()
    rng = random.Random(1)
    wild = [-2 ** 31, -2 ** 31 + 1, -1, 0, 1, 2, 7, 100, 2 ** 31 - 2, 2 ** 31 - 1]
    cases = [(a, b, n, k) for a in wild for b in wild for n in (0, 1, 7, 2 ** 31 - 1) for k in (0, 1, 5, 2 ** 31 - 1)]
    cases += [(rng.randint(-20, 40), rng.randint(-20, 40), rng.randint(0, 25), rng.randint(0, 9)) for _ in range(5000)]
    for a, b, n, k in cases:
        place(a, b, n, k, out)
        first, count = out
        assert 0 <= first and 0 <= count <= k and first + count <= n, (a, b, n, k, first, count)
        if 0 <= a <= b <= n:
            assert (first, count) == (a, min(b - a, k))
