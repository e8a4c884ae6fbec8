"""The fp8 and read-out calls without a GPU: refusals of the C ABI (fake
pointers in a child process that sees no device), and checks of the tests' own
references."""
import json
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import fp8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "exact_int8_gemm_amd", "libprism.so")
OK, INVALID, ALIGN, UNSUP = 0, -1, -2, -3
A = 0x7F0000000000
F32, F16, BF16 = 0, 1, 2
KMAX = 131040

_CHILD = r"""
import ctypes, json, sys
lib = ctypes.CDLL(sys.argv[1])
hip = ctypes.CDLL("libamdhip64.so.7")
count = ctypes.c_int(0)
if hip.hipGetDeviceCount(ctypes.byref(count)) == 0 and count.value > 0:
    print(json.dumps({"device_visible": count.value}))
    sys.exit(0)
p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
sig = {"prism_quantize_blocks_fp8": [p, i32, i64, p, p, i64, i64, p],
       "prism_quantize_tiles_fp8": [p, i32, i64, p, p, i64, i64, p],
       "prism_swiglu_quantize_fp8": [p, p, i32, i64, p, p, i64, i64, p],
       "prism_gemm_fp8_blockscale": [p, p, p, p, p, i32, i64, i64, i64, p],
       "prism_token_logprobs": [p, i32, i64, p, i64, i32, p, p, p, p, p, p, i64, i64, i64, p]}
for n, a in sig.items():
    getattr(lib, n).restype = i32
    getattr(lib, n).argtypes = a
ws = lib.prism_token_logprobs_workspace
ws.restype = i32
ws.argtypes = [i64, i64, i32, p]
out = []
for fn, args in json.loads(sys.argv[2]):
    if fn == "prism_token_logprobs_workspace":
        n = i64(-7)
        out.append([ws(*args, ctypes.addressof(n)), n.value])
    else:
        out.append(getattr(lib, fn)(*args))
print(json.dumps({"status": out}))
"""


def _b(x=A, t=F32, ld=64, q=A, s=A, M=4, K=64):
    return [x, t, ld, q, s, M, K, None]


def _s(g=A, u=A, t=F32, ld=128, q=A, s=A, M=4, K=64):
    return [g, u, t, ld, q, s, M, K, None]


def _g(q=A, sa=A, w=A, sw=A, y=A, t=BF16, M=4, N=16, K=64):
    return [q, sa, w, sw, y, t, M, N, K, None]


def _l(z=A, t=F32, ld=100, tok=A, T=1, top=2, lp=A, lse=A, ent=A, ids=A, tlp=A, ws=None, wb=0, M=4, V=100):
    return [z, t, ld, tok, T, top, lp, lse, ent, ids, tlp, ws, wb, M, V, None]


CASES = []
for _fn in ("prism_quantize_blocks_fp8", "prism_quantize_tiles_fp8"):
    CASES += [(_fn, a, e) for a, e in [
        (_b(), UNSUP),                              # valid: only the device is missing
        (_b(t=F16), UNSUP), (_b(t=BF16, ld=72), UNSUP), (_b(K=KMAX, ld=KMAX), UNSUP),
        (_b(M=0), OK), (_b(None, F32, 0, None, None, 0, 0), OK),
        (_b(M=-1), INVALID), (_b(K=0), INVALID), (_b(K=-16), INVALID), (_b(K=KMAX + 16, ld=KMAX + 16), INVALID),
        (_b(t=3), INVALID), (_b(t=-1), INVALID), (_b(t=3, M=0), INVALID),
        (_b(ld=48), INVALID),                       # rows overlap
        (_b(ld=1 << 62), INVALID), (_b(M=1 << 31), INVALID),
        (_b(x=None), INVALID), (_b(q=None), INVALID), (_b(s=None), INVALID),
        (_b(K=40), ALIGN), (_b(x=A + 4), ALIGN), (_b(q=A + 8), ALIGN), (_b(s=A + 2), ALIGN),
        (_b(ld=66), ALIGN), (_b(t=BF16, ld=68), ALIGN),
    ]]
CASES += [("prism_swiglu_quantize_fp8", a, e) for a, e in [
    (_s(), UNSUP), (_s(M=0), OK), (_s(M=-1), INVALID), (_s(K=0), INVALID), (_s(t=9), INVALID), (_s(ld=32), INVALID),
    (_s(g=None), INVALID), (_s(u=None), INVALID), (_s(q=None), INVALID), (_s(s=None), INVALID),
    (_s(K=24), ALIGN), (_s(g=A + 8), ALIGN), (_s(u=A + 8), ALIGN), (_s(q=A + 4), ALIGN), (_s(s=A + 1), ALIGN),
    (_s(ld=130), ALIGN)]]
CASES += [("prism_gemm_fp8_blockscale", a, e) for a, e in [
    (_g(), UNSUP), (_g(t=F32), UNSUP), (_g(t=F16, y=A + 2), UNSUP), (_g(N=1, K=16), UNSUP),
    (_g(M=0), OK), (_g(None, None, None, None, None, F32, 0, 0, 0), OK),
    (_g(M=-1), INVALID), (_g(N=-1), INVALID), (_g(K=-16), INVALID), (_g(N=0), INVALID), (_g(K=0), INVALID),
    (_g(t=3), INVALID), (_g(t=3, M=0), INVALID), (_g(t=-1), INVALID), (_g(K=KMAX + 16), INVALID),
    (_g(M=1 << 31), INVALID), (_g(N=1 << 31), INVALID), (_g(M=(1 << 31) - 1, N=(1 << 31) - 1), INVALID),
    (_g(q=None), INVALID), (_g(sa=None), INVALID), (_g(w=None), INVALID), (_g(sw=None), INVALID), (_g(y=None), INVALID),
    (_g(K=72), ALIGN), (_g(q=A + 8), ALIGN), (_g(w=A + 8), ALIGN), (_g(sa=A + 2), ALIGN), (_g(sw=A + 2), ALIGN),
    (_g(y=A + 1), ALIGN), (_g(t=F32, y=A + 2), ALIGN)]]
# grids of 2^32 threads: 16 rows by two blocks a workgroup of 256 (one where the call is small), tiles
CASES += [(fn, a, e) for fn, a, e in [
    ("prism_quantize_blocks_fp8", _b(M=(1 << 28) - 16, K=256, ld=256, t=BF16), UNSUP),
    ("prism_quantize_blocks_fp8", _b(M=1 << 28, K=256, ld=256, t=BF16), INVALID),
    ("prism_swiglu_quantize_fp8", _s(M=(1 << 28) - 16, K=256, ld=512, t=BF16), UNSUP),
    ("prism_swiglu_quantize_fp8", _s(M=1 << 28, K=256, ld=512, t=BF16), INVALID),
    ("prism_quantize_blocks_fp8", _b(M=(1 << 28) - 16, K=128, ld=128, t=BF16), UNSUP),
    ("prism_quantize_tiles_fp8", _b(M=(1 << 31) - 128, K=128, ld=128, t=BF16), UNSUP),
    ("prism_quantize_tiles_fp8", _b(M=(1 << 31) - 127, K=128, ld=128, t=BF16), INVALID)]]
# grids of 2^32 threads: 16 columns a workgroup of 256, 64 x 64 and 128 x 128 tiles
CASES += [("prism_gemm_fp8_blockscale", a, e) for a, e in [
    (_g(M=1, N=1 << 28, K=16), INVALID), (_g(M=1, N=(1 << 28) - 16, K=16), UNSUP),
    (_g(M=8, N=1 << 28, K=16, t=F16), INVALID), (_g(M=4, N=(1 << 31) - 1, K=16, t=F32), INVALID),
    (_g(M=9, N=1 << 30, K=16, t=F32), INVALID), (_g(M=9, N=(1 << 30) - 64, K=16, t=F32), UNSUP),
    (_g(M=9, N=1 << 30, K=16, t=F16), INVALID), (_g(M=9, N=1 << 30, K=16), UNSUP),
    (_g(M=9, N=(1 << 31) - 1, K=16), INVALID), (_g(M=(1 << 31) - 1, N=16, K=16), INVALID),
    (_g(M=(1 << 31) - 128, N=16, K=16), UNSUP), (_g(M=1 << 20, N=1 << 20, K=16), INVALID)]]
_BIG = 1 << 20   # a vocabulary of several chunks
CASES += [("prism_token_logprobs", a, e) for a, e in [
    (_l(), UNSUP), (_l(t=BF16, z=A + 2), UNSUP), (_l(tok=None, T=0, lp=None), UNSUP),
    (_l(top=0, ids=None, tlp=None), UNSUP), (_l(lse=None, ent=None), UNSUP), (_l(top=32, V=1, ld=1), UNSUP),
    (_l(M=0), OK), (_l(None, F32, 0, None, 0, 0, None, None, None, None, None, None, 0, 0, 0), OK),
    (_l(M=-1), INVALID), (_l(V=0), INVALID), (_l(V=-1), INVALID), (_l(T=-1), INVALID), (_l(top=-1), INVALID),
    (_l(top=33), INVALID), (_l(top=33, M=0), INVALID), (_l(t=4), INVALID), (_l(ld=99), INVALID), (_l(wb=-1), INVALID),
    (_l(M=1 << 31), INVALID), (_l(V=1 << 31, ld=1 << 31), INVALID), (_l(ld=1 << 62), INVALID),
    (_l(z=None), INVALID), (_l(tok=None), INVALID), (_l(lp=None), INVALID), (_l(ids=None), INVALID),
    (_l(tlp=None), INVALID),
    (_l(V=_BIG, ld=_BIG), INVALID),                                   # workspace missing
    (_l(V=_BIG, ld=_BIG, ws=A, wb=64), INVALID),                      # too small
    (_l(V=_BIG, ld=_BIG, ws=A, wb=1 << 30), UNSUP), (_l(V=_BIG, ld=_BIG, ws=A + 4, wb=1 << 30), ALIGN),
    (_l(z=A + 2), ALIGN), (_l(t=F16, z=A + 1), ALIGN), (_l(tok=A + 4), ALIGN), (_l(lp=A + 2), ALIGN),
    (_l(lse=A + 2), ALIGN), (_l(ent=A + 2), ALIGN), (_l(ids=A + 4), ALIGN), (_l(tlp=A + 2), ALIGN)]]
# grids of 2^32 threads: a wave for each 4096 logits, in fours; a wave or, with many keys, four to join a row's
CASES += [("prism_token_logprobs", a, e) for a, e in [
    (_l(M=(1 << 26) - 4, top=0), UNSUP), (_l(M=1 << 26, top=0), INVALID),
    (_l(M=1 << 24, V=4100, ld=4100, t=F16, ws=A, wb=1 << 40), UNSUP),
    (_l(M=(1 << 25) - 2, V=4100, ld=4100, t=F16, ws=A, wb=1 << 40), UNSUP),
    (_l(M=1 << 25, V=4100, ld=4100, t=F16, ws=A, wb=1 << 40), INVALID),
    (_l(M=1 << 20, V=100003, ld=100003, top=32, ws=A, wb=1 << 40), UNSUP)]]
WS = "prism_token_logprobs_workspace"
WS_CASES = [([0, 0, 0], OK), ([4, 100, 20], OK), ([4, _BIG, 0], OK), ([4, _BIG, 32], OK), ([-1, 4, 0], INVALID),
            ([1, -4, 0], INVALID), ([1, 4, 33], INVALID), ([1, 4, -1], INVALID), ([1 << 31, 4, 0], INVALID),
            ([1, 1 << 31, 0], INVALID)]


@pytest.fixture(scope="module")
def results():
    if not os.path.exists(LIB):
        from exact_int8_gemm_amd import build
        build.build_library()
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", CUDA_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    payload = json.dumps([[fn, a] for fn, a, _ in CASES] + [[WS, a] for a, _ in WS_CASES])
    out = subprocess.run([sys.executable, "-c", _CHILD, LIB, payload], env=env, capture_output=True, text=True,
                         timeout=120)
    assert out.returncode == 0, out.stderr
    res = json.loads(out.stdout.strip().splitlines()[-1])
    if "device_visible" in res:
        pytest.skip("a HIP device is visible despite HIP_VISIBLE_DEVICES=-1: fake-pointer calls not made")
    return res["status"]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_refusals(results, i):
    fn, args, expect = CASES[i]
    assert results[i] == expect, (fn, args)


@pytest.mark.parametrize("i", range(len(WS_CASES)))
def test_workspace(results, i):
    args, expect = WS_CASES[i]
    status, n = results[len(CASES) + i]
    assert status == expect
    if expect != OK:
        assert n == -7          # nothing written
    else:
        M, V, top = args
        assert n >= 0 and (n == 0 or (V > 1000 and n >= M * (8 * top + 12)))


def test_python_refuses_host_tensors():
    from exact_int8_gemm_amd import prism
    x = torch.zeros((4, 128))
    for call in (lambda: prism.quantize_blocks_fp8(x), lambda: prism.quantize_tiles_fp8(x),
                 lambda: prism.swiglu_quantize_fp8(x, x), lambda: prism.token_logprobs(x),
                 lambda: prism.gemm_fp8_blockscale(x.to(torch.float8_e4m3fn), x, x, x)):
        with pytest.raises(ValueError, match="HIP device"):
            call()


def test_reference_values_are_torchs():
    """The e4m3 table against torch's type, over every code."""
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(ref.E4M3))
    assert np.array_equal(t[~np.isnan(t)], ref.E4M3[~np.isnan(t)])


def test_reference_rounding_by_hand():
    # spacing 2 in [16, 32): 17 and 19 are ties, to the even codes 16 and 20
    assert list(ref.round_e4m3([17.0, 19.0, 17.001, 18.999, -19.0])) == [16, 20, 18, 18, -20]
    # subnormals: spacing 2^-9, tie 2^-10 goes to 0, 3 * 2^-10 to 2 * 2^-9
    assert list(ref.round_e4m3([2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 1.01 * 2.0 ** -10])) == \
        [0, 2.0 ** -8, 2.0 ** -9, 2.0 ** -9]
    assert list(ref.round_e4m3([448, 1e9, -np.inf])) == [448, 448, -448]


def test_reference_rounding_is_nearest():
    """Against a search over all values, on random numbers and at every tie's neighbours."""
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.uniform(-448, 448, 2000), np.exp(rng.uniform(-8, 6, 2000)), np.nextafter(ref._MID, 0),
                        np.nextafter(ref._MID, 1000)])
    got = ref.round_e4m3(x)
    near = np.abs(x[:, None] - ref.E4M3[~np.isnan(ref.E4M3)]).min(axis=1)
    assert np.array_equal(np.abs(x - got), near)


def test_reference_quantizer_by_hand():
    x = np.zeros((2, 130), np.float32)
    x[0, 0], x[0, 1], x[0, 129] = 448, 17, -2       # block 0: s = 1; block 1: s = 2 / 448
    v, s = ref.quantize(x, 1)
    assert s.shape == (2, 2) and s[0, 0] == 1 and s[0, 1] == np.float32(2) / np.float32(448) and s[1, 0] == 0
    assert v[0, 0] == 448 and v[0, 1] == 16 and v[0, 129] == -448 and not v[1].any()


def test_reference_logprobs_by_hand():
    z = np.log(np.array([[0.5, 0.25, 0.25, 0.0]], np.float64), where=[[1, 1, 1, 0]], out=np.full((1, 4), -np.inf))
    lp, lse, ent, ids, tlp = ref.logprobs(z, np.array([[0, 3, 4]]), 4)
    assert math.isclose(lp[0, 0], math.log(0.5)) and lp[0, 1] == -np.inf and np.isnan(lp[0, 2])
    assert abs(lse[0]) < 1e-12 and math.isclose(ent[0], 1.5 * math.log(2))
    assert list(ids[0]) == [0, 1, 2, -1] and tlp[0, 3] == -np.inf
