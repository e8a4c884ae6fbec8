"""The mixture-of-experts calls without a GPU: refusals of the C ABI (fake pointers in a child process that sees no
device), and checks of the tests' own references."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import moe_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "exact_int8_gemm_amd", "libprism.so")
OK, INVALID, ALIGN, UNSUP = 0, -1, -2, -3
A = 0x7F0000000000
F32, F16, BF16 = 0, 1, 2
IMAX = (1 << 31) - 1

_CHILD = r"""
import ctypes, json, sys
lib = ctypes.CDLL(sys.argv[1])
hip = ctypes.CDLL("libamdhip64.so.7")
count = ctypes.c_int(0)
if hip.hipGetDeviceCount(ctypes.byref(count)) == 0 and count.value > 0:
    print(json.dumps({"device_visible": count.value}))
    sys.exit(0)
p, i64, i32, f32, f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_double
norm = [p, i32, i64, p, i64, p, i64, i32, p, i32, f64, p, p, p, i64, i64, p]
sig = {"prism_add_rmsnorm_quantize_fp8": norm, "prism_add_rmsnorm_quantize_rows": norm,
       "prism_route_experts": [p, i32, i64, p, i32, i32, f32, i32, p, p, p, p, p, p, i64, i64, i64, p],
       "prism_gemm_fp8_grouped": [p, p, p, p, p, p, p, i32, i64, i64, i64, i64, i64, p],
       "prism_combine_experts": [p, i32, p, p, p, p, i32, i64, i64, i64, i64, p]}
for n, a in sig.items():
    getattr(lib, n).restype = i32
    getattr(lib, n).argtypes = a
ws = lib.prism_route_experts_workspace
ws.restype = i32
ws.argtypes = [i64, i64, p]
out = []
for fn, args in json.loads(sys.argv[2]):
    if fn == "prism_route_experts_workspace":
        n = i64(-7)
        out.append([ws(*args, ctypes.addressof(n)), n.value])
    else:
        out.append(getattr(lib, fn)(*args))
print(json.dumps({"status": out}))
"""


def _n(x=A, t=BF16, ld=64, res=A, rld=64, out=A, old=64, rt=BF16, gain=A, gt=F32, eps=1e-6, norm=A, q=A, s=A, M=4,
       K=64):
    return [x, t, ld, res, rld, out, old, rt, gain, gt, eps, norm, q, s, M, K, None]


def _r(z=A, t=F32, ld=64, bias=A, score=0, renorm=1, scale=1.0, top=4, ids=A, w=A, off=A, rows=A, slots=A, ws=None,
       wb=0, M=4, E=64):
    return [z, t, ld, bias, score, renorm, scale, top, ids, w, off, rows, slots, ws, wb, M, E, None]


def _g(q=A, sa=A, rows=A, off=A, w=A, sw=A, y=A, t=BF16, M=4, R=8, E=4, N=16, K=64):
    return [q, sa, rows, off, w, sw, y, t, M, R, E, N, K, None]


def _c(x=A, t=BF16, w=A, slots=A, add=A, y=A, yt=BF16, R=8, M=4, top=2, N=33):
    return [x, t, w, slots, add, y, yt, R, M, top, N, None]


NAN, INF = float("nan"), float("inf")
CASES = []
for _fn in ("prism_add_rmsnorm_quantize_fp8", "prism_add_rmsnorm_quantize_rows"):
    CASES += [(_fn, a, e) for a, e in [
        (_n(), UNSUP),                                  # valid: only the device is missing
        (_n(rt=F32), UNSUP), (_n(t=F16, rt=F16, gt=BF16), UNSUP), (_n(t=F32, rt=F32), UNSUP), (_n(norm=None), UNSUP),
        (_n(out=None, old=0), UNSUP), (_n(res=None, rld=0, out=None, old=0, rt=9), UNSUP), (_n(eps=0.0), UNSUP),
        (_n(K=65536, ld=65536, rld=65536, old=65536), UNSUP), (_n(out=A + 4096, old=80), UNSUP),
        (_n(M=0), OK), (_n(None, BF16, 0, None, 0, None, 0, BF16, None, F32, 0.0, None, None, None, 0, 0), OK),
        (_n(M=-1), INVALID), (_n(K=-16), INVALID), (_n(K=0), INVALID), (_n(M=1 << 31), INVALID),
        (_n(K=65552, ld=65552, rld=65552, old=65552), INVALID),
        (_n(t=3), INVALID), (_n(gt=-1), INVALID), (_n(t=3, M=0), INVALID), (_n(rt=F16), INVALID),
        (_n(t=F32, rt=BF16), INVALID), (_n(rt=3), INVALID),
        (_n(eps=-1e-9), INVALID), (_n(eps=NAN), INVALID), (_n(eps=INF), INVALID), (_n(eps=NAN, M=0), INVALID),
        (_n(ld=48), INVALID), (_n(rld=48), INVALID), (_n(old=48), INVALID), (_n(ld=1 << 62), INVALID),
        (_n(rld=1 << 62), INVALID), (_n(old=1 << 62), INVALID),
        (_n(old=72), INVALID),                          # in place with another stride
        (_n(res=None), INVALID),                        # an output without its input
        (_n(x=None), INVALID), (_n(gain=None), INVALID), (_n(q=None), INVALID), (_n(s=None), INVALID),
        (_n(K=40), ALIGN), (_n(x=A + 8), ALIGN), (_n(res=A + 8, out=A), ALIGN), (_n(out=A + 8), ALIGN),
        (_n(gain=A + 4), ALIGN), (_n(norm=A + 8), ALIGN), (_n(q=A + 8), ALIGN), (_n(s=A + 2), ALIGN),
        (_n(ld=68), ALIGN), (_n(rld=68, old=68), ALIGN), (_n(out=A + 4096, old=68), ALIGN),
        (_n(rt=F32, rld=66, old=66), ALIGN),
        (_n(M=(1 << 26) - 1), UNSUP), (_n(M=1 << 26), INVALID),   # 2^32 threads
    ]]
CASES += [("prism_route_experts", a, e) for a, e in [
    (_r(), UNSUP), (_r(t=BF16, z=A + 2), UNSUP), (_r(bias=None), UNSUP), (_r(score=1, renorm=0), UNSUP),
    (_r(E=1024, ld=1024, top=32), UNSUP), (_r(E=1, ld=1, top=1), UNSUP), (_r(E=7, ld=7), UNSUP), (_r(M=32), UNSUP),
    (_r(M=0), OK), (_r(None, F32, 0, None, 0, 0, 1.0, 1, None, None, None, None, None, None, 0, 0, 0), OK),
    (_r(M=-1), INVALID), (_r(E=-1), INVALID), (_r(E=0), INVALID), (_r(t=3), INVALID), (_r(t=-1, M=0), INVALID),
    (_r(score=2), INVALID), (_r(score=-1), INVALID), (_r(scale=NAN), INVALID), (_r(scale=INF), INVALID),
    (_r(top=0), INVALID), (_r(top=33), INVALID), (_r(top=65, E=64), INVALID), (_r(top=8, E=7, ld=7), INVALID),
    (_r(E=1025, ld=1025), INVALID), (_r(ld=63), INVALID), (_r(ld=1 << 62), INVALID), (_r(wb=-1), INVALID),
    (_r(M=(1 << 24) + 1, ws=A, wb=1 << 40), INVALID),
    (_r(M=1 << 24, ws=A, wb=1 << 40), UNSUP),
    (_r(M=1 << 24, top=32, E=64, ws=A, wb=1 << 40), UNSUP),
    (_r(z=None), INVALID), (_r(ids=None), INVALID), (_r(w=None), INVALID), (_r(off=None), INVALID),
    (_r(rows=None), INVALID), (_r(slots=None), INVALID),
    (_r(M=1000), INVALID), (_r(M=1000, ws=A, wb=64), INVALID), (_r(M=1000, ws=A, wb=1 << 20), UNSUP),
    (_r(M=1000, ws=A + 4, wb=1 << 20), ALIGN),
    (_r(z=A + 2), ALIGN), (_r(t=F16, z=A + 1), ALIGN), (_r(bias=A + 2), ALIGN), (_r(ids=A + 2), ALIGN),
    (_r(w=A + 2), ALIGN), (_r(off=A + 2), ALIGN), (_r(rows=A + 2), ALIGN), (_r(slots=A + 2), ALIGN)]]
CASES += [("prism_gemm_fp8_grouped", a, e) for a, e in [
    (_g(), UNSUP), (_g(rows=None, M=8), UNSUP), (_g(t=F32), UNSUP), (_g(t=F16, y=A + 2), UNSUP), (_g(E=1024), UNSUP),
    (_g(N=1, K=16), UNSUP), (_g(R=1), UNSUP), (_g(M=IMAX // 64, R=100), UNSUP),
    (_g(R=0), OK), (_g(None, None, None, None, None, None, None, F32, 0, 0, 0, 0, 0), OK),
    (_g(M=-1), INVALID), (_g(R=-1), INVALID), (_g(E=-1), INVALID), (_g(N=-1), INVALID), (_g(K=-16), INVALID),
    (_g(M=0), INVALID), (_g(E=0), INVALID), (_g(N=0), INVALID), (_g(K=0), INVALID), (_g(E=1025), INVALID),
    (_g(K=131056), INVALID), (_g(M=1 << 31), INVALID), (_g(R=1 << 31), INVALID), (_g(N=1 << 31), INVALID),
    (_g(t=3), INVALID), (_g(t=3, R=0), INVALID), (_g(t=-1), INVALID),
    (_g(rows=None, M=7), INVALID),                       # without rows every row of y is one of q
    (_g(M=1 << 25, K=64), INVALID),                      # 2^31 codes behind row numbers
    (_g(M=1 << 25, R=1 << 25, K=64, rows=None), UNSUP),
    (_g(R=IMAX, N=IMAX, M=4), INVALID),                  # grid
    # wide tiles: their rows are counted in whole tiles, in 32 bits
    (_g(R=IMAX, N=256, K=640), INVALID), (_g(R=IMAX - 255, N=256, K=640), INVALID),
    (_g(R=IMAX - 256, N=256, K=640), UNSUP),
    (_g(q=None), INVALID), (_g(sa=None), INVALID), (_g(off=None), INVALID), (_g(w=None), INVALID),
    (_g(sw=None), INVALID), (_g(y=None), INVALID),
    (_g(K=72), ALIGN), (_g(q=A + 8), ALIGN), (_g(w=A + 8), ALIGN), (_g(sa=A + 2), ALIGN), (_g(sw=A + 2), ALIGN),
    (_g(rows=A + 2), ALIGN), (_g(off=A + 2), ALIGN), (_g(y=A + 1), ALIGN), (_g(t=F32, y=A + 2), ALIGN)]]
CASES += [("prism_combine_experts", a, e) for a, e in [
    (_c(), UNSUP), (_c(yt=F32), UNSUP), (_c(t=F32, yt=F32), UNSUP), (_c(t=F16, yt=F16, x=A + 2, y=A + 2, add=A + 2), UNSUP),
    (_c(add=None), UNSUP), (_c(R=0, x=None), UNSUP), (_c(top=32), UNSUP), (_c(N=1), UNSUP),
    (_c(M=0), OK), (_c(None, F32, None, None, None, None, F32, 0, 0, 1, 0), OK),
    (_c(R=-1), INVALID), (_c(M=-1), INVALID), (_c(N=-1), INVALID), (_c(N=0), INVALID), (_c(top=0), INVALID),
    (_c(top=33), INVALID), (_c(t=3), INVALID), (_c(yt=F16), INVALID), (_c(t=F32, yt=BF16), INVALID),
    (_c(yt=3, M=0), INVALID), (_c(R=1 << 31), INVALID), (_c(M=1 << 31), INVALID), (_c(N=1 << 31), INVALID),
    (_c(M=IMAX, N=IMAX), INVALID), (_c(M=1 << 30, N=32), INVALID),     # grid
    (_c(x=None), INVALID), (_c(w=None), INVALID), (_c(slots=None), INVALID), (_c(y=None), INVALID),
    (_c(x=A + 1), ALIGN), (_c(w=A + 2), ALIGN), (_c(slots=A + 2), ALIGN), (_c(add=A + 1), ALIGN), (_c(y=A + 1), ALIGN),
    (_c(yt=F32, y=A + 2), ALIGN), (_c(yt=F32, add=A + 2), ALIGN)]]
WS = "prism_route_experts_workspace"
WS_CASES = [([0, 0], OK), ([1, 64], OK), ([32, 1024], OK), ([8192, 256], OK), ([1 << 24, 1024], OK), ([-1, 4], INVALID),
            ([1, -4], INVALID), ([(1 << 24) + 1, 4], INVALID), ([1, 1025], INVALID)]


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
    assert n == -7 if expect != OK else n >= 0      # a refused call writes nothing
    if expect == OK and args[0] >= 8192:
        assert 0 < n <= 1 << 20 or args[0] > 8192


def test_limits_of_the_binding_are_the_headers():
    import re
    from exact_int8_gemm_amd import prism
    text = open(os.path.join(ROOT, "include", "prism.h")).read()
    d = {k: int(v) for k, v in re.findall(r"#define\s+(PRISM_\w+)\s+\(?(-?\d+)\)?", text)}
    assert (d["PRISM_NORM_K_MAX"], d["PRISM_EXPERTS_MAX"], d["PRISM_ROUTE_M_MAX"]) == \
        (prism.NORM_K_MAX, prism.EXPERTS_MAX, prism.ROUTE_M_MAX)
    assert {"softmax": d["PRISM_SCORE_SOFTMAX"], "sigmoid": d["PRISM_SCORE_SIGMOID"]} == prism.SCORES


def test_python_refuses_host_tensors():
    from exact_int8_gemm_amd import prism
    x = torch.zeros((4, 128))
    i = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: prism.add_rmsnorm_quantize_fp8(x, x[0]), lambda: prism.add_rmsnorm_quantize_rows(x, x[0]),
                 lambda: prism.route_experts(x, 2), lambda: prism.combine_experts(x, x, i),
                 lambda: prism.gemm_fp8_grouped(x.to(torch.float8_e4m3fn), x, x, x, i)):
        with pytest.raises(ValueError, match="HIP device"):
            call()


# ------------------------------------------------------------ the references themselves

def test_reference_norm_by_hand():
    h = np.array([[3.0, 4.0], [0.0, 0.0]], np.float32)
    y = ref.norm(h, [1.0, 2.0], 0.0)
    inv = np.float32(1 / np.sqrt(12.5))
    assert y[0, 0] == np.float32(3) * inv and y[0, 1] == np.float32(4) * inv * 2 and np.isnan(y[1]).all()
    assert not ref.norm(h, [1.0, 2.0], 1e-6)[1].any()


def test_reference_int8_by_hand():
    q, s = ref.quantize_int8([[127.0, 1.5, 2.5, -126.5], [0, 0, 0, 0], [np.inf, 1, 2, 3]])
    one = np.float32(127) * (np.float32(1) / np.float32(127))
    assert list(q[0]) == [127, 2, 2, -126] and s[0] == one == 1      # ties to even
    assert not q[1].any() and s[1] == 0 and not q[2].any() and np.isnan(s[2])


def test_reference_route_by_hand():
    z = np.log([[0.2, 0.4, 0.4, 1e-9]])
    ids, w, off, rows, slots = ref.route(z, 2)
    assert list(ids[0]) == [1, 2] and np.allclose(w[0], 0.5) and list(off) == [0, 0, 1, 2, 2]
    assert list(rows) == [0, 0] and list(slots[0]) == [0, 1]
    ids, w, *_ = ref.route(z, 2, bias=[0.3, 0, 0, 0], renormalize=False, scale=2.0)
    assert list(ids[0]) == [0, 1] and np.allclose(w[0], [0.4, 0.8])
    ids, w, off, rows, slots = ref.route([[-np.inf, 1.0], [-np.inf, -np.inf], [np.nan, 0]], 2, score="sigmoid")
    assert ids.tolist() == [[1, -1], [-1, -1], [-1, -1]] and w[0, 0] == 1 and not w[1].any() and np.isnan(w[2]).all()
    assert list(off) == [0, 0, 1] and list(rows) == [0] + [-1] * 5 and slots.tolist() == [[0, -1], [-1, -1], [-1, -1]]


def test_reference_dispatch_keeps_the_order_of_the_tokens():
    off, rows, slots = ref.dispatch(np.array([[1, 0], [1, -1], [0, 1]]), 3)
    assert list(off) == [0, 2, 5, 5] and list(rows) == [0, 2, 0, 1, 2, -1]
    assert slots.tolist() == [[2, 0], [3, -1], [1, 4]]


def test_reference_combine_by_hand():
    x = [[1.0, 2.0], [10.0, 20.0]]
    y, mag = ref.combine(x, [[0.5, -1.0]], np.array([[1, 0]]), [[100.0, 0.0]])
    assert y.tolist() == [[104.0, 8.0]] and mag.tolist() == [[106.0, 12.0]]
    y, _ = ref.combine(x, [[0.5, 1.0], [np.nan, 0]], np.array([[-1, 2], [-1, -1]]))
    assert not y[0].any() and np.isnan(y[1]).all()
