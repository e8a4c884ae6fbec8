"""The norm with an 8-bit output on the GPU against its definition step by step in numpy.

Every output is compared exactly: the sum of squares is held in 64 bits on both sides, where the order changes 2^-50 of
it at the most, so inv's rounding to fp32 can differ in one row of 2^26; all that follows is single fp32 roundings.
"""
import numpy as np
import pytest
import torch

import moe_ref as ref
from exact_int8_gemm_amd import prism
from gpu_util import DEV

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PAIRS = [("f32", None), ("f32", "f32"), ("f16", None), ("f16", "f16"), ("f16", "f32"), ("bf16", None), ("bf16", "bf16"),
         ("bf16", "f32")]
EPS = 1e-6


def call(to, *args, **kw):
    return (prism.add_rmsnorm_quantize_fp8 if to == "fp8" else prism.add_rmsnorm_quantize_rows)(*args, **kw)


def inputs(seed, m, k, kind, res, gain="f32"):
    """On the CPU: x, residual (or None), gain."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, k), generator=g).to(TYPES[kind])
    loud = torch.where(torch.rand((k,), generator=g) < 0.02, 20.0, 1.0)
    r = None if res is None else (torch.randn((m, k), generator=g) * loud).to(TYPES[res])
    return x, r, (1 + 0.2 * torch.randn((k,), generator=g)).to(TYPES[gain])


def expect(to, x, r, gain, eps=EPS):
    """-> codes as float32, scales, h, y (fp32); all numpy but h."""
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    y = ref.norm(h.float().numpy(), gain.float().numpy(), eps)
    q, s = ref.quantize_fp8(y) if to == "fp8" else ref.quantize_int8(y)
    return q.astype(np.float32), s, h, y


def check(to, got, want, kind, norm):
    q, s, h, y = want
    assert np.array_equal(got.scale.cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(got.q.float().cpu().numpy(), q)
    if got.residual is not None:
        assert torch.equal(got.residual.cpu(), h)
    if norm:
        assert torch.equal(got.norm.cpu(), torch.from_numpy(y).to(TYPES[kind]))
    else:
        assert got.norm is None


def on(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("to", ["fp8", "int8"])
@pytest.mark.parametrize("kind,res", PAIRS)
@pytest.mark.parametrize("m,k", [(1, 16), (1, 5120), (2, 112), (3, 144), (17, 400), (33, 1040), (130, 2064), (5, 4112),
                                 (3, 9680), (2, 17408), (1, 33040), (2, 65536)])
def test_against_the_definition(m, k, kind, res, to):
    norm = (m + k) % 3 != 0
    x, r, gain = inputs(m * 1000 + k, m, k, kind, res)
    got = call(to, on(x), on(gain), EPS, residual=on(r), norm=norm)
    assert got.q.dtype == (prism.FP8 if to == "fp8" else torch.int8)
    check(to, got, expect(to, x, r, gain), kind, norm)


@pytest.mark.parametrize("to", ["fp8", "int8"])
@pytest.mark.parametrize("gain", list(TYPES))
def test_types_of_the_gain(gain, to):
    x, r, g = inputs(5, 9, 656, "bf16", "bf16", gain)
    check(to, call(to, on(x), on(g), 1e-5, residual=on(r)), expect(to, x, r, g, 1e-5), "bf16", False)


@pytest.mark.parametrize("to", ["fp8", "int8"])
@pytest.mark.parametrize("kind,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_strided_rows_and_given_outputs(kind, res, to):
    m, k = 21, 400
    x, r, g = inputs(6, m, k, kind, res)
    want = expect(to, x, r, g)
    wide_x = torch.full((m, 1024), 9.0, dtype=TYPES[kind], device=DEV)
    wide_r = torch.full((m, 768), 9.0, dtype=TYPES[res], device=DEV)
    wide_o = torch.full((m, 528), 9.0, dtype=TYPES[res], device=DEV)
    wide_x[:, 256:656].copy_(x)
    wide_r[:, 64:464].copy_(r)
    q = torch.empty((m, k), dtype=prism.FP8 if to == "fp8" else torch.int8, device=DEV)
    s = torch.empty(want[1].shape, device=DEV)
    y = torch.empty((m, k), dtype=TYPES[kind], device=DEV)
    out = wide_o[:, 32:432]
    got = call(to, wide_x[:, 256:656], on(g), EPS, residual=wide_r[:, 64:464], residual_out=out, norm=y, q=q, scale=s)
    assert got.q is q and got.scale is s and got.residual is out and got.norm is y
    check(to, got, want, kind, True)
    assert (wide_o[:, :32] == 9).all() and (wide_o[:, 432:] == 9).all()
    assert torch.equal(wide_r[:, 64:464].cpu(), r) and torch.equal(wide_x[:, 256:656].cpu(), x)
    # the residual in its own place, as a layer keeps it
    place = wide_r[:, 64:464]
    got = call(to, wide_x[:, 256:656], on(g), EPS, residual=place, residual_out=place)
    check(to, got, want, kind, False)
    assert (wide_r[:, :64] == 9).all() and (wide_r[:, 464:] == 9).all()


@pytest.mark.parametrize("to", ["fp8", "int8"])
def test_special_values(to):
    """Zeros, subnormals, the largest values, infinities and NaN, each in a row of its own; eps 0 and large."""
    k = 272
    g = torch.Generator().manual_seed(7)
    x = torch.randn((12, k), generator=g)
    x[0] = 0
    x[1] = -0.0
    x[2] *= 1e-40
    x[3] = torch.finfo(torch.float32).max
    x[4, 3] = float("inf")
    x[5, 130] = float("nan")
    x[6] *= 1e-20
    x[7] *= 1e30
    x[8, 1:] = 0                    # one value
    x[9, :] = 1e-45
    x[10, 5], x[10, 6] = float("inf"), -float("inf")
    gain = torch.randn((k,), generator=g)
    gain[::7] = 0
    for eps in (0.0, 1e-6, 1e-30, 3.0):
        want = expect(to, x, None, gain, eps)
        got = call(to, on(x), on(gain), eps, norm=True)
        assert np.array_equal(got.scale.cpu().numpy(), want[1], equal_nan=True), eps
        assert np.array_equal(got.q.float().cpu().numpy(), want[0]), eps
        assert np.array_equal(got.norm.cpu().numpy(), want[3], equal_nan=True), eps
    assert np.isnan(want[1].reshape(-1, 12)[:, 5]).all()


@pytest.mark.parametrize("to", ["fp8", "int8"])
def test_the_residual_is_rounded_before_it_is_normed(to):
    """x far below the residual's last bit: the norm is that of the stored residual; fp16 sums over its largest value
    are infinities, as stored."""
    k = 128
    r = torch.full((2, k), 256.0).bfloat16()
    x = torch.full((2, k), 0.5).bfloat16()
    got = call(to, on(x), on(torch.ones(k)), EPS, residual=on(r), norm=True)
    assert torch.equal(got.residual.cpu(), r)
    check(to, got, expect(to, x, r, torch.ones(k)), "bf16", True)
    r, x = torch.full((1, k), 60000.0).half(), torch.full((1, k), 10000.0).half()
    got = call(to, on(x), on(torch.ones(k)), EPS, residual=on(r))
    assert torch.isinf(got.residual).all() and torch.isnan(got.scale).all() and not got.q.float().any()


@pytest.mark.parametrize("to", ["fp8", "int8"])
@pytest.mark.parametrize("k", [144, 2576, 5120, 17408])
def test_rows_do_not_depend_on_the_batch(k, to):
    m = 1030
    x, r, g = inputs(8, m, k, "bf16", "f32")
    x, r, g = on(x), on(r), on(g)
    whole = call(to, x, g, EPS, residual=r, norm=True)
    scale = whole.scale if to == "fp8" else whole.scale[None]
    for lo, hi in ((0, 1), (1029, 1030), (500, 516), (3, 259)):
        part = call(to, x[lo:hi], g, EPS, residual=r[lo:hi], norm=True)
        assert torch.equal(part.q.view(torch.uint8), whole.q[lo:hi].view(torch.uint8))
        assert torch.equal(part.scale if to == "fp8" else part.scale[None], scale[:, lo:hi])
        assert torch.equal(part.residual, whole.residual[lo:hi]) and torch.equal(part.norm, whole.norm[lo:hi])


@pytest.mark.parametrize("to", ["fp8", "int8"])
def test_does_not_write_outside(to):
    m, k = 19, 272
    x, r, g = inputs(9, m, k, "bf16", "bf16")
    q = torch.full((m + 8, k), 3.0, device=DEV).to(prism.FP8 if to == "fp8" else torch.int8)
    count = 3 * m if to == "fp8" else m
    s = torch.full((count + 64,), 7.0, device=DEV)
    y = torch.full((m + 8, k), 5.0, dtype=torch.bfloat16, device=DEV)
    h = torch.full((m + 8, k), 6.0, dtype=torch.bfloat16, device=DEV)
    got = call(to, on(x), on(g), EPS, residual=on(r), residual_out=h[:m], norm=y[:m], q=q[:m],
               scale=s[:count].view(3, m) if to == "fp8" else s[:count])
    check(to, got, expect(to, x, r, g), "bf16", True)
    assert (q[m:].float() == 3).all() and (s[count:] == 7).all() and (y[m:] == 5).all() and (h[m:] == 6).all()


@pytest.mark.parametrize("to", ["fp8", "int8"])
def test_inputs_and_outputs_past_32_bit_offsets(to):
    m, k = 70000, 32768
    assert m * k > 2 ** 31
    x = torch.zeros((m, k), dtype=torch.bfloat16, device=DEV)
    some = torch.tensor([0, 1, 34567, m - 2, m - 1])
    xs, _, g = inputs(10, 5, k, "bf16", None)
    x[some] = on(xs)
    got = call(to, x, on(g), EPS, residual=x, residual_out=x)
    want = expect(to, xs, xs, g)
    scale = got.scale[:, some] if to == "fp8" else got.scale[some]
    assert np.array_equal(scale.cpu().numpy(), want[1])
    codes = got.q.view(torch.uint8)
    assert np.array_equal(codes[some].view(got.q.dtype).float().cpu().numpy(), want[0])
    assert torch.equal(x[some].cpu(), want[2])
    assert not codes[2:34567].any() and not codes[34568:m - 2].any()
    del x, codes, got
    torch.cuda.empty_cache()


def test_feeds_the_products_as_the_quantizers_do():
    """The fp8 codes of a norm kept in fp32 are those of the plain quantizer on it, the int8 ones nearly, and go into both products."""
    x, r, g = inputs(11, 40, 640, "f32", "f32")
    a = prism.add_rmsnorm_quantize_fp8(on(x), on(g), EPS, residual=on(r), norm=True)
    b = prism.add_rmsnorm_quantize_rows(on(x), on(g), EPS, residual=on(r))
    q, s = prism.quantize_blocks_fp8(a.norm)
    assert torch.equal(q.view(torch.uint8), a.q.view(torch.uint8)) and torch.equal(s, a.scale)
    qi, si = prism.quantize_rows(a.norm)
    # its row scale is a quotient, one step from the product at the most; codes then differ next to ties only
    assert ((si / b.scale - 1).abs() <= 2.0 ** -22).all() and (qi.int() - b.q.int()).abs().max() <= 1
    assert (qi != b.q).float().mean() <= 1e-3
    w = torch.randn((96, 640), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    y = prism.gemm_fp8_blockscale(a.q, a.scale, *prism.quantize_tiles_fp8(w))
    wi, swi = prism.quantize_rows(w)
    z = prism.gemm_w8a8(b.q, b.scale, wi, swi)
    exact = a.norm.double() @ w.double().t().contiguous()
    # one rounding to e4m3 on either side, 2^-4 / sqrt 3 of a value rms each; to int8, 1 / 254 of a row's largest
    assert torch.linalg.norm(y - exact) <= 0.06 * torch.linalg.norm(exact)
    assert torch.linalg.norm(z - exact) <= 0.06 * torch.linalg.norm(exact)


def test_streams_and_graphs():
    x, r, g = inputs(12, 50, 1296, "bf16", "f32")
    x, r, g = on(x), on(r), on(g)
    torch.cuda.synchronize()

    def step(x):
        h = prism.add_rmsnorm_quantize_fp8(x * 2, g, EPS, residual=r, norm=True)
        return h, prism.add_rmsnorm_quantize_rows(h.norm, g, EPS, residual=h.residual)

    eager = step(x)
    side = torch.cuda.Stream(device=DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        for a, b in zip(step(x), eager):
            for u, v in zip(a, b):
                assert (u is None and v is None) or torch.equal(u.float(), v.float())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x)
    for rep in range(4):
        for a in got:
            a.scale.fill_(float("nan"))
            a.residual.fill_(float("nan"))
        torch.randn((500, 500), device=DEV).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            for u, v in zip(a, b):
                assert (u is None and v is None) or torch.equal(u.float(), v.float()), rep


def test_refusals_of_the_binding():
    x, r, g = (on(t) for t in inputs(13, 4, 256, "bf16", "bf16"))
    f = prism.add_rmsnorm_quantize_fp8
    with pytest.raises(TypeError):
        f(x.double(), g)
    with pytest.raises(TypeError):
        f(x, g.double())
    with pytest.raises(ValueError, match="gain"):
        f(x, g[:128])
    with pytest.raises(ValueError, match="gain"):
        f(x, g.cpu())
    with pytest.raises(TypeError, match="residual"):
        f(x, g, residual=r.half())
    with pytest.raises(TypeError, match="residual"):
        f(x.float(), g, residual=r)
    with pytest.raises(ValueError, match="residual"):
        f(x, g, residual=r[:2])
    with pytest.raises(ValueError, match="residual"):
        f(x, g, residual_out=r)
    with pytest.raises(ValueError, match="residual_out"):
        f(x, g, residual=r, residual_out=r.float())
    with pytest.raises(ValueError, match="overlapping"):
        f(x, g, residual=r, residual_out=r[:1].expand(4, 256))
    with pytest.raises(ValueError, match="contiguous rows"):
        f(x.t(), g[:4])
    with pytest.raises(TypeError):
        f(x, g, norm=torch.empty((4, 256), device=DEV))
    with pytest.raises(TypeError):
        f(x, g, q=torch.empty((4, 256), dtype=torch.int8, device=DEV))
    with pytest.raises(ValueError, match="scale"):
        f(x, g, scale=torch.empty((4, 2), device=DEV))
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(prism.PrismError):
            f(x, g, eps)
    with pytest.raises(prism.PrismError) as e:
        f(x[:, 1:129], g[:128])
    assert e.value.status == -2
    with pytest.raises(prism.PrismError) as e:
        f(x, g, residual=torch.zeros((4, 264), dtype=torch.bfloat16, device=DEV)[:, 4:260])
    assert e.value.status == -2
    with pytest.raises(prism.PrismError):
        f(torch.zeros((1, 65552), device=DEV), torch.zeros((65552,), device=DEV))


@pytest.mark.parametrize("to", ["fp8", "int8"])
def test_empty_batches(to):
    x = torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)
    got = call(to, x, torch.ones((256,), device=DEV), EPS, residual=x, norm=True)
    assert got.q.shape == (0, 256) and got.residual.shape == (0, 256) and got.norm.shape == (0, 256)
    assert got.scale.shape == ((2, 0) if to == "fp8" else (0,))
