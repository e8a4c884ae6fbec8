"""Routing and the weighted sum of expert outputs on the GPU against plain 64-bit references.

Ids, offsets, rows and slots are compared exactly: keys are logits, or sums in 64 bits that two different experts of
these inputs do not share.  A weight is a few 64-bit operations, below 2^-50, and one rounding to fp32: within 2^-24 +
2^-40 of its value, or the smallest subnormal.

Weighted sum: one fma for each choice in fp32, each off by at most 2^-24 of the magnitudes added so far, T in all:
    |y - exact| <= top 2^-24 (1 + 2^-20) T + eps / 2 (|exact| + that) + the smallest subnormal of a 16-bit y.
"""
import numpy as np
import pytest
import torch

import moe_ref as ref
from exact_int8_gemm_amd import prism
from gpu_util import DEV

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = {"f32": 2.0 ** -23, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}


def host(t):
    return t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def logits(seed, m, e, kind, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((m, e), generator=g) * 2 + torch.randn((e,), generator=g)
    if masked:
        z[torch.rand((m, e), generator=g) < masked] = -float("inf")
    return z.to(TYPES[kind])


def check_route(z, r, top, **kw):
    ids, w, off, rows, slots = ref.route(z.float().numpy(), top, **kw)
    assert np.array_equal(host(r.ids), ids)
    assert np.array_equal(host(r.offsets), off)
    assert np.array_equal(host(r.rows), rows)
    assert np.array_equal(host(r.slots), slots)
    got = r.weights.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(w))
    live = ~np.isnan(w)
    assert (np.abs(got[live] - w[live]) <= (2.0 ** -24 + 2.0 ** -40) * np.abs(w[live]) + 2.0 ** -149).all()


SHAPES = [(1, 1, 1), (1, 2, 2), (1, 64, 8), (3, 8, 2), (4, 128, 8), (31, 61, 6), (32, 64, 4), (33, 65, 5), (64, 7, 7),
          (65, 160, 6), (100, 256, 8), (257, 512, 10), (40, 1024, 32), (500, 60, 4), (1001, 128, 8)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("m,e,top", SHAPES)
def test_route(m, e, top, kind):
    z = logits(m * 31 + e, m, e, kind)
    check_route(z, prism.route_experts(z.to(DEV), top), top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("m,e,top", [(1, 64, 8), (5, 61, 6), (40, 256, 8), (70, 300, 3), (35, 1000, 16)])
def test_scores_and_bias(m, e, top, biased, renormalize, score):
    z = logits(m + e, m, e, "f32", masked=0.2)
    bias = torch.randn((e,), generator=torch.Generator().manual_seed(e)) * 0.3 if biased else None
    r = prism.route_experts(z.to(DEV), top, score=score, bias=None if bias is None else bias.to(DEV),
                            renormalize=renormalize, scale=2.5)
    check_route(z, r, top, score=score, bias=None if bias is None else bias.numpy(), renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("m", [5, 40, 203])
def test_masks_and_special_values(m, biased):
    """Rows with fewer open experts than choices, none at all, NaN and infinities; experts that a bias closes."""
    e, top = 70, 6
    z = logits(m, m, e, "f32", masked=0.93)
    z[0] = -float("inf")
    z[1, :] = -float("inf")
    z[1, 69] = -1000.0
    z[2, 5] = float("nan")
    z[3, 64] = float("inf")
    z[4] = 0.0
    z[4, 10] = -0.0
    if m > 5:
        z[7] = -3.0e38
        z[8] = torch.linspace(-400, 400, e)
    bias = None
    if biased:
        bias = torch.randn((e,), generator=torch.Generator().manual_seed(1))
        bias[3], bias[66], bias[20] = -float("inf"), float("nan"), 30.0
    for score in ("softmax", "sigmoid"):
        r = prism.route_experts(z.to(DEV), top, score=score, bias=None if bias is None else bias.to(DEV))
        check_route(z, r, top, score=score, bias=None if bias is None else bias.numpy())


@pytest.mark.parametrize("kind", list(TYPES))
def test_equal_logits_go_to_the_lower_index(kind):
    """Few different values, so that ties stand at the border of the choice in every row."""
    g = torch.Generator().manual_seed(3)
    z = torch.randint(-2, 3, (90, 200), generator=g).to(TYPES[kind])
    bias = torch.randint(0, 2, (200,), generator=g).float() * 0.25
    check_route(z, prism.route_experts(z.to(DEV), 9), 9)
    check_route(z, prism.route_experts(z.to(DEV), 9, score="sigmoid", bias=bias.to(DEV)), 9, score="sigmoid",
                bias=bias.numpy())


@pytest.mark.parametrize("kind", list(TYPES))
def test_strided_and_unaligned_rows(kind):
    z = logits(4, 50, 61, kind)
    wide = torch.full((50, 131), float("nan"), dtype=TYPES[kind], device=DEV)
    wide[:, 3:64] = z.to(DEV)
    check_route(z, prism.route_experts(wide[:, 3:64], 5), 5)


def test_one_expert_gets_all_and_others_none():
    z = torch.zeros((300, 64))
    z[:, 63] = 5
    z[:, 0] = 4
    check_route(z, prism.route_experts(z.to(DEV), 2), 2)


def sorted_by_torch(ids, e):
    key = torch.where(ids < 0, e, ids).view(-1).long()
    ordered, order = torch.sort(key, stable=True)
    off = torch.searchsorted(ordered, torch.arange(e + 1, device=ids.device))
    rows = torch.where(ordered < e, order // ids.shape[1], -1)
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order), device=ids.device)
    return off, rows, torch.where(ids < 0, -1, place.view(ids.shape))


@pytest.mark.parametrize("m,e,top", [(16384, 64, 8), (16385, 256, 4), (40000, 33, 3), (100003, 128, 2)])
def test_many_tokens(m, e, top):
    """More than one pass a workgroup: the choices against torch's sort, the list against a stable one."""
    z = logits(5, m, e, "f32").to(DEV)
    z[11::97] = -float("inf")
    r = prism.route_experts(z, top)
    best, at = torch.sort(z, dim=1, descending=True, stable=True)
    ids = torch.where(best[:, :top] == -float("inf"), -1, at[:, :top])
    assert torch.equal(r.ids.long(), ids)
    for got, want in zip((r.offsets, r.rows, r.slots), sorted_by_torch(r.ids, e)):
        assert torch.equal(got.long(), want)


def test_tokens_do_not_depend_on_the_batch():
    z = logits(6, 700, 128, "bf16").to(DEV)
    bias = torch.randn((128,), generator=torch.Generator().manual_seed(2)).to(DEV)
    for kw in ({}, {"score": "sigmoid", "bias": bias}, {"renormalize": False}):
        whole = prism.route_experts(z, 8, **kw)
        for lo, hi in ((0, 1), (699, 700), (40, 72), (100, 300)):
            part = prism.route_experts(z[lo:hi], 8, **kw)
            assert torch.equal(part.ids, whole.ids[lo:hi]) and torch.equal(part.weights, whole.weights[lo:hi])
        again = prism.route_experts(z, 8, **kw)
        for a, b in zip(again, whole):
            assert torch.equal(a, b)


def test_route_with_a_given_workspace_and_graphs():
    """Two captured calls that share a workspace, replayed with eager work in between."""
    z1, z2 = logits(7, 90, 64, "f32").to(DEV), logits(8, 300, 64, "f32").to(DEV)
    ws = torch.empty((prism.route_experts_workspace(300, 64) + 64,), dtype=torch.uint8, device=DEV)
    eager = [prism.route_experts(z, 4, workspace=ws) for z in (z1, z2)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for z in (z1, z2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(prism.route_experts(z, 4, workspace=ws))
        graphs.append(g)
    for rep in range(4):
        for r in got:
            for t in r:
                t.fill_(-7)
        ws.fill_(255)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            for u, v in zip(a, b):
                assert torch.equal(u, v), rep


def test_route_refusals():
    z = torch.zeros((40, 64), device=DEV)
    with pytest.raises(TypeError):
        prism.route_experts(z.double(), 2)
    with pytest.raises(ValueError):
        prism.route_experts(z, 0)
    with pytest.raises(ValueError):
        prism.route_experts(z, 33)
    with pytest.raises(prism.PrismError):
        prism.route_experts(z[:, :4], 5)
    with pytest.raises(ValueError, match="score"):
        prism.route_experts(z, 2, score="relu")
    with pytest.raises(ValueError, match="bias"):
        prism.route_experts(z, 2, bias=torch.zeros((63,), device=DEV))
    with pytest.raises(TypeError):
        prism.route_experts(z, 2, bias=torch.zeros((64,), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(prism.PrismError):
        prism.route_experts(z, 2, workspace=torch.empty((8,), dtype=torch.uint8, device=DEV))
    with pytest.raises(prism.PrismError):
        prism.route_experts(z, 2, scale=float("nan"))
    with pytest.raises(prism.PrismError):
        prism.route_experts(torch.zeros((2, 1025), device=DEV), 2)


def test_route_empty_batch():
    r = prism.route_experts(torch.empty((0, 64), device=DEV), 4)
    assert r.ids.shape == (0, 4) and r.rows.shape == (0,) and torch.equal(r.offsets, torch.zeros_like(r.offsets))


# ------------------------------------------------------------ weighted sum

def combine_input(seed, m, top, n, kind, out, add, holes=0.1):
    g = torch.Generator().manual_seed(seed)
    r = m * top + 3
    x = torch.randn((r, n), generator=g).to(TYPES[kind])
    w = torch.randn((m, top), generator=g)
    slots = torch.randint(0, r, (m, top), generator=g).to(torch.int32)
    slots[torch.rand((m, top), generator=g) < holes] = -1
    slots[torch.rand((m, top), generator=g) < holes / 4] = r
    a = torch.randn((m, n), generator=g).to(TYPES[out]) if add else None
    return x, w, slots, a


def check_combine(x, w, slots, a, y, out):
    want, mag = ref.combine(x.float().numpy(), w.numpy(), slots.numpy(), None if a is None else a.float().numpy())
    sums = slots.shape[1] * 2.0 ** -24 * (1 + 2.0 ** -20) * mag
    tol = sums + (0 if out == "f32" else EPS[out] / 2 * (np.abs(want) + sums) + 2.0 ** -25)
    assert (np.abs(y.cpu().double().numpy() - want) <= tol).all()


@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("m,top,n", [(1, 1, 1), (1, 8, 2560), (3, 2, 7), (5, 8, 33), (17, 9, 264), (64, 32, 100),
                                     (130, 6, 1021), (40, 4, 4096)])
@pytest.mark.parametrize("add", [False, True])
def test_combine(m, top, n, kind, out, add):
    x, w, slots, a = combine_input(m + top + n, m, top, n, kind, out, add)
    y = prism.combine_experts(x.to(DEV), w.to(DEV), slots.to(DEV), add=None if a is None else a.to(DEV),
                              out_dtype=TYPES[out])
    check_combine(x, w, slots, a, y, out)


@pytest.mark.parametrize("kind", list(TYPES))
def test_combine_in_place_unaligned_and_not_outside(kind):
    m, top, n = 9, 3, 77
    x, w, slots, a = combine_input(1, m, top, n, kind, kind, True)
    buf = torch.full((m * n + 64,), 5.0, dtype=TYPES[kind], device=DEV)
    y = buf[1:1 + m * n].view(m, n)
    y.copy_(a)
    wide = torch.zeros((x.numel() + 1,), dtype=TYPES[kind], device=DEV)
    xs = wide[1:].view(x.shape)
    xs.copy_(x)
    got = prism.combine_experts(xs, w.to(DEV), slots.to(DEV), add=y, y=y)
    assert got is y and buf[0] == 5 and (buf[1 + m * n:] == 5).all()
    check_combine(x, w, slots, a, y, kind)


def test_combine_empty_choices_and_nan_weights():
    x = torch.full((4, 40), float("nan"), device=DEV)
    slots = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    w = torch.zeros((3, 2), device=DEV)
    add = torch.randn((3, 40), device=DEV)
    assert not prism.combine_experts(x, w, slots).any()          # rows that no slot names are not looked at
    assert torch.equal(prism.combine_experts(x, w, slots, add=add), add)
    w[1] = float("nan")                                          # a token without a valid routing shows
    y = prism.combine_experts(x, w, slots, add=add)
    assert torch.isnan(y[1]).all() and torch.equal(y[[0, 2]], add[[0, 2]])
    assert not prism.combine_experts(x[:0], torch.ones_like(w), slots + 1).any()


def test_combine_rows_do_not_depend_on_the_batch():
    x, w, slots, a = (t.to(DEV) for t in combine_input(2, 300, 8, 1003, "bf16", "bf16", True))
    whole = prism.combine_experts(x, w, slots, add=a)
    for lo, hi in ((0, 1), (299, 300), (17, 90)):
        part = prism.combine_experts(x, w[lo:hi].contiguous(), slots[lo:hi].contiguous(), add=a[lo:hi].contiguous())
        assert torch.equal(part, whole[lo:hi])


@pytest.mark.parametrize("kind,n", [("bf16", 8200), ("f16", 8197), ("f32", 4100)])
def test_combine_of_more_than_the_caches_hold(kind, n):
    """Over 256 MB of x: whole numbers and weights that are powers of two, exact in any order."""
    m, top = 2100, 8
    g = torch.Generator(device=DEV).manual_seed(n)
    x = torch.randint(-3, 4, (m * top, n), generator=g, device=DEV).to(TYPES[kind])
    assert x.numel() * x.element_size() > 2 ** 28
    w = torch.exp2(torch.randint(-1, 2, (m, top), generator=g, device=DEV).float())
    slots = torch.randperm(m * top, generator=g, device=DEV).view(m, top).to(torch.int32)
    slots[::5, 3] = -1
    add = torch.randint(-3, 4, (m, n), generator=g, device=DEV).to(TYPES[kind])
    want = add.float().clone()
    for j in range(top):
        part = x[slots[:, j].clamp(min=0).long()].float() * w[:, j, None]
        want += torch.where(slots[:, j, None] >= 0, part, 0.0)
    y = add.clone()
    assert prism.combine_experts(x, w, slots, add=y, y=y) is y
    assert torch.equal(y, want.to(TYPES[kind]))
    assert torch.equal(prism.combine_experts(x, w, slots, add=add), y)


def test_combine_past_32_bit_offsets():
    r, n = 131200, 16500
    assert r * n > 2 ** 31
    x = torch.zeros((r, n), dtype=torch.bfloat16, device=DEV)
    x[-1] = torch.arange(n, device=DEV) % 64
    x[-2] = 3
    slots = torch.tensor([[r - 1, r - 2], [0, r - 1]], dtype=torch.int32, device=DEV)
    y = prism.combine_experts(x, torch.tensor([[1.0, 2.0], [5.0, 0.5]], device=DEV), slots)
    base = (torch.arange(n, device=DEV) % 64).bfloat16()
    assert torch.equal(y[0], base + 6) and torch.equal(y[1], base / 2)
    del x
    torch.cuda.empty_cache()


def test_combine_refusals():
    x, w = torch.zeros((8, 16), device=DEV), torch.zeros((4, 2), device=DEV)
    s = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        prism.combine_experts(x, w, s.long())
    with pytest.raises(ValueError):
        prism.combine_experts(x, w[:2], s)
    with pytest.raises(TypeError):
        prism.combine_experts(x, w, s, out_dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        prism.combine_experts(x.bfloat16(), w, s, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        prism.combine_experts(x, w, s, add=torch.zeros((4, 15), device=DEV))
    with pytest.raises(TypeError):
        prism.combine_experts(x.bfloat16(), w, s, add=torch.zeros((4, 16), device=DEV), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        prism.combine_experts(x.t(), w, s)
    with pytest.raises(prism.PrismError):
        prism.combine_experts(x, torch.zeros((1, 33), device=DEV), torch.zeros((1, 33), dtype=torch.int32, device=DEV))
    assert prism.combine_experts(x, w[:0], s[:0]).shape == (0, 16)
