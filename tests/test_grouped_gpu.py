"""The fp8 GEMM grouped by expert on the GPU.

Its definition is the dense product's, row by row, and so are its bits: each group is compared bit for bit with
gemm_fp8_blockscale on the same rows and that expert's weights, whose own tests hold it to 64-bit references; and small
integers with powers of two for scales, where every sum is exact in any order, are compared with exact results.
"""
import numpy as np
import pytest
import torch

from exact_int8_gemm_amd import prism
from gpu_util import DEV

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)


def operands(seed, m, e, n, k, integers=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kb, nb = -(-k // 128), -(-n // 128)
    if integers:
        q = torch.randint(-2, 3, (m, k), generator=g, device=DEV).float().to(prism.FP8)
        w = torch.randint(-2, 3, (e, n, k), generator=g, device=DEV).float().to(prism.FP8)
        sa = torch.exp2(torch.randint(-2, 3, (kb, m), generator=g, device=DEV).float())
        sw = torch.exp2(torch.randint(-2, 3, (e, nb, kb), generator=g, device=DEV).float())
        return q, sa, w, sw
    x = torch.randn((m, k), generator=g, device=DEV)
    x *= torch.where(torch.rand((k,), generator=g, device=DEV) < 0.01, 20.0, 1.0)
    q, sa = prism.quantize_blocks_fp8(x)
    w = torch.empty((e, n, k), dtype=prism.FP8, device=DEV)
    sw = torch.empty((e, nb, kb), device=DEV)
    for i in range(e):
        prism.quantize_tiles_fp8(torch.randn((n, k), generator=g, device=DEV) * 0.02, q=w[i], scale=sw[i])
    return q, sa, w, sw


def take(q, sa, rows):
    """The rows of the codes and their scales; zeros where a row is outside."""
    ok = (rows >= 0) & (rows < q.shape[0])
    at = torch.where(ok, rows, 0).long()
    qi = torch.where(ok[:, None], q.view(torch.uint8)[at], 0).view(prism.FP8)
    return qi, torch.where(ok[None], sa[:, at], 0.0).contiguous()


def dense(q, sa, w, sw, counts, kind):
    """Group by group through the dense product."""
    parts, at = [], 0
    for i, c in enumerate(counts):
        if c:
            parts.append(prism.gemm_fp8_blockscale(q[at:at + c], sa[:, at:at + c].contiguous(), w[i], sw[i],
                                                   out_dtype=TYPES[kind]))
        at += c
    return torch.cat(parts)


def ragged(rng, rows, e, empty=0.3):
    p = rng.random(e) ** 2 * (rng.random(e) >= empty) + 1e-9
    return rng.multinomial(rows, p / p.sum())


SHAPES = [(1, 1, 1, 16), (1, 4, 33, 128), (3, 2, 129, 144), (8, 64, 320, 2064), (17, 5, 100, 400), (40, 130, 272, 528),
          (64, 3, 200, 1040), (100, 9, 1030, 272), (130, 16, 257, 640), (300, 7, 128, 4112), (600, 60, 144, 1168),
          (1000, 4, 640, 384), (2500, 11, 300, 272), (2000, 2, 520, 1296), (1500, 257, 130, 144), (700, 1024, 48, 80)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("r,e,n,k", SHAPES)
def test_bits_of_the_dense_product(r, e, n, k, gather, kind):
    rng = np.random.default_rng(r + e + n + k)
    counts = ragged(rng, r, e)
    m = max(1, r // 3) if gather else r
    q, sa, w, sw = operands(r + e, m, e, n, k)
    rows = torch.from_numpy(rng.integers(0, m, r).astype(np.int32)).to(DEV) if gather else None
    y = prism.gemm_fp8_grouped(q, sa, w, sw, offsets_of(counts), rows=rows, out_dtype=TYPES[kind])
    if gather:
        q, sa = take(q, sa, rows)
    assert torch.equal(bits(y), bits(dense(q, sa, w, sw, counts, kind)))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("r,e,n,k", SHAPES)
def test_exact_on_small_integers(r, e, n, k, kind):
    rng = np.random.default_rng(r * e + n + k)
    counts = ragged(rng, r, e)
    m = max(1, r // 2)
    q, sa, w, sw = operands(r + 1, m, e, n, k, integers=True)
    rows = torch.from_numpy(rng.integers(0, m, r).astype(np.int32)).to(DEV)
    y = prism.gemm_fp8_grouped(q, sa, w, sw, offsets_of(counts), rows=rows, out_dtype=TYPES[kind])
    a = (q.double() * sa.double().repeat_interleave(128, 0)[:k].t())[rows.long()]
    at = 0
    for i, c in enumerate(counts):
        if c:
            b = w[i].double() * sw[i].double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
            assert torch.equal(y[at:at + c], torch.mm(a[at:at + c], b.t().contiguous()).to(TYPES[kind])), i
        at += c


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,n,k", [
    ([700, 0, 1, 300, 2000, 129, 0, 0, 255], 1300, 400), ([0, 0, 5000], 640, 272), ([4096], 1300, 272),
    ([1] * 64, 2576, 400), ([16] * 40, 1300, 656), ([15, 17] * 30, 640, 1040), ([64] * 33, 2048, 528),
    ([128, 127, 129] * 10, 2176, 272), ([256] * 24, 2560, 400), ([300] * 40, 1472, 272), ([1000, 3] * 12, 1024, 528)])
def test_groups_of_many_sizes(counts, n, k, gather, kind):
    """Groups around every tile's size, many of them, and one that holds all."""
    r, e = sum(counts), len(counts)
    m = r // 4 + 1 if gather else r
    q, sa, w, sw = operands(r, m, e, n, k)
    rows = torch.randint(0, m, (r,), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(torch.int32)
    y = prism.gemm_fp8_grouped(q, sa, w, sw, offsets_of(counts), rows=rows if gather else None, out_dtype=TYPES[kind])
    if gather:
        q, sa = take(q, sa, rows)
    assert torch.equal(bits(y), bits(dense(q, sa, w, sw, counts, kind)))


# Sizes at which a bf16 y takes the kernel of 256-column tiles: heights of 64 to 256 rows, tiles cut in the last round,
# one to eight rounds, an odd number of blocks, a partial last one, the fewest blocks it takes, over 64 groups.
WIDE = [([1, 64, 65, 128, 129, 192, 193, 256, 257, 320, 449, 600, 1000, 0, 700], 2560, 656),
        ([3000, 5, 2000], 2576, 640), ([8192], 2560, 768), ([260] * 64, 2560, 1152), ([512] * 20, 5000, 1040),
        ([0] * 7 + [150] * 100, 2560, 656), ([200] * 300, 1280, 656), ([64, 640] * 12, 2560, 5120),
        ([320] * 16, 2560, 1296)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,n,k", WIDE)
def test_wide_tiles(counts, n, k, gather):
    r, e = sum(counts), len(counts)
    m = r // 5 if gather else r
    q, sa, w, sw = operands(r + k, m, e, n, k)
    rows = torch.randint(0, m, (r,), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).to(torch.int32)
    off = offsets_of(counts)
    y = prism.gemm_fp8_grouped(q, sa, w, sw, off, rows=rows if gather else None, out_dtype=torch.bfloat16)
    again = prism.gemm_fp8_grouped(q, sa, w, sw, off, rows=rows if gather else None, out_dtype=torch.bfloat16)
    if gather:
        q, sa = take(q, sa, rows)
    assert torch.equal(bits(y), bits(dense(q, sa, w, sw, counts, "bf16")))
    assert torch.equal(bits(y), bits(again))


@pytest.mark.parametrize("gather", [False, True])
def test_wide_tiles_exact_and_not_outside(gather):
    """Whole numbers, exact in any order; offsets from behind 0 to before the end, rows outside q, y at an odd element
    with memory around it, codes at any 16 bytes with NaN around them, NaN scales and codes."""
    counts, lead, n, k = [700, 0, 1300, 64, 1900], 37, 2569, 656
    used, e = sum(counts), len(counts)
    r = lead + used + 91
    m = 900 if gather else r
    q, sa, w, sw = operands(12, m, e, n, k, integers=True)
    bq = torch.full((m * k + 256,), 0x7F, dtype=torch.uint8, device=DEV)
    bw = torch.full((e * n * k + 256,), 0x7F, dtype=torch.uint8, device=DEV)
    q1, w1 = bq[48:48 + m * k].view(m, k), bw[112:112 + e * n * k].view(e, n, k)
    q1.copy_(q.view(torch.uint8))
    w1.copy_(w.view(torch.uint8))
    rows = torch.randint(-3, m + 3, (r,), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    rows = rows.to(torch.int32) if gather else torch.arange(r, dtype=torch.int32, device=DEV)
    if gather:
        rows[lead + 5], rows[lead + used - 1] = -2 ** 31, 2 ** 31 - 1
    off = offsets_of(counts) + lead
    buf = torch.full((r * n + 513,), 5.0, dtype=torch.bfloat16, device=DEV)
    y = buf[1:1 + r * n].view(r, n)
    prism.gemm_fp8_grouped(q1.view(prism.FP8), sa, w1.view(prism.FP8), sw, off, rows=rows if gather else None, y=y)
    assert (buf[:1 + lead * n] == 5).all() and (buf[1 + (lead + used) * n:] == 5).all()
    ok = (rows >= 0) & (rows < m)
    a = (q.double() * sa.double().repeat_interleave(128, 0)[:k].t())[torch.where(ok, rows, 0).long()]
    a = torch.where(ok[:, None], a, 0.0)
    at = lead
    want = []
    for i, c in enumerate(counts):
        b = w[i].double() * sw[i].double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
        want.append(torch.mm(a[at:at + c], b.t().contiguous()).to(torch.bfloat16))
        at += c
    want = torch.cat(want)
    assert torch.equal(y[lead:lead + used], want)
    # a NaN scale of one row of q, a NaN code of one column of an expert
    sa[2, 7] = float("nan")
    w1[2, n - 1, k - 1] = 0x7F
    prism.gemm_fp8_grouped(q1.view(prism.FP8), sa, w1.view(prism.FP8), sw, off, rows=rows if gather else None, y=y)
    bad = torch.zeros((used, n), dtype=torch.bool, device=DEV)
    bad[(rows == 7)[lead:lead + used]] = True
    bad[700:2000, n - 1] = True
    got = y[lead:lead + used]
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], want[~bad])


def test_wide_tiles_with_descending_offsets():
    """What is written of y is not specified; nothing else is."""
    r, n, k, e = 5005, 2576, 656, 9
    q, sa, w, sw = operands(13, r, e, n, k)
    buf = torch.full((r * n + 512,), 5.0, dtype=torch.bfloat16, device=DEV)
    for off in ([0, r, 0, r, -1, r, 3, r, 2 ** 31 - 1, 0], [r, 0, r, 0, r, 0, r, 0, r, 0], [-2 ** 31] * 9 + [2 ** 31 - 1]):
        prism.gemm_fp8_grouped(q, sa, w, sw, torch.tensor(off, dtype=torch.int32, device=DEV), y=buf[:r * n].view(r, n))
        assert (buf[r * n:] == 5).all()
    want = prism.gemm_fp8_blockscale(q, sa, w[8], sw[8], out_dtype=torch.bfloat16)
    assert torch.equal(bits(buf[:r * n].view(r, n)), bits(want))      # the last list is in order: all rows are expert 8's


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("r", [3, 70, 900])
def test_rows_outside_the_groups_are_left(r, kind):
    """Offsets that begin behind 0 and end before R, row numbers outside q, and memory around y."""
    n, k, e, m = 161, 272, 6, 50
    q, sa, w, sw = operands(r, m, e, n, k)
    lo, hi = r // 3, r - r // 3
    cut = np.sort(np.random.default_rng(r).integers(lo, hi + 1, e - 1))
    off = torch.tensor([lo, *cut, hi], dtype=torch.int32, device=DEV)
    rows = torch.randint(-5, m + 5, (r,), generator=torch.Generator(device=DEV).manual_seed(r), device=DEV).to(torch.int32)
    rows[lo] = -2 ** 31
    rows[hi - 1] = 2 ** 31 - 1
    buf = torch.full((r * n + 512,), 5.0, dtype=TYPES[kind], device=DEV)
    y = buf[:r * n].view(r, n)
    assert prism.gemm_fp8_grouped(q, sa, w, sw, off, rows=rows, y=y) is y
    assert (y[:lo] == 5).all() and (buf[hi * n:] == 5).all()
    qi, si = take(q, sa, rows[lo:hi])
    want = dense(qi, si, w, sw, np.diff([lo, *cut, hi]), kind)
    assert torch.equal(bits(y[lo:hi]), bits(want))


@pytest.mark.parametrize("r", [40, 1200])
def test_offsets_outside_the_rows(r):
    """Taken as clamped; where they descend, y holds something, and nothing else is written."""
    n, k, e = 130, 144, 4
    q, sa, w, sw = operands(1, r, e, n, k)
    want = dense(q, sa, w, sw, [r // 2, 0, r - r // 2, 0], "f32")
    off = torch.tensor([-9, r // 2, r // 2, 2 ** 31 - 1, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    assert torch.equal(prism.gemm_fp8_grouped(q, sa, w, sw, off), want)
    buf = torch.full((r * n + 512,), 5.0, device=DEV)
    off = torch.tensor([0, r, -2 ** 31, r, 0], dtype=torch.int32, device=DEV)
    prism.gemm_fp8_grouped(q, sa, w, sw, off, y=buf[:r * n].view(r, n))
    assert (buf[r * n:] == 5).all()
    off = torch.zeros_like(off)
    y = torch.full((r, n), 5.0, device=DEV)
    assert (prism.gemm_fp8_grouped(q, sa, w, sw, off, y=y) == 5).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_rows_do_not_depend_on_the_batch(kind):
    """The same rows in calls of few and of many others, in groups of any size, gathered or not."""
    n, k, e = 528, 1040, 8
    q, sa, w, sw = operands(3, 64, e, n, k)
    rng = np.random.default_rng(3)

    def run(lists):
        rows = torch.tensor(sum(lists, []), dtype=torch.int32, device=DEV)
        y = bits(prism.gemm_fp8_grouped(q, sa, w, sw, offsets_of([len(v) for v in lists]), rows=rows,
                                        out_dtype=TYPES[kind]))
        at = np.cumsum([0] + [len(v) for v in lists])
        return [y[a:b] for a, b in zip(at, at[1:])]

    alone = [run([[5] if j == i else [] for j in range(e)])[i] for i in range(e)]
    for per in (1, 3, 16, 40, 130, 300, 700):
        lists = [list(map(int, rng.integers(0, 64, rng.integers(1, 2 * per)))) for _ in range(e)]
        for v in lists:
            v[len(v) // 2] = 5
        got = run(lists)
        for i in range(e):
            assert torch.equal(got[i][len(lists[i]) // 2], alone[i][0]), (per, i)
        for a, b in zip(got, run(lists)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("r", [5, 90, 1000])
def test_special_values(r, kind):
    """NaN scales and codes spoil their own row, or their expert's column, only."""
    n, k, e = 200, 400, 3
    q, sa, w, sw = operands(4, r, e, n, k)
    counts = [r // 2, 0, r - r // 2]
    off = offsets_of(counts)
    clean = prism.gemm_fp8_grouped(q, sa, w, sw, off, out_dtype=TYPES[kind])
    sa2, qd, wd = sa.clone(), q.view(torch.uint8).clone(), w.view(torch.uint8).clone()
    sa2[1, r - 1] = float("nan")
    qd[0, 399] = 0x7F
    wd[2, 199, 0] = 0xFF
    wd[1] = 0x7F                      # an expert without rows
    y = prism.gemm_fp8_grouped(qd.view(prism.FP8), sa2, wd.view(prism.FP8), sw, off, out_dtype=TYPES[kind])
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0] = bad[r - 1] = True
    bad[counts[0]:, 199] = True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("r,n,k", [(6, 33, 144), (300, 161, 272), (1500, 129, 400)])
def test_unaligned_output_and_codes(r, n, k, kind):
    """y at an odd element, and codes that start at any 16 bytes, with NaN codes around them."""
    e = 3
    counts = [r // 3, r - r // 3 - 1, 1]
    q, sa, w, sw = operands(5, r, e, n, k)
    want = dense(q, sa, w, sw, counts, kind)
    bq = torch.full((r * k + 256,), 0x7F, dtype=torch.uint8, device=DEV)
    bw = torch.full((e * n * k + 256,), 0x7F, dtype=torch.uint8, device=DEV)
    q1, w1 = bq[48:48 + r * k].view(r, k), bw[112:112 + e * n * k].view(e, n, k)
    q1.copy_(q.view(torch.uint8))
    w1.copy_(w.view(torch.uint8))
    buf = torch.zeros((r * n + 1,), dtype=TYPES[kind], device=DEV)
    y = prism.gemm_fp8_grouped(q1.view(prism.FP8), sa, w1.view(prism.FP8), sw, offsets_of(counts), y=buf[1:].view(r, n))
    assert torch.equal(bits(y), bits(want))


def test_weights_past_32_bit_offsets():
    e, n, k = 70, 8200, 8208
    assert e * n * k > 2 ** 32
    g = torch.Generator(device=DEV).manual_seed(6)
    w = torch.zeros((e, n, k), dtype=torch.uint8, device=DEV)
    w[e - 1] = torch.randint(0, 120, (n, k), generator=g, device=DEV).to(torch.uint8)
    w = w.view(prism.FP8)
    sw = torch.rand((e, -(-n // 128), -(-k // 128)), generator=g, device=DEV)
    for r in (3, 200, 2000):
        q, sa = prism.quantize_blocks_fp8(torch.randn((r, k), generator=g, device=DEV))
        counts = [1] + [0] * (e - 2) + [r - 1]
        y = prism.gemm_fp8_grouped(q, sa, w, sw, offsets_of(counts), out_dtype=torch.bfloat16)
        assert torch.equal(bits(y), bits(dense(q, sa, w, sw, counts, "bf16"))) and (y[1:] != 0).any()
    del w, sw
    torch.cuda.empty_cache()


def test_outputs_and_rows_past_32_bit_offsets():
    """More than 2^31 outputs, and codes of more than 2^31 bytes where no row numbers are given."""
    r, n, k = 140000, 15500, 16
    assert r * n > 2 ** 31
    q, sa, w, sw = operands(7, r, 2, n, k, integers=True)
    y = prism.gemm_fp8_grouped(q, sa, w, sw, offsets_of([r - 500, 500]), out_dtype=torch.bfloat16)
    tail = dense(q[-900:], sa[:, -900:].contiguous(), w, sw, [400, 500], "bf16")
    assert torch.equal(y[-900:], tail)
    del y, q, sa, w, sw
    torch.cuda.empty_cache()
    r, n, k = 270000, 40, 8192
    assert r * k > 2 ** 31
    q = torch.zeros((r, k), dtype=torch.uint8, device=DEV).view(prism.FP8)
    tq, ts, w, sw = operands(8, 300, 2, n, k)
    q[-300:].view(torch.uint8).copy_(tq.view(torch.uint8))
    sa = torch.ones((k // 128, r), device=DEV)
    sa[:, -300:] = ts
    y = prism.gemm_fp8_grouped(q, sa, w, sw, offsets_of([r - 200, 200]))
    assert torch.equal(y[-300:], dense(tq, ts, w, sw, [100, 200], "f32")) and (y[:-300] == 0).all()
    del y, q, sa
    torch.cuda.empty_cache()


def test_streams_and_graphs():
    """Captured with offsets and rows that change between the replays, as routing makes them."""
    n, k, e, top = 300, 528, 16, 4
    w, sw = operands(9, 1, e, n, k)[2:]
    sizes = (3, 50, 600)
    q = [operands(10 + m, m, 1, 1, k)[:2] for m in sizes]
    z = [torch.randn((m, e), device=DEV) for m in sizes]

    def step():
        out = []
        for (qi, si), zi in zip(q, z):
            r = prism.route_experts(zi, top)
            out.append((r, prism.gemm_fp8_grouped(qi, si, w, sw, r.offsets, rows=r.rows, out_dtype=torch.bfloat16)))
        return out

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(4):
        for zi in z:
            zi.normal_()
        for _, y in got:
            y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream(device=DEV)
        with torch.cuda.stream(side):
            eager = step()
        side.synchronize()
        for (ra, ya), (rb, yb) in zip(got, eager):
            assert torch.equal(ra.rows, rb.rows) and torch.equal(bits(ya), bits(yb)), rep


def test_refusals():
    q, sa, w, sw = operands(11, 8, 3, 48, 256)
    off = offsets_of([3, 0, 5])
    rows = torch.zeros((8,), dtype=torch.int32, device=DEV)
    f = prism.gemm_fp8_grouped
    with pytest.raises(TypeError):
        f(q.view(torch.int8), sa, w, sw, off)
    with pytest.raises(ValueError):
        f(q, sa, w[0], sw, off)
    with pytest.raises(ValueError, match="w "):
        f(q, sa, w[:, :, :128].contiguous(), sw, off)
    with pytest.raises(ValueError, match="s_a"):
        f(q, sa[:1], w, sw, off)
    with pytest.raises(ValueError, match="s_w"):
        f(q, sa, w, sw[:2], off)
    with pytest.raises(ValueError, match="offsets"):
        f(q, sa, w, sw, off[:3])
    with pytest.raises(TypeError):
        f(q, sa, w, sw, off.long())
    with pytest.raises(TypeError):
        f(q, sa, w, sw, off, rows=rows.long())
    with pytest.raises(ValueError, match="rows"):
        f(q, sa, w, sw, off, rows=rows.view(2, 4))
    with pytest.raises(ValueError):
        f(q, sa, w, sw, off.cpu())
    with pytest.raises(ValueError, match="y "):
        f(q, sa, w, sw, off, rows=rows[:7], y=torch.empty((8, 48), device=DEV))
    with pytest.raises(TypeError):
        f(q, sa, w, sw, off, out_dtype=torch.float64)
    with pytest.raises(prism.PrismError) as e:
        q2, sa2, w2, sw2 = (torch.zeros((8, 40), dtype=torch.uint8, device=DEV).view(prism.FP8), sa[:1],
                            torch.zeros((3, 48, 40), dtype=torch.uint8, device=DEV).view(prism.FP8), sw[:, :, :1].contiguous())
        f(q2, sa2, w2, sw2, off)
    assert e.value.status == -2
    assert f(q, sa, w, sw, off, rows=rows[:0]).shape == (0, 48)
    assert f(q[:0], sa[:, :0].contiguous(), w, sw, torch.zeros_like(off)).shape == (0, 48)
