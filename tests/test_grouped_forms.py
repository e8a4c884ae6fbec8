"""The grouped fp8 GEMM, kernel by kernel: the query that names the kernel of a call (no GPU), and on the GPU, where each
test makes sure of the kernel it is about, offsets that descend, groups of a tile and a half, and weights and outputs past
32-bit offsets.  Bits are compared with the dense product's, group by group.
"""
import pytest
import torch

from exact_int8_gemm_amd import prism
from gpu_util import DEV
from test_grouped_gpu import bits, dense, offsets_of, operands, take

gpu = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def form(r, e, n, k, kind):
    return prism.gemm_fp8_grouped_form(r, e, n, k, TYPES[kind])


# ------------------------------------------------------------ the query

def test_every_form_is_named_and_reached():
    met = {kind: set() for kind in TYPES}
    for kind in TYPES:
        for e in (1, 8, 64):
            for r in (1, 8, 50, 300, 2000, 9000, 40000):
                for n in (16, 640, 2560):
                    for k in (144, 2560):
                        met[kind].add(form(r, e, n, k, kind))
    assert met["f32"] == met["f16"] == {"few", "64x64", "128x128"}
    assert met["bf16"] == {"64x64", "64x128", "128x128", "wide"}


def test_few_blocks_are_not_for_the_wide_kernel():
    assert form(40000, 8, 2560, 640, "bf16") == "wide" and form(40000, 8, 2560, 512, "bf16") != "wide"
    assert form(40000, 8, 2560, 528, "bf16") != "wide"


@pytest.mark.parametrize("r,e,n,k,status", [
    (0, 4, 16, 64, -1), (-1, 4, 16, 64, -1), (1 << 31, 4, 16, 64, -1), (8, 0, 16, 64, -1), (8, 1025, 16, 64, -1),
    (8, 4, 0, 64, -1), (8, 4, 1 << 31, 64, -1), (8, 4, 16, 0, -1), (8, 4, 16, 131056, -1), (8, 4, 16, 72, -2),
    ((1 << 31) - 1, 4, (1 << 31) - 1, 64, -1)])
def test_sizes_that_the_call_refuses(r, e, n, k, status):
    with pytest.raises(prism.PrismError) as err:
        form(r, e, n, k, "bf16")
    assert err.value.status == status


def test_unknown_types_are_refused():
    assert prism.lib().prism_gemm_fp8_grouped_form(3, 8, 4, 16, 64) == -1
    assert prism.lib().prism_gemm_fp8_grouped_form(-1, 8, 4, 16, 64) == -1
    with pytest.raises(TypeError):
        prism.gemm_fp8_grouped_form(8, 4, 16, 64, torch.float64)


# ------------------------------------------------------------ on the GPU

def gathered(gather, r, m, q, sa, seed=2):
    """(rows or None, the codes and scales that each row of y is made from)"""
    if not gather:
        return None, q, sa
    rows = torch.randint(0, m, (r,), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(torch.int32)
    return (rows, *take(q, sa, rows))


DESCENDING = [(5005, 3, 2576, 640, "bf16", "wide"), (9001, 9, 2576, 656, "bf16", "wide"), (700, 9, 528, 400, "bf16", "64x64"),
              (1100, 6, 1300, 400, "bf16", "64x128"), (5005, 9, 2576, 656, "bf16", "128x128"),
              (40, 9, 528, 400, "f32", "few"), (700, 9, 528, 400, "f16", "64x64"), (5005, 9, 1300, 400, "f32", "128x128")]


@gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("r,e,n,k,kind,name", DESCENDING)
def test_descending_offsets(r, e, n, k, kind, name, gather):
    """What is written of y is not specified; nothing else is, and an ordered list afterwards is whole."""
    assert form(r, e, n, k, kind) == name
    m = r // 3 if gather else r
    q, sa, w, sw = operands(r + e, m, e, n, k)
    rows, qr, sr = gathered(gather, r, m, q, sa)
    buf = torch.full((r * n + 1024,), 5.0, dtype=TYPES[kind], device=DEV)
    y = buf[512:512 + r * n].view(r, n)
    up, down = [0, r] * e, [r, 0] * e
    edges = ([-2 ** 31, 2 ** 31 - 1] * e)
    for off in (up[:e + 1], down[:e + 1], edges[:e + 1], list(range(r, r - e - 1, -1)), [r // 2] + up[:e]):
        prism.gemm_fp8_grouped(q, sa, w, sw, torch.tensor(off, dtype=torch.int32, device=DEV), rows=rows, y=y)
        assert (buf[:512] == 5).all() and (buf[512 + r * n:] == 5).all(), off
    counts = [0] * (e - 1) + [r]
    prism.gemm_fp8_grouped(q, sa, w, sw, offsets_of(counts), rows=rows, y=y)
    assert torch.equal(bits(y), bits(dense(qr, sr, w, sw, counts, kind)))


@gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,n,k", [([320] * 28, 2560, 1296), ([320] * 16, 5000, 656), ([129] * 50, 2560, 784)])
def test_wide_tiles_of_a_tile_and_a_half(counts, n, k, gather):
    r, e = sum(counts), len(counts)
    assert form(r, e, n, k, "bf16") == "wide"
    m = r // 5 if gather else r
    q, sa, w, sw = operands(r + k, m, e, n, k)
    rows, qr, sr = gathered(gather, r, m, q, sa)
    y = prism.gemm_fp8_grouped(q, sa, w, sw, offsets_of(counts), rows=rows, out_dtype=torch.bfloat16)
    assert torch.equal(bits(y), bits(dense(qr, sr, w, sw, counts, "bf16")))


@gpu
@pytest.mark.parametrize("r,e,n,k,kind,name", [(6, 210, 2560, 8208, "f32", "few"), (6, 210, 2560, 8208, "f16", "few"),
                                               (20000, 70, 8200, 8208, "bf16", "wide"),
                                               (20000, 70, 8200, 8208, "f32", "128x128"),
                                               (300, 70, 8200, 8208, "f16", "64x64")])
def test_weights_past_32_bit_offsets(r, e, n, k, kind, name):
    assert form(r, e, n, k, kind) == name and e * n * k > 2 ** 32
    g = torch.Generator(device=DEV).manual_seed(r)
    w = torch.zeros((e, n, k), dtype=torch.uint8, device=DEV)
    w[e - 2:] = torch.randint(0, 120, (2, n, k), generator=g, device=DEV).to(torch.uint8)
    w = w.view(prism.FP8)
    sw = torch.rand((e, -(-n // 128), -(-k // 128)), generator=g, device=DEV)
    q, sa = prism.quantize_blocks_fp8(torch.randn((r, k), generator=g, device=DEV))
    counts = [1] + [0] * (e - 3) + [r // 2, r - 1 - r // 2]
    y = prism.gemm_fp8_grouped(q, sa, w, sw, offsets_of(counts), out_dtype=TYPES[kind])
    assert torch.equal(bits(y), bits(dense(q, sa, w, sw, counts, kind)))
    assert not y[0].any() and (y[1:] != 0).any(1).all()
    del w, sw, y
    torch.cuda.empty_cache()


@gpu
@pytest.mark.parametrize("kind,name", [("bf16", "wide"), ("f16", "128x128")])
def test_outputs_past_32_bit_offsets(kind, name):
    r, n, k = 140000, 15500, 640
    assert r * n > 2 ** 31 and form(r, 2, n, k, kind) == name
    q, sa, w, sw = operands(17, r, 2, n, k)
    y = prism.gemm_fp8_grouped(q, sa, w, sw, offsets_of([r - 500, 500]), out_dtype=TYPES[kind])
    for lo in (0, 138400, r - 900):            # element 2^31 is in row 138547
        hi = lo + 900
        counts = [min(hi, r - 500) - lo, max(0, hi - (r - 500))]
        part = dense(q[lo:hi], sa[:, lo:hi].contiguous(), w, sw, counts, kind)
        assert torch.equal(bits(y[lo:hi]), bits(part)), lo
    del y, q, sa
    torch.cuda.empty_cache()


def test_the_lists_of_this_file_are_of_every_form():
    assert {c[5] for c in DESCENDING} == set(prism.GROUPED_FORMS)
