"""The norm with an 8-bit output on batches whose residual is written past the caches (128 MiB and more of it): every output
against the same call on parts below that size, and some rows against the definition.  All exactly, as in
test_norm_quant_gpu.py.
"""
import pytest
import torch

from exact_int8_gemm_amd import prism
from gpu_util import DEV
from test_norm_quant_gpu import TYPES, call, check, expect

pytestmark = pytest.mark.gpu

# one, two and eight chunks a thread
SHAPES = [(32300, 1040), (6601, 5120), (4100, 8192), (2003, 17408)]


@pytest.mark.parametrize("to", ["fp8", "int8"])
@pytest.mark.parametrize("kind,res", [("bf16", "f32"), ("f16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("m,k", SHAPES)
def test_residuals_larger_than_the_limit(m, k, kind, res, to):
    m *= 4 // torch.empty(0, dtype=TYPES[res]).element_size()
    g = torch.Generator(device=DEV).manual_seed(m + k)
    x = torch.randn((m, k), generator=g, device=DEV).to(TYPES[kind])
    r = (torch.randn((m, k), generator=g, device=DEV) * 3).to(TYPES[res])
    gain = 1 + 0.2 * torch.randn((k,), generator=g, device=DEV)
    assert r.numel() * r.element_size() >= 2 ** 27
    whole = call(to, x, gain, residual=r, norm=True)
    parts = 3
    for i in range(parts):
        lo, hi = m * i // parts, m * (i + 1) // parts
        part = call(to, x[lo:hi], gain, residual=r[lo:hi], norm=True)
        assert part.residual.numel() * part.residual.element_size() < 2 ** 27
        assert torch.equal(whole.q[lo:hi].view(torch.uint8), part.q.view(torch.uint8))
        assert torch.equal(whole.scale[:, lo:hi] if to == "fp8" else whole.scale[lo:hi], part.scale)
        assert torch.equal(whole.residual[lo:hi], part.residual) and torch.equal(whole.norm[lo:hi], part.norm)
    some = torch.tensor([0, 1, m // 2, m - 1], device=DEV)
    want = expect(to, x[some].cpu(), r[some].cpu(), gain.cpu())
    got = prism.NormQuantized(whole.q.view(torch.uint8)[some].view(whole.q.dtype),
                              whole.scale[:, some] if to == "fp8" else whole.scale[some], whole.residual[some],
                              whole.norm[some])
    check(to, got, want, kind, True)
    # the residual in its own place, with rows apart
    wide = torch.full((m, k + 64), 9.0, dtype=TYPES[res], device=DEV)
    place = wide[:, 32:32 + k]
    place.copy_(r)
    again = call(to, x, gain, residual=place, residual_out=place)
    assert torch.equal(place, whole.residual) and (wide[:, :32] == 9).all() and (wide[:, 32 + k:] == 9).all()
    assert torch.equal(again.q.view(torch.uint8), whole.q.view(torch.uint8)) and torch.equal(again.scale, whole.scale)
