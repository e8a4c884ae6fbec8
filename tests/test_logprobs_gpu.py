"""token_logprobs on the GPU against a plain 64-bit reference.

Tolerances.  S is a sum of at most a few hundred partial sums in fp32, each
term's exp good to a few 2^-23 where it matters: log S is off by less than
2^-17; the difference z - m, the log and the final subtraction round at
2^-24 of values up to |result|:  |lp - exact| <= 2^-17 + 2^-22 |exact|, the
same for lse.  The entropy's two terms carry that error relative to
themselves: 2^-16 (1 + H).  Token ids are compared exactly.
"""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from exact_int8_gemm_amd import prism
from gpu_util import DEV

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NEG = -np.inf


def close(got, exact, tol, what):
    got = got.cpu().numpy().astype(np.float64)
    fin = np.isfinite(exact)
    assert np.array_equal(np.isnan(got), np.isnan(exact)), what
    assert np.array_equal(got[~fin & ~np.isnan(exact)], exact[~fin & ~np.isnan(exact)]), what
    err = np.abs(got[fin] - exact[fin])
    assert (err <= tol(exact[fin])).all(), (what, float(err.max(initial=0)))


def check(z, tokens, top, r=None):
    """z a tensor on the GPU, tokens numpy int64 [M, T]."""
    r = prism.token_logprobs(z, torch.from_numpy(tokens).to(DEV), top=top) if r is None else r
    lp, lse, ent, ids, tlp = ref.logprobs(z.float().cpu().numpy(), tokens, top)

    def tol(x):
        return 2.0 ** -17 + 2.0 ** -22 * np.abs(x)
    close(r.logprobs, lp, tol, "logprobs")
    close(r.lse, lse, tol, "lse")
    close(r.entropy, ent, lambda h: 2.0 ** -16 * (1 + h), "entropy")
    assert np.array_equal(r.top_ids.cpu().numpy(), ids)
    close(r.top_logprobs, tlp, tol, "top_logprobs")
    return r


def tensor(a, kind):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(TYPES[kind]).to(DEV)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("m,v,t,top", [(1, 1, 1, 3), (3, 2, 2, 2), (2, 7, 0, 0), (5, 64, 1, 20), (2, 1000, 3, 32),
                                       (3, 4095, 1, 5), (2, 4096, 1, 5), (2, 4097, 1, 5), (2, 8191, 2, 5),
                                       (2, 8192, 1, 1), (3, 8193, 8, 20), (1, 50001, 4, 20), (3, 131072, 1, 8),
                                       (2, 200001, 5, 32), (40, 16387, 1, 0)])
def test_against_64_bits(m, v, t, top, kind):
    rng = np.random.default_rng(m * 100 + v + t)
    z = tensor(3 * rng.standard_normal((m, v)), kind)
    check(z, rng.integers(0, v, (m, t)), top)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("v", [100, 5000, 20011])
def test_masked_rows(v, kind):
    rng = np.random.default_rng(v)
    lowest = float(torch.finfo(TYPES[kind]).min)
    z = 2 * rng.standard_normal((10, v))
    z[0] = NEG                                       # nothing left
    z[1, :] = NEG
    z[1, v - 1] = -3.0                               # one token left
    z[2, rng.random(v) < 0.98] = NEG
    z[3, :v - 2] = NEG
    z[4, : v // 2] = NEG
    z[5, :] = lowest                                 # masked by the type's lowest value: uniform
    z[6, rng.random(v) < 0.9] = lowest
    z[7, 1:] = lowest
    z[8, ::2] = NEG
    z[9] = NEG
    z[9, 3] = lowest
    tok = rng.integers(0, v, (10, 3))
    tok[1, 0] = v - 1
    check(tensor(z, kind), tok, 20)


@pytest.mark.parametrize("v", [300, 9000, 30000])
def test_rows_that_are_no_distribution(v):
    rng = np.random.default_rng(v + 1)
    z = rng.standard_normal((8, v))
    z[0, 5] = np.nan
    z[1, v - 1] = np.inf
    z[2] = np.nan
    z[3, :] = NEG
    z[3, 2] = np.inf
    z[4, :] = NEG
    z[4, v - 3] = np.nan
    z[5, 0] = -np.nan
    r = check(tensor(z, "f32"), rng.integers(0, v, (8, 2)), 6)
    assert (r.top_ids[:6] == -1).all() and torch.isnan(r.top_logprobs[:6]).all()


def test_tokens_outside_the_vocabulary():
    z = tensor(np.random.default_rng(2).standard_normal((3, 500)), "f32")
    check(z, np.array([[0, -1, 499], [500, 3, 1 << 40], [-(1 << 62), 2, 2]]), 2)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("v", [40, 3000, 8192, 25000])
def test_ties(v, kind):
    """Equal values everywhere, few distinct values, ascending and descending rows, signed zeros."""
    rng = np.random.default_rng(v + 7)
    z = np.zeros((8, v))
    z[1] = rng.integers(0, 3, v)
    z[2] = np.arange(v) / v * 8
    z[3] = -np.arange(v) / v * 8
    z[4] = np.where(rng.random(v) < 0.5, 0.0, -0.0)
    z[5] = -5
    z[5, rng.permutation(v)[:10]] = 1.5
    z[6] = np.repeat(rng.standard_normal(-(-v // 9)), 9)[:v]
    z[7] = np.sort(rng.standard_normal(v))
    check(tensor(z, kind), rng.integers(0, v, (8, 1)), 32)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("v", [4000, 21000])
def test_large_values_in_few_lanes(v, kind):
    """Large values that fall to a few lanes of a wave only: too many of their pieces, or too many values, for the
    places they are collected in."""
    rng = np.random.default_rng(v + 13)
    i = np.arange(v)
    for vec in (4, 8):
        lane = i // vec % 64
        z = rng.permutation(v)[None, :].repeat(6, 0) / v * 2
        z[0, lane < 20] += 8                          # 20 lanes, all of their values
        z[1, (lane < 10) & (i % vec == 1)] += 8       # 10 lanes, a value per piece
        z[2, lane < 31] += 8
        z[3] = -65504
        z[3, lane < 3] = rng.integers(0, 4, (lane < 3).sum())
        z[4] = np.where(lane < 12, 8 - lane / 8, 0)   # ties within and over the lanes
        z[5] = np.where((lane < 20) & (i % vec == 0), 3, -np.inf)
        check(tensor(z, kind), rng.integers(0, v, (6, 1)), 32)
        check(tensor(z, kind), rng.integers(0, v, (6, 1)), 11)


def test_large_values_and_peaked_rows():
    rng = np.random.default_rng(4)
    v = 20000
    z = rng.standard_normal((7, v))
    z[0] += 1e4
    z[1] -= 1e4
    z[2] *= 1e4
    z[3] = -80
    z[3, 17] = 0
    z[4] = -1000
    z[4, 9000] = 0
    z[5] *= 1e-6
    z[6] = -30 * np.arange(v)
    check(tensor(z, "f32"), rng.integers(0, v, (7, 4)), 10)


@pytest.mark.parametrize("v", [9, 4096, 20000])
def test_values_whose_multiples_overflow(v):
    rng = np.random.default_rng(v + 11)
    z = rng.uniform(2.0, 3.2, (4, v)) * 1e38
    z[1] *= -1
    z[2] = 1e30
    z[3, 1:] = -3e38
    z[3, 0] = -1e30
    check(tensor(z, "f32"), rng.integers(0, v, (4, 3)), 6)


@pytest.mark.parametrize("kind", list(TYPES))
def test_strided_and_unaligned_rows(kind):
    rng = np.random.default_rng(5)
    big = tensor(rng.standard_normal((6, 20101)), kind)
    for lo, v in ((0, 20101), (1, 9001), (3, 20000), (7, 130)):
        check(big[:, lo:lo + v], rng.integers(0, v, (6, 2)), 7)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("v", [777, 8192, 33001])
def test_rows_do_not_depend_on_the_batch(v, kind):
    rng = np.random.default_rng(v + 9)
    z = tensor(3 * rng.standard_normal((300, v)), kind)
    tok = torch.from_numpy(rng.integers(0, v, (300, 2))).to(DEV)
    whole = prism.token_logprobs(z, tok, top=9)
    again = prism.token_logprobs(z, tok, top=9)
    for a, b in zip(whole, again):
        assert torch.equal(a, b)
    for i in (0, 1, 150, 299):
        one = prism.token_logprobs(z[i:i + 1].contiguous(), tok[i:i + 1], top=9)
        for a, b in zip(one, whole):
            assert torch.equal(a[0], b[i])
    # the sums do not depend on `top` or the tokens either
    assert torch.equal(prism.token_logprobs(z).lse, whole.lse)


def test_given_workspace_and_no_writes_outside():
    rng = np.random.default_rng(6)
    z = tensor(rng.standard_normal((5, 70001)), "f32")
    need = prism.token_logprobs_workspace(5, 70001, 8)
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device=DEV)
    tok = rng.integers(0, 70001, (5, 1))
    r = prism.token_logprobs(z, torch.from_numpy(tok).to(DEV), top=8, workspace=ws[:need])
    check(z, tok, 8, r)
    assert (ws[need:] == 77).all()
    assert prism.token_logprobs_workspace(5, 100, 8) == 0


def test_logits_past_32_bit_offsets():
    m, v = 66, (1 << 25) + 3
    z = torch.zeros((m, v), dtype=torch.float16, device=DEV)
    z[m - 1, v - 1] = 5
    z[m - 1, 7] = 4
    tok = torch.full((m, 1), v - 1, dtype=torch.int64, device=DEV)
    r = prism.token_logprobs(z, tok, top=3)
    lse = np.log(v - 2 + np.exp(5.0) + np.exp(4.0))
    assert abs(float(r.lse[m - 1]) - lse) < 1e-4 and abs(float(r.logprobs[m - 1, 0]) - (5 - lse)) < 1e-4
    assert r.top_ids[m - 1].tolist() == [v - 1, 7, 0] and r.top_ids[0].tolist() == [0, 1, 2]
    assert abs(float(r.lse[0]) - np.log(v)) < 1e-4 and abs(float(r.entropy[0]) - np.log(v)) < 1e-3
    del z
    torch.cuda.empty_cache()


@pytest.mark.parametrize("mask", [-1e5, -2.0 ** 20, -1e9, -2e9, -1e10, -1e12, -1e20, -9e29, -1e30, -1e38])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("v,top", [(3000, 7), (20011, 0), (20011, 6), (100003, 20), (300000, 3)])
def test_finite_masks_of_any_size(v, top, kind, mask):
    """Logits masked by a finite value: a few tokens left, spread out, in the first or in the last values only (whole
    chunks of 4096 and a cut last one have nothing but the mask), and none."""
    rng = np.random.default_rng(v + top)
    z = 2 * rng.standard_normal((5, v))
    z[0, rng.random(v) < 0.99] = mask
    z[1, 100:] = mask
    z[2, :v - 50] = mask
    z[3] = mask
    z[4, v // 2] = mask
    check(tensor(z, kind), rng.integers(0, v, (5, 3)), top)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("v", [50, 4096, 9000])
def test_rows_of_any_magnitude(v, kind):
    """Uniform rows, rows a few logits wide where the type holds them, and rows spread over their magnitude, of both
    signs and every power of ten, and at 2^20 and its neighbours."""
    rng = np.random.default_rng(v + 17)
    near = [2.0 ** 20, np.nextafter(np.float32(2.0 ** 20), np.float32(0)), 2.0 ** 20 + 0.125, 2.0 ** 20 * 1.0078125]
    sizes = [10.0 ** k for k in range(3, 39)] + [float(x) for x in near] + [1.5e9, 1.7e9, 3e9, 7e9, 0.99e30]
    rows = []
    for b in sizes:
        for sign in (1, -1):
            rows.append(np.full(v, sign * b))
            rows.append(sign * b - 12 * rng.random(v))
            rows.append(sign * b * rng.uniform(0.4, 1, v))
    z = np.stack(rows)
    check(tensor(z, kind), rng.integers(0, v, (len(z), 2)), 5)
