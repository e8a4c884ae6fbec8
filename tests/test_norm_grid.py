"""The norms' grid limit: what is refused is a launch of 2^32 threads, not fewer.

A row of K values takes the least whole number of 64s of threads that hold 8 values each up to 512 threads, 16 up to
1024, and 64 beyond.  Without a GPU the calls are made with fake pointers in a child process that sees no device, so that
a valid one ends with the missing device.
"""
import json
import os
import subprocess
import sys

import pytest

from test_moe_cpu import _CHILD, _n, INVALID, LIB, UNSUP


def threads(k):
    for values in (8, 16, 64):
        n = -(-k // (64 * values)) * 64
        if n <= {8: 512, 16: 1024, 64: 1024}[values]:
            return n


WIDTHS = [16, 64, 512, 528, 4096, 4112, 5120, 8192, 16384, 16400, 33040, 65536]
CALLS = [(fn, k, more) for fn in ("prism_add_rmsnorm_quantize_fp8", "prism_add_rmsnorm_quantize_rows")
         for k in WIDTHS for more in (0, 1)]


@pytest.fixture(scope="module")
def statuses():
    if not os.path.exists(LIB):
        from exact_int8_gemm_amd import build
        build.build_library()
    calls = [[fn, _n(M=(2 ** 32 - 1) // threads(k) + more, K=k, ld=k, rld=k, old=k)] for fn, k, more in CALLS]
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", CUDA_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    out = subprocess.run([sys.executable, "-c", _CHILD, LIB, json.dumps(calls)], env=env, capture_output=True, text=True,
                         timeout=120)
    assert out.returncode == 0, out.stderr
    res = json.loads(out.stdout.strip().splitlines()[-1])
    if "device_visible" in res:
        pytest.skip("a HIP device is visible despite HIP_VISIBLE_DEVICES=-1: fake-pointer calls not made")
    return res["status"]


@pytest.mark.parametrize("i", range(len(CALLS)))
def test_rows_up_to_the_grid_limit(statuses, i):
    assert statuses[i] == (INVALID if CALLS[i][2] else UNSUP), CALLS[i]


@pytest.mark.gpu
@pytest.mark.parametrize("to", ["fp8", "int8"])
def test_more_rows_than_threads_of_eight_values_allow(to):
    import numpy as np
    import torch
    from exact_int8_gemm_amd import prism
    from gpu_util import DEV
    from test_norm_quant_gpu import call, expect, inputs
    m, k = 524800, 65536
    assert m * (k // 8) > 2 ** 32
    x = torch.zeros((m, k), dtype=torch.bfloat16, device=DEV)
    some = torch.tensor([0, 1, 524287, 524288, m - 1])
    xs, _, g = inputs(14, 5, k, "bf16", None)
    x[some] = xs.to(DEV)
    got = call(to, x, g.to(DEV))
    want = expect(to, xs, None, g)
    scale = got.scale[:, some] if to == "fp8" else got.scale[some]
    assert np.array_equal(scale.cpu().numpy(), want[1])
    codes = got.q.view(torch.uint8)
    assert np.array_equal(codes[some].view(got.q.dtype).float().cpu().numpy(), want[0])
    live = (got.scale != 0).any(0) if to == "fp8" else got.scale != 0
    assert torch.equal(live.nonzero()[:, 0].cpu(), some)     # every other row was written, as zeros
    for lo in range(0, m, 65600):
        rows = codes[lo:lo + 65600].view(torch.int64)
        assert torch.equal((rows != 0).any(1), live[lo:lo + 65600])
    del x, got, codes
    torch.cuda.empty_cache()
