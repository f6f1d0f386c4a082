"""GEMV clusters whose last split of K is nearly empty: its CTA has its partial
sums ready long before the CTA that it hands them to."""

import numpy as np
import pytest

import oracle
import seeded_inputs as si
from gpu_util import assert_within_matmul_tol, device, to_dev, to_host64, torch

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,N", [(257, 96), (1025, 512), (2049, 4096), (4097, 1024), (8193, 256)])
@pytest.mark.parametrize("M", [1, 2])
def test_uneven_splits(M, K, N):
    A, B = si.activations_f32(M, K, seed=K), si.q4_weights(K, N, seed=N)
    a, b = to_dev(A), to_dev(B)
    outs = [torch.empty((M, N), dtype=torch.float32, device=device()) for _ in range(40)]
    for c in outs:      # one after another: the next launch's CTAs start while the last ones finish
        q4.q4_matmul_ex(c, a, b, M, N, K)
    torch.cuda.synchronize()
    C64, S = oracle.matmul(A, B, M, N, K)
    assert_within_matmul_tol(to_host64(outs[0]), C64, S, f"M={M} K={K} N={N}")
    assert all(torch.equal(outs[0], c) for c in outs[1:])
    assert q4.q4_get_device_status() == q4.Q4_OK
