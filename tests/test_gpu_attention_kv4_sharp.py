"""Attention over the paged 4-bit cache against fp64 within kv4_sharp's bound (about
0.001 to 0.003 of a head's output), over lengths, head groups, pages, windows, masks,
ragged batches and both kernels, the log-sum-exp included."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv4_sharp import assert_close, assert_lse, dequantised, exact
from kv4_util import BF16, F16, paged, random_cache
from parity_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


def qg():
    import int4_quantized_gemm_b200 as q
    return q


def run(lens, new, Hq, H, D, P, dtype, ragged=False, causal=True, window=0, scale=None):
    q = qg()
    seed = sum(lens) + sum(new) + Hq
    table, pages = paged(lens, P, seed)
    cache = random_cache(q, pages, H, D, P, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    qs = torch.randn(sum(new), Hq, D, generator=g, device="cuda").to(dtype)
    starts = None
    if ragged or len(set(new)) > 1:
        starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    lse = torch.full(qs.shape[:2], float("nan"), device="cuda")
    got = q.attention_kv4(qs, cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                          q_starts=starts, scale=scale, causal=causal, window=window, lse=lse)
    q.check_device_errors()
    out, l, bound, lse_bound = exact(qs, dequantised(cache, table, lens), new, scale or D ** -0.5, causal, window)
    assert_close(got, out, bound)
    assert_lse(lse, l, lse_bound)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 500, 1025])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_single_tokens(L, D, dtype):
    run([L, max(1, L - 1), 1], [1, 1, 1], 8, 2, D, 16, dtype)


@pytest.mark.parametrize("Hq,H", [(1, 1), (5, 1), (14, 2), (16, 1), (24, 2), (40, 1), (32, 32)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 20])
def test_head_groups(Hq, H, D, n):
    run([77, 300], [n, n], Hq, H, D, 32, F16)


@pytest.mark.parametrize("P", [16, 32, 48, 80, 256, 1024])
@pytest.mark.parametrize("n", [1, 40])
def test_page_sizes(P, n):
    run([200, P + 40, P + 41, 40], [n] * 4, 8, 2, 128, P, F16)


@pytest.mark.parametrize("n", [2, 4, 8, 9, 17, 31, 64, 130])
@pytest.mark.parametrize("Hq,H", [(4, 1), (2, 2), (7, 1)])
@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, F16)])
def test_several_tokens(n, Hq, H, D, dtype):
    run([n, n + 1, n + 90, 257 + n], [n] * 4, Hq, H, D, 16, dtype)


@pytest.mark.parametrize("n", [1, 4, 40, 150])
@pytest.mark.parametrize("window", [1, 16, 63, 65, 100, 1000])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_windows_and_masks(n, window, D, causal):
    run([400, n, 150], [n] * 3, 4, 2, D, 32, F16, causal=causal, window=window)


@pytest.mark.parametrize("n", [1, 5, 50, 140])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_without_a_causal_mask(n, dtype):
    run([200, n, 333], [n] * 3, 4, 2, 128, 64, dtype, causal=False)


@pytest.mark.parametrize("lens,new", [
    ([300, 0, 17, 64, 1, 90, 5], [40, 0, 1, 64, 1, 0, 3]), ([300, 20, 700], [1, 1, 1]), ([1000, 130, 256, 640], [300, 130, 1, 2]),
    ([700, 33, 3, 5000, 64], [3, 4, 1, 2, 4]), ([700, 33, 3, 5000, 64], [1, 3, 3, 5, 4])])
@pytest.mark.parametrize("Hq,H", [(8, 2), (20, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_ragged_batches(lens, new, Hq, H, D):
    run(lens, new, Hq, H, D, 16, F16, ragged=True)
    run(lens, new, Hq, H, D, 64, BF16, ragged=True, window=100)


@pytest.mark.parametrize("D", [64, 128])
def test_a_ragged_batch_of_many_row_tiles(D):
    """Enough of them that no tile's keys are split: the kernel that leaves no parts."""
    run([700, 33, 400, 513], [400, 1, 300, 256], 40, 40, D, 64, F16)


def test_more_queries_than_keys():
    for n in (1, 20, 200):
        run([0, n // 2, n], [n] * 3, 4, 2, 128, 16, F16)


@pytest.mark.parametrize("D", [64, 128])
def test_long_sequences(D):
    run([20000, 3, 700, 1, 9000], [1] * 5, 8, 2, D, 64, F16)
    run([12000, 500], [4, 4], 8, 2, D, 128, BF16)
    run([5000, 400], [70, 70], 4, 2, D, 64, F16)
    run([3000], [256], 2, 1, D, 64, F16)
    run([1024], [1024], 2, 1, D, 64, BF16)


@pytest.mark.parametrize("scale", [1e-4, 0.02, 0.3])
@pytest.mark.parametrize("n", [1, 30])
def test_scales(scale, n):
    run([333, 64], [n, n], 8, 2, 64, 16, F16, scale=scale)
