"""Queries of any size in attention over the 4-bit cache: what one row holds does not
reach the others, and rows without a score to speak of weigh every key alike."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv4_sharp import assert_close, dequantised, exact
from kv4_util import BF16, F16, paged, random_cache
from parity_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]
L, P = 300, 16


def qg():
    import int4_quantized_gemm_b200 as q
    return q


def setup(D, seed=0, offset=1.0):
    q = qg()
    table, pages = paged([L], P, seed)
    cache = random_cache(q, pages, 2, D, P, seed, offset=offset)
    call = lambda qs, **kw: q.attention_kv4(qs, cache, torch.from_numpy(table).cuda(),
                                            torch.tensor([L], dtype=torch.int32, device="cuda"), **kw)
    return call, dequantised(cache, table, [L])


def queries(n, D, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, 8, D, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype,bad", [(F16, float("nan")), (F16, float("inf")), (F16, 6e4), (BF16, float("nan")),
                                       (BF16, float("-inf")), (BF16, 2.0 ** 40), (BF16, 2.0 ** 110)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 40, 150])
def test_one_row_does_not_reach_the_others(dtype, bad, D, n):
    """A NaN, an infinity or a huge value in one head's query of one token."""
    call, kv = setup(D)
    qs = queries(n, D, dtype)
    ref, _, bound, _ = exact(qs, kv, [n], D ** -0.5)
    at = [(n // 2, 3), (n - 1, 6)]
    rest = torch.ones(n, 8, dtype=torch.bool, device="cuda")
    for t, h in at:
        qs[t, h, 5] = bad
        rest[t, h] = False
    got = call(qs)
    assert_close(got[rest], ref[rest], bound[rest])
    if bad != bad:
        assert torch.isnan(got[~rest]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 40])
def test_rows_of_very_different_sizes(D, n):
    """Rows near one between rows of 2^20 to 2^100."""
    call, kv = setup(D)
    qs = queries(n, D, BF16)
    rng = np.random.default_rng(0)
    sizes = torch.from_numpy(np.where(rng.random((n, 8)) < 0.5, 1.0, 2.0 ** rng.integers(20, 101, (n, 8)))).cuda()
    ref, _, bound, _ = exact(qs, kv, [n], D ** -0.5)
    got = call((qs.double() * sizes[..., None]).to(BF16))
    one = sizes == 1.0
    assert one.any() and not one.all()
    assert_close(got[one], ref[one], bound[one])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("scale", [1e-20, 1e-30, 1e-37])
def test_zero_and_small_queries_with_a_small_scale(dtype, n, scale):
    """Every visible key has the same weight."""
    call, kv = setup(64)
    qs = queries(n, 64, dtype)
    qs[:, ::2] = 0
    qs[:, 1] *= 2.0 ** -10
    ref, _, bound, _ = exact(qs, kv, [n], scale)
    assert_close(call(qs, scale=scale), ref, bound)
