"""Queries of any size in attention over the 4-bit cache: what one row holds does not
reach the others, large and zero rows have their softmax's limit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv4_sharp import U, assert_close, dequantised, exact
from kv4_util import BF16, F16, half_step, paged, random_cache
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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("size", [2.0 ** 80, 2.0 ** 118, 2.0 ** 124])
def test_huge_queries_take_their_best_key(D, n, size):
    """Scores so far apart that all of the weight is on one key, also where they pass binary32."""
    call, kv = setup(D, offset=0.0)
    qs = (queries(n, D, BF16).clamp(-7, 7).float() * size).to(BF16)
    lse = torch.empty(n, 8, device="cuda")
    got = call(qs, lse=lse).double()
    k, v, _, r = kv[0]
    some = 0
    for h in range(8):
        x = qs[:, h].double() @ k[h // 4].T * D ** -0.5
        x = torch.where(torch.arange(L, device="cuda") <= torch.arange(L - n, L, device="cuda")[:, None], x, -torch.inf)
        top = x.topk(2, 1)
        spread = torch.sqrt(qs[:, h].double() ** 2 @ (k[h // 4] ** 2).T).amax(1) * D ** -0.5
        clear = top.values[:, 0] - top.values[:, 1] > 20 * U * spread      # no rounding of a key changes the order
        best = top.indices[:, 0]
        # weight and value round to fp16 once each, the output to its type
        allowed = (2 * U + 2 * half_step(BF16)) * (v[h // 4][best].abs() + r[h // 4][best])
        assert ((got[:, h] - v[h // 4][best]).abs() <= allowed)[clear].all()
        some += int(clear.sum())
    assert some >= 4 * n


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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 40, 2.0 ** 86])
def test_the_log_sum_of_large_queries(D, n, size):
    """Finite and right up to queries of 2^90."""
    call, kv = setup(D)
    qs = (queries(n, D, BF16).clamp(-7, 7).float() * size).to(BF16)
    lse = torch.empty(n, 8, device="cuda")
    out = call(qs, lse=lse)
    assert torch.isfinite(out).all()
    ref = exact(qs, kv, [n], D ** -0.5)[1]
    k = kv[0][0].abs()
    most = torch.stack([(qs[:, h].double().abs() @ k[h // 4].T).amax(1) for h in range(8)], 1) * D ** -0.5
    # every product of the best key's score rounds by u at most, twice; binary32 sums and products
    assert ((lse.double() - ref).abs() <= (2 * U + 2.0 ** -18) * most + 0.01).all()
