"""What a query does not see does not change what it gives: wide windows with more
queries than keys, and tokens of a draft that hold NaN, infinities or large values."""
from __future__ import annotations

import pytest
import torch

from kv4_sharp import assert_close, dequantised, exact
from kv4_util import BF16, F16, paged, random_cache
from parity_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


def qg():
    import int4_quantized_gemm_b200 as q
    return q


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 40, 1 << 20])
@pytest.mark.parametrize("L,n", [(5, 16), (0, 9), (100, 110), (70, 300), (200, 200)])
@pytest.mark.parametrize("causal", [True, False])
def test_a_window_wider_than_every_sequence_hides_nothing(window, L, n, causal):
    q = qg()
    table, pages = paged([L, 7], 16, 0)
    cache = random_cache(q, pages, 1, 64, 16, 0)
    qs = torch.randn(2 * n, 1, 64, device="cuda").to(F16)
    args = torch.from_numpy(table).cuda(), torch.tensor([L, 7], dtype=torch.int32, device="cuda")
    lse = torch.empty(2, 2 * n, 1, device="cuda")
    want = q.attention_kv4(qs, cache, *args, causal=causal, lse=lse[0])
    got = q.attention_kv4(qs, cache, *args, causal=causal, window=window, lse=lse[1])
    assert torch.equal(want, got) and torch.equal(lse[0], lse[1])


def _draft(D, Hq, n, what, where, window=0, small=2.0 ** -9):
    """(output, exact output and bounds without the odd token) of n draft tokens; where: position of a token whose
    value's params are `what` (a factor, or NaN or an infinity)."""
    q = qg()
    L, P = 300, 16
    table, pages = paged([L], P, 0)
    cache = random_cache(q, pages, 2, D, P, 0)
    cache.v_params.mul_(small)
    g = torch.Generator(device="cuda").manual_seed(n)
    qs = torch.randn(n, Hq, D, generator=g, device="cuda").to(BF16)
    ref, _, bound, _ = exact(qs, dequantised(cache, table, [L]), [n], D ** -0.5, True, window)
    page, row = int(table[0, where // P]), where % P
    cache.v_params[page, :, row] *= what
    if what == what and abs(what) != float("inf"):
        seen, _, seen_bound, _ = exact(qs, dequantised(cache, table, [L]), [n], D ** -0.5, True, window)
    else:
        seen = seen_bound = None
    out = q.attention_kv4(qs, cache, torch.from_numpy(table).cuda(), torch.tensor([L], dtype=torch.int32, device="cuda"),
                          window=window)
    q.check_device_errors()
    return out, ref, bound, seen, seen_bound


@pytest.mark.parametrize("n,Hq", [(2, 4), (3, 4), (4, 4), (2, 8), (3, 8), (4, 8), (9, 8)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_a_draft_token_that_is_not_finite_is_not_seen_before_it(n, Hq, D, what):
    out, ref, bound, _, _ = _draft(D, Hq, n, what, 299)
    assert_close(out[:n - 1], ref[:n - 1], bound[:n - 1])
    assert not torch.isfinite(out[n - 1]).any()


@pytest.mark.parametrize("n,Hq", [(2, 4), (4, 4), (3, 8), (4, 8), (9, 8)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", [2.0 ** 10, 2.0 ** 20])
def test_a_large_draft_token_does_not_cost_the_tokens_before_it_digits(n, Hq, D, what):
    out, ref, bound, seen, seen_bound = _draft(D, Hq, n, what, 299)
    assert_close(out[:n - 1], ref[:n - 1], bound[:n - 1])
    assert_close(out[n - 1:], seen[n - 1:], seen_bound[n - 1:])


@pytest.mark.parametrize("n,Hq", [(2, 4), (4, 8)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", [2.0 ** 20, float("nan")])
@pytest.mark.parametrize("window", [100, 250])
def test_a_large_token_that_the_window_has_passed(n, Hq, D, what, window):
    """The oldest token that the first of the draft sees, and none of the others."""
    out, ref, bound, seen, seen_bound = _draft(D, Hq, n, what, 300 - n - window + 1, window)
    assert_close(out[1:], ref[1:], bound[1:])
    if seen is not None:
        assert_close(out[:1], seen[:1], seen_bound[:1])
    else:
        assert not torch.isfinite(out[0]).any()
