"""What a query does not see does not change what it gives: wide windows with more
queries than keys, and tokens of a draft that hold NaN, infinities or large values."""
from __future__ import annotations

import pytest
import torch

from kv4_util import F16, paged, random_cache
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
