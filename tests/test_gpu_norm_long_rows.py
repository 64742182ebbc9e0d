"""Rows next to the longest that the norm and the row reader take, 2^31 - 1 elements."""
from __future__ import annotations

import pytest
import torch

from kv4_util import F16
from parity_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


def test_rows_next_to_2_to_the_31():
    import int4_quantized_gemm_b200 as q
    n, step = 1 << 31, 1 << 26
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(n, dtype=F16, device="cuda")
    for a in range(0, n, step):                       # small integers: every thread's sum of squares is exact
        x[a:a + step] = torch.randint(-2, 3, (step,), generator=g, device="cuda", dtype=torch.int8)
    w = torch.ones(n, dtype=F16, device="cuda")
    w[n - 9:] = 2
    x[n - 9:] = 2                                     # the row's largest product, 4, is at its end
    codes = torch.empty(n, dtype=torch.int8, device="cuda")
    y = torch.empty(n, dtype=F16, device="cuda")
    for K in (n - 1, n - 8):
        codes.fill_(77)
        y.fill_(7)
        _, s, _ = q.rmsnorm_quantize_int8(x[None, :K], w[:K], eps=1e-5, out=codes[None, :K])
        q.dequantize_rowwise_int8(codes[None, :K], s, out=y[None, :K])
        total = 0.0
        for a in range(0, K, step):
            b = min(K, a + step)
            total += float(x[a:b].double().square().sum())
            ref = torch.round(x[a:b].float() * w[a:b].float() * torch.tensor(127.0 / 4.0, device="cuda")).to(torch.int8)
            assert torch.equal(codes[a:b], ref)
            assert torch.equal(y[a:b], (ref.float() * s).half())
        assert (codes[K:] == 77).all() and (y[K:] == 7).all()
        want = 4.0 / 127.0 / (total / K + 1e-5) ** 0.5
        assert abs(float(s[0]) - want) <= 40 * 2.0 ** -24 * want      # the threads' sums joined: 5 + 16 roundings, halved; six more
