"""RMS norm with residual addition and int8 codes (rmsnorm_quantize_int8), and
the int8 row reader (dequantize_rowwise_int8), against their definitions.

Codes are bit-exact: products of two 16-bit values are exact in binary32 and
every later step is one IEEE operation.  The scale takes a binary32 sum of K
squares in any order (relative error at most K 2^-24 of a positive sum, halved
by the square root) and six more roundings.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv4_util import BF16, F16, F32, half_step
from parity_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


def qg():
    import int4_quantized_gemm_b200 as q
    return q


def rows(M, K, dtype, seed, scale=1.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = (K + 15) // 16 * 16 + pad
    t = torch.full((M, ld), float("nan") if dtype.is_floating_point else 0, dtype=dtype, device="cuda")[:, :K]
    if dtype.is_floating_point:
        t.copy_(torch.randn(M, K, generator=g, device="cuda") * scale)
    return t


def reference(x, w, res, eps):
    """(codes, scale fp64, h) by the definition."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    hf = h.float().cpu().numpy()
    p = hf * w.float().cpu().numpy()
    a = np.maximum(np.abs(p).max(1), np.float32(1e-30))
    q = np.clip(np.rint(p * (np.float32(127) / a)[:, None]), -127, 127).astype(np.int8)
    r = 1 / np.sqrt((hf.astype(np.float64) ** 2).mean(1) + eps)
    return q, a.astype(np.float64) / 127 * r, h


SHAPES = [(1, 1), (1, 7), (3, 8), (2, 33), (5, 1000), (9, 1024), (4, 1025), (7, 4096), (3, 4100), (2, 11008),
          (2, 16384), (2, 16385), (3, 20007), (300, 64), (1000, 129)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("residual", [False, True])
def test_codes_scale_and_residual(M, K, dtype, residual):
    x, w = rows(M, K, dtype, 1), rows(1, K, dtype, 2)[0].contiguous()
    res = rows(M, K, dtype, 3, 4.0, pad=16) if residual else None
    q, s, h = qg().rmsnorm_quantize_int8(x, w, res, eps=1e-5)
    rq, rs, rh = reference(x, w, res, 1e-5)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert (np.abs(s.double().cpu().numpy() - rs) <= (K * 2.0 ** -25 + 6 * 2.0 ** -24) * rs).all()
    assert (h is None) == (res is None)
    if residual:
        assert torch.equal(h, rh)
    assert q.dtype == torch.int8 and q.shape == (M, K)


@pytest.mark.parametrize("K", [100, 4096, 20000])
def test_residual_in_place(K):
    """residual_out may be the residual or x."""
    for where in ("residual", "x"):
        x, res, w = rows(6, K, F16, 4), rows(6, K, F16, 5), rows(1, K, F16, 6)[0].contiguous()
        rq, rs, rh = reference(x, w, res, 1e-5)
        dst = res if where == "residual" else x
        q, _, h = qg().rmsnorm_quantize_int8(x, w, res, residual_out=dst)
        assert h is dst and torch.equal(dst, rh) and np.array_equal(q.cpu().numpy(), rq)


def test_zero_tiny_and_huge_rows():
    K = 512
    x = torch.zeros(6, K, dtype=F16, device="cuda")
    x[1] = 2.0 ** -24                      # smallest subnormal everywhere
    x[2, 3] = 65504.0
    x[3] = 1000.0
    x[4, ::2] = -2.0 ** -14
    w = torch.ones(K, dtype=F16, device="cuda")
    q, s, _ = qg().rmsnorm_quantize_int8(x, w, eps=1e-5)
    rq, rs, _ = reference(x, w, None, 1e-5)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert (np.abs(s.double().cpu().numpy() - rs) <= (K * 2.0 ** -25 + 6 * 2.0 ** -24) * rs).all()
    assert not q[0].any() and not q[5].any() and torch.isfinite(s).all()


@pytest.mark.parametrize("dtype,value", [(F16, float("nan")), (F16, float("inf")), (BF16, float("-inf")),
                                         (BF16, 3e38), (BF16, 1e25)])
def test_rows_that_are_not_finite(dtype, value):
    """A NaN, an infinity, or a product or square sum beyond binary32: scale NaN, codes 0, that row only."""
    for at in (0, 129, 130):
        x = rows(3, 131, dtype, 7)
        x[1, at] = value
        w = torch.full((131,), 2.0, dtype=dtype, device="cuda")
        q, s, _ = qg().rmsnorm_quantize_int8(x, w)
        assert torch.isnan(s[1]) and not q[1].any()
        assert torch.isfinite(s[[0, 2]]).all() and q[0].any() and q[2].any()
    s = rows(2, 64, F16, 8)
    s[0, 1] = 60000.0                                # the sum leaves fp16
    q, sc, h = qg().rmsnorm_quantize_int8(s, torch.ones(64, dtype=F16, device="cuda"), s.clone())
    assert torch.isinf(h[0, 1]) and torch.isnan(sc[0]) and torch.isfinite(sc[1])


def test_padding_columns_and_other_rows_are_left_alone():
    K = 100
    x, w = rows(4, K, BF16, 9), rows(1, K, BF16, 10)[0].contiguous()
    buf = torch.full((6, 128), 77, dtype=torch.int8, device="cuda")
    qg().rmsnorm_quantize_int8(x, w, out=buf[1:5, :K])
    assert (buf[0] == 77).all() and (buf[5] == 77).all() and (buf[1:5, K:] == 77).all()


@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 8), (17, 1000), (64, 4096), (2, 70001), (10000, 40)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_dequantize_rowwise(M, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    q = torch.zeros(M, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :K]
    q.copy_(torch.randint(-128, 128, (M, K), generator=g, device="cuda"))
    s = torch.rand(M, generator=g, device="cuda") + 1e-3
    y = qg().dequantize_rowwise_int8(q, s, out_dtype=dtype)
    ref = (q.float() * s[:, None]).to(dtype)                # binary32 product, rounded once
    assert y.dtype == dtype and torch.equal(y, ref)


def test_codes_times_scale_is_the_norm():
    """The two together: the normed row to half a code's step."""
    x, w, res = rows(33, 4096, BF16, 11), rows(1, 4096, BF16, 12)[0].contiguous(), rows(33, 4096, BF16, 13)
    q, s, h = qg().rmsnorm_quantize_int8(x, w, res, eps=1e-6)
    y = qg().dequantize_rowwise_int8(q, s, out_dtype=F32).double()
    hd = h.double()
    ref = hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + 1e-6) * w.double()
    step = ref.abs().amax(1, keepdim=True) / 127
    # half a step, 127 roundings of the inverse and product (2^-23 each), the scale's error
    assert ((y - ref).abs() <= step * (0.5 + 127 * 2.0 ** -22) + ref.abs() * 4096 * 2.0 ** -25).all()


def test_a_plan_in_a_graph_equals_the_call():
    q = qg()
    x, w, res = rows(16, 4096, F16, 14), rows(1, 4096, F16, 15)[0].contiguous(), rows(16, 4096, F16, 16)
    want = q.rmsnorm_quantize_int8(x, w, res)
    p = q.plan_rmsnorm_quantize_int8(x, w, res)
    p.launch()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.launch()
    for t in p.out:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, p.out):
        assert torch.equal(a, b)


def test_on_another_stream():
    q = qg()
    x, w = rows(64, 4096, F16, 17), rows(1, 4096, F16, 18)[0].contiguous()
    want = q.rmsnorm_quantize_int8(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = q.rmsnorm_quantize_int8(x, w)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_the_operand_of_the_w8a8_product():
    """rmsnorm_quantize_int8 -> gemm_w8a8 against the fp64 product of the codes' values."""
    q = qg()
    x, w, res = rows(40, 512, F16, 19), rows(1, 512, F16, 20)[0].contiguous(), rows(40, 512, F16, 21)
    wt = rows(96, 512, F16, 22, 0.05)
    wq, ws = q.quantize_rowwise_int8(wt)
    xq, xs, _ = q.rmsnorm_quantize_int8(x, w, res)
    y = q.gemm_w8a8(xq, wq, xs, ws, out_dtype=F32).double()
    ref = (xq.double() * xs.double()[:, None]) @ (wq.double() * ws.double()[:, None]).T
    # exact integer sum, then two binary32 products
    assert ((y - ref).abs() <= 4 * half_step(F32) * ref.abs() + 1e-30).all()
    q.check_device_errors()
