"""The norm, row reader, cache writer and reader at sizes where they take another block
shape or more work a thread (thresholds: four blocks, 512 loads of 8 codes or 1024 threads
an SM), with ends that are no multiple of it: bit for bit against the definitions."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv4_util import BF16, F16, F32, codes_of, quantise_ref
from parity_util import requires_cuda
from test_gpu_norm_int8 import reference, rows

pytestmark = [pytest.mark.gpu, requires_cuda]


def qg():
    import int4_quantized_gemm_b200 as q
    return q


@pytest.mark.parametrize("M,K", [(701, 1000), (593, 513), (601, 4096), (593, 2049), (151, 10007), (149, 16384), (149, 8193),
                                 (597, 500), (592, 1024), (592, 4096), (148, 9000)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_many_rows(M, K, dtype, residual):
    x, w = rows(M, K, dtype, 1), rows(1, K, dtype, 2)[0].contiguous()
    res = rows(M, K, dtype, 3, 4.0, pad=16) if residual else None
    x[M // 2] = 0
    q, s, h = qg().rmsnorm_quantize_int8(x, w, res, eps=1e-5)
    rq, rs, rh = reference(x, w, res, 1e-5)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert (np.abs(s.double().cpu().numpy() - rs) <= (K * 2.0 ** -25 + 6 * 2.0 ** -24) * rs).all()
    assert (h is None) if res is None else torch.equal(h, rh)


@pytest.mark.parametrize("M,K", [(41, 20000), (31, 20007), (150, 4101), (701, 1000), (80001, 13), (2001, 2047), (19001, 33)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_many_int8_rows_read_back(M, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(M)
    q = torch.zeros(M, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :K]
    q.copy_(torch.randint(-128, 128, (M, K), generator=g, device="cuda"))
    s = torch.rand(M, generator=g, device="cuda") + 1e-3
    out = torch.full((M + 1, (K + 15) // 16 * 16), 7.0, dtype=dtype, device="cuda")
    qg().dequantize_rowwise_int8(q, s, out_dtype=dtype, out=out[:M, :K])
    assert torch.equal(out[:M, :K], (q.float() * s[:, None]).to(dtype))
    assert (out[M] == 7).all() and (out[:, K:] == 7).all()


@pytest.mark.parametrize("T,H,D,P", [(4743, 16, 64, 16), (4741, 16, 64, 48), (4739, 8, 128, 64), (4738, 8, 64, 32)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_many_tokens_written_and_read(T, H, D, P, dtype):
    q = qg()
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn(T, H, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    pages = -(-T // P) + 1
    cache = q.kv4_cache(pages, H, D, P)
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:T].contiguous()
    slots[5], slots[T - 1] = -1, -3
    q.quantize_kv4(k, v, cache, slots)
    q.check_device_errors()
    keep = slots >= 0
    at, used = slots[keep], torch.zeros(pages * P, dtype=torch.bool, device="cuda")
    used[at] = True
    rest = (~used).nonzero()[:, 0]
    want = {}
    for name, x in (("k", k), ("v", v)):
        words, params = getattr(cache, name + "_codes"), getattr(cache, name + "_params")
        c, s, o = quantise_ref(x[keep])
        assert np.array_equal(codes_of(words[at // P, :, at % P]), c)
        p = params[at // P, :, at % P].cpu().numpy()
        assert np.array_equal(p[..., 0], s) and np.array_equal(p[..., 1], o)
        assert not words[rest // P, :, rest % P].any() and not params[rest // P, :, rest % P].any()
        sf, of = (torch.from_numpy(a).float()[..., None] for a in (s, o))
        want[name] = (torch.from_numpy(c).float().view(*sf.shape[:3], 64) * sf + of).view(-1, H, D).cuda()
    for out_dtype in (F32, F16, BF16):
        buf = torch.full((2, T + 4, H, D), 7.0, dtype=out_dtype, device="cuda")
        q.dequantize_kv4(cache, slots, out_dtype=out_dtype, out=(buf[0, :T], buf[1, :T]))
        for x, name in zip(buf, "kv"):
            assert torch.equal(x[:T][keep], want[name].to(out_dtype))
            assert not x[:T][~keep].any() and (x[T:] == 7).all()
