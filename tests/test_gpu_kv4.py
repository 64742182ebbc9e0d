"""The paged 4-bit cache's writer and reader (quantize_kv4, dequantize_kv4):
codes, scales and offsets bit for bit against the definition."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv4_util import BF16, F16, F32, codes_of, quantise_ref, values_of
from parity_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


def qg():
    import int4_quantized_gemm_b200 as q
    return q


def _kv(T, H, D, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda: (torch.randn(T, H, D, generator=g, device="cuda") * scale).to(dtype)
    return mk() + (2 * torch.randn(H, D, generator=g, device="cuda")).to(dtype), mk()


def _check(cache, slots, x, name):
    """The cache at `slots` holds the definition's codes and params of x."""
    P = cache.page_size
    words, params = getattr(cache, name + "_codes"), getattr(cache, name + "_params")
    got_c = codes_of(words[slots // P, :, slots % P])
    got_p = params[slots // P, :, slots % P].cpu().numpy()
    c, s, o = quantise_ref(x)
    assert np.array_equal(got_p[..., 0], s, equal_nan=True) and np.array_equal(got_p[..., 1], o, equal_nan=True)
    assert np.array_equal(got_c, c)


def _slots(T, pages, P, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randperm(pages * P, generator=g, device="cuda")[:T].contiguous()


@pytest.mark.parametrize("T,H,D,P", [(1, 1, 64, 16), (1, 8, 128, 16), (7, 3, 128, 48), (33, 5, 64, 64), (130, 2, 128, 256),
                                     (1000, 8, 128, 64), (5, 32, 128, 32)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_written_codes_and_params(T, H, D, P, dtype):
    q = qg()
    k, v = _kv(T, H, D, dtype, T + H)
    pages = -(-T // P) + 2
    cache, slots = q.kv4_cache(pages, H, D, P), _slots(T, pages, P, T)
    before = [t.clone() for t in cache]
    assert q.quantize_kv4(k, v, cache, slots) is cache
    _check(cache, slots, k, "k")
    _check(cache, slots, v, "v")
    rest = torch.ones(pages * P, dtype=torch.bool, device="cuda")
    rest[slots] = False
    rest = rest.nonzero()[:, 0]
    for t, b in zip(cache, before):               # nothing else changes
        assert torch.equal(t[rest // P, :, rest % P], b[rest // P, :, rest % P])
    q.check_device_errors()


@pytest.mark.parametrize("T,H,D,P", [(1, 1, 64, 16), (9, 3, 128, 48), (257, 8, 64, 32), (1000, 2, 128, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_values_read_back(T, H, D, P, dtype):
    q = qg()
    k, v = _kv(T, H, D, F16, T)
    pages = -(-T // P) + 1
    cache, slots = q.kv4_cache(pages, H, D, P), _slots(T, pages, P, T + 1)
    q.quantize_kv4(k, v, cache, slots)
    got = q.dequantize_kv4(cache, slots, out_dtype=dtype)
    for name, x in zip("kv", got):
        c, p = getattr(cache, name + "_codes"), getattr(cache, name + "_params")
        p32 = p[slots // P, :, slots % P].float()
        code = torch.from_numpy(codes_of(c[slots // P, :, slots % P])).float().cuda().view(T, H, D // 64, 64)
        # scale * code is exact in binary32, so the sum is one rounding; then one to the type
        want = (code * p32[..., 0, None] + p32[..., 1, None]).view(T, H, D).to(dtype)
        assert x.dtype == dtype and torch.equal(x, want)


def test_a_value_is_off_by_half_a_step_at_most():
    q = qg()
    k, v = _kv(300, 4, 128, F16, 3)
    cache, slots = q.kv4_cache(5, 4, 128, 64), torch.arange(300, device="cuda")
    q.quantize_kv4(k, v, cache, slots)
    for x, name in ((k, "k"), (v, "v")):
        p = getattr(cache, name + "_params")[slots // 64, :, slots % 64].double().cpu().numpy()
        got = values_of(getattr(cache, name + "_codes")[slots // 64, :, slots % 64],
                        getattr(cache, name + "_params")[slots // 64, :, slots % 64])
        step = p[..., 0].repeat(64, -1)
        # half a step; the scale's fp16 rounding (2^-11) moves the largest code's value by up to 15 of its parts
        assert (np.abs(got - x.double().cpu().numpy()) <= step * (0.5 + 15 * 2.0 ** -11)).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_ties_flat_groups_and_extreme_values(dtype):
    """Values on the half-steps, groups of one value, subnormals, the type's largest, infinities and NaN."""
    q = qg()
    i = torch.arange(64, device="cuda")
    g = [0.25 * (i % 31) * 0.5,                             # every half step of scale 0.25
         1.0 + 0.125 * (i % 16), -3.0 - 0.5 * (i % 31) / 2, 0.0 * i, 0.0 * i - 7.25, 1e-6 * i, 2.0 ** -24 * i,
         torch.where(i == 5, 65504.0, -65504.0), torch.where(i == 9, float("inf"), 1.0 * i),
         torch.where(i == 0, float("-inf"), 1.0 * i), torch.where(i == 63, float("nan"), 1.0 * i),
         torch.full((64,), float("nan"), device="cuda"), torch.where(i % 2 == 0, float("inf"), float("-inf")),
         3.0e4 + 16.0 * (i % 7)]
    if dtype == BF16:
        g += [1e30 * (i - 32.0), 3e38 * torch.ones(64, device="cuda"), 1e-38 * i, 100.0 + 0.01 * i]
    x = torch.stack([a.float() for a in g]).to(dtype)        # [n, 64]
    x = torch.cat([x, x.flip(0)], 1).view(len(g), 1, 128)
    cache, slots = q.kv4_cache(2, 1, 128, 32), torch.arange(len(g), device="cuda")
    q.quantize_kv4(x, x, cache, slots)
    _check(cache, slots, x, "k")
    _check(cache, slots, x, "v")


def test_random_ties():
    """fp16 values on a coarse grid: quotients that are exact half-integers are common."""
    q = qg()
    g = torch.Generator(device="cuda").manual_seed(5)
    x = (torch.randint(-31, 32, (2000, 2, 64), generator=g, device="cuda") * 0.125).to(F16)
    x[:, :, 0], x[:, :, 1] = -3.875, 3.625                  # scale 0.5: odd multiples of 0.125 * 2 tie
    cache, slots = q.kv4_cache(32, 2, 64, 64), torch.arange(2000, device="cuda")
    q.quantize_kv4(x, x, cache, slots)
    _check(cache, slots, x, "k")


def test_strided_inputs_of_a_fused_projection():
    q = qg()
    T, Hq, H, D = 19, 8, 2, 128
    qkv = torch.randn(T, (Hq + 2 * H) * D, device="cuda").to(F16)
    k, v = qkv[:, Hq * D:(Hq + H) * D].view(T, H, D), qkv[:, (Hq + H) * D:].view(T, H, D)
    assert not k.is_contiguous()
    cache, slots = q.kv4_cache(3, H, D, 16), torch.arange(5, 5 + T, device="cuda")
    q.quantize_kv4(k, v, cache, slots)
    _check(cache, slots, k, "k")
    _check(cache, slots, v, "v")
    out = torch.zeros(T, (Hq + 2 * H) * D, dtype=F16, device="cuda")
    ko, vo = out[:, Hq * D:(Hq + H) * D].view(T, H, D), out[:, (Hq + H) * D:].view(T, H, D)
    q.dequantize_kv4(cache, slots, out=(ko, vo))
    want = q.dequantize_kv4(cache, slots)
    assert torch.equal(ko, want[0]) and torch.equal(vo, want[1]) and not out[:, :Hq * D].any()
    # head-major storage
    kt = torch.randn(H, T, D, device="cuda").to(BF16).transpose(0, 1)
    q.quantize_kv4(kt, kt, cache, slots)
    _check(cache, slots, kt, "v")


def test_skipped_and_bad_slots():
    """Negative slots are padding; slots behind the cache are skipped and reported."""
    q = qg()
    k, v = _kv(6, 2, 64, F16, 8)
    cache = q.kv4_cache(2, 2, 64, 16)
    slots = torch.tensor([-1, 3, -7, 31, 0, -1], device="cuda")
    q.quantize_kv4(k, v, cache, slots)
    q.check_device_errors()
    keep = slots >= 0
    _check(cache, slots[keep], k[keep], "k")
    ko, vo = q.dequantize_kv4(cache, slots)
    assert not ko[~keep].any() and not vo[~keep].any() and ko[keep].any()
    before = [t.clone() for t in cache]
    bad = torch.full((6,), 32, device="cuda")
    q.quantize_kv4(k, v, cache, bad)
    with pytest.raises(q.QGError) as e:
        q.check_device_errors()
    assert e.value.status == q.QG_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(before, cache))
    ko, _ = q.dequantize_kv4(cache, bad)
    assert not ko.any()
    with pytest.raises(q.QGError):
        q.check_device_errors()
    q.check_device_errors()                                   # the report is cleared


def test_nothing_to_do_and_the_same_slot_twice():
    q = qg()
    cache = q.kv4_cache(1, 2, 64, 16)
    e = torch.empty(0, 2, 64, dtype=F16, device="cuda")
    q.quantize_kv4(e, e, cache, torch.empty(0, dtype=torch.int64, device="cuda"))
    k, v = _kv(2, 2, 64, F16, 9)
    q.quantize_kv4(k, v, cache, torch.tensor([4, 4], device="cuda"))      # either token's words
    assert not cache.k_codes[0, :, :4].any() and not cache.k_codes[0, :, 5:].any()
    q.quantize_kv4(k[:1].repeat(2, 1, 1), v[:1].repeat(2, 1, 1), cache, torch.tensor([4, 4], device="cuda"))
    _check(cache, torch.tensor([4], device="cuda"), k[:1], "k")


def test_offsets_past_32_bits():
    """A pool whose code array is larger than 2^32 bytes: its last page is written and read in place."""
    q = qg()
    H, D, P = 8, 128, 256
    pages = (1 << 32) // (H * P * D // 2) + 3
    cache = q.kv4_cache(pages, H, D, P)
    k, v = _kv(4, H, D, F16, 10)
    slots = torch.tensor([0, 5 * P, (pages - 1) * P + 7, pages * P - 1], device="cuda")
    q.quantize_kv4(k, v, cache, slots)
    _check(cache, slots, k, "k")
    _check(cache, slots, v, "v")
    small = q.kv4_cache(1, H, D, P)
    q.quantize_kv4(k, v, small, torch.arange(4, device="cuda"))
    for a, b in zip(q.dequantize_kv4(cache, slots), q.dequantize_kv4(small, torch.arange(4, device="cuda"))):
        assert torch.equal(a, b)
    q.check_device_errors()


def test_a_plan_in_a_graph():
    q = qg()
    k, v = _kv(16, 8, 128, BF16, 11)
    slots = torch.arange(16, device="cuda")
    want, cache = q.kv4_cache(2, 8, 128, 64), q.kv4_cache(2, 8, 128, 64)
    p = q.plan_quantize_kv4(k, v, cache, slots)
    p.launch()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.launch()
    slots += 64                                                # new slots and values, same buffers
    k.mul_(2)
    q.quantize_kv4(k, v, want, slots)
    for t in cache:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, cache))
