"""The calls of a decoder layer's attention half as they are used together: norm
with residual and int8 codes -> W8A8 projection -> new keys and values into the
4-bit cache -> attention over it -> rowwise int8 -> W8A8 projection -> the next
norm with the residual.

Each stage is held to its definition (fp64) on the values that it was given, so
every bound is that stage's own: codes are exact; a W8A8 output of n-bit type is
an exact integer times two binary32 scales (two roundings of 2^-24) and one
rounding to the type; attention has kv4_util's bound."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv4_util import (BF16, F16, assert_attention, attention_ref, codes_of, half_step, paged, quantise_ref, smallest)
from parity_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


def qg():
    import int4_quantized_gemm_b200 as q
    return q


class Layer:
    """Random weights and a cache for `lens` tokens a sequence."""

    def __init__(self, Hq, H, D, E, P, lens, dtype, seed):
        q = qg()
        self.Hq, self.H, self.D, self.dtype = Hq, H, D, dtype
        g = torch.Generator(device="cuda").manual_seed(seed)
        def weight(n, k):
            return q.quantize_rowwise_int8((torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).half())
        self.norm1, self.norm2 = (1 + 0.1 * torch.randn(2, E, generator=g, device="cuda")).to(dtype).unbind(0)
        self.wqkv, self.sqkv = weight((Hq + 2 * H) * D, E)
        self.wo, self.so = weight(E, Hq * D)
        self.table, pages = paged(lens, P, seed)
        self.block_table = torch.from_numpy(self.table).cuda()
        self.cache = q.kv4_cache(pages, H, D, P)

    def __call__(self, x, res, slots, lens, starts=None, window=0):
        """Every intermediate value, in order."""
        q, T, s = qg(), x.shape[0], {}
        s["xq"], s["xs"], s["h"] = q.rmsnorm_quantize_int8(x, self.norm1, res)
        s["qkv"] = q.gemm_w8a8(s["xq"], self.wqkv, s["xs"], self.sqkv, out_dtype=self.dtype)
        s["q"], s["k"], s["v"] = s["qkv"].view(T, -1, self.D).split([self.Hq, self.H, self.H], 1)
        q.quantize_kv4(s["k"], s["v"], self.cache, slots)
        s["attn"] = q.attention_kv4(s["q"], self.cache, self.block_table, lens, q_starts=starts, window=window)
        s["aq"], s["as"] = q.quantize_rowwise_int8(s["attn"].reshape(T, -1).half())
        s["o"] = q.gemm_w8a8(s["aq"], self.wo, s["as"], self.so, out_dtype=self.dtype)
        s["yq"], s["ys"], s["y"] = q.rmsnorm_quantize_int8(s["o"], self.norm2, s["h"])
        return s

    def slots(self, at):
        """Slots of (sequence, position) pairs."""
        P = self.cache.page_size
        return torch.tensor([int(self.table[b, t // P]) * P + t % P for b, t in at], dtype=torch.int64, device="cuda")


def check_norm(x, w, res, xq, xs, h):
    assert torch.equal(h, (x.float() + res.float()).to(x.dtype))
    hf, K = h.float().cpu().numpy(), x.shape[1]
    p = hf * w.float().cpu().numpy()
    a = np.abs(p).max(1)
    assert np.array_equal(xq.cpu().numpy(), np.clip(np.rint(p * (np.float32(127) / a)[:, None]), -127, 127))
    s = a.astype(np.float64) / 127 / np.sqrt((hf.astype(np.float64) ** 2).mean(1) + 1e-5)
    # a sum of K squares (K 2^-24, halved by the root) and six roundings
    assert (np.abs(xs.double().cpu().numpy() - s) <= (K * 2.0 ** -25 + 6 * 2.0 ** -24) * s).all()


def check_gemm(y, xq, xs, wq, ws):
    ref = (xq.double() @ wq.double().T) * xs.double()[:, None] * ws.double()[None, :]   # integers below 2^53: exact
    off = 3 * 2.0 ** -24 * ref.abs()
    assert ((y.double() - ref).abs() <= off + half_step(y.dtype) * (ref.abs() + off) + smallest(y.dtype)).all()


def check(layer, s, x, res, slots, lens, new, window=0):
    check_norm(x, layer.norm1, res, s["xq"], s["xs"], s["h"])
    check_gemm(s["qkv"], s["xq"], s["xs"], layer.wqkv, layer.sqkv)
    P = layer.cache.page_size
    page, row = slots // P, slots % P
    for t, codes, params in ((s["k"], layer.cache.k_codes, layer.cache.k_params),
                             (s["v"], layer.cache.v_codes, layer.cache.v_params)):
        c, sc, o = quantise_ref(t)
        assert np.array_equal(codes_of(codes[page, :, row]), c)
        got = params[page, :, row].cpu().numpy()
        assert np.array_equal(got[..., 0], sc) and np.array_equal(got[..., 1], o)
    ref, _, bound, _ = attention_ref(s["q"], layer.cache, layer.table, lens, new, layer.D ** -0.5, True, window)
    assert_attention(s["attn"], ref, bound)
    check_gemm(s["o"], s["aq"], s["as"], layer.wo, layer.so)
    check_norm(s["o"], layer.norm2, s["h"], s["yq"], s["ys"], s["y"])


@pytest.mark.parametrize("Hq,H,D,E,P", [(8, 2, 128, 1024, 64), (14, 2, 64, 896, 16), (4, 4, 64, 256, 32)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompts_then_single_tokens(Hq, H, D, E, P, dtype):
    """A ragged batch of prompts, then tokens one by one, eagerly and from a graph that
    is captured once and replayed while slots and lengths change in place."""
    q = qg()
    prompts, steps = [70, 1, 200], 4
    layer = Layer(Hq, H, D, E, P, [n + steps for n in prompts], dtype, 3)
    T = sum(prompts)
    x, res = (torch.randn(T, E, device="cuda").to(dtype) for _ in range(2))
    slots = layer.slots([(b, t) for b, n in enumerate(prompts) for t in range(n)])
    starts = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]), dtype=torch.int32, device="cuda")
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    check(layer, layer(x, res, slots, lens, starts), x, res, slots, prompts, prompts)

    B = len(prompts)
    xs, rs = ([torch.randn(B, E, device="cuda").to(dtype) for _ in range(steps)] for _ in range(2))
    x, res = xs[0].clone(), rs[0].clone()
    slots = layer.slots([(b, n) for b, n in enumerate(prompts)])
    lens += 1
    layer(x, res, slots, lens)                           # warm-up of the capture: writes what step 0 writes again
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = layer(x, res, slots, lens)
    for i in range(steps):
        now = [n + i + 1 for n in prompts]
        x.copy_(xs[i])
        res.copy_(rs[i])
        slots.copy_(layer.slots([(b, n - 1) for b, n in enumerate(now)]))
        lens.copy_(torch.tensor(now))
        graph.replay()
        check(layer, s, x, res, slots, now, [1] * B)
        eager = layer(x, res, slots, lens)
        assert all(torch.equal(s[name], eager[name]) for name in s)
    q.check_device_errors()


def test_a_padded_batch_and_plans():
    """Unused entries of a fixed batch: slot -1, length 0; plans give what the calls give."""
    q = qg()
    B, Hq, H, D, E, P, dtype = 5, 8, 2, 128, 512, 16, F16
    lens = [33, 0, 90, 0, 17]
    layer = Layer(Hq, H, D, E, P, lens, dtype, 5)
    old = layer.slots([(b, t) for b, n in enumerate(lens) for t in range(n - 1)])
    kv = torch.randn(2, old.numel(), H, D, device="cuda").to(dtype)
    q.quantize_kv4(kv[0], kv[1], layer.cache, old)
    x, res = (torch.randn(B, E, device="cuda").to(dtype) for _ in range(2))
    slots = torch.full((B,), -1, dtype=torch.int64, device="cuda")
    live = [b for b, n in enumerate(lens) if n]
    slots[live] = layer.slots([(b, lens[b] - 1) for b in live])
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s = layer(x, res, slots, n, window=40)
    assert not s["attn"][[1, 3]].any()
    ref, _, bound, _ = attention_ref(s["q"], layer.cache, layer.table, lens, [1] * B, D ** -0.5, True, 40)
    assert_attention(s["attn"], ref, bound)

    p1 = q.plan_rmsnorm_quantize_int8(x, layer.norm1, res)
    xq, xsc, h = p1.out
    p2 = q.plan_gemm_w8a8(xq, layer.wqkv, xsc, layer.sqkv, out_dtype=dtype)
    qh, k, v = p2.out.view(B, -1, D).split([Hq, H, H], 1)
    p3 = q.plan_quantize_kv4(k, v, layer.cache, slots)
    p4 = q.plan_attention_kv4(qh, layer.cache, layer.block_table, n, window=40)
    before = [t.clone() for t in layer.cache]
    for p in (p1, p2, p3, p4):
        p.launch()
    assert torch.equal(p4.out, s["attn"]) and torch.equal(h, s["h"])
    assert all(torch.equal(a, b) for a, b in zip(before, layer.cache))
    q.check_device_errors()
