"""fp64 references of the norm, 4-bit cache and attention operators, and the
bounds their kernels are held to."""
from __future__ import annotations

import math

import numpy as np
import torch

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def half_step(dtype) -> float:
    """Largest relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def smallest(dtype) -> float:
    """Half the spacing of the type's subnormal values: the absolute rounding error near zero."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------------------
# 4-bit cache
# ---------------------------------------------------------------------------
def quantise_ref(x: torch.Tensor):
    """x [T, H, D] fp16/bf16 -> (codes int64 [T, H, D], scale, offset fp16 [T, H, D/64]) by
    the definition, every step an IEEE binary32 (or fp16) operation."""
    T, H, D = x.shape
    v = x.detach().float().cpu().numpy().reshape(T, H, D // 64, 64)
    bad = np.isnan(v).any(-1)
    c = np.clip(np.where(np.isnan(v), np.float32(0), v), np.float32(-65504), np.float32(65504))
    lo, hi = c.min(-1), c.max(-1)
    s = np.maximum((hi - lo) / np.float32(15), np.float32(1e-5)).astype(np.float16)
    o = lo.astype(np.float16)
    q = np.rint((c - o.astype(np.float32)[..., None]) / s.astype(np.float32)[..., None])
    q = np.clip(q, 0, 15).astype(np.int64)
    q[bad] = 0
    s[bad] = np.nan
    o[bad] = np.nan
    return q.reshape(T, H, D), s, o


def codes_of(words: torch.Tensor) -> np.ndarray:
    """codes int32 [..., 8, G] -> int64 [..., 64 G]: channel 64 g + 8 j + i is nibble i of word [j, g]."""
    w = words.detach().cpu().numpy().view(np.uint32).astype(np.int64)
    G = w.shape[-1]
    out = np.zeros((*w.shape[:-2], 64 * G), dtype=np.int64)
    for g in range(G):
        for j in range(8):
            for i in range(8):
                out[..., 64 * g + 8 * j + i] = (w[..., j, g] >> (4 * i)) & 15
    return out


def values_of(words: torch.Tensor, params: torch.Tensor) -> np.ndarray:
    """fp64 values scale * code + offset."""
    p = params.detach().cpu().numpy().astype(np.float64)
    lead, G = tuple(words.shape[:-2]), words.shape[-1]
    with np.errstate(invalid="ignore"):
        return (codes_of(words).reshape(*lead, G, 64) * p[..., 0, None] + p[..., 1, None]).reshape(*lead, 64 * G)


def paged(lens, page_size, seed, spare=2):
    """(block table int32 [B, W], pages in the pool): pages of each sequence anywhere in the
    pool; entries behind a sequence's pages hold -1, which must not be read."""
    rng = np.random.default_rng(seed)
    need = [-(-a // page_size) for a in lens]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(need), 1) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def attention_ref(q, cache, table, lens, new, scale, causal=True, window=0):
    """fp64 (out [T, Hq, D], lse [T, Hq], bound [T, Hq, D], lse_bound [T, Hq]) of attention over the cache.

    bound: the arithmetic error that the kernels may make besides the output's rounding.
    With u = 2^-11 (one rounding to fp16), S = scale * sum_d |q_d| (|k_d| + r) (r: the
    group's range 15 * scale, since code and offset round apart), every key rounds to
    fp16 in two steps (offset shift, value: 2 u of its parts), so a score moves by at
    most e = 2 u S plus (D + 8) 2^-23 S for its binary32 sum, its p by a factor
    exp(+-e); p (times a value's scale) and the value round to fp16 once or twice more
    (3 u); the binary32 sums over n keys and their joins add (n + 16) 2^-23.  All of it
    acts on sum_j p_j (|v_j| + r_j), and the normalised sum can move by the same
    relative amount once more.
    lse_bound: every p_j moves by a factor of at most exp(+-e'), e' the exponent above, so
    the logarithm of their sum moves by e' at most, and by the sum's binary32 error
    (n + 16) 2^-23; its own rounding and that of the maximum's scaling add 2^-22 of the
    largest score and of the result."""
    u = 2.0 ** -11
    T, Hq, D = q.shape
    P, H = cache.page_size, cache.num_heads
    qd = q.detach().double().cpu().numpy()
    out, lse, bound = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf), np.zeros((T, Hq, D))
    lse_bound = np.zeros((T, Hq))
    at = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        pages = torch.from_numpy(table[b, : -(-L // P)].astype(np.int64)).to(cache.k_codes.device)
        val, rng = [], []
        for c, p in ((cache.k_codes, cache.k_params), (cache.v_codes, cache.v_params)):
            val.append(values_of(c[pages], p[pages]).transpose(1, 0, 2, 3).reshape(H, len(pages) * P, D)[:, :L])
            r = 15 * np.abs(p[pages].double().cpu().numpy()[..., 0]).repeat(64, -1)
            rng.append(r.transpose(1, 0, 2, 3).reshape(H, len(pages) * P, D)[:, :L])
        pos = np.arange(L - n, L)[:, None]
        key = np.arange(L)
        seen = np.ones((n, L), dtype=bool)
        if causal:
            seen &= key <= pos
        if window:
            seen &= key > pos - window
        for hq in range(Hq):
            h = hq // (Hq // H)
            k, v = val[0][h], val[1][h]
            x = np.where(seen, scale * qd[at:at + n, hq] @ k.T, -np.inf)
            big = scale * np.abs(qd[at:at + n, hq]) @ (np.abs(k) + rng[0][h]).T
            m = x.max(1, initial=-np.inf, keepdims=True)
            w = np.exp(x - np.where(np.isinf(m), 0, m))
            total = w.sum(1, keepdims=True)
            ok = total[:, 0] > 0
            w = w / np.where(total > 0, total, 1)
            out[at:at + n, hq] = w @ v
            lse[at:at + n, hq][ok] = (m + np.log(np.where(total > 0, total, 1)))[ok, 0]
            most = np.where(seen, big, 0).max(1, initial=0)
            e = np.expm1((2 * u + (D + 8) * 2.0 ** -23) * most)[:, None]
            lse_bound[at:at + n, hq] = ((2 * u + (D + 8) * 2.0 ** -23) * most + (L + 16) * 2.0 ** -23
                                        + 2.0 ** -22 * (most + np.log(L + 2.0)))
            bound[at:at + n, hq] = (2 * e + 3 * u + (L + 16) * 2.0 ** -22) * (w @ (np.abs(v) + rng[1][h]))
        at += n
    return out, lse, bound, lse_bound


def assert_attention(got: torch.Tensor, ref: np.ndarray, bound: np.ndarray, what: str = "") -> None:
    g = got.detach().double().cpu().numpy()
    assert np.isfinite(g).all(), f"{what}: not finite"
    allowed = bound + half_step(got.dtype) * (np.abs(ref) + bound) + smallest(got.dtype)
    err = np.abs(g - ref)
    assert (err <= allowed).all(), f"{what}: {(err > allowed).sum()} outputs off, worst {np.max(err / allowed):.3g} of the bound"


def random_cache(qg, pages, H, D, P, seed, dtype=F16, device="cuda", offset=1.0):
    """A cache whose every token holds quantised random keys and values."""
    g = torch.Generator(device=device).manual_seed(seed)
    k = torch.randn(pages * P, H, D, generator=g, device=device) + offset * torch.randn(H, D, generator=g, device=device)
    v = torch.randn(pages * P, H, D, generator=g, device=device) + 0.5
    cache = qg.kv4_cache(pages, H, D, P, device=device)
    slots = torch.arange(pages * P, device=device)
    qg.quantize_kv4(k.to(dtype), v.to(dtype), cache, slots)
    return cache
