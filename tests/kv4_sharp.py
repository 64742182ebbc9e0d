"""Attention over the 4-bit cache in fp64 and how far a right kernel may be from
it: one bound per query token and head, on the Euclidean norm of the difference
over the head's channels.

The kernels' roundings are independent of one another, so their squares add
instead of their magnitudes.  With u = 2^-11, the half step of fp16, a rounding
is an error of at most u and of u / sqrt(3) root mean square, relative to what
is rounded.  For p_j the weights, v_j the values, o the output, r the range (15
scales) of a value's group:
  * a key's rounding moves its score by s_j = scale u / sqrt(3) |q k_j| (the norm of the
    products over the channels), binary32 sums of D terms by scale 2^-22 sqrt(D) |q (|k_j| + r_j)|:
    the output moves by p_j s_j (v_j - o)
  * the weight's and the value's roundings: p_j sqrt(2) u / sqrt(3) (|v_j| + r_j / 2)
The root of their summed squares over keys and channels is the error's standard
deviation; five of them are allowed (one key alone reaches sqrt(3)).  Beside it,
as plain sums because binary32 accumulators may cut rather than round: (n / 16 + 32) 2^-23
of sum_j p_j (|v_j| + r_j) for n keys, 2^-22 of the largest score as a factor of the
output, and the output's own rounding to its type (half a step).

The logarithm of the sum moves by the scores' part, sqrt(sum (p_j s_j)^2), five times,
by (n / 4 + 32) 2^-24 and by 2^-22 of the largest score and of itself."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -11


def dequantised(cache, table, lens):
    """(keys, values, key ranges, value ranges), fp64 [H, L, D], of each sequence."""
    got = []
    P, H, G = cache.page_size, cache.num_heads, cache.head_dim // 64
    shift = torch.arange(0, 32, 4, device=cache.k_codes.device)
    for row, L in zip(torch.as_tensor(table).tolist(), lens):
        pages = torch.tensor(row[: -(-L // P)], dtype=torch.long, device=cache.k_codes.device)
        values, ranges = [], []
        for words, params in ((cache.k_codes, cache.k_params), (cache.v_codes, cache.v_params)):
            c = (words[pages].long().transpose(-1, -2)[..., None] >> shift) & 15      # [n, H, P, G, 8, 8]
            s, o = params[pages].double().unbind(-1)
            x = c.double() * s[..., None, None] + o[..., None, None]
            values.append(x.reshape(-1, H, P, 64 * G).transpose(0, 1).reshape(H, -1, 64 * G)[:, :L])
            r = (15 * s.abs()).repeat_interleave(64, -1)
            ranges.append(r.transpose(0, 1).reshape(H, -1, 64 * G)[:, :L])
        got.append((*values, *ranges))
    return got


def exact(q, kv, new, scale, causal=True, window=0):
    """fp64 (out [T, Hq, D], lse [T, Hq], bound on |error| of a head's output before its own rounding
    [T, Hq], bound of the lse [T, Hq]); kv: `dequantised`'s, or the like."""
    T, Hq, D = q.shape
    x64 = dict(dtype=torch.float64, device=q.device)
    out, bound = torch.zeros(T, Hq, D, **x64), torch.zeros(T, Hq, **x64)
    lse, lse_bound = torch.full((T, Hq), -math.inf, **x64), torch.zeros(T, Hq, **x64)
    at = 0
    for (k, v, rk, rv), n in zip(kv, new):
        H, L, _ = k.shape
        if n == 0:
            continue
        pos = torch.arange(L - n, L, device=q.device)[:, None]
        key = torch.arange(L, device=q.device)
        seen = torch.ones(n, L, dtype=torch.bool, device=q.device)
        if causal:
            seen &= key <= pos
        if window:
            seen &= key > pos - window
        for hq in range(Hq):
            h = hq // (Hq // H)
            qd, kk, vv = q[at:at + n, hq].double(), k[h], v[h]
            x = torch.where(seen, scale * qd @ kk.T, -math.inf)
            if L == 0:
                continue
            lse[at:at + n, hq] = l = torch.logsumexp(x, 1)
            some = torch.isfinite(l)
            p = torch.where(some[:, None], torch.exp(x - torch.where(some, l, 0.0)[:, None]), 0.0)
            o = out[at:at + n, hq] = p @ vv
            s = scale * (U / 3 ** 0.5 * torch.sqrt(qd ** 2 @ (kk ** 2).T)
                         + 2.0 ** -22 * D ** 0.5 * torch.sqrt(qd ** 2 @ ((kk.abs() + rk[h]) ** 2).T))
            w = (p * s) ** 2
            apart = w @ (vv ** 2).sum(1) - 2 * ((w @ vv) * o).sum(1) + w.sum(1) * (o ** 2).sum(1)
            own = 2 * U ** 2 / 3 * (p ** 2 @ ((vv.abs() + rv[h] / 2) ** 2).sum(1))
            most = torch.where(seen, (scale * qd @ kk.T).abs(), 0.0).amax(1)
            count = seen.sum(1)
            bound[at:at + n, hq] = (5 * torch.sqrt(apart.clamp(min=0) + own) + 2.0 ** -22 * most * o.norm(dim=1)
                                    + (count / 16 + 32) * 2.0 ** -23 * (p @ (vv.abs() + rv[h])).norm(dim=1))
            lse_bound[at:at + n, hq] = (5 * torch.sqrt(w.sum(1)) + (count / 4 + 32) * 2.0 ** -24
                                        + 2.0 ** -22 * (most + torch.where(some, l, 0.0).abs() + 1))
        at += n
    return out, lse, bound, lse_bound


def assert_close(got, ref, bound, what=""):
    """Every head's output within its bound and its type's rounding."""
    g, t = got.detach().double(), torch.finfo(got.dtype)
    err, size = (g - ref).norm(dim=-1), ref.norm(dim=-1)
    allowed = bound + t.eps / 2 * (size + bound) + ref.shape[-1] ** 0.5 * t.smallest_normal * t.eps / 2
    off = ~(err <= allowed)                                  # a NaN is off
    assert not off.any(), f"{what}: {int(off.sum())} of {off.numel()} heads off, worst {float((err / allowed).nan_to_num(math.inf).max()):.3g} of the bound"


def assert_lse(got, ref, bound, what=""):
    l, some = got.detach().double(), torch.isfinite(ref)
    assert torch.equal(torch.isneginf(l), ~some), f"{what}: rows that see nothing"
    err = torch.where(some, (l - torch.where(some, ref, 0.0)).abs(), 0.0)
    assert (err <= bound)[some].all(), f"{what}: lse off, worst {float((err / bound)[some].max()):.3g} of the bound"
