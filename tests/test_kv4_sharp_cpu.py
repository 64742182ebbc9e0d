"""The bound that attention over the 4-bit cache is held to tells right from
wrong: what a right kernel rounds passes, each of several mistakes does not.
The mistakes are made here, in fp64, on the CPU."""
from __future__ import annotations

import pytest
import torch

from kv4_sharp import assert_close, assert_lse, exact
from kv4_util import BF16, F16, quantise_ref

SHAPES = [  # lengths, new tokens, query heads, KV heads, head size, window
    ([500], [1], 8, 2, 64, 0), ([77, 300], [1, 1], 8, 1, 128, 0), ([1025], [1], 4, 4, 128, 0), ([200, 333], [4, 4], 8, 2, 128, 0),
    ([300], [40], 4, 2, 128, 0), ([700], [200], 2, 1, 128, 0), ([150, 400], [6, 6], 4, 2, 128, 100), ([400], [40], 4, 2, 64, 64)]


def inputs(lens, new, Hq, H, D, dtype, seed=0):
    """Queries, and keys and values as a cache holds them (distributions of the GPU tests)."""
    g = torch.Generator().manual_seed(seed)
    kv = []
    mean = torch.randn(H, D, generator=g)
    for L in lens:
        both = []
        for x in (torch.randn(L, H, D, generator=g) + mean, torch.randn(L, H, D, generator=g) + 0.5):
            c, s, o = (torch.from_numpy(a) for a in quantise_ref(x.to(F16)))
            both.append(((c.view(L, H, D // 64, 64) * s.double()[..., None] + o.double()[..., None]).view(L, H, D).transpose(0, 1),
                         (15 * s.double()).repeat_interleave(64, -1).transpose(0, 1)))
        (k, rk), (v, rv) = both
        kv.append((k, v, rk, rv))
    return torch.randn(sum(new), Hq, D, generator=g).to(dtype), kv


def rounded(q, kv, new, scale, window):
    """What the tensor cores round: keys and values to fp16, weights to fp16 under 2^7, the output to its type."""
    half = [(k.half().double(), v.half().double(), rk, rv) for k, v, rk, rv in kv]
    out, lse = torch.zeros(q.shape, dtype=torch.float64), exact(q, half, new, scale, True, window)[1]
    at = 0
    for (k, v, _, _), n in zip(half, new):
        H, L, _ = k.shape
        pos, key = torch.arange(L - n, L)[:, None], torch.arange(L)
        seen = (key <= pos) & (key > pos - window if window else True)
        for hq in range(q.shape[1]):
            h = hq // (q.shape[1] // H)
            x = torch.where(seen, scale * q[at:at + n, hq].double() @ k[h].T, -torch.inf)
            e = torch.exp(x - x.amax(1, keepdim=True))
            out[at:at + n, hq] = (e * 128).half().double() @ v[h] / 128 / e.sum(1, keepdim=True)
        at += n
    return out.to(q.dtype), lse


def mistakes(q, kv, lens, new, scale, window):
    """(name, output) of attention done wrong."""
    ref = exact(q, kv, new, scale, True, window)[0]
    yield "zeros", torch.zeros_like(ref)
    yield "5 % more", 1.05 * ref
    yield "negated queries", exact(-q, kv, new, scale, True, window)[0]
    yield "uniform weights", exact(0 * q, kv, new, scale, True, window)[0]
    yield "scale 3 % off", exact(q, kv, new, 1.03 * scale, True, window)[0]
    yield "query heads in reverse", ref.flip(1)
    yield "values of the next channel", ref.roll(1, -1)
    if q.dtype == F16 or max(lens) <= 500:  # the weight of one key of 1000 is within bf16's half step
        yield "the last key dropped", without(q, kv, new, scale, window, 0, 1)
    yield "16 keys dropped", without(q, kv, new, scale, window, 32, 48)
    if window:
        yield "window one longer", exact(q, kv, new, scale, True, window + 1)[0]
        yield "window one shorter", exact(q, kv, new, scale, True, window - 1)[0]
    if max(new) > 1:
        yield "no causal mask", exact(q, kv, new, scale, False, window)[0]


def without(q, kv, new, scale, window, lo, hi):
    """Attention that misses the keys lo .. hi - 1 from each sequence's end."""
    out, at = torch.zeros(q.shape, dtype=torch.float64), 0
    for (k, v, _, _), n in zip(kv, new):
        H, L, _ = k.shape
        pos, key = torch.arange(L - n, L)[:, None], torch.arange(L)
        seen = (key <= pos) & ((key < L - hi) | (key >= L - lo)) & (key > pos - window if window else True)
        for hq in range(q.shape[1]):
            h = hq // (q.shape[1] // H)
            x = torch.where(seen, scale * q[at:at + n, hq].double() @ k[h].T, -1e300)
            out[at:at + n, hq] = torch.softmax(x, 1) @ v[h]
        at += n
    return out


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_the_kernels_roundings_pass_and_mistakes_do_not(shape, dtype):
    lens, new, Hq, H, D, window = shape
    q, kv = inputs(lens, new, Hq, H, D, dtype)
    scale = D ** -0.5
    ref, lse, bound, lse_bound = exact(q, kv, new, scale, True, window)
    got, got_lse = rounded(q, kv, new, scale, window)
    assert_close(got, ref, bound)
    assert_lse(got_lse, lse, lse_bound)
    for name, wrong in mistakes(q, kv, lens, new, scale, window):
        with pytest.raises(AssertionError, match=name):
            assert_close(wrong.to(dtype), ref, bound, name)
    with pytest.raises(AssertionError):
        assert_lse(lse + 0.01, lse, lse_bound)
