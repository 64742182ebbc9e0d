"""Attention over the paged 4-bit cache (attention_kv4) against fp64, within the
bound that kv4_util.attention_ref derives."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from kv4_util import BF16, F16, assert_attention, attention_ref, paged, random_cache
from parity_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


def qg():
    import int4_quantized_gemm_b200 as q
    return q


def _case(lens, new, Hq, H, D, P, dtype, seed=0, **kw):
    """Random cache and queries; returns (out, lse, reference, lse reference, their bounds)."""
    q = qg()
    table, pages = paged(lens, P, seed)
    cache = random_cache(q, pages, H, D, P, seed)
    T = sum(new)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    qs = torch.randn(T, Hq, D, generator=g, device="cuda").to(dtype)
    lse = torch.full((T, Hq), float("nan"), device="cuda")
    starts = None
    if len(set(new)) > 1 or kw.pop("ragged", False):
        starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    scale = kw.get("scale") or D ** -0.5
    out = torch.full_like(qs, float("nan"))
    got = q.attention_kv4(qs, cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                          q_starts=starts, out=out, lse=lse, **kw)
    assert got is out
    q.check_device_errors()
    ref, rl, bound, lb = attention_ref(qs, cache, table, lens, new, scale, kw.get("causal", True), kw.get("window", 0))
    return out, lse, ref, rl, bound, lb


def _run(lens, new, Hq, H, D, P, dtype, **kw):
    out, lse, ref, rl, bound, lb = _case(lens, new, Hq, H, D, P, dtype, **kw)
    assert_attention(out, ref, bound, str((lens, new, Hq, H, D, P, dtype, kw)))
    l = lse.double().cpu().numpy()
    some = np.isfinite(rl)
    assert np.array_equal(np.isneginf(l), ~some)
    assert (np.abs(l - rl)[some] <= lb[some]).all()


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 500, 1025])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_single_tokens_of_every_length(L, D, dtype):
    _run([L, max(1, L - 1), 1], [1, 1, 1], 8, 2, D, 16, dtype, seed=L)


@pytest.mark.parametrize("Hq,H", [(1, 1), (2, 2), (5, 1), (7, 1), (8, 1), (14, 2), (16, 1), (24, 2), (40, 1), (32, 32)])
@pytest.mark.parametrize("D", [64, 128])
def test_head_groups(Hq, H, D):
    _run([77, 300], [1, 1], Hq, H, D, 32, F16, seed=Hq)


@pytest.mark.parametrize("P", [16, 32, 48, 64, 80, 128, 256, 1024])
def test_page_sizes(P):
    _run([200, P, P + 1, 1], [1] * 4, 8, 2, 128, P, F16, seed=P)
    _run([200, P + 40], [40, 40], 8, 2, 128, P, F16, seed=P)


@pytest.mark.parametrize("n", [2, 3, 4, 5, 8, 9, 16, 17, 31, 33, 64, 100, 130])
@pytest.mark.parametrize("Hq,H", [(4, 1), (2, 2), (7, 1)])
def test_several_query_tokens(n, Hq, H):
    _run([n, n + 1, n + 90, 257 + n], [n] * 4, Hq, H, 128, 16, F16, seed=n)


@pytest.mark.parametrize("n", [1, 2, 6, 40, 150])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 1000])
@pytest.mark.parametrize("D", [64, 128])
def test_windows(n, window, D):
    _run([400, n, 150], [n] * 3, 4, 2, D, 32, F16, seed=window, window=window)


@pytest.mark.parametrize("n", [1, 5, 50, 140])
@pytest.mark.parametrize("window", [0, 30])
def test_without_a_causal_mask(n, window):
    _run([200, n, 333], [n] * 3, 4, 2, 128, 64, BF16, seed=n, causal=False, window=window)


def test_ragged_query_lengths_and_empty_sequences():
    _run([300, 0, 17, 64, 1, 90, 5], [40, 0, 1, 64, 1, 0, 3], 8, 2, 128, 16, F16)
    _run([300, 20, 700], [1, 1, 1], 8, 2, 64, 16, BF16, ragged=True)
    _run([1000, 130, 256, 640], [300, 130, 1, 2], 4, 1, 64, 64, F16)
    _run([60, 70], [0, 0], 4, 1, 64, 64, F16, ragged=True)


@pytest.mark.parametrize("Hq,H,n", [(4, 2, 1), (4, 2, 20), (4, 1, 200)])
def test_more_queries_than_keys(Hq, H, n):
    """The first queries then stand before the sequence: nothing is visible, zeros."""
    out, lse, ref, rl, bound, lb = _case([0, max(n // 2, 0), n], [n] * 3, Hq, H, 128, 16, F16, seed=n)
    assert_attention(out, ref, bound)
    empty = np.isneginf(rl)
    assert empty.any() and not out.cpu().numpy()[empty].any()
    assert torch.isneginf(lse).cpu().numpy()[empty].all()


def test_long_and_short_together():
    _run([20000, 3, 700, 1, 9000], [1] * 5, 8, 2, 128, 64, F16, seed=1)
    _run([30011], [1], 8, 1, 64, 16, BF16, seed=2)
    _run([12000, 500], [4, 4], 8, 2, 64, 128, F16, seed=3)
    _run([5000, 400], [70, 70], 4, 2, 128, 64, F16, seed=4)


def test_many_sequences():
    rng = np.random.default_rng(0)
    lens = [int(a) for a in rng.integers(1, 200, 600)]
    _run(lens, [1] * 600, 2, 1, 64, 16, F16)


def test_scales():
    for scale in (1e-4, 0.5, 2.0):
        _run([333, 64], [1, 1], 8, 2, 64, 16, F16, scale=scale)
        _run([333, 64], [30, 30], 8, 2, 64, 16, F16, scale=scale)


@pytest.mark.parametrize("n", [1, 40])
def test_the_result_does_not_depend_on_what_lies_behind_a_sequence(n):
    """Stale pages, codes, infinities and NaN behind the last token, also inside its page."""
    q = qg()
    lens, P = [37, 100, 64], 32
    table, pages = paged(lens, P, 0)
    a = random_cache(q, pages, 2, 128, P, 0)
    b = q.KV4Cache(*(t.clone() for t in a))
    used = torch.zeros(pages, P, dtype=torch.bool, device="cuda")
    for r, L in zip(table, lens):
        for t in range(L):
            used[r[t // P], t % P] = True
    for codes, params in ((b.k_codes, b.k_params), (b.v_codes, b.v_params)):
        codes.transpose(1, 2)[~used] = -1
        params.transpose(1, 2)[~used] = float("nan")
        params.transpose(1, 2)[:, ::3][~used[:, ::3]] = float("inf")
    qs = torch.randn(3 * n, 8, 128, device="cuda").to(F16)
    args = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    x, y = q.attention_kv4(qs, a, *args), q.attention_kv4(qs, b, *args)
    assert torch.isfinite(y).all() and torch.equal(x, y)


@pytest.mark.parametrize("n", [1, 40])
def test_infinities_and_nan_in_masked_places(n):
    """A key outside the window may hold NaN; a visible one gives NaN to its own sequence only."""
    q = qg()
    lens, P = [200, 200], 16
    table, pages = paged(lens, P, 0)
    cache = random_cache(q, pages, 1, 64, P, 0)
    qs = torch.randn(2 * n, 4, 64, device="cuda").to(F16)
    args = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = q.attention_kv4(qs, cache, *args, window=50)
    for t in range(0, 200 - n - 50):                     # positions that no query's window reaches
        cache.k_params[int(table[0, t // P]), :, t % P] = float("nan")
        cache.v_params[int(table[0, t // P]), :, t % P] = float("nan")
    got = q.attention_kv4(qs, cache, *args, window=50)
    assert torch.equal(want, got)
    got = q.attention_kv4(qs, cache, *args)
    assert torch.isnan(got[:n]).all() and torch.isfinite(got[n:]).all()
    if n > 1:                                            # queries before a NaN key do not see it
        clean = random_cache(q, pages, 1, 64, P, 0)
        want = q.attention_kv4(qs, clean, *args)
        t = 199
        clean.v_params[int(table[0, t // P]), :, t % P] = float("nan")
        got = q.attention_kv4(qs, clean, *args)
        assert torch.equal(want[:n - 1], got[:n - 1]) and torch.isnan(got[n - 1]).all() and torch.equal(want[n:], got[n:])


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("size", [1e-4, 1e-2, 30.0, 500.0])
def test_values_of_any_size(n, size):
    """Small and large values keep their relative accuracy (their scales differ by powers of ten)."""
    q = qg()
    L, P = 150, 16
    table, pages = paged([L], P, 0)
    cache = random_cache(q, pages, 2, 64, P, 0)
    cache.v_params.mul_(size)
    qs = torch.randn(n, 4, 64, device="cuda").to(BF16)
    out = q.attention_kv4(qs, cache, torch.from_numpy(table).cuda(), torch.tensor([L], dtype=torch.int32, device="cuda"))
    ref, _, bound, _ = attention_ref(qs, cache, table, [L], [n], 0.125)
    # scales of 1e-4 are fp16 subnormals only below 6e-5: the cache itself is exact as given
    assert_attention(out, ref, bound + (2.0 ** -24 if size < 1e-2 else 0), f"{size}")


@pytest.mark.parametrize("n", [1, 20])
def test_values_whose_scale_grows_along_the_sequence(n):
    q = qg()
    L, P = 700, 16
    table, pages = paged([L], P, 0)
    cache = random_cache(q, pages, 1, 128, P, 0)
    for t in range(L):
        f = 2.0 ** (16 * t / L - 10)
        cache.v_params[int(table[0, t // P]), :, t % P] *= f
    qs = torch.randn(n, 8, 128, device="cuda").to(F16)
    out = q.attention_kv4(qs, cache, torch.from_numpy(table).cuda(), torch.tensor([L], dtype=torch.int32, device="cuda"))
    ref, _, bound, _ = attention_ref(qs, cache, table, [L], [n], 128 ** -0.5)
    assert_attention(out, ref, bound)


@pytest.mark.parametrize("n", [1, 20])
def test_sharp_and_large_scores(n):
    """One key far above the others, first, middle or last, and queries of any size."""
    q = qg()
    L, P = 300, 16
    table, pages = paged([L], P, 0)
    for at in (0, 150, L - n):
        for size in (1e-3, 1.0, 60.0):
            cache = random_cache(q, pages, 1, 64, P, 0, offset=0.0)
            cache.k_params[int(table[0, at // P]), :, at % P] *= 4
            qs = (torch.randn(n, 4, 64, device="cuda") * size).to(BF16)
            out = q.attention_kv4(qs, cache, torch.from_numpy(table).cuda(),
                                  torch.tensor([L], dtype=torch.int32, device="cuda"))
            ref, _, bound, _ = attention_ref(qs, cache, table, [L], [n], 0.125)
            assert_attention(out, ref, bound, f"{at} {size}")


@pytest.mark.parametrize("n", [1, 24])
def test_strided_queries_and_outputs_and_rows_behind_the_last_sequence(n):
    q = qg()
    lens, P = [50, 90], 16
    table, pages = paged(lens, P, 0)
    cache = random_cache(q, pages, 2, 128, P, 0)
    buf = torch.randn(2 * n + 3, 12 * 128, device="cuda").to(F16)      # a fused projection with three rows of padding
    qs = buf[:, :8 * 128].view(-1, 8, 128)
    starts = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    out = torch.full((2 * n + 3, 10, 128), 7.0, dtype=F16, device="cuda")
    tb = torch.full((2, 40), 12345678, dtype=torch.int32, device="cuda")
    tb[:, :table.shape[1]] = torch.from_numpy(table)
    args = tb[:, :table.shape[1]], torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.full((2 * n + 3, 8), 5.0, device="cuda")
    q.attention_kv4(qs, cache, *args, q_starts=starts, out=out[:, 1:9], lse=lse)
    want = q.attention_kv4(qs[:2 * n].contiguous(), cache, *args)
    assert torch.equal(out[:2 * n, 1:9], want)
    assert (out[:, 0] == 7).all() and (out[:, 9] == 7).all() and (out[2 * n:] == 7).all() and (lse[2 * n:] == 5).all()
    # head-major queries
    hm = qs[:2 * n].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(q.attention_kv4(hm, cache, *args), want)


@pytest.mark.parametrize("n", [1, 40])
def test_the_same_call_twice_gives_the_same_bits(n):
    q = qg()
    lens, P = [5000, 77, 1200], 64
    table, pages = paged(lens, P, 0)
    cache = random_cache(q, pages, 2, 128, P, 0)
    qs = torch.randn(3 * n, 8, 128, device="cuda").to(F16)
    args = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = q.attention_kv4(qs, cache, *args)
    for _ in range(5):
        assert torch.equal(a, q.attention_kv4(qs, cache, *args))


@pytest.mark.parametrize("n", [1, 40])
def test_shared_pages(n):
    """Two sequences with a common prefix share its pages."""
    q = qg()
    P, L = 16, 130
    table, pages = paged([L, L], P, 0)
    table[1, :5] = table[0, :5]
    cache = random_cache(q, pages, 2, 64, P, 0)
    qs = torch.randn(2 * n, 4, 64, device="cuda").to(F16)
    out = q.attention_kv4(qs, cache, torch.from_numpy(table).cuda(), torch.tensor([L, L], dtype=torch.int32, device="cuda"))
    ref, _, bound, _ = attention_ref(qs, cache, table, [L, L], [n, n], 0.125)
    assert_attention(out, ref, bound)


def test_bad_device_data_is_reported_and_not_followed():
    """Page indices outside the cache, lengths beyond the table, starts outside q: never read or written."""
    q = qg()
    cache = random_cache(q, 4, 2, 64, 16, 0)
    dev = dict(dtype=torch.int32, device="cuda")
    for n in (1, 40):
        qs = torch.randn(2 * n, 4, 64, device="cuda").to(F16)
        good = torch.tensor([[0, 1], [2, 3]], **dev)
        for table, lens, starts in (([[0, 9], [2, 3]], [20, 20], None), ([[0, -5], [2, 3]], [20, 20], None),
                                    ([[0, 1], [2, 3]], [20, 1000], None), ([[0, 1], [2, 3]], [-3, 20], None),
                                    ([[0, 1], [2, 3]], [20, 20], [0, n, 2 * n + 5]),
                                    ([[0, 1], [2, 3]], [20, 20], [0, 2 * n, n]), ([[0, 1], [2, 3]], [20, 20], [-2, n, 2 * n])):
            st = None if starts is None else torch.tensor(starts, **dev)
            q.attention_kv4(qs, cache, torch.tensor(table, **dev), torch.tensor(lens, **dev), q_starts=st)
            with pytest.raises(q.QGError) as e:
                q.check_device_errors()
            assert e.value.status == q.QG_ERR_INVALID_ARG, (table, lens, starts)
        q.attention_kv4(qs, cache, good, torch.tensor([20, 32], **dev))
        q.check_device_errors()


def test_two_calls_on_two_streams_and_two_graphs():
    """Scratch is each call's own: calls in flight together do not touch one another's."""
    q = qg()
    lens, P = [9000, 1], 64
    table, pages = paged(lens, P, 0)
    cache = random_cache(q, pages, 2, 128, P, 0)
    args = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = [torch.randn(2, 8, 128, device="cuda").to(F16) for _ in range(2)]
    want = [q.attention_kv4(x, cache, *args) for x in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(q.attention_kv4(qs[i], cache, *args))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], x) for x in got[i])
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(q.attention_kv4(qs[i], cache, *args))
        graphs.append(g)
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    q.check_device_errors()


@pytest.mark.parametrize("n", [1, 40])
def test_a_plan_follows_its_buffers(n):
    """A decode loop: lengths, table and queries change in place between launches."""
    q = qg()
    P, B = 16, 3
    cache = random_cache(q, 30, 2, 128, P, 0)
    qs = torch.randn(B * n, 8, 128, device="cuda").to(F16)
    table = torch.randperm(30, device="cuda").to(torch.int32).view(3, 10)
    lens = torch.tensor([n, n + 5, n + 70], dtype=torch.int32, device="cuda")
    p = q.plan_attention_kv4(qs, cache, table, lens)
    p.launch()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.launch()
    for step in range(3):
        lens += step
        qs.mul_(0.9)
        want = q.attention_kv4(qs, cache, table, lens)
        p.out.zero_()
        p.launch() if step == 1 else g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, p.out)
    q.check_device_errors()


def test_offsets_past_32_bits():
    """Pages behind 2^32 bytes of codes."""
    q = qg()
    H, D, P = 8, 128, 256
    pages = (1 << 32) // (H * P * D // 2) + 3
    big, small = q.kv4_cache(pages, H, D, P), random_cache(q, 2, H, D, P, 0)
    for a, b in zip(big, small):
        a[-2:] = b
    for n in (1, 40):
        qs = torch.randn(n, 8, 128, device="cuda").to(F16)
        lens = torch.tensor([400], dtype=torch.int32, device="cuda")
        x = q.attention_kv4(qs, big, torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device="cuda"), lens)
        y = q.attention_kv4(qs, small, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), lens)
        assert torch.equal(x, y)


def test_merging_by_the_log_sum_exp():
    """Two disjoint ranges of keys (a window and the whole) joined through lse give the whole."""
    q = qg()
    L, P = 256, 16
    table, pages = paged([L], P, 0)
    cache = random_cache(q, pages, 2, 64, P, 0)
    qs = torch.randn(1, 4, 64, device="cuda").to(F16)
    tb = torch.from_numpy(table).cuda()
    la, lb, lw = (torch.empty(1, 4, device="cuda") for _ in range(3))
    dev = dict(dtype=torch.int32, device="cuda")
    a = q.attention_kv4(qs, cache, tb, torch.tensor([L], **dev), window=96, lse=la).double()
    b = q.attention_kv4(qs, cache, tb, torch.tensor([L - 96], **dev), lse=lb).double()
    w = q.attention_kv4(qs, cache, tb, torch.tensor([L], **dev), lse=lw).double()
    wa, wb = torch.exp((la - lw).double())[..., None], torch.exp((lb - lw).double())[..., None]
    ref, _, bound, _ = attention_ref(qs, cache, table, [L], [1], 0.125)
    tol = torch.from_numpy(3 * bound).cuda() + 3 * 2.0 ** -11 * (wa * a.abs() + wb * b.abs() + w.abs())
    assert ((wa * a + wb * b - w).abs() <= tol).all()


@pytest.mark.parametrize("n,L", [(300, 300), (513, 700), (1024, 1024), (256, 3000), (130, 6000)])
@pytest.mark.parametrize("D", [64, 128])
def test_long_prompts(n, L, D):
    """Many steps over the keys by both row tiles, one share of the keys a block (many heads) and several (one)."""
    _run([L], [n], 2, 1, D, 64, F16, seed=n)
    q = qg()
    table, pages = paged([L], 64, 1)
    one = random_cache(q, pages, 1, D, 64, 1)
    many = q.KV4Cache(*(t.expand(-1, 160, *t.shape[2:]).contiguous() for t in one))
    qs = torch.randn(n, 1, D, device="cuda").to(F16)
    args = torch.from_numpy(table).cuda(), torch.tensor([L], dtype=torch.int32, device="cuda")
    x = q.attention_kv4(qs.expand(-1, 160, -1).contiguous(), many, *args)
    q.check_device_errors()
    ref, _, bound, _ = attention_ref(qs, one, table, [L], [n], D ** -0.5)
    assert_attention(x[:, :1], ref, bound)
    assert torch.equal(x, x[:, :1].expand(-1, 160, -1))


@pytest.mark.parametrize("new", [[3, 4, 1, 2, 4], [4, 0, 4, 4, 3], [1, 3, 3, 5, 4], [2, 1, 1, 2, 2]])
@pytest.mark.parametrize("D", [64, 128])
def test_ragged_drafts(new, D):
    """Sequences of a few tokens each, one of them with more rows than the others' kernel takes; idle ones between."""
    lens = [700, 33, 3, 5000, 64]
    _run(lens, new, 8, 2, D, 16, F16, seed=sum(new))
    _run(lens, new, 8, 2, D, 64, BF16, seed=sum(new), window=100)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [[1, 40, 1], [1, 300, 300], [20, 20, 20]])
def test_prompts_and_tokens_in_one_call_follow_what_came_before(new, D):
    """The two kernels of a ragged call overlap: neither starts before the cache's writer, nor does a later kernel
    start before both."""
    q = qg()
    lens, P, H, Hq = [3000, 600, 900], 16, 2, 8
    table, pages = paged(lens, P, 0)
    T = sum(new)
    tb, n = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    slots = torch.arange(pages * P, device="cuda")
    ks = [torch.randn(pages * P, H, D, device="cuda").to(F16) for _ in range(4)]
    qs = torch.randn(T, Hq, D, device="cuda").to(F16)
    want = []
    for k in ks:
        cache = q.kv4_cache(pages, H, D, P)
        q.quantize_kv4(k, k, cache, slots)
        torch.cuda.synchronize()
        want.append(q.attention_kv4(qs, cache, tb, n, q_starts=starts))
        torch.cuda.synchronize()
    cache = q.kv4_cache(pages, H, D, P)
    out = [torch.empty_like(qs) for _ in ks]
    codes = [torch.empty(T, Hq * D, dtype=torch.int8, device="cuda") for _ in ks]
    scales = [torch.empty(T, device="cuda") for _ in ks]

    def step():
        for i, k in enumerate(ks):
            q.quantize_kv4(k, k, cache, slots)
            q.attention_kv4(qs, cache, tb, n, q_starts=starts, out=out[i])
            q.quantize_rowwise_int8(out[i].view(T, -1), out=codes[i], scale_out=scales[i])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        for o in out:
            o.zero_()
        graph.replay()
        for i in range(len(ks)):
            assert torch.equal(out[i], want[i])
            a, b = q.quantize_rowwise_int8(want[i].view(T, -1))
            assert torch.equal(codes[i], a) and torch.equal(scales[i], b)
    q.check_device_errors()


@pytest.mark.parametrize("new", [[1, 1, 40, 1], [3, 4, 4, 3], [1, 300, 1, 1]])
def test_ragged_calls_see_lengths_and_tables_written_just_before(new):
    """Lengths, starts and table change on the device right before each call of a replayed graph."""
    q = qg()
    B, P, H, Hq, D, pages, calls = len(new), 16, 2, 8, 128, 600, 6
    cache = random_cache(q, pages, H, D, P, 0)
    rng = np.random.default_rng(0)
    qs = torch.randn(sum(new), Hq, D, device="cuda").to(F16)
    tables = [torch.from_numpy(rng.permutation(pages)[:B * 100].reshape(B, 100).astype(np.int32)).cuda() for _ in range(calls)]
    lens = [torch.from_numpy(rng.integers(max(new), 1600, B).astype(np.int32)).cuda() for _ in range(calls)]
    orders = [rng.permutation(new) for _ in range(calls)]
    starts = [torch.tensor(np.concatenate([[0], np.cumsum(o)]), dtype=torch.int32, device="cuda") for o in orders]
    want = []
    for i in range(calls):
        want.append(q.attention_kv4(qs, cache, tables[i], lens[i], q_starts=starts[i]))
        torch.cuda.synchronize()
    t, n, s = (torch.empty_like(x[0]) for x in (tables, lens, starts))
    outs = [torch.empty_like(qs) for _ in range(calls)]

    def step():
        for i in range(calls):
            t.copy_(tables[i])
            s.copy_(starts[i])
            n.copy_(lens[i])
            q.attention_kv4(qs, cache, t, n, q_starts=s, out=outs[i])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(30):
        for o in outs:
            o.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    q.check_device_errors()
