"""The norm, cache and attention kernels in the debug library (libqg_debug.so):
its device-side checks of every bulk copy's source, place and size report
nothing, and the results equal the release library's bit for bit."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest
import torch

from kv4_util import BF16, F16, paged, random_cache
from parity_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


def qg():
    import int4_quantized_gemm_b200 as q
    return q


@pytest.fixture(scope="module")
def debug():
    q = qg()
    if not os.path.exists(q.DEBUG_LIB_PATH):
        pytest.fail("libqg_debug.so is missing: build it with int4_quantized_gemm_b200/build.py --debug")
    lib = ctypes.CDLL(q.DEBUG_LIB_PATH)
    for name, (args, res) in q.SIGNATURES.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res
    assert lib.qg_debug_checks() == 1
    return lib


def _both(debug, call):
    """Outputs of call() through the release and the debug library."""
    q, release, outs = qg(), qg().raw, []
    try:
        for lib in (release, debug):
            q.raw = lib
            outs.append([t.clone() for t in call()])
            q.check_device_errors()
    finally:
        q.raw = release
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("P", [16, 48, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [[1, 1, 1], [4, 4, 4], [1, 70, 300], [200, 200, 200], [3, 0, 2]])
@pytest.mark.parametrize("window", [0, 100])
def test_attention(debug, P, D, new, window):
    q = qg()
    lens = [1000, 333, 700]
    table, pages = paged(lens, P, 0)
    cache = random_cache(q, pages, 2, D, P, 0)
    qs = torch.randn(sum(new), 8, D, device="cuda").to(F16)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    args = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    _both(debug, lambda: [q.attention_kv4(qs, cache, *args, q_starts=starts if len(set(new)) > 1 else None, window=window)])


@pytest.mark.parametrize("D", [64, 128])
def test_cache_and_norm(debug, D):
    q = qg()
    k, v = torch.randn(2, 500, 3, D, device="cuda").to(BF16)
    slots = torch.randperm(512, device="cuda")[:500].contiguous()

    def cache():
        c = q.kv4_cache(32, 3, D, 16)
        q.quantize_kv4(k, v, c, slots)
        return [*c, *q.dequantize_kv4(c, slots, out_dtype=torch.float32)]

    _both(debug, cache)
    x, r = torch.randn(2, 33, 1000, device="cuda").to(F16)

    def norm():
        a, s, h = q.rmsnorm_quantize_int8(x, x[0].contiguous(), r)
        return [a, s, h, q.dequantize_rowwise_int8(a, s)]

    _both(debug, norm)
