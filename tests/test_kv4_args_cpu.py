"""Argument checks of the norm, 4-bit cache and attention entry points: every
refusal happens on the host, before a device is looked for."""
from __future__ import annotations

import ctypes

import pytest
import torch

import int4_quantized_gemm_b200 as qg

F = 0x10000  # 16-byte aligned, never dereferenced
R = qg.raw


def vp(x):
    return ctypes.c_void_p(x) if x is not None else None


def norm(x=F, ldx=64, res=None, ldr=0, w=F, dtype=qg.QG_F16, eps=1e-5, xq=F, ldq=64, xs=F, ro=None, ldo=0, M=4, K=64):
    return R.qg_rmsnorm_quantize_int8(vp(x), ldx, vp(res), ldr, vp(w), dtype, eps, vp(xq), ldq, vp(xs), vp(ro), ldo, M, K,
                                      None)


def cache(kc=F, kp=F, vc=F, vpar=F, pages=4, heads=2, page=16, dim=64):
    return ctypes.byref(qg._CKV4Cache(kc, kp, vc, vpar, pages, heads, page, dim))


def write(c=None, k=F, kt=128, kh=64, v=F, vt=128, vh=64, dtype=qg.QG_F16, slots=F, T=3):
    return R.qg_quantize_kv4(vp(k), kt, kh, vp(v), vt, vh, dtype, vp(slots), c or cache(), T, None)


def read(c=None, k=F, kt=128, kh=64, v=F, vt=128, vh=64, dtype=qg.QG_F16, slots=F, T=3):
    return R.qg_dequantize_kv4(c or cache(), vp(slots), vp(k), kt, kh, vp(v), vt, vh, dtype, T, None)


def attend(c=None, q=F, qt=256, qh=64, table=F, ld=2, lens=F, starts=None, scale=0.125, causal=1, window=0, out=F, ot=256,
           oh=64, dtype=qg.QG_F16, lse=None, B=2, T=2, Hq=4, pages=2, ws=F, wsn=1 << 40):
    return R.qg_attention_kv4(vp(q), qt, qh, c or cache(), vp(table), ld, vp(lens), vp(starts), scale, causal, window,
                              vp(out), ot, oh, dtype, vp(lse), B, T, Hq, pages, vp(ws), wsn, None)


I, A, U = qg.QG_ERR_INVALID_ARG, qg.QG_ERR_ALIGNMENT, qg.QG_ERR_UNSUPPORTED


@pytest.mark.parametrize("st,kw", [
    (I, dict(M=-1)), (I, dict(K=0)), (I, dict(dtype=qg.QG_F32)), (I, dict(dtype=9)), (I, dict(eps=0.0)), (I, dict(eps=-1.0)),
    (I, dict(eps=float("nan"))), (I, dict(eps=float("inf"))), (I, dict(x=None)), (I, dict(w=None)), (I, dict(xq=None)),
    (I, dict(xs=None)), (I, dict(res=F, ldr=64)), (I, dict(ro=F, ldo=64)), (I, dict(ldx=56)), (A, dict(x=F + 2)),
    (A, dict(ldx=68)), (A, dict(w=F + 8)), (A, dict(ldq=72)), (A, dict(res=F, ldr=68, ro=F, ldo=64)), (A, dict(xs=F + 2)),
    (U, dict(M=1 << 31)), (qg.QG_OK, dict(M=0))])
def test_norm_refusals(st, kw):
    assert norm(**kw) == st


@pytest.mark.parametrize("st,kw", [
    (I, dict(T=-1)), (I, dict(k=None)), (I, dict(v=None)), (I, dict(slots=None)), (A, dict(k=F + 8)), (A, dict(kt=132)),
    (A, dict(vh=68)), (I, dict(kt=-8)), (A, dict(slots=F + 4)), (I, dict(dtype=qg.QG_I32)), (qg.QG_OK, dict(T=0)),
    (U, dict(c=cache(dim=96))), (U, dict(c=cache(dim=256))), (I, dict(c=cache(page=24))), (I, dict(c=cache(page=0))),
    (I, dict(c=cache(heads=0))), (I, dict(c=cache(pages=-1))), (I, dict(c=cache(kc=None))), (A, dict(c=cache(vpar=F + 4))),
    (U, dict(c=cache(pages=1 << 31)))])
def test_cache_refusals(st, kw):
    assert write(**kw) == st
    assert read(**kw) == st
    assert R.qg_quantize_kv4(vp(F), 128, 64, vp(F), 128, 64, 1, vp(F), None, 3, None) == I


def test_only_the_reader_takes_float32():
    assert write(dtype=qg.QG_F32) == I
    assert read(dtype=qg.QG_F32, kt=130) == A and read(dtype=qg.QG_F32, T=0) == qg.QG_OK


@pytest.mark.parametrize("st,kw", [
    (I, dict(B=-1)), (I, dict(T=-2)), (I, dict(Hq=0)), (I, dict(Hq=3)), (I, dict(scale=0.0)), (I, dict(scale=-1.0)),
    (I, dict(scale=float("nan"))), (I, dict(scale=float("inf"))), (I, dict(window=-1)), (I, dict(pages=-1)), (I, dict(T=3)),
    (U, dict(B=4097, T=4097)), (I, dict(q=None)), (I, dict(out=None)), (I, dict(table=None)), (I, dict(ld=1)),
    (I, dict(lens=None)), (A, dict(q=F + 2)), (A, dict(qt=260)), (A, dict(oh=60)), (A, dict(lse=F + 2)), (A, dict(lens=F + 2)),
    (I, dict(dtype=qg.QG_F32)), (U, dict(T=1 << 30, B=2)), (U, dict(pages=1 << 28, ld=1 << 28)), (qg.QG_OK, dict(T=0)),
    (qg.QG_OK, dict(B=0, T=0)), (U, dict(c=cache(dim=192)))])
def test_attention_refusals(st, kw):
    assert attend(**kw) == st


def test_attention_asks_for_its_workspace():
    need = R.qg_attention_kv4_workspace_size(2, 2, 4, 2, 64, 0)
    assert R.qg_attention_kv4_workspace_size(0, 0, 4, 2, 64, 0) == 0
    assert R.qg_attention_kv4_workspace_size(2, 2, 5, 2, 64, 0) == 0      # not a multiple: no such call
    assert need < 1 << 30
    if need:
        assert attend(ws=None, wsn=0) == I and attend(wsn=need - 1) == I and attend(ws=F + 4, wsn=need) == A


def test_plans_repeat_the_direct_calls_status():
    h = ctypes.c_void_p()
    for create, args, st in (
            (R.qg_plan_rmsnorm_quantize_int8, (vp(F), 64, None, 0, vp(F), qg.QG_F16, 0.0, vp(F), 64, vp(F), None, 0, 4, 64), I),
            (R.qg_plan_quantize_kv4, (vp(F), 128, 64, vp(F), 128, 64, 9, vp(F), cache(), 3), I),
            (R.qg_plan_quantize_kv4, (vp(F), 128, 64, vp(F), 128, 64, 1, vp(F), cache(dim=32), 3), U),
            (R.qg_plan_attention_kv4, (vp(F), 256, 64, cache(), vp(F), 2, vp(F), None, 0.0, 1, 0, vp(F), 256, 64, 1, None, 2,
                                       2, 4, 2, vp(F), 1 << 40), I)):
        assert create(ctypes.byref(h), *args) == qg.QG_OK
        assert R.qg_plan_launch(h, None) == st
        R.qg_plan_destroy(h)
        assert create(None, *args) == I
    assert R.qg_plan_quantize_kv4(ctypes.byref(h), vp(F), 128, 64, vp(F), 128, 64, 1, vp(F), None, 3) == I


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_report_no_device():
    assert norm() == qg.QG_ERR_NO_DEVICE and write() == qg.QG_ERR_NO_DEVICE and read() == qg.QG_ERR_NO_DEVICE
    assert attend() == qg.QG_ERR_NO_DEVICE
    assert R.qg_dequantize_rowwise_int8(vp(F), 64, vp(F), vp(F), 1, 64, 4, 64, None) == qg.QG_ERR_NO_DEVICE


def test_dequantize_rowwise_refusals():
    f = lambda xq=F, ldq=64, xs=F, y=F, dt=1, ldy=64, M=4, K=64: R.qg_dequantize_rowwise_int8(
        vp(xq), ldq, vp(xs), vp(y), dt, ldy, M, K, None)
    assert f(dt=3) == I and f(M=-1) == I and f(xq=None) == I and f(y=None) == I and f(xs=None) == I and f(ldy=32) == I
    assert f(xq=F + 8) == A and f(ldq=72) == A and f(ldy=68) == A and f(y=F + 4) == A
    assert f(M=0) == qg.QG_OK and f(K=0) == qg.QG_OK


def test_the_binding_refuses_cpu_tensors_and_wrong_shapes():
    c = qg.kv4_cache(2, 2, 64, 16, device="cpu")
    assert c.num_pages == 2 and c.num_heads == 2 and c.page_size == 16 and c.head_dim == 64
    h = torch.zeros(3, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        qg.quantize_kv4(h, h, c, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        qg.dequantize_kv4(c, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        qg.attention_kv4(h, c, torch.zeros(3, 1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        qg.rmsnorm_quantize_int8(h[:, 0], h[0, 0])
    with pytest.raises(ValueError):
        qg.dequantize_rowwise_int8(torch.zeros(2, 16, dtype=torch.int8), torch.zeros(2))
    for bad in (dict(head_dim=80), dict(page_size=24), dict(page_size=0)):
        with pytest.raises(ValueError):
            qg.kv4_cache(**{**dict(num_pages=1, num_heads=1, head_dim=64, page_size=16, device="cpu"), **bad})
    with pytest.raises(TypeError):
        qg._heads3(h, "k", torch.bfloat16, (3, 2, 64))
    with pytest.raises(ValueError):
        qg._heads3(h.transpose(1, 2), "k", torch.float16, (3, 64, 2))
    with pytest.raises(ValueError):
        qg._cache_arg(c._replace(v_params=c.v_params[:1]))
    with pytest.raises(ValueError):
        qg._cache_arg(c._replace(k_codes=c.k_codes.transpose(0, 1)))
