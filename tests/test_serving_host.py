"""Refusals of the single-token serving entry points: every argument error
comes back before any CUDA call, so these run without a GPU."""
import ctypes

import pytest
import torch

import block_scaled_fp4_reduce_b200 as fp4
from block_scaled_fp4_reduce_b200 import build as fp4_build

P = 1 << 20     # a fake, aligned "device" address (never dereferenced)
Q = P + 4       # misaligned


@pytest.fixture(scope="module")
def L():
    fp4_build.build()
    return fp4.lib()


def cache(fmt=fp4.NVFP4, heads=2, head_dim=128, page_size=64, num_pages=4, kp=P, ks=P, vp=P, vs=P, kg=P, vg=P):
    return fp4.KVCacheStruct(fmt, heads, head_dim, page_size, num_pages, kp, ks, vp, vs, kg, vg)


def ref(c):
    return ctypes.addressof(c)


BAD_CACHES = [
    (dict(fmt=2), fp4.ERR_INVALID_ARG), (dict(heads=0), fp4.ERR_INVALID_ARG), (dict(head_dim=0), fp4.ERR_INVALID_ARG),
    (dict(page_size=-16), fp4.ERR_INVALID_ARG), (dict(num_pages=0), fp4.ERR_INVALID_ARG),
    (dict(page_size=24), fp4.ERR_SHAPE), (dict(head_dim=48), fp4.ERR_SHAPE), (dict(head_dim=2048), fp4.ERR_SHAPE),
    (dict(heads=1 << 14), fp4.ERR_SHAPE), (dict(num_pages=1 << 40), fp4.ERR_SHAPE),
    (dict(kp=None), fp4.ERR_INVALID_ARG), (dict(vs=None), fp4.ERR_INVALID_ARG), (dict(kg=None), fp4.ERR_INVALID_ARG),
    (dict(vp=Q), fp4.ERR_ALIGN), (dict(ks=P + 8), fp4.ERR_ALIGN), (dict(vg=P + 2), fp4.ERR_ALIGN),
]


@pytest.mark.parametrize("bad,want", BAD_CACHES, ids=lambda v: str(v))
def test_cache_refusals(L, bad, want):
    c = cache(**bad)
    assert L.fp4_kv_write(ref(c), P, P, fp4.BF16, 4, 256, 256, P, 0, P, None) == want
    assert L.fp4_kv_read(ref(c), P, 4, P, P, fp4.BF16, 256, 256, P, None) == want
    assert L.fp4_kv_attention(ref(c), P, fp4.BF16, 1, 1, 2, 256, P, 4, P, 1.0, 0, P, P, P, 1 << 30, P, None) == want
    assert L.fp4_kv_attention_workspace_bytes(ref(c), 1, 1, 2, 4) == 0
    assert L.fp4_kv_write(None, P, P, fp4.BF16, 4, 256, 256, P, 0, P, None) == fp4.ERR_INVALID_ARG


def test_write_and_read_refusals(L):
    c = cache()
    w = lambda k=P, v=P, dt=fp4.BF16, T=4, ks=256, vs=256, s=P, rule=0, st=P: L.fp4_kv_write(  # noqa: E731
        ref(c), k, v, dt, T, ks, vs, s, rule, st, None)
    r = lambda k=P, v=P, dt=fp4.BF16, T=4, ks=256, vs=256, s=P, rule=0, st=P: L.fp4_kv_read(  # noqa: E731
        ref(c), s, T, k, v, dt, ks, vs, st, None)
    for f in (w, r):
        assert f(dt=2) == fp4.ERR_INVALID_ARG
        assert f(T=-1) == fp4.ERR_INVALID_ARG
        assert f(T=0, k=None, v=None, s=None) == fp4.OK             # nothing to do
        assert f(st=None) == fp4.ERR_INVALID_ARG
        assert f(k=None) == fp4.ERR_INVALID_ARG and f(s=None) == fp4.ERR_INVALID_ARG
        assert f(ks=255) == fp4.ERR_SHAPE                            # shorter than a token
        assert f(vs=1 << 62) == fp4.ERR_SHAPE
        assert f(k=P + 16) == fp4.ERR_ALIGN and f(vs=264) == fp4.ERR_ALIGN and f(s=Q) == fp4.ERR_ALIGN
    assert w(rule=2) == fp4.ERR_INVALID_ARG


def test_attention_refusals(L):
    def f(c=None, q=P, dt=fp4.BF16, B=2, T=1, HQ=4, qs=512, pt=P, width=4, lens=P, scale=1.0, window=0, out=P, lse=P,
          ws=P, wsn=1 << 30, st=P):
        c = c or cache()
        return L.fp4_kv_attention(ref(c), q, dt, B, T, HQ, qs, pt, width, lens, scale, window, out, lse, ws, wsn, st, None)
    assert f(dt=9) == fp4.ERR_INVALID_ARG and f(st=None) == fp4.ERR_INVALID_ARG
    assert f(window=-1) == fp4.ERR_INVALID_ARG
    assert f(scale=float("nan")) == fp4.ERR_INVALID_ARG and f(scale=float("inf")) == fp4.ERR_INVALID_ARG
    assert f(B=-1) == fp4.ERR_INVALID_ARG and f(T=-1) == fp4.ERR_INVALID_ARG and f(HQ=0) == fp4.ERR_INVALID_ARG
    assert f(width=-1) == fp4.ERR_INVALID_ARG
    assert f(B=0) == fp4.OK and f(T=0) == fp4.OK
    assert f(HQ=3) == fp4.ERR_SHAPE                                  # not whole groups
    assert f(c=cache(head_dim=96), qs=512) == fp4.ERR_SHAPE
    assert f(qs=511) == fp4.ERR_SHAPE
    assert f(width=1 << 31) == fp4.ERR_SHAPE and f(B=1 << 31) == fp4.ERR_SHAPE and f(T=1 << 30, HQ=4) == fp4.ERR_SHAPE
    assert f(q=None) == fp4.ERR_INVALID_ARG and f(out=None) == fp4.ERR_INVALID_ARG
    assert f(lens=None) == fp4.ERR_INVALID_ARG and f(pt=None) == fp4.ERR_INVALID_ARG
    assert f(q=P + 8) == fp4.ERR_ALIGN and f(qs=516) == fp4.ERR_ALIGN and f(out=Q) == fp4.ERR_ALIGN
    assert f(lens=P + 2) == fp4.ERR_ALIGN and f(lse=P + 2) == fp4.ERR_ALIGN and f(ws=P + 8) == fp4.ERR_ALIGN
    assert f(ws=None) == fp4.ERR_WORKSPACE and f(wsn=0) == fp4.ERR_WORKSPACE
    c = cache()
    need = L.fp4_kv_attention_workspace_bytes(ref(c), 2, 1, 4, 4)
    assert need >= 16 and f(wsn=need - 1) == fp4.ERR_WORKSPACE


def test_linear_refusals(L):
    def f(fmt=fp4.NVFP4, x=P, dt=fp4.BF16, rows=4, K=256, xs=256, pk=P, sc=P, g=P, N=100, y=P, odt=fp4.BF16, ws=P,
          wsn=1 << 40, st=P):
        return L.fp4_linear(fmt, x, dt, rows, K, xs, pk, sc, g, N, y, odt, ws, wsn, st, None)
    assert f(fmt=2) == fp4.ERR_INVALID_ARG and f(dt=2) == fp4.ERR_INVALID_ARG and f(odt=2) == fp4.ERR_INVALID_ARG
    assert f(rows=-1) == fp4.ERR_INVALID_ARG and f(N=-1) == fp4.ERR_INVALID_ARG and f(K=-1) == fp4.ERR_INVALID_ARG
    assert f(st=None) == fp4.ERR_INVALID_ARG
    assert f(K=240, xs=240) == fp4.ERR_SHAPE                         # 15 blocks of 16: the row pitch is not whole vectors
    assert f(rows=1 << 31) == fp4.ERR_SHAPE and f(N=1 << 31) == fp4.ERR_SHAPE
    assert f(xs=255) == fp4.ERR_SHAPE
    assert f(rows=0) == fp4.OK and f(N=0) == fp4.OK
    assert f(x=None) == fp4.ERR_INVALID_ARG and f(pk=None) == fp4.ERR_INVALID_ARG and f(y=None) == fp4.ERR_INVALID_ARG
    assert f(g=None) == fp4.ERR_INVALID_ARG
    assert f(x=P + 1) == fp4.ERR_ALIGN and f(pk=P + 8) == fp4.ERR_ALIGN and f(sc=P + 8) == fp4.ERR_ALIGN
    assert f(y=P + 1) == fp4.ERR_ALIGN and f(odt=fp4.F32, y=P + 2) == fp4.ERR_ALIGN
    assert f(ws=None) == fp4.ERR_WORKSPACE and f(wsn=0) == fp4.ERR_WORKSPACE and f(ws=P + 4) == fp4.ERR_ALIGN


def test_sizes_below_zero_and_overflow_give_no_workspace(L):
    assert L.fp4_linear_workspace_bytes(-1, 4) == 0 and L.fp4_linear_workspace_bytes(4, -1) == 0
    assert L.fp4_linear_workspace_bytes(1 << 40, 32) == 0


@pytest.mark.parametrize("rows,n,dt,want", [
    (1, 65535 * 128, fp4.BF16, None), (1, 65535 * 128 + 1, fp4.BF16, fp4.ERR_SHAPE), (1, (1 << 63) - 1, fp4.BF16, fp4.ERR_SHAPE),
    ((1 << 23) - 1, 8, fp4.BF16, None), (1 << 23, 8, fp4.BF16, fp4.ERR_SHAPE), (65535 * 80, 8, fp4.F32, None),
    (65535 * 80 + 1, 8, fp4.F32, fp4.ERR_SHAPE)])
def test_linear_s_largest_shapes(L, rows, n, dt, want):
    """Up to the grid's limits a call gets as far as its workspace (refused here: none is given)."""
    got = L.fp4_linear(fp4.NVFP4, P, dt, rows, 32, 32, P, P, P, n, P, fp4.BF16, None, 0, P, None)
    assert got == (fp4.ERR_WORKSPACE if want is None else want)


def test_status_string_of_a_bad_index(L):
    assert L.fp4_status_string(fp4.ERR_INDEX) == b"slot, page or length out of range"


def test_binding_refuses_cpu_tensors_and_wrong_types():
    t = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        fp4.KVCache(fp4.NVFP4, t, t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        fp4.LinearWeight(fp4.NVFP4, torch.zeros(4, 16, dtype=torch.uint8), t, torch.ones(1), 4, 32)


def test_linear_weight_refuses_cpu_tensors():
    """Before the layout kernel is launched on host addresses."""
    t = torch.zeros(4, 16, dtype=torch.uint8)
    q = fp4.Quantized(fp4.NVFP4, t, torch.zeros(4, 2, dtype=torch.uint8), torch.ones(1), torch.zeros(1, dtype=torch.int32), 4, 32)
    with pytest.raises(ValueError, match="CUDA"):
        fp4.linear_weight(q)


@pytest.mark.parametrize("k,fits", [(16, False), (48, False), (240, False), (225, False), (224, True), (255, True), (32, True)])
def test_linear_weight_names_the_k_it_takes(k, fits):
    """An NVFP4 weight of an odd number of 16-blocks is refused when it is laid out, not by every call with it."""
    t = torch.zeros(4, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA" if fits else "multiple of 32"):
        fp4.LinearWeight(fp4.NVFP4, t, t, torch.ones(1), 4, k)
    with pytest.raises(ValueError, match="CUDA"):
        fp4.LinearWeight(fp4.MXFP4, t, t, None, 4, k)
