"""Refusals of the training and serving entry points: every one is made on the host, before
anything is enqueued (the pointers here are never dereferenced)."""
import ctypes

import pytest

from adaptive_block_sparse_hilbert_b200 import fva

P = ctypes.c_void_p
F = ctypes.c_float


def _bwd(s, mask=None, size=1 << 40, **change):
    m = fva.fva_mask(16, 16, 10, 16, 16, 16, 10, 16, 16) if mask is None else mask
    a = dict(q=256, k=512, v=768, o=1024, do=1280, lse=1536, dq=2048, dk=2304, dv=2560, ws=4096)
    a.update(change)
    x = {n: P(p) for n, p in a.items()}
    return fva.call_raw("fva_sparse_attn_bwd", ctypes.byref(s), x["q"], x["k"], x["v"], x["o"], x["do"], x["lse"],
                        ctypes.byref(m), x["dq"], x["dk"], x["dv"], F(0.0), x["ws"], size, None, None)


def test_gradient_refusals():
    s = fva.make_shape(1, 2, 128, 2, 16, 16, "bf16")
    for name in ("q", "k", "v", "o", "do", "lse", "dq", "dk", "dv", "ws"):
        assert _bwd(s, **{name: None}) == fva.FVA_ERR_INVALID_ARG, name
        assert _bwd(s, **{name: 8}) == fva.FVA_ERR_ALIGNMENT, name
    for out in ("dq", "dk", "dv"):
        for other in (256, 512, 768, 1024, 1280):
            assert _bwd(s, **{out: other}) == fva.FVA_ERR_INVALID_ARG, out
    assert _bwd(s, dq=2304) == fva.FVA_ERR_INVALID_ARG     # dq is dk
    assert _bwd(s, dv=2048) == fva.FVA_ERR_INVALID_ARG     # dv is dq
    assert _bwd(s, mask=fva.fva_mask(16, 16, 10, 16, None, 16, 10, 16, 16)) == fva.FVA_ERR_INVALID_ARG
    need = fva.fva_sparse_attn_bwd_workspace_bytes(s)
    assert _bwd(s, size=need - 1) == fva.FVA_ERR_WORKSPACE
    for bad in (fva.make_shape(1, 2, 32, 2, 16, 16, "bf16"), fva.make_shape(1, 2, 256, 2, 16, 16, "bf16"),
                fva.make_shape(1, 2, 256, 2, 16, 16, "f32"), fva.make_shape(1, 2, 64, 0, 16, 16, "bf16"),
                fva.make_shape(1, 600, 64, 1, 1024, 128, "bf16")):  # the last: 600 * 2048^2 list entries
        assert fva.fva_sparse_attn_bwd_workspace_bytes(bad) == 0
        assert _bwd(bad) == fva.FVA_ERR_UNSUPPORTED_SHAPE
    assert fva.fva_sparse_attn_bwd_workspace_bytes(fva.make_shape(1, 2, 32, 2, 16, 16, "f32")) > 0


def test_forward_lse_refusals():
    s = fva.make_shape(1, 2, 128, 2, 16, 16, "bf16")
    m = fva.fva_mask(16, 16, 10, 16, 16, 16, 10, 16, 16)
    go = lambda lse, o=1024: fva.call_raw("fva_sparse_attn_lse", ctypes.byref(s), P(256), P(512), P(768), fva.FVA_F16,  # noqa: E731
                                          ctypes.byref(m), P(o), P(lse), F(0.0), None, None)
    assert go(None) == fva.FVA_ERR_INVALID_ARG
    assert go(1544) == fva.FVA_ERR_ALIGNMENT
    assert go(2048, 256) == fva.FVA_ERR_INVALID_ARG


def _cache(dtype=fva.FVA_BF16, d=128, Hkv=4, n_pages=10, **change):
    a = dict(k=256, v=512, key_mean=768, mass=1024)
    a.update(change)
    return fva.fva_cache(a["k"], a["v"], a["key_mean"], a["mass"], n_pages, Hkv, d, dtype)


def _seqs(B=2, max_blocks=8, table=4096, length=8192):
    return fva.fva_seqs(table, length, B, max_blocks)


BIG = 1 << 50


def _append(c=None, s=None, k=256, v=512, tokens=20, stride=512, ptr=64, most=10):
    return fva.call_raw("fva_cache_append", ctypes.byref(c or _cache()), ctypes.byref(s or _seqs()), P(k), P(v), tokens, stride,
                        P(ptr), most, None, None)


def _route(c=None, s=None, q=256, H=8, stride=1024, p=0.9, floor=2, recent=1, kept=512, n=768, ws=4096, size=BIG):
    return fva.call_raw("fva_cache_route", ctypes.byref(c or _cache()), ctypes.byref(s or _seqs()), P(q), H, stride, p,
                        floor, recent, F(0.0), P(kept), P(n), P(ws), size, None, None)


def _attn(c=None, s=None, q=256, H=8, stride=1024, kept=512, n=768, o=2048, lse=None, acc=0, ws=4096, size=BIG):
    return fva.call_raw("fva_cache_attn", ctypes.byref(c or _cache()), ctypes.byref(s or _seqs()), P(q), H, stride,
                        P(kept), P(n), P(o), P(lse), F(0.0), acc, P(ws), size, None, None)


def _evict(c=None, s=None, keep=100, sink=4, recent=8, dst=64, blocks=2, kept=512, n=768, ws=4096, size=BIG):
    return fva.call_raw("fva_cache_evict", ctypes.byref(c or _cache()), ctypes.byref(s or _seqs()), keep, sink, recent,
                        P(dst), blocks, P(kept), P(n), P(ws), size, None, None)


@pytest.mark.parametrize("call", [_append, _route, _attn, _evict])
def test_cache_refusals(call):
    for name in ("k", "v", "key_mean"):
        assert call(c=_cache(**{name: None})) == fva.FVA_ERR_INVALID_ARG
        assert call(c=_cache(**{name: 264})) == fva.FVA_ERR_ALIGNMENT
    assert call(c=_cache(mass=1028)) == fva.FVA_ERR_ALIGNMENT
    for change in (dict(d=96), dict(d=32), dict(d=256), dict(dtype=7), dict(Hkv=0), dict(Hkv=65536), dict(n_pages=0)):
        assert call(c=_cache(**change)) == fva.FVA_ERR_UNSUPPORTED_SHAPE, change
    for change in (dict(B=0), dict(B=65536), dict(max_blocks=0), dict(max_blocks=16385)):
        assert call(s=_seqs(**change)) == fva.FVA_ERR_UNSUPPORTED_SHAPE, change
    assert call(s=_seqs(table=None)) == fva.FVA_ERR_INVALID_ARG
    assert call(s=_seqs(length=None)) == fva.FVA_ERR_INVALID_ARG


def test_append_refusals():
    assert _append(k=None) == _append(v=None) == _append(ptr=None) == fva.FVA_ERR_INVALID_ARG
    assert _append(stride=511) == fva.FVA_ERR_INVALID_ARG    # narrower than a token's heads
    assert _append(stride=516) == fva.FVA_ERR_ALIGNMENT
    assert _append(k=260) == fva.FVA_ERR_ALIGNMENT
    assert _append(most=-1) == _append(tokens=-1) == fva.FVA_ERR_INVALID_ARG
    assert _append(most=0) == fva.FVA_OK                     # nothing to append


@pytest.mark.parametrize("call", [_route, _attn])
def test_query_refusals(call):
    assert call(q=None) == fva.FVA_ERR_INVALID_ARG
    assert call(H=6) == call(H=0) == call(H=65536 * 4) == fva.FVA_ERR_UNSUPPORTED_SHAPE
    assert call(H=516, stride=516 * 128) == fva.FVA_ERR_UNSUPPORTED_SHAPE  # 129 query heads per key head
    assert call(stride=1023) == fva.FVA_ERR_INVALID_ARG
    assert call(stride=1028) == fva.FVA_ERR_ALIGNMENT
    assert call(q=264) == fva.FVA_ERR_ALIGNMENT
    assert call(ws=None) == fva.FVA_ERR_INVALID_ARG
    assert call(size=16) == fva.FVA_ERR_WORKSPACE
    assert call(kept=None) == call(n=None) == fva.FVA_ERR_INVALID_ARG
    assert call(kept=520) == fva.FVA_ERR_ALIGNMENT


def test_route_attn_evict_refusals():
    for p in (0.0, -1.0, 1.5, float("nan")):
        assert _route(p=p) == fva.FVA_ERR_INVALID_ARG
    assert _route(floor=-1) == _route(recent=-1) == fva.FVA_ERR_INVALID_ARG
    assert _attn(o=None) == _attn(o=256) == fva.FVA_ERR_INVALID_ARG
    assert _attn(acc=1, c=_cache(mass=None)) == fva.FVA_ERR_INVALID_ARG
    assert _evict(c=_cache(mass=None)) == fva.FVA_ERR_INVALID_ARG
    assert _evict(keep=0) == _evict(keep=(1 << 20) + 1) == _evict(sink=-1) == _evict(recent=-1) == fva.FVA_ERR_INVALID_ARG
    assert _evict(sink=60, recent=41) == fva.FVA_ERR_INVALID_ARG
    assert _evict(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == fva.FVA_ERR_INVALID_ARG
    assert _evict(c=_cache(Hkv=65535)) == fva.FVA_ERR_UNSUPPORTED_SHAPE
    assert _evict(blocks=1) == fva.FVA_ERR_CAPACITY
    assert _evict(dst=None) == _evict(kept=None) == _evict(n=None) == _evict(ws=None) == fva.FVA_ERR_INVALID_ARG
    assert _evict(size=0) == fva.FVA_ERR_WORKSPACE


def test_workspace_queries():
    class Fake:
        def c(self):
            return _cache()
    for q in (lambda b, m: fva.fva_cache_route_workspace_bytes(Fake(), b, m, 8),
              lambda b, m: fva.fva_cache_attn_workspace_bytes(Fake(), b, m, 8, True),
              lambda b, m: fva.fva_cache_evict_workspace_bytes(Fake(), b, m)):
        assert q(0, 8) == q(2, 0) == q(2, 16385) == 0
        assert 0 < q(2, 8) <= q(64, 8) <= q(64, 16384)
