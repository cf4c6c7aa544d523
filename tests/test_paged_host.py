"""Refusals of the paged-cache calls and of the head norms: every bad argument
is turned down on the host, before any device work."""
import ctypes

import numpy as np
import pytest

from rotated_codebook_kv_tq_b200 import native


@pytest.fixture(scope="module")
def L():
    from rotated_codebook_kv_tq_b200.build import build
    build()
    return native.lib()


@pytest.fixture(scope="module")
def codec(L):
    """A codec without device memory (no sketch, Walsh-Hadamard rotation)."""
    def make(d):
        desc = native.CodecDesc(d, 3, 0, 3, np.ones(d, np.int8).ctypes.data, None, None)
        signs = np.ones(d, np.int8)
        desc.rotation_signs = signs.ctypes.data
        h = ctypes.c_void_p()
        assert L.tq_codec_create(ctypes.byref(desc), ctypes.byref(h)) == native.TQ_OK
        return h
    return {d: make(d) for d in (64, 128, 1536)}


X = 0x10000   # stands for a device buffer: refused calls never read it


def cache(pages=4, heads=2, page=64, **kw):
    f = dict(kcode=X, kscale=X, vcode=X, vnorm=X, B=pages, Hkv=heads, rows_cap=page)
    f.update(kw)
    return native.CacheDesc(**f)


def batch(**kw):
    f = dict(page_table=X, q_start=X, seq_lens=X, table_stride=2, num_seqs=3, max_pages=2, max_new=8,
             max_seq_len=128)
    f.update(kw)
    return native.PagedBatchDesc(**f)


def quantize(L, c, k=X, v=X, dtype=1, N=8, rc=None, rs=None, rn=0, ca=None, b=None, status=None):
    return L.tq_paged_quantize_kv(c, k, v, dtype, N, 256, 64, rc, rs, rn, ctypes.byref(ca or cache()),
                                  ctypes.byref(b or batch()), status, None)


def dequantize(L, c, k=X, v=X, dtype=1, N=8, ca=None, b=None):
    return L.tq_paged_dequantize(c, ctypes.byref(ca or cache()), ctypes.byref(b or batch()), N, k, v, dtype, None)


def attention(L, c, q=X, dtype=1, N=8, Hq=4, scale=0.1, rc=None, rs=None, rn=0, ws=X, wsb=1 << 40, out=X,
              odt=1, ca=None, b=None):
    return L.tq_paged_attention(c, q, dtype, N, Hq, 256, 64, ctypes.byref(ca or cache()),
                                ctypes.byref(b or batch()), scale, rc, rs, rn, ws, wsb, out, odt, None)


BAD_BATCH = [
    (dict(num_seqs=-1), native.TQ_ERR_INVALID_ARG), (dict(max_new=-1), native.TQ_ERR_INVALID_ARG),
    (dict(max_seq_len=129), native.TQ_ERR_INVALID_ARG), (dict(max_pages=-1), native.TQ_ERR_INVALID_ARG),
    (dict(num_seqs=65536), native.TQ_ERR_INVALID_ARG), (dict(page_table=None), native.TQ_ERR_INVALID_ARG),
    (dict(q_start=None), native.TQ_ERR_INVALID_ARG), (dict(seq_lens=None), native.TQ_ERR_INVALID_ARG),
    (dict(table_stride=1), native.TQ_ERR_INVALID_ARG), (dict(q_start=X + 2), native.TQ_ERR_ALIGNMENT),
]
BAD_CACHE = [
    (dict(kcode=None), native.TQ_ERR_INVALID_ARG), (dict(B=0), native.TQ_ERR_INVALID_ARG),
    (dict(rows_cap=16), native.TQ_ERR_INVALID_ARG), (dict(rows_cap=96), native.TQ_ERR_INVALID_ARG),
    (dict(rows_cap=1 << 21), native.TQ_ERR_INVALID_ARG), (dict(vcode=X + 8), native.TQ_ERR_ALIGNMENT),
    (dict(kscale=X + 4), native.TQ_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("call", [quantize, dequantize, attention])
def test_every_paged_call_refuses_bad_batches_and_caches(L, codec, call):
    for kw, code in BAD_BATCH:
        assert call(L, codec[128], b=batch(**kw)) == code, kw
    for kw, code in BAD_CACHE:
        assert call(L, codec[128], ca=cache(**kw)) == code, kw
    assert call(L, None) == native.TQ_ERR_INVALID_ARG
    assert call(L, codec[1536]) == native.TQ_ERR_UNSUPPORTED
    assert call(L, codec[128], N=-1) == native.TQ_ERR_INVALID_ARG
    assert call(L, codec[128], N=(1 << 24) + 1) == native.TQ_ERR_INVALID_ARG
    # nothing to do: accepted without device work
    assert call(L, codec[128], N=0) == native.TQ_OK
    assert call(L, codec[128], b=batch(num_seqs=0)) == native.TQ_OK
    assert call(L, codec[128], b=batch(max_new=0)) == native.TQ_OK


def test_quantize_refusals(L, codec):
    c = codec[64]
    assert quantize(L, c, k=None) == native.TQ_ERR_INVALID_ARG
    assert quantize(L, c, dtype=2) == native.TQ_ERR_INVALID_ARG
    assert quantize(L, c, rc=X) == native.TQ_ERR_INVALID_ARG
    assert quantize(L, c, rc=X, rs=X, rn=127) == native.TQ_ERR_INVALID_ARG
    assert quantize(L, c, k=X + 1) == native.TQ_ERR_ALIGNMENT
    assert quantize(L, c, dtype=0, v=X + 2) == native.TQ_ERR_ALIGNMENT
    assert b"paged_quantize" in L.tq_last_error()


def test_dequantize_refusals(L, codec):
    c = codec[64]
    assert dequantize(L, c, k=None, v=None) == native.TQ_ERR_INVALID_ARG
    assert dequantize(L, c, dtype=5) == native.TQ_ERR_INVALID_ARG
    assert dequantize(L, c, k=X + 8) == native.TQ_ERR_ALIGNMENT


def test_attention_refusals(L, codec):
    c = codec[64]
    assert attention(L, c, q=None) == native.TQ_ERR_INVALID_ARG
    assert attention(L, c, out=None) == native.TQ_ERR_INVALID_ARG
    assert attention(L, c, Hq=5) == native.TQ_ERR_INVALID_ARG
    assert attention(L, c, Hq=0) == native.TQ_ERR_INVALID_ARG
    assert attention(L, c, scale=float("nan")) == native.TQ_ERR_INVALID_ARG
    assert attention(L, c, dtype=3) == native.TQ_ERR_INVALID_ARG
    assert attention(L, c, odt=3) == native.TQ_ERR_INVALID_ARG
    assert attention(L, c, rs=X) == native.TQ_ERR_INVALID_ARG
    assert attention(L, c, rc=X, rs=X, rn=1) == native.TQ_ERR_INVALID_ARG
    assert attention(L, c, out=X + 8) == native.TQ_ERR_ALIGNMENT
    n = ctypes.c_size_t(0)
    assert L.tq_paged_attention_workspace(c, ctypes.byref(batch()), 8, 4, 2, ctypes.byref(n)) == native.TQ_OK
    assert n.value > 0
    assert attention(L, c, wsb=n.value - 1) == native.TQ_ERR_WORKSPACE
    assert attention(L, c, ws=None) == native.TQ_ERR_WORKSPACE
    assert attention(L, c, ws=X + 8) == native.TQ_ERR_ALIGNMENT
    # limits of empty and of very large steps
    for kw in (dict(num_seqs=0), dict(max_new=0), dict(max_seq_len=0), dict(max_new=(1 << 31) - 1)):
        assert L.tq_paged_attention_workspace(c, ctypes.byref(batch(**kw)), 8, 4, 2, ctypes.byref(n)) == native.TQ_OK
    for bad in (dict(N=-1), dict(Hq=3), dict(Hkv=0)):
        a = dict(N=8, Hq=4, Hkv=2)
        a.update(bad)
        assert L.tq_paged_attention_workspace(c, ctypes.byref(batch()), a["N"], a["Hq"], a["Hkv"],
                                              ctypes.byref(n)) == native.TQ_ERR_INVALID_ARG


def heads(**kw):
    f = dict(x=X, y=X, weight=None, x_stride_t=512, x_stride_h=64, y_stride_t=512, y_stride_h=64, heads=4)
    f.update(kw)
    return native.HeadsDesc(**f)


def norm(L, q=None, k=None, dtype=1, wd=1, d=64, N=4, eps=1e-6, pos=X, rc=None, rs=None, rn=0):
    return L.tq_qk_norm_rope(None if q is None else ctypes.byref(q), None if k is None else ctypes.byref(k),
                             dtype, wd, d, N, eps, pos, rc, rs, rn, None)


def test_norm_rope_refusals(L):
    assert norm(L) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(), d=96) == native.TQ_ERR_UNSUPPORTED
    assert norm(L, heads(), dtype=4) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(), wd=4) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(), N=-1) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(), eps=-1.0) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(), eps=float("nan")) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(x=None)) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(heads=-1)) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(heads=4097)) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(), heads(y=None)) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(x=X + 1)) == native.TQ_ERR_ALIGNMENT
    assert norm(L, heads(), rc=X) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(), rc=X, rs=X, rn=0) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(), rc=X, rs=X, rn=5, pos=None) == native.TQ_ERR_INVALID_ARG
    assert norm(L, heads(), N=0) == native.TQ_OK
    assert norm(L, heads(heads=0)) == native.TQ_OK


def test_binding_refusals():
    import torch
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError):
        native.PagedBatch(i(2, 3), i(2), i(2), 1, 32).desc()
    with pytest.raises(TypeError):
        native.PagedBatch(i(2, 3).long(), i(3), i(2), 1, 32).desc()
    with pytest.raises(ValueError):
        native.PagedBatch(i(3, 2).t(), i(3), i(2), 1, 32).desc()
    x = torch.zeros((2, 3, 64))
    with pytest.raises(ValueError):
        native.qk_norm_rope(None, None, None, None, 1e-6, None, None, None)
    with pytest.raises(ValueError):
        native.qk_norm_rope(x, None, None, None, 1e-6, None, x[:, :2], None)
    with pytest.raises(ValueError):
        native.qk_norm_rope(x, None, torch.ones(32), None, 1e-6, None, x, None)
    with pytest.raises(ValueError):
        native.qk_norm_rope(x, None, None, None, 1e-6, i(3), x, None)
    with pytest.raises(ValueError):
        native.qk_norm_rope(x.transpose(1, 2), None, None, None, 1e-6, None, x, None)
    with pytest.raises(TypeError):
        native.qk_norm_rope(x.half(), None, None, None, 1e-6, None, x.half(), None)


def test_row_limits_of_a_call(L, codec):
    """Row counts that no launch could cover are refused, not cut off."""
    c, n = codec[64], ctypes.c_size_t(0)
    many = dict(N=1 << 24, ca=cache(heads=256))
    assert quantize(L, c, **many) == native.TQ_ERR_INVALID_ARG
    assert dequantize(L, c, **many) == native.TQ_ERR_INVALID_ARG
    assert attention(L, c, Hq=256, **many) == native.TQ_ERR_INVALID_ARG
    assert attention(L, c, N=1 << 24, Hq=256, ca=cache(heads=1)) == native.TQ_ERR_INVALID_ARG
    assert quantize(L, c, ca=cache(heads=65536)) == native.TQ_ERR_INVALID_ARG
    for N, Hq in ((1 << 24, 256), ((1 << 24) + 1, 4), (8, 65536 * 2)):
        assert L.tq_paged_attention_workspace(c, ctypes.byref(batch()), N, Hq, 1,
                                              ctypes.byref(n)) == native.TQ_ERR_INVALID_ARG
    # more work than a call counts: refused before any device work
    long = batch(num_seqs=65535, max_pages=1 << 24, table_stride=1 << 24, max_new=1, max_seq_len=1 << 30)
    assert attention(L, c, N=65535, Hq=8, ca=cache(heads=8), b=long) == native.TQ_ERR_INVALID_ARG
    # a limit on new tokens far above the call's tokens counts as the call's
    for Hq in (8, 160):
        sizes = []
        for most in (8, (1 << 31) - 1):
            assert L.tq_paged_attention_workspace(c, ctypes.byref(batch(max_new=most)), 8, Hq, 1,
                                                  ctypes.byref(n)) == native.TQ_OK
            sizes.append(n.value)
        assert sizes[0] == sizes[1]


def test_binding_refuses_host_tensors():
    import torch
    if torch.cuda.is_available():
        pytest.skip("covered there with a device")
    x = torch.zeros((2, 3, 64))
    with pytest.raises(ValueError, match="current CUDA device"):
        native.qk_norm_rope(x, None, None, None, 1e-6, None, x, None)
