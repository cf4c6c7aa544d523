"""Paged-cache calls at their limits: waits that give up, wide head groups, limits
larger than the call, tensors that are not on the current device."""
import math

import numpy as np
import pytest
import torch

from rotated_codebook_kv_tq_b200 import native
import paged_testlib as pt
import tq_testlib as tl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    tl.require_cuda()


def bf16(g, *shape):
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).cuda().to(torch.bfloat16)


def attend(ncodec, q, cache, b, Hkv, ws_fill=None):
    N, Hq, d = q.shape
    out = torch.full((N, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, native.paged_attention_workspace(ncodec, b, N, Hq, Hkv)), dtype=torch.uint8,
                     device="cuda")
    if ws_fill is not None:
        ws.fill_(ws_fill)
    native.paged_attention(ncodec, q, cache, b, 1 / math.sqrt(d), out, ws)
    return out


@pytest.mark.parametrize("d,new", [(128, 1), (128, 5), (128, 300), (64, 300)])
def test_attention_wait_give_up_is_answered_with_nan(monkeypatch, d, new):
    """TQ_WAIT_LIMIT=0 makes every bounded wait run out at once: the kernels let
    their own copies and products land, answer NaN, and the next call is whole."""
    Hq, Hkv, page = 8, 2, 64
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    batch = pt.Batch([(700, new), (333, new)], page)
    cache, b = pt.upload(pt.random_pages(ocodec, batch.pool, Hkv, page), ncodec), batch.device()
    q = bf16(np.random.default_rng(1), batch.N, Hq, d)
    good = attend(ncodec, q, cache, b, Hkv)
    assert torch.isfinite(good).all()
    monkeypatch.setenv("TQ_WAIT_LIMIT", "0")
    bad = attend(ncodec, q, cache, b, Hkv)
    torch.cuda.synchronize()
    assert torch.isnan(bad).all()
    monkeypatch.delenv("TQ_WAIT_LIMIT")
    assert torch.equal(attend(ncodec, q, cache, b, Hkv), good)


def test_append_and_read_back_wait_give_up_is_reported(monkeypatch):
    d, Hkv, page, T = 128, 8, 64, 1500
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    batch = pt.Batch([(T, T)], page)
    b = batch.device()
    kv = bf16(np.random.default_rng(2), T, 2 * Hkv, d)
    cache = native.alloc_cache(ncodec, batch.pool, Hkv, page)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(4)]

    def call(k, v):
        status.zero_()
        native.paged_quantize_kv(ncodec, kv[:, :Hkv], kv[:, Hkv:], cache, b, status=status)
        native.paged_dequantize(ncodec, cache, b, k, v)
        torch.cuda.synchronize()
        return int(status.item())

    assert call(outs[0], outs[1]) == 0
    monkeypatch.setenv("TQ_WAIT_LIMIT", "0")
    assert call(outs[2], outs[3]) < 0          # bit 31
    # every group issues its first tile, waits and gives up: all its rows are NaN
    assert torch.isnan(outs[2]).all() and torch.isnan(outs[3]).all()
    monkeypatch.delenv("TQ_WAIT_LIMIT")
    assert call(outs[2], outs[3]) == 0
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])


@pytest.mark.parametrize("G,Hkv,new", [(160, 1, 40), (130, 2, 1), (128, 1, 3), (71, 2, 2)])
def test_attention_of_wide_head_groups(G, Hkv, new):
    d, page = 64, 32
    ocodec, ncodec = pt.codecs(d, 3, True, 3)
    batch = pt.Batch([(150, new), (new, new)], page, extra_rows=1)
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    q = bf16(np.random.default_rng(3), batch.N, G * Hkv, d)
    out = attend(ncodec, q, pt.upload(planes, ncodec), batch.device(), Hkv).float().cpu().numpy()
    ref, sigma = pt.attention_ref(planes, ocodec, batch, q.float().cpu().numpy().astype(np.float64),
                                  1 / math.sqrt(d), None)
    known = ~np.isnan(ref)
    assert np.all(out[~known] == 7.0)
    err = np.linalg.norm((out - ref)[known]) / np.linalg.norm(ref[known])
    assert err <= pt.attention_tolerance(sigma, torch.bfloat16), err


RAGGED = [
    # d, Hq, Hkv, sequences, longest, most new tokens
    (64, 4, 2, 40, 300, 1), (128, 8, 1, 40, 700, 2), (64, 4, 4, 300, 150, 3), (128, 4, 2, 1100, 40, 1),
    (128, 8, 2, 3, 9000, 6), (64, 6, 2, 5, 5000, 4), (128, 12, 1, 33, 400, 9)]


@pytest.mark.parametrize("case", RAGGED, ids=[f"d{c[0]}h{c[1]}-{c[2]}s{c[3]}n{c[5]}" for c in RAGGED])
def test_ragged_batches_of_few_rows(case):
    """Sequences of very unequal lengths, some without new tokens, some without
    any token: work that is cut inside sequences, and blocks with several."""
    d, Hq, Hkv, S, longest, most = case
    page = 32
    ocodec, ncodec = pt.codecs(d, 3, True, 4)
    g = np.random.default_rng(S)
    lens = np.maximum(g.integers(-3, longest, S), 0)
    lens[:3] = longest, 1, 0
    news = np.minimum(g.integers(0, most + 1, S), lens)
    news[0] = most
    news[2] = 1                                    # a token without a position
    batch = pt.Batch([(int(a), int(b)) for a, b in zip(lens, news)], page, seed=S, start=2, extra_rows=1)
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    cache, b = pt.upload(planes, ncodec), batch.device()
    q = bf16(g, batch.N, Hq, d)
    got = attend(ncodec, q, cache, b, Hkv, ws_fill=255)
    out = got.float().cpu().numpy()
    ref, sigma = pt.attention_ref(planes, ocodec, batch, q.float().cpu().numpy().astype(np.float64),
                                  1 / math.sqrt(d), None)
    known = ~np.isnan(ref)
    assert np.all(out[~known] == 7.0)
    tol = pt.attention_tolerance(sigma, torch.bfloat16)
    for r in range(batch.N):
        for h in range(Hq):
            if known[r, h, 0]:
                n, e = np.linalg.norm(ref[r, h]), np.linalg.norm(out[r, h] - ref[r, h])
                assert e <= 4 * tol * n, (r, h, e, n)
    assert np.linalg.norm((out - ref)[known]) <= tol * np.linalg.norm(ref[known])
    # the same again, bit by bit
    assert torch.equal(attend(ncodec, q, cache, b, Hkv, ws_fill=0), got)


@pytest.mark.parametrize("new", [1, 3, 90])
def test_limits_larger_than_the_call_do_not_change_it(new):
    """max_new and max_seq_len are limits: generous ones give the same rows (the
    splits of the keys, and so the order of sums, may differ), whatever the
    workspace held."""
    d, Hq, Hkv, page = 128, 8, 2, 64
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    batch = pt.Batch([(500, new), (77, min(new, 77)), (1, 1)], page)
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    cache, b = pt.upload(planes, ncodec), batch.device()
    q = bf16(np.random.default_rng(4), batch.N, Hq, d)
    out = attend(ncodec, q, cache, b, Hkv)
    wide = torch.full((3, 400), -1, dtype=torch.int32, device="cuda")
    wide[:, :b.page_table.shape[1]] = b.page_table
    big = native.PagedBatch(wide, b.q_start, b.seq_lens, (1 << 31) - 1, 400 * page)
    other = attend(ncodec, q, cache, big, Hkv, ws_fill=255)
    ref, sigma = pt.attention_ref(planes, ocodec, batch, q.float().cpu().numpy().astype(np.float64),
                                  1 / math.sqrt(d), None)
    for o in (out, other):
        err = np.linalg.norm(o.float().cpu().numpy() - ref) / np.linalg.norm(ref)
        assert err <= pt.attention_tolerance(sigma, torch.bfloat16), err
    back = [torch.empty((batch.N, Hkv, d), device="cuda") for _ in range(2)]
    native.paged_dequantize(ncodec, cache, b, back[0], None)
    native.paged_dequantize(ncodec, cache, big, back[1], None)
    assert torch.equal(back[0], back[1])


def test_tensors_elsewhere_are_refused():
    d, Hkv, page = 64, 2, 32
    ocodec, ncodec = pt.codecs(d, 3, True, 3)
    batch = pt.Batch([(40, 4)], page)
    cache, b = native.alloc_cache(ncodec, batch.pool, Hkv, page), batch.device()
    host = native.PagedBatch(b.page_table, b.q_start.cpu(), b.seq_lens.cpu(), 4, 40)
    x = torch.zeros((4, 4, d), dtype=torch.bfloat16, device="cuda")
    k = x[:, :Hkv].contiguous()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    rope = (torch.zeros(64, d // 2), torch.zeros(64, d // 2))
    for call in (lambda: native.paged_quantize_kv(ncodec, k.cpu(), k.cpu(), cache, b),
                 lambda: native.paged_quantize_kv(ncodec, k, k, cache, b, rope=rope),
                 lambda: native.paged_quantize_kv(ncodec, k, k, cache, host),
                 lambda: native.paged_dequantize(ncodec, cache, b, k, k.cpu()),
                 lambda: native.paged_dequantize(ncodec, cache, host, k, None),
                 lambda: native.paged_attention(ncodec, x, cache, b, 0.1, torch.empty_like(x), ws.cpu()),
                 lambda: native.paged_attention(ncodec, x, cache, b, 0.1, x.cpu(), ws),
                 lambda: native.qk_norm_rope(x, None, None, None, 1e-6, pos.cpu(), x, None),
                 lambda: native.qk_norm_rope(x, None, torch.ones(d), None, 1e-6, pos, x, None)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
