"""Paged cache on the GPU against 64-bit references: append, read-back and
attention over ragged batches, their edges, and a run of them together."""
import math

import numpy as np
import pytest
import torch

from oracle import codec as oc
from oracle.rotation import apply_rope
from rotated_codebook_kv_tq_b200 import native, synth
import paged_testlib as pt
import tq_testlib as tl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    tl.require_cuda()


def dev(x, dtype):
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def attend(ncodec, q, cache, batch, Hkv, rope=None, out_dtype=torch.bfloat16, fill=7.0, scale=None, ws=None):
    b = batch if isinstance(batch, native.PagedBatch) else batch.device()
    N, Hq, d = q.shape
    out = torch.full((N, Hq, d), fill, dtype=out_dtype, device="cuda")
    if ws is None:
        ws = torch.empty(max(16, native.paged_attention_workspace(ncodec, b, N, Hq, Hkv)),
                         dtype=torch.uint8, device="cuda")
    native.paged_attention(ncodec, q, cache, b, 1 / math.sqrt(d) if scale is None else scale, out, ws,
                           rope=rope)
    return out


def check_answers(out, ref, sigma, out_dtype=torch.bfloat16, fill=7.0):
    got = host(out)
    known = ~np.isnan(ref)
    assert np.all(got[~known] == fill), "rows of no sequence were touched"
    tol = pt.attention_tolerance(sigma, out_dtype)
    err = np.linalg.norm((got - ref)[known]) / max(np.linalg.norm(ref[known]), 1e-30)
    assert np.isfinite(got).all() and err <= tol, (err, tol)
    # no single answer row is lost among the others: its own share at the same rule
    for r in range(ref.shape[0]):
        for h in range(ref.shape[1]):
            if known[r, h, 0]:
                n = np.linalg.norm(ref[r, h])
                e = np.linalg.norm(got[r, h] - ref[r, h])
                assert e <= 4 * tol * max(n, 1e-30) if n > 0 else e == 0.0, (r, h, e, n)


# ------------------------------------------------------------------ append

APPEND = [
    # d, bits_k, qjl, bits_v, Hkv, page, seqs, dtype, rope, haar
    (128, 4, True, 4, 2, 64, [(1, 1), (70, 1), (64, 1)], "bf16", True, False),
    (128, 4, True, 4, 2, 32, [(200, 137), (33, 2), (5, 5), (40, 0)], "bf16", True, False),
    (64, 3, True, 3, 3, 32, [(100, 100), (31, 31), (95, 33)], "bf16", True, False),
    (64, 2, True, 2, 1, 128, [(129, 129)], "fp32", False, False),
    (128, 5, True, 1, 1, 64, [(65, 65), (1, 1)], "fp32", True, False),
    (128, 3, False, 3, 2, 64, [(90, 80)], "bf16", False, False),
    (64, 1, False, 4, 2, 32, [(64, 64)], "bf16", True, False),
    (128, 4, True, 4, 1, 64, [(70, 65)], "bf16", True, True),
    (64, 3, True, 2, 2, 32, [(40, 40), (1, 1)], "bf16", False, True),
    (128, 4, True, 4, 8, 64, [(1024, 1024), (700, 699)], "bf16", True, False),
    (64, 3, True, 3, 5, 32, [(900, 900), (801, 800)], "bf16", True, False),
    (128, 5, True, 1, 4, 64, [(700, 600), (500, 500)], "fp32", True, False),
    (128, 2, True, 2, 8, 32, [(513, 513), (70, 69)], "bf16", False, False),
    (128, 3, False, 3, 6, 128, [(1000, 900)], "fp32", False, False),
    (128, 4, False, 2, 6, 32, [(800, 790)], "bf16", True, False),
    (64, 2, True, 4, 3, 64, [(1500, 1400), (129, 128)], "fp32", True, False),
    (64, 1, False, 1, 6, 32, [(800, 799)], "bf16", True, False),
    (64, 5, True, 2, 6, 32, [(800, 799)], "bf16", False, False),
    (64, 4, False, 3, 7, 64, [(640, 600)], "fp32", True, False),
    (128, 4, True, 4, 8, 32, [(33, 33)] * 17, "bf16", True, False),
]


def encode_ref(planes, ocodec, batch, K, V, rope):
    """The planes after the append, by the oracle's row encoders."""
    P, Hkv = batch.page, K.shape[1]
    new = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in planes.items()}
    todo = [(r, batch.page_of(s, p), p) for r, s, p in batch.rows() if p >= 0]
    todo = [x for x in todo if x[1] is not None]
    rows = np.array([x[0] for x in todo])
    pages = np.array([x[1] for x in todo])
    pos = np.array([x[2] for x in todo])
    for h in range(Hkv):
        k = K[rows, h]
        if rope is not None:
            k = apply_rope(k, rope[0], rope[1], pos)
        ek = pt.encode_keys(k, ocodec)
        kc, ks = oc.pack_keys(ek, ocodec)
        new["kcode"][pages, h, pos % P] = kc
        new["kscale"][pages, h, pos % P] = ks
        ev = pt.encode_values(V[rows, h], ocodec)
        new["vnorm"][pages, h, pos % P] = ev["nu16"]
        for i in range(len(rows)):
            w = new["vcode"][pages[i], h, (pos[i] % P) // 32]
            bit = np.uint32(1 << int(pos[i] % 32))
            for p in range(ocodec.bits_v):
                on = ((ev["idx"][i] >> p) & 1).astype(bool)
                w[p] = np.where(on, w[p] | bit, w[p] & ~bit)
    return new


def make_kv(batch, Hkv, d, dtype, seed=3):
    g = np.random.default_rng(seed)
    x = g.standard_normal((batch.N, 2 * Hkv, d)) * np.exp(g.standard_normal((2 * Hkv, d)))
    t = dev(x, dtype)
    return t, host(t)


def same_planes(cache, ref):
    got = tl.download_cache(cache)
    for key in ("kcode", "vcode"):
        bad = np.argwhere(got[key] != ref[key])
        assert not len(bad), (key, len(bad), bad[:4].tolist())
    assert np.all(tl.fp16_close(got["kscale"], ref["kscale"]))
    assert np.all(tl.fp16_close(got["vnorm"], ref["vnorm"]))


@pytest.mark.parametrize("case", APPEND, ids=[f"d{c[0]}k{c[1]}{'q' if c[2] else ''}v{c[3]}p{c[5]}{c[7]}{'haar' if c[9] else ''}-{i}"
                                              for i, c in enumerate(APPEND)])
def test_append_codes_are_those_of_exact_arithmetic(case):
    d, bk, qjl, bv, Hkv, page, seqs, dtype, with_rope, haar = case
    ocodec, ncodec = pt.codecs(d, bk, qjl, bv, haar=haar)
    batch = pt.Batch(seqs, page, seed=d + bk, start=2, extra_rows=3)
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    cache = pt.upload(planes, ncodec)
    kv, kvh = make_kv(batch, Hkv, d, dtype)
    rope = synth.rope_table(batch.max_len, d, 1e4) if with_rope else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.paged_quantize_kv(ncodec, kv[:, :Hkv], kv[:, Hkv:], cache, batch.device(),
                             rope=tl.rope_device(rope), status=status)
    if haar:
        # the dense rotation is given in fp32: its 64-bit values are those
        ocodec.Pi = native.haar_rotation(synth.haar_gaussian(d, 11)).astype(np.float64)
    ref = encode_ref(planes, ocodec, batch, kvh[:, :Hkv], kvh[:, Hkv:], rope)
    same_planes(cache, ref)
    assert int(status.item()) == 0


def test_append_of_bad_rows_missing_pages_and_short_sequences():
    d, Hkv, page = 128, 2, 32
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    # the last sequence has more new tokens than tokens
    batch = pt.Batch([(50, 40), (40, 40), (3, 5)], page, seed=4)
    batch.table[1, 0] = batch.pool          # behind the pool
    batch.table[0, 1] = -5
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    cache = pt.upload(planes, ncodec)
    kv, kvh = make_kv(batch, Hkv, d, "fp32")
    kv[3, 0, 5] = float("nan")
    kv[4, 3, 0] = float("inf")
    kv[6, 1] *= 1e5                          # norm beyond fp16
    kv[7] = 0.0
    kvh = host(kv)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.paged_quantize_kv(ncodec, kv[:, :Hkv], kv[:, Hkv:], cache, batch.device(), status=status)
    with np.errstate(invalid="ignore"):
        ref = encode_ref(planes, ocodec, batch, kvh[:, :Hkv], kvh[:, Hkv:], None)
    same_planes(cache, ref)
    lost = sum(1 for _, s, p in batch.rows() if p >= 0 and batch.page_of(s, p) is None)
    assert int(status.item()) == 3 + 2 * Hkv * lost


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp32")])
def test_append_of_bad_rows_in_a_large_call(d, dtype):
    """Rows that are zero, tiny, huge, not finite or on a border, missing pages, and
    a sequence with more new tokens than tokens, in a call of full tiles."""
    Hkv, page = 5, 64
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    batch = pt.Batch([(700, 600), (300, 320), (90, 90)], page, seed=4, start=1, extra_rows=1)
    batch.table[0, 3] = batch.pool
    batch.table[2, 0] = -1
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    cache = pt.upload(planes, ncodec)
    kv, _ = make_kv(batch, Hkv, d, dtype)
    r0 = int(batch.q_start[1])
    kv[r0 + 30, 0, 5] = float("nan")
    kv[r0 + 31, Hkv + 3, 0] = float("inf")
    kv[r0 + 32, 1] *= 1e6                     # norm beyond fp16
    kv[r0 + 33, :] = 0.0
    kv[r0 + 34, :] = -0.0
    kv[r0 + 35, :] *= 1e-14
    kv[r0 + 36, :] *= 1e-30
    kv[r0 + 37, :] = 1.0                      # one coordinate carries the row
    kv[r0 + 38, :] = 0.0
    kv[r0 + 38, :, 3] = -2.0                  # all coordinates equal in size
    for i, e in enumerate((65503.0, 65504.0, 65519.0, 65521.0, 66000.0)):
        kv[r0 + 40 + i, :] = 0.0
        kv[r0 + 40 + i, :, 1] = e             # norms around fp16's end
    kvh = host(kv)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.paged_quantize_kv(ncodec, kv[:, :Hkv], kv[:, Hkv:], cache, batch.device(), status=status)
    with np.errstate(invalid="ignore", over="ignore"):
        ref = encode_ref(planes, ocodec, batch, kvh[:, :Hkv], kvh[:, Hkv:], None)
    same_planes(cache, ref)
    norm = np.sqrt((kvh * kvh).sum(-1))
    with np.errstate(over="ignore", invalid="ignore"):
        bad = ~np.isfinite(norm.astype(np.float16))
    count = 0
    for r, s, p in batch.rows():
        if p >= 0:
            count += 2 * Hkv if batch.page_of(s, p) is None else int(bad[r].sum())
    assert int(status.item()) == count


def test_append_does_not_depend_on_the_chunks():
    """A prompt appended whole, in odd chunks and token by token: the same bytes."""
    d, Hkv, page, T = 128, 8, 64, 1500
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    rope = tl.rope_device(synth.rope_table(T, d, 5e5))
    whole = pt.Batch([(T, T)], page, seed=1)
    kv, _ = make_kv(whole, Hkv, d, "bf16")
    caches = []
    for chunks in ([T], [700, 33, 1, 500, 266], [T - 20] + [1] * 20):
        cache = native.alloc_cache(ncodec, whole.pool, Hkv, page)
        at = 0
        for n in chunks:
            b = native.PagedBatch(torch.from_numpy(whole.table).cuda(),
                                  torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                  torch.tensor([at + n], dtype=torch.int32, device="cuda"), n, at + n)
            part = kv[at:at + n]
            native.paged_quantize_kv(ncodec, part[:, :Hkv], part[:, Hkv:], cache, b, rope=rope)
            at += n
        caches.append(tl.download_cache(cache))
    for other in caches[1:]:
        for key in ("kcode", "vcode"):
            assert np.array_equal(caches[0][key], other[key]), key
        for key in ("kscale", "vnorm"):
            assert np.all(tl.fp16_close(caches[0][key], other[key])), key


# ------------------------------------------------------------------ read-back

READ = [
    # d, bits_k, qjl, bits_v, page, dtype, haar, tokens of the long sequence (0: none)
    (128, 4, True, 4, 64, torch.bfloat16, False, 0), (128, 5, True, 1, 32, torch.float32, False, 0),
    (64, 3, True, 3, 32, torch.float32, False, 0), (64, 4, False, 2, 128, torch.bfloat16, False, 0),
    (128, 2, True, 2, 64, torch.float32, True, 0), (64, 2, True, 4, 32, torch.float32, False, 0),
    (128, 4, True, 4, 64, torch.bfloat16, False, 1500), (128, 5, True, 2, 32, torch.bfloat16, False, 1400),
    (64, 3, True, 3, 128, torch.bfloat16, False, 1501), (64, 4, False, 4, 32, torch.bfloat16, False, 1400),
    (128, 3, False, 1, 64, torch.bfloat16, False, 1400), (64, 5, True, 4, 64, torch.bfloat16, False, 1601),
    (128, 4, True, 4, 64, torch.bfloat16, True, 1400), (128, 4, True, 4, 64, torch.float32, False, 1400)]


@pytest.mark.parametrize("case", READ, ids=[f"d{c[0]}k{c[1]}v{c[3]}p{c[4]}-{i}" for i, c in enumerate(READ)])
def test_read_back(case):
    d, bk, qjl, bv, page, dtype, haar, long = case
    Hkv = 3
    ocodec, ncodec = pt.codecs(d, bk, qjl, bv, haar=haar)
    seqs = [(page + 1, page + 1), (1, 1), (200, 77), (10, 12), (50, 0)]
    batch = pt.Batch(seqs + ([(long + 70, long)] if long else []), page, seed=9, start=1, extra_rows=2)
    batch.table[2, -(-200 // page) - 1] = -1
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    # rows behind the last token of a sequence may hold anything
    planes["kscale"][batch.table[0, 1], :, 1:] = np.nan
    planes["vnorm"][batch.table[0, 1], :, 1:] = np.nan
    cache = pt.upload(planes, ncodec)
    outs = [torch.full((batch.N, Hkv, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    native.paged_dequantize(ncodec, cache, batch.device(), outs[0], outs[1])
    ref = np.full((2, batch.N, Hkv, d), 7.0)
    for s, (n, m) in enumerate(zip(batch.lens, batch.news)):
        r0 = int(batch.q_start[s])
        for h in range(Hkv):
            k, v, there = pt.sequence_rows(planes, ocodec, batch, s, h, n)
            for i in range(m):
                p = n - m + i
                ref[0, r0 + i, h] = k[p] if p >= 0 else 0.0
                ref[1, r0 + i, h] = v[p] if p >= 0 else 0.0
    # fp32 answers: sums of at most 2 d terms (sketch, rotation), each add off
    # by at most an ulp of the running sum, bounded by the sum of the terms' sizes
    # over sqrt(d): |c| + coef rho sum_i |(S Pi)_ij| <= 2 sqrt(d) in all.
    # bf16 answers: their rounding, 2^-8 of the value at most, and before it the
    # fp16 operands, 2^-11 of each term: |c| <= 2 for uniform codes (Cauchy-Schwarz
    # over d terms of size |c| / sqrt(d)), and the sketch's terms, coef rho and
    # S H D both rounded: 2 * 1.2533 rho * 1.1 with rho <= 0.4 and a tenth for |S v| / sqrt(d).
    for got, want, top in ((host(outs[0]), ref[0], np.nanmax(planes["kscale"][..., 0])),
                           (host(outs[1]), ref[1], np.nanmax(planes["vnorm"]))):
        top = float(top)
        tol = top * 2.0 * math.sqrt(d) * (2 * d + 16) * 2.0 ** -23 * 0.25
        if dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(want) + top * 2.0 ** -11 * (2.0 + 2.8 * 0.4)
        assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want))
        rel = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert rel <= (1e-5 if dtype == torch.float32 else 4 * math.sqrt(2.0 ** -16 / 3 + 3 * 2.0 ** -22)), rel
    only = torch.empty_like(outs[1])
    native.paged_dequantize(ncodec, cache, batch.device(), None, only)
    used = slice(int(batch.q_start[0]), int(batch.q_start[-1]))
    assert torch.equal(only[used], outs[1][used])
    native.paged_dequantize(ncodec, cache, batch.device(), only, None)
    assert torch.equal(only[used], outs[0][used])


# ------------------------------------------------------------------ attention

ATTN = [
    # d, bits_k, qjl, bits_v, Hq, Hkv, page, seqs, rope, q dtype, out dtype
    (128, 4, True, 4, 8, 2, 64, [(1, 1), (64, 1), (65, 1), (1000, 1)], True, "bf16", "bf16"),
    (128, 4, True, 4, 4, 4, 32, [(31, 1), (33, 1)], True, "bf16", "bf16"),
    (128, 2, True, 2, 16, 2, 32, [(500, 6), (37, 3), (6, 6), (100, 0)], False, "bf16", "bf16"),
    (128, 5, True, 1, 14, 2, 64, [(130, 9), (700, 16)], True, "fp32", "fp32"),
    (128, 3, False, 3, 8, 1, 128, [(300, 2), (129, 129)], True, "bf16", "fp32"),
    (64, 3, True, 3, 4, 4, 32, [(257, 257), (100, 64)], True, "bf16", "bf16"),
    (64, 2, True, 4, 8, 2, 64, [(2000, 1), (77, 1)], True, "bf16", "bf16"),
    (64, 4, False, 2, 6, 2, 32, [(90, 33), (400, 31)], False, "bf16", "bf16"),
    (128, 4, True, 4, 8, 2, 64, [(600, 300), (1, 1), (130, 129)], True, "bf16", "bf16"),
    (128, 4, True, 4, 32, 1, 64, [(333, 1), (90, 5)], True, "bf16", "bf16"),
    (64, 5, True, 4, 20, 20, 32, [(130, 130)], True, "bf16", "bf16"),
    (128, 4, True, 3, 8, 2, 64, [(513, 100), (257, 257), (128, 128), (129, 1)], True, "bf16", "fp32"),
]


@pytest.mark.parametrize("case", ATTN, ids=[f"d{c[0]}k{c[1]}v{c[3]}h{c[4]}-{c[5]}p{c[6]}-{i}"
                                            for i, c in enumerate(ATTN)])
def test_attention(case):
    d, bk, qjl, bv, Hq, Hkv, page, seqs, with_rope, qd, od = case
    ocodec, ncodec = pt.codecs(d, bk, qjl, bv)
    batch = pt.Batch(seqs, page, seed=Hq, start=1, extra_rows=2)
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    cache = pt.upload(planes, ncodec)
    g = np.random.default_rng(5)
    # rows wider than the heads: strides of a packed projection
    q = dev(g.standard_normal((batch.N, Hq + 3, d)), qd)[:, 2:2 + Hq]
    rope = synth.rope_table(batch.max_len, d, 1e4) if with_rope else None
    odt = torch.bfloat16 if od == "bf16" else torch.float32
    out = attend(ncodec, q, cache, batch, Hkv, tl.rope_device(rope), odt)
    ref, sigma = pt.attention_ref(planes, ocodec, batch, host(q), 1 / math.sqrt(d), rope)
    check_answers(out, ref, sigma, odt)


def test_attention_dense_rotation():
    d, Hq, Hkv, page = 128, 8, 2, 64
    ocodec, ncodec = pt.codecs(d, 4, True, 4, haar=True)
    for seqs in ([(300, 1), (64, 4)], [(400, 200)]):
        batch = pt.Batch(seqs, page)
        planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
        q = dev(np.random.default_rng(5).standard_normal((batch.N, Hq, d)), "bf16")
        out = attend(ncodec, q, pt.upload(planes, ncodec), batch, Hkv)
        ref, sigma = pt.attention_ref(planes, ocodec, batch, host(q), 1 / math.sqrt(d), None)
        check_answers(out, ref, sigma)


@pytest.mark.parametrize("new", [1, 5, 150])
def test_attention_missing_pages_and_empty_rows(new):
    """Pages outside the pool are not seen; a query with nothing to see, or
    without a position, gets zeros."""
    d, Hq, Hkv, page = 128, 8, 2, 32
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    batch = pt.Batch([(200, new), (32, min(new, 32)), (2, new), (160, new)], page, max_new=new)
    batch.table[0, 2] = -1
    batch.table[0, 6] = 1 << 30
    batch.table[1, 0] = batch.pool
    batch.table[3, :] = -7
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    # what lies in pages that no one may see
    for key in ("kscale", "vnorm"):
        used = np.zeros(batch.pool, bool)
        for s in range(4):
            for p in batch.table[s]:
                if 0 <= p < batch.pool:
                    used[p] = True
        planes[key][~used] = np.nan
    q = dev(np.random.default_rng(6).standard_normal((batch.N, Hq, d)), "bf16")
    out = attend(ncodec, q, pt.upload(planes, ncodec), batch, Hkv)
    ref, sigma = pt.attention_ref(planes, ocodec, batch, host(q), 1 / math.sqrt(d), None)
    check_answers(out, ref, sigma)


@pytest.mark.parametrize("new", [1, 4, 140])
def test_attention_rows_behind_the_sequence_do_not_count(new):
    """NaN and infinite scales in rows behind a sequence's last token, inside its last page."""
    d, Hq, Hkv, page = 64, 4, 2, 128
    ocodec, ncodec = pt.codecs(d, 3, True, 3)
    batch = pt.Batch([(max(new, 140) + 1, new), (5, min(new, 5))], page)
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    for s in range(2):
        n = batch.lens[s]
        p = batch.table[s, (n - 1) // page]
        planes["kscale"][p, :, (n - 1) % page + 1:] = np.inf
        planes["vnorm"][p, :, (n - 1) % page + 1:] = np.nan
    q = dev(np.random.default_rng(6).standard_normal((batch.N, Hq, d)), "bf16")
    out = attend(ncodec, q, pt.upload(planes, ncodec), batch, Hkv)
    ref, sigma = pt.attention_ref(planes, ocodec, batch, host(q), 1 / math.sqrt(d), None)
    check_answers(out, ref, sigma)


@pytest.mark.parametrize("new", [1, 200])
def test_attention_shared_prefix_and_large_logits(new):
    """Two sequences over the same pages; logits of a hundred and more."""
    d, Hq, Hkv, page = 128, 4, 1, 64
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    batch = pt.Batch([(500, new), (500, new)], page)
    batch.table[1, :4] = batch.table[0, :4]
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page, nu=60.0)
    q = dev(np.random.default_rng(8).standard_normal((batch.N, Hq, d)), "bf16")
    out = attend(ncodec, q, pt.upload(planes, ncodec), batch, Hkv)
    ref, sigma = pt.attention_ref(planes, ocodec, batch, host(q), 1 / math.sqrt(d), None)
    check_answers(out, ref, sigma)


def test_attention_zero_query_is_the_mean():
    d, Hq, Hkv, page = 64, 4, 2, 32
    ocodec, ncodec = pt.codecs(d, 3, True, 3)
    for new in (1, 100):
        batch = pt.Batch([(333, new)], page)
        planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
        q = torch.zeros((batch.N, Hq, d), dtype=torch.bfloat16, device="cuda")
        out = attend(ncodec, q, pt.upload(planes, ncodec), batch, Hkv)
        ref, sigma = pt.attention_ref(planes, ocodec, batch, host(q), 1 / math.sqrt(d), None)
        check_answers(out, ref, sigma)


def test_offsets_beyond_32_bits():
    """Pages at the end of a pool whose planes are larger than 2^31 bytes."""
    d, Hq, Hkv, page, pool = 128, 8, 8, 64, 70000
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    batch = pt.Batch([(150, 70), (100, 1)], page)
    cache = native.alloc_cache(ncodec, pool, Hkv, page)
    assert cache.kcode.numel() > 1 << 31
    shift = pool - batch.pool
    batch.table[batch.table >= 0] += shift
    b = batch.device()
    kv, kvh = make_kv(batch, Hkv, d, "bf16")
    native.paged_quantize_kv(ncodec, kv[:, :Hkv], kv[:, Hkv:], cache, b)
    small = native.Cache(cache.kcode[shift:], cache.kscale[shift:], cache.vcode[shift:], cache.vnorm[shift:],
                         batch.pool, Hkv, page)
    planes = tl.download_cache(small)
    batch.table[batch.table >= 0] -= shift
    zero = {k: (np.zeros_like(v) if isinstance(v, np.ndarray) else v) for k, v in planes.items()}
    same_planes(small, encode_ref(zero, ocodec, batch, kvh[:, :Hkv], kvh[:, Hkv:], None))
    q = dev(np.random.default_rng(8).standard_normal((batch.N, Hq, d)), "bf16")
    out = attend(ncodec, q, cache, b, Hkv)
    ref, sigma = pt.attention_ref(planes, ocodec, batch, host(q), 1 / math.sqrt(d), None)
    check_answers(out, ref, sigma)
    back = [torch.empty((batch.N, Hkv, d), device="cuda") for _ in range(2)]
    native.paged_dequantize(ncodec, cache, b, back[0], back[1])
    near = [torch.empty((batch.N, Hkv, d), device="cuda") for _ in range(2)]
    native.paged_dequantize(ncodec, small, batch.device(), near[0], near[1])
    assert torch.equal(back[0], near[0]) and torch.equal(back[1], near[1])


@pytest.mark.parametrize("new,dtype", [(3, "bf16"), (300, "bf16"), (300, "fp32")])
def test_rows_off_16_byte_boundaries(new, dtype):
    """Tensors whose rows start on odd elements: the same answers and codes."""
    d, Hq, Hkv, page = 128, 8, 4, 64
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    batch = pt.Batch([(700, new), (400, new)] * (1 if new < 100 else 2), page)
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    b, rope = batch.device(), tl.rope_device(synth.rope_table(batch.max_len, d, 1e4))
    g = np.random.default_rng(3)
    whole = dev(g.standard_normal((batch.N, (Hq + 2 * Hkv) * d + 3)), dtype)
    w = whole.shape[1]
    odd = lambda at, H: whole.as_strided((batch.N, H, d), (w, d, 1), 1 + at * d)
    q, k, v = odd(0, Hq), odd(Hq, Hkv), odd(Hq + Hkv, Hkv)
    out = []
    for f in (lambda t: t, lambda t: t.contiguous()):
        cache = pt.upload(planes, ncodec)
        native.paged_quantize_kv(ncodec, f(k), f(v), cache, b, rope=rope)
        out.append((tl.download_cache(cache), attend(ncodec, f(q), pt.upload(planes, ncodec), b, Hkv, rope=rope)))
    for key in ("kcode", "vcode"):
        assert np.array_equal(out[0][0][key], out[1][0][key]), key
    for key in ("kscale", "vnorm"):
        assert np.all(tl.fp16_close(out[0][0][key], out[1][0][key])), key
    assert torch.equal(out[0][1], out[1][1])


# ------------------------------------------------------------------ use

def test_empty_batches_touch_nothing():
    ocodec, ncodec = pt.codecs(64, 3, True, 3)
    cache = native.alloc_cache(ncodec, 2, 2, 32)
    before = tl.download_cache(cache)
    for seqs in ([], [(40, 0)], [(0, 0)], [(0, 3)]):
        batch = pt.Batch(seqs, 32, extra_rows=2)
        b = batch.device()
        kv = torch.ones((batch.N, 4, 64), dtype=torch.bfloat16, device="cuda")
        native.paged_quantize_kv(ncodec, kv[:, :2], kv[:, 2:], cache, b)
        out = attend(ncodec, kv, cache, b, 2)
        k = torch.full((batch.N, 2, 64), 5.0, device="cuda")
        native.paged_dequantize(ncodec, cache, b, k, None)
        n = sum(batch.news)
        assert (out[:n] == 0).all() and (out[n:] == 7).all()
        assert (k[:n] == 0).all() and (k[n:] == 5).all()
    after = tl.download_cache(cache)
    for key in ("kcode", "kscale", "vcode", "vnorm"):
        assert np.array_equal(before[key], after[key])


@pytest.mark.parametrize("new", [1, 120])
def test_captured_calls_follow_their_inputs(new):
    """Append and attention in a CUDA graph: replay after the starts, lengths,
    pages and tensors have changed, on another stream than the capture's."""
    d, Hq, Hkv, page = 128, 8, 2, 64
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    batch = pt.Batch([(400, new), (333, new)], page, seed=2)
    planes = pt.random_pages(ocodec, batch.pool, Hkv, page)
    cache = pt.upload(planes, ncodec)
    b = batch.device()
    rope = synth.rope_table(batch.max_len, d, 1e4)
    rd = tl.rope_device(rope)
    kv, kvh = make_kv(batch, Hkv, d, "bf16")
    q = dev(np.random.default_rng(8).standard_normal((batch.N, Hq, d)), "bf16")
    out = torch.zeros((batch.N, Hq, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(native.paged_attention_workspace(ncodec, b, batch.N, Hq, Hkv) + 16, dtype=torch.uint8,
                     device="cuda")

    def step():
        native.paged_quantize_kv(ncodec, kv[:, :Hkv], kv[:, Hkv:], cache, b, rope=rd)
        native.paged_attention(ncodec, q, cache, b, 1 / math.sqrt(d), out, ws, rope=rd)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # another step: shorter sequences, pages swapped, other data, a used workspace
    batch.lens = [300, 201]
    batch.table[:, :2] = batch.table[::-1, :2].copy()
    b.seq_lens.copy_(torch.tensor(batch.lens, dtype=torch.int32))
    b.page_table.copy_(torch.from_numpy(batch.table))
    kv.mul_(0.5)
    q.mul_(-1.0)
    ws.fill_(255)
    cache2 = pt.upload(planes, ncodec)
    for name in ("kcode", "kscale", "vcode", "vnorm"):
        getattr(cache, name).copy_(getattr(cache2, name))
    graph.replay()
    torch.cuda.synchronize()
    now = encode_ref(planes, ocodec, batch, host(kv)[:, :Hkv], host(kv)[:, Hkv:], rope)
    same_planes(cache, now)
    ref, sigma = pt.attention_ref(now, ocodec, batch, host(q), 1 / math.sqrt(d), rope)
    check_answers(out, ref, sigma)


def test_two_streams_at_once_give_the_same_answers():
    d, Hq, Hkv, page = 128, 8, 2, 64
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    jobs = []
    for i, new in enumerate((1, 130)):
        batch = pt.Batch([(900, new), (777, new)], page, seed=i)
        planes = pt.random_pages(ocodec, batch.pool, Hkv, page, seed=i)
        q = dev(np.random.default_rng(i).standard_normal((batch.N, Hq, d)), "bf16")
        cache, b = pt.upload(planes, ncodec), batch.device()
        jobs.append((q, cache, b, attend(ncodec, q, cache, b, Hkv)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(10):
        for i, (q, cache, b, _) in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i].append(attend(ncodec, q, cache, b, Hkv))
    torch.cuda.synchronize()
    for i, job in enumerate(jobs):
        for o in got[i]:
            assert torch.equal(o, job[3])


def test_norms_append_and_attention_as_a_server_runs_them():
    """Two sequences: their prompts in two chunks, then decode steps, head norms
    and rotation first; every answer against 64-bit attention over what the
    cache holds, and the cache against the 64-bit codes of the rotated keys."""
    d, Hq, Hkv, page, eps = 128, 8, 2, 32, 1e-6
    ocodec, ncodec = pt.codecs(d, 4, True, 4)
    g = np.random.default_rng(12)
    limit = 160
    rope = synth.rope_table(limit, d, 1e4)
    rd = tl.rope_device(rope)
    wq, wk = (dev(1 + 0.2 * g.standard_normal(d), "bf16") for _ in range(2))
    steps = [[60, 33], [41, 50], [1, 1], [1, 1], [1, 0], [3, 1]]
    total = np.sum(steps, axis=0)
    full = pt.Batch([(int(n), 0) for n in total], page, seed=3)
    planes = pt.random_pages(ocodec, full.pool, Hkv, page)
    cache = pt.upload(planes, ncodec)
    have = np.zeros(2, int)
    for news in steps:
        have = have + news
        batch = pt.Batch([(int(n), int(m)) for n, m in zip(have, news)], page)
        batch.table, batch.pool, batch.max_pages = full.table, full.pool, full.max_pages
        b = batch.device()
        pos = np.concatenate([np.arange(n - m, n) for n, m in zip(have, news)]).astype(np.int32)
        x = dev(2 * g.standard_normal((batch.N, Hq + 2 * Hkv, d)), "bf16")
        q, k = torch.empty_like(x[:, :Hq]), torch.empty_like(x[:, Hq:Hq + Hkv])
        native.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], wq, wk, eps, torch.from_numpy(pos).cuda(), q, k,
                            rope=rd)
        v = x[:, Hq + Hkv:].contiguous()
        native.paged_quantize_kv(ncodec, k.contiguous(), v, cache, b)
        out = attend(ncodec, q, cache, b, Hkv)
        xh = host(x)
        for got, part, w in ((q, xh[:, :Hq], wq), (k, xh[:, Hq:Hq + Hkv], wk)):
            y = part / np.sqrt(np.mean(part * part, -1, keepdims=True) + eps) * host(w)
            want = apply_rope(y.transpose(1, 0, 2), rope[0], rope[1], pos).transpose(1, 0, 2)
            assert np.all(np.abs(host(got) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5)
        planes = encode_ref(planes, ocodec, batch, host(k), host(v), None)
        same_planes(cache, planes)
        planes = tl.download_cache(cache)     # norms may differ by an fp16 ulp
        ref, sigma = pt.attention_ref(planes, ocodec, batch, host(q), 1 / math.sqrt(d), None)
        check_answers(out, ref, sigma)
