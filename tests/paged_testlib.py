"""Helpers of the paged-cache tests: ragged batches, random coded pages, and
64-bit references of the append, the read-back and the attention, built from
the oracle's row functions."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import codec as oc
from oracle.rotation import apply_rope
from rotated_codebook_kv_tq_b200 import native, synth
import tq_testlib as tl


def codecs(d, bits_k, qjl, bits_v, seed=11, haar=False):
    w = synth.Workload("paged", seed, 1, 1, 1, d, 32, bits_k, qjl, bits_v, "bf16", None, None, 0, 1.0, 0)
    return tl.codecs(w, haar=haar)


class Batch:
    """A ragged batch on host and device.  seqs: (tokens, new tokens) each.
    pool pages are handed out in a random order; page tables of unequal length
    are padded with -1.  start: packed rows before the first sequence."""

    def __init__(self, seqs, page, seed=0, spare=3, extra_rows=0, start=0, max_new=None, max_len=None):
        g = np.random.default_rng(seed)
        self.page, self.lens, self.news = page, [a for a, _ in seqs], [b for _, b in seqs]
        per = [-(-n // page) for n in self.lens]
        self.pool = sum(per) + spare
        order = g.permutation(self.pool)
        self.max_pages = max(per + [1])
        self.table = np.full((len(seqs), self.max_pages), -1, np.int32)
        at = 0
        for i, n in enumerate(per):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.q_start = (start + np.concatenate([[0], np.cumsum(self.news)])).astype(np.int32)
        self.N = int(self.q_start[-1]) + extra_rows
        self.max_new = max(self.news + [0]) if max_new is None else max_new
        self.max_len = max(self.lens + [0]) if max_len is None else max_len

    def device(self):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()
        return native.PagedBatch(t(self.table), t(self.q_start), t(np.array(self.lens)), self.max_new,
                                 self.max_len)

    def rows(self):
        """(packed row, sequence, position) of every new token that has one."""
        for s, (n, m) in enumerate(zip(self.lens, self.news)):
            for i in range(m):
                yield int(self.q_start[s]) + i, s, n - m + i

    def page_of(self, s, pos):
        p = int(self.table[s, pos // self.page])
        return p if 0 <= p < self.pool else None


def random_pages(ocodec, pool, Hkv, page, seed=0, nu=3.0):
    """Planes of random codes: uniform code bits, norms around ``nu``."""
    g = np.random.default_rng(seed)
    d = ocodec.d
    shape = (pool, Hkv, page)
    kscale = np.stack([nu * np.exp(0.4 * g.standard_normal(shape)), 0.4 * g.random(shape)], -1)
    if not ocodec.qjl_k:
        kscale[..., 1] = 0.0
    return dict(
        kcode=g.integers(0, 256, shape + (ocodec.planes_k, d // 8), dtype=np.uint8),
        kscale=kscale.astype(np.float16),
        vcode=g.integers(0, 1 << 32, (pool, Hkv, page // 32, ocodec.bits_v, d), dtype=np.uint32),
        vnorm=(nu * np.exp(0.4 * g.standard_normal(shape))).astype(np.float16), rows_cap=page)


def upload(planes, ncodec):
    pool, Hkv = planes["kcode"].shape[:2]
    return tl.upload_cache(planes, ncodec, pool, Hkv)


def _exact_codes(u, thresholds32):
    """#{k : u >= t_k} in 64 bits (the oracle rounds u to fp32 first, which
    decides differently where u is within half an fp32 step of a threshold)."""
    return np.sum(u[..., None] >= thresholds32.astype(np.float64), axis=-1).astype(np.int64)


def encode_keys(x, ocodec):
    e = oc.quantize_keys(x, ocodec)
    e["idx"] = _exact_codes(e["u"], ocodec.cb_k.thresholds32)
    if ocodec.qjl_k:
        r = e["u"] - ocodec.cb_k.centroids32.astype(np.float64)[e["idx"]]
        rho = np.sqrt(np.sum(r * r, axis=-1))
        e.update(r=r, rho=rho, rho16=rho.astype(np.float16), sigma=r @ ocodec.S.T >= 0)
    return e


def encode_values(x, ocodec):
    e = oc.quantize_values(x, ocodec)
    e["idx"] = _exact_codes(e["u"], ocodec.cb_v.thresholds32)
    return e


def page_rows(planes, ocodec, page, h):
    """Unpacked rows of one page and head."""
    return oc.cache_rows(planes, ocodec, page, h, planes["rows_cap"])


def sequence_rows(planes, ocodec, batch, s, h, n):
    """Dequantized keys and values [n, d] of a sequence's first n tokens, and
    which of them have a page."""
    P, d = batch.page, ocodec.d
    keys, vals, there = np.zeros((n, d)), np.zeros((n, d)), np.zeros(n, bool)
    for a in range(0, n, P):
        page, m = batch.page_of(s, a), min(P, n - a)
        if page is None:
            continue
        ik, sg, nk, rk, iv, nv = page_rows(planes, ocodec, page, h)
        keys[a:a + m] = oc.dequant_keys(ik, sg, nk, rk, ocodec)[:m]
        vals[a:a + m] = oc.dequant_values(iv, nv, ocodec)[:m]
        there[a:a + m] = True
    return keys, vals, there


def attention_ref(planes, ocodec, batch, q, scale, rope):
    """Answers [N, Hq, d] in 64 bits (NaN in rows that belong to no sequence)
    and the largest spread of a query's visible logits."""
    N, Hq, d = q.shape
    Hkv = planes["kcode"].shape[1]
    G = Hq // Hkv
    out = np.full((N, Hq, d), np.nan)
    sigma = 0.0
    for s, (n, m) in enumerate(zip(batch.lens, batch.news)):
        if m == 0:
            continue
        r0 = int(batch.q_start[s])
        pos = np.arange(n - m, n)
        for h in range(Hkv):
            keys, vals, there = sequence_rows(planes, ocodec, batch, s, h, n)
            for g in range(h * G, (h + 1) * G):
                x = q[r0:r0 + m, g]
                if rope is not None:
                    x = apply_rope(x, rope[0], rope[1], np.maximum(pos, 0))
                see = (np.arange(n)[None, :] <= pos[:, None]) & there[None, :]
                lg = np.where(see, scale * (x @ keys.T), -np.inf)
                for i in range(m):
                    if not see[i].any():
                        out[r0 + i, g] = 0.0
                        continue
                    v = lg[i][see[i]]
                    sigma = max(sigma, float(np.std(v)))
                    p = np.exp(v - v.max())
                    out[r0 + i, g] = p @ vals[see[i]] / p.sum()
    return out, sigma


def attention_tolerance(sigma, out_dtype):
    """Relative 2-norm bound of the answers.  Roundings at work, each at its rms
    size (a third root below the half step) and independent over the sums:
    the query and the key in fp16 (2^-11 of an element) shift a logit by up to
    2^-11 of the logits' spread each; a weight and a value in bf16 (2^-8 / sqrt 3
    each) and the answer's own rounding.  The spread is taken at the half step
    (not its rms) and four times the sum allowed."""
    half = 2.0 ** -8 / math.sqrt(3.0)
    o = half if out_dtype == torch.bfloat16 else 0.0
    return 4.0 * math.sqrt(2.0 * (2.0 ** -11 * max(sigma, 1.0)) ** 2 + 2.0 * half ** 2 + o ** 2)
