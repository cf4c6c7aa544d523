"""Plain forms and measured cases of the paged-cache operators.

Four operators work on one ragged batch: new tokens of several sequences,
packed back to back, over a compressed KV cache that is cut into pages.

* ``norm_rope``: RMS norm of every query and key head, then the rotate-half
  position rotation.
* ``append``: the new tokens' keys and values are rotated by position, coded
  (norm, randomized Walsh-Hadamard rotation, Lloyd-Max codes, sign sketch of the
  key residual) and written into their pages.  A quantized cache is compared
  through the values it stands for, so a pass also reads the new rows back.
* ``read_back``: rows of a paged cache as vectors.
* ``attention``: the new tokens' queries, each over the cached tokens up to its
  own position, straight from the pages.

The plain forms are elementary torch operations in fp32 (in fp64 where a value
next to a code border decides the code).
"""
import functools
import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases

def _attention(name, d, bits_k, bits_v, Hq, Hkv, page, seqs, new, ctx, theta):
    return {"name": name, "op": "attention", "d": d, "bits_k": bits_k, "bits_v": bits_v, "Hq": Hq,
            "Hkv": Hkv, "page": page, "seqs": seqs, "new": new, "ctx": ctx, "theta": theta}


def listed():
    return [
        # norms and rotation of 16 decoding sequences' heads: launch latency
        {"name": "norm_rope decode", "op": "norm_rope", "tokens": 16, "Hq": 32, "Hkv": 8, "d": 128,
         "dtype": "bf16", "theta": 5e5},
        # a long prompt of the Llama-shaped layer: HBM
        {"name": "norm_rope prompt", "op": "norm_rope", "tokens": 16384, "Hq": 32, "Hkv": 8, "d": 128,
         "dtype": "bf16", "theta": 5e5},
        # the ESM-shaped heads in fp32, an odd token count
        {"name": "norm_rope fp32", "op": "norm_rope", "tokens": 997, "Hq": 20, "Hkv": 20, "d": 64,
         "dtype": "fp32", "theta": 1e4},
        # one decode step of 64 sequences: one token each into 64 different pages
        {"name": "append decode", "op": "append", "d": 128, "bits_k": 4, "bits_v": 4, "Hkv": 8,
         "page": 64, "seqs": 64, "new": 1, "ctx": 4096, "theta": 5e5, "dtype": "bf16"},
        # prompts of four sequences, ragged, one of them continued inside a page
        {"name": "append prompts", "op": "append", "d": 128, "bits_k": 4, "bits_v": 4, "Hkv": 8,
         "page": 64, "seqs": 4, "new": 4096, "ctx": 5000, "theta": 5e5, "dtype": "bf16"},
        # a 32768-token prefix read back (moved to another engine, or re-encoded)
        {"name": "read_back prefix", "op": "read_back", "d": 128, "bits_k": 4, "bits_v": 4, "Hkv": 8,
         "page": 128, "seqs": 1, "new": 32768, "ctx": 32768, "dtype": "bf16"},
        # the last tokens of a few short sequences, ESM-shaped 3-bit codec
        {"name": "read_back tails", "op": "read_back", "d": 64, "bits_k": 3, "bits_v": 3, "Hkv": 20,
         "page": 32, "seqs": 8, "new": 33, "ctx": 201, "dtype": "bf16"},
        # one new token over a long context, the Llama-shaped decode layer
        _attention("decode one", 128, 4, 4, 32, 8, 64, 1, 1, 32768, 5e5),
        # a decode step of 64 sequences of 4096 to 8192 tokens
        _attention("decode batch", 128, 4, 4, 32, 8, 64, 64, 1, 8192, 5e5),
        # six drafted tokens each of eight sequences, the 2-bit long-context codec
        _attention("draft check", 128, 2, 2, 32, 8, 32, 8, 6, 16001, 0.0),
        # one chunk of a long prompt: 2048 new tokens behind 30720 cached ones
        _attention("prompt chunk", 128, 4, 4, 32, 8, 64, 1, 2048, 32768, 5e5),
        # whole prompts of sixteen sequences, ESM-shaped heads
        _attention("prompts", 64, 3, 3, 20, 20, 32, 16, 1024, 1024, 1e4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "read_back", "attention", "attention"])
    d, Hkv, G = rng.choice([(128, 8, 4), (128, 8, 4), (64, 20, 1), (128, 4, 8), (64, 8, 4), (128, 2, 7)])
    bits_k, bits_v = rng.choice([(4, 4), (4, 4), (3, 3), (2, 2), (5, 4), (3, 2)])
    theta = rng.choice([5e5, 1e4])
    page = rng.choice([32, 64, 128])
    if op == "norm_rope":
        return {"op": op, "tokens": _log(rng, 1, 16000), "Hq": Hkv * G, "Hkv": Hkv, "d": d,
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "theta": theta}
    if op in ("append", "read_back"):
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, max(2, 14000 // seqs))
        c = {"op": op, "d": d, "bits_k": bits_k, "bits_v": bits_v, "Hkv": Hkv, "page": page, "seqs": seqs,
             "new": new, "ctx": new + rng.randrange(0, 1000), "dtype": "bf16"}
        if op == "append":
            c["theta"] = theta
            c["dtype"] = rng.choice(["bf16", "bf16", "fp32"])
        return c
    kind = rng.choice(["decode", "draft", "chunk"])
    if kind == "chunk":
        seqs = _log(rng, 1, 8)
        new = _log(rng, 33, max(64, 2000 // seqs))
        ctx = new + _log(rng, 1, max(2, 24000 // seqs))
    else:
        seqs = _log(rng, 1, 64)
        new = 1 if kind == "decode" else rng.randrange(2, 17)
        ctx = new + _log(rng, 16, max(32, 200000 // max(seqs, 6)))
    return {"op": "attention", "d": d, "bits_k": bits_k, "bits_v": bits_v, "Hq": Hkv * G, "Hkv": Hkv,
            "page": page, "seqs": seqs, "new": new, "ctx": ctx, "theta": theta}


def _lengths(case):
    """(tokens of each sequence, new tokens among them): ragged between half and
    all of the case's context and new tokens, every sequence with at least one."""
    S, ctx, new = case["seqs"], case["ctx"], case["new"]
    lens = [max(1, ctx - (i * ctx) // (2 * S)) for i in range(S)]
    news = [min(lens[i], max(1, new - (i * new) // (2 * S))) for i in range(S)]
    return lens, news


def work(case):
    d = case["d"]
    if case["op"] == "norm_rope":
        es = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * (case["Hq"] + case["Hkv"]) * d
        return {"bytes": 2 * n * es + case["tokens"] * d * 4, "flops": 7 * n}
    lens, news = _lengths(case)
    Hkv = case["Hkv"]
    row = d // 8 * (case["bits_k"] + case["bits_v"]) + 6       # compressed bytes of a token and head
    N = sum(news)
    es = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if case["op"] == "append":
        # inputs, the rows written, the vectors read back; the sketch S r and its transpose
        return {"bytes": N * Hkv * (2 * d * es + row + 2 * d * 2) + N * d * 4,
                "flops": N * Hkv * 4 * d * d}
    if case["op"] == "read_back":
        return {"bytes": N * Hkv * (row + 2 * d * 2), "flops": N * Hkv * 2 * d * d}
    seen = sum(n * L - n * (n - 1) // 2 for L, n in zip(lens, news))
    return {"bytes": sum(lens) * Hkv * row + 2 * N * case["Hq"] * d * 2, "flops": 4 * d * case["Hq"] * seen}


# ------------------------------------------------------------------ the codec

@functools.lru_cache(maxsize=None)
def _codebook(d, bits):
    """Lloyd-Max centroids and thresholds (fp32) of the coordinate law
    (1 - x^2)^((d-3)/2) on [-1, 1]."""
    n = 1 << bits
    gx, gw = np.polynomial.legendre.leggauss(160)
    c = np.array([(2 * i + 1 - n) / n for i in range(n)]) * 2.5 / math.sqrt(d)
    for _ in range(100000):
        e = np.concatenate([[-1.0], (c[1:] + c[:-1]) / 2, [1.0]])
        mid, half = (e[1:] + e[:-1]) / 2, (e[1:] - e[:-1]) / 2
        x = mid[:, None] + half[:, None] * gx[None, :]
        f = gw[None, :] * np.exp((d - 3) / 2 * np.log1p(-x * x))
        new = (f * x).sum(1) / f.sum(1)
        new = (new - new[::-1]) / 2
        done = np.max(np.abs(new - c)) < 1e-16
        c = new
        if done:
            break
    return c.astype(np.float32), ((c[1:] + c[:-1]) / 2).astype(np.float32)


@functools.lru_cache(maxsize=None)
def _signs_and_sketch(d):
    """The rotation signs D and the sketch S (bf16 values) of every codec here."""
    g = np.random.Generator(np.random.PCG64(1000 + d))
    signs = np.where(g.integers(0, 2, size=d) == 1, 1, -1).astype(np.int8)
    S = torch.from_numpy(g.standard_normal((d, d), dtype=np.float32)).to(torch.bfloat16)
    return signs, S


@functools.lru_cache(maxsize=None)
def _handle(d, bits_k, bits_v):
    """The codec handle that a user's program keeps."""
    from rotated_codebook_kv_tq_b200 import native
    signs, S = _signs_and_sketch(d)
    return native.Codec(d, bits_k, True, bits_v, signs, S.view(torch.int16).numpy().view(np.uint16))


@functools.lru_cache(maxsize=None)
def _tables(d, bits_k, bits_v):
    """Device copies of the codec's constants for the plain forms."""
    signs, S = _signs_and_sketch(d)
    H = torch.ones((1, 1), dtype=torch.float64)
    while H.shape[0] < d:
        H = torch.cat([torch.cat([H, H], 1), torch.cat([H, -H], 1)], 0)
    Pi = H * torch.from_numpy(signs.astype(np.float64))[None, :] / math.sqrt(d)
    ck, tk = _codebook(d, bits_k - 1)
    cv, tv = _codebook(d, bits_v)
    dev = lambda a: torch.as_tensor(a).cuda()
    return {"Pi": dev(Pi), "S": dev(S.to(torch.float64)), "ck": dev(ck), "tk": dev(tk), "cv": dev(cv),
            "tv": dev(tv)}


def _rope_table(n, d, theta):
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * (
        theta ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") * 2.0 / d))[None, :]
    return ang.cos().float().contiguous(), ang.sin().float().contiguous()


def _rotate(x, cos, sin):
    """Rotate-half of x [N, H, d] with cos, sin [N, d/2]."""
    h = x.shape[-1] // 2
    c, s = cos[:, None, :].to(x.dtype), sin[:, None, :].to(x.dtype)
    return torch.cat([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], -1)


# ------------------------------------------------------------------ inputs

def _channel_scales(g, heads, d):
    """Lognormal channel scales with four outlier channels a head."""
    s = torch.exp(torch.randn((heads, d), generator=g, device="cuda"))
    hot = torch.rand((heads, d), generator=g, device="cuda").topk(4, dim=1).indices
    return s.scatter(1, hot, s.gather(1, hot) * 20.0)


def _encoded(g, case, pages):
    """Planes of a pool of ``pages`` pages that hold coded tokens."""
    d, Hkv, P, bits_k, bits_v = (case[k] for k in ("d", "Hkv", "page", "bits_k", "bits_v"))
    t = _tables(d, bits_k, bits_v)
    Pi, S = t["Pi"].float(), t["S"].float()
    sk, sv = _channel_scales(g, Hkv, d), _channel_scales(g, Hkv, d)
    kcode = torch.empty((pages, Hkv, P, bits_k, d // 8), dtype=torch.uint8, device="cuda")
    kscale = torch.empty((pages, Hkv, P, 2), dtype=torch.float16, device="cuda")
    vcode = torch.empty((pages, Hkv, P // 32, bits_v, d), dtype=torch.int32, device="cuda")
    vnorm = torch.empty((pages, Hkv, P), dtype=torch.float16, device="cuda")
    step = max(1, (1 << 23) // (Hkv * P * d))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = torch.randn((n, Hkv, P, d), generator=g, device="cuda") * sk[None, :, None, :]
        nu = x.norm(dim=-1)
        u = (x @ Pi.T) / nu[..., None]
        idx = torch.bucketize(u, t["tk"], right=True)
        r = u - t["ck"][idx]
        planes = [(idx >> p) & 1 for p in range(bits_k - 1)] + [(r @ S.T >= 0).long()]
        kcode[a:a + n] = _bytes(torch.stack(planes, 3))
        kscale[a:a + n] = torch.stack([nu, r.norm(dim=-1)], -1).half()
        x = torch.randn((n, Hkv, P, d), generator=g, device="cuda") * sv[None, :, None, :]
        nu = x.norm(dim=-1)
        idx = torch.bucketize((x @ Pi.T) / nu[..., None], t["tv"], right=True)
        idx = idx.view(n, Hkv, P // 32, 32, d)
        at = torch.arange(32, device="cuda")[:, None]
        for p in range(bits_v):
            vcode[a:a + n, :, :, p] = (((idx >> p) & 1) << at).sum(3).to(torch.int32)
        vnorm[a:a + n] = nu.half()
    return kcode, kscale, vcode, vnorm


def _bytes(bits):
    """[..., d] of 0/1 -> [..., d/8] bytes, coordinate i at byte i / 8, bit i % 8."""
    w = 1 << torch.arange(8, device=bits.device)
    return (bits.reshape(bits.shape[:-1] + (-1, 8)) * w).sum(-1).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    d, Hkv = case["d"], case["Hkv"]
    dt = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
    s = {"case": case}
    if case["op"] == "norm_rope":
        N, Hq = case["tokens"], case["Hq"]
        limit = 2 * N + 64
        # the heads as one projection leaves them: queries, keys and values of a token side by side
        s["qkv"] = torch.randn((N, Hq + 2 * Hkv, d), generator=g, device="cuda").mul_(2.0).to(dt)
        s["q"], s["k"] = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv]
        s["wq"] = (1.0 + 0.2 * torch.randn((d,), generator=g, device="cuda")).to(dt)
        s["wk"] = (1.0 + 0.2 * torch.randn((d,), generator=g, device="cuda")).to(dt)
        s["rope"] = _rope_table(limit, d, case["theta"])
        s["positions"] = torch.randint(0, limit, (N,), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.empty((N, Hq, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((N, Hkv, d), dtype=dt, device="cuda")
        return s
    lens, news = _lengths(case)
    P, S, N = case["page"], case["seqs"], sum(news)
    per = [-(-n // P) for n in lens]
    pool = sum(per) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((S, max(per)), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    s["kcode"], s["kscale"], s["vcode"], s["vnorm"] = _encoded(g, case, pool)
    s["table"] = table
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device="cuda")
    s["N"], s["max_new"], s["max_len"] = N, max(news), max(lens)
    s["rope"] = _rope_table(max(lens), d, case["theta"]) if case.get("theta") else None
    if case["op"] == "append":
        # keys and values of a token side by side, as the projection leaves them
        scale = torch.cat([_channel_scales(g, Hkv, d), _channel_scales(g, Hkv, d)])
        s["kv"] = (torch.randn((N, 2 * Hkv, d), generator=g, device="cuda") * scale[None]).to(dt)
        s["k"], s["v"] = s["kv"][:, :Hkv], s["kv"][:, Hkv:]
    if case["op"] in ("append", "read_back"):
        s["k_out"] = torch.empty((N, Hkv, d), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty((N, Hkv, d), dtype=torch.bfloat16, device="cuda")
    else:
        s["q"] = torch.randn((N, case["Hq"], d), generator=g, device="cuda").to(torch.bfloat16)
        s["out"] = torch.empty((N, case["Hq"], d), dtype=torch.bfloat16, device="cuda")
    if own:
        from rotated_codebook_kv_tq_b200 import native
        s["codec"] = _handle(d, case["bits_k"], case["bits_v"])
        s["cache"] = native.Cache(s["kcode"], s["kscale"], s["vcode"], s["vnorm"], pool, Hkv, P)
        s["batch"] = native.PagedBatch(s["table"], s["q_start"], s["seq_lens"], s["max_new"], s["max_len"])
        if case["op"] == "attention":
            n = native.paged_attention_workspace(s["codec"], s["batch"], N, case["Hq"], Hkv)
            s["ws"] = torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _owner(s):
    """(sequence, position) of every new token."""
    n = torch.arange(s["N"], device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].long(), n, right=True)
    pos = s["seq_lens"].long()[seq] - (s["q_start"].long()[seq + 1] - n)
    return seq, pos


def _unit(x, Pi):
    """norm and rotated unit vector, in 64 bits: the codes hang on borders."""
    x = x.double()
    nu = x.square().sum(-1).sqrt()
    return nu, (x @ Pi.T) / torch.where(nu > 0, nu, 1.0)[..., None]


def _plain_append(s):
    case = s["case"]
    P, bits_k, bits_v = case["page"], case["bits_k"], case["bits_v"]
    t = _tables(case["d"], bits_k, bits_v)
    seq, pos = _owner(s)
    page, row = s["table"].long()[seq, pos // P], pos % P
    k = s["k"].double()
    if s["rope"] is not None:
        k = _rotate(k, s["rope"][0][pos], s["rope"][1][pos])
    nu, u = _unit(k, t["Pi"])
    idx = torch.bucketize(u, t["tk"].double(), right=True)
    r = u - t["ck"].double()[idx]
    code = torch.stack([(idx >> p) & 1 for p in range(bits_k - 1)] + [(r @ t["S"].T >= 0).long()], 2)
    s["kcode"][page, :, row] = _bytes(code)
    s["kscale"][page, :, row] = torch.stack([nu, r.square().sum(-1).sqrt()], -1).half()
    nu, u = _unit(s["v"], t["Pi"])
    idx = torch.bucketize(u, t["tv"].double(), right=True)
    s["vnorm"][page, :, row] = nu.half()
    # 32-token words: the bits of new tokens replaced, the others kept
    Hkv, d = case["Hkv"], case["d"]
    words = s["vcode"].view(-1, bits_v, d)
    at = (page[:, None] * Hkv + torch.arange(Hkv, device="cuda")) * (P // 32) + (row // 32)[:, None]
    bit = (1 << (row % 32)).to(torch.int32)[:, None, None, None]
    planes = torch.stack([(idx >> p) & 1 for p in range(bits_v)], 2).to(torch.int32)
    new = torch.zeros_like(words).index_put_((at,), planes * bit, accumulate=True)
    mask = torch.zeros_like(words).index_put_((at,), bit.expand_as(planes), accumulate=True)
    words.copy_((words & ~mask) | new)


def _gathered(s, page, row):
    """Centroids, signs and scales (fp32) of the given cache rows: page, row [...]."""
    case = s["case"]
    d, bits_k, bits_v = case["d"], case["bits_k"], case["bits_v"]
    t = _tables(d, bits_k, bits_v)
    byte = s["kcode"][page, :, row]                              # [..., Hkv, planes, d/8]
    bits = ((byte[..., None] >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1).flatten(-2)
    idx = sum(bits[..., p, :].int() << p for p in range(bits_k - 1))
    scale = s["kscale"][page, :, row].float()
    word = s["vcode"][page, :, row // 32]                        # [..., Hkv, bits_v, d]
    vb = (word >> (row % 32).to(torch.int32)[..., None, None, None]) & 1
    vidx = sum(vb[..., p, :] << p for p in range(bits_v))
    return (t["ck"][idx], bits[..., bits_k - 1, :].float() * 2 - 1, scale[..., 0], scale[..., 1],
            t["cv"][vidx], s["vnorm"][page, :, row].float())


def _plain_read_back(s):
    case = s["case"]
    d, P = case["d"], case["page"]
    t = _tables(d, case["bits_k"], case["bits_v"])
    seq, pos = _owner(s)
    c, sg, nu, rho, cv, nv = _gathered(s, s["table"].long()[seq, pos // P], pos % P)
    coef = math.sqrt(math.pi / 2) / d
    y = c + coef * rho[..., None] * (sg @ t["S"].float())
    Pi = t["Pi"].float()
    return (nu[..., None] * (y @ Pi)).bfloat16(), (nv[..., None] * (cv @ Pi)).bfloat16()


def _plain_attention(s):
    case = s["case"]
    d, P, S, Hq, Hkv = case["d"], case["page"], case["seqs"], case["Hq"], case["Hkv"]
    t = _tables(d, case["bits_k"], case["bits_v"])
    Pi, Sk = t["Pi"].float(), t["S"].float()
    seq, pos = _owner(s)
    q = s["q"].float()
    if s["rope"] is not None:
        q = _rotate(q, s["rope"][0][pos], s["rope"][1][pos])
    q1 = q @ Pi.T
    # padded: [sequence, new token, head] and [sequence, cached token, head]
    slot = torch.arange(s["N"], device="cuda") - s["q_start"].long()[seq]
    M, L = s["max_new"], s["max_len"]
    qp = torch.zeros((S, M, Hkv, Hq // Hkv, d), device="cuda")
    qp[seq, slot] = q1.view(-1, Hkv, Hq // Hkv, d)
    qpos = torch.full((S, M), -1, device="cuda", dtype=torch.long)
    qpos[seq, slot] = pos
    j = torch.arange(L, device="cuda")
    c, sg, nu, rho, cv, nv = _gathered(s, s["table"].long()[:, j // P], (j % P).expand(S, L))
    coef = math.sqrt(math.pi / 2) / d
    key = c + coef * rho[..., None] * (sg @ Sk)                  # <q', S^T sg> = <S q', sg>
    key = (key * nu[..., None] / math.sqrt(d)).permute(0, 2, 3, 1)          # [S, Hkv, d, L]
    value = (cv * nv[..., None]).transpose(1, 2)                            # [S, Hkv, L, d]
    rows = qp.permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, d)                 # (head of the group, token)
    logit = (rows @ key).view(S, Hkv, Hq // Hkv, M, L)
    logit.masked_fill_((j > qpos[..., None])[:, None, None], -math.inf)
    logit.sub_(logit.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    o = logit.view(S, Hkv, -1, L) @ value
    o = o / logit.view(S, Hkv, -1, L).sum(-1, keepdim=True).clamp_min(1e-30)
    o = (o @ Pi).view(S, Hkv, Hq // Hkv, M, d).permute(0, 3, 1, 2, 4)       # [S, M, Hkv, G, d]
    return o[seq, slot].reshape(-1, Hq, d).bfloat16()


def _plain_norm_rope(s):
    cos, sin = s["rope"]
    p = s["positions"].long()
    c, n = cos[p], sin[p]

    def one(x, w):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        return _rotate(y, c, n)
    return one(s["q"], s["wq"]).to(s["q"].dtype), one(s["k"], s["wk"]).to(s["k"].dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        from rotated_codebook_kv_tq_b200 import native
        if op == "norm_rope":
            native.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], EPS, s["positions"], s["q_out"],
                                s["k_out"], rope=s["rope"])
            return s["q_out"], s["k_out"]
        if op == "attention":
            native.paged_attention(s["codec"], s["q"], s["cache"], s["batch"],
                                   1 / math.sqrt(s["case"]["d"]), s["out"], s["ws"], rope=s["rope"])
            return s["out"]
        if op == "append":
            native.paged_quantize_kv(s["codec"], s["k"], s["v"], s["cache"], s["batch"], rope=s["rope"])
        native.paged_dequantize(s["codec"], s["cache"], s["batch"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if op == "norm_rope":
        return _plain_norm_rope(s)
    if op == "attention":
        return _plain_attention(s)
    if op == "append":
        _plain_append(s)
    return _plain_read_back(s)


# ------------------------------------------------------------------ 64 bits

def _exact_rope(x, cos, sin):
    """Complex rotation of x [..., n, d] by angles with cos, sin [n, d/2]."""
    h = x.shape[-1] // 2
    z = torch.complex(x[..., :h], x[..., h:]) * torch.complex(cos.double(), sin.double())
    return torch.cat([z.real, z.imag], -1)


def _exact_rows(s, seq, head, n):
    """Dequantized keys and values of tokens 0..n-1 of a sequence's KV head, in
    the rotated domain, from the planes, by integer arithmetic on whole words."""
    case = s["case"]
    d, P, bits_k, bits_v = case["d"], case["page"], case["bits_k"], case["bits_v"]
    t = _tables(d, bits_k, bits_v)
    pages = s["table"][seq, :-(-n // P)].long()
    by = s["kcode"][pages, head].reshape(-1, bits_k, d // 8)[:n].to(torch.int64)
    idx = torch.zeros((n, d), dtype=torch.int64, device="cuda")
    sg = None
    for p in range(bits_k):
        bit = torch.stack([by[:, p] // (1 << e) % 2 for e in range(8)], -1).reshape(n, d)
        if p < bits_k - 1:
            idx += bit * (1 << p)
        else:
            sg = 2.0 * bit.double() - 1.0
    sc = s["kscale"][pages, head].reshape(-1, 2)[:n].double()
    key = t["ck"].double()[idx] + (math.sqrt(math.pi / 2) / d) * sc[:, 1:] * torch.einsum("ij,ni->nj", t["S"], sg)
    w = s["vcode"][pages, head].reshape(-1, bits_v, d).to(torch.int64) % (1 << 32)
    j = torch.arange(n, device="cuda")
    vi = torch.zeros((n, d), dtype=torch.int64, device="cuda")
    for p in range(bits_v):
        vi += (w[j // 32, p] >> (j % 32)[:, None]) % 2 * (1 << p)
    nv = s["vnorm"][pages, head].reshape(-1)[:n].double()
    return key * sc[:, :1], t["cv"].double()[vi] * nv[:, None]


def _exact_codes(x, t, centroids, thresholds):
    """norm, rotated unit vector and its centroids, by counting thresholds."""
    nu = torch.sqrt((x * x).sum(-1))
    u = torch.einsum("ij,...j->...i", t["Pi"], x) / nu[..., None]
    n = torch.zeros_like(u, dtype=torch.int64)
    for th in thresholds.double():
        n += u >= th
    return nu, u, centroids.double()[n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        p = s["positions"].long()
        out = []
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            x = x.double()
            y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
            out.append(_exact_rope(y.transpose(0, 1), s["rope"][0][p], s["rope"][1][p]).transpose(0, 1))
        return out
    d, Hkv, P = case["d"], case["Hkv"], case["page"]
    lens, news = _lengths(case)
    t = _tables(d, case["bits_k"], case["bits_v"])
    if case["op"] == "append":
        # what the new rows stand for, without the planes
        pos = torch.cat([torch.arange(L - n, L, device="cuda") for L, n in zip(lens, news)])
        k = s["k"].double()
        if s["rope"] is not None:
            k = _exact_rope(k.transpose(0, 1), s["rope"][0][pos], s["rope"][1][pos]).transpose(0, 1)
        nu, u, c = _exact_codes(k, t, t["ck"], t["tk"])
        r = u - c
        sg = torch.where(torch.einsum("ij,...j->...i", t["S"], r) >= 0, 1.0, -1.0).double()
        rho = torch.sqrt((r * r).sum(-1)).half().double()
        y = c + math.sqrt(math.pi / 2) / d * rho[..., None] * torch.einsum("ij,...i->...j", t["S"], sg)
        key = nu.half().double()[..., None] * torch.einsum("ij,...i->...j", t["Pi"], y)
        nu, u, c = _exact_codes(s["v"].double(), t, t["cv"], t["tv"])
        return [key, nu.half().double()[..., None] * torch.einsum("ij,...i->...j", t["Pi"], c)]
    N, Hq = sum(news), case.get("Hq", 0)
    G = Hq // Hkv
    at = [0] + list(np.cumsum(news))
    if case["op"] == "read_back":
        key = torch.empty((N, Hkv, d), dtype=torch.float64, device="cuda")
        value = torch.empty_like(key)
        for i in range(len(lens)):
            for h in range(Hkv):
                kr, vr = _exact_rows(s, i, h, lens[i])
                key[at[i]:at[i + 1], h] = kr[lens[i] - news[i]:] @ t["Pi"]
                value[at[i]:at[i + 1], h] = vr[lens[i] - news[i]:] @ t["Pi"]
        return [key, value]
    out = torch.empty((N, Hq, d), dtype=torch.float64, device="cuda")
    for i in range(len(lens)):
        q = s["q"][at[i]:at[i + 1]].double().transpose(0, 1)             # [Hq, n, d]
        pos = torch.arange(lens[i] - news[i], lens[i], device="cuda")
        if s["rope"] is not None:
            q = _exact_rope(q, s["rope"][0][pos], s["rope"][1][pos])
        q = q @ t["Pi"].T
        hidden = torch.arange(lens[i], device="cuda")[None, :] > pos[:, None]
        for h in range(Hkv):
            kr, vr = _exact_rows(s, i, h, lens[i])
            for g in range(h * G, (h + 1) * G):
                w = torch.softmax((q[g] @ kr.T / math.sqrt(d)).masked_fill(hidden, -math.inf), -1)
                out[at[i]:at[i + 1], g] = (w @ vr) @ t["Pi"]
    return out
