"""Head norms with the position rotation against 64-bit references."""
import numpy as np
import pytest
import torch

from oracle.rotation import apply_rope
from rotated_codebook_kv_tq_b200 import native, synth
import tq_testlib as tl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    tl.require_cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def reference(x, w, eps, pos, rope):
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    if w is not None:
        y = y * w
    if rope is None:
        return y
    return apply_rope(y.transpose(1, 0, 2), rope[0], rope[1], pos).transpose(1, 0, 2)


def close(got, x, w, eps, pos, rope, dtype):
    """The final rounding, and fp32 sums and products before it: the mean of d
    squares, its root, three products and the rotation's sum, (d + 12) half
    steps on terms no larger than the pair's sizes."""
    want = reference(x, w, eps, pos, rope)
    d = x.shape[-1]
    y = reference(x, w, eps, pos, None)
    pair = np.abs(y) + np.abs(np.roll(y, d // 2, -1))
    tol = torch.finfo(dtype).eps / 2 * np.abs(want) + (d + 12) * 2.0 ** -24 * pair * (1 + torch.finfo(dtype).eps)
    assert np.all(np.abs(host(got) - want) <= tol + 1e-38), np.max(np.abs(host(got) - want) - tol)


CASES = [
    # tokens, Hq, Hk, d, dtype, weight dtype, rope, padding of a token's row (elements)
    (1, 1, 1, 128, torch.bfloat16, torch.bfloat16, True, 0),
    (5, 32, 8, 128, torch.bfloat16, torch.bfloat16, True, 256),
    (33, 7, 3, 64, torch.bfloat16, torch.float32, True, 64),
    (17, 5, 2, 128, torch.float32, torch.float32, True, 0),
    (64, 20, 20, 64, torch.float32, torch.bfloat16, False, 3),
    (9, 4, 2, 128, torch.bfloat16, torch.bfloat16, True, 3),
    (1001, 14, 2, 128, torch.bfloat16, None, True, 128),
    (300, 1, 33, 64, torch.bfloat16, torch.bfloat16, True, 1),
]


@pytest.mark.parametrize("case", CASES, ids=[f"n{c[0]}h{c[1]}-{c[2]}d{c[3]}-{i}" for i, c in enumerate(CASES)])
def test_matches_64_bits(case):
    N, Hq, Hk, d, dtype, wd, with_rope, pad = case
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    width = (Hq + Hk) * d + pad
    buf = torch.randn((N, width), generator=g, device="cuda").mul_(3).to(dtype)
    q = buf.as_strided((N, Hq, d), (width, d, 1))
    k = buf.as_strided((N, Hk, d), (width, d, 1), Hq * d)
    wq = None if wd is None else (1 + 0.3 * torch.randn((d,), generator=g, device="cuda")).to(wd)
    wk = None if wd is None else (1 + 0.3 * torch.randn((d,), generator=g, device="cuda")).to(wd)
    limit = 77
    rope = synth.rope_table(limit, d, 1e4) if with_rope else None
    pos = torch.randint(-2, limit + 3, (N,), generator=g, device="cuda", dtype=torch.int32)
    at = np.clip(pos.cpu().numpy(), 0, limit - 1)
    qo, ko = torch.empty((N, Hq, d), dtype=dtype, device="cuda"), torch.empty((N, Hk, d), dtype=dtype, device="cuda")
    before = buf.clone()
    native.qk_norm_rope(q, k, wq, wk, 1e-5, pos if with_rope else None, qo, ko, rope=tl.rope_device(rope))
    hw = lambda w: None if w is None else host(w)
    close(qo, host(q), hw(wq), 1e-5, at, rope, dtype)
    close(ko, host(k), hw(wk), 1e-5, at, rope, dtype)
    assert torch.equal(buf, before)
    # one side alone gives the same, and so does writing over the input
    q2 = torch.empty_like(qo)
    native.qk_norm_rope(q, None, wq, None, 1e-5, pos if with_rope else None, q2, None, rope=tl.rope_device(rope))
    assert torch.equal(q2, qo)
    native.qk_norm_rope(q, k, wq, wk, 1e-5, pos if with_rope else None, q, k, rope=tl.rope_device(rope))
    assert torch.equal(q, qo) and torch.equal(k, ko)
    if pad:
        assert torch.equal(buf[:, (Hq + Hk) * d:], before[:, (Hq + Hk) * d:])


def test_zero_tiny_and_huge_rows():
    d = 128
    x = torch.zeros((4, 1, d), dtype=torch.float32, device="cuda")
    x[1] = 1e-12
    x[2] = 1e15
    x[3, 0, 7] = -5.0
    y = torch.empty_like(x)
    native.qk_norm_rope(x, None, None, None, 1e-6, None, y, None)
    close(y, host(x), None, 1e-6, None, None, torch.float32)
    assert (y[0] == 0).all()


def test_empty_call():
    x = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    native.qk_norm_rope(x, x, None, None, 1e-6, None, x, x)


def test_captured_call_follows_positions():
    d, N = 64, 6
    rope = synth.rope_table(50, d, 1e4)
    rd = tl.rope_device(rope)
    x = torch.randn((N, 3, d), device="cuda")
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    native.qk_norm_rope(x, None, None, None, 1e-6, pos, y, None, rope=rd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        native.qk_norm_rope(x, None, None, None, 1e-6, pos, y, None, rope=rd)
    x.mul_(-2.0).add_(1.0)
    pos.add_(17)
    graph.replay()
    torch.cuda.synchronize()
    close(y, host(x), None, 1e-6, pos.cpu().numpy(), rope, torch.float32)
