"""Head norms with rotary positions and cache appends on the GPU against 64 bits.

Tolerance of a normed and rotated element y = a c - b s: rounding to bf16 is off by at most
half a step, 2^-8 |y|. Before it, in fp32: the angle is rounded to 2^-25 half turns (pi 2^-25
absolute in cos and sin, whose own error is below 2^-22), the products and the sum to 2^-24
each, and the norm's factor carries d/8 + 7 roundings of the sum of squares (half of them
after the root), 2^-22 of the root and 2 products: below 2^-19 of |a| + |b| all together."""
import numpy as np
import pytest
import torch

import block_sparse_long_06_b200 as bsa
from oracle import tokens_oracle as TO

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def close(got, y, size):
    got = f64(got)
    off = np.abs(got - y)
    assert (off <= 2.0 ** -8 * np.abs(y) + 2.0 ** -19 * size).all(), float((off - 2.0 ** -8 * np.abs(y)).max())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def qkv_rows(N, Hq, Hkv, d, dtype, seed):
    x = (torch.randn(N, Hq + 2 * Hkv, d, generator=gen(seed), device="cuda") * 1.5).to(dtype)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def weights(d, seed):
    return (1.0 + 0.3 * torch.randn(d, generator=gen(seed), device="cuda")).float()


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (64, 64), (128, 64), (128, 80), (128, 128),
                                   (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope_matches_64_bits(dtype, d, rot, interleaved, norm):
    N, Hq, Hkv = 5, 6, 2
    q, k, _ = qkv_rows(N, Hq, Hkv, d, dtype, 1)
    pos = ints([0, 1, 777, 1 << 20, (1 << 21) - 1])
    f, factor = (bsa.rope_frequencies(rot, 500000.0, "ramp", 8.0) if rot else ([], 1.0))
    rope = bsa.Rope(bsa.rope_steps(f).cuda(), interleaved, factor) if rot else None
    wq, wk = (weights(d, 2), weights(d, 3)) if norm else (None, None)
    tok = bsa.Tokens(N=N, B=1, Hq=Hq, Hkv=Hkv, d=d, T=1 << 21, positions=pos, rope=rope, norm=norm,
                     eps=1e-5, q_weight=wq, k_weight=wk)
    q_out = torch.full((N, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((Hkv, N, d), 7.0, dtype=torch.bfloat16, device="cuda")   # head by head
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.bsa_norm_rope(tok, q, q_out, k, k_out.transpose(0, 1), status)
    assert int(status.item()) == 0
    for x, w, out in ((q, wq, q_out), (k, wk, k_out.transpose(0, 1))):
        close(out, *TO.norm_rope(f64(x), pos.cpu().numpy(), f, interleaved, factor,
                                 None if w is None else f64(w), 1e-5, norm))


@pytest.mark.parametrize("N,Hq,Hkv", [(1, 1, 1), (3, 16, 1), (2371, 4, 4), (2500, 6, 3)])
def test_norm_rope_row_counts_in_place_and_one_side(N, Hq, Hkv):
    """One row up to several rows a block, with heads that do not fill it; in place; q alone."""
    d = 64
    q, k, _ = qkv_rows(N, Hq, Hkv, d, torch.bfloat16, 5)
    f, _ = bsa.rope_frequencies(d)
    rope = bsa.Rope.make(d)
    tok = bsa.Tokens(N=N, B=1, Hq=Hq, Hkv=Hkv, d=d, T=N + 9, rope=rope, norm=True)
    pos = np.arange(9, N + 9)          # the newest N tokens of a sequence of T
    want_q = TO.norm_rope(f64(q), pos, f, norm=True, eps=1e-6)
    want_k = TO.norm_rope(f64(k), pos, f, norm=True, eps=1e-6)
    alone = torch.empty(N, Hq, d, dtype=torch.bfloat16, device="cuda")
    bsa.bsa_norm_rope(tok, q, alone)
    close(alone, *want_q)
    bsa.bsa_norm_rope(tok, q, q, k, k)
    close(q, *want_q)
    close(k, *want_k)
    assert torch.equal(q.contiguous(), alone)


def test_norm_rope_padding_rows_and_sequences():
    """Rows behind the last sequence keep what they held; empty sequences take no rows."""
    d, N = 128, 11
    q, _, _ = qkv_rows(N, 2, 1, d, torch.float16, 6)
    tok = bsa.Tokens(N=N, B=4, Hq=2, Hkv=1, d=d, T=100, cu_seqlens=ints([0, 3, 3, 8, 8]),
                     seq_lens=ints([3, 50, 90, 0]), rope=bsa.Rope.make(d))
    out = torch.full((N, 2, d), 5.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.bsa_norm_rope(tok, q, out, dev_status=status)
    assert int(status.item()) == 0
    f, _ = bsa.rope_frequencies(d)
    close(out[:8], *TO.norm_rope(f64(q[:8]), [0, 1, 2, 85, 86, 87, 88, 89], f))
    assert (out[8:] == 5.0).all()
    # a sequence shorter than its rows: they are reported and left
    tok.seq_lens = ints([2, 50, 90, 0])
    out.fill_(5.0)
    bsa.bsa_norm_rope(tok, q, out, dev_status=status)
    assert int(status.item()) == bsa.BSA_DEV_BAD_LENGTH
    assert (out[0] == 5.0).all()
    close(out[1:3], *TO.norm_rope(f64(q[1:3]), [0, 1], f))


def test_norm_of_zero_and_huge_heads():
    d = 128
    x = torch.zeros(3, 1, d, dtype=torch.float32, device="cuda")
    x[1] = 1e15
    x[2, 0, 3] = 1e-12
    tok = bsa.Tokens(N=3, B=1, Hq=1, Hkv=1, d=d, T=3, norm=True, eps=1e-6)
    out = torch.empty(3, 1, d, dtype=torch.bfloat16, device="cuda")
    bsa.bsa_norm_rope(tok, x, out)
    close(out, *TO.norm_rope(f64(x), [0, 0, 0], norm=True, eps=1e-6))


# ------------------------------------------------------------------ append
def pools(pages, Hkv, d, seed):
    g = gen(seed)
    return [torch.randn(pages, Hkv, 64, w, generator=g, device="cuda").to(torch.bfloat16)
            for w in (d, d, 16)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,Hq,Hkv,interleaved", [(128, 8, 2, False), (64, 4, 4, True)])
@pytest.mark.parametrize("with_q,with_idx", [(True, True), (False, False)])
def test_append_ragged_paged(dtype, d, Hq, Hkv, interleaved, with_q, with_idx):
    new, total = [3, 0, 130, 1, 64], [3, 40, 195, 65, 128]
    N = sum(new) + 4                       # padding rows
    q, k, v = qkv_rows(N, Hq, Hkv, d, dtype, 7)
    idx = torch.randn(N, Hkv, 16, generator=gen(8), device="cuda").to(dtype)
    K, V, I = pools(23, Hkv, d, 9)
    pt = torch.randperm(23, generator=gen(10), device="cuda").to(torch.int32)[:20].reshape(5, 4)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    wk = weights(d, 11)
    rope = bsa.Rope.make(d, interleaved=interleaved)
    tok = bsa.Tokens(N=N, B=5, Hq=Hq, Hkv=Hkv, d=d, T=256, cu_seqlens=ints(cu), seq_lens=ints(total),
                     rope=rope, norm=True, k_weight=wk)
    before = [x.clone() for x in (K, V, I)]
    q_out = torch.full((N, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.bsa_append_kv(tok, k, v, bsa.paged_cache(K, pt), bsa.paged_cache(V, pt),
                      k_idx=idx if with_idx else None,
                      kidx_cache=bsa.paged_cache(I, pt) if with_idx else None,
                      q=q if with_q else None, q_out=q_out if with_q else None, dev_status=status)
    assert int(status.item()) == 0
    f, _ = bsa.rope_frequencies(d)
    at = [t for t in TO.row_tokens(cu, total, N) if t[0] >= 0]
    pos = np.array([t for _, t in at])
    n = len(at)
    page = pt.cpu().numpy()[[b for b, _ in at], pos // 64]
    kw = TO.norm_rope(f64(k[:n]), pos, f, interleaved, 1.0, f64(wk), 1e-6, True)
    close(K[page, :, pos % 64], *kw)
    assert torch.equal(V[page, :, pos % 64], v[:n].to(torch.bfloat16))
    if with_idx:
        assert torch.equal(I[page, :, pos % 64], idx[:n].to(torch.bfloat16))
    if with_q:
        close(q_out[:n], *TO.norm_rope(f64(q[:n]), pos, f, interleaved, 1.0, None, 1e-6, True))
        assert (q_out[n:] == 3.0).all()
    # every other slot is as it was
    for x, old, wrote in ((K, before[0], True), (V, before[1], True), (I, before[2], with_idx)):
        if wrote:
            x[page, :, pos % 64] = old[page, :, pos % 64]
        assert torch.equal(x, old)


def test_append_one_token_each_contiguous_and_positions():
    """N = B without cu_seqlens, contiguous caches of a length that ends inside a block, and
    rotations that differ from the slots."""
    B, H, d, T = 6, 2, 128, 100
    _, k, v = qkv_rows(B, 4, H, d, torch.bfloat16, 12)
    lens = [1, 64, 65, 100, 99, 2]
    pos = ints([1000 + n for n in lens])
    K = torch.zeros(B, H, T, d, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    tok = bsa.Tokens(N=B, B=B, Hq=4, Hkv=H, d=d, T=T, seq_lens=ints(lens), positions=pos,
                     rope=bsa.Rope.make(d))
    bsa.bsa_append_kv(tok, k, v, bsa.contiguous_cache(K), bsa.contiguous_cache(V))
    f, _ = bsa.rope_frequencies(d)
    y = TO.norm_rope(f64(k), pos.cpu().numpy(), f)
    b = torch.arange(B)
    at = torch.tensor(lens) - 1
    close(K[b, :, at], *y)
    assert torch.equal(V[b, :, at], v)
    assert int((V != 0).any(-1).sum()) == B * H


def test_append_bad_pages_and_lengths_are_reported_and_skipped():
    B, H, d = 4, 2, 64
    _, k, v = qkv_rows(B, 2, H, d, torch.float32, 13)
    K, V, _ = pools(4, H, d, 14)
    before = K.clone(), V.clone()
    pt = ints([[0, 1], [2, 99], [-1, 3], [3, 3]])
    tok = bsa.Tokens(N=B, B=B, Hq=2, Hkv=H, d=d, T=128, seq_lens=ints([5, 70, 1, 300]))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.bsa_append_kv(tok, k, v, bsa.paged_cache(K, pt), bsa.paged_cache(V, pt), dev_status=status)
    assert int(status.item()) == bsa.BSA_DEV_BAD_PAGE | bsa.BSA_DEV_BAD_LENGTH
    assert torch.equal(K[0, :, 4], k[0].to(torch.bfloat16))
    K[0, :, 4], V[0, :, 4] = before[0][0, :, 4], before[1][0, :, 4]
    assert torch.equal(K, before[0]) and torch.equal(V, before[1])


@pytest.mark.parametrize("B", [33, 1025, 1100])
def test_append_finds_sequences_in_large_batches(B):
    """Two rounds of the sequence search, with empty sequences between."""
    H, d = 1, 64
    new = [(b * 7) % 3 for b in range(B)]
    cu = np.concatenate([[0], np.cumsum(new)])
    N = int(cu[-1])
    _, k, v = qkv_rows(N, 1, H, d, torch.bfloat16, 15)
    K = torch.zeros(B, H, 64, d, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    tok = bsa.Tokens(N=N, B=B, Hq=1, Hkv=H, d=d, T=64, cu_seqlens=ints(cu.tolist()),
                     seq_lens=ints([n + b % 5 for b, n in enumerate(new)]))
    bsa.bsa_append_kv(tok, k, v, bsa.contiguous_cache(K), bsa.contiguous_cache(V))
    at = TO.row_tokens(cu.tolist(), [n + b % 5 for b, n in enumerate(new)], N) if B < 100 else [
        (b, b % 5 + i) for b, n in enumerate(new) for i in range(n)]
    b, t = np.array(at).T
    assert torch.equal(V[b, :, t], v) and torch.equal(K[b, :, t], k)
    assert int((V != 0).any(-1).sum()) == N


def test_append_replays_in_a_graph_with_new_lengths():
    B, H, d = 3, 2, 128
    K, V, _ = pools(6, H, d, 16)
    pt = ints([[0, 1], [2, 3], [4, 5]])
    lens = ints([1, 64, 100])
    _, k, v = qkv_rows(B, 2, H, d, torch.bfloat16, 17)
    tok = bsa.Tokens(N=B, B=B, Hq=2, Hkv=H, d=d, T=128, seq_lens=lens, rope=bsa.Rope.make(d))
    call = lambda: bsa.bsa_append_kv(tok, k, v, bsa.paged_cache(K, pt), bsa.paged_cache(V, pt))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        call()
    lens.copy_(ints([30, 65, 128]))
    g.replay()
    torch.cuda.synchronize()
    f, _ = bsa.rope_frequencies(d)
    y = TO.norm_rope(f64(k), [29, 64, 127], f)
    close(torch.stack([K[0, :, 29], K[3, :, 0], K[5, :, 63]]), *y)


@pytest.mark.parametrize("bad", ["K", "V", "I", "extent"])
def test_append_writes_all_caches_or_none(bad):
    """Tables of their own for K, V and index keys, one of them with a page that does not exist
    (or a pool that ends before it): the row's other slots stay as they were, its query comes."""
    B, H, d = 3, 2, 128
    q, k, v = qkv_rows(B, 4, H, d, torch.bfloat16, 18)
    idx = torch.randn(B, H, 16, generator=gen(19), device="cuda").to(torch.bfloat16)
    pool = dict(zip("KVI", pools(6, H, d, 20)))
    table = dict(K=ints([[0, 1], [2, 3], [4, 5]]), V=ints([[5, 4], [3, 2], [1, 0]]),
                 I=ints([[2, 3], [4, 5], [0, 1]]))
    if bad in table:
        table[bad][1, 1] = 77
    caches = {n: bsa.paged_cache(pool[n], table[n]) for n in "KVI"}
    if bad == "extent":           # the index keys' page 5 (sequence 1) is cut off
        caches["I"] = bsa.paged_cache(pool["I"][:5], table["I"])
        caches["I"].num_pages = 6
    before = {n: x.clone() for n, x in pool.items()}
    tok = bsa.Tokens(N=B, B=B, Hq=4, Hkv=H, d=d, T=128, seq_lens=ints([3, 70, 128]),
                     rope=bsa.Rope.make(d))
    q_out = torch.zeros(B, 4, d, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.bsa_append_kv(tok, k, v, caches["K"], caches["V"], idx, caches["I"], q, q_out, status)
    assert int(status.item()) == bsa.BSA_DEV_BAD_PAGE
    f, _ = bsa.rope_frequencies(d)
    close(q_out, *TO.norm_rope(f64(q), [2, 69, 127], f))
    want = TO.norm_rope(f64(k), [2, 69, 127], f)
    for b, pos in ((0, 2), (2, 127)):
        at = {n: (int(table[n][b, pos // 64]), slice(None), pos % 64) for n in "KVI"}
        close(pool["K"][at["K"]], want[0][b], want[1][b])
        assert torch.equal(pool["V"][at["V"]], v[b]) and torch.equal(pool["I"][at["I"]], idx[b])
        for n in "KVI":
            pool[n][at[n]] = before[n][at[n]]
    for n in "KVI":
        assert torch.equal(pool[n], before[n])
