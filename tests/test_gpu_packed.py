"""Dense packed attention and shared-prefix decode on the GPU against 64 bits.

Tolerances. With s the largest scale * sum |q_c k_c| of a row: a score is a sum of d products
of bf16 values (exact in fp32) with one rounding of at most 2^-23 (of what it adds up) each,
so it is off by at most e = d 2^-23 s; the base-2 exponential adds 2^-17. P is rounded to bf16
(2^-8 relative), O adds n products with 2^-23 each. So |o - o_exact| is at most
(2^-8 + 2 (e + 2^-17) + n 2^-23) sum_j p_j |v_j| before it is rounded to bf16 (2^-8 |o|), and
lse is off by at most e + 2^-17 + n 2^-24 + 2^-22 |lse|."""
import math

import numpy as np
import pytest
import torch

import block_sparse_long_06_b200 as bsa
from oracle import tokens_oracle as TO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(*shape, seed=0, scale=1.0):
    return (torch.randn(*shape, generator=gen(seed), device="cuda") * scale).to(torch.bfloat16)


class Paged:
    """Pools with scattered pages; every slot behind a sequence's end holds NaN or infinity."""

    def __init__(self, lens, Hkv, d, seed, spare=3, T=None):
        nb = [-(-n // 64) for n in lens]
        width = max(1, max(nb) if T is None else -(-T // 64))
        P = sum(nb) + spare
        self.K, self.V = (randn(P, Hkv, 64, d, seed=seed + i) for i in (0, 1))
        order = torch.randperm(P, generator=torch.Generator().manual_seed(seed))
        self.pt = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(nb):
            self.pt[b, :n] = order[at:at + n]
            at += n
        for p in order[at:].tolist():
            self.K[p], self.V[p] = float("nan"), float("inf")
        for b, n in enumerate(lens):
            if n % 64:
                p = int(self.pt[b, nb[b] - 1])
                self.K[p, :, n % 64:], self.V[p, :, n % 64:] = float("nan"), float("-inf")
        self.pt = self.pt.cuda()
        self.lens, self.T = lens, 64 * width if T is None else T

    def caches(self):
        return bsa.paged_cache(self.K, self.pt), bsa.paged_cache(self.V, self.pt)

    def keys(self, X, b, n):
        """[Hkv, n, d] of sequence b, in 64 bits."""
        pages = self.pt[b, :-(-n // 64)].long()
        return f64(X[pages]).transpose(1, 0, 2, 3).reshape(X.shape[1], -1, X.shape[3])[:, :n]


def exact(q, mem, cu, lens, causal, G, scale=None, hide=None):
    """(o, lse, spread, size, n) over all rows; rows of no sequence keep lse = nan."""
    N, Hq, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    o, spread = np.zeros((N, Hq, d)), np.zeros((N, Hq, d))
    lse, size = np.full((N, Hq), np.nan), np.zeros((N, Hq))
    qq = f64(q)
    for b, n in enumerate(lens):
        r = slice(cu[b], cu[b + 1])
        c = cu[b + 1] - cu[b]
        K, V = mem.keys(mem.K, b, n), mem.keys(mem.V, b, n)
        vis = np.ones((c, n), bool)
        if causal:
            vis = np.arange(n)[None, :] <= (n - c + np.arange(c))[:, None]
        if hide is not None:
            vis = vis & ~hide(b, np.arange(n))[None, :]
        for h in range(Hq):
            o[r, h], lse[r, h], spread[r, h], size[r, h] = TO.attend_rows(
                qq[r, h], K[h // G], V[h // G], scale, vis)
    return o, lse, spread, size


def check(step, want, keys, d):
    o, lse, spread, size = want
    live = ~np.isnan(lse)
    e = d * 2.0 ** -23 * size + 2.0 ** -17
    got32, got, gl = f64(step.o_f32), f64(step.o), f64(step.lse)
    bound = (2.0 ** -8 + 2 * e + keys * 2.0 ** -23)[..., None] * spread
    off = np.abs(got32 - o)
    assert np.isfinite(got32[live]).all()
    assert (off <= bound)[live].all(), float((off - bound)[live].max())
    assert torch.equal(step.o_f32.to(torch.bfloat16)[torch.from_numpy(live)], step.o[torch.from_numpy(live)])
    none = live & np.isinf(lse)
    assert (gl[none] == -np.inf).all() and not got[none].any()
    some = live & np.isfinite(lse)
    off = np.abs(gl[some] - lse[some])
    bound = (e + keys * 2.0 ** -24)[some] + 2.0 ** -22 * np.abs(lse[some])
    assert (off <= bound).all(), float((off - bound).max())


def sums(x):
    return [0] + list(np.cumsum(x))


def run_attend(q, mem, cu, lens, Hkv, causal=True, pad=0, status=0, **kw):
    N, Hq, d = q.shape
    tok = bsa.Tokens(N=N, B=len(lens), Hq=Hq, Hkv=Hkv, d=d, T=mem.T, cu_seqlens=ints(cu),
                     seq_lens=ints(lens), causal=causal, **kw)
    step = bsa.PackedAttention(tok)
    for x in (step.o, step.lse, step.o_f32):
        x.fill_(77.0)
    step.run(q, *mem.caches())
    assert int(step.status.item()) == status
    for x in (step.o, step.lse, step.o_f32):
        assert (x[cu[-1]:] == 77.0).all()       # padding rows
    return step


# ------------------------------------------------------------------ packed attention
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_batch(d, G, causal):
    """Prompts, chunks behind a cache, single tokens, a sequence without rows, page and tile
    ends inside sequences, garbage behind every end."""
    Hkv = 2
    new, lens = [1, 70, 0, 257, 1, 33], [1, 70, 5, 300, 515, 129]
    cu = sums(new)
    mem = Paged(lens, Hkv, d, seed=G + d)
    q = randn(cu[-1] + 3, Hkv * G, d, seed=9, scale=1.5)
    step = run_attend(q, mem, cu, lens, Hkv, causal)
    check(step, exact(q, mem, cu, lens, causal, G), 515, d)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 640])
def test_prompt_lengths(n):
    d, G, Hkv = 128, 4, 1
    mem = Paged([n], Hkv, d, seed=n)
    q = randn(n, G, d, seed=n + 1, scale=1.5)
    step = run_attend(q, mem, [0, n], [n], Hkv)
    check(step, exact(q, mem, [0, n], [n], True, G), n, d)


@pytest.mark.parametrize("lens", [[4097], [1, 3000, 64, 0, 128, 5000]])
def test_single_tokens_split_over_keys(lens):
    """One row a sequence (an empty sequence has a row too: it sees nothing)."""
    d, G, Hkv = 128, 4, 2
    B = len(lens)
    mem = Paged(lens, Hkv, d, seed=21)
    q = randn(B, Hkv * G, d, seed=22, scale=2.0)
    bad = bsa.BSA_DEV_BAD_LENGTH if 0 in lens else 0     # no token, but a row
    step = run_attend(q, mem, list(range(B + 1)), lens, Hkv, status=bad)
    check(step, exact(q, mem, list(range(B + 1)), lens, True, G), max(lens), d)
    # the same rows without cu_seqlens
    tok = bsa.Tokens(N=B, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, T=mem.T, seq_lens=ints(lens))
    again = bsa.PackedAttention(tok)
    again.run(q, *mem.caches())
    assert torch.equal(again.o, step.o) and torch.equal(again.lse, step.lse)


@pytest.mark.parametrize("d", [64, 128])
def test_one_row_over_many_splits(d):
    """More splits than a warp has lanes are joined; three kv heads."""
    n, G, Hkv = 40000, 4, 3
    mem = Paged([n], Hkv, d, seed=23)
    q = randn(1, Hkv * G, d, seed=24, scale=2.0)
    step = run_attend(q, mem, [0, 1], [n], Hkv)
    check(step, exact(q, mem, [0, 1], [n], True, G), n, d)


def test_the_same_call_gives_the_same_bits():
    d, G, Hkv = 128, 4, 2
    lens, new = [1500, 700, 3000, 64], [200, 1, 3, 64]
    cu = sums(new)
    mem = Paged(lens, Hkv, d, seed=25)
    q = randn(cu[-1], Hkv * G, d, seed=26)
    first = run_attend(q, mem, cu, lens, Hkv)
    for _ in range(5):
        again = run_attend(q, mem, cu, lens, Hkv)
        assert torch.equal(first.o_f32, again.o_f32) and torch.equal(first.lse, again.lse)


def test_two_streams_at_once():
    """Two objects, each with a workspace of its own, on two streams; inputs of one made on the
    other's stream are waited for by the caller."""
    d, G, Hkv = 128, 4, 2
    lens, new = [900, 3000], [100, 1]
    cu = sums(new)
    mem = Paged(lens, Hkv, d, seed=27)
    qs = [randn(cu[-1], Hkv * G, d, seed=28 + i) for i in range(2)]
    steps, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for q in qs:
        tok = bsa.Tokens(N=cu[-1], B=2, Hq=Hkv * G, Hkv=Hkv, d=d, T=mem.T, cu_seqlens=ints(cu),
                         seq_lens=ints(lens))
        steps.append(bsa.PackedAttention(tok))
    torch.cuda.synchronize()
    for _ in range(4):
        for q, step, stream in zip(qs, steps, streams):
            step.run(q, *mem.caches(), stream=stream)
    torch.cuda.synchronize()
    for q, step in zip(qs, steps):
        assert int(step.status.item()) == 0
        check(step, exact(q, mem, cu, lens, True, G), 3000, d)


def test_growing_scores_move_the_maximum():
    """Each block of keys has larger scores than the ones before, so O is rescaled many times;
    one key late in the row takes nearly all the weight."""
    d, G, Hkv, n = 128, 2, 1, 700
    mem = Paged([n], Hkv, d, seed=30)
    q = randn(40, G, d, seed=31)
    mean = q.float().mean((0, 1))
    mean /= mean.norm()
    for i in range(n):
        p, r = int(mem.pt[0, i // 64]), i % 64
        mem.K[p, 0, r] = (mean * (i / 8.0)).to(torch.bfloat16)
    q = (q.float() + mean * 6.0).to(torch.bfloat16)
    step = run_attend(q, mem, [0, 40], [n], Hkv)
    want = exact(q, mem, [0, 40], [n], True, G)
    assert (want[1].max() > 40)
    check(step, want, n, d)


def test_contiguous_caches_strided_queries_and_scale():
    d, G, Hkv, B, T = 64, 4, 2, 3, 150
    lens, new = [150, 77, 3], [20, 77, 1]
    cu = sums(new)
    K, V = randn(B, Hkv, T, d, seed=40), randn(B, Hkv, T, d, seed=41)
    qkv = randn(cu[-1], Hkv * (G + 2), d, seed=42)
    q = qkv[:, :Hkv * G]
    tok = bsa.Tokens(N=cu[-1], B=B, Hq=Hkv * G, Hkv=Hkv, d=d, T=T, cu_seqlens=ints(cu),
                     seq_lens=ints(lens), attn_scale=0.3)
    step = bsa.PackedAttention(tok)
    step.run(q, bsa.contiguous_cache(K), bsa.contiguous_cache(V))
    assert int(step.status.item()) == 0

    class Flat:
        pass
    mem = Flat()
    mem.K, mem.V = K, V
    mem.keys = lambda X, b, n: f64(X[b, :, :n])
    check(step, exact(q, mem, cu, lens, True, G, scale=0.3), 150, d)


def test_equal_rows_without_lengths():
    """No cu_seqlens and no seq_lens: B sequences of T tokens, all of them rows."""
    d, Hkv, G, B, T = 64, 1, 8, 2, 200
    mem = Paged([T] * B, Hkv, d, seed=43, T=T)
    q = randn(B * T, G, d, seed=44)
    tok = bsa.Tokens(N=B * T, B=B, Hq=G, Hkv=Hkv, d=d, T=T)
    step = bsa.PackedAttention(tok)
    step.run(q, *mem.caches())
    check(step, exact(q, mem, [0, T, 2 * T], [T, T], True, G), T, d)


@pytest.mark.parametrize("causal", [True, False])
def test_bad_pages_are_left_out(causal):
    d, G, Hkv = 128, 4, 2
    lens, new = [500, 300], [100, 1]
    cu = sums(new)
    mem = Paged(lens, Hkv, d, seed=50)
    q = randn(cu[-1], Hkv * G, d, seed=51)
    good = mem.pt.clone()
    mem.pt[0, 2], mem.pt[0, 7], mem.pt[1, 0] = -5, 10 ** 6, 1 << 30
    step = run_attend(q, mem, cu, lens, Hkv, causal, status=bsa.BSA_DEV_BAD_PAGE)
    mem.pt = good
    hide = lambda b, j: np.isin(j // 64, [2, 7] if b == 0 else [0])
    check(step, exact(q, mem, cu, lens, causal, G, hide=hide), 500, d)


def test_bad_lengths_write_nothing_or_clamp():
    d, Hkv = 64, 1
    mem = Paged([100, 100], Hkv, d, seed=52)
    q = randn(10, 2, d, seed=53)
    for cu in ([0, 6, 4], [0, 4, 11], [1, 4, 10], [0, -1, 10]):
        tok = bsa.Tokens(N=10, B=2, Hq=2, Hkv=Hkv, d=d, T=mem.T, cu_seqlens=ints(cu),
                         seq_lens=ints([100, 100]))
        step = bsa.PackedAttention(tok)
        step.o.fill_(77.0)
        step.lse.fill_(77.0)
        step.run(q, *mem.caches())
        assert int(step.status.item()) == bsa.BSA_DEV_BAD_LENGTH
        assert (step.o == 77.0).all() and (step.lse == 77.0).all()
    # a sequence shorter than its rows: the first ones see nothing
    step = run_attend(q, mem, [0, 5, 10], [3, 100], Hkv, status=bsa.BSA_DEV_BAD_LENGTH)
    assert (step.lse[:2] == -math.inf).all() and not step.o[:2].any()
    want = exact(q, mem, [0, 5, 10], [3, 100], True, 2)
    check(step, want, 100, d)


def test_many_short_sequences():
    d, G, Hkv, B = 64, 2, 1, 1500
    new = [1 + b % 3 for b in range(B)]
    cu = sums(new)
    K, V = randn(B, Hkv, 64, d, seed=54), randn(B, Hkv, 64, d, seed=55)
    q = randn(cu[-1], G, d, seed=56)
    tok = bsa.Tokens(N=cu[-1], B=B, Hq=G, Hkv=Hkv, d=d, T=64, cu_seqlens=ints(cu),
                     seq_lens=ints([n + b % 50 for b, n in enumerate(new)]))
    step = bsa.PackedAttention(tok)
    step.run(q, bsa.contiguous_cache(K), bsa.contiguous_cache(V))
    lens = [n + b % 50 for b, n in enumerate(new)]

    class Flat:
        pass
    mem = Flat()
    mem.K, mem.V = K, V
    kk, vv = f64(K), f64(V)
    mem.keys = lambda X, b, n: (kk if X is K else vv)[b, :, :n]
    check(step, exact(q, mem, cu, lens, True, G), 64, d)


def test_graph_replay_with_new_lengths_and_a_second_stream():
    d, G, Hkv = 128, 4, 2
    mem = Paged([700, 700, 700], Hkv, d, seed=60)
    N = 300
    q = randn(N, Hkv * G, d, seed=61)
    cu, lens = ints([0, 100, 200, 300]), ints([700, 700, 700])
    tok = bsa.Tokens(N=N, B=3, Hq=Hkv * G, Hkv=Hkv, d=d, T=mem.T, cu_seqlens=cu, seq_lens=lens)
    step = bsa.PackedAttention(tok)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run(q, *mem.caches())
    side.synchronize()
    first = step.o.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        step.run(q, *mem.caches())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.o, first)
    for cu1, len1 in (([0, 1, 2, 3], [700, 1, 350]), ([0, 0, 299, 299], [9, 640, 0])):
        cu.copy_(ints(cu1))
        lens.copy_(ints(len1))
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert int(step.status.item()) == 0
        part = Paged.__new__(Paged)
        part.__dict__.update(mem.__dict__)
        want = exact(q, part, cu1, len1, True, G)
        # the pools hold garbage only behind 700, so shorter lengths read real keys
        check(step, want, 700, d)


# ------------------------------------------------------------------ shared prefixes
def run_shared(q, mem, cu, lens, Hkv, own, **kw):
    N, Hq, d = q.shape
    tok = bsa.Tokens(N=N, B=len(lens), Hq=Hq, Hkv=Hkv, d=d, T=mem.T, cu_seqlens=ints(cu),
                     seq_lens=ints(lens))
    step = bsa.SharedPrefixDecode(tok)
    for x in (step.o, step.lse, step.o_f32):
        x.fill_(77.0)
    step.run(q, *mem.caches(), *own)
    assert int(step.status.item()) == 0
    for x in (step.o, step.lse, step.o_f32):
        assert (x[cu[-1]:] == 77.0).all()
    return step


def exact_shared(q, mem, cu, lens, G, own):
    o, lse, spread, size = exact(q, mem, cu, lens, False, G)
    if own[0] is None:
        return o, lse, spread, size
    oo, ll = f64(own[0]), f64(own[1])
    live = ~np.isnan(lse)
    om, lm, wa, wb = TO.merge(o, np.where(live, lse, 0.0), oo, ll)
    spread = wa[..., None] * spread + np.where(wb[..., None] > 0, np.abs(oo), 0.0) * wb[..., None]
    return om, np.where(live, lm, np.nan), spread, size


@pytest.mark.parametrize("d,G", [(64, 1), (128, 4), (128, 16)])
@pytest.mark.parametrize("rows,lens", [([1], [1]), ([40], [777]), ([3, 0, 65, 2], [600, 64, 1, 0])])
@pytest.mark.parametrize("with_own", [True, False])
def test_shared_prefix(d, G, rows, lens, with_own):
    Hkv = 2
    cu = sums(rows)
    N = cu[-1] + 2
    mem = Paged(lens, Hkv, d, seed=70)
    q = randn(N, Hkv * G, d, seed=71, scale=1.5)
    own = (None, None)
    if with_own:
        o_own = torch.randn(N, Hkv * G, d, generator=gen(72), device="cuda")
        lse_own = 5.0 + 3.0 * torch.randn(N, Hkv * G, generator=gen(73), device="cuda")
        lse_own[0, 0] = -math.inf           # a sequence with no tokens of its own yet
        o_own[0, 0] = float("nan")
        own = (o_own, lse_own)
    step = run_shared(q, mem, cu, lens, Hkv, own)
    check(step, exact_shared(q, mem, cu, lens, G, own), max(lens), d)


@pytest.mark.parametrize("d,G,Hkv", [(128, 4, 8), (64, 8, 3)])
def test_work_dealt_to_the_sms_in_equal_parts(d, G, Hkv):
    """Few tiles of very different lengths, a prefix without tokens and one of a single block
    among them: tiles are cut wherever an SM's share ends."""
    rows, lens = [30, 1, 64, 2, 17], [9000, 0, 2500, 64, 5001]
    cu = sums(rows)
    mem = Paged(lens, Hkv, d, seed=78)
    q = randn(cu[-1], Hkv * G, d, seed=79, scale=1.5)
    own = (torch.randn(cu[-1], Hkv * G, d, generator=gen(80), device="cuda"),
           8.0 + torch.randn(cu[-1], Hkv * G, generator=gen(81), device="cuda"))
    step = run_shared(q, mem, cu, lens, Hkv, own)
    check(step, exact_shared(q, mem, cu, lens, G, own), max(lens), d)


def test_shared_prefix_bad_ranges_write_nothing():
    mem = Paged([100, 100], 1, 64, seed=82)
    q = randn(10, 2, 64, seed=83)
    good = bsa.Tokens(N=10, B=2, Hq=2, Hkv=1, d=64, T=mem.T, cu_seqlens=ints([0, 5, 10]),
                      seq_lens=ints([100, 100]))
    step = bsa.SharedPrefixDecode(good)
    step.run(q, *mem.caches())                   # leaves results in the workspace
    for cu in ([0, 6, 4], [0, 4, 11], [1, 4, 10]):
        good.cu_seqlens = ints(cu)
        step.status.zero_()
        step.o.fill_(77.0)
        step.lse.fill_(77.0)
        step.run(q, *mem.caches())
        assert int(step.status.item()) == bsa.BSA_DEV_BAD_LENGTH
        assert (step.o == 77.0).all() and (step.lse == 77.0).all()


def test_shared_prefix_outputs_may_be_the_own_part():
    d, G, Hkv = 128, 4, 2
    mem = Paged([300], Hkv, d, seed=74)
    q = randn(9, Hkv * G, d, seed=75)
    o_own = torch.randn(9, Hkv * G, d, generator=gen(76), device="cuda")
    lse_own = torch.randn(9, Hkv * G, generator=gen(77), device="cuda") + 5
    step = run_shared(q, mem, [0, 9], [300], Hkv, (o_own, lse_own))
    bsa.bsa_decode_shared(step.tok, q, *mem.caches(), o_own, lse_own, step.o, lse_own, o_own,
                          step.workspace, step.status)
    assert torch.equal(o_own, step.o_f32) and torch.equal(lse_own, step.lse)


# ------------------------------------------------------------------ together
def test_prompt_append_attend_then_shared_decode():
    """As a server runs them: a shared document and the sequences' own prompts are appended
    (normed and rotated) and attended; then a decode step appends a token to every sequence,
    block-sparse decode covers its own tokens and the document is joined to it."""
    d, Hq, Hkv, G, B, doc = 128, 8, 2, 4, 3, 333
    own_lens = [70, 1, 200]
    g = gen(80)
    T = 320
    nb = T // 64
    pages = 6 + B * nb
    K, V, I = (torch.full((pages, Hkv, 64, w), float("nan"), dtype=torch.bfloat16, device="cuda")
               for w in (d, d, 16))
    pt = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    doc_pt, own_pt = pt[:6].reshape(1, 6).contiguous(), pt[6:].reshape(B, nb).contiguous()
    rope = bsa.Rope.make(d, theta=500000.0)
    w = (1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).float()
    common = dict(Hq=Hq, Hkv=Hkv, d=d, rope=rope, norm=True, q_weight=w, k_weight=w)
    f, _ = bsa.rope_frequencies(d, 500000.0)
    new = lambda n: [torch.randn(n, h, x, generator=g, device="cuda").to(torch.bfloat16)
                     for h, x in ((Hq, d), (Hkv, d), (Hkv, d), (Hkv, 16))]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(tok, x, table):
        q, k, v, idx = x
        q_out = torch.empty_like(q)
        bsa.bsa_append_kv(tok, k, v, bsa.paged_cache(K, table), bsa.paged_cache(V, table), idx,
                          bsa.paged_cache(I, table), q, q_out, status)
        return q_out

    # the document
    x_doc = new(doc)
    tok = bsa.Tokens(N=doc, B=1, T=6 * 64, seq_lens=ints([doc]), **common)
    q_doc = append(tok, x_doc, doc_pt)
    att = bsa.PackedAttention(tok)
    att.run(q_doc, bsa.paged_cache(K, doc_pt), bsa.paged_cache(V, doc_pt))
    mem = Paged.__new__(Paged)
    mem.K, mem.V, mem.pt, mem.T = K, V, doc_pt, 6 * 64
    check(att, exact(q_doc, mem, [0, doc], [doc], True, G), doc, d)

    # a decode step: the sequences' tokens so far, then one more each
    for lens, rows in ((own_lens, own_lens), ([n + 1 for n in own_lens], [1] * B)):
        cu = sums(rows)
        x = new(cu[-1])
        pos = np.concatenate([doc + n - c + np.arange(c) for n, c in zip(lens, rows)])
        tok = bsa.Tokens(N=cu[-1], B=B, T=T, cu_seqlens=ints(cu), seq_lens=ints(lens),
                         positions=ints(pos.tolist()), **common)
        q = append(tok, x, own_pt)
        want_q = TO.norm_rope(f64(x[0]), pos, f, weight=f64(w), eps=1e-6, norm=True)
        assert (np.abs(f64(q) - want_q[0]) <= 2.0 ** -8 * np.abs(want_q[0]) + 2.0 ** -19 * want_q[1]).all()
    prob = bsa.Problem(phase=bsa.PHASE_DECODE, B=B, Hq=Hq, Hkv=Hkv, d=d, T=T, n_sink=1, n_local=2,
                       k_max=8, p=1.0, seq_lens=ints(lens))
    sparse = bsa.DecodeStep(prob)
    q_idx = torch.randn(B, Hq, 16, generator=g, device="cuda").to(torch.bfloat16)
    for page in own_pt.flatten().tolist():       # block-sparse decode wants finite rows
        K[page], V[page], I[page] = K[page].nan_to_num(), V[page].nan_to_num(), I[page].nan_to_num()
    sparse.run(q, q_idx, bsa.paged_cache(I, own_pt), bsa.paged_cache(K, own_pt),
               bsa.paged_cache(V, own_pt))
    assert int(sparse.status.item()) == 0 and int(status.item()) == 0
    tok = bsa.Tokens(N=B, B=1, Hq=Hq, Hkv=Hkv, d=d, T=6 * 64, seq_lens=ints([doc]))
    shared = bsa.SharedPrefixDecode(tok)
    shared.run(q, bsa.paged_cache(K, doc_pt), bsa.paged_cache(V, doc_pt), sparse.o_f32, sparse.lse)
    # every block was kept: the sum is dense attention over the document and all own tokens
    kd, vd = mem.keys(K, 0, doc), mem.keys(V, 0, doc)
    want = [np.zeros((B, Hq, d)), np.zeros((B, Hq)), np.zeros((B, Hq, d)), np.zeros((B, Hq))]
    mem.pt = own_pt
    for b, n in enumerate(lens):
        ko, vo = mem.keys(K, b, n), mem.keys(V, b, n)
        for h in range(Hq):
            kk, vv = np.concatenate([kd[h // G], ko[h // G]]), np.concatenate([vd[h // G], vo[h // G]])
            r = TO.attend_rows(f64(q)[b:b + 1, h], kk, vv, 1 / math.sqrt(d), np.ones((1, len(kk)), bool))
            for a, y in zip(want, r):
                a[b, h] = y[0]
    check(shared, want, doc + max(lens), d)


# ------------------------------------------------------------------ both ways to plan
PLANS = [
    # new, lens, Hkv, G, d, causal
    ([1] * 31, [1 + 83 * b for b in range(31)], 2, 4, 128, True),      # a block plans for itself
    ([1] * 32, [1 + 83 * b for b in range(32)], 2, 4, 128, True),      # 33 tiles: the plan kernel
    ([2] * 40, [2600 - 64 * b for b in range(40)], 1, 4, 64, False),
    ([800], [2900], 4, 8, 64, True),           # 25 tiles of 4 heads, cut: two units a block
    ([800], [2900], 4, 8, 64, False),
    ([600], [1500], 37, 1, 64, True),          # at most 4 tiles of 37 heads: as many as SMs
    ([600], [1500], 38, 1, 64, True),
    ([33, 0, 65, 1], [1600, 0, 1537, 1], 3, 4, 128, True),
]


@pytest.mark.parametrize("new,lens,Hkv,G,d,causal", PLANS)
def test_units_of_both_plans(new, lens, Hkv, G, d, causal):
    cu = sums(new)
    mem = Paged(lens, Hkv, d, seed=90)
    q = randn(cu[-1] + 2, Hkv * G, d, seed=91, scale=1.5)
    step = run_attend(q, mem, cu, lens, Hkv, causal)
    check(step, exact(q, mem, cu, lens, causal, G), max(lens), d)


@pytest.mark.parametrize("B", [3, 40])
@pytest.mark.parametrize("T", [128, 4096])
def test_bad_ranges_are_refused_by_both_plans(B, T):
    mem = Paged([100] * B, 1, 64, seed=92, T=T)
    q = randn(3 * B, 2, 64, seed=93)
    good = list(range(0, 3 * B + 1, 3))
    tok = bsa.Tokens(N=3 * B, B=B, Hq=2, Hkv=1, d=64, T=T, cu_seqlens=ints(good),
                     seq_lens=ints([100] * B))
    step = bsa.PackedAttention(tok)
    step.run(q, *mem.caches())                   # leaves results in the workspace
    assert int(step.status.item()) == 0
    for at, value in ((0, 1), (1, 0x7fffffff), (1, -2147483648), (B - 1, 0), (B, 3 * B + 1)):
        cu = list(good)
        cu[at] = value
        tok.cu_seqlens = ints(cu)
        step.status.zero_()
        for x in (step.o, step.lse, step.o_f32):
            x.fill_(77.0)
        step.run(q, *mem.caches())
        assert int(step.status.item()) == bsa.BSA_DEV_BAD_LENGTH
        assert all((x == 77.0).all() for x in (step.o, step.lse, step.o_f32))


@pytest.mark.parametrize("n", [100, 1500])
def test_outputs_that_start_at_16_bytes(n):
    """32-byte stores are for outputs on 32-byte boundaries."""
    d, G, Hkv = 128, 4, 2
    mem = Paged([n], Hkv, d, seed=94)
    q = randn(70, Hkv * G, d, seed=95)
    want = run_attend(q, mem, [0, 70], [n], Hkv)
    size = 70 * Hkv * G * d
    o = torch.zeros(size + 8, dtype=torch.bfloat16, device="cuda")[8:].view(70, Hkv * G, d)
    o_f32 = torch.zeros(size + 4, device="cuda")[4:].view(70, Hkv * G, d)
    lse = torch.zeros(70, Hkv * G, device="cuda")
    for a, b in ((o, want.o_f32), (want.o, o_f32), (o, o_f32), (o, None)):
        for x in (o, o_f32, lse):
            x.zero_()
        b = torch.empty_like(want.o_f32) if b is want.o_f32 else b
        a = torch.empty_like(want.o) if a is want.o else a
        bsa.bsa_attend_packed(want.tok, q, *mem.caches(), a, lse, b, want.workspace, want.status)
        assert torch.equal(a, want.o) and torch.equal(lse, want.lse)
        assert b is None or torch.equal(b, want.o_f32)


@pytest.mark.parametrize("lens", [[100, 0, 64], [5000, 0, 300]])
@pytest.mark.parametrize("rows", [[2, 1, 40], [70, 3, 300]])
def test_the_own_part_is_joined_once(rows, lens):
    """By the unit that has a row alone, or by the merge of its splits."""
    d, G, Hkv = 128, 4, 2
    cu = sums(rows)
    mem = Paged(lens, Hkv, d, seed=96)
    q = randn(cu[-1] + 1, Hkv * G, d, seed=97, scale=1.5)
    own = (torch.randn(cu[-1] + 1, Hkv * G, d, generator=gen(98), device="cuda"),
           8.0 + torch.randn(cu[-1] + 1, Hkv * G, generator=gen(99), device="cuda"))
    own[1][0, :2], own[1][cu[1], :] = 200.0, -math.inf
    step = run_shared(q, mem, cu, lens, Hkv, own)
    check(step, exact_shared(q, mem, cu, lens, G, own), max(lens), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [[1, 20, 3], [90, 2, 33]])
def test_what_other_rows_hold_has_no_effect(d, rows):
    """Padding rows and other sequences' rows share tiles with a sequence's: NaN or infinite
    there, its bits stay."""
    G, Hkv = 8, 2
    lens = [1700, 300, 129]
    cu = sums(rows)
    mem = Paged(lens, Hkv, d, seed=100)
    q = randn(cu[-1] + 40, Hkv * G, d, seed=101, scale=1.5)
    want = run_attend(q, mem, cu, lens, Hkv)
    bad = q.clone()
    bad[cu[1]:] = float("nan")
    bad[cu[1] + 1::2] = float("inf")
    got = run_attend(bad, mem, cu, lens, Hkv)
    for a, b in ((got.o, want.o), (got.lse, want.lse), (got.o_f32, want.o_f32)):
        assert torch.equal(a[:cu[1]], b[:cu[1]])


@pytest.mark.parametrize("d", [64, 128])
def test_units_of_odd_numbers_of_steps(d):
    """A block's units with one tile of rows and with two, of one step and of many, one after the
    other: buffers of scores and stages go on where the last unit left them."""
    G, Hkv = 4, 1
    new = [1, 64, 1, 33, 2, 70, 1, 5, 64, 1, 1, 40] * 40
    lens = [n + (b * 97) % 700 for b, n in enumerate(new)]
    cu = sums(new)
    mem = Paged(lens, Hkv, d, seed=102)
    q = randn(cu[-1], Hkv * G, d, seed=103, scale=1.5)
    step = run_attend(q, mem, cu, lens, Hkv)
    check(step, exact(q, mem, cu, lens, True, G), max(lens), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 40, 300])
def test_maxima_that_rise_at_every_step(d, new):
    """Later keys are ever longer, so that O is rescaled at most steps, in some rows of a warp and
    not in others."""
    G, Hkv, n = 4, 2, 1400
    mem = Paged([n], Hkv, d, seed=104)
    pages = mem.pt[0].long()
    for j, p in enumerate(pages[:-(-n // 64)].tolist()):
        mem.K[p] = (mem.K[p].float() * (1.0 + 1.5 * j)).to(torch.bfloat16)
    q = randn(new, Hkv * G, d, seed=105, scale=1.5)
    q[::3] *= 0.05
    step = run_attend(q, mem, [0, new], [n], Hkv)
    check(step, exact(q, mem, [0, new], [n], True, G), n, d)


@pytest.mark.parametrize("B,shared", [(3, False), (40, False), (3, True), (40, True)])
def test_a_captured_plan_follows_the_lengths(B, shared):
    """Splits, rows and the number of tiles change from replay to replay, in both ways to plan; an
    outsider's results with the same lengths are the same bits."""
    d, G, Hkv, T = 128, 4, 2, 4096
    N = 4 * B
    mem = Paged([T] * B, Hkv, d, seed=110, T=T)
    q = randn(N, Hkv * G, d, seed=111, scale=1.5)
    own = ()
    if shared:
        own = (torch.randn(N, Hkv * G, d, generator=gen(112), device="cuda"),
               8.0 + torch.randn(N, Hkv * G, generator=gen(113), device="cuda"))
    cu, lens = ints([4 * b for b in range(B + 1)]), ints([T] * B)
    make = bsa.SharedPrefixDecode if shared else bsa.PackedAttention
    tok = lambda c, n: bsa.Tokens(N=N, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, T=T, cu_seqlens=c, seq_lens=n)
    step = make(tok(cu, lens))
    caches = mem.caches()
    step.run(q, *caches, *own)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run(q, *caches, *own)
    for seed in range(4):
        r = np.random.default_rng(seed)
        rows = [0, 1, 4, 2][seed] + r.integers(0, 1 + [4, 3, 0, 1][seed], B)
        have = r.integers(4, [T, 200, T, 1500][seed] + 1, B)
        cu.copy_(ints(sums(rows.tolist())))
        lens.copy_(ints(have.tolist()))
        for x in (step.o, step.lse, step.o_f32):
            x.fill_(77.0)
        graph.replay()
        other = make(tok(cu.clone(), lens.clone()))
        for x in (other.o, other.lse, other.o_f32):
            x.fill_(77.0)
        other.run(q, *caches, *own)
        assert int(step.status.item()) == 0 and int(other.status.item()) == 0
        for a, b in ((step.o, other.o), (step.lse, other.lse), (step.o_f32, other.o_f32)):
            assert torch.equal(a, b)
        n = int(rows.sum())
        assert (step.lse[n:] == 77.0).all() and (step.lse[:n] != 77.0).all()
    # the last batch against 64 bits
    c = sums(rows.tolist())
    want = (exact_shared(q, mem, c, have.tolist(), G, own) if shared
            else exact(q, mem, c, have.tolist(), True, G))
    check(step, want, T, d)


@pytest.mark.parametrize("d", [64, 128])
def test_own_part_in_place_with_and_without_splits(d):
    """o_f32 is o_own and lse is lse_own, for rows that the merge writes and rows that it does not."""
    G, Hkv, rows, lens = 4, 2, [3, 5, 70], [6000, 100, 3001]
    cu = sums(rows)
    mem = Paged(lens, Hkv, d, seed=120)
    q = randn(cu[-1], Hkv * G, d, seed=121, scale=1.5)
    o_own = torch.randn(cu[-1], Hkv * G, d, generator=gen(122), device="cuda")
    lse_own = 8.0 + torch.randn(cu[-1], Hkv * G, generator=gen(123), device="cuda")
    step = run_shared(q, mem, cu, lens, Hkv, (o_own, lse_own))
    check(step, exact_shared(q, mem, cu, lens, G, (o_own, lse_own)), max(lens), d)
    bsa.bsa_decode_shared(step.tok, q, *mem.caches(), o_own, lse_own, step.o, lse_own, o_own,
                          step.workspace, step.status)
    assert torch.equal(o_own, step.o_f32) and torch.equal(lse_own, step.lse)


@pytest.mark.parametrize("new", [1, 70])
def test_bad_value_pages_of_a_table_with_rows_of_its_own(new):
    """K's and V's tables start at the same address, V's rows are closer together: a bad page of
    V's alone, behind the first 32 blocks, is found as one of K's is."""
    d, G, Hkv, nb = 64, 4, 2, 40
    n = nb * 64 - 5
    K, V = randn(2 * nb, Hkv, 64, d, seed=130), randn(2 * nb, Hkv, 64, d, seed=131)
    table = torch.full((4 * nb,), -1, dtype=torch.int32)
    kt, vt = table.view(2, 2 * nb), table[:2 * nb].view(2, nb)
    kt[0, :nb], kt[1, :nb] = torch.arange(nb), torch.arange(nb, 2 * nb)
    vt[1] = torch.arange(nb).flip(0)
    table[nb + 35] = 1 << 20                        # block 35 of V's second sequence
    table = table.cuda()
    kt, vt = table.view(2, 2 * nb), table[:2 * nb].view(2, nb)
    caches = bsa.paged_cache(K, kt), bsa.paged_cache(V, vt)
    assert kt.data_ptr() == vt.data_ptr()
    cu = [0, new, 2 * new]
    q = randn(2 * new, Hkv * G, d, seed=132, scale=1.5)
    tok = bsa.Tokens(N=2 * new, B=2, Hq=Hkv * G, Hkv=Hkv, d=d, T=nb * 64, cu_seqlens=ints(cu),
                     seq_lens=ints([n, n]))
    step = bsa.PackedAttention(tok)
    step.run(q, *caches)
    assert int(step.status.item()) == bsa.BSA_DEV_BAD_PAGE

    class Two:
        pass
    mem = Two()
    mem.K, mem.V = K, V
    mem.keys = lambda X, b, m: f64(X[(kt if X is K else vt)[b, :nb].long().clamp(max=2 * nb - 1)]).transpose(
        1, 0, 2, 3).reshape(Hkv, -1, d)[:, :m]
    hide = lambda b, j: (j // 64 == 35) if b == 1 else np.zeros(len(j), bool)
    check(step, exact(q, mem, cu, [n, n], True, G, hide=hide), n, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1 << 20, 1 << 17])
def test_sums_of_many_equal_scores_behind_a_larger_one(n, d):
    """So many rows that no unit is split. Every key behind the first has the same score, so that
    each of n equal terms is added to a sum that has grown: lse is off by at most 2.8e-6 (an
    exponential), 2^-21 (its argument and the ex2), 64 2^-24 (a step's sum), 2^-23 (their sum) and
    2^-22 of itself, less than 2^-16 together at any length."""
    G, Hkv, N = 16, 8, 16 * 74
    K = torch.zeros(2, Hkv, 64, d, device="cuda", dtype=torch.bfloat16)
    K[..., :8] = 0.25 * torch.arange(8, device="cuda").to(torch.bfloat16)
    K[0, :, 0] *= 1.125
    V = randn(2, Hkv, 64, d, seed=140)
    pt = torch.ones(1, n // 64, dtype=torch.int32)
    pt[0, 0] = 0
    q = torch.zeros(N, Hkv * G, d, device="cuda", dtype=torch.bfloat16)
    q[..., :8] = randn(N, 1, 8, seed=141)
    scale = 0.7
    tok = bsa.Tokens(N=N, B=1, Hq=Hkv * G, Hkv=Hkv, d=d, T=n, attn_scale=scale)
    step = bsa.SharedPrefixDecode(tok, keep_f32=False)
    assert bsa.bsa_packed_workspace_size(tok, bsa.OP_DECODE_SHARED) < 1 << 20     # no splits
    step.run(q, bsa.paged_cache(K, pt.cuda()), bsa.paged_cache(V, pt.cuda()))
    assert int(step.status.item()) == 0
    first, other = (f64(q[:, 0, :8]) @ f64(K[0, 0, r, :8]) * float(np.float32(scale)) for r in (0, 1))
    want = np.logaddexp(first, np.log(n - 1.0) + other)
    assert (np.abs(f64(step.lse) - want[:, None]) <= 2.0 ** -16).all(), np.abs(f64(step.lse) - want[:, None]).max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 70])
def test_scores_beyond_fp32_make_their_rows_nan(d, new):
    """inf - inf is NaN in 32 bits, wherever in a step the key is; rows without one stay."""
    G, Hkv, n = 2, 1, 300
    for key in (0, 13, 14, 15, 130, 229):
        mem = Paged([n], Hkv, d, seed=150)
        q = randn(new, G, d, seed=151)
        q[:, 0] = 0.0
        want = run_attend(q, mem, [0, new], [n], Hkv)
        mem.K[int(mem.pt[0, key // 64]), 0, key % 64, 0] = 2.0 ** 100
        q[:, 1, 0] = 2.0 ** 100
        step = run_attend(q, mem, [0, new], [n], Hkv)
        for x, y in ((step.o, want.o), (step.o_f32, want.o_f32), (step.lse, want.lse)):
            assert torch.isnan(x[:, 1]).all() and torch.equal(x[:, 0], y[:, 0])


# ------------------------------------------------------------------ weights in one or two parts
def check_parts(step, want, keys, d, parts):
    """As check, with weights that are off by 2^-8 (one part) or 2^-15 (two) where they meet V."""
    o, lse, spread, size = want
    live = ~np.isnan(lse)
    e = d * 2.0 ** -23 * size + 2.0 ** -17
    bound = ((2.0 ** -8 if parts == 1 else 2.0 ** -15) + 2 * e + keys * 2.0 ** -23)[..., None] * spread
    off = np.abs(f64(step.o_f32) - o)
    assert (off <= bound)[live].all(), float((off - bound)[live].max())
    check(step, want, keys, d)


@pytest.mark.parametrize("d,G", [(64, 1), (64, 8), (128, 4), (128, 16)])
@pytest.mark.parametrize("parts", [0, 1, 2])
@pytest.mark.parametrize("rows,lens", [([1, 1, 1], [3000, 64, 1]), ([90, 2, 33], [700, 1500, 129])])
def test_weights_in_one_or_two_parts(d, G, parts, rows, lens):
    """Two where a call's rows fill no more than a tile a sequence, unless the caller says."""
    Hkv = 2
    cu = sums(rows)
    mem = Paged(lens, Hkv, d, seed=160)
    q = randn(cu[-1], Hkv * G, d, seed=161, scale=1.5)
    step = run_attend(q, mem, cu, lens, Hkv, p_parts=parts)
    want = exact(q, mem, cu, lens, True, G)
    few = cu[-1] * G <= 128 * len(lens)
    got = parts or (2 if few else 1)
    check_parts(step, want, max(lens), d, got)
    for other in (1, 2):
        same = torch.equal(run_attend(q, mem, cu, lens, Hkv, p_parts=other).o_f32, step.o_f32)
        assert same == (other == got)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,lens", [([40, 1], [5000, 300]), ([200, 90], [700, 2600])])
def test_shared_prefixes_join_parts_of_one_precision(d, rows, lens):
    """As exact as the own parts that bsa_decode gives, where the caller asks for it or the rows
    are few; the own part's weight may be all but nothing, or all."""
    G, Hkv = 4, 2
    cu = sums(rows)
    mem = Paged(lens, Hkv, d, seed=162)
    q = randn(cu[-1], Hkv * G, d, seed=163, scale=1.5)
    own = (torch.randn(cu[-1], Hkv * G, d, generator=gen(164), device="cuda"),
           8.0 + 6.0 * torch.randn(cu[-1], Hkv * G, generator=gen(165), device="cuda"))
    tok = bsa.Tokens(N=cu[-1], B=2, Hq=Hkv * G, Hkv=Hkv, d=d, T=mem.T, cu_seqlens=ints(cu),
                     seq_lens=ints(lens), p_parts=2)
    step = bsa.SharedPrefixDecode(tok)
    step.run(q, *mem.caches(), *own)
    assert int(step.status.item()) == 0
    check_parts(step, exact_shared(q, mem, cu, lens, G, own), max(lens), d, 2)


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,lens,causal", [([1, 1], [5000, 700], True), ([300, 1, 70], [900, 64, 1000], True),
                                              ([17], [333], False), ([130] * 40, [200 + 3 * b for b in range(40)], False),
                                              ([700, 220, 500, 640], [4500, 1500, 2500, 700], True)])
def test_every_row_of_v_counts(parts, d, rows, lens, causal):
    """With q = 0 all weights are 1 and a row's result is the mean of the n values it sees, from
    n / 16 sums of 16 products each, off by 2^-22 at most of the sizes added up (and 20 steps for
    parts and the division): not one key may be missing or counted twice, which is 1 / n."""
    G, Hkv = 4, 2
    cu = sums(rows)
    mem = Paged(lens, Hkv, d, seed=166)
    q = torch.zeros(cu[-1], Hkv * G, d, dtype=torch.bfloat16, device="cuda")
    step = run_attend(q, mem, cu, lens, Hkv, causal, p_parts=parts)
    for b, n in enumerate(lens):
        V = mem.keys(mem.V, b, n)
        total, size = np.cumsum(V, 1), np.cumsum(np.abs(V), 1)
        seen = np.arange(n - rows[b], n) if causal else np.full(rows[b], n - 1)
        mean, size = (np.repeat(x[:, seen].transpose(1, 0, 2), G, 1) / (seen + 1.0)[:, None, None]
                      for x in (total, size))
        off = np.abs(f64(step.o_f32[cu[b]:cu[b + 1]]) - mean)
        assert (off <= (n / 8 + 20) * 2.0 ** -23 * size).all(), float((off / size).max())


# ------------------------------------------------------------------ the plan kernel's own cases
PLAN_KERNEL = [
    # new, lens, Hkv, G, d, causal, the kernel plans, some unit is cut
    ([1] * 32, [1 + 83 * b for b in range(32)], 2, 4, 128, True, False, None),   # 32 tiles
    ([1] * 33, [1 + 83 * b for b in range(33)], 2, 4, 128, True, True, True),    # 33
    ([600], [1500], 49, 1, 64, True, False, None),       # 3 tiles of 49 heads, 147 units, and of 50
    ([600], [1500], 50, 1, 64, True, True, False),
    # 35 tiles of up to 32 tokens, most of them two tiles of rows, over long and short contexts
    ([400, 100, 250, 300], [4500, 1500, 2500, 700], 1, 8, 64, True, True, True),
    ([400, 100, 250, 300], [4500, 1500, 2500, 700], 1, 8, 64, False, True, True),
    ([400, 100, 250, 300], [4500, 1500, 2500, 700], 1, 8, 128, True, True, True),
    ([400, 100, 250, 300], [4500, 1500, 2500, 700], 1, 8, 128, False, True, True),
    # the same between sequences without rows or without tokens, rows of one tile among them
    # (763 rows of 6 sequences make 29 tiles at most, 963 make 35)
    ([0, 333, 7, 0, 420, 1], [900, 3001, 4000, 0, 2111, 77], 2, 8, 128, True, False, None),
    ([0, 433, 7, 0, 520, 1], [900, 3001, 4000, 0, 2111, 77], 2, 8, 128, True, True, True),
]


@pytest.mark.parametrize("new,lens,Hkv,G,d,causal,kernel,cut", PLAN_KERNEL)
def test_the_plan_kernel_cuts_units_of_one_and_two_tiles(new, lens, Hkv, G, d, causal, kernel, cut):
    """Which way a call is planned shows in the first words of its workspace: the plan kernel writes
    the number of entries, and whether a tile has several."""
    assert torch.cuda.get_device_properties(0).multi_processor_count == 148    # what the cases count on
    cu = sums(new)
    mem = Paged(lens, Hkv, d, seed=170)
    q = randn(cu[-1] + 2, Hkv * G, d, seed=171, scale=1.5)
    tok = bsa.Tokens(N=cu[-1] + 2, B=len(lens), Hq=Hkv * G, Hkv=Hkv, d=d, T=mem.T, cu_seqlens=ints(cu),
                     seq_lens=ints(lens), causal=causal)
    step = bsa.PackedAttention(tok)
    step.workspace.fill_(0xff)
    step.o_f32.fill_(77.0)
    step.run(q, *mem.caches())
    entries, _, any_cut, _ = step.workspace[:16].view(torch.int32).tolist()
    assert int(step.status.item()) == 0
    assert (entries != -1) == kernel
    if kernel:
        tiles = sum(-(-n // (256 // G)) for n in new)
        assert any_cut == cut and (entries > tiles) == cut
    assert (step.o_f32[cu[-1]:] == 77.0).all()
    check(step, exact(q, mem, cu, lens, causal, G), max(lens), d)
