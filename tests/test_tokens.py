"""Operators around the caches, on the CPU: rotary tables against 64-bit angles, the oracle's
pins, and the arguments that the entry points refuse before any launch."""
import copy
import ctypes
import math
import pickle

import numpy as np
import pytest
import torch

import block_sparse_long_06_b200 as bsa
from oracle import tokens_oracle as TO


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(bsa.LIB_PATH):
        from block_sparse_long_06_b200 import build
        build.build()
    return bsa.load_library()


# ------------------------------------------------------------------ rotary tables
@pytest.mark.parametrize("dim,theta,scaling", [
    (64, 10000.0, dict()), (128, 500000.0, dict(scaling="linear", factor=4.0)),
    (128, 10000.0, dict(scaling="ntk", factor=8.0)),
    (128, 500000.0, dict(scaling="ramp", factor=16.0, original=4096))])
def test_rope_steps_give_the_angle_at_far_positions(dim, theta, scaling):
    f, _ = bsa.rope_frequencies(dim, theta, **scaling)
    steps = bsa.rope_steps(f)
    for pos in (0, 1, 12345, 1 << 20, (1 << 21) - 1, -7):
        for i in (0, 1, dim // 4, dim // 2 - 1):
            turns = (pos * int(steps[i])) % 2 ** 64 / 2.0 ** 64
            from fractions import Fraction
            want = Fraction(float(f[i])) * pos / Fraction(2 * math.pi)
            want = float(want - math.floor(want))
            off = abs(turns - want)
            # the step is 2^-53 of itself off (64-bit frequency), the product pos times that
            assert min(off, 1 - off) <= abs(pos) * 2.0 ** -54 + 2.0 ** -52


def test_rope_scalings():
    base, one = bsa.rope_frequencies(64, 10000.0)
    assert one == 1.0 and base[0] == 1.0
    f, _ = bsa.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert torch.equal(f, base / 4)
    f, _ = bsa.rope_frequencies(64, 10000.0, "ntk", 4.0)
    assert f[0] == 1.0 and math.isclose(float(f[-1]), float(base[-1]) / 4, rel_tol=1e-12)
    f, factor = bsa.rope_frequencies(64, 10000.0, "ramp", 4.0, original=4096, low=1.0, high=32.0)
    turns = 4096 * base / (2 * math.pi)
    assert torch.equal(f[turns >= 32], base[turns >= 32])
    assert torch.equal(f[turns <= 1], base[turns <= 1] / 4)
    assert math.isclose(factor, 0.1 * math.log(4.0) + 1.0)
    for bad in (dict(dim=63), dict(dim=64, theta=0.0), dict(dim=64, factor=0.5),
                dict(dim=64, scaling="no"), dict(dim=64, scaling="ramp", low=2.0, high=2.0)):
        with pytest.raises(bsa.BsaError):
            bsa.rope_frequencies(**bad)


# ------------------------------------------------------------------ the oracle's pins
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_is_complex_multiplication(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 24))
    f = 100.0 ** -(np.arange(8) / 8)
    pos = np.array([0, 1, 2, 77, -3])
    y, _ = TO.norm_rope(x, pos, f, interleaved, 1.25)
    z = (x[..., 0:16:2] + 1j * x[..., 1:16:2]) if interleaved else (x[..., :8] + 1j * x[..., 8:16])
    z = z * 1.25 * np.exp(1j * pos[:, None] * f)[:, None, :]
    got = (y[..., 0:16:2] + 1j * y[..., 1:16:2]) if interleaved else (y[..., :8] + 1j * y[..., 8:16])
    assert np.allclose(got, z, atol=1e-13)
    assert np.array_equal(y[..., 16:], x[..., 16:])


def test_oracle_norm_attention_and_merge():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 2, 16))
    y, _ = TO.norm_rope(x, np.zeros(4), weight=np.full(16, 2.0), norm=True)
    assert np.allclose((y ** 2).mean(-1), 4.0)
    q, K, V = rng.standard_normal((3, 8)), rng.standard_normal((20, 8)), rng.standard_normal((20, 8))
    vis = np.arange(20) < np.array([13, 20, 6])[:, None]
    o, lse, spread, size = TO.attend_rows(q, K, V, 0.3, vis)
    t = torch.nn.functional.scaled_dot_product_attention(
        torch.tensor(q)[None], torch.tensor(K)[None], torch.tensor(V)[None], scale=0.3,
        attn_mask=torch.tensor(vis)[None])
    assert np.allclose(o, t.numpy()[0])
    assert np.allclose(np.exp(lse), (np.exp(q @ K.T * 0.3) * vis).sum(1))
    assert (spread >= np.abs(o) - 1e-12).all() and (size > 0).all()
    early = np.arange(20) < 5
    a, b = (TO.attend_rows(q, K, V, 0.3, vis & x)[:2] for x in (early, ~early))
    om, lm, wa, wb = TO.merge(*a, *b)
    assert np.allclose(om, o) and np.allclose(lm, lse) and np.allclose(wa + wb, 1.0)
    om, lm, _, _ = TO.merge(*a, np.full((3, 8), np.nan), np.full(3, -np.inf))
    assert np.allclose(om, a[0]) and np.allclose(lm, a[1])
    K[19] = np.nan                                 # a key that nobody sees
    o2 = TO.attend_rows(q[::2], K, V, 0.3, vis[::2])[0]
    assert np.allclose(o2, o[::2])
    o, lse, _, _ = TO.attend_rows(q, K, V, 0.3, np.zeros((3, 20), bool))
    assert (lse == -np.inf).all() and not o.any()
    om, lm, _, _ = TO.merge(o, lse, o, lse)
    assert (lm == -np.inf).all() and not om.any()


def test_row_tokens():
    assert TO.row_tokens([0, 2, 2, 3], [5, 9, 1], 5) == [(0, 3), (0, 4), (2, 0), (-1, -1), (-1, -1)]


# ------------------------------------------------------------------ refusals
def tokens(**kw):
    base = dict(N=4, B=2, Hq=8, Hkv=2, d=128, r=16, block=64, T=256, cu_seqlens=0x1000,
                seq_lens=0x2000, rope_steps=0x3000, rope_dim=128, rope_factor=1.0, norm=1,
                eps=1e-6, causal=1)
    base.update(kw)
    t = bsa.CTokens()
    for name, v in base.items():
        setattr(t, name, v)
    return t


def rows(base=0x10000, ts=1024, hs=128, kind=0):
    return bsa.CRows(base, ts, hs, kind)


def cache(base=0x40000, width=128, T=256, **kw):
    c = bsa.CCache(base, 2 * T * width, 64 * width, T * width, None, 0, 0, 2 * 2 * T * width)
    for name, v in kw.items():
        setattr(c, name, v)
    return c


NONE = bsa.CRows(None, 0, 0, 0)

BAD_TOKENS = [
    (dict(N=-1), bsa.BSA_ERR_INVALID_ARG), (dict(B=0), bsa.BSA_ERR_INVALID_ARG),
    (dict(Hq=7), bsa.BSA_ERR_INVALID_ARG), (dict(T=-1), bsa.BSA_ERR_INVALID_ARG),
    (dict(N=5, cu_seqlens=None), bsa.BSA_ERR_INVALID_ARG),
    (dict(rope_factor=float("inf")), bsa.BSA_ERR_INVALID_ARG),
    (dict(eps=-1.0), bsa.BSA_ERR_INVALID_ARG), (dict(norm=2), bsa.BSA_ERR_INVALID_ARG),
    (dict(rope_interleaved=3), bsa.BSA_ERR_INVALID_ARG),
    (dict(rope_dim=-16), bsa.BSA_ERR_INVALID_ARG), (dict(rope_dim=144), bsa.BSA_ERR_INVALID_ARG),
    (dict(rope_steps=None), bsa.BSA_ERR_INVALID_ARG), (dict(causal=2), bsa.BSA_ERR_INVALID_ARG),
    (dict(q_stride=4), bsa.BSA_ERR_INVALID_ARG), (dict(attn_scale=-1.0), bsa.BSA_ERR_INVALID_ARG),
    (dict(block=32), bsa.BSA_ERR_UNSUPPORTED), (dict(r=8), bsa.BSA_ERR_UNSUPPORTED),
    (dict(d=96, rope_dim=96), bsa.BSA_ERR_UNSUPPORTED),
    (dict(rope_dim=24), bsa.BSA_ERR_UNSUPPORTED), (dict(T=64 * 32769), bsa.BSA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_TOKENS)
def test_bad_token_problems_are_refused(lib, kw, code):
    t = ctypes.byref(tokens(**kw))
    assert lib.bsa_norm_rope(t, rows(), rows(0x20000), NONE, NONE, None, None) == code
    assert lib.bsa_append_kv(t, rows(), rows(), NONE, cache(), cache(), bsa.CCache(), NONE, NONE,
                             None, None) == code
    assert lib.bsa_attend_packed(t, 0x10000, cache(), cache(), 0x20000, 0x30000, None, 0x100000,
                                 1 << 40, None, None) == code
    out = ctypes.c_size_t(0)
    assert lib.bsa_packed_workspace_size(t, bsa.OP_ATTEND_PACKED, ctypes.byref(out)) == code


def test_bad_rows_are_refused(lib):
    t = ctypes.byref(tokens())
    E = bsa.BSA_ERR_INVALID_ARG
    call = lib.bsa_norm_rope
    assert call(t, NONE, NONE, NONE, NONE, None, None) == E
    for bad in (rows(0x10008), rows(ts=1020), rows(hs=4), rows(kind=3), rows(ts=-8)):
        assert call(t, bad, rows(0x20000), NONE, NONE, None, None) == E
        assert call(t, NONE, NONE, bad, rows(0x20000), None, None) == E
        assert lib.bsa_append_kv(t, bad, rows(), NONE, cache(), cache(), bsa.CCache(), NONE, NONE,
                                 None, None) == E
    assert call(t, rows(), NONE, NONE, NONE, None, None) == E               # no output
    assert call(t, rows(), rows(0x20000, kind=2), NONE, NONE, None, None) == E   # outputs are bf16
    assert call(t, rows(), rows(0x20000), rows(kind=1), rows(0x30000), None, None) == E  # two types
    assert call(t, rows(), rows(ts=2048), NONE, NONE, None, None) == E      # in place, other rows
    assert call(t, rows(kind=2), rows(), NONE, NONE, None, None) == E       # in place, other type
    for bad in (rows(0x20000, ts=0), rows(0x20000, hs=0), rows(0x20000, hs=64)):   # heads overlap
        assert call(t, rows(), bad, NONE, NONE, None, None) == E
    app = lib.bsa_append_kv
    assert app(t, rows(), rows(kind=1), NONE, cache(), cache(), bsa.CCache(), NONE, NONE, None,
               None) == E
    for bad in (cache(None), cache(0x40008), cache(block_stride=0), cache(head_stride=64),
                cache(page_table=0x5000, num_pages=0), cache(page_table=0x5000, num_pages=9,
                                                             page_table_stride=3), cache(extent=0)):
        assert app(t, rows(), rows(), NONE, bad, cache(), bsa.CCache(), NONE, NONE, None, None) == E
        assert app(t, rows(), rows(), NONE, cache(), bad, bsa.CCache(), NONE, NONE, None, None) == E
        assert lib.bsa_attend_packed(t, 0x10000, cache(), bad, 0x20000, 0x30000, None, 0x100000,
                                     1 << 40, None, None) == E
    assert app(t, rows(), rows(), rows(), cache(), cache(), bsa.CCache(), NONE, NONE, None,
               None) == E                                                   # index keys, no cache


def test_packed_calls_refuse(lib):
    t = ctypes.byref(tokens())
    E = bsa.BSA_ERR_INVALID_ARG
    att, sh = lib.bsa_attend_packed, lib.bsa_decode_shared
    ok = (0x20000, 0x30000, None)
    for q, o, lse, f32 in ((None, *ok), (0x10008, *ok), (0x10000, None, 0x30000, None),
                           (0x10000, 0x20008, 0x30000, None), (0x10000, 0x20000, None, None),
                           (0x10000, 0x20000, 0x30000, 0x50004)):
        assert att(t, q, cache(), cache(), o, lse, f32, 0x100000, 1 << 40, None, None) == E
        assert sh(t, q, cache(), cache(), None, None, o, lse, f32, 0x100000, 1 << 40, None,
                  None) == E
    assert sh(t, 0x10000, cache(), cache(), 0x60000, None, *ok, 0x100000, 1 << 40, None, None) == E
    assert att(ctypes.byref(tokens(q_stride=512)), 0x10000, cache(), cache(), *ok, 0x100000,
               1 << 40, None, None) == E                                    # rows overlap
    assert att(ctypes.byref(tokens(Hq=6)), 0x10000, cache(), cache(), *ok, 0x100000, 1 << 40, None,
               None) == bsa.BSA_ERR_UNSUPPORTED                             # G = 3
    for ws, n in ((None, 1 << 40), (0x100080, 1 << 40), (0x100000, 64)):
        assert att(t, 0x10000, cache(), cache(), *ok, ws, n, None, None) == bsa.BSA_ERR_WORKSPACE
    assert att(t, 0x10000, cache(extent=(1 << 31) * 128), cache(), *ok, 0x100000, 1 << 40, None,
               None) == bsa.BSA_ERR_UNSUPPORTED


def test_no_rows_is_nothing_to_do(lib):
    t = ctypes.byref(tokens(N=0))
    assert lib.bsa_norm_rope(t, NONE, NONE, NONE, NONE, None, None) == 0
    assert lib.bsa_append_kv(t, NONE, NONE, NONE, bsa.CCache(), bsa.CCache(), bsa.CCache(), NONE,
                             NONE, None, None) == 0
    assert lib.bsa_attend_packed(t, None, bsa.CCache(), bsa.CCache(), None, None, None, None, 0,
                                 None, None) == 0


def test_workspace_sizes(lib):
    def size(op=bsa.OP_ATTEND_PACKED, **kw):
        out = ctypes.c_size_t(0)
        assert lib.bsa_packed_workspace_size(ctypes.byref(tokens(**kw)), op, ctypes.byref(out)) == 0
        return out.value
    big = size(N=65536, B=1, Hq=32, Hkv=8, T=65536)
    assert big < 1 << 20                       # enough units: no splits, no partial results
    assert size(N=1, B=1, Hq=32, Hkv=8, T=65536) < 2 << 20
    # a row's own part is joined where the row is written: no more for shared prefixes
    assert size(op=bsa.OP_DECODE_SHARED, N=65536, B=1, Hq=32, Hkv=8, T=65536) == big
    out = ctypes.c_size_t(0)
    assert lib.bsa_packed_workspace_size(ctypes.byref(tokens()), bsa.OP_DECODE,
                                         ctypes.byref(out)) == bsa.BSA_ERR_INVALID_ARG


def test_python_checks_raise_before_the_library():
    tok = bsa.Tokens(N=2, B=2, Hq=4, Hkv=2, d=64, T=64)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(bsa.BsaError):
        bsa.bsa_norm_rope(tok, q, q)                        # not on the GPU
    with pytest.raises(bsa.BsaError):
        bsa.bsa_norm_rope(tok, None, None)
    with pytest.raises(bsa.BsaError):
        bsa.bsa_norm_rope(tok, q, None)
    with pytest.raises(bsa.BsaError):
        bsa.bsa_norm_rope(tok, q[:1], q[:1])
    with pytest.raises(bsa.BsaError):
        bsa.bsa_norm_rope(tok, q.double(), q)
    with pytest.raises(bsa.BsaError):
        bsa.Tokens(N=2, B=2, Hq=4, Hkv=2, d=64, T=64,
                   seq_lens=torch.zeros(2, dtype=torch.int64)).c()


# ------------------------------------------------------------------ queries of the binding
def test_queries_whose_rows_overlap_are_refused():
    """A stride of 0 would be taken for the default, rows behind the buffer's end for queries."""
    tok = bsa.Tokens(N=3, B=3, Hq=4, Hkv=2, d=64, T=64)
    one = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    close = torch.zeros(2 * 128 + 256, dtype=torch.bfloat16).as_strided((3, 4, 64), (128, 64, 1))
    c = bsa.contiguous_cache(torch.zeros(3, 2, 64, 64, dtype=torch.bfloat16))
    for call in (lambda q: bsa.bsa_attend_packed(tok, q, c, c, None, None, None, None),
                 lambda q: bsa.bsa_decode_shared(tok, q, c, c, None, None, None, None, None, None)):
        for q in (one.expand(3, 4, 64), close):
            with pytest.raises(bsa.BsaError, match="overlap"):
                call(q)
        for q in (torch.zeros(3, 4, 64, dtype=torch.bfloat16),
                  torch.zeros(3, 8, 64, dtype=torch.bfloat16)[:, 2:6]):
            with pytest.raises(bsa.BsaError, match="GPU"):
                call(q)


# ------------------------------------------------------------------ structs of the binding
def test_described_caches_and_tokens_can_be_copied():
    pool = torch.zeros(3, 2, 64, 16, dtype=torch.bfloat16)
    c = bsa.paged_cache(pool, torch.zeros(2, 4, dtype=torch.int32))
    tok = bsa.Tokens(N=2, B=2, Hq=4, Hkv=2, d=64, T=64, eps=0.5)
    before = bytes(c.c()), bytes(tok.c())
    for one in (copy.deepcopy(c), copy.copy(c), pickle.loads(pickle.dumps(c))):
        struct = one.c()
        assert struct.base == one.tensor.data_ptr()
        assert struct.page_table == one.page_table.data_ptr() and struct.page_table_stride == 4
    for one in (copy.deepcopy(tok), copy.copy(tok), pickle.loads(pickle.dumps(tok))):
        one.N = 1
        assert one.c().N == 1 and one.c().eps == 0.5
    assert (bytes(c.c()), bytes(tok.c())) == before


def test_structs_are_the_callers_own():
    c = bsa.contiguous_cache(torch.zeros(1, 2, 64, 16, dtype=torch.bfloat16))
    tok = bsa.Tokens(N=2, B=2, Hq=4, Hkv=2, d=64, T=64)
    for what, name in ((c, "extent"), (tok, "N")):
        one, other = what.c(), what.c()
        setattr(one, name, 1 << 20)
        assert getattr(other, name) == getattr(what.c(), name) != 1 << 20


def test_sizes_follow_tensors_changed_in_place():
    pool, table = torch.zeros(8, 2, 64, 16, dtype=torch.bfloat16), torch.zeros(2, 6, dtype=torch.int32)
    c = bsa.paged_cache(pool, table)
    for struct in (c.c, c._struct):
        assert struct().extent == pool.numel() and struct().page_table_stride == 6
    pool.resize_(3, 2, 64, 16)
    table.resize_(2, 3)
    for struct in (c.c, c._struct):
        assert struct().extent == 3 * 2 * 64 * 16 and struct().page_table_stride == 3
    c.tensor.data = torch.zeros(1, 2, 64, 16, dtype=torch.bfloat16)
    assert c._struct().extent == 2 * 64 * 16 and c._struct().base == c.tensor.data_ptr()


def test_lengths_changed_in_place_are_checked_again(monkeypatch):
    monkeypatch.setattr(bsa, "_on_gpu", lambda t: True)
    lens = torch.zeros(2, dtype=torch.int32)
    tok = bsa.Tokens(N=2, B=2, Hq=4, Hkv=2, d=64, T=64, seq_lens=lens)
    assert tok.c().seq_lens == lens.data_ptr()
    lens.resize_(1)
    with pytest.raises(bsa.BsaError, match="seq_lens"):
        tok.c()


# ------------------------------------------------------------------ what is written, once
def test_outputs_whose_rows_overlap_are_refused(lib):
    """Head h + 1 of a row may not be head h of the next, in no order of rows and heads."""
    E = bsa.BSA_ERR_INVALID_ARG
    two = lambda **kw: ctypes.byref(tokens(**kw))           # N = 4 rows, 8 and 2 heads, d = 128
    for bad in (rows(0x20000, ts=128, hs=128), rows(0x20000, ts=1016, hs=128),
                rows(0x20000, ts=128, hs=504), rows(0x20000, ts=256, hs=128)):
        assert lib.bsa_norm_rope(two(), rows(), bad, NONE, NONE, None, None) == E
        assert lib.bsa_append_kv(two(), rows(), rows(), NONE, cache(), cache(), bsa.CCache(),
                                 rows(), bad, None, None) == E
    assert lib.bsa_norm_rope(two(), NONE, NONE, rows(), rows(0x20000, ts=128, hs=128), None,
                             None) == E


W, T = 128, 200                                  # B = 2, Hkv = 2
LAYOUTS = [
    # (fits, cache fields): head by head, of T tokens or more
    (True, dict(T=T)), (True, dict(T=256)), (False, dict(T=100)), (False, dict(T=199)),
    # block by block, heads inside
    (True, dict(block_stride=2 * 64 * W, head_stride=64 * W, seq_stride=8 * 64 * W)),
    (False, dict(block_stride=2 * 64 * W, head_stride=64 * W, seq_stride=7 * 64 * W)),
    (False, dict(block_stride=2 * 64 * W, head_stride=63 * W, seq_stride=8 * 64 * W)),
    # sequence inside head
    (True, dict(block_stride=64 * W, seq_stride=T * W, head_stride=2 * T * W)),
    (False, dict(block_stride=64 * W, seq_stride=T * W, head_stride=T * W)),
    (False, dict(seq_stride=0, T=T)), (False, dict(block_stride=63 * W, T=T)),
    # pages: sequences share the pool, unless they have one each
    (True, dict(page_table=0x5000, page_table_stride=4, num_pages=9, seq_stride=0,
                block_stride=2 * 64 * W, head_stride=64 * W)),
    (True, dict(page_table=0x5000, page_table_stride=4, num_pages=9, seq_stride=0,
                block_stride=64 * W, head_stride=9 * 64 * W)),
    (False, dict(page_table=0x5000, page_table_stride=4, num_pages=9, seq_stride=0,
                 block_stride=64 * W, head_stride=64 * W)),
    (False, dict(page_table=0x5000, page_table_stride=4, num_pages=9, seq_stride=8 * 2 * 64 * W,
                 block_stride=2 * 64 * W, head_stride=64 * W)),
]


@pytest.mark.parametrize("fits,kw", LAYOUTS)
def test_appends_go_into_caches_whose_slots_are_apart(lib, fits, kw):
    """A token of the capacity T behind the end of its head's rows would overwrite the next
    head's. Where K's layout is fine, V's size is what is refused."""
    large = cache(extent=(1 << 31) * 128, T=256)
    k = cache(extent=1 << 30, **kw)
    t = ctypes.byref(tokens(T=T))
    got = lib.bsa_append_kv(t, rows(), rows(), NONE, k, large, bsa.CCache(), NONE, NONE, None, None)
    assert got == (bsa.BSA_ERR_UNSUPPORTED if fits else bsa.BSA_ERR_INVALID_ARG)


def test_appends_check_values_and_index_keys_too(lib):
    app, E = lib.bsa_append_kv, bsa.BSA_ERR_INVALID_ARG
    t = ctypes.byref(tokens(T=T))
    good, short = cache(T=256), cache(T=100, extent=1 << 30)
    assert app(t, rows(), rows(), NONE, good, short, bsa.CCache(), NONE, NONE, None, None) == E
    assert app(t, rows(), rows(), rows(), good, good, cache(width=16, T=100, extent=1 << 30), NONE,
               NONE, None, None) == E
    # capacity 0 has no slots, one sequence and one head no neighbours
    large = cache(extent=(1 << 31) * 128)
    for kw in (dict(T=0), dict(B=1, N=4, Hkv=1, Hq=8, T=256)):
        assert app(ctypes.byref(tokens(**kw)), rows(), rows(), NONE, cache(T=64, head_stride=0, seq_stride=0,
                   extent=1 << 20), large, bsa.CCache(), NONE, NONE, None,
                   None) == bsa.BSA_ERR_UNSUPPORTED


def test_page_tables_are_checked_before_a_call(monkeypatch):
    """A table of too few rows, of another type or with rows apart would be read past its end or
    as other pages."""
    seen = []
    monkeypatch.setattr(bsa, "_launch", lambda fn, what, dev, *args: seen.append(what))
    monkeypatch.setattr(bsa, "_rows", lambda *a: None)
    monkeypatch.setattr(bsa, "_raw_stream", lambda *a: 0)
    pool = torch.zeros(5, 2, 64, 64, dtype=torch.bfloat16)
    idx = torch.zeros(5, 2, 64, 16, dtype=torch.bfloat16)
    table = torch.zeros(3, 4, dtype=torch.int32)
    tok = bsa.Tokens(N=3, B=3, Hq=4, Hkv=2, d=64, T=256)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)

    def make(pool, t):
        c = bsa.paged_cache(pool, table)
        c.page_table = t
        return c

    append = lambda k, v, i: bsa.bsa_append_kv(tok, x, x, make(pool, k), make(pool, v), x,
                                               make(idx, i))
    append(table, table, table)
    append(torch.zeros(4, 4, dtype=torch.int32), table, table)
    assert seen == ["bsa_append_kv"] * 2
    for bad in (table[:2], table.long(), torch.zeros(3, 8, dtype=torch.int32)[:, :4], table[0],
                table[:, :3].contiguous()):
        for three in ((bad, table, table), (table, bad, table), (table, table, bad)):
            with pytest.raises(bsa.BsaError, match="page table"):
                append(*three)
    for bad in (table[:2], table.long()):       # the attention calls' caches go the same way
        for two in ((bad, table), (table, bad)):
            with pytest.raises(bsa.BsaError, match="page table"):
                bsa._structs(tok, -1, *(make(pool, t) for t in two))


@pytest.mark.parametrize("parts", [-1, 3])
def test_parts_of_a_weight_are_one_or_two(lib, parts):
    assert lib.bsa_attend_packed(ctypes.byref(tokens(p_parts=parts)), 0x10000, cache(), cache(), 0x20000,
                                 0x30000, None, 0x100000, 1 << 40, None, None) == bsa.BSA_ERR_INVALID_ARG
