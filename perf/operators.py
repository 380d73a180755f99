"""What is measured of the operators around the caches: head norms with rotary positions,
appending to the paged caches, dense causal attention over packed rows, and decode attention
over prefixes that a batch shares.

A case is a plain dict; `prepare` makes its inputs on the GPU, `run` makes one pass (the
library's calls where `own` is true, elementary torch operations in 32 bits elsewhere),
`exact` gives the same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

PAGE = 64
INDEX = 16
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 32 sequences at far positions: latency alone counts
        dict(name="rotate_decode_b32", op="rotate", rows=32, Hq=32, Hkv=8, d=128, type="bf16",
             rot=128, interleaved=False, norm=True, scaled=False, far=131072, split=False),
        # a ragged batch of prompts, half of each head rotated in pairs, fp32 projections
        dict(name="rotate_ragged_pairs_f32", op="rotate", rows=5003, Hq=16, Hkv=2, d=128,
             type="f32", rot=64, interleaved=True, norm=False, scaled=False, far=8192, split=False),
        # the 64K prompt of the block-sparse prefill, written head by head as prefill reads it
        dict(name="rotate_prompt_64k", op="rotate", rows=65536, Hq=32, Hkv=8, d=128, type="bf16",
             rot=128, interleaved=False, norm=True, scaled=True, far=65536, split=True),
        # one new token for each of 32 sequences
        dict(name="append_decode_b32", op="append", B=32, new=1, past=8191, mix=3, Hq=32, Hkv=8,
             d=128, type="bf16", rot=128, interleaved=False, norm=True, scaled=False),
        # packed prompts of all lengths up to 4K, 16-bit floats in, half heads
        dict(name="append_prompts_16k", op="append", B=9, new=4096, past=700, mix=5, Hq=32,
             Hkv=8, d=128, type="f16", rot=128, interleaved=True, norm=False, scaled=True),
        # a handful of short prompts of a small model: the smallest call
        dict(name="attend_short_d64", op="attend", B=5, new=130, past=0, mix=1, Hq=8, Hkv=2, d=64),
        # dense decode of 8 sequences of up to 32K tokens, one token each
        dict(name="attend_decode_32k", op="attend", B=8, new=1, past=32767, mix=2, Hq=32, Hkv=8,
             d=128),
        # chunks of prompts behind what the cache holds already, odd lengths
        dict(name="attend_chunks_ragged", op="attend", B=7, new=2047, past=6001, mix=4, Hq=32,
             Hkv=8, d=128),
        # one whole prompt of 32K
        dict(name="attend_prompt_32k", op="attend", B=1, new=32768, past=0, mix=0, Hq=32, Hkv=8,
             d=128),
        # four sequences behind a system prompt of a thousand tokens
        dict(name="shared_b4_1k", op="shared", rows=4, groups=1, prefix=1003, mix=0, Hq=8, Hkv=2,
             d=64),
        # the decode batch of 32 behind one document of 32K
        dict(name="shared_b32_32k", op="shared", rows=32, groups=1, prefix=32768, mix=0, Hq=32,
             Hkv=8, d=128),
        # 200 sequences behind three documents of up to 64K
        dict(name="shared_b200_3x64k", op="shared", rows=200, groups=3, prefix=65500, mix=7, Hq=64,
             Hkv=8, d=128),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "attend", "attend", "shared"])
    d = rng.choice([64, 128, 128])
    Hkv, G = rng.choice([(1, 8), (2, 4), (4, 16), (8, 1), (8, 2), (8, 4), (4, 8)])
    c = dict(op=op, Hq=Hkv * G, Hkv=Hkv, d=d)
    if op in ("rotate", "append"):
        c.update(type=rng.choice(["bf16", "bf16", "f16", "f32"]), interleaved=rng.random() < 0.4,
                 rot=rng.choice([16, d // 2, d // 2 + 16, d, d]), norm=rng.random() < 0.6,
                 scaled=rng.random() < 0.4)
    if op == "rotate":
        c.update(rows=_spread(rng, 1, 40000), far=_spread(rng, 64, 1 << 20),
                 split=rng.random() < 0.3)
        c["far"] = max(c["far"], c["rows"])
    elif op == "append":
        B = _spread(rng, 1, 48)
        c.update(B=B, new=_spread(rng, 1, max(2, 20000 // B)), past=_spread(rng, 1, 8000),
                 mix=rng.randrange(1000))
    elif op == "attend":
        B = _spread(rng, 1, 24)
        new = _spread(rng, 1, 12000 // B) if rng.random() < 0.7 else 1
        c.update(B=B, new=new, past=_spread(rng, 1, 16000), mix=rng.randrange(1000))
    else:
        c.update(rows=_spread(rng, 2, 200), groups=rng.choice([1, 1, 2, 4]),
                 prefix=_spread(rng, 70, 40000), mix=rng.randrange(1000))
        c["groups"] = min(c["groups"], c["rows"])
    return c


def _lens(case):
    """(new rows, tokens before them) of each sequence: the first has the largest of both."""
    r = random.Random(case["mix"])
    new = [case["new"]] + [r.randint(1, case["new"]) for _ in range(case["B"] - 1)]
    past = [case["past"]] + [r.randint(0, case["past"]) for _ in range(case["B"] - 1)]
    return new, past


def _groups(case):
    """(rows, prefix length) of each group of sequences that share a prefix."""
    r = random.Random(case["mix"])
    n, g = case["rows"], case["groups"]
    cuts = sorted(r.sample(range(1, n), g - 1)) if g > 1 else []
    rows = [b - a for a, b in zip([0] + cuts, cuts + [n])]
    return rows, [case["prefix"]] + [r.randint(1, case["prefix"]) for _ in range(g - 1)]


def _sums(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


# --------------------------------------------------------------------------- inputs
def _frequencies(case):
    """Radians a position of each rotated pair, in 64 bits. `scaled`: the long wavelengths
    (over 8192 positions) turn 8 times more slowly, the short ones (under 2048) as they are,
    those between by a ramp on their number of turns; cos and sin then get a factor."""
    half = case["rot"] // 2
    f = 500000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    if not case["scaled"]:
        return f, 1.0
    turns = 8192.0 * f / (2 * math.pi)
    keep = ((turns - 1.0) / 3.0).clamp(0.0, 1.0)
    return f * keep + f / 8.0 * (1.0 - keep), 0.1 * math.log(8.0) + 1.0


def _steps(f):
    """The same in 2^-64 turns, as the 64-bit integers that the library's calls read."""
    turns = f / (2 * math.pi)
    high = torch.floor(turns * 2.0 ** 32)
    low = torch.floor((turns * 2.0 ** 32 - high) * 2.0 ** 32)
    return high.to(torch.int64) * 2 ** 32 + low.to(torch.int64)


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(generator=g)


def _table(lens, g):
    """A page table [B, widest] of scattered pages, and how many pages there are."""
    blocks = [-(-n // PAGE) for n in lens]
    pages = sum(blocks)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(blocks + [1]), dtype=torch.int32, device="cuda")
    for b, at in enumerate(_sums(blocks)[:-1]):
        table[b, :blocks[b]] = order[at:at + blocks[b]]
    return table, max(pages, 1)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, Hq, Hkv, d = case["op"], case["Hq"], case["Hkv"], case["d"]
    s = dict(case=case)
    if op in ("rotate", "append"):
        f, factor = _frequencies(case)
        s.update(freq=f.cuda(), steps=_steps(f).cuda(), factor=factor)
        s.update({w: 1.0 + 0.2 * _normal(g, d, dtype=torch.float32) if case["norm"] else None
                  for w in ("wq", "wk")})
    if op == "rotate":
        n = case["rows"]
        # q and k lie side by side in the rows of one projection
        s["qkv"] = _normal(g, n, Hq + 2 * Hkv, d, dtype=TYPES[case["type"]]) * 1.7
        start = torch.randint(0, case["far"] - n + 1, (1,), generator=g, device="cuda")
        pos = start + torch.arange(n, device="cuda")
        if n <= 4096:     # a batch: every row at a position of its own
            pos = torch.randint(0, case["far"], (n,), generator=g, device="cuda")
        s["pos"] = pos.to(torch.int32)
        shape = (lambda h: (h, n, d)) if case["split"] else (lambda h: (n, h, d))
        s["q_out"] = torch.empty(shape(Hq), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(shape(Hkv), dtype=torch.bfloat16, device="cuda")
    elif op == "append":
        new, past = _lens(case)
        n = sum(new)
        total = [a + b for a, b in zip(new, past)]
        s["qkv"] = _normal(g, n, Hq + 2 * Hkv, d, dtype=TYPES[case["type"]]) * 1.7
        s["idx"] = _normal(g, n, Hkv, INDEX, dtype=TYPES[case["type"]])
        s["table"], pages = _table(total, g)
        s["K"] = _normal(g, pages, Hkv, PAGE, d)
        s["V"] = _normal(g, pages, Hkv, PAGE, d)
        s["I"] = _normal(g, pages, Hkv, PAGE, INDEX)
        s["cu"], s["total"] = _ints(_sums(new)), _ints(total)
        s["q_out"] = torch.empty(n, Hq, d, dtype=torch.bfloat16, device="cuda")
    elif op == "attend":
        new, past = _lens(case)
        n = sum(new)
        total = [a + b for a, b in zip(new, past)]
        s["q"] = _normal(g, n, Hq, d) * 1.5
        s["table"], pages = _table(total, g)
        s["K"], s["V"] = _normal(g, pages, Hkv, PAGE, d), _normal(g, pages, Hkv, PAGE, d)
        s["K"][:, :, 5] *= 2.0          # a few keys that many rows look at
        s["cu"], s["total"] = _ints(_sums(new)), _ints(total)
        s["lens"] = (new, total)
    else:
        rows, prefix = _groups(case)
        n = sum(rows)
        s["q"] = _normal(g, n, Hq, d) * 1.5
        s["table"], pages = _table(prefix, g)
        s["K"], s["V"] = _normal(g, pages, Hkv, PAGE, d), _normal(g, pages, Hkv, PAGE, d)
        s["K"][:, :, 5] *= 2.0
        # what the attention over each sequence's own tokens gave
        s["o_own"] = _normal(g, n, Hq, d, dtype=torch.float32) * 0.2
        s["lse_own"] = math.log(case["prefix"]) + _normal(g, n, Hq, dtype=torch.float32)
        s["cu"], s["total"] = _ints(_sums(rows)), _ints(prefix)
        s["lens"] = (rows, prefix)
    return s


# ----------------------------------------------------------------------- one pass
def _norm_rope(x, w, s, pos):
    """Plain form of the head norm and the rotation: x [n, H, d]."""
    case = s["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    rot = case["rot"]
    # angles in 64 bits: at far positions 32 bits keep no digit of the fast pairs' turns
    angle = pos.double()[:, None] * s["freq"]
    cos = (torch.cos(angle) * s["factor"]).float()[:, None, :]
    sin = (torch.sin(angle) * s["factor"]).float()[:, None, :]
    out = x.clone()
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return out.to(torch.bfloat16)


def _split(s):
    Hq, Hkv = s["case"]["Hq"], s["case"]["Hkv"]
    return s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]


def _rotate_plain(s):
    q, k, _ = _split(s)
    q, k = _norm_rope(q, s["wq"], s, s["pos"]), _norm_rope(k, s["wk"], s, s["pos"])
    if s["case"]["split"]:
        q, k = q.transpose(0, 1), k.transpose(0, 1)
    s["q_out"].copy_(q)
    s["k_out"].copy_(k)
    return {"q": s["q_out"], "k": s["k_out"]}


def _slots(s):
    """(position, page, row of the page) of every new token, from the lengths."""
    cu, total, n = s["cu"].long(), s["total"].long(), s["qkv"].shape[0]
    row = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    pos = total[b] - cu[b + 1] + row
    return pos, s["table"].long()[b, pos // PAGE], pos % PAGE


def _append_plain(s):
    q, k, v = _split(s)
    pos, page, row = _slots(s)
    s["q_out"].copy_(_norm_rope(q, s["wq"], s, pos))
    s["K"][page, :, row] = _norm_rope(k, s["wk"], s, pos)
    s["V"][page, :, row] = v.to(torch.bfloat16)
    s["I"][page, :, row] = s["idx"].to(torch.bfloat16)
    return {"K": s["K"], "V": s["V"], "I": s["I"], "q": s["q_out"]}


def _keys(s, name, b, n, dtype):
    """The first n tokens of a sequence's cache: [Hkv, n, d]."""
    x = s[name][s["table"][b, :-(-n // PAGE)].long()].to(dtype)
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _attention(q, k, v, first):
    """softmax(q k^T / sqrt(d)) v over the keys 0 .. first + row, or over all (first None), and
    the log of the sums. q [n, Hq, d], k and v [Hkv, m, d]."""
    n, Hq, d = q.shape
    Hkv, m = k.shape[:2]
    q = q.reshape(n, Hkv, Hq // Hkv, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
    x = (q @ k.transpose(1, 2)) * (1.0 / math.sqrt(d))
    if first is not None:
        x = x.reshape(Hkv, -1, n, m)
        limit = first + torch.arange(n, device=q.device)
        x = x.masked_fill(torch.arange(m, device=q.device) > limit[:, None], -math.inf)
        x = x.reshape(Hkv, -1, m)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    o, lse = (x @ v) / total, top + torch.log(total)
    back = (lambda y: y.reshape(Hkv, Hq // Hkv, n, -1).permute(2, 0, 1, 3).reshape(n, Hq, -1))
    return back(o), back(lse)[..., 0]


def _attend(s, dtype, rows):
    """All sequences in turn, `rows` query rows at a time (the scores of all would not fit)."""
    o, lse = [], []
    new, total = s["lens"]
    for b, at in enumerate(_sums(new)[:-1]):
        k, v = _keys(s, "K", b, total[b], dtype), _keys(s, "V", b, total[b], dtype)
        for r in range(0, new[b], rows):
            n = min(rows, new[b] - r)
            first = total[b] - new[b] + r
            x = _attention(s["q"][at + r:at + r + n].to(dtype), k[:, :first + n],
                           v[:, :first + n], first)
            o.append(x[0])
            lse.append(x[1])
    return torch.cat(o), torch.cat(lse)


def _shared(s, dtype, merge):
    o, lse = [], []
    rows, prefix = s["lens"]
    for b, at in enumerate(_sums(rows)[:-1]):
        k, v = _keys(s, "K", b, prefix[b], dtype), _keys(s, "V", b, prefix[b], dtype)
        x = _attention(s["q"][at:at + rows[b]].to(dtype), k, v, None)
        o.append(x[0])
        lse.append(x[1])
    return merge(torch.cat(o), torch.cat(lse), s["o_own"].to(dtype), s["lse_own"].to(dtype))


def _merge(o, lse, o_own, lse_own):
    top = torch.maximum(lse, lse_own)
    a, b = torch.exp(lse - top), torch.exp(lse_own - top)
    both = (a[..., None] * o + b[..., None] * o_own) / (a + b)[..., None]
    return both, top + torch.log(a + b)


def _handle(s):
    """What a program keeps beside its inputs: the problem's description, outputs, workspace."""
    if "handle" not in s:
        import block_sparse_long_06_b200 as bsa
        case = s["case"]
        op, Hq, Hkv, d = case["op"], case["Hq"], case["Hkv"], case["d"]
        if op in ("rotate", "append"):
            rope = bsa.Rope(s["steps"], interleaved=case["interleaved"], factor=s["factor"])
            q, k, v = _split(s)
            more = dict(rope=rope, norm=case["norm"], eps=EPS, q_weight=s["wq"], k_weight=s["wk"])
        if op == "rotate":
            n = case["rows"]
            tok = bsa.Tokens(N=n, B=1, Hq=Hq, Hkv=Hkv, d=d, T=case["far"], positions=s["pos"],
                             **more)
            out = [x.transpose(0, 1) if case["split"] else x for x in (s["q_out"], s["k_out"])]
            s["handle"] = (bsa, tok, q, k, *out)
        elif op == "append":
            T = s["table"].shape[1] * PAGE
            tok = bsa.Tokens(N=s["qkv"].shape[0], B=case["B"], Hq=Hq, Hkv=Hkv, d=d, T=T,
                             cu_seqlens=s["cu"], seq_lens=s["total"], **more)
            caches = [bsa.paged_cache(s[x], s["table"]) for x in "KVI"]
            s["handle"] = (bsa, tok, q, k, v, *caches)
        else:
            tok = bsa.Tokens(N=s["q"].shape[0], B=len(s["lens"][0]), Hq=Hq, Hkv=Hkv, d=d,
                             T=s["table"].shape[1] * PAGE, cu_seqlens=s["cu"],
                             seq_lens=s["total"], causal=op == "attend")
            make = bsa.PackedAttention if op == "attend" else bsa.SharedPrefixDecode
            caches = [bsa.paged_cache(s[x], s["table"]) for x in "KV"]
            s["handle"] = (make(tok, keep_f32=False), *caches)
    return s["handle"]


def _run_own(s):
    op, h = s["case"]["op"], _handle(s)
    if op == "rotate":
        bsa, tok, q, k, q_out, k_out = h
        bsa.bsa_norm_rope(tok, q, q_out, k, k_out)
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        bsa, tok, q, k, v, K, V, I = h
        bsa.bsa_append_kv(tok, k, v, K, V, k_idx=s["idx"], kidx_cache=I, q=q, q_out=s["q_out"])
        return {"K": s["K"], "V": s["V"], "I": s["I"], "q": s["q_out"]}
    step, K, V = h
    if op == "attend":
        step.run(s["q"], K, V)
    else:
        step.run(s["q"], K, V, s["o_own"], s["lse_own"])
    return {"o": step.o, "lse": step.lse}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "rotate":
        return _rotate_plain(state)
    if op == "append":
        return _append_plain(state)
    o, lse = (_attend(state, torch.float32, 1024) if op == "attend"
              else _shared(state, torch.float32, _merge))
    return {"o": o.to(torch.bfloat16), "lse": lse}


# --------------------------------------------------------------------------- work
def work(case):
    op, Hq, Hkv, d = case["op"], case["Hq"], case["Hkv"], case["d"]
    if op in ("rotate", "append"):
        size = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
        if op == "rotate":
            n, wide = case["rows"], (Hq + Hkv) * d
        else:
            n, wide = sum(_lens(case)[0]), (Hq + 2 * Hkv) * d + Hkv * INDEX
        return {"bytes": n * wide * (size + 2) + 4 * n, "flops": 6 * n * (Hq + Hkv) * d}
    if op == "attend":
        new, past = _lens(case)
        keys = sum(a + b for a, b in zip(new, past))
        pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, past))
        n, own_part = sum(new), 0
    else:
        rows, prefix = _groups(case)
        keys, pairs = sum(prefix), sum(a * b for a, b in zip(rows, prefix))
        n = sum(rows)
        own_part = n * Hq * (4 * d + 4)
    return {"bytes": 4 * keys * Hkv * d + n * Hq * (4 * d + 4) + own_part,
            "flops": 4 * pairs * Hq * d}


# -------------------------------------------------------------------- in 64 bits
def _turned(x, w, s, pos):
    """Head norm and rotation of x [n, H, d] in 64 bits, as products of complex numbers."""
    case = s["case"]
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    rot = case["rot"]
    head, tail = x[..., :rot], x[..., rot:]
    n, H = x.shape[:2]
    pair = (head.reshape(n, H, rot // 2, 2) if case["interleaved"]
            else head.reshape(n, H, 2, rot // 2).transpose(2, 3)).contiguous()
    turn = torch.polar(torch.full_like(s["freq"], s["factor"]).expand(n, -1).contiguous(),
                       torch.outer(pos.double(), s["freq"]))
    pair = torch.view_as_real(torch.view_as_complex(pair) * turn[:, None])
    head = (pair if case["interleaved"] else pair.transpose(2, 3)).reshape(n, H, rot)
    return torch.cat([head, tail], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, Hq, Hkv = case["op"], case["Hq"], case["Hkv"]
    if op == "rotate":
        q = _turned(s["qkv"][:, :Hq], s["wq"], s, s["pos"])
        k = _turned(s["qkv"][:, Hq:Hq + Hkv], s["wk"], s, s["pos"])
        return {"q": q.transpose(0, 1) if case["split"] else q,
                "k": k.transpose(0, 1) if case["split"] else k}
    if op == "append":
        new, past = _lens(case)
        pos = torch.cat([torch.arange(p, p + n) for n, p in zip(new, past)]).cuda()
        seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)]).cuda()
        page = s["table"][seq, pos // PAGE].long()
        out = {name: s[name].double() for name in "KVI"}
        out["K"][page, :, pos % PAGE] = _turned(s["qkv"][:, Hq:Hq + Hkv], s["wk"], s, pos)
        out["V"][page, :, pos % PAGE] = s["qkv"][:, Hq + Hkv:].double()
        out["I"][page, :, pos % PAGE] = s["idx"].double()
        out["q"] = _turned(s["qkv"][:, :Hq], s["wq"], s, pos)
        return out
    return _exact_attention(case, s)


def _exact_attention(case, s):
    """One head at a time: probabilities from torch's softmax in 64 bits; a sequence's own part
    (shared prefixes) is one more key, whose score is its log-sum and whose value its output."""
    op, d, G = case["op"], case["d"], case["Hq"] // case["Hkv"]
    rows, total = _lens(case) if op == "attend" else _groups(case)
    if op == "attend":
        total = [a + b for a, b in zip(rows, total)]
    n = sum(rows)
    o = torch.empty(n, case["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.empty(n, case["Hq"], dtype=torch.float64, device="cuda")
    at = 0
    for b, count in enumerate(rows):
        m = total[b]
        page = s["table"][b, :-(-m // PAGE)].long()
        for h in range(case["Hq"]):
            k = s["K"][page, h // G].reshape(-1, d)[:m].double()
            v = s["V"][page, h // G].reshape(-1, d)[:m].double()
            for r in range(0, count, 4096):
                i = slice(at + r, at + min(r + 4096, count))
                x = s["q"][i, h].double() @ k.T / math.sqrt(d)
                if op == "attend":
                    limit = torch.arange(m - count + r, m - count + r + x.shape[0], device="cuda")
                    x[torch.arange(m, device="cuda")[None, :] > limit[:, None]] = -math.inf
                    o[i, h], lse[i, h] = torch.softmax(x, -1) @ v, torch.logsumexp(x, -1)
                else:
                    x = torch.cat([x, s["lse_own"][i, h, None].double()], 1)
                    p = torch.softmax(x, -1)
                    o[i, h] = p[:, :-1] @ v + p[:, -1:] * s["o_own"][i, h].double()
                    lse[i, h] = torch.logsumexp(x, -1)
        at += count
    return {"o": o, "lse": lse}
