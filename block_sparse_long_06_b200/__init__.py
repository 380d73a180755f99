"""Python binding of libbsa.so: dynamic block-sparse attention on B200 (sm_100a).

Thin ctypes marshalling over the C ABI in include/bsa.h. Every step of the method
runs in the library's CUDA kernels; torch only owns device memory and streams.
Importing this package does not load the library; the first call does, and it
raises if libbsa.so is missing (build it with ``python -m
block_sparse_long_06_b200.build``). There is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsa.so")

BSA_OK, BSA_ERR_INVALID_ARG, BSA_ERR_UNSUPPORTED, BSA_ERR_WORKSPACE, BSA_ERR_CUDA = range(5)
BSA_DEV_BAD_PAGE, BSA_DEV_BAD_KEPT, BSA_DEV_NONFINITE, BSA_DEV_TIMEOUT, BSA_DEV_FP16_RANGE = (
    0x1, 0x2, 0x4, 0x8, 0x10)
BSA_DEV_BAD_LENGTH = 0x20
PHASE_DECODE, PHASE_PREFILL = 0, 1
OP_SCORE, OP_SELECT, OP_DECODE, OP_PREFILL, OP_PBS_PERMUTE = 0, 1, 2, 3, 4
OP_ATTEND_PACKED, OP_DECODE_SHARED = 5, 6
BLOCK = 64

EXPORTED = ["bsa_max_kept", "bsa_workspace_size", "bsa_score_blocks", "bsa_select_top_p",
            "bsa_decode", "bsa_prefill", "bsa_status_string", "bsa_last_cuda_error",
            "bsa_decode_noalloc", "bsa_quantize_index_keys", "bsa_score_blocks_q",
            "bsa_pbs_permute", "bsa_norm_rope", "bsa_append_kv", "bsa_attend_packed",
            "bsa_decode_shared", "bsa_packed_workspace_size"]
NOALLOC_SCRATCH_BYTES = 8 << 20
IDX_FP4, IDX_INT4 = 1, 2
QIDX_RECORD_BYTES = 576


class BsaError(RuntimeError):
    pass


class CCache(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("seq_stride", ctypes.c_int64),
                ("block_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("page_table", ctypes.c_void_p), ("page_table_stride", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("extent", ctypes.c_int64)]


class CQCache(ctypes.Structure):
    _fields_ = [("records", ctypes.c_void_p), ("gscale", ctypes.c_void_p),
                ("seq_stride", ctypes.c_int64), ("block_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("page_table_stride", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("extent", ctypes.c_int64), ("format", ctypes.c_int32)]


class CProblem(ctypes.Structure):
    _fields_ = [("phase", ctypes.c_int32), ("B", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("r", ctypes.c_int32),
                ("block", ctypes.c_int32), ("T", ctypes.c_int32), ("seq_lens", ctypes.c_void_p),
                ("n_sink", ctypes.c_int32), ("n_local", ctypes.c_int32),
                ("k_max", ctypes.c_int32), ("k_min", ctypes.c_int32), ("p", ctypes.c_float),
                ("idx_scale", ctypes.c_float), ("attn_scale", ctypes.c_float),
                ("head_w", ctypes.c_void_p), ("head_p", ctypes.c_void_p),
                ("idx_heads", ctypes.c_int32), ("segment", ctypes.c_int32),
                ("key_pos", ctypes.c_void_p), ("group_size", ctypes.c_int32),
                ("k_groups", ctypes.c_int32), ("group_scores", ctypes.c_void_p),
                ("kept_groups", ctypes.c_void_p)]


class CRows(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("type", ctypes.c_int32)]


class CTokens(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("B", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("r", ctypes.c_int32),
                ("block", ctypes.c_int32), ("T", ctypes.c_int32),
                ("cu_seqlens", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("rope_steps", ctypes.c_void_p),
                ("rope_dim", ctypes.c_int32), ("rope_interleaved", ctypes.c_int32),
                ("rope_factor", ctypes.c_float), ("norm", ctypes.c_int32),
                ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("causal", ctypes.c_int32),
                ("attn_scale", ctypes.c_float), ("q_stride", ctypes.c_int64),
                ("p_parts", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libbsa.so once and declare its signatures; raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise BsaError(f"{path} not found: build it with `python -m block_sparse_long_06_b200.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(CProblem)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.bsa_max_kept.argtypes = [P]
    lib.bsa_max_kept.restype = ctypes.c_int32
    lib.bsa_workspace_size.argtypes = [P, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]
    lib.bsa_workspace_size.restype = ctypes.c_int
    lib.bsa_score_blocks.argtypes = [P, vp, CCache, vp, vp, vp]
    lib.bsa_score_blocks.restype = ctypes.c_int
    lib.bsa_select_top_p.argtypes = [P, vp, vp, vp, vp, vp]
    lib.bsa_select_top_p.restype = ctypes.c_int
    for name in ("bsa_decode", "bsa_prefill"):
        f = getattr(lib, name)
        f.argtypes = [P, vp, CCache, CCache, vp, vp, vp, vp, vp, vp, sz, vp, vp]
        f.restype = ctypes.c_int
    lib.bsa_decode_noalloc.argtypes = [P, vp, CCache, CCache, vp, vp, vp, vp, vp, vp, vp]
    lib.bsa_decode_noalloc.restype = ctypes.c_int
    lib.bsa_quantize_index_keys.argtypes = [P, CCache, CQCache, vp, vp]
    lib.bsa_quantize_index_keys.restype = ctypes.c_int
    lib.bsa_score_blocks_q.argtypes = [P, vp, CQCache, vp, vp, vp]
    lib.bsa_score_blocks_q.restype = ctypes.c_int
    lib.bsa_pbs_permute.argtypes = [P, vp, CCache, CCache, CCache, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.bsa_pbs_permute.restype = ctypes.c_int
    TP = ctypes.POINTER(CTokens)
    lib.bsa_norm_rope.argtypes = [TP, CRows, CRows, CRows, CRows, vp, vp]
    lib.bsa_append_kv.argtypes = [TP, CRows, CRows, CRows, CCache, CCache, CCache, CRows, CRows,
                                  vp, vp]
    lib.bsa_attend_packed.argtypes = [TP, vp, CCache, CCache, vp, vp, vp, vp, sz, vp, vp]
    lib.bsa_decode_shared.argtypes = [TP, vp, CCache, CCache, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.bsa_packed_workspace_size.argtypes = [TP, ctypes.c_int32, ctypes.POINTER(sz)]
    for name in ("bsa_norm_rope", "bsa_append_kv", "bsa_attend_packed", "bsa_decode_shared",
                 "bsa_packed_workspace_size"):
        getattr(lib, name).restype = ctypes.c_int
    lib.bsa_status_string.argtypes = [ctypes.c_int]
    lib.bsa_status_string.restype = ctypes.c_char_p
    lib.bsa_last_cuda_error.argtypes = []
    lib.bsa_last_cuda_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != BSA_OK:
        lib = load_library()
        msg = lib.bsa_status_string(status).decode()
        if status == BSA_ERR_CUDA:
            msg += ": " + lib.bsa_last_cuda_error().decode()
        raise BsaError(f"{what}: {msg} (status {status})")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ------------------------------------------------------------------ problem / caches
@dataclass
class Problem:
    phase: int
    B: int
    Hq: int
    Hkv: int
    d: int
    T: int
    n_sink: int
    n_local: int
    k_max: int
    p: float
    k_min: int = 0
    r: int = 16
    block: int = BLOCK
    idx_scale: float = 0.0        # 0 -> 1/sqrt(r)
    attn_scale: float = 0.0       # 0 -> 1/sqrt(d)
    seq_lens: Optional[torch.Tensor] = None   # device int32 [B] (decode)
    head_w: Optional[torch.Tensor] = None     # device float32 [Hq]
    head_p: Optional[torch.Tensor] = None     # device float32 [Hkv]: per-kv-head p (<= 0: local head)
    idx_heads: int = 0                        # 0: an index head per query head; 1: one per kv group
    segment: int = 0                          # prefill: PBS segment length in tokens (0: none)
    key_pos: Optional[torch.Tensor] = None    # prefill with segment: device int32 [B, Hkv, T]
    group_size: int = 0                       # decode: two-level routing group (16/32/64; 0: off)
    k_groups: int = 0                         # decode with group_size: kept groups per row
    group_scores: Optional[torch.Tensor] = None   # device float32 [B, Hkv, nb * 64 / group_size]
    kept_groups: Optional[torch.Tensor] = None    # device int32 [B, Hkv, max_kept] bitmasks

    @property
    def G(self):
        return self.Hq // self.Hkv

    @property
    def nb(self):
        return (self.T + BLOCK - 1) // BLOCK

    def c(self) -> CProblem:
        return CProblem(self.phase, self.B, self.Hq, self.Hkv, self.d, self.r, self.block, self.T,
                        _ptr(self.seq_lens), self.n_sink, self.n_local, self.k_max, self.k_min,
                        float(self.p), float(self.idx_scale), float(self.attn_scale),
                        _ptr(self.head_w), _ptr(self.head_p), int(self.idx_heads),
                        int(self.segment), _ptr(self.key_pos), int(self.group_size),
                        int(self.k_groups), _ptr(self.group_scores), _ptr(self.kept_groups))


_I32 = torch.int32


@dataclass
class Cache:
    """A bf16 cache tensor (K, V or index keys) and its addressing (bsa_cache_t)."""
    tensor: torch.Tensor
    seq_stride: int
    block_stride: int
    head_stride: int
    page_table: Optional[torch.Tensor] = None
    num_pages: int = 0

    _kept = None                               # the last call's struct, not part of the state

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_kept":
            object.__setattr__(self, "_kept", None)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_kept"}

    def _struct(self, table=None) -> CCache:
        """The struct kept between calls until a field changes: for one call, by value. What a
        tensor says of itself is read every time. table: what _table says of the page table."""
        c = self._kept
        if c is None:
            c = self._kept = CCache(None, self.seq_stride, self.block_stride, self.head_stride,
                                    None, 0, self.num_pages, 0)
        c.base, c.extent = self.tensor.data_ptr(), self.tensor.numel()
        if self.page_table is not None:
            c.page_table, c.page_table_stride = table or (self.page_table.data_ptr(),
                                                          self.page_table.shape[1])
        return c

    def c(self) -> CCache:
        return CCache.from_buffer_copy(self._struct())


def contiguous_cache(t: torch.Tensor) -> Cache:
    """[B, Hkv, T, w] contiguous bf16 tensor."""
    assert t.is_contiguous() and t.dtype == torch.bfloat16 and t.dim() == 4
    B, H, T, w = t.shape
    return Cache(t, H * T * w, BLOCK * w, T * w)


def paged_cache(pool: torch.Tensor, page_table: torch.Tensor) -> Cache:
    """[P, Hkv, 64, w] contiguous bf16 pool with a [B, nb] int32 page table."""
    assert pool.is_contiguous() and pool.dtype == torch.bfloat16 and pool.shape[2] == BLOCK
    assert page_table.dtype == torch.int32 and page_table.is_contiguous()
    P, H, _, w = pool.shape
    return Cache(pool, 0, H * BLOCK * w, BLOCK * w, page_table, P)


@dataclass
class QCache:
    """A 4-bit index-key cache (bsa_qcache_t): 576-byte records of 64 tokens, plus
    the cache scale. `records` is a uint8 tensor, `gscale` a float32 [1] tensor."""
    records: torch.Tensor
    gscale: torch.Tensor
    fmt: int
    seq_stride: int
    block_stride: int
    head_stride: int
    page_table: Optional[torch.Tensor] = None
    num_pages: int = 0

    def c(self) -> CQCache:
        pt = self.page_table
        return CQCache(self.records.data_ptr(), self.gscale.data_ptr(), self.seq_stride,
                       self.block_stride, self.head_stride, None if pt is None else pt.data_ptr(),
                       0 if pt is None else pt.shape[1], self.num_pages,
                       self.records.numel() // QIDX_RECORD_BYTES, self.fmt)


def contiguous_qcache(B: int, Hkv: int, T: int, fmt: int, device=None) -> QCache:
    """Zeroed [B, Hkv, nb] records (nb = ceil(T/64))."""
    nb = (T + BLOCK - 1) // BLOCK
    rec = torch.zeros(B * Hkv * nb * QIDX_RECORD_BYTES, dtype=torch.uint8, device=device)
    gs = torch.zeros(1, dtype=torch.float32, device=device)
    return QCache(rec, gs, fmt, Hkv * nb, 1, nb)


def paged_qcache(num_pages: int, Hkv: int, page_table: torch.Tensor, fmt: int, device=None) -> QCache:
    """Zeroed [P, Hkv] records addressed through a [B, nb] int32 page table."""
    assert page_table.dtype == torch.int32 and page_table.is_contiguous()
    rec = torch.zeros(num_pages * Hkv * QIDX_RECORD_BYTES, dtype=torch.uint8, device=device)
    gs = torch.zeros(1, dtype=torch.float32, device=device)
    return QCache(rec, gs, fmt, 0, Hkv, 1, page_table, num_pages)


# ------------------------------------------------------------------ new token rows
def rope_frequencies(dim: int, theta: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, original: int = 8192, low: float = 1.0,
                     high: float = 32.0):
    """Rotary frequencies (radians per position, float64 [dim / 2] on the host) and the factor
    on cos and sin. theta^(-2i/dim), and for contexts `factor` times the `original` length:

    * ``linear``: every frequency divided by `factor`;
    * ``ntk``: theta raised to theta * factor^(dim / (dim - 2)), which divides the slowest
      frequency by `factor` and leaves the fastest;
    * ``ramp``: by the turns a pair makes over `original` positions: at most `low` turns:
      divided by `factor`, at least `high`: as they are, a linear ramp between; the factor on
      cos and sin is 0.1 ln(factor) + 1.
    """
    if dim <= 0 or dim % 2 or not theta > 0 or not factor >= 1:
        raise BsaError("rope_frequencies: dim even and > 0, theta > 0, factor >= 1")
    i = torch.arange(dim // 2, dtype=torch.float64) * 2 / dim
    if scaling == "none":
        return theta ** -i, 1.0
    if scaling == "linear":
        return theta ** -i / factor, 1.0
    if scaling == "ntk":
        if dim == 2:
            raise BsaError("rope_frequencies: ntk needs more than one pair")
        return (theta * factor ** (dim / (dim - 2))) ** -i, 1.0
    if scaling == "ramp":
        if not 0 <= low < high:
            raise BsaError("rope_frequencies: 0 <= low < high")
        f = theta ** -i
        keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    raise BsaError(f"rope_frequencies: unknown scaling {scaling!r}")


def rope_steps(frequencies: torch.Tensor) -> torch.Tensor:
    """What each pair turns by per position, in units of 2^-64 turns (int64, modulo 2^64)."""
    turns = torch.remainder(frequencies.detach().double() / (2 * math.pi), 1.0)
    high = torch.floor(turns * 2.0 ** 32)
    low = torch.floor((turns * 2.0 ** 32 - high) * 2.0 ** 32)
    high, low = high.to(torch.int64), low.to(torch.int64)
    return torch.where(high >= 2 ** 31, high - 2 ** 32, high) * 2 ** 32 + low


@dataclass
class Rope:
    """Rotary positions of the leading 2 * len(steps) elements of each head: pairs
    (i, i + half) or, interleaved, (2i, 2i + 1). `steps` is a device int64 tensor
    (rope_steps); `factor` multiplies cos and sin."""
    steps: torch.Tensor
    interleaved: bool = False
    factor: float = 1.0

    @classmethod
    def make(cls, dim: int, theta: float = 10000.0, interleaved: bool = False, device="cuda",
             **scaling) -> "Rope":
        """Steps of rope_frequencies(dim, theta, **scaling), on `device`."""
        f, factor = rope_frequencies(dim, theta, **scaling)
        return cls(rope_steps(f).to(device), interleaved, factor)


@dataclass
class Tokens:
    """Packed new token rows (bsa_tokens_t). Rows [cu_seqlens[b], cu_seqlens[b+1]) are the
    newest tokens of sequence b, which has seq_lens[b] tokens with them; rows behind the last
    sequence are padding."""
    N: int
    B: int
    Hq: int
    Hkv: int
    d: int
    T: int                                     # capacity: tokens of a sequence at most
    cu_seqlens: Optional[torch.Tensor] = None  # device int32 [B+1]; None: N / B rows each
    seq_lens: Optional[torch.Tensor] = None    # device int32 [B]; None: T each
    positions: Optional[torch.Tensor] = None   # device int32 [N]; None: the token number
    rope: Optional[Rope] = None
    norm: bool = False
    eps: float = 1e-6
    q_weight: Optional[torch.Tensor] = None    # device float32 [d]; None: ones
    k_weight: Optional[torch.Tensor] = None
    causal: bool = True
    attn_scale: float = 0.0                    # 0 -> 1/sqrt(d)
    q_stride: int = 0                          # elements between tokens of q; 0 -> Hq * d
    r: int = 16
    block: int = BLOCK
    p_parts: int = 0                           # bf16 parts of a softmax weight (1, 2); 0 -> by rows

    _kept = None                               # the last call's description, not part of the state

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_kept":
            object.__setattr__(self, "_kept", None)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_kept"}

    def tensors(self):
        rope = self.rope
        return (self.cu_seqlens, self.seq_lens, self.positions, self.q_weight, self.k_weight,
                None if rope is None else rope.steps)

    def _description(self):
        """(struct, device index or -1), kept between calls until a field changes: for one call, by
        value. Checked once, and again where a tensor has another size."""
        kept, rope = self._kept, self.rope
        if kept is None or (rope is not None and (kept[3] is not rope.steps or
                                                  kept[4] != (rope.interleaved, rope.factor))):
            kept = self._describe_again()
        c = kept[0]
        for name, size, address, n in kept[2]:
            if size() != n:
                self._describe_again()
                return self._description()
            setattr(c, name, address())
        return c, kept[1]

    def _describe_again(self):
        self._kept, rope = None, self.rope
        names = ("cu_seqlens", "seq_lens", "positions", "q_weight", "k_weight", "rope_steps")
        tensors = [(n, t) for n, t in zip(names, self.tensors()) if t is not None]
        self._kept = (self._describe(), tensors[0][1].get_device() if tensors else -1,
                      [(n, t.numel, t.data_ptr, t.numel()) for n, t in tensors],
                      None if rope is None else rope.steps,
                      None if rope is None else (rope.interleaved, rope.factor))
        return self._kept

    def c(self) -> CTokens:
        return CTokens.from_buffer_copy(self._description()[0])

    def _describe(self) -> CTokens:
        _want("cu_seqlens", self.cu_seqlens, torch.int32, (self.B + 1,))
        _want("seq_lens", self.seq_lens, torch.int32, (self.B,))
        _want("positions", self.positions, torch.int32, (self.N,))
        _want("q_weight", self.q_weight, torch.float32, (self.d,))
        _want("k_weight", self.k_weight, torch.float32, (self.d,))
        rope, dim = self.rope, 0
        if rope is not None:
            _want("rope.steps", rope.steps, torch.int64, (rope.steps.numel(),))
            dim = 2 * rope.steps.numel()
        if len({t.get_device() for t in self.tensors() if t is not None}) > 1:
            raise BsaError("Tokens: tensors on several devices")
        return CTokens(self.N, self.B, self.Hq, self.Hkv, self.d, self.r, self.block, self.T,
                       None, None, None, None, dim, int(rope is not None and rope.interleaved),
                       1.0 if rope is None else float(rope.factor), int(self.norm),
                       float(self.eps), None, None, int(self.causal), float(self.attn_scale),
                       int(self.q_stride), int(self.p_parts))


_ROW_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _want(name, t, dtype, shape):
    """Raise unless t is None or a contiguous device tensor of this type and shape."""
    if t is None:
        return
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise BsaError(f"{name}: contiguous {dtype} {tuple(shape)} wanted, got {t.dtype} "
                       f"{tuple(t.shape)} with strides {t.stride()}")
    if not _on_gpu(t):
        raise BsaError(f"{name}: has to be on the GPU")


def _on_gpu(t):
    return t.is_cuda


def _table(name, pt, B, T, dev):
    """(address, row length) of a page table for B sequences of up to T tokens; None: none."""
    if pt is None:
        return None
    shape = pt.shape
    if (len(shape) != 2 or shape[0] < B or shape[1] * BLOCK < T or pt.dtype is not _I32 or
            not pt.is_contiguous()):
        raise BsaError(f"{name}: a contiguous int32 page table of {B} rows and {-(-T // BLOCK)} "
                       f"pages a row at least wanted, got {pt.dtype} {tuple(shape)} with strides "
                       f"{pt.stride()}")
    if pt.get_device() != dev:
        _check_device(dev, pt)
    return pt.data_ptr(), shape[1]


_NO_CACHE = CCache()


def _structs(tok, dev, k, v, x=None):
    """The structs of a call's caches of keys, values and index keys (None: none) on device `dev`,
    most of which share a page table."""
    B, T, pt = tok.B, tok.T, k.page_table
    if k.tensor.get_device() != dev or v.tensor.get_device() != dev:
        _check_device(dev, k.tensor, v.tensor)
    table = _table("k", pt, B, T, dev)
    ks = k._struct(table)
    vs = v._struct(table if v.page_table is pt else _table("v", v.page_table, B, T, dev))
    if x is None:
        return ks, vs, _NO_CACHE
    _check_device(dev, x.tensor)
    return ks, vs, x._struct(table if x.page_table is pt else
                             _table("k_idx", x.page_table, B, T, dev))


_NO_ROWS = CRows(None, 0, 0, 0)


def _rows(name, t, N, heads, width, dev, out=False) -> CRows:
    """Head rows [N, heads, width] on device `dev`, of any token and head stride; None: no
    rows. Outputs are bfloat16."""
    if t is None:
        return _NO_ROWS
    kind = _ROW_TYPES.get(t.dtype)
    if kind is None or (out and kind != 0):
        raise BsaError(f"{name}: {'bfloat16' if out else 'bfloat16, float16 or float32'} wanted, "
                       f"got {t.dtype}")
    if t.shape != (N, heads, width) or (stride := t.stride())[2] != 1:
        raise BsaError(f"{name}: [{N}, {heads}, {width}] with contiguous heads wanted, got "
                       f"{tuple(t.shape)} with strides {t.stride()}")
    if t.get_device() != dev or dev < 0:
        raise BsaError(f"{name}: on {t.device}, wanted on the GPU and where the others are")
    return CRows(t.data_ptr(), stride[0], stride[1], kind)


def _check_device(dev, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise BsaError(f"a tensor on {t.device}, wanted on cuda:{dev} as the others")


def _tokens_on(tok, dev) -> CTokens:
    c, at = tok._description()
    if at != dev and at != -1:
        raise BsaError(f"the description's tensors are on cuda:{at}, the others on cuda:{dev}")
    return c


def _raw_stream(stream, dev) -> int:
    """The stream's handle; None: the current stream of device `dev`."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _launch(fn, what, dev, *args):
    """Call an entry point with `dev` as the current device (kernels and streams belong to
    it) and raise on a status."""
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status != BSA_OK:
        _check(status, what)


# ------------------------------------------------------------------ the C entry points
def bsa_max_kept(prob: Problem) -> int:
    return load_library().bsa_max_kept(ctypes.byref(prob.c()))


def bsa_workspace_size(prob: Problem, op: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().bsa_workspace_size(ctypes.byref(prob.c()), op, ctypes.byref(out)),
           "bsa_workspace_size")
    return out.value


def bsa_score_blocks(prob: Problem, q_idx, k_idx: Cache, block_scores, dev_status=None,
                     stream=None):
    _check(load_library().bsa_score_blocks(ctypes.byref(prob.c()), _ptr(q_idx), k_idx.c(),
                                           _ptr(block_scores), _ptr(dev_status), _stream(stream)),
           "bsa_score_blocks")


def bsa_quantize_index_keys(prob: Problem, k_idx: Cache, out: QCache, dev_status=None,
                            stream=None):
    _check(load_library().bsa_quantize_index_keys(ctypes.byref(prob.c()), k_idx.c(), out.c(),
                                                  _ptr(dev_status), _stream(stream)),
           "bsa_quantize_index_keys")


def bsa_score_blocks_q(prob: Problem, q_idx, k_idx: QCache, block_scores, dev_status=None,
                       stream=None):
    _check(load_library().bsa_score_blocks_q(ctypes.byref(prob.c()), _ptr(q_idx), k_idx.c(),
                                             _ptr(block_scores), _ptr(dev_status), _stream(stream)),
           "bsa_score_blocks_q")


def bsa_select_top_p(prob: Problem, block_scores, kept, kept_count, dev_status=None, stream=None):
    _check(load_library().bsa_select_top_p(ctypes.byref(prob.c()), _ptr(block_scores), _ptr(kept),
                                           _ptr(kept_count), _ptr(dev_status), _stream(stream)),
           "bsa_select_top_p")


def bsa_decode(prob: Problem, q, k: Cache, v: Cache, kept, kept_count, o, lse, o_f32, workspace,
               dev_status=None, stream=None):
    _check(load_library().bsa_decode(ctypes.byref(prob.c()), _ptr(q), k.c(), v.c(), _ptr(kept),
                                     _ptr(kept_count), _ptr(o), _ptr(lse), _ptr(o_f32),
                                     _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                     _ptr(dev_status), _stream(stream)),
           "bsa_decode")


def bsa_prefill(prob: Problem, q, k: Cache, v: Cache, kept, kept_count, o, lse, o_f32, workspace,
                dev_status=None, stream=None):
    _check(load_library().bsa_prefill(ctypes.byref(prob.c()), _ptr(q), k.c(), v.c(), _ptr(kept),
                                      _ptr(kept_count), _ptr(o), _ptr(lse), _ptr(o_f32),
                                      _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                      _ptr(dev_status), _stream(stream)),
           "bsa_prefill")


def bsa_decode_noalloc(prob: Problem, q, k: Cache, v: Cache, kept, kept_count, o, lse, o_f32,
                       dev_status=None, stream=None):
    """bsa_decode without a workspace argument, for callers that cannot allocate device
    memory: the split-K scratch lives in the library's fixed 8 MiB device array. Calls
    that overlap on the GPU share that array and must be serialised by the caller."""
    _check(load_library().bsa_decode_noalloc(ctypes.byref(prob.c()), _ptr(q), k.c(), v.c(),
                                             _ptr(kept), _ptr(kept_count), _ptr(o), _ptr(lse),
                                             _ptr(o_f32), _ptr(dev_status), _stream(stream)),
           "bsa_decode_noalloc")


def bsa_pbs_permute(prob: Problem, q, k: Cache, v: Cache, k_idx: Cache, k_perm, v_perm,
                    kidx_perm, key_pos, workspace, dev_status=None, stream=None):
    _check(load_library().bsa_pbs_permute(ctypes.byref(prob.c()), _ptr(q), k.c(), v.c(),
                                          k_idx.c(), _ptr(k_perm), _ptr(v_perm),
                                          _ptr(kidx_perm), _ptr(key_pos), _ptr(workspace),
                                          0 if workspace is None else workspace.numel(),
                                          _ptr(dev_status), _stream(stream)),
           "bsa_pbs_permute")


def bsa_norm_rope(tok: Tokens, q, q_out, k=None, k_out=None, dev_status=None, stream=None):
    """Norm (tok.norm) and rotate (tok.rope) the heads of q [N, Hq, d] into q_out and of
    k [N, Hkv, d] into k_out (bf16; either pair may be None, outputs may be the inputs)."""
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or q is k is None:
        raise BsaError("bsa_norm_rope: q and q_out, k and k_out come together, one pair at least")
    dev = (k if q is None else q).get_device()
    N, d, c = tok.N, tok.d, _tokens_on(tok, dev)
    if dev_status is not None:
        _check_device(dev, dev_status)
    _launch(load_library().bsa_norm_rope, "bsa_norm_rope", dev, c,
            _rows("q", q, N, tok.Hq, d, dev), _rows("q_out", q_out, N, tok.Hq, d, dev, True),
            _rows("k", k, N, tok.Hkv, d, dev), _rows("k_out", k_out, N, tok.Hkv, d, dev, True),
            None if dev_status is None else dev_status.data_ptr(), _raw_stream(stream, dev))


def bsa_append_kv(tok: Tokens, k, v, k_cache: Cache, v_cache: Cache, k_idx=None,
                  kidx_cache: Optional[Cache] = None, q=None, q_out=None, dev_status=None,
                  stream=None):
    """Append k (normed and rotated) and v [N, Hkv, d] and, where given, the index keys
    k_idx [N, Hkv, r] to their sequences' caches; q [N, Hq, d], where given, is normed and
    rotated into q_out by the same launch."""
    if (q is None) != (q_out is None) or (k_idx is None) != (kidx_cache is None):
        raise BsaError("bsa_append_kv: q and q_out, k_idx and kidx_cache come together")
    dev = k.get_device()
    N, d, H, c = tok.N, tok.d, tok.Hkv, _tokens_on(tok, dev)
    if dev_status is not None:
        _check_device(dev, dev_status)
    _launch(load_library().bsa_append_kv, "bsa_append_kv", dev, c,
            _rows("k", k, N, H, d, dev), _rows("v", v, N, H, d, dev),
            _rows("k_idx", k_idx, N, H, tok.r, dev), *_structs(tok, dev, k_cache, v_cache, kidx_cache),
            _rows("q", q, N, tok.Hq, d, dev), _rows("q_out", q_out, N, tok.Hq, d, dev, True),
            None if dev_status is None else dev_status.data_ptr(), _raw_stream(stream, dev))


def bsa_packed_workspace_size(tok: Tokens, op: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().bsa_packed_workspace_size(ctypes.byref(tok.c()), op, ctypes.byref(out)),
           "bsa_packed_workspace_size")
    return out.value


def _packed_call(name, tok, q, k, v, own, o, lse, o_f32, workspace, dev_status, stream):
    dev = q.get_device()
    N, Hq, d = tok.N, tok.Hq, tok.d
    stride = q.stride()
    if q.dtype != torch.bfloat16 or q.shape != (N, Hq, d) or (
            N > 0 and (stride[2] != 1 or stride[1] != d)):
        raise BsaError(f"{name}: q has to be bfloat16 [{N}, {Hq}, {d}], a token's heads side by "
                       f"side, got {q.dtype} {tuple(q.shape)} {q.stride()}")
    if N > 1 and stride[0] < Hq * d:      # (0 in the struct is the default, not one row for all)
        raise BsaError(f"{name}: q's rows overlap: {stride[0]} elements between tokens, wanted "
                       f"{Hq * d} at least")
    if dev < 0:
        raise BsaError(f"{name}: q has to be on the GPU")
    c = _tokens_on(tok, dev)
    _check_device(dev, o, lse, o_f32, workspace, dev_status, *own)
    _want("o", o, torch.bfloat16, (N, Hq, d))
    _want("lse", lse, torch.float32, (N, Hq))
    _want("o_f32", o_f32, torch.float32, (N, Hq, d))
    if N > 1:
        if tok.q_stride not in (0, stride[0]):
            raise BsaError(f"{name}: q_stride {tok.q_stride}, but q has {stride[0]}")
        if stride[0] != Hq * d:
            c = CTokens.from_buffer_copy(c)
            c.q_stride = stride[0]
    args = [c, q.data_ptr(), *_structs(tok, dev, k, v)[:2]]
    if own:
        _want("o_own", own[0], torch.float32, (N, Hq, d))
        _want("lse_own", own[1], torch.float32, (N, Hq))
        args += [None if t is None else t.data_ptr() for t in own]
    _launch(getattr(load_library(), name), name, dev, *args, o.data_ptr(), lse.data_ptr(),
            None if o_f32 is None else o_f32.data_ptr(),
            None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel() * workspace.element_size(),
            None if dev_status is None else dev_status.data_ptr(), _raw_stream(stream, dev))


def bsa_attend_packed(tok: Tokens, q, k: Cache, v: Cache, o, lse, o_f32, workspace,
                      dev_status=None, stream=None):
    """Dense attention of packed rows q [N, Hq, d] over their sequences' caches."""
    _packed_call("bsa_attend_packed", tok, q, k, v, (), o, lse, o_f32, workspace, dev_status,
                 stream)


def bsa_decode_shared(tok: Tokens, q, k: Cache, v: Cache, o_own, lse_own, o, lse, o_f32,
                      workspace, dev_status=None, stream=None):
    """Decode attention over shared prefixes (tok.B of them, caches k and v), joined with the
    attention over each row's own tokens (o_own, lse_own; both None: none)."""
    _packed_call("bsa_decode_shared", tok, q, k, v, (o_own, lse_own), o, lse, o_f32, workspace,
                 dev_status, stream)


def bsa_status_string(status: int) -> str:
    return load_library().bsa_status_string(status).decode()


# ------------------------------------------------------------------ pipelines
class DecodeStep:
    """Buffers for one decode problem and the score -> select -> attend chain.

    Outputs live in this object (torch-allocated once); ``run`` enqueues the three
    entry points on the current stream and returns nothing (no host sync)."""

    def __init__(self, prob: Problem, device="cuda", keep_f32=True):
        assert prob.phase == PHASE_DECODE
        self.prob = prob
        dev = torch.device(device)
        mk = bsa_max_kept(prob)
        self.scores = torch.empty(prob.B, prob.Hkv, prob.nb, dtype=torch.float32, device=dev)
        self.kept = torch.empty(prob.B, prob.Hkv, mk, dtype=torch.int32, device=dev)
        self.kept_count = torch.empty(prob.B, prob.Hkv, dtype=torch.int32, device=dev)
        self.o = torch.empty(prob.B, prob.Hq, prob.d, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(prob.B, prob.Hq, dtype=torch.float32, device=dev)
        self.o_f32 = (torch.empty(prob.B, prob.Hq, prob.d, dtype=torch.float32, device=dev)
                      if keep_f32 else None)
        if prob.group_size > 0:   # two-level routing: group scores and kept-group masks
            prob.group_scores = torch.empty(prob.B, prob.Hkv, prob.nb * BLOCK // prob.group_size,
                                            dtype=torch.float32, device=dev)
            prob.kept_groups = torch.empty(prob.B, prob.Hkv, mk, dtype=torch.int32, device=dev)
            self.group_scores, self.kept_groups = prob.group_scores, prob.kept_groups
        ws = bsa_workspace_size(prob, OP_DECODE)
        self.workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def run(self, q, q_idx, k_idx, k: Cache, v: Cache, stream=None):
        """k_idx: a bf16 index-key Cache or a 4-bit QCache."""
        p = self.prob
        if isinstance(k_idx, QCache):
            bsa_score_blocks_q(p, q_idx, k_idx, self.scores, self.status, stream)
        else:
            bsa_score_blocks(p, q_idx, k_idx, self.scores, self.status, stream)
        bsa_select_top_p(p, self.scores, self.kept, self.kept_count, self.status, stream)
        bsa_decode(p, q, k, v, self.kept, self.kept_count, self.o, self.lse, self.o_f32,
                   self.workspace, self.status, stream)


class Prefill:
    """Buffers for one prefill problem and the score -> select -> attend chain."""

    def __init__(self, prob: Problem, device="cuda", keep_f32=True):
        assert prob.phase == PHASE_PREFILL
        self.prob = prob
        dev = torch.device(device)
        nqb = prob.nb
        mk = bsa_max_kept(prob)
        self.scores = torch.empty(prob.B, prob.Hkv, nqb, nqb, dtype=torch.float32, device=dev)
        self.kept = torch.empty(prob.B, prob.Hkv, nqb, mk, dtype=torch.int32, device=dev)
        self.kept_count = torch.empty(prob.B, prob.Hkv, nqb, dtype=torch.int32, device=dev)
        self.o = torch.empty(prob.B, prob.Hq, prob.T, prob.d, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(prob.B, prob.Hq, prob.T, dtype=torch.float32, device=dev)
        self.o_f32 = (torch.empty(prob.B, prob.Hq, prob.T, prob.d, dtype=torch.float32, device=dev)
                      if keep_f32 else None)
        ws = bsa_workspace_size(prob, OP_PREFILL)
        self.workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def select(self, q_idx, k_idx: Cache, stream=None):
        bsa_score_blocks(self.prob, q_idx, k_idx, self.scores, self.status, stream)
        bsa_select_top_p(self.prob, self.scores, self.kept, self.kept_count, self.status, stream)

    def attend(self, q, k: Cache, v: Cache, stream=None):
        bsa_prefill(self.prob, q, k, v, self.kept, self.kept_count, self.o, self.lse, self.o_f32,
                    self.workspace, self.status, stream)

    def run(self, q, q_idx, k_idx: Cache, k: Cache, v: Cache, stream=None):
        self.select(q_idx, k_idx, stream)
        self.attend(q, k, v, stream)


class PbsPrefill:
    """Block-sparse prefill over a segment-permuted key order (PBS-Attn): permute the
    keys inside segments of `prob.segment` tokens by importance, then score, select
    and attend on the permuted caches. Buffers live in this object; ``run`` enqueues
    the four entry points on the current stream."""

    def __init__(self, prob: Problem, device="cuda", keep_f32=True):
        assert prob.phase == PHASE_PREFILL and prob.segment > 0
        dev = torch.device(device)
        B, H, T, d = prob.B, prob.Hkv, prob.T, prob.d
        self.k_perm = torch.empty(B, H, T, d, dtype=torch.bfloat16, device=dev)
        self.v_perm = torch.empty(B, H, T, d, dtype=torch.bfloat16, device=dev)
        self.kidx_perm = torch.empty(B, H, T, prob.r, dtype=torch.bfloat16, device=dev)
        self.key_pos = torch.empty(B, H, T, dtype=torch.int32, device=dev)
        prob.key_pos = self.key_pos
        self.prob = prob
        ws = bsa_workspace_size(prob, OP_PBS_PERMUTE)
        self.pws = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
        self.pf = Prefill(prob, device=device, keep_f32=keep_f32)
        self.status = self.pf.status

    def permute(self, q, k: Cache, v: Cache, k_idx: Cache, stream=None):
        bsa_pbs_permute(self.prob, q, k, v, k_idx, self.k_perm, self.v_perm, self.kidx_perm,
                        self.key_pos, self.pws, self.status, stream)

    def run(self, q, q_idx, k_idx: Cache, k: Cache, v: Cache, stream=None):
        self.permute(q, k, v, k_idx, stream)
        self.pf.run(q, q_idx, contiguous_cache(self.kidx_perm), contiguous_cache(self.k_perm),
                    contiguous_cache(self.v_perm), stream)


class _PackedBuffers:
    def __init__(self, tok: Tokens, op: int, device, keep_f32):
        dev = torch.device(device)
        self.tok = tok
        self.o = torch.empty(tok.N, tok.Hq, tok.d, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(tok.N, tok.Hq, dtype=torch.float32, device=dev)
        self.o_f32 = (torch.empty(tok.N, tok.Hq, tok.d, dtype=torch.float32, device=dev)
                      if keep_f32 else None)
        ws = bsa_packed_workspace_size(tok, op)
        self.workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)


class PackedAttention(_PackedBuffers):
    """Outputs and workspace for dense attention of packed rows. ``run`` enqueues
    bsa_attend_packed on the current stream; lengths are read on the device, so the same
    object (or a graph captured from ``run``) serves every batch of up to N rows."""

    def __init__(self, tok: Tokens, device="cuda", keep_f32=True):
        super().__init__(tok, OP_ATTEND_PACKED, device, keep_f32)

    def run(self, q, k: Cache, v: Cache, stream=None):
        bsa_attend_packed(self.tok, q, k, v, self.o, self.lse, self.o_f32, self.workspace,
                          self.status, stream)


class SharedPrefixDecode(_PackedBuffers):
    """Outputs and workspace for decode over shared prefixes. ``run`` takes what a DecodeStep
    over each sequence's own tokens left in its o_f32 and lse, or nothing."""

    def __init__(self, tok: Tokens, device="cuda", keep_f32=True):
        super().__init__(tok, OP_DECODE_SHARED, device, keep_f32)

    def run(self, q, k: Cache, v: Cache, o_own=None, lse_own=None, stream=None):
        bsa_decode_shared(self.tok, q, k, v, o_own, lse_own, self.o, self.lse, self.o_f32,
                          self.workspace, self.status, stream)


def problem_for(w, seq_lens: Optional[torch.Tensor] = None,
                head_w: Optional[torch.Tensor] = None) -> Problem:
    """Problem description of a synthetic workload (see workloads.Workload)."""
    phase = PHASE_DECODE if w.phase == "decode" else PHASE_PREFILL
    return Problem(phase=phase, B=w.B, Hq=w.Hq, Hkv=w.Hkv, d=w.d, T=w.T, n_sink=w.n_sink,
                   n_local=w.n_local, k_max=w.k_max, k_min=w.k_min, p=w.p, r=w.r,
                   idx_scale=1.0 / math.sqrt(w.r), attn_scale=1.0 / math.sqrt(w.d),
                   seq_lens=seq_lens if phase == PHASE_DECODE else None, head_w=head_w)


def caches_for(inputs: dict):
    """(k_idx, K, V) caches of a generated input dict."""
    k_idx = contiguous_cache(inputs["k_idx"])
    if inputs.get("page_table") is not None:
        pt = inputs["page_table"]
        return k_idx, paged_cache(inputs["K"], pt), paged_cache(inputs["V"], pt)
    return k_idx, contiguous_cache(inputs["K"]), contiguous_cache(inputs["V"])


class DecodeGraph:
    """One decode step from host buffers as a single CUDA graph launch.

    The graph holds, on fixed device buffers: the copy of the new query (q, q_idx)
    from pinned host tensors, score -> select -> attend (the kernels keep their
    programmatic dependent-launch edges), and the copy of o and lse back into pinned
    host tensors. New queries are written into ``q_host`` / ``q_idx_host`` in place;
    ``launch`` enqueues the step, ``run`` also waits for the host outputs."""

    def __init__(self, step: DecodeStep, q_host, q_idx_host, k_idx, k: Cache, v: Cache,
                 o_host, lse_host):
        self.step, self.k_idx, self.k, self.v = step, k_idx, k, v
        self.q_host, self.q_idx_host, self.o_host, self.lse_host = q_host, q_idx_host, o_host, lse_host
        self.q_dev = torch.empty(q_host.shape, dtype=q_host.dtype, device="cuda")
        self.q_idx_dev = torch.empty(q_idx_host.shape, dtype=q_idx_host.dtype, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self._body()          # first launches (function attributes, tensor maps) uncaptured
        side.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        # "relaxed": the entry points set kernel attributes on the host while capturing
        with torch.cuda.graph(self.graph, capture_error_mode="relaxed"):
            self._body()
        torch.cuda.synchronize()

    def _body(self):
        self.q_dev.copy_(self.q_host, non_blocking=True)
        self.q_idx_dev.copy_(self.q_idx_host, non_blocking=True)
        self.step.run(self.q_dev, self.q_idx_dev, self.k_idx, self.k, self.v)
        self.o_host.copy_(self.step.o, non_blocking=True)
        self.lse_host.copy_(self.step.lse, non_blocking=True)

    def launch(self):
        self.graph.replay()

    def run(self):
        self.graph.replay()
        torch.cuda.current_stream().synchronize()


def decode_step_host(step: DecodeStep, q_host, q_idx_host, k_idx, k: Cache, v: Cache,
                     o_host, lse_host, q_dev=None, q_idx_dev=None, stream=None):
    """One decode step from host buffers: copy the new query (q, q_idx; pinned host
    tensors) to the device, run score -> select -> attend, copy o and lse back into
    the pinned host tensors, and wait for them. The KV and index-key caches stay
    resident on the device."""
    stream = torch.cuda.current_stream() if stream is None else stream
    q_dev = torch.empty(q_host.shape, dtype=q_host.dtype, device="cuda") if q_dev is None else q_dev
    q_idx_dev = (torch.empty(q_idx_host.shape, dtype=q_idx_host.dtype, device="cuda")
                 if q_idx_dev is None else q_idx_dev)
    with torch.cuda.stream(stream):
        q_dev.copy_(q_host, non_blocking=True)
        q_idx_dev.copy_(q_idx_host, non_blocking=True)
        step.run(q_dev, q_idx_dev, k_idx, k, v, stream)
        o_host.copy_(step.o, non_blocking=True)
        lse_host.copy_(step.lse, non_blocking=True)
    stream.synchronize()
