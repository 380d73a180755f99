// C ABI of libbsa.so: argument validation, workspace sizing, TMA descriptor
// creation and kernel launches. No allocation, no synchronisation.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "bsa_internal.h"
#include "tokens_internal.h"

namespace {

thread_local char g_last_cuda_error[256] = "";

bsa_status_t cuda_fail(cudaError_t e) {
  std::snprintf(g_last_cuda_error, sizeof(g_last_cuda_error), "%s: %s", cudaGetErrorName(e),
                cudaGetErrorString(e));
  return BSA_ERR_CUDA;
}

// SM count of the current device, read once per device.
int num_sms_current(int* out_dev = nullptr) {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
  if (out_dev) *out_dev = dev;
  if (dev < 0 || dev >= 64) {
    int n = 148;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
  }
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 148;
    cache[dev] = n;
  }
  return cache[dev];
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 2-D map over rows of `width` 16-bit elements, 64-wide boxes of `box_rows` rows,
// 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int width, bool fp16,
              int box_rows = 64) {
  auto enc = get_encode();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(width) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                   const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool is_pow2_group(int G) { return G == 1 || G == 2 || G == 4 || G == 8 || G == 16; }

int nblocks(int T) { return (T + 63) / 64; }

// Shape checks shared by every entry point.
bsa_status_t check_problem(const bsa_problem_t* p) {
  if (p == nullptr) return BSA_ERR_INVALID_ARG;
  if (p->phase != BSA_PHASE_DECODE && p->phase != BSA_PHASE_PREFILL) return BSA_ERR_INVALID_ARG;
  if (p->B <= 0 || p->Hq <= 0 || p->Hkv <= 0 || p->T < 0) return BSA_ERR_INVALID_ARG;
  if (p->Hq % p->Hkv != 0) return BSA_ERR_INVALID_ARG;
  if (p->n_sink < 0 || p->n_local < 0 || p->k_max < 0 || p->k_min < 0) return BSA_ERR_INVALID_ARG;
  if (p->k_min > p->k_max) return BSA_ERR_INVALID_ARG;
  if (!std::isfinite(p->p) || !std::isfinite(p->idx_scale) || !std::isfinite(p->attn_scale))
    return BSA_ERR_INVALID_ARG;
  if (p->idx_scale < 0.f || p->attn_scale < 0.f) return BSA_ERR_INVALID_ARG;
  if (p->block != 64 || p->r != 16) return BSA_ERR_UNSUPPORTED;
  if (p->d != 64 && p->d != 128) return BSA_ERR_UNSUPPORTED;
  if (!is_pow2_group(p->Hq / p->Hkv)) return BSA_ERR_UNSUPPORTED;
  if (p->k_max > 8192) return BSA_ERR_UNSUPPORTED;
  if (nblocks(p->T) > 32768) return BSA_ERR_UNSUPPORTED;
  if (p->phase == BSA_PHASE_PREFILL && p->seq_lens != nullptr) return BSA_ERR_UNSUPPORTED;
  if (p->phase == BSA_PHASE_PREFILL && p->T <= 0) return BSA_ERR_INVALID_ARG;
  if (p->idx_heads != 0 && p->idx_heads != 1 && p->idx_heads != p->Hq / p->Hkv)
    return BSA_ERR_UNSUPPORTED;
  if (p->segment != 0) {
    if (p->phase != BSA_PHASE_PREFILL || p->segment < 0 || p->segment % 64 != 0)
      return BSA_ERR_INVALID_ARG;
    if (p->segment > 8192) return BSA_ERR_UNSUPPORTED;
  }
  if (p->group_size != 0) {
    if (p->phase != BSA_PHASE_DECODE || p->k_groups < 0) return BSA_ERR_INVALID_ARG;
    if (p->group_size != 16 && p->group_size != 32 && p->group_size != 64)
      return BSA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(p->k_max) * (64 / p->group_size) > 8192) return BSA_ERR_UNSUPPORTED;
  }
  return BSA_OK;
}

// Blocks per segment of a permuted key order (1 when the keys keep their order).
int seg_blocks_of(const bsa_problem_t* p) { return p->segment > 0 ? p->segment / 64 : 1; }

// Index heads per kv group: one per query head (the default) or one per group
// (SparDA, Main innovations §2: a compact indexer with one head per GQA group).
int idx_group(const bsa_problem_t* p) { return p->idx_heads == 1 ? 1 : p->Hq / p->Hkv; }

float idx_scale_of(const bsa_problem_t* p) {
  return p->idx_scale > 0.f ? p->idx_scale : 1.0f / std::sqrt(static_cast<float>(p->r));
}
float attn_scale_of(const bsa_problem_t* p) {
  return p->attn_scale > 0.f ? p->attn_scale : 1.0f / std::sqrt(static_cast<float>(p->d));
}

// Cache checks: non-null 16-byte aligned base, strides that keep every row 16-byte
// aligned and (for K/V, read through TMA) whole rows of `width`.
bsa_status_t check_cache(const bsa_cache_t& c, const bsa_problem_t* p, int width, bool rows_tma) {
  if (c.base == nullptr || !aligned16(c.base) || c.extent <= 0) return BSA_ERR_INVALID_ARG;
  const int64_t unit = rows_tma ? width : 8;
  if (c.seq_stride < 0 || c.block_stride <= 0 || c.head_stride < 0) return BSA_ERR_INVALID_ARG;
  if (c.seq_stride % unit || c.block_stride % unit || c.head_stride % unit)
    return BSA_ERR_INVALID_ARG;
  if (c.page_table != nullptr) {
    if (c.num_pages <= 0 || c.page_table_stride < nblocks(p->T)) return BSA_ERR_INVALID_ARG;
  }
  if (rows_tma && c.extent / width > 0x7fffffffLL) return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}

bsa::CacheView view(const bsa_cache_t& c) {
  bsa::CacheView v;
  v.base = c.base;
  v.seq_stride = c.seq_stride;
  v.block_stride = c.block_stride;
  v.head_stride = c.head_stride;
  v.page_table = c.page_table;
  v.pt_stride = c.page_table_stride;
  v.num_pages = c.num_pages;
  v.extent = c.extent;
  return v;
}

struct DecodePlan {
  int splits, split_len, units;
  size_t part_o_bytes, part_ml_bytes;
};

DecodePlan decode_plan(const bsa_problem_t* p, int num_sms) {
  DecodePlan pl;
  const int rows = p->B * p->Hkv;
  const int mk = bsa_max_kept(p);
  bsa::decode_split_plan(rows, mk, num_sms, &pl.splits, &pl.split_len);
  pl.units = rows * pl.splits;
  const int G = p->Hq / p->Hkv;
  pl.part_o_bytes = static_cast<size_t>(pl.units) * G * p->d * sizeof(float);
  pl.part_ml_bytes = static_cast<size_t>(pl.units) * G * 2 * sizeof(float);
  return pl;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// 4-bit index-key cache checks: 16-byte aligned records, record strides >= 0,
// a valid format and a scale pointer.
bsa_status_t check_qcache(const bsa_qcache_t& c, const bsa_problem_t* p) {
  if (c.records == nullptr || !aligned16(c.records) || c.gscale == nullptr || c.extent <= 0)
    return BSA_ERR_INVALID_ARG;
  if (c.format != BSA_IDX_FP4 && c.format != BSA_IDX_INT4) return BSA_ERR_INVALID_ARG;
  if (c.seq_stride < 0 || c.block_stride <= 0 || c.head_stride < 0) return BSA_ERR_INVALID_ARG;
  if (c.page_table != nullptr) {
    if (c.num_pages <= 0 || c.page_table_stride < nblocks(p->T)) return BSA_ERR_INVALID_ARG;
  }
  return BSA_OK;
}

bsa::CacheView qview(const bsa_qcache_t& c) {
  bsa::CacheView v;
  v.base = c.records;
  v.seq_stride = c.seq_stride;
  v.block_stride = c.block_stride;
  v.head_stride = c.head_stride;
  v.page_table = c.page_table;
  v.pt_stride = c.page_table_stride;
  v.num_pages = c.num_pages;
  v.extent = c.extent;
  return v;
}

// ---------------------------------------------------------------- new token rows
// Shape checks of a bsa_tokens_t.
bsa_status_t check_tokens(const bsa_tokens_t* t) {
  if (t == nullptr) return BSA_ERR_INVALID_ARG;
  if (t->N < 0 || t->B <= 0 || t->Hq <= 0 || t->Hkv <= 0 || t->T < 0) return BSA_ERR_INVALID_ARG;
  if (t->Hq % t->Hkv != 0) return BSA_ERR_INVALID_ARG;
  if (t->cu_seqlens == nullptr && t->N % t->B != 0) return BSA_ERR_INVALID_ARG;
  if (!std::isfinite(t->rope_factor) || !std::isfinite(t->eps) || !std::isfinite(t->attn_scale))
    return BSA_ERR_INVALID_ARG;
  if (t->eps < 0.f || t->attn_scale < 0.f) return BSA_ERR_INVALID_ARG;
  if ((t->norm != 0 && t->norm != 1) || (t->causal != 0 && t->causal != 1) ||
      (t->rope_interleaved != 0 && t->rope_interleaved != 1))
    return BSA_ERR_INVALID_ARG;
  if (t->rope_dim < 0 || t->rope_dim > t->d || (t->rope_dim > 0 && t->rope_steps == nullptr))
    return BSA_ERR_INVALID_ARG;
  if (t->q_stride < 0 || t->q_stride % 8 != 0) return BSA_ERR_INVALID_ARG;
  if (t->p_parts < 0 || t->p_parts > 2) return BSA_ERR_INVALID_ARG;
  if (t->block != 64 || t->r != 16) return BSA_ERR_UNSUPPORTED;
  if (t->d != 64 && t->d != 128) return BSA_ERR_UNSUPPORTED;
  if (t->rope_dim % 16 != 0) return BSA_ERR_UNSUPPORTED;
  if (nblocks(t->T) > 32768) return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}

// Head rows of type `type`: every head starts on a 16-byte boundary.
bsa_status_t check_rows(const bsa_rows_t& x, int type) {
  if (x.base == nullptr || !aligned16(x.base) || x.type != type) return BSA_ERR_INVALID_ARG;
  const int64_t unit = type == BSA_TYPE_F32 ? 4 : 8;
  if (x.token_stride < 0 || x.head_stride < 0 || x.token_stride % unit || x.head_stride % unit)
    return BSA_ERR_INVALID_ARG;
  return BSA_OK;
}

// Output rows (bf16) of N tokens and `heads` heads: no two overlap, with a token's heads between
// those of other tokens or the other way round.
bsa_status_t check_out(const bsa_rows_t& x, const bsa_tokens_t* t, int heads) {
  bsa_status_t st = check_rows(x, BSA_TYPE_BF16);
  if (st != BSA_OK) return st;
  if ((t->N > 1 && x.token_stride < t->d) || (heads > 1 && x.head_stride < t->d))
    return BSA_ERR_INVALID_ARG;
  // in 128 bits: the strides are the caller's
  if (t->N > 1 && heads > 1 &&
      x.token_stride < static_cast<__int128>(heads - 1) * x.head_stride + t->d &&
      x.head_stride < static_cast<__int128>(t->N - 1) * x.token_stride + t->d)
    return BSA_ERR_INVALID_ARG;
  return BSA_OK;
}

// An output that starts where its input does has to be the same rows.
bool same_or_apart(const bsa_rows_t& in, const bsa_rows_t& out) {
  return in.base != out.base || (in.type == out.type && in.token_stride == out.token_stride &&
                                 in.head_stride == out.head_stride);
}

// Cache checks for a capacity of T tokens (see check_cache).
bsa_status_t check_token_cache(const bsa_cache_t& c, const bsa_tokens_t* t, int width, bool rows_tma) {
  bsa_problem_t p{};
  p.T = t->T;
  return check_cache(c, &p, width, rows_tma);
}

// Cache checks for appends: besides, no two token slots overlap (a token of the capacity T behind
// the end of its head's rows would land in the next head's). Each stride of the nest, from the
// smallest, has to span what lies inside it. Sequences of a page table share the pool, where the
// table says who has which page, unless seq_stride gives them one each.
bsa_status_t check_append_cache(const bsa_cache_t& c, const bsa_tokens_t* t, int width, bool rows_tma) {
  const bsa_status_t st = check_token_cache(c, t, width, rows_tma);
  if (st != BSA_OK || t->T == 0) return st;
  const bool paged = c.page_table != nullptr;
  struct Dim {
    int64_t count, stride;
    bool blocks;
  } dims[3] = {{paged ? c.num_pages : nblocks(t->T), c.block_stride, true},
               {t->Hkv, c.head_stride, false},
               {paged && c.seq_stride == 0 ? 1 : t->B, c.seq_stride, false}};
  std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  __int128 span = static_cast<__int128>(paged ? 64 : std::min(64, t->T)) * width;
  const __int128 block = span;
  for (const Dim& x : dims) {
    if (x.count <= 1) continue;
    if (x.stride < span) return BSA_ERR_INVALID_ARG;
    const __int128 last = static_cast<__int128>(x.count - 1) * x.stride;
    // the last block of a head's rows may be a part
    if (x.blocks && !paged && span == block)
      span = last + static_cast<__int128>(t->T - (x.count - 1) * 64) * width;
    else
      span += last;
  }
  return BSA_OK;
}

bsa::RowsView rows_view(const bsa_rows_t& x) {
  bsa::RowsView v;
  v.base = x.base;
  v.token_stride = x.token_stride;
  v.head_stride = x.head_stride;
  return v;
}

// Fields shared by bsa_norm_rope and bsa_append_kv.
bsa::HeadsArgs heads_args(const bsa_tokens_t* t, int type, int32_t* dev_status) {
  bsa::HeadsArgs a{};
  a.cu = t->cu_seqlens;
  a.seq_lens = t->seq_lens;
  a.positions = t->positions;
  a.rope_steps = t->rope_steps;
  a.norm = t->norm;
  a.q_weight = t->norm ? t->q_weight : nullptr;
  a.k_weight = t->norm ? t->k_weight : nullptr;
  a.eps = t->eps;
  a.status = dev_status;
  a.N = t->N;
  a.B = t->B;
  a.Hq = t->Hq;
  a.Hkv = t->Hkv;
  a.d = t->d;
  a.T = t->T;
  a.type = type;
  a.rope_dim = t->rope_dim;
  a.rope_interleaved = t->rope_interleaved;
  a.rope_factor = t->rope_factor == 0.f ? 1.0f : t->rope_factor;
  return a;
}

// Workspace of the packed attention. Splits of the key axis: enough for about four units
// an SM when the rows fill as few units as they can.
struct PackedWorkspace {
  int smax, max_entries;
  size_t offs, entries, row_splits, ml, o, total;
};
PackedWorkspace packed_workspace(const bsa_tokens_t* t, int num_sms) {
  PackedWorkspace w;
  const int per = bsa::packed_unit_tokens(t->Hq / t->Hkv);
  const int64_t rows = t->N > 0 ? t->N : 1;
  const int64_t least = (rows + per - 1) / per;
  const int64_t want = (4ll * num_sms + least * t->Hkv - 1) / (least * t->Hkv);
  // the most tiles that N rows of up to B sequences can make
  const int64_t seqs = std::min<int64_t>(rows, t->B), most = seqs + (rows - seqs) / per;
  const int64_t steps = (t->T + 127) / 128;
  w.smax = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, 64), steps)));
  // A merge costs as much as 4 to 6 steps of one tile: halving 12 of them gains little, and without
  // splits no merge is launched (4 rows behind 1,024 keys: 16 us, 20 with a merge that finds
  // nothing to do).
  if (steps * (t->N > per / 2 ? 2 : 1) <= 12) w.smax = 1;
  w.max_entries = static_cast<int>(most * w.smax);
  w.offs = 256;
  w.entries = w.offs + align256((static_cast<size_t>(t->B) + 1) * sizeof(int32_t));
  w.row_splits = w.entries + align256(static_cast<size_t>(w.max_entries) * 2 * sizeof(int4));
  w.ml = w.row_splits + align256(static_cast<size_t>(rows) * sizeof(int32_t));
  const size_t parts = w.smax > 1 ? static_cast<size_t>(w.smax) * rows * t->Hq : 0;
  w.o = w.ml + align256(parts * 2 * sizeof(float));
  w.total = w.o + align256(parts * t->d * sizeof(float));
  return w;
}

// 3-D map over q [N, Hq, d] (bf16, `stride` elements a token): boxes of the G heads of one
// kv group for 128 / G tokens, 64 elements wide, 128-byte swizzle. The box's rows lie in
// shared memory as (token, head).
bool make_q_map(CUtensorMap* m, const void* q, const bsa_tokens_t* t, int64_t stride) {
  auto enc = get_encode();
  if (!enc) return false;
  const int G = t->Hq / t->Hkv;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(t->d), static_cast<cuuint64_t>(t->Hq),
                        static_cast<cuuint64_t>(t->N)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(t->d) * 2, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(128 / G)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box,
                   estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Whether every block that a valid page number (or a token below T) leads to lies whole inside
// the extent.
bool inside_extent(const bsa_cache_t& c, const bsa_tokens_t* t) {
  const int64_t blocks = c.page_table != nullptr ? c.num_pages : nblocks(t->T);
  if (blocks == 0) return true;
  // in 128 bits: the strides are the caller's
  const __int128 last = static_cast<__int128>(t->B - 1) * c.seq_stride +
                        static_cast<__int128>(blocks - 1) * c.block_stride +
                        static_cast<__int128>(t->Hkv - 1) * c.head_stride + 64ll * t->d;
  return last <= c.extent;
}

bsa_status_t packed_attention(const bsa_tokens_t* t, bool shared, const void* q, const bsa_cache_t& k,
                              const bsa_cache_t& v, const float* o_own, const float* lse_own, void* o,
                              float* lse, float* o_f32, void* workspace, size_t workspace_bytes,
                              int32_t* dev_status, void* stream) {
  bsa_status_t st = check_tokens(t);
  if (st != BSA_OK) return st;
  if (!is_pow2_group(t->Hq / t->Hkv)) return BSA_ERR_UNSUPPORTED;
  if (t->N == 0) return BSA_OK;
  if (q == nullptr || o == nullptr || lse == nullptr) return BSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(o_f32) || !aligned16(o_own))
    return BSA_ERR_INVALID_ARG;
  if ((o_own == nullptr) != (lse_own == nullptr)) return BSA_ERR_INVALID_ARG;
  const int64_t stride = t->q_stride > 0 ? t->q_stride : static_cast<int64_t>(t->Hq) * t->d;
  if (stride < static_cast<int64_t>(t->Hq) * t->d) return BSA_ERR_INVALID_ARG;
  if ((st = check_token_cache(k, t, t->d, true)) != BSA_OK) return st;
  if ((st = check_token_cache(v, t, t->d, true)) != BSA_OK) return st;
  const int num_sms = num_sms_current();
  const PackedWorkspace w = packed_workspace(t, num_sms);
  if (workspace == nullptr || workspace_bytes < w.total || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return BSA_ERR_WORKSPACE;
  CUtensorMap tq, tk, tv;
  if (!make_q_map(&tq, q, t, stride) || !make_map(&tk, k.base, k.extent / t->d, t->d, false) ||
      !make_map(&tv, v.base, v.extent / t->d, t->d, false))
    return cuda_fail(cudaErrorInvalidValue);
  bsa::PackedArgs a{};
  char* ws = static_cast<char*>(workspace);
  a.q = q;
  a.k = view(k);
  a.v = view(v);
  a.cu = t->cu_seqlens;
  a.seq_lens = t->seq_lens;
  a.o_own = o_own;
  a.lse_own = lse_own;
  a.o = o;
  a.lse = lse;
  a.o_f32 = o_f32;
  a.status = dev_status;
  a.head = reinterpret_cast<int32_t*>(ws);
  a.offs = reinterpret_cast<int32_t*>(ws + w.offs);
  a.entries = reinterpret_cast<int4*>(ws + w.entries);
  a.row_splits = reinterpret_cast<int32_t*>(ws + w.row_splits);
  a.part_ml = reinterpret_cast<float*>(ws + w.ml);
  a.part_o = reinterpret_cast<float*>(ws + w.o);
  a.N = t->N;
  a.B = t->B;
  a.Hq = t->Hq;
  a.Hkv = t->Hkv;
  a.G = t->Hq / t->Hkv;
  a.d = t->d;
  a.T = t->T;
  a.causal = shared ? 0 : t->causal;
  a.smax = w.smax;
  a.max_entries = w.max_entries;
  a.num_sms = num_sms;
  // plan_in_warp has the reason. With more tiles than SMs, two rounds of units would be too coarse.
  const int max_tiles = w.max_entries / w.smax;
  a.in_block = t->B <= 32 && max_tiles <= 32 && max_tiles * t->Hkv <= num_sms;
  while ((1 << a.lgG) < a.G) ++a.lgG;
  a.k_safe = inside_extent(k, t);
  a.v_safe = inside_extent(v, t);
  a.scale_log2 = (t->attn_scale > 0.f ? t->attn_scale : 1.0f / std::sqrt(static_cast<float>(t->d))) *
                 1.4426950408889634f;
  // With no more rows than fill a tile a sequence, the keys' arrival takes the time (one row each
  // of 8 sequences over 32K keys: 136 us with one part, 148 with two), with more the products do
  // (a prompt of 32K: 7.8 and 10.4 ms).
  const bool few = static_cast<int64_t>(t->N) * a.G <= 128ll * t->B;
  a.p_parts = t->p_parts != 0 ? t->p_parts : few ? 2 : 1;
  const cudaError_t e = bsa::launch_packed(a, tq, tk, tv, num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

// Workspace of bsa_pbs_permute: per-chunk row statistics, row log-sum-exps, importance.
struct PbsWorkspace {
  size_t ml, lse2, imp, total;
};
PbsWorkspace pbs_workspace(const bsa_problem_t* p) {
  const size_t bh = static_cast<size_t>(p->B) * p->Hkv;
  const size_t rows = bh * (p->Hq / p->Hkv) * 64;
  PbsWorkspace w;
  w.ml = 0;
  w.lse2 = align256(rows * bsa::pbs_chunks(p->T) * 2 * sizeof(float));
  w.imp = w.lse2 + align256(rows * sizeof(float));
  w.total = w.imp + align256(bh * static_cast<size_t>(p->T) * sizeof(float));
  return w;
}

}  // namespace

namespace bsa {
bsa_status_t record_cuda_error(cudaError_t e) { return cuda_fail(e); }
}  // namespace bsa

extern "C" {

int32_t bsa_max_kept(const bsa_problem_t* p) {
  if (p == nullptr) return 0;
  const int32_t base = p->n_sink + p->n_local + p->k_max;
  if (p->phase != BSA_PHASE_PREFILL) return base;
  return base + (p->segment > 0 ? p->segment / 64 : 1);
}

bsa_status_t bsa_workspace_size(const bsa_problem_t* p, int32_t op, size_t* bytes) {
  if (bytes == nullptr) return BSA_ERR_INVALID_ARG;
  *bytes = 0;
  bsa_status_t st = check_problem(p);
  if (st != BSA_OK) return st;
  switch (op) {
    case BSA_OP_SCORE:
    case BSA_OP_SELECT:
      return BSA_OK;
    case BSA_OP_DECODE: {
      if (p->phase != BSA_PHASE_DECODE) return BSA_ERR_INVALID_ARG;
      const DecodePlan pl = decode_plan(p, num_sms_current());
      *bytes = align256(pl.part_o_bytes) + align256(pl.part_ml_bytes);
      return BSA_OK;
    }
    case BSA_OP_PREFILL: {
      if (p->phase != BSA_PHASE_PREFILL) return BSA_ERR_INVALID_ARG;
      const int64_t Tpad = static_cast<int64_t>(nblocks(p->T)) * 64;
      *bytes = align256(static_cast<size_t>(p->B) * p->Hkv * Tpad * p->d * 2) + 256;
      return BSA_OK;
    }
    case BSA_OP_PBS_PERMUTE: {
      if (p->phase != BSA_PHASE_PREFILL || p->segment <= 0) return BSA_ERR_INVALID_ARG;
      *bytes = pbs_workspace(p).total;
      return BSA_OK;
    }
    default:
      return BSA_ERR_INVALID_ARG;
  }
}

bsa_status_t bsa_score_blocks(const bsa_problem_t* p, const void* q_idx, bsa_cache_t k_idx,
                              float* block_scores, int32_t* dev_status, void* stream) {
  bsa_status_t st = check_problem(p);
  if (st != BSA_OK) return st;
  if (q_idx == nullptr || block_scores == nullptr || !aligned16(q_idx)) return BSA_ERR_INVALID_ARG;
  if (p->group_size > 0 && (p->group_scores == nullptr || !aligned16(p->group_scores)))
    return BSA_ERR_INVALID_ARG;
  if ((st = check_cache(k_idx, p, p->r, false)) != BSA_OK) return st;
  const int num_sms = num_sms_current();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (p->phase == BSA_PHASE_DECODE) {
    bsa::ScoreDecodeArgs a{};
    a.q_idx = q_idx;
    a.kidx = view(k_idx);
    a.seq_lens = p->seq_lens;
    a.head_w = p->head_w;
    a.head_p = p->head_p;
    a.k_min = p->k_min;
    a.scores = block_scores;
    a.status = dev_status;
    a.B = p->B;
    a.G = idx_group(p);
    a.Hq = p->Hkv * a.G;   // index heads: q_idx rows and head weights
    a.Hkv = p->Hkv;
    a.T = p->T;
    a.nb_max = nblocks(p->T);
    const int cb = bsa::score_decode_chunk_blocks();
    a.chunks_per_row = (a.nb_max + cb - 1) / cb;
    a.total_items = static_cast<int64_t>(p->B) * p->Hkv * a.chunks_per_row;
    a.idx_scale = idx_scale_of(p);
    a.group_size = p->group_size;
    a.group_scores = p->group_scores;
    e = bsa::launch_score_decode(a, num_sms, s);
  } else {
    bsa::ScorePrefillArgs a{};
    a.q_idx = q_idx;
    a.kidx = view(k_idx);
    a.head_w = p->head_w;
    a.head_p = p->head_p;
    a.k_min = p->k_min;
    a.scores = block_scores;
    a.status = dev_status;
    a.B = p->B;
    a.G = idx_group(p);
    a.Hq = p->Hkv * a.G;   // index heads: q_idx rows and head weights
    a.Hkv = p->Hkv;
    a.T = p->T;
    a.nqb = nblocks(p->T);
    a.idx_scale = idx_scale_of(p);
    e = bsa::launch_score_prefill(a, num_sms, s);
  }
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

bsa_status_t bsa_quantize_index_keys(const bsa_problem_t* p, bsa_cache_t k_idx, bsa_qcache_t out,
                                     int32_t* dev_status, void* stream) {
  bsa_status_t st = check_problem(p);
  if (st != BSA_OK) return st;
  if (p->phase != BSA_PHASE_DECODE) return BSA_ERR_UNSUPPORTED;
  if ((st = check_cache(k_idx, p, p->r, false)) != BSA_OK) return st;
  if ((st = check_qcache(out, p)) != BSA_OK) return st;
  bsa::QuantArgs a{};
  a.src = view(k_idx);
  a.dst = qview(out);
  a.gscale = out.gscale;
  a.seq_lens = p->seq_lens;
  a.status = dev_status;
  a.B = p->B;
  a.Hkv = p->Hkv;
  a.T = p->T;
  a.nb = nblocks(p->T);
  a.fmt = out.format;
  const cudaError_t e = bsa::launch_quantize_index(a, num_sms_current(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

bsa_status_t bsa_score_blocks_q(const bsa_problem_t* p, const void* q_idx, bsa_qcache_t k_idx,
                                float* block_scores, int32_t* dev_status, void* stream) {
  bsa_status_t st = check_problem(p);
  if (st != BSA_OK) return st;
  if (p->phase != BSA_PHASE_DECODE) return BSA_ERR_UNSUPPORTED;
  if (q_idx == nullptr || block_scores == nullptr || !aligned16(q_idx)) return BSA_ERR_INVALID_ARG;
  if (p->group_size > 0 && (p->group_scores == nullptr || !aligned16(p->group_scores)))
    return BSA_ERR_INVALID_ARG;
  if ((st = check_qcache(k_idx, p)) != BSA_OK) return st;
  bsa::ScoreDecodeArgs a{};
  a.q_idx = q_idx;
  a.kidx = qview(k_idx);
  a.seq_lens = p->seq_lens;
  a.head_w = p->head_w;
    a.head_p = p->head_p;
    a.k_min = p->k_min;
  a.scores = block_scores;
  a.status = dev_status;
  a.B = p->B;
  a.G = idx_group(p);
  a.Hq = p->Hkv * a.G;   // index heads: q_idx rows and head weights
  a.Hkv = p->Hkv;
  a.T = p->T;
  a.nb_max = nblocks(p->T);
  const int cb = bsa::score_decode_chunk_blocks();
  a.chunks_per_row = (a.nb_max + cb - 1) / cb;
  a.total_items = static_cast<int64_t>(p->B) * p->Hkv * a.chunks_per_row;
  a.idx_scale = idx_scale_of(p);
  a.kfmt = k_idx.format;
  a.gscale = k_idx.gscale;
  a.group_size = p->group_size;
  a.group_scores = p->group_scores;
  const cudaError_t e = bsa::launch_score_decode(a, num_sms_current(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

bsa_status_t bsa_select_top_p(const bsa_problem_t* p, const float* block_scores, int32_t* kept,
                              int32_t* kept_count, int32_t* dev_status, void* stream) {
  bsa_status_t st = check_problem(p);
  if (st != BSA_OK) return st;
  if (block_scores == nullptr || kept == nullptr || kept_count == nullptr)
    return BSA_ERR_INVALID_ARG;
  if (p->group_size > 0 && (p->group_scores == nullptr || p->kept_groups == nullptr))
    return BSA_ERR_INVALID_ARG;
  bsa::SelectArgs a{};
  a.scores = block_scores;
  a.kept = kept;
  a.kept_count = kept_count;
  a.seq_lens = p->phase == BSA_PHASE_DECODE ? p->seq_lens : nullptr;
  a.status = dev_status;
  a.phase = p->phase;
  a.B = p->B;
  a.Hkv = p->Hkv;
  a.T = p->T;
  a.nb_max = nblocks(p->T);
  a.nqb = nblocks(p->T);
  a.max_kept = bsa_max_kept(p);
  a.n_sink = p->n_sink;
  a.n_local = p->n_local;
  a.k_max = p->k_max;
  a.k_min = p->k_min;
  a.p = p->p;
  a.head_p = p->head_p;
  a.seg_blocks = seg_blocks_of(p);
  cudaError_t e = bsa::launch_select(a, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess && p->group_size > 0) {
    // level 2: the best token groups of the kept blocks
    bsa::GroupSelectArgs ga{};
    ga.group_scores = p->group_scores;
    ga.kept = kept;
    ga.kept_count = kept_count;
    ga.seq_lens = p->seq_lens;
    ga.kept_groups = p->kept_groups;
    ga.status = dev_status;
    ga.B = p->B;
    ga.Hkv = p->Hkv;
    ga.T = p->T;
    ga.nb_max = nblocks(p->T);
    ga.max_kept = a.max_kept;
    ga.n_sink = p->n_sink;
    ga.n_local = p->n_local;
    ga.group_size = p->group_size;
    ga.k_groups = p->k_groups;
    ga.max_cand = p->k_max * (64 / p->group_size);
    e = bsa::launch_select_groups(ga, static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

bsa_status_t bsa_decode(const bsa_problem_t* p, const void* q, bsa_cache_t k, bsa_cache_t v,
                        const int32_t* kept, const int32_t* kept_count, void* o, float* lse,
                        float* o_f32, void* workspace, size_t workspace_bytes,
                        int32_t* dev_status, void* stream) {
  bsa_status_t st = check_problem(p);
  if (st != BSA_OK) return st;
  if (p->phase != BSA_PHASE_DECODE) return BSA_ERR_INVALID_ARG;
  if (q == nullptr || kept == nullptr || kept_count == nullptr || o == nullptr || lse == nullptr)
    return BSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o)) return BSA_ERR_INVALID_ARG;
  if ((st = check_cache(k, p, p->d, true)) != BSA_OK) return st;
  if ((st = check_cache(v, p, p->d, true)) != BSA_OK) return st;
  const int num_sms = num_sms_current();
  const DecodePlan pl = decode_plan(p, num_sms);
  const size_t need = align256(pl.part_o_bytes) + align256(pl.part_ml_bytes);
  if (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return BSA_ERR_WORKSPACE;
  if (p->group_size > 0 && p->kept_groups == nullptr) return BSA_ERR_INVALID_ARG;
  bsa::DecodeMaps maps;
  if (!make_map(&maps.k, k.base, k.extent / p->d, p->d, false) ||
      !make_map(&maps.v, v.base, v.extent / p->d, p->d, false))
    return cuda_fail(cudaErrorInvalidValue);
  if (p->group_size > 0) {
    if (!make_map(&maps.k16, k.base, k.extent / p->d, p->d, false, 16) ||
        !make_map(&maps.v16, v.base, v.extent / p->d, p->d, false, 16))
      return cuda_fail(cudaErrorInvalidValue);
  } else {
    // not read: every kept block is copied whole
    maps.k16 = maps.k;
    maps.v16 = maps.v;
  }
  bsa::DecodeArgs a{};
  a.q = q;
  a.k = view(k);
  a.v = view(v);
  a.kept = kept;
  a.kept_count = kept_count;
  a.seq_lens = p->seq_lens;
  a.o = o;
  a.lse = lse;
  a.o_f32 = o_f32;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256(pl.part_o_bytes));
  a.status = dev_status;
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.G = p->Hq / p->Hkv;
  a.d = p->d;
  a.T = p->T;
  a.max_kept = bsa_max_kept(p);
  a.splits = pl.splits;
  a.split_len = pl.split_len;
  a.scale_log2 = attn_scale_of(p) * 1.4426950408889634f;
  a.kept_groups = p->group_size > 0 ? p->kept_groups : nullptr;
  a.group_size = p->group_size;
  cudaError_t e = bsa::launch_decode(a, maps, pl.units, num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

bsa_status_t bsa_prefill(const bsa_problem_t* p, const void* q, bsa_cache_t k, bsa_cache_t v,
                         const int32_t* kept, const int32_t* kept_count, void* o, float* lse,
                         float* o_f32, void* workspace, size_t workspace_bytes,
                         int32_t* dev_status, void* stream) {
  bsa_status_t st = check_problem(p);
  if (st != BSA_OK) return st;
  if (p->phase != BSA_PHASE_PREFILL) return BSA_ERR_INVALID_ARG;
  if (q == nullptr || kept == nullptr || kept_count == nullptr || o == nullptr || lse == nullptr)
    return BSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || (o_f32 && !aligned16(o_f32))) return BSA_ERR_INVALID_ARG;
  if (p->segment > 0 && p->key_pos == nullptr) return BSA_ERR_INVALID_ARG;
  if ((st = check_cache(k, p, p->d, true)) != BSA_OK) return st;
  if ((st = check_cache(v, p, p->d, false)) != BSA_OK) return st;
  const int nqb = nblocks(p->T);
  const int64_t Tpad = static_cast<int64_t>(nqb) * 64;
  const size_t v16_bytes = align256(static_cast<size_t>(p->B) * p->Hkv * Tpad * p->d * 2);
  const size_t need = v16_bytes + 256;
  if (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return BSA_ERR_WORKSPACE;
  const int64_t qrows = static_cast<int64_t>(p->B) * p->Hq * p->T;
  const int64_t vrows = static_cast<int64_t>(p->B) * p->Hkv * Tpad;
  if (qrows > 0x7fffffffLL || vrows > 0x7fffffffLL) return BSA_ERR_UNSUPPORTED;
  CUtensorMap tq, tk, tv;
  if (!make_map(&tq, q, qrows, p->d, false) || !make_map(&tk, k.base, k.extent / p->d, p->d, false) ||
      !make_map(&tv, workspace, vrows, p->d, true))
    return cuda_fail(cudaErrorInvalidValue);
  bsa::PrefillArgs a{};
  a.q = q;
  a.k = view(k);
  a.v = view(v);
  a.v16 = workspace;
  a.kept = kept;
  a.kept_count = kept_count;
  a.o = o;
  a.lse = lse;
  a.o_f32 = o_f32;
  a.status = dev_status;
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.G = p->Hq / p->Hkv;
  a.d = p->d;
  a.T = p->T;
  a.nqb = nqb;
  a.Tpad = static_cast<int>(Tpad);
  a.max_kept = bsa_max_kept(p);
  a.scale_log2 = attn_scale_of(p) * 1.4426950408889634f;
  a.seg_blocks = seg_blocks_of(p);
  a.key_pos = p->segment > 0 ? p->key_pos : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = bsa::launch_v_to_f16(a, s);
  if (e != cudaSuccess) return cuda_fail(e);
  int* unit_counter = reinterpret_cast<int*>(static_cast<char*>(workspace) + v16_bytes);
  e = bsa::launch_prefill_tc(a, tq, tk, tv, unit_counter, num_sms_current(), s);
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

bsa_status_t bsa_pbs_permute(const bsa_problem_t* p, const void* q, bsa_cache_t k, bsa_cache_t v,
                             bsa_cache_t k_idx, void* k_perm, void* v_perm, void* kidx_perm,
                             int32_t* key_pos, void* workspace, size_t workspace_bytes,
                             int32_t* dev_status, void* stream) {
  bsa_status_t st = check_problem(p);
  if (st != BSA_OK) return st;
  if (p->phase != BSA_PHASE_PREFILL || p->segment <= 0) return BSA_ERR_INVALID_ARG;
  if (q == nullptr || k_perm == nullptr || v_perm == nullptr || kidx_perm == nullptr ||
      key_pos == nullptr)
    return BSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_perm) || !aligned16(v_perm) || !aligned16(kidx_perm) ||
      !aligned16(key_pos))
    return BSA_ERR_INVALID_ARG;
  if ((st = check_cache(k, p, p->d, false)) != BSA_OK) return st;
  if ((st = check_cache(v, p, p->d, false)) != BSA_OK) return st;
  if ((st = check_cache(k_idx, p, p->r, false)) != BSA_OK) return st;
  const PbsWorkspace ws = pbs_workspace(p);
  if (workspace == nullptr || workspace_bytes < ws.total ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return BSA_ERR_WORKSPACE;
  bsa::PbsArgs a{};
  a.q = q;
  a.k = view(k);
  a.v = view(v);
  a.kidx = view(k_idx);
  a.k_perm = k_perm;
  a.v_perm = v_perm;
  a.kidx_perm = kidx_perm;
  a.key_pos = key_pos;
  char* w = static_cast<char*>(workspace);
  a.ml = reinterpret_cast<float*>(w + ws.ml);
  a.lse2 = reinterpret_cast<float*>(w + ws.lse2);
  a.imp = reinterpret_cast<float*>(w + ws.imp);
  a.status = dev_status;
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.G = p->Hq / p->Hkv;
  a.d = p->d;
  a.T = p->T;
  a.nqb = nblocks(p->T);
  a.nchunk = bsa::pbs_chunks(p->T);
  a.segment = p->segment;
  a.scale_log2 = attn_scale_of(p) * 1.4426950408889634f;
  const cudaError_t e =
      bsa::launch_pbs_permute(a, num_sms_current(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

bsa_status_t bsa_norm_rope(const bsa_tokens_t* t, bsa_rows_t q, bsa_rows_t q_out, bsa_rows_t k,
                           bsa_rows_t k_out, int32_t* dev_status, void* stream) {
  bsa_status_t st = check_tokens(t);
  if (st != BSA_OK) return st;
  if (t->N == 0) return BSA_OK;
  if (q.base == nullptr && k.base == nullptr) return BSA_ERR_INVALID_ARG;
  const int type = q.base != nullptr ? q.type : k.type;
  if (type != BSA_TYPE_BF16 && type != BSA_TYPE_F16 && type != BSA_TYPE_F32)
    return BSA_ERR_INVALID_ARG;
  bsa::HeadsArgs a = heads_args(t, type, dev_status);
  if (q.base != nullptr) {
    if ((st = check_rows(q, type)) != BSA_OK || (st = check_out(q_out, t, t->Hq)) != BSA_OK)
      return st;
    if (!same_or_apart(q, q_out)) return BSA_ERR_INVALID_ARG;
    a.q = rows_view(q);
    a.q_out = rows_view(q_out);
  }
  if (k.base != nullptr) {
    if ((st = check_rows(k, type)) != BSA_OK || (st = check_out(k_out, t, t->Hkv)) != BSA_OK)
      return st;
    if (!same_or_apart(k, k_out)) return BSA_ERR_INVALID_ARG;
    a.k = rows_view(k);
    a.k_out = rows_view(k_out);
  }
  // a row's sequence says its position, or whether it is padding
  a.needs_slot = t->cu_seqlens != nullptr || (t->positions == nullptr && t->rope_dim > 0);
  const cudaError_t e =
      bsa::launch_token_heads(a, num_sms_current(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

bsa_status_t bsa_append_kv(const bsa_tokens_t* t, bsa_rows_t k, bsa_rows_t v, bsa_rows_t kidx,
                           bsa_cache_t k_cache, bsa_cache_t v_cache, bsa_cache_t kidx_cache,
                           bsa_rows_t q, bsa_rows_t q_out, int32_t* dev_status, void* stream) {
  bsa_status_t st = check_tokens(t);
  if (st != BSA_OK) return st;
  if (t->N == 0) return BSA_OK;
  const int type = k.type;
  if (type != BSA_TYPE_BF16 && type != BSA_TYPE_F16 && type != BSA_TYPE_F32)
    return BSA_ERR_INVALID_ARG;
  if ((st = check_rows(k, type)) != BSA_OK || (st = check_rows(v, type)) != BSA_OK) return st;
  if ((st = check_append_cache(k_cache, t, t->d, true)) != BSA_OK) return st;
  if ((st = check_append_cache(v_cache, t, t->d, true)) != BSA_OK) return st;
  bsa::HeadsArgs a = heads_args(t, type, dev_status);
  a.k = rows_view(k);
  a.v = rows_view(v);
  a.k_cache = view(k_cache);
  a.v_cache = view(v_cache);
  if (kidx.base != nullptr) {
    if ((st = check_rows(kidx, type)) != BSA_OK) return st;
    if ((st = check_append_cache(kidx_cache, t, t->r, false)) != BSA_OK) return st;
    a.kidx = rows_view(kidx);
    a.kidx_cache = view(kidx_cache);
  }
  if (q.base != nullptr) {
    if ((st = check_rows(q, type)) != BSA_OK || (st = check_out(q_out, t, t->Hq)) != BSA_OK)
      return st;
    if (!same_or_apart(q, q_out)) return BSA_ERR_INVALID_ARG;
    a.q = rows_view(q);
    a.q_out = rows_view(q_out);
  }
  a.cached = 1;
  a.needs_slot = 1;
  const cudaError_t e =
      bsa::launch_token_heads(a, num_sms_current(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

bsa_status_t bsa_packed_workspace_size(const bsa_tokens_t* t, int32_t op, size_t* bytes) {
  if (bytes == nullptr) return BSA_ERR_INVALID_ARG;
  *bytes = 0;
  bsa_status_t st = check_tokens(t);
  if (st != BSA_OK) return st;
  if (op != BSA_OP_ATTEND_PACKED && op != BSA_OP_DECODE_SHARED) return BSA_ERR_INVALID_ARG;
  if (!is_pow2_group(t->Hq / t->Hkv)) return BSA_ERR_UNSUPPORTED;
  *bytes = packed_workspace(t, num_sms_current()).total;
  return BSA_OK;
}

bsa_status_t bsa_attend_packed(const bsa_tokens_t* t, const void* q, bsa_cache_t k, bsa_cache_t v,
                               void* o, float* lse, float* o_f32, void* workspace,
                               size_t workspace_bytes, int32_t* dev_status, void* stream) {
  return packed_attention(t, false, q, k, v, nullptr, nullptr, o, lse, o_f32, workspace,
                          workspace_bytes, dev_status, stream);
}

bsa_status_t bsa_decode_shared(const bsa_tokens_t* t, const void* q, bsa_cache_t k, bsa_cache_t v,
                               const float* o_own, const float* lse_own, void* o, float* lse,
                               float* o_f32, void* workspace, size_t workspace_bytes,
                               int32_t* dev_status, void* stream) {
  return packed_attention(t, true, q, k, v, o_own, lse_own, o, lse, o_f32, workspace,
                          workspace_bytes, dev_status, stream);
}

const char* bsa_status_string(bsa_status_t s) {
  switch (s) {
    case BSA_OK: return "ok";
    case BSA_ERR_INVALID_ARG: return "invalid argument";
    case BSA_ERR_UNSUPPORTED: return "unsupported shape or parameter";
    case BSA_ERR_WORKSPACE: return "workspace missing or too small";
    case BSA_ERR_CUDA: return "CUDA error";
    default: return "unknown status";
  }
}

const char* bsa_last_cuda_error(void) { return g_last_cuda_error; }

}  // extern "C"
