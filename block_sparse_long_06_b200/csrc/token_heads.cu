// Head norms with rotary positions, into tensors (bsa_norm_rope) or, with the values and
// index keys beside them, into the caches (bsa_append_kv).
//
// A head row x of d elements at position p:
//   y = x * w / sqrt(mean(x^2) + eps), then every pair (a, b) of the rotated part turns by
//   the angle p * f_i:  (a, b) -> factor * (a cos - b sin, b cos + a sin).
// The angle is kept in turns: f_i / 2pi as a 64-bit fraction, so p * step wraps to the
// fraction of a turn by itself and no far position loses digits (an fp32 product p * f is
// off by 0.06 rad at p = 2^20).
//
// One group of d/8 lanes holds one head, 8 elements a lane: 16-byte loads and stores of
// 16-bit types, the norm by shuffles inside the group. Halves of a head are rot/2 apart, a
// multiple of 8 elements, so a pair's other element is at the same place of another lane. A
// block takes a few token rows and all their heads: cos and sin of a row are computed once,
// into shared memory, and serve its Hq + Hkv heads. Each element is read and written once:
// the kernel is bound by HBM for many rows, by latency for few.
#include <type_traits>

#include "bsa_common.cuh"
#include "bsa_internal.h"

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTok = 4;             // token rows a block takes at most
constexpr int kAhead = 4;              // head rows in flight a lane group

template <typename In>
struct Raw8 {                          // 8 elements as loaded
  static constexpr int kWords = sizeof(In) * 2;
  uint32_t w[kWords];
};

template <typename In>
BSA_DEVFN Raw8<In> load8(const void* base, int64_t elem) {
  Raw8<In> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const In*>(base) + elem);
#pragma unroll
  for (int i = 0; i < Raw8<In>::kWords / 4; ++i) {
    const uint4 v = p[i];
    r.w[4 * i] = v.x;
    r.w[4 * i + 1] = v.y;
    r.w[4 * i + 2] = v.z;
    r.w[4 * i + 3] = v.w;
  }
  return r;
}

template <typename In>
BSA_DEVFN void widen(const Raw8<In>& r, float (&x)[8]) {
  if constexpr (std::is_same<In, float>::value) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 v;
      if constexpr (std::is_same<In, __half>::value)
        v = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
      else
        v = unpack_bf16(r.w[i]);
      x[2 * i] = v.x;
      x[2 * i + 1] = v.y;
    }
  }
}

// Sequence of row n: the last b with cu[b] <= n, by a 32-way search (one round of loads for
// up to 32 sequences, two for up to 1024). B when the row lies behind the last sequence.
BSA_DEVFN int sequence_of(const int32_t* cu, int B, int n, int lane) {
  int lo = 0, size = B;                // the answer is in [lo, lo + size]
  while (size > 0) {
    const int step = (size + 31) / 32;
    const int at = lo + min((lane + 1) * step, size);
    const bool below = (lane * step < size) && cu[at] <= n;   // all of [.., at) end by n
    const int hits = __popc(__ballot_sync(0xffffffffu, below));
    const int next = lo + min(hits * step, size);
    size = min(step - 1, lo + size - next);
    if (step == 1) size = 0;
    lo = next;
  }
  return lo;
}

// Element offset of token slot `pos` of (b, head 0) in cache c, or -1 where it is bad.
BSA_DEVFN int64_t slot_of(const CacheView& c, int b, int pos, int heads, int width) {
  int64_t phys = pos / kBlock;
  if (c.page_table != nullptr) {
    phys = c.page_table[static_cast<int64_t>(b) * c.pt_stride + pos / kBlock];
    if (phys < 0 || phys >= c.num_pages) return -1;
  }
  const int64_t off = static_cast<int64_t>(b) * c.seq_stride + phys * c.block_stride +
                      static_cast<int64_t>(pos % kBlock) * width;
  if (off < 0 || off + static_cast<int64_t>(heads - 1) * c.head_stride + width > c.extent) return -1;
  return off;
}

struct RowInfo {
  int64_t k, v, x;       // cache offsets of the row's slots (head 0), -1: not written
  int live;
};

template <int D, typename In>
__global__ void __launch_bounds__(kThreads) token_heads_kernel(const HeadsArgs a, const int tok_per_block) {
  constexpr int kLanes = D / 8;                  // lanes a head
  constexpr int kGroups = kThreads / kLanes;     // heads in flight a block
  __shared__ float2 turn[kMaxTok][D / 2];        // factor * (cos, sin) of each pair
  __shared__ RowInfo rows[kMaxTok];
  __shared__ int64_t where[kMaxTok];             // position the row is rotated to
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * tok_per_block;
  const int ntok = min(tok_per_block, a.N - n0);
  const int half = a.rope_dim / 2;

  if (warp < ntok) {                             // one warp a row: where it goes
    const int n = n0 + warp;
    RowInfo R = {-1, -1, -1, 1};
    int64_t pos = a.positions != nullptr ? a.positions[n] : 0;
    if (a.needs_slot) {
      const int b = a.cu != nullptr ? sequence_of(a.cu, a.B, n, lane) : n / (a.N / a.B);
      int64_t token = -1;
      if (b < a.B) {
        const int first = a.cu != nullptr ? a.cu[b] : b * (a.N / a.B);
        const int last = a.cu != nullptr ? a.cu[b + 1] : first + a.N / a.B;
        const int len = a.seq_lens != nullptr ? a.seq_lens[b] : a.T;
        token = static_cast<int64_t>(len) - (static_cast<int64_t>(last) - n);
        if (n < first || n >= last || last > a.N || len > a.T || token < 0) token = -1;
      }
      if (token < 0) {
        R.live = 0;
        if (b < a.B && lane == 0) report(a.status, BSA_DEV_BAD_LENGTH);
      } else if (a.cached) {
        R.k = slot_of(a.k_cache, b, static_cast<int>(token), a.Hkv, D);
        R.v = slot_of(a.v_cache, b, static_cast<int>(token), a.Hkv, D);
        if (a.kidx.base != nullptr) R.x = slot_of(a.kidx_cache, b, static_cast<int>(token), a.Hkv, kR);
        if (lane == 0 && (R.k < 0 || R.v < 0 || (a.kidx.base != nullptr && R.x < 0)))
          report(a.status, BSA_DEV_BAD_PAGE);
      }
      if (a.positions == nullptr) pos = token;
    }
    if (lane == 0) {
      rows[warp] = R;
      where[warp] = pos;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < ntok * half; i += kThreads) {
    const int t = i / half, p = i - t * half;
    // the fraction of a turn, in 2^-64 turns; its top 32 bits as a signed half turn
    const uint64_t angle = static_cast<uint64_t>(where[t]) * a.rope_steps[p];
    const float x = static_cast<float>(static_cast<int32_t>(angle >> 32)) * 4.656612873077393e-10f;
    float s, c;
    sincospif(x, &s, &c);                        // x = angle / pi in [-1, 1)
    turn[t][p] = make_float2(c * a.rope_factor, s * a.rope_factor);
  }
  __syncthreads();

  // head rows of the block: per token q heads, k heads and (to the caches) v heads
  const int sub = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int nq = a.q.base != nullptr ? a.Hq : 0, nk = a.k.base != nullptr ? a.Hkv : 0;
  const int nv = a.cached ? a.Hkv : 0;
  const int per_tok = nq + nk + nv, total = ntok * per_tok;
  const int parts = half / 8;                    // lanes that hold one half of the rotated part
  float wq[8], wk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wq[i] = a.q_weight != nullptr ? a.q_weight[sub * 8 + i] : 1.f;
    wk[i] = a.k_weight != nullptr ? a.k_weight[sub * 8 + i] : 1.f;
  }
  // the whole block runs the loop the same number of times: the shuffles need every lane
  for (int base = 0; base < total; base += kGroups * kAhead) {
    Raw8<In> raw[kAhead];
    int tok[kAhead], head[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int item = base + u * kGroups + group;
      tok[u] = item < total ? item / per_tok : -1;
      head[u] = item - tok[u] * per_tok;
      if (tok[u] >= 0 && !rows[tok[u]].live) tok[u] = -1;
      if (tok[u] >= 0) {
        const int64_t n = n0 + tok[u];
        const int h = head[u];
        const RowsView& src = h < nq ? a.q : h < nq + nk ? a.k : a.v;
        const int hh = h < nq ? h : h < nq + nk ? h - nq : h - nq - nk;
        raw[u] = load8<In>(src.base, n * src.token_stride + hh * src.head_stride + sub * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (base + u * kGroups >= total) break;    // the same for the whole block
      float x[8];
      if (tok[u] >= 0) {
        widen<In>(raw[u], x);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
      }
      const int h = head[u];
      const bool is_q = h < nq, is_v = h >= nq + nk;
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
        if (!is_v) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= inv * (is_q ? wq[i] : wk[i]);
        }
      }
      if (half > 0) {
        const int t = tok[u] >= 0 ? tok[u] : 0;
        if (a.rope_interleaved) {
          if (sub < 2 * parts && !is_v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 cs = turn[t][sub * 4 + i];
              const float p = x[2 * i], r = x[2 * i + 1];
              x[2 * i] = p * cs.x - r * cs.y;
              x[2 * i + 1] = r * cs.x + p * cs.y;
            }
          }
        } else {
          // the lane with the other element of each pair
          const int other = sub < parts ? sub + parts : sub < 2 * parts ? sub - parts : sub;
          const int src = (lane & ~(kLanes - 1)) + other;
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], src);
          if (sub < 2 * parts && !is_v) {
            const int first = (sub < parts ? sub : sub - parts) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 cs = turn[t][first + i];
              x[i] = x[i] * cs.x + (sub < parts ? -y[i] : y[i]) * cs.y;
            }
          }
        }
      }
      if (tok[u] < 0) continue;
      const uint4 out = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                   pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
      const int64_t n = n0 + tok[u];
      __nv_bfloat16* dst = nullptr;
      if (is_q) {
        dst = static_cast<__nv_bfloat16*>(a.q_out.base) + n * a.q_out.token_stride + h * a.q_out.head_stride;
      } else if (!a.cached) {
        dst = static_cast<__nv_bfloat16*>(a.k_out.base) + n * a.k_out.token_stride +
              (h - nq) * a.k_out.head_stride;
      } else {
        const CacheView& c = is_v ? a.v_cache : a.k_cache;
        const int64_t off = is_v ? rows[tok[u]].v : rows[tok[u]].k;
        if (off >= 0)
          dst = static_cast<__nv_bfloat16*>(const_cast<void*>(c.base)) + off +
                static_cast<int64_t>(h - nq - (is_v ? nk : 0)) * c.head_stride;
      }
      if (dst != nullptr) *reinterpret_cast<uint4*>(dst + sub * 8) = out;
    }
  }

  // index keys: two lanes a head
  if (a.cached && a.kidx.base != nullptr) {
    for (int i = threadIdx.x; i < ntok * a.Hkv * 2; i += kThreads) {
      const int t = i / (a.Hkv * 2), h = (i >> 1) % a.Hkv, c8 = (i & 1) * 8;
      if (!rows[t].live || rows[t].x < 0) continue;
      const int64_t n = n0 + t;
      const Raw8<In> r = load8<In>(a.kidx.base, n * a.kidx.token_stride + h * a.kidx.head_stride + c8);
      float x[8];
      widen<In>(r, x);
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(const_cast<void*>(a.kidx_cache.base)) +
                           rows[t].x + static_cast<int64_t>(h) * a.kidx_cache.head_stride + c8;
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                  pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
  }
}

template <int D>
cudaError_t launch_d(const HeadsArgs& a, int num_sms, cudaStream_t s) {
  // one row a block while that leaves SMs idle (decode), four rows (one cos/sin a thread at
  // d = 128) where there are many
  const int tok = a.N >= 4 * num_sms * kMaxTok ? kMaxTok : 1;
  const dim3 grid((a.N + tok - 1) / tok);
  switch (a.type) {
    case BSA_TYPE_BF16: return launch_pdl(token_heads_kernel<D, __nv_bfloat16>, grid, dim3(kThreads), 0, s, a, tok);
    case BSA_TYPE_F16: return launch_pdl(token_heads_kernel<D, __half>, grid, dim3(kThreads), 0, s, a, tok);
    default: return launch_pdl(token_heads_kernel<D, float>, grid, dim3(kThreads), 0, s, a, tok);
  }
}

}  // namespace

cudaError_t launch_token_heads(const HeadsArgs& a, int num_sms, cudaStream_t s) {
  return a.d == 128 ? launch_d<128>(a, num_sms, s) : launch_d<64>(a, num_sms, s);
}

}  // namespace bsa
