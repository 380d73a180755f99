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
// One group of d/8 lanes holds one head, two runs of 4 elements a lane: where pairs are rot/2
// apart the runs are too, so that both elements of a pair are in the same lane (no exchange),
// and a group's runs still cover whole 32-byte sectors. The norm's sum goes through shuffles
// inside the group. A warp takes heads of one token row, so its cos and sin stay in registers
// for all of them, and the loads of four heads a lane are in flight. Each element is read and
// written once: the kernel is bound by HBM for many rows, by latency for few, where several
// warps share a row's heads.
#include <type_traits>

#include "tokens_common.cuh"
#include "tokens_internal.h"

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;              // head rows in flight a lane group

template <typename In>
struct Run4 {                          // 4 elements as loaded
  static constexpr int kWords = sizeof(In);
  uint32_t w[kWords];
};

template <typename In>
BSA_DEVFN Run4<In> load4(const In* from) {
  Run4<In> r;
  if constexpr (sizeof(In) == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(from);
    r.w[0] = v.x;
    r.w[1] = v.y;
    r.w[2] = v.z;
    r.w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(from);
    r.w[0] = v.x;
    r.w[1] = v.y;
  }
  return r;
}

template <typename In>
BSA_DEVFN void widen(const Run4<In>& r, float* x) {
  if constexpr (std::is_same<In, float>::value) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
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

BSA_DEVFN void store4(__nv_bfloat16* to, const float* x) {
  *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
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

// share: warps that share a row's heads (a power of two up to kWarps).
// 32 warps an SM where the registers of 4 heads in flight allow it (measured at 65,536 rows of
// 40 bf16 heads: 242 us, with 24 warps 261; fp32 spills at 32: 20.0 us against 17.2 at 5003 rows).
template <int D, typename In>
__global__ void __launch_bounds__(kThreads, sizeof(In) == 4 ? 3 : 4) token_heads_kernel(const HeadsArgs a, const int share) {
  constexpr int kLanes = D / 8;                  // lanes a head
  constexpr int kHeads = 32 / kLanes;            // heads a warp holds at a time
  __shared__ float2 turns[kWarps][D / 2];        // factor * (cos, sin) of the warp's row
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int n = static_cast<int>(unit / share), part = static_cast<int>(unit % share);
  if (n >= a.N) return;
  const int sub = lane % kLanes;
  const int base = part * kHeads;                // of the warp's first heads
  const int stride = share * kHeads;
  // the lane's two runs of elements
  const int half = a.rope_dim / 2;
  const bool apart = !a.rope_interleaved && sub < half / 4;
  const int run0 = apart ? sub * 4 : sub * 8, run1 = apart ? half + sub * 4 : sub * 8 + 4;

  // the row's sequence, token number, slots and position
  int64_t kslot = -1, vslot = -1, xslot = -1;
  int64_t pos = a.positions != nullptr ? a.positions[n] : 0;
  if (a.needs_slot) {
    const int each = a.N / a.B;
    const int b = a.cu != nullptr ? sequence_of(a.cu, a.B, n, lane) : n / each;
    if (b >= a.B) return;                        // padding
    const int row0 = a.cu != nullptr ? a.cu[b] : b * each;
    const int row1 = a.cu != nullptr ? a.cu[b + 1] : row0 + each;
    const int len = a.seq_lens != nullptr ? a.seq_lens[b] : a.T;
    const int64_t token = static_cast<int64_t>(len) - (static_cast<int64_t>(row1) - n);
    if (n < row0 || n >= row1 || row1 > a.N || len > a.T || token < 0) {
      if (lane == 0) report(a.status, BSA_DEV_BAD_LENGTH);
      return;
    }
    if (a.cached) {
      kslot = slot_of(a.k_cache, b, static_cast<int>(token), a.Hkv, D);
      vslot = slot_of(a.v_cache, b, static_cast<int>(token), a.Hkv, D);
      if (a.kidx.base != nullptr) xslot = slot_of(a.kidx_cache, b, static_cast<int>(token), a.Hkv, kR);
      if (kslot < 0 || vslot < 0 || (a.kidx.base != nullptr && xslot < 0)) {
        if (lane == 0) report(a.status, BSA_DEV_BAD_PAGE);
        kslot = vslot = xslot = -1;              // all of a token's slots or none
      }
    }
    if (a.positions == nullptr) pos = token;
  }

  // cos and sin of the row, two pairs a lane, then those of the lane's 4 pairs in registers
  float2 cs[4];
  if (half > 0) {
    for (int p = lane; p < half; p += 32) {
      // the fraction of a turn, in 2^-64 turns; its top 32 bits as a signed half turn
      const uint64_t angle = static_cast<uint64_t>(pos) * a.rope_steps[p];
      const float x = static_cast<float>(static_cast<int32_t>(angle >> 32)) * 4.656612873077393e-10f;
      float s, c;
      sincospif(x, &s, &c);                      // x = angle / pi in [-1, 1)
      turns[warp][p] = make_float2(c * a.rope_factor, s * a.rope_factor);
    }
    __syncwarp();
  }
  const bool turned = sub < half / 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = turned ? turns[warp][sub * 4 + i] : make_float2(1.f, 0.f);

  // Heads of one kind: from `src` to `dst` (null: nowhere), both at the row. w: norm weights.
  // The lane groups run the loop the same number of times: the shuffles need the whole warp.
  auto heads = [&](auto prepare, const RowsView& from, int count, __nv_bfloat16* dst, int64_t dst_step,
                   const float* w) {
    constexpr bool kPrepare = decltype(prepare)::value;
    const In* src = static_cast<const In*>(from.base) + n * from.token_stride;
    float wt[8];
    if constexpr (kPrepare) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wt[i] = w != nullptr ? w[run0 + i] : 1.f;
        wt[4 + i] = w != nullptr ? w[run1 + i] : 1.f;
      }
    }
    for (int h0 = base; h0 < count; h0 += stride * kAhead) {
      Run4<In> r0[kAhead], r1[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int h = min(h0 + u * stride + lane / kLanes, count - 1);
        r0[u] = load4<In>(src + h * from.head_stride + run0);
        r1[u] = load4<In>(src + h * from.head_stride + run1);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (h0 + u * stride >= count) break;     // the same for the whole warp
        float x[8];
        widen<In>(r0[u], x);
        widen<In>(r1[u], x + 4);
        if constexpr (kPrepare) {
          if (a.norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= inv * wt[i];
          }
          if (turned && a.rope_interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {        // pairs next to each other
              const float p = x[2 * i], q = x[2 * i + 1];
              x[2 * i] = p * cs[i].x - q * cs[i].y;
              x[2 * i + 1] = q * cs[i].x + p * cs[i].y;
            }
          } else if (turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {        // across the two runs
              const float p = x[i], q = x[4 + i];
              x[i] = p * cs[i].x - q * cs[i].y;
              x[4 + i] = q * cs[i].x + p * cs[i].y;
            }
          }
        }
        const int h = h0 + u * stride + lane / kLanes;
        if (h < count && dst != nullptr) {
          store4(dst + h * dst_step + run0, x);
          store4(dst + h * dst_step + run1, x + 4);
        }
      }
    }
  };
  using Out = __nv_bfloat16;
  const std::true_type prepared;
  const std::false_type copied;
  if (a.q.base != nullptr)
    heads(prepared, a.q, a.Hq, static_cast<Out*>(a.q_out.base) + n * a.q_out.token_stride,
          a.q_out.head_stride, a.q_weight);
  if (a.cached) {
    Out* kbase = static_cast<Out*>(const_cast<void*>(a.k_cache.base));
    Out* vbase = static_cast<Out*>(const_cast<void*>(a.v_cache.base));
    heads(prepared, a.k, a.Hkv, kslot < 0 ? nullptr : kbase + kslot, a.k_cache.head_stride, a.k_weight);
    heads(copied, a.v, a.Hkv, vslot < 0 ? nullptr : vbase + vslot, a.v_cache.head_stride, nullptr);
    // index keys: two lanes a head
    if (xslot >= 0) {
      Out* xbase = static_cast<Out*>(const_cast<void*>(a.kidx_cache.base)) + xslot;
      for (int i = part * 32 + lane; i < a.Hkv * 2; i += share * 32) {
        const int h = i >> 1, c8 = (i & 1) * 8;
        const In* src = static_cast<const In*>(a.kidx.base) + n * a.kidx.token_stride +
                        h * a.kidx.head_stride + c8;
        float x[8];
        widen<In>(load4<In>(src), x);
        widen<In>(load4<In>(src + 4), x + 4);
        store4(xbase + h * a.kidx_cache.head_stride + c8, x);
        store4(xbase + h * a.kidx_cache.head_stride + c8 + 4, x + 4);
      }
    }
  } else if (a.k.base != nullptr) {
    heads(prepared, a.k, a.Hkv, static_cast<Out*>(a.k_out.base) + n * a.k_out.token_stride,
          a.k_out.head_stride, a.k_weight);
  }
}

template <int D>
cudaError_t launch_d(const HeadsArgs& a, int num_sms, cudaStream_t s) {
  // warps that share a row: as many as it has work for while that leaves SMs with less than
  // 16 warps
  const int heads = a.Hq + 2 * a.Hkv, per = 32 / (D / 8);
  int share = 1;
  while (share < kWarps && share * per < heads && static_cast<int64_t>(a.N) * share * 2 <= 16ll * num_sms)
    share *= 2;
  const int64_t warps = static_cast<int64_t>(a.N) * share;
  const dim3 grid(static_cast<unsigned>((warps + kWarps - 1) / kWarps));
  switch (a.type) {
    case BSA_TYPE_BF16: return launch_pdl(token_heads_kernel<D, __nv_bfloat16>, grid, dim3(kThreads), 0, s, a, share);
    case BSA_TYPE_F16: return launch_pdl(token_heads_kernel<D, __half>, grid, dim3(kThreads), 0, s, a, share);
    default: return launch_pdl(token_heads_kernel<D, float>, grid, dim3(kThreads), 0, s, a, share);
  }
}

}  // namespace

cudaError_t launch_token_heads(const HeadsArgs& a, int num_sms, cudaStream_t s) {
  return a.d == 128 ? launch_d<128>(a, num_sms, s) : launch_d<64>(a, num_sms, s);
}

}  // namespace bsa
