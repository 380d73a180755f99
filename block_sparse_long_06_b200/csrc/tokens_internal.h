// Internal launch interface of the operators on new token rows (token_heads.cu,
// packed_attn.cu), as bsa_internal.h is for the other kernels.
#pragma once

#include "bsa_internal.h"

namespace bsa {

// Device-side copy of a bsa_rows_t.
struct RowsView {
  void* base;
  int64_t token_stride, head_stride;
};

// Head norms and rotary positions of new token rows, into tensors or the caches.
struct HeadsArgs {
  RowsView q, k, v, kidx;     // inputs of one type (bsa_type_t); base null: none
  RowsView q_out, k_out;      // bf16; k_out unused when `cached`
  CacheView k_cache, v_cache, kidx_cache;   // when `cached`: where k, v and kidx go
  const int32_t* cu;          // [B+1] or null
  const int32_t* seq_lens;    // [B] or null
  const int32_t* positions;   // [N] or null
  const uint64_t* rope_steps; // [rope_dim / 2]
  const float* q_weight;      // [d] or null
  const float* k_weight;      // [d] or null
  int32_t* status;
  int N, B, Hq, Hkv, d, T, type, cached, needs_slot;   // needs_slot: rows look up their sequence
  int rope_dim, rope_interleaved, norm;
  float rope_factor, eps;
};

// Dense attention of packed rows (workspace pointers: the plan kernel's results, partials).
struct PackedArgs {
  const void* q;
  CacheView k, v;
  const int32_t* cu;          // [B+1] or null
  const int32_t* seq_lens;    // [B] or null
  const float* o_own;         // [N, Hq, d] or null: joined by who writes the row
  const float* lse_own;       // [N, Hq]
  void* o;                    // [N, Hq, d] bf16
  float* lse;                 // [N, Hq]
  float* o_f32;               // [N, Hq, d] or null
  int32_t* status;
  int32_t* head;              // plan: [0] entries, [1] unit counter, [2] any row split, [3] no unit has two tiles
  int32_t* offs;              // plan: [B+1] first tile of each sequence
  int4* entries;              // plan: two int4 an entry
  int32_t* row_splits;        // plan: [N] partial results of each row (0: row not written)
  float* part_ml;             // [smax, N, Hq, 2] (max, sum) in log2 units
  float* part_o;              // [smax, N, Hq, d] fp32, not normalised
  int N, B, Hq, Hkv, G, d, T, causal, smax;
  int in_block;               // few tiles: every block plans for itself
  int max_entries, num_sms, lgG;   // lgG: log2(G)
  int k_safe, v_safe;         // every page (or block) of the cache lies inside its extent
  float scale_log2;
  int p_parts;                // bf16 parts of P: 1 or 2
};

cudaError_t launch_token_heads(const HeadsArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_packed(const PackedArgs& a, const CUtensorMap& tq, const CUtensorMap& tk,
                          const CUtensorMap& tv, int num_sms, cudaStream_t s);
// Query rows (tokens) of one unit of the packed attention: two tiles of 128 (token, head) rows.
constexpr int packed_unit_tokens(int G) { return 256 / G; }

}  // namespace bsa
