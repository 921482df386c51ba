// What the kernels of a sampling step (norms of query and key heads with their
// rotation, attention of requests that share a prefix) take, beyond serving.cuh.
#pragma once

#include "serving.cuh"

namespace fa {

// a / b for a >= 0, b > 0, in 32 bits where both fit
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  return (((unsigned long long)a | (unsigned long long)b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// Norms of heads with the rotation (see fa_qk_norm_rope in fa.h).
struct NormRopeParams {
  const void* q;             // inputs of the forward
  const void* k;
  const void* dyq;           // gradients of its outputs (backward)
  const void* dyk;
  void* q_out;               // outputs, or the gradients of the inputs
  void* k_out;
  const void* wq;            // [d] bf16, or fp32 with w_fp32
  const void* wk;
  const int* positions;      // [n_axes, T]
  float* dw_part;            // backward: [blocks, d] sums of each block, q's blocks first
  long long q_stride, k_stride, dyq_stride, dyk_stride, q_out_stride, k_out_stride;  // elements between rows
  int T, Hq, Hkv;
  int w_fp32;
  float eps;
  int heads_per_thread;      // set by the launch
  int q_chunks, k_chunks;    //   thread chunks of a token's query and of its key heads
  int q_blocks;              //   blocks that work on query heads (backward)
  signed char axis[64];      // axis of pair p, -1: not rotated
  uint64_t turn[64];         // its frequency: fraction of a turn per position, in 2^-64
};
cudaError_t launch_norm_rope(NormRopeParams& p, int D, bool neighbours, cudaStream_t stream);
int norm_rope_bwd_blocks(int T, int Hq, int Hkv, int D, int* q_blocks);  // blocks of the backward, those of q's heads
cudaError_t launch_norm_rope_bwd(NormRopeParams& p, int D, bool neighbours, float* dwq, float* dwk, cudaStream_t stream);

// Attention of requests that share prefixes (see fa_decode_paged_shared in fa.h).
constexpr int kSharedTile = 128;  // keys per tile, rows per tile of rows

// Keys that the query tokens of an entry meet together: a group's shared keys,
// or a request's own.
struct SharedEntry {
  int tok0, ntok;      // query tokens tok0 .. tok0 + ntok - 1 (token = request * Nq + its query)
  int row;             // of the block table
  int lo, end;         // keys
  int all_lo, all_hi;  // the keys that every query token (of a request with keys) sees, if any
  int tiles;           // of 128 keys from lo rounded down to a TMA box; few rows: of 16 keys
  int kind;            // 0: a group's shared keys, 1: a request's own
};
struct SharedList {
  SharedEntry* entry;  // those that have keys
  long long* cum;      // weight before each
};
struct SharedHead {
  long long total[3];  // weight of the entries with many rows, of those with few dealt early, and late
  int shares[3];       // they are dealt to: CTAs, warps
  int count[2];        // entries of the lists
  int queue;           // shares of few rows that warps have taken
};
// What a call's first kernel leaves for the others, in the workspace.
struct SharedPlan {
  SharedHead* head;
  SharedList list[2];  // [G + B] entries with many rows, with few
  int2* of_request;    // [B] entries of its group's shared keys and of its own: 2 number + list, -1: none
  int* g_shared;       // [G] keys that the group shares, its entry of them, the keys of its shortest request (that has
  int* g_of;           //   some), of its longest: where groups are too many for the first kernel's shared memory
  int* g_least;
  unsigned long long* g_most;
};
struct SharedParams {
  const int* block_table;    // [B, max_blocks]
  const int* seq_lens;       // [B]
  const int* starts;         // [G + 1]
  const int* shared_lens;    // [G]
  const float* k_scale;      // [num_pages, Hkv], of 8-bit pages
  const float* v_scale;
  const void* q;             // [B, Nq, Hq, d] bf16
  void* o;                   // the same
  float* lse;                // [B, Hq, Nq]
  float* part_o;             // results of units inside one share, [4][rows][d] (shared / own keys, two runs each), then of the
  float* part_lse;           //   pieces that shares' borders cut, two a share, [2][128][d] of many rows, [few][d] of few: each
                             //   normalised; log2 of its mass
  SharedPlan plan;
  int B, Nq, Hq, Hkv, heads; // heads: query heads of a K/V head
  int G, tile_tokens;        // groups; query tokens of a tile of rows
  int page_size, num_pages, max_blocks, max_len;
  int win_left;              // -1: no window
  int box_rows;              // keys per TMA box: 16 .. 128, divides the page and the tile
  int shares;                // CTAs
  int warps;                 // of a CTA, that attend for few rows
  int few;                   // most rows of an entry that a warp attends for: 0, 8 or 16
  float few_cost;            // of a CTA's time a slot of few rows' weight takes
  float scale_log2, tau;
  unsigned* err;
  unsigned long long timeout_ns;
};
int shared_few(int Nq, int heads, int D, bool kv8);
size_t shared_part_rows(int B, int Nq, int Hq, int heads, int shares);
size_t shared_plan_bytes(int B, int G);
void shared_plan_at(SharedPlan& plan, void* at, int B, int G);
bool make_tmap_queries(CUtensorMap* m, const void* ptr, int D, int Hq, long long tokens, int heads, int tile_tokens);
bool make_tmap_pages(CUtensorMap* m, const void* ptr, int D, int Hkv, int page_size, int num_pages, int box_rows);
cudaError_t launch_decode_shared(const CUtensorMap (&maps)[5], SharedParams& p, int D, bool kv8, cudaStream_t stream);  // q; k, v; k, v by 16 keys

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2, int c3,
                                            int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
// Whether the phase with the given parity has completed (mbar_try_wait may wait a while for it).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// As tmem_ld32_max, of 16 columns.
__device__ __forceinline__ void tmem_ld16_max(uint32_t taddr, uint32_t* r, float& m) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, [%17];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=f"(m)
      : "r"(taddr));
}
// As idesc_bf16, with f16 inputs.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16(M, N, a_mn, b_mn) & ~(1u << 7 | 1u << 10);
}

// Four e4m3 codes as f16, exactly, in their order.
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(x));
}

}  // namespace fa
