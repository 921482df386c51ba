// What the kernels of a sampling step (norms of query and key heads with their
// rotation, attention of requests that share a prefix) take, beyond serving.cuh.
#pragma once

#include "serving.cuh"

namespace fa {

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
  int tiles;           // of 128 keys from lo rounded down to a TMA box
  int kind;            // 0: a group's shared keys, 1: a request's own
};
// What a call's first kernel leaves for the others, in the workspace.
struct SharedPlan {
  int* count;          // [1] entries that have keys
  long long* total;    // [1] weight of all
  SharedEntry* entry;  // [G + B]
  long long* cum;      // [G + B + 1] weight before each entry
  int* of_group;       // [G] entry of its shared keys, -1: none
  int* of_request;     // [B] entry of its own keys
  int* group;          // [B] its group
  int* g_shared;       // [G] keys that the group shares (as used)
  int* start_entry;    // [shares] where each share begins
  long long* start_off;
};
struct SharedParams {
  const int* block_table;    // [B, max_blocks]
  const int* seq_lens;       // [B]
  const int* starts;         // [G + 1]
  const int* shared_lens;    // [G]
  void* o;                   // [B, Nq, Hq, d] bf16
  float* lse;                // [B, Hq, Nq]
  float* part_o;             // results of units inside one share, [4][rows][d] (shared / own keys, two runs each), then of
  float* part_lse;           //   the pieces that a share's borders cut, [2 * shares][2][128][d]: each normalised; log2 of its mass
  SharedPlan plan;
  int B, Nq, Hq, Hkv, heads; // heads: query heads of a K/V head
  int G, tile_tokens;        // groups; query tokens of a tile of rows
  int page_size, num_pages, max_blocks, max_len;
  int win_left;              // -1: no window
  int box_rows;              // keys per TMA box: 16 .. 128, divides the page and the tile
  int shares, lead;          // tiles that a unit counts for its start and end
  float scale_log2, tau;
  unsigned* err;
  unsigned long long timeout_ns;
};
size_t shared_plan_bytes(int B, int G, int shares);
void shared_plan_at(SharedPlan& plan, void* at, int B, int G, int shares);
bool make_tmap_queries(CUtensorMap* m, const void* ptr, int D, int Hq, long long tokens, int heads, int tile_tokens);
bool make_tmap_pages(CUtensorMap* m, const void* ptr, int D, int Hkv, int page_size, int num_pages, int box_rows);
cudaError_t launch_decode_shared(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const SharedParams& p,
                                 int D, cudaStream_t stream);

}  // namespace fa
