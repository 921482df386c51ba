// What the kernels of a serving step (page planning, rotary positions, the
// 8-bit cache and the attention over it) share beyond ptx.cuh: their launch
// parameters and a few more instructions.
#pragma once

#include <cuda_fp16.h>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

constexpr int kSms = 152;  // of a GB300: the rules that fill it were measured there
constexpr unsigned FA_DEVERR_OUT_OF_PAGES = 0x2002u;  // a plan needs more pages than the free stack has

// Planning a step (see fa_page_plan in fa.h).
constexpr int kPlanMaxB = 16384;  // requests at most
struct PlanParams {
  const int* ctx_lens;       // [B]
  const int* new_lens;       // [B]
  const int* free_pages;     // [num_pages]
  const int* free_count;     // [1]
  int* block_table;          // [B, max_blocks]
  int* seq_lens;             // [B], may be ctx_lens
  int* cu_new;               // [B + 1]
  int* page;                 // [max_tokens] x 3
  int* slot;
  int* position;
  int* free_count_out;       // [1], may be free_count
  int B;
  int max_tokens;
  int page_size;
  int num_pages;
  int max_blocks;
  int totals_later;          // set by the launch: seq_lens and free_count_out come from a second kernel
  unsigned* err;
};
cudaError_t launch_page_plan(PlanParams& p, cudaStream_t stream);

// Rotary positions (see fa_rope_axes in fa.h).
struct RopeParams {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const int* positions;      // [n_axes, T]
  long long q_stride, k_stride, q_out_stride, k_out_stride;  // elements between rows
  int T, Hq, Hkv;
  int inverse;
  int heads_per_thread;      // set by the launch
  int chunks;                //   thread chunks of a token's Hq + Hkv heads
  signed char axis[64];      // axis of pair p, -1: not rotated
  uint64_t turn[64];         // its frequency: fraction of a turn per position, in 2^-64
};
cudaError_t launch_rope(RopeParams& p, int D, bool neighbours, cudaStream_t stream);

// 8-bit paged cache, write side (see fa_kv8_append in fa.h).
struct Kv8AppendParams {
  const void* k_new;
  const void* v_new;
  void* k_codes;
  void* v_codes;
  float* k_scale;
  float* v_scale;
  const int* page;           // [n]
  const int* slot;           // [n]
  const int* copy_src;       // [n] or nullptr
  long long k_stride, v_stride;
  int n, Hkv, page_size, num_pages;
  int split;                 // warps that share 32 rows' runs, set by the launch
  unsigned* err;
};
cudaError_t launch_kv8_append(Kv8AppendParams& p, int D, cudaStream_t stream);

// Attention over the 8-bit paged cache (see fa_decode_kv8 in fa.h).
constexpr int kKv8Tile = 128;  // keys per tile
struct Kv8DecodeParams {
  const void* q;             // [B, Nq, Hq, d] bf16
  const uint8_t* k_codes;    // [num_pages, Hkv, page_size, d]
  const uint8_t* v_codes;
  const float* k_scale;      // [num_pages, Hkv]
  const float* v_scale;
  const int* block_table;    // [B, max_blocks]
  const int* seq_lens;       // [B]
  void* o;
  float* lse;
  float* part_o;             // [2 * shares, RT, d] fp32: the pieces a share's borders cut, each normalised
  float* part_lse;           // [2 * shares, RT] log2 of each piece's softmax mass
  int B, Nq, Hq, Hkv, group;
  int page_size, num_pages, max_blocks, max_len;
  int win_left;              // -1: no window
  int box_rows;              // keys per TMA box: 16 .. 128, divides the page and the tile
  int lead;                  // tiles that a unit counts for its start and end, set by the launch
  int row_tiles;             // tiles of query rows per K/V head, set by the launch
  float scale_log2;
  unsigned* err;
  unsigned long long timeout_ns;
};
int kv8_auto_shares(int B, int Nq, int Hkv, int group, int span);
int kv8_most_shares(int Nq, int group);  // that kv8_auto_shares can choose on the current device
int kv8_row_tile(int rows);  // query rows of a CTA for `rows` rows per K/V head
// 3-D uint8 tensor map of the codes, [heads of pages][page_size][D], swizzled at the row's length.
bool make_tmap_codes(CUtensorMap* m, const void* ptr, int D, int page_size, long long page_heads, int box_rows);
cudaError_t launch_decode_kv8(const CUtensorMap& tk, const CUtensorMap& tv, Kv8DecodeParams& p, int D, int shares, int span,
                              cudaStream_t stream);

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Four bytes global -> shared without a register; cp_async_arrive has the
// thread's earlier ones, when they are there, arrive once on an mbarrier.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// As smem_desc_sw128, for rows of 64 bytes and the 64-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo_bytes >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo_bytes >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1u << 46;  // descriptor version for tcgen05
  d |= (uint64_t)4u << 61;  // swizzle mode: 64-byte
  return d;
}

// The same for rows of 32 bytes and the 32-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc_sw32(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo_bytes >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo_bytes >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1u << 46;  // descriptor version for tcgen05
  d |= (uint64_t)6u << 61;  // swizzle mode: 32-byte
  return d;
}

// Instruction descriptor for kind::f8f6f4 with e4m3 operands, either of them MN-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
  return idesc_e4m3(M, N) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16);
}

// The same with A of e4m3 and B of e5m2.
__host__ __device__ constexpr uint32_t idesc_e4m3_e5m2(int M, int N, bool a_mn, bool b_mn) {
  return idesc_e4m3(M, N, a_mn, b_mn) | (1u << 10);
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

// Two floats -> two e4m3 codes, e0 in the low byte; two codes -> their values, exact.
__device__ __forceinline__ uint32_t pack_e4m3x2(float e0, float e1) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(e0), "f"(e1));
  return r;
}
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Two floats -> f16x2, e0 in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float e0, float e1) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(h) : "f"(e0), "f"(e1));
  return h;
}
// Two f16 whose upper bytes are the nearest e5m2 to the given ones, below 61440 in
// magnitude (a tie goes up; a NaN does not stay one, but 0x7fff, as conversions
// and arithmetic make it, carries nothing into its neighbour); and `more` times what
// those bytes leave, exact where it is no subnormal.
__device__ __forceinline__ uint32_t e5m2_round(uint32_t two) { return two + 0x00800080u; }
__device__ __forceinline__ uint32_t e5m2_rest(uint32_t two, uint32_t rounded, float more) {
  const uint32_t up = rounded & 0xff00ff00u;
  const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&two), *reinterpret_cast<const __half2*>(&up));
  const __half2 r = __hmul2(rest, __float2half2_rn(more));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The largest of a warp's 32 values, in every lane.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

}  // namespace fa
