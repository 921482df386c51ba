// Attention of a few query tokens per request over the 8-bit paged cache.
//     s_j = scale * k_scale(page_j) * q . k8_j
//     O = sum_j softmax(s)_j * v_scale(page_j) * v8_j,   lse = log sum_j e^(s_j)
// A CTA takes a chunk of one request's keys for one query row and leaves a
// normalised partial (O_c, lse_c in base 2); a second kernel merges the
// partials, lse = log sum_c e^(lse_c), O = sum_c e^(lse_c - lse) O_c.
#include "fa_internal.h"
#include "ptx.cuh"

#include <cmath>
#include <cuda_fp16.h>

namespace fa {

namespace {

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A request's length as the kernels use it: clamped into [0, max_len], a length outside reported.
__device__ __forceinline__ int kv8_len(const Kv8DecodeParams& p, int b, bool report) {
  int n = p.seq_lens[b];
  if (n < 0 || n > p.max_len) {
    if (report) atomicCAS(p.err, 0u, FA_DEVERR_BAD_SEQLEN);
    n = n < 0 ? 0 : p.max_len;
  }
  return n;
}

// First key any of the request's queries sees, rounded down to a tile.
__device__ __forceinline__ int kv8_begin(const Kv8DecodeParams& p, int len) {
  if (p.win_left < 0) return 0;
  const int lo = len - p.Nq - p.win_left;
  return lo <= 0 ? 0 : lo / kKv8Tile * kKv8Tile;
}

}  // namespace

// Simple form: one warp per (query row, chunk), a lane holding d / 32 elements.
template <int D>
__global__ void __launch_bounds__(128) fa_decode_kv8_simple_kernel(const __grid_constant__ Kv8DecodeParams p) {
  constexpr int E = D / 32;
  const int lane = lane_id(), warp = threadIdx.x >> 5;
  const int b = blockIdx.y, c = blockIdx.x;
  const int r = (int)blockIdx.z * 4 + warp;  // (query token, head)
  if (r >= p.Nq * p.Hq) return;
  const int iq = r / p.Hq, h = r - iq * p.Hq, hk = h / p.group;
  const int len = kv8_len(p, b, threadIdx.x == 0);
  const int beg = kv8_begin(p, len) + c * p.chunk, end = min(len, beg + p.chunk);
  const int pos = len - p.Nq + iq;
  const size_t row = ((size_t)b * p.Nq + iq) * p.Hq + h;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[row * D + lane * E + e]) * p.scale_log2;
    o[e] = 0.f;
  }
  const int lo = p.win_left >= 0 ? max(beg, pos - p.win_left) : beg;
  for (int j = lo; j < end && j <= pos; ++j) {
    int page = p.block_table[(size_t)b * p.max_blocks + j / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) atomicCAS(p.err, 0u, FA_DEVERR_BAD_PAGE);
      page = 0;
    }
    const size_t ph = (size_t)page * p.Hkv + hk, at = (ph * p.page_size + j % p.page_size) * D + lane * E;
    float s = 0.f, kf[E], vf[E];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 a = e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(p.k_codes + at + e));
      const float2 v = e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(p.v_codes + at + e));
      kf[e] = a.x, kf[e + 1] = a.y, vf[e] = v.x, vf[e + 1] = v.y;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], kf[e], s);
#pragma unroll
    for (int t = 16; t > 0; t >>= 1) s += __shfl_xor_sync(0xffffffffu, s, t);
    s *= p.k_scale[ph];
    const float mn = fmaxf(m, s), al = ex2_sfu(m - mn), w = ex2_sfu(s - mn), wv = w * p.v_scale[ph];
    l = fmaf(l, al, w);
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], al, wv * vf[e]);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) p.part_o[(row * p.splits + c) * D + lane * E + e] = o[e] * inv;
  if (lane == 0) p.part_lse[row * p.splits + c] = l > 0.f ? m + __log2f(l) : -INFINITY;
}

// Log-sum-exp merge; one warp per query row.
template <int D>
__global__ void __launch_bounds__(256) fa_decode_kv8_combine_kernel(const __grid_constant__ Kv8DecodeParams p) {
  constexpr int E = D / 32;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = lane_id();
  if (row >= (long long)p.B * p.Nq * p.Hq) return;
  const float* pl = p.part_lse + row * p.splits;
  float m = -INFINITY;
  for (int c = lane; c < p.splits; c += 32) m = fmaxf(m, pl[c]);
#pragma unroll
  for (int t = 16; t > 0; t >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, t));
  float acc[E], wsum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (m != -INFINITY) {
    for (int c = 0; c < p.splits; ++c) {
      const float w = ex2_sfu(pl[c] - m);
      wsum += w;
      const float* src = p.part_o + (row * p.splits + c) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, src[e], acc[e]);
    }
  }
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) {
    const int h = (int)(row % p.Hq);
    const long long bi = row / p.Hq;
    const int i = (int)(bi % p.Nq);
    const long long b = bi / p.Nq;
    p.lse[(b * p.Hq + h) * p.Nq + i] = wsum > 0.f ? (m + __log2f(wsum)) * 0.69314718055994531f : -INFINITY;
  }
}

int kv8_auto_splits(int B, int Nq, int Hkv, int group, int span) {
  (void)Nq;
  (void)group;
  int dev = 0, n_sm = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  const long long ctas = (long long)B * Hkv;
  long long s = (8LL * n_sm + ctas - 1) / ctas;
  const long long most = ((long long)span + kKv8Tile - 1) / kKv8Tile;
  s = s > most ? most : s;
  return s < 1 ? 1 : (int)s;
}

template <int D>
static cudaError_t launch_decode_kv8_t(const Kv8DecodeParams& p, cudaStream_t stream) {
  const dim3 grid(p.splits, p.B, (p.Nq * p.Hq + 3) / 4);
  fa_decode_kv8_simple_kernel<D><<<grid, 128, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long rows = (long long)p.B * p.Nq * p.Hq;
  fa_decode_kv8_combine_kernel<D><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_decode_kv8(const Kv8DecodeParams& p, int D, cudaStream_t stream) {
  if (D == 64) return launch_decode_kv8_t<64>(p, stream);
  if (D == 128) return launch_decode_kv8_t<128>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fa
