// Rotary positions with several axes, forward and gradient in one kernel (the
// gradient of a rotation by a is the rotation by -a).
//
// Pair p of a head turns by a = pos[axis_p][t] * inv_freq_p.  Only a modulo a
// turn matters, and far positions make a large, so the frequency is held as a
// 64-bit binary fraction of a turn, f = frac(inv_freq / 2 pi) * 2^64: the top
// 32 bits of pos * f, an integer product that wraps, are the angle's fraction
// of a turn to 2^-32, at any position.  The sine and cosine of that fraction
// (|angle| <= pi) are the fast ones, whose error there is 2^-21, against the
// 2^-9 of the result's bf16.
//
// Bound by HBM: each element of q and k is read and written once.  A thread
// holds 8 pairs (two 16-byte vectors) of a token, takes their sines once and
// rotates heads_per_thread heads with them.
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

}  // namespace

template <int D, bool NB>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int TPT = D / 16;  // threads per token and head: 8 pairs each
  const long long item = ((long long)blockIdx.x * kRopeThreads + threadIdx.x) / TPT;
  const int j = threadIdx.x % TPT;
  const long long t = item / p.chunks;
  if (t >= p.T) return;
  const int h0 = (int)(item - t * p.chunks) * p.heads_per_thread;
  const int h1 = min(h0 + p.heads_per_thread, p.Hq + p.Hkv);

  float co[8], si[8];
  uint32_t turned = 0;  // bit e: pair 8j + e turns
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int ax = p.axis[8 * j + e];
    const uint64_t f = p.turn[8 * j + e];
    co[e] = 1.f;
    si[e] = 0.f;
    if (ax >= 0) {
      const int pos = p.positions[(size_t)ax * p.T + t];
      const uint32_t frac = (uint32_t)(((uint64_t)(long long)pos * f) >> 32);
      const float a = (float)(int)frac * 1.4629180792671596e-9f;  // 2 pi / 2^32
      co[e] = __cosf(a);
      si[e] = p.inverse ? -__sinf(a) : __sinf(a);
      turned |= 1u << e;
    }
  }
  // element offsets of the thread's two vectors within a head
  const int o0 = NB ? 16 * j : 8 * j, o1 = NB ? 16 * j + 8 : 8 * j + D / 2;
  for (int h = h0; h < h1; ++h) {
    const bool isq = h < p.Hq;
    const int hh = isq ? h : h - p.Hq;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(isq ? p.q : p.k) +
                               t * (isq ? p.q_stride : p.k_stride) + (size_t)hh * D;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(isq ? p.q_out : p.k_out) +
                         t * (isq ? p.q_out_stride : p.k_out_stride) + (size_t)hh * D;
    const uint4 u = *reinterpret_cast<const uint4*>(src + o0), v = *reinterpret_cast<const uint4*>(src + o1);
    const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
    uint32_t ra[4], rb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (NB) {  // word i of a is pair 8j + i, word i of b pair 8j + 4 + i
        const float2 x = bf2(a[i]), y = bf2(b[i]);
        ra[i] = pack_bf16x2(x.x * co[i] - x.y * si[i], x.x * si[i] + x.y * co[i]);
        rb[i] = pack_bf16x2(y.x * co[4 + i] - y.y * si[4 + i], y.x * si[4 + i] + y.y * co[4 + i]);
        if (!(turned >> i & 1)) ra[i] = a[i];
        if (!(turned >> (4 + i) & 1)) rb[i] = b[i];
      } else {  // words i hold the two halves of pairs 8j + 2i and 8j + 2i + 1
        const float2 x = bf2(a[i]), y = bf2(b[i]);
        ra[i] = pack_bf16x2(x.x * co[2 * i] - y.x * si[2 * i], x.y * co[2 * i + 1] - y.y * si[2 * i + 1]);
        rb[i] = pack_bf16x2(x.x * si[2 * i] + y.x * co[2 * i], x.y * si[2 * i + 1] + y.y * co[2 * i + 1]);
        // a pair that does not turn is copied: 0 times an infinity would not be
        const uint32_t keep = ((turned >> (2 * i) & 1) ? 0u : 0xffffu) | ((turned >> (2 * i + 1) & 1) ? 0u : 0xffff0000u);
        ra[i] = (ra[i] & ~keep) | (a[i] & keep);
        rb[i] = (rb[i] & ~keep) | (b[i] & keep);
      }
    }
    *reinterpret_cast<uint4*>(dst + o0) = make_uint4(ra[0], ra[1], ra[2], ra[3]);
    *reinterpret_cast<uint4*>(dst + o1) = make_uint4(rb[0], rb[1], rb[2], rb[3]);
  }
}

cudaError_t launch_rope(RopeParams& p, int D, bool neighbours, cudaStream_t stream) {
  p.heads_per_thread = 1;
  p.chunks = p.Hq + p.Hkv;
  const long long threads = (long long)p.T * p.chunks * (D / 16);
  const long long blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks);
  if (D == 64)
    neighbours ? fa_rope_kernel<64, true><<<grid, kRopeThreads, 0, stream>>>(p)
               : fa_rope_kernel<64, false><<<grid, kRopeThreads, 0, stream>>>(p);
  else
    neighbours ? fa_rope_kernel<128, true><<<grid, kRopeThreads, 0, stream>>>(p)
               : fa_rope_kernel<128, false><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
