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
// rotates heads_per_thread heads with them, four at a time: their loads are all
// asked for before the first is used, which takes 80 registers, 24 warps per SM
// (and, with pairs in halves, five more that wait in local memory).
// Measured: 16384 tokens of 32 + 8 heads of 128 53 us, 6.3 TB/s; the gradient of
// 12289 tokens of 16 + 16 heads of 64, neighbouring pairs, 18 us, 5.5 TB/s; 64 tokens
// of 32 + 8 heads 2.9 us, a launch.
#include "serving.cuh"

namespace fa {

namespace {

constexpr int kRopeThreads = 128;  // (256: 12289 tokens of 16 + 16 heads of 64 19.0 us for 18.3, a longer last wave)
constexpr long long kRopeFull = kSms * 512;  // threads that keep the SMs busy
constexpr int kRopeHeads = 8;               // heads of a thread at most

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

}  // namespace

template <int D, bool NB, int BATCH>
__global__ void __launch_bounds__(kRopeThreads, 6) fa_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int TPT = D / 16;  // threads per token and head: 8 pairs each
  // Lanes with different pairs would read the plan, where it lies among the
  // parameters, one after the other (64 tokens of 32 + 8 heads: 3.4 us, and 2.9 from here).
  __shared__ uint64_t s_turn[8][TPT];  // pair 8j + e at [e][j]
  __shared__ int s_axis[8][TPT];
  if (threadIdx.x < D / 2) {
    s_turn[threadIdx.x % 8][threadIdx.x / 8] = p.turn[threadIdx.x];
    s_axis[threadIdx.x % 8][threadIdx.x / 8] = p.axis[threadIdx.x];
  }
  __syncthreads();
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
    const int ax = s_axis[e][j];
    const uint64_t f = s_turn[e][j];
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
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride;
  __nv_bfloat16* qo = static_cast<__nv_bfloat16*>(p.q_out) + t * p.q_out_stride;
  __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(p.k_out) + t * p.k_out_stride;
  // the loads of BATCH heads first, then their stores: outputs may be the
  // inputs, so the compiler could not move a load past a store by itself
  for (int h = h0; h < h1; h += BATCH) {
    uint4 u[BATCH], v[BATCH];
#pragma unroll
    for (int x = 0; x < BATCH; ++x) {
      if (h + x < h1) {
        const __nv_bfloat16* src = h + x < p.Hq ? q + (size_t)(h + x) * D : k + (size_t)(h + x - p.Hq) * D;
        u[x] = *reinterpret_cast<const uint4*>(src + o0);
        v[x] = *reinterpret_cast<const uint4*>(src + o1);
      }
    }
#pragma unroll
    for (int x = 0; x < BATCH; ++x) {
      if (h + x >= h1) break;
      const uint32_t a[4] = {u[x].x, u[x].y, u[x].z, u[x].w}, b[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
      uint32_t ra[4], rb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = bf2(a[i]), z = bf2(b[i]);
        if constexpr (NB) {  // word i of a is pair 8j + i, word i of b pair 8j + 4 + i
          ra[i] = pack_bf16x2(y.x * co[i] - y.y * si[i], y.x * si[i] + y.y * co[i]);
          rb[i] = pack_bf16x2(z.x * co[4 + i] - z.y * si[4 + i], z.x * si[4 + i] + z.y * co[4 + i]);
        } else {  // words i hold the two halves of pairs 8j + 2i and 8j + 2i + 1
          ra[i] = pack_bf16x2(y.x * co[2 * i] - z.x * si[2 * i], y.y * co[2 * i + 1] - z.y * si[2 * i + 1]);
          rb[i] = pack_bf16x2(y.x * si[2 * i] + z.x * co[2 * i], y.y * si[2 * i + 1] + z.y * co[2 * i + 1]);
        }
      }
      if (turned != 0xffu) {  // pairs that do not turn are copied: 0 times an infinity would not be
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (NB) {
            if (!(turned >> i & 1)) ra[i] = a[i];
            if (!(turned >> (4 + i) & 1)) rb[i] = b[i];
          } else {
            const uint32_t keep =
                ((turned >> (2 * i) & 1) ? 0u : 0xffffu) | ((turned >> (2 * i + 1) & 1) ? 0u : 0xffff0000u);
            ra[i] = (ra[i] & ~keep) | (a[i] & keep);
            rb[i] = (rb[i] & ~keep) | (b[i] & keep);
          }
        }
      }
      __nv_bfloat16* dst = h + x < p.Hq ? qo + (size_t)(h + x) * D : ko + (size_t)(h + x - p.Hq) * D;
      *reinterpret_cast<uint4*>(dst + o0) = make_uint4(ra[0], ra[1], ra[2], ra[3]);
      *reinterpret_cast<uint4*>(dst + o1) = make_uint4(rb[0], rb[1], rb[2], rb[3]);
    }
  }
}

template <int D, bool NB>
static void launch_rope_t(const RopeParams& p, unsigned blocks, cudaStream_t stream) {
  if (p.heads_per_thread == 1)
    fa_rope_kernel<D, NB, 1><<<blocks, kRopeThreads, 0, stream>>>(p);
  else
    fa_rope_kernel<D, NB, 4><<<blocks, kRopeThreads, 0, stream>>>(p);
}

cudaError_t launch_rope(RopeParams& p, int D, bool neighbours, cudaStream_t stream) {
  const int H = p.Hq + p.Hkv, tpt = D / 16;
  const long long one = (long long)p.T * H * tpt;  // threads with a head each
  // More heads a thread share its sines, as long as enough threads are left.
  // Microseconds with 1 / 4 / 8 / 16 heads, 32 + 8 heads of 128: 64 tokens 2.9 /
  // 3.5 / 4.3 / 5.9, 1024 8.2 / 5.7 / 6.0 / 6.3, 2048 14.0 / 8.4 / 8.1 / 9.3, 16384 99 /
  // 56 / 53 / 56.
  const long long heads = (one + kRopeFull - 1) / kRopeFull;
  p.heads_per_thread = (int)(heads < kRopeHeads ? heads : kRopeHeads);
  p.chunks = (H + p.heads_per_thread - 1) / p.heads_per_thread;
  p.heads_per_thread = (H + p.chunks - 1) / p.chunks;
  p.chunks = (H + p.heads_per_thread - 1) / p.heads_per_thread;
  const long long blocks = ((long long)p.T * p.chunks * tpt + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  if (D == 64)
    neighbours ? launch_rope_t<64, true>(p, (unsigned)blocks, stream) : launch_rope_t<64, false>(p, (unsigned)blocks, stream);
  else
    neighbours ? launch_rope_t<128, true>(p, (unsigned)blocks, stream) : launch_rope_t<128, false>(p, (unsigned)blocks, stream);
  return cudaGetLastError();
}

}  // namespace fa
