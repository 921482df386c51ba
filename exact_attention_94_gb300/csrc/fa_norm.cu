// Root-mean-square norms of query and key heads with the rotation of their
// pairs in the same pass, and the gradients.  A head x of d elements with
// weights w at a token whose pairs turn by the angles a:
//     r = (mean(x^2) + eps)^(-1/2),   n = x r,   y = Rot(a) (w n).
// Backward, from g = Rot(-a) dy:
//     dw = sum over tokens and heads of g n,
//     dx = r (u - n mean(u n)),  u = w g.
//
// Bound by HBM: each element is read and written once (backward: x and dy are
// read, dx is written).  A thread holds 8 pairs of a head (two 16-byte vectors),
// d / 16 threads a head; they add up their squares by shuffles, so the norm
// costs no second pass.  A thread keeps its pairs' sines and weights over the
// heads of a token.  Angles are reduced as in fa_rope.cu; the sines are good to
// 2^-23, for the weights' gradients are given in fp32.
//
// Measured, d = 128, 32 + 8 heads, replayed graphs of many calls: 16384 tokens 61 us
// (5.5 TB/s of 6.8 that a copy reaches), the gradient 109 us (4.6 TB/s); 64 tokens
// 3.2 us.  15 instructions an element at half the issue slots bounded it at 67 and
// 111: pairs of elements in one instruction, weights and rotation as one product of
// each pair, a series for the sines and a head's loads ahead of the one in work are what is
// gained since.  (Of four heads at a time 1000 tokens took 8.5 us and not 6.4; a tile of
// tokens whose sines a block makes once for all heads 73 and 126 us; four blocks of the
// gradient to an SM 114 us.)
//
// dw: a block adds up its share of the rows in registers, its threads' sums in a
// fixed order in shared memory, and a second kernel the blocks' sums: the same
// call gives the same bits.
#include "sampling.cuh"

namespace fa {

namespace {

constexpr int kNormThreads = 128;

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Element e of pairs of elements.
__device__ __forceinline__ void f2_part(const uint64_t (&x)[8], int e, float& y) {
  float lo, hi;
  f2_unpack(x[e >> 1], lo, hi);
  y = e & 1 ? hi : lo;
}

// Which of a thread's 16 elements is which: x[e] and x[8 + e] are pair 8j + e.
template <bool NB>
__device__ __forceinline__ void unpack(uint4 a, uint4 b, float (&x)[16]) {
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = bf2(wa[i]), z = bf2(wb[i]);
    if constexpr (NB) {  // word i of a is pair 8j + i, word i of b pair 8j + 4 + i
      x[i] = y.x, x[8 + i] = y.y, x[4 + i] = z.x, x[12 + i] = z.y;
    } else {  // words i hold the two halves of pairs 8j + 2i and 8j + 2i + 1
      x[2 * i] = y.x, x[2 * i + 1] = y.y, x[8 + 2 * i] = z.x, x[9 + 2 * i] = z.y;
    }
  }
}
template <bool NB>
__device__ __forceinline__ void pack(const float (&x)[16], uint4& a, uint4& b) {
  uint32_t wa[4], wb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (NB) {
      wa[i] = pack_bf16x2(x[i], x[8 + i]);
      wb[i] = pack_bf16x2(x[4 + i], x[12 + i]);
    } else {
      wa[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
      wb[i] = pack_bf16x2(x[8 + 2 * i], x[9 + 2 * i]);
    }
  }
  a = make_uint4(wa[0], wa[1], wa[2], wa[3]);
  b = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}
// Offset within a head of the thread's element e of 16.
template <int D, bool NB>
__device__ __forceinline__ int offset(int j, int e) {
  return NB ? 16 * j + 2 * (e & 7) + (e >> 3) : 8 * j + (e & 7) + (e >> 3) * (D / 2);
}

// The plan where lanes with different pairs read it together (as in fa_rope.cu).
template <int D>
struct PlanSmem {
  uint64_t turn[8][D / 16];  // pair 8j + e at [e][j]
  int axis[8][D / 16];
  __device__ __forceinline__ void load(const NormRopeParams& p) {
    if (threadIdx.x < D / 2) {
      turn[threadIdx.x % 8][threadIdx.x / 8] = p.turn[threadIdx.x];
      axis[threadIdx.x % 8][threadIdx.x / 8] = p.axis[threadIdx.x];
    }
  }
};
// Sine and cosine of frac 2^-32 turns: the nearest quarter is the top bits, and what is left, at
// most an eighth of a turn, goes into their Taylor series, whose first terms left out are below
// 2^-28 of a sine and 2^-33.  (The library's functions took a quarter of the kernel's instructions.)
__device__ __forceinline__ void turn_sincos(uint32_t frac, float& si, float& co) {
  const uint32_t quarter = (frac + 0x20000000u) >> 30;
  const float x = (float)(int)(frac - (quarter << 30)) * 1.4629180792671596e-9f, y = x * x;  // 2 pi 2^-32
  float a = fmaf(y, 2.7557319e-6f, -1.9841270e-4f), b = fmaf(y, -2.7557319e-7f, 2.4801587e-5f);
  a = fmaf(y, a, 8.3333333e-3f), b = fmaf(y, b, -1.3888889e-3f);
  a = fmaf(y, a, -0.16666667f), b = fmaf(y, b, 4.1666667e-2f);
  a = fmaf(x * y, a, x), b = fmaf(y, fmaf(y, b, -0.5f), 1.f);
  si = quarter & 1 ? b : a, co = quarter & 1 ? a : b;
  si = __uint_as_float(__float_as_uint(si) ^ (quarter & 2) << 30);
  co = __uint_as_float(__float_as_uint(co) ^ (quarter + 1 & 2) << 30);
}
// Cosines and sines of a token's pairs 8j .. 8j + 7; bit e of the result: pair 8j + e turns.
template <int D>
__device__ __forceinline__ uint32_t angles(const NormRopeParams& p, const PlanSmem<D>& plan, int j, long long t,
                                           float (&co)[8], float (&si)[8]) {
  uint32_t turned = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int ax = plan.axis[e][j];
    co[e] = 1.f;
    si[e] = 0.f;
    if (ax >= 0) {
      const int pos = p.positions[(size_t)ax * p.T + t];
      const uint32_t frac = (uint32_t)(((uint64_t)(long long)pos * plan.turn[e][j]) >> 32);
      turn_sincos(frac, si[e], co[e]);
      turned |= 1u << e;
    }
  }
  return turned;
}

template <int D, bool NB>
__device__ __forceinline__ void load_weights(const void* w, int fp32, int j, float (&out)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int o = offset<D, NB>(j, e);
    out[e] = fp32 ? static_cast<const float*>(w)[o] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[o]);
  }
}

// Sum over the threads of a head (the same bits in each of them).
template <int TPT>
__device__ __forceinline__ float head_sum(float v, uint32_t mask) {
#pragma unroll
  for (int o = 1; o < TPT; o <<= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}

__device__ __forceinline__ float squares(const float (&x)[16]) {
  uint64_t a = 0ull, b = 0ull;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const uint64_t y = f2_pack(x[i], x[i + 1]), z = f2_pack(x[i + 2], x[i + 3]);
    a = f2_fma(y, y, a), b = f2_fma(z, z, b);
  }
  float lo, hi;
  f2_unpack(f2_add(a, b), lo, hi);
  return lo + hi;
}
// Sums of squares outside these are taken again of x 2^-68 or x 2^64: values beyond
// 2^64 would square to infinity, and those below 2^-50 count where eps is as small.
// (128 squares of what is below 2^60 add up to less than 2^127.)
__device__ __forceinline__ float other_scale(float sum, float eps) {
  if (!(sum < 1e37f)) return 0x1p-68f;
  return sum < 1e-30f && eps < 1e-24f ? 0x1p64f : 1.f;
}

}  // namespace

template <int D, bool NB, int BATCH>
__global__ void __launch_bounds__(kNormThreads) fa_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int TPT = D / 16;  // threads per head
  __shared__ PlanSmem<D> plan;
  const long long item = ((long long)blockIdx.x * kNormThreads + threadIdx.x) / TPT;
  const int j = threadIdx.x % TPT, chunks = p.q_chunks + p.k_chunks;
  const uint32_t mask = ((1u << TPT) - 1u) << ((threadIdx.x & 31) / TPT * TPT);  // the head's lanes
  const long long t = div_ll(item, chunks);
  const bool live = t < p.T;  // (of all of a head's lanes)
  const int c = (int)(item - t * chunks);
  const bool is_q = c < p.q_chunks;
  const int H = is_q ? p.Hq : p.Hkv, h0 = (is_q ? c : c - p.q_chunks) * p.heads_per_thread;
  const int h1 = min(h0 + p.heads_per_thread, H);
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_q ? p.q : p.k) + t * (is_q ? p.q_stride : p.k_stride);
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_q ? p.q_out : p.k_out) + t * (is_q ? p.q_out_stride : p.k_out_stride);
  const int o0 = NB ? 16 * j : 8 * j, o1 = NB ? 16 * j + 8 : 8 * j + D / 2;
  // a batch of heads is asked for before the angles are made, the next ones before the last is worked on
  uint4 u[BATCH], v[BATCH], u_next[BATCH], v_next[BATCH];
  auto load = [&](int h) {
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      if (h + b < h1) {
        u_next[b] = *reinterpret_cast<const uint4*>(src + (size_t)(h + b) * D + o0);
        v_next[b] = *reinterpret_cast<const uint4*>(src + (size_t)(h + b) * D + o1);
      }
    }
  };
  if (live) load(h0);
  plan.load(p);
  __syncthreads();
  if (!live) return;
  float co[8], si[8], w[16];
  load_weights<D, NB>(is_q ? p.wq : p.wk, p.w_fp32, j, w);
  const uint32_t turned = angles<D>(p, plan, j, t, co, si);
  // weights and rotation as one: y = (n0 c0 + n1 c1, n0 c2 + n1 c3) for each pair, two pairs at a time
  uint64_t c0[4], c1[4], c2[4], c3[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 2 * i;
    c0[i] = f2_pack(co[e] * w[e], co[e + 1] * w[e + 1]), c1[i] = f2_pack(-si[e] * w[8 + e], -si[e + 1] * w[9 + e]);
    c2[i] = f2_pack(si[e] * w[e], si[e + 1] * w[e + 1]), c3[i] = f2_pack(co[e] * w[8 + e], co[e + 1] * w[9 + e]);
  }
  for (int h = h0; h < h1; h += BATCH) {
#pragma unroll
    for (int b = 0; b < BATCH; ++b) u[b] = u_next[b], v[b] = v_next[b];
    if (h + BATCH < h1) load(h + BATCH);
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      if (h + b >= h1) break;
      float x[16], y[16];
      unpack<NB>(u[b], v[b], x);
      float s = squares(x);
      s = head_sum<TPT>(s, mask);
      const float f = other_scale(s, p.eps);
      if (f != 1.f) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= f;
        s = head_sum<TPT>(squares(x), mask);
      }
      const float r = rsqrtf(fmaf(s, 1.f / D, p.eps * f * f));
      const uint64_t r2 = f2_pack(r, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t n0 = f2_mul(f2_pack(x[2 * i], x[2 * i + 1]), r2), n1 = f2_mul(f2_pack(x[8 + 2 * i], x[9 + 2 * i]), r2);
        f2_unpack(f2_fma(n0, c0[i], f2_mul(n1, c1[i])), y[2 * i], y[2 * i + 1]);
        f2_unpack(f2_fma(n0, c2[i], f2_mul(n1, c3[i])), y[8 + 2 * i], y[9 + 2 * i]);
      }
      if (turned != 0xffu) {  // pairs that do not turn: 0 times an infinity would not be 0
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!(turned >> e & 1)) y[e] = x[e] * r * w[e], y[8 + e] = x[8 + e] * r * w[8 + e];
      }
      pack<NB>(y, u[b], v[b]);
      *reinterpret_cast<uint4*>(dst + (size_t)(h + b) * D + o0) = u[b];
      *reinterpret_cast<uint4*>(dst + (size_t)(h + b) * D + o1) = v[b];
    }
  }
}

template <int D, bool NB, int BATCH>
__global__ void __launch_bounds__(kNormThreads) fa_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int TPT = D / 16, HEADS = kNormThreads / TPT;  // heads of a block at a time
  __shared__ PlanSmem<D> plan;
  __shared__ float s_dw[kNormThreads / 32][D];
  const bool is_q = (int)blockIdx.x < p.q_blocks;
  const int block = is_q ? blockIdx.x : blockIdx.x - p.q_blocks, blocks = is_q ? p.q_blocks : gridDim.x - p.q_blocks;
  const int H = is_q ? p.Hq : p.Hkv, chunks = is_q ? p.q_chunks : p.k_chunks;
  const int j = threadIdx.x % TPT, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t mask = ((1u << TPT) - 1u) << (lane / TPT * TPT);
  const __nv_bfloat16* xs = static_cast<const __nv_bfloat16*>(is_q ? p.q : p.k);
  const __nv_bfloat16* gs = static_cast<const __nv_bfloat16*>(is_q ? p.dyq : p.dyk);
  __nv_bfloat16* ds = static_cast<__nv_bfloat16*>(is_q ? p.q_out : p.k_out);
  const long long x_stride = is_q ? p.q_stride : p.k_stride, g_stride = is_q ? p.dyq_stride : p.dyk_stride;
  const long long d_stride = is_q ? p.q_out_stride : p.k_out_stride;
  const int o0 = NB ? 16 * j : 8 * j, o1 = NB ? 16 * j + 8 : 8 * j + D / 2;
  const long long items = (long long)p.T * chunks, step = (long long)blocks * HEADS;
  // a batch of heads of an item (a token's chunk); the next one is asked for before this one is worked on
  struct At {
    long long item, t;
    int h, h1;
  };
  auto begin = [&](At& at) {
    at.t = div_ll(at.item, chunks);
    at.h = (int)(at.item - at.t * chunks) * p.heads_per_thread;
    at.h1 = min(at.h + p.heads_per_thread, H);
  };
  uint4 xa[BATCH], xb[BATCH], ga[BATCH], gb[BATCH], xa_next[BATCH], xb_next[BATCH], ga_next[BATCH], gb_next[BATCH];
  auto load = [&](const At& at) {
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      if (at.h + b < at.h1) {
        const __nv_bfloat16 *x = xs + at.t * x_stride + (size_t)(at.h + b) * D, *g = gs + at.t * g_stride + (size_t)(at.h + b) * D;
        xa_next[b] = *reinterpret_cast<const uint4*>(x + o0), xb_next[b] = *reinterpret_cast<const uint4*>(x + o1);
        ga_next[b] = *reinterpret_cast<const uint4*>(g + o0), gb_next[b] = *reinterpret_cast<const uint4*>(g + o1);
      }
    }
  };
  At next{(long long)block * HEADS + threadIdx.x / TPT, 0, 0, 0};
  if (next.item < items) {
    begin(next);
    load(next);
  }
  plan.load(p);
  __syncthreads();
  float w[16];
  uint64_t dw2[8];  // (pairs of elements)
  load_weights<D, NB>(is_q ? p.wq : p.wk, p.w_fp32, j, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw2[i] = 0ull;
  float co[8], si[8];
  uint32_t turned = 0;
  long long angles_of = -1;
  while (next.item < items) {
    const long long t = next.t;
    const int h = next.h, h1 = next.h1;
#pragma unroll
    for (int b = 0; b < BATCH; ++b) xa[b] = xa_next[b], xb[b] = xb_next[b], ga[b] = ga_next[b], gb[b] = gb_next[b];
    next.h += BATCH;
    if (next.h >= next.h1) {
      next.item += step;
      if (next.item < items) begin(next);
    }
    if (next.item < items) load(next);
    if (t != angles_of) turned = angles<D>(p, plan, j, t, co, si);
    angles_of = t;
    {
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        if (h + b >= h1) break;
        float x[16], y[16], g[16];
        unpack<NB>(xa[b], xb[b], x);
        unpack<NB>(ga[b], gb[b], y);
        uint64_t g2[8], u2[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // the rotation back
          const uint64_t y0 = f2_pack(y[2 * i], y[2 * i + 1]), y1 = f2_pack(y[8 + 2 * i], y[9 + 2 * i]);
          const uint64_t c = f2_pack(co[2 * i], co[2 * i + 1]), sn = f2_pack(si[2 * i], si[2 * i + 1]);
          const uint64_t neg = f2_pack(-si[2 * i], -si[2 * i + 1]);
          g2[i] = f2_fma(y0, c, f2_mul(y1, sn));
          g2[4 + i] = f2_fma(y1, c, f2_mul(y0, neg));
        }
        if (turned != 0xffu) {
#pragma unroll
          for (int e = 0; e < 16; ++e) f2_part(g2, e, g[e]);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!(turned >> e & 1)) g[e] = y[e], g[8 + e] = y[8 + e];
#pragma unroll
          for (int i = 0; i < 8; ++i) g2[i] = f2_pack(g[2 * i], g[2 * i + 1]);
        }
        uint64_t x2[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u2[i] = f2_mul(g2[i], f2_pack(w[2 * i], w[2 * i + 1])), x2[i] = f2_pack(x[2 * i], x[2 * i + 1]);
        auto sums = [&](float& s, float& m) {
          uint64_t a[2] = {0ull, 0ull}, c[2] = {0ull, 0ull};
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i & 1] = f2_fma(x2[i], x2[i], a[i & 1]), c[i & 1] = f2_fma(u2[i], x2[i], c[i & 1]);
          float lo, hi;
          f2_unpack(f2_add(a[0], a[1]), lo, hi);
          s = head_sum<TPT>(lo + hi, mask);
          f2_unpack(f2_add(c[0], c[1]), lo, hi);
          m = head_sum<TPT>(lo + hi, mask);
        };
        float s, m;
        sums(s, m);
        const float f = other_scale(s, p.eps);
        // The products u x may leave fp32 where u n does not (at its lower end too, if eps lets r be beyond 2^14):
        // then n comes first.
        const bool far = f != 1.f || !(fabsf(m) < 1e37f) || (fabsf(m) < 1e-30f && p.eps < 1e-8f);
        if (far) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x2[i] = f2_mul(x2[i], f2_pack(f, f));
          sums(s, m);
        }
        const float r = rsqrtf(fmaf(s, 1.f / D, p.eps * f * f));
        if (far) {
          uint64_t c = 0ull;
#pragma unroll
          for (int i = 0; i < 8; ++i) c = f2_fma(u2[i], f2_mul(x2[i], f2_pack(r * (1.f / D), r * (1.f / D))), c);
          float lo, hi;
          f2_unpack(c, lo, hi);
          m = head_sum<TPT>(lo + hi, mask);
        } else {
          m *= r * (1.f / D);  // mean(u n)
        }
        const uint64_t r2 = f2_pack(r, r), m2 = f2_pack(-m, -m), rf2 = f2_pack(r * f, r * f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t n = f2_mul(x2[i], r2);
          dw2[i] = f2_fma(g2[i], n, dw2[i]);
          f2_unpack(f2_mul(f2_fma(n, m2, u2[i]), rf2), y[2 * i], y[2 * i + 1]);
        }
        uint4 a, c;
        pack<NB>(y, a, c);
        __nv_bfloat16* d = ds + t * d_stride + (size_t)(h + b) * D;
        *reinterpret_cast<uint4*>(d + o0) = a;
        *reinterpret_cast<uint4*>(d + o1) = c;
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;");  // the blocks' sums may be set up; they wait for this grid's end
  // the block's sums: lanes with the same pairs, then the warps
  __syncwarp();
  float dw[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) f2_part(dw2, e, dw[e]);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
#pragma unroll
    for (int o = TPT; o < 32; o <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
    if (lane < TPT) s_dw[warp][offset<D, NB>(j, e)] = dw[e];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) v += s_dw[i][threadIdx.x];
    p.dw_part[(size_t)blockIdx.x * D + threadIdx.x] = v;
  }
}

// The blocks' sums of eight elements of dw added up: 32 rows of threads, then a tree.
__global__ void __launch_bounds__(256) fa_norm_dw_kernel(const float* part, int D, int q_blocks, int blocks, float* dwq,
                                                         float* dwk) {
  __shared__ float s[32][8];
  const int col = threadIdx.x % 8, row = threadIdx.x / 8, e = blockIdx.x * 8 + col;
  float* out = blockIdx.y == 0 ? dwq : dwk;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the sums are there
  if (out == nullptr) return;
  const int b0 = blockIdx.y == 0 ? 0 : q_blocks, b1 = blockIdx.y == 0 ? q_blocks : blocks;
  float v = 0.f;
  for (int b = b0 + row; b < b1; b += 32) v += part[(size_t)b * D + e];
  s[row][col] = v;
  __syncthreads();
#pragma unroll
  for (int n = 16; n > 0; n >>= 1) {
    if (row < n) s[row][col] += s[row + n][col];
    __syncthreads();
  }
  if (row == 0) out[e] = s[0][col];
}

namespace {

constexpr int kNormHeads = 8;                   // heads of a thread at most
constexpr long long kNormFull = kSms * 512;     // threads that keep the SMs busy

void set_chunks(NormRopeParams& p, int D) {
  // more heads a thread share its sines and weights, as long as enough threads are left
  const long long one = (long long)p.T * (p.Hq + p.Hkv) * (D / 16);
  const long long heads = (one + kNormFull - 1) / kNormFull;
  p.heads_per_thread = heads < 1 ? 1 : (int)(heads < kNormHeads ? heads : kNormHeads);  // (no tokens: 1, it divides)
  p.q_chunks = (p.Hq + p.heads_per_thread - 1) / p.heads_per_thread;
  p.k_chunks = (p.Hkv + p.heads_per_thread - 1) / p.heads_per_thread;
}

template <int D, bool NB>
void launch_norm_rope_t(const NormRopeParams& p, unsigned blocks, cudaStream_t stream) {
  if (p.heads_per_thread == 1)
    fa_norm_rope_kernel<D, NB, 1><<<blocks, kNormThreads, 0, stream>>>(p);
  else
    fa_norm_rope_kernel<D, NB, 2><<<blocks, kNormThreads, 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeParams& p, int D, bool neighbours, cudaStream_t stream) {
  set_chunks(p, D);
  const long long blocks = ((long long)p.T * (p.q_chunks + p.k_chunks) * (D / 16) + kNormThreads - 1) / kNormThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  if (D == 64)
    neighbours ? launch_norm_rope_t<64, true>(p, (unsigned)blocks, stream) : launch_norm_rope_t<64, false>(p, (unsigned)blocks, stream);
  else
    neighbours ? launch_norm_rope_t<128, true>(p, (unsigned)blocks, stream) : launch_norm_rope_t<128, false>(p, (unsigned)blocks, stream);
  return cudaGetLastError();
}

// Blocks in proportion to the heads of each side, one at least for a side that has heads, no more than there is work for.
int norm_rope_bwd_blocks(int T, int Hq, int Hkv, int D, int* q_blocks) {
  constexpr int kMost = kSms * 6;  // twice what stands on the SMs at once (three blocks of 148 registers a thread each)
  const int heads = kNormThreads / (D / 16);
  auto most = [&](int H) { return ((long long)T * H + heads - 1) / heads; };
  long long nq = Hq > 0 ? (long long)kMost * Hq / (Hq + Hkv) : 0;
  if (Hq > 0 && nq < 1) nq = 1;
  if (Hkv > 0 && nq >= kMost) nq = kMost - 1;
  long long nk = Hkv > 0 ? kMost - nq : 0;
  if (nq > most(Hq)) nq = most(Hq);
  if (nk > most(Hkv)) nk = most(Hkv);
  *q_blocks = (int)nq;
  return (int)(nq + nk);
}

cudaError_t launch_norm_rope_bwd(NormRopeParams& p, int D, bool neighbours, float* dwq, float* dwk, cudaStream_t stream) {
  set_chunks(p, D);
  const int blocks = norm_rope_bwd_blocks(p.T, p.Hq, p.Hkv, D, &p.q_blocks);
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(D / 8, 2);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  if (blocks > 0) {
    auto kern = D == 64 ? (neighbours ? fa_norm_rope_bwd_kernel<64, true, 1> : fa_norm_rope_bwd_kernel<64, false, 1>)
                        : (neighbours ? fa_norm_rope_bwd_kernel<128, true, 1> : fa_norm_rope_bwd_kernel<128, false, 1>);
    kern<<<blocks, kNormThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cfg.attrs = &a;  // (its launch overlaps the first kernel's end)
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, fa_norm_dw_kernel, (const float*)p.dw_part, D, p.q_blocks, blocks, dwq, dwk);
}

}  // namespace fa
