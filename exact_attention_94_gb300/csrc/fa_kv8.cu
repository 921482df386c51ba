// The 8-bit paged cache, write side: quantise new tokens into pages of e4m3
// codes with one power-of-two scale per page and K/V head ("efficient-
// attention/flash-2-3", sections "FP8, and the outlier problem": one scale per
// block, and "Paged KV caches, a preview of serving").
//
//   own   = 2^e, smallest e with amax <= 448 * 2^e over the run's finite values
//   scale = max(own, the page's scale)   (own alone for a run from slot 0)
//   code  = e4m3(x / scale);  older codes of the page: e4m3(code * old / scale)
// A power of two makes the division exact and the move of older codes exact
// but for those that fall below e4m3's normal range, and e4m3, a floating
// format, loses no precision to it.
//
// A run is a maximal sequence of rows with one page and consecutive slots.
// One warp takes a run's rows of one K/V head, for K or for V: the largest
// magnitude first, then the codes.  Bound by HBM for prompts (2 bytes read and
// 1 written per element), by latency for a step of single tokens.  Measured, 8
// K/V heads of 128: 9 prompts of 2047 tokens each into pages of 32 25 us, 4.4 TB/s (27 of
// them 62 us, 5.5 TB/s); 64 requests of a token 3.3 us, a launch.
#include "serving.cuh"

namespace fa {

namespace {

constexpr int kAppendWarps = 4;
constexpr int kAppendBlocks = 7;  // CTAs per SM: all the registers allow (9 prompts of 2047: 26.1 us, and 27.8 with four)
constexpr int kHeld = 8;  // vectors of a run that a lane holds in registers (with 4, 28.9 us; with 16, four CTAs, 25.8)

__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  const float2 a = unpack_e4m3x2(w & 0xffffu), b = unpack_e4m3x2(w >> 16);
  return pack_e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

// 16-bit halves with a magnitude of 0x7f80 or more are infinities and NaNs.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t mags) {
  if ((mags & 0xffffu) >= 0x7f80u) mags &= 0xffff0000u;
  if ((mags >> 16) >= 0x7f80u) mags &= 0x0000ffffu;
  return mags;
}

// The scale of a largest magnitude, given as bf16 bits; 0 for 0.
__device__ __forceinline__ float pow2_scale(uint32_t amax_bits) {
  if (amax_bits == 0) return 0.f;
  // bits = 1.m * 2^(E - 127); 448 = 1.75 * 2^8, and 1.m > 1.75 needs one more
  int e = (int)(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7fu) > 0x60u ? 1 : 0);
  e = max(e, -126);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Eight bf16 values times inv -> eight codes.  The conversion keeps a NaN; an
// infinity, which it would saturate, has to be made one first (ODD).
template <bool ODD>
__device__ __forceinline__ uint2 encode8(const uint4& u, float inv) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = ODD && isinf(f[i]) ? __uint_as_float(0x7fffffffu) : f[i] * inv;
  return make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
}

}  // namespace

// pass 0: every run; 1: runs that copy an older page first; 2: the others.  With
// copies, 1 and 2 are two launches: an in-place run may rescale the very page
// that another run copies from, and the copy has to read it first.
template <int D>
__global__ void __launch_bounds__(32 * kAppendWarps, kAppendBlocks) fa_kv8_append_kernel(const Kv8AppendParams p, int pass) {
  constexpr int LPR = D / 8;     // lanes per row, 8 elements each
  constexpr int RPI = 32 / LPR;  // rows per iteration
  const int lane = lane_id();
  const long long unit = (long long)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const long long part = unit / (2 * p.Hkv);
  const int which = (int)(unit - part * 2 * p.Hkv);
  const long long tile = part / p.split;
  const int turn = (int)(part - tile * p.split);  // this warp's runs of the tile: every split-th one from here
  const int head = which % p.Hkv;
  const bool is_v = which >= p.Hkv;
  const long long r0 = tile * 32;
  if (r0 >= p.n) return;
  const int rows = (int)min(32ll, p.n - r0);

  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(is_v ? p.v_new : p.k_new) + (size_t)head * D;
  const long long xs = is_v ? p.v_stride : p.k_stride;
  uint8_t* codes = static_cast<uint8_t*>(is_v ? p.v_codes : p.k_codes);
  float* scales = is_v ? p.v_scale : p.k_scale;
  const int sub = lane / LPR, seg = lane % LPR;

  // ---- rows of this tile that begin a run
  int pg = -1, sl = -1, pg2 = -1, sl2 = -1;  // of row r0 + lane, and of r0 + 32 + lane, where runs may end
  bool lead = false;
  if (r0 + 32 + lane < p.n) {
    pg2 = p.page[r0 + 32 + lane];
    sl2 = p.slot[r0 + 32 + lane];
  }
  if (lane < rows) {
    const long long i = r0 + lane;
    pg = p.page[i];
    sl = p.slot[i];
    lead = pg != -1;
    if (lead && i > 0 && sl > 0 && sl < p.page_size) lead = !(p.page[i - 1] == pg && p.slot[i - 1] == sl - 1);
  }
  uint32_t todo = __ballot_sync(0xffffffffu, lead);
  const int rank = __popc(todo & ((1u << lane) - 1u));
  todo = __ballot_sync(0xffffffffu, lead && (unsigned)rank % (unsigned)p.split == (unsigned)turn);
  while (todo != 0) {
    const int l = __ffs(todo) - 1;
    todo &= todo - 1;
    const int page = __shfl_sync(0xffffffffu, pg, l), first = __shfl_sync(0xffffffffu, sl, l);
    const long long row = r0 + l;
    const int src = p.copy_src != nullptr ? p.copy_src[row] : -1;
    if (page < 0 || page >= p.num_pages || first < 0 || first >= p.page_size || src >= p.num_pages || src < -1) {
      if (lane == 0) atomicCAS(p.err, 0u, FA_DEVERR_BAD_PAGE);
      continue;
    }
    if (pass == 1 && src < 0) continue;
    if (pass == 2 && src >= 0) continue;
    // ---- length of the run
    const int most = (int)min((long long)(p.page_size - first), p.n - row);
    uint32_t ends = ~__ballot_sync(0xffffffffu, lane < l || (pg == page && sl == first + lane - l));
    int len = ends != 0 ? __ffs(ends) - 1 - l : 32 - l;
    bool goes_on = ends == 0;
    if (goes_on) {
      ends = ~__ballot_sync(0xffffffffu, pg2 == page && sl2 == first + 32 + lane - l);
      len += ends != 0 ? __ffs(ends) - 1 : 32;
      goes_on = ends == 0;
    }
    len = min(len, most);
    while (goes_on && len < most) {
      const int i = len + lane;
      const bool on = i < most && p.page[row + i] == page && p.slot[row + i] == first + i;
      const uint32_t m = __ballot_sync(0xffffffffu, on);
      const int more = __ffs(~m) - 1;  // rows before the first that does not go on; -1: all 32 do
      len += more < 0 ? 32 : more;
      if (more >= 0) break;
    }
    // ---- largest finite magnitude (as bf16 bits: they order like the values).
    // A run of up to kHeld * RPI rows stays in registers; a longer one is read
    // again for its codes.
    const __nv_bfloat16* rows_at = x + row * xs + seg * 8;
    uint4 held[kHeld];
    uint32_t mx = 0;
    auto load = [&](int i0) {
#pragma unroll
      for (int c = 0; c < kHeld; ++c) {
        const int i = i0 + sub + c * RPI;
        held[c] = make_uint4(0u, 0u, 0u, 0u);
        if (i < len) held[c] = *reinterpret_cast<const uint4*>(rows_at + i * xs);
      }
    };
    for (int i0 = 0; i0 < len; i0 += kHeld * RPI) {
      load(i0);
#pragma unroll
      for (int c = 0; c < kHeld; ++c) {
        if (i0 + c * RPI >= len) break;
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(held[c].x & 0x7fff7fffu, held[c].y & 0x7fff7fffu),
                                   __vmaxu2(held[c].z & 0x7fff7fffu, held[c].w & 0x7fff7fffu)));
      }
    }
    uint32_t amax = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
    const bool odd = amax >= 0x7f80u;  // an infinity or a NaN in the run: again, without them
    if (odd) {
      mx = 0;
      for (int i = sub; i < len; i += RPI) {
        const uint4 u = *reinterpret_cast<const uint4*>(rows_at + i * xs);
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(finite_or_zero(u.x & 0x7fff7fffu), finite_or_zero(u.y & 0x7fff7fffu)),
                                   __vmaxu2(finite_or_zero(u.z & 0x7fff7fffu), finite_or_zero(u.w & 0x7fff7fffu))));
      }
      amax = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
    }
    const float own = pow2_scale(amax);
    const size_t to = (size_t)page * p.Hkv + head;
    const size_t from = (size_t)(src >= 0 ? src : page) * p.Hkv + head;
    const float old = first > 0 ? scales[from] : 0.f;
    const float scale = fmaxf(old, own);
    const float inv = scale > 0.f ? 1.f / scale : 0.f;
    __syncwarp();
    if (lane == 0) scales[to] = scale;
    uint8_t* dst = codes + to * p.page_size * D + seg * 8;
    // ---- older codes of the page
    if (first > 0 && (src >= 0 || scale != old)) {
      const uint8_t* old_codes = codes + from * p.page_size * D + seg * 8;
      const float ratio = old > 0.f ? old * inv : 0.f;
      for (int i = sub; i < first; i += RPI) {
        uint2 c = *reinterpret_cast<const uint2*>(old_codes + (size_t)i * D);
        if (ratio != 1.f) c = make_uint2(recode4(c.x, ratio), recode4(c.y, ratio));
        *reinterpret_cast<uint2*>(dst + (size_t)i * D) = c;
      }
    }
    // ---- new codes
    dst += (size_t)first * D;
    if (odd) {
      for (int i = sub; i < len; i += RPI)
        *reinterpret_cast<uint2*>(dst + (size_t)i * D) = encode8<true>(*reinterpret_cast<const uint4*>(rows_at + i * xs), inv);
      continue;
    }
    for (int i0 = 0; i0 < len; i0 += kHeld * RPI) {
      if (len > kHeld * RPI) load(i0);
#pragma unroll
      for (int c = 0; c < kHeld; ++c) {
        const int i = i0 + sub + c * RPI;
        if (i0 + c * RPI >= len) break;
        if (i < len) *reinterpret_cast<uint2*>(dst + (size_t)i * D) = encode8<false>(held[c], inv);
      }
    }
  }
}

template <int D>
static cudaError_t launch_kv8_append_t(Kv8AppendParams& p, cudaStream_t stream) {
  // A warp looks at 32 rows and takes every split-th run that begins there: all
  // of them where there are many rows (prompts: a run or two), fewer where the
  // rows alone would leave SMs idle (a step of single tokens: 32 runs).  64 single
  // tokens take 3.5 us so and 36 with split 1; 9 prompts of 1024 tokens 16.4, and 55
  // with split 32.
  const long long tiles = ((long long)p.n + 31) / 32 * 2 * p.Hkv;
  const long long split = (long long)kSms * kAppendBlocks * kAppendWarps / tiles;
  p.split = (int)(split < 1 ? 1 : split > 32 ? 32 : split);
  const long long blocks = (tiles * p.split + kAppendWarps - 1) / kAppendWarps;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  for (int pass = p.copy_src != nullptr ? 1 : 0; pass <= (p.copy_src != nullptr ? 2 : 0); ++pass) {
    fa_kv8_append_kernel<D><<<(unsigned)blocks, 32 * kAppendWarps, 0, stream>>>(p, pass);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_kv8_append(Kv8AppendParams& p, int D, cudaStream_t stream) {
  if (D == 64) return launch_kv8_append_t<64>(p, stream);
  if (D == 128) return launch_kv8_append_t<128>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fa
