// Attention of a few query tokens per request over the 8-bit paged cache.
//     s_j = scale * k_scale(page_j) * q . k8_j
//     O = sum_j softmax(s)_j * v_scale(page_j) * v8_j,   lse = log sum_j e^(s_j)
// A split kernel takes a chunk of a request's keys and leaves a normalised
// partial (O_c, lse_c in base 2); a second kernel merges the partials,
// lse = log sum_c e^(lse_c), O = sum_c e^(lse_c - lse) O_c.
//
// The step is bound by HBM (2 d bytes per key and K/V head), so what matters
// is that the codes meet no work of their own: both products run on the fifth-
// generation tensor cores on the e4m3 codes as they lie in the cache, and no
// code ever passes through a register.  The keys take the M side, 128 of them,
// and the few query rows of a K/V head (its group's heads times the request's
// query tokens) the N side:
//     S^T [128 keys x rows] = K8 Q^T        A = K tile, B = Q
//     O^T [d x rows]        = V8^T P^T      A = V tile read MN-major, B = P
// B is then what has to be made 8-bit, and it is made so without loss that
// counts, as a sum of e4m3 numbers 16 times apart, each part a column of its
// own:  q = 2^k (q1 + q2 / 16) exactly (a bf16 has 8 significant bits, an e4m3
// 4) for what is within 2^13 of the row's largest, and within 2^-23 of the
// largest below;  p = (p1 + p2 / 16 + p3 / 256) / 256 to 2^-12 of itself, or of
// 2^-14 of the tile's largest.  Page scales are one factor per key: k_scale
// joins the score, v_scale (over the tile's largest) the probability.
//
// CTA: one chunk of one request and K/V head, RT query rows.
//   warps 0-3  thread = key of the tile for S and P (TMEM lane), and one of the
//              d output elements for O, which sums over the tiles in registers
//   warp 4     producer: block table and scales, one TMA box per page into a
//              ring of K and V tiles
//   warp 5     issues the products
// S is double buffered in TMEM (the next tile's scores are ready when a tile's
// softmax starts), O and P are not: P of a tile is written after O of the one
// before has been read.
#include "fa_internal.h"
#include "ptx.cuh"

#include <cmath>

namespace fa {

namespace {

constexpr int kThreads = 192;

template <int D, int RT>
struct Layout {
  static constexpr uint32_t kSlot = 128u * D;                       // a tile of K or V
  static constexpr int kSlots = D == 128 ? 6 : 12;                  // ring: K0 V0 K1 V1 ...
  static constexpr int kNS = 2 * RT < 16 ? 16 : 2 * RT;             // columns of S
  static constexpr int kNP = (3 * RT + 15) / 16 * 16;               // columns of P and O
  static constexpr uint32_t kCols = 2 * kNS + kNP <= 64 ? 64 : 128; // TMEM columns
  static constexpr uint32_t kPOff = kSlots * kSlot;
  static constexpr uint32_t kQOff = kPOff + kNP * 128u;
  static constexpr uint32_t kScOff = kQOff + kNS * (uint32_t)D;     // per V slot: 8 key scales, 8 value scales, factor
  static constexpr uint32_t kScBytes = 80;
  static constexpr uint32_t kMaxOff = kScOff + kSlots / 2 * kScBytes;  // [2][4][RT] warps' maxima
  static constexpr uint32_t kRowOff = kMaxOff + 2 * 4 * RT * 4;     // [RT] query scales, [RT] positions
  static constexpr uint32_t kBarOff = (kRowOff + 2 * RT * 4 + 15) / 16 * 16;
  static constexpr uint32_t kBytes = kBarOff + 8 * (2 * kSlots + 6) + 16 + 1024;
  static_assert(2 * kNS + kNP <= 128, "TMEM columns");
};

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

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t* r) {
  if constexpr (N >= 16) {
    tmem_ld16(addr, r);
    if constexpr (N > 16) tmem_load<N - 16>(addr + 16, r + 16);
  } else if constexpr (N > 0) {
    static_assert(N == 8, "columns in eights");
    tmem_ld8(addr, r);
  }
}

__device__ __forceinline__ void sts_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

}  // namespace

template <int D, int RT>
__global__ void __launch_bounds__(kThreads, 2)
    fa_decode_kv8_split_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                               const __grid_constant__ Kv8DecodeParams p) {
  using L = Layout<D, RT>;
  constexpr int NSL = L::kSlots;
  const int c = blockIdx.x, b = blockIdx.y;
  const int hk = (int)blockIdx.z / p.row_tiles, rt = (int)blockIdx.z - hk * p.row_tiles;
  const int row0 = rt * RT, rows = min(RT, p.Nq * p.group - row0);  // rows of this K/V head: token * group + head
  const int warp = warp_id(), lane = lane_id();

  const int len = kv8_len(p, b, threadIdx.x == 0);
  const int beg = kv8_begin(p, len) + c * p.chunk, end = min(len, beg + p.chunk);
  const int tiles = beg < end ? (end - beg + kKv8Tile - 1) / kKv8Tile : 0;
  // row r of the CTA: query token, and its row of q and o
  auto q_row = [&](int r) {
    const int i = (row0 + r) / p.group, g = row0 + r - i * p.group;
    return ((size_t)b * p.Nq + i) * p.Hq + (size_t)hk * p.group + g;
  };
  if (tiles == 0) {  // nothing to read: an empty partial, or the result for no keys
    for (int r = warp; r < rows; r += kThreads / 32) {
      const size_t row = q_row(r);
      if (p.splits > 1) {
        if (lane == 0) p.part_lse[row * p.splits + c] = -INFINITY;
      } else {
        uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + row * D);
        for (int e = lane; e < D / 2; e += 32) o[e] = 0u;
        const int i = (row0 + r) / p.group;
        if (lane == 0)
          p.lse[((size_t)b * p.Hq + (size_t)hk * p.group + row0 + r - i * p.group) * p.Nq + i] = -INFINITY;
      }
    }
    return;
  }

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sb = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBarOff;
  auto FULL = [&](int s) { return bars + 8u * (uint32_t)s; };
  auto EMPTY = [&](int s) { return bars + 8u * (uint32_t)(NSL + s); };
  const uint32_t SF = bars + 16u * NSL;  // S_full[2], then P_full, O_full, exchange, Q ready
  const uint32_t PF = SF + 16, OF = SF + 24, XB = SF + 32, QB = SF + 40;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sb + L::kBarOff + 16 * NSL + 48);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sb + L::kBarOff + 16 * NSL + 52);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * NSL; ++s) mbar_init(FULL(s), 1);
    mbar_init(SF, 1);
    mbar_init(SF + 8, 1);
    mbar_init(PF, 4);
    mbar_init(OF, 1);
    mbar_init(XB, 4);
    mbar_init(QB, 4);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(base + L::kBarOff + 16 * NSL + 52, L::kCols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tO = tmem + 2 * L::kNS;
  const WaitCtx w{abort_flag, p.timeout_ns, p.err};
  bool ok = true;

  if (warp == 4) {
    // ============================================================ producer
    // Lane i of a batch of four tiles owns 16 keys: their page and its scales.
    // The next batch's are read while this one's tiles are loaded.
    const int g_first = beg / 16, g_end = (end + 15) / 16;
    const int bpb = p.box_rows / 16;  // 16-key groups per TMA box
    auto page_of = [&](int batch, int& page, int& off) {
      const int g = g_first + batch * 32 + lane;
      page = 0;
      off = 0;
      if (g >= g_end) return false;
      const int blk = g * 16 / p.page_size;
      off = g * 16 - blk * p.page_size;
      page = p.block_table[(size_t)b * p.max_blocks + blk];
      return true;
    };
    auto checked = [&](int page, bool on) {  // report, and read a valid page instead
      if (on && (page < 0 || page >= p.num_pages)) {
        atomicCAS(p.err, 0u, FA_DEVERR_BAD_PAGE);
        return 0;
      }
      return page;
    };
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    int page, off, page_n = 0, off_n = 0;
    float ks = 0.f, vs = 0.f, ks_n = 0.f, vs_n = 0.f;
    bool on = page_of(0, page, off), on_n = false;
    page = checked(page, on);
    if (on) {
      ks = p.k_scale[(size_t)page * p.Hkv + hk];
      vs = p.v_scale[(size_t)page * p.Hkv + hk];
    }
    for (int t = 0; t < tiles; ++t) {
      const int i = t & 3;
      if (i == 0) {
        if (t > 0) {
          page = page_n, off = off_n, on = on_n, ks = ks_n, vs = vs_n;
        }
        on_n = page_of((t >> 2) + 1, page_n, off_n);
      }
      const bool mine = (lane >> 3) == i && on;
      const int boxes = (min(8, g_end - (g_first + 8 * t)) + bpb - 1) / bpb;
      const uint32_t bytes = (uint32_t)(boxes * p.box_rows * D);
      const bool issue = mine && (lane & (bpb - 1)) == 0;
      const uint32_t at = (uint32_t)(lane & 7) * 16u * D;
      const int ph = page * p.Hkv + hk;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int slot = (2 * t + v) % NSL, use = (2 * t + v) / NSL;
        if (use > 0) ok = mbar_wait(EMPTY(slot), (use - 1) & 1, w, 51);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (v == 1) {
          float mv = vs;
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
          if ((lane >> 3) == i) {
            float* sc = reinterpret_cast<float*>(sb + L::kScOff + (slot >> 1) * L::kScBytes);
            sc[lane & 7] = ks;
            sc[8 + (lane & 7)] = mv > 0.f ? vs / mv : 0.f;
            if ((lane & 7) == 0) sc[16] = mv * (1.f / 256.f);
          }
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(FULL(slot), bytes);
        __syncwarp();
        if (issue) tma_load_3d(base + slot * L::kSlot + at, v ? &tm_v : &tm_k, FULL(slot), 0, off, ph);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (i == 2) {  // a next batch exists only if this one is full
        page_n = checked(page_n, on_n);
        if (on_n) {
          ks_n = p.k_scale[(size_t)page_n * p.Hkv + hk];
          vs_n = p.v_scale[(size_t)page_n * p.Hkv + hk];
        } else {
          ks_n = vs_n = 0.f;
        }
      }
    }
  } else if (warp == 5) {
    // ============================================================ products
    constexpr uint32_t IDESC_S = idesc_e4m3(128, L::kNS), IDESC_O = idesc_e4m3(D, L::kNP, true);
    const uint32_t qa = base + L::kQOff, pa = base + L::kPOff;
    const uint64_t qd = D == 128 ? smem_desc_sw128(qa, 16, 1024) : smem_desc_sw64(qa, 16, 512);
    const uint64_t pd = smem_desc_sw128(pa, 16, 1024);
    ok = mbar_wait(QB, 0, w, 52);
    for (int t = 0; t <= tiles && __all_sync(0xffffffffu, ok); ++t) {
      if (t < tiles) {
        const int slot = (2 * t) % NSL;
        ok = mbar_wait(FULL(slot), (2 * t / NSL) & 1, w, 53);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint32_t ka = base + slot * L::kSlot;
        const uint64_t kd = D == 128 ? smem_desc_sw128(ka, 16, 1024) : smem_desc_sw64(ka, 16, 512);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          mma_ss_f8_w(tS + (t & 1) * L::kNS, desc_add(kd, kk * 32), desc_add(qd, kk * 32), IDESC_S, kk > 0);
        mma_commit_w(EMPTY(slot));
        mma_commit_w(SF + 8u * (t & 1));
      }
      if (t > 0) {
        const int slot = (2 * t - 1) % NSL;
        ok = mbar_wait(PF, (t - 1) & 1, w, 54);
        if (__all_sync(0xffffffffu, ok)) ok = mbar_wait(FULL(slot), ((2 * t - 1) / NSL) & 1, w, 55);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint32_t va = base + slot * L::kSlot;
        const uint64_t vd = D == 128 ? smem_desc_sw128(va, 16, 1024) : smem_desc_sw64(va, 16, 512);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss_f8_w(tO, desc_add(vd, kk * 32 * D), desc_add(pd, kk * 32), IDESC_O, kk > 0);
        mma_commit_w(EMPTY(slot));
        mma_commit_w(OF);
      }
    }
  } else {
    // ============================================================ softmax and sums
    float* s_max = reinterpret_cast<float*>(sb + L::kMaxOff);
    float* s_qsc = reinterpret_cast<float*>(sb + L::kRowOff);
    int* s_pos = reinterpret_cast<int*>(sb + L::kRowOff + 4 * RT);
    // ---- Q: a warp per row, split into two e4m3 parts at the row's power of two
    for (int r = warp; r < RT; r += 4) {
      constexpr int E = D / 32;
      float q[E];
      float mx = 0.f;
      bool odd = false;  // an infinity or a NaN in the row
#pragma unroll
      for (int e = 0; e < E; ++e) q[e] = 0.f;
      if (r < rows) {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + q_row(r) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = __bfloat162float(src[e]);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        odd |= !(fabsf(q[e]) <= 3.4e38f);
        mx = fmaxf(mx, fabsf(q[e]));
      }
      mx = fminf(warp_max(mx), 3.39e38f);
      odd = __any_sync(0xffffffffu, odd);
      // 2^k with mx / 2^k in [128, 256)
      const int ex = max((int)(__float_as_uint(mx) >> 23) - 7, 1);  // biased exponent of 2^k
      const float inv = mx > 0.f ? __uint_as_float((uint32_t)min(254 - ex, 254) << 23) : 1.f;
      const float sc = mx > 0.f ? __uint_as_float((uint32_t)ex << 23) : 1.f;
      uint32_t c1[E / 2], c2[E / 2];
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float x = odd ? __uint_as_float(0x7fffffffu) : q[e] * inv, y = odd ? __uint_as_float(0x7fffffffu) : q[e + 1] * inv;
        c1[e / 2] = pack_e4m3x2(x, y);
        const float2 h = unpack_e4m3x2(c1[e / 2]);
        c2[e / 2] = pack_e4m3x2((x - h.x) * 16.f, (y - h.y) * 16.f);
      }
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const int n = part * RT + r;
        if constexpr (D == 128) {
          const uint32_t v = part ? (c2[0] | c2[1] << 16) : (c1[0] | c1[1] << 16);
          *reinterpret_cast<uint32_t*>(sb + L::kQOff + n * 128 + (((lane >> 2) ^ (n & 7)) << 4) + (lane & 3) * 4) = v;
        } else {
          const uint32_t v = part ? c2[0] : c1[0];
          *reinterpret_cast<uint16_t*>(sb + L::kQOff + n * 64 + (((lane >> 3) ^ ((n >> 1) & 3)) << 4) + (lane & 7) * 2) =
              (uint16_t)v;
        }
      }
      if (lane == 0) {
        s_qsc[r] = sc * p.scale_log2;
        s_pos[r] = len - p.Nq + (row0 + r) / p.group;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(QB);
    ok = mbar_wait(QB, 0, w, 56);

    const uint32_t lane_sel = (uint32_t)warp << 21;  // TMEM lane 32 * warp
    const int key = warp * 32 + lane;                // key of the tile
    // this thread's byte of P in row n: 128-byte rows, 128-byte swizzle
    const uint32_t p_at = base + L::kPOff + (key & 15);
    float m[RT], l[RT], acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) m[r] = -INFINITY, l[r] = 0.f, acc[r] = 0.f;
    float c_prev = 0.f;

    auto add_o = [&](int t) {  // O of tile t joins the sums, which stand at the reference it was made with
      if (!__all_sync(0xffffffffu, mbar_wait(OF, t & 1, w, 57))) return false;
      tc_fence_after();
      uint32_t o[L::kNP];
      tmem_load<(3 * RT + 7) / 8 * 8>(tO + lane_sel, o);
      tmem_ld_wait();
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float x = fmaf(__uint_as_float(o[2 * RT + r]), 0.0625f, __uint_as_float(o[RT + r]));
        acc[r] = fmaf(fmaf(x, 0.0625f, __uint_as_float(o[r])), c_prev, acc[r]);
      }
      return true;
    };

    for (int t = 0; t < tiles && __all_sync(0xffffffffu, ok); ++t) {
      const int vslot = (2 * t + 1) % NSL;
      ok = mbar_wait(SF + 8u * (t & 1), (t >> 1) & 1, w, 58);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      uint32_t sr[2 * RT];
      tmem_load<2 * RT>(tS + (t & 1) * L::kNS + lane_sel, sr);
      ok = mbar_wait(FULL(vslot), ((2 * t + 1) / NSL) & 1, w, 59);
      if (!__all_sync(0xffffffffu, ok)) break;
      const float* sc = reinterpret_cast<const float*>(sb + L::kScOff + (vslot >> 1) * L::kScBytes);
      const float ks = sc[key >> 4], vn = sc[8 + (key >> 4)] * 256.f, c_now = sc[16];
      tmem_ld_wait();
      float s[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r)
        s[r] = fmaf(__uint_as_float(sr[RT + r]), 0.0625f, __uint_as_float(sr[r])) * (ks * s_qsc[r]);
      // ---- keys that some row does not see
      const int j0 = beg + t * kKv8Tile, j = j0 + key;
      const bool partial = j0 + kKv8Tile > len - p.Nq + 1 || (p.win_left >= 0 && j0 < len - 1 - p.win_left);
      if (partial) {
        bool any = false;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const int pos = s_pos[r];
          const bool sees = j <= pos && (p.win_left < 0 || j >= pos - p.win_left);
          any |= sees && r < rows;
          if (!sees) s[r] = -INFINITY;
        }
        if (!any) {  // its value row may hold anything: 0 * NaN would not be 0
          uint4* row = reinterpret_cast<uint4*>(sb + vslot * L::kSlot + key * D);
#pragma unroll
          for (int e = 0; e < D / 16; ++e) row[e] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      // ---- the tile's largest score of each row, over the four warps
      {
        float mw[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) mw[r] = warp_max(s[r]);
        float4* dst = reinterpret_cast<float4*>(s_max + ((t & 1) * 4 + warp) * RT);
        if (lane == 0) {
#pragma unroll
          for (int r = 0; r < RT; r += 4) dst[r / 4] = make_float4(mw[r], mw[r + 1], mw[r + 2], mw[r + 3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(XB);
      }
      ok = mbar_wait(XB, t & 1, w, 60);
      if (!__all_sync(0xffffffffu, ok)) break;
      // ---- O of the tile before; P's buffer is free with it
      if (t > 0) {
        ok = add_o(t - 1);
        if (!ok) break;
      }
      c_prev = c_now;
      // ---- reference, probabilities, their three parts
#pragma unroll
      for (int r4 = 0; r4 < RT; r4 += 4) {
        float4 a = *reinterpret_cast<const float4*>(s_max + ((t & 1) * 4) * RT + r4);
#pragma unroll
        for (int x = 1; x < 4; ++x) {
          const float4 bq = *reinterpret_cast<const float4*>(s_max + ((t & 1) * 4 + x) * RT + r4);
          a.x = fmaxf(a.x, bq.x), a.y = fmaxf(a.y, bq.y), a.z = fmaxf(a.z, bq.z), a.w = fmaxf(a.w, bq.w);
        }
        const float tm[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          float pv[2];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int r = r4 + e + f;
            const float mn = fmaxf(m[r], tm[e + f]), ref = mn == -INFINITY ? 0.f : mn;
            const float al = ex2_sfu(m[r] - ref), pr = ex2_sfu(s[r] - ref);
            l[r] = fmaf(l[r], al, pr);
            acc[r] *= al;
            m[r] = mn;
            pv[f] = pr * vn;
          }
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            const uint32_t two = pack_e4m3x2(pv[0], pv[1]);
            const int n = part * RT + r4 + e;
            sts_u8(p_at + n * 128 + ((((uint32_t)key >> 4) ^ (n & 7)) << 4), two & 0xffu);
            sts_u8(p_at + (n + 1) * 128 + ((((uint32_t)key >> 4) ^ ((n + 1) & 7)) << 4), two >> 8);
            if (part < 2) {
              const float2 h = unpack_e4m3x2(two);
              pv[0] = (pv[0] - h.x) * 16.f;
              pv[1] = (pv[1] - h.y) * 16.f;
            }
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(PF);
    }
    if (__all_sync(0xffffffffu, ok)) ok = add_o(tiles - 1);
    // ---- each row's sum over the 128 key lanes
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
    }
    // s_max's other half is free: every warp is past the exchange that used it
    float* s_l = s_max + (tiles & 1) * 4 * RT;
    if (lane == 0) {
#pragma unroll
      for (int r = 0; r < RT; ++r) s_l[warp * RT + r] = l[r];
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(XB);
    if (__all_sync(0xffffffffu, ok)) ok = mbar_wait(XB, tiles & 1, w, 61);
    if (__all_sync(0xffffffffu, ok)) {
      // output element of this thread: TMEM lane; an M = 64 product uses lanes 0 .. 15 of each warp's 32
      const int e = D == 128 ? key : warp * 16 + lane;
      const bool has = D == 128 || lane < 16;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (r >= rows) break;
        const float sum = s_l[r] + s_l[RT + r] + s_l[2 * RT + r] + s_l[3 * RT + r];
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        const float lse2 = sum > 0.f ? m[r] + __log2f(sum) : (sum == 0.f ? -INFINITY : sum);
        const size_t row = q_row(r);
        if (p.splits > 1) {
          if (has) p.part_o[(row * p.splits + c) * D + e] = acc[r] * inv;
          if (threadIdx.x == 0) p.part_lse[row * p.splits + c] = lse2;
        } else {
          if (has) static_cast<__nv_bfloat16*>(p.o)[row * D + e] = __float2bfloat16_rn(acc[r] * inv);
          const int i = (row0 + r) / p.group;
          if (threadIdx.x == 0)
            p.lse[((size_t)b * p.Hq + (size_t)hk * p.group + row0 + r - i * p.group) * p.Nq + i] =
                lse2 * 0.69314718055994531f;
        }
      }
    }
    tc_fence_before();
  }
  if (!ok) {  // let copies and products in flight land before the CTA's memory goes
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
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
  for (int c = 0; c < p.splits; ++c) {
    const float lc = pl[c];
    if (lc == -INFINITY) continue;  // an empty chunk: its O was not written
    const float w = ex2_sfu(lc - m);
    wsum += w;
    const float* src = p.part_o + (row * p.splits + c) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, src[e], acc[e]);
  }
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) {
    const int h = (int)(row % p.Hq);
    const long long bi = row / p.Hq;
    const int i = (int)(bi % p.Nq);
    const long long b = bi / p.Nq;
    p.lse[(b * p.Hq + h) * p.Nq + i] = wsum == 0.f ? -INFINITY : (m + __log2f(wsum)) * 0.69314718055994531f;
  }
}

// Query rows of one CTA.
static int kv8_row_tile(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }

int kv8_auto_splits(int B, int Nq, int Hkv, int group, int span) {
  int dev = 0, n_sm = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  const int rows = Nq * group, tile = kv8_row_tile(rows);
  const long long ctas = (long long)B * Hkv * ((rows + tile - 1) / tile);
  long long s = (8LL * n_sm + ctas - 1) / ctas;
  const long long most = ((long long)span + kKv8Tile - 1) / kKv8Tile;
  s = s > most ? most : s;
  return s < 1 ? 1 : (s > 65535 ? 65535 : (int)s);
}

template <int D, int RT>
static cudaError_t launch_split(const CUtensorMap& tk, const CUtensorMap& tv, Kv8DecodeParams& p, cudaStream_t stream) {
  auto kern = fa_decode_kv8_split_kernel<D, RT>;
  constexpr uint32_t smem = Layout<D, RT>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  p.row_tiles = (p.Nq * p.group + RT - 1) / RT;
  if ((long long)p.Hkv * p.row_tiles > 65535) return cudaErrorInvalidValue;
  kern<<<dim3(p.splits, p.B, p.Hkv * p.row_tiles), kThreads, smem, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_decode_kv8_t(const CUtensorMap& tk, const CUtensorMap& tv, Kv8DecodeParams& p,
                                       cudaStream_t stream) {
  cudaError_t e;
  switch (kv8_row_tile(p.Nq * p.group)) {
    case 4: e = launch_split<D, 4>(tk, tv, p, stream); break;
    case 8: e = launch_split<D, 8>(tk, tv, p, stream); break;
    default: e = launch_split<D, 16>(tk, tv, p, stream); break;
  }
  if (e != cudaSuccess || p.splits == 1) return e;
  const long long rows = (long long)p.B * p.Nq * p.Hq;
  fa_decode_kv8_combine_kernel<D><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_decode_kv8(const CUtensorMap& tk, const CUtensorMap& tv, Kv8DecodeParams& p, int D,
                              cudaStream_t stream) {
  if (D == 64) return launch_decode_kv8_t<64>(tk, tv, p, stream);
  if (D == 128) return launch_decode_kv8_t<128>(tk, tv, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fa
