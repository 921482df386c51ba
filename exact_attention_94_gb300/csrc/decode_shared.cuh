// Attention of a few query tokens per request over a paged cache, for a batch
// whose requests come in groups that share their first tokens.
//     s_j = scale q . k_j,   O = sum_j softmax(s)_j v_j,   lse = log sum_j e^(s_j)
//
// A group's shared keys meet the queries of all its requests as one product,
// and are read once for up to 256 rows at a time; each request's own keys meet
// its own queries; the parts are merged by their masses:
//     lse = log sum_c e^(lse_c),   O = sum_c e^(lse_c - lse) O_c.
//
// Three kernels, the launch of each overlapping the one before:
//  - the plan, one CTA: an entry for each group's shared keys and each request's
//    own (query tokens, keys, table row), in two lists: entries of many rows, whose
//    (entry, K/V head, 256 rows) units are tiles of 128 keys, and of few (8 or 16),
//    whose (entry, K/V head) units are steps of 16 keys.  Each list is cut in shares
//    of equal weight, a unit weighing more for its start and end.
//  - the main kernel, one CTA per SM.  A CTA of the first has a share of tiles; the
//    warps of the others begin with a share of few rows each, and all warps take the
//    rest of those from a queue as they come to an end.  So products that tensor cores
//    bound run beside keys that HBM bounds.  (Own keys as tiles too, an eighth of their
//    128 rows used: 64 requests with 16385 shared and 100 to 2000 own tokens 101 us
//    and not 85, 256 with 32768 and 1 to 512 376 and not 257.)
//    Tiles: rows take the M side of both tcgen05 products: S [128 x 128 keys] = Q K^T,
//    O [128 x d] += P V with P in TMEM over S, two tiles in turn, so one's products run
//    while the other's softmax does.  Units of more than 128 rows are two tiles of rows
//    that meet the same keys; units of up to 128 are one tile of rows, whose key tiles
//    the two take in turn, and both results are merged at the end.
//    Few rows: decode_few.cuh.
//  - the merge, a warp for up to 8 query rows: results of whole units (at their rows) or
//    of the pieces that shares' borders cut.
//
// Rows of a tile are query tokens times the query heads of one K/V head, as they
// lie in Q: a TMA box of [tokens][heads][64 elements].
//
// Main kernel's warps, of tiles: 2 walks over the share and announces its pieces; 0
// loads K and 3 loads Q and V (K and V into one ring, across units); 1 issues the
// products; 4-7 and 8-11 are the softmax of the two tiles, a thread per row; 12-15
// convert 8-bit tiles.
//
// A TMA box is a page's keys (128 at most) of one head, all d of them: a tile of K or
// V lies in shared memory as [8 keys][64 elements of d][8 x 128 bytes], so that one
// box fills whole eights of keys.
//
// Measured, 64 heads over 8, d = 128, replayed graphs (bf16 pages / 8-bit):
//   64 requests, 16385 shared, 100 to 2000 own            85 / 104 us
//   256 requests, 32768 shared, 1 to 512 own              257 / 393 us
//   256 requests, 32768 shared, one own                   226 / 318 us, 1.2 / 0.86 PFLOP/s
//   32 requests, 131072 shared (256 rows)                 140 / 172 us
//   64 requests, 8192 own                                 354 us, 6.1 TB/s / 272 us, 4.0 TB/s
//   4 requests, 777 shared, 32 heads over 8               20 / 22 us
// (at 2070 MHz; over bf16 pages the power cap holds 256 requests at 1980 to 2040).
// bf16 tiles are bound by the products (1570 cycles a job of two 128 x 128 x 128 products
// that take 1280: 171 us of 226 for 216 jobs an SM; start and merge are some 25 more, and
// 30 are not accounted for).  8-bit ones are bound by the softmax warps, with which the
// converting ones share issue slots and registers: 2400 cycles a job.  The smallest
// calls are the three kernels' latencies one after the other: plan 5 us, main 11, merge 4.
#pragma once

#include "sampling.cuh"

#include <cmath>

namespace fa {

namespace {

constexpr int kPlanThreads = 1024;
// What units weigh.  Of many rows, in half microseconds about: of one and of two tiles of
// rows, and each of their tiles of keys.  Of few rows: their start and end, in 16 keys.
constexpr int kLeadOne = 5, kTileOne = 2, kLeadTwo = 12, kTileTwo = 3, kLeadFew = 6;
constexpr float kFew = 0.17f;                  // of a CTA's half microseconds 16 keys of few rows take, d = 128
constexpr int kFewEarly = 12, kFewLate = 16;   // shares of few rows for each CTA at most, that warps begin with and that they take
constexpr float kFew8 = 1.f;                   // what 16 keys of 8 bits take of that
constexpr int kFewLateOf = 2;                  // one in so many of few rows' weight is dealt late,
constexpr int kFewLateFrom = 64;               //   where a warp's share is this much at least
constexpr int kFewLeast = 8, kFewLateLeast = 24;  // weight of those shares at least
constexpr int kPlanSmem = 1024;                // groups, entries in the plan's shared memory
constexpr int kMergeRows = 8;                  // of a warp of the merge
constexpr int kPieces = 6;                     // announced ahead

// The main kernel over bf16 pages, and over pages of 8-bit codes (KV8), whose tiles four more
// warps convert.
// Warps of a CTA that attend for few rows: the softmax warps, and of 8-bit pages those that
// convert, of d = 64 all of them (of d = 128 their rings have no room).
__host__ __device__ constexpr int few_warps(int D, bool kv8) { return kv8 || D == 64 ? 12 : 8; }

template <int D, bool KV8>
struct SharedLayout {
  static constexpr int kThreads = KV8 ? 512 : 384;
  static constexpr uint32_t kTile = 128u * D * 2u;  // a tile of Q, K or V
  static constexpr uint32_t kRawTile = 128u * D;    // of codes, which land in their slot's second half
  static constexpr uint32_t kChunk = 128u * 128u;   // of Q: 128 rows x 128 bytes (one 128-byte swizzle column)
  static constexpr int kStages = 640 / D;                  // K/V ring slots
  static constexpr int kScales = KV8 ? 1024 / D : 0;       // key tiles whose scales are kept
  static constexpr uint32_t kQOff = 0;                     // two tiles of Q
  static constexpr uint32_t kKVOff = 2 * kTile;
  static constexpr uint32_t kMiscOff = kKVOff + kStages * kTile;
  static constexpr uint32_t kMisc = D == 64 ? 4096 : 2048;  // barriers, pieces
  static constexpr uint32_t kBytes = kMiscOff + kMisc + 1024;  // alignment slack
};
static_assert(SharedLayout<128, false>::kBytes <= 227 * 1024 && SharedLayout<128, true>::kBytes <= 227 * 1024, "shared memory");

// Tiles t0 .. t1 - 1 of a unit, as the walk announces them; t0 = t1 marks the end.
struct Piece {
  long long place;     // row of the results: of the query row itself (times Hq: whole units), or of a cut piece's first
  int side;            // rows between the two runs' or tiles' results (cut pieces); 0: the unit's only piece
  int kind;            // 0: shared keys, 1: a request's own
  int tok0, ntok;      // query tokens of the unit
  int head;            // K/V head
  int row;             // of the block table
  int lo, end, all_lo, all_hi, beg;
  int t0, t1, pad;
};

__device__ __forceinline__ int chunks_of(const SharedParams& p, bool few, int ntok) {  // of 256 rows
  return few ? 1 : (ntok + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
}
// What a unit weighs: its start and end, and each of its tiles of keys.  Slot
// lead + tile * t of its weight is where tile t begins.
struct Weight {
  int lead, tile;
};
__device__ __forceinline__ Weight weight_of(const SharedParams& p, bool few, int ntok) {
  return few ? Weight{kLeadFew, 1} : ntok > p.tile_tokens ? Weight{kLeadTwo, kTileTwo} : Weight{kLeadOne, kTileOne};
}

// `total` slots of weight in n equal shares: the first `more` have each + 1.
struct Equal {
  long long total, each, more;
  int n;
  __device__ __forceinline__ Equal(long long t, int shares)
      : total(t), each(shares > 0 ? div_ll(t, shares) : 0), more(shares > 0 ? t - each * shares : 0), n(shares) {}
  __device__ __forceinline__ long long begin(long long k) const { return each * k + (k < more ? k : more); }
  __device__ __forceinline__ int of(long long slot) const {
    return (int)(slot < more * (each + 1) ? div_ll(slot, each + 1) : more + div_ll(slot - more * (each + 1), each));
  }
};
// The shares of a list: early ones, then late ones.
struct Deal {
  Equal early, late;
  __device__ __forceinline__ long long begin(int k) const {
    return k < early.n ? early.begin(k) : early.total + late.begin(k - early.n);
  }
  __device__ __forceinline__ int of(long long slot) const {
    return slot < early.total ? early.of(slot) : early.n + late.of(slot - early.total);
  }
};
__device__ __forceinline__ Deal deal_of(const SharedHead& h, bool few) {
  return few ? Deal{Equal(h.total[1], h.shares[1]), Equal(h.total[2], h.shares[2])}
             : Deal{Equal(h.total[0], h.shares[0]), Equal(0, 0)};
}

// The units' pieces of a share, one after the other.
struct Walk {
  const SharedEntry* entries;
  SharedEntry ent, ahead;
  long long begin, at, to, off;
  int e, count;
  // Share k of a list of n entries; called by whole warps.
  __device__ __forceinline__ void start(const SharedList& list, int n, const Deal& deal, int k) {
    begin = at = deal.begin(k), to = deal.begin(k + 1);
    int lo = 0, hi = n;  // the last entry that begins at or before it: 32 at a time
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, i = lo + lane_id() * step;
      const unsigned votes = __ballot_sync(0xffffffffu, i < hi && list.cum[i] <= at);
      lo += (__popc(votes) - 1) * step;
      hi = min(hi, lo + step);
    }
    entries = list.entry;
    e = lo, count = n;
    ent = entries[e];
    off = at - list.cum[e];
    if (e + 1 < count) ahead = entries[e + 1];
  }
  // Tiles t0 .. t1 - 1 of unit u of `ent`; later: the unit begins behind the share's first slot.  False: the share is over.
  __device__ __forceinline__ bool next(const SharedParams& p, bool few, int& u, int& t0, int& t1, bool& later) {
    while (at < to) {
      const Weight wt = weight_of(p, few, ent.ntok);
      const int weight = wt.lead + wt.tile * ent.tiles, chunks = chunks_of(p, few, ent.ntok);
      if (off >= (long long)weight * p.Hkv * chunks) {
        off = 0;
        ++e;
        ent = ahead;
        if (e + 1 < count) ahead = entries[e + 1];
        continue;
      }
      u = (int)div_ll(off, weight);
      const int w0 = (int)(off - (long long)u * weight), w1 = (int)(to - at < weight - w0 ? w0 + (to - at) : weight);
      later = w0 == 0 && at > begin;
      off += w1 - w0;
      at += w1 - w0;
      t0 = w0 <= wt.lead ? 0 : (w0 - wt.lead + wt.tile - 1) / wt.tile;
      t1 = w1 <= wt.lead ? 0 : (w1 - wt.lead + wt.tile - 1) / wt.tile;
      if (t0 < t1) return true;
    }
    return false;
  }
};
// Place of the results of a share's cut pieces (two: it begins inside a unit, or it ends inside one).
__device__ __forceinline__ long long cut_place(const SharedParams& p, bool few, int k, bool later) {
  const long long rows = (long long)p.B * p.Nq * p.Hq, slot = 2 * (long long)k + (later ? 1 : 0);
  return 4 * rows + (few ? 512ll * p.shares + slot * p.few : slot * 2 * kSharedTile);
}

}  // namespace

// ---------------------------------------------------------------- main

// 8-bit pages: codes are exact in f16, so K and V tiles become f16, and what they meet:
//  - a row of queries times a power of two of its own, exact for what is within 2^28 of its largest;
//  - probabilities times value scales, against a reference per row at which that is kAtRef: rounded by
//    2^-11 of themselves, or by 2^-32 of the row's largest.  The row sums share the reference.  They
//    are of the probabilities alone, of which none that counts is below 2^-110 or above 2^95 of it;
//    it may move by more than 2^126 from one page to the next, so they go along in two halves.
constexpr float kAtRefLog2 = 7.f, kMaxTau = 8.f;
constexpr float kLeastScale = -80.f;  // log2 of a value scale, from below
__device__ __forceinline__ float scale_log2(float v) { return v > 0.f && v < INFINITY ? fmaxf(__log2f(v), kLeastScale) : kLeastScale; }
// Barrier `id` of 128 threads, and whether `ok` holds in all of them.
__device__ __forceinline__ bool all_of_128(int id, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %2, 0;\n\t"
      "bar.red.and.pred p, %1, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(id), "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}
__device__ __forceinline__ void load_8(const float* at, float (&x)[8]) {  // of shared memory
  const uint32_t a = smem_u32(at);
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(a) : "memory");
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]) : "r"(a + 16) : "memory");
}
// The factor that takes a row with this largest |bf16| to 2^14 .. 2^15, and what undoes it.
struct RowScale {
  float to, back;
  __device__ __forceinline__ explicit RowScale(uint32_t largest) {
    const uint32_t e = max(largest >> 7, 15u);
    to = __uint_as_float((268u - e) << 23), back = __uint_as_float((e - 14u) << 23);
  }
};
__device__ __forceinline__ uint32_t bf16_f16(uint32_t x, float scale) {
  return pack_f16x2(__uint_as_float(x << 16) * scale, __uint_as_float(x & 0xffff0000u) * scale);
}
__device__ __forceinline__ uint4 bf16_f16(uint4 x, float scale) {
  return make_uint4(bf16_f16(x.x, scale), bf16_f16(x.y, scale), bf16_f16(x.z, scale), bf16_f16(x.w, scale));
}
__device__ __forceinline__ uint32_t largest_bf16(uint32_t m, uint4 x) {  // two maxima
  const uint32_t a = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(m, x.x & a), __vmaxu2(__vmaxu2(x.y & a, x.z & a), x.w & a));
}

#include "decode_few.cuh"

template <int D, int NR, bool KV8>
__global__ void __launch_bounds__((SharedLayout<D, KV8>::kThreads), 1)
    fa_decode_shared_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k16,
                            const __grid_constant__ CUtensorMap tm_v16, const __grid_constant__ SharedParams p) {
  using L = SharedLayout<D, KV8>;
  constexpr int NS = L::kStages, RAW = KV8 ? NS : 0, SCALES = L::kScales, CH = D / 64;
  constexpr uint32_t TILE = L::kTile, CHUNK = L::kChunk;
  const int warp = warp_id(), lane = lane_id();

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sb = smem_raw + (base - raw);
  const uint32_t q_s = base + L::kQOff, kv_s = base + L::kKVOff;

  // Rings: K/V tiles, pieces.  RAW_FULL: a tile's codes have landed.  Q[s]: a tile of Q has landed; its last S product is
  // done.  Per tile t in turn: S ready, P's first and second 64 keys ready, the last
  // product of a run of key tiles done (O), and O read.  X: the softmax warps of a
  // tile, and of both, have come this far.  Q_READY: a tile of Q is f16.
  enum { KV_FULL = 0, KV_EMPTY = NS, PC_FULL = 2 * NS, PC_EMPTY = PC_FULL + kPieces, Q_FULL = PC_EMPTY + kPieces,
         Q_EMPTY = Q_FULL + 2, S_FULL = Q_EMPTY + 2, P_FULL = S_FULL + 2, O_FINAL = P_FULL + 4, O_EMPTY = O_FINAL + 2,
         XB = O_EMPTY + 2, DRAIN = XB + 3, RAW_FULL = DRAIN + 1, Q_READY = RAW_FULL + RAW,
         NBARS = Q_READY + (KV8 ? 2 : 0) };
  const uint32_t bar0 = base + L::kMiscOff;
  auto BAR = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  constexpr uint32_t SLOT = L::kMiscOff + (8 * NBARS + 15) / 16 * 16, PIECES = SLOT + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sb + SLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Piece* s_piece = reinterpret_cast<Piece*>(sb + PIECES);                              // [kPieces]
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(sb + PIECES + 64 * kPieces);           // [2 groups][2][4]
  float* s_scale = reinterpret_cast<float*>(sb + PIECES + 64 * kPieces + 64);          // KV8: [SCALES][8 of keys, 8 of values, 8 logarithms of these]
  static_assert(sizeof(Piece) == 64 && PIECES % 16 == 0, "pieces; scales are read 16 bytes at a time");
  static_assert(PIECES + 64 * kPieces + 64 + SCALES * 96 <= L::kMiscOff + L::kMisc, "misc area");
  // Few rows, once the tiles are done with: a warp's region, and what it keeps beside its rings.
  constexpr int FEW = few_warps(D, KV8);
  constexpr bool ALL = !KV8 && FEW == 12;  // the warps that load and multiply are among them
  constexpr uint32_t FEW_BYTES = L::kMiscOff / FEW / 1024 * 1024, FEW_OWN = KV8 ? FEW_BYTES - 256 : FEW_BYTES;
  static_assert(KV8 || PIECES + FEW * sizeof(FewState) <= L::kMiscOff + L::kMisc, "misc area");
  static_assert(sizeof(FewState) <= 256, "misc area");

  if (threadIdx.x == 0) {
    for (int i = 0; i < NBARS; ++i) {
      int n = 1;
      if (KV8 && i < NS) n = 4;  // the warps that convert
      if (i >= Q_READY) n = 8;
      if (i >= PC_EMPTY && i < PC_EMPTY + kPieces) n = KV8 ? 15 : 11;  // who loads, converts, multiplies, eight warps of softmax
      if ((i >= P_FULL && i < P_FULL + 4) || i == O_EMPTY || i == O_EMPTY + 1) n = 128;
      if (i == XB || i == XB + 1) n = 4;
      if (i == XB + 2) n = 8;
      mbar_init(BAR(i), n);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx w{abort_flag, p.timeout_ns, p.err};
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is there
  asm volatile("griddepcontrol.launch_dependents;");  // the merge may be set up; it waits for this grid's end

  // the next piece announced, read by every lane of a warp
  auto take = [&](int piece, Piece& s, unsigned site) {
    const int slot = piece % kPieces;
    if (!__all_sync(0xffffffffu, mbar_wait(BAR(PC_FULL + slot), piece / kPieces & 1, w, site))) return false;
    s = s_piece[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(PC_EMPTY + slot));
    return true;
  };
  // Ring places of key tile `it`: its K comes before the V of the tile in front, as
  // the products take them.
  auto k_place = [](int it) { return it == 0 ? 0 : 2 * it - 1; };
  auto v_place = [](int it) { return 2 * it + 2; };

  // CTAs begin with a share of the entries with many rows, or with shares of few rows for their warps
  const int n_many = p.plan.head->shares[0];
  const bool many = (int)blockIdx.x < n_many;
  const bool few = NR > 0 && (!many || p.plan.head->shares[2] > 0);  // (behind the tiles there are the late shares alone)
  // Registers go where a row's 128 scores are held: 56 x 4 warps + 224 x 8 is what 168 x 12 was
  // (and is again, where all twelve attend for few rows); of 8-bit pages
  // (56 + 72) x 4 + 192 x 8, and then 56 x 4 + 152 x 12, what 128 x 16 was.  A CTA without tiles
  // goes to the latter at once, one with tiles behind a barrier: where the warps that convert
  // could grow before the softmax warps have, they would take what those wait for forever.
  auto few_rows = [&]() {
    if constexpr (NR > 0) {
      const int x = ALL ? warp : warp - 4, others = (int)gridDim.x - n_many;
      if (few)
        attend_few<D, NR, KV8, FEW_OWN>(p, tm_k16, tm_v16, w, many ? -1 : x * others + (int)blockIdx.x - n_many, base + x * FEW_BYTES,
                                        sb + x * FEW_BYTES,
                                        reinterpret_cast<FewState*>(KV8 ? sb + x * FEW_BYTES + FEW_OWN : sb + PIECES + x * sizeof(FewState)));
    }
  };
  if (warp < 4) {
    if (!ALL || many) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (!many) {
    } else if (warp == 2) {
      // ============================================================ walk over the share
      Walk walk;
      walk.start(p.plan.list[0], p.plan.head->count[0], deal_of(*p.plan.head, false), (int)blockIdx.x);
      bool left = true;
      for (int pieces = 0; left; ++pieces) {
        Piece s = {};
        int u;
        bool later;
        left = walk.next(p, false, u, s.t0, s.t1, later);
        if (left) {  // (else t0 = t1: the end)
          const SharedEntry& ent = walk.ent;
          const int chunks = chunks_of(p, false, ent.ntok);
          s.head = (int)((unsigned)u / (unsigned)chunks);
          const int c = u - s.head * chunks;
          s.tok0 = ent.tok0 + c * 2 * p.tile_tokens;
          s.ntok = min(2 * p.tile_tokens, ent.ntok - c * 2 * p.tile_tokens);
          s.lo = ent.lo, s.end = ent.end, s.all_lo = ent.all_lo, s.all_hi = ent.all_hi;
          s.beg = ent.lo / p.box_rows * p.box_rows;
          s.kind = ent.kind;
          s.row = ent.row;
          s.side = s.t0 == 0 && s.t1 == ent.tiles ? 0 : kSharedTile;
          s.place = s.side == 0 ? 2 * (long long)ent.kind * p.B * p.Nq * p.Hq : cut_place(p, false, (int)blockIdx.x, later);
        }
        const int slot = pieces % kPieces;
        if (pieces >= kPieces &&
            !__all_sync(0xffffffffu, mbar_wait(BAR(PC_EMPTY + slot), (pieces / kPieces - 1) & 1, w, 70)))
          break;
        if (lane == 0) {
          s_piece[slot] = s;
          mbar_arrive(BAR(PC_FULL + slot));
        }
        __syncwarp();
      }
    } else if (warp == 0 || warp == 3) {
      // ============================================================ loads of K, and of Q and V
      const CUtensorMap* map = warp == 0 ? &tm_k : &tm_v;
      if (lane == 0) {
        tma_prefetch_desc(map);
        if (warp == 3) tma_prefetch_desc(&tm_q);
      }
      const int boxes = kSharedTile / p.box_rows, shift = __ffs(p.box_rows) - 5;  // TMA boxes of a tile; 16-key groups of one, log2
      bool ok = true, more = true;
      Piece pc;
      pc.t0 = pc.t1 = 0;
      int t_next = 0, piece = 0;
      struct Batch {  // up to four tiles of a piece, lane i owning 16 keys; their pages are read two batches ahead
        int n, rows8, page, head, last;  // rows8: of the cache, in eights, less the page's; last: 16-key groups there are
        int tok0, ntok;                  // a piece's first batch: its query tokens; else 0
      };
      auto fetch = [&](Batch& q) {
        q.n = q.ntok = 0;
        if (!more) return;
        if (t_next == pc.t1) {
          more = take(piece++, pc, 73) && pc.t0 < pc.t1;
          t_next = pc.t0;
          if (!more) return;
          q.tok0 = pc.tok0, q.ntok = pc.ntok;
        }
        q.n = min(4, pc.t1 - t_next);
        const int g0 = (pc.beg + t_next * kSharedTile) / 16, g = g0 + lane;
        q.last = (pc.end + 15) / 16 - g0;
        q.head = pc.head;
        q.page = q.rows8 = 0;
        t_next += q.n;
        if (lane < 8 * q.n && lane < q.last) {
          const int blk = (int)((unsigned)(g * 16) / (unsigned)p.page_size);
          q.rows8 = 2 * g - blk * (p.page_size / 8);
          q.page = p.block_table[(size_t)pc.row * p.max_blocks + blk];
        }
      };
      int place = warp == 0 ? 0 : 2, qt = 0;  // ring places, as k_place and v_place count; tiles of Q so far
      Batch now, then;
      fetch(now);
      fetch(then);
      while (ok && now.n > 0) {
        if (now.page < 0 || now.page >= p.num_pages) {  // report, and read a valid page instead
          atomicCAS(p.err, 0u, FA_DEVERR_BAD_PAGE);
          now.page = 0;
        }
        if (warp == 3) {  // Q, before the first values (which are needed later)
          for (int x = 0; x < now.ntok && ok; x += p.tile_tokens, ++qt) {
            const int slot = qt & 1;
            if (qt >= 2) ok = __all_sync(0xffffffffu, mbar_wait(BAR(Q_EMPTY + slot), (qt / 2 - 1) & 1, w, 72));
            if (ok && elect_one()) {
              mbar_arrive_expect_tx(BAR(Q_FULL + slot), (uint32_t)(p.tile_tokens * p.heads * D * 2));
#pragma unroll
              for (int c = 0; c < CH; ++c)
                tma_load_3d(q_s + slot * TILE + c * CHUNK, &tm_q, BAR(Q_FULL + slot), c * 64, now.head * p.heads, now.tok0 + x);
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        const int at8 = KV8 ? now.rows8 * 8 : now.page * (p.page_size / 8) + now.rows8;  // row of the page, or eight of all pages'
        const int plane = now.page * p.Hkv + now.head;
        float k_scale = 0.f, v_scale = 0.f;
        if constexpr (KV8) {
          if (warp == 0 && lane < 8 * now.n && lane < now.last) k_scale = p.k_scale[plane], v_scale = p.v_scale[plane];
        }
        constexpr int FULL = KV8 ? (int)RAW_FULL : (int)KV_FULL;
        for (int i = 0; i < now.n; ++i) {
          const int slot = place % NS, here = min(boxes, (max(now.last - 8 * i, 0) + (1 << shift) - 1) >> shift);
          if (place >= NS) ok = __all_sync(0xffffffffu, mbar_wait(BAR(KV_EMPTY + slot), (place / NS - 1) & 1, w, 74));
          if (!ok) break;
          if (KV8 && warp == 0) {  // scales, which the softmax warps read when the keys' scores are there
            const int sc_slot = (place + 1) / 2 % (SCALES + !SCALES);
            if (lane >> 3 == i) {
              float* sc = s_scale + sc_slot * 24 + (lane & 7);
              // (a value scale that is no number is a NaN)
              sc[0] = k_scale, sc[8] = fabsf(v_scale) < INFINITY ? v_scale : __uint_as_float(0x7fffffffu), sc[16] = scale_log2(v_scale);
            }
            __syncwarp();
          }
          if (elect_one()) mbar_arrive_expect_tx(BAR(FULL + slot), (uint32_t)(here * p.box_rows * D * (KV8 ? 1 : 2)));
          __syncwarp();
          const uint32_t dst = kv_s + slot * TILE + (KV8 ? L::kRawTile : 0), bar = BAR(FULL + slot);
          for (int x = 0; x < here; ++x) {  // (one lane issues, with the same operands in all)
            const int row = __shfl_sync(0xffffffffu, at8, 8 * i + (x << shift));
            if constexpr (KV8) {
              const int pl = __shfl_sync(0xffffffffu, plane, 8 * i + (x << shift));
              if (elect_one()) tma_load_3d(dst + x * p.box_rows * D, map, bar, 0, row, pl);
            } else {
              if (elect_one()) tma_load_5d(dst + x * p.box_rows * D * 2, map, bar, 0, 0, 0, row, now.head);
            }
          }
          place += place == 0 ? 1 : 2;
        }
        now = then;
        fetch(then);
      }
      if (!ok) {  // let copies already in flight land before the CTA's shared memory goes away
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
      }
    } else if (warp == 1) {
      // ============================================================ products
      // Job n is a tile of rows times a tile of keys; jobs take S, P and O of tile n & 1.
      // S of job n is issued before the product of job n - 1's P, which waits for its softmax.
      constexpr uint32_t IDESC_S = KV8 ? idesc_f16(128, 128, false, false) : idesc_bf16(128, 128, false, false);
      constexpr uint32_t IDESC_O = KV8 ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);
      constexpr int QUERIES = KV8 ? (int)Q_READY : (int)Q_FULL;
      struct Job {
        uint32_t vslot, vphase;
        bool on, first, last, frees;  // first, last of its tile's run in the piece; the last to read its values
      } before{};
      uint32_t n = 0, qt = 0, runs[2] = {0, 0}, ps[2] = {0, 0};
      uint32_t sk = 0, pk = 0, sv = 2, pv = 0;  // ring slots and phases of the tile's K and V
      bool ok = true, start = true;
      auto advance = [](uint32_t& slot, uint32_t& phase, uint32_t by) {
        slot += by;
        if (slot >= (uint32_t)NS) slot -= NS, phase ^= 1u;
      };
      auto there = [&](uint32_t bar, uint32_t phase) { return (bool)__all_sync(0xffffffffu, mbar_test(bar, phase)); };
      auto wait = [&](uint32_t bar, uint32_t phase, unsigned site) {
        return there(bar, phase) || __all_sync(0xffffffffu, mbar_wait(bar, phase, w, site));
      };
      auto product = [&](const Job& j, uint32_t t) {  // O_t (+)= P V
        if (!wait(BAR(KV_FULL) + 8 * j.vslot, j.vphase, 75)) return false;
        if (j.first && runs[t] > 0 && !wait(BAR(O_EMPTY) + 8 * t, (runs[t] - 1) & 1, 76)) return false;  // the run before has been read
        if (!wait(BAR(P_FULL) + 16 * t, ps[t] & 1, 77)) return false;
        tc_fence_after();
        const uint64_t vd = smem_desc_sw128(kv_s + j.vslot * TILE, 1024, CH * 1024);
        const uint32_t dst = tmem + 256u + (t ? (uint32_t)D : 0u), pa = tmem + (t ? 128u : 0u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts_w(dst, pa + kk * 8, desc_add(vd, kk * CH * 2048), IDESC_O, (!j.first || kk > 0) ? 1u : 0u);
        if (!wait(BAR(P_FULL) + 16 * t + 8, ps[t] & 1, 78)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 4; kk < 8; ++kk) mma_ts_w(dst, pa + kk * 8, desc_add(vd, kk * CH * 2048), IDESC_O, 1u);
        ++ps[t];
        if (j.first) ++runs[t];
        if (j.frees) mma_commit_w(BAR(KV_EMPTY) + 8 * j.vslot);
        if (j.last) mma_commit_w(BAR(O_FINAL) + 8 * t);
        return true;
      };
      Piece s;
      for (int piece = 0; ok && take(piece, s, 79) && s.t0 < s.t1; ++piece) {
        const int tiles = s.t1 - s.t0, subs = s.ntok > p.tile_tokens ? 2 : 1;
        const int alone = 3 - subs;  // jobs between a tile's jobs on the same S: key tiles in turn, or every one
        for (int x = 0; x < tiles && ok; ++x) {
          bool here = there(BAR(KV_FULL) + 8 * sk, pk);
          for (int sub = 0; sub < subs; ++sub, ++n) {
            const uint32_t t = n & 1, q = qt + sub, qs = q & 1;
            if (x == 0 && here) here = there(BAR(QUERIES) + 8 * qs, q >> 1 & 1);
            if (!here) {
              // Inputs that have not come yet: the last job's product need not wait for them.  (Not
              // for the second tile of rows: its values' place in the ring may be these keys'.)
              if (sub == 0) {
                if (before.on && !(ok = product(before, t ^ 1))) break;
                before.on = false;
              }
              ok = wait(BAR(KV_FULL) + 8 * sk, pk, 81);
              if (ok && x == 0) ok = wait(BAR(QUERIES) + 8 * qs, q >> 1 & 1, 80);
              if (!ok) break;
              here = true;
            }
            tc_fence_after();
            const uint64_t qd = smem_desc_sw128(q_s + qs * TILE, 16, 1024), kd = smem_desc_sw128(kv_s + sk * TILE, 16, CH * 1024);
            const uint32_t dst = tmem + (t ? 128u : 0u);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t o = (kk % 4) * 32;
              mma_ss_w(dst, desc_add(qd, (kk / 4) * CHUNK + o), desc_add(kd, (kk / 4) * 1024 + o), IDESC_S, kk > 0);
            }
            mma_commit_w(BAR(S_FULL) + 8 * t);
            if (x == tiles - 1) mma_commit_w(BAR(Q_EMPTY) + 8 * qs);
            if (sub == subs - 1) mma_commit_w(BAR(KV_EMPTY) + 8 * sk);
            if (before.on && !(ok = product(before, t ^ 1))) break;
            before = {sv, pv, true, x < alone, x >= tiles - alone, sub == subs - 1};
          }
          advance(sk, pk, start ? 1u : 2u);  // (as k_place and v_place count)
          advance(sv, pv, 2u);
          start = false;
        }
        qt += subs;
      }
      if (ok && before.on) ok = product(before, (n - 1) & 1);
      // Drain: every product and every earlier commit's arrival has landed
      // before TMEM is released and the CTA's shared memory goes away.
      mma_commit_w(BAR(DRAIN));
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(BAR(DRAIN), 0) && globaltimer_ns() - t0 < p.timeout_ns) {
      }
    }
    __syncwarp();
    if (many) __syncthreads();  // shared memory changes hands, and registers
    if (ALL) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
  } else {
    if (KV8 && warp >= 12) {
      if constexpr (KV8) {
        if (many) {
          asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
          // ============================================================ codes to f16
          // A tile of codes as TMA lays it, 16-byte chunks swizzled over the banks, becomes one of
          // f16 as the products take it, in its place: the codes are its second half, and those
          // of the last 64 keys wait in registers until all have been read.  (With the codes in a ring
          // of their own there was room for three tiles, and products waited 1000 cycles each.)
          const int me = threadIdx.x & 127;
          auto convert = [&](int place) {
            const int slot = place % NS;
            const bool ok = mbar_wait(BAR(RAW_FULL + slot), place / NS & 1, w, 91);
            uint8_t* tile = sb + L::kKVOff + slot * TILE;
            const uint4* raw = reinterpret_cast<const uint4*>(tile + L::kRawTile);
            constexpr int N = D / 32;  // chunks of a thread in half a tile
            uint4 x[N], late[N];
            auto put = [&](const uint4& codes, int at) {
              const int key = at / (D / 16), c = (at % (D / 16)) ^ (D == 128 ? key & 7 : key >> 1 & 3);
              uint4 y[2];
              codes_f16(codes.x, y[0].x, y[0].y), codes_f16(codes.y, y[0].z, y[0].w);
              codes_f16(codes.z, y[1].x, y[1].y), codes_f16(codes.w, y[1].z, y[1].w);
              uint8_t* row = tile + (key >> 3) * CH * 1024 + (c >> 2) * 1024 + (key & 7) * 128;
              const int odd = c >> 2 & 1;  // (d = 128: half the lanes store their second half first, to other banks)
              *reinterpret_cast<uint4*>(row + ((((2 * c + odd) & 7) ^ (key & 7)) << 4)) = odd ? y[1] : y[0];
              *reinterpret_cast<uint4*>(row + ((((2 * c + 1 - odd) & 7) ^ (key & 7)) << 4)) = odd ? y[0] : y[1];
            };
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = raw[i * 128 + me];
#pragma unroll
            for (int i = 0; i < N; ++i) put(x[i], i * 128 + me);
#pragma unroll
            for (int i = 0; i < N; ++i) late[i] = raw[(N + i) * 128 + me];
            // (where a warp's wait has run out all four stop here: none waits for it again)
            if (!all_of_128(1, ok)) return false;
#pragma unroll
            for (int i = 0; i < N; ++i) put(late[i], (N + i) * 128 + me);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(KV_FULL + slot));
            return true;
          };
          bool ok = true;
          int it = 0;
          Piece s;
          for (int piece = 0; ok && take(piece, s, 93) && s.t0 < s.t1; ++piece)
            for (int x = s.t0; x < s.t1 && ok; ++x, ++it) ok = convert(k_place(it)) && (it == 0 || convert(v_place(it - 1)));
          if (ok && it > 0) convert(v_place(it - 1));
        }
      }
      __syncwarp();
      if (many) __syncthreads();
      asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    } else {
      if (!KV8 && (!ALL || many)) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
      else if (KV8 && many) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
      if (many) {
        // ============================================================ softmax
        const int t = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_off + (t ? 128u : 0u), tO = tmem + lane_off + 256u + (t ? (uint32_t)D : 0u);
        float sl2 = p.scale_log2;
        const float tau = KV8 ? fminf(p.tau, kMaxTau) : p.tau;
        int qt = 0;  // tiles of Q so far
        const int my_tok = r / p.heads, my_head = r - my_tok * p.heads;
        const long long rows = (long long)p.B * p.Nq * p.Hq;
        bool ok = true;
        int n0 = 0, it0 = 0, phase = 0, runs = 0;  // jobs and key tiles before the piece; S phases and runs of this tile
        uint32_t xg = 0, xb = 0, flip = 0;
        Piece s;
        for (int piece = 0; ok && take(piece, s, 82) && s.t0 < s.t1; ++piece) {
          const int tiles = s.t1 - s.t0;
          const bool pair = s.ntok > p.tile_tokens;
          const int side = (t ^ n0) & 1;  // pair: tile of rows; else: which of the two runs of key tiles
          const int tok = s.tok0 + (pair ? side * p.tile_tokens : 0) + my_tok;
          const bool valid = my_tok < p.tile_tokens && tok < s.tok0 + s.ntok;
          // the keys this row sees: [key_lo, key_hi)
          int key_lo = 0, key_hi = 0;
          if (valid) {
            const int b = p.Nq == 1 ? tok : (int)((unsigned)tok / (unsigned)p.Nq);
            const int len = s.kind == 1 ? s.end : min(max(p.seq_lens[b], 0), p.max_len), pos = len - p.Nq + tok - b * p.Nq;
            key_lo = p.win_left >= 0 ? max(s.lo, pos - p.win_left) : s.lo;
            key_hi = min(s.end, pos + 1);
          }
          const bool live = __any_sync(0xffffffffu, valid);  // some row of the warp is there
          if constexpr (KV8) {  // queries to f16, a row times its own scale
            const int q = qt + (pair ? side : 0), slot = q & 1;
            ok = mbar_wait(BAR(Q_FULL + slot), q >> 1 & 1, w, 95);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            uint8_t* row = sb + L::kQOff + slot * TILE + r * 128;
            uint32_t most = 0;
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
              most = largest_bf16(most, *reinterpret_cast<const uint4*>(row + (c >> 3) * CHUNK + (((c & 7) ^ (r & 7)) << 4)));
            const RowScale rs(max(most >> 16, most & 0xffffu));
            sl2 = p.scale_log2 * rs.back;
            if (!pair) {  // each group converts half, when both have seen it
              __syncwarp();
              if (lane == 0) mbar_arrive(BAR(XB + 2));
              ok = mbar_wait(BAR(XB + 2), xb++ & 1, w, 96);
              if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
              }
            }
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              uint4* at = reinterpret_cast<uint4*>(row + (c >> 3) * CHUNK + (((c & 7) ^ (r & 7)) << 4));
              if (pair || c / (D / 16) == side) *at = bf16_f16(*at, rs.to);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(BAR(Q_READY + slot));
              if (pair) mbar_arrive(BAR(Q_READY + slot));
            }
            qt += pair ? 2 : 1;
          }
          float m_ref = -INFINITY, l = 0.f;
          bool poison = false;
          const int x_step = pair ? 1 : 2, x_first = pair ? 0 : side;
          for (int x = x_first; x < tiles; x += x_step, ++phase) {
            const int j0 = s.beg + (s.t0 + x) * kSharedTile;
            ok = mbar_wait(BAR(S_FULL + t), phase & 1, w, 83);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const float* sc = s_scale + (it0 + x) % (SCALES + !SCALES) * 24;
            const bool inside = j0 >= s.all_lo && j0 + kSharedTile <= s.all_hi;  // every row sees every key
            if (!inside) {
              // Some rows do not see some keys of the tile, and 0 times a NaN or an infinity
              // is not 0.  What no row sees (it may be anything) counts as zero; a value row
              // that some see, and that holds one, counts as zero too, and its rows get a NaN.
              const int uv = v_place(it0 + x), vslot = uv % NS;
              ok = mbar_wait(BAR(KV_FULL + vslot), uv / NS & 1, w, 84);
              if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
              }
              const int key = j0 + r;
              const bool out = key < s.lo || key >= s.end;
              uint4* row = reinterpret_cast<uint4*>(sb + L::kKVOff + vslot * TILE + (r >> 3) * CH * 1024 + (r & 7) * 128);
              // (a value scale that is no number makes all its page's values such)
              bool odd = KV8 && !out && !(fabsf(sc[8 + (r >> 4)]) < INFINITY);
              if (KV8 || max(j0, s.lo) < s.all_lo || min(j0 + kSharedTile, s.end) > s.all_hi) {
                if (!out && (key < s.all_lo || key >= s.all_hi)) {
                  uint32_t bad = 0;
#pragma unroll 1
                  for (int i = 0; i < 8 * CH; ++i) {
                    const uint4 v = row[(i >> 3) * 64 + (i + lane & 7)];  // (other banks for each lane)
                    constexpr uint32_t E = KV8 ? 0x7c007c00u : 0x7f807f80u;
                    bad |= __vcmpeq2(v.x & E, E) | __vcmpeq2(v.y & E, E) | __vcmpeq2(v.z & E, E) | __vcmpeq2(v.w & E, E);
                  }
                  odd |= bad != 0;
                }
                const uint32_t votes = __ballot_sync(0xffffffffu, odd);
                uint32_t* slot = s_bad + 8 * t + 4 * (flip++ & 1);
                if (lane == 0) {
                  slot[quarter] = votes;
                  mbar_arrive(pair ? BAR(XB + 2) : BAR(XB + t));
                }
                // (pairs: both tiles' warps have read the values before either clears them)
                ok = pair ? mbar_wait(BAR(XB + 2), xb++ & 1, w, 85) : mbar_wait(BAR(XB + t), xg++ & 1, w, 86);
                if (!__all_sync(0xffffffffu, ok)) {
                  ok = false;
                  break;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int a = min(max(key_lo - j0 - 32 * i, 0), 32), z = min(max(key_hi - j0 - 32 * i, 0), 32);
                  const uint32_t sees = z > a ? (0xffffffffu >> (32 - (z - a))) << a : 0u;
                  poison |= (slot[i] & sees) != 0;
                }
              }
              if (side == 0 || !pair) {  // (the other tile's product comes behind this one's)
                if (out || odd) {
#pragma unroll
                  for (int i = 0; i < 8 * CH; ++i) row[(i >> 3) * 64 + (i + lane & 7)] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
              }
            }
            if (live) {
              uint32_t sr[4][32], none = 0;  // bit c: no row of the warp sees any of the c-th 32 keys
              constexpr int G = KV8 ? 8 : 4;  // loads, each with its maximum
              float mq[G], mul[KV8 ? 8 : 1];  // what scores of each load's keys are multiplied by
              float v_mul[KV8 ? 8 : 1], v_log[KV8 ? 8 : 1];
              if constexpr (KV8) {
                // (the scales are asked for here, in whole vectors: read where they are used, each was
                // waited for, 1000 cycles a tile)
                load_8(sc, mul), load_8(sc + 16, v_log), load_8(sc + 8, v_mul);
#pragma unroll
                for (int g = 0; g < 8; ++g) tmem_ld16_max(tS + 16 * g, &sr[g >> 1][16 * (g & 1)], mq[g]);
#pragma unroll
                for (int g = 0; g < 8; ++g) mul[g] *= sl2;
                if (!inside) {  // (who sees values whose scale is no number has a NaN by `poison`)
#pragma unroll
                  for (int g = 0; g < 8; ++g) v_mul[g] = v_mul[g] == v_mul[g] ? v_mul[g] : 0.f;
                }
              } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_max(tS + 32 * c, sr[c], mq[c]);
                mul[0] = sl2;
              }
              tmem_ld_wait();
              if (!inside) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const int a = min(max(key_lo - j0 - 32 * c, 0), 32), z = min(max(key_hi - j0 - 32 * c, 0), 32);
                  const uint32_t sees = z > a ? (0xffffffffu >> (32 - (z - a))) << a : 0u;
                  if (__any_sync(0xffffffffu, ~sees)) {
                    none |= __any_sync(0xffffffffu, sees) ? 0u : 1u << c;
#pragma unroll
                    for (int h = 0; h < G / 4; ++h) {
                      float m = -INFINITY;
#pragma unroll
                      for (int i = h * (128 / G); i < (h + 1) * (128 / G); i += 2) {
                        // (times its scale first: -inf times 0 is no number)
                        if constexpr (KV8) {
                          sr[c][i] = __float_as_uint(__uint_as_float(sr[c][i]) * mul[2 * c + h]);
                          sr[c][i + 1] = __float_as_uint(__uint_as_float(sr[c][i + 1]) * mul[2 * c + h]);
                        }
                        if (!(sees >> i & 1)) sr[c][i] = 0xff800000u;
                        if (!(sees >> (i + 1) & 1)) sr[c][i + 1] = 0xff800000u;
                        m = max3f(m, __uint_as_float(sr[c][i]), __uint_as_float(sr[c][i + 1]));
                      }
                      mq[c * (G / 4) + h] = m;
                      if constexpr (KV8) mul[2 * c + h] = 1.f;
                    }
                  }
                }
              }
              float m_new = -INFINITY;
              if constexpr (KV8) {
#pragma unroll
                for (int g = 0; g < 8; g += 2) m_new = max3f(m_new, fmaf(mq[g], mul[g], v_log[g]), fmaf(mq[g + 1], mul[g + 1], v_log[g + 1]));
                m_new -= kAtRefLog2;
              } else {
                m_new = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * sl2;
              }
              float alpha = 1.f, half = 1.f;  // KV8: alpha = half^2
              const bool moves = m_new > m_ref + tau;
              if (moves) {
                if constexpr (KV8) half = ex2_sfu(0.5f * (m_ref - m_new)), alpha = half * half;
                else alpha = ex2_sfu(m_ref - m_new);
                m_ref = m_new;
              }
              if (x != x_first && __any_sync(0xffffffffu, moves)) {
                // rows whose reference moved: O *= alpha (alpha = 1 for the others)
#pragma unroll 1
                for (int c = 0; c < D; c += 8) {
                  uint32_t ov[8];
                  tmem_ld8(tO + c, ov);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 8; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                  tmem_st8(tO + c, ov);
                }
              }
              const float mb = m_ref == -INFINITY ? 0.f : m_ref;
              const uint64_t nmb2 = f2_pack(-mb, -mb);
              uint64_t acc[2] = {0ull, 0ull};
              uint32_t pk[32];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                if (!(none >> c & 1)) {
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    const int g = KV8 ? 2 * c + (i >> 3) : 0;
                    float y0, y1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c][2 * i]), __uint_as_float(sr[c][2 * i + 1])),
                                     f2_pack(mul[g], mul[g]), nmb2), y0, y1);
                    float p0 = ex2_sfu(y0), p1 = ex2_sfu(y1);
                    acc[i & 1] = f2_add(acc[i & 1], f2_pack(p0, p1));
                    if constexpr (KV8) {
                      f2_unpack(f2_mul(f2_pack(p0, p1), f2_pack(v_mul[g], v_mul[g])), p0, p1);
                      pk[16 * (c & 1) + i] = pack_f16x2(p0, p1);
                    } else {
                      pk[16 * (c & 1) + i] = pack_bf16x2(p0, p1);
                    }
                  }
                } else {  // keys that no row of the warp sees
#pragma unroll
                  for (int i = 0; i < 16; ++i) pk[16 * (c & 1) + i] = 0u;
                }
                if (c & 1) {  // 64 keys: their product may begin
                  tmem_st32(tS + 16 * (c - 1), pk);
                  tmem_st_wait();
                  tc_fence_before();
                  mbar_arrive(BAR(P_FULL + 2 * t + (c >> 1)));
                }
              }
              float s0, s1;
              f2_unpack(f2_add(acc[0], acc[1]), s0, s1);
              // (value scales move the reference by up to 2^160, which half leaves in range; l stays there)
              l = KV8 ? fmaf(l * half, half, s0 + s1) : fmaf(l, alpha, s0 + s1);
            } else {
              tc_fence_before();
              mbar_arrive(BAR(P_FULL + 2 * t));
              mbar_arrive(BAR(P_FULL + 2 * t + 1));
            }
          }
          if (!ok) break;
          n0 += pair ? 2 * tiles : tiles;
          it0 += tiles;
          // ---------------------------------------------------------- results of the run
          const int h = s.head * p.heads + my_head;
          const long long place = s.side == 0 ? s.place + (pair ? 0 : side) * rows + (long long)tok * p.Hq + h
                                              : s.place + side * s.side + r;
          if (x_first >= tiles) {  // one tile of keys: the other run has none
            if (valid) p.part_lse[place] = -INFINITY;
            continue;
          }
          ok = mbar_wait(BAR(O_FINAL + t), runs & 1, w, 87);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          ++runs;
          if (live) {
            tc_fence_after();
            const float inv = poison ? __uint_as_float(0x7fffffffu) : 1.f / l;
            float* dst = p.part_o + place * D;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              tmem_ld32(tO + 32 * c, ov);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * inv);
              if (valid && l != 0.f) {
#pragma unroll
                for (int i = 0; i < 32; i += 8) st_global_v8(dst + 32 * c + i, ov + i);
              }
            }
            // l = 0: the row sees none of these keys (a NaN passes through)
            if (valid) p.part_lse[place] = l == 0.f ? -INFINITY : m_ref + __log2f(l);
            tc_fence_before();
          }
          mbar_arrive(BAR(O_EMPTY + t));
        }
      }
      __syncwarp();
      if (many) {
        fence_proxy_async_smem();
        __syncthreads();
      }
      if (KV8) {
        if (many) asm volatile("setmaxnreg.dec.sync.aligned.u32 152;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
      } else if (ALL) {
        if (many) asm volatile("setmaxnreg.dec.sync.aligned.u32 168;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
      } else {
        few_rows();
      }
    }
    if (KV8) few_rows();
  }
  if (ALL) few_rows();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The main kernel: p.shares CTAs, behind the plan (cfg has the stream and the attribute that lets it start early).
template <int D, int NR, bool KV8>
static cudaError_t launch_shared_t(const CUtensorMap (&maps)[5], const SharedParams& p, cudaLaunchConfig_t& cfg) {
  auto kern = fa_decode_shared_kernel<D, NR, KV8>;
  constexpr uint32_t smem = SharedLayout<D, KV8>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)p.shares);
  cfg.blockDim = dim3(SharedLayout<D, KV8>::kThreads);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], maps[3], maps[4], p);
}
template <int D, bool KV8>
static cudaError_t launch_shared_main(const CUtensorMap (&maps)[5], const SharedParams& p, cudaLaunchConfig_t& cfg) {
  switch (p.few) {
    case 8: return launch_shared_t<D, 1, KV8>(maps, p, cfg);
    case 16:
      if constexpr (!(KV8 && D == 128)) return launch_shared_t<D, 2, KV8>(maps, p, cfg);
      else return cudaErrorInvalidValue;  // (shared_few gives these to tiles)
    default: return launch_shared_t<D, 0, KV8>(maps, p, cfg);
  }
}

}  // namespace fa
