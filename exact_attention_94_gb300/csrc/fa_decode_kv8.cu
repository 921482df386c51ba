// Attention of a few query tokens per request over the 8-bit paged cache.
//     s_j = scale * k_scale(page_j) * q . k8_j
//     O = sum_j softmax(s)_j * v_scale(page_j) * v8_j,   lse = log sum_j e^(s_j)
//
// The step is bound by HBM (2 d bytes per key and K/V head), so what matters
// is that the codes meet no work of their own: both products run on the fifth-
// generation tensor cores on the e4m3 codes as they lie in the cache, and no
// code ever passes through a register.  The keys take the M side, 128 of them,
// and the few query rows of a K/V head (its group's heads times the request's
// query tokens) the N side:
//     S^T [128 keys x rows] = K8 Q^T        A = K tile, B = Q
//     O^T [d x rows]       += V8^T P^T      A = V tile read MN-major, B = P
// B is then what has to be made 8-bit, and it is made so without loss that
// counts, as a sum of 8-bit numbers, each part a column of its own:
//     q = 2^k (q1 + q2 / 16), e4m3, exactly (a bf16 has 8 significant bits, an e4m3 4)
//         for what is within 2^13 of the row's largest, to 2^-22 of the largest below
//     p = p1 + p2 / 8 + p3 / 128, e5m2, exactly for p rounded to f16
// p's rounding is what the products lose: 2^-11 of a probability, or 2^-35 of the
// row's largest (its reference, below) where that is more.  (Three e4m3 parts 16 times
// apart hold the f16 too, but nothing below 2^-24 of the reference: of a first key
// 17 above 32767 others whose values alone count, nothing was left of O = 0.00135.
// Four e5m2 parts cut off, not rounded, need a fourth of P's columns more.)  Page
// scales are one factor per key: k_scale joins the score, v_scale the probability.
// P lies by key (N-major), so a thread, which has all rows of a key, stores 16 codes
// at a time.
//
// O stays in TMEM over the tiles.  It is made against a reference per row, in
// log2 units of probability times value scale, at which p = 4096: the reference
// moves only when a p would pass what rounds to e5m2's largest (2^3.9 times the
// largest at the reference's making), and O is rescaled then.  A tile costs a vote of the four
// softmax warps on that, and no exchange of maxima.  The row sums share the
// reference, so they are a row's mass divided by the value scale of its loudest
// key: fp32 holds them for value scales of 2^-80 to 2^80, and beyond drops keys
// (with scales of 2^L what is below 2^(L - 126) of the largest).
//
// Work: the tiles of 128 keys of all (request, K/V head, row tile) units in
// one list, dealt in equal shares to the CTAs (two or three per SM), which
// balances requests of any lengths; a unit counts some tiles more than it has,
// for its start and end.  A unit inside one share is finished there; one that
// a share's border cuts leaves normalised partials, which a second kernel
// merges: lse = log sum_c e^(lse_c), O = sum_c e^(lse_c - lse) O_c.  (Merged by
// the unit's last CTA instead, in the one kernel, a single request of 777
// tokens took 13.3 us and not 9.6, 32 rows 78.8 and not 72.3: the fences and
// the count cost more than a launch that overlaps the main kernel's end.)
//
// CTA:
//   warps 0-3  thread = key of the tile (TMEM lane) for S and P, and one of the
//              d output elements at a unit's end (for 32 rows, warps 0-7)
//   next       producer: block table and scales, a TMA box per page into rings
//              of K and of V tiles, across the units' borders
//   last       issues the products
// S is double buffered in TMEM (the next tile's scores are ready when a tile's
// softmax starts); P is not: it is written when the product before has read it.
//
// Measured, d = 128 unless said, pages of 16 to 64, replayed graphs of many calls:
//   64 requests of 16385 to 32768 tokens, 64 heads over 8      479 us  6.74 TB/s
//   256 requests of 1 to 2048, 64 heads over 8                  97 us  5.6 TB/s
//   8 requests of 1000 to 8192, 32 heads over 32                54 us  5.5 TB/s
//   16 requests of 100 to 16384, 4 drafts, 64 heads over 8      59 us  4.6 TB/s
//   the same with 8 drafts, 64 rows in two tiles                99 us  2.8 TB/s
//   4096 requests of 1 to 128, 64 heads over 8                 229 us  2.9 TB/s
//   32 requests, a window of 4096, 16 heads over 4, d = 64      20 us  3.0 TB/s
//   1 request of 777, 32 heads over 8                          8.4 us
// The first is as fast as the card copies.  The calls of 20 to 60 us lose some
// 5 us to the start (lengths, page numbers, pages: three reads one after the
// other before the first tile) and the merge.  Units of one tile are a chain of
// exchanges between the warps, 3.2 us each, three at once per SM.  32 rows are
// bound by the softmax warps' instructions (issue slots 51% busy) and their
// waits for one another: they came from 82 us with one group of warps and a
// byte store per code, by two groups (72), P by key and its split in half
// precision (66), all scores read at once (62.5), packed fp32 arithmetic (60) and
// parts of P that are bytes of an f16 (59).  More than 32 rows are tiles of 32 that
// follow one another in a share, so each reads the cache again (64 rows: 1.6
// times its bytes from HBM, the rest from L2) and pays for 32 rows: 33 cost 64's.
#include "serving.cuh"

#include <cmath>

namespace fa {

namespace {

constexpr int kParts = 3;            // of a P
constexpr float kAtRef = 4096.f;     // p at the reference
constexpr float kHeadroom = 3.9f;    // log2(61440 / 4096), rounded down: from 61440 on p1 would be infinite
// log2 of a value scale, from below: a page of zeros counts as one of 2^-80 (with
// 2^-100 the sums of a long row times kAtRef could overflow)
constexpr float kLeastScale = -80.f;
// What a unit's start and end cost, in tiles.  Against none at all: 16 requests
// of 100 to 16384 tokens with 32 rows 82 -> 60 us, with 8 rows 53.3 -> 51.9; 128 up
// to 2000, d = 64, 49 -> 37; a window of 4096 24.3 -> 20.6.  With 2 the 32 rows take
// 63.5; with 6 the 128 requests take 40.
constexpr int kLead(int RT) { return 3 + RT / 16; }
constexpr float kNoRef = -3.0e38f;   // reference of a row that has seen no key

// CTAs per SM: three where registers and shared memory allow it, for the loads
// and the units in flight (two: 4096 requests up to 128 tokens, 8 rows, 331 us, and
// not 229; 128 up to 2000, d = 64, 39.8 and not 37.2; only 16 or more tiles a unit
// would have it the other way, by 2%).
constexpr int kv8_ctas_per_sm(int RT) { return RT <= 8 ? 3 : 2; }

template <int D, int RT>
struct Layout {
  // Softmax warps come in groups of four (one for each quarter of a tile's
  // keys); 32 rows are two groups' work, 16 rows each (one group, when both were
  // measured, 66 us for the 62.5 of two; for 16 rows and fewer two gain nothing).
  static constexpr int kGroups = RT == 32 ? 2 : 1;
  static_assert(RT / kGroups <= 16, "rows of a group");
  static constexpr int kThreads = (4 * kGroups + 2) * 32;
  static constexpr uint32_t kSlot = 128u * D;                                // a tile of K or V
  static constexpr int kCtas = kv8_ctas_per_sm(RT);
  // Rings of K and of V tiles.  A V tile is held longer, until its product has
  // been made, so where CTAs are two, V's ring has a tile more than K's (with as
  // many, four drafts of eight heads 62.1 us, not 59.4).
  static constexpr int kKs = 256 / D;
  static constexpr int kVs = kCtas == 3 ? 256 / D : 384 / D;
  static constexpr int kSlots = kKs + kVs;
  static constexpr int kNS = 2 * RT < 16 ? 16 : 2 * RT;                      // columns of S
  // Columns of P and O: three parts of RT, and what is left of a strip's 32,
  // which holds anything and is not read.  P lies in strips of 32 columns, a
  // key's 32 bytes after another's, so that its thread writes 16 at a time.
  static constexpr int kNP = (kParts * RT + 31) / 32 * 32;
  static constexpr uint32_t kStrip = kKv8Tile * 32u;
  static constexpr uint32_t kUsed = 2 * kNS + kNP;
  static constexpr uint32_t kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : 256;  // TMEM columns, two CTAs' 512 at most
  static constexpr uint32_t kPOff = kSlots * kSlot;
  static constexpr uint32_t kQOff = kPOff + kKv8Tile * (uint32_t)kNP;
  static constexpr uint32_t kScOff = kQOff + kNS * (uint32_t)D;              // per V slot: 8 key scales, 8 value scales
  static constexpr uint32_t kScBytes = 64;
  // [4][RT] each: warps' maxima, sums, references, factors, output rows
  static constexpr uint32_t kMaxOff = kScOff + kVs * kScBytes;
  static constexpr uint32_t kRowOff = kMaxOff + 20 * RT * 4;                 // two of: [RT] query scales, [RT] positions
  static constexpr uint32_t kMiscOff = (kRowOff + 2 * 2 * RT * 4 + 15) / 16 * 16;  // votes, scan, start
  // the piece announced ahead of its tiles, with its rows of Q as they lie in memory
  static constexpr uint32_t kPieceOff = kMiscOff + 192;
  static constexpr uint32_t kStageOff = (kPieceOff + 32 + 127) / 128 * 128;
  static constexpr uint32_t kStage = RT * D * 2u;
  static constexpr uint32_t kBarOff = kStageOff + kStage;
  static constexpr int kBars = 2 * kSlots + 10;
  static constexpr uint32_t kBytes = kBarOff + 8 * kBars + 16 + 1024;
  static_assert(kUsed <= 256, "TMEM columns");
};

// A request's length as the kernels use it: clamped into [0, max_len], a length outside reported.
__device__ __forceinline__ int kv8_clamp(const Kv8DecodeParams& p, int n) {
  if (n < 0 || n > p.max_len) {
    atomicCAS(p.err, 0u, FA_DEVERR_BAD_SEQLEN);
    n = n < 0 ? 0 : p.max_len;
  }
  return n;
}
__device__ __forceinline__ int kv8_len(const Kv8DecodeParams& p, int b) { return kv8_clamp(p, p.seq_lens[b]); }

// First key any of the request's queries sees, rounded down to a tile; tiles from there.
__device__ __forceinline__ int kv8_begin(const Kv8DecodeParams& p, int len) {
  if (p.win_left < 0) return 0;
  const int lo = len - p.Nq - p.win_left;
  return lo <= 0 ? 0 : lo / kKv8Tile * kKv8Tile;
}
__device__ __forceinline__ int kv8_tiles(const Kv8DecodeParams& p, int len) {
  return (len - kv8_begin(p, len) + kKv8Tile - 1) / kKv8Tile;
}

// a / b for a >= 0, b > 0, in 32 bits where both fit (a 64-bit division takes some hundred instructions)
__host__ __device__ __forceinline__ long long quick_div(long long a, long long b) {
  return (((unsigned long long)a | (unsigned long long)b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// First slot of a CTA's share of the whole weight.
__host__ __device__ __forceinline__ long long share_begin(long long total, int shares, int k) {
  const long long each = quick_div(total, shares), more = total - each * shares;  // the first `more` shares have one slot more
  return each * k + (k < more ? k : more);
}

// A unit weighs its tiles and p.lead more, what its start and end cost a CTA in
// tiles; slot p.lead + t of its weight is tile t.
__device__ __forceinline__ long long kv8_weight(const Kv8DecodeParams& p, int tiles) {
  return tiles > 0 ? tiles + p.lead : 0;
}

// A piece of a share: tiles t0 .. t1 - 1 of unit u (K/V head and row tile) of
// request b; t0 = t1 marks the share's end.
struct Piece {
  int b, u, t0, t1, tiles, len, beg, pad;
};

// Where the requests' weights begin: thread t of the block adds up requests b0 .. b1 - 1.
struct Scan {
  long long before, mine, total;  // weight before the thread's requests, of them, of all
  int b0, b1;
};
template <int WARPS>
__device__ __forceinline__ Scan kv8_scan(const Kv8DecodeParams& p, int units, long long* s_scan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = (p.B + 32 * WARPS - 1) / (32 * WARPS);
  Scan c{0, 0, 0, min(p.B, tid * n), min(p.B, tid * n + n)};
  for (int b = c.b0; b < c.b1; ++b) c.mine += kv8_weight(p, kv8_tiles(p, kv8_len(p, b))) * units;
  long long sum = c.mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += x;
  }
  if (lane == 31) s_scan[warp] = sum;
  __syncthreads();
  c.before = sum - c.mine;
#pragma unroll
  for (int x = 0; x < WARPS; ++x) {
    if (x < warp) c.before += s_scan[x];
    c.total += s_scan[x];
  }
  return c;
}
// The request that holds a slot of the whole weight, by the thread that has it:
// its number, the slot within it, its tiles and its length.
__device__ __forceinline__ void kv8_find(const Kv8DecodeParams& p, int units, const Scan& c, long long slot,
                                         volatile long long* out) {
  if (slot < c.before || slot >= c.before + c.mine) return;
  long long at = c.before;
  for (int b = c.b0; b < c.b1; ++b) {
    const int len = kv8_len(p, b), tiles = kv8_tiles(p, len);
    if (slot < at + kv8_weight(p, tiles) * units) {
      out[0] = b;
      out[1] = slot - at;
      out[2] = (long long)tiles << 32 | (unsigned)len;
      return;
    }
    at += kv8_weight(p, tiles) * units;
  }
}

// Row tile and K/V head of a unit.
__device__ __forceinline__ int row_tile(const Kv8DecodeParams& p, int u) {
  return p.row_tiles == 1 ? 0 : (int)((unsigned)u % (unsigned)p.row_tiles);
}
__device__ __forceinline__ int kv_head(const Kv8DecodeParams& p, int u) {
  return p.row_tiles == 1 ? u : (int)((unsigned)u / (unsigned)p.row_tiles);
}

// The producer's walk over the share, piece by piece.
struct Walk {
  long long left;  // weight of the share still to come
  long long off;   // next slot within the weight of the request's units
  int b, tiles, len;
  int len_next;    // seq_lens[b + 1], read long before it is needed

  __device__ __forceinline__ Piece next(const Kv8DecodeParams& p, int units) {
    Piece s{};
    while (left > 0) {
      const int each = tiles + p.lead;
      if (tiles == 0 || off >= (long long)each * units) {  // the request's units are done (or it has no keys)
        off = 0;
        ++b;
        len = kv8_clamp(p, len_next);
        tiles = kv8_tiles(p, len);
        len_next = b + 1 < p.B ? p.seq_lens[b + 1] : 0;
        continue;
      }
      const int u = (int)quick_div(off, each);
      const int w0 = (int)(off - (long long)u * each), w1 = (int)(left < each - w0 ? w0 + left : each);
      off += w1 - w0;
      left -= w1 - w0;
      s = {b, u, max(w0 - p.lead, 0), max(w1 - p.lead, 0), tiles, len, kv8_begin(p, len), 0};
      if (s.t0 < s.t1) return s;
    }
    s.t0 = s.t1 = 0;
    return s;
  }
};

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t* r) {
  if constexpr (N >= 16) {
    tmem_ld16(addr, r);
    if constexpr (N > 16) tmem_load<N - 16>(addr + 16, r + 16);
  } else if constexpr (N > 0) {
    static_assert(N == 8 || N == 4, "columns in fours");
    if constexpr (N == 8)
      tmem_ld8(addr, r);
    else
      tmem_ld4(addr, r);
  }
}

template <int N>
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t* r) {
  if constexpr (N >= 8) {
    tmem_st8(addr, r);
    if constexpr (N > 8) tmem_store<N - 8>(addr + 8, r + 8);
  } else if constexpr (N > 0) {
    static_assert(N == 4, "columns in fours");
    tmem_st4(addr, r);
  }
}

// Sums v[r] of the warp's lanes for every r: lane r * (32 / RT) gets the total
// of row r.  Halves the rows while it adds (31 shuffles for 32 rows, not 160).
template <int RT>
__device__ __forceinline__ float warp_row_sums(float (&v)[RT], int lane) {
  int o = 16;
#pragma unroll
  for (int n = RT / 2; n > 0; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n];
      v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  float x = v[0];
#pragma unroll
  for (int b = 16 / RT; b > 0; b >>= 1) x += __shfl_xor_sync(0xffffffffu, x, b);
  return x;
}

}  // namespace

template <int D, int RT>
__global__ void __launch_bounds__(Layout<D, RT>::kThreads, Layout<D, RT>::kCtas)
    fa_decode_kv8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ Kv8DecodeParams p) {
  using L = Layout<D, RT>;
  constexpr int KS = L::kKs, VS = L::kVs, NSL = L::kSlots;
  constexpr int GROUPS = L::kGroups, SOFT = 4 * GROUPS, kThreads = L::kThreads;  // softmax warps, then the two others
  const int k = blockIdx.x, units = p.Hkv * p.row_tiles;
  const int warp = warp_id(), lane = lane_id();

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sb = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBarOff;
  // barriers and tiles of the rings: K's slots, then V's
  auto FULL = [&](int s) { return bars + 8u * (uint32_t)s; };
  auto EMPTY = [&](int s) { return bars + 8u * (uint32_t)(NSL + s); };
  auto TILE = [&](int s) { return base + L::kSlot * (uint32_t)s; };
  const uint32_t SF = bars + 16u * NSL;  // S ready [2]; then P ready, O ready, the warps' exchange, Q ready
  const uint32_t PF = SF + 16, OF = SF + 24, QB = SF + 32, XB = SF + 40;           // (an exchange for each group, one for all)
  const uint32_t HERE = SF + 64, TAKEN = SF + 72;                                   // piece announced, and taken by all its readers
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sb + L::kBarOff + 8 * L::kBars);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sb + L::kBarOff + 8 * L::kBars + 4);
  Piece* s_piece = reinterpret_cast<Piece*>(sb + L::kPieceOff);
  int* s_vote = reinterpret_cast<int*>(sb + L::kMiscOff);                       // [2][SOFT]
  long long* s_scan = reinterpret_cast<long long*>(sb + L::kMiscOff + 64);      // [SOFT + 2] warps' sums
  volatile long long* s_start = reinterpret_cast<volatile long long*>(sb + L::kMiscOff + 144);  // b, off, tiles and len

  if (warp == SOFT + 1) {
    tmem_alloc(base + L::kBarOff + 8 * L::kBars + 4, L::kCols);
    tmem_relinquish();
    tc_fence_before();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < NSL; ++s) {
      mbar_init(FULL(s), s < KS ? 1 : 9);  // (values: the copy's bytes, and eight lanes' scales)
      mbar_init(EMPTY(s), 1);
    }
    mbar_init(SF, 1);
    mbar_init(SF + 8, 1);
    mbar_init(PF, SOFT);
    mbar_init(OF, 1);
    mbar_init(QB, SOFT);
    mbar_init(XB, 4);
    mbar_init(XB + 8, 4);
    mbar_init(XB + 16, SOFT);
    mbar_init(HERE, 1);
    mbar_init(TAKEN, SOFT + 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  const Scan scan = kv8_scan<kThreads / 32>(p, units, s_scan);
  const long long from = share_begin(scan.total, (int)gridDim.x, k), to = share_begin(scan.total, (int)gridDim.x, k + 1);
  kv8_find(p, units, scan, from, s_start);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tO = tmem + 2 * L::kNS;
  const WaitCtx w{abort_flag, p.timeout_ns, p.err};
  bool ok = true;
  asm volatile("griddepcontrol.launch_dependents;");  // the merge may be set up; it waits for this grid's end

  if (warp == SOFT) {
    // ============================================================ producer
    // With the ring full, every load of the SM waits behind the ring's bytes, 2
    // to 4 us, so no register waits for one that was just asked for.  Tiles go in
    // batches of four of a piece, lane i owning 16 keys.  Page numbers are read
    // two batches ahead (and moved to their place one later, when they have
    // come); scales are copied asynchronously to the tile's place, and arrive on
    // its barrier.  A piece is announced, with its rows of Q, before its first
    // tile is asked for.  (That waits until the piece before has been taken, which
    // needs no tile that has not been asked for.  Announcing two or three pieces
    // ahead where shared memory allows it gained nothing.)
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    struct Batch {
      int n;     // tiles, 0: none left
      int page;  // this lane's 16 keys: page, slot of the first, whether they exist
      int off;
      bool on;
      int hk;
      bool first;  // the piece's first batch
      Piece pc;
    };
    Walk walk{to - from, 0, 0, 0, 0, 0};
    if (to > from) {
      const int b = (int)s_start[0];
      walk = {to - from, s_start[1], b, (int)(s_start[2] >> 32), (int)(s_start[2] & 0xffffffffll),
              b + 1 < p.B ? p.seq_lens[b + 1] : 0};
    }
    const int bpb = p.box_rows / 16;  // 16-key groups per TMA box
    Piece pc{};
    int t_next = 0, pieces = 0;  // next tile of pc to fetch; pieces fetched
    bool more = true;
    auto announce = [&](const Piece& pc) {
      if (pieces > 0) ok = __all_sync(0xffffffffu, mbar_wait(TAKEN, (pieces - 1) & 1, w, 50));
      if (!ok) return;
      const int x0 = row_tile(p, pc.u) * RT, rows = pc.t0 < pc.t1 ? min(RT, p.Nq * p.group - x0) : 0;
      if (lane == 0) {
        *s_piece = pc;
        mbar_arrive_expect_tx(HERE, (uint32_t)(rows * D * 2));
      }
      __syncwarp();
      if (lane < rows) {
        const int x = x0 + lane, i = p.Nq == 1 ? 0 : (int)((unsigned)x / (unsigned)p.group);
        const int h = kv_head(p, pc.u) * p.group + x - i * p.group;
        bulk_load(base + L::kStageOff + lane * D * 2,
                  static_cast<const __nv_bfloat16*>(p.q) + (((size_t)pc.b * p.Nq + i) * p.Hq + h) * D, D * 2, HERE);
      }
      ++pieces;
    };
    auto fetch = [&](Batch& q) {
      q = {};
      if (!more) return;
      if (t_next == pc.t1) {
        pc = walk.next(p, units);
        t_next = pc.t0;
        more = pc.t0 < pc.t1;
        if (!more) return;
        q.first = true;
        q.pc = pc;
      }
      q.n = min(4, pc.t1 - t_next);
      const int g = (pc.beg + t_next * kKv8Tile) / 16 + lane;
      // (pages that no query's window reaches may be gone; a box that it reaches lies in one that is not)
      const int lo = p.win_left < 0 ? 0 : max(0, pc.len - p.Nq - p.win_left) / 16 / bpb * bpb;
      q.on = lane < 8 * q.n && g < (pc.len + 15) / 16 && g >= lo;
      q.hk = kv_head(p, pc.u);
      t_next += q.n;
      if (q.on) {
        const int blk = (int)((unsigned)(g * 16) / (unsigned)p.page_size);
        q.off = g * 16 - blk * p.page_size;
        q.page = p.block_table[(size_t)pc.b * p.max_blocks + blk];
      }
    };
    Batch now, next;
    fetch(now);
    fetch(next);
    int it = 0;  // tiles of the share so far
    while (ok && now.n > 0) {
      if (now.on && (now.page < 0 || now.page >= p.num_pages)) {  // report, and read a valid page instead
        atomicCAS(p.err, 0u, FA_DEVERR_BAD_PAGE);
        now.page = 0;
      }
      if (now.first) announce(now.pc);
      if (!ok) break;
      const int ph = now.page * p.Hkv + now.hk;
      const uint32_t on = __ballot_sync(0xffffffffu, now.on);
      for (int i = 0; i < now.n; ++i, ++it) {
        const int boxes = (__popc(on >> (8 * i) & 0xffu) + bpb - 1) / bpb;
        const uint32_t bytes = (uint32_t)(boxes * p.box_rows * D);
        const bool mine = (lane >> 3) == i, issue = mine && now.on && (lane & (bpb - 1)) == 0;
        const uint32_t at = (uint32_t)(lane & 7) * 16u * D;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int slot = v ? KS + it % VS : it % KS, use = v ? it / VS : it / KS;
          if (use > 0) ok = mbar_wait(EMPTY(slot), (use - 1) & 1, w, 51);
          if (!__all_sync(0xffffffffu, ok)) break;
          if (lane == 0) mbar_arrive_expect_tx(FULL(slot), bytes);
          __syncwarp();
          if (issue) tma_load_3d(TILE(slot) + at, v ? &tm_v : &tm_k, FULL(slot), 0, now.off, ph);
          if (v == 1 && mine) {
            float* sc = reinterpret_cast<float*>(sb + L::kScOff + (it % VS) * L::kScBytes) + (lane & 7);
            if (now.on) {
              cp_async4(smem_u32(sc), p.k_scale + ph);
              cp_async4(smem_u32(sc + 8), p.v_scale + ph);
              cp_async_arrive(FULL(slot));  // one of the barrier's eight more arrivals, when the copies are there
            } else {
              sc[0] = sc[8] = 0.f;
              mbar_arrive(FULL(slot));
            }
          }
          __syncwarp();
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      now = next;
      fetch(next);
    }
    if (ok) announce(pc);  // the end
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == SOFT + 1) {
    // ============================================================ products
    constexpr uint32_t IDESC_S = idesc_e4m3(128, L::kNS), IDESC_O = idesc_e4m3_e5m2(D, L::kNP, true, true);
    const uint32_t qa = base + L::kQOff, pa = base + L::kPOff;
    const uint64_t qd = D == 128 ? smem_desc_sw128(qa, 16, 1024) : smem_desc_sw64(qa, 16, 512);
    const uint64_t pd = smem_desc_sw32(pa, L::kStrip, 256);
    auto pv = [&](int it, bool first) {  // O (+)= V^T P^T of tile `it`
      const int slot = KS + it % VS;
      bool good = mbar_wait(PF, it & 1, w, 54);
      if (__all_sync(0xffffffffu, good)) good = mbar_wait(FULL(slot), it / VS & 1, w, 55);
      if (!__all_sync(0xffffffffu, good)) return false;
      tc_fence_after();
      const uint32_t va = TILE(slot);
      const uint64_t vd = D == 128 ? smem_desc_sw128(va, 16, 1024) : smem_desc_sw64(va, 16, 512);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_ss_f8_w(tO, desc_add(vd, kk * 32 * D), desc_add(pd, kk * 32 * 32), IDESC_O, (kk > 0 || !first) ? 1u : 0u);
      mma_commit_w(EMPTY(slot));
      mma_commit_w(OF);
      return true;
    };
    for (int it = 0, piece = 0; ok; ++piece) {
      ok = __all_sync(0xffffffffu, mbar_wait(HERE, piece & 1, w, 56));
      if (!ok) break;
      const int n = s_piece->t1 - s_piece->t0;
      __syncwarp();
      if (lane == 0) mbar_arrive(TAKEN);
      if (n == 0) break;
      ok = __all_sync(0xffffffffu, mbar_wait(QB, piece & 1, w, 52));
      for (int t = 0; t < n && ok; ++t, ++it) {
        const int slot = it % KS;
        ok = __all_sync(0xffffffffu, mbar_wait(FULL(slot), it / KS & 1, w, 53));
        if (!ok) break;
        tc_fence_after();
        const uint32_t ka = TILE(slot);
        const uint64_t kd = D == 128 ? smem_desc_sw128(ka, 16, 1024) : smem_desc_sw64(ka, 16, 512);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          mma_ss_f8_w(tS + (it & 1) * L::kNS, desc_add(kd, kk * 32), desc_add(qd, kk * 32), IDESC_S, kk > 0);
        mma_commit_w(EMPTY(slot));
        mma_commit_w(SF + 8u * (it & 1));
        if (t > 0) ok = pv(it - 1, t == 1);
      }
      if (ok) ok = pv(it - 1, n == 1);
    }
  } else {
    // ============================================================ softmax
    constexpr int RG = RT / GROUPS;                  // rows of a group
    const int group = warp >> 2, quarter = warp & 3, g0 = group * RG;
    float* my_max = reinterpret_cast<float*>(sb + L::kMaxOff) + warp * RG;
    float* my_sum = my_max + 4 * RT;
    float* my_neg = my_max + 8 * RT;                 // this warp's copies: the rows' references, negated,
    float* my_al = my_max + 12 * RT;                 //   what a moved one multiplies sums by,
    int* my_at = reinterpret_cast<int*>(my_max + 16 * RT);  // and where the results go
    const float* g_max = my_max - quarter * RG;      // the group's four warps'
    const float* g_sum = my_sum - quarter * RG;
    const uint32_t lane_sel = (uint32_t)quarter << 21;  // TMEM lane 32 * quarter
    const int key = quarter * 32 + lane;             // key of the tile
    // column c of this thread's key in P: its strip, the key's 32 bytes, their swizzle
    uint8_t* p_row = sb + L::kPOff + key * 32;
    const int p_flip = key << 2 & 16;
    auto p_at = [&](int c) { return p_row + (c >> 5) * L::kStrip + ((c & 31) ^ p_flip); };
    const int group16 = key >> 4;                    // of the tile's keys: where its scales are
    auto rows_of = [&](const Piece& s) { return min(RT, p.Nq * p.group - row_tile(p, s.u) * RT); };
    // row r of a piece: its row of q and o, its query token
    auto q_row = [&](const Piece& s, int r, int& i, int& h) {
      const int x = row_tile(p, s.u) * RT + r;
      i = p.Nq == 1 ? 0 : (int)((unsigned)x / (unsigned)p.group);
      h = kv_head(p, s.u) * p.group + x - i * p.group;
      return ((size_t)s.b * p.Nq + i) * p.Hq + h;
    };
    // ---- the next piece, and its Q: rows in turn for the warps, split into two
    // e4m3 parts at each row's power of two
    auto take = [&](int piece, Piece& s) {
      if (!__all_sync(0xffffffffu, mbar_wait(HERE, piece & 1, w, 63))) return false;
      s = *s_piece;
      float* s_qsc = reinterpret_cast<float*>(sb + L::kRowOff + (piece & 1) * 2 * RT * 4);
      int* s_pos = reinterpret_cast<int*>(s_qsc + RT);
      const int rows = s.t0 == s.t1 ? 0 : rows_of(s);
      constexpr int LPR = D / 8, RPW = 32 / LPR;                // lanes per row, rows per warp and pass
      constexpr int PASSES = (RT + SOFT * RPW - 1) / (SOFT * RPW);
      const int sub = lane / LPR, seg = lane % LPR;
      uint4 q[PASSES];
#pragma unroll
      for (int x = 0; x < PASSES; ++x) {
        const int r = (x * SOFT + warp) * RPW + sub;
        q[x] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) q[x] = *reinterpret_cast<const uint4*>(sb + L::kStageOff + r * D * 2 + seg * 16);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(TAKEN);
      if (rows == 0) return true;
#pragma unroll
      for (int x = 0; x < PASSES; ++x) {
        const int r = (x * SOFT + warp) * RPW + sub;
        const uint32_t wd[4] = {q[x].x, q[x].y, q[x].z, q[x].w};
        float f[8], mx = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] = __uint_as_float(e & 1 ? wd[e / 2] & 0xffff0000u : wd[e / 2] << 16);
          mx = fmaxf(mx, fabsf(f[e]));
        }
        bool odd = false;  // an infinity or a NaN in the row
#pragma unroll
        for (int e = 0; e < 8; ++e) odd |= !(fabsf(f[e]) <= 3.4e38f);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = fminf(mx, 3.39e38f);
        odd = (__ballot_sync(0xffffffffu, odd) >> (sub * LPR) & ((1u << LPR) - 1u)) != 0;
        // 2^k with mx / 2^k in [128, 256)
        const int ex = max((int)(__float_as_uint(mx) >> 23) - 7, 1);  // biased exponent of 2^k
        const float inv = mx > 0.f ? __uint_as_float((uint32_t)(254 - ex) << 23) : 1.f;
        const float sc = mx > 0.f ? __uint_as_float((uint32_t)ex << 23) : 1.f;
        uint32_t c1[4], c2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = odd ? __uint_as_float(0x7fffffffu) : f[2 * e] * inv;
          const float z = odd ? __uint_as_float(0x7fffffffu) : f[2 * e + 1] * inv;
          c1[e] = pack_e4m3x2(y, z);
          const float2 g = unpack_e4m3x2(c1[e]);
          c2[e] = pack_e4m3x2((y - g.x) * 16.f, (z - g.y) * 16.f);
        }
        if (r < RT) {
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const int col = part * RT + r;
            const uint32_t* c = part ? c2 : c1;
            const uint32_t at = D == 128 ? col * 128 + (((seg >> 1) ^ (col & 7)) << 4)
                                         : col * 64 + (((seg >> 1) ^ ((col >> 1) & 3)) << 4);
            *reinterpret_cast<uint2*>(sb + L::kQOff + at + (seg & 1) * 8) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
          }
          if (seg == 0) {
            const int y = row_tile(p, s.u) * RT + r;
            s_qsc[r] = sc * p.scale_log2;
            s_pos[r] = s.len - p.Nq + (p.Nq == 1 || r >= rows ? 0 : (int)((unsigned)y / (unsigned)p.group));
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(QB);
      return true;
    };

    int it = 0, piece = 0;
    uint32_t xphase = 0;  // phase of the warps' exchange
    auto exchange = [&]() {  // every warp of the group has written what the others read next
      __syncwarp();
      if (lane == 0) mbar_arrive(XB + 8 * group);
      return __all_sync(0xffffffffu, mbar_wait(XB + 8 * group, xphase++ & 1, w, 60));
    };
    uint32_t bphase = 0;
    auto both = [&]() {  // all softmax warps have come this far
      __syncwarp();
      if (lane == 0) mbar_arrive(XB + 16);
      return __all_sync(0xffffffffu, mbar_wait(XB + 16, bphase++ & 1, w, 64));
    };
    Piece pc;
    ok = take(0, pc);
    while (ok && pc.t0 < pc.t1) {
      const float* s_qsc = reinterpret_cast<const float*>(sb + L::kRowOff + (piece & 1) * 2 * RT * 4) + g0;
      const int* s_pos = reinterpret_cast<const int*>(s_qsc + RT);  // (both from the group's first row)
      const int rows = rows_of(pc);
      // positions of the tile's first and last row; between them they rise by one or not at all
      const int x0 = row_tile(p, pc.u) * RT, at0 = pc.len - p.Nq;
      const int pos_first = p.Nq == 1 ? at0 : at0 + (int)((unsigned)x0 / (unsigned)p.group);
      const int pos_last = p.Nq == 1 ? at0 : at0 + (int)((unsigned)(x0 + rows - 1) / (unsigned)p.group);
      ok = __all_sync(0xffffffffu, mbar_wait(QB, piece & 1, w, 56));
      uint64_t l2[RG / 2];  // rows' sums of this key lane, in twos
#pragma unroll
      for (int r = 0; r < RG / 2; ++r) l2[r] = 0;
      __syncwarp();
      if (lane < RG) my_neg[lane] = 0.f;
      __syncwarp();

      for (int t = pc.t0; t < pc.t1 && ok; ++t, ++it) {
        const int vslot = KS + it % VS;
        ok = mbar_wait(SF + 8u * (it & 1), (it >> 1) & 1, w, 58);
        if (__all_sync(0xffffffffu, ok)) ok = mbar_wait(FULL(vslot), it / VS & 1, w, 59);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float* sc = reinterpret_cast<const float*>(sb + L::kScOff + (it % VS) * L::kScBytes);
        const float ks = sc[group16], vs0 = sc[8 + group16];
        const bool odd_scale = !(fabsf(vs0) <= 3.4e38f);  // (an infinity would pass as e4m3's largest)
        const float vs = odd_scale ? __uint_as_float(0x7fffffffu) : vs0, lvs = fmaxf(__log2f(vs), kLeastScale);
        const int j0 = pc.beg + t * kKv8Tile, j = j0 + key;
        // some row does not see some key of the tile
        const bool partial = j0 + kKv8Tile > pc.len - p.Nq + 1 || (p.win_left >= 0 && j0 < pc.len - 1 - p.win_left);
        auto sees = [&](int r) { return j <= s_pos[r] && (p.win_left < 0 || j >= s_pos[r] - p.win_left); };
        // A key's value row may hold NaN, and 0 * NaN is not 0.  Where no row sees
        // the key (it may be anything behind the last or before the window), its
        // values count as zero.
        // Where some rows do and some don't (drafts), a row with a NaN counts as zero
        // too, and as NaN to the rows that see it: in all their elements.  So does every
        // row of a page whose scale is no number.
        bool poison = odd_scale, any = true, all = true;
        if (partial) {
          any = j <= pos_last && (p.win_left < 0 || j >= pos_first - p.win_left);
          all = j <= pos_first && (p.win_left < 0 || j >= pos_last - p.win_left);
          uint4* row = reinterpret_cast<uint4*>(sb + vslot * L::kSlot + key * D);
          auto turn = [&](int e) { return (e + (D == 128 ? lane : lane >> 1)) & (D / 16 - 1); };  // (other banks for each lane)
          if (any && !all) {
            uint32_t nan = 0;
#pragma unroll 1
            for (int e = 0; e < D / 16; ++e) {
              const uint4 v = row[turn(e)];
              nan |= __vcmpeq4(v.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                     __vcmpeq4(v.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
            }
            poison |= nan != 0;
          }
          poison &= any;
          if (GROUPS > 1) {  // (one group's row is the other's: both have read it before either writes)
            // every softmax warp passes here: the tile is partial for all of them
            ok = both();
            if (!ok) break;
          }
          if (!any || poison) {
#pragma unroll
            for (int e = 0; e < D / 16; ++e) row[turn(e)] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        float s[RG];
        for (bool settled = false;;) {
          // ---- scores less the references, in log2 units
          uint32_t s1[RG], s2[RG];
          tmem_load<RG>(tS + (it & 1) * L::kNS + lane_sel + g0, s1);
          tmem_load<RG>(tS + (it & 1) * L::kNS + lane_sel + RT + g0, s2);
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < RG; r += 4) {
            const ulonglong2 qsc = *reinterpret_cast<const ulonglong2*>(s_qsc + r);
            const ulonglong2 neg = *reinterpret_cast<const ulonglong2*>(my_neg + r);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {  // (two rows an instruction)
              const uint64_t x = f2_fma(f2_pack(__uint_as_float(s2[r + e]), __uint_as_float(s2[r + e + 1])),
                                        f2_pack(0.0625f, 0.0625f),
                                        f2_pack(__uint_as_float(s1[r + e]), __uint_as_float(s1[r + e + 1])));
              f2_unpack(f2_fma(x, f2_mul(e ? qsc.y : qsc.x, f2_pack(ks, ks)), e ? neg.y : neg.x), s[r + e], s[r + e + 1]);
            }
          }
          if (!all) {
#pragma unroll
            for (int r = 0; r < RG; ++r) s[r] = any && sees(r) ? s[r] : -INFINITY;
          }
          if (settled) break;
          if (t == pc.t0) {  // a piece's first tile makes the references (0 so far): its largest
#pragma unroll
            for (int r = 0; r < RG; r += 4) {
              float x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = warp_max(s[r + e] + lvs);
              if (lane == 0) *reinterpret_cast<float4*>(my_max + r) = make_float4(x[0], x[1], x[2], x[3]);
            }
            ok = exchange();
            if (!ok) break;
            if (lane < RG) {  // (of a row that sees no key yet, kNoRef)
              const float x = fmaxf(fmaxf(g_max[lane], g_max[RG + lane]), fmaxf(g_max[2 * RG + lane], g_max[3 * RG + lane]));
              my_neg[lane] = -fmaxf(x, kNoRef);
            }
            __syncwarp();
            if constexpr (RG > 4) {
#pragma unroll
              for (int r = 0; r < RG; ++r) s[r] += my_neg[r];
              break;
            } else {
              // (four rows are faster read again: a window of 4096, d = 64, 20.9 us, and 22.1; eight are
              // not: 512 requests with a window of 128 64.5, and 61.8)
              settled = true;
              continue;
            }
          }
          // ---- another moves them if one of its p passes what e5m2 holds
          float top = fmaxf(s[0], s[1]);
#pragma unroll
          for (int r = 2; r < RG; r += 2) top = max3f(top, s[r], s[r + 1]);
          const bool move = __any_sync(0xffffffffu, top > kHeadroom - lvs);
          if (lane == 0) s_vote[(it & 1) * SOFT + warp] = move;
          ok = exchange();
          if (!ok) break;
          const int4 votes = *reinterpret_cast<const int4*>(s_vote + (it & 1) * SOFT + group * 4);
          if ((votes.x | votes.y | votes.z | votes.w) == 0) break;
          // ---- new references: the largest up to here (rolled loops: rare, and the code is long already)
          constexpr int G = RG > 8 ? 8 : RG;  // rows at a time
#pragma unroll 1
          for (int r = 0; r < RG; r += G) {
            uint32_t s1[G], s2[G];
            tmem_load<G>(tS + (it & 1) * L::kNS + lane_sel + g0 + r, s1);
            tmem_load<G>(tS + (it & 1) * L::kNS + lane_sel + RT + g0 + r, s2);
            tmem_ld_wait();
            float x[G];
#pragma unroll
            for (int e = 0; e < G; ++e) {
              x[e] = fmaf(__uint_as_float(s2[e]), 0.0625f, __uint_as_float(s1[e])) * (ks * s_qsc[r + e]) + lvs;
              if (!all && !(any && sees(r + e))) x[e] = -INFINITY;
              x[e] = warp_max(x[e]);
            }
            if (lane == 0) {
#pragma unroll
              for (int e = 0; e < G; e += 4)
                *reinterpret_cast<float4*>(my_max + r + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            }
          }
          ok = exchange();
          if (!ok) break;
          if (lane < RG) {
            const float x = fmaxf(fmaxf(g_max[lane], g_max[RG + lane]), fmaxf(g_max[2 * RG + lane], g_max[3 * RG + lane]));
            const float old = -my_neg[lane], now = fmaxf(old, x);  // (a row that sees no key yet has -inf in x)
            my_neg[lane] = -now;
            my_al[lane] = ex2_sfu(old - now);
          }
          __syncwarp();
#pragma unroll
          for (int r = 0; r < RG; r += 2) l2[r / 2] = f2_mul(l2[r / 2], f2_pack(my_al[r], my_al[r + 1]));
          // O stands at the old ones
          ok = __all_sync(0xffffffffu, mbar_wait(OF, (it - 1) & 1, w, 62));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int part = 0; part < kParts; ++part) {
            uint32_t o[RG];
            tmem_load<RG>(tO + lane_sel + part * RT + g0, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < RG; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * my_al[e]);
            tmem_store<RG>(tO + lane_sel + part * RT + g0, o);
          }
          tmem_st_wait();
          settled = true;
        }
        if (!ok) break;
        // ---- probabilities; P's buffer is free when the product before has read it
        if (t > pc.t0) {
          ok = __all_sync(0xffffffffu, mbar_wait(OF, (it - 1) & 1, w, 57));
          if (!ok) break;
        }
        // p rounded to f16, by 2^-11 of itself at most.  An e5m2 is an f16's upper byte:
        // the first part is that byte, rounded, which leaves 2^-3 at most, in eight
        // bits; the second leaves 2^-7, a multiple of 2^-10 that the third is exactly.
        // (Below 2^-13 the parts' own steps end; with the f16's they lose 2^-23 at most,
        // 2^-35 of the reference.)
        const float vn = poison || !any ? 0.f : vs * kAtRef;
        uint32_t code[kParts][RG / 4];
#pragma unroll
        for (int r = 0; r < RG; r += 4) {
          uint32_t x[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p0 = ex2_sfu(s[r + 2 * e]), p1 = ex2_sfu(s[r + 2 * e + 1]);
            l2[r / 2 + e] = f2_add(l2[r / 2 + e], f2_pack(p0, p1));
            float y0, y1;
            f2_unpack(f2_mul(f2_pack(p0, p1), f2_pack(vn, vn)), y0, y1);
            x[e] = pack_f16x2(y0, y1);
          }
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            const uint32_t up[2] = {e5m2_round(x[0]), e5m2_round(x[1])};
            code[part][r / 4] = __byte_perm(up[0], up[1], 0x7531);
            if (part + 1 < kParts) {
              const float more = part == 0 ? 8.f : 16.f;
              x[0] = e5m2_rest(x[0], up[0], more), x[1] = e5m2_rest(x[1], up[1], more);
            }
          }
        }
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          const uint32_t* c = code[part];
          uint8_t* at = p_at(part * RT + g0);
          if constexpr (RG == 16)
            *reinterpret_cast<uint4*>(at) = make_uint4(c[0], c[1], c[2], c[3]);
          else if constexpr (RG == 8)
            *reinterpret_cast<uint2*>(at) = make_uint2(c[0], c[1]);
          else
            *reinterpret_cast<uint32_t*>(at) = c[0];
        }
        if (poison) {
#pragma unroll 1
          for (int r = 0; r < RG; ++r)
            if (sees(r)) *p_at(g0 + r) = 0x7f;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(PF);
      }
      if (!ok) break;
      // ---- the next piece's Q, while this one's last products run (its scores are all read, so Q is free)
      const Piece done = pc;
      ok = take(piece + 1, pc);
      if (!ok) break;
      // ---- each row's sum over the 128 key lanes
      float l[RG];
#pragma unroll
      for (int r = 0; r < RG; r += 2) f2_unpack(l2[r / 2], l[r], l[r + 1]);
      const float row_sum = warp_row_sums<RG>(l, lane);
      if (lane % (32 / RG) == 0) my_sum[lane / (32 / RG)] = row_sum;
      ok = exchange();
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(OF, (it - 1) & 1, w, 61));
      if (!ok) break;
      tc_fence_after();
      // output element of this thread: its TMEM lane; an M = 64 product uses lanes 0 .. 15 of each warp's 32
      const int e = D == 128 ? key : quarter * 16 + lane;
      const bool has = D == 128 || lane < 16;
      const bool whole = done.t0 == 0 && done.t1 == done.tiles;
      // lane r works out row r of the group for its warp: where it goes, what its sums are divided by; the row's lse
      const int mine = min(RG, rows - g0);
      if (lane < mine) {
        const float sum = g_sum[lane] + g_sum[RG + lane] + g_sum[2 * RG + lane] + g_sum[3 * RG + lane];
        // sum = 0: the row sees none of these keys (a NaN passes through)
        const float lse2 = sum == 0.f ? -INFINITY : __log2f(sum) - my_neg[lane];
        my_al[lane] = sum == 0.f ? 0.f : 1.f / (sum * kAtRef);
        if (whole) {
          int i, h;
          my_at[lane] = (int)q_row(done, g0 + lane, i, h);  // (below 2^30)
          if (quarter == 0) p.lse[((size_t)done.b * p.Hq + h) * p.Nq + i] = lse2 * 0.69314718055994531f;
        } else {
          const size_t part = 2 * (size_t)k + (piece > 0 ? 1 : 0);  // a share's first piece, or its last
          my_at[lane] = (int)(part * RT) + g0 + lane;
          if (quarter == 0) p.part_lse[part * RT + g0 + lane] = lse2;
        }
      }
      __syncwarp();
      constexpr int OB = 4;  // rows at a time (8 are more code: 4096 requests up to 512 tokens 538 us, and 506)
#pragma unroll 1
      for (int r0 = 0; r0 < mine; r0 += OB) {
        uint32_t o1[OB], o2[OB], o3[OB];
        tmem_load<OB>(tO + lane_sel + g0 + r0, o1);
        tmem_load<OB>(tO + lane_sel + RT + g0 + r0, o2);
        tmem_load<OB>(tO + lane_sel + 2 * RT + g0 + r0, o3);
        tmem_ld_wait();
#pragma unroll
        for (int x0 = 0; x0 < OB; x0 += 4) {
          const float4 f4 = *reinterpret_cast<const float4*>(my_al + r0 + x0);
          const int4 a4 = *reinterpret_cast<const int4*>(my_at + r0 + x0);
          const float f[4] = {f4.x, f4.y, f4.z, f4.w};
          const int at[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int x = x0 + z;
            if (r0 + x < mine && has) {
              const float y = fmaf(fmaf(__uint_as_float(o3[x]), 0.0625f, __uint_as_float(o2[x])), 0.125f, __uint_as_float(o1[x]));
              const float val = f[z] == 0.f ? 0.f : y * f[z];  // (0 * NaN would not be 0)
              if (whole)
                static_cast<__nv_bfloat16*>(p.o)[(size_t)at[z] * D + e] = __float2bfloat16_rn(val);
              else
                p.part_o[(size_t)at[z] * D + e] = val;
            }
          }
        }
      }
      tc_fence_before();
      ok = exchange();  // the sums' places are free again
      if (!ok) break;
      ++piece;
    }
    tc_fence_before();
  }
  if (!ok) {  // let copies and products in flight land before the CTA's memory goes
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  __syncthreads();
  if (warp == SOFT + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// What the shares' borders cut, and requests without keys.  Block x looks at
// unit x, or, where units are more than shares, at the border behind share x
// and the unit that begins in that share and goes on behind it.  A unit that lies
// in the shares first .. last is merged, W warps to a row, each four shares at a
// time.  Where that is, is worked out from the lengths again, which needs
// nothing of the main kernel and so is done while that one ends.
//   Blocks for units always: 16384 requests up to 64 tokens, whose lengths every
// block of theirs adds up, 536 us, and 370 so.  Blocks for borders always: 8
// requests up to 1000 tokens 17.2 us, and 12.5.  One warp to a row always: a request of
// 131072 tokens 62 us, and 52.5.
template <int D, int W, bool BY_UNIT>
__global__ void __launch_bounds__(256) fa_decode_kv8_merge_kernel(const __grid_constant__ Kv8DecodeParams p, int RT,
                                                                  int shares) {
  constexpr int E = D / 32, ROWS = 8 / W;
  const int units = p.Hkv * p.row_tiles, lane = lane_id(), warp = threadIdx.x >> 5, row = warp / W, part = warp % W;
  __shared__ long long s_sum[16], s_at[3];
  __shared__ float s_m[8], s_w[8], s_o[W > 1 ? 8 : 1][D];
  long long each, more;
  auto share_of = [&](long long t) {
    return (int)(t < more * (each + 1) ? quick_div(t, each + 1) : more + quick_div(t - more * (each + 1), each));
  };
  int b, u, first = 0, last = -1;
  long long u0 = 0;
  if constexpr (BY_UNIT) {
    b = blockIdx.x / units;
    u = blockIdx.x - b * units;
    long long before = 0, total = 0;
    for (int x = threadIdx.x; x < p.B; x += 256) {
      const long long weight = kv8_weight(p, kv8_tiles(p, kv8_len(p, x))) * units;
      total += weight;
      if (x < b) before += weight;
    }
    const long long weight = kv8_weight(p, kv8_tiles(p, kv8_len(p, b)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      before += __shfl_xor_sync(0xffffffffu, before, o);
      total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane == 0) s_sum[warp] = before, s_sum[8 + warp] = total;
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int x = 0; x < 8; ++x) before += s_sum[x], total += s_sum[8 + x];
    each = quick_div(total, shares), more = total - each * shares;
    u0 = before + u * weight;
    if (weight > 0) first = share_of(u0 + p.lead), last = share_of(u0 + weight - 1);
  } else {
    const Scan scan = kv8_scan<8>(p, units, s_sum);
    each = quick_div(scan.total, shares), more = scan.total - each * shares;
    const long long border = share_begin(scan.total, shares, blockIdx.x + 1);
    kv8_find(p, units, scan, border, s_at);
    __syncthreads();
    b = u = 0;
    if (border < scan.total) {
      b = (int)s_at[0];
      const int weight = (int)(s_at[2] >> 32) + p.lead;
      u = (int)quick_div(s_at[1], weight);
      u0 = border - s_at[1] + (long long)u * weight;
      first = share_of(u0 + p.lead);
      if (first == (int)blockIdx.x) last = share_of(u0 + weight - 1);
    }
  }
  for (int x0 = blockIdx.x; x0 < p.B; x0 += gridDim.x) {  // requests without keys
    if (kv8_len(p, x0) > 0) continue;
    const int n = p.Nq * p.Hq;
    for (int x = blockIdx.y * 256 + threadIdx.x; x < n * (D / 8); x += gridDim.y * 256)
      static_cast<uint4*>(p.o)[(size_t)x0 * n * (D / 8) + x] = make_uint4(0u, 0u, 0u, 0u);
    for (int x = blockIdx.y * 256 + threadIdx.x; x < n; x += gridDim.y * 256) p.lse[(size_t)x0 * n + x] = -INFINITY;
  }
  const int rows = min(RT, p.Nq * p.group - row_tile(p, u) * RT);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the main kernel's grid is done
  if (last <= first) return;
  for (int r0 = blockIdx.y * ROWS; r0 < rows; r0 += gridDim.y * ROWS) {
    const int r = min(r0 + row, rows - 1);
    float acc[E], wsum = 0.f, m = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int k0 = first + part; k0 <= last; k0 += 4 * W) {
      float lc[4], v[4][E];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const bool on = k0 + W * y <= last;
        const int kk = on ? k0 + W * y : k0;
        // the share's last piece, if it begins before the unit, or its first
        const long long sl = (2 * (long long)kk + (each * kk + (kk < more ? kk : more) < u0 ? 1 : 0)) * RT + r;
        lc[y] = on ? p.part_lse[sl] : -INFINITY;
        const float* src = p.part_o + sl * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) v[y][e] = src[e];
      }
      const float mn = fmaxf(fmaxf(fmaxf(lc[0], lc[1]), fmaxf(lc[2], lc[3])), m), ref = mn == -INFINITY ? 0.f : mn;
      const float al = ex2_sfu(m - ref);
      m = mn;
      wsum *= al;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= al;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float wc = ex2_sfu(lc[y] - ref);
        wsum += wc;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wc, v[y][e], acc[e]);
      }
    }
    if constexpr (W > 1) {  // the warps' parts, against their largest
#pragma unroll
      for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
      if (lane == 0) s_m[warp] = m, s_w[warp] = wsum;
      __syncthreads();
      const int w0 = row * W;
#pragma unroll
      for (int y = 0; y < W; ++y) m = fmaxf(m, s_m[w0 + y]);
      const float ref = m == -INFINITY ? 0.f : m;
      wsum = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
      for (int y = 0; y < W; ++y) {
        const float f = ex2_sfu(s_m[w0 + y] - ref);
        wsum = fmaf(f, s_w[w0 + y], wsum);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(f, s_o[w0 + y][lane * E + e], acc[e]);
      }
      __syncthreads();
    }
    if (part == 0 && r0 + row < rows) {
      const int x = row_tile(p, u) * RT + r, i = p.Nq == 1 ? 0 : (int)((unsigned)x / (unsigned)p.group);
      const int h = kv_head(p, u) * p.group + x - i * p.group;
      const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
      const size_t out = ((size_t)b * p.Nq + i) * p.Hq + h;
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + out * D + lane * E);
#pragma unroll
      for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
      if (lane == 0)
        p.lse[((size_t)b * p.Hq + h) * p.Nq + i] = wsum == 0.f ? -INFINITY : (m + __log2f(wsum)) * 0.69314718055994531f;
    }
  }
}

// Query rows of one CTA.  A tile of fewer rows leaves room for a third CTA and
// has less to do at a unit's start and end: 4 rows take 20.6 us in a tile of 4,
// 22.9 in one of 8 and 27.6 in one of 16 (32 requests, a window of 4096, d = 64);
// 8 rows 37 and 56 in tiles of 8 and 16 (128 requests up to 2000, d = 64); 16 rows
// 53.9 and 57.0 in tiles of 16 and 32 (two drafts of eight heads); and 32 rows 60
// in one tile and 79 in two, which read the cache twice (four drafts).
int kv8_row_tile(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

// CTAs that run at once, the most shares dealt of the library's own choice, and the most tiles a call can have.
int kv8_most_shares(int Nq, int group) {
  int dev = 0, n_sm = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  return n_sm * kv8_ctas_per_sm(kv8_row_tile(Nq * group));
}
static long long kv8_most_tiles(int B, int Nq, int Hkv, int group, int span) {
  const int rows = Nq * group, rt = kv8_row_tile(rows);
  return (long long)B * Hkv * ((rows + rt - 1) / rt) * (((long long)span + kKv8Tile - 1) / kKv8Tile);
}

int kv8_auto_shares(int B, int Nq, int Hkv, int group, int span) {
  const long long tiles = kv8_most_tiles(B, Nq, Hkv, group, span);
  const int ctas = kv8_most_shares(Nq, group);
  return (int)(tiles < 1 ? 1 : tiles < ctas ? tiles : ctas);
}

template <int D, int RT>
static cudaError_t launch_main(const CUtensorMap& tk, const CUtensorMap& tv, Kv8DecodeParams& p, int shares, int span,
                               cudaStream_t stream) {
  auto kern = fa_decode_kv8_kernel<D, RT>;
  constexpr uint32_t smem = Layout<D, RT>::kBytes;
  static_assert((smem + 1024) * Layout<D, RT>::kCtas <= 228 * 1024, "CTAs per SM");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  p.row_tiles = (p.Nq * p.group + RT - 1) / RT;
  // Where a share is a tile or less, nothing is gained by making room for starts.
  p.lead = kv8_most_tiles(p.B, p.Nq, p.Hkv, p.group, span) > kv8_most_shares(p.Nq, p.group) ? kLead(RT) : 0;
  kern<<<shares, Layout<D, RT>::kThreads, smem, stream>>>(tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the merge's launch overlaps the main kernel (programmatic dependent launch); its blocks wait for the grid's end
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  // four warps to a row where units lie in four shares or more
  const long long units = (long long)p.B * p.Hkv * p.row_tiles;
  const bool by_unit = units <= shares, wide = 4 * units <= shares;
  cfg.gridDim = dim3((unsigned)(by_unit ? units : shares), wide ? RT / 2 : (RT + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &a;
  cfg.numAttrs = 1;
  auto merge = wide      ? fa_decode_kv8_merge_kernel<D, 4, true>
               : by_unit ? fa_decode_kv8_merge_kernel<D, 1, true>
                         : fa_decode_kv8_merge_kernel<D, 1, false>;
  return cudaLaunchKernelEx(&cfg, merge, static_cast<const Kv8DecodeParams&>(p), (int)RT, shares);
}

template <int D>
static cudaError_t launch_decode_kv8_t(const CUtensorMap& tk, const CUtensorMap& tv, Kv8DecodeParams& p, int shares, int span,
                                       cudaStream_t stream) {
  switch (kv8_row_tile(p.Nq * p.group)) {
    case 4: return launch_main<D, 4>(tk, tv, p, shares, span, stream);
    case 8: return launch_main<D, 8>(tk, tv, p, shares, span, stream);
    case 16: return launch_main<D, 16>(tk, tv, p, shares, span, stream);
    default: return launch_main<D, 32>(tk, tv, p, shares, span, stream);
  }
}

cudaError_t launch_decode_kv8(const CUtensorMap& tk, const CUtensorMap& tv, Kv8DecodeParams& p, int D, int shares, int span,
                              cudaStream_t stream) {
  if (D == 64) return launch_decode_kv8_t<64>(tk, tv, p, shares, span, stream);
  if (D == 128) return launch_decode_kv8_t<128>(tk, tv, p, shares, span, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fa
