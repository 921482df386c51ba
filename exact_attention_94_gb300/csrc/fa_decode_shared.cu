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
//    own (query tokens, keys, table row), and where each CTA's share of the work
//    begins.  The work is one list of tiles of 128 keys, of all (entry, K/V head,
//    256 rows) units, dealt in equal shares; a unit counts `lead` tiles more, for
//    its start and end.
//  - the main kernel, one CTA per SM.  Rows take the M side of both tcgen05
//    products: S [128 x 128 keys] = Q K^T, O [128 x d] += P V with P in TMEM over
//    S, two tiles in turn, so one's products run while the other's softmax does.
//    Units of more than 128 rows are two tiles of rows that meet the same keys;
//    units of up to 128 are one tile of rows, whose key tiles the two take in
//    turn, and both results are merged at the end.
//  - the merge, a warp per query row: results of whole units (at their rows) or of
//    the pieces that shares' borders cut.
//
// Rows of a tile are query tokens times the query heads of one K/V head, as they
// lie in Q: a TMA box of [tokens][heads][64 elements].
//
// Main kernel's warps: 2 walks over the shares and announces their pieces; 0 loads
// K and 3 loads Q and V (K and V into one ring, across units); 1 issues the products;
// 4-7 and 8-11 are the softmax of the two tiles, a thread per row.
//
// A TMA box is a page's keys (128 at most) of one head, all d of them: a tile of K or
// V lies in shared memory as [8 keys][64 elements of d][8 x 128 bytes], so that one
// box fills whole eights of keys.
#include "sampling.cuh"

#include <cmath>

namespace fa {

namespace {

constexpr int kPlanThreads = 1024;
// What units weigh.  Of many rows, in half microseconds about: of one and of two tiles of
// rows, and each of their tiles of keys.  Of few rows: their start and end, in 16 keys.
constexpr int kLeadOne = 5, kTileOne = 2, kLeadTwo = 12, kTileTwo = 3, kLeadFew = 6;
constexpr float kFew = 0.17f;                  // of a CTA's half microseconds 16 keys of few rows take, d = 128
constexpr int kWarps = 8;                      // of a CTA, that attend for few rows
constexpr int kFewEarly = 8, kFewLate = 16;    // shares of few rows for each CTA at most, that warps begin with and that they take
constexpr int kFewLateOf = 2;                  // one in so many of few rows' weight is dealt late,
constexpr int kFewLateFrom = 64;               //   where a warp's share is this much at least
constexpr int kFewLeast = 8, kFewLateLeast = 24;  // weight of those shares at least
constexpr int kPlanSmem = 1024;                // groups, entries in the plan's shared memory
constexpr int kMergeRows = 8;                  // of a warp of the merge
constexpr int kPieces = 6;                     // announced ahead

template <int D>
struct SharedLayout {
  static constexpr uint32_t kTile = 128u * D * 2u;  // a tile of Q, K or V
  static constexpr uint32_t kChunk = 128u * 128u;   // of Q: 128 rows x 128 bytes (one 128-byte swizzle column)
  static constexpr int kStages = D == 64 ? 10 : 5;  // K/V ring slots
  static constexpr uint32_t kQOff = 0;              // two tiles of Q
  static constexpr uint32_t kKVOff = 2 * kTile;
  static constexpr uint32_t kMiscOff = kKVOff + kStages * kTile;
  static constexpr uint32_t kMisc = D == 64 ? 3072 : 2048;   // barriers, pieces
  static constexpr uint32_t kBytes = kMiscOff + kMisc + 1024;  // alignment slack
  // Warps that attend for few rows, once the tiles are done with: of each a ring of 16 keys
  // and values, and queries.
  static constexpr uint32_t kWarpBytes = kMiscOff / kWarps / 1024 * 1024;
  static constexpr uint32_t kFewTile = 16u * D * 2u;
};
static_assert(SharedLayout<128>::kBytes <= 227 * 1024 && SharedLayout<64>::kBytes <= 227 * 1024, "shared memory");
constexpr int kThreads = 384;

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

// a / b for a >= 0, b > 0, in 32 bits where both fit
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  return (((unsigned long long)a | (unsigned long long)b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
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

// ---------------------------------------------------------------- plan

__global__ void __launch_bounds__(kPlanThreads, 1) fa_shared_plan_kernel(const __grid_constant__ SharedParams p) {
  __shared__ long long s_w[2][32];
  __shared__ int s_n[2][32];
  __shared__ int s_starts[kPlanSmem + 1], s_shared[kPlanSmem], s_least[kPlanSmem];
  __shared__ int s_of[kPlanSmem];
  __shared__ unsigned long long s_most[kPlanSmem];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const SharedPlan& pl = p.plan;
  asm volatile("griddepcontrol.launch_dependents;");
  const bool small = p.G <= kPlanSmem;  // groups' numbers in shared memory
  const int* starts = small ? s_starts : p.starts;
  int *least = small ? s_least : pl.g_least, *shared = small ? s_shared : pl.g_shared;
  unsigned long long* most = small ? s_most : pl.g_most;  // longest length, and the first request that has it
  int* of_group = small ? s_of : pl.g_of;                 // its entry of shared keys
  const int len0 = tid < p.B ? p.seq_lens[tid] : 0;       // (asked for early; of the thread's first entry too)
  const int len1 = tid >= p.G && tid - p.G < p.B ? p.seq_lens[tid - p.G] : 0;
  // groups that do not cut the batch into runs are reported, and nothing counts as shared
  bool bad = false;
  for (int g = tid; g <= p.G; g += kPlanThreads) {
    const int s = p.starts[g], s0 = g > 0 ? p.starts[g - 1] : 0;
    bad |= g == 0 ? s != 0 : s < s0;
    bad |= g == p.G && s != p.B;
    if (small) s_starts[g] = s;
    if (g < p.G) {
      int n = p.shared_lens[g];
      if (n < 0 || n > p.max_len) {
        atomicCAS(p.err, 0u, FA_DEVERR_BAD_SEQLEN);
        n = 0;
      }
      shared[g] = n, least[g] = 0x7fffffff, most[g] = 0;
    }
  }
  const bool grouped = __syncthreads_or(bad) == 0;
  if (!grouped && tid == 0) atomicCAS(p.err, 0u, FA_DEVERR_BAD_SEQLEN);
  auto group_of = [&](int b) {  // the group that begins last at or before b, and has requests
    int g = 0, z = p.G;
    while (z - g > 1) {
      const int m = (g + z) / 2;
      if (starts[m] <= b) g = m; else z = m;
    }
    return g;
  };
  // each group's longest request and shortest with keys
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int g = -1, len = 0;
    if (b < p.B) {
      len = b0 == 0 ? len0 : p.seq_lens[b];
      if (len < 0 || len > p.max_len) {
        atomicCAS(p.err, 0u, FA_DEVERR_BAD_SEQLEN);
        len = len < 0 ? 0 : p.max_len;
      }
      if (grouped) g = group_of(b);
    }
    const unsigned long long key = (unsigned long long)(unsigned)len << 32 | (unsigned)(0x7fffffff - b);
    int same;
    __match_all_sync(0xffffffffu, g, &same);
    if (same) {  // one group's: the warp's together
      const unsigned top = __reduce_max_sync(0xffffffffu, (unsigned)len);
      const unsigned who = __ballot_sync(0xffffffffu, (unsigned)len == top);
      const int low = __reduce_min_sync(0xffffffffu, len > 0 ? len : 0x7fffffff);
      if (g >= 0 && lane == __ffs(who) - 1) {
        atomicMax(&most[g], key);
        atomicMin(&least[g], low);
      }
    } else if (g >= 0) {
      atomicMax(&most[g], key);
      if (len > 0) atomicMin(&least[g], len);
    }
  }
  __syncthreads();
  // keys that group g shares, as used: none for a request alone, whose keys are all its own
  auto shares_of = [&](int g) {
    const int n = starts[g + 1] - starts[g] < 2 ? 0 : shared[g];
    return min(n, (int)(most[g] >> 32));
  };
  // Entries: groups' shared keys, then requests' own, a block's threads at a time.  Those that
  // have keys get the next places of their list.
  long long total[2] = {0, 0};
  int count[2] = {0, 0};
  for (int i0 = 0; i0 < p.G + p.B; i0 += kPlanThreads) {
    const int g = i0 + tid, b = g - p.G;
    SharedEntry e{};
    int n = 0, of = -1;  // n: keys that the group shares; of: a request's group
    if (b < 0) {
      n = grouped ? shares_of(g) : 0;
      if (n > 0) {
        const int b0 = starts[g], top = (int)(most[g] >> 32), low = least[g];
        e = {b0 * p.Nq, (starts[g + 1] - b0) * p.Nq, 0x7fffffff - (int)(unsigned)most[g], 0, n, 0, 0, 0, 0};
        if (p.win_left >= 0) {
          e.lo = max(0, low - p.Nq - p.win_left);
          e.all_lo = top - 1 - p.win_left;
        }
        e.all_lo = max(e.all_lo, e.lo);
        e.all_hi = min(n, low - p.Nq + 1);
      }
    } else if (b < p.B) {
      const int len = min(max(i0 == 0 ? len1 : p.seq_lens[b], 0), p.max_len);
      if (grouped) of = group_of(b);
      e = {b * p.Nq, p.Nq, b, of >= 0 ? min(shares_of(of), len) : 0, len, 0, 0, 0, 1};
      if (p.win_left >= 0) {
        e.lo = max(e.lo, len - p.Nq - p.win_left);
        e.all_lo = len - 1 - p.win_left;
      }
      e.all_lo = max(e.all_lo, e.lo);
      e.all_hi = len - p.Nq + 1;
      if (len == 0) of = -1;  // (all_lo, all_hi of the shared keys leave it out)
    }
    const bool few = (long long)e.ntok * p.heads <= p.few;
    if (e.lo < e.end) e.tiles = few ? (e.end - e.lo / 16 * 16 + 15) / 16 : (e.end - e.lo / p.box_rows * p.box_rows + kSharedTile - 1) / kSharedTile;
    const Weight u = weight_of(p, few, e.ntok);
    const long long w = e.tiles > 0 ? (u.lead + (long long)u.tile * e.tiles) * p.Hkv * chunks_of(p, few, e.ntok) : 0;
    int at = -1;
    long long sum[2];
    unsigned votes[2];
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      sum[l] = few == (l == 1) ? w : 0;
      votes[l] = __ballot_sync(0xffffffffu, sum[l] > 0);
      if (votes[l] != 0) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, sum[l], o);
          if (lane >= o) sum[l] += x;
        }
      }
      if (lane == 31) s_w[l][warp] = sum[l], s_n[l][warp] = __popc(votes[l]);
    }
    __syncthreads();
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      long long ws = s_w[l][lane], before = total[l];
      int ns = s_n[l][lane], place = count[l];
      if (__any_sync(0xffffffffu, ns > 0)) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, ws, o);
          const int y = __shfl_up_sync(0xffffffffu, ns, o);
          if (lane >= o) ws += x, ns += y;
        }
        const long long ahead_w = __shfl_sync(0xffffffffu, ws, (warp + 31) & 31);
        const int ahead_n = __shfl_sync(0xffffffffu, ns, (warp + 31) & 31);
        if (warp > 0) before += ahead_w, place += ahead_n;
        total[l] += __shfl_sync(0xffffffffu, ws, 31);
        count[l] += __shfl_sync(0xffffffffu, ns, 31);
      }
      if (w > 0 && few == (l == 1)) {
        place += __popc(votes[l] & ((1u << lane) - 1u));
        pl.list[l].entry[place] = e;
        pl.list[l].cum[place] = before + sum[l] - w;
        at = 2 * place + l;
      }
    }
    if (b < 0) of_group[g] = at;
    __syncthreads();  // (groups come before requests, and every warp has read the sums)
    if (b >= 0 && b < p.B) pl.of_request[b] = make_int2(of >= 0 ? of_group[of] : -1, at);
  }
  // Shares.  Of many rows one for each of so many CTAs as their part of all work is, no
  // shorter than a tile (or a unit's piece could be empty).  Of few rows one for each warp of
  // the others, and the rest in smaller ones, which warps take as they come to an end.
  SharedHead head{};
  auto shares_in = [&](long long most, long long weight, int least) { return (int)min(most, weight / least); };
  const float few_time = (float)total[1] * p.few_cost;
  const float part = (float)total[0] / fmaxf((float)total[0] + few_time, 1.f);
  head.total[0] = total[0];
  head.shares[0] = shares_in(min((long long)p.shares, (long long)(part * (float)p.shares + 1.f)), total[0], kTileTwo);
  if (total[1] > 0) {
    const int others = p.shares - head.shares[0];
    const bool late = total[1] >= (long long)kFewLateFrom * kWarps * others;
    head.total[2] = late ? total[1] / (others > 0 ? kFewLateOf : 1) : 0;
    head.shares[2] = shares_in((long long)kFewLate * p.shares, head.total[2], kFewLateLeast);
    if (late && head.shares[2] == 0) head.shares[2] = 1;
    head.total[1] = total[1] - head.total[2];
    head.shares[1] = head.total[1] > 0 ? max(shares_in((long long)kWarps * others, head.total[1], kFewLeast), 1) : 0;
  }
  head.count[0] = count[0], head.count[1] = count[1];
  head.queue = head.shares[1];
  if (tid == 0) *pl.head = head;
}

// ---------------------------------------------------------------- main

#include "decode_few.cuh"

template <int D, int NR>
__global__ void __launch_bounds__(kThreads, 1)
    fa_decode_shared_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k16,
                            const __grid_constant__ CUtensorMap tm_v16, const __grid_constant__ SharedParams p) {
  using L = SharedLayout<D>;
  constexpr int NS = L::kStages, CH = D / 64;
  constexpr uint32_t TILE = L::kTile, CHUNK = L::kChunk;
  const int warp = warp_id(), lane = lane_id();

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sb = smem_raw + (base - raw);
  const uint32_t q_s = base + L::kQOff, kv_s = base + L::kKVOff;

  // Rings: K/V tiles, pieces.  Q[s]: a tile of Q has landed; its last S product is
  // done.  Per tile t in turn: S ready, P's first and second 64 keys ready, the last
  // product of a run of key tiles done (O), and O read.  X: the softmax warps of a
  // tile, and of both, have come this far.  FEW: of each warp that attends for few rows,
  // 16 keys and values have landed.
  enum { KV_FULL = 0, KV_EMPTY = NS, PC_FULL = 2 * NS, PC_EMPTY = PC_FULL + kPieces, Q_FULL = PC_EMPTY + kPieces,
         Q_EMPTY = Q_FULL + 2, S_FULL = Q_EMPTY + 2, P_FULL = S_FULL + 2, O_FINAL = P_FULL + 4, O_EMPTY = O_FINAL + 2,
         XB = O_EMPTY + 2, DRAIN = XB + 3, FEW = DRAIN + 1, NBARS = FEW + kWarps * kFewStages };
  const uint32_t bar0 = base + L::kMiscOff;
  auto BAR = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  constexpr uint32_t SLOT = L::kMiscOff + 8 * NBARS, PIECES = SLOT + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sb + SLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Piece* s_piece = reinterpret_cast<Piece*>(sb + PIECES);                              // [kPieces]
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(sb + PIECES + 64 * kPieces);           // [2 groups][2][4]
  FewPiece* s_few = reinterpret_cast<FewPiece*>(sb + PIECES);                          // [kWarps][kFewPieces], once those are done with
  static_assert(sizeof(Piece) == 64 && PIECES % 8 == 0, "pieces");
  static_assert(PIECES + 64 * kPieces + 64 <= L::kMiscOff + L::kMisc, "misc area");
  static_assert(PIECES + kWarps * kFewPieces * sizeof(FewPiece) <= L::kMiscOff + L::kMisc, "misc area");

  if (threadIdx.x == 0) {
    for (int i = 0; i < NBARS; ++i) {
      int n = 1;
      if (i >= PC_EMPTY && i < PC_EMPTY + kPieces) n = 11;  // who loads, who multiplies, eight warps of softmax
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
  asm volatile("griddepcontrol.launch_dependents;");  // the merge may be set up from the plan; it waits for this grid's end

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
  // (registers go where a row's 128 scores are held: 56 x 4 warps + 224 x 8 is what 168 x 12 was)
  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
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
      const int at8 = now.page * (p.page_size / 8) + now.rows8;
      for (int i = 0; i < now.n; ++i) {
        const int slot = place % NS, here = min(boxes, (max(now.last - 8 * i, 0) + (1 << shift) - 1) >> shift);
        if (place >= NS) ok = __all_sync(0xffffffffu, mbar_wait(BAR(KV_EMPTY + slot), (place / NS - 1) & 1, w, 74));
        if (!ok) break;
        if (elect_one()) mbar_arrive_expect_tx(BAR(KV_FULL + slot), (uint32_t)(here * p.box_rows * D * 2));
        __syncwarp();
        const uint32_t dst = kv_s + slot * TILE, bar = BAR(KV_FULL + slot);
        for (int x = 0; x < here; ++x) {  // (one lane issues, with the same operands in all)
          const int row8 = __shfl_sync(0xffffffffu, at8, 8 * i + (x << shift));
          if (elect_one()) tma_load_5d(dst + x * p.box_rows * D * 2, map, bar, 0, 0, 0, row8, now.head);
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
    constexpr uint32_t IDESC_S = idesc_bf16(128, 128, false, false), IDESC_O = idesc_bf16(128, D, false, true);
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
          if (x == 0 && here) here = there(BAR(Q_FULL) + 8 * qs, q >> 1 & 1);
          if (!here) {
            // inputs that have not come yet: the last job's product need not wait for them
            if (before.on && !(ok = product(before, t ^ 1))) break;
            before.on = false;
            ok = wait(BAR(KV_FULL) + 8 * sk, pk, 81);
            if (ok && x == 0) ok = wait(BAR(Q_FULL) + 8 * qs, q >> 1 & 1, 80);
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
  if (few && many) __syncthreads();  // shared memory changes hands
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    if (many) {
    // ============================================================ softmax
    const int t = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + (t ? 128u : 0u), tO = tmem + lane_off + 256u + (t ? (uint32_t)D : 0u);
    const float sl2 = p.scale_log2;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
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
          bool odd = false;
          if (max(j0, s.lo) < s.all_lo || min(j0 + kSharedTile, s.end) > s.all_hi) {
            if (!out && (key < s.all_lo || key >= s.all_hi)) {
              uint32_t bad = 0;
#pragma unroll 1
              for (int i = 0; i < 8 * CH; ++i) {
                const uint4 v = row[(i >> 3) * 64 + (i + lane & 7)];  // (other banks for each lane)
                bad |= __vcmpeq2(v.x & 0x7f807f80u, 0x7f807f80u) | __vcmpeq2(v.y & 0x7f807f80u, 0x7f807f80u) |
                       __vcmpeq2(v.z & 0x7f807f80u, 0x7f807f80u) | __vcmpeq2(v.w & 0x7f807f80u, 0x7f807f80u);
              }
              odd = bad != 0;
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
          float mq[4];                   // each load's maximum over its 32 columns
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_max(tS + 32 * c, sr[c], mq[c]);
          tmem_ld_wait();
          if (!inside) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int a = min(max(key_lo - j0 - 32 * c, 0), 32), z = min(max(key_hi - j0 - 32 * c, 0), 32);
              const uint32_t sees = z > a ? (0xffffffffu >> (32 - (z - a))) << a : 0u;
              if (__any_sync(0xffffffffu, ~sees)) {
                float m = -INFINITY;
                none |= __any_sync(0xffffffffu, sees) ? 0u : 1u << c;
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  if (!(sees >> i & 1)) sr[c][i] = 0xff800000u;
                  if (!(sees >> (i + 1) & 1)) sr[c][i + 1] = 0xff800000u;
                  m = max3f(m, __uint_as_float(sr[c][i]), __uint_as_float(sr[c][i + 1]));
                }
                mq[c] = m;
              }
            }
          }
          const float m_new = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * sl2;
          float alpha = 1.f;
          const bool moves = m_new > m_ref + p.tau;
          if (moves) {
            alpha = ex2_sfu(m_ref - m_new);
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
                float y0, y1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c][2 * i]), __uint_as_float(sr[c][2 * i + 1])), sl2x2, nmb2), y0, y1);
                const float p0 = ex2_sfu(y0), p1 = ex2_sfu(y1);
                acc[i & 1] = f2_add(acc[i & 1], f2_pack(p0, p1));
                pk[16 * (c & 1) + i] = pack_bf16x2(p0, p1);
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
          l = fmaf(l, alpha, s0 + s1);
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
    if constexpr (NR > 0) {
      if (few && many) {
        fence_proxy_async_smem();
        __syncthreads();
      }
      const int x = warp - 4, others = (int)gridDim.x - n_many;
      if (few) attend_few<D, NR>(p, tm_k16, tm_v16, w, many ? -1 : x * others + (int)blockIdx.x - n_many, base + x * L::kWarpBytes,
                        sb + x * L::kWarpBytes, BAR(FEW + x * kFewStages), s_few + x * kFewPieces);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- merge

// A warp for R query rows of a token and K/V head, one where all are on the GPU at once: the
// results of the group's shared keys and of the request's own.  Lane i looks at part i; a
// part without mass has lse = -inf, and its O is not read.
template <int D, int R>
__global__ void __launch_bounds__(256, R == 1 ? 4 : 2) fa_decode_shared_merge_kernel(const __grid_constant__ SharedParams p) {
  constexpr int E = D / 32, U = R == 1 ? 8 : 1;  // U: parts read at a time
  const int lane = threadIdx.x & 31, fours = (p.heads + R - 1) / R;
  const long long rows = (long long)p.B * p.Nq * p.Hq, x = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (x >= (long long)p.B * p.Nq * p.Hkv * fours) return;
  const long long of_four = div_ll(x, fours);
  const int h0 = (int)(x - of_four * fours) * R, tok = (int)div_ll(of_four, p.Hkv), head = (int)(of_four - (long long)tok * p.Hkv);
  const int b = tok / p.Nq, nr = min(R, p.heads - h0);
  const long long row = (long long)tok * p.Hq + head * p.heads + h0;
  // (the plan, which the main kernel's CTAs have all waited for; read past L1)
  const int2 entries = __ldcg(p.plan.of_request + b);
  // parts of each kind: n of them, `runs` in each of the shares from `first` on
  int n[2] = {0, 0}, runs[2] = {1, 1}, first[2] = {0, 0};
  long long base[2] = {0, 0}, begin[2] = {0, 0};  // place of the first part, or of the row in a slot; the unit's begin
  bool cut[2] = {false, false}, few[2] = {false, false};
  SharedHead totals;
  const longlong2 t0 = __ldcg(reinterpret_cast<const longlong2*>(p.plan.head)),
                  t1 = __ldcg(reinterpret_cast<const longlong2*>(p.plan.head) + 1);
  totals.total[0] = t0.x, totals.total[1] = t0.y, totals.total[2] = t1.x;
  totals.shares[0] = (int)t1.y, totals.shares[1] = (int)(t1.y >> 32), totals.shares[2] = __ldcg(&p.plan.head->shares[2]);
  const Deal deals[2] = {deal_of(totals, false), deal_of(totals, true)};
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const int of = kind == 0 ? entries.x : entries.y;
    if (of < 0) continue;
    few[kind] = of & 1;
    const SharedList& list = p.plan.list[of & 1];
    const Deal& deal = (of & 1) ? deals[1] : deals[0];
    const SharedEntry* at = list.entry + (of >> 1);
    const int tok0 = __ldcg(&at->tok0), ntok = __ldcg(&at->ntok), tiles = __ldcg(&at->tiles);
    const long long cum = __ldcg(list.cum + (of >> 1));
    const Weight wt = weight_of(p, few[kind], ntok);
    const int weight = wt.lead + wt.tile * tiles, chunks = chunks_of(p, few[kind], ntok);
    const int c = few[kind] ? 0 : (tok - tok0) / (2 * p.tile_tokens), in = tok - tok0 - c * 2 * p.tile_tokens;
    const bool pair = few[kind] || ntok - c * 2 * p.tile_tokens > p.tile_tokens;
    begin[kind] = cum + (long long)weight * ((long long)head * chunks + c);
    first[kind] = deal.of(begin[kind] + wt.lead);
    const int last = deal.of(begin[kind] + weight - wt.tile);  // where the last tile begins
    cut[kind] = first[kind] != last;
    runs[kind] = pair ? 1 : 2;
    n[kind] = (last - first[kind] + 1) * runs[kind];
    const int side = few[kind] ? 0 : in / p.tile_tokens;
    base[kind] = cut[kind] ? side * kSharedTile + (in - side * p.tile_tokens) * p.heads + h0 : 2 * kind * rows + row;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the main kernel's grid is done
  float acc[R][E], mass[R], m[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    mass[r] = 0.f, m[r] = -INFINITY;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[r][i] = 0.f;
  }
  for (int i0 = 0; i0 < n[0] + n[1]; i0 += 32) {
    float lc[R], f[R];
    long long place = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) lc[r] = -INFINITY;
    if (i0 + lane < n[0] + n[1]) {
      const bool own_part = i0 + lane >= n[0];
      const int i = i0 + lane - (own_part ? n[0] : 0);
      const bool two = (own_part ? runs[1] : runs[0]) == 2;
      const int run = two ? i & 1 : 0, k = (own_part ? first[1] : first[0]) + (two ? i >> 1 : i);
      // a cut unit's: of the share's last piece, if it begins before the unit, or its first
      const bool in_few = own_part ? few[1] : few[0], later = (in_few ? deals[1] : deals[0]).begin(k) < (own_part ? begin[1] : begin[0]);
      place = own_part ? base[1] : base[0];
      place += (own_part ? cut[1] : cut[0]) ? cut_place(p, in_few, k, later) + run * kSharedTile : run * rows;
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < nr) lc[r] = p.part_lse[place + r];
    }
    unsigned todo = 0, has[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = lc[r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));  // (a NaN is left out)
      const float mn = fmaxf(m[r], top), ref = mn == -INFINITY ? 0.f : mn, al = ex2_sfu(m[r] - ref);
      m[r] = mn;
      mass[r] *= al;
#pragma unroll
      for (int i = 0; i < E; ++i) acc[r][i] *= al;
      f[r] = ex2_sfu(lc[r] - ref);
      has[r] = __ballot_sync(0xffffffffu, lc[r] != -INFINITY);
      todo |= has[r];
    }
    while (todo) {
      float v[U][R][E], fu[U][R];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int from = todo ? __ffs(todo) - 1 : 0;
        const long long at = __shfl_sync(0xffffffffu, place, from);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float weight = __shfl_sync(0xffffffffu, f[r], from);
          const bool on = todo != 0 && (has[r] >> from & 1);
          fu[u][r] = on ? weight : 0.f;
          const float* src = p.part_o + (at + r) * D + lane * E;
#pragma unroll
          for (int i = 0; i < E; ++i) v[u][r][i] = 0.f;
          if (on) {
            if constexpr (E == 4) {
              const float4 y = *reinterpret_cast<const float4*>(src);
              v[u][r][0] = y.x, v[u][r][1] = y.y, v[u][r][2] = y.z, v[u][r][3] = y.w;
            } else {
              const float2 y = *reinterpret_cast<const float2*>(src);
              v[u][r][0] = y.x, v[u][r][1] = y.y;
            }
          }
        }
        todo &= todo - 1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          mass[r] += fu[u][r];
#pragma unroll
          for (int i = 0; i < E; ++i) acc[r][i] = fmaf(fu[u][r], v[u][r][i], acc[r][i]);
        }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= nr) break;
    const float inv = mass[r] == 0.f ? 0.f : 1.f / mass[r];
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + (row + r) * D + lane * E);
#pragma unroll
    for (int i = 0; i < E; i += 2) dst[i / 2] = pack_bf16x2(acc[r][i] * inv, acc[r][i + 1] * inv);
    if (lane == 0)
      p.lse[((long long)b * p.Hq + head * p.heads + h0 + r) * p.Nq + tok - b * p.Nq] =
          mass[r] == 0.f ? -INFINITY : (m[r] + __log2f(mass[r])) * 0.69314718055994531f;
  }
}

// ---------------------------------------------------------------- host

static size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// The plan's arrays one after the other from `at` (or their bytes alone).
static size_t plan_layout(SharedPlan* plan, void* at, int B, int G) {
  uint8_t* base = static_cast<uint8_t*>(at);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* here = base + off;
    off += up16(bytes);
    return here;
  };
  SharedPlan pl;
  pl.head = reinterpret_cast<SharedHead*>(take(sizeof(SharedHead)));
  for (SharedList& l : pl.list) {
    l.entry = reinterpret_cast<SharedEntry*>(take(sizeof(SharedEntry) * ((size_t)G + B)));
    l.cum = reinterpret_cast<long long*>(take(8 * ((size_t)G + B)));
  }
  pl.of_request = reinterpret_cast<int2*>(take(8 * (size_t)B));
  pl.g_shared = reinterpret_cast<int*>(take(4 * (size_t)G));
  pl.g_of = reinterpret_cast<int*>(take(4 * (size_t)G));
  pl.g_least = reinterpret_cast<int*>(take(4 * (size_t)G));
  pl.g_most = reinterpret_cast<unsigned long long*>(take(8 * (size_t)G));
  if (plan != nullptr) *plan = pl;
  return off;
}
int shared_few(int Nq, int heads) {
  const int rows = Nq * heads;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 0;
}
size_t shared_part_rows(int B, int Nq, int Hq, int heads, int shares) {
  return 4 * (size_t)B * Nq * Hq + 512 * (size_t)shares + 2 * (size_t)shared_few(Nq, heads) * (kFewEarly + kFewLate) * shares;
}
size_t shared_plan_bytes(int B, int G) { return plan_layout(nullptr, nullptr, B, G); }
void shared_plan_at(SharedPlan& plan, void* at, int B, int G) { plan_layout(&plan, at, B, G); }

template <int D, int NR>
static cudaError_t launch_t(const CUtensorMap (&maps)[5], const SharedParams& p, cudaStream_t stream) {
  auto kern = fa_decode_shared_kernel<D, NR>;
  constexpr uint32_t smem = SharedLayout<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  fa_shared_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.shares);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &a;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], maps[3], maps[4], p)) != cudaSuccess) return e;
  const long long tokens = (long long)p.B * p.Nq * p.Hkv;
  const bool one = tokens * p.heads <= 32ll * kSms;
  const long long warps = tokens * (one ? p.heads : (p.heads + kMergeRows - 1) / kMergeRows);
  cfg.gridDim = dim3((unsigned)((warps + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return one ? cudaLaunchKernelEx(&cfg, fa_decode_shared_merge_kernel<D, 1>, p)
             : cudaLaunchKernelEx(&cfg, fa_decode_shared_merge_kernel<D, kMergeRows>, p);
}

template <int D>
static cudaError_t launch_d(const CUtensorMap (&maps)[5], SharedParams p, cudaStream_t stream) {
  p.few_cost = kFew * D / 128;
  switch (p.few) {
    case 8: return launch_t<D, 1>(maps, p, stream);
    case 16: return launch_t<D, 2>(maps, p, stream);
    case 32: return launch_t<D, 4>(maps, p, stream);
    default: return launch_t<D, 0>(maps, p, stream);
  }
}

cudaError_t launch_decode_shared(const CUtensorMap (&maps)[5], const SharedParams& p, int D, cudaStream_t stream) {
  if (D == 64) return launch_d<64>(maps, p, stream);
  if (D == 128) return launch_d<128>(maps, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fa
