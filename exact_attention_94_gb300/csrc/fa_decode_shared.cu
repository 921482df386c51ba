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
// Main kernel's warps: 0 loads (Q, and a TMA box per page into a ring of K and V
// tiles, across units), 1 issues the products, 4-7 and 8-11 are the softmax of
// the two tiles, a thread per row.
#include "sampling.cuh"

#include <cmath>

namespace fa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPieces = 4;  // announced ahead

template <int D>
struct SharedLayout {
  static constexpr uint32_t kTile = 128u * D * 2u;  // a tile of Q, K or V
  static constexpr uint32_t kChunk = 128u * 128u;   // 128 rows x 128 bytes (one 128-byte swizzle column)
  static constexpr int kStages = D == 64 ? 8 : 4;   // K/V ring slots
  static constexpr uint32_t kQOff = 0;              // two tiles of Q
  static constexpr uint32_t kKVOff = 2 * kTile;
  static constexpr uint32_t kMiscOff = kKVOff + kStages * kTile;
  static constexpr uint32_t kBytes = kMiscOff + 1024 + 1024;  // pieces, barriers; alignment slack
};
constexpr int kThreads = 384;

// Tiles t0 .. t1 - 1 of a unit, as the producer announces them; t0 = t1 marks the share's end.
struct Piece {
  int tok0, ntok;      // query tokens of the unit
  int head;            // K/V head
  int lo, end, all_lo, all_hi, beg;
  int t0, t1;
  int whole;           // the unit's only piece
  int kind;            // 0: shared keys, 1: a request's own
  int slot;            // where a cut piece's results go
  int pad[3];
};

__device__ __forceinline__ int shared_len(const SharedParams& p, int b) {
  int n = p.seq_lens[b];
  if (n < 0 || n > p.max_len) {
    atomicCAS(p.err, 0u, FA_DEVERR_BAD_SEQLEN);
    n = n < 0 ? 0 : p.max_len;
  }
  return n;
}

__device__ __forceinline__ int chunks_of(const SharedParams& p, int ntok) {  // of 256 rows
  return (ntok + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
}
__device__ __forceinline__ long long units_of(const SharedParams& p, int ntok) {
  return (long long)p.Hkv * chunks_of(p, ntok);
}

// a / b for a >= 0, b > 0, in 32 bits where both fit
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  return (((unsigned long long)a | (unsigned long long)b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}
__device__ __forceinline__ long long share_begin(long long total, int shares, long long k) {
  const long long each = div_ll(total, shares), more = total - each * shares;  // the first `more` shares have one more
  return each * k + (k < more ? k : more);
}

}  // namespace

// ---------------------------------------------------------------- plan

__global__ void __launch_bounds__(kPlanThreads) fa_shared_plan_kernel(const __grid_constant__ SharedParams p) {
  __shared__ long long s_w[32];
  __shared__ int s_n[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const SharedPlan& pl = p.plan;
  asm volatile("griddepcontrol.launch_dependents;");
  // groups that do not cut the batch into runs are reported, and nothing counts as shared
  bool bad = false;
  for (int g = tid; g <= p.G; g += kPlanThreads) {
    const int s = p.starts[g];
    bad |= g == 0 ? s != 0 : s < p.starts[g - 1];
    bad |= g == p.G && s != p.B;
  }
  const bool grouped = __syncthreads_or(bad) == 0;
  if (!grouped && tid == 0) atomicCAS(p.err, 0u, FA_DEVERR_BAD_SEQLEN);
  // a group's shared keys: a warp each
  for (int g = warp; g < p.G; g += 32) {
    const int b0 = grouped ? p.starts[g] : 0, b1 = grouped ? p.starts[g + 1] : 0;
    int most = 0, least = 0x7fffffff, at = b1;
    for (int b = b0 + lane; b < b1; b += 32) {
      const int n = shared_len(p, b);
      pl.group[b] = g;
      if (n > most) most = n, at = b;
      if (n > 0) least = min(least, n);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const int m2 = __shfl_xor_sync(0xffffffffu, most, o), a2 = __shfl_xor_sync(0xffffffffu, at, o);
      if (m2 > most || (m2 == most && a2 < at)) most = m2, at = a2;
      least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    }
    if (lane == 0) {
      int n = p.shared_lens[g];
      if (n < 0 || n > p.max_len) {
        atomicCAS(p.err, 0u, FA_DEVERR_BAD_SEQLEN);
        n = 0;
      }
      if (b1 - b0 < 2) n = 0;  // a request alone: all its keys are its own
      n = min(n, most);
      pl.g_shared[g] = n;
      SharedEntry e{b0 * p.Nq, (b1 - b0) * p.Nq, at, 0, n, 0, 0, 0, 0};
      if (n > 0) {
        if (p.win_left >= 0) {
          e.lo = max(0, least - p.Nq - p.win_left);
          e.all_lo = max(0, most - 1 - p.win_left);
        }
        e.all_lo = max(e.all_lo, e.lo);
        e.all_hi = min(n, least - p.Nq + 1);
        if (e.lo < n) e.tiles = (n - e.lo / p.box_rows * p.box_rows + kSharedTile - 1) / kSharedTile;
      }
      // (each group's before its place in the list is known: at the end of the array of entries)
      pl.entry[p.G + p.B + g] = e;
    }
  }
  __syncthreads();
  // the list: groups, then requests, those with keys
  const int items = p.G + p.B, n = (items + kPlanThreads - 1) / kPlanThreads;
  auto make = [&](int i) {
    if (i < p.G) return pl.entry[p.G + p.B + i];
    const int b = i - p.G, len = shared_len(p, b);
    SharedEntry e{b * p.Nq, p.Nq, b, 0, len, 0, 0, 0, 1};
    if (grouped) e.lo = min(pl.g_shared[pl.group[b]], len);
    if (p.win_left >= 0) {
      e.lo = max(e.lo, len - p.Nq - p.win_left);
      e.all_lo = len - 1 - p.win_left;
    }
    e.all_lo = max(e.all_lo, e.lo);
    e.all_hi = len - p.Nq + 1;
    if (e.lo < len) e.tiles = (len - e.lo / p.box_rows * p.box_rows + kSharedTile - 1) / kSharedTile;
    return e;
  };
  const int i0 = min(items, tid * n), i1 = min(items, i0 + n);
  long long w = 0;
  int c = 0;
  for (int i = i0; i < i1; ++i) {
    const SharedEntry e = make(i);
    if (e.tiles > 0) w += (e.tiles + p.lead) * units_of(p, e.ntok), ++c;
  }
  long long ws = w;
  int cs = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, ws, o);
    const int y = __shfl_up_sync(0xffffffffu, cs, o);
    if (lane >= o) ws += x, cs += y;
  }
  if (lane == 31) s_w[warp] = ws, s_n[warp] = cs;
  __syncthreads();
  long long total = 0;
  int count = 0;
  ws -= w, cs -= c;
#pragma unroll
  for (int x = 0; x < 32; ++x) {
    if (x < warp) ws += s_w[x], cs += s_n[x];
    total += s_w[x], count += s_n[x];
  }
  for (int i = i0; i < i1; ++i) {
    const SharedEntry e = make(i);
    const bool on = e.tiles > 0;
    if (on) {
      pl.entry[cs] = e;
      pl.cum[cs] = ws;
    }
    (i < p.G ? pl.of_group[i] : pl.of_request[i - p.G]) = on ? cs : -1;
    if (on) ws += (e.tiles + p.lead) * units_of(p, e.ntok), ++cs;
  }
  if (!grouped)
    for (int b = tid; b < p.B; b += kPlanThreads) pl.group[b] = -1;
  if (tid == 0) {
    *pl.count = count;
    *pl.total = total;
    pl.cum[count] = total;
  }
  __syncthreads();
  // where the shares begin
  for (int k = tid; k < p.shares; k += kPlanThreads) {
    const long long at = share_begin(total, p.shares, k);
    int a = 0, z = count;  // the last entry that begins at or before it
    while (z - a > 1) {
      const int m = (a + z) / 2;
      if (pl.cum[m] <= at) a = m; else z = m;
    }
    pl.start_entry[k] = a;
    pl.start_off[k] = count > 0 ? at - pl.cum[a] : 0;
  }
}

// ---------------------------------------------------------------- main

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    fa_decode_shared_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ SharedParams p) {
  using L = SharedLayout<D>;
  constexpr int NS = L::kStages, CH = D / 64;
  constexpr uint32_t TILE = L::kTile, CHUNK = L::kChunk;
  const int warp = warp_id(), lane = lane_id();

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sb = smem_raw + (base - raw);
  const uint32_t q_s = base + L::kQOff, kv_s = base + L::kKVOff;

  Piece* s_piece = reinterpret_cast<Piece*>(sb + L::kMiscOff);                         // [kPieces]
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(sb + L::kMiscOff + 64 * kPieces);      // [2 groups][2][4]
  static_assert(sizeof(Piece) == 64, "pieces");
  const uint32_t bar0 = base + L::kMiscOff + 64 * kPieces + 64;
  // Rings: K/V tiles, pieces.  Q[s]: a tile of Q has landed; its last S product is
  // done.  Per tile t in turn: S ready, P ready, the last product of a run of key
  // tiles done (O), and O read.  X: the softmax warps of a tile, and of both, have
  // come this far.
  enum { KV_FULL = 0, KV_EMPTY = NS, PC_FULL = 2 * NS, PC_EMPTY = PC_FULL + kPieces, Q_FULL = PC_EMPTY + kPieces,
         Q_EMPTY = Q_FULL + 2, S_FULL = Q_EMPTY + 2, P_FULL = S_FULL + 2, O_FINAL = P_FULL + 2, O_EMPTY = O_FINAL + 2,
         XB = O_EMPTY + 2, DRAIN = XB + 3, NBARS = DRAIN + 1 };
  static_assert(64 * kPieces + 64 + 8 * NBARS + 16 <= 1024, "misc area");
  auto BAR = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sb + L::kMiscOff + 64 * kPieces + 64 + 8 * NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NBARS; ++i) {
      int n = 1;
      if (i >= PC_EMPTY && i < PC_EMPTY + kPieces) n = 9;  // the products' warp and eight of softmax
      if (i == P_FULL || i == P_FULL + 1 || i == O_EMPTY || i == O_EMPTY + 1) n = 128;
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
  asm volatile("griddepcontrol.launch_dependents;");  // the merge may be set up; it waits for this grid's end
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is there

  if (warp == 0) {
    // ============================================================ loads
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    bool ok = true;
    const int k = blockIdx.x;
    const long long total = *p.plan.total, from = share_begin(total, p.shares, k), to = share_begin(total, p.shares, k + 1);
    const int count = *p.plan.count;
    const int bpb = p.box_rows / 16;  // 16-key groups per TMA box
    // the walk over the share
    long long at = from, off = p.plan.start_off[k];
    int e = p.plan.start_entry[k], pieces = 0, row = 0;
    SharedEntry ent = {}, ahead = {};
    if (from < to) {
      ent = p.plan.entry[e];
      if (e + 1 < count) ahead = p.plan.entry[e + 1];
    }
    auto next = [&]() {  // the share's next piece; t0 = t1: none is left
      Piece s = {};
      while (at < to) {
        const int weight = ent.tiles + p.lead;
        const int chunks = chunks_of(p, ent.ntok);
        if (off >= (long long)weight * p.Hkv * chunks) {
          off = 0;
          ++e;
          ent = ahead;
          if (e + 1 < count) ahead = p.plan.entry[e + 1];  // (read long before it is needed)
          continue;
        }
        const int u = (int)div_ll(off, weight), w0 = (int)(off - (long long)u * weight);
        const int w1 = (int)(to - at < weight - w0 ? w0 + (to - at) : weight);
        const bool later = w0 == 0 && at > from;  // the unit begins behind the share's first slot
        off += w1 - w0;
        at += w1 - w0;
        s.t0 = max(w0 - p.lead, 0), s.t1 = max(w1 - p.lead, 0);
        if (s.t0 == s.t1) continue;
        s.head = (int)((unsigned)u / (unsigned)chunks);
        const int c = u - s.head * chunks;
        s.tok0 = ent.tok0 + c * 2 * p.tile_tokens;
        s.ntok = min(2 * p.tile_tokens, ent.ntok - c * 2 * p.tile_tokens);
        s.lo = ent.lo, s.end = ent.end, s.all_lo = ent.all_lo, s.all_hi = ent.all_hi;
        s.beg = ent.lo / p.box_rows * p.box_rows;
        s.whole = s.t0 == 0 && s.t1 == ent.tiles;
        s.kind = ent.kind;
        s.slot = 2 * k + (later ? 1 : 0);
        row = ent.row;
        return s;
      }
      s.t0 = s.t1 = 0;
      return s;
    };
    struct Batch {  // up to four tiles of a piece, lane i owning 16 keys
      int n, page, off, head;
      bool on, first;
      Piece pc;
    };
    Piece pc = {};
    int t_next = 0;
    bool more = true;
    auto fetch = [&](Batch& q) {
      q.n = 0, q.on = q.first = false;
      if (!more) return;
      if (t_next == pc.t1) {
        pc = next();
        t_next = pc.t0;
        more = pc.t0 < pc.t1;
        if (!more) return;
        q.first = true;
      }
      q.pc = pc;
      q.n = min(4, pc.t1 - t_next);
      const int g = (pc.beg + t_next * kSharedTile) / 16 + lane;
      q.on = lane < 8 * q.n && g < (pc.end + 15) / 16;
      q.head = pc.head;
      t_next += q.n;
      if (q.on) {
        const int blk = (int)((unsigned)(g * 16) / (unsigned)p.page_size);
        q.off = g * 16 - blk * p.page_size;
        q.page = p.block_table[(size_t)row * p.max_blocks + blk];
      }
    };
    auto announce = [&](const Piece& s) {
      const int slot = pieces % kPieces;
      if (pieces >= kPieces) ok = __all_sync(0xffffffffu, mbar_wait(BAR(PC_EMPTY + slot), (pieces / kPieces - 1) & 1, w, 70));
      if (!ok) return;
      if (lane == 0) {
        s_piece[slot] = s;
        mbar_arrive(BAR(PC_FULL + slot));
      }
      ++pieces;
    };
    int it = 0, qt = 0;  // key tiles, tiles of Q so far
    Batch now, then;
    fetch(now);
    fetch(then);
    while (ok && now.n > 0) {
      if (now.on && (now.page < 0 || now.page >= p.num_pages)) {  // report, and read a valid page instead
        atomicCAS(p.err, 0u, FA_DEVERR_BAD_PAGE);
        now.page = 0;
      }
      if (now.first) announce(now.pc);
      const uint32_t on = __ballot_sync(0xffffffffu, now.on);
      for (int i = 0; i < now.n && ok; ++i, ++it) {
        const int boxes = (__popc(on >> (8 * i) & 0xffu) + bpb - 1) / bpb;
        const bool issue = (lane >> 3) == i && now.on && (lane & (bpb - 1)) == 0;
        const uint32_t dst = (uint32_t)(lane & 7) * 16u * 128u;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int u = 2 * it + v, slot = u % NS;
          if (u >= NS) ok = mbar_wait(BAR(KV_EMPTY + slot), (u / NS - 1) & 1, w, 71);
          if (!__all_sync(0xffffffffu, ok)) break;
          if (lane == 0) mbar_arrive_expect_tx(BAR(KV_FULL + slot), (uint32_t)(boxes * p.box_rows * D * 2));
          __syncwarp();
          if (issue) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
              tma_load_4d(kv_s + slot * TILE + c * CHUNK + dst, v ? &tm_v : &tm_k, BAR(KV_FULL + slot), c * 64, now.head,
                          now.off, now.page);
          }
          __syncwarp();
        }
        ok = __all_sync(0xffffffffu, ok);
        if (ok && i == 0 && now.first) {  // Q behind the first keys, which need no room that the last unit's Q holds
          const int tiles = now.pc.ntok > p.tile_tokens ? 2 : 1;
          for (int x = 0; x < tiles && ok; ++x, ++qt) {
            const int slot = qt & 1;
            if (qt >= 2) ok = __all_sync(0xffffffffu, mbar_wait(BAR(Q_EMPTY + slot), (qt / 2 - 1) & 1, w, 72));
            if (ok && lane == 0) {
              mbar_arrive_expect_tx(BAR(Q_FULL + slot), (uint32_t)(p.tile_tokens * p.heads * D * 2));
#pragma unroll
              for (int c = 0; c < CH; ++c)
                tma_load_3d(q_s + slot * TILE + c * CHUNK, &tm_q, BAR(Q_FULL + slot), c * 64, now.head * p.heads,
                            now.pc.tok0 + x * p.tile_tokens);
            }
            __syncwarp();
          }
        }
      }
      now = then;
      fetch(then);
    }
    if (ok) announce(pc);  // the end
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
      int vslot, vphase;
      bool on, first, last, frees;  // first, last of its tile's run in the piece; the last to read its values
    } before{};
    int n = 0, it = 0, qt = 0, runs[2] = {0, 0}, ps[2] = {0, 0};
    bool ok = true;
    auto product = [&](const Job& j, int t) {  // O_t (+)= P V
      bool good = mbar_wait(BAR(KV_FULL + j.vslot), j.vphase, w, 73);
      if (__all_sync(0xffffffffu, good)) good = mbar_wait(BAR(P_FULL + t), ps[t] & 1, w, 74);
      if (__all_sync(0xffffffffu, good) && j.first && runs[t] > 0)  // the run before has been read
        good = mbar_wait(BAR(O_EMPTY + t), (runs[t] - 1) & 1, w, 75);
      if (!__all_sync(0xffffffffu, good)) return false;
      ++ps[t];
      if (j.first) ++runs[t];
      tc_fence_after();
      const uint32_t va = kv_s + j.vslot * TILE, dst = tmem + 256u + (t ? (uint32_t)D : 0u), pa = tmem + (t ? 128u : 0u);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ts_w(dst, pa + kk * 8, smem_desc_sw128(va + kk * 2048, CHUNK, 1024), IDESC_O, (!j.first || kk > 0) ? 1u : 0u);
      if (j.frees) mma_commit_w(BAR(KV_EMPTY + j.vslot));
      if (j.last) mma_commit_w(BAR(O_FINAL + t));
      return true;
    };
    for (int piece = 0; ok; ++piece) {
      const int pslot = piece % kPieces;
      ok = __all_sync(0xffffffffu, mbar_wait(BAR(PC_FULL + pslot), piece / kPieces & 1, w, 76));
      if (!ok) break;
      const int tiles = s_piece[pslot].t1 - s_piece[pslot].t0, subs = s_piece[pslot].ntok > p.tile_tokens ? 2 : 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(PC_EMPTY + pslot));
      if (tiles == 0) break;
      for (int x = 0; x < tiles && ok; ++x, ++it) {
        const int uk = 2 * it, sk = uk % NS, uv = uk + 1;
        for (int sub = 0; sub < subs && ok; ++sub, ++n) {
          const int t = n & 1, qs = (qt + sub) & 1;
          if (x == 0) ok = __all_sync(0xffffffffu, mbar_wait(BAR(Q_FULL + qs), (qt + sub) / 2 & 1, w, 77));
          if (ok && sub == 0) ok = __all_sync(0xffffffffu, mbar_wait(BAR(KV_FULL + sk), uk / NS & 1, w, 78));
          if (!ok) break;
          tc_fence_after();
          const uint32_t qa = q_s + qs * TILE, ka = kv_s + sk * TILE, dst = tmem + (t ? 128u : 0u);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (kk / 4) * CHUNK + (kk % 4) * 32;
            mma_ss_w(dst, smem_desc_sw128(qa + o, 16, 1024), smem_desc_sw128(ka + o, 16, 1024), IDESC_S, kk > 0);
          }
          mma_commit_w(BAR(S_FULL + t));
          if (x == tiles - 1) mma_commit_w(BAR(Q_EMPTY + qs));
          if (sub == subs - 1) mma_commit_w(BAR(KV_EMPTY + sk));
          if (before.on) ok = product(before, t ^ 1);
          const int alone = 3 - subs;  // jobs between a tile's jobs on the same S: key tiles in turn, or every one
          before = {uv % NS, uv / NS & 1, true, x < alone, x >= tiles - alone, sub == subs - 1};
        }
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
  } else if (warp >= 4) {
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
    for (int piece = 0; ok; ++piece) {
      const int pslot = piece % kPieces;
      ok = __all_sync(0xffffffffu, mbar_wait(BAR(PC_FULL + pslot), piece / kPieces & 1, w, 79));
      if (!ok) break;
      const Piece s = s_piece[pslot];
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(PC_EMPTY + pslot));
      const int tiles = s.t1 - s.t0;
      if (tiles == 0) break;
      const bool pair = s.ntok > p.tile_tokens;
      const int side = (t ^ n0) & 1;  // pair: tile of rows; else: which of the two runs of key tiles
      const int tok = s.tok0 + (pair ? side * p.tile_tokens : 0) + my_tok;
      const bool valid = my_tok < p.tile_tokens && tok < s.tok0 + s.ntok;
      // the keys this row sees: [key_lo, key_hi)
      int key_lo = 0, key_hi = 0;
      if (valid) {
        const int b = p.Nq == 1 ? tok : (int)((unsigned)tok / (unsigned)p.Nq);
        const int len = min(max(p.seq_lens[b], 0), p.max_len), pos = len - p.Nq + tok - b * p.Nq;
        key_lo = p.win_left >= 0 ? max(s.lo, pos - p.win_left) : s.lo;
        key_hi = min(s.end, pos + 1);
      }
      const bool live = __any_sync(0xffffffffu, valid);  // some row of the warp is there
      float m_ref = -INFINITY, l = 0.f;
      bool poison = false;
      const int x_step = pair ? 1 : 2, x_first = pair ? 0 : side;
      for (int x = x_first; x < tiles; x += x_step, ++phase) {
        const int uv = 2 * (it0 + x) + 1, vslot = uv % NS;
        const int j0 = s.beg + (s.t0 + x) * kSharedTile;
        ok = mbar_wait(BAR(S_FULL + t), phase & 1, w, 80);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (j0 < s.all_lo || j0 + kSharedTile > s.all_hi) {
          // Some rows do not see some keys of the tile, and 0 times a NaN or an infinity
          // is not 0.  What no row sees (it may be anything) counts as zero; a value row
          // that some see, and that holds one, counts as zero too, and its rows get a NaN.
          ok = mbar_wait(BAR(KV_FULL + vslot), uv / NS & 1, w, 81);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          const int key = j0 + r;
          const bool out = key < s.lo || key >= s.end;
          uint4* row = reinterpret_cast<uint4*>(sb + L::kKVOff + vslot * TILE + r * 128);
          bool odd = false;
          if (max(j0, s.lo) < s.all_lo || min(j0 + kSharedTile, s.end) > s.all_hi) {
            if (!out && (key < s.all_lo || key >= s.all_hi)) {
              uint32_t bad = 0;
#pragma unroll 1
              for (int i = 0; i < 8 * CH; ++i) {
                const uint4 v = row[(i >> 3) * (CHUNK / 16) + (i + lane & 7)];  // (other banks for each lane)
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
            ok = pair ? mbar_wait(BAR(XB + 2), xb++ & 1, w, 82) : mbar_wait(BAR(XB + t), xg++ & 1, w, 83);
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
              for (int i = 0; i < 8 * CH; ++i) row[(i >> 3) * (CHUNK / 16) + (i + lane & 7)] = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
        }
        if (live) {
          uint32_t sr[4][32];
          float mq[4];  // each load's maximum over its 32 columns
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_max(tS + 32 * c, sr[c], mq[c]);
          tmem_ld_wait();
          float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
          float v[128];
#pragma unroll
          for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(sr[i / 32][i % 32]);
          if (j0 < key_lo || j0 + kSharedTile > key_hi) {  // a tile the row sees only in part, or not at all
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (j0 + i < key_lo || j0 + i >= key_hi) v[i] = -INFINITY;
            float mg[8];
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              float m = fmaxf(v[16 * g], v[16 * g + 1]);
#pragma unroll
              for (int i = 2; i < 16; i += 2) m = max3f(m, v[16 * g + i], v[16 * g + i + 1]);
              mg[g] = m;
            }
            mx = max3f(max3f(mg[0], mg[1], mg[2]), max3f(mg[3], mg[4], mg[5]), fmaxf(mg[6], mg[7]));
          }
          const float m_new = mx * sl2;
          float alpha = 1.f;
          const bool moves = m_new > m_ref + p.tau;
          if (moves) {
            alpha = ex2_sfu(m_ref - m_new);
            m_ref = m_new;
          }
          const float mb = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t nmb2 = f2_pack(-mb, -mb);
          uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
          uint32_t pk[2][32];
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            float y0, y1;
            f2_unpack(f2_fma(f2_pack(v[2 * i], v[2 * i + 1]), sl2x2, nmb2), y0, y1);
            const float p0 = ex2_sfu(y0), p1 = ex2_sfu(y1);
            acc[i & 3] = f2_add(acc[i & 3], f2_pack(p0, p1));
            pk[i / 32][i % 32] = pack_bf16x2(p0, p1);
            if (i == 31) tmem_st32(tS, pk[0]);  // the first half out early: frees registers
          }
          const uint64_t sum = f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3]));
          float s0, s1;
          f2_unpack(sum, s0, s1);
          l = fmaf(l, alpha, s0 + s1);
          if (x != x_first && __any_sync(0xffffffffu, moves)) {
            // rows whose reference moved: O *= alpha (alpha = 1 for the others)
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              tmem_ld32(tO + 32 * c, ov);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
              tmem_st32(tO + 32 * c, ov);
            }
          }
          tmem_st32(tS + 32, pk[1]);
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(BAR(P_FULL + t));
      }
      if (!ok) break;
      n0 += pair ? 2 * tiles : tiles;
      it0 += tiles;
      // ---------------------------------------------------------- results of the run
      const int h = s.head * p.heads + my_head;
      const long long place = s.whole ? (long long)(2 * s.kind + (pair ? 0 : side)) * rows + (long long)tok * p.Hq + h
                                      : 4 * rows + ((long long)s.slot * 2 + side) * 128 + r;
      if (x_first >= tiles) {  // one tile of keys: the other run has none
        if (valid) p.part_lse[place] = -INFINITY;
        continue;
      }
      ok = mbar_wait(BAR(O_FINAL + t), runs & 1, w, 84);
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
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<uint4*>(dst + 32 * c)[i] = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
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
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- merge

// A warp per query row: the results of the group's shared keys and of the
// request's own.  A part without mass has lse = -inf, and its O is not read.
template <int D>
__global__ void __launch_bounds__(256) fa_decode_shared_merge_kernel(const __grid_constant__ SharedParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)p.B * p.Nq * p.Hq, x = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the main kernel's grid is done
  if (x >= rows) return;
  const long long token = div_ll(x, p.Hq);
  const int tok = (int)token, h = (int)(x - token * p.Hq), head = h / p.heads, b = tok / p.Nq;
  const long long total = *p.plan.total, each = div_ll(total, p.shares), more = total - each * p.shares;
  auto share_of = [&](long long s) {
    return (int)(s < more * (each + 1) ? div_ll(s, each + 1) : more + div_ll(s - more * (each + 1), each));
  };
  float acc[E], mass = 0.f, m = -INFINITY;
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = 0.f;
  auto add = [&](long long place) {
    const float lc = p.part_lse[place];
    if (lc == -INFINITY) return;
    const float* src = p.part_o + place * D + lane * E;
    float v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = src[i];
    const float mn = fmaxf(m, lc), ref = mn == -INFINITY ? 0.f : mn;  // (lc may be NaN)
    const float al = ex2_sfu(m - ref), f = ex2_sfu(lc - ref);
    m = mn;
    mass = fmaf(mass, al, f);
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = fmaf(acc[i], al, f * v[i]);
  };
  const int g = p.plan.group[b];
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const int e = kind == 0 ? (g >= 0 ? p.plan.of_group[g] : -1) : p.plan.of_request[b];
    if (e < 0) continue;
    const SharedEntry ent = p.plan.entry[e];
    const int weight = ent.tiles + p.lead, chunks = chunks_of(p, ent.ntok);
    const int c = (tok - ent.tok0) / (2 * p.tile_tokens), in = tok - ent.tok0 - c * 2 * p.tile_tokens;
    const bool pair = ent.ntok - c * 2 * p.tile_tokens > p.tile_tokens;
    const long long u0 = p.plan.cum[e] + (long long)weight * ((long long)head * chunks + c);
    const int first = share_of(u0 + p.lead), last = share_of(u0 + weight - 1);
    if (first == last) {
      add((2 * kind) * rows + x);
      if (!pair) add((2 * kind + 1) * rows + x);
      continue;
    }
    const int side = in / p.tile_tokens, r = (in - side * p.tile_tokens) * p.heads + h - head * p.heads;
    for (int k = first; k <= last; ++k) {
      // the share's last piece, if it begins before the unit, or its first
      const long long slot = 2 * (long long)k + (each * k + (k < more ? k : more) < u0 ? 1 : 0);
      if (pair) {
        add(4 * rows + (slot * 2 + side) * 128 + r);
      } else {
        add(4 * rows + slot * 256 + r);
        add(4 * rows + slot * 256 + 128 + r);
      }
    }
  }
  const float inv = mass == 0.f ? 0.f : 1.f / mass;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + x * D + lane * E);
#pragma unroll
  for (int i = 0; i < E; i += 2) dst[i / 2] = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
  if (lane == 0)
    p.lse[((long long)b * p.Hq + h) * p.Nq + tok - b * p.Nq] = mass == 0.f ? -INFINITY : (m + __log2f(mass)) * 0.69314718055994531f;
}

// ---------------------------------------------------------------- host

static size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// The plan's arrays one after the other from `at` (or their bytes alone).
static size_t plan_layout(SharedPlan* plan, void* at, int B, int G, int shares) {
  uint8_t* base = static_cast<uint8_t*>(at);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* here = base + off;
    off += up16(bytes);
    return here;
  };
  SharedPlan pl;
  const size_t n = (size_t)B + G;
  pl.total = reinterpret_cast<long long*>(take(8));
  pl.count = reinterpret_cast<int*>(take(4));
  pl.entry = reinterpret_cast<SharedEntry*>(take(sizeof(SharedEntry) * (n + G)));  // (and the groups', before they have a place)
  pl.cum = reinterpret_cast<long long*>(take(8 * (n + 1)));
  pl.of_group = reinterpret_cast<int*>(take(4 * (size_t)G));
  pl.of_request = reinterpret_cast<int*>(take(4 * (size_t)B));
  pl.group = reinterpret_cast<int*>(take(4 * (size_t)B));
  pl.g_shared = reinterpret_cast<int*>(take(4 * (size_t)G));
  pl.start_entry = reinterpret_cast<int*>(take(4 * (size_t)shares));
  pl.start_off = reinterpret_cast<long long*>(take(8 * (size_t)shares));
  if (plan != nullptr) *plan = pl;
  return off;
}
size_t shared_plan_bytes(int B, int G, int shares) { return plan_layout(nullptr, nullptr, B, G, shares); }
void shared_plan_at(SharedPlan& plan, void* at, int B, int G, int shares) { plan_layout(&plan, at, B, G, shares); }

template <int D>
static cudaError_t launch_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const SharedParams& p,
                            cudaStream_t stream) {
  auto kern = fa_decode_shared_kernel<D>;
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
  if ((e = cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, p)) != cudaSuccess) return e;
  const long long rows = (long long)p.B * p.Nq * p.Hq;
  cfg.gridDim = dim3((unsigned)((rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, fa_decode_shared_merge_kernel<D>, p);
}

cudaError_t launch_decode_shared(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const SharedParams& p,
                                 int D, cudaStream_t stream) {
  if (D == 64) return launch_t<64>(tq, tk, tv, p, stream);
  if (D == 128) return launch_t<128>(tq, tk, tv, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fa
