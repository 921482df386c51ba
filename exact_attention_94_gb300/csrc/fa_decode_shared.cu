// The plan and the merge of decode_shared.cuh, and its main kernel over bf16 pages.
#include "decode_shared.cuh"

namespace fa {

cudaError_t launch_shared_main8(const CUtensorMap (&maps)[5], const SharedParams& p, int D, cudaLaunchConfig_t& cfg);

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
    const bool late = total[1] >= (long long)kFewLateFrom * p.warps * others;
    head.total[2] = late ? total[1] / (others > 0 ? kFewLateOf : 1) : 0;
    head.shares[2] = shares_in((long long)kFewLate * p.shares, head.total[2], kFewLateLeast);
    if (late && head.shares[2] == 0) head.shares[2] = 1;
    head.total[1] = total[1] - head.total[2];
    head.shares[1] = head.total[1] > 0 ? max(shares_in((long long)p.warps * others, head.total[1], kFewLeast), 1) : 0;
  }
  head.count[0] = count[0], head.count[1] = count[1];
  head.queue = head.shares[1];
  if (tid == 0) *pl.head = head;
}

// ---------------------------------------------------------------- merge

// What the merge reads of the plan: EARLY, while its writes need not be visible yet, past L1; else through it, for all
// warps of an SM read the same (past it 4096 rows took 8 us more).
template <bool EARLY, class T>
__device__ __forceinline__ T seen(const T* at) {
  if constexpr (sizeof(T) == 16) {
    longlong2 x;
    if constexpr (EARLY) asm volatile("ld.relaxed.gpu.global.v2.s64 {%0, %1}, [%2];" : "=l"(x.x), "=l"(x.y) : "l"(at) : "memory");
    else asm volatile("ld.global.v2.s64 {%0, %1}, [%2];" : "=l"(x.x), "=l"(x.y) : "l"(at) : "memory");
    return x;
  } else if constexpr (sizeof(T) == 8) {
    long long x;
    if constexpr (EARLY) asm volatile("ld.relaxed.gpu.global.s64 %0, [%1];" : "=l"(x) : "l"(at) : "memory");
    else asm volatile("ld.global.s64 %0, [%1];" : "=l"(x) : "l"(at) : "memory");
    return x;
  } else {
    int x;
    if constexpr (EARLY) asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(x) : "l"(at) : "memory");
    else asm volatile("ld.global.s32 %0, [%1];" : "=r"(x) : "l"(at) : "memory");
    return x;
  }
}
struct SeenPlan {
  int entry[2];                   // of_request
  int tok0[2], ntok[2], tiles[2];
  long long cum[2];
  longlong2 head[2];              // totals, shares of the first two lists
  int last;                       // shares of the third
  // What is at the places `of` of the lists, and the head.
  template <bool EARLY>
  __device__ __forceinline__ void read(const SharedParams& p, const int (&of)[2]) {
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      tok0[kind] = ntok[kind] = tiles[kind] = 0, cum[kind] = 0;
      if (of[kind] < 0) continue;
      const SharedList& list = p.plan.list[of[kind] & 1];
      const int i = min(of[kind] >> 1, p.G + p.B - 1);  // (an entry there is, whatever has been read)
      const SharedEntry* e = list.entry + i;
      tok0[kind] = seen<EARLY>(&e->tok0), ntok[kind] = seen<EARLY>(&e->ntok), tiles[kind] = seen<EARLY>(&e->tiles);
      cum[kind] = seen<EARLY>(list.cum + i);
    }
    const longlong2* h = reinterpret_cast<const longlong2*>(p.plan.head);
    head[0] = seen<EARLY>(h), head[1] = seen<EARLY>(h + 1), last = seen<EARLY>(&p.plan.head->shares[2]);
  }
  template <bool EARLY>
  __device__ __forceinline__ void read_entries(const SharedParams& p, int b) {
    const long long x = seen<EARLY>(reinterpret_cast<const long long*>(p.plan.of_request + b));
    entry[0] = (int)x, entry[1] = (int)(x >> 32);
  }
  __device__ __forceinline__ bool operator==(const SeenPlan& o) const {
    bool same = head[0].x == o.head[0].x && head[0].y == o.head[0].y && head[1].x == o.head[1].x && head[1].y == o.head[1].y &&
                last == o.last;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
      same = same && entry[kind] == o.entry[kind] && tok0[kind] == o.tok0[kind] && ntok[kind] == o.ntok[kind] &&
             tiles[kind] == o.tiles[kind] && cum[kind] == o.cum[kind];
    return same;
  }
};

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
  // parts of each kind: n of them, `runs` in each of the shares from `first` on
  int n[2], runs[2], first[2];
  long long base[2], begin[2];  // place of the first part, or of the row in a slot; the unit's begin
  bool cut[2], few[2];
  Deal deals[2] = {{{0, 0}, {0, 0}}, {{0, 0}, {0, 0}}};
  // The plan's writes are sure to be visible behind the wait alone, but until then the main kernel works: they are
  // read and worked on before it, and read behind it once more, all at once, to compare.  (1 us of a call; 4 to 8
  // where all of this begins behind the wait.)
  SeenPlan plan;
  for (bool early = true;; early = false) {
    plan.read_entries<true>(p, b);
    plan.read<true>(p, plan.entry);
    SharedHead totals;
    totals.total[0] = plan.head[0].x, totals.total[1] = plan.head[0].y, totals.total[2] = plan.head[1].x;
    totals.shares[0] = (int)plan.head[1].y, totals.shares[1] = (int)(plan.head[1].y >> 32), totals.shares[2] = plan.last;
    deals[0] = deal_of(totals, false), deals[1] = deal_of(totals, true);
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      n[kind] = 0, runs[kind] = 1, first[kind] = 0, base[kind] = begin[kind] = 0, cut[kind] = few[kind] = false;
      const int of = plan.entry[kind];
      if (of < 0) continue;
      few[kind] = of & 1;
      const Deal& deal = (of & 1) ? deals[1] : deals[0];
      const Weight wt = weight_of(p, few[kind], plan.ntok[kind]);
      const int weight = wt.lead + wt.tile * plan.tiles[kind], chunks = chunks_of(p, few[kind], plan.ntok[kind]);
      const int c = few[kind] ? 0 : (tok - plan.tok0[kind]) / (2 * p.tile_tokens), in = tok - plan.tok0[kind] - c * 2 * p.tile_tokens;
      const bool pair = few[kind] || plan.ntok[kind] - c * 2 * p.tile_tokens > p.tile_tokens;
      begin[kind] = plan.cum[kind] + (long long)weight * ((long long)head * chunks + c);
      first[kind] = deal.of(begin[kind] + wt.lead);
      const int last = deal.of(begin[kind] + weight - wt.tile);  // where the last tile begins
      cut[kind] = first[kind] != last;
      runs[kind] = pair ? 1 : 2;
      n[kind] = (last - first[kind] + 1) * runs[kind];
      const int side = few[kind] ? 0 : in / p.tile_tokens;
      base[kind] = cut[kind] ? side * kSharedTile + (in - side * p.tile_tokens) * p.heads + h0 : 2 * kind * rows + row;
    }
    if (!early) break;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the main kernel's grid is done, and the plan before it
    SeenPlan now;
    now.read_entries<false>(p, b);
    now.read<false>(p, plan.entry);
    if (__all_sync(0xffffffffu, now == plan)) break;
  }
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
// The most rows of an entry that a warp attends for, if a request's own keys meet no more;
// 0: tiles for all.  (64 requests of 4096 tokens, 64 heads over 8, d = 128: 16 rows 224 us by
// warps and 193 by tiles, but 4 drafts of 4 heads behind shared prompts 38 and 41; 32 rows 367
// and 197.  8-bit pages, whose conversions take registers: 16 rows 386 and 267, of d = 64 98 and 146.
// Rows alone decide: where 16 rows of bf16 meet long own keys, tiles would be the better choice.)
int shared_few(int Nq, int heads, int D, bool kv8) {
  const int rows = Nq * heads;
  return rows <= 8 ? 8 : rows <= 16 && !(kv8 && D == 128) ? 16 : 0;
}
size_t shared_part_rows(int B, int Nq, int Hq, int heads, int shares) {
  return 4 * (size_t)B * Nq * Hq + 512 * (size_t)shares + 2 * (size_t)shared_few(Nq, heads, 64, false) * (kFewEarly + kFewLate) * shares;
}
size_t shared_plan_bytes(int B, int G) { return plan_layout(nullptr, nullptr, B, G); }
void shared_plan_at(SharedPlan& plan, void* at, int B, int G) { plan_layout(&plan, at, B, G); }

template <int D>
static cudaError_t launch_merge(const SharedParams& p, cudaLaunchConfig_t& cfg) {
  const long long tokens = (long long)p.B * p.Nq * p.Hkv;
  const bool one = tokens * p.heads <= 32ll * kSms;
  const long long warps = tokens * (one ? p.heads : (p.heads + kMergeRows - 1) / kMergeRows);
  cfg.gridDim = dim3((unsigned)((warps + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return one ? cudaLaunchKernelEx(&cfg, fa_decode_shared_merge_kernel<D, 1>, p)
             : cudaLaunchKernelEx(&cfg, fa_decode_shared_merge_kernel<D, kMergeRows>, p);
}

cudaError_t launch_decode_shared(const CUtensorMap (&maps)[5], SharedParams& p, int D, bool kv8, cudaStream_t stream) {
  if (D != 64 && D != 128) return cudaErrorInvalidValue;
  p.few_cost = kFew * D / 128 * (kv8 ? kFew8 : 1.f);
  p.few = shared_few(p.Nq, p.heads, D, kv8);
  p.warps = few_warps(D, kv8);
  fa_shared_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = &a;
  cfg.numAttrs = 1;
  e = kv8 ? launch_shared_main8(maps, p, D, cfg)
          : D == 64 ? launch_shared_main<64, false>(maps, p, cfg) : launch_shared_main<128, false>(maps, p, cfg);
  if (e != cudaSuccess) return e;
  return D == 64 ? launch_merge<64>(p, cfg) : launch_merge<128>(p, cfg);
}

}  // namespace fa
