// Attention for entries of few rows (16 query rows at most), a warp by itself for each
// piece of a unit, beside or behind the tiles of many rows: included by
// decode_shared.cuh, within its namespace.
//
// What bounds it is HBM: a row of keys meets 8 rows of queries, a 16th of what the
// 128 rows of a tensor-memory tile do, and such a tile's exchanges between warps
// cost 5.6 us a unit.  Here keys take the M side of small warp-wide products, 16
// of them a step, and 8 NR rows the N side:
//     S^T [16 keys x rows] = K Q^T,    O^T [d x rows] += V^T P^T,
// so 8 rows fill a product, P^T becomes the second one's operand by transposing
// 8 x 8 blocks between lanes, and O^T stays in registers.  A warp has its own ring of
// steps in shared memory, filled by TMA across units' borders, and meets no other warp
// until its results are merged.
//
// A warp alone takes some 1300 to 1570 cycles a step, dependent instructions and
// instruction fetches, so eight of an SM take 80 GB/s of d = 128, and of d = 64 (a step
// is half the bytes) 48, twelve 70 (HBM's share of an SM is 45; beside 130 CTAs of tiles they
// get that).  64 requests of 4096 own tokens, 16 heads of 64 over 16: 198 us, 5.4 TB/s.
constexpr int kFewStages = 5;  // of a warp's ring, at most
constexpr int kFewPieces = 4;  // a warp knows of: one it works on, those it loads

struct FewPiece {
  int slot;  // of the results: 2 share + later; -1: the unit's only piece
  int head_kind;
  int tok0, ntok;
  int lo, end, all_lo, all_hi;
  int t0, t1;
};
// What a warp keeps in shared memory beside its rings.
struct FewState {
  FewPiece ring[kFewPieces];
  unsigned long long bars[kFewStages];  // a step has landed
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Of a row of queries (at `row`, as copied), the second product operand for step x of 16 elements of d
// against codes: a lane's four codes are d .. d + 3.
__device__ __forceinline__ void few_queries(uint32_t& b0, uint32_t& b1, const uint8_t* row, int x, int q, int r) {
  const int c = 8 * (x >> 2) + 2 * q + (x >> 1 & 1);
  const uint2 v = *reinterpret_cast<const uint2*>(row + ((c ^ r) << 4) + 8 * (x & 1));
  b0 = v.x, b1 = v.y;
}
// 16 bytes to shared memory, or zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// k: the warp's first share, -1: none; at, mem: its shared memory, of BYTES.
template <int D, int NR, bool KV8, uint32_t BYTES>
__device__ __forceinline__ void attend_few(const SharedParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const WaitCtx& w,
                                           int k, uint32_t at, uint8_t* mem, FewState* state) {
  constexpr int ROWS = 8 * NR, CH = D / 64, C16 = D / 8;  // C16: 16-byte chunks of a row of bf16
  constexpr uint32_t TILE = 16u * D * (KV8 ? 1 : 2), QBYTES = ROWS * D * 2u, SCALES = KV8 ? 8 * kFewStages : 0;
  constexpr int FIT = (int)((BYTES - QBYTES - SCALES) / (2 * TILE)), NST = FIT < kFewStages ? FIT : kFewStages;
  static_assert(NST >= 2, "ring");
  FewPiece* ring = state->ring;
  const uint32_t bars = smem_u32(state->bars);
  float2* s_scale = reinterpret_cast<float2*>(mem + NST * 2 * TILE + QBYTES);  // KV8: of a step's keys, values
  constexpr uint32_t QAT = NST * 2 * TILE;
  const int lane = lane_id(), quad = lane >> 2, q2 = 2 * (lane & 3);
  const SharedList& list = p.plan.list[1];
  const Deal deal = deal_of(*p.plan.head, true);
  const int early = deal.early.n, all = early + deal.late.n, entries = p.plan.head->count[1];
  const float sl2 = p.scale_log2, tau = KV8 ? fminf(p.tau, kMaxTau) : p.tau;
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  // ------------------------------------------------------------ loads: shares, their pieces, batches of 32 steps
  Walk walk;
  walk.at = walk.to = 0;
  bool more = all > 0;
  if (k >= 0 && k < early) walk.start(list, entries, deal, k);
  int taken = 0, started = 0, queried = 0;  // pieces: known, worked on, whose queries were asked for
  int t_next = 0, t_end = 0, beg = 0, row = 0, head = 0;
  struct Batch {
    int n, page, rows8, head;  // lane i: step i's page and its place in there, in eights of keys
  };
  auto fetch = [&](Batch& b) {
    b.n = 0;
    if (t_next == t_end) {
      int u;
      bool later;
      int t0, t1;
      while (!walk.next(p, true, u, t0, t1, later)) {
        if (early == all) {
          k = all;
        } else {
          if (lane == 0) k = atomicAdd(&p.plan.head->queue, 1);
          k = __shfl_sync(0xffffffffu, k, 0);
        }
        if (k >= all) {
          more = false;
          return;
        }
        walk.start(list, entries, deal, k);
      }
      const SharedEntry& e = walk.ent;
      t_next = t0, t_end = t1;
      beg = e.lo / 16, row = e.row, head = u;
      if (lane == 0)
        ring[taken % kFewPieces] = {t0 == 0 && t1 == e.tiles ? -1 : 2 * k + (later ? 1 : 0), 2 * u + e.kind, e.tok0, e.ntok,
                                    e.lo, e.end, e.all_lo, e.all_hi, t0, t1};
      __syncwarp();
      ++taken;
    }
    b.n = min(32, t_end - t_next);
    b.head = head;
    b.page = b.rows8 = 0;
    if (lane < b.n) {
      const int g = beg + t_next + lane, blk = (int)((unsigned)(g * 16) / (unsigned)p.page_size);
      b.rows8 = 2 * g - blk * (p.page_size / 8);
      b.page = p.block_table[(size_t)row * p.max_blocks + blk];
    }
    t_next += b.n;
  };
  Batch now, then;
  now.n = then.n = 0;
  int i_now = 0, row_at = 0, plane = 0, issued = 0, done = 0, st_in = 0;
  float k_scale = 0.f, v_scale = 0.f;
  // ------------------------------------------------------------ the piece in work
  float o[D / 16][NR][4], m_ref[NR][2], l[NR][2];
  uint32_t qf[NR][D / 8];
  float q_back[KV8 ? NR : 1][2];  // what undoes the rows' scales
  int key_lo[NR][2], key_hi[NR][2];
  uint32_t poison = 0;
  FewPiece pc = {};
  int t = 0, st = 0;
  uint32_t phase = 0;
  bool ok = true;
  const uint32_t k_row = (uint32_t)((lane >> 3 & 1) * CH * 1024 + (lane & 7) * 128);  // ldmatrix: keys by matrix & 1, chunks by >> 1
  const uint32_t v_row = (uint32_t)((lane >> 4) * CH * 1024 + (lane & 7) * 128);      // keys by matrix >> 1, chunks by & 1
  const uint32_t x7 = lane & 7;
  for (;;) {
    // ---- ask for what there is room for
    if (more && then.n == 0 && (t_next < t_end || taken < started + kFewPieces - 1)) fetch(then);
    while (issued - done < NST) {
      if (i_now == now.n) {
        if (then.n == 0) break;
        now = then;
        i_now = 0;
        if (now.page < 0 || now.page >= p.num_pages) {  // report, and read a valid page instead
          atomicCAS(p.err, 0u, FA_DEVERR_BAD_PAGE);
          now.page = 0;
        }
        row_at = KV8 ? now.rows8 * 8 : now.page * (p.page_size / 8) + now.rows8;  // row of the page, or eight of all pages'
        plane = now.page * p.Hkv + now.head;
        if constexpr (KV8) {
          if (lane < now.n) k_scale = p.k_scale[plane], v_scale = p.v_scale[plane];
        }
        then.n = 0;
      }
      const int row = __shfl_sync(0xffffffffu, row_at, i_now), pl = KV8 ? __shfl_sync(0xffffffffu, plane, i_now) : 0;
      const uint32_t bar = bars + 8 * st_in, dst = at + st_in * 2 * TILE;
      if (KV8 && lane == i_now) s_scale[st_in] = make_float2(k_scale, v_scale);
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, 2 * TILE);
        if constexpr (KV8) {
          tma_load_3d(dst, &tm_k, bar, 0, row, pl);
          tma_load_3d(dst + TILE, &tm_v, bar, 0, row, pl);
        } else {
          tma_load_5d(dst, &tm_k, bar, 0, 0, 0, row, now.head);
          tma_load_5d(dst + TILE, &tm_v, bar, 0, 0, 0, row, now.head);
        }
      }
      __syncwarp();
      if (++st_in == NST) st_in = 0;
      ++i_now;
      ++issued;
    }
    if (queried < taken && queried <= started) {
      const FewPiece& f = ring[queried % kFewPieces];
      const int n = f.ntok * p.heads, h0 = (f.head_kind >> 1) * p.heads;
      for (int i = lane; i < ROWS * C16; i += 32) {
        const int r = i / C16, c = i % C16, tk = r < n ? r / p.heads : 0, h = r < n ? r - tk * p.heads : 0;
        const char* src = static_cast<const char*>(p.q) + (((long long)(f.tok0 + tk) * p.Hq + h0 + h) * D + c * 8) * 2;
        copy16(at + QAT + r * (D * 2) + ((c ^ (r & 7)) << 4), src, r < n);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      ++queried;
    }
    if (t == pc.t1) {  // the next piece
      if (done == issued) break;
      pc = ring[started % kFewPieces];
      t = pc.t0;
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      if constexpr (KV8) {  // queries to f16, a row times its own scale: four lanes a row
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          uint8_t* q_row = mem + QAT + (8 * nr + quad) * (D * 2);
          uint32_t most = 0;
#pragma unroll
          for (int c = lane & 3; c < C16; c += 4) most = largest_bf16(most, *reinterpret_cast<const uint4*>(q_row + ((c ^ quad) << 4)));
          most = max(most >> 16, most & 0xffffu);
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const RowScale rs(most);
#pragma unroll
          for (int c = lane & 3; c < C16; c += 4) {
            uint4* x = reinterpret_cast<uint4*>(q_row + ((c ^ quad) << 4));
            *x = bf16_f16(*x, rs.to);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) q_back[nr][j] = __shfl_sync(0xffffffffu, rs.back, 4 * (q2 + j));
        }
        __syncwarp();
      }
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int c = 0; c < C16; c += 4) {
          if constexpr (KV8) {  // two steps of 16 elements of d
#pragma unroll
            for (int i = 0; i < 2; ++i)
              few_queries(qf[nr][c + 2 * i], qf[nr][c + 2 * i + 1], mem + QAT + (8 * nr + quad) * (D * 2), c / 2 + i, lane & 3, quad);
          } else {
            uint32_t r[4];
            ldsm4(r, at + QAT + (8 * nr + x7) * (D * 2) + (((c + (lane >> 3)) ^ x7) << 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) qf[nr][c + i] = r[i];
          }
        }
      __syncwarp();
      ++started;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = 8 * nr + q2 + j, tk = r / p.heads, tok = pc.tok0 + tk;
          key_lo[nr][j] = key_hi[nr][j] = 0;
          if (tk < pc.ntok) {
            const int b = p.Nq == 1 ? tok : (int)((unsigned)tok / (unsigned)p.Nq);
            const int len = pc.head_kind & 1 ? pc.end : min(max(p.seq_lens[b], 0), p.max_len), pos = len - p.Nq + tok - b * p.Nq;
            key_lo[nr][j] = p.win_left >= 0 ? max(pc.lo, pos - p.win_left) : pc.lo;
            key_hi[nr][j] = min(pc.end, pos + 1);
          }
          m_ref[nr][j] = -INFINITY;
          l[nr][j] = 0.f;
        }
#pragma unroll
      for (int x = 0; x < D / 16; ++x)
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[x][nr][j] = 0.f;
      poison = 0;
    }
    // ---- a step: 16 keys
    const int j0 = (pc.lo / 16 + t) * 16;
    const uint32_t ks = at + st * 2 * TILE, vs = ks + TILE;
    ok = mbar_wait(bars + 8 * st, phase, w, 90);
    if (!__all_sync(0xffffffffu, ok)) break;
    const bool inside = j0 >= pc.all_lo && j0 + 16 <= pc.all_hi;  // every row sees every key
    if (!KV8 && !inside) {
      // 0 times a NaN or an infinity is not 0: what no row sees (it may be anything) counts as
      // zero; a value row that some see, and that holds one, counts as zero too, and its
      // rows get a NaN.
      const int kk = lane >> 1, key = j0 + kk;  // two lanes a key
      const bool out = key < pc.lo || key >= pc.end, some = !out && (key < pc.all_lo || key >= pc.all_hi);
      uint4* v = reinterpret_cast<uint4*>(mem + st * 2 * TILE + TILE + (kk >> 3) * CH * 1024 + (kk & 7) * 128);
      uint32_t bad = 0;
      if (some) {
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i) {
          const int c = (lane & 1) * 4 * CH + i;
          const uint4 x = v[(c >> 3) * 64 + (c & 7)];
          bad |= __vcmpeq2(x.x & 0x7f807f80u, 0x7f807f80u) | __vcmpeq2(x.y & 0x7f807f80u, 0x7f807f80u) |
                 __vcmpeq2(x.z & 0x7f807f80u, 0x7f807f80u) | __vcmpeq2(x.w & 0x7f807f80u, 0x7f807f80u);
        }
      }
      uint32_t odd = __ballot_sync(0xffffffffu, bad != 0);  // bit 2 key: either of its lanes
      odd = (odd | odd >> 1) & 0x55555555u;
      if (odd) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int a = min(max(key_lo[nr][j] - j0, 0), 16), z = min(max(key_hi[nr][j] - j0, 0), 16);
            const uint32_t sees = z > a ? (0xffffffffu >> (32 - 2 * (z - a))) << (2 * a) : 0u;
            if (odd & sees) poison |= 1u << (2 * nr + j);
          }
      }
      if (out || (odd >> (2 * kk) & 1)) {
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i) {
          const int c = (lane & 1) * 4 * CH + i;
          v[(c >> 3) * 64 + (c & 7)] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();  // (the copy that fills the place next comes behind these writes)
      __syncwarp();
    }
    float s[NR][2][4];  // two chains of dependent products
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[nr][0][j] = s[nr][1][j] = 0.f;
    uint4 kc[KV8 ? 2 : 1][KV8 ? CH : 1];  // codes: a key's chunks lane & 3 and, d = 128, 4 behind it
    float mul = sl2, v_mul = 1.f, lv = 0.f;  // lv: of the value scale, less the reference's own
    uint32_t odd = 0;  // 16 keys with values to poison who sees them
    if constexpr (KV8) {
      const float2 sc = s_scale[st];
      mul = sl2 * sc.x, v_mul = sc.y;
      lv = scale_log2(v_mul) - kAtRefLog2;
      if (!(fabsf(v_mul) < INFINITY)) v_mul = 0.f, odd = 0xffffu;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const int key = quad + 8 * h, c = (lane & 3) + 4 * j;
          kc[h][j] = *reinterpret_cast<const uint4*>(mem + st * 2 * TILE + key * D + ((c ^ (D == 128 ? key & 7 : key >> 1 & 3)) << 4));
        }
    }
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      uint32_t a[4];
      if constexpr (KV8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4& c = kc[h][x >> 2];
          const uint32_t word = (x & 3) == 0 ? c.x : (x & 3) == 1 ? c.y : (x & 3) == 2 ? c.z : c.w;
          codes_f16(word, a[h], a[2 + h]);
        }
      } else
        ldsm4(a, ks + k_row + (x >> 2) * 1024 + (((2 * (x & 3) + (lane >> 4)) ^ x7) << 4));
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) mma16816<KV8>(s[nr][x % 2], a, qf[nr][2 * x], qf[nr][2 * x + 1]);
    }
    bool moves = false;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
      for (int j = 0; j < 4; ++j) s[nr][0][j] = (s[nr][0][j] + s[nr][1][j]) * (KV8 ? mul * q_back[nr][j & 1] : mul);
      if (!inside) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = j0 + quad + 8 * (j >> 1);
          if (key < key_lo[nr][j & 1] || key >= key_hi[nr][j & 1]) s[nr][0][j] = -INFINITY;
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) moves |= fmaxf(s[nr][0][j], s[nr][0][j + 2]) + lv > m_ref[nr][j] + tau;
    }
    if (__any_sync(0xffffffffu, moves)) {  // some row's reference moves: O, l *= alpha
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float m = fmaxf(s[nr][0][j], s[nr][0][j + 2]);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
          m += lv;
          if (m > m_ref[nr][j] + tau) {
            const float half = KV8 ? ex2_sfu(0.5f * (m_ref[nr][j] - m)) : 1.f;  // (as for tiles)
            const float alpha = KV8 ? half * half : ex2_sfu(m_ref[nr][j] - m);
            m_ref[nr][j] = m;
            l[nr][j] = KV8 ? l[nr][j] * half * half : l[nr][j] * alpha;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) o[x][nr][j] *= alpha, o[x][nr][j + 2] *= alpha;
          }
        }
    }
    uint32_t pb[NR][2];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      float e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float m = m_ref[nr][j & 1] == -INFINITY ? 0.f : m_ref[nr][j & 1];
        e[j] = ex2_sfu(s[nr][0][j] - m);
      }
      l[nr][0] += e[0] + e[2];
      l[nr][1] += e[1] + e[3];
      if constexpr (KV8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] *= v_mul;
      }
      pb[nr][0] = transpose8(KV8 ? pack_f16x2(e[0], e[1]) : pack_bf16x2(e[0], e[1]));
      pb[nr][1] = transpose8(KV8 ? pack_f16x2(e[2], e[3]) : pack_bf16x2(e[2], e[3]));
    }
    uint32_t vc[4], nan_v[2] = {0, 0};
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      uint32_t a[4];
      if constexpr (KV8) {
        // pairs of codes, transposed by two chunks: of a chunk, d = 2 quad is row quad of O^T's
        // tile, d = 2 quad + 1 row quad + 8
        if (x % 2 == 0) {
          const int key = (lane >> 3 & 1) * 8 + (lane & 7), c = x + (lane >> 4);
          ldsm4t(vc, vs + key * D + ((c ^ (D == 128 ? key & 7 : key >> 1 & 3)) << 4));
          if (!inside) {  // (0 times a NaN is not 0)
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const uint32_t nan = __vcmpeq4(vc[h] & 0x7f7f7f7fu, 0x7f7f7f7fu);
              vc[h] &= ~nan;
              nan_v[h & 1] |= nan;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) codes_f16(__byte_perm(vc[2 * (x % 2) + h], 0u, 0x3120), a[2 * h], a[2 * h + 1]);
      } else
        ldsm4t(a, vs + v_row + (x >> 2) * 1024 + (((2 * (x & 3) + (lane >> 3 & 1)) ^ x7) << 4));
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) mma16816<KV8>(o[x][nr], a, pb[nr][0], pb[nr][1]);
    }
    if (KV8 && (odd != 0 || (!inside && __any_sync(0xffffffffu, (nan_v[0] | nan_v[1]) != 0)))) {
      // a NaN among values that not all rows see, or a value scale that is no number, is a NaN
      // in all elements of the rows that see it
#pragma unroll
      for (int h = 0; h < 2; ++h)
        odd |= ((nan_v[h] & 0xffffu ? 1u : 0u) | (nan_v[h] >> 16 ? 2u : 0u)) << (8 * h + q2);
      odd = __reduce_or_sync(0xffffffffu, odd);
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int a = min(max(key_lo[nr][j] - j0, 0), 16), z = min(max(key_hi[nr][j] - j0, 0), 16);
          const uint32_t sees = z > a ? (0xffffu >> (16 - (z - a))) << a : 0u;
          if (odd & sees) poison |= 1u << (2 * nr + j);
        }
    }
    __syncwarp();  // every lane has read the step
    ++done;
    if (++st == NST) st = 0, phase ^= 1u;
    if (++t < pc.t1) continue;
    // ---- results of the piece
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = l[nr][j];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int r = 8 * nr + q2 + j;
        if (r >= pc.ntok * p.heads) continue;
        const int tk = r / p.heads, kind = pc.head_kind & 1;
        const long long rows = (long long)p.B * p.Nq * p.Hq;
        const long long place = pc.slot < 0 ? 2 * kind * rows + (long long)(pc.tok0 + tk) * p.Hq + (pc.head_kind >> 1) * p.heads + r - tk * p.heads
                                            : cut_place(p, true, pc.slot >> 1, pc.slot & 1) + r;
        // sum = 0: the row sees none of these keys (a NaN passes through)
        if (quad == 0) p.part_lse[place] = sum == 0.f ? -INFINITY : m_ref[nr][j] + __log2f(sum);
        if (sum == 0.f) continue;
        const float inv = poison >> (2 * nr + j) & 1 ? __uint_as_float(0x7fffffffu) : 1.f / sum;
        float* dst = p.part_o + place * D;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const float a = o[x][nr][j] * inv, b = o[x][nr][j + 2] * inv;
          if constexpr (KV8) *reinterpret_cast<float2*>(dst + 16 * x + 2 * quad) = make_float2(a, b);
          else dst[16 * x + quad] = a, dst[16 * x + quad + 8] = b;
        }
      }
  }
  if (!ok) {  // let copies already in flight land before the CTA's shared memory goes away
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
}
