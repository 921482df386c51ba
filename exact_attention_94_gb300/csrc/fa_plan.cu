// Planning a serving step on the GPU: block tables, slot maps and packed
// offsets from the requests' lengths ("efficient-attention/flash-2-3",
// section "Paged KV caches, a preview of serving": a block table maps a
// sequence's logical blocks to pages, and a page is taken from the free list
// only when the last one fills).
//
// With c_b cached and n_b new tokens and pages of P:
//     need_b = ceil((c_b + n_b) / P) - ceil(c_b / P)
//     cu = exclusive sum of n,  base = exclusive sum of need
//     token c_b + i of request b: row cu_b + i, block (c_b + i) / P, whose page
//     is the table's for a block held before, else
//     free[count - 1 - (base_b + block - ceil(c_b / P))].
// A few thousand integers come in, 12 bytes go out per row; the step is bound by
// latency: a launch, two barriers and three reads one after the other (lengths,
// free page, its entry).  256 requests of a token take 3.4 us, where a kernel that
// does next to nothing takes 2.8; the 1.5 MB of 61 prompts take 5.4.
//
// Every CTA scans all requests for itself (the sums stay in its shared memory;
// nothing passes between CTAs) and serves its part of the rows.  One CTA does a
// step of few rows.  Where there are many, the CTAs that read ctx_lens and
// free_count have no order among themselves, so seq_lens and free_count_out,
// where they are the same arrays, are then written by a second launch of one
// CTA, from cu_new and the old count.
#include "serving.cuh"

namespace fa {

namespace {

// a / b rounded up, for a >= 0, b > 0, without a 64-bit division
__device__ __forceinline__ int div_up(int a, int b) {
  const unsigned q = (unsigned)a / (unsigned)b;
  return (int)(q + (q * (unsigned)b != (unsigned)a ? 1u : 0u));
}

__device__ __forceinline__ long long warp_incl_sum(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

}  // namespace

template <int THREADS>
__global__ void __launch_bounds__(THREADS) fa_page_plan_kernel(const PlanParams p) {
  constexpr int WARPS = THREADS / 32;
  extern __shared__ int s_mem[];
  int* s_cu = s_mem;                // [B + 1] first row of each request
  int* s_ctx = s_cu + p.B + 1;      // [B] tokens held before
  int* s_base = s_ctx + p.B;        // [B] stack position of its first new page, counted from the top
  __shared__ long long s_tok[WARPS], s_need[WARPS];
  __shared__ int s_free;

  const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;

  // ---- sums over the requests: thread t takes requests t*k .. t*k + k - 1
  const int k = (p.B + THREADS - 1) / THREADS;
  const int b0 = min(p.B, tid * k), b1 = min(p.B, b0 + k);
  long long tok = 0, need = 0;
  bool bad = false;
  if (tid == 0) s_free = *p.free_count;
  for (int b = b0; b < b1; ++b) {
    int c = p.ctx_lens[b], n = p.new_lens[b];
    s_ctx[b] = c;
    if (c < 0 || n < 0 || (long long)c + n > (long long)p.max_blocks * p.page_size || (long long)c + n > 0x7fffffffll) {
      bad = true;
      c = n = 0;
    }
    s_cu[b] = (int)min(tok, 0x7fffffffll);
    s_base[b] = (int)min(need, 0x7fffffffll);
    tok += n;
    need += div_up(c + n, p.page_size) - div_up(c, p.page_size);
  }
  const long long tok_in = warp_incl_sum(tok, lane), need_in = warp_incl_sum(need, lane);
  if (lane == 31) {
    s_tok[warp] = tok_in;
    s_need[warp] = need_in;
  }
  const bool any_bad = __syncthreads_or(bad);
  long long tok0 = tok_in - tok, need0 = need_in - need, tok_all = 0, need_all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) {
      tok0 += s_tok[w];
      need0 += s_need[w];
    }
    tok_all += s_tok[w];
    need_all += s_need[w];
  }
  const int free_n = s_free;
  unsigned code = 0;
  if (any_bad || tok_all > p.max_tokens || free_n < 0 || free_n > p.num_pages)
    code = FA_DEVERR_BAD_SEQLEN;
  else if (need_all > free_n)
    code = FA_DEVERR_OUT_OF_PAGES;
  const bool ok = code == 0;
  if (ok) {  // otherwise nothing below reads the sums
    for (int b = b0; b < b1; ++b) {
      s_cu[b] += (int)tok0;
      s_base[b] += (int)need0;
    }
  }
  if (tid == 0) s_cu[p.B] = ok ? (int)tok_all : 0;
  __syncthreads();

  if (blockIdx.x == 0) {
    for (int b = tid; b <= p.B; b += THREADS) {
      p.cu_new[b] = ok ? s_cu[b] : 0;
      if (b < p.B && !p.totals_later) p.seq_lens[b] = s_ctx[b] + (ok ? s_cu[b + 1] - s_cu[b] : 0);
    }
    if (tid == 0) {
      if (!p.totals_later) *p.free_count_out = ok ? free_n - (int)need_all : free_n;
      if (!ok) atomicCAS(p.err, 0u, code);
    }
  }

  // ---- rows
  const int total = s_cu[p.B];
  for (long long row = (long long)blockIdx.x * THREADS + tid; row < p.max_tokens; row += (long long)gridDim.x * THREADS) {
    int page = -1, slot = -1, pos = 0;
    if (row < total) {
      int lo = 0, hi = p.B - 1;  // the last request whose first row is at most this one
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_cu[mid] <= row)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int ctx = s_ctx[lo];
      pos = ctx + (int)row - s_cu[lo];
      const int blk = (int)((unsigned)pos / (unsigned)p.page_size), held = div_up(ctx, p.page_size);
      slot = pos - blk * p.page_size;
      int* entry = p.block_table + (size_t)lo * p.max_blocks + blk;
      page = blk < held ? *entry : p.free_pages[free_n - 1 - (s_base[lo] + blk - held)];
      if (page < 0 || page >= p.num_pages) {
        atomicCAS(p.err, 0u, FA_DEVERR_BAD_PAGE);
        page = slot = -1;
      } else if (slot == 0) {
        *entry = page;  // the first token of a new page
      }
    }
    p.page[row] = page;
    p.slot[row] = slot;
    p.position[row] = pos;
  }
}

// The lengths and the free count after a step whose rows many CTAs have written.
__global__ void __launch_bounds__(1024) fa_page_plan_totals_kernel(const PlanParams p) {
  long long need = 0;
  for (int b = threadIdx.x; b < p.B; b += 1024) {
    const int c = p.ctx_lens[b], n = p.cu_new[b + 1] - p.cu_new[b];  // (a refused step: n = 0, any c)
    p.seq_lens[b] = c + n;
    if (n > 0) need += div_up(c + n, p.page_size) - div_up(c, p.page_size);
  }
  __shared__ long long s_need[32];
  const long long in_warp = warp_incl_sum(need, lane_id());
  if (lane_id() == 31) s_need[threadIdx.x >> 5] = in_warp;
  __syncthreads();
  if (threadIdx.x == 0) {
    long long all = 0;
    for (int w = 0; w < 32; ++w) all += s_need[w];
    *p.free_count_out = *p.free_count - (int)all;
  }
}

static constexpr size_t plan_smem(int B) { return (3 * (size_t)B + 1) * sizeof(int); }

template <int THREADS>
static cudaError_t launch_page_plan_t(const PlanParams& p, int ctas, cudaStream_t stream) {
  const size_t smem = plan_smem(p.B);
  // More than the 48 KiB that every launch may have, less the kernel's static
  // part, is asked for, and always as much as the largest batch takes: the limit
  // belongs to the process, and a call on another thread may set it between here
  // and the launch.
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(fa_page_plan_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)plan_smem(kPlanMaxB));
    if (e != cudaSuccess) return e;
  }
  fa_page_plan_kernel<THREADS><<<ctas, THREADS, smem, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_page_plan(PlanParams& p, cudaStream_t stream) {
  // One small CTA for few rows: it starts and synchronises sooner (256 requests of
  // a token: 3.5 us, and 5.1 with 1024 threads; 1024 requests 6.8 and 6.5).  CTAs of
  // 1024 rows for more (2048 requests 7.0 us, and 8.4 in one CTA; the 126,000 rows
  // of 61 prompts 5.4 and 108).
  if (p.max_tokens <= 1024 && p.B <= 1024) {
    p.totals_later = 0;
    return launch_page_plan_t<256>(p, 1, stream);
  }
  const int ctas = (p.max_tokens - 1) / 1024 + 1;  // (1 for no rows)
  p.totals_later = ctas > 1 && (p.seq_lens == p.ctx_lens || p.free_count_out == p.free_count);
  const cudaError_t e = launch_page_plan_t<1024>(p, ctas < 2 * kSms ? ctas : 2 * kSms, stream);
  if (e != cudaSuccess || !p.totals_later) return e;
  fa_page_plan_totals_kernel<<<1, 1024, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
