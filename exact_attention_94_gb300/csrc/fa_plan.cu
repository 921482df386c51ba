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
// The step is bound by latency: a few thousand integers in, 12 bytes out per
// row.  So one launch does all of it.  Every CTA scans all requests for itself
// (the sums stay in its shared memory; nothing passes between CTAs through
// device memory) and serves every k-th block of 1024 rows.  The CTAs form one
// thread-block cluster, whose barrier separates the last read of ctx_lens and
// free_count from the first write of seq_lens and free_count_out, so both may
// be updated in place.
#include "fa_internal.h"
#include "ptx.cuh"

#include <cooperative_groups.h>

namespace fa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanRows = 4;
constexpr int kPlanWarps = kPlanThreads / 32;

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

__global__ void __launch_bounds__(kPlanThreads) fa_page_plan_kernel(const PlanParams p) {
  extern __shared__ int s_mem[];
  int* s_cu = s_mem;                // [B + 1] first row of each request
  int* s_ctx = s_cu + p.B + 1;      // [B] tokens held before
  int* s_base = s_ctx + p.B;        // [B] stack position of its first new page, counted from the top
  __shared__ long long s_tok[kPlanWarps], s_need[kPlanWarps];
  __shared__ int s_free;

  const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
  const auto cluster = cooperative_groups::this_cluster();
  const int rank = (int)blockIdx.x, ranks = (int)gridDim.x;

  // ---- sums over the requests: thread t takes requests t*k .. t*k + k - 1
  const int k = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(p.B, tid * k), b1 = min(p.B, b0 + k);
  long long tok = 0, need = 0;
  bool bad = false;
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
  if (tid == 0) s_free = *p.free_count;
  const long long tok_in = warp_incl_sum(tok, lane), need_in = warp_incl_sum(need, lane);
  if (lane == 31) {
    s_tok[warp] = tok_in;
    s_need[warp] = need_in;
  }
  const bool any_bad = __syncthreads_or(bad);
  long long tok0 = tok_in - tok, need0 = need_in - need, tok_all = 0, need_all = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
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
  // every CTA has read the lengths and the count: they may be overwritten now
  if (ranks > 1)
    cluster.sync();
  else
    __syncthreads();

  if (rank == 0) {
    for (int b = tid; b <= p.B; b += kPlanThreads) {
      p.cu_new[b] = ok ? s_cu[b] : 0;
      if (b < p.B) p.seq_lens[b] = s_ctx[b] + (ok ? s_cu[b + 1] - s_cu[b] : 0);
    }
    if (tid == 0) {
      *p.free_count_out = ok ? free_n - (int)need_all : free_n;
      if (!ok) atomicCAS(p.err, 0u, code);
    }
  }

  // ---- rows, kPlanRows of a thread at a time: their searches and page loads overlap
  const int total = s_cu[p.B];
  const long long step = (long long)ranks * kPlanThreads;
  for (long long r0 = (long long)rank * kPlanThreads + tid; r0 < p.max_tokens; r0 += step * kPlanRows) {
    int page[kPlanRows], slot[kPlanRows], pos[kPlanRows], lo[kPlanRows], hi[kPlanRows];
    int* entry[kPlanRows];
#pragma unroll
    for (int x = 0; x < kPlanRows; ++x) lo[x] = 0, hi[x] = p.B - 1;
    for (int n = p.B; n > 1; n = (n + 1) >> 1) {  // the last request whose first row is at most this one
#pragma unroll
      for (int x = 0; x < kPlanRows; ++x) {
        const int mid = (lo[x] + hi[x] + 1) >> 1;
        const bool up = s_cu[mid] <= r0 + x * step;
        lo[x] = up ? mid : lo[x];
        hi[x] = up ? hi[x] : max(lo[x], mid - 1);
      }
    }
#pragma unroll
    for (int x = 0; x < kPlanRows; ++x) {
      page[x] = slot[x] = -1;
      pos[x] = 0;
      entry[x] = nullptr;
      if (r0 + x * step < total) {
        const int ctx = s_ctx[lo[x]];
        pos[x] = ctx + (int)(r0 + x * step) - s_cu[lo[x]];
        const int blk = (int)((unsigned)pos[x] / (unsigned)p.page_size), held = div_up(ctx, p.page_size);
        slot[x] = pos[x] - blk * p.page_size;
        entry[x] = p.block_table + (size_t)lo[x] * p.max_blocks + blk;
        page[x] = *(blk < held ? entry[x] : p.free_pages + (free_n - 1 - (s_base[lo[x]] + blk - held)));
      }
    }
#pragma unroll
    for (int x = 0; x < kPlanRows; ++x) {
      const long long row = r0 + x * step;
      if (row >= p.max_tokens) break;
      if (entry[x] != nullptr) {
        if (page[x] < 0 || page[x] >= p.num_pages) {
          atomicCAS(p.err, 0u, FA_DEVERR_BAD_PAGE);
          page[x] = slot[x] = -1;
        } else if (slot[x] == 0) {
          *entry[x] = page[x];  // the first token of a new page
        }
      }
      p.page[row] = page[x];
      p.slot[row] = slot[x];
      p.position[row] = pos[x];
    }
  }
}

cudaError_t launch_page_plan(const PlanParams& p, cudaStream_t stream) {
  const size_t smem = (3 * (size_t)p.B + 1) * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(fa_page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  if (p.max_tokens <= 4 * kPlanThreads) {
    fa_page_plan_kernel<<<1, kPlanThreads, smem, stream>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(8);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = cfg.gridDim.x;
  a.val.clusterDim.y = a.val.clusterDim.z = 1;
  cfg.attrs = &a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_page_plan_kernel, p);
}

}  // namespace fa
