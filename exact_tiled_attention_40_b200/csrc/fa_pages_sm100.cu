// Block tables, positions and cache slots of one step's new tokens, built on the GPU
// from request lengths and a list of free pages.
//
// With need_b = ceil((len_b + new_b) / 16) - ceil(len_b / 16), P_b and T_b the sums of
// need and new over the sequences before b: sequence b takes the pages
// free[count - 1 - P_b - i], i < need_b, and the token rows T_b ... T_b + new_b - 1.
//
// One launch.  Each CTA of the cluster scans all lengths (a few thousand at most) into
// its own shared memory; the cluster then meets, so that the lengths and the page count
// may be written in place, and its threads share the new pages and the token rows, each
// finding its sequence by binary search.  Few tokens: one CTA, bound by the latency of
// one scan.
#include <algorithm>

#include "fa_internal.h"
#include "ptx_sm100.cuh"
#include "../../include/fa.h"

namespace fa {
namespace {

constexpr int kThreads = 1024;
constexpr int kPage = 16;
constexpr int kClusterMax = 8;          // portable cluster size
constexpr int kTokensOneCta = 4096;     // token rows that one CTA deals with by itself

struct ExtendParams {
  int32_t* table;
  const int32_t *lens, *news, *free_pages, *free_count;
  int32_t *lens_out, *free_count_out, *cu, *positions;
  long long* slots;
  int B, max_pages, num_pages, max_tokens;
  int* err;
};

__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }

// Largest b in [0, n) with start[b] <= x (start[0] <= x, non-decreasing): the sequence
// that owns item x, empty ones before it skipped.
__device__ __forceinline__ int owner(const int* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_ctas() {
  unsigned n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}

__global__ void __launch_bounds__(kThreads) fa_extend_pages_kernel(const ExtendParams p) {
  extern __shared__ int sm[];
  int* tok0 = sm;                        // [B] first token row of each sequence
  int* pg0 = sm + p.B;                   // [B] pages taken before it
  int* len0 = sm + 2 * p.B;              // [B] cached length
  __shared__ long long warp_tok[32], warp_pg[32];
  __shared__ long long carry_tok, carry_pg;
  __shared__ unsigned long long total_tok, total_pg;   // of the admitted sequences
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool lead = blockIdx.x == 0;
  // a count outside the list is flagged and leaves nothing to take
  int count = __ldcg(p.free_count);
  if (count < 0 || count > p.num_pages) {
    if (lead && tid == 0) atomicOr(p.err, kErrBadIndex);
    count = 0;
  }
  if (tid == 0) {
    carry_tok = carry_pg = 0;
    total_tok = total_pg = 0;
  }
  __syncthreads();
  const long long cap = static_cast<long long>(p.max_pages) * kPage;
  for (int base = 0; base < p.B; base += kThreads) {
    const int b = base + tid;
    int len = 0, add = 0, need = 0;
    if (b < p.B) {
      len = __ldcg(p.lens + b);
      add = __ldcg(p.news + b);
      if (len < 0 || add < 0 || static_cast<long long>(len) + add > cap) {
        if (lead) atomicOr(p.err, kErrBadIndex);
        add = 0;                         // the sequence stays as it is
      } else {
        need = pages_of(len + add) - pages_of(len);
      }
    }
    long long x = add, y = need;         // inclusive warp scans
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long xu = __shfl_up_sync(0xffffffffu, x, d);
      const long long yu = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) {
        x += xu;
        y += yu;
      }
    }
    if (lane == 31) {
      warp_tok[warp] = x;
      warp_pg[warp] = y;
    }
    __syncthreads();
    if (warp == 0) {
      long long wx = warp_tok[lane], wy = warp_pg[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long xu = __shfl_up_sync(0xffffffffu, wx, d);
        const long long yu = __shfl_up_sync(0xffffffffu, wy, d);
        if (lane >= d) {
          wx += xu;
          wy += yu;
        }
      }
      warp_tok[lane] = wx;
      warp_pg[lane] = wy;
    }
    __syncthreads();
    const long long tok_end = carry_tok + (warp > 0 ? warp_tok[warp - 1] : 0) + x;
    const long long pg_end = carry_pg + (warp > 0 ? warp_pg[warp - 1] : 0) + y;
    // both sums only grow: from the first sequence that does not fit on, none does
    const bool admitted = tok_end <= p.max_tokens && pg_end <= count;
    if (b < p.B) {
      len0[b] = len;
      if (admitted) {
        tok0[b] = static_cast<int>(tok_end - add);
        pg0[b] = static_cast<int>(pg_end - need);
        atomicMax(&total_tok, static_cast<unsigned long long>(tok_end));
        atomicMax(&total_pg, static_cast<unsigned long long>(pg_end));
      } else {
        tok0[b] = -1;                    // set to the totals below
        if (lead) atomicOr(p.err, kErrNoPages);
      }
    }
    __syncthreads();
    if (tid == kThreads - 1) {
      carry_tok = tok_end;
      carry_pg = pg_end;
    }
    __syncthreads();
  }
  const int tokens = static_cast<int>(total_tok), pages = static_cast<int>(total_pg);
  for (int b = tid; b < p.B; b += kThreads)
    if (tok0[b] < 0) {
      tok0[b] = tokens;
      pg0[b] = pages;
    }
  cluster_sync();                        // every CTA has read the lengths and the count
  if (lead) {
    for (int b = tid; b < p.B; b += kThreads) {
      p.cu[b] = tok0[b];
      p.lens_out[b] = len0[b] + (b + 1 < p.B ? tok0[b + 1] : tokens) - tok0[b];
    }
    if (tid == 0) {
      p.cu[p.B] = tokens;
      *p.free_count_out = count - pages;
    }
  }
  // (unsigned: max_tokens may be close to 2^31)
  const unsigned step = cluster_ctas() * kThreads;
  const unsigned first = blockIdx.x * kThreads + tid;
  for (unsigned i = first; i < static_cast<unsigned>(pages); i += step) {
    const int b = owner(pg0, p.B, i);
    const int id = __ldg(p.free_pages + count - 1 - i);
    if (id < 0 || id >= p.num_pages) atomicOr(p.err, kErrBadIndex);
    p.table[static_cast<size_t>(b) * p.max_pages + pages_of(len0[b]) + i - pg0[b]] = id;
  }
  for (unsigned i = first; i < static_cast<unsigned>(p.max_tokens); i += step) {
    int pos = 0;
    long long slot = -1;
    if (i < static_cast<unsigned>(tokens)) {
      const int b = owner(tok0, p.B, i);
      const int len = len0[b];
      pos = len + i - tok0[b];
      const int pg = pos / kPage, own = pages_of(len);
      // a page that the sequence had (only its last, part-filled one can be) or a new one
      const int id = pg < own ? __ldcg(p.table + static_cast<size_t>(b) * p.max_pages + pg)
                              : __ldg(p.free_pages + count - 1 - pg0[b] - (pg - own));
      if (id < 0 || id >= p.num_pages)
        atomicOr(p.err, kErrBadIndex);
      else
        slot = static_cast<long long>(id) * kPage + pos % kPage;
    }
    p.positions[i] = pos;
    p.slots[i] = slot;
  }
}

}  // namespace

int launch_extend_pages(const ExtendArgs& a, cudaStream_t stream, int device) {
  ExtendParams prm;
  prm.table = a.block_table;
  prm.lens = a.seq_lens;
  prm.news = a.new_lens;
  prm.free_pages = a.free_pages;
  prm.free_count = a.free_count;
  prm.lens_out = a.seq_lens_out;
  prm.free_count_out = a.free_count_out;
  prm.cu = a.cu_seqlens_q;
  prm.positions = a.positions;
  prm.slots = reinterpret_cast<long long*>(a.slot_map);
  prm.B = a.B;
  prm.max_pages = a.max_pages_per_seq;
  prm.num_pages = a.num_pages;
  prm.max_tokens = a.max_tokens;
  prm.err = device_error_word(device);
  if (!prm.err) return set_error(FA_ERR_CUDA, "device error word unavailable");
  const int ctas = a.max_tokens <= kTokensOneCta ? 1 : kClusterMax;
  const int smem = 3 * a.B * static_cast<int>(sizeof(int));
  int rc = raise_smem_limit(reinterpret_cast<const void*>(fa_extend_pages_kernel),
                            3 * kMaxExtendSeqs * static_cast<int>(sizeof(int)), device,
                            kSmemExtend);
  if (rc != FA_OK) return rc;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fa_extend_pages_kernel, prm);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    return set_error(FA_ERR_CUDA, "page extension launch: %s", cudaGetErrorString(e));
  return FA_OK;
}

}  // namespace fa
