// Block tables, positions and cache slots of one step's new tokens, built on the GPU
// from request lengths and a list of free pages.
//
// With need_b = ceil((len_b + new_b) / 16) - ceil(len_b / 16), P_b and T_b the sums of
// need and new over the sequences before b: sequence b takes the pages
// free[count - 1 - P_b - i], i < need_b, and the token rows T_b ... T_b + new_b - 1.
//
// Each CTA of a cluster scans all lengths (a few thousand at most) into its own shared
// memory; the cluster then meets, so that the lengths and the page count may be written in
// place, and its threads share the new pages, each finding its sequence by binary search.
// Few token rows are dealt with by the same (one) CTA; many by a second grid over all SMs,
// which reads what the first has written.  Bound by latency: 4.0-4.2 us for 64 sequences of
// one token, 7.5-8.1 us for 301 with 262 k rows (one cluster for all: 24.1 us).
#include <algorithm>

#include "fa_internal.h"
#include "ptx_sm100.cuh"
#include "../../include/fa.h"

namespace fa {
namespace {

constexpr int kRowThreads = 512;
constexpr int kPage = 16;
constexpr int kClusterMax = 8;          // portable cluster size
// Token rows that the scanning CTA deals with by itself: 2048 rows 7.1 us so and 7.5 with
// the second grid, 3200 7.5 and 7.5, 8192 11.8 and 9.5; a second launch costs the host 2 us.
constexpr int kTokensOneCta = 4096;

struct ExtendParams {
  int32_t* table;
  const int32_t *lens, *news, *free_pages, *free_count;
  int32_t *lens_out, *free_count_out, *cu, *positions;
  long long* slots;
  int B, max_pages, num_pages, max_tokens;
  bool rows;             // write the token rows too
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

// The pool slot of position pos on page id; an id outside the pool is flagged.
__device__ __forceinline__ long long slot_of(const ExtendParams& p, int id, int pos) {
  if (id >= 0 && id < p.num_pages) return static_cast<long long>(id) * kPage + pos % kPage;
  atomicOr(p.err, kErrBadIndex);
  return -1;
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

template <int THREADS>
__global__ void __launch_bounds__(THREADS) fa_extend_pages_kernel(const ExtendParams p) {
  constexpr int WARPS = THREADS / 32;
  extern __shared__ int sm[];
  int* tok0 = sm;                        // [B] first token row of each sequence
  int* pg0 = sm + p.B;                   // [B] pages taken before it
  int* len0 = sm + 2 * p.B;              // [B] cached length
  __shared__ long long warp_tok[WARPS], warp_pg[WARPS];
  __shared__ long long carry_tok, carry_pg;
  __shared__ unsigned total_tok, total_pg;             // of the admitted sequences
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool lead = blockIdx.x == 0;
  pdl_launch_dependents();               // (the rows' grid waits for this one's results)
  int count = __ldcg(p.free_count);
  int next_len = 0, next_add = 0;        // the next pass's, on their way
  if (tid < p.B) {
    next_len = __ldcg(p.lens + tid);
    next_add = __ldcg(p.news + tid);
  }
  // a count outside the list is flagged and leaves nothing to take
  if (count < 0 || count > p.num_pages) {
    if (lead && tid == 0) atomicOr(p.err, kErrBadIndex);
    count = 0;
  }
  if (tid == 0) {
    carry_tok = carry_pg = 0;
    total_tok = total_pg = 0;
  }
  const long long cap = static_cast<long long>(p.max_pages) * kPage;
  for (int base = 0; base < p.B; base += THREADS) {
    const int b = base + tid;
    const int len = next_len;
    int add = next_add, need = 0;
    next_len = next_add = 0;
    if (b + THREADS < p.B) {
      next_len = __ldcg(p.lens + b + THREADS);
      next_add = __ldcg(p.news + b + THREADS);
    }
    if (b < p.B) {
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
      long long wx = lane < WARPS ? warp_tok[lane] : 0, wy = lane < WARPS ? warp_pg[lane] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long xu = __shfl_up_sync(0xffffffffu, wx, d);
        const long long yu = __shfl_up_sync(0xffffffffu, wy, d);
        if (lane >= d) {
          wx += xu;
          wy += yu;
        }
      }
      if (lane < WARPS) {
        warp_tok[lane] = wx;
        warp_pg[lane] = wy;
      }
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
      } else {
        tok0[b] = -1;                    // set to the totals below
        if (lead) atomicOr(p.err, kErrNoPages);
      }
    }
    // (admitted sums fit 31 bits: they are bounded by max_tokens and the count)
    const bool in = b < p.B && admitted;
    const unsigned tok_max = __reduce_max_sync(0xffffffffu, in ? static_cast<unsigned>(tok_end) : 0u);
    const unsigned pg_max = __reduce_max_sync(0xffffffffu, in ? static_cast<unsigned>(pg_end) : 0u);
    if (lane == 0) {
      atomicMax(&total_tok, tok_max);
      atomicMax(&total_pg, pg_max);
    }
    __syncthreads();
    if (tid == THREADS - 1) {
      carry_tok = tok_end;
      carry_pg = pg_end;
    }
    __syncthreads();
  }
  __syncthreads();                       // (no sequence: the loop did not meet)
  const int tokens = static_cast<int>(total_tok), pages = static_cast<int>(total_pg);
  for (int b = tid; b < p.B; b += THREADS)
    if (tok0[b] < 0) {
      tok0[b] = tokens;
      pg0[b] = pages;
    }
  cluster_sync();                        // every CTA has read the lengths and the count
  if (lead) {
    for (int b = tid; b < p.B; b += THREADS) {
      p.cu[b] = tok0[b];
      p.lens_out[b] = len0[b] + (b + 1 < p.B ? tok0[b + 1] : tokens) - tok0[b];
    }
    if (tid == 0) {
      p.cu[p.B] = tokens;
      *p.free_count_out = count - pages;
    }
  }
  // (unsigned: max_tokens may be close to 2^31)
  const unsigned step = cluster_ctas() * THREADS;
  const unsigned first = blockIdx.x * THREADS + tid;
  for (unsigned i = first; i < static_cast<unsigned>(pages); i += step) {
    const int b = owner(pg0, p.B, i);
    const int id = __ldg(p.free_pages + count - 1 - i);
    if (id < 0 || id >= p.num_pages) atomicOr(p.err, kErrBadIndex);
    p.table[static_cast<size_t>(b) * p.max_pages + pages_of(len0[b]) + i - pg0[b]] = id;
  }
  if (!p.rows) return;
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
      slot = slot_of(p, id, pos);
    }
    p.positions[i] = pos;
    p.slots[i] = slot;
  }
}

// The token rows from the offsets, lengths and tables that the first kernel wrote.
__global__ void __launch_bounds__(kRowThreads) fa_extend_rows_kernel(const ExtendParams p) {
  extern __shared__ int sm[];            // [B + 1] first token row of each sequence
  pdl_wait();
  for (int b = threadIdx.x; b <= p.B; b += kRowThreads) sm[b] = __ldcg(p.cu + b);
  __syncthreads();
  const int tokens = sm[p.B];
  const unsigned step = gridDim.x * kRowThreads;
  for (unsigned i = blockIdx.x * kRowThreads + threadIdx.x;
       i < static_cast<unsigned>(p.max_tokens); i += step) {
    int pos = 0;
    long long slot = -1;
    if (i < static_cast<unsigned>(tokens)) {
      const int b = owner(sm, p.B, i);
      pos = __ldcg(p.lens_out + b) - (sm[b + 1] - static_cast<int>(i));
      slot = slot_of(p, __ldcg(p.table + static_cast<size_t>(b) * p.max_pages + pos / kPage), pos);
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
  prm.rows = a.max_tokens <= kTokensOneCta;
  const int nsm = device_sm_count(device);
  if (nsm <= 0) return set_error(FA_ERR_CUDA, "cannot read the SM count of device %d", device);
  // Few sequences and rows: fewer threads meet sooner (64 of one token 5.9 us with 256
  // threads, 6.6 with 1024; 256 with 1024 rows 8.4 and 7.7).
  const bool few = a.B <= 256 && a.max_tokens <= 256;
  auto* kernel = few ? fa_extend_pages_kernel<256> : fa_extend_pages_kernel<1024>;
  int rc = FA_OK;
  if (!few)
    rc = raise_smem_limit(reinterpret_cast<const void*>(kernel),
                          3 * kMaxExtendSeqs * static_cast<int>(sizeof(int)), device, kSmemExtend);
  if (rc == FA_OK && !prm.rows)
    rc = raise_smem_limit(reinterpret_cast<const void*>(fa_extend_rows_kernel),
                          (kMaxExtendSeqs + 1) * static_cast<int>(sizeof(int)), device,
                          kSmemExtendRows);
  if (rc != FA_OK) return rc;
  const int ctas = prm.rows ? 1 : kClusterMax;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(few ? 256 : 1024);
  cfg.dynamicSmemBytes = 3 * a.B * static_cast<int>(sizeof(int));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, prm);
  if (e == cudaSuccess && !prm.rows) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    // (max_tokens > 0 here, and close to 2^31 at most: nothing is added to it)
    cfg.gridDim = dim3(std::min(1 + (a.max_tokens - 1) / kRowThreads, 2 * nsm));
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = (a.B + 1) * static_cast<int>(sizeof(int));
    e = cudaLaunchKernelEx(&cfg, fa_extend_rows_kernel, prm);
  }
  if (e != cudaSuccess)
    return set_error(FA_ERR_CUDA, "page extension launch: %s", cudaGetErrorString(e));
  return FA_OK;
}

}  // namespace fa
