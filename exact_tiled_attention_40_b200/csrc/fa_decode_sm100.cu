// Split-KV decode over a paged KV cache for sm_100a.
//
// Decode (cabseo.com, "Advanced techniques for enhancing LLM throughput",
// sections "Memory requirements" and "Autoregressive and memory-bound
// operations") attends one new query token per sequence over the whole KV
// cache, a matrix-vector product bound by HBM bandwidth.  The cache is paged
// (section "Paged attention"): fixed pages of 16 token slots, each slot holding
// all KV heads, reached through a per-sequence block table.
//
// Within a warp each half-warp takes one token and each of its 16 lanes a
// 16-byte slice (8 elements) of the 256-byte head row.  Partial dot products for
// the G query heads that share the KV head are folded across the 16 lanes with a
// transposing butterfly (each exchange halves the number of live heads), leaving
// every lane with the full score of one head.  An online softmax (running max,
// rescale by exp2(m_old - m_new), unnormalised accumulator) runs over the keys,
// and each chunk's normalised output and LSE go to a workspace that a combine
// kernel merges by LSE -- the softmax merge of unite.ai, "Flash Attention:
// Revolutionizing Transformer Efficiency", section "The Mathematics of Flash
// Attention", formula 2.
//
// Two schedules:
//  * Hkv <= 8 (streamed): one persistent CTA per SM.  All sequences' caches form
//    one list of half-pages (8 token slots: 8 * Hkv * 256 bytes of K and as many
//    of V, each contiguous in the pool); CTA c takes the equal share
//    [c*H/C, (c+1)*H/C) of the H half-pages, whatever the sequence lengths.  A
//    producer warp streams them through a shared-memory ring with TMA tensor
//    copies (128-byte swizzle, head-major boxes); eight consumer warps (warp g <-> KV head g) compute scores and
//    outputs with warp-level tensor-core MMAs from shared memory and emit one
//    partial result per (CTA, sequence) segment, stored in
//    slot c + b (unique: along the list either c or b or both grow by one); a
//    merge kernel combines each sequence's segments.
//  * otherwise (direct): grid (chunk, sequence) of fixed page chunks, cache read
//    straight from HBM with 16-byte non-allocating loads.
//
// SHARED instantiations serve batches whose sequences share their first pages: the
// shared keys are the business of fa_prefix_sm100.cu, the kernels here stream each
// sequence's own keys behind them, and the merge joins both.  A sequence shorter than
// the shared pages does not take part: all of its keys are streamed as its own.  They
// always stream: where there are more KV heads than the 8 consumer warps, a sequence is
// cut into groups of heads that go through all kernels as sequences of their own (q, o
// and the LSE of a group are contiguous, and a stage's box starts at the group's first
// head).  33 sequences of about 150 own keys, 16 heads, 4000 shared keys: 51.0 us direct,
// 33.2 us cut in two.
#include <cstdio>
#include <cstring>
#include <algorithm>
#include <mutex>
#include <vector>

#include "fa_internal.h"
#include "prefix_split.cuh"
#include "ptx_sm100.cuh"
#include "../../include/fa.h"

namespace fa {
namespace {

constexpr int kDecD = 128;
constexpr int kPage = 16;
constexpr int kDecWarps = 8;
constexpr int kDecThreads = kDecWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;

// streamed schedule
constexpr int kHalf = 8;                        // token slots per stage
// SHARED: a stage is a page.  The consumers' chain of a stage (scores, maximum, exponents,
// weights) is what bounds a CTA, and twice the tokens lengthen it little: a page of 8 KV
// heads takes an SM 0.92 us, two half-pages 1.36 us; of 4 heads or fewer 0.68 and 1.16 us.
constexpr int stage_tokens(bool shared) { return shared ? kPage : kHalf; }
constexpr int kConsumerWarps = kDecWarps;       // one per KV head (see the stream kernel)
constexpr int kStreamThreads = 12 * 32;          // 8 consumer warps + a producer warpgroup
// Register split (setmaxnreg): the producer warpgroup (warps 8-11, one of them
// working) gives registers to the two consumer warpgroups; 40 x 128 + 224 x 256
// stays within the 384 x 168 the block is launched with.
constexpr uint32_t kRegsProducer = 48;
constexpr uint32_t kRegsConsumer = 224;
static_assert(kRegsProducer * 128 + kRegsConsumer * 256 <= 384 * 168, "register split");
constexpr int kMaxStages = 8;
constexpr int kStreamSmemBudget = 200 * 1024;
// Streamed schedule: the half-page list is split into equal contiguous shares,
// one per CTA.  The first 15/16 of each share is streamed by its own CTA; the
// last 16th is cut into units of kDynUnit half-pages that go to whichever CTA
// asks first, so CTAs that stream more slowly (SMs differ in the bandwidth they
// get) finish with the others.  Keeping each share's units next to it spreads
// them over all sequences, so no sequence collects many partials.
constexpr int kDynDiv = 16;    // 1 / kDynDiv of each share is dynamic
constexpr int kDynUnit = 8;    // half-pages per dynamic unit (at least)
// SHARED: the CTAs that the shared-prefix kernel keeps waiting only take dynamic units, and
// how long they wait is estimated, so more is dynamic where most wait: a quarter (256
// sequences of about 256 own and 32768 shared keys, where 124 of 148 wait: 168 us, 177 with
// an eighth), else a 16th (64 of about 2050 own and 4096 shared, 11 wait: 102.8 us, with a
// quarter 109.4).
constexpr int kDynDivWait = 4;
constexpr int dyn_unit(bool shared) { return shared ? 4 : kDynUnit; }
constexpr int kMaxUnitsPerCta = 4;
constexpr int kMaxStreamCtas = 204;                       // so a sequence has <= 1024 partials
constexpr int kMaxMergeSlots = kMaxStreamCtas * (1 + kMaxUnitsPerCta);
// SHARED, nothing attended together: a list of at most this many sequences, too short for
// dynamic units, is summed up by every CTA itself instead of a kernel of its own (8 + 2
// heads, us with that kernel / so: 7 sequences of 65 pages 13.4 / 11.3, 64 of 15 17.6 / 15.9,
// but 256 of 3 19.6 / 20.4).
constexpr int kScanHere = 128;
constexpr int merge_warps(bool shared) { return shared ? 8 : 32; }
constexpr int kHbSmemMax = 4096;   // sequences whose offsets the producer keeps in shared memory

struct DecodeParams {
  const uint16_t* q;
  const uint16_t* kc;
  const uint16_t* vc;
  const int32_t* block_table;
  const int32_t* seq_lens;
  uint16_t* o;
  float* lse;
  float* ws_o;     // partial outputs, [slot][Hq][128] normalised
  float* ws_lse;   // partial LSE (natural log), [slot][Hq]
  int* hb;         // streamed: hb[b] = half-pages before sequence b, hb[B] = total
  int* dyn_next;   // streamed: next dynamic unit to hand out (zeroed by the scan kernel)
  int B, Hq, Hkv, max_pages, num_pages;
  int pps, nsplit;             // direct schedule
  int nctas, nstages;          // streamed schedule
  int dyn_units_cap;           // streamed: partial slots reserved for dynamic units
  int hb_in_smem;              // streamed: the producer copies hb to shared memory
  float scale_log2;
  int* err;
  int merge_split;             // SHARED: warps of the merge that share a row (1, 2, 4 or 8)
  int groups;                  // SHARED: head groups of a sequence (B, Hq, Hkv count these)
  PrefixWork pw;               // SHARED: the shared pages and how their work is split
  const float* pre_o;          // SHARED: segments' partial outputs [slot][256][128]
  const float* pre_lse;        // SHARED: their LSE [slot][256]
  const int32_t* prefix_table; // SHARED: ids of the shared pages
  bool scan_here;              // SHARED: a short list, without a scan kernel (see kScanHere)
};

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ int checked_len(const DecodeParams& p, int b) {
  const int len = p.seq_lens[b];
  if (len < 0 || len > p.max_pages * kPage) return -1;
  return len;
}

// The sequence that entry b of the batch belongs to.
template <bool SHARED>
__device__ __forceinline__ int seq_of(const DecodeParams& p, int b) {
  return SHARED ? b / p.groups : b;
}

// The keys that sequence b does not share: their number (-1: invalid length) and the
// block-table entry they start at; `shared` is the batch's number of shared pages.
struct OwnKeys {
  int len, page0;
};
template <bool SHARED>
__device__ __forceinline__ OwnKeys own_keys(int len, int shared) {
  OwnKeys k;
  k.len = len;
  k.page0 = 0;
  if (SHARED && len >= shared * kPage) {
    k.len -= shared * kPage;
    k.page0 = shared;
  }
  return k;
}

// SHARED, short list: pages of entry b, and the CTAs that share H of them.
__device__ __forceinline__ int listed_pages(const DecodeParams& p, int b, bool flag) {
  const int len = checked_len(p, b / p.groups);
  if (len < 0 && flag) atomicOr(p.err, kErrBadIndex);
  return len < 0 ? 0 : (len + kPage - 1) / kPage;
}
__device__ __forceinline__ int short_list_ctas(const DecodeParams& p, int H) {
  return min(p.nctas, max(1, H / kOwnMinPages));
}

// Fold G partial sums held by 16 lanes (lane bits 0-3 = sub) into one full sum
// per lane: lane `sub` ends with the total of head sub >> (4 - log2 G).
template <int G>
__device__ __forceinline__ float fold_heads(float (&v)[G], int sub) {
  constexpr int LG = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : G == 8 ? 3 : 4;
#pragma unroll
  for (int step = 0; step < LG; ++step) {
    const int mask = 8 >> step;
    const bool upper = (sub & mask) != 0;
    const int n = G >> (step + 1);
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float keep = upper ? v[k + n] : v[k];
      const float send = upper ? v[k] : v[k + n];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
    }
  }
  float x = v[0];
#pragma unroll
  for (int mask = 8 >> LG; mask >= 1; mask >>= 1) x += __shfl_xor_sync(0xffffffffu, x, mask);
  return x;
}

template <int G>
__global__ void __launch_bounds__(kDecThreads) fa_decode_split_kernel(const DecodeParams p) {
  constexpr int LG = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3;
  constexpr int SHIFT = 4 - LG;       // lane `h << SHIFT` holds head h after the fold
  constexpr int NI = G >= 8 ? 4 : 8;  // token pairs per iteration
  __shared__ __align__(16) float pbuf[kDecWarps][NI][2][G];

  const int b = blockIdx.y;
  const int split = blockIdx.x;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int half = lane >> 4;
  const int sub = lane & 15;
  const int my_head = sub >> SHIFT;

  const int len = checked_len(p, b);
  if (len < 0) {
    if (threadIdx.x == 0 && split == 0) atomicOr(p.err, kErrBadIndex);
    return;
  }
  const int npages = (len + kPage - 1) / kPage;
  const int pbeg = split * p.pps;
  if (pbeg >= npages) return;
  const int pend = min(pbeg + p.pps, npages);
  const size_t tok_stride = static_cast<size_t>(p.Hkv) * kDecD;   // elements between slots

  for (int g = warp; g < p.Hkv; g += kDecWarps) {
    const int hq0 = g * G;
    float qf[G][8];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const uint4 u = *reinterpret_cast<const uint4*>(
          p.q + (static_cast<size_t>(b) * p.Hq + hq0 + h) * kDecD + sub * 8);
      bf16x8_to_f32(u, qf[h]);
#pragma unroll
      for (int e = 0; e < 8; ++e) qf[h][e] *= p.scale_log2;
    }
    float m[G], l[G], acc[G][8];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[h][e] = 0.f;
    }
    float m_mine = -INFINITY;

    for (int pg = pbeg; pg < pend; ++pg) {
      const int page = p.block_table[static_cast<size_t>(b) * p.max_pages + pg];
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicOr(p.err, kErrBadIndex);
        continue;
      }
      const int ntok = min(kPage, len - pg * kPage);
      const uint16_t* kbase = p.kc + (static_cast<size_t>(page) * kPage * p.Hkv + g) * kDecD + sub * 8;
      const uint16_t* vbase = p.vc + (static_cast<size_t>(page) * kPage * p.Hkv + g) * kDecD + sub * 8;
#pragma unroll 1
      for (int t0 = 0; t0 < kPage; t0 += 2 * NI) {
        uint4 kr[NI], vr[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int t = t0 + 2 * i + half;
          if (t < ntok) {
            kr[i] = ld_stream(kbase + t * tok_stride);
            vr[i] = ld_stream(vbase + t * tok_stride);
          } else {
            kr[i] = make_uint4(0, 0, 0, 0);
            vr[i] = make_uint4(0, 0, 0, 0);
          }
        }
        float sc[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          float kf[8];
          bf16x8_to_f32(kr[i], kf);
          float part[G];
#pragma unroll
          for (int h = 0; h < G; ++h) {
            float a = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) a = fmaf(qf[h][e], kf[e], a);
            part[h] = a;
          }
          sc[i] = fold_heads<G>(part, sub);
          if (t0 + 2 * i + half >= ntok) sc[i] = -INFINITY;
        }
        // chunk maximum of this lane's head over both half-warps' tokens
        float mx = sc[0];
#pragma unroll
        for (int i = 1; i < NI; ++i) mx = fmaxf(mx, sc[i]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float m_new_mine = fmaxf(m_mine, mx);
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float mh = fmaxf(m[h], __shfl_sync(0xffffffffu, mx, h << SHIFT));
          const float alpha = (m[h] == -INFINITY) ? 0.f : ex2(m[h] - mh);
          l[h] *= alpha;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[h][e] *= alpha;
          m[h] = mh;
        }
        m_mine = m_new_mine;
        float pv[NI];
        float psum = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          pv[i] = (sc[i] == -INFINITY) ? 0.f : ex2(sc[i] - m_mine);
          psum += pv[i];
        }
        psum += __shfl_xor_sync(0xffffffffu, psum, 16);
#pragma unroll
        for (int h = 0; h < G; ++h) l[h] += __shfl_sync(0xffffffffu, psum, h << SHIFT);
        if ((sub & ((1 << SHIFT) - 1)) == 0) {
#pragma unroll
          for (int i = 0; i < NI; ++i) pbuf[warp][i][half][my_head] = pv[i];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          float vf[8];
          bf16x8_to_f32(vr[i], vf);
          float pp[G];
#pragma unroll
          for (int h = 0; h < G; ++h) pp[h] = pbuf[warp][i][half][h];
#pragma unroll
          for (int h = 0; h < G; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[h][e] = fmaf(pp[h], vf[e], acc[h][e]);
        }
        __syncwarp();
      }
    }
    // the two half-warps accumulated different tokens of the same slices
#pragma unroll
    for (int h = 0; h < G; ++h)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[h][e] += __shfl_xor_sync(0xffffffffu, acc[h][e], 16);
    if (half == 0) {
      const size_t base = (static_cast<size_t>(b) * p.nsplit + split) * p.Hq + hq0;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float inv = l[h] == 0.f ? 0.f : 1.f / l[h];      // 0: no key (a NaN is one)
        float4* dst = reinterpret_cast<float4*>(p.ws_o + (base + h) * kDecD + sub * 8);
        dst[0] = make_float4(acc[h][0] * inv, acc[h][1] * inv, acc[h][2] * inv, acc[h][3] * inv);
        dst[1] = make_float4(acc[h][4] * inv, acc[h][5] * inv, acc[h][6] * inv, acc[h][7] * inv);
        if (sub == 0)
          p.ws_lse[base + h] = l[h] == 0.f ? -INFINITY : (m[h] + __log2f(l[h])) * kLn2;
      }
    }
  }
}


// A stage holds, for K and for V, two TMA boxes (head dimension halves) of
// [Hkv heads][8 tokens][64 elements] with 128-byte swizzle: the 128-byte row of
// (head g, token t) keeps its 16-byte chunk c at position c ^ t, so the 8 token
// rows of one head are read by ldmatrix without bank conflicts.
// (SHARED: of 16 tokens, whose swizzle is that of token % 8.)
__host__ __device__ constexpr int box_bytes(int Hkv, int tokens) { return Hkv * tokens * 64 * 2; }
__host__ __device__ constexpr int stage_kv_bytes(int Hkv, int tokens) {
  return 2 * box_bytes(Hkv, tokens);
}

// hb[b] = sum over b' < b of ceil(len_b' / 8); hb[B] = total.  One block.
// (SHARED: of the lengths without the shared keys.)
template <bool SHARED>
__global__ void __launch_bounds__(1024) fa_decode_scan_kernel(const DecodeParams p) {
  __shared__ int warp_sums[32];
  __shared__ int carry;
  constexpr int TS = stage_tokens(SHARED);
  const int shared = SHARED && p.pw.together ? shared_pages(p.pw) : 0;
  pdl_launch_dependents();   // the stream kernel may launch now; it waits for hb itself
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    carry = 0;
    *p.dyn_next = 0;
  }
  __syncthreads();
  for (int base = 0; base < p.B; base += 1024) {
    const int b = base + threadIdx.x;
    int v = 0;
    if (b < p.B) {
      const int len = checked_len(p, seq_of<SHARED>(p, b));
      if (len < 0)
        atomicOr(p.err, kErrBadIndex);
      else
        v = (own_keys<SHARED>(len, shared).len + TS - 1) / TS;
    }
    int x = v;   // inclusive warp scan
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int w = warp_sums[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += y;
      }
      warp_sums[lane] = w;   // inclusive prefix of warp totals
    }
    __syncthreads();
    const int before = carry + (warp > 0 ? warp_sums[warp - 1] : 0) + x - v;
    if (b < p.B) p.hb[b] = before;
    __syncthreads();
    if (threadIdx.x == 1023) carry = before + v;
    __syncthreads();
  }
  if (threadIdx.x == 0) p.hb[p.B] = carry;
}

// Share of CTA c: [x0, x1) = [c*H/C, (c+1)*H/C); its own part [x0, y) and its
// dynamic part [y, x1) of d = (x1 - x0) / kDynDiv half-pages, cut into units of
// U half-pages; unit k of CTA c is global unit c * NUc + k (it may be empty).
// At most cap units in all (cap < C: no dynamic parts).  The partial of a
// segment of sequence b goes to slot c + b (own part of CTA c) or
// C + B + u + b (unit u): along the list the sequence index and the share or
// unit index never both stay the same, so the slots are distinct.
struct StreamSplit {
  int U, NUc, div;         // the last 1 / div of a share is dynamic
};
// (grid: CTAs with or without a share)
template <bool SHARED>
__device__ __forceinline__ StreamSplit stream_split(int H, int C, int cap, int grid) {
  StreamSplit sp;
  sp.div = SHARED && 2 * C < grid ? kDynDivWait : kDynDiv;
  sp.U = dyn_unit(SHARED);
  sp.NUc = 0;
  // (SHARED: cap is kMaxUnitsPerCta for every CTA of the grid, however many have shares)
  const int per_cta = SHARED ? cap / C : min(cap / C, kMaxUnitsPerCta);
  const int dmax = ((H + C - 1) / C) / sp.div;
  // (SHARED: a part of less than a unit would only add partials)
  if (per_cta > 0 && dmax >= (SHARED ? sp.U : 1)) {
    if ((dmax + sp.U - 1) / sp.U > per_cta) sp.U = (dmax + per_cta - 1) / per_cta;
    sp.NUc = (dmax + sp.U - 1) / sp.U;
  }
  return sp;
}
struct Share {
  int x0, y, x1;
};
__device__ __forceinline__ Share share_of(int c, int H, int C, const StreamSplit& sp) {
  Share sh;
  sh.x0 = share_edge(c, H, C);
  sh.x1 = share_edge(c + 1, H, C);
  sh.y = sh.x1 - (sp.NUc > 0 ? (sh.x1 - sh.x0) / sp.div : 0);
  return sh;
}

struct StageMeta {
  int b, hh, flags, len;   // flags: 1 = first of segment, 2 = last of segment, 4 = page valid,
                           //        8 = no more stages
  int slot0;               // partial slot of this segment = slot0 + b
};

template <int G, bool SHARED>
__global__ void __launch_bounds__(kStreamThreads, 1)
    fa_decode_stream_kernel(const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const DecodeParams p) {
  // Consumer warp g owns KV head g and its G <= 8 query heads.  Scores and
  // outputs use warp-level tensor-core MMAs: S (16 x 8) = Q (16 query-head rows,
  // G used) x K^T per 8-token stage, then O (16 x 128) += P (16 x 8) x V; the
  // score fragment becomes the P operand in registers, and every lane's rows
  // are its own query head, so the online softmax needs no broadcasts.
  extern __shared__ __align__(1024) uint8_t dsm_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages];
  __shared__ StageMeta meta[kMaxStages];
  __shared__ int abort_sm;

  const int c = blockIdx.x;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int NS = p.nstages;
  constexpr int TS = stage_tokens(SHARED);
  const int HB = box_bytes(p.Hkv, TS);              // one TMA box (half of the head dimension)
  const int SKV = stage_kv_bytes(p.Hkv, TS);        // bytes per stage for K (and for V)
  // swizzled TMA destinations must be 1024-byte aligned
  const uint32_t sbase = (smem_u32(dsm_raw) + 1023u) & ~1023u;
  auto full = [&](int st) { return smem_u32(&bars[st]); };
  auto empty = [&](int st) { return smem_u32(&bars[kMaxStages + st]); };
  volatile int* abort_flag = &abort_sm;
  if (threadIdx.x == 0) {
    for (int st = 0; st < NS; ++st) {
      mbar_init(full(st), 1);
      mbar_init(empty(st), kConsumerWarps);
    }
    abort_sm = 0;
    fence_barrier_init();
  }
  // Everything above overlaps the scan kernel; the half-page offsets are its output.
  // SHARED: the shared-prefix kernel stands in between and lets this one launch only
  // after the scan has finished; its own output is not read here, so this grid starts
  // on every SM that one has left and waits for it at the very end.
  // (Where the shared keys are streamed like the others, it does not stand there.)
  // (With a short list this is the first kernel of the call.)
  if (!SHARED || !p.pw.together) pdl_wait();
  // The merge kernel may launch once every CTA is past this point, so its launch
  // implies that the scan has finished: it reads the offsets before its own wait.
  pdl_launch_dependents();
  // C: the CTAs with shares of the list
  const bool scan_here = SHARED && p.scan_here;
  int shared = 0, listed = 0, C = gridDim.x, H = 0;
  StreamSplit sp = {1, 0, 1};
  Share own = {0, 0, 0};
  if constexpr (SHARED) {
    if (!p.pw.together) listed = shared_pages(p.pw);   // pages to be read by prefix_table
    if (!scan_here) {
      const PrefixSplit ps = prefix_split(p.pw, C);
      shared = ps.pages;
      C = ps.own_ctas;
    }
  }
  if (!scan_here) {
    H = SHARED ? __ldcg(p.hb + p.B) : p.hb[p.B];
    sp = stream_split<SHARED>(H, C, p.dyn_units_cap, gridDim.x);
    if (c < C) own = share_of(c, H, C, sp);
  }
  __syncthreads();

  if (warp >= kConsumerWarps) {
    regs_dec<kRegsProducer>();
    if (warp != kConsumerWarps) return;
    // ---------------------------------------------------------------- producer
    // The sequence offsets are searched for every stage: keep them in shared
    // memory (after the stage ring) when they fit.
    const int* hbp = p.hb;
    if (p.hb_in_smem) {
      int* hb_sm = reinterpret_cast<int*>(dsm_raw + (sbase - smem_u32(dsm_raw)) + NS * 2 * SKV);
      if (scan_here) {
        for (int b0 = 0; b0 < p.B; b0 += 32) {
          const int v = b0 + lane < p.B ? listed_pages(p, b0 + lane, c == 0) : 0;
          int x = v;                             // inclusive warp scan
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
          }
          if (b0 + lane < p.B) hb_sm[b0 + lane] = H + x - v;
          H += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) hb_sm[p.B] = H;
        C = short_list_ctas(p, H);
        if (c < C) own = share_of(c, H, C, sp);
      } else {
        for (int i = lane; i <= p.B; i += 32) hb_sm[i] = __ldcg(p.hb + i);
      }
      __syncwarp();
      hbp = hb_sm;
    }
    // Ranges of the half-page list: this CTA's static share, then dynamic units
    // while any are left.  For each range the whole warp resolves the next 32
    // stages (sequence, half-page, page id, length) with independent loads and
    // lane 0 issues them in order.  A last stage flagged 8 ends the consumers.
    int issued = 0;
    bool ok = true;
    auto acquire_stage = [&](int& st) {
      st = issued % NS;
      return mbar_wait_sleepy(empty(st), ((issued / NS) & 1) ^ 1, abort_flag, p.err, kWaitLimitNs);
    };
    auto run_range = [&](int xs, int cnt, int slot0) {
      for (int base = 0; base < cnt && ok; base += 32) {
        const int i = base + lane;
        int bq = 0, hh = 0, page = -1, len = 0, flags = 0;
        if (i < cnt) {
          const int x = xs + i;
          int lo = 0, hi = p.B;                  // hb[lo] <= x < hb[hi]
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (hbp[mid] <= x) lo = mid; else hi = mid;
          }
          bq = lo;
          const int hb_b = hbp[bq], hb_n = hbp[bq + 1];
          hh = x - hb_b;
          const int seq = seq_of<SHARED>(p, bq);
          const OwnKeys mine = own_keys<SHARED>(p.seq_lens[seq], shared);
          len = mine.len;
          bool valid;
          if (SHARED && hh < listed && len >= listed * kPage) {
            page = p.prefix_table[hh];
            valid = true;
            if (page < 0 || page >= p.num_pages) {
              atomicOr(p.err, kErrBadIndex);
              page = p.num_pages;                // past the pool: zeros
            }
          } else {
            page = p.block_table[static_cast<size_t>(seq) * p.max_pages + mine.page0 +
                                 (SHARED ? hh : hh >> 1)];
            valid = page >= 0 && page < p.num_pages;
          }
          flags = ((i == 0 || hh == 0) ? 1 : 0) | ((i == cnt - 1 || x + 1 == hb_n) ? 2 : 0) |
                  (valid ? 4 : 0);
        }
        const int cnt_here = min(32, cnt - base);
        for (int k = 0; k < cnt_here; ++k) {
          const int kb = __shfl_sync(0xffffffffu, bq, k);
          const int khh = __shfl_sync(0xffffffffu, hh, k);
          const int kpage = __shfl_sync(0xffffffffu, page, k);
          const int klen = __shfl_sync(0xffffffffu, len, k);
          const int kflags = __shfl_sync(0xffffffffu, flags, k);
          if (lane == 0) {
            int st;
            if (!acquire_stage(st)) {
              ok = false;
            } else {
              StageMeta md;
              md.b = kb;
              md.hh = khh;
              md.len = klen;
              md.flags = kflags;
              md.slot0 = slot0;
              meta[st] = md;
              if (kflags & 4) {
                const int tok0 = kpage * kPage + (SHARED ? 0 : (khh & 1) * kHalf);
                const uint32_t kdst = sbase + st * 2 * SKV;
                mbar_arrive_expect_tx(full(st), 2 * SKV);
                const int head0 = SHARED ? (kb % p.groups) * p.Hkv : 0;
                tma_load_3d(kdst, &tmK, full(st), 0, tok0, head0);
                tma_load_3d(kdst + HB, &tmK, full(st), 64, tok0, head0);
                tma_load_3d(kdst + SKV, &tmV, full(st), 0, tok0, head0);
                tma_load_3d(kdst + SKV + HB, &tmV, full(st), 64, tok0, head0);
              } else {
                atomicOr(p.err, kErrBadIndex);   // consumers skip this stage
                mbar_arrive(full(st));
              }
              ++issued;
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
        }
      }
    };
    if (own.y > own.x0) run_range(own.x0, own.y - own.x0, c);
    const int n_units = C * sp.NUc;
    while (ok && n_units > 0) {
      int u = 0;
      if (lane == 0) u = atomicAdd(p.dyn_next, 1);
      u = __shfl_sync(0xffffffffu, u, 0);
      if (u >= n_units) break;
      const Share sh = share_of(u / sp.NUc, H, C, sp);
      const int xs = sh.y + (u % sp.NUc) * sp.U;
      if (xs < sh.x1) run_range(xs, min(sh.x1, xs + sp.U) - xs, C + p.B + u);
    }
    if (lane == 0) {
      int st;
      if (ok && acquire_stage(st)) {             // end marker: no copy behind it
        StageMeta md;
        md.b = 0;
        md.hh = 0;
        md.len = 0;
        md.flags = 8;
        md.slot0 = 0;
        meta[st] = md;
        mbar_arrive(full(st));
        ++issued;
      }
      // copies still in flight must land before the CTA exits
      volatile int no_abort = 0;
      for (int i = max(0, issued - NS); i < issued; ++i)
        mbar_wait(full(i % NS), (i / NS) & 1, &no_abort, p.err, kWaitLimitNs);
      // this grid may only complete after the shared-prefix kernel: the merge waits for
      // this grid and then reads the partials of both
      if constexpr (SHARED) pdl_wait();
    }
    return;
  }

  regs_inc<kRegsConsumer>();
  // ------------------------------------------------------------------ consumers
  // Fragment layout (m16n8k16 / m16n8k8, gq = lane / 4, tq = lane % 4): score and
  // output rows are query heads gq (rows gq + 8 are unused and stay zero),
  // columns are tokens 2 tq, 2 tq + 1 of the stage (scores) or output columns
  // 8 n + 2 tq, 8 n + 2 tq + 1 (chunk n of O).
  const int gq = lane >> 2;
  const int tq = lane & 3;
  const int g = warp;                          // KV head of this warp (idle when g >= Hkv)
  const bool active = g < p.Hkv;
  const bool my_row = gq < G;                  // this lane's rows are real query heads
  const int hq = g * G + (my_row ? gq : 0);
  uint32_t qa[8][2];                           // Q A-fragments per 16-wide d chunk
  float o[16][4];
  float m_run = -INFINITY, l_run = 0.f;
  // ldmatrix: lane supplies row (head g, token lane % 8) of matrix lane / 8; for the
  // 32-wide group dg that is swizzled chunk ((dg & 1) * 4 + lane / 8) ^ (lane % 8)
  // in box dg / 2.
  const int lt = lane & 7;
  const uint32_t row_off = static_cast<uint32_t>((g * TS + lt) * 128);
  uint32_t ld_off[4];
#pragma unroll
  for (int dg = 0; dg < 4; ++dg)
    ld_off[dg] = static_cast<uint32_t>((dg >> 1) * HB) + row_off +
                 static_cast<uint32_t>((((dg & 1) * 4 + (lane >> 3)) ^ lt) << 4);
  for (int i = 0;; ++i) {
    const int st = i % NS;
    const bool ready = mbar_wait(full(st), (i / NS) & 1, abort_flag, p.err, kWaitLimitNs);
    if (!__all_sync(0xffffffffu, ready)) return;
    const StageMeta md = meta[st];
    if (md.flags & 8) break;                   // the producer has no more stages
    if (active) {
      if (md.flags & 1) {                      // a new sequence segment begins
        m_run = -INFINITY;
        l_run = 0.f;
        const uint32_t* qrow = reinterpret_cast<const uint32_t*>(
            p.q + (static_cast<size_t>(md.b) * p.Hq + hq) * kDecD);
#pragma unroll
        for (int kc = 0; kc < 8; ++kc) {
          qa[kc][0] = my_row ? qrow[kc * 8 + tq] : 0u;       // elements 16 kc + 2 tq, +1
          qa[kc][1] = my_row ? qrow[kc * 8 + 4 + tq] : 0u;   // elements 16 kc + 8 + 2 tq, +1
        }
#pragma unroll
        for (int nn = 0; nn < 16; ++nn) o[nn][0] = o[nn][1] = o[nn][2] = o[nn][3] = 0.f;
      }
      if (md.flags & 4) {
        const int ntok = min(TS, md.len - md.hh * TS);
        const uint32_t kaddr = sbase + st * 2 * SKV;
        const uint32_t vaddr = kaddr + SKV;
        // S = Q K^T over the 128-wide head dimension, 32 columns per ldmatrix; eight
        // tokens (1024 bytes on) to a score tile
        constexpr int TILES = TS / kHalf;
        float sa[TILES][4] = {};
#pragma unroll
        for (int dg = 0; dg < 4; ++dg) {
#pragma unroll
          for (int tt = 0; tt < TILES; ++tt) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4(kaddr + ld_off[dg] + tt * kHalf * 128, b0, b1, b2, b3);
            mma_bf16_16816(sa[tt], qa[2 * dg][0], 0u, qa[2 * dg][1], 0u, b0, b1);
            mma_bf16_16816(sa[tt], qa[2 * dg + 1][0], 0u, qa[2 * dg + 1][1], 0u, b2, b3);
          }
        }
        const int t0 = 2 * tq;
        float sc[TILES][2];
        float mx = -INFINITY;
#pragma unroll
        for (int tt = 0; tt < TILES; ++tt) {
          sc[tt][0] = tt * kHalf + t0 < ntok ? sa[tt][0] * p.scale_log2 : -INFINITY;
          sc[tt][1] = tt * kHalf + t0 + 1 < ntok ? sa[tt][1] * p.scale_log2 : -INFINITY;
          mx = fmaxf(mx, fmaxf(sc[tt][0], sc[tt][1]));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = fmaxf(m_run, mx);
        const float alpha = (m_run == -INFINITY) ? 0.f : ex2(m_run - m_new);
        m_run = m_new;
        float psum = 0.f;
        uint32_t pa[TILES];                      // P A-fragments: row gq, tokens 2 tq, 2 tq + 1
#pragma unroll
        for (int tt = 0; tt < TILES; ++tt) {
          const float p0 = (sc[tt][0] == -INFINITY) ? 0.f : ex2(sc[tt][0] - m_run);
          const float p1 = (sc[tt][1] == -INFINITY) ? 0.f : ex2(sc[tt][1] - m_run);
          psum += p0 + p1;
          pa[tt] = pack_bf16x2(p0, p1);
        }
        l_run = l_run * alpha + psum;
#pragma unroll
        for (int nn = 0; nn < 16; ++nn) {
          o[nn][0] *= alpha;
          o[nn][1] *= alpha;
        }
        // slots behind the sequence's last token hold whatever the pool held: their
        // weights are zero, and so must their values be (zero times NaN is NaN)
        uint32_t v_keep[TILES];
#pragma unroll
        for (int tt = 0; tt < TILES; ++tt)
          v_keep[tt] = (tt * kHalf + t0 < ntok ? 0x0000ffffu : 0u) |
                       (tt * kHalf + t0 + 1 < ntok ? 0xffff0000u : 0u);
#pragma unroll
        for (int ng = 0; ng < 4; ++ng) {
          uint32_t v[TILES][4];
#pragma unroll
          for (int tt = 0; tt < TILES; ++tt) {
            ldsm_x4_t(vaddr + ld_off[ng] + tt * kHalf * 128, v[tt][0], v[tt][1], v[tt][2],
                      v[tt][3]);
            if (ntok < TS) {
#pragma unroll
              for (int i4 = 0; i4 < 4; ++i4) v[tt][i4] &= v_keep[tt];
            }
          }
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            if constexpr (TILES == 2)
              mma_bf16_16816(o[4 * ng + i4], pa[0], 0u, pa[1], 0u, v[0][i4], v[1][i4]);
            else
              mma_bf16_1688(o[4 * ng + i4], pa[0], 0u, v[0][i4]);
          }
        }
      }

      if (md.flags & 2) {                      // segment ends: its partial goes to slot0 + b
        float l_tot = l_run;
        l_tot += __shfl_xor_sync(0xffffffffu, l_tot, 1);
        l_tot += __shfl_xor_sync(0xffffffffu, l_tot, 2);
        if (my_row) {
          const float inv = l_tot == 0.f ? 0.f : 1.f / l_tot;  // 0: no key (a NaN is one)
          const size_t rowi = (static_cast<size_t>(md.slot0) + md.b) * p.Hq + hq;
          float* dst = p.ws_o + rowi * kDecD + 2 * tq;
#pragma unroll
          for (int nn = 0; nn < 16; ++nn)
            *reinterpret_cast<float2*>(dst + 8 * nn) = make_float2(o[nn][0] * inv, o[nn][1] * inv);
          if (tq == 0)
            p.ws_lse[rowi] = l_tot == 0.f ? -INFINITY : (m_run + __log2f(l_tot)) * kLn2;
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty(st));
  }
}

// Streamed schedule, merge: one block per sequence b.  The partials of b sit in
// slot c + b for every CTA c whose own part meets b, and in slot C + B + u + b
// for every dynamic unit u that meets b; warp 0 lists them in shared memory
// (lanes over CTAs), then each warp merges query heads by their LSE (formula 2
// of the softmax merge), lane i owning output columns [4i, 4i + 4).
//
// The offsets are the scan kernel's output, which has finished by the time this
// grid launches (the stream kernel signals its dependents only after its own
// wait on the scan), so the slot list is built while the stream kernel still
// runs; after the wait only the partials are read, the LSEs and the first
// kMergeBatch partial rows of a head in one round of independent loads.
constexpr int kMergeBatch = 8;

// n partial results of one (sequence, query head) joined by their LSE: lse_at(k) and
// row_at(k) (the lane's four columns) give the k-th.  32 partials at a time (one
// sequence rarely has more): one LSE per lane and the first kMergeBatch rows load
// together; a later chunk with a larger maximum rescales what is accumulated so far.  A
// partial whose scores had a NaN has a NaN LSE, which the maximum passes over and the sum
// of the weights takes up: only partials with an LSE of -inf, those of no key, are nothing.
struct Joined {
  float4 acc;       // the lane's columns, weighted by exp(LSE - mx)
  float wsum, mx;   // sum of the weights (all lanes), their reference
};
template <class LseAt, class RowAt>
__device__ __forceinline__ Joined join_partials(int n, int lane, LseAt lse_at, RowAt row_at) {
  float wsum = 0.f, mx = -INFINITY;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < n; k0 += 32) {
    const int cnt = min(32, n - k0);
    const float ls = lane < cnt ? lse_at(k0 + lane) : -INFINITY;
    float4 v[kMergeBatch];
#pragma unroll
    for (int j = 0; j < kMergeBatch; ++j)
      if (j < cnt) v[j] = row_at(k0 + j);
    float m = ls;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    m = fmaxf(m, mx);
    // every LSE so far is -inf (warp-uniform)
    if (m == -INFINITY && !__any_sync(0xffffffffu, ls != -INFINITY)) continue;
    const float sc = ex2((mx - m) * kLog2e);   // 0 on the first finite chunk
    acc.x *= sc;
    acc.y *= sc;
    acc.z *= sc;
    acc.w *= sc;
    wsum *= sc;
    mx = m;
    const float w = (ls == -INFINITY) ? 0.f : ex2((ls - mx) * kLog2e);
    wsum += w;
    for (int j0 = 0; j0 < cnt; j0 += kMergeBatch) {
      if (j0 > 0) {
#pragma unroll
        for (int j = 0; j < kMergeBatch; ++j)
          if (j0 + j < cnt) v[j] = row_at(k0 + j0 + j);
      }
#pragma unroll
      for (int j = 0; j < kMergeBatch; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
        if (j0 + j < cnt) {
          acc.x = fmaf(wj, v[j].x, acc.x);
          acc.y = fmaf(wj, v[j].y, acc.y);
          acc.z = fmaf(wj, v[j].z, acc.z);
          acc.w = fmaf(wj, v[j].w, acc.w);
        }
      }
    }
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, d);
  return {acc, wsum, mx};
}
__device__ __forceinline__ void store_joined(const Joined& r, int lane, uint16_t* o, float* lse) {
  const float inv = r.wsum == 0.f ? 0.f : 1.f / r.wsum;
  *reinterpret_cast<uint2*>(o + lane * 4) = make_uint2(
      pack_bf16x2(r.acc.x * inv, r.acc.y * inv), pack_bf16x2(r.acc.z * inv, r.acc.w * inv));
  if (lse && lane == 0) *lse = r.wsum == 0.f ? -INFINITY : r.mx + __log2f(r.wsum) * kLn2;
}

// The segments of the shared prefix that hold row (b, h): n of them, the k-th at row
// row0 + k step of the segments' workspace.
struct PrefixRows {
  int n;
  size_t row0, step;
};
__device__ __forceinline__ PrefixRows prefix_rows(const DecodeParams& p, const PrefixSplit& sp,
                                                  int b, int h) {
  const int G = p.Hq / p.Hkv;
  const int row = b / p.groups * G + h % G;
  const int group = (row >> 8) / p.pw.team, member = (row >> 8) - group * p.pw.team;
  const int item = (b % p.groups * p.Hkv + h / G) * p.pw.pair_groups + group;
  const int c0 = cta_of(static_cast<long long>(item) * sp.nt, sp.units, sp.teams);
  const int c1 = cta_of(static_cast<long long>(item + 1) * sp.nt - 1, sp.units, sp.teams);
  PrefixRows r;
  r.n = c1 - c0 + 1;
  r.row0 = (static_cast<size_t>(c0 + item) * p.pw.team + member) * 256 + (row & 255);
  r.step = static_cast<size_t>(p.pw.team) * 256;
  return r;
}

// SHARED: blocks of 8 warps, `p.merge_split` of which share a row's partials, so that few
// rows with many partials (a long prefix, a small batch) use more warps than they are: as
// many as keep all warps resident.  Two sequences of 1024 pages, 32 + 8 heads: 33.9 us a
// warp a row, 29.8 us so; 7 sequences of 65 pages, 8 + 2 heads: 15.2 and 13.0 us.
template <bool SHARED>
__global__ void __launch_bounds__(merge_warps(SHARED) * 32) fa_decode_stream_merge_kernel(
    const DecodeParams p) {
  constexpr int kWarps = merge_warps(SHARED);
  const int split = SHARED ? p.merge_split : 1;
  const int rows = kWarps / split;             // heads of the block at a time
  const int head_step = SHARED ? gridDim.y * rows : kWarps;
  const int head0 = SHARED ? blockIdx.y * rows : 0;
  __shared__ Joined parts[SHARED ? kWarps : 1][32];
  __shared__ int slots[kMaxMergeSlots];
  __shared__ int n_slots_sm;
  const int b = blockIdx.x;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  int xs, xe, H;                               // the entry's part of the list, its length
  const bool scan_here = SHARED && p.scan_here;
  if (scan_here) {
    __shared__ int sums[3];
    if (threadIdx.x < 3) sums[threadIdx.x] = 0;
    __syncthreads();
    int before = 0, mine = 0, total = 0;
    for (int i = threadIdx.x; i < p.B; i += kWarps * 32) {
      const int n = listed_pages(p, i, false);
      total += n;
      if (i < b) before += n;
      if (i == b) mine = n;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    mine = __reduce_add_sync(0xffffffffu, mine);
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) {
      atomicAdd(&sums[0], before);
      atomicAdd(&sums[1], mine);
      atomicAdd(&sums[2], total);
    }
    __syncthreads();
    xs = sums[0];
    xe = xs + sums[1];
    H = sums[2];
  } else {
    xs = __ldcg(p.hb + b);
    xe = __ldcg(p.hb + b + 1);
    H = __ldcg(p.hb + p.B);
  }
  PrefixSplit ps = {};
  bool sees = false;                           // the sequence has the shared keys
  if (scan_here) {
    ps.own_ctas = short_list_ctas(p, H);
  } else if constexpr (SHARED) {
    ps = prefix_split(p.pw, p.pw.ctas);
    sees = ps.pages > 0 && checked_len(p, seq_of<SHARED>(p, b)) >= ps.pages * kPage;
  }
  if (xe <= xs && !sees) {                     // no keys (or an invalid length): O = 0, LSE = -inf
    pdl_wait();
    for (int h = head0 + warp; warp < rows && h < p.Hq; h += head_step) {
      const size_t wid = static_cast<size_t>(b) * p.Hq + h;
      *reinterpret_cast<uint2*>(p.o + wid * kDecD + lane * 4) = make_uint2(0, 0);
      if (p.lse && lane == 0) p.lse[wid] = -INFINITY;
    }
    return;
  }
  const int C = SHARED ? ps.own_ctas : p.nctas;
  StreamSplit sp = {1, 0, 1};
  if (!scan_here) sp = stream_split<SHARED>(H, C, p.dyn_units_cap, p.nctas);
  if (warp == 0) {
    int base = 0;
    // no own keys: an empty range
    const int c_first = xe > xs ? cta_of(xs, H, C) : 0;
    const int c_last = xe > xs ? cta_of(xe - 1, H, C) : -1;
    for (int c0 = c_first; c0 <= c_last; c0 += 32) {
      const int cc = c0 + lane;
      Share sh;
      int own = 0, k0 = 0, k1 = -1;
      if (cc <= c_last) {
        sh = share_of(cc, H, C, sp);
        own = max(xs, sh.x0) < min(xe, sh.y) ? 1 : 0;
        const int lo = max(xs, sh.y), hi = min(xe, sh.x1);
        if (lo < hi) {
          k0 = (lo - sh.y) / sp.U;
          k1 = (hi - 1 - sh.y) / sp.U;
        }
      }
      const int cnt = own + (k1 - k0 + 1);
      int incl = cnt;                          // inclusive prefix over the lanes
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      int at = base + incl - cnt;
      if (own && at < kMaxMergeSlots) slots[at] = cc + b;
      at += own;
      for (int k = k0; k <= k1; ++k, ++at)
        if (at < kMaxMergeSlots) slots[at] = C + p.B + cc * sp.NUc + k + b;
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) n_slots_sm = min(base, kMaxMergeSlots);
  }
  __syncthreads();
  const int ns = n_slots_sm;
  pdl_wait();                                  // the stream kernel's partials
  const float4* wo = reinterpret_cast<const float4*>(p.ws_o);
  const float4* po = reinterpret_cast<const float4*>(p.pre_o);
  const int share = SHARED ? warp % split : 0; // partials share, share + split, ... are the warp's
  for (int h0 = head0; h0 < p.Hq; h0 += head_step) {
    const int h = h0 + (SHARED ? warp / split : warp);
    const size_t wid = static_cast<size_t>(b) * p.Hq + h;
    Joined r = {make_float4(0.f, 0.f, 0.f, 0.f), 0.f, -INFINITY};
    if (h < p.Hq) {
      PrefixRows pr;
      pr.n = 0;
      pr.row0 = pr.step = 0;
      if (SHARED && sees) pr = prefix_rows(p, ps, b, h);
      r = join_partials(
          (ns + pr.n - share + split - 1) / split, lane,
          [&](int k) {
            if (SHARED) k = share + k * split;
            if (SHARED && k >= ns)
              return __ldcg(p.pre_lse + pr.row0 + (k - ns) * pr.step);
            return __ldcg(p.ws_lse + static_cast<size_t>(slots[k]) * p.Hq + h);
          },
          [&](int k) {
            if (SHARED) k = share + k * split;
            if (SHARED && k >= ns)
              return __ldcg(po + (pr.row0 + (k - ns) * pr.step) * (kDecD / 4) + lane);
            return __ldcg(wo + (static_cast<size_t>(slots[k]) * p.Hq + h) * (kDecD / 4) + lane);
          });
    }
    if (SHARED && split > 1) {
      parts[warp][lane] = r;
      __syncthreads();
      if (share == 0) {
        float mx = r.mx;
        for (int i = 1; i < split; ++i) mx = fmaxf(mx, parts[warp + i][lane].mx);
        Joined all = {make_float4(0.f, 0.f, 0.f, 0.f), 0.f, mx};
        // (a NaN in a part without a finite LSE stays one under its weight of zero)
        for (int i = 0; i < split; ++i) {
          const Joined q = parts[warp + i][lane];
          const float w = q.mx == -INFINITY ? 0.f : ex2((q.mx - mx) * kLog2e);
          all.acc.x = fmaf(w, q.acc.x, all.acc.x);
          all.acc.y = fmaf(w, q.acc.y, all.acc.y);
          all.acc.z = fmaf(w, q.acc.z, all.acc.z);
          all.acc.w = fmaf(w, q.acc.w, all.acc.w);
          all.wsum = fmaf(w, q.wsum, all.wsum);
        }
        r = all;
      }
      __syncthreads();                         // read before the next heads' are written
    }
    if (h < p.Hq && share == 0)
      store_joined(r, lane, p.o + wid * kDecD, p.lse ? p.lse + wid : nullptr);
  }
}

// One CTA of 128 threads per (sequence, query head); thread d owns output column d.
__global__ void __launch_bounds__(kDecD) fa_decode_combine_kernel(const DecodeParams p) {
  const int bh = blockIdx.x;
  const int b = bh / p.Hq;
  const int h = bh - b * p.Hq;
  const int d = threadIdx.x;
  const int len = checked_len(p, b);
  const int npages = len > 0 ? (len + kPage - 1) / kPage : 0;
  const int ns = (npages + p.pps - 1) / p.pps;
  float out = 0.f, lse = -INFINITY;
  if (ns > 0) {
    const size_t base = static_cast<size_t>(b) * p.nsplit * p.Hq + h;
    float mx = -INFINITY;
    bool any = false;                          // a partial with keys (a NaN's LSE is NaN)
    for (int s = 0; s < ns; ++s) {
      const float ls = p.ws_lse[base + static_cast<size_t>(s) * p.Hq];
      any |= ls != -INFINITY;
      mx = fmaxf(mx, ls);
    }
    if (any) {
      float wsum = 0.f, acc = 0.f;
      for (int s = 0; s < ns; ++s) {
        const size_t idx = base + static_cast<size_t>(s) * p.Hq;
        const float ls = p.ws_lse[idx];
        const float w = (ls == -INFINITY) ? 0.f : ex2((ls - mx) * kLog2e);
        wsum += w;
        acc = fmaf(w, p.ws_o[idx * kDecD + d], acc);
      }
      out = acc / wsum;
      lse = mx + __log2f(wsum) * kLn2;
    }
  }
  uint32_t packed = pack_bf16x2(out, 0.f);
  p.o[static_cast<size_t>(bh) * kDecD + d] = static_cast<uint16_t>(packed & 0xffffu);
  if (p.lse && d == 0) p.lse[bh] = lse;
}

struct DevicePool {
  cudaMemPool_t pool = nullptr;
};
std::mutex g_pool_mu;
std::vector<DevicePool> g_pools;

int get_pool(int device, cudaMemPool_t* out) {
  std::lock_guard<std::mutex> g(g_pool_mu);
  if (static_cast<int>(g_pools.size()) <= device) g_pools.resize(device + 1);
  if (!g_pools[device].pool) {
    cudaMemPoolProps props = {};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = device;
    cudaMemPool_t pool;
    cudaError_t e = cudaMemPoolCreate(&pool, &props);
    if (e != cudaSuccess)
      return set_error(FA_ERR_CUDA, "cudaMemPoolCreate: %s", cudaGetErrorString(e));
    uint64_t keep = ~0ull;   // keep freed workspace cached in the pool between calls
    cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep);
    g_pools[device].pool = pool;
  }
  *out = g_pools[device].pool;
  return FA_OK;
}

int sm_count(int device) {
  static int cached[64] = {};
  static std::mutex mu;
  std::lock_guard<std::mutex> g(mu);
  if (device < 0 || device >= 64) return 0;
  if (!cached[device]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) n = 0;
    cached[device] = n;
  }
  return cached[device];
}

// The shared prefix of a SHARED call: its page ids, how its work is split, and the
// workspace of its segments.
struct SharedPrefix {
  int B = 0, Hq = 0, Hkv = 0, groups = 1;      // of the call; head groups of a sequence
  bool scan_here = false;
  const int32_t* table = nullptr;
  PrefixWork work;
  float* ws_o = nullptr;
  float* ws_lse = nullptr;
  float scale = 0.f;
};

// Launch geometry and workspace size of one decode call.
struct DecodePlan {
  bool streamed = false;
  int pps = 0, nsplit = 0;     // direct schedule
  int nctas = 0, nstages = 0;  // streamed schedule
  int dyn_units_cap = 0;       // streamed: dynamic units the partial slots allow
  size_t n_part = 0;           // partial rows (slot x head)
  size_t bytes = 0;            // workspace bytes
};

// Direct schedule: pages per chunk so that a full-length batch makes ~2048 CTAs.
int direct_pps(int B, int max_pages_per_seq) {
  const long long want = (static_cast<long long>(B) * max_pages_per_seq + 2047) / 2048;
  int pps = 4;
  while (pps < want && pps < 64) pps *= 2;
  return pps;
}

void finish_plan(DecodePlan& pl, int B, int Hq, int Hkv) {
  if (pl.streamed) {
    // slots: C + B static, then (units + B) dynamic when there are units
    const size_t dyn_slots = pl.dyn_units_cap > 0 ? static_cast<size_t>(pl.dyn_units_cap) + B : 0;
    pl.n_part = (static_cast<size_t>(pl.nctas) + B + dyn_slots) * Hq;
    pl.bytes = pl.n_part * (kDecD + 1) * sizeof(float) + (static_cast<size_t>(B) + 2) * sizeof(int);
  } else {
    pl.n_part = static_cast<size_t>(B) * pl.nsplit * Hq;
    pl.bytes = pl.n_part * (kDecD + 1) * sizeof(float);
  }
}

DecodePlan make_plan(int B, int Hq, int Hkv, int max_pages_per_seq, int nsm,
                     bool shared = false) {
  DecodePlan pl;
  // streamed: one consumer warp per KV head, its G <= 8 query heads as MMA rows
  pl.streamed = Hkv <= kDecWarps && nsm > 0;
  if (pl.streamed) {
    pl.nctas = std::min(nsm, kMaxStreamCtas);
    pl.nstages = kStreamSmemBudget / (2 * stage_kv_bytes(Hkv, stage_tokens(shared)));
    if (pl.nstages > kMaxStages) pl.nstages = kMaxStages;
    // enough units for the dynamic part of every share of the longest possible list
    const long long h_max = 2LL * B * max_pages_per_seq;
    const long long per_cta =
        ((h_max + pl.nctas - 1) / pl.nctas) / (shared ? kDynDivWait : kDynDiv) / dyn_unit(shared) + 1;
    pl.dyn_units_cap = static_cast<int>(std::min<long long>(per_cta * pl.nctas, 1 << 24));
  } else {
    pl.pps = direct_pps(B, max_pages_per_seq);
    pl.nsplit = (max_pages_per_seq + pl.pps - 1) / pl.pps;
  }
  finish_plan(pl, B, Hq, Hkv);
  return pl;
}

template <int G, bool SHARED>
int launch_kernels(const DecodeParams& prm, const DecodePlan& pl, const CUtensorMap& tmK,
                   const CUtensorMap& tmV, const SharedPrefix* pre, cudaStream_t stream,
                   int device) {
  if (pl.streamed) {
    const int smem = pl.nstages * 2 * stage_kv_bytes(prm.Hkv, stage_tokens(SHARED)) + 1024 +
                     (prm.hb_in_smem ? (prm.B + 1) * 4 : 0);
    {
      // the shared-memory limit is a property of the function on each device
      static int attr_gen[64] = {};
      static std::mutex mu;
      std::lock_guard<std::mutex> g(mu);
      if (device < 0 || device >= 64) return set_error(FA_ERR_CUDA, "device ordinal out of range");
      if (attr_gen[device] != cache_generation()) {
        cudaError_t e = cudaFuncSetAttribute(fa_decode_stream_kernel<G, SHARED>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kStreamSmemBudget + 1024 + kHbSmemMax * 4);
        if (e != cudaSuccess)
          return set_error(FA_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        attr_gen[device] = cache_generation();
      }
    }
    // The stream and merge kernels are launched with programmatic serialization:
    // each may start while its predecessor runs and waits (griddepcontrol.wait)
    // before it reads the predecessor's output, which hides the launch gaps.
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    if (!prm.scan_here) fa_decode_scan_kernel<SHARED><<<1, 1024, 0, stream>>>(prm);
    if constexpr (SHARED) {
      // right after the scan, overlapping it and the stream kernel
      if (prm.pw.together) {
        const int rc = launch_prefix(prm.q, prm.kc, prm.vc, prm.pw, pre->table, pre->ws_o,
                                     pre->ws_lse, pre->B, pre->Hq, pre->Hkv, prm.num_pages,
                                     pre->scale, stream, device);
        if (rc != FA_OK) return rc;
      }
    }
    cfg.gridDim = dim3(pl.nctas);
    cfg.blockDim = dim3(kStreamThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.numAttrs = prm.scan_here ? 0 : 1;        // (then the call's first kernel)
    cudaLaunchKernelEx(&cfg, fa_decode_stream_kernel<G, SHARED>, tmK, tmV, prm);
    cfg.numAttrs = 1;
    constexpr int mw = merge_warps(SHARED);
    cfg.gridDim = dim3(prm.B, SHARED ? (prm.Hq * prm.merge_split + mw - 1) / mw : 1);
    cfg.blockDim = dim3(mw * 32);
    cfg.dynamicSmemBytes = 0;
    cudaLaunchKernelEx(&cfg, fa_decode_stream_merge_kernel<SHARED>, prm);
  } else if constexpr (!SHARED) {
    dim3 grid(pl.nsplit, prm.B);
    fa_decode_split_kernel<G><<<grid, kDecThreads, 0, stream>>>(prm);
    fa_decode_combine_kernel<<<prm.B * prm.Hq, kDecD, 0, stream>>>(prm);
  }
  return FA_OK;
}

// Runs one decode with the given workspace (at least pl.bytes, 256-byte aligned).
int run_decode(const void* q, const void* kcache, const void* vcache, const int32_t* block_table,
               const int32_t* seq_lens, void* o, float* lse, int B, int Hq, int Hkv,
               int max_pages_per_seq, int num_pages, float scale, const DecodePlan& pl, void* ws,
               cudaStream_t stream, int device, const SharedPrefix* pre = nullptr) {
  const int G = Hq / Hkv;
  DecodeParams prm;
  prm.q = static_cast<const uint16_t*>(q);
  prm.kc = static_cast<const uint16_t*>(kcache);
  prm.vc = static_cast<const uint16_t*>(vcache);
  prm.block_table = block_table;
  prm.seq_lens = seq_lens;
  prm.o = static_cast<uint16_t*>(o);
  prm.lse = lse;
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.max_pages = max_pages_per_seq;
  prm.num_pages = num_pages;
  prm.pps = pl.pps;
  prm.nsplit = pl.nsplit;
  prm.nctas = pl.nctas;
  prm.nstages = pl.nstages;
  prm.dyn_units_cap = pl.dyn_units_cap;
  prm.hb_in_smem = B + 1 <= kHbSmemMax ? 1 : 0;
  prm.scale_log2 = scale * kLog2e;
  prm.err = device_error_word(device);
  if (!prm.err) return set_error(FA_ERR_CUDA, "device error word unavailable");
  prm.groups = pre ? pre->groups : 1;
  prm.merge_split = 1;
  while (pre && prm.merge_split < 8 && 2LL * prm.merge_split * B * Hq <= 8LL * 3 * pl.nctas)
    prm.merge_split *= 2;
  prm.pw = PrefixWork{};
  prm.pre_o = prm.pre_lse = nullptr;
  prm.prefix_table = pre ? pre->table : nullptr;
  prm.scan_here = pre && pre->scan_here;
  if (pre) {
    prm.pw = pre->work;
    prm.pw.err = prm.err;
    prm.pre_o = pre->ws_o;
    prm.pre_lse = pre->ws_lse;
  }
  if (!pl.streamed && (pl.nsplit > 65535 || B > 65535))
    return set_error(FA_ERR_UNSUPPORTED, "too many sequences or chunks for one launch");
  if (static_cast<long long>(B) * Hq > 0x7fffffffLL)
    return set_error(FA_ERR_UNSUPPORTED, "B * Hq too large");
  prm.ws_o = static_cast<float*>(ws);
  prm.ws_lse = prm.ws_o + pl.n_part * kDecD;
  prm.hb = reinterpret_cast<int*>(prm.ws_lse + pl.n_part);
  prm.pw.own_total = prm.hb + B;
  prm.dyn_next = prm.hb + (B + 1);
  CUtensorMap tmK, tmV;
  if (pl.streamed) {
    // K and V caches viewed as [Hkv][num_pages * 16 tokens][128]: box {64, 8, Hkv}
    const uint64_t dims[3] = {static_cast<uint64_t>(kDecD),
                              static_cast<uint64_t>(num_pages) * kPage,
                              static_cast<uint64_t>(Hkv) * prm.groups};
    const uint64_t strides[2] = {static_cast<uint64_t>(Hkv) * prm.groups * kDecD * 2,
                                 static_cast<uint64_t>(kDecD) * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(stage_tokens(pre != nullptr)),
                             static_cast<uint32_t>(Hkv)};
    int rc = encode_tensor_map_16bit(&tmK, kcache, true, 3, dims, strides, box);
    if (rc == FA_OK) rc = encode_tensor_map_16bit(&tmV, vcache, true, 3, dims, strides, box);
    if (rc != FA_OK) return rc;
  } else {
    memset(&tmK, 0, sizeof(tmK));
    memset(&tmV, 0, sizeof(tmV));
  }
  int lrc;
#define FA_DECODE_G(G_)                                                                  \
  lrc = pre ? launch_kernels<G_, true>(prm, pl, tmK, tmV, pre, stream, device)             \
            : launch_kernels<G_, false>(prm, pl, tmK, tmV, pre, stream, device)
  switch (G) {
    case 1: FA_DECODE_G(1); break;
    case 2: FA_DECODE_G(2); break;
    case 4: FA_DECODE_G(4); break;
    default: FA_DECODE_G(8); break;
  }
#undef FA_DECODE_G
  if (lrc != FA_OK) return lrc;
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(FA_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
  return FA_OK;
}

}  // namespace

int launch_decode(const void* q, const void* kcache, const void* vcache, const int32_t* block_table,
                  const int32_t* seq_lens, void* o, float* lse, int B, int Hq, int Hkv, int D,
                  int page_size, float scale, int max_pages_per_seq, int num_pages,
                  cudaStream_t stream, int device) {
  if (D != kDecD) return set_error(FA_ERR_UNSUPPORTED, "decode supports D == 128 only (got %d)", D);
  if (page_size != kPage)
    return set_error(FA_ERR_UNSUPPORTED, "decode supports page_size == 16 only (got %d)", page_size);
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8)
    return set_error(FA_ERR_UNSUPPORTED, "decode supports Hq/Hkv in {1,2,4,8} (got %d)", G);
  const DecodePlan pl = make_plan(B, Hq, Hkv, max_pages_per_seq, sm_count(device));
  cudaMemPool_t pool;
  int rc = get_pool(device, &pool);
  if (rc != FA_OK) return rc;
  void* ws = nullptr;
  cudaError_t e = cudaMallocFromPoolAsync(&ws, pl.bytes, pool, stream);
  if (e != cudaSuccess)
    return set_error(FA_ERR_CUDA, "workspace allocation (%zu bytes): %s", pl.bytes,
                     cudaGetErrorString(e));
  rc = run_decode(q, kcache, vcache, block_table, seq_lens, o, lse, B, Hq, Hkv, max_pages_per_seq,
                  num_pages, scale, pl, ws, stream, device);
  cudaError_t ef = cudaFreeAsync(ws, stream);
  if (rc != FA_OK) {
    cudaGetLastError();                // of the release: the first error is the one reported
    return rc;
  }
  if (ef != cudaSuccess)
    return set_error(FA_ERR_CUDA, "workspace release: %s", cudaGetErrorString(ef));
  return FA_OK;
}

int launch_decode_shared(const void* q, const void* kcache, const void* vcache,
                         const int32_t* block_table, const int32_t* seq_lens,
                         const int32_t* prefix_table, const int32_t* prefix_pages,
                         int max_prefix_pages, void* o, float* lse, int B, int Hq, int Hkv,
                         float scale, int max_pages_per_seq, int num_pages, cudaStream_t stream,
                         int device) {
  const int G = Hq / Hkv;
  const int nsm = sm_count(device);
  if (nsm <= 0) return set_error(FA_ERR_CUDA, "cannot read the SM count of device %d", device);
  SharedPrefix pre;
  pre.B = B;
  pre.Hq = Hq;
  pre.Hkv = Hkv;
  while (Hkv % pre.groups != 0 || Hkv / pre.groups > kConsumerWarps) ++pre.groups;
  const int gq = Hq / pre.groups, gkv = Hkv / pre.groups;
  const long long entries = static_cast<long long>(B) * pre.groups;
  if (2 * entries * max_pages_per_seq > 0x7fffffffLL)
    return set_error(FA_ERR_UNSUPPORTED, "shared prefix: too many keys for one call");
  const int gb = static_cast<int>(entries);
  DecodePlan pl = make_plan(gb, gq, gkv, max_pages_per_seq, nsm, true);
  // a CTA never gets more units than this, so no more slots are needed either
  pl.dyn_units_cap = std::min(pl.dyn_units_cap, pl.nctas * kMaxUnitsPerCta);
  finish_plan(pl, gb, gq, gkv);
  pre.table = prefix_table;
  pre.scale = scale;
  pre.work.pages = prefix_pages;
  pre.work.max_pages = max_prefix_pages;
  const long long pairs = (static_cast<long long>(B) * G + 255) / 256;
  pre.work.pair_groups = static_cast<int>((pairs + kPrefixTeam - 1) / kPrefixTeam);
  pre.work.team =
      static_cast<int>((pairs + pre.work.pair_groups - 1) / pre.work.pair_groups);
  const long long items = static_cast<long long>(Hkv) * pre.work.pair_groups;
  const long long tiles =
      (static_cast<long long>(max_prefix_pages) * kPage + kPrefixTile - 1) / kPrefixTile;
  if (items * tiles > 0x7fffffffLL - nsm || static_cast<long long>(B) * Hq > 0x7fffffffLL - 256)
    return set_error(FA_ERR_UNSUPPORTED, "shared prefix: too much work for one call");
  pre.work.pairs = static_cast<int>(pairs);
  pre.work.items = static_cast<int>(items);
  // Few copies of few shared pages are streamed with the own ones: the copies come from L2,
  // and the prefix kernel's start and end cost about 7 us.  The launches are chosen here, by
  // the bound on the pages; the count itself is on the device.  32 + 8 heads, together / apart:
  // 7 sequences of 32 pages 17.2 / 12.2 us, of 130 19.0 / 15.5, of 260 20.3 / 20.2;
  // 64 of 16 19.5 / 17.7, of 32 20.2 / 24.7.
  pre.work.together = entries * max_prefix_pages > 1536;
  // (64 pages a CTA are the least of which a 16th makes a dynamic unit)
  pre.scan_here = !pre.work.together && entries <= kScanHere &&
                  entries * max_pages_per_seq < 64LL * pl.nctas;
  // Measured on an SM: a key tile against two row tiles 1.9 to 2.3 us, against one 1.8 us;
  // a page of 8 KV heads 0.92 us (of 4 or fewer 0.68: one number for all counts those a
  // quarter too dear).  What matters is their ratio.  us of 256 sequences with
  // 32768 shared keys / 64 with 4096 at 2050 and 350 ns: 318 / 106, 700: 181 / 106, 1000:
  // 170 / 107, 1400: 178 / 126, 2000: 190 / 150, 3000: 219 / 199; in a long run at the power
  // limit, where tiles take longer, 195 / 112 at 750 and 194 / 112 at 850.
  pre.work.tile_ns = static_cast<long long>(B) * G > 128 ? 2050 : 1800;
  pre.work.page_ns = 850;
  pre.work.ctas = nsm;
  // segments write to slot (team + item) * team size + member
  const size_t pre_rows = pre.work.together ? (nsm + items * pre.work.team) * size_t(256) : 0;
  const size_t pre_bytes = (pre_rows * (kDecD + 1) * sizeof(float) + 255) & ~size_t(255);
  cudaMemPool_t pool;
  int rc = get_pool(device, &pool);
  if (rc != FA_OK) return rc;
  void* ws = nullptr;
  cudaError_t e = cudaMallocFromPoolAsync(&ws, pre_bytes + pl.bytes, pool, stream);
  if (e != cudaSuccess)
    return set_error(FA_ERR_CUDA, "workspace allocation (%zu bytes): %s", pre_bytes + pl.bytes,
                     cudaGetErrorString(e));
  pre.ws_o = static_cast<float*>(ws);
  pre.ws_lse = pre.ws_o + pre_rows * kDecD;
  rc = run_decode(q, kcache, vcache, block_table, seq_lens, o, lse, gb, gq, gkv,
                  max_pages_per_seq, num_pages, scale, pl, static_cast<char*>(ws) + pre_bytes,
                  stream, device, &pre);
  cudaError_t ef = cudaFreeAsync(ws, stream);
  if (rc != FA_OK) {
    cudaGetLastError();                // of the release: the first error is the one reported
    return rc;
  }
  if (ef != cudaSuccess)
    return set_error(FA_ERR_CUDA, "workspace release: %s", cudaGetErrorString(ef));
  return FA_OK;
}

void release_decode_resources() {
  std::lock_guard<std::mutex> g(g_pool_mu);
  for (auto& dp : g_pools) {
    if (dp.pool) {
      cudaMemPoolDestroy(dp.pool);
      dp.pool = nullptr;
    }
  }
}

}  // namespace fa

// ---------------------------------------------------------------- no-allocation variant
//
// Same kernels as launch_decode, but the chunk partials live in a fixed array
// compiled into this library instead of memory obtained at call time, for
// callers that cannot allocate device memory during a decode step.  The array
// is part of the library's device image: every GPU on which the library's
// kernels are loaded holds these bytes until the process exits.  Every call
// shares it and it keeps the previous call's contents; nothing in it has to
// start at zero when the call begins: each call writes everything it later reads
// (the prefix offsets and every partial the merge reads).  Two calls whose kernels
// overlap on the GPU (for example on two streams) use the same bytes and race.
namespace fa {

static __device__ __align__(256) float g_decode_scratch[kNoAllocScratchBytes / sizeof(float)];

namespace {
std::mutex g_scratch_mu;
float* g_scratch_ptr[64] = {};
int g_scratch_gen[64] = {};

// Device address of g_decode_scratch on `device` (which must be current).  In
// host code the array's name is only a host-side stand-in; the address a kernel
// may use comes from cudaGetSymbolAddress, looked up once per device (and again
// after fa_release(), which a caller makes after resetting the device).
int scratch_address(int device, float** out) {
  if (device < 0 || device >= 64) return set_error(FA_ERR_CUDA, "device ordinal out of range");
  std::lock_guard<std::mutex> g(g_scratch_mu);
  const int gen = cache_generation();
  if (!g_scratch_ptr[device] || g_scratch_gen[device] != gen) {
    void* p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_decode_scratch);
    if (e != cudaSuccess || p == nullptr)
      return set_error(FA_ERR_CUDA, "cudaGetSymbolAddress(decode scratch): %s",
                       cudaGetErrorString(e));
    g_scratch_ptr[device] = static_cast<float*>(p);
    g_scratch_gen[device] = gen;
  }
  *out = g_scratch_ptr[device];
  return FA_OK;
}

// Direct schedule with its page chunks widened until the partials fit.
DecodePlan widen_direct(int B, int Hq, int Hkv, int max_pages_per_seq) {
  DecodePlan pl;
  pl.streamed = false;
  pl.pps = direct_pps(B, max_pages_per_seq);
  pl.nsplit = (max_pages_per_seq + pl.pps - 1) / pl.pps;
  finish_plan(pl, B, Hq, Hkv);
  while (pl.bytes > kNoAllocScratchBytes && pl.nsplit > 1) {
    pl.pps *= 2;
    pl.nsplit = (max_pages_per_seq + pl.pps - 1) / pl.pps;
    finish_plan(pl, B, Hq, Hkv);
  }
  return pl;
}

// Plan that fits the fixed scratch on a device with `nsm` SMs (0: no device
// known, which plans the direct schedule, the one with the smallest need).
// The streamed schedule (Hkv <= 8) is kept when it fits, if need be with fewer
// dynamic units (each then covers more half-pages) or none; otherwise the
// direct schedule with widened chunks, which needs only B * Hq rows at one
// chunk per sequence.
int plan_noalloc(int B, int Hq, int Hkv, int max_pages_per_seq, int nsm, DecodePlan* out) {
  DecodePlan pl = make_plan(B, Hq, Hkv, max_pages_per_seq, nsm);
  if (pl.streamed && pl.bytes > kNoAllocScratchBytes) {
    const long long rows_fit =
        (static_cast<long long>(kNoAllocScratchBytes) - (static_cast<long long>(B) + 2) * 4) /
        ((kDecD + 1) * 4) / Hq;
    const long long cap = rows_fit - pl.nctas - 2LL * B;
    pl.dyn_units_cap = cap > 0 ? static_cast<int>(std::min<long long>(cap, pl.dyn_units_cap)) : 0;
    finish_plan(pl, B, Hq, Hkv);
  }
  if (pl.bytes > kNoAllocScratchBytes) pl = widen_direct(B, Hq, Hkv, max_pages_per_seq);
  if (pl.bytes > kNoAllocScratchBytes)
    return set_error(FA_ERR_INVALID_ARG,
                     "fa_decode_paged_noalloc: this problem needs %zu bytes of scratch; the fixed "
                     "scratch holds %zu bytes (partial rows of %d bytes: at least B * Hq = %lld)",
                     pl.bytes, kNoAllocScratchBytes, (kDecD + 1) * 4,
                     static_cast<long long>(B) * Hq);
  *out = pl;
  return FA_OK;
}
}  // namespace

int check_decode_noalloc(int B, int Hq, int Hkv, int max_pages_per_seq, int nsm) {
  DecodePlan pl;
  return plan_noalloc(B, Hq, Hkv, max_pages_per_seq, nsm, &pl);
}

// Kernels are loaded at their first launch otherwise, and loading one may take device
// memory: the first call on a device loads all that any later one can need.
static int load_noalloc_kernels(int device) {
  static int gen[64] = {};
  static std::mutex mu;
  std::lock_guard<std::mutex> g(mu);
  if (device < 0 || device >= 64) return set_error(FA_ERR_CUDA, "device ordinal out of range");
  if (gen[device] == cache_generation()) return FA_OK;
  const void* const kernels[] = {
      reinterpret_cast<const void*>(fa_decode_scan_kernel<false>),
      reinterpret_cast<const void*>(fa_decode_stream_kernel<1, false>),
      reinterpret_cast<const void*>(fa_decode_stream_kernel<2, false>),
      reinterpret_cast<const void*>(fa_decode_stream_kernel<4, false>),
      reinterpret_cast<const void*>(fa_decode_stream_kernel<8, false>),
      reinterpret_cast<const void*>(fa_decode_stream_merge_kernel<false>),
      reinterpret_cast<const void*>(fa_decode_split_kernel<1>),
      reinterpret_cast<const void*>(fa_decode_split_kernel<2>),
      reinterpret_cast<const void*>(fa_decode_split_kernel<4>),
      reinterpret_cast<const void*>(fa_decode_split_kernel<8>),
      reinterpret_cast<const void*>(fa_decode_combine_kernel)};
  for (const void* k : kernels) {
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, k);
    if (e != cudaSuccess)
      return set_error(FA_ERR_CUDA, "cudaFuncGetAttributes: %s", cudaGetErrorString(e));
  }
  gen[device] = cache_generation();
  return FA_OK;
}

int launch_decode_noalloc(const void* q, const void* kcache, const void* vcache,
                          const int32_t* block_table, const int32_t* seq_lens, void* o, float* lse,
                          int B, int Hq, int Hkv, int max_pages_per_seq, int num_pages,
                          float scale, cudaStream_t stream, int device) {
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8)
    return set_error(FA_ERR_UNSUPPORTED, "decode supports Hq/Hkv in {1,2,4,8} (got %d)", G);
  DecodePlan pl;
  int rc = plan_noalloc(B, Hq, Hkv, max_pages_per_seq, sm_count(device), &pl);
  if (rc != FA_OK) return rc;
  float* scratch = nullptr;
  if ((rc = scratch_address(device, &scratch)) != FA_OK) return rc;
  if ((rc = load_noalloc_kernels(device)) != FA_OK) return rc;
  return run_decode(q, kcache, vcache, block_table, seq_lens, o, lse, B, Hq, Hkv,
                    max_pages_per_seq, num_pages, scale, pl, scratch, stream, device);
}

}  // namespace fa
