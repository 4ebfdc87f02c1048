// Per-head RMS norm and rotary position rotation of queries and keys in one pass,
// the same with K and V written into the page pool, and the backward pass.
//
// For a head row x of D elements with weight w,
//     xhat = x / sqrt(mean(x^2) + eps),   y = R (w * xhat),
// where R turns element pair j by the angle whose cosine and sine are column j of
// the token's row of a table.  The backward pass of dy is
//     g = R^T dy,   dw = sum over rows of g * xhat,
//     dx = (w * g - xhat * mean(w * g * xhat)) / sqrt(mean(x^2) + eps).
//
// Bound by memory: 4 bytes an element forward, 6 backward, against a few dozen
// instructions.  A group of D / 8 lanes owns a token and a few of its heads, a
// lane 8 elements of every row: four pairs, both elements of each, so neither the
// rotation nor its inverse exchanges anything between lanes; only the sums over a
// row do (xor shuffles inside the group).  The lane's four cosines and sines are
// read once for all of the group's heads.  Everything is computed in fp32 and
// rounded once.
#include <algorithm>

#include "fa_internal.h"
#include "ptx_sm100.cuh"
#include "../../include/fa.h"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;        // head rows of one group's task

struct RowParams {
  const uint16_t *q, *k, *v;     // token-major rows, q_stride (...) elements between tokens
  const uint16_t *wq, *wk;       // [D] or null: no norm
  const float* table;            // [max_pos, rot]: cosines of the rot / 2 pairs, then sines
  const int32_t* pos;            // [n_axes, T]
  const uint8_t* axis;           // [rot / 2] axis of every pair, or null: axis 0
  uint16_t *qo, *ko, *vo;        // outputs (append: ko and vo are the pools)
  const long long* slots;        // append: pool slot of every token, negative: padding
  long long q_stride, k_stride, v_stride, num_slots;
  int T, N, Hq, Hkv;             // heads first: outputs [T / N, H, N, D]; N = 0: [T, H, D]
  int rot, n_axes, max_pos;
  float eps;
  int* err;
};

// The lane's eight elements of a row: [a, a + 4) and [b, b + 4).  Pairs are
// (a + i, b + i) when rotating halves against each other, adjacent elements when
// interleaved (then b = a + 4); a lane of elements that are not rotated
// (8 * lane >= rot) just owns eight of them.
template <bool INTER>
struct Lane {
  int a, b, pair;
  bool turns;
  __device__ Lane(int l, int rot) {
    turns = 8 * l < rot;
    pair = 4 * l;
    if (INTER || !turns) {
      a = 8 * l;
      b = a + 4;
    } else {
      a = 4 * l;
      b = rot / 2 + 4 * l;
    }
  }
};

struct Raw {
  uint2 a, b;
};
__device__ __forceinline__ Raw load_row(const uint16_t* row, int a, int b) {
  Raw r;
  r.a = __ldg(reinterpret_cast<const uint2*>(row + a));
  r.b = __ldg(reinterpret_cast<const uint2*>(row + b));
  return r;
}
__device__ __forceinline__ void store_row(uint16_t* row, int a, int b, const Raw& r) {
  *reinterpret_cast<uint2*>(row + a) = r.a;
  *reinterpret_cast<uint2*>(row + b) = r.b;
}
template <bool BF16>
__device__ __forceinline__ void unpack2(uint32_t u, float& lo, float& hi) {
  if constexpr (BF16) {
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float(u & 0xffff0000u);
  } else {
    unpack_f16x2(u, lo, hi);
  }
}
template <bool BF16>
__device__ __forceinline__ void unpack(const Raw& r, float (&f)[8]) {
  unpack2<BF16>(r.a.x, f[0], f[1]);
  unpack2<BF16>(r.a.y, f[2], f[3]);
  unpack2<BF16>(r.b.x, f[4], f[5]);
  unpack2<BF16>(r.b.y, f[6], f[7]);
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return BF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}
template <bool BF16>
__device__ __forceinline__ Raw pack(const float (&f)[8]) {
  Raw r;
  r.a = make_uint2(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]));
  r.b = make_uint2(pack2<BF16>(f[4], f[5]), pack2<BF16>(f[6], f[7]));
  return r;
}

// Sum over the LANES lanes of a group (a power of two, aligned in the warp).
template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int d = LANES / 2; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// Cosines and sines of the lane's four pairs at token t.  A position outside the
// table and an axis outside [0, n_axes) are flagged and read as 0.
template <bool INTER>
__device__ __forceinline__ void load_angles(const RowParams& p, const Lane<INTER>& ln, int t,
                                            float (&c)[4], float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (!ln.turns) return;
  if (p.axis == nullptr) {
    int ps = __ldg(p.pos + t);
    if (ps < 0 || ps >= p.max_pos) {
      atomicOr(p.err, kErrBadIndex);
      ps = 0;
    }
    const float* row = p.table + static_cast<size_t>(ps) * p.rot + ln.pair;
    const float4 cv = __ldg(reinterpret_cast<const float4*>(row));
    const float4 sv = __ldg(reinterpret_cast<const float4*>(row + p.rot / 2));
    c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
    s[0] = sv.x, s[1] = sv.y, s[2] = sv.z, s[3] = sv.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int ax = __ldg(p.axis + ln.pair + i);
      bool bad = ax >= p.n_axes;
      int ps = __ldg(p.pos + static_cast<size_t>(bad ? 0 : ax) * p.T + t);
      if (ps < 0 || ps >= p.max_pos) {
        bad = true;
        ps = 0;
      }
      if (bad) atomicOr(p.err, kErrBadIndex);
      const float* row = p.table + static_cast<size_t>(ps) * p.rot + ln.pair + i;
      c[i] = __ldg(row);
      s[i] = __ldg(row + p.rot / 2);
    }
  }
}

// Turns the lane's pairs by the angle (inverse: by minus the angle).
template <bool INTER, bool INVERSE>
__device__ __forceinline__ void turn(float (&f)[8], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = INTER ? 2 * i : i, v = INTER ? 2 * i + 1 : i + 4;
    const float x = f[u], y = f[v];
    const float sn = INVERSE ? -s[i] : s[i];
    f[u] = x * c[i] - y * sn;
    f[v] = y * c[i] + x * sn;
  }
}

__device__ __forceinline__ size_t out_row(const RowParams& p, int t, int h, int H) {
  if (p.N == 0) return static_cast<size_t>(t) * H + h;
  const int b = t / p.N;
  return (static_cast<size_t>(b) * H + h) * p.N + (t - b * p.N);
}

// A task is (token, up to kHeads heads of q, k or, when appending, v).
struct Chunks {
  int nq, nk, nv;
  __host__ __device__ Chunks(int Hq, int Hkv, bool append)
      : nq((Hq + kHeads - 1) / kHeads), nk((Hkv + kHeads - 1) / kHeads), nv(append ? nk : 0) {}
  __host__ __device__ int per_token() const { return nq + nk + nv; }
};

template <int D, bool BF16, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kThreads) fa_norm_rope_kernel(const RowParams p) {
  constexpr int LANES = D / 8;
  const Chunks ch(p.Hq, p.Hkv, APPEND);
  const int l = threadIdx.x % LANES;
  const long long task =
      (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / LANES;
  const int per = ch.per_token();
  const bool live = task < static_cast<long long>(p.T) * per;
  const int t = live ? static_cast<int>(task / per) : 0;
  int c = live ? static_cast<int>(task - static_cast<long long>(t) * per) : 0;
  int kind = 0;                                // 0: q, 1: k, 2: v
  if (c >= ch.nq) {
    c -= ch.nq;
    kind = 1;
    if (c >= ch.nk) {
      c -= ch.nk;
      kind = 2;
    }
  }
  const int H = kind == 0 ? p.Hq : p.Hkv;
  const int h0 = c * kHeads;
  const int nh = live ? min(kHeads, H - h0) : 0;
  long long slot = 0;
  bool write = live;
  if constexpr (APPEND) {
    if (live) slot = __ldg(p.slots + t);
    if (slot < 0) write = false;               // padding: nothing of the token is written
    if (slot >= p.num_slots) {
      atomicOr(p.err, kErrBadIndex);
      write = false;
    }
  }
  const Lane<INTER> own(l, p.rot);
  const Lane<true> plain(l, 0);                // v rows are copied: eight adjacent elements
  const int a = kind == 2 ? plain.a : own.a, b = kind == 2 ? plain.b : own.b;
  const uint16_t* in = kind == 0 ? p.q + t * p.q_stride
                                 : kind == 1 ? p.k + t * p.k_stride : p.v + t * p.v_stride;
  in += h0 * D;
  Raw raw[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (i < nh && write) raw[i] = load_row(in + i * D, a, b);
    else raw[i].a = raw[i].b = make_uint2(0, 0);
  const uint16_t* weight = kind == 0 ? p.wq : p.wk;
  float w[8], cs[4], sn[4];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = 1.f;
  const bool norm = weight != nullptr && kind != 2;
  const bool turns = own.turns && write && kind != 2;
  if (norm) unpack<BF16>(load_row(weight, a, b), w);
  if (turns) load_angles<INTER>(p, own, t, cs, sn);
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    float f[8];
    unpack<BF16>(raw[i], f);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
    ss = group_sum<LANES>(ss);
    if (norm) {
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] * r * w[e];
    }
    if (turns) turn<INTER, false>(f, cs, sn);
    if (i < nh && write) {
      uint16_t* out;
      if (kind == 0)
        out = p.qo + out_row(p, t, h0 + i, p.Hq) * D;
      else if (APPEND)
        out = (kind == 1 ? p.ko : p.vo) + (static_cast<size_t>(slot) * p.Hkv + h0 + i) * D;
      else
        out = p.ko + out_row(p, t, h0 + i, p.Hkv) * D;
      store_row(out, a, b, kind == 2 ? raw[i] : pack<BF16>(f));
    }
  }
}

struct BwdParams {
  RowParams r;                   // q, k, weights, angles and sizes of the forward
  const uint16_t *dqo, *dko;     // gradients of the outputs, in the outputs' layout
  uint16_t *dq, *dk;             // gradients of the inputs, token-major
  long long dq_stride, dk_stride;
  float* partial;                // [2][gridDim.x][D]: every block's sum over its rows
  float *dwq, *dwk;
};

// Tasks of q, then of k, dealt to the groups of the grid in turn; the group's share of
// dw stays in registers over all of its rows, the block's is one row of `partial`.
template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads) fa_norm_rope_bwd_kernel(const BwdParams bp) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  __shared__ float sums[GROUPS][D];
  const RowParams& p = bp.r;
  const int l = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Lane<INTER> own(l, p.rot);
  for (int kind = 0; kind < 2; ++kind) {
    const int H = kind == 0 ? p.Hq : p.Hkv;
    const int per = (H + kHeads - 1) / kHeads;
    const long long tasks = static_cast<long long>(p.T) * per;
    const uint16_t* weight = kind == 0 ? p.wq : p.wk;
    const bool norm = weight != nullptr;
    float w[8], acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] = 1.f;
      acc[e] = 0.f;
    }
    if (norm) unpack<BF16>(load_row(weight, own.a, own.b), w);
    // the whole block goes round together: the sums over a row use full warps
    for (long long first = static_cast<long long>(blockIdx.x) * GROUPS; first < tasks;
         first += static_cast<long long>(gridDim.x) * GROUPS) {
      const long long task = first + group;
      const bool live = task < tasks;
      const int t = live ? static_cast<int>(task / per) : 0;
      const int h0 = live ? static_cast<int>(task - static_cast<long long>(t) * per) * kHeads : 0;
      const int nh = live ? min(kHeads, H - h0) : 0;
      const uint16_t* x = (kind == 0 ? p.q + t * p.q_stride : p.k + t * p.k_stride) + h0 * D;
      const uint16_t* dy = kind == 0 ? bp.dqo : bp.dko;
      uint16_t* dx =
          (kind == 0 ? bp.dq + t * bp.dq_stride : bp.dk + t * bp.dk_stride) + h0 * D;
      Raw rx[kHeads], rg[kHeads];
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        rx[i].a = rx[i].b = rg[i].a = rg[i].b = make_uint2(0, 0);
        if (i < nh) {
          rx[i] = load_row(x + i * D, own.a, own.b);
          rg[i] = load_row(dy + out_row(p, t, h0 + i, H) * D, own.a, own.b);
        }
      }
      float cs[4], sn[4];
      const bool turns = own.turns && live;
      if (turns) load_angles<INTER>(p, own, t, cs, sn);
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        float f[8], g[8];
        unpack<BF16>(rx[i], f);
        unpack<BF16>(rg[i], g);
        if (turns) turn<INTER, true>(g, cs, sn);
        if (norm) {
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss = fmaf(f[e], f[e], ss);
            dot = fmaf(g[e] * w[e], f[e], dot);
          }
          ss = group_sum<LANES>(ss);
          dot = group_sum<LANES>(dot);
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const float m = dot * r * (1.f / D);         // mean(w * g * xhat)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float xh = f[e] * r;
            acc[e] = fmaf(g[e], xh, acc[e]);
            g[e] = r * (g[e] * w[e] - xh * m);
          }
        }
        if (i < nh) store_row(dx + i * D, own.a, own.b, pack<BF16>(g));
      }
    }
    if (norm) {
      *reinterpret_cast<float4*>(&sums[group][own.a]) =
          make_float4(acc[0], acc[1], acc[2], acc[3]);
      *reinterpret_cast<float4*>(&sums[group][own.b]) =
          make_float4(acc[4], acc[5], acc[6], acc[7]);
      __syncthreads();
      if (threadIdx.x < D) {
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) s += sums[g][threadIdx.x];
        bp.partial[(static_cast<size_t>(kind) * gridDim.x + blockIdx.x) * D + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

// dw: the blocks' rows of `partial` summed in a fixed order (the same bits every
// call).  Block (column group, q or k): 32 columns, 32 warps over the rows.
__global__ void __launch_bounds__(1024) fa_norm_rope_dw_kernel(const BwdParams bp, int D,
                                                               int rows) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kind = blockIdx.y, d = blockIdx.x * 32 + lane;
  float* out = kind == 0 ? bp.dwq : bp.dwk;
  pdl_wait();
  if ((kind == 0 ? bp.r.wq : bp.r.wk) == nullptr) return;
  float s = 0.f;
  for (int r = warp; r < rows; r += 32)
    s += __ldcg(bp.partial + (static_cast<size_t>(kind) * rows + r) * D + d);
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) total += sums[i][lane];
    out[d] = total;
  }
}

void fill(RowParams* r, const NormRopeArgs& a, int device) {
  r->q = static_cast<const uint16_t*>(a.q);
  r->k = static_cast<const uint16_t*>(a.k);
  r->v = static_cast<const uint16_t*>(a.v);
  r->wq = static_cast<const uint16_t*>(a.q_weight);
  r->wk = static_cast<const uint16_t*>(a.k_weight);
  r->table = a.table;
  r->pos = a.positions;
  r->axis = a.n_axes > 1 ? a.pair_axis : nullptr;
  r->qo = static_cast<uint16_t*>(a.q_out);
  r->ko = static_cast<uint16_t*>(a.k_out);
  r->vo = static_cast<uint16_t*>(a.v_out);
  r->slots = reinterpret_cast<const long long*>(a.slot_map);
  r->q_stride = a.q_stride;
  r->k_stride = a.k_stride;
  r->v_stride = a.v_stride;
  r->num_slots = a.num_slots;
  r->T = a.T;
  r->N = a.heads_first ? a.N : 0;
  r->Hq = a.Hq;
  r->Hkv = a.Hkv;
  r->rot = a.rot_dim;
  r->n_axes = a.n_axes;
  r->max_pos = a.max_pos;
  r->eps = a.eps;
  r->err = device_error_word(device);
}

template <int D, bool BF16, bool INTER>
void launch_rows(const RowParams& r, bool append, unsigned blocks, cudaStream_t stream) {
  if constexpr (BF16) {
    if (append) {
      fa_norm_rope_kernel<D, true, INTER, true><<<blocks, kThreads, 0, stream>>>(r);
      return;
    }
  }
  fa_norm_rope_kernel<D, BF16, INTER, false><<<blocks, kThreads, 0, stream>>>(r);
}

}  // namespace

int launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream, int device) {
  RowParams r;
  fill(&r, a, device);
  if (!r.err) return set_error(FA_ERR_CUDA, "device error word unavailable");
  const bool append = a.slot_map != nullptr;
  const long long lanes =
      static_cast<long long>(a.T) * Chunks(a.Hq, a.Hkv, append).per_token() * (a.D / 8);
  const long long blocks = (lanes + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return set_error(FA_ERR_UNSUPPORTED, "too many rows for one launch");
  const unsigned n = static_cast<unsigned>(blocks);
#define FA_ROWS(D_, BF_, IN_) launch_rows<D_, BF_, IN_>(r, append, n, stream)
#define FA_ROWS_T(D_, BF_) (a.interleaved ? FA_ROWS(D_, BF_, true) : FA_ROWS(D_, BF_, false))
  if (a.D == 128)
    a.bf16 ? FA_ROWS_T(128, true) : FA_ROWS_T(128, false);
  else
    a.bf16 ? FA_ROWS_T(64, true) : FA_ROWS_T(64, false);
#undef FA_ROWS_T
#undef FA_ROWS
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess)
    return set_error(FA_ERR_CUDA, "norm + rotation launch: %s", cudaGetErrorString(e));
  return FA_OK;
}

int launch_norm_rope_bwd(const NormRopeArgs& a, const NormRopeGrads& g, cudaStream_t stream,
                         int device) {
  BwdParams bp;
  fill(&bp.r, a, device);
  if (!bp.r.err) return set_error(FA_ERR_CUDA, "device error word unavailable");
  bp.dqo = static_cast<const uint16_t*>(g.dq_out);
  bp.dko = static_cast<const uint16_t*>(g.dk_out);
  bp.dq = static_cast<uint16_t*>(g.dq);
  bp.dk = static_cast<uint16_t*>(g.dk);
  bp.dq_stride = g.dq_stride;
  bp.dk_stride = g.dk_stride;
  bp.partial = g.scratch;
  bp.dwq = g.dq_weight;
  bp.dwk = g.dk_weight;
  const int nsm = device_sm_count(device);
  if (nsm <= 0) return set_error(FA_ERR_CUDA, "cannot read the SM count of device %d", device);
  const int groups = kThreads / (a.D / 8);
  const Chunks ch(a.Hq, a.Hkv, false);
  const long long tasks = static_cast<long long>(a.T) * std::max(ch.nq, ch.nk);
  const int blocks = static_cast<int>(std::min<long long>(
      std::max<long long>((tasks + groups - 1) / groups, 1),
      std::min(4 * nsm, FA_QK_NORM_ROPE_SCRATCH_ROWS)));
#define FA_BWD(D_, BF_, IN_) \
  fa_norm_rope_bwd_kernel<D_, BF_, IN_><<<blocks, kThreads, 0, stream>>>(bp)
#define FA_BWD_T(D_, BF_)    \
  if (a.interleaved)         \
    FA_BWD(D_, BF_, true);   \
  else                       \
    FA_BWD(D_, BF_, false)
  if (a.D == 128) {
    if (a.bf16) { FA_BWD_T(128, true); } else { FA_BWD_T(128, false); }
  } else {
    if (a.bf16) { FA_BWD_T(64, true); } else { FA_BWD_T(64, false); }
  }
#undef FA_BWD_T
#undef FA_BWD
  if (a.q_weight || a.k_weight)
    fa_norm_rope_dw_kernel<<<dim3(a.D / 32, 2), 1024, 0, stream>>>(bp, a.D, blocks);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess)
    return set_error(FA_ERR_CUDA, "norm + rotation backward launch: %s", cudaGetErrorString(e));
  return FA_OK;
}

}  // namespace fa
