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
// Memory's share is 4 bytes an element forward, 6 backward; next to it stands the issue of
// instructions (108 and 154 warp instructions for two rows of 128, half of the time each).
// A group of D / 8 lanes owns a token and a few of its heads, a lane 8 elements of every
// row: four pairs, both elements of each, so neither the rotation nor its inverse
// exchanges anything between lanes; only the sums over a row do, four at a time.  The
// lane's four cosines and sines are read once for all of the group's heads.  Everything
// is computed in fp32, in packed pairs, and rounded once.
//
// 8192 tokens of 32 + 8 heads of 128 in bf16 (events around graph replays, inputs of three
// times L2; each input and output byte counted once): forward 32.7 us, 5.3 TB/s; with K and V
// to the pool 37.5 us, 5.5 TB/s; backward 45.5 us, 5.6 TB/s (copy: 6.55 TB/s); 64 tokens to
// the pool 3.0 us.
#include <algorithm>
#include <type_traits>

#include "fa_internal.h"
#include "ptx_sm100.cuh"
#include "../../include/fa.h"

namespace fa {
namespace {

using Yes = std::true_type;
using No = std::false_type;

// (8192 tokens of 32 + 8 heads of 128, four heads a task: 37.8 us with 256 threads, 33.3
// with 128, 32.7 with 64, which are slower for heads of 64.)
constexpr int kThreads = 128;
constexpr int kFewHeads = 4;     // head rows of one group's task: few or many of them
constexpr int kManyHeads = 8;
// Backward, same size: 3 blocks an SM 45.4 us, 4 (128 registers) 46.6; 5 leave L1 too small
// (75 us before the cases of the inner loop were compiled apart, 4 then 53).
constexpr int kBwdThreads = 128;
constexpr int kBwdHeads = 4;
constexpr int kBwdBlocks = 3;
constexpr int kBwdStages = 2;    // tasks of a group in shared memory
constexpr int kBwdPieces = 2 * kBwdHeads + 2;   // 16-byte pieces of a lane and task
constexpr int kBwdSmem = kBwdStages * kBwdPieces * kBwdThreads * 16;

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

// Eight elements in fp32 as four pairs (u[i], v[i]), two of each to a register pair, for
// the packed fp32 instructions: half the issue slots, which bound these kernels before
// memory does.
struct Eight {
  uint64_t u[2], v[2];
};
template <bool BF16>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
  if constexpr (BF16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
  } else {
    unpack_f16x2(w, lo, hi);
  }
}
template <bool BF16, bool INTER>
__device__ __forceinline__ Eight unpack(const Raw& r) {
  float f[8];
  unpack2<BF16>(r.a.x, f[0], f[1]);
  unpack2<BF16>(r.a.y, f[2], f[3]);
  unpack2<BF16>(r.b.x, f[4], f[5]);
  unpack2<BF16>(r.b.y, f[6], f[7]);
  Eight e;
  if constexpr (INTER) {
    e.u[0] = f2_pack(f[0], f[2]);
    e.u[1] = f2_pack(f[4], f[6]);
    e.v[0] = f2_pack(f[1], f[3]);
    e.v[1] = f2_pack(f[5], f[7]);
  } else {
    e.u[0] = f2_pack(f[0], f[1]);
    e.u[1] = f2_pack(f[2], f[3]);
    e.v[0] = f2_pack(f[4], f[5]);
    e.v[1] = f2_pack(f[6], f[7]);
  }
  return e;
}
// The elements in the order of the row: four from a, four from b.
template <bool INTER>
__device__ __forceinline__ void in_order(const Eight& e, float (&f)[8]) {
  if constexpr (INTER) {
    f2_unpack(e.u[0], f[0], f[2]);
    f2_unpack(e.u[1], f[4], f[6]);
    f2_unpack(e.v[0], f[1], f[3]);
    f2_unpack(e.v[1], f[5], f[7]);
  } else {
    f2_unpack(e.u[0], f[0], f[1]);
    f2_unpack(e.u[1], f[2], f[3]);
    f2_unpack(e.v[0], f[4], f[5]);
    f2_unpack(e.v[1], f[6], f[7]);
  }
}
template <bool BF16, bool INTER>
__device__ __forceinline__ Raw pack(const Eight& e) {
  float f[8];
  in_order<INTER>(e, f);
  auto two = [](float lo, float hi) { return BF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi); };
  Raw r;
  r.a = make_uint2(two(f[0], f[1]), two(f[2], f[3]));
  r.b = make_uint2(two(f[4], f[5]), two(f[6], f[7]));
  return r;
}
// Sum of x * y over the lane's eight elements.
__device__ __forceinline__ float dot8(const Eight& x, const Eight& y) {
  const uint64_t s0 = f2_fma(x.u[1], y.u[1], f2_mul(x.u[0], y.u[0]));
  const uint64_t s1 = f2_fma(x.v[1], y.v[1], f2_mul(x.v[0], y.v[0]));
  float lo, hi;
  f2_unpack(f2_add(s0, s1), lo, hi);
  return lo + hi;
}
__device__ __forceinline__ Eight mul8(const Eight& x, const Eight& y) {
  return {{f2_mul(x.u[0], y.u[0]), f2_mul(x.u[1], y.u[1])},
          {f2_mul(x.v[0], y.v[0]), f2_mul(x.v[1], y.v[1])}};
}
__device__ __forceinline__ Eight mul8(const Eight& x, float y) {
  const uint64_t yy = f2_pack(y, y);
  return {{f2_mul(x.u[0], yy), f2_mul(x.u[1], yy)}, {f2_mul(x.v[0], yy), f2_mul(x.v[1], yy)}};
}
__device__ __forceinline__ Eight fma8(const Eight& x, const Eight& y, const Eight& z) {
  return {{f2_fma(x.u[0], y.u[0], z.u[0]), f2_fma(x.u[1], y.u[1], z.u[1])},
          {f2_fma(x.v[0], y.v[0], z.v[0]), f2_fma(x.v[1], y.v[1], z.v[1])}};
}
__device__ __forceinline__ Eight fma8(const Eight& x, float y, const Eight& z) {
  const uint64_t yy = f2_pack(y, y);
  return fma8(x, Eight{{yy, yy}, {yy, yy}}, z);
}

// The sums over a group's LANES lanes (a power of two, aligned in the warp) of four
// values, one to a quarter of the group: lane bits LANES / 2 and LANES / 4 choose the
// value.  Five shuffles at 16 lanes, where a butterfly for each value takes sixteen.
template <int LANES>
__device__ __forceinline__ float fold4(const float (&v)[4], int l) {
  const bool high = l & (LANES / 2), odd = l & (LANES / 4);
  float a = high ? v[2] : v[0], b = high ? v[3] : v[1];
  a += __shfl_xor_sync(0xffffffffu, high ? v[0] : v[2], LANES / 2);
  b += __shfl_xor_sync(0xffffffffu, high ? v[1] : v[3], LANES / 2);
  float x = odd ? b : a;
  x += __shfl_xor_sync(0xffffffffu, odd ? a : b, LANES / 4);
#pragma unroll
  for (int d = LANES / 8; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
// Value i of a fold, from a lane that holds it.
template <int LANES>
__device__ __forceinline__ float from_fold(float x, int i) {
  return __shfl_sync(0xffffffffu, x, (i & 2 ? LANES / 2 : 0) + (i & 1 ? LANES / 4 : 0), LANES);
}

// Cosines and sines of the lane's four pairs.
struct Angles {
  uint64_t c[2], s[2];
};
// At token t.  A position outside the table and an axis outside [0, n_axes) are flagged
// (where `flag` is set) and read as 0.
template <bool INTER>
__device__ __forceinline__ Angles load_angles(const RowParams& p, const Lane<INTER>& ln,
                                              unsigned t, bool flag) {
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (ln.turns) {
    if (p.axis == nullptr) {
      int ps = __ldg(p.pos + t);
      if (ps < 0 || ps >= p.max_pos) {
        if (flag) atomicOr(p.err, kErrBadIndex);
        ps = 0;
      }
      const float* row = p.table + static_cast<size_t>(ps) * p.rot + ln.pair;
      c = __ldg(reinterpret_cast<const float4*>(row));
      s = __ldg(reinterpret_cast<const float4*>(row + p.rot / 2));
    } else {
      float cs[4], sn[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ax = __ldg(p.axis + ln.pair + i);
        bool bad = ax >= p.n_axes;
        int ps = __ldg(p.pos + static_cast<size_t>(bad ? 0 : ax) * p.T + t);
        if (ps < 0 || ps >= p.max_pos) {
          bad = true;
          ps = 0;
        }
        if (bad && flag) atomicOr(p.err, kErrBadIndex);
        const float* row = p.table + static_cast<size_t>(ps) * p.rot + ln.pair + i;
        cs[i] = __ldg(row);
        sn[i] = __ldg(row + p.rot / 2);
      }
      c = make_float4(cs[0], cs[1], cs[2], cs[3]);
      s = make_float4(sn[0], sn[1], sn[2], sn[3]);
    }
  }
  return {{f2_pack(c.x, c.y), f2_pack(c.z, c.w)}, {f2_pack(s.x, s.y), f2_pack(s.z, s.w)}};
}

// Turns the pairs by the angle (inverse: by minus the angle).
template <bool INVERSE>
__device__ __forceinline__ void turn(Eight& e, const Angles& a) {
  const uint64_t minus = f2_pack(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t neg = f2_mul(a.s[i], minus);
    const uint64_t x = e.u[i], y = e.v[i];
    e.u[i] = f2_fma(y, INVERSE ? a.s[i] : neg, f2_mul(x, a.c[i]));
    e.v[i] = f2_fma(x, INVERSE ? neg : a.s[i], f2_mul(y, a.c[i]));
  }
}

// Rows of one token in an output or its gradient: the first row of head h0, and the
// elements from one head to the next.
struct OutRows {
  size_t at, step;
  __device__ OutRows(const RowParams& p, unsigned t, int h0, int H, int D) {
    if (p.N == 0) {
      at = (static_cast<size_t>(t) * H + h0) * D;
      step = D;
    } else {
      const unsigned b = t / static_cast<unsigned>(p.N), n = t - b * p.N;
      at = ((static_cast<size_t>(b) * H + h0) * p.N + n) * D;
      step = static_cast<size_t>(p.N) * D;
    }
  }
};

// A task is (token, up to HEADS heads of q, k or, when appending, v); a group of LANES
// lanes takes one.  Neighbouring groups of a block take neighbours in memory: heads of a
// token where the outputs are token-major, tokens of a head chunk where they are heads
// first (8192 tokens of 32 + 8 heads of 128, four heads a task: 33.7 us against 35.1 the
// other way round there, 39.6 against 41.6 token-major with K and V to the pool).
struct Tasks {
  unsigned chunks, blocks;
  __host__ __device__ Tasks(unsigned T, int H, int heads, bool heads_first, int groups) {
    chunks = (H + heads - 1) / heads;
    blocks = heads_first ? (T + groups - 1) / groups * chunks : (T * chunks + groups - 1) / groups;
  }
  // group `group` of block `block`: its token (T or more: none) and chunk
  __device__ void task(unsigned block, unsigned group, unsigned groups, bool heads_first,
                       unsigned& t, unsigned& c) const {
    if (heads_first) {
      const unsigned tg = block / chunks;
      c = block - tg * chunks;
      t = tg * groups + group;
    } else {
      const unsigned i = block * groups + group;
      t = i / chunks;
      c = i - t * chunks;
    }
  }
};

template <int D, bool BF16, bool INTER, bool APPEND, int HEADS>
__global__ void __launch_bounds__(kThreads) fa_norm_rope_kernel(const RowParams p) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  // q's blocks, then k's, then v's
  const bool first = !APPEND && p.N > 0;
  Tasks tasks(p.T, p.Hq, HEADS, first, GROUPS);
  unsigned block = blockIdx.x;
  int kind = 0;                                // 0: q, 1: k, 2: v
  if (block >= tasks.blocks) {
    block -= tasks.blocks;
    kind = 1;
    tasks = Tasks(p.T, p.Hkv, HEADS, first, GROUPS);
    if (APPEND && block >= tasks.blocks) {
      block -= tasks.blocks;
      kind = 2;
    }
  }
  const int H = kind == 0 ? p.Hq : p.Hkv;
  const int l = threadIdx.x % LANES;
  unsigned mine, c;
  tasks.task(block, threadIdx.x / LANES, GROUPS, first, mine, c);
  const int h0 = c * HEADS;
  const int nh = min(HEADS, H - h0);
  bool write = mine < static_cast<unsigned>(p.T);
  const unsigned t = write ? mine : p.T - 1;   // behind the last token: reads, writes nothing
  long long slot = 0;
  if constexpr (APPEND) {
    slot = __ldg(p.slots + t);
    if (slot < 0) write = false;               // padding: nothing of the token is written
    if (slot >= p.num_slots) {
      if (write) atomicOr(p.err, kErrBadIndex);
      write = false;
    }
  }
  const Lane<INTER> own(l, p.rot);
  if (APPEND && kind == 2) {                   // v rows are copied
    const uint16_t* in = p.v + t * p.v_stride + h0 * D + 8 * l;
    uint16_t* out = p.vo + (static_cast<size_t>(slot) * p.Hkv + h0) * D + 8 * l;
    uint4 raw[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i)
      if (i < nh) raw[i] = __ldg(reinterpret_cast<const uint4*>(in + i * D));
    if (write)
#pragma unroll
      for (int i = 0; i < HEADS; ++i)
        if (i < nh) *reinterpret_cast<uint4*>(out + i * D) = raw[i];
    return;
  }
  const uint16_t* in = (kind == 0 ? p.q + t * p.q_stride : p.k + t * p.k_stride) + h0 * D;
  Raw raw[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    raw[i].a = raw[i].b = make_uint2(0, 0);
    if (i < nh) raw[i] = load_row(in + i * D, own.a, own.b);
  }
  const uint16_t* weight = kind == 0 ? p.wq : p.wk;
  const bool norm = weight != nullptr;
  Eight w;
  if (norm) w = unpack<BF16, INTER>(load_row(weight, own.a, own.b));
  const Angles ang = load_angles<INTER>(p, own, t, write);
  float r[HEADS / 4];                          // four rows' factors, one to a quarter of the group
  if (norm) {
#pragma unroll
    for (int i = 0; i < HEADS; i += 4) {
      float ss[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Eight x = unpack<BF16, INTER>(raw[i + j]);
        ss[j] = dot8(x, x);
      }
      r[i / 4] = rsqrtf(fold4<LANES>(ss, l) * (1.f / D) + p.eps);
    }
  }
  uint16_t* out;
  size_t step;
  if (APPEND && kind == 1) {
    out = p.ko + (static_cast<size_t>(slot) * p.Hkv + h0) * D;
    step = D;
  } else {
    const OutRows rows(p, t, h0, H, D);
    out = (kind == 0 ? p.qo : p.ko) + rows.at;
    step = rows.step;
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    Eight x = unpack<BF16, INTER>(raw[i]);
    if (norm) x = mul8(mul8(x, from_fold<LANES>(r[i / 4], i & 3)), w);
    if (own.turns) turn<false>(x, ang);
    if (i < nh && write) store_row(out + i * step, own.a, own.b, pack<BF16, INTER>(x));
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

// (.cg: not through L1, of which the stages in shared memory leave little)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(read ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Tasks (token group, heads) of q, then of k, dealt to the blocks of the grid in turn; a
// group's share of dw stays in registers over all of its rows, the block's is one row of
// `partial`.  While a task is computed the rows and angles of the next one are on their
// way to shared memory, to places that only the group reads.  ALL: every element is turned
// (rot == D).  What the branches on that, on a weight and on a last chunk of fewer heads
// cost inside the loop over rows (53 us against 46 at 8192 tokens of 32 + 8 heads of 128)
// is taken out of it by compiling each case.
template <int D, bool BF16, bool INTER, bool ALL>
__global__ void __launch_bounds__(kBwdThreads, kBwdBlocks)
    fa_norm_rope_bwd_kernel(const BwdParams bp) {
  constexpr int LANES = D / 8, GROUPS = kBwdThreads / LANES;
  extern __shared__ uint4 pieces[];            // [stage][piece][thread]
  __shared__ __align__(16) float sums[GROUPS][D];   // (written 16 bytes at a time)
  static_assert(__alignof__(sums) >= 16 && D % 4 == 0, "alignment of the float4 stores");
  const RowParams& p = bp.r;
  const int l = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Lane<INTER> own(l, p.rot);
  const unsigned token_groups = (static_cast<unsigned>(p.T) + GROUPS - 1) / GROUPS;
  const unsigned per_q = (p.Hq + kBwdHeads - 1) / kBwdHeads;
  const unsigned per_k = (p.Hkv + kBwdHeads - 1) / kBwdHeads;
  const unsigned q_tasks = token_groups * per_q, all_tasks = q_tasks + token_groups * per_k;

  struct Task {
    int kind, h0, nh;
    unsigned t;
    bool live;
  };
  auto task_at = [&](unsigned i) {
    Task k;
    k.kind = i >= q_tasks;
    if (k.kind) i -= q_tasks;
    const unsigned per = k.kind ? per_k : per_q;
    const unsigned tg = i / per;
    k.h0 = (i - tg * per) * kBwdHeads;
    k.nh = min(kBwdHeads, (k.kind ? p.Hkv : p.Hq) - k.h0);
    k.t = tg * GROUPS + group;
    k.live = k.t < static_cast<unsigned>(p.T);
    if (!k.live) k.t = p.T - 1;
    return k;
  };
  // table rows of the lane's pairs (one row, or four), read a task ahead of their use
  int row[4] = {0, 0, 0, 0};
  auto load_rows = [&](const Task& k) {
    if (!ALL && !own.turns) return;
    if (p.axis == nullptr) {
      row[0] = __ldg(p.pos + k.t);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ax = __ldg(p.axis + own.pair + i);
        const bool bad = ax >= p.n_axes;
        row[i] = __ldg(p.pos + static_cast<size_t>(bad ? 0 : ax) * p.T + k.t);
        if (bad && k.live) atomicOr(p.err, kErrBadIndex);
      }
    }
  };
  auto checked = [&](int ps, bool flag) {
    if (ps >= 0 && ps < p.max_pos) return ps;
    if (flag) atomicOr(p.err, kErrBadIndex);
    return 0;
  };
  auto piece = [&](int stage, int i) {
    return pieces + (stage * kBwdPieces + i) * kBwdThreads + threadIdx.x;
  };
  auto issue = [&](const Task& k, int stage) {
    const int H = k.kind ? p.Hkv : p.Hq;
    const uint16_t* x = (k.kind ? p.k + k.t * p.k_stride : p.q + k.t * p.q_stride) + k.h0 * D;
    const OutRows rows(p, k.t, k.h0, H, D);
    const uint16_t* dy = (k.kind ? bp.dko : bp.dqo) + rows.at;
#pragma unroll
    for (int i = 0; i < kBwdHeads; ++i) {
      const bool read = k.live && i < k.nh;    // (zeros otherwise: they add nothing to dw)
      const int at = i < k.nh ? i : 0;
      cp_async16(smem_u32(piece(stage, 2 * i)), x + at * D + 8 * l, read);
      cp_async16(smem_u32(piece(stage, 2 * i + 1)), dy + at * rows.step + 8 * l, read);
    }
    if (ALL || own.turns) {
      if (p.axis == nullptr) {
        const float* c = p.table + static_cast<size_t>(checked(row[0], k.live)) * p.rot + own.pair;
        cp_async16(smem_u32(piece(stage, 2 * kBwdHeads)), c, true);
        cp_async16(smem_u32(piece(stage, 2 * kBwdHeads + 1)), c + p.rot / 2, true);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* c =
              p.table + static_cast<size_t>(checked(row[i], k.live)) * p.rot + own.pair + i;
          cp_async4(smem_u32(piece(stage, 2 * kBwdHeads)) + 4 * i, c);
          cp_async4(smem_u32(piece(stage, 2 * kBwdHeads + 1)) + 4 * i, c + p.rot / 2);
        }
      }
    }
  };

  unsigned i = blockIdx.x;
  Task cur = {}, next = {};
  if (i < all_tasks) {
    cur = task_at(i);
    load_rows(cur);
    issue(cur, 0);
    if (i + gridDim.x < all_tasks) {
      next = task_at(i + gridDim.x);
      load_rows(next);
    }
  }
  cp_async_commit();
  int stage = 0;
  for (int kind = 0; kind < 2; ++kind) {
    const uint16_t* weight = kind == 0 ? p.wq : p.wk;
    const bool norm = weight != nullptr;
    const unsigned end = kind == 0 ? q_tasks : all_tasks;
    Eight w, acc = {{0, 0}, {0, 0}};
    if (norm) w = unpack<BF16, INTER>(load_row(weight, own.a, own.b));
    for (; i < end; i += gridDim.x) {
      const bool more = i + gridDim.x < all_tasks;
      Task after = {};
      if (more) {
        issue(next, stage ^ 1);
        if (i + 2 * gridDim.x < all_tasks) {
          after = task_at(i + 2 * gridDim.x);
          load_rows(after);
        }
      }
      cp_async_commit();
      cp_async_wait<1>();
      __syncwarp();                            // the group's lanes copied each other's elements
      uint16_t* dx = (kind == 0 ? bp.dq + cur.t * bp.dq_stride : bp.dk + cur.t * bp.dk_stride) +
                     cur.h0 * D;
      Angles ang;
      const ulonglong2 cs = *reinterpret_cast<const ulonglong2*>(piece(stage, 2 * kBwdHeads));
      const ulonglong2 sn = *reinterpret_cast<const ulonglong2*>(piece(stage, 2 * kBwdHeads + 1));
      ang.c[0] = cs.x, ang.c[1] = cs.y;
      ang.s[0] = sn.x, ang.s[1] = sn.y;
      auto staged = [&](int i) {               // the lane's elements of row i of the group
        const uint16_t* r = reinterpret_cast<const uint16_t*>(
            pieces + (stage * kBwdPieces + i) * kBwdThreads + group * LANES);
        Raw raw;
        raw.a = *reinterpret_cast<const uint2*>(r + own.a);
        raw.b = *reinterpret_cast<const uint2*>(r + own.b);
        return raw;
      };
      auto rows = [&](auto norm_c, auto full_c) {
        constexpr bool NORM = decltype(norm_c)::value, FULL = decltype(full_c)::value;
#pragma unroll
        for (int i0 = 0; i0 < kBwdHeads; i0 += 2) {  // two rows: four sums at a time
          if (!FULL && i0 >= cur.nh) break;
          Eight f[2], g[2], wg[2];
          float v[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            f[j] = unpack<BF16, INTER>(staged(2 * (i0 + j)));
            g[j] = unpack<BF16, INTER>(staged(2 * (i0 + j) + 1));
            if (ALL || own.turns) turn<true>(g[j], ang);
            if (NORM) {
              wg[j] = mul8(g[j], w);
              v[2 * j] = dot8(f[j], f[j]);
              v[2 * j + 1] = dot8(wg[j], f[j]);
            }
          }
          if (NORM) {
            const float sum = fold4<LANES>(v, l);
            const float rs = rsqrtf(sum * (1.f / D) + p.eps);   // of the lanes with a square
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float r = from_fold<LANES>(rs, 2 * j);
              const float k = from_fold<LANES>(sum, 2 * j + 1) * r * (-1.f / D) * r * r;
              acc = fma8(mul8(g[j], r), f[j], acc);
              g[j] = fma8(f[j], k, mul8(wg[j], r));  // r (w g - xhat mean(w g xhat))
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if ((FULL || i0 + j < cur.nh) && cur.live)
              store_row(dx + (i0 + j) * D, own.a, own.b, pack<BF16, INTER>(g[j]));
        }
      };
      const bool full = cur.nh == kBwdHeads;
      if (norm)
        full ? rows(Yes{}, Yes{}) : rows(Yes{}, No{});
      else
        full ? rows(No{}, Yes{}) : rows(No{}, No{});
      __syncwarp();                            // read by all before it is written again
      cur = next;
      next = after;
      stage ^= 1;
    }
    if (norm) {
      float a[8];
      in_order<INTER>(acc, a);
      *reinterpret_cast<float4*>(&sums[group][own.a]) = make_float4(a[0], a[1], a[2], a[3]);
      *reinterpret_cast<float4*>(&sums[group][own.b]) = make_float4(a[4], a[5], a[6], a[7]);
      __syncthreads();
      for (int d = threadIdx.x; d < D; d += kBwdThreads) {
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) s += sums[g][d];
        bp.partial[(static_cast<size_t>(kind) * gridDim.x + blockIdx.x) * D + d] = s;
      }
      __syncthreads();
    }
  }
  cp_async_wait<0>();
  pdl_launch_dependents();
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
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  const float* from = bp.partial + static_cast<size_t>(kind) * rows * D + d;
#pragma unroll 2
  for (int r = warp; r < rows; r += 128)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + 32 * i < rows) s[i] += __ldcg(from + static_cast<size_t>(r + 32 * i) * D);
  sums[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
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

template <int D, bool BF16>
void launch_rows(const RowParams& r, bool append, bool interleaved, int nsm,
                 cudaStream_t stream) {
  const int groups = kThreads / (D / 8);
  const bool first = r.N > 0;
  auto blocks = [&](int heads) {
    const unsigned kv = Tasks(r.T, r.Hkv, heads, first, groups).blocks;
    return Tasks(r.T, r.Hq, heads, first, groups).blocks + (append ? 2 * kv : kv);
  };
  // Eight heads a task read the weights and angles half as often and keep more bytes in
  // flight; four make twice the blocks.  32 + 8 heads of 128, us of four / eight: 64 tokens
  // 2.9 / 3.3, 512 3.9 / 4.1, 1024 (640 blocks of eight) 4.9 / 5.1, 2048 (1280) 8.24 / 8.21,
  // 8192 33.5 / 32.5, 16384 62.4 / 57.8; 8186 of 8 + 8 heads of 64 (1024) 9.0 / 8.0.
  const bool many = blocks(kManyHeads) >= 5u * nsm;
  auto run = [&](auto inter, auto app, auto heads) {
    constexpr int HEADS = decltype(heads)::value;
    fa_norm_rope_kernel<D, BF16, decltype(inter)::value, decltype(app)::value, HEADS>
        <<<blocks(HEADS), kThreads, 0, stream>>>(r);
  };
  auto run_heads = [&](auto inter, auto app) {
    many ? run(inter, app, std::integral_constant<int, kManyHeads>{})
         : run(inter, app, std::integral_constant<int, kFewHeads>{});
  };
  if constexpr (BF16) {                        // the page pool is bf16
    if (append) {
      interleaved ? run_heads(Yes{}, Yes{}) : run_heads(No{}, Yes{});
      return;
    }
  }
  interleaved ? run_heads(Yes{}, No{}) : run_heads(No{}, No{});
}

template <int D, bool BF16>
void launch_bwd(const BwdParams& bp, bool interleaved, int blocks, cudaStream_t stream) {
  auto run = [&](auto inter, auto all) {
    fa_norm_rope_bwd_kernel<D, BF16, decltype(inter)::value, decltype(all)::value>
        <<<blocks, kBwdThreads, kBwdSmem, stream>>>(bp);
  };
  const bool all = bp.r.rot == D;
  if (interleaved)
    all ? run(Yes{}, Yes{}) : run(Yes{}, No{});
  else
    all ? run(No{}, Yes{}) : run(No{}, No{});
}

}  // namespace

int launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream, int device) {
  RowParams r;
  fill(&r, a, device);
  if (!r.err) return set_error(FA_ERR_CUDA, "device error word unavailable");
  const bool append = a.slot_map != nullptr;
  const int nsm = device_sm_count(device);
  if (nsm <= 0) return set_error(FA_ERR_CUDA, "cannot read the SM count of device %d", device);
  if (a.D == 128)
    a.bf16 ? launch_rows<128, true>(r, append, a.interleaved, nsm, stream)
           : launch_rows<128, false>(r, append, a.interleaved, nsm, stream);
  else
    a.bf16 ? launch_rows<64, true>(r, append, a.interleaved, nsm, stream)
           : launch_rows<64, false>(r, append, a.interleaved, nsm, stream);
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
  const int groups = kBwdThreads / (a.D / 8);
  const long long chunks =
      (a.Hq + kBwdHeads - 1) / kBwdHeads + (a.Hkv + kBwdHeads - 1) / kBwdHeads;
  const long long tasks = (static_cast<long long>(a.T) + groups - 1) / groups * chunks;
  const int blocks = static_cast<int>(std::min<long long>(
      std::max<long long>(tasks, 1), std::min(kBwdBlocks * nsm, FA_QK_NORM_ROPE_SCRATCH_ROWS)));
  if (a.D == 128)
    a.bf16 ? launch_bwd<128, true>(bp, a.interleaved, blocks, stream)
           : launch_bwd<128, false>(bp, a.interleaved, blocks, stream);
  else
    a.bf16 ? launch_bwd<64, true>(bp, a.interleaved, blocks, stream)
           : launch_bwd<64, false>(bp, a.interleaved, blocks, stream);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && (a.q_weight || a.k_weight)) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.D / 32, 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, fa_norm_rope_dw_kernel, bp, a.D, blocks);
  }
  if (e != cudaSuccess)
    return set_error(FA_ERR_CUDA, "norm + rotation backward launch: %s", cudaGetErrorString(e));
  return FA_OK;
}

}  // namespace fa
