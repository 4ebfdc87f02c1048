// Attention of a whole decode batch over the keys that all of its sequences share.
//
// One query token per sequence makes decode a matrix-vector product per sequence.
// Over a prefix that every sequence shares it is a matrix-matrix product: the rows of
// KV head g are the G = Hq / Hkv query heads of all B sequences, B * G of them, and the
// prefix is read once for all instead of once per sequence.  Per key the rows cost
// 4 * B * Hq * 128 flops against 4 * 128 * Hkv bytes, so a batch of a few dozen rows a
// KV head is bound by HBM and one of a few hundred by the tensor cores.
//
// The work is a list of (KV head, group of pairs of 128-row tiles, 128-key tile) units for
// teams of CTAs, a pair each; of the C teams that prefix_split.cuh gives it, team c takes
// the equal contiguous share [c W / C, (c + 1) W / C) of its W units, whatever the prefix
// length, so that few rows over a long prefix still use every SM.  A share that spans
// several (head, group) items is cut into segments; every segment writes its normalised
// partial output and LSE in fp32 to a member's slot of c + item (unique: along the list c,
// item or both grow by one), and the decode merge joins a row's segments with the partials
// of its own keys by their LSE.
//
// Within a segment this is the online-softmax pipeline of the forward kernel on
// tcgen05 (see there for the roles and the tensor-memory plan): a producer warp gathers
// the 16-token pages of K and V by TMA into a ring of four 128-key tiles, one warp
// issues S = Q K^T and O += P V, two softmax warpgroups own a row tile each.
//
// 256 sequences of 32 + 8 heads over 37888 shared keys (1024 rows a KV head, 158 GFLOP):
// 146 us, 1085 TFLOP/s; from one key count to the next 2.0 us a unit, the forward kernel's
// rate, and 18 us for two segments' starts and ends.  With every page id the same (L2)
// 140 us: the chain of S, softmax and P V bounds it, not memory.  (This kernel alone: in a
// call of 256 sequences over 32768 keys its last CTA ends at 136 of 169 us, the own keys'
// last at 151, the merge at 169.)  33 rows a KV head, 16 heads: 1.8 us a unit (one row
// tile), 5.4 TB/s.
#include <algorithm>

#include "fa_internal.h"
#include "ptx_sm100.cuh"
#include "prefix_split.cuh"
#include "../../include/fa.h"

namespace fa {
namespace {

constexpr int kD = 128;
constexpr int kBM = 128;         // query rows per tile = TMEM lanes
constexpr int kBN = kPrefixTile; // keys per tile
constexpr int kPageTok = 16;
constexpr float kTau = 8.0f;     // lazy-rescale threshold (log2 units), as in the forward
constexpr int kThreads = 384;
constexpr uint32_t kRegsControl = 72;    // warps 8-11
constexpr uint32_t kRegsSoftmax = 216;   // warps 0-7
static_assert(kRegsControl * 128 + kRegsSoftmax * 256 <= 384 * 168, "register split");

constexpr int kChunks = kD / 64;           // 128-byte swizzle atoms along D
constexpr int kChunkBytes = kBM * 128;
constexpr int kTileBytes = kBM * kD * 2;
constexpr int kSlots = 4;
constexpr int kQOff = 0;
constexpr int kKVOff = 2 * kTileBytes;
constexpr int kBarOff = kKVOff + kSlots * kTileBytes;
constexpr int kNumBars = 2 + 2 * kSlots + 2 + 4 + 2 + 1 + 1;
constexpr int kMiscOff = kBarOff + kNumBars * 8;
constexpr int kStageOff = (kMiscOff + 16 + 127) & ~127;
constexpr int kStageBytes = 32 * 128;      // a warp's 32 rows x 32 fp32 columns
constexpr int kSmemBytes = kStageOff + 8 * kStageBytes + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct PrefixParams {
  PrefixWork w;
  const int32_t* table;
  float* ws_o;       // [slot][256][128] normalised partial outputs
  float* ws_lse;     // [slot][256] natural log
  int B, G, Hkv, num_pages;
  float scale_log2;
  int* err;
  uint64_t timeout_ns;
};

// A segment: key tiles [j0, j1) of rows [256 pair, 256 pair + 256) of KV head hkv, whose
// partial results go to slot `slot`.
struct Segment {
  int slot, hkv, pair, j0, j1;
  bool two;          // the pair's second row tile holds rows
};
struct SegmentWalker {
  int u, u1, nt, team, member;
  __device__ SegmentWalker(int cta, const PrefixWork& w, const PrefixSplit& sp) {
    nt = sp.nt;
    u = u1 = 0;
    team = cta / w.team;
    member = cta - team * w.team;
    if (team < sp.teams) {
      u = share_edge(team, sp.units, sp.teams);
      u1 = share_edge(team + 1, sp.units, sp.teams);
    }
  }
  __device__ bool next(const PrefixParams& p, Segment& s) {
    while (u < u1) {
      const int item = u / nt;
      s.slot = (team + item) * p.w.team + member;
      s.j0 = u - item * nt;
      s.j1 = min(nt, s.j0 + (u1 - u));
      s.hkv = item / p.w.pair_groups;
      s.pair = (item - s.hkv * p.w.pair_groups) * p.w.team + member;
      s.two = s.pair * 256 + kBM < p.B * p.G;
      u += s.j1 - s.j0;
      if (s.pair < p.w.pairs) return true;       // else the last group has fewer pairs
    }
    return false;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    fa_prefix_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const PrefixParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int C = gridDim.x;
  const int cta = blockIdx.x;

  auto bar = [&](int i) -> uint32_t { return sbase + kBarOff + 8 * i; };
  auto q_full = [&](int t) { return bar(t); };
  auto kv_full = [&](int s) { return bar(2 + s); };
  auto kv_empty = [&](int s) { return bar(2 + kSlots + s); };
  auto s_full = [&](int t) { return bar(2 + 2 * kSlots + t); };
  auto p_half = [&](int t, int h) { return bar(4 + 2 * kSlots + 2 * t + h); };
  auto o_full = [&](int t) { return bar(8 + 2 * kSlots + t); };
  const uint32_t mma_done = bar(10 + 2 * kSlots);
  const uint32_t q_empty = bar(11 + 2 * kSlots);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kMiscOff + 4);

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 1);
      mbar_init(s_full(t), 1);
      mbar_init(p_half(t, 0), kBM);
      mbar_init(p_half(t, 1), kBM);
      mbar_init(o_full(t), 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 1);
    }
    mbar_init(mma_done, 1);
    mbar_init(q_empty, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // Everything above overlaps the scan of the lengths; its sum decides the split.
  pdl_wait();
  const PrefixSplit sp = prefix_split(p.w, C);
  // The next kernel of the stream reads the scan's output without waiting for this grid:
  // the scan has finished.
  pdl_launch_dependents();
  const int pages = sp.pages;
  const int n_keys = pages * kPageTok;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    regs_dec<kRegsControl>();
    if (warp == 8) {
      // ------------------------------------------------------------ TMA producer
      // A key tile is eight pages: lane pg * kChunks + ch reads page pg's id and issues
      // its 64-column box ch.  Pages past the prefix lie past the pool for the tensor
      // map, which fills them with zeros (their scores are masked, and zeros times a
      // zero weight stay zero whatever the pool holds); so do ids outside the pool,
      // which are flagged.
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
      }
      auto wait_all = [&](uint32_t br, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(br, parity, abort_flag, p.err, p.timeout_ns));
      };
      constexpr int kBoxes = (kBN / kPageTok) * kChunks;
      const int pg = lane / kChunks, ch = lane % kChunks;
      int pos = 0, segs = 0;
      bool ok = true;
      SegmentWalker walk(cta, p.w, sp);
      Segment s;
      while (ok && walk.next(p, s)) {
        if (segs > 0 && !wait_all(q_empty, (segs - 1) & 1)) break;
        if (lane == 0) {
          for (int t = 0; t < 2; ++t) {
            mbar_arrive_expect_tx(q_full(t), kTileBytes);
            const uint32_t dst = sbase + kQOff + t * kTileBytes;
            for (int c2 = 0; c2 < kChunks; ++c2)   // [B, Hq, D]: box {64, G, 128 / G}
              tma_load_3d(dst + c2 * kChunkBytes, &tmQ, q_full(t), c2 * 64, s.hkv * p.G,
                          (s.pair * 256 + t * kBM) / p.G);
          }
        }
        ++segs;
        for (int j = s.j0; j < s.j1 && ok; ++j) {
          int page = p.num_pages;                  // past the pool: zeros
          if (lane < kBoxes) {
            const int k = j * (kBN / kPageTok) + pg;
            if (k < pages) {
              page = __ldg(p.table + k);
              if (page < 0 || page >= p.num_pages) {
                atomicOr(p.err, kErrBadIndex);
                page = p.num_pages;
              }
            }
          }
          for (int w = 0; w < 2; ++w, ++pos) {
            const int slot = pos % kSlots;
            const uint32_t ph = (pos / kSlots) & 1;
            if (!wait_all(kv_empty(slot), ph ^ 1)) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(kv_full(slot), kTileBytes);
            __syncwarp();
            const uint32_t dst = sbase + kKVOff + slot * kTileBytes;
            const void* tm = w ? static_cast<const void*>(&tmV) : static_cast<const void*>(&tmK);
            if (lane < kBoxes)
              tma_load_3d(dst + ch * kChunkBytes + pg * kPageTok * 128, tm, kv_full(slot),
                          ch * 64, s.hkv, page * kPageTok);
          }
        }
      }
      // Every issued copy must land before the CTA may exit (also on abort).
      if (lane == 0) {
        volatile int no_abort = 0;
        if (segs > 0)
          for (int t = 0; t < 2; ++t)
            mbar_wait(q_full(t), (segs - 1) & 1, &no_abort, p.err, p.timeout_ns);
        for (int sl = 0; sl < kSlots && sl < pos; ++sl) {
          const int last = sl + ((pos - 1 - sl) / kSlots) * kSlots;
          mbar_wait(kv_full(sl), (last / kSlots) & 1, &no_abort, p.err, p.timeout_ns);
        }
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------ MMA issuer
      const bool leader = elect_one();
      constexpr uint32_t idesc_s = idesc_f16(kBM, kBN, true, false);
      constexpr uint32_t idesc_pv = idesc_f16(kBM, kD, true, true);
      auto slot_of = [&](int pos) { return pos % kSlots; };
      auto phase_of = [&](int pos) { return static_cast<uint32_t>((pos / kSlots) & 1); };
      auto wait = [&](uint32_t br, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(br, parity, abort_flag, p.err, p.timeout_ns));
      };
      auto commit = [&](uint32_t br) {
        if (leader) tc_commit(br);
      };
      const uint64_t desc_q0 = smem_desc_sw128(sbase + kQOff, 16, 1024);
      const uint64_t desc_q1 = smem_desc_sw128(sbase + kQOff + kTileBytes, 16, 1024);
      const uint64_t desc_k = smem_desc_sw128(sbase + kKVOff, 16, 1024);            // K-major
      const uint64_t desc_v = smem_desc_sw128(sbase + kKVOff, kChunkBytes, 1024);   // MN-major
      auto issue_s = [&](int t, int slot) {
        const uint64_t a0 = t ? desc_q1 : desc_q0;
        const uint64_t b0 = desc_k + static_cast<uint64_t>((slot * kTileBytes) >> 4);
        const uint32_t d = tmem + t * 128;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk) {
            const uint64_t off =
                static_cast<uint64_t>(((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4);
            mma_ss(d, a0 + off, b0 + off, idesc_s, kk > 0 ? 1u : 0u);
          }
          tc_commit(s_full(t));
        }
      };
      auto issue_pv_half = [&](int t, int slot, int h, bool accumulate) {
        const uint64_t b0 = desc_v + static_cast<uint64_t>((slot * kTileBytes) >> 4);
        const uint32_t d = tmem + 256 + t * kD;
        const uint32_t a = tmem + t * 128 + 64;   // P: 16-bit pairs in S's columns 64-127
        if (leader) {
#pragma unroll
          for (int k4 = 0; k4 < kBN / 32; ++k4) {
            const int kk = h * (kBN / 32) + k4;
            mma_ts(d, a + kk * 8, b0 + static_cast<uint64_t>((kk * 16 * 128) >> 4), idesc_pv,
                   (accumulate || kk > 0) ? 1u : 0u);
          }
        }
      };
      bool ok = true;
      int pos = 0, segs = 0;
      int tiles[2] = {0, 0};   // S tiles of each row tile in earlier segments (phases)
      SegmentWalker walk(cta, p.w, sp);
      Segment s;
      while (ok && walk.next(p, s)) {
        const int n = s.j1 - s.j0;
        const int nts = s.two ? 2 : 1;
        ok = wait(q_full(0), segs & 1);
        if (ok) ok = wait(q_full(1), segs & 1);
        if (ok) ok = wait(kv_full(slot_of(pos)), phase_of(pos));
        if (!ok) break;
        ++segs;
        tc_fence_after();
        for (int t = 0; t < nts; ++t) issue_s(t, slot_of(pos));
        commit(kv_empty(slot_of(pos)));
        if (n == 1) commit(q_empty);
        for (int j = 0; j < n && ok; ++j) {
          const int vpos = pos + 2 * j + 1;
          const int kpos = pos + 2 * j + 2;
          const bool has_next = j + 1 < n;
          ok = wait(kv_full(slot_of(vpos)), phase_of(vpos));
          bool k_ready = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || t >= nts) continue;
            const uint32_t par = static_cast<uint32_t>((tiles[t] + j) & 1);
            ok = wait(p_half(t, 0), par);
            if (!ok) continue;
            tc_fence_after();
            issue_pv_half(t, slot_of(vpos), 0, j > 0);
            ok = wait(p_half(t, 1), par);
            if (!ok) continue;
            tc_fence_after();
            issue_pv_half(t, slot_of(vpos), 1, true);
            if (has_next) {
              if (!k_ready) {
                ok = wait(kv_full(slot_of(kpos)), phase_of(kpos));
                k_ready = true;
                if (!ok) continue;
                tc_fence_after();
              }
              issue_s(t, slot_of(kpos));
            } else {
              commit(o_full(t));
            }
          }
          if (!ok) break;
          if (j + 2 == n) commit(q_empty);       // the segment's last S MMAs are issued
          commit(kv_empty(slot_of(vpos)));
          if (has_next) commit(kv_empty(slot_of(kpos)));
        }
        pos += 2 * n;
        tiles[0] += n;
        if (s.two) tiles[1] += n;
      }
      // All issued MMAs must complete before TMEM is released (also on abort).
      commit(mma_done);
      volatile int no_abort = 0;
      mbar_wait(mma_done, 0, &no_abort, p.err, p.timeout_ns);
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax warpgroups
    const int t = warp >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + t * 128;
    const uint32_t tP = tS + 64;
    const uint32_t tO = tmem + lane_base + 256 + t * kD;
    uint8_t* stage = smem + kStageOff + warp * kStageBytes;
    int tiles = 0, outs = 0;
    bool ok = true;
    SegmentWalker walk(cta, p.w, sp);
    Segment s;
    while (ok && walk.next(p, s)) {
      if (t == 1 && !s.two) continue;
      const int n = s.j1 - s.j0;
      float m_used = -INFINITY;
      float l = 0.f;
      for (int j = 0; j < n; ++j) {
        // tcgen05.ld/st/wait are warp-collective: every branch around them is
        // made warp-uniform, also on the abort path.
        const bool got = mbar_wait(s_full(t), (tiles + j) & 1, abort_flag, p.err, p.timeout_ns);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sv[128];
        tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]), p.err);
        tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]), p.err);
        tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[64]), p.err);
        tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sv[96]), p.err);
        tmem_wait_ld(p.err);
        const int kbase = (s.j0 + j) * kBN;
        if (n_keys - kbase < kBN) {              // the prefix ends inside this tile
          const int lim = n_keys - 1 - kbase;
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (e > lim) sv[e] = __float_as_uint(-INFINITY);
        }
        // row maximum: four independent three-input-max chains
        float acc[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = __uint_as_float(sv[k]);
#pragma unroll
        for (int e = 4; e + 8 <= 128; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            acc[k] = fmax3(acc[k], __uint_as_float(sv[e + k]), __uint_as_float(sv[e + 4 + k]));
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = fmaxf(acc[k], __uint_as_float(sv[124 + k]));
        const float m_tile =
            fmaxf(fmaxf(acc[0], acc[1]), fmaxf(acc[2], acc[3])) * p.scale_log2;
        const bool move = m_tile > m_used + kTau;
        float alpha = 1.f;
        if (move) {
          alpha = ex2(m_used - m_tile);          // 0 on the first tile
          l *= alpha;
          m_used = m_tile;
        }
        if (j > 0 && __any_sync(0xffffffffu, move)) {
#pragma unroll 1
          for (int c = 0; c < kD / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(tO + 32 * c, ov, p.err);
            tmem_wait_ld(p.err);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32(tO + 32 * c, ov, p.err);
          }
        }
        const float neg_m = (m_used == -INFINITY) ? 0.f : -m_used;
        const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
        const uint64_t nm2 = f2_pack(neg_m, neg_m);
        uint64_t sum2[4] = {0, 0, 0, 0};
        // P is rounded to bf16 for the second product (each weight by at most 2^-8 of
        // itself, independently); the row sum is of the unrounded fp32 weights.
        auto exp_cols = [&](int c, uint32_t (&pk)[16]) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[32 * c + 2 * e]),
                                     __uint_as_float(sv[32 * c + 2 * e + 1])), c2, nm2), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            sum2[e & 3] = f2_add(sum2[e & 3], f2_pack(p0, p1));
            pk[e] = pack_bf16x2(p0, p1);
          }
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {            // released in halves of 64 keys
#pragma unroll
          for (int c = 2 * h; c < 2 * h + 2; ++c) {
            uint32_t pk[16];
            exp_cols(c, pk);
            tmem_st16(tP + 16 * c, pk, p.err);
          }
          tmem_wait_st(p.err);
          tc_fence_before();
          mbar_arrive(p_half(t, h));
        }
        float sa, sb;
        f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), sa, sb);
        l += sa + sb;
      }
      if (!ok) break;
      tiles += n;
      const bool fin = mbar_wait(o_full(t), outs & 1, abort_flag, p.err, p.timeout_ns);
      ++outs;
      if (!__all_sync(0xffffffffu, fin)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // The warp's 32 rows, 32 columns at a time: through its staging box (16-byte chunk
      // k of row r at k ^ (r & 7)), so that 8 lanes write 128 contiguous bytes of a row.
      const float inv_l = l == 0.f ? 0.f : 1.f / l;   // 0: every score was -inf (then LSE is)
      const size_t row0 = static_cast<size_t>(s.slot) * 256 + t * kBM + (warp & 3) * 32;
      const int rows = min(32, p.B * p.G - (s.pair * 256 + t * kBM + (warp & 3) * 32));
#pragma unroll 1
      for (int c = 0; c < kD / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(tO + 32 * c, ov, p.err);
        tmem_wait_ld(p.err);
        __syncwarp();                            // the box's previous columns are out
#pragma unroll
        for (int v = 0; v < 8; ++v)
          *reinterpret_cast<float4*>(stage + lane * 128 + ((v ^ (lane & 7)) << 4)) = make_float4(
              __uint_as_float(ov[4 * v]) * inv_l, __uint_as_float(ov[4 * v + 1]) * inv_l,
              __uint_as_float(ov[4 * v + 2]) * inv_l, __uint_as_float(ov[4 * v + 3]) * inv_l);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = i * 4 + (lane >> 3), v = lane & 7;
          if (rr < rows)
            *reinterpret_cast<float4*>(p.ws_o + (row0 + rr) * kD + 32 * c + 4 * v) =
                *reinterpret_cast<const float4*>(stage + rr * 128 + ((v ^ (rr & 7)) << 4));
        }
      }
      if (lane < rows) p.ws_lse[row0 + lane] = (m_used + __log2f(l)) * 0.69314718055994530942f;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

int launch_prefix(const void* q, const void* kcache, const void* vcache, const PrefixWork& w,
                  const int32_t* prefix_table, float* ws_o, float* ws_lse, int B, int Hq, int Hkv,
                  int num_pages, float scale, cudaStream_t stream, int device) {
  const int G = Hq / Hkv;
  int rc = raise_smem_limit(reinterpret_cast<const void*>(fa_prefix_kernel), kSmemBytes, device,
                            kSmemPrefix);
  if (rc != FA_OK) return rc;
  CUtensorMap tq, tk, tv;
  {
    const uint64_t dims[3] = {kD, static_cast<uint64_t>(Hq), static_cast<uint64_t>(B)};
    const uint64_t strides[2] = {kD * 2, static_cast<uint64_t>(Hq) * kD * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(kBM / G)};
    if ((rc = encode_tensor_map_16bit(&tq, q, true, 3, dims, strides, box)) != FA_OK) return rc;
  }
  {
    const uint64_t dims[3] = {kD, static_cast<uint64_t>(Hkv),
                              static_cast<uint64_t>(num_pages) * kPageTok};
    const uint64_t strides[2] = {kD * 2, static_cast<uint64_t>(Hkv) * kD * 2};
    const uint32_t box[3] = {64, 1, kPageTok};
    rc = encode_tensor_map_16bit(&tk, kcache, true, 3, dims, strides, box);
    if (rc == FA_OK) rc = encode_tensor_map_16bit(&tv, vcache, true, 3, dims, strides, box);
    if (rc != FA_OK) return rc;
  }
  PrefixParams prm;
  prm.w = w;
  prm.table = prefix_table;
  prm.ws_o = ws_o;
  prm.ws_lse = ws_lse;
  prm.B = B;
  prm.G = G;
  prm.Hkv = Hkv;
  prm.num_pages = num_pages;
  prm.scale_log2 = scale * 1.4426950408889634f;
  prm.err = device_error_word(device);
  prm.timeout_ns = kWaitLimitNs;
  if (!prm.err) return set_error(FA_ERR_CUDA, "device error word unavailable");
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(w.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fa_prefix_kernel, tq, tk, tv, prm);
  if (e != cudaSuccess)
    return set_error(FA_ERR_CUDA, "shared-prefix launch: %s", cudaGetErrorString(e));
  return FA_OK;
}

}  // namespace fa
