// How the shared-prefix attention is split: used by the kernel that computes the
// segments and by the merge that reads them.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "ptx_sm100.cuh"

namespace fa {

// floor(c * H / C) for 0 <= c <= C
__device__ __forceinline__ int share_edge(int c, int H, int C) {
  const long long prod = static_cast<long long>(c) * H;
  if (prod <= 0x7fffffffLL)
    return static_cast<int>(static_cast<uint32_t>(prod) / static_cast<uint32_t>(C));
  return static_cast<int>(prod / C);
}
// The largest c in [0, C) with share_edge(c) <= x, for 0 <= x < H: the share that holds
// entry x.
__device__ __forceinline__ int cta_of(long long x, long long H, long long C) {
  if ((x + 1) * C <= 0x7fffffffLL)             // the usual case: 32-bit division
    return static_cast<int>((static_cast<uint32_t>(x + 1) * static_cast<uint32_t>(C) - 1u) /
                            static_cast<uint32_t>(H));
  return static_cast<int>(((x + 1) * C - 1) / H);
}

// Number of shared pages, read on the device; a count outside [0, max_pages] is flagged
// and stands for no sharing.
__device__ __forceinline__ int shared_pages(const PrefixWork& w) {
  const int n = __ldg(w.pages);
  if (n < 0 || n > w.max_pages) {
    atomicOr(w.err, kErrBadIndex);
    return 0;
  }
  return n;
}

// Key tiles of so many shared pages (whose tokens may be close to 2^31).
__host__ __device__ constexpr int prefix_tiles(int pages) {
  constexpr int kTilePages = kPrefixTile / 16;
  return pages / kTilePages + (pages % kTilePages != 0);
}
static_assert(prefix_tiles(0x7fffffff / 16) == 1 << 24, "the longest prefix");

// A unit is a key tile of a KV head for a team of CTAs, each of which takes a pair of row
// tiles: they read the same keys at about the same time, so that HBM is read once and not
// once a pair (256 sequences of 32 + 8 heads, 4 pairs a KV head, 32768 shared keys: 178.0
// and 176.4 us a call, 204.3 and 197.8 in a long run at the power limit).
//
// The prefix kernel and the stream kernel are both bound by what an SM does (tiles, pages),
// so the SMs are divided between them in proportion to their work: the teams' CTAs take
// prefix tiles, and the stream kernel's blocks, as many as there are SMs left, which start at
// once on the others, share the sequences' own pages.
struct PrefixSplit {
  int pages;       // shared pages that are attended at once
  int nt;          // key tiles of the prefix
  int units;       // items * nt
  int teams;       // teams that take a share of the units (0: no prefix)
  int own_ctas;    // CTAs that take a share of the streamed pages (1 to C)
};
// Read after the scan of the lengths has finished.
__device__ __forceinline__ PrefixSplit prefix_split(const PrefixWork& w, int C) {
  PrefixSplit s;
  s.pages = w.together ? shared_pages(w) : 0;
  s.nt = prefix_tiles(s.pages);
  s.units = w.items * s.nt;
  const long long prefix = static_cast<long long>(s.units) * w.team * w.tile_ns;
  const int own_pages = __ldcg(w.own_total);
  const long long own = static_cast<long long>(own_pages) * w.page_ns;
  s.teams = 0;
  if (s.units > 0) {
    const int ctas = static_cast<int>((prefix * C + prefix + own - 1) / (prefix + own));
    s.teams = max(1, min((ctas + w.team / 2) / w.team, min(C / w.team, s.units)));
  }
  const int ctas = s.teams * w.team;
  s.own_ctas = min(ctas < C ? C - ctas : C, max(1, own_pages / kOwnMinPages));
  return s;
}

}  // namespace fa
