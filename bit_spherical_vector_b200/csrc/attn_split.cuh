// attn_split.cuh -- how decode attention cuts its work (shared by the kernel and
// the host test of the split).  The line of all 16-key tiles, in (request, head,
// tile) order, is cut into equal ranges: one per CTA, and each of those one per
// warp.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define SVQ_HD __host__ __device__ __forceinline__
#else
#define SVQ_HD inline
#endif

namespace svq {

constexpr int kAttnTile = 16;            // keys per tile

// First place of range i of n over places [0, total).
SVQ_HD long long range_start(long long total, int i, int n) { return total * i / n; }
// The range that place g lies in: the last i with range_start(i) <= g.
SVQ_HD int range_of(long long g, long long total, int n) { return (int)(((g + 1) * n - 1) / total); }

// CTAs that take part: each of their warps gets a tile at least.
SVQ_HD int attn_ctas(long long total, int grid, int warps) {
  const long long c = (total + warps - 1) / warps;
  return c < grid ? (int)c : grid;
}

// The requests of a call as every CTA keeps them: tiles before request b, and
// its row with the number of keys missing in its last tile.
struct AttnSeqs {
  const int* pre;                        // [n + 1]
  const uint32_t* meta;                  // [n]: row << 4 | missing keys
  SVQ_HD int tiles(int b) const { return pre[b + 1] - pre[b]; }
  SVQ_HD int row(int b) const { return (int)(meta[b] >> 4); }
  SVQ_HD int len(int b) const { return tiles(b) * kAttnTile - (int)(meta[b] & 15u); }
};

// A place on the line: tile t of nt of head (and row tile) h of request b.
struct AttnCursor {
  int b, h, t, nt;
  SVQ_HD void set(const AttnSeqs& s, int n, int heads, long long g) {
    const int gq = (int)(g / heads);
    int lo = 0, hi = n;
    while (hi - lo > 1) {                // last b with pre[b] <= gq: a request with tiles
      const int mid = (lo + hi) >> 1;
      if (s.pre[mid] <= gq) lo = mid; else hi = mid;
    }
    b = lo;
    nt = s.tiles(b);
    const long long r = g - (long long)s.pre[b] * heads;
    h = (int)(r / nt);
    t = (int)(r - (long long)h * nt);
  }
  // The next place; called only where there is one.
  SVQ_HD void next(const AttnSeqs& s, int n, int heads) {
    if (++t < nt) return;
    t = 0;
    if (++h < heads) return;
    h = 0;
    do ++b; while (b < n && s.tiles(b) == 0);
    nt = b < n ? s.tiles(b) : 1;
  }
  SVQ_HD long long unit(int heads) const { return (long long)b * heads + h; }
};

}  // namespace svq
