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

// Quotient of nonnegative numbers: a 64-bit division is ten times a 32-bit one
// and only lines beyond 2^32 tiles need it.
SVQ_HD long long div_places(long long a, long long b) {
  if (((unsigned long long)a | (unsigned long long)b) >> 32 == 0) return (long long)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// Quotient of a number below 2^31 by a divisor that the host knows: with m =
// floor(2^(31 + s) / d) + 1 and 2^(s - 1) < d <= 2^s the product's high part is
// exact (T. Granlund and P. Montgomery, Division by Invariant Integers using
// Multiplication, 1994).
struct FastDiv {
  uint32_t d, m;
  int s;
  FastDiv() = default;
  explicit FastDiv(int divisor) : d((uint32_t)divisor), s(0) {
    while ((1ull << s) < d) ++s;
    m = (uint32_t)((1ull << (31 + s)) / d + 1);
  }
  SVQ_HD int div(int n) const { return (int)(((unsigned long long)(uint32_t)n * m) >> (31 + s)); }
};

// Places [0, total) in n ranges of equal size, the first ranges one longer.
struct AttnLine {
  long long size, longer;                // size of the shorter ranges, how many are longer
  int n;
  SVQ_HD AttnLine(long long total, int ranges)
      : size(div_places(total, ranges)), longer(total - size * ranges), n(ranges) {}
  SVQ_HD long long start(int i) const { return size * i + (i < longer ? i : longer); }
  SVQ_HD int range_of(long long g) const {             // the range that place g lies in
    const long long split = longer * (size + 1);
    return (int)(g < split ? div_places(g, size + 1) : longer + div_places(g - split, size));
  }
};

// CTAs that take part in an even split: each of their warps gets a tile at least.
SVQ_HD int attn_ctas(long long total, int grid, int warps) {
  const long long c = (total + warps - 1) / warps;
  return c < grid ? (c > 0 ? (int)c : 1) : grid;
}

// Parts of one unit are joined `fan` at a time, level by level; on a level the
// parts left stand `stride` (a power of fan) apart.  First part of part x's group
// and the group's size, for a unit of n parts.
SVQ_HD int attn_group(int n, int fan, int stride, int x, int* members) {
  const int span = stride * fan, first = x / span * span;
  const int left = (n - 1 - first) / stride + 1;
  *members = left < fan ? left : fan;
  return first;
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
  SVQ_HD void set(const AttnSeqs& s, int n, int heads, const FastDiv& by_heads, long long g) {
    const int gq = g >> 31 ? (int)(g / heads) : by_heads.div((int)g);
    int lo = 0, hi = n;
    while (hi - lo > 1) {                // last b with pre[b] <= gq: a request with tiles
      const int mid = (lo + hi) >> 1;
      if (s.pre[mid] <= gq) lo = mid; else hi = mid;
    }
    b = lo;
    nt = s.tiles(b);
    const long long r = g - (long long)s.pre[b] * heads;
    h = (int)div_places(r, nt);
    t = (int)(r - (long long)h * nt);
  }
  SVQ_HD int unit(int heads) const { return b * heads + h; }   // at most 2^22
};

// Tiles [s0, s1) of a CTA: one unit (short requests, as many CTAs as units), or
// its range of the even split.  False: none.
SVQ_HD bool attn_share(const AttnSeqs& s, int n, int heads, const FastDiv& by_heads, bool by_unit, const AttnLine& line,
                       int cta, long long* s0, long long* s1) {
  if (by_unit) {
    if (cta >= n * heads) return false;
    const int b = by_heads.div(cta), nt = s.tiles(b);
    *s0 = (long long)s.pre[b] * heads + (long long)(cta - b * heads) * nt;
    *s1 = *s0 + nt;
    return nt > 0;
  }
  if (cta >= line.n) return false;
  *s0 = line.start(cta);
  *s1 = line.start(cta + 1);
  return *s1 > *s0;
}

}  // namespace svq
