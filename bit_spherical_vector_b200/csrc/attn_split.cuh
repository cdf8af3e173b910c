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

// A range boundary moved to the nearer end of the unit that it would cut, if the
// unit has at most `most` tiles (a cut costs a join).  Places at the line's end stay.
SVQ_HD long long attn_snap(const AttnSeqs& s, int n, int heads, const FastDiv& by_heads, long long total, int most,
                           long long g) {
  if (g <= 0 || g >= total) return g;
  AttnCursor c;
  c.set(s, n, heads, by_heads, g);
  if (c.nt > most) return g;
  return 2 * c.t <= c.nt ? g - c.t : g - c.t + c.nt;
}

// Longest units that boundaries do not cut: what a boundary moves is read by one
// SM or warp more and another less, so only units of a few tiles, and for warps of
// at most twice their share, are worth it.
constexpr int kSnap = 8;
SVQ_HD int attn_warp_snap(long long tiles, int warps) {
  const long long share = 2 * tiles / warps;
  return share < kSnap ? (int)share : kSnap;
}

// The cut of the line: `by_unit` gives each unit to a CTA (short requests, as many
// CTAs as units), else CTAs and their warps get even ranges but for the short units
// at their ends, if there are any (`shorts`).
struct AttnCut {
  AttnSeqs s;
  AttnLine line;
  FastDiv by_heads;
  long long total;
  int n, heads;
  bool by_unit, shorts;
  SVQ_HD AttnCut(const AttnSeqs& seqs, int n_seqs, int n_heads, const FastDiv& div, bool unit_each, bool any_short,
                 int grid, int warps)
      : s(seqs),
        line((long long)seqs.pre[n_seqs] * n_heads, attn_ctas((long long)seqs.pre[n_seqs] * n_heads, grid, warps)),
        by_heads(div),
        total((long long)seqs.pre[n_seqs] * n_heads),
        n(n_seqs),
        heads(n_heads),
        by_unit(unit_each),
        shorts(any_short) {}
  SVQ_HD bool moves() const { return shorts && !by_unit; }         // edges are not simply the even ranges
  SVQ_HD int ctas() const { return by_unit ? n * heads : line.n; }
  // First place of CTA c's range, 0 <= c <= ctas() (a range may be empty).
  SVQ_HD long long edge(int c) const {
    if (!by_unit) {
      const long long g = line.start(c);
      return moves() ? attn_snap(s, n, heads, by_heads, total, kSnap, g) : g;
    }
    const int b = by_heads.div(c);
    return b == n ? total : (long long)s.pre[b] * heads + (long long)(c - b * heads) * s.tiles(b);
  }
  // First place of warp w's range in the CTA's [s0, s1), 0 <= w <= warps.
  SVQ_HD long long warp_edge(long long s0, long long s1, int w, int warps) const {
    if (w == 0) return s0;
    if (w == warps) return s1;
    const AttnLine part(s1 - s0, warps);
    long long g = s0 + part.start(w);
    if (!moves()) return g;
    g = attn_snap(s, n, heads, by_heads, total, attn_warp_snap(s1 - s0, warps), g);
    return g < s0 ? s0 : g > s1 ? s1 : g;
  }
  // CTAs that share the unit of tiles [u0, u1) if any boundary cuts it.  Boundaries
  // inside such a unit have not been moved and others not into it, so they are those
  // that the even ranges give.
  SVQ_HD int first_cta(long long u0) const { return line.range_of(u0); }
  SVQ_HD int last_cta(long long u1) const { return line.range_of(u1 - 1); }
};

}  // namespace svq
