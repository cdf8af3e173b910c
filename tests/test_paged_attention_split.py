"""Host logic of decode attention's split (no GPU): the kernel's own range and cursor functions, compiled into
a host program and walked the way the kernel walks them.

For seeded batches (one to 600 requests, lengths 0 to thousands, 1 to 64 heads and row tiles, 4 and 8 warps,
148 CTAs and fewer) every tile of every unit must be visited exactly once, in order; every unit must be
written exactly once: by the one warp that has all of it, by the one CTA that has all of it, or by the last
of the CTAs from that of its first tile to that of its last, which are exactly the CTAs that leave a part of
it; no CTA uses a workspace slot twice, no warp a part slot twice, and a counter (that of the unit's first CTA)
belongs to one unit and gets as many arrivals as the unit has CTAs.  Places beyond 2^31 are checked on the range
functions alone."""
import os
import shutil
import subprocess

import pytest

from bit_spherical_vector_b200 import build as svq_build

HARNESS = r"""
#include <algorithm>
#include <cstdio>
#include <map>
#include <random>
#include <set>
#include <vector>
#include "attn_split.cuh"
using namespace svq;
static long long bad = 0, cases = 0, split_units = 0, units = 0;
#define CHECK(c, ...) do { if (!(c)) { if (++bad < 20) { printf(__VA_ARGS__); printf("\n"); } } } while (0)

static void walk(const std::vector<int>& lens, int heads, int grid, int W) {
  const int n = (int)lens.size();
  std::vector<int> pre(n + 1, 0);
  std::vector<uint32_t> meta(n);
  for (int b = 0; b < n; ++b) {
    const int nt = (lens[b] + kAttnTile - 1) / kAttnTile;
    pre[b + 1] = pre[b] + nt;
    meta[b] = ((uint32_t)b << 4) | (uint32_t)(nt * kAttnTile - lens[b]);
  }
  const AttnSeqs s{pre.data(), meta.data()};
  for (int b = 0; b < n; ++b) CHECK(s.len(b) == lens[b] && s.row(b) == b, "meta %d", b);
  const long long total = (long long)pre[n] * heads;
  const FastDiv by_heads(heads);
  int longest = 0;
  for (int b = 0; b < n; ++b) longest = std::max(longest, s.tiles(b));
  const bool by_unit = longest <= 4 * W && (long long)n * heads <= grid;
  bool shorts = false;
  for (int b = 0; b < n; ++b) shorts |= s.tiles(b) > 0 && s.tiles(b) <= kSnap;
  const AttnCut cut(s, n, heads, by_heads, by_unit, shorts, grid, W);
  ++cases;
  units += by_unit;
  std::map<long long, int> written;                       // unit -> times written
  std::map<int, std::pair<long long, int>> counter;       // counter -> unit, arrivals
  std::map<long long, std::set<int>> far;                 // unit -> CTAs that left a part
  long long expect_b = 0, expect_h = 0, expect_t = -1;    // the line in order
  int eb = -1;
  CHECK(cut.ctas() <= grid && cut.edge(0) == 0 && cut.edge(cut.ctas()) == total, "ends of the line");
  for (int c = 0; c < cut.ctas(); ++c) {
    const long long s0 = cut.edge(c), s1 = cut.edge(c + 1);
    CHECK(s1 >= s0, "CTA ranges overlap");
    if (s1 <= s0) continue;
    CHECK(cut.warp_edge(s0, s1, 0, W) == s0 && cut.warp_edge(s0, s1, W, W) == s1, "ends of a CTA");
    std::vector<long long> part(2 * W, -1);
    for (int w = 0; w < W; ++w) {
      const long long w0 = cut.warp_edge(s0, s1, w, W), w1 = cut.warp_edge(s0, s1, w + 1, W);
      CHECK(s0 <= w0 && w0 <= w1 && w1 <= s1, "warp ranges overlap");
      if (w0 >= w1) continue;
      AttnCursor cur;
      bool fresh = true, from_start = true;
      for (long long g = w0; g < w1; ++g) {
        cur.set(s, n, heads, by_heads, g);
        if (fresh) from_start = cur.t == 0;
        fresh = false;
        // the place is the next one of the line
        if (expect_t >= 0) {
          if (++expect_t == s.tiles(eb)) {
            expect_t = 0;
            if (++expect_h == heads) {
              expect_h = 0;
              do ++eb; while (eb < n && s.tiles(eb) == 0);
            }
          }
        } else {
          expect_t = 0;
          eb = 0;
          while (s.tiles(eb) == 0) ++eb;
        }
        CHECK(cur.b == eb && cur.h == expect_h && cur.t == expect_t && cur.nt == s.tiles(eb), "place %lld", g);
        CHECK(cur.b < n && cur.t * kAttnTile < lens[cur.b], "beyond a request");
        const bool ue = cur.t == cur.nt - 1, re = g == w1 - 1;
        if (ue || re) {
          if (ue && from_start) written[cur.unit(heads)]++;
          else {
            const int slot = re ? 1 : 0;
            CHECK(part[2 * w + slot] < 0, "part slot twice");
            part[2 * w + slot] = cur.unit(heads);
          }
          fresh = true;
        }
      }
    }
    bool used[2] = {false, false};
    for (int a = 0; a < 2 * W;) {
      if (part[a] < 0) { ++a; continue; }
      const long long unit = part[a];
      int e = a + 1;
      while (e < 2 * W && (part[e] < 0 || part[e] == unit)) ++e;
      // the kernel counts a unit's parts as slots 1 of consecutive warps and perhaps a last slot 0
      int last = e - 1, at = a;
      while (part[last] < 0) --last;
      for (int x = 0; x < last / 2 - a / 2 + 1; ++x) {
        const int y = std::min(2 * (a / 2 + x) + 1, last);
        while (at < e && part[at] < 0) ++at;
        CHECK(y == at, "part %d of unit %lld", x, unit);
        ++at;
      }
      while (at < e && part[at] < 0) ++at;
      CHECK(at == e, "parts of unit %lld left over", unit);
      const int b = (int)(unit / heads), h = (int)(unit % heads);
      const long long u0 = (long long)pre[b] * heads + (long long)h * s.tiles(b), u1 = u0 + s.tiles(b);
      if (u0 >= s0 && u1 <= s1) written[unit]++;
      else {
        const int slot = u0 >= s0;
        CHECK(!used[slot], "workspace slot twice");
        used[slot] = true;
        const int c0 = cut.first_cta(u0), c1 = cut.last_cta(u1);
        CHECK(!by_unit && c0 <= c && c <= c1 && c1 > c0, "CTAs of a unit");
        CHECK((slot == 1) == (c == c0), "slot of the first CTA");
        CHECK(far[unit].insert(c).second, "two parts of a unit in one CTA");
        auto& k = counter[c0];
        if (k.second == 0) k.first = unit;
        CHECK(k.first == unit, "counter shared");
        if (++k.second == c1 - c0 + 1) written[unit]++;      // joined below, level by level
      }
      a = e;
    }
  }
  split_units += (long long)far.size();
  // The joins: CTAs arrive in random order, the last of a group adds its parts and goes on for them.
  static std::mt19937 shuffle(11);
  for (int fan : {8, 16, 32}) {
    std::map<std::pair<int, int>, std::pair<long long, int>> at;       // (level, counter) -> unit, arrivals
    for (auto& f : far) {
      const int c0 = *f.second.begin(), n = (int)f.second.size();
      CHECK(*f.second.rbegin() == c0 + n - 1, "CTAs of a unit are neighbours");
      std::vector<int> order(f.second.begin(), f.second.end());
      std::shuffle(order.begin(), order.end(), shuffle);
      std::vector<std::set<int>> holds(n);                  // parts summed in each place
      for (int i = 0; i < n; ++i) holds[i] = {i};
      int done = 0;
      for (int c : order) {
        for (int stride = 1, level = 0;; stride *= fan, ++level) {
          CHECK(level < 3, "levels");
          int m;
          const int first = attn_group(n, fan, stride, c - c0, &m);
          if (m > 1) {
            auto& k = at[{level, c0 + first}];
            if (k.second == 0) k.first = f.first;
            CHECK(k.first == f.first, "counter shared on a level");
            if (++k.second < m) break;
          }
          for (int x = 1; x < m; ++x) {
            CHECK(first + x * stride < n, "beyond the unit");
            for (int v : holds[first + x * stride]) CHECK(holds[first].insert(v).second, "added twice");
            holds[first + x * stride].clear();
          }
          if (stride * fan > n - 1) {
            ++done;
            CHECK(first == 0 && (int)holds[0].size() == n, "all parts in the sum");
            break;
          }
        }
      }
      CHECK(done == 1, "joined %d times", done);
    }
  }
  for (auto& k : counter)
    CHECK((int)far[k.second.first].size() == k.second.second, "arrivals");
  for (int b = 0; b < n; ++b)
    for (int h = 0; h < heads; ++h) {
      const auto it = written.find((long long)b * heads + h);
      CHECK((it == written.end() ? 0 : it->second) == (s.tiles(b) ? 1 : 0), "unit %d %d written", b, h);
    }
}

int main() {
  std::mt19937 r(7);
  auto u = [&](int a, int b) { return a + (int)(r() % (unsigned)(b - a + 1)); };
  for (int W : {4, 8, 10})
    for (int len : {0, 1, 15, 16, 17, 127, 128, 512, 4096, 40000})
      for (int heads : {1, 8})
        walk({len}, heads, 148, W);
  for (int i = 0; i < 400; ++i) {
    const int n = u(1, i % 10 ? 40 : 600), heads = u(1, i % 7 ? 8 : 64), most = 1 << u(2, 12);
    std::vector<int> lens(n);
    for (auto& l : lens) l = u(0, 4) ? u(0, most) : 0;
    walk(lens, heads, i % 3 ? 148 : u(1, 160), i % 4 == 0 ? 4 : i % 4 == 1 ? 10 : 8);
  }
  // ranges far beyond 32 bits
  for (int i = 0; i < 2000; ++i) {
    const long long total = ((long long)r() << 9) + r() % 1000 + 1;
    const int n = u(1, 148);
    if (total < n) continue;
    const int c = u(0, n - 1);
    const AttnLine line(total, n);
    const long long a = line.start(c), b = line.start(c + 1);
    CHECK(a < b && line.range_of(a) == c && line.range_of(b - 1) == c, "range of %lld", total);
    CHECK(line.start(0) == 0 && line.start(n) == total, "ends of %lld", total);
  }
  // quotients by known divisors, at the ends of their range and around multiples
  for (int i = 0; i < 200000; ++i) {
    const int d = i < 5000 ? i + 1 : 1 + (int)(r() >> (1 + r() % 31)) , k = (int)(r() >> 1) / d;
    const FastDiv f(d);
    for (long long x : {(long long)k * d - 1, (long long)k * d, (long long)k * d + d - 1, (long long)(r() >> 1), 0x7FFFFFFFll, 0ll})
      if (x >= 0 && x <= 0x7FFFFFFF) CHECK(f.div((int)x) == x / d, "%lld / %d", x, d);
  }
  printf("cases=%lld split=%lld units=%lld bad=%lld\n", cases, split_units, units, bad);
  return bad ? 1 : 0;
}
"""


def test_every_tile_once_and_every_unit_written_once(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "split.cpp", tmp_path / "split"
    src.write_text(HARNESS)
    hdr = tmp_path / "attn_split.cuh"
    hdr.write_text(open(os.path.join(svq_build.CSRC, "attn_split.cuh")).read())
    r = subprocess.run([cxx, "-O1", "-std=c++17", "-I", str(tmp_path), str(src), "-o", str(exe)], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    counts = dict(kv.split("=") for kv in r.stdout.split())
    assert int(counts["cases"]) > 400 and int(counts["split"]) > 1000 and int(counts["units"]) > 20
