// paged_attention.cu -- attention of one new token per request over a paged
// key/value cache.
//
//   s_j = scale * q . k_j,  p_j = e^(s_j - max s),  o = sum_j p_j v_j / sum_j p_j,   j < len
//
// Every key and value is read once for all query heads that share it, up to 16
// (a larger group reads it again for each row tile of 16), so the cache's bytes bound
// the call; everything here serves to keep loads in flight on every SM whatever the
// lengths are.
//
// Split.  A unit is one (request, key head, row tile of at most 8 or 16 query
// heads); its keys are cut into tiles of 16.  All tiles of the call, in (request,
// head, tile) order, form one line that is cut into equal ranges, one per CTA and
// again one per warp, with no regard for where units begin: long and short
// requests balance by construction and the host need not know the lengths.  Each
// warp streams its own range through its own ring of shared-memory stages
// (16-byte cp.async, no block barrier in the loop), across unit boundaries.
//
// Products.  The scores are formed as K q^T and the output as V^T p^T: the 16
// keys of a tile (then 16 entries of a head) are the M side of mma.m16n8k16 and
// the queries the N side, so a group of up to 8 heads fills the instruction
// (row tiles of 8: NQ = 1) and K and V come from shared memory by ldmatrix as
// they lie.  At the rate that HBM delivers the cache the tensor work is a few
// per cent of this path's rate, so the 128-row tcgen05 form has nothing to win.
// P is rounded to the cache's type twice, a high part and the remainder, and
// both are multiplied: with one rounding to bf16 (2^-9 of each weight) the
// result would lose more than its own output rounding.  fp16 also lacks the
// range: weights below 2^-25 of the largest would vanish, and over 10^5 keys they
// can be a per cent of the sum; so P is formed 2^15 times as large (at most
// 32768), which the final division removes.
//
// Join.  A unit cut by a range boundary leaves a part (running maximum, sum and
// unnormalised output, fp32): the warps' parts are joined inside the CTA after
// the loop, the CTAs' parts through the workspace by the CTA that arrives last
// (a counter per CTA that wraps back to zero), in CTA order, so results do not
// depend on timing.  Nothing waits on another CTA.
//
// B200, in a CUDA graph, heads of 128, 4 query heads to a key head, 8 key heads: one
// request of 131072 keys 87 us = 6.2 TB/s (7.1 in the loop; the front takes 2.6 us, the
// joins 5), 128 requests of up to 4096 keys 184 us = 6.1 TB/s, both bound by HBM (copy
// rate 6.6); one of 512 keys 8 us, a chain of dependent loads and one join.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_params.h"
#include "attn_split.cuh"
#include "sm100.cuh"
#include "svq.h"
#include "svq_internal.h"

namespace svq {
namespace {

constexpr int kTile = kAttnTile;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr uint32_t kNoRow = ~0u;         // a request without a row in this step

template <int D>
struct Shape {
  // Bytes on their way are what HBM wants (two stages of each warp at least, 128 KB
  // an SM), warps what hides the chain of a tile, which is as long for 4 KB as for 8:
  // heads of 64 take ten warps of four stages (67 requests of up to 4510 keys, 48
  // heads on 4: 41.2 us; eight of five: 45.0 us; twelve of three, 96 KB: 48 us).
  static constexpr int kWarps = D == 256 ? 4 : D == 128 ? 8 : 10;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = D == 64 ? 4 : 3;
  static constexpr int kRow = D * 2;                       // bytes of one key
  static constexpr int kStage = kTile * kRow * 2;          // K tile, then V tile
  static constexpr int kRing = kWarps * kStages * kStage;
  // A unit of up to 4 tiles per warp is not worth a join: when all are, and there
  // are CTAs enough, each gets one (three more tiles take a warp as long as the
  // join of CTAs, about 2 us: 1 request of 512 keys, 8 key heads of 128, 7.7 us
  // against 8.3 us split over four CTAs each).
  static constexpr int kUnitTiles = 4 * kWarps;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {      // a in the low half
  if (BF16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (BF16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// One instruction that makes a pair of floats NaN if one of four numbers is (also, for
// nothing, where their products run over).
__device__ __forceinline__ void probe_nan(unsigned long long& probe, const float (&v)[4]) {
  unsigned long long a, b;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(v[0]), "f"(v[1]));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(v[2]), "f"(v[3]));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(probe) : "l"(a), "l"(b));
}
__device__ __forceinline__ bool is_nan(unsigned long long probe) {
  const float s = __uint_as_float((uint32_t)probe) + __uint_as_float((uint32_t)(probe >> 32));
  return s != s;
}
// Weight of a part with maximum m in a join whose maximum is M (both in units of
// log2): a part that saw no key has m = -inf and weight 0.  Any other weighs the least
// positive number at least: an infinite sum stays infinite, and to finite ones it adds
// 2^-149 of the part's at most.
__device__ __forceinline__ float part_weight(float m, float M) {
  return m == kNegInf ? 0.f : fmaxf(ex2(m - M), 1.401298464e-45f);
}

// Where a unit's result goes: row of the output, first query head << 8 | heads,
// and the CTAs that share the unit.
struct UnitOut {
  int row, heads, c0, c1;
};

__device__ __forceinline__ void weigh(float4& acc, float f, const float4& v) {
  acc.x = fmaf(v.x, f, acc.x);
  acc.y = fmaf(v.y, f, acc.y);
  acc.z = fmaf(v.z, f, acc.z);
  acc.w = fmaf(v.w, f, acc.w);
}

// An infinite value that counts.  A weight is multiplied in two terms, of which one may be
// 0 or negative, so the products make NaN of a sum that is infinite.  A warp that has met
// NaN among its sums goes through its range [w0, w1) of the line once more: weights of
// finite scores are positive, so infinite values of one sign give that infinity; both
// signs, a NaN or an infinity whose score is -inf (0 times infinity) give NaN, and so does
// a score that is NaN or +inf (then all of a row is NaN).  Sums are found where the loop
// has left them: parts in `part0` or `part1` (slots 0 and 1), Pitch apart, whole units in
// the output.  The values of a unit with NaN are read once more for all its rows, a lane
// D / 32 entries of a key (128 requests of up to 4096 keys, an infinity in each: 0.8 ms).
// Calls without infinities and NaN never come here; what they pay is the look at the sums
// where a warp leaves a unit, D / 16 instructions for each 8 heads: 0.1 to 0.2 us of short
// calls (1 request of 3 keys: 4.1 -> 4.2 us), nothing of long ones but with thousands of
// short units of wide heads (245 requests of 186 keys, 96 heads of 256 on 8: 134 -> 138 us).
template <int D, int R, int Pitch, bool BF16>
__device__ __noinline__ void mend_sums(const PagedAttnParams& p, const int* pre, float* part0, float* part1, long long w0,
                                       long long w1) {
  constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;      // infinity: larger magnitudes are NaN
  constexpr int E = D / 32;                                // entries of a lane
  constexpr uint32_t kAll = (1u << E) - 1u;
  const AttnSeqs seqs{pre, reinterpret_cast<const uint32_t*>(pre + p.n_seqs + 1)};
  const uint32_t out_inf = p.out_bf16 ? 0x7F80u : 0x7C00u;
  const int lane = threadIdx.x & 31, heads = p.kv.n_heads * p.row_tiles;
  __syncwarp();                                            // the sums are written
  for (long long g = w0; g < w1;) {
    AttnCursor c;
    c.set(seqs, p.n_seqs, heads, p.by_heads, g);
    const long long end = min(w1, g + c.nt - c.t);
    const bool whole = c.t == 0 && end == g + c.nt;
    float* part = (end == w1 ? part1 : part0) + lane * E;
    // (unsigned: a loop's last step passes a length next to 2^31)
    const unsigned j0 = c.t * kTile, j1 = min((unsigned)seqs.len(c.b), (c.t + (unsigned)(end - g)) * kTile);
    g = end;
    const int kv_head = p.by_row_tiles.div(c.h), rt = c.h - kv_head * p.row_tiles, count = min(R, p.group - rt * R);
    const int64_t at_row = ((int64_t)seqs.row(c.b) * p.n_q + kv_head * p.group + rt * R) * D;
    const uint16_t* q = p.q + at_row;
    uint16_t* out = p.out + at_row + lane * E;
    auto nans = [&](int r) {                               // the lane's entries of row r that are NaN
      uint32_t m = 0;
      for (int e = 0; e < E; ++e) {
        const bool nan = whole ? (__ldcg(out + r * D + e) & 0x7FFFu) > out_inf : part[r * Pitch + e] != part[r * Pitch + e];
        m |= (uint32_t)nan << e;
      }
      return m;
    };
    auto place_of = [&](unsigned j) -> int64_t {           // of a key's first entry, -1: none that counts
      if (j >= j1) return -1;
      const int jp = p.by_page.div((int)j), page = p.table[(int64_t)c.b * p.width + jp];
      if ((unsigned)page >= (unsigned)p.kv.n_pages) return -1;
      return (int64_t)page * p.kv.page_stride + (int64_t)((int)j - jp * p.kv.page_size) * p.kv.token_stride +
             (int64_t)kv_head * p.kv.head_stride;
    };
    bool any = false;
    for (int r = 0; r < count; ++r) any |= nans(r) != 0;
    if (!__any_sync(0xFFFFFFFFu, any)) continue;

    uint32_t up = 0, down = 0, nan = 0, zero[R];           // bit e: what the values of the lane's entry hold
#pragma unroll
    for (int r = 0; r < R; ++r) zero[r] = 0;               // an infinity without weight in row r
    for (unsigned j = j0; j < j1 && !__all_sync(0xFFFFFFFFu, nan == kAll); j += 32) {
      const int64_t mine = place_of(j + lane);
      constexpr int kBatch = 8;
#pragma unroll 1
      for (int x0 = 0; x0 < 32; x0 += kBatch) {
        uint32_t w[kBatch][E / 2];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int64_t at = __shfl_sync(0xFFFFFFFFu, mine, x0 + x);
          const uint32_t* v = reinterpret_cast<const uint32_t*>(p.kv.v + (at < 0 ? 0 : at) + lane * E);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) w[x][e] = at < 0 ? 0u : v[e];
        }
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          uint32_t here = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const uint32_t v = w[x][e >> 1] >> (16 * (e & 1)) & 0xFFFFu, bit = 1u << e;
            if ((v & 0x7FFFu) > kInf) nan |= bit;
            if ((v & 0x7FFFu) != kInf) continue;
            here |= bit;
            (v & 0x8000u ? down : up) |= bit;
          }
          if (!__any_sync(0xFFFFFFFFu, here != 0)) continue;
          const uint16_t* k = p.kv.k + __shfl_sync(0xFFFFFFFFu, mine, x0 + x);
#pragma unroll 1
          for (int r = 0; r < count; ++r) {
            float s = 0.f;
            for (int e = lane * 2; e < D; e += 64) {
              const float2 a = unpack2<BF16>(*reinterpret_cast<const uint32_t*>(q + r * D + e));
              const float2 b = unpack2<BF16>(*reinterpret_cast<const uint32_t*>(k + e));
              s = fmaf(a.x, b.x, fmaf(a.y, b.y, s));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            if (s * p.scale_log2 != kNegInf) continue;
#pragma unroll
            for (int i = 0; i < R; ++i) zero[i] |= i == r ? here : 0u;
          }
        }
      }
    }
#pragma unroll 1
    for (int r = 0; r < count; ++r) {
      const uint32_t have = nans(r);
      uint32_t fix = have & ~nan & (up ^ down);
#pragma unroll
      for (int i = 0; i < R; ++i) fix &= i == r ? ~zero[i] : ~0u;
      if (!__any_sync(0xFFFFFFFFu, fix != 0)) continue;
      if (__all_sync(0xFFFFFFFFu, have == kAll)) {         // all of a row: its scores may be the reason
        bool lost = false;
        for (unsigned j = j0; j < j1 && !__any_sync(0xFFFFFFFFu, lost); j += 32) {
          const int64_t at = place_of(j + lane);
          float s = 0.f;
          for (int e = 0; e < D && at >= 0; e += 8) {
            const uint4 a4 = *reinterpret_cast<const uint4*>(q + r * D + e);
            const uint4 b4 = *reinterpret_cast<const uint4*>(p.kv.k + at + e);
            const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 u = unpack2<BF16>(a[i]), t = unpack2<BF16>(b[i]);
              s = fmaf(u.x, t.x, fmaf(u.y, t.y, s));
            }
          }
          lost = !(s * p.scale_log2 < -kNegInf);
        }
        if (__any_sync(0xFFFFFFFFu, lost)) continue;
      }
      for (int e = 0; e < E; ++e) {
        if (!((fix >> e) & 1)) continue;
        const bool plus = (up >> e) & 1;
        if (whole) out[r * D + e] = (uint16_t)(out_inf | (plus ? 0u : 0x8000u));
        else part[r * Pitch + e] = plus ? -kNegInf : kNegInf;
      }
    }
  }
  __syncwarp();
}

template <int D, int NQ, bool BF16>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
  using S = Shape<D>;
  constexpr int W = S::kWarps, T = S::kThreads, R = NQ * 8;        // R: query heads per unit, padded
  constexpr int KS = D / 16;                                       // 16-wide steps along a head
  constexpr int CPR = D / 8;                                       // 16-byte chunks of a key
  constexpr int kPitch = D + 4;                                    // floats between heads of a warp's part
  constexpr int kPartWords = R * D + 2 * R;                        // a CTA's part: entries, then (maximum, sum) pairs
  constexpr float kShift = BF16 ? 0.f : 15.f;                      // P is kept 2^kShift times as large
  extern __shared__ __align__(128) unsigned char smem[];
  int* pre = reinterpret_cast<int*>(smem + S::kRing);
  uint32_t* meta = reinterpret_cast<uint32_t*>(pre + p.n_seqs + 1);
  constexpr int P = 2 * W;                                         // parts of a CTA at most: two per warp
  static_assert(P <= 32, "one lane for each part");
  __shared__ float2 part_ml[P][R];                                 // (maximum, sum) of a part
  __shared__ UnitOut part_to[P];
  __shared__ int part_unit[P];                                     // unit of a part, -1: none
  __shared__ int2 note[W][S::kStages];                             // tile in a stage: keys that count and flags; unit
  __shared__ int2 wsum[W];
  __shared__ bool spoilt[W];                                       // NaN among the warp's sums
  __shared__ bool joined[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = p.n_seqs, heads = p.kv.n_heads * p.row_tiles;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- prefix sums of the requests' tiles
  int kinds;                                               // of requests that the call has
  constexpr int kLong = 1, kEmpty = 2, kShort = 4;         // more than kUnitTiles tiles, a row but no key, 1 to kSnap tiles
  {
    const int per = (n + T - 1) / T, b0 = min(n, tid * per), b1 = min(n, b0 + per);
    const int most = p.width * p.kv.page_size;
    int sum = 0;
    kinds = 0;
    for (int b = b0; b < b1; ++b) {
      int len = p.lens[b], row = b;
      bool skip = false;
      if (p.cu_rows) {
        const int r1 = p.cu_rows[b + 1];
        row = r1 - 1;
        skip = p.cu_rows[b] >= r1;                                 // no row in this step
      }
      if (!skip && (row < 0 || row >= p.n_rows)) {
        skip = true;
        *p.status = SVQ_ERR_INVALID_ARG;
      }
      if (!skip && (len < 0 || len > most)) {
        len = len < 0 ? 0 : most;
        *p.status = SVQ_ERR_INVALID_ARG;
      }
      if (skip) len = 0;
      const int nt = (len + kTile - 1) / kTile;
      pre[b] = nt;
      meta[b] = skip ? kNoRow : ((uint32_t)row << 4) | (uint32_t)(nt * kTile - len);
      sum += nt;
      kinds |= nt > S::kUnitTiles ? kLong : nt > kSnap ? 0 : nt > 0 ? kShort : skip ? 0 : kEmpty;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += v;
    }
    kinds = __reduce_or_sync(0xFFFFFFFFu, kinds);
    if (lane == 31) wsum[warp] = make_int2(inc, kinds);
    __syncthreads();
    int before = inc - sum, all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int2 v = wsum[w];
      before += w < warp ? v.x : 0;
      all += v.x;
      kinds |= v.y;
    }
    for (int b = b0; b < b1; ++b) {
      const int nt = pre[b];
      pre[b] = before;
      before += nt;
    }
    if (tid == 0) pre[n] = all;
    __syncthreads();
  }
  const AttnSeqs seqs{pre, meta};
  // rows without a key: zeros, and the logarithm of an empty sum
  for (int b = blockIdx.x; (kinds & kEmpty) && b < n; b += gridDim.x) {
    if (seqs.tiles(b) != 0 || meta[b] == kNoRow) continue;
    const int64_t row = seqs.row(b);
    for (int i = tid; i < p.n_q * (D / 2); i += T) reinterpret_cast<uint32_t*>(p.out + row * p.n_q * D)[i] = 0u;
    if (p.lse)
      for (int i = tid; i < p.n_q; i += T) p.lse[row * p.n_q + i] = kNegInf;
  }
  const int cta = blockIdx.x;
  const AttnCut cut(seqs, n, heads, p.by_heads, !(kinds & kLong) && n * heads <= (int)gridDim.x, kinds & kShort,
                    gridDim.x, W);
  if (cta >= cut.ctas()) return;
  long long s0, s1, w0, w1;                                // tiles of this CTA, of this warp
  if (cut.moves()) {                                       // two edges, each with a search: side by side in two lanes
    long long edge = cut.edge(cta + (lane & 1));
    s0 = __shfl_sync(0xFFFFFFFFu, edge, 0);
    s1 = __shfl_sync(0xFFFFFFFFu, edge, 1);
    edge = cut.warp_edge(s0, s1, warp + (lane & 1), W);
    w0 = __shfl_sync(0xFFFFFFFFu, edge, 0);
    w1 = __shfl_sync(0xFFFFFFFFu, edge, 1);
  } else {
    s0 = cut.edge(cta);
    s1 = cut.edge(cta + 1);
    const AttnLine part(s1 - s0, W);
    w0 = s0 + part.start(warp);
    w1 = s0 + part.start(warp + 1);
  }
  if (s1 <= s0) return;

  const uint32_t ring = sm100::smem_u32(smem) + warp * S::kStages * S::kStage;
  const int g8 = lane >> 2, t2 = (lane & 3) * 2;
  if (lane < 2) part_unit[2 * warp + lane] = -1;
  if (lane == 0) spoilt[warp] = false;

  // the shift is taken off the sum, which is exact; m - kShift would round a small m to the
  // size of 15 (lse of 1, 2 and 4 keys off by 3.4, 2.2 and 1.5e-7 of itself, so by 1.9, 1.3
  // and 0.9e-7)
  auto log_sum = [](float m, float l) {
    return l == 0.f ? kNegInf : fmaf(m, 0.6931471805599453f, logf(l * (BF16 ? 1.f : 0x1p-15f)));
  };
  auto put4 = [&](int64_t row, int head, int d, float2 ml, const float4& acc) {
    const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
    const float v[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
    *reinterpret_cast<uint2*>(p.out + (row * p.n_q + head) * D + d) =
        p.out_bf16 ? make_uint2(pack2<true>(v[0], v[1]), pack2<true>(v[2], v[3]))
                   : make_uint2(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]));
    if (p.lse && d == 0) p.lse[row * p.n_q + head] = log_sum(ml.x, ml.y);
  };

  // The drained ring takes both parts of its warp.  A part left in mid-range waits
  // in the workspace until then.
  static_assert(2 * R * kPitch * 4 <= S::kStages * S::kStage, "two parts in a warp's ring");
  auto part_room = [&](int w, int slot) {
    return reinterpret_cast<float*>(smem + (size_t)w * S::kStages * S::kStage) + (slot ? 0 : R * kPitch);
  };
  float* spilled = p.warp_part + ((int64_t)cta * W + warp) * R * kPitch;
  const int todo = (int)(w1 - w0);
  if (todo > 0) {
    // ---- this warp's stream of tiles.  Every 32 tiles each lane finds the place of
    // one of them: request, head and tile, its first page and the keys that count.
    const bool whole = p.kv.page_size % kTile == 0;        // a tile lies in one page
    int64_t at_base = 0;                                   // of lane's tile: element of its first key (or of its head)
    int at_key = 0, at_req = 0, at_unit = 0, at_info = 0;  // info: keys | unit begins << 8 | unit ends << 9
    auto look_up = [&](int first) {
      if (first + lane >= todo) return;
      AttnCursor c;
      c.set(seqs, n, heads, p.by_heads, w0 + first + lane);
      at_key = c.t * kTile;
      at_req = c.b;
      at_unit = c.unit(heads);
      at_base = (int64_t)p.by_row_tiles.div(c.h) * p.kv.head_stride;
      int keys = min(kTile, seqs.len(c.b) - at_key);
      if (whole) {
        const int j = p.by_page.div(at_key);
        const int page = p.table[(int64_t)c.b * p.width + j];
        if ((unsigned)page < (unsigned)p.kv.n_pages) {
          at_base += (int64_t)page * p.kv.page_stride + (int64_t)(at_key - j * p.kv.page_size) * p.kv.token_stride;
        } else {                                           // keys on a page that does not exist do not count
          keys = 0;
          *p.status = SVQ_ERR_INVALID_ARG;
        }
      }
      at_info = keys | (c.t == 0) << 8 | (c.t == c.nt - 1) << 9;
    };
    constexpr int kStep = 32 / CPR;                        // keys copied by one instruction of the warp
    const int chunk = lane % CPR, r_lane = lane / CPR;
    auto load_tile = [&](int i, int stage) {               // tile i of the range
      const int src = i & 31;
      const int64_t base = __shfl_sync(0xFFFFFFFFu, at_base, src) + chunk * 8;
      const int keys = __shfl_sync(0xFFFFFFFFu, at_info, src) & 255;
      const uint32_t dst = ring + stage * S::kStage + r_lane * S::kRow;
      uint32_t okm;
      if (whole) {
        okm = (1u << keys) - 1u;
        const int64_t step = kStep * p.kv.token_stride;
        int64_t a = base + r_lane * p.kv.token_stride;
#pragma unroll
        for (int r = 0; r < kTile; r += kStep) {
          const bool in = r + r_lane < keys;               // else the row is filled with zeros, and nothing is read
          const int64_t e = in ? a : 0;
          const uint32_t d = dst + r * S::kRow + ((chunk ^ ((r + r_lane) & 7)) << 4);
          cp_async16(d, p.kv.k + e, in ? 16 : 0);
          cp_async16(d + kTile * S::kRow, p.kv.v + e, in ? 16 : 0);
          a += step;
        }
      } else {                                             // each key looks its own page up
        const int key = __shfl_sync(0xFFFFFFFFu, at_key, src) + (lane & 15);
        const int req = __shfl_sync(0xFFFFFFFFu, at_req, src), j = p.by_page.div(key);
        int64_t mine = 0;
        bool ok = false;
        if ((lane & 15) < keys) {
          const int page = p.table[(int64_t)req * p.width + j];
          ok = (unsigned)page < (unsigned)p.kv.n_pages;
          if (ok) mine = (int64_t)page * p.kv.page_stride + (int64_t)(key - j * p.kv.page_size) * p.kv.token_stride;
          else *p.status = SVQ_ERR_INVALID_ARG;
        }
        okm = __ballot_sync(0xFFFFFFFFu, ok) & 0xFFFFu;
#pragma unroll
        for (int r = 0; r < kTile; r += kStep) {
          const int64_t key_at = __shfl_sync(0xFFFFFFFFu, mine, r + r_lane);
          const bool in = (okm >> (r + r_lane)) & 1;
          const int64_t e = in ? base + key_at : 0;
          const uint32_t d = dst + r * S::kRow + ((chunk ^ ((r + r_lane) & 7)) << 4);
          cp_async16(d, p.kv.k + e, in ? 16 : 0);
          cp_async16(d + kTile * S::kRow, p.kv.v + e, in ? 16 : 0);
        }
      }
      if (lane == src) note[warp][stage] = make_int2((at_info & 0x300) << 8 | (int)okm, at_unit);
    };

    float o[KS][NQ][4];
    float mx[NQ][2], ls[NQ][2];
    uint32_t qf[KS][NQ][2];
    UnitOut to;
    bool fresh = true;                                     // a unit begins here (for this warp)
    bool from_start = true;                                // this warp has the unit from its first tile on
    int use = 0, put_stage = 0;
    for (int i = 1 - S::kStages; i < todo; ++i) {
      // tile i is used, tile i + kStages - 1 goes into the stage that tile i - 1 has left
      cp_wait<S::kStages - 2>();
      __syncwarp();
      auto load_next = [&]() {
        const int next = i + S::kStages - 1;
        if (next < todo) {
          if ((next & 31) == 0) look_up(next);
          load_tile(next, put_stage);
        }
        cp_commit();
        put_stage = put_stage + 1 == S::kStages ? 0 : put_stage + 1;
      };
      if (i < 0) {
        load_next();
        continue;
      }
      const int2 nb = note[warp][use];
      const uint32_t okm = (uint32_t)nb.x & 0xFFFFu;
      const int unit = nb.y;
      const uint32_t kt = ring + use * S::kStage, vt = kt + kTile * S::kRow;
      use = use + 1 == S::kStages ? 0 : use + 1;
      if (fresh) {
        // what is known of the unit, worked out while its first keys are on their way
        const int b = p.by_heads.div(unit), h = unit - b * heads, kv_head = p.by_row_tiles.div(h);
        const int rt = h - kv_head * p.row_tiles, nt = seqs.tiles(b);
        const int count = min(R, p.group - rt * R);
        const long long u0 = (long long)seqs.pre[b] * heads + (long long)h * nt, u1 = u0 + nt;
        to.row = seqs.row(b);
        to.heads = (kv_head * p.group + rt * R) << 8 | count;
        to.c0 = to.c1 = cta;
        if (u0 < s0 || u1 > s1) {
          to.c0 = cut.first_cta(u0);
          to.c1 = cut.last_cta(u1);
        }
        const uint16_t* qr = p.q + ((int64_t)to.row * p.n_q + (to.heads >> 8)) * D;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          const int r = q * 8 + g8;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const uint16_t* a = qr + r * D + ks * 16 + t2;
            qf[ks][q][0] = r < count ? *reinterpret_cast<const uint32_t*>(a) : 0u;
            qf[ks][q][1] = r < count ? *reinterpret_cast<const uint32_t*>(a + 8) : 0u;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[q][e] = kNegInf;
            ls[q][e] = 0.f;
          }
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[ks][q][e] = 0.f;
        }
        from_start = (nb.x >> 16) & 1;
        fresh = false;
      }

      // scores of 16 keys: rows g8 and g8 + 8, query heads t2 and t2 + 1
      // two chains of products, half as long, where registers allow
      constexpr bool kTwo = D < 256;
      float sc[NQ][4], sd[NQ][4];
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[q][e] = sd[q][e] = 0.f;
      const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t a[4];
        ldsm4(kt + lrow * S::kRow + (((2 * ks + (lane >> 4)) ^ (lane & 7)) << 4), a);
#pragma unroll
        for (int q = 0; q < NQ; ++q) mma<BF16>(kTwo && (ks & 1) ? sd[q] : sc[q], a, qf[ks][q][0], qf[ks][q][1]);
      }
      load_next();                                         // issued while the products are on their way
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (kTwo) sc[q][e] += sd[q][e];
      const bool ok0 = (okm >> g8) & 1, ok1 = (okm >> (g8 + 8)) & 1;
      uint32_t ph[NQ][2], pl[NQ][2];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        float a0 = ok0 ? sc[q][0] * p.scale_log2 : kNegInf, a1 = ok0 ? sc[q][1] * p.scale_log2 : kNegInf;
        float b0 = ok1 ? sc[q][2] * p.scale_log2 : kNegInf, b1 = ok1 ? sc[q][3] * p.scale_log2 : kNegInf;
        float m0 = fmaxf(a0, b0), m1 = fmaxf(a1, b1);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          m0 = fmaxf(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, x));
          m1 = fmaxf(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, x));
        }
        if (__any_sync(0xFFFFFFFFu, m0 > mx[q][0] || m1 > mx[q][1])) {
          const float n0 = fmaxf(mx[q][0], m0), n1 = fmaxf(mx[q][1], m1);
          const float f0 = part_weight(mx[q][0], n0), f1 = part_weight(mx[q][1], n1);
          mx[q][0] = n0;
          mx[q][1] = n1;
          ls[q][0] *= f0;
          ls[q][1] *= f1;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            o[ks][q][0] *= f0;
            o[ks][q][1] *= f1;
            o[ks][q][2] *= f0;
            o[ks][q][3] *= f1;
          }
        }
        const float r0 = mx[q][0] == kNegInf ? 0.f : mx[q][0] - kShift;
        const float r1 = mx[q][1] == kNegInf ? 0.f : mx[q][1] - kShift;
        a0 = ex2(a0 - r0);
        b0 = ex2(b0 - r0);
        a1 = ex2(a1 - r1);
        b1 = ex2(b1 - r1);
        ls[q][0] += a0 + b0;
        ls[q][1] += a1 + b1;
        // (key, two heads) -> (head, two keys); high part and remainder
        const uint32_t h0 = pack2<BF16>(a0, a1), h1 = pack2<BF16>(b0, b1);
        const float2 w0f = unpack2<BF16>(h0), w1f = unpack2<BF16>(h1);
        ph[q][0] = transpose8(h0);
        ph[q][1] = transpose8(h1);
        pl[q][0] = transpose8(pack2<BF16>(a0 - w0f.x, a1 - w0f.y));
        pl[q][1] = transpose8(pack2<BF16>(b0 - w1f.x, b1 - w1f.y));
      }
      const int vrow = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t a[4];
        ldsm4t(vt + vrow * S::kRow + (((2 * ks + ((lane >> 3) & 1)) ^ (lane & 7)) << 4), a);
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          mma<BF16>(o[ks][q], a, ph[q][0], ph[q][1]);
          mma<BF16>(o[ks][q], a, pl[q][0], pl[q][1]);
        }
      }

      const bool unit_ends = (nb.x >> 17) & 1, range_ends = i == todo - 1;
      if (!unit_ends && !range_ends) continue;
      fresh = true;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          ls[q][0] += __shfl_xor_sync(0xFFFFFFFFu, ls[q][0], x);
          ls[q][1] += __shfl_xor_sync(0xFFFFFFFFu, ls[q][1], x);
        }
      unsigned long long probe = 0;                        // two floats, NaN if a sum is
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) probe_nan(probe, o[ks][q]);
      if (is_nan(probe)) spoilt[warp] = true;
      if (!(unit_ends && from_start)) {
        // A part: in mid-range (the ring is in use) to the workspace, else to the
        // ring, which is drained: every tile of the range has been waited for.
        const int slot = range_ends;
        float* dst = slot ? part_room(warp, 1) : spilled;
        __syncwarp();
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          float* d0 = dst + (q * 8 + t2) * kPitch + g8;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            d0[ks * 16] = o[ks][q][0];
            d0[ks * 16 + kPitch] = o[ks][q][1];
            d0[ks * 16 + 8] = o[ks][q][2];
            d0[ks * 16 + 8 + kPitch] = o[ks][q][3];
          }
          if (g8 == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) part_ml[2 * warp + slot][q * 8 + t2 + e] = make_float2(mx[q][e], ls[q][e]);
          }
        }
        if (lane == 0) {
          part_unit[2 * warp + slot] = unit;
          part_to[2 * warp + slot] = to;
        }
        continue;
      }
      // The whole unit is this warp's: it goes straight out.
      const int head0 = to.heads >> 8, count = to.heads & 255;
      const int64_t row = to.row;
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const float i0 = ls[q][0] == 0.f ? 0.f : 1.f / ls[q][0], i1 = ls[q][1] == 0.f ? 0.f : 1.f / ls[q][1];
        const int r = q * 8 + t2;
        // 8 x 8 transposes turn (entry, two heads) into (head, two entries): 4-byte stores
        const int rr = q * 8 + g8;
        uint16_t* dst = p.out + (row * p.n_q + head0 + rr) * D + t2;
#pragma unroll
        for (int x = 0; x < 2 * KS; ++x) {
          const float u = o[x >> 1][q][2 * (x & 1)] * i0, w = o[x >> 1][q][2 * (x & 1) + 1] * i1;
          const uint32_t t = transpose8(p.out_bf16 ? pack2<true>(u, w) : pack2<false>(u, w));
          if (rr < count) *reinterpret_cast<uint32_t*>(dst + x * 8) = t;
        }
        if (p.lse && g8 == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (r + e < count) p.lse[row * p.n_q + head0 + r + e] = log_sum(mx[q][e], ls[q][e]);
        }
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncwarp();
  const bool parked = part_unit[2 * warp] >= 0, nan_met = spoilt[warp];
  if (nan_met) mend_sums<D, R, kPitch, BF16>(p, pre, spilled, part_room(warp, 1), w0, w1);
  if (parked) {
    const float4* src = reinterpret_cast<const float4*>(spilled);
    float4* dst = reinterpret_cast<float4*>(part_room(warp, 0));
#pragma unroll 8
    for (int i = lane; i < R * kPitch / 4; i += 32) dst[i] = __ldcg(src + i);
  }
  __syncthreads();

  // ---- join the warps' parts.  Parts of one unit are neighbours in the order
  // (warp, slot): slots 1 of consecutive warps, then perhaps a slot 0.  A warp
  // takes a row (or two of 64 entries) of a unit at a time, a lane V times 4
  // entries; no condition stands before a load, so the loads do not queue.
  constexpr int V = D == 256 ? 2 : 1, kRows = D == 64 ? 2 : 1;
  constexpr int kItems = R / kRows;                        // of a unit
  const int r_sub = D == 64 ? lane >> 4 : 0, d_lane = D == 64 ? (lane & 15) * 4 : lane * 4;    // + 128 for V = 1
  const int my_unit = lane < P ? part_unit[lane] : -1;
  const uint32_t have = __ballot_sync(0xFFFFFFFFu, my_unit >= 0);
  const uint32_t lower = have & ((1u << lane) - 1u);
  const int prev = __shfl_sync(0xFFFFFFFFu, my_unit, lower ? 31 - __clz(lower) : lane);
  const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, my_unit >= 0 && (!lower || prev != my_unit));
  // part x of a unit: CTA c0 + x's, in its place 1 if the unit begins there and else in place 0
  auto cta_part = [&](const UnitOut& u, int x) { return p.cta_part + ((u.c0 + x) * 2 + (x == 0)) * kPartWords; };
#pragma unroll 1
  for (int it = warp; it < __popc(firsts) * kItems; it += W) {
    uint32_t left = firsts;
#pragma unroll 1
    for (int k = it / kItems; k > 0; --k) left &= left - 1;
    const int a = __ffs(left) - 1;
    const uint32_t later = left & (left - 1);              // the next unit's first part
    const uint32_t members = have & ~((1u << a) - 1u) & (later ? (later & (0u - later)) - 1u : ~0u);
    const int last = 31 - __clz(members), w0p = a >> 1, n_parts = (last >> 1) - w0p + 1;
    const UnitOut u = part_to[a];
    const int r = it % kItems * kRows + r_sub;
    if (it % kItems * kRows >= (u.heads & 255)) continue;
    // part x is slot 1 of warp w0p + x, but for the last, which is `last`
    float M = kNegInf, L = 0.f;
#pragma unroll 4
    for (int x = 0; x < n_parts; ++x) M = fmaxf(M, part_ml[min(2 * (w0p + x) + 1, last)][r].x);
    float4 acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = 0; x < n_parts; ++x) {
      const int y = min(2 * (w0p + x) + 1, last);
      const float2 ml = part_ml[y][r];
      const float f = part_weight(ml.x, M);
      L = fmaf(f, ml.y, L);
      const float* src = part_room(y >> 1, y & 1) + r * kPitch + d_lane;
#pragma unroll
      for (int k = 0; k < V; ++k) weigh(acc[k], f, reinterpret_cast<const float4*>(src)[k * 32]);
    }
    if (r >= (u.heads & 255)) continue;
    if (u.c0 != u.c1) {
      float* far = cta_part(u, cta - u.c0);
#pragma unroll
      for (int k = 0; k < V; ++k) reinterpret_cast<float4*>(far + r * D + d_lane)[k * 32] = acc[k];
      if (d_lane == 0) *reinterpret_cast<float2*>(far + R * D + 2 * r) = make_float2(M, L);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) put4(u.row, (u.heads >> 8) + r, d_lane + k * 128, make_float2(M, L), acc[k]);
    }
  }
  // The CTA's first unit may have begun in another CTA, its last may go on in one.
  if (!firsts) return;
  const int a0 = __ffs(firsts) - 1, a1 = 31 - __clz(firsts);
  const bool from_before = part_to[a0].c0 < cta, goes_on = part_to[a1].c0 == cta && part_to[a1].c1 > cta;
  if (!from_before && !goes_on) return;

  // ---- join the CTAs' parts, up to kFan neighbours at a time: the last of them to
  // get here adds them and goes on in their place (a wide unit on many CTAs would
  // keep a single one busy for longer than the whole loop).  The wider a part, the
  // fewer at a time: 32 of 4 KB save a level (1 x 131072 of 8 heads of 128: 88.3 us
  // against 89.6 us with 16), 32 of 16 KB cost 7 us against 16 (8 wide).
  constexpr int kFan = D == 64 ? 16 : R * D <= 1024 ? 32 : R * D <= 2048 ? 16 : 8;
  auto arrive = [&](const UnitOut& u, int stride, int level) {
    int members;
    const int first = attn_group(u.c1 - u.c0 + 1, kFan, stride, cta - u.c0, &members);
    if (members == 1) return true;
    // Release of this CTA's part (a barrier puts all threads' stores before it)
    // and acquire of the others'; the counter wraps to zero with the last.
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                 : "=r"(old)
                 : "l"(p.counters + level * (int)gridDim.x + u.c0 + first), "r"((unsigned)(members - 1))
                 : "memory");
    return old == (unsigned)(members - 1);
  };
  constexpr int kLanes = 32 / kRows;                       // lanes of a row: lane x looks at part x
  static_assert(kFan <= kLanes, "a lane for each part of a group");
#pragma unroll 1
  for (int stride = 1, level = 0;; stride *= kFan, ++level) {
    __syncthreads();                                       // the parts of this CTA are written
    if (tid < 2) {
      const bool mine = level == 0 ? (tid ? goes_on : from_before) : joined[tid];
      joined[tid] = mine && arrive(part_to[tid ? a1 : a0], stride, level);
    }
    __syncthreads();
    if (!joined[0] && !joined[1]) return;
#pragma unroll 1
    for (int it = warp; it < 2 * kItems; it += W) {
      const int s = it / kItems;
      if (!joined[s]) continue;
      const UnitOut u = part_to[s ? a1 : a0];
      const int r = it % kItems * kRows + r_sub;
      if (it % kItems * kRows >= (u.heads & 255)) continue;
      int members;
      const int first = attn_group(u.c1 - u.c0 + 1, kFan, stride, cta - u.c0, &members);
      const float* base = cta_part(u, first);
      // parts beyond the first stand 2 * stride places apart, in place 0
      const float* rest = cta_part(u, first + stride);
      const int64_t pitch = (int64_t)stride * 2 * kPartWords;
      auto part_at = [&](int x) { return x == 0 ? base : rest + (x - 1) * pitch; };
      const int mine = min(lane % kLanes, members - 1);
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(part_at(mine) + R * D + 2 * r));
      constexpr int kBatch = 8;
      float4 v[kBatch][V];
#pragma unroll
      for (int x = 0; x < kBatch; ++x)                     // beyond the last: loaded again, without weight
#pragma unroll
        for (int k = 0; k < V; ++k)
          v[x][k] = __ldcg(reinterpret_cast<const float4*>(part_at(min(x, members - 1)) + r * D + d_lane) + k * 32);
      float M = lane % kLanes < members ? ml.x : kNegInf;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
      const float f = lane % kLanes < members ? part_weight(ml.x, M) : 0.f;
      float L = lane % kLanes < members ? f * ml.y : 0.f;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
      float4 acc[V];
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int x0 = 0;; x0 += kBatch) {
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const float g = __shfl_sync(0xFFFFFFFFu, f, x0 + x, kLanes);
          const bool in = x0 + x < members;
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const float4 t = v[x][k];
            weigh(acc[k], g, make_float4(in ? t.x : 0.f, in ? t.y : 0.f, in ? t.z : 0.f, in ? t.w : 0.f));
          }
        }
        if (x0 + kBatch >= members) break;
#pragma unroll
        for (int x = 0; x < kBatch; ++x)
#pragma unroll
          for (int k = 0; k < V; ++k)
            v[x][k] = __ldcg(
                reinterpret_cast<const float4*>(part_at(min(x0 + kBatch + x, members - 1)) + r * D + d_lane) + k * 32);
      }
      if (r >= (u.heads & 255)) continue;
      if (stride * kFan > u.c1 - u.c0) {
#pragma unroll
        for (int k = 0; k < V; ++k) put4(u.row, (u.heads >> 8) + r, d_lane + k * 128, make_float2(M, L), acc[k]);
      } else {
        float* far = const_cast<float*>(base);
#pragma unroll
        for (int k = 0; k < V; ++k) reinterpret_cast<float4*>(far + r * D + d_lane)[k * 32] = acc[k];
        if (d_lane == 0) *reinterpret_cast<float2*>(far + R * D + 2 * r) = make_float2(M, L);
      }
    }
    __syncthreads();
    if (tid < 2 && joined[tid]) {
      const UnitOut u = part_to[tid ? a1 : a0];
      joined[tid] = stride * kFan <= u.c1 - u.c0;          // not yet the whole unit
    }
    __syncthreads();
    if (!joined[0] && !joined[1]) return;
  }
}

// Rows of the output from natural order to that of their consumer, in place: entry
// i to column order[i], a row (of a request with a row in this step) to a CTA, by
// way of shared memory.  Two-byte stores straight from the attention kernel, a
// sector each, made it a third slower (158 requests of up to 1276 keys, 32 heads of
// 128: 68 us against 48 us in natural order).
constexpr int kOrderThreads = 256;

__global__ void __launch_bounds__(kOrderThreads) order_rows_kernel(const __grid_constant__ PagedAttnParams p, int words) {
  extern __shared__ __align__(16) uint16_t line[];         // [words]
  const int b = blockIdx.x;
  for (int i = threadIdx.x * 8; i < words; i += kOrderThreads * 8)       // columns that no entry goes to
    *reinterpret_cast<uint4*>(line + i) = make_uint4(0u, 0u, 0u, 0u);
  // the first columns before the previous kernel has finished: order is a weight
  constexpr int kAhead = 2;
  int4 first[kAhead][2];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = (threadIdx.x + k * kOrderThreads) * 8;
    if (i < words) {
      first[k][0] = __ldg(reinterpret_cast<const int4*>(p.order + i));
      first[k][1] = __ldg(reinterpret_cast<const int4*>(p.order + i + 4));
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int row = b;
  if (p.cu_rows) {
    const int r1 = p.cu_rows[b + 1];
    if (p.cu_rows[b] >= r1) return;
    row = r1 - 1;
  }
  if (row < 0 || row >= p.n_rows) return;                  // reported by the attention kernel
  __syncthreads();
  uint16_t* out = p.out + (int64_t)row * words;
  auto scatter = [&](int i, const int4& o0, const int4& o1) {
    const uint4 v = *reinterpret_cast<const uint4*>(out + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const int at[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if ((unsigned)at[e] < (unsigned)words) line[at[e]] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      else *p.status = SVQ_ERR_INVALID_ARG;
    }
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = (threadIdx.x + k * kOrderThreads) * 8;
    if (i < words) scatter(i, first[k][0], first[k][1]);
  }
  for (int i = (threadIdx.x + kAhead * kOrderThreads) * 8; i < words; i += kOrderThreads * 8)
    scatter(i, __ldg(reinterpret_cast<const int4*>(p.order + i)), __ldg(reinterpret_cast<const int4*>(p.order + i + 4)));
  __syncthreads();
  for (int i = threadIdx.x * 8; i < words; i += kOrderThreads * 8)
    *reinterpret_cast<uint4*>(out + i) = *reinterpret_cast<const uint4*>(line + i);
}

cudaError_t order_rows(const PagedAttnParams& p, int words, cudaStream_t st) {
  static std::atomic<int> have[64];
  const cudaError_t e = allow_smem(order_rows_kernel, kMaxOrdered * 2, have);
  if (e != cudaSuccess) return e;
  return launch_dependent(order_rows_kernel, dim3((unsigned)p.n_seqs), kOrderThreads, (size_t)words * 2, 1, st, p, words);
}

template <int D>
constexpr size_t smem_bytes(int n_seqs) { return Shape<D>::kRing + (size_t)(2 * n_seqs + 1) * 4; }

template <int D>
void plan_d(int n_seqs, PagedAttnPlan* plan) {
  plan->warps = Shape<D>::kWarps;
  plan->smem = smem_bytes<D>(n_seqs);
}

template <int D, int NQ, bool BF16>
cudaError_t launch_dq(const PagedAttnParams& p, const PagedAttnPlan& plan, cudaStream_t st) {
  // the most any call needs, so that concurrent first calls agree
  static std::atomic<int> have[64];
  const cudaError_t e = allow_smem(paged_attn_kernel<D, NQ, BF16>, smem_bytes<D>(kMaxSeqs), have);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_attn_kernel<D, NQ, BF16>, (unsigned)plan.ctas, Shape<D>::kThreads, plan.smem, 1, st,
                          p);
}

template <int D>
cudaError_t launch_d(const PagedAttnParams& p, const PagedAttnPlan& plan, int kv_bf16, cudaStream_t st) {
  if (plan.rows == 8) return kv_bf16 ? launch_dq<D, 1, true>(p, plan, st) : launch_dq<D, 1, false>(p, plan, st);
  return kv_bf16 ? launch_dq<D, 2, true>(p, plan, st) : launch_dq<D, 2, false>(p, plan, st);
}

}  // namespace

bool plan_paged_attn(int n_q, int n_kv, int head_dim, int n_seqs, int num_sms, PagedAttnPlan* plan) {
  if (n_kv < 1 || n_q < n_kv || n_q % n_kv != 0) return false;
  plan->ctas = num_sms;                                    // one per SM: the ring fills its shared memory
  plan->rows = n_q / n_kv <= 8 ? 8 : 16;
  switch (head_dim) {
    case 64: plan_d<64>(n_seqs, plan); break;
    case 128: plan_d<128>(n_seqs, plan); break;
    case 256: plan_d<256>(n_seqs, plan); break;
    default: return false;
  }
  // Counters at the start, in the region that the GEMV keeps its own in (both
  // leave them at zero), then the parts.
  const size_t cta_bytes = (size_t)plan->ctas * 2 * (plan->rows * head_dim + 2 * plan->rows) * 4;
  plan->cta_part = kGemvCounterBytes;
  plan->warp_part = (plan->cta_part + cta_bytes + 255) / 256 * 256;
  plan->ws_total = plan->warp_part + (size_t)plan->ctas * plan->warps * plan->rows * (head_dim + 4) * 4;
  return true;
}

cudaError_t launch_paged_attn(const PagedAttnParams& p, const PagedAttnPlan& plan, int head_dim, int kv_bf16,
                              cudaStream_t st) {
  const cudaError_t e = head_dim == 64    ? launch_d<64>(p, plan, kv_bf16, st)
                        : head_dim == 128 ? launch_d<128>(p, plan, kv_bf16, st)
                                          : launch_d<256>(p, plan, kv_bf16, st);
  if (e != cudaSuccess || !p.order) return e;
  return order_rows(p, p.n_q * head_dim, st);
}

}  // namespace svq
