// paged_attention.cu -- attention of one new token per request over a paged
// key/value cache.
//
//   s_j = scale * q . k_j,  p_j = e^(s_j - max s),  o = sum_j p_j v_j / sum_j p_j,   j < len
//
// Every key and value is read once for the whole group of query heads that
// shares it, so the cache's bytes bound the call; everything here serves to keep
// loads in flight on every SM whatever the lengths are.
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
  static constexpr int kWarps = D == 256 ? 4 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = D == 64 ? 5 : 3;
  static constexpr int kRow = D * 2;                       // bytes of one key
  static constexpr int kStage = kTile * kRow * 2;          // K tile, then V tile
  static constexpr int kRing = kWarps * kStages * kStage;
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
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
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
__device__ __forceinline__ uint16_t out16(float v, int bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Weight of a part with maximum m in a join whose maximum is M (both in units of
// log2): a part that saw no key has m = -inf and weight 0.
__device__ __forceinline__ float part_weight(float m, float M) { return m == kNegInf ? 0.f : ex2(m - M); }

template <int D, int NQ, bool BF16>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
  using S = Shape<D>;
  constexpr int W = S::kWarps, T = S::kThreads, R = NQ * 8;        // R: query heads per unit, padded
  constexpr int KS = D / 16;                                       // 16-wide steps along a head
  constexpr int CPR = D / 8;                                       // 16-byte chunks of a key
  constexpr float kShift = BF16 ? 0.f : 15.f;                      // P is kept 2^kShift times as large
  extern __shared__ __align__(128) unsigned char smem[];
  int* pre = reinterpret_cast<int*>(smem + S::kRing);
  uint32_t* meta = reinterpret_cast<uint32_t*>(pre + p.n_seqs + 1);
  __shared__ float part_m[W][2][R], part_l[W][2][R];
  __shared__ long long part_unit[W][2];                            // unit of a part, -1: none
  __shared__ uint32_t live[W][S::kStages];                         // keys of a stage that count
  __shared__ int wsum[W];
  __shared__ unsigned joined[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = p.n_seqs, heads = p.kv.n_heads * p.row_tiles;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- prefix sums of the requests' tiles
  {
    const int per = (n + T - 1) / T, b0 = min(n, tid * per), b1 = min(n, b0 + per);
    const int most = p.width * p.kv.page_size;
    int sum = 0;
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
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int before = inc - sum;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    for (int b = b0; b < b1; ++b) {
      const int nt = pre[b];
      pre[b] = before;
      before += nt;
    }
    if (tid == 0) {
      int all = 0;
      for (int w = 0; w < W; ++w) all += wsum[w];
      pre[n] = all;
    }
    __syncthreads();
  }
  const AttnSeqs seqs{pre, meta};
  // rows without a key: zeros, and the logarithm of an empty sum
  for (int b = blockIdx.x; b < n; b += gridDim.x) {
    if (seqs.tiles(b) != 0 || meta[b] == kNoRow) continue;
    const int64_t row = seqs.row(b);
    for (int i = tid; i < p.n_q * (D / 2); i += T) reinterpret_cast<uint32_t*>(p.out + row * p.n_q * D)[i] = 0u;
    if (p.lse)
      for (int i = tid; i < p.n_q; i += T) p.lse[row * p.n_q + i] = kNegInf;
  }
  const long long total = (long long)pre[n] * heads;
  const int ctas = attn_ctas(total, gridDim.x, W);
  const int cta = blockIdx.x;
  if (cta >= ctas) return;
  const long long s0 = range_start(total, cta, ctas), s1 = range_start(total, cta + 1, ctas);
  const long long w0 = s0 + range_start(s1 - s0, warp, W), w1 = s0 + range_start(s1 - s0, warp + 1, W);

  const uint32_t ring = sm100::smem_u32(smem) + warp * S::kStages * S::kStage;
  float o[KS][NQ][4];
  float mx[NQ][2], ls[NQ][2];
  uint32_t qf[KS][NQ][2];
  const int g8 = lane >> 2, t2 = (lane & 3) * 2;
  if (lane < 2) part_unit[warp][lane] = -1;

  // Writes the running part of unit (b, h) of this warp: slot 0 to the
  // workspace in mid-range (the ring is in use), slot 1 to the drained ring.
  auto leave_part = [&](const AttnCursor& c, int slot) {
    float* dst = slot == 0 ? p.warp_part + ((int64_t)cta * W + warp) * R * D
                           : reinterpret_cast<float*>(smem + (size_t)warp * S::kStages * S::kStage);
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const int d = i * 16 + g8, r = q * 8 + t2;
        dst[r * D + d] = o[i][q][0];
        dst[(r + 1) * D + d] = o[i][q][1];
        dst[r * D + d + 8] = o[i][q][2];
        dst[(r + 1) * D + d + 8] = o[i][q][3];
      }
      if (g8 == 0) {
        part_m[warp][slot][q * 8 + t2] = mx[q][0];
        part_m[warp][slot][q * 8 + t2 + 1] = mx[q][1];
        part_l[warp][slot][q * 8 + t2] = ls[q][0];
        part_l[warp][slot][q * 8 + t2 + 1] = ls[q][1];
      }
    }
    if (lane == 0) part_unit[warp][slot] = c.unit(heads);
  };
  // Heads of a unit: first query head and how many of the R rows are real.
  auto unit_heads = [&](int h, int* count) {
    const int kv_head = h / p.row_tiles, rt = h - kv_head * p.row_tiles;
    *count = min(R, p.group - rt * R);
    return kv_head * p.group + rt * R;
  };
  auto put = [&](int64_t row, int head, int d, float v) {
    const int i = head * D + d;
    int at = i;
    if (p.order) {
      at = p.order[i];
      if ((unsigned)at >= (unsigned)(p.n_q * D)) {
        *p.status = SVQ_ERR_INVALID_ARG;
        return;
      }
    }
    p.out[row * p.n_q * D + at] = out16(v, p.out_bf16);
  };
  auto log_sum = [](float m, float l) {
    return l == 0.f ? kNegInf : fmaf(m - kShift, 0.6931471805599453f, logf(l));
  };
  // A unit that lies wholly inside this warp's range goes straight out.
  auto write_unit = [&](const AttnCursor& c) {
    int count;
    const int head0 = unit_heads(c.h, &count);
    const int64_t row = seqs.row(c.b);
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const float i0 = ls[q][0] == 0.f ? 0.f : 1.f / ls[q][0], i1 = ls[q][1] == 0.f ? 0.f : 1.f / ls[q][1];
      const int r = q * 8 + t2;
      if (p.order) {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const int d = i * 16 + g8;
          if (r < count) {
            put(row, head0 + r, d, o[i][q][0] * i0);
            put(row, head0 + r, d + 8, o[i][q][2] * i0);
          }
          if (r + 1 < count) {
            put(row, head0 + r + 1, d, o[i][q][1] * i1);
            put(row, head0 + r + 1, d + 8, o[i][q][3] * i1);
          }
        }
      } else {
        // 8 x 8 transposes turn (entry, two heads) into (head, two entries): 4-byte stores
        const int rr = q * 8 + g8;
        uint16_t* dst = p.out + (row * p.n_q + head0 + rr) * D + t2;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const uint32_t lo = p.out_bf16 ? pack2<true>(o[i][q][0] * i0, o[i][q][1] * i1)
                                         : pack2<false>(o[i][q][0] * i0, o[i][q][1] * i1);
          const uint32_t hi = p.out_bf16 ? pack2<true>(o[i][q][2] * i0, o[i][q][3] * i1)
                                         : pack2<false>(o[i][q][2] * i0, o[i][q][3] * i1);
          const uint32_t a = transpose8(lo), b = transpose8(hi);
          if (rr < count) {
            *reinterpret_cast<uint32_t*>(dst + i * 16) = a;
            *reinterpret_cast<uint32_t*>(dst + i * 16 + 8) = b;
          }
        }
      }
      if (p.lse && g8 == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (r + e < count)
            p.lse[row * p.n_q + head0 + r + e] = log_sum(mx[q][e], ls[q][e]);
      }
    }
  };

  if (w0 < w1) {
    // ---- this warp's stream of tiles
    AttnCursor put_c, get_c;                                   // next tile to load, next tile to use
    get_c.set(seqs, n, heads, w0);
    put_c = get_c;
    const int todo = (int)(w1 - w0);
    int loaded = 0;                                        // tiles whose loads have been issued
    int page, off;                                         // of key (lane & 15) of the next tile to load
    bool in;
    auto look_up = [&]() {
      const int key = put_c.t * kTile + (lane & 15);
      const int j = key / p.kv.page_size;
      off = key - j * p.kv.page_size;
      in = key < seqs.len(put_c.b);
      page = in ? __ldg(p.table + (int64_t)put_c.b * p.width + j) : 0;
    };
    auto load_tile = [&](int stage) {
      if (loaded < todo) {
        const bool ok = in && (unsigned)page < (unsigned)p.kv.n_pages;
        if (in && !ok) *p.status = SVQ_ERR_INVALID_ARG;    // a key on a page that does not exist does not count
        const uint32_t okm = __ballot_sync(0xFFFFFFFFu, ok) & 0xFFFFu;
        const int64_t base =
            ok ? (int64_t)page * p.kv.page_stride + (int64_t)off * p.kv.token_stride : (int64_t)0;
        const uint16_t* kh = p.kv.k + (int64_t)(put_c.h / p.row_tiles) * p.kv.head_stride;
        const uint16_t* vh = p.kv.v + (int64_t)(put_c.h / p.row_tiles) * p.kv.head_stride;
        const uint32_t dst = ring + stage * S::kStage;
        const int chunk = lane % CPR;
#pragma unroll
        for (int i = 0; i < kTile * CPR / 32; ++i) {
          const int r = i * (32 / CPR) + lane / CPR;
          const int64_t a = __shfl_sync(0xFFFFFFFFu, base, r) + chunk * 8;
          const int bytes = (okm >> r) & 1 ? 16 : 0;       // 0: the row is filled with zeros
          const uint32_t d = dst + r * S::kRow + ((chunk ^ (r & 7)) << 4);
          cp_async16(d, kh + a, bytes);
          cp_async16(d + kTile * S::kRow, vh + a, bytes);
        }
        if (lane == 0) live[warp][stage] = okm;
        if (++loaded < todo) {
          put_c.next(seqs, n, heads);
          look_up();
        }
      }
      cp_commit();
    };
    look_up();
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) load_tile(i);

    bool fresh = true;                                     // a unit begins here (for this warp)
    bool from_start = get_c.t == 0;                        // this warp has the unit from its first tile on
    int stage = 0;
    for (int i = 0; i < todo; ++i) {
      if (fresh) {
        int count;
        const int head0 = unit_heads(get_c.h, &count);
        const uint16_t* qr = p.q + ((int64_t)seqs.row(get_c.b) * p.n_q + head0) * D;
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
        fresh = false;
      }
      cp_wait<S::kStages - 2>();
      __syncwarp();
      const uint32_t okm = live[warp][stage];
      {
        const int ahead = stage == 0 ? S::kStages - 1 : stage - 1;   // the stage used one tile ago
        load_tile(ahead);
      }
      const uint32_t kt = ring + stage * S::kStage, vt = kt + kTile * S::kRow;
      stage = stage + 1 == S::kStages ? 0 : stage + 1;

      // scores of 16 keys: rows g8 and g8 + 8, query heads t2 and t2 + 1
      float sc[NQ][4];
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[q][e] = 0.f;
      const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t a[4];
        ldsm4(kt + lrow * S::kRow + (((2 * ks + (lane >> 4)) ^ (lane & 7)) << 4), a);
#pragma unroll
        for (int q = 0; q < NQ; ++q) mma<BF16>(sc[q], a, qf[ks][q][0], qf[ks][q][1]);
      }
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

      const bool unit_ends = get_c.t == get_c.nt - 1, range_ends = i == todo - 1;
      if (unit_ends || range_ends) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) {
            ls[q][0] += __shfl_xor_sync(0xFFFFFFFFu, ls[q][0], x);
            ls[q][1] += __shfl_xor_sync(0xFFFFFFFFu, ls[q][1], x);
          }
        if (unit_ends && from_start) {
          write_unit(get_c);
        } else if (range_ends) {
          cp_wait<0>();
          __syncwarp();                                    // every lane is done with the ring
          leave_part(get_c, 1);
        } else {
          leave_part(get_c, 0);
        }
        fresh = true;
        from_start = true;
      }
      if (!range_ends) get_c.next(seqs, n, heads);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();

  // ---- join the warps' parts.  Parts of one unit are neighbours in the order
  // (warp, slot); units that reach beyond this CTA leave a part in the workspace.
  const int part_words = R * D + 2 * R;
  auto cta_part = [&](int c, int slot) { return p.cta_part + ((int64_t)c * 2 + slot) * part_words; };
  long long far_unit[2] = {-1, -1};                        // units that other CTAs share, and their CTAs
  int far_c0[2], far_c1[2];
  for (int a = 0; a < 2 * W;) {
    const long long unit = part_unit[a >> 1][a & 1];
    if (unit < 0) {
      ++a;
      continue;
    }
    int e = a + 1;
    while (e < 2 * W && (part_unit[e >> 1][e & 1] < 0 || part_unit[e >> 1][e & 1] == unit)) ++e;
    const int b = (int)(unit / heads), h = (int)(unit - (long long)b * heads);
    const long long u0 = (long long)seqs.pre[b] * heads + (long long)h * seqs.tiles(b), u1 = u0 + seqs.tiles(b);
    int count;
    const int head0 = unit_heads(h, &count);
    const bool whole = u0 >= s0 && u1 <= s1;
    float* far = nullptr;
    if (!whole) {
      const int slot = u0 >= s0;                           // 1: the unit begins here, 0: it began before
      far_unit[slot] = unit;
      far_c0[slot] = range_of(u0, total, ctas);
      far_c1[slot] = range_of(u1 - 1, total, ctas);
      far = cta_part(cta, slot);
    }
    const int64_t row = seqs.row(b);
    for (int i = tid; i < count * D; i += T) {
      const int r = i / D, d = i - r * D;
      float M = kNegInf;
      for (int x = a; x < e; ++x)
        if (part_unit[x >> 1][x & 1] == unit) M = fmaxf(M, part_m[x >> 1][x & 1][r]);
      float acc = 0.f, L = 0.f;
      for (int x = a; x < e; ++x) {
        if (part_unit[x >> 1][x & 1] != unit) continue;
        const float f = part_weight(part_m[x >> 1][x & 1][r], M);
        const float v = x & 1 ? reinterpret_cast<const float*>(smem + (size_t)(x >> 1) * S::kStages * S::kStage)[i]
                              : __ldcg(p.warp_part + ((int64_t)cta * W + (x >> 1)) * R * D + i);
        acc = fmaf(f, v, acc);
        L = fmaf(f, part_l[x >> 1][x & 1][r], L);
      }
      if (far) {
        far[i] = acc;
        if (d == 0) {
          far[R * D + r] = M;
          far[R * D + R + r] = L;
        }
      } else {
        put(row, head0 + r, d, L == 0.f ? 0.f : acc / L);
        if (p.lse && d == 0)
          p.lse[row * p.n_q + head0 + r] = log_sum(M, L);
      }
    }
    a = e;
  }
  if (far_unit[0] < 0 && far_unit[1] < 0) return;

  // ---- join the CTAs' parts: the last of the unit's CTAs to get here adds them.
  __threadfence();
  __syncthreads();
  if (tid < 2) {
    unsigned last = 0;
    const long long unit = tid ? far_unit[1] : far_unit[0];
    if (unit >= 0) {
      const int c0 = tid ? far_c0[1] : far_c0[0], c1 = tid ? far_c1[1] : far_c1[0];
      last = atomicInc(p.counters + c0, (unsigned)(c1 - c0)) == (unsigned)(c1 - c0);    // wraps to zero
      __threadfence();
    }
    joined[tid] = last;
  }
  __syncthreads();
  float* wts = reinterpret_cast<float*>(smem);             // [parts][R]
  for (int s = 0; s < 2; ++s) {
    if (!joined[s]) continue;
    const int c0 = far_c0[s], c1 = far_c1[s], k = c1 - c0 + 1;
    const long long unit = far_unit[s];
    const int b = (int)(unit / heads), h = (int)(unit - (long long)b * heads);
    int count;
    const int head0 = unit_heads(h, &count);
    float* psum = wts + k * R;                             // [parts][R] sums
    float* sums = psum + k * R;                            // [R] maxima, [R] sums
    for (int i = tid; i < k * R; i += T) {
      const float* ml = cta_part(c0 + i / R, i / R == 0) + R * D + i % R;
      wts[i] = __ldcg(ml);
      psum[i] = __ldcg(ml + R);
    }
    __syncthreads();
    if (tid < count) {
      float M = kNegInf, L = 0.f;
      for (int x = 0; x < k; ++x) M = fmaxf(M, wts[x * R + tid]);
      for (int x = 0; x < k; ++x) {
        const float f = part_weight(wts[x * R + tid], M);
        wts[x * R + tid] = f;
        L = fmaf(f, psum[x * R + tid], L);
      }
      sums[tid] = M;
      sums[R + tid] = L;
    }
    __syncthreads();
    const int64_t row = seqs.row(b);
    for (int i = tid; i < count * D; i += T) {
      const int r = i / D, d = i - r * D;
      float acc = 0.f;
#pragma unroll 8
      for (int x = 0; x < k; ++x) acc = fmaf(wts[x * R + r], __ldcg(cta_part(c0 + x, x == 0) + i), acc);
      const float L = sums[R + r];
      put(row, head0 + r, d, L == 0.f ? 0.f : acc / L);
      if (p.lse && d == 0)
        p.lse[row * p.n_q + head0 + r] = log_sum(sums[r], L);
    }
    __syncthreads();
  }
}

template <int D>
void plan_d(int n_seqs, PagedAttnPlan* plan) {
  plan->warps = Shape<D>::kWarps;
  plan->smem = Shape<D>::kRing + (size_t)(2 * n_seqs + 1) * 4;
}

template <int D, int NQ, bool BF16>
cudaError_t launch_dq(const PagedAttnParams& p, const PagedAttnPlan& plan, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<D, NQ, BF16>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan.smem);
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
  plan->ws_total = plan->warp_part + (size_t)plan->ctas * plan->warps * plan->rows * head_dim * 4;
  return true;
}

cudaError_t launch_paged_attn(const PagedAttnParams& p, const PagedAttnPlan& plan, int head_dim, int kv_bf16,
                              cudaStream_t st) {
  switch (head_dim) {
    case 64: return launch_d<64>(p, plan, kv_bf16, st);
    case 128: return launch_d<128>(p, plan, kv_bf16, st);
    default: return launch_d<256>(p, plan, kv_bf16, st);
  }
}

}  // namespace svq
