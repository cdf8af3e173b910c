// rope_cache.cu -- between the q|k|v linears and the attention: per-head RMS
// norms of the queries and keys, rotary positions, and the new keys and values
// written into their slots of the paged cache, in one pass.
//
//   n = x * gamma / sqrt(mean(x^2) + eps)            (per head, fp32; no gamma: n = x)
//   (u, w) -> factor * (u cos a - w sin a, u sin a + w cos a),  a = position * inv_freq[i]
// for the pairs (i, i + rot / 2) or (2i, 2i + 1) of the first rot entries, each
// result rounded once.
//
// The angle is what needs care: at position 10^6 an fp32 product is off by
// 0.03 rad.  It is formed in turns in fp64 (position * (inv_freq / 2 pi)), the
// whole turns are dropped there, and only the remaining half turn goes to fp32
// (sincospi): off by less than 5e-7 rad at the largest int32 position (the fp64 product
// 4e-7, its rounding to fp32 1e-7), by the 1e-7 alone near 0.
//
// One read of q|k|v and one write of q, k and v bounds long calls in principle,
// latency short ones.  A warp takes heads of one kind (queries, keys or values) of
// one row.  A head is spread over D / 8 lanes, each with two chunks of 4 entries
// that lie half the rotated part apart (or half the rest of the head), so both
// entries of a half-split pair are in one lane, as those of a neighbour pair are.
// The sines are formed once for the warp's heads, a share by each of the 256 / D
// lanes that need the same ones, and multiplied with gamma.  Nothing else is
// exchanged but the sum of squares, and warps do not wait for one another.
// (A CTA per row with the sines in shared memory: 16.5 us where this took 13.6,
// 2.1 us for one row against 1.5.)
//
// B200, in a CUDA graph: 2048 rows of 32 + 8 + 8 heads of 128, bf16, 12.9 us =
// 3.9 TB/s (copy rate 6.6); 777 rows of 14 + 2 + 2 heads of 64 3.2 us, one row 1.5 to 1.7 us.
// The 2048 rows are bound by latency on too few warps: 71 registers leave 28 warps an
// SM, so their 8192 warps run in two waves, each through its own chain of slot,
// position, sines and loads; schedulers issue in 57 % of the cycles, and HBM is at 59 %
// of the copy rate.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "attn_params.h"
#include "svq.h"

namespace svq {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <bool BF16>
__device__ __forceinline__ float to_f32(uint16_t v) {
  return BF16 ? __bfloat162float(__ushort_as_bfloat16(v)) : __half2float(__ushort_as_half(v));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {      // a in the low half
  if (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two fp32 operations in one instruction (each rounded as alone).
struct F2 {
  unsigned long long v;
  __device__ F2() {}
  __device__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ float2 get() const {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
  }
};
__device__ __forceinline__ F2 mul2(const F2& a, const F2& b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(const F2& a, const F2& b, const F2& c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Four entries of type XT (0 fp32, 1 fp16, 2 bf16) as they are stored.
template <int XT>
struct Chunk {
  uint32_t w[XT == 0 ? 4 : 2];
  static constexpr int kSize = XT == 0 ? 4 : 2;            // bytes of an entry
  __device__ void load(const void* p) {
    if constexpr (XT == 0) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    }
  }
  __device__ float get(int i) const {
    if constexpr (XT == 0) return __uint_as_float(w[i]);
    else return to_f32<XT == 2>((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
  }
};

// BF16: type of the cache and q_out; IL: neighbour pairs.  A step is 256 / D heads;
// a warp takes p.steps of them, U at a time with the next U on their way (U = 1:
// one step, and no loop).
template <int D, int XT, bool BF16, bool IL, int U>
__global__ void __launch_bounds__(kThreads) rope_cache_kernel(const __grid_constant__ RopeCacheParams p) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;      // lanes of a head, heads of a step
  const int lane = threadIdx.x & 31, n_kv = p.kv.n_heads;
  // the warp's row and slice of its heads; kind: 0 queries, 1 keys, 2 values
  const int wid = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int m = p.by_slices.div(wid), y = wid - m * (int)p.by_slices.d;
  if (m >= p.M) return;
  const int kind = y < p.q_slices ? 0 : y < p.q_slices + p.kv_slices ? 1 : 2;
  const int heads = kind == 0 ? p.n_q : n_kv;
  const int first = (y - (kind == 0 ? 0 : kind == 1 ? p.q_slices : p.q_slices + p.kv_slices)) * p.steps * kHeads;
  const uint16_t* gamma = kind == 0 ? p.q_gamma : kind == 1 ? p.k_gamma : nullptr;
  const int half = p.rot >> 1, i = lane % kLanes;
  // the lane's chunks: entries c0.. and c1.. of its heads
  const bool turned = i * 8 < p.rot;
  const int c0 = turned ? i * 4 : p.rot + (i * 4 - half);
  const int c1 = c0 + (turned ? half : (D - p.rot) >> 1);
  // its pairs e = 0..3: (c0 + e, c1 + e) if half split, else two neighbour pairs in each chunk
  auto pair_of = [&](int e) { return IL ? ((e & 2 ? c1 : c0) >> 1) + (e & 1) : c0 + e; };

  // weights and constants, before the previous kernel has finished
  constexpr int kShare = 4 / kHeads;                       // pairs whose sines this lane forms
  const int e0 = lane / kLanes * kShare;
  double freq[kShare];
  Chunk<1> g0, g1;
  if (kind < 2) {
#pragma unroll
    for (int e = 0; e < kShare; ++e)                       // turns per position
      freq[e] = turned ? __ldg(p.inv_freq + pair_of(e0 + e)) * 0.15915494309189533577 : 0.0;
  }
  if (gamma) {
    g0.load(gamma + c0);
    g1.load(gamma + c1);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int slot = p.slots[m], position = p.positions[m];
  const int h0 = first + lane / kLanes;                    // the lane's heads: h0, h0 + kHeads, ..
  // both read and write pointer walk from step to step
  const char* src = reinterpret_cast<const char*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                    (m * (kind == 0 ? p.ldq : kind == 1 ? p.ldk : p.ldv) + h0 * D + c0) * Chunk<XT>::kSize;
  const int src_c1 = (c1 - c0) * Chunk<XT>::kSize;
  const int my_steps = min(p.steps, (heads - h0 + kHeads - 1) / kHeads);     // with a head for this lane
  using Batch = Chunk<XT>[U][2];
  auto load = [&](Batch& x, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u < my_steps) {
        x[u][0].load(src);
        x[u][1].load(src + src_c1);
      }
      src += kHeads * D * Chunk<XT>::kSize;
    }
  };
  Batch xa, xb;
  load(xa, 0);
  if (slot < 0) return;                                    // a padding row
  const int page = slot / p.kv.page_size;
  if (page >= p.kv.n_pages) {
    if (lane == 0) *p.status = SVQ_ERR_INVALID_ARG;
    return;
  }
  const int64_t at = (int64_t)page * p.kv.page_stride + (int64_t)(slot - page * p.kv.page_size) * p.kv.token_stride;
  const int64_t head_step = kind == 0 ? D : p.kv.head_stride, step = kHeads * head_step;
  const int steps = min(p.steps, (heads - first + kHeads - 1) / kHeads);     // of the warp
  uint16_t* dst = (kind == 0 ? p.q_out + (int64_t)m * p.n_q * D : (kind == 1 ? p.kv.k : p.kv.v) + at) + h0 * head_step + c0;

  // (u, w) -> (u a - w b, u c + w d): the rotation times gamma, for the lane's pairs
  float ra[4], rb[4], rc[4], rd[4];
  if (kind < 2) {
    float cs[kShare], sn[kShare];
#pragma unroll
    for (int e = 0; e < kShare; ++e) {
      const double t = (double)position * freq[e];
      const float f = (float)(t - rint(t));                // turns in [-1/2, 1/2]
      sincospif(2.f * f, &sn[e], &cs[e]);
      cs[e] = turned ? cs[e] * p.factor : 1.f;
      sn[e] *= p.factor;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c = __shfl_sync(0xFFFFFFFFu, cs[e % kShare], i + e / kShare * kLanes);
      const float s = __shfl_sync(0xFFFFFFFFu, sn[e % kShare], i + e / kShare * kLanes);
      float gu = 1.f, gw = 1.f;
      if (gamma) {
        gu = IL ? (e & 2 ? g1 : g0).get((e & 1) * 2) : g0.get(e);
        gw = IL ? (e & 2 ? g1 : g0).get((e & 1) * 2 + 1) : g1.get(e);
      }
      ra[e] = gu * c;
      rb[e] = gw * s;
      rc[e] = gu * s;
      rd[e] = gw * c;
    }
  }

  auto compute = [&](const Batch& x, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= steps) break;
      float v[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[0][e] = x[u][0].get(e);
        v[1][e] = x[u][1].get(e);
      }
      if (kind < 2) {
        float inv = 1.f;
        if (gamma) {
          F2 s2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const F2 t(v[e >> 1][(e & 1) * 2], v[e >> 1][(e & 1) * 2 + 1]);
            s2 = fma2(t, t, s2);
          }
          float ss = s2.get().x + s2.get().y;
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
          inv = __frsqrt_rn(ss * (1.0f / D) + p.eps);
        }
        if (turned && !IL) {
          const F2 inv2(inv, inv);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const F2 a(v[0][e], v[0][e + 1]), b(v[1][e], v[1][e + 1]);
            const F2 a2 = mul2(fma2(b, F2(-rb[e], -rb[e + 1]), mul2(a, F2(ra[e], ra[e + 1]))), inv2);
            const F2 b2 = mul2(fma2(a, F2(rc[e], rc[e + 1]), mul2(b, F2(rd[e], rd[e + 1]))), inv2);
            v[0][e] = a2.get().x;
            v[0][e + 1] = a2.get().y;
            v[1][e] = b2.get().x;
            v[1][e + 1] = b2.get().y;
          }
        } else if (turned) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& a = v[e >> 1][(e & 1) * 2];
            float& b = v[e >> 1][(e & 1) * 2 + 1];
            const float t = fmaf(a, ra[e], -(b * rb[e])) * inv;
            b = fmaf(a, rc[e], b * rd[e]) * inv;
            a = t;
          }
        } else {                                           // gamma alone: an infinity beside it stays where it is
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            (IL ? v[e >> 1][(e & 1) * 2] : v[0][e]) *= ra[e] * inv;
            (IL ? v[e >> 1][(e & 1) * 2 + 1] : v[1][e]) *= rd[e] * inv;
          }
        }
      }
      if (s + u < my_steps) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(v[0][0], v[0][1]), pack2<BF16>(v[0][2], v[0][3]));
        *reinterpret_cast<uint2*>(dst + (c1 - c0)) = make_uint2(pack2<BF16>(v[1][0], v[1][1]), pack2<BF16>(v[1][2], v[1][3]));
      }
      dst += step;
    }
  };
  if constexpr (U == 1) {
    compute(xa, 0);
  } else {
#pragma unroll 1
    for (int s = 0; s < steps; s += 2 * U) {
      load(xb, s + U);
      compute(xa, s);
      load(xa, s + 2 * U);
      compute(xb, s + U);
    }
  }
}

template <int D, int XT, bool BF16>
cudaError_t launch_dx(RopeCacheParams p, int num_sms, cudaStream_t st) {
  // Few rows: a step per warp, so that latency is all there is.  Many: as many
  // steps as leave 48 warps for each SM (the sines of a row are formed anew in every
  // warp), a power of two up to sixteen so that slices are mostly whole turns of the
  // loop (2048 rows of 48 heads of 128: 12.9 us in eights, 14.2 us in sixes), and no
  // more than the longest kind of head has (which may be odd).  48 is measured, not the
  // warps that an SM holds: 28 takes those rows by sixteens, 17.5 us, though 64 rows of
  // 64 + 8 + 8 heads of 256 gain (4.1 -> 3.4 us); 96 takes them by fours, 12.8 us, and 365
  // rows of 20 + 4 + 4 heads of 256 lose (5.2 -> 6.0 us).
  constexpr int kHeads = 256 / D;
  const int q_steps = (p.n_q + kHeads - 1) / kHeads, kv_steps = (p.kv.n_heads + kHeads - 1) / kHeads;
  const long long all = (long long)p.M * (q_steps + 2 * kv_steps), warps = (long long)num_sms * 48;
  const long long steps = (all + warps - 1) / warps;
  p.steps = 1;
  while (p.steps < steps && p.steps < 16) p.steps *= 2;
  p.steps = std::min(p.steps, std::max(q_steps, kv_steps));
  p.q_slices = (q_steps + p.steps - 1) / p.steps;
  p.kv_slices = (kv_steps + p.steps - 1) / p.steps;
  const int slices = p.q_slices + 2 * p.kv_slices;
  p.by_slices = FastDiv(slices);
  const unsigned ctas = (unsigned)(((long long)p.M * slices + kWarps - 1) / kWarps);
  const auto kern = p.interleaved ? (p.steps == 1 ? rope_cache_kernel<D, XT, BF16, true, 1> : rope_cache_kernel<D, XT, BF16, true, 2>)
                                  : (p.steps == 1 ? rope_cache_kernel<D, XT, BF16, false, 1> : rope_cache_kernel<D, XT, BF16, false, 2>);
  return launch_dependent(kern, dim3(ctas), kThreads, 0, 1, st, p);
}

template <int D>
cudaError_t launch_d(const RopeCacheParams& p, int x_dtype, int kv_bf16, int num_sms, cudaStream_t st) {
  switch (x_dtype * 2 + kv_bf16) {
    case 0: return launch_dx<D, 0, false>(p, num_sms, st);
    case 1: return launch_dx<D, 0, true>(p, num_sms, st);
    case 2: return launch_dx<D, 1, false>(p, num_sms, st);
    case 3: return launch_dx<D, 1, true>(p, num_sms, st);
    case 4: return launch_dx<D, 2, false>(p, num_sms, st);
    default: return launch_dx<D, 2, true>(p, num_sms, st);
  }
}

}  // namespace

cudaError_t launch_rope_cache(const RopeCacheParams& p, int head_dim, int x_dtype, int kv_bf16, int num_sms,
                              cudaStream_t st) {
  switch (head_dim) {
    case 64: return launch_d<64>(p, x_dtype, kv_bf16, num_sms, st);
    case 128: return launch_d<128>(p, x_dtype, kv_bf16, num_sms, st);
    default: return launch_d<256>(p, x_dtype, kv_bf16, num_sms, st);
  }
}

}  // namespace svq
