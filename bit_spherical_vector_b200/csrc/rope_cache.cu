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
// (sincospi): off by 2e-7 at any position an int32 holds up to 10^8.
//
// One read of q|k|v and one write of q, k and v bounds it.  A warp takes U
// consecutive heads of one row, a lane D / 32 consecutive entries of each: rows
// are read and written whole, the norm is a butterfly, the partner of a
// half-split pair is one shuffle away (rot / 2 is a multiple of D / 32), and the
// sines of a row are formed once for the U heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (BF16)
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(a)) |
           ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(b)) << 16);
  return (uint32_t)__half_as_ushort(__float2half_rn(a)) | ((uint32_t)__half_as_ushort(__float2half_rn(b)) << 16);
}

// E consecutive 32-bit words (E = 1, 2 or 4 per vector access).
template <int N>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
      w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[N]) {
  if constexpr (N == 1) *reinterpret_cast<uint32_t*>(p) = w[0];
  else if constexpr (N == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// XT: type of q|k|v (0 fp32, 1 fp16, 2 bf16); BF16: type of the cache and q_out.
template <int D, int XT, bool BF16, int U>
__global__ void __launch_bounds__(kThreads) rope_cache_kernel(const __grid_constant__ RopeCacheParams p) {
  constexpr int E = D / 32;                        // entries per lane
  constexpr int XW = XT == 0 ? E : E / 2;          // 32-bit words per lane and head, read
  const int lane = threadIdx.x & 31;
  const int n_kv = p.kv.n_heads, roped = p.n_q + n_kv, heads = roped + n_kv;
  const int chunks = (heads + U - 1) / U;
  const long long wid = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int m = (int)(wid / chunks), h0 = (int)(wid - (long long)m * chunks) * U;
  const int j0 = lane * E;
  const int half = p.rot >> 1;
  const bool turned = j0 < p.rot;

  // weights and constants, before the previous kernel has finished
  double freq[E];
  if (turned && h0 < roped) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int j = j0 + e;
      const int i = p.interleaved ? (j >> 1) : (j < half ? j : j - half);
      freq[e] = __ldg(p.inv_freq + i) * 0.15915494309189533577;        // 1 / (2 pi): turns per position
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (m >= p.M) return;
  const int slot = p.slots[m];
  if (slot < 0) return;                            // a padding row: nothing of it is read or written
  const int page = slot / p.kv.page_size;
  if (page >= p.kv.n_pages) {
    if (lane == 0) *p.status = SVQ_ERR_INVALID_ARG;
    return;
  }

  uint32_t raw[U][XW];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u;
    if (h < heads) {
      const char* x = reinterpret_cast<const char*>(h < p.n_q ? p.q : h < roped ? p.k : p.v);
      const int64_t ld = h < p.n_q ? p.ldq : h < roped ? p.ldk : p.ldv;
      const int hh = h < p.n_q ? h : h < roped ? h - p.n_q : h - roped;
      load_words<XW>(x + (m * ld + (int64_t)hh * D + j0) * (XT == 0 ? 4 : 2), raw[u]);
    }
  }

  float c[E], s[E];                                // s carries the sign of the partner's term
#pragma unroll
  for (int e = 0; e < E; ++e) {
    c[e] = 1.f;
    s[e] = 0.f;
  }
  if (turned && h0 < roped) {
    const double pos = (double)p.positions[m];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int j = j0 + e;
      if (p.interleaved && (e & 1)) {              // the same angle as the entry before
        c[e] = c[e - 1];
        s[e] = -s[e - 1];
      } else {
        const double t = pos * freq[e];
        const float f = (float)(t - rint(t));      // turns in [-1/2, 1/2]
        float sn, cs;
        sincospif(2.f * f, &sn, &cs);
        c[e] = cs * p.factor;
        s[e] = (p.interleaved || j < half ? -sn : sn) * p.factor;
      }
    }
  }
  const int mate = j0 < half ? lane + half / E : lane - half / E;     // lane of the half-split partner
  const int64_t at = (int64_t)page * p.kv.page_stride + (int64_t)(slot - page * p.kv.page_size) * p.kv.token_stride;

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u;
    if (h >= heads) break;
    float v[E];
#pragma unroll
    for (int w = 0; w < XW; ++w) {
      if constexpr (XT == 0) {
        v[w] = __uint_as_float(raw[u][w]);
      } else {
        v[2 * w] = to_f32<XT == 2>((uint16_t)(raw[u][w] & 0xFFFFu));
        v[2 * w + 1] = to_f32<XT == 2>((uint16_t)(raw[u][w] >> 16));
      }
    }
    if (h < roped) {
      const uint16_t* gamma = h < p.n_q ? p.q_gamma : p.k_gamma;
      if (gamma) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(v[e], v[e], ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float inv = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
        uint32_t g[E / 2];
        load_words<E / 2>(gamma + j0, g);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = v[e] * inv * to_f32<false>((uint16_t)(g[e / 2] >> (16 * (e & 1))));
      }
      if (p.interleaved) {
        if (turned) {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float a = v[e], b = v[e + 1];
            v[e] = fmaf(b, s[e], a * c[e]);
            v[e + 1] = fmaf(a, s[e + 1], b * c[e + 1]);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float b = __shfl_sync(0xFFFFFFFFu, v[e], turned ? mate : lane);
          if (turned) v[e] = fmaf(b, s[e], v[e] * c[e]);
        }
      }
    }
    uint32_t o[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) o[e / 2] = pack2<BF16>(v[e], v[e + 1]);
    uint16_t* dst;
    if (h < p.n_q) dst = p.q_out + ((int64_t)m * p.n_q + h) * D;
    else if (h < roped) dst = p.kv.k + at + (int64_t)(h - p.n_q) * p.kv.head_stride;
    else dst = p.kv.v + at + (int64_t)(h - roped) * p.kv.head_stride;
    store_words<E / 2>(dst + j0, o);
  }
}

template <int D, int XT, bool BF16>
cudaError_t launch_dx(const RopeCacheParams& p, int num_sms, cudaStream_t st) {
  const long long heads = p.n_q + 2LL * p.kv.n_heads;
  // One head per warp while that leaves the SMs short of warps, else eight (the
  // sines of a row are then formed once for eight heads).
  if (p.M * heads <= (long long)num_sms * 64) {
    const long long warps = p.M * heads;
    return launch_dependent(rope_cache_kernel<D, XT, BF16, 1>, (unsigned)((warps + kWarps - 1) / kWarps), kThreads, 0,
                            1, st, p);
  }
  const long long warps = p.M * ((heads + 7) / 8);
  return launch_dependent(rope_cache_kernel<D, XT, BF16, 8>, (unsigned)((warps + kWarps - 1) / kWarps), kThreads, 0, 1,
                          st, p);
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
