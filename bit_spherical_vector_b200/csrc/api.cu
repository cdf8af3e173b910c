// api.cu -- the extern "C" boundary of libsvq (declared in include/svq.h):
// argument validation, workspace sizing, the device status word, dispatch to
// the kernel launchers.  No entry point allocates or frees memory.
#include <cuda_runtime.h>

#include <mutex>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "attn_params.h"
#include "layout.cuh"
#include "svq.h"
#include "gemm_params.h"
#include "moe_params.h"
#include "svq_internal.h"
#include "calib.h"

namespace {

__device__ int g_status_word;   // set by kernels whose bounded waits run out

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? SVQ_OK : SVQ_ERR_CUDA; }

int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

int check_matrix(const svq_matrix* W) {
  if (!W) return SVQ_ERR_INVALID_ARG;
  if (W->b_d < 1 || W->b_d > 10) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (W->K % 8 != 0 || !svq::layout_supported(W->N, W->K)) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (!W->packed || !W->codebook) return SVQ_ERR_INVALID_ARG;
  if (W->radius_lut) {
    // per-row radius table: at most 16 levels (b_r <= 4)
    if (10 - W->b_d > svq::kLutMaxBits) return SVQ_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(W->radius_lut, 2)) return SVQ_ERR_INVALID_ARG;
  } else {
    if (!W->radius_scale || !W->radius_offset) return SVQ_ERR_INVALID_ARG;
    if (!aligned(W->radius_scale, 2) || !aligned(W->radius_offset, 2)) return SVQ_ERR_INVALID_ARG;
  }
  if (!aligned(W->packed, 16) || !aligned(W->codebook, 16) || (W->perm && !aligned(W->perm, 4)))
    return SVQ_ERR_INVALID_ARG;
  return SVQ_OK;
}

svq::GemvMatDesc desc_of(const svq_matrix& W, const uint16_t* x, void* y) {
  svq::GemvMatDesc d;
  d.N = W.N; d.K = W.K; d.b_d = W.b_d;
  d.packed = W.packed; d.codebook = W.codebook; d.scale = W.radius_scale; d.offset = W.radius_offset;
  d.perm = W.perm; d.lut = W.radius_lut; d.x = x; d.y = y;
  return d;
}

int plan_group(const svq_matrix* mats, int n_mats, int M, svq::GemvPlan* plan,
               svq::GemvMatDesc* descs, const uint16_t* const* x, void* const* y) {
  if (!mats || n_mats < 1 || n_mats > svq::kGemvMaxMats) return SVQ_ERR_INVALID_ARG;
  if (M < 1 || M > 16) return SVQ_ERR_INVALID_ARG;
  for (int i = 0; i < n_mats; ++i) {
    const int st = check_matrix(&mats[i]);
    if (st != SVQ_OK) return st;
    // one grouped launch: every matrix with a radius table, or none
    if ((mats[i].radius_lut != nullptr) != (mats[0].radius_lut != nullptr)) return SVQ_ERR_INVALID_ARG;
    descs[i] = desc_of(mats[i], x ? x[i] : nullptr, y ? y[i] : nullptr);
  }
  const int sms = num_sms();
  if (sms <= 0) return SVQ_ERR_CUDA;
  // The plan depends only on the shapes, M and the SM count: keep the last few
  // (a decode loop calls the same layers over and over).
  struct Key {
    int sms, M, n, dims[3 * svq::kGemvMaxMats];
    bool operator==(const Key& o) const {
      if (sms != o.sms || M != o.M || n != o.n) return false;
      for (int i = 0; i < 3 * n; ++i)
        if (dims[i] != o.dims[i]) return false;
      return true;
    }
  };
  struct Entry {
    Key key;
    svq::GemvPlan plan;
    bool used;
  };
  static Entry cache[32];
  static int next_slot = 0;
  static std::mutex mu;
  Key key{};
  key.sms = sms; key.M = M; key.n = n_mats;
  for (int i = 0; i < n_mats; ++i) {
    // b_d, plus 16 when the matrix carries a radius table (its shared memory differs)
    key.dims[3 * i] = mats[i].N; key.dims[3 * i + 1] = mats[i].K;
    key.dims[3 * i + 2] = mats[i].b_d + (mats[i].radius_lut ? 16 : 0);
  }
  {
    std::lock_guard<std::mutex> lock(mu);
    for (const Entry& e : cache)
      if (e.used && e.key == key) {
        *plan = e.plan;
        return SVQ_OK;
      }
  }
  if (!svq::plan_gemv(descs, n_mats, M, sms, plan)) return SVQ_ERR_UNSUPPORTED_SHAPE;
  std::lock_guard<std::mutex> lock(mu);
  cache[next_slot] = Entry{key, *plan, true};
  next_slot = (next_slot + 1) % 32;
  return SVQ_OK;
}

// Scratch for svq_linear_gemv_noalloc: split-K partial sums and completion
// counters of one call.  Every GPU that loads the library holds these bytes
// until the process exits.
constexpr size_t kNoAllocScratchBytes = 1u << 20;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

// Device address of g_noalloc_scratch for the current device, looked up (and
// the scratch zero-filled on `stream`) on the first call per device.  In host
// code the array's name is only a host-side stand-in; kernels must be given the
// address returned by cudaGetSymbolAddress.
void* noalloc_scratch(cudaStream_t stream) {
  static void* ptr[64] = {nullptr};
  static std::mutex mu;                          // first calls from several host threads
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) return nullptr;
    // Completion counters must start at zero; every completed call leaves them zero.
    if (cudaMemsetAsync(p, 0, kNoAllocScratchBytes, stream) != cudaSuccess) return nullptr;
    ptr[dev] = p;
  }
  return ptr[dev];
}

int* status_word() {
  static int* ptr[64] = {nullptr};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess) return nullptr;
    ptr[dev] = static_cast<int*>(p);
  }
  return ptr[dev];
}

// A paged cache as the kernels take it: heads of 64, 128 or 256 entries, whole
// 16-byte chunks everywhere, and a slot number (page * page_size + token) that
// fits 32 bits.
int check_cache(const svq_kv_cache* c) {
  if (!c || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return SVQ_ERR_INVALID_ARG;
  if (c->dtype != SVQ_F16 && c->dtype != SVQ_BF16) return SVQ_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->page_size < 1 || c->n_heads < 1 || c->reserved != 0) return SVQ_ERR_INVALID_ARG;
  if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0 || c->page_stride % 8 || c->token_stride % 8 ||
      c->head_stride % 8)
    return SVQ_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if ((int64_t)c->n_pages * c->page_size > INT32_MAX || c->n_heads > 1024) return SVQ_ERR_UNSUPPORTED_SHAPE;
  return SVQ_OK;
}

svq::KvView view_of(const svq_kv_cache& c) {
  svq::KvView v;
  v.k = static_cast<uint16_t*>(c.k); v.v = static_cast<uint16_t*>(c.v);
  v.page_stride = c.page_stride; v.token_stride = c.token_stride; v.head_stride = c.head_stride;
  v.n_pages = c.n_pages; v.page_size = c.page_size; v.n_heads = c.n_heads;
  return v;
}

}  // namespace

extern "C" {

const char* svq_status_string(int status) {
  switch (status) {
    case SVQ_OK: return "ok";
    case SVQ_ERR_INVALID_ARG: return "invalid argument (null or misaligned pointer, bad enum or batch size)";
    case SVQ_ERR_UNSUPPORTED_SHAPE:
      return "unsupported shape (needs K % 8 == 0, 1 <= b_d <= 10; radius tables b_r <= 4; MoE K % 128 == 0 and N % 4 == 0)";
    case SVQ_ERR_WORKSPACE: return "workspace missing or too small";
    case SVQ_ERR_CUDA: return "CUDA runtime error";
    case SVQ_ERR_TIMEOUT: return "a kernel's bounded wait timed out";
    default: return "unknown status";
  }
}

int svq_version(void) { return 100; }

size_t svq_packed_bytes(int N, int K) {
  if (!svq::layout_supported(N, K)) return 0;
  return svq::packed_bytes(N, K);
}

size_t svq_canonical_bytes(int N, int K) {
  if (N <= 0 || K <= 0 || K % 8) return 0;
  return (size_t)N * (((size_t)(K / 8) * 18 + 7) / 8);
}

int svq_repack(const uint8_t* canonical, int N, int K, int b_d, void* packed_out, svq_stream_t stream) {
  if (!canonical || !packed_out) return SVQ_ERR_INVALID_ARG;
  if (b_d < 1 || b_d > 10 || !svq::layout_supported(N, K)) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(packed_out, 16)) return SVQ_ERR_INVALID_ARG;
  return cuda_status(svq::launch_repack(canonical, N, K, b_d, packed_out, (cudaStream_t)stream));
}

int svq_unpack_fields(const void* packed, int N, int K, int b_d, uint8_t* signs, uint16_t* idx,
                      uint16_t* code, svq_stream_t stream) {
  if (!packed || !signs || !idx || !code) return SVQ_ERR_INVALID_ARG;
  if (b_d < 1 || b_d > 10 || !svq::layout_supported(N, K)) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(packed, 16) || !aligned(idx, 2) || !aligned(code, 2)) return SVQ_ERR_INVALID_ARG;
  return cuda_status(svq::launch_unpack(packed, N, K, b_d, signs, idx, code, (cudaStream_t)stream));
}

int svq_dequantize(const svq_matrix* W, int out_dtype, void* w_out, svq_stream_t stream) {
  const int st = check_matrix(W);
  if (st != SVQ_OK) return st;
  if (!w_out || !aligned(w_out, 16)) return SVQ_ERR_INVALID_ARG;
  if (out_dtype != SVQ_F16 && out_dtype != SVQ_BF16) return SVQ_ERR_INVALID_ARG;
  return cuda_status(svq::launch_dequant(W->packed, W->N, W->K, W->b_d, W->codebook, W->radius_scale,
                                         W->radius_offset, W->radius_lut, out_dtype == SVQ_BF16, (uint16_t*)w_out,
                                         (cudaStream_t)stream));
}

int svq_linear_gemv_batched_workspace_size(const svq_matrix* mats, int n_mats, int M, size_t* bytes) {
  if (!bytes) return SVQ_ERR_INVALID_ARG;
  svq::GemvPlan plan;
  svq::GemvMatDesc descs[svq::kGemvMaxMats];
  const int st = plan_group(mats, n_mats, M, &plan, descs, nullptr, nullptr);
  if (st != SVQ_OK) return st;
  *bytes = plan.ws_total;
  return SVQ_OK;
}

int svq_linear_gemv_workspace_size(const svq_matrix* W, int M, size_t* bytes) {
  return svq_linear_gemv_batched_workspace_size(W, 1, M, bytes);
}

int svq_workspace_init(void* workspace, size_t bytes, svq_stream_t stream) {
  if (bytes == 0) return SVQ_OK;
  if (!workspace) return SVQ_ERR_INVALID_ARG;
  return cuda_status(cudaMemsetAsync(workspace, 0, bytes, (cudaStream_t)stream));
}

// Checks and plans a grouped GEMV call (nothing is enqueued).
static int prepare_batched(const svq_matrix* mats, int n_mats, const uint16_t* const* x, int M, void* const* y,
                           int y_dtype, void* workspace, size_t workspace_bytes, svq::GemvPlan* plan,
                           svq::GemvMatDesc* descs) {
  if (!x || !y) return SVQ_ERR_INVALID_ARG;
  if (y_dtype != SVQ_F16 && y_dtype != SVQ_F32) return SVQ_ERR_INVALID_ARG;
  if (n_mats < 1 || n_mats > svq::kGemvMaxMats) return SVQ_ERR_INVALID_ARG;
  for (int i = 0; i < n_mats; ++i) {
    if (!x[i] || !y[i]) return SVQ_ERR_INVALID_ARG;
    if (!aligned(x[i], 2) || !aligned(y[i], y_dtype == SVQ_F32 ? 4 : 2)) return SVQ_ERR_INVALID_ARG;
  }
  const int st = plan_group(mats, n_mats, M, plan, descs, x, y);
  if (st != SVQ_OK) return st;
  if (plan->ws_total > 0 && (!workspace || workspace_bytes < plan->ws_total || !aligned(workspace, 256)))
    return SVQ_ERR_WORKSPACE;
  return SVQ_OK;
}

int svq_linear_gemv_batched(const svq_matrix* mats, int n_mats, const uint16_t* const* x, int M,
                            void* const* y, int y_dtype, void* workspace, size_t workspace_bytes,
                            svq_stream_t stream) {
  svq::GemvPlan plan;
  svq::GemvMatDesc descs[svq::kGemvMaxMats];
  const int st = prepare_batched(mats, n_mats, x, M, y, y_dtype, workspace, workspace_bytes, &plan, descs);
  if (st != SVQ_OK) return st;
  return cuda_status(svq::launch_gemv(descs, plan, y_dtype == SVQ_F32, workspace, (cudaStream_t)stream));
}

int svq_linear_gemv_batched_host(const svq_matrix* mats, int n_mats, const uint16_t* x_host, uint16_t* x_dev,
                                 int M, void* y_host, void* y_dev, int y_dtype, void* workspace,
                                 size_t workspace_bytes, svq_stream_t stream) {
  if (!mats || !x_host || !x_dev || !y_host || !y_dev) return SVQ_ERR_INVALID_ARG;
  if (n_mats < 1 || n_mats > svq::kGemvMaxMats || M < 1) return SVQ_ERR_INVALID_ARG;
  if (y_dtype != SVQ_F16 && y_dtype != SVQ_F32) return SVQ_ERR_INVALID_ARG;
  const size_t ysz = y_dtype == SVQ_F32 ? 4 : 2;
  const uint16_t* xs[svq::kGemvMaxMats];
  void* ys[svq::kGemvMaxMats];
  size_t xo = 0, yo = 0;                             // elements of x, bytes of y
  for (int i = 0; i < n_mats; ++i) {
    if (mats[i].N < 1 || mats[i].K < 1) return SVQ_ERR_INVALID_ARG;
    xs[i] = x_dev + xo;
    ys[i] = reinterpret_cast<char*>(y_dev) + yo;
    xo += (size_t)M * mats[i].K;
    yo += (size_t)M * mats[i].N * ysz;
  }
  svq::GemvPlan plan;
  svq::GemvMatDesc descs[svq::kGemvMaxMats];
  // every check passes before anything is enqueued
  const int st = prepare_batched(mats, n_mats, xs, M, ys, y_dtype, workspace, workspace_bytes, &plan, descs);
  if (st != SVQ_OK) return st;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaMemcpyAsync(x_dev, x_host, xo * 2, cudaMemcpyHostToDevice, s);
  if (e != cudaSuccess) return cuda_status(e);
  e = svq::launch_gemv(descs, plan, y_dtype == SVQ_F32, workspace, s);
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(cudaMemcpyAsync(y_host, y_dev, yo, cudaMemcpyDeviceToHost, s));
}

int svq_linear_gemv(const svq_matrix* W, const uint16_t* x, int M, void* y, int y_dtype, void* workspace,
                    size_t workspace_bytes, svq_stream_t stream) {
  void* yy[1] = {y};
  const uint16_t* xx[1] = {x};
  if (!x || !y) return SVQ_ERR_INVALID_ARG;
  return svq_linear_gemv_batched(W, 1, xx, M, yy, y_dtype, workspace, workspace_bytes, stream);
}

int svq_linear_gemv_noalloc(const svq_matrix* W, const uint16_t* x, int M, void* y, int y_dtype,
                            svq_stream_t stream) {
  if (!x || !y) return SVQ_ERR_INVALID_ARG;
  if (y_dtype != SVQ_F16 && y_dtype != SVQ_F32) return SVQ_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(y, y_dtype == SVQ_F32 ? 4 : 2)) return SVQ_ERR_INVALID_ARG;
  svq::GemvPlan plan;
  svq::GemvMatDesc descs[1];
  const uint16_t* xx[1] = {x};
  void* yy[1] = {y};
  const int st = plan_group(W, 1, M, &plan, descs, xx, yy);
  if (st != SVQ_OK) return st;
  if (plan.ws_total > kNoAllocScratchBytes) return SVQ_ERR_WORKSPACE;
  void* scratch = noalloc_scratch((cudaStream_t)stream);
  if (!scratch) return SVQ_ERR_CUDA;
  return cuda_status(svq::launch_gemv(descs, plan, y_dtype == SVQ_F32, scratch, (cudaStream_t)stream));
}

int svq_linear_gemm_workspace_size(const svq_matrix* W, int M, size_t* bytes) {
  if (!bytes) return SVQ_ERR_INVALID_ARG;
  const int st = check_matrix(W);
  if (st != SVQ_OK) return st;
  if (M < 1) return SVQ_ERR_INVALID_ARG;
  const int sms = num_sms();
  if (sms <= 0) return SVQ_ERR_CUDA;
  *bytes = svq::plan_gemm(W->N, W->K, M, sms).ws_bytes;
  return SVQ_OK;
}

int svq_linear_gemm(const svq_matrix* W, const uint16_t* x, int x_dtype, int M, void* y, int y_dtype,
                    void* workspace, size_t workspace_bytes, svq_stream_t stream) {
  const int st = check_matrix(W);
  if (st != SVQ_OK) return st;
  if (!x || !y || M < 1) return SVQ_ERR_INVALID_ARG;
  if (x_dtype != SVQ_BF16 && x_dtype != SVQ_F16) return SVQ_ERR_INVALID_ARG;
  if (y_dtype != SVQ_BF16 && y_dtype != SVQ_F32) return SVQ_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(y, 16)) return SVQ_ERR_INVALID_ARG;
  if (!W->perm && !aligned(x, 16)) return SVQ_ERR_INVALID_ARG;     // read directly by TMA
  const int sms = num_sms();
  if (sms <= 0) return SVQ_ERR_CUDA;
  const svq::GemmPlan g = svq::plan_gemm(W->N, W->K, M, sms);
  if (!workspace || workspace_bytes < g.ws_bytes || !aligned(workspace, 256)) return SVQ_ERR_WORKSPACE;
  int* status = status_word();
  if (!status) return SVQ_ERR_CUDA;
  svq::GemmMatDesc d;
  d.N = W->N; d.K = W->K; d.b_d = W->b_d; d.M = M;
  d.packed = W->packed; d.codebook = W->codebook; d.scale = W->radius_scale; d.offset = W->radius_offset;
  d.lut = W->radius_lut;
  d.perm = W->perm; d.x = x; d.x_bf16 = x_dtype == SVQ_BF16; d.y = y; d.y_f32 = y_dtype == SVQ_F32;
  return cuda_status(svq::launch_gemm(d, g, workspace, status, (cudaStream_t)stream));
}

int svq_moe_grouped_gemv_workspace_size(int n_mats, int n_items, int N, int accumulate, size_t* bytes) {
  if (!bytes || n_mats < 1 || n_items < 0 || N < 1) return SVQ_ERR_INVALID_ARG;
  *bytes = svq::moe_workspace_layout(n_mats, n_items, N, accumulate ? 1 : 0).total;
  return SVQ_OK;
}

int svq_moe_grouped_gemv(const svq_matrix* mats, int n_mats, int N, int K, int max_b_d, const svq_group_item* items,
                         int n_items, int max_items_per_matrix, const void* x, int x_mode, int n_x_rows, float* y,
                         int n_out_rows, int accumulate, void* workspace, size_t workspace_bytes,
                         svq_stream_t stream) {
  if (!mats || !items || !x || !y || n_mats < 1 || n_items < 1 || n_out_rows < 1 || n_x_rows < 1)
    return SVQ_ERR_INVALID_ARG;
  // the grouped MoE kernel takes only shapes that need no padding
  if (max_b_d < 1 || max_b_d > 10 || !svq::layout_supported(N, K) || N % 4 != 0 || K % 128 != 0)
    return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (n_mats > 16384 || max_items_per_matrix < 1) return SVQ_ERR_INVALID_ARG;
  if (x_mode != SVQ_X_F16 && x_mode != SVQ_X_SWIGLU_F32) return SVQ_ERR_INVALID_ARG;
  if (!aligned(mats, 8) || !aligned(items, 4) || !aligned(y, 4) || !aligned(x, x_mode == SVQ_X_F16 ? 2 : 4))
    return SVQ_ERR_INVALID_ARG;
  const int mt = max_items_per_matrix == 1 ? 1 : (max_items_per_matrix == 2 ? 2 : 4);
  if (svq::moe_smem_bytes(max_b_d, K, mt, n_mats, n_items) > 220 * 1024) return SVQ_ERR_UNSUPPORTED_SHAPE;
  const svq::MoeWorkspace w = svq::moe_workspace_layout(n_mats, n_items, N, accumulate ? 1 : 0);
  if (!workspace || workspace_bytes < w.total || !aligned(workspace, 256)) return SVQ_ERR_WORKSPACE;
  const int sms = num_sms();
  int* status = status_word();
  if (sms <= 0 || !status) return SVQ_ERR_CUDA;
  char* b = reinterpret_cast<char*>(workspace);
  svq::MoeKParams p;
  p.mats = mats; p.n_mats = n_mats; p.N = N; p.K = K; p.max_b_d = max_b_d;
  p.items = items; p.n_items = n_items; p.x = x; p.x_mode = x_mode; p.n_x_rows = n_x_rows; p.y = y;
  p.n_out_rows = n_out_rows; p.accumulate = accumulate ? 1 : 0;
  p.offsets = reinterpret_cast<int*>(b + w.offsets);
  p.cursor = reinterpret_cast<int*>(b + w.cursor);
  p.sorted = reinterpret_cast<int*>(b + w.sorted);
  p.active = reinterpret_cast<int*>(b + w.active);
  p.n_active = reinterpret_cast<int*>(b + w.n_active);
  p.costpre = reinterpret_cast<int*>(b + w.costpre);
  p.mt = mt;
  p.local_route = svq::moe_local_route(n_mats, n_items) ? 1 : 0;
  p.item_out = accumulate ? reinterpret_cast<float*>(b + w.item_out) : nullptr;
  p.status = status;
  return cuda_status(svq::launch_moe(p, mt, n_out_rows, sms, (cudaStream_t)stream));
}

int svq_rmsnorm_permute(const uint16_t* h, int h_dtype, const uint16_t* gamma, float eps, int M, int K,
                        const int32_t* const* perms, uint16_t* const* outs, int n_out, svq_stream_t stream) {
  if (h_dtype != SVQ_F16 && h_dtype != SVQ_BF16) return SVQ_ERR_INVALID_ARG;
  if (n_out < 1 || n_out > svq::kMaxProducerOuts || !outs) return SVQ_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return SVQ_ERR_INVALID_ARG;   // rejects NaN and infinity
  if (M < 0 || M > 65535) return SVQ_ERR_INVALID_ARG;
  if (K < 8 || K % 8 != 0) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return SVQ_OK;                     // nothing to read or write
  if (!h || !gamma || !aligned(h, 16) || !aligned(gamma, 16)) return SVQ_ERR_INVALID_ARG;
  for (int g = 0; g < n_out; ++g) {
    if (!outs[g] || !aligned(outs[g], 16)) return SVQ_ERR_INVALID_ARG;
    if (perms && perms[g] && !aligned(perms[g], 4)) return SVQ_ERR_INVALID_ARG;
  }
  return cuda_status(svq::launch_rmsnorm_permute(h, h_dtype == SVQ_BF16, gamma, eps, M, K, perms, outs, n_out,
                                                 (cudaStream_t)stream));
}

int svq_swiglu_permute(const float* gate, const float* up, int M, int I, const int32_t* perm, uint16_t* x,
                       svq_stream_t stream) {
  if (M < 0 || M > 65535) return SVQ_ERR_INVALID_ARG;
  if (I < 8 || I % 8 != 0) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return SVQ_OK;                     // nothing to read or write
  if (!gate || !up || !x || !aligned(gate, 16) || !aligned(up, 16) || !aligned(x, 16)) return SVQ_ERR_INVALID_ARG;
  if (perm && !aligned(perm, 4)) return SVQ_ERR_INVALID_ARG;
  return cuda_status(svq::launch_swiglu_permute(gate, up, M, I, perm, x, (cudaStream_t)stream));
}

int svq_rope_frequencies(int rot_dim, double base, int scaling, double scale, int trained_len, double* inv_freq,
                         float* factor) {
  if (!inv_freq || !factor) return SVQ_ERR_INVALID_ARG;
  if (rot_dim < 16 || rot_dim > 256 || rot_dim % 16 != 0) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (!(base > 1.0) || base > 1e300) return SVQ_ERR_INVALID_ARG;
  if (scaling < SVQ_ROPE_PLAIN || scaling > SVQ_ROPE_YARN) return SVQ_ERR_INVALID_ARG;
  if (scaling != SVQ_ROPE_PLAIN && (!(scale >= 1.0) || scale > 1e6)) return SVQ_ERR_INVALID_ARG;
  if (scaling == SVQ_ROPE_YARN && trained_len < 1) return SVQ_ERR_INVALID_ARG;
  const int half = rot_dim / 2;
  *factor = 1.0f;
  if (scaling == SVQ_ROPE_NTK) base *= std::pow(scale, (double)rot_dim / (rot_dim - 2));
  for (int i = 0; i < half; ++i) inv_freq[i] = std::pow(base, -2.0 * i / rot_dim);
  if (scaling == SVQ_ROPE_LINEAR)
    for (int i = 0; i < half; ++i) inv_freq[i] /= scale;
  if (scaling == SVQ_ROPE_YARN) {
    // pair index whose frequency makes the given number of turns over the trained length
    const double two_pi = 6.283185307179586476925;
    const auto at = [&](double turns) {
      return rot_dim * std::log(trained_len / (turns * two_pi)) / (2.0 * std::log(base));
    };
    const double lo = std::fmax(std::floor(at(32.0)), 0.0), hi = std::fmin(std::ceil(at(1.0)), rot_dim - 1.0);
    for (int i = 0; i < half; ++i) {
      // (the ramp's ends lie inside the head, so over a few positions its upper one would be below pair 0)
      const double ramp = i >= at(1.0) ? 1.0 : std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      inv_freq[i] = inv_freq[i] / scale * ramp + inv_freq[i] * (1.0 - ramp);
    }
    *factor = (float)(0.1 * std::log(scale) + 1.0);
  }
  return SVQ_OK;
}

int svq_kv_assign(const int32_t* lens, const int32_t* n_new, int n_seqs, int page_size, int32_t* block_table,
                  int max_pages, int32_t* free_pages, int n_pages, const int32_t* n_free, int32_t* lens_out,
                  int32_t* n_free_out, int32_t* cu_rows, int32_t* positions, int32_t* slots, int max_rows,
                  svq_stream_t stream) {
  if (n_seqs < 1 || page_size < 1 || max_pages < 1 || n_pages < 1 || max_rows < 0) return SVQ_ERR_INVALID_ARG;
  if (n_seqs > svq::kMaxSeqs || (int64_t)n_seqs * max_pages > INT32_MAX || (int64_t)max_pages * page_size > INT32_MAX ||
      (int64_t)n_pages * page_size > INT32_MAX || max_rows > (1 << 30))
    return SVQ_ERR_UNSUPPORTED_SHAPE;
  const void* ptrs[] = {lens, n_new, block_table, free_pages, n_free, lens_out, n_free_out, cu_rows};
  for (const void* q : ptrs)
    if (!q || !aligned(q, 4)) return SVQ_ERR_INVALID_ARG;
  if (max_rows > 0 && (!positions || !slots || !aligned(positions, 4) || !aligned(slots, 4)))
    return SVQ_ERR_INVALID_ARG;
  int* status = status_word();
  if (!status) return SVQ_ERR_CUDA;
  svq::KvAssignParams p;
  p.lens = lens; p.n_new = n_new; p.table = block_table; p.free_pages = free_pages; p.n_free = n_free;
  p.lens_out = lens_out; p.n_free_out = n_free_out; p.cu_rows = cu_rows; p.positions = positions; p.slots = slots;
  p.status = status;
  p.by_page = svq::FastDiv(page_size);
  p.n_seqs = n_seqs; p.width = max_pages; p.page_size = page_size; p.n_pages = n_pages; p.max_rows = max_rows;
  return cuda_status(svq::launch_kv_assign(p, (cudaStream_t)stream));
}

int svq_qk_norm_rope_cache(const void* q, const void* k, const void* v, int x_dtype, int64_t ldq, int64_t ldk,
                           int64_t ldv, int M, int n_q_heads, const uint16_t* q_gamma, const uint16_t* k_gamma,
                           float eps, const svq_rope* rope, const int32_t* positions, const int32_t* slots,
                           const svq_kv_cache* cache, uint16_t* q_out, svq_stream_t stream) {
  const int st = check_cache(cache);
  if (st != SVQ_OK) return st;
  if (x_dtype != SVQ_F32 && x_dtype != SVQ_F16 && x_dtype != SVQ_BF16) return SVQ_ERR_INVALID_ARG;
  if (!rope || !rope->inv_freq || !aligned(rope->inv_freq, 8) || rope->reserved != 0) return SVQ_ERR_INVALID_ARG;
  if (rope->interleaved != 0 && rope->interleaved != 1) return SVQ_ERR_INVALID_ARG;
  if (!(rope->factor >= -3.0e38f && rope->factor <= 3.0e38f)) return SVQ_ERR_INVALID_ARG;
  if (rope->rot_dim < 16 || rope->rot_dim > cache->head_dim || rope->rot_dim % 16 != 0)
    return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return SVQ_ERR_INVALID_ARG;
  if (M < 0 || M > (1 << 20) || n_q_heads < 1 || n_q_heads > 1024) return SVQ_ERR_INVALID_ARG;
  if (M == 0) return SVQ_OK;                     // nothing to read or write
  const int64_t q_row = (int64_t)n_q_heads * cache->head_dim, kv_row = (int64_t)cache->n_heads * cache->head_dim;
  if (ldq < q_row || ldk < kv_row || ldv < kv_row || ldq % 8 || ldk % 8 || ldv % 8) return SVQ_ERR_INVALID_ARG;
  if (!q || !k || !v || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !q_out || !aligned(q_out, 16))
    return SVQ_ERR_INVALID_ARG;
  if ((q_gamma && !aligned(q_gamma, 16)) || (k_gamma && !aligned(k_gamma, 16))) return SVQ_ERR_INVALID_ARG;
  if (!positions || !slots || !aligned(positions, 4) || !aligned(slots, 4)) return SVQ_ERR_INVALID_ARG;
  const int sms = num_sms();
  int* status = status_word();
  if (sms <= 0 || !status) return SVQ_ERR_CUDA;
  svq::RopeCacheParams p;
  p.q = q; p.k = k; p.v = v; p.ldq = ldq; p.ldk = ldk; p.ldv = ldv;
  p.q_gamma = q_gamma; p.k_gamma = k_gamma; p.inv_freq = rope->inv_freq; p.positions = positions; p.slots = slots;
  p.q_out = q_out; p.status = status; p.kv = view_of(*cache); p.eps = eps; p.factor = rope->factor;
  p.M = M; p.n_q = n_q_heads; p.rot = rope->rot_dim; p.interleaved = rope->interleaved;
  return cuda_status(svq::launch_rope_cache(p, cache->head_dim, x_dtype == SVQ_F32 ? 0 : x_dtype == SVQ_F16 ? 1 : 2,
                                            cache->dtype == SVQ_BF16, sms, (cudaStream_t)stream));
}

int svq_paged_attention_workspace_size(const svq_kv_cache* cache, int n_q_heads, size_t* bytes) {
  if (!bytes) return SVQ_ERR_INVALID_ARG;
  const int st = check_cache(cache);
  if (st != SVQ_OK) return st;
  const int sms = num_sms();
  if (sms <= 0) return SVQ_ERR_CUDA;
  svq::PagedAttnPlan plan;
  if (!svq::plan_paged_attn(n_q_heads, cache->n_heads, cache->head_dim, 1, sms, &plan))
    return SVQ_ERR_UNSUPPORTED_SHAPE;
  *bytes = plan.ws_total;
  return SVQ_OK;
}

int svq_paged_attention(const uint16_t* q, int n_rows, int n_q_heads, const svq_kv_cache* cache, const int32_t* lens,
                        const int32_t* cu_rows, int n_seqs, const int32_t* block_table, int max_pages, float scale,
                        const int32_t* order, void* out, int out_dtype, float* lse, void* workspace,
                        size_t workspace_bytes, svq_stream_t stream) {
  const int st = check_cache(cache);
  if (st != SVQ_OK) return st;
  if (out_dtype != SVQ_F16 && out_dtype != SVQ_BF16) return SVQ_ERR_INVALID_ARG;
  const float scale_log2 = scale * 1.4426950408889634f;    // the kernel's scores are in units of log2
  if (!(scale_log2 >= -3.0e38f && scale_log2 <= 3.0e38f)) return SVQ_ERR_INVALID_ARG;      // rejects NaN and infinities
  if (n_seqs < 0 || n_rows < 0 || max_pages < 1) return SVQ_ERR_INVALID_ARG;
  // the tiles of all requests are counted in 32 bits
  if (n_seqs > svq::kMaxSeqs || n_rows > (1 << 26) || (int64_t)max_pages * cache->page_size > INT32_MAX - 16 ||
      n_seqs * ((int64_t)max_pages * cache->page_size / 16 + 1) > INT32_MAX || n_q_heads > 1024)
    return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (order && (int64_t)n_q_heads * cache->head_dim > svq::kMaxOrdered) return SVQ_ERR_UNSUPPORTED_SHAPE;
  svq::PagedAttnPlan plan;
  const int sms = num_sms();
  if (n_q_heads < 1 || n_q_heads % cache->n_heads != 0) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (n_seqs == 0 || n_rows == 0) return SVQ_OK; // nothing to read or write
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !lens || !aligned(lens, 4) || !block_table ||
      !aligned(block_table, 4))
    return SVQ_ERR_INVALID_ARG;
  if ((cu_rows && !aligned(cu_rows, 4)) || (order && !aligned(order, 16)) || (lse && !aligned(lse, 4)))
    return SVQ_ERR_INVALID_ARG;
  if (sms <= 0) return SVQ_ERR_CUDA;
  if (!svq::plan_paged_attn(n_q_heads, cache->n_heads, cache->head_dim, n_seqs, sms, &plan))
    return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || workspace_bytes < plan.ws_total || !aligned(workspace, 256)) return SVQ_ERR_WORKSPACE;
  int* status = status_word();
  if (!status) return SVQ_ERR_CUDA;
  char* w = static_cast<char*>(workspace);
  svq::PagedAttnParams p;
  p.q = q; p.lens = lens; p.cu_rows = cu_rows; p.table = block_table; p.order = order;
  p.out = static_cast<uint16_t*>(out); p.lse = lse; p.status = status;
  p.counters = reinterpret_cast<unsigned*>(w);
  p.cta_part = reinterpret_cast<float*>(w + plan.cta_part);
  p.warp_part = reinterpret_cast<float*>(w + plan.warp_part);
  p.kv = view_of(*cache);
  p.scale_log2 = scale_log2;
  p.n_seqs = n_seqs; p.width = max_pages; p.n_q = n_q_heads; p.n_rows = n_rows;
  p.group = n_q_heads / cache->n_heads;
  p.row_tiles = (p.group + plan.rows - 1) / plan.rows;
  p.by_heads = svq::FastDiv(cache->n_heads * p.row_tiles);
  p.by_row_tiles = svq::FastDiv(p.row_tiles);
  p.by_page = svq::FastDiv(cache->page_size);
  p.out_bf16 = out_dtype == SVQ_BF16;
  return cuda_status(svq::launch_paged_attn(p, plan, cache->head_dim, cache->dtype == SVQ_BF16, (cudaStream_t)stream));
}

int svq_esg(const float* x_cal, int T, int K, double gamma, double* energy, int32_t* perm, float* weights,
            svq_stream_t stream) {
  if (T < 1 || K < 8 || K % 8 != 0) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (!x_cal || !energy || !perm) return SVQ_ERR_INVALID_ARG;
  if (!aligned(x_cal, 4) || !aligned(energy, 8) || !aligned(perm, 4) || (weights && !aligned(weights, 4)))
    return SVQ_ERR_INVALID_ARG;
  if (!(gamma == gamma)) return SVQ_ERR_INVALID_ARG;               // NaN exponent
  return cuda_status(svq::launch_esg(x_cal, T, K, gamma, energy, perm, weights, (cudaStream_t)stream));
}

int svq_radius_grid(const float* W, int N, int K, const int32_t* perm, int b_d, uint16_t* scale, uint16_t* offset,
                    svq_stream_t stream) {
  if (N < 1 || K < 8 || K % 8 != 0 || b_d < 1 || b_d > 10) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (!W || !scale || !offset) return SVQ_ERR_INVALID_ARG;
  if (!aligned(W, 4) || !aligned(scale, 2) || !aligned(offset, 2) || (perm && !aligned(perm, 4)))
    return SVQ_ERR_INVALID_ARG;
  return cuda_status(svq::launch_radius_grid(W, N, K, perm, b_d, scale, offset, (cudaStream_t)stream));
}

int svq_encode(const float* W, int N, int K, int b_d, const int32_t* perm, const float* weights,
               const uint16_t* codebook, const uint16_t* scale, const uint16_t* offset, const uint16_t* radius_lut,
               uint8_t* canonical, double* row_err, svq_stream_t stream) {
  if (N < 1 || K < 8 || K % 8 != 0 || b_d < 1 || b_d > 10) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (radius_lut && 10 - b_d > svq::kLutMaxBits) return SVQ_ERR_UNSUPPORTED_SHAPE;
  if (!W || !codebook || !canonical || (!radius_lut && (!scale || !offset))) return SVQ_ERR_INVALID_ARG;
  if (!aligned(W, 4) || !aligned(codebook, 2) || (scale && !aligned(scale, 2)) || (offset && !aligned(offset, 2)) ||
      (radius_lut && !aligned(radius_lut, 2)) || (perm && !aligned(perm, 4)) || (weights && !aligned(weights, 4)) ||
      (row_err && !aligned(row_err, 8)))
    return SVQ_ERR_INVALID_ARG;
  return cuda_status(svq::launch_encode(W, N, K, b_d, perm, weights, codebook, scale, offset, radius_lut, canonical,
                                        row_err, (cudaStream_t)stream));
}

int svq_abs_select(const double* row_err, int n_cand, int N, double* totals, int32_t* best, svq_stream_t stream) {
  if (n_cand < 1 || n_cand > svq::kAbsMaxCandidates || N < 1) return SVQ_ERR_INVALID_ARG;
  if (!row_err || !best || !aligned(row_err, 8) || !aligned(best, 4) || (totals && !aligned(totals, 8)))
    return SVQ_ERR_INVALID_ARG;
  return cuda_status(svq::launch_abs_select(row_err, n_cand, N, totals, best, (cudaStream_t)stream));
}

unsigned svq_debug_set_wait_polls(unsigned polls) { return svq::set_wait_polls(polls); }

int svq_get_device_status(svq_stream_t stream) {
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return SVQ_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_status_word, sizeof(int)) != cudaSuccess) return SVQ_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(g_status_word, &zero, sizeof(int)) != cudaSuccess) return SVQ_ERR_CUDA;
  return v;
}

}  // extern "C"
