// kv_assign.cu -- block tables and slot maps of one step, built on the GPU from
// the requests' lengths.
//
// With ps tokens to a page, held_b = ceil(len_b / ps) pages of request b are in
// its table row.  n_b >= 0 new tokens take need_b = ceil((len_b + n_b) / ps) -
// held_b pages; n_b < 0 says that the request is done and releases its held_b.
// The free pages are a stack: the n_free entries of the list, then the released
// pages in request order; the k-th page that the step needs (request order) is
// entry top - 1 - k.  Row r of the step belongs to the request with
// cu[b] <= r < cu[b + 1], stands at position len_b + r - cu[b] and is kept in
// slot page * ps + position % ps.
//
// The work is three prefix sums over the requests and a few words per row, so
// latency bounds it: every CTA computes the prefix sums for itself (two loads
// and one block scan), then the rows, the new table entries and the free list
// are spread over all threads, each entry found by a binary search in shared
// memory; no CTA reads what another writes.  The CTAs of a call form one
// cluster and meet at its barrier once all of them have read the lengths and
// the free count, so those two may be updated in place (a captured decode step
// replayed again and again).  B200, in a CUDA graph: 16 decode rows 2.7 us, 256
// requests with 8192 rows 6.2 us.
#include "attn_params.h"
#include "svq.h"

namespace svq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Last i in [0, n) with a[i] <= v, for nondecreasing a with a[0] <= v.
__device__ __forceinline__ int find_segment(const int* a, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

struct Stack {                           // the step's free pages, bottom to top
  const KvAssignParams& p;
  const int* gone;                       // [n_seqs + 1] released pages before request b
  int n_free;
  __device__ int released(int i) const {
    const int b = find_segment(gone, p.n_seqs, i);
    return p.table[(size_t)b * p.width + (i - gone[b])];
  }
  __device__ int at(int i) const { return i < n_free ? p.free_pages[i] : released(i - n_free); }
};

__global__ void __launch_bounds__(kThreads) kv_assign_kernel(const __grid_constant__ KvAssignParams p) {
  extern __shared__ int sm[];
  const int n = p.n_seqs, ps = p.page_size;
  // pages of l tokens, 0 <= l <= width * page size (any other l refuses the call)
  auto pages_of = [&](int l) { return l > 0 ? p.by_page.div(l - 1) + 1 : 0; };
  int* len = sm;                         // [n] tokens, -1: done
  int* cu = len + n;                     // [n + 1] rows before request b
  int* need = cu + n + 1;                // [n + 1] pages needed before request b
  int* gone = need + n + 1;              // [n + 1] pages released before request b
  __shared__ long long w_rows[kWarps];
  __shared__ int w_need[kWarps], w_gone[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, ctas = gridDim.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Each thread takes a run of consecutive requests.  Row counts are summed in
  // 64 bits: a nonsense count must not wrap into a plausible total.  The page
  // sums stay below 2^31 whenever the call is not refused (the host checks
  // n_seqs * width, and need <= rows + n).
  const int n_free = *p.n_free;
  const long long room = (long long)p.width * ps;
  const int per = (n + kThreads - 1) / kThreads;
  const int b0 = min(n, tid * per), b1 = min(n, b0 + per);
  long long rows_t = 0;
  int need_t = 0, gone_t = 0;
  bool bad = n_free < 0 || n_free > p.n_pages;
  for (int b = b0; b < b1; ++b) {
    const int l = p.lens[b], a = p.n_new[b];
    const long long to = (long long)l + max(a, 0);
    bad |= l < 0 || to > room;
    const int held = pages_of(l);
    len[b] = l;
    cu[b] = a;                           // the new count for now
    rows_t += max(a, 0);
    need_t += a < 0 ? 0 : pages_of((int)to) - held;
    gone_t += a < 0 ? held : 0;
  }
  // inclusive sums over the lanes of the first `lanes`
  auto scan = [&](long long& r, int& s, int& t, int lanes) {
    for (int o = 1; o < lanes; o <<= 1) {
      const long long r1 = __shfl_up_sync(0xFFFFFFFFu, r, o);
      const int s1 = __shfl_up_sync(0xFFFFFFFFu, s, o), t1 = __shfl_up_sync(0xFFFFFFFFu, t, o);
      if (lane >= o) {
        r += r1;
        s += s1;
        t += t1;
      }
    }
  };
  long long rows_i = rows_t;
  int need_i = need_t, gone_i = gone_t;
  scan(rows_i, need_i, gone_i, 32);
  if (lane == 31) {
    w_rows[warp] = rows_i;
    w_need[warp] = need_i;
    w_gone[warp] = gone_i;
  }
  bad = __syncthreads_or(bad);
  long long rows_w = w_rows[lane % kWarps];                // every warp adds up the warps' sums
  int need_w = w_need[lane % kWarps], gone_w = w_gone[lane % kWarps];
  scan(rows_w, need_w, gone_w, kWarps);
  const long long rows_all = __shfl_sync(0xFFFFFFFFu, rows_w, kWarps - 1);
  const int need_all = __shfl_sync(0xFFFFFFFFu, need_w, kWarps - 1);
  const int gone_all = __shfl_sync(0xFFFFFFFFu, gone_w, kWarps - 1);
  long long rows = __shfl_sync(0xFFFFFFFFu, rows_w, (warp + 31) % 32);
  int need_b = __shfl_sync(0xFFFFFFFFu, need_w, (warp + 31) % 32);
  int gone_b = __shfl_sync(0xFFFFFFFFu, gone_w, (warp + 31) % 32);
  rows = (warp ? rows : 0) + rows_i - rows_t;
  need_b = (warp ? need_b : 0) + need_i - need_t;
  gone_b = (warp ? gone_b : 0) + gone_i - gone_t;
  const long long top = (long long)n_free + gone_all;
  const bool refuse = bad || rows_all > p.max_rows || need_all > top || top > p.n_pages;
  for (int b = b0; b < b1; ++b) {
    const int l = len[b], a = cu[b];
    const int held = pages_of(l);
    if (a < 0) len[b] = -1;              // done: it has no row, only its pages count
    cu[b] = (int)rows;
    need[b] = need_b;
    gone[b] = gone_b;
    rows += max(a, 0);
    need_b += a < 0 ? 0 : pages_of(l + a) - held;
    gone_b += a < 0 ? held : 0;
    if (rank == 0) p.cu_rows[b] = refuse ? 0 : cu[b];
  }
  if (tid == 0) {
    cu[n] = (int)rows_all;
    need[n] = need_all;
    gone[n] = gone_all;
    if (rank == 0) p.cu_rows[n] = refuse ? 0 : (int)rows_all;
  }
  // All CTAs have read the lengths and the free count (also the barrier that
  // publishes the prefix sums inside each CTA).
  if (ctas > 1) {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  if (rank == 0) {
    for (int b = b0; b < b1; ++b) {
      const int l = len[b];
      p.lens_out[b] = refuse ? p.lens[b] : l < 0 ? 0 : l + (cu[b + 1] - cu[b]);
    }
    if (tid == 0) {
      *p.n_free_out = refuse ? n_free : (int)(top - need_all);
      if (refuse) *p.status = SVQ_ERR_INVALID_ARG;
    }
  }
  const int g = rank * kThreads + tid, gn = ctas * kThreads;
  if (refuse) {
    for (int r = g; r < p.max_rows; r += gn) {
      p.positions[r] = -1;
      p.slots[r] = -1;
    }
    return;
  }
  const Stack stack{p, gone, n_free};
  const int itop = (int)top;
  // Four entries at a time: their loads are on their way together before the first store.
  constexpr int kBatch = 4;
  for (int r0 = g; r0 < p.max_rows; r0 += kBatch * gn) {
    int pos[kBatch], page[kBatch], off[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k * gn;
      pos[k] = -1;
      page[k] = off[k] = 0;
      if (r >= (int)rows_all) continue;
      const int b = find_segment(cu, n, r), l = len[b];
      pos[k] = l + (r - cu[b]);
      const int held = pages_of(l), j = p.by_page.div(pos[k]);
      off[k] = pos[k] - j * ps;
      page[k] = j < held ? p.table[(size_t)b * p.width + j] : stack.at(itop - 1 - (need[b] + j - held));
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k * gn;
      if (r >= p.max_rows) break;
      const bool ok = (unsigned)page[k] < (unsigned)p.n_pages;
      if (!ok) *p.status = SVQ_ERR_INVALID_ARG;
      p.positions[r] = pos[k];
      p.slots[r] = pos[k] >= 0 && ok ? page[k] * ps + off[k] : -1;
    }
  }
  for (int k0 = g; k0 < need_all; k0 += kBatch * gn) {
    int at[kBatch], page[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = k0 + k * gn;
      at[k] = page[k] = 0;
      if (i >= need_all) continue;
      const int b = find_segment(need, n, i);
      at[k] = b * p.width + pages_of(len[b]) + (i - need[b]);
      page[k] = stack.at(itop - 1 - i);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (k0 + k * gn < need_all) p.table[at[k]] = page[k];
  }
  // Released pages that the step does not take go onto the list, entry by entry where
  // they are few.  Where every warp has kRun * 32 of them they mostly lie in long
  // runs, the rows of done requests: a warp looks up the two runs that its next kRun
  // * 32 begin in, takes what lies there with kRun loads a lane on their way (from an
  // index held inside the runs: a load behind a condition would wait for the one
  // before), and goes entry by entry from the third run on (1024 requests of up to 16384
  // pages of one token, a tenth of them done: 271 -> 46 us).
  // (Unsigned: they can be close to 2^31, and the last step of a loop passes that.)
  // A page outside the pool goes onto the list like any other, and is reported here: the
  // step that takes it may be far (`worst` is looked at once: a branch at every store made
  // long releases half as slow again).
  const unsigned kept = max(itop - need_all - n_free, 0);
  unsigned worst = 0;
  auto report = [&] {
    if (worst >= (unsigned)p.n_pages) *p.status = SVQ_ERR_INVALID_ARG;
  };
  auto keep = [&](unsigned from, unsigned to, unsigned step) {
    for (unsigned i0 = from; i0 < to; i0 += kBatch * step) {
      int page[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) page[k] = i0 + k * step < to ? stack.released((int)(i0 + k * step)) : 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) worst = max(worst, (unsigned)page[k]);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i0 + k * step < to) p.free_pages[n_free + i0 + k * step] = page[k];
    }
  };
  constexpr unsigned kRun = 16;
  if (kept < kRun * gn) {
    keep(g, kept, gn);
    report();
    return;
  }
  for (unsigned i0 = g / 32 * (kRun * 32); i0 < kept; i0 += kRun * gn) {
    const unsigned to = min(kept, i0 + kRun * 32);
    const int b0 = find_segment(gone, n, (int)i0);
    const unsigned end0 = gone[b0 + 1];
    const int b1 = end0 < to ? find_segment(gone, n, (int)end0) : b0;
    const unsigned end = min(to, (unsigned)gone[b1 + 1]);
    const int* row0 = p.table + (size_t)b0 * p.width - gone[b0];
    const int* row1 = p.table + (size_t)b1 * p.width - gone[b1];
    int page[kRun];
#pragma unroll
    for (unsigned k = 0; k < kRun; ++k) {
      const unsigned i = min(i0 + k * 32 + lane, end - 1);
      page[k] = (i < end0 ? row0 : row1)[i];
    }
#pragma unroll
    for (unsigned k = 0; k < kRun; ++k) worst = max(worst, (unsigned)page[k]);
#pragma unroll
    for (unsigned k = 0; k < kRun; ++k) {
      const unsigned i = i0 + k * 32 + lane;
      if (i < end) p.free_pages[n_free + i] = page[k];
    }
    keep(end + lane, to, 32);
  }
  report();
}

}  // namespace

cudaError_t launch_kv_assign(const KvAssignParams& p, cudaStream_t st) {
  const size_t smem = (size_t)(4 * p.n_seqs + 3) * sizeof(int);
  // One CTA where there is little to spread, which a cluster makes 0.3 us slower (16
  // decode rows: 2.7 us against 3.0 us); a cluster where rows are many (543 requests
  // and 3339 rows: 4.8 us against 6.9 us) or the table is large, since a done request
  // may release a long row of it (63 requests of up to 3909 pages: 7.5 us against 30 us).
  const bool small = p.max_rows <= 2 * kThreads && (long long)p.n_seqs * p.width <= 8192;
  const unsigned ctas = small ? 1 : 8;
  if (smem > 48 * 1024) {                // the most any call needs, so that concurrent first calls agree
    static std::atomic<int> have[64];
    const cudaError_t e = allow_smem(kv_assign_kernel, (size_t)(4 * kMaxSeqs + 3) * sizeof(int), have);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(kv_assign_kernel, ctas, kThreads, smem, ctas, st, p);
}

}  // namespace svq
