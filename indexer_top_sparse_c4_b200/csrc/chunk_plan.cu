// chunk_plan.cu -- block tables and slot maps of a serving step, built on the
// GPU from the requests' lengths ("QSA HiSparse" README: page size 64, all KV
// resident; the tables every other call of this library reads).
//
//   cu[b]   = sum_{i<b} n_new[i]            kv[b] = n_cached[b] + n_new[b]
//   token t of request b = the one with cu[b] <= t < cu[b+1]:
//   pos     = n_cached[b] + t - cu[b]       slot  = page(b, pos / 64) * 64 + pos % 64
//   page(b, i) = page_table[b][i] below ceil(n_cached[b] / 64), and behind it
//                free_pages[base[b] + i - ceil(n_cached[b] / 64)], base the
//                prefix sum of the pages the requests grow by
//
// The work is a few bytes per request and 12 per token, so a call costs what
// its launch and the chain of dependent reads cost.  One launch does all of
// it: every CTA scans all requests' lengths itself (they are L2 hits after the
// first CTA), keeps both prefix sums in shared memory and then serves its own
// slice of tokens and of new table entries by binary search, so no CTA waits
// for another and no second launch is needed.  Pages that a token needs are
// taken from the free list, never from the table entries other CTAs write.
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxReq = 8192;
constexpr int kTokens = 4 * kThreads;  // tokens per CTA

struct PlanReq {
  int cached, fresh;
};
__device__ __forceinline__ PlanReq load_req(const PlanArgs& a, int b, bool report) {
  int c = a.n_cached[b], n = a.n_new[b];
  if (report && (c < 0 || n < 0)) flag(a.status, QSA_DEV_ROW_RANGE);
  return PlanReq{max(c, 0), max(n, 0)};
}
__device__ __forceinline__ int pages_of(const PlanArgs& a, long long tokens) {
  const long long p = (tokens + kPageTokens - 1) / kPageTokens;
  return p < a.pt_stride ? (int)p : a.pt_stride;
}
__device__ __forceinline__ int find(const int* v, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Exclusive prefix sum over the CTA plus carry (64 bits: lengths are the caller's).
__device__ __forceinline__ long long scan(long long v, long long* warp_sum, long long& carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  __syncthreads();
  const long long out = carry + before + x - v;
  carry += total;
  return out;
}

__global__ void __launch_bounds__(kThreads) chunk_plan_kernel(PlanArgs a) {
  extern __shared__ long long smem[];             // all of the kernel's: plan_smem below counts it
  long long* warp_sum = smem;                     // [kThreads / 32]
  int* cu = reinterpret_cast<int*>(smem + kThreads / 32);   // [B + 1] tokens before each request, cut at T
  int* base = cu + a.B + 1;                       // [B + 1] free pages taken before each request
  const int tid = threadIdx.x;
  const bool first = blockIdx.x == 0;
  pdl_wait();
  pdl_launch_dependents();

  long long tokens = 0, taken = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    PlanReq r{0, 0};
    if (b < a.B) r = load_req(a, b, first);
    const long long before = scan(r.fresh, warp_sum, tokens);
    // tokens past T are cut: the request keeps those that fit
    const int lo = (int)min(before, (long long)a.T);
    const int hi = (int)min(before + r.fresh, (long long)a.T);
    const long long kv = (long long)r.cached + (hi - lo);
    const int has = pages_of(a, r.cached), need = pages_of(a, kv);
    const long long pages = scan(need - has, warp_sum, taken);
    if (b < a.B) {
      cu[b] = lo;
      base[b] = (int)min(pages, 0x7fffffffll);
      if (first) {
        a.cu_new[b] = lo;
        a.kv_len[b] = (int)min(kv, 0x7fffffffll);
        if (before + r.fresh > a.T || kv > (long long)a.pt_stride * kPageTokens) flag(a.status, QSA_DEV_ROW_RANGE);
      }
    }
  }
  const int used = (int)min(tokens, (long long)a.T);
  const int grown = (int)min(taken, 0x7fffffffll);
  if (tid == 0) {
    cu[a.B] = used;
    base[a.B] = grown;
    if (first) {
      a.cu_new[a.B] = used;
      a.n_taken[0] = min(grown, a.n_free);
      if (grown > a.n_free) flag(a.status, QSA_DEV_NO_PAGE);
    }
  }
  __syncthreads();

  // new table entries
  for (int g = blockIdx.x * kThreads + tid; g < grown; g += gridDim.x * kThreads) {
    const int b = find(base, a.B, g);
    const int page = g < a.n_free ? a.free_pages[g] : -1;
    if (g < a.n_free && (page < 0 || page >= a.num_pages)) flag(a.status, QSA_DEV_BAD_PAGE);
    a.page_table[(size_t)b * a.pt_stride + pages_of(a, load_req(a, b, false).cached) + (g - base[b])] = page;
  }
  // tokens
#pragma unroll
  for (int i = 0; i < kTokens / kThreads; ++i) {
    const int t = blockIdx.x * kTokens + i * kThreads + tid;
    if (t >= a.T) break;
    int req = -1, pos = -1, slot = -1;
    if (t < used) {
      req = find(cu, a.B, t);
      const PlanReq r = load_req(a, req, false);
      const long long p = (long long)r.cached + (t - cu[req]);
      pos = (int)min(p, 0x7fffffffll);
      const long long lp = p / kPageTokens;
      if (lp < a.pt_stride) {
        const int has = pages_of(a, r.cached);
        int page;
        if (lp < has) {
          page = a.page_table[(size_t)req * a.pt_stride + lp];
          if (page < 0 || page >= a.num_pages) flag(a.status, QSA_DEV_BAD_PAGE);
        } else {
          const long long g = (long long)base[req] + (lp - has);
          page = g < a.n_free ? a.free_pages[g] : -1;
        }
        if (page >= 0 && page < a.num_pages) slot = page * kPageTokens + (int)(p % kPageTokens);
      }
    }
    a.q_req[t] = req;
    a.q_pos[t] = pos;
    a.slot[t] = slot;
  }
}

constexpr size_t plan_smem(int B) { return kThreads / 32 * sizeof(long long) + 2 * ((size_t)B + 1) * sizeof(int); }

}  // namespace

int chunk_plan_max_requests() { return kMaxReq; }

cudaError_t launch_chunk_plan(const PlanArgs& a, cudaStream_t s) {
  const int grid = a.T > 0 ? (a.T + kTokens - 1) / kTokens : 1;
  const size_t smem = plan_smem(a.B);
  if (smem > 48 * 1024) {       // more than a kernel has without asking
    const cudaError_t e = cudaFuncSetAttribute(chunk_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)plan_smem(kMaxReq));
    if (e != cudaSuccess) return e;
  }
  return launch_k(chunk_plan_kernel, dim3(grid), dim3(kThreads), smem, s, 1, a);
}

}  // namespace qsa
