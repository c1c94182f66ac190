// chunk_attn.cu -- causal attention of each request's new tokens over all of
// its cached tokens in the paged cache: the dense counterpart of stage 4
// (TensorRT-LLM "QSASparseAttentionConfig", seq_len_threshold: sequences up to
// the threshold attend densely; "QSA in brief": all KV stays resident).
//
//   p = kv_len[b] - n_new[b] + i    (position of new token i of request b)
//   out = sum_{j <= p} softmax(scale q . k_j) v_j,   lse = log sum_{j <= p} exp(scale q . k_j)
//
// This file holds the general kernel (every dtype pair, FP32 arithmetic on the
// CUDA cores), the combine kernel that merges tiles several workers share, and
// the choice between the general kernel and those on the tensor cores.
//
// General kernel: a CTA takes a tile of 32 query rows (whole tokens: all query
// heads of one KV head) against one page of 64 keys at a time.  256 threads
// hold 2 x 4 logits each; the page's keys and values go through shared memory
// in FP32 and are read back as float4 (32 multiply-adds per 6 shared loads),
// the running maximum and sum of the softmax stay in registers, 16 threads to
// a row.  It serves float32 models, whose values the tensor cores would round,
// and is bound by the FP32 pipes for long prompts; a tiny model's (437 tokens,
// 4/1 heads of D 64: 18 us) by the launch and one tile's latency.  128 threads
// of 4 x 4 logits share loads better, but leave a scheduler one warp to hide
// latencies with, and took as long.
#include <math.h>

#include "chunk_common.cuh"

namespace qsa {

// chunk_attn_tc.cu
bool chunk_tc_supported(const ChunkArgs& a);
int chunk_tc_rows();
// chunk_attn_few.cu
cudaError_t launch_chunk_attn_few(const ChunkArgs& a, const ChunkWs& ws, int rows, int grid, float qk_scale_log2,
                                  float vmul, cudaStream_t s);
cudaError_t launch_chunk_attn_tc(const ChunkArgs& a, const ChunkWs& ws, int grid, float qk_scale_log2, float vmul,
                                 cudaStream_t s);

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

constexpr int kThreads = 256;
constexpr int kR = 2;                  // query rows of a thread
constexpr int kRows = 32;              // query rows of a tile
constexpr int kKeys = kPageTokens;     // keys of a block: one page

template <int D>
struct SimtSmem {
  float q[kRows][D];
  float k[kKeys][D + 4];               // + 4: 8 rows' float4 fall into distinct banks
  float v[kKeys][D];
  float p[kRows][kKeys + 4];
  ChunkSched sched;
};

template <int D, typename QT, typename KVT>
__global__ void __launch_bounds__(kThreads) chunk_simt_kernel(ChunkArgs a, ChunkWs ws, float qk_scale_log2, float vmul) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SimtSmem<D>& sm = *reinterpret_cast<SimtSmem<D>*>(smem_raw);
  const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15;
  const int G = a.Hq / a.Hkv, TPT = kRows / G;
  constexpr int C4 = D / 64;           // float4 columns of O per thread
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0 && blockIdx.x < kChunkMaxCtas) ws.desc[blockIdx.x].n_parts = 0;
  chunk_sched_build(a, sm.sched, TPT, kKeys, blockIdx.x, gridDim.x, false, 2);
  ChunkWalk walk;
  walk.begin(a, sm.sched, blockIdx.x, gridDim.x);
  const QT* q = reinterpret_cast<const QT*>(a.q);
  const KVT* kc = reinterpret_cast<const KVT*>(a.k_pages);
  const KVT* vc = reinterpret_cast<const KVT*>(a.v_pages);
  ChunkItem it;
  while (walk.next(a, sm.sched, TPT, kKeys, it)) {
    const int rows = it.ntok * G;
    __syncthreads();
    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < rows) {
        const size_t src = ((size_t)(it.t0 + r / G) * a.Hq + it.kvh * G + r % G) * D + d;
        VecLoad<QT, 4>::get(q, src, x);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sm.q[r][d + j] = x[j] * qk_scale_log2;
    }
    int lim[kR];                        // keys each of this thread's rows sees
    float m[kR], l[kR], o[kR][C4 * 4];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int r = rg * kR + i;
      lim[i] = r < rows ? min(it.p0 + r / G + 1, it.kv) : it.kv;   // rows past the tile are not stored
      m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < C4 * 4; ++c) o[i][c] = 0.f;
    }
    const int32_t* pt = a.page_table + (size_t)it.b * a.pt_stride;
    for (int blk = it.blk_lo; blk < it.blk_hi; ++blk) {
      const int key0 = blk * kKeys;
      const int live = min(kKeys, it.kv - key0);   // keys of the page that hold tokens
      int page = live > 0 ? pt[blk] : -1;
      if (live > 0 && (page < 0 || page >= a.num_pages)) {
        if (tid == 0) flag(a.status, QSA_DEV_BAD_PAGE);
        page = -1;
      }
      __syncthreads();
      for (int i = tid; i < kKeys * (D / 4); i += kThreads) {
        const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
        if (page >= 0 && r < live) {
          const size_t src = (((size_t)page * kPageTokens + r) * a.Hkv + it.kvh) * D + d;
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = Elem<KVT>::get(kc, src + j), y[j] = Elem<KVT>::get(vc, src + j);
        }
        *reinterpret_cast<float4*>(&sm.k[r][d]) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(&sm.v[r][d]) = make_float4(y[0], y[1], y[2], y[3]);
      }
      __syncthreads();
      // logits (base 2) of rows rg * kR and the next, keys cg + 16 j
      float s[kR][4] = {};
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 x[kR], y[4];
#pragma unroll
        for (int i = 0; i < kR; ++i) x[i] = *reinterpret_cast<const float4*>(&sm.q[rg * kR + i][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(&sm.k[cg + 16 * j][d]);
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
            s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
            s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
            s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
          }
      }
      bool whole = page >= 0;          // every row sees every key of the page
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const int seen = page >= 0 ? lim[i] - key0 : 0;
        whole = whole && seen >= kKeys;
        float mx = m[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (cg + 16 * j >= seen) s[i][j] = -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int d = 8; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float base = mx == -INFINITY ? 0.f : mx;
        const float alpha = m[i] == mx ? 1.f : exp2f(m[i] - base);
        m[i] = mx;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2f(s[i][j] - base);
          sum += e;
          sm.p[rg * kR + i][cg + 16 * j] = e;
        }
#pragma unroll
        for (int d = 8; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l[i] = l[i] * alpha + sum;
#pragma unroll
        for (int c = 0; c < C4 * 4; ++c) o[i][c] *= alpha;
      }
      __syncwarp();                    // a row's 16 threads share a warp
      if (page >= 0) {
        for (int j = 0; j < live; ++j) {
          float p[kR];
#pragma unroll
          for (int i = 0; i < kR; ++i) p[i] = sm.p[rg * kR + i][j];
#pragma unroll
          for (int c = 0; c < C4; ++c) {
            const float4 y = *reinterpret_cast<const float4*>(&sm.v[j][cg * 4 + 64 * c]);
#pragma unroll
            for (int i = 0; i < kR; ++i) {
              // a value a row does not see must not reach it, not even as 0 * inf
              if (whole || key0 + j < lim[i]) {
                o[i][4 * c] = fmaf(p[i], y.x, o[i][4 * c]);
                o[i][4 * c + 1] = fmaf(p[i], y.y, o[i][4 * c + 1]);
                o[i][4 * c + 2] = fmaf(p[i], y.z, o[i][4 * c + 2]);
                o[i][4 * c + 3] = fmaf(p[i], y.w, o[i][4 * c + 3]);
              }
            }
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int r = rg * kR + i;
      if (r >= rows) continue;
      if (it.part < 0) {
        const size_t row = (size_t)(it.t0 + r / G) * a.Hq + it.kvh * G + r % G;
        const float inv = l[i] == 0.f ? 0.f : vmul / l[i];
        QT* op = reinterpret_cast<QT*>(a.out) + row * D;
#pragma unroll
        for (int c = 0; c < C4; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float y = l[i] == 0.f ? 0.f : o[i][4 * c + j] * inv;
            if constexpr (sizeof(QT) == 4) op[cg * 4 + 64 * c + j] = y;
            else op[cg * 4 + 64 * c + j] = __float2bfloat16_rn(y);
          }
        if (a.lse && cg == 0) a.lse[row] = l[i] == 0.f ? -INFINITY : m[i] * kLn2 + logf(l[i]);
      } else {
        const size_t prow = (size_t)it.part * kRows + r;
#pragma unroll
        for (int c = 0; c < C4; ++c)
          *reinterpret_cast<float4*>(ws.o + prow * D + cg * 4 + 64 * c) =
              make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]);
        if (cg == 0) ws.ml[prow] = make_float2(m[i], l[i]);
      }
    }
    if (it.n_parts > 0 && tid == 0) ws.desc[blockIdx.x] = ChunkDesc{it.n_parts, it.t0, it.ntok, it.kvh};
  }
}

// Merges a tile that several workers share: blockIdx.x = the worker that opened
// it, blockIdx.y walks its rows.  Up to 8 partials (chunks): a warp joins a row
// by itself.  More (long decode rows): a row's partials are spread over the 8
// warps and joined in shared memory.  The order of the sums is fixed.
constexpr int kCombineThreads = 256;
// CTAs to a worker's tile.  Narrow tiles: 8, as most of a small step's only find
// that nothing is shared (one token behind 63: 9.5 us, 10.7 with 16); else
// 16 (8: float32 prompts 23 us instead of 20).
constexpr int kCombineFew = 8, kCombineWide = 16;
template <int D, typename OT>
__global__ void __launch_bounds__(kCombineThreads) chunk_combine_kernel(ChunkArgs a, ChunkWs ws, int tile_rows,
                                                                        float vmul) {
  constexpr int VPT = D / 32;
  constexpr int W = kCombineThreads / 32;
  __shared__ float o_s[W][D];
  __shared__ float ml_s[W][2];
  pdl_wait();
  pdl_launch_dependents();
  const ChunkDesc dsc = ws.desc[blockIdx.x];
  if (dsc.n_parts == 0) return;
  const int G = a.Hq / a.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = 2 * blockIdx.x + 1;                 // then 2 (blockIdx.x + i), i = 1 .. n_parts - 1
  if (dsc.n_parts <= W) {
    for (int r = blockIdx.y * W + warp; r < dsc.ntok * G; r += gridDim.y * W) {
      // lane i: the maximum and sum of part i, and its weight
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < dsc.n_parts) ml = ws.ml[(size_t)(lane == 0 ? first : 2 * (blockIdx.x + lane)) * tile_rows + r];
      float mx = ml.x;
#pragma unroll
      for (int d = 4; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      mx = __shfl_sync(0xffffffffu, mx, 0);
      const float w = ml.x == mx ? 1.f : exp2f(ml.x - (mx == -INFINITY ? 0.f : mx));
      float total = 0.f, o[VPT];
#pragma unroll
      for (int j = 0; j < VPT; ++j) o[j] = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (i >= dsc.n_parts) break;
        float x[VPT];
        VecLoad<float, VPT>::get(ws.o, ((size_t)(i == 0 ? first : 2 * (blockIdx.x + i)) * tile_rows + r) * D + lane * VPT, x);
        const float wi = __shfl_sync(0xffffffffu, w, i);
        total += __shfl_sync(0xffffffffu, ml.y, i) * wi;
#pragma unroll
        for (int j = 0; j < VPT; ++j) o[j] = fmaf(x[j], wi, o[j]);
      }
      const int tok = r / G;
      const size_t row = (size_t)(dsc.t0 + tok) * a.Hq + dsc.kvh * G + (r - tok * G);
      const float inv = total == 0.f ? 0.f : vmul / total;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        o[j] = total == 0.f ? 0.f : o[j] * inv;
        if constexpr (sizeof(OT) == 4) reinterpret_cast<float*>(a.out)[row * D + lane * VPT + j] = o[j];
        else reinterpret_cast<__nv_bfloat16*>(a.out)[row * D + lane * VPT + j] = __float2bfloat16_rn(o[j]);
      }
      if (a.lse && lane == 0) a.lse[row] = total == 0.f ? -INFINITY : mx * kLn2 + logf(total);
    }
    return;
  }
  for (int r = blockIdx.y; r < dsc.ntok * G; r += gridDim.y) {
    float m = -INFINITY, l = 0.f, o[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) o[j] = 0.f;
    for (int i = warp; i < dsc.n_parts; i += W) {
      const size_t row = (size_t)(i == 0 ? first : 2 * (blockIdx.x + i)) * tile_rows + r;
      const float2 ml = ws.ml[row];
      float x[VPT];
      VecLoad<float, VPT>::get(ws.o, row * D + lane * VPT, x);
      const float mn = fmaxf(m, ml.x);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float w0 = m == mn ? 1.f : exp2f(m - base), w1 = ml.x == mn ? 1.f : exp2f(ml.x - base);
      m = mn;
      l = l * w0 + ml.y * w1;
#pragma unroll
      for (int j = 0; j < VPT; ++j) o[j] = o[j] * w0 + x[j] * w1;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) o_s[warp][lane * VPT + j] = o[j];
    if (lane == 0) ml_s[warp][0] = m, ml_s[warp][1] = l;
    __syncthreads();
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) mx = fmaxf(mx, ml_s[w][0]);
    const float base = mx == -INFINITY ? 0.f : mx;
    float wt[W], total = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      wt[w] = ml_s[w][0] == mx ? 1.f : exp2f(ml_s[w][0] - base);
      total += ml_s[w][1] * wt[w];
    }
    const size_t out_row = (size_t)(dsc.t0 + r / G) * a.Hq + dsc.kvh * G + r % G;
    for (int d = threadIdx.x; d < D; d += kCombineThreads) {
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) y += o_s[w][d] * wt[w];
      y = total == 0.f ? 0.f : y * (vmul / total);
      if constexpr (sizeof(OT) == 4) reinterpret_cast<float*>(a.out)[out_row * D + d] = y;
      else reinterpret_cast<__nv_bfloat16*>(a.out)[out_row * D + d] = __float2bfloat16_rn(y);
    }
    if (a.lse && threadIdx.x == 0) a.lse[out_row] = total == 0.f ? -INFINITY : mx * kLn2 + logf(total);
    __syncthreads();
  }
}

template <int D, typename QT, typename KVT>
cudaError_t launch_simt(const ChunkArgs& a, const ChunkWs& ws, int grid, float qk, float vmul, cudaStream_t s) {
  auto kern = chunk_simt_kernel<D, QT, KVT>;
  const size_t smem = sizeof(SimtSmem<D>);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(grid), dim3(kThreads), smem, s, 1, a, ws, qk, vmul);
}
template <int D, typename QT>
cudaError_t launch_simt_kv(const ChunkArgs& a, const ChunkWs& ws, int grid, float qk, float vmul, cudaStream_t s) {
  switch (a.kv_dt) {
    case QSA_F32: return launch_simt<D, QT, float>(a, ws, grid, qk, vmul, s);
    case QSA_BF16: return launch_simt<D, QT, __nv_bfloat16>(a, ws, grid, qk, vmul, s);
    default: return launch_simt<D, QT, __nv_fp8_e4m3>(a, ws, grid, qk, vmul, s);
  }
}
// Query rows of a tile of the few-rows kernel (8 or 16), or 0: the wide tiles
// serve better.  The host knows the batch's tokens, not each request's.  Above
// 16 rows the narrow tiles read the cache once per 16.
// Measured, 16/2 heads, narrow against wide (us):
//   rows  batch         D 256 BF16  FP8        D 128 BF16  FP8
//   8     8 x 65,000    163 : 210   95 : 216   88 : 173    56 : 184
//   16    8 x 65,000    180 : 212   126 : 214  93 : 167    80 : 183
//   24    8 x 65,000    330 : 213   206 : 213  165 : 170   138 : 184
//   32    8 x 65,000    332 : 198   218 : 205  167 : 147   150 : 160
//   32    64 x 300      46 : 32     45 : 36    29 : 24     28 : 29
// The average misses batches that are far from it: a T padded from 8 to 160
// tokens puts 8 x 65,000 FP8 on the wide tiles (211 us instead of 92), and 64
// tokens behind 3,000 beside a prompt of 2,000 take 248 us in one call, 59 + 110
// in two (BF16: 128 against 74 + 54).
int few_rows(const ChunkArgs& a) {
  const int G = a.Hq / a.Hkv;
  const int rows = (a.T + a.B - 1) / a.B * G;   // of an average request
  const int most = 16 + (a.kv_dt == QSA_FP8_E4M3 ? 8 : 0) + (a.D <= 128 ? 8 : 0);
  return rows <= 8 ? 8 : rows <= most ? 16 : 0;
}

template <int D>
cudaError_t launch_d(const ChunkArgs& a, void* wsp, int grid, float qk, float vmul, cudaStream_t s) {
  const bool tc = chunk_tc_supported(a);
  const int few = tc ? few_rows(a) : 0;
  const int rows = few ? few : tc ? chunk_tc_rows() : kRows;
  const ChunkWs ws = chunk_ws(wsp, D);
  cudaError_t e;
  if (few) e = launch_chunk_attn_few(a, ws, few, grid, qk, vmul, s);
  else if (tc) e = launch_chunk_attn_tc(a, ws, grid, qk, vmul, s);
  else if (a.q_dt == QSA_F32) e = launch_simt_kv<D, float>(a, ws, grid, qk, vmul, s);
  else e = launch_simt_kv<D, __nv_bfloat16>(a, ws, grid, qk, vmul, s);
  if (e != cudaSuccess) return e;
  auto comb = a.q_dt == QSA_F32 ? chunk_combine_kernel<D, float> : chunk_combine_kernel<D, __nv_bfloat16>;
  const int workers = tc && !few ? grid / 2 : grid;   // who may have opened a tile that others finish
  return launch_k(comb, dim3(workers, few ? kCombineFew : kCombineWide), dim3(kCombineThreads), 0, s, 1, a, ws, rows, vmul);
}

}  // namespace

int chunk_attn_max_requests() { return kChunkMaxReq; }

size_t chunk_attn_ws_bytes(int T, int B, int Hq, int Hkv, int D, qsa_dtype_t kv_dt) {
  (void)T, (void)B, (void)Hq, (void)Hkv, (void)kv_dt;
  return chunk_ws_bytes(D);
}

cudaError_t launch_chunk_attn(const ChunkArgs& a, void* ws, cudaStream_t s) {
  const float scale = a.sm_scale > 0.f ? a.sm_scale : 1.f / sqrtf((float)a.D);
  const bool fp8 = a.kv_dt == QSA_FP8_E4M3;
  const float qk = scale * kLog2e * (fp8 ? a.k_scale : 1.f);
  const float vmul = fp8 ? a.v_scale : 1.f;
  int dev = 0, sms = kChunkMaxCtas;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int grid = sms < kChunkMaxCtas ? sms : kChunkMaxCtas;
  switch (a.D) {
    case 64: return launch_d<64>(a, ws, grid, qk, vmul, s);
    case 128: return launch_d<128>(a, ws, grid, qk, vmul, s);
    default: return launch_d<256>(a, ws, grid, qk, vmul, s);
  }
}

}  // namespace qsa
