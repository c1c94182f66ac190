// chunk_common.cuh -- what the kernels of the chunk attention share: the
// reading of a request's lengths, the cut of the work into tiles of query rows
// and blocks of keys, and the share of it of each worker (a CTA, or a pair).
#pragma once
#include "umma.cuh"

namespace qsa {

constexpr int kChunkMaxReq = 1024;   // requests per chunk-attention call
constexpr int kChunkMaxTiles = 1024; // query tiles per KV head of a call whose tiles are split over workers
constexpr int kChunkMaxCtas = 148;   // CTAs that leave partials (one per SM of a B200; half as many pairs)

// A request as the device arrays give it.  `kv` is capped to the tokens a row
// of the page table can address.
struct ChunkReq {
  int t0, n, p0, kv;  // first query token, tokens, position of the first one, cached tokens
};
__device__ __forceinline__ ChunkReq chunk_req(const ChunkArgs& a, int b, bool report) {
  int lo = a.cu_new[b], hi = a.cu_new[b + 1], kv = a.kv_len[b];
  const int cap = a.pt_stride * kPageTokens;
  if (report && (lo < 0 || hi < lo || hi > a.T || kv < 0 || kv > cap)) flag(a.status, QSA_DEV_ROW_RANGE);
  lo = min(max(lo, 0), a.T);
  hi = min(max(hi, lo), a.T);
  kv = max(kv, 0);
  return ChunkReq{lo, hi - lo, kv - (hi - lo), min(kv, cap)};
}

// One worker's piece of work: key blocks [blk_lo, blk_hi) of a tile of query
// tokens and one KV head.
struct ChunkItem {
  int b, kvh, t0, ntok, p0, kv;
  int blk_lo, blk_hi, nblk;
  int part;      // -1: the whole tile; otherwise the slot its partial goes to
  int n_parts;   // > 0: this piece holds the tile's first block, and so many pieces share the tile
};

// What a combine CTA needs to know of a tile that several workers share; entry
// c is written by worker c (n_parts = 0: none of its pieces opens a shared
// tile).  Partial slots: 2c + 1 for a piece that opens a tile worker c does not
// finish, 2c for a piece that starts inside a tile (its first).
struct ChunkDesc {
  int n_parts, t0, ntok, kvh;
};

// The cut of a call's work.  Query tiles hold TPT tokens of one request (all
// query heads of one KV head); their keys fall into blocks of KT.  With few
// tiles the linear (KV head, tile, unit) space is divided evenly over the
// workers, whatever the requests' lengths, and tiles that several share are
// merged by the combine kernel.  A tile's units are its key blocks behind a
// lead: what its start and end cost, in blocks, so that a worker with many
// short tiles does not finish last.  With many tiles (four per worker, or
// more than the table holds) every tile is one worker's; neighbours then walk
// the same keys at about the same time and share them in L2, and rounds run
// in alternating order so that the causal tiles' growing lengths even out.
struct ChunkSched {
  int first[kChunkMaxReq + 1];    // query tiles before each request
  int blk[kChunkMaxTiles + 1];    // shared tiles: units before each query tile (its lead and its key blocks)
  int warp_sum[32];
  int nq, shared_tiles, lead;
  // shared tiles: where this worker starts and ends, and its first tile
  long long u, u1;
  int ctas, kvh, q, x, b;         // ctas: workers that have work; x: unit within the tile; b: request
};

// Exclusive prefix sum of v over the CTA's threads plus `carry`; returns this
// thread's prefix and adds the total to carry.
__device__ __forceinline__ int chunk_scan(int v, int* warp_sum, int& carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < nw; ++w) {
    const int s = warp_sum[w];
    if (w < warp) before += s;
    total += s;
  }
  __syncthreads();
  const int out = carry + before + x - v;
  carry += total;
  return out;
}

__device__ __forceinline__ int chunk_tile_blocks(const ChunkReq& r, int tile, int TPT, int KT) {
  const int last = min(r.n, (tile + 1) * TPT) - 1;          // the tile's last token
  const int seen = min(r.p0 + last + 1, r.kv);              // keys it may see
  return max(1, (seen + KT - 1) / KT);                      // an empty tile still writes its zeros
}

// The last index i of [0, n) with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int chunk_find(const int* v, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Called by every thread of the CTA for worker `me` of `all` (a CTA, or a pair
// of them); the table is ready on return.  share: tiles are split over workers
// however many there are (as far as the table holds them).
__device__ __forceinline__ void chunk_sched_build(const ChunkArgs& a, ChunkSched& s, int TPT, int KT, int me, int all,
                                                  bool share, int lead) {
  int carry = 0;
  for (int base = 0; base < a.B; base += blockDim.x) {
    const int b = base + threadIdx.x;
    int n = 0;
    if (b < a.B) n = (chunk_req(a, b, blockIdx.x == 0).n + TPT - 1) / TPT;
    const int before = chunk_scan(n, s.warp_sum, carry);
    if (b < a.B) s.first[b] = before;
  }
  const int nq = carry;
  const bool shared = nq <= kChunkMaxTiles && (share || (long long)nq * a.Hkv < 4ll * all);
  if (threadIdx.x == 0) {
    s.first[a.B] = nq;
    s.nq = nq;
    s.lead = lead;
    s.shared_tiles = shared;
    s.u = s.u1 = 0;
    s.ctas = all;
  }
  __syncthreads();
  if (!shared || nq == 0) return;
  carry = 0;
  for (int base = 0; base < nq; base += blockDim.x) {
    const int q = base + threadIdx.x;
    int n = 0;
    if (q < nq) {
      const int b = chunk_find(s.first, a.B, q);
      n = lead + chunk_tile_blocks(chunk_req(a, b, false), q - s.first[b], TPT, KT);
    }
    const int before = chunk_scan(n, s.warp_sum, carry);
    if (q < nq) s.blk[q] = before;
  }
  if (threadIdx.x == 0) s.blk[nq] = carry;
  __syncthreads();
  const int wq = carry;
  const long long total = (long long)wq * a.Hkv;
  const int ctas = total < all ? (int)total : all;
  long long u = 0, u1 = 0;
  int kvh = 0;
  if (me < ctas) {
    if (total < (1 << 23)) {   // 32-bit divisions are several times cheaper
      const uint32_t t = (uint32_t)total;
      u = t * (uint32_t)me / (uint32_t)ctas;
      u1 = t * (uint32_t)(me + 1) / (uint32_t)ctas;
      kvh = (int)((uint32_t)u / (uint32_t)wq);
    } else {
      u = total * me / ctas;
      u1 = total * (me + 1) / ctas;
      kvh = (int)(u / wq);
    }
  }
  // the thread whose tile holds the first unit writes the start down
  const int y = (int)(u - (long long)kvh * wq);
  for (int q = threadIdx.x; q < nq; q += blockDim.x) {
    if (s.blk[q] <= y && y < s.blk[q + 1]) {
      s.u = u, s.u1 = u1, s.ctas = ctas, s.kvh = kvh;
      s.q = q, s.x = y - s.blk[q], s.b = chunk_find(s.first, a.B, q);
    }
  }
  __syncthreads();
}

// The walk of worker `me` of `all` (a CTA, or a pair of them) over its pieces;
// every warp role runs its own copy.  A step costs a few shared-memory reads:
// the next tile follows from the last one, only the first is searched for.
struct ChunkWalk {
  long long u, u1, total;  // shared tiles: units left to walk; otherwise u counts rounds
  int me, all, ctas;       // ctas: workers that have work
  int kvh, q, x, b;        // shared tiles: KV head, tile, unit within the tile, request

  __device__ __forceinline__ void begin(const ChunkArgs& a, const ChunkSched& s, int me_, int all_) {
    me = me_, all = all_;
    u = s.u, u1 = s.u1, ctas = s.ctas, total = 0;
    kvh = q = x = b = 0;
    if (s.shared_tiles && s.nq > 0) {
      total = (long long)s.blk[s.nq] * a.Hkv;
      kvh = s.kvh, q = s.q, x = s.x, b = s.b;
    }
  }
  __device__ __forceinline__ bool next(const ChunkArgs& a, const ChunkSched& s, int TPT, int KT, ChunkItem& it) {
    int tile;
    if (s.shared_tiles) {
      for (;;) {   // a piece that would hold no block (a tile's lead alone) is passed over
        if (u >= u1) return false;
        while (s.first[b + 1] <= q) ++b;
        const int units = s.blk[q + 1] - s.blk[q], nblk = units - s.lead;
        const int take = u1 - u < units - x ? (int)(u1 - u) : units - x;
        it.kvh = kvh, it.b = b, it.nblk = nblk;
        it.blk_lo = max(0, x - s.lead), it.blk_hi = x + take - s.lead;
        it.part = -1, it.n_parts = 0;
        tile = q - s.first[b];
        if (it.blk_lo > 0) {
          it.part = 2 * me;
        } else if (it.blk_hi < nblk) {
          it.part = 2 * me + 1;
          const long long last = u + (units - x) - 1;                  // the tile's last unit
          // the worker whose share holds it
          const int owner = total < (1 << 23) ? (int)(((uint32_t)(last + 1) * (uint32_t)ctas - 1) / (uint32_t)total)
                                              : (int)(((last + 1) * ctas - 1) / total);
          it.n_parts = owner - me + 1;
        }
        u += take;
        x += take;
        if (x == units) {
          x = 0;
          if (++q == s.nq) q = 0, b = 0, ++kvh;
        }
        if (it.blk_hi > it.blk_lo) break;
      }
    } else {
      const long long idx = u * all + ((u & 1) ? all - 1 - me : me);
      if (u * all >= (long long)s.nq * a.Hkv) return false;
      ++u;
      if (idx >= (long long)s.nq * a.Hkv) return false;  // only in the last round
      it.kvh = (int)(idx / s.nq);
      q = (int)(idx - (long long)it.kvh * s.nq);
      it.part = -1, it.n_parts = 0;
      it.b = chunk_find(s.first, a.B, q);
      tile = q - s.first[it.b];
    }
    const ChunkReq r = chunk_req(a, it.b, false);
    if (!s.shared_tiles) {
      it.nblk = chunk_tile_blocks(r, tile, TPT, KT);
      it.blk_lo = 0, it.blk_hi = it.nblk;
    }
    it.t0 = r.t0 + tile * TPT;
    it.ntok = min(TPT, r.n - tile * TPT);
    it.p0 = r.p0 + tile * TPT;
    it.kv = r.kv;
    return true;
  }
};

// Partials of the split tiles: unnormalised outputs [slot][row][D], then
// (running maximum in base 2, sum) [slot][row], then the tiles' descriptors.
// Two slots a worker; workers x rows of a tile is at most kChunkMaxCtas x 128.
constexpr size_t kChunkWsRows = (size_t)2 * kChunkMaxCtas * 128;
struct ChunkWs {
  float* o;
  float2* ml;
  ChunkDesc* desc;
};
__host__ __device__ __forceinline__ size_t chunk_ws_bytes(int D) {
  return kChunkWsRows * (D * sizeof(float) + sizeof(float2)) + kChunkMaxCtas * sizeof(ChunkDesc);
}
__host__ __device__ __forceinline__ ChunkWs chunk_ws(void* ws, int D) {
  ChunkWs w;
  w.o = reinterpret_cast<float*>(ws);
  w.ml = reinterpret_cast<float2*>(w.o + kChunkWsRows * D);
  w.desc = reinterpret_cast<ChunkDesc*>(w.ml + kChunkWsRows);
  return w;
}

// 3-D map over a cache seen as [token rows, Hkv, D]: boxes of `cols` values of
// one head of `rows` tokens, swizzled over 128 or 64 bytes or (0) not at all.
inline bool chunk_cache_map(CUtensorMap* m, const void* base, const ChunkArgs& a, bool fp8, int cols, int rows,
                            int swizzle) {
  umma::EncodeTiledFn fn = umma::encode_fn();
  if (!fn) return false;
  const cuuint64_t e = fp8 ? 1 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages * kPageTokens};
  const cuuint64_t strides[2] = {(cuuint64_t)a.D * e, (cuuint64_t)a.D * a.Hkv * e};
  const cuuint32_t box[3] = {(cuuint32_t)cols, 1u, (cuuint32_t)rows};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                           : swizzle == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace qsa
