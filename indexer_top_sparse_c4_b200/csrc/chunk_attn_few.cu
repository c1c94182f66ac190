// chunk_attn_few.cu -- the chunk attention for requests of a few query rows
// (decode steps, drafts): BF16 queries over a BF16 or FP8 E4M3 paged cache.
//
// With up to 16 query rows per KV head a call reads each key and value for 2
// to 32 multiply-adds per byte, so it is bound by the cache read, and the work
// per byte on the SM decides whether the read runs at full rate.  The products
// are taken transposed, S^T = K Q^T and O^T += V^T P^T, as 16 x 8 x 16 register
// products (mma.sync): the keys or head dimensions fill the 16 rows and 8 or
// 16 query rows the columns, so little of a product is padding, keys and
// values go from shared memory through registers once, and FP8 codes are
// widened there (e4m3 is a subset of FP16) without a second trip through
// shared memory.  The wide tcgen05 tiles spend shared-memory traffic on
// widened copies and on rows that do not exist: 211 us where this kernel takes
// 91 (8 x 65,000 tokens, 16/2 heads of D 256, FP8).
//
// Measured, 8 x 262,144 tokens, FP8: 316 us, 6.8 TB/s, 1.04 of what a plain copy
// reaches.  What a warp issues counts as much as what memory gives: per SM
// sub-partition a product takes 8 cycles, a conversion of two codes 2 (4 for the
// upper two of a word), a byte permutation 2; a clock read and two votes less
// per step took the call from 365 us to 325, and under the power limit, at 1.75
// GHz, copies issued under elect.sync and shorter softmax steps from 375 to 342.
// BF16 at D 256: 165 us for 8 x 65,000 tokens, 0.98 of the copy rate.
//
//  * registers: up to 255 a thread; at 16 rows the D 256 forms spill (FP8 72 bytes
//    stored, BF16 4), the others nothing.
//  * every warp works on its own: it takes every W-th step of 16 keys of the
//    CTA's piece, loads keys and values by TMA into its own ring (one lane
//    issues, an mbarrier per slot, the next piece's first steps behind this
//    one's last), and keeps its own softmax state and O^T in registers; nothing
//    in the loop waits for another warp.
//  * accumulator layouts: S^T and O^T both have the query rows in columns
//    2 (lane % 4) and the next, so maxima, sums and rescaling are per thread;
//    P^T becomes the B operand of the second product by one 8 x 8 transpose
//    (movmatrix) per fragment.  The order of the contraction over head
//    dimensions and of O^T's rows is free: FP8 fragments take the four
//    consecutive dimensions that a thread's 32-bit word holds.
//  * the softmax reference moves (and O^T is rescaled) only when a logit has
//    outgrown it by 2^8; for an FP8 cache P is kept 2^7 larger, so that small
//    probabilities stay in FP16's normal range down to 2^-21 of the largest
//    (smaller ones are rounded by 2^-32 of the largest).
//  * the warps' results are merged in shared memory at the end of a piece, the
//    pieces of a tile by the combine kernel, both in a fixed order.
//  * FP8 queries: see the power-of-two row scale of chunk_attn_tc.cu.
//  * steps with keys that some row does not see ("edge" steps): a zero
//    probability does not silence NaN or infinity, so non-finite values and
//    those past the last token are cleared in registers; what a row does see
//    is added back to its output.
#include "chunk_common.cuh"
#include "umma.cuh"

namespace qsa {
namespace {

using namespace mbar;

constexpr float kGrow = 8.f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kStep = 16;  // keys of a step
constexpr int kLead = 4;   // what a tile costs beside its blocks of 64 keys, in blocks

template <int D, bool FP8, int NT>
struct FewCfg {
  static constexpr int E = FP8 ? 1 : 2;
  static constexpr int RB = D * E < 128 ? D * E : 128;   // bytes of a box row
  static constexpr int kBoxes = D * E / RB;
  static constexpr int kSlot = kStep * D * E;            // a step's keys, or its values
  // Warps: four for BF16 at D 256 (six: 176 instead of 167 us for 8 x 65,000
  // tokens); twelve where a step's codes are few and its fixed part weighs
  // (FP8 at D 128: 56 us, eight 61); else eight (twelve at D 256 FP8: 332 instead
  // of 342 us for 8 x 262,144 tokens when power holds the clock down, but 48.4
  // instead of 46.7 for 64 x 3,000).
  static constexpr int W = kSlot >= 8192 ? 4 : FP8 && D <= 128 && NT == 1 ? 12 : 8;
  // 96 KB of rings, twice what 6.5 TB/s keep in flight.  More is slower, as if
  // memory served fewer streams better: 8 x 262,144 tokens FP8 316 us with 96
  // KB, 330 with 128 or 160, 327 with 64; 8 x 65,000 BF16 165, 173, 180, 171.
  static constexpr int kRing = 96 * 1024;
  static constexpr int S = kRing / (W * kSlot) < 8 ? kRing / (W * kSlot) : 8;
};

template <int D, bool FP8, int NT>
struct FewSmem {
  using C = FewCfg<D, FP8, NT>;
  alignas(1024) unsigned char ring[C::W][C::S][C::kSlot];
  float merge[C::W / 2][NT * (D / 16) * 4][32];          // O^T fragments of half of the warps
  float2 ml[C::W][NT * 8];
  float2 row[NT * 8];                                    // maximum and sum over the warps
  alignas(8) uint64_t full[C::W][C::S];
  int poison[2], abort_flag;   // poison: by piece
  ChunkSched sched;
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(saddr(dst)), "l"(map), "r"(saddr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same onto zero
template <bool F16>
__device__ __forceinline__ void mma16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t widen(uint32_t codes) {  // two e4m3 codes (low 16 bits) to FP16
  uint32_t r;
  asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(r) : "r"(codes));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t nonfinite16(uint32_t w) {  // mask of the non-finite halves of w
  constexpr uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  return ((w & e) == e ? 0xffffu : 0u) | ((w & (e << 16)) == (e << 16) ? 0xffff0000u : 0u);
}

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(FewCfg<D, FP8, NT>::W * 32, 1)
    chunk_few_kernel(ChunkArgs a, ChunkWs ws, float qk_scale_log2, float vmul, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v) {
  using C = FewCfg<D, FP8, NT>;
  constexpr int W = C::W, S = C::S, MT = D / 16, kRows = 8 * NT;
  constexpr float kShift = FP8 ? 7.f : 0.f;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  FewSmem<D, FP8, NT>& sm =
      *reinterpret_cast<FewSmem<D, FP8, NT>*>(smem_raw + ((1024 - ((uintptr_t)smem_raw & 1023)) & 1023));
  // the warp number by shuffle: the compiler then knows it, and what follows
  // from it, as the same in all lanes
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31, lr = lane >> 2, lc = lane & 3;
  volatile int* abort_flag = &sm.abort_flag;
  const int G = a.Hq / a.Hkv, TPT = kRows / G;
  constexpr int KT = kPageTokens;
  const uint32_t g_inv = 65536u / G + 1;   // x / G = x * g_inv >> 16 for a tile's rows

  if (threadIdx.x == 0) {
    for (int w = 0; w < W; ++w)
      for (int s = 0; s < S; ++s) mbar_init(&sm.full[w][s], 1);
    sm.abort_flag = 0;
    sm.poison[0] = sm.poison[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) ws.desc[blockIdx.x].n_parts = 0;
  chunk_sched_build(a, sm.sched, TPT, KT, blockIdx.x, gridDim.x, true, kLead);

  // Keys this tile's last row sees, and the steps of a piece that hold any.
  auto steps_of = [&](const ChunkItem& x) {
    const int seen = min(x.p0 + x.ntok, x.kv) - x.blk_lo * KT;
    return max(0, min((x.blk_hi - x.blk_lo) * (KT / kStep), (seen + kStep - 1) / kStep));
  };

  // ---- the load stream: K and V of this warp's steps, piece after piece
  ChunkWalk lwalk;
  lwalk.begin(a, sm.sched, blockIdx.x, gridDim.x);
  ChunkWalk walk = lwalk;
  ChunkItem lit;
  int ls = 0, lns = 0, lwin = -1, lpage = 0, ly = 0;
  uint32_t issued = 0, badmask = 0;   // slots armed; by slot: a bad page
  uint32_t islot = 0;
  bool lk = true, more = true, dead = false;       // dead: a wait has given up
  auto next_piece = [&]() {
    do {
      more = lwalk.next(a, sm.sched, TPT, KT, lit);
      if (!more) return;
      ls = warp, lns = steps_of(lit), lwin = -1;
    } while (ls >= lns);
  };
  auto issue = [&]() {
    if (!more || dead) return;
    if (lk) {
      const int lp = lit.blk_lo + ls / (KT / kStep);
      if (lwin < 0 || lp - lwin >= 32) {
        lwin = lp;
        const int n_pages = (lit.kv + kPageTokens - 1) / kPageTokens;
        lpage = 0;
        if (lp + lane < min(n_pages, lit.blk_hi)) {
          lpage = __ldg(a.page_table + (size_t)lit.b * a.pt_stride + lp + lane);
          if (lpage < 0 || lpage >= a.num_pages) {
            flag(a.status, QSA_DEV_BAD_PAGE);
            lpage = -1;
          }
        }
      }
      const int page = __shfl_sync(0xffffffffu, lpage, lp - lwin);
      // a bad page reads the rows behind the cache: zeros
      ly = page < 0 ? -1 : page * kPageTokens + (ls % (KT / kStep)) * kStep;
    }
    badmask = (badmask & ~(1u << islot)) | ((ly < 0 ? 1u : 0u) << islot);
    if (elect_one()) {
      mbar_arrive_tx(&sm.full[warp][islot], C::kSlot);
      const int y = ly < 0 ? a.num_pages * kPageTokens : ly;
#pragma unroll
      for (int b = 0; b < C::kBoxes; ++b)
        tma_load_3d(sm.ring[warp][islot] + b * (kStep * C::RB), lk ? &map_k : &map_v, &sm.full[warp][islot],
                    b * (C::RB / C::E), lit.kvh, y);
    }
    __syncwarp();
    ++issued;
    if (++islot == S) islot = 0;
    lk = !lk;
    if (lk) {
      ls += W;
      if (ls >= lns) next_piece();
    }
  };
  next_piece();
  for (int i = 0; i < S; ++i) issue();

  // ---- the pieces
  ChunkItem it;
  uint32_t slot = 0, phase = 0, parity = 0;
  auto wait_slot = [&]() {
    // One look first: reading the clock for a bounded wait costs more than most
    // waits of an FP8 cache (8 x 262,144 tokens at D 256: 325 us, 365 without).
    // BF16 waits for memory nearly always.
    if (FP8 && __all_sync(0xffffffffu, mbar_test(&sm.full[warp][slot], phase))) return;
    dead = dead || !__all_sync(0xffffffffu, !*abort_flag && mbar_wait(&sm.full[warp][slot], phase, abort_flag, a.status));
  };
  auto release = [&]() {
    __syncwarp();
    if (++slot == S) slot = 0, phase ^= 1;
    issue();
  };
  // This lane's row in a fragment load: matrices (keys 0-7, 8-15) x (chunk,
  // chunk + 1), chunk even.  Chunk c of key k lies at c ^ swizzle(k) of its
  // row, so a lane's addresses differ by an exclusive or and the box.
  const int fkey = (lane & 7) + ((lane >> 3) & 1) * 8;
  const int fsw = C::RB == 128 ? fkey & 7 : (fkey >> 1) & 3;
  const uint32_t flane = fkey * C::RB + (((lane >> 4) ^ fsw) << 4);
  auto frag_addr = [&](uint32_t base, int chunk) {
    constexpr int CPB = C::RB / 16;
    return ((base + flane) ^ ((chunk % CPB) << 4)) + (chunk / CPB) * (kStep * C::RB);
  };

  while (walk.next(a, sm.sched, TPT, KT, it)) {
    const int ns = steps_of(it), rows = it.ntok * G;
    const int lim0 = max(0, min(it.p0 + 1, it.kv));  // keys every row sees
    // Q as B operand: row n = lr + 8 nt
    uint32_t qf[NT][MT][2];
    float sc[NT][2], m[NT][2], l[NT][2];
    float neg[NT][2], top[NT][2];                    // -m (0 while m is -infinity), and what a logit may reach
    int lim[NT][2];
    float o[NT][MT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = lr + 8 * nt;
      const bool live = r < rows;
      const __nv_bfloat16* qrow = reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                  ((size_t)(it.t0 + (live ? r / G : 0)) * a.Hq + it.kvh * G + (live ? r % G : 0)) * D;
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        if constexpr (FP8) {                         // dimensions 16 k + 4 lc .. + 3
          const uint2 v = live ? *reinterpret_cast<const uint2*>(qrow + 16 * k + 4 * lc) : make_uint2(0, 0);
          qf[nt][k][0] = v.x, qf[nt][k][1] = v.y;
        } else {                                     // 16 k + 2 lc, + 1 and 8 further
          qf[nt][k][0] = live ? *reinterpret_cast<const uint32_t*>(qrow + 16 * k + 2 * lc) : 0u;
          qf[nt][k][1] = live ? *reinterpret_cast<const uint32_t*>(qrow + 16 * k + 8 + 2 * lc) : 0u;
        }
      }
      float undo = 1.f;
      if constexpr (FP8) {
        uint32_t top = 11u;                          // the row's largest exponent field
#pragma unroll
        for (int k = 0; k < MT; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) top = max(top, max((qf[nt][k][j] >> 7) & 0xffu, (qf[nt][k][j] >> 23) & 0xffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = min(top, 254u);
        const float up = __uint_as_float((264u - top) << 23);      // the largest lands in 2^10 .. 2^11
#pragma unroll
        for (int k = 0; k < MT; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w = qf[nt][k][j];
            qf[nt][k][j] = pack16<true>(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
          }
        undo = __uint_as_float((top - 10u) << 23);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {                  // rows 2 lc + j of the accumulators
        const int rr = 2 * lc + j + 8 * nt;
        // FP8: never 0, 0 x -inf would be NaN where the logit is 0
        sc[nt][j] = FP8 ? fmaxf(qk_scale_log2 * __shfl_sync(0xffffffffu, undo, (2 * lc + j) * 4), 1.2e-38f) : qk_scale_log2;
        lim[nt][j] = rr < rows ? min(it.p0 + rr / G + 1, it.kv) : it.kv;
        m[nt][j] = -INFINITY, l[nt][j] = 0.f;
        neg[nt][j] = 0.f, top[nt][j] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
    }

    for (int s = warp; s < ns; s += W) {
      const int key0 = it.blk_lo * KT + s * kStep;
      const bool edge = key0 + kStep > lim0;
      // ---- S^T = K Q^T, CH chains of products each
      constexpr int CH = 2;
      float sx[NT][CH][4];
      wait_slot();
      const bool bad = (badmask >> slot) & 1;
      {
        const uint32_t base = saddr(sm.ring[warp][slot]);
#pragma unroll
        for (int k = 0; k < MT; k += FP8 ? 2 : 1) {
          uint32_t r[4];
          ldm4(r, frag_addr(base, FP8 ? k : 2 * k));
          if constexpr (FP8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t x = r[2 * h], y = r[2 * h + 1];
              const uint32_t a0 = widen(x), a1 = widen(y), a2 = widen(x >> 16), a3 = widen(y >> 16);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (k + h < CH) mma16816_zero<true>(sx[nt][(k + h) % CH], a0, a1, a2, a3, qf[nt][k + h][0], qf[nt][k + h][1]);
                else mma16816<true>(sx[nt][(k + h) % CH], a0, a1, a2, a3, qf[nt][k + h][0], qf[nt][k + h][1]);
              }
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (k < CH) mma16816_zero<false>(sx[nt][k % CH], r[0], r[1], r[2], r[3], qf[nt][k][0], qf[nt][k][1]);
              else mma16816<false>(sx[nt][k % CH], r[0], r[1], r[2], r[3], qf[nt][k][0], qf[nt][k][1]);
            }
          }
        }
      }
      release();
      // ---- softmax: this thread holds keys key0 + lr and + 8 of rows 2 lc, 2 lc + 1
      uint32_t pf[NT][2];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x = sx[nt][0][j];
#pragma unroll
          for (int c = 1; c < CH; ++c) x += sx[nt][c][j];
          x *= sc[nt][j & 1];
          if (edge || bad) {
            if (bad || key0 + lr + (j >> 1) * 8 >= lim[nt][j & 1]) x = -INFINITY;
          }
          sx[nt][0][j] = x;
          grow = grow || x > top[nt][j & 1];
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = fmaxf(sx[nt][0][j], sx[nt][0][j + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m[nt][j], mx - kShift);
            const float alpha = m[nt][j] == mn ? 1.f : ex2(m[nt][j] - mn);
            m[nt][j] = mn;
            l[nt][j] *= alpha;
            neg[nt][j] = mn == -INFINITY ? 0.f : -mn;
            top[nt][j] = mn + (kGrow + kShift);
#pragma unroll
            for (int i = 0; i < MT; ++i) o[nt][i][j] *= alpha, o[nt][i][j + 2] *= alpha;
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p[j] = ex2(sx[nt][0][j] + neg[nt][j & 1]);
          l[nt][j & 1] += p[j];
        }
        pf[nt][0] = transpose8(pack16<FP8>(p[0], p[1]));
        pf[nt][1] = transpose8(pack16<FP8>(p[2], p[3]));
      }
      // ---- O^T += V^T P^T
      wait_slot();
      const uint32_t base = saddr(sm.ring[warp][slot]);
      const int kleft = it.kv - key0 - 2 * lc;       // keys 2 lc, + 1 (and 8 further) of the step below kv
      auto pv = [&](auto edge_tag) {
        constexpr bool EDGE = decltype(edge_tag)::value;
        bool odd = false;
        auto clean = [&](uint32_t x, int off) {      // keys 2 lc + off, + 1
          if constexpr (EDGE) {
            const uint32_t past = (kleft <= off ? 0xffffu : 0u) | (kleft <= off + 1 ? 0xffff0000u : 0u);
            x &= ~past;
            const uint32_t nf = nonfinite16<FP8>(x);
            odd = odd || nf;
            x &= ~nf;
          }
          return x;
        };
#pragma unroll
        for (int i = 0; i < MT; i += FP8 ? 2 : 1) {
          uint32_t r[4];
          ldm4t(r, frag_addr(base, FP8 ? i : 2 * i));
          if constexpr (FP8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // bytes (key, dim), (key, dim + 1), (key + 1, dim), (key + 1, dim + 1): pair the keys
              const uint32_t x = __byte_perm(r[2 * h], 0, 0x3120), y = __byte_perm(r[2 * h + 1], 0, 0x3120);
              const uint32_t a0 = clean(widen(x), 0), a1 = clean(widen(x >> 16), 0);
              const uint32_t a2 = clean(widen(y), 8), a3 = clean(widen(y >> 16), 8);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<true>(o[nt][i + h], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
            }
          } else {
            const uint32_t a0 = clean(r[0], 0), a1 = clean(r[2], 0), a2 = clean(r[1], 8), a3 = clean(r[3], 8);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<false>(o[nt][i], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
          }
        }
        if (EDGE && odd) sm.poison[parity] = 1;
      };
      if (edge) pv(std::true_type{});
      else pv(std::false_type{});
      release();
    }

    // ---- merge of the warps, output of the piece
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], d);
        if (lane < 4) sm.ml[warp][nt * 8 + 2 * lc + j] = make_float2(m[nt][j], l[nt][j]);
      }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) mx = fmaxf(mx, sm.ml[w][nt * 8 + 2 * lc + j].x);
        const float f = m[nt][j] == mx ? 1.f : ex2(m[nt][j] - mx);
#pragma unroll
        for (int i = 0; i < MT; ++i) o[nt][i][j] *= f, o[nt][i][j + 2] *= f;
      }
    if (threadIdx.x < kRows) {
      float mx = -INFINITY, total = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) mx = fmaxf(mx, sm.ml[w][threadIdx.x].x);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 v = sm.ml[w][threadIdx.x];
        total += v.x == mx ? v.y : v.y * ex2(v.x - mx);
      }
      sm.row[threadIdx.x] = make_float2(mx, total);
    }
    if (warp >= W / 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) sm.merge[warp - W / 2][(nt * MT + i) * 4 + j][lane] = o[nt][i][j];
    }
    __syncthreads();
    if (warp < W / 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) sm.merge[warp][(nt * MT + i) * 4 + j][lane] += o[nt][i][j];
    }
    __syncthreads();
    const bool poison = sm.poison[parity] != 0;
    // adds the non-finite values of the edge steps that token tok sees
    auto seen_nonfinite = [&](int tok, int d, float (&y)[2]) {
      const int from = max(it.blk_lo * KT, lim0 / kStep * kStep);
      const int to = min(min(it.p0 + tok + 1, it.kv), it.blk_hi * KT);
      for (int t = from; t < to; ++t) {
        const int page = __ldg(a.page_table + (size_t)it.b * a.pt_stride + t / kPageTokens);
        if (page < 0 || page >= a.num_pages) continue;
        const size_t src = (((size_t)page * kPageTokens + t % kPageTokens) * a.Hkv + it.kvh) * D + d;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v;
          if constexpr (FP8) v = Elem<__nv_fp8_e4m3>::get(reinterpret_cast<const __nv_fp8_e4m3*>(a.v_pages), src + e);
          else v = Elem<__nv_bfloat16>::get(reinterpret_cast<const __nv_bfloat16*>(a.v_pages), src + e);
          if (!isfinite(v)) y[e] += v;
        }
      }
    };
    if (threadIdx.x == 0) sm.poison[parity ^ 1] = 0;   // last read a piece ago, set again behind this piece's last barrier
    // a thread keeps its pair of dimensions and walks over the rows
    constexpr int RP = W * 32 / (D / 2);
    const int d = (threadIdx.x % (D / 2)) * 2;
#pragma unroll 8
    for (int n = threadIdx.x / (D / 2); n < kRows; n += RP) {
      if (n >= rows) break;
      const float mx = sm.row[n].x, total = sm.row[n].y;
      float y[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int q = FP8 ? (d & 15) >> 1 : (d & 7) + e, hi = FP8 ? e : (d >> 3) & 1;
        const int reg = ((n >> 3) * MT + (d >> 4)) * 4 + hi * 2 + (n & 1), ln = q * 4 + ((n & 7) >> 1);
        y[e] = 0.f;
#pragma unroll
        for (int w = 0; w < W / 2; ++w) y[e] += sm.merge[w][reg][ln];
      }
      const int tok = (int)((uint32_t)n * g_inv >> 16);
      if (total == 0.f) y[0] = y[1] = 0.f;
      else if (poison) seen_nonfinite(tok, d, y);
      if (it.part < 0) {
        const float inv = total == 0.f ? 0.f : vmul / total;
        const size_t row = (size_t)(it.t0 + tok) * a.Hq + it.kvh * G + (n - tok * G);
        *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(a.out) + row * D + d) =
            pack16<false>(y[0] * inv, y[1] * inv);
        if (d == 0 && a.lse) a.lse[row] = total == 0.f ? -INFINITY : mx * kLn2 + logf(total);
      } else {
        const size_t row = (size_t)it.part * kRows + n;
        *reinterpret_cast<float2*>(ws.o + row * D + d) = make_float2(y[0], y[1]);
        if (d == 0) ws.ml[row] = make_float2(mx, total);
      }
    }
    if (it.n_parts > 0 && threadIdx.x == 0) ws.desc[blockIdx.x] = ChunkDesc{it.n_parts, it.t0, it.ntok, it.kvh};
    __syncthreads();
    parity ^= 1;
  }
  if (*abort_flag && lane == 0)            // no copy may still be in flight when the CTA leaves
    for (uint32_t i = issued < S ? 0 : issued - S; i < issued; ++i) mbar_drain(&sm.full[warp][i % S], (i / S) & 1);
}

template <int D, bool FP8, int NT>
cudaError_t launch(const ChunkArgs& a, const ChunkWs& ws, int grid, float qk, float vmul, cudaStream_t s) {
  using C = FewCfg<D, FP8, NT>;
  CUtensorMap mk, mv;
  constexpr int sw = C::RB == 128 ? 128 : 64;
  if (!chunk_cache_map(&mk, a.k_pages, a, FP8, C::RB / C::E, kStep, sw) ||
      !chunk_cache_map(&mv, a.v_pages, a, FP8, C::RB / C::E, kStep, sw))
    return cudaErrorInvalidValue;
  auto kern = chunk_few_kernel<D, FP8, NT>;
  constexpr size_t smem = sizeof(FewSmem<D, FP8, NT>) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(grid), dim3(C::W * 32), smem, s, 1, a, ws, qk, vmul, mk, mv);
}
template <int D, bool FP8>
cudaError_t launch_nt(const ChunkArgs& a, const ChunkWs& ws, int rows, int grid, float qk, float vmul, cudaStream_t s) {
  return rows == 8 ? launch<D, FP8, 1>(a, ws, grid, qk, vmul, s) : launch<D, FP8, 2>(a, ws, grid, qk, vmul, s);
}
template <int D>
cudaError_t launch_kv(const ChunkArgs& a, const ChunkWs& ws, int rows, int grid, float qk, float vmul, cudaStream_t s) {
  return a.kv_dt == QSA_FP8_E4M3 ? launch_nt<D, true>(a, ws, rows, grid, qk, vmul, s)
                                 : launch_nt<D, false>(a, ws, rows, grid, qk, vmul, s);
}

}  // namespace

// rows: query rows of a tile, 8 or 16
cudaError_t launch_chunk_attn_few(const ChunkArgs& a, const ChunkWs& ws, int rows, int grid, float qk, float vmul,
                                  cudaStream_t s) {
  switch (a.D) {
    case 64: return launch_kv<64>(a, ws, rows, grid, qk, vmul, s);
    case 128: return launch_kv<128>(a, ws, rows, grid, qk, vmul, s);
    default: return launch_kv<256>(a, ws, rows, grid, qk, vmul, s);
  }
}

}  // namespace qsa
