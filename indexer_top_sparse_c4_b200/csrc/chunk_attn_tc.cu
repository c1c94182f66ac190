// chunk_attn_tc.cu -- the chunk attention on the 5th-generation tensor cores:
// BF16 queries over a BF16 or FP8 E4M3 paged cache, drafts to whole prompts
// (requests of a few rows: chunk_attn_few.cu).
//
//   S = Q K^T (FP32),  P = exp2(scale log2(e) S - m),  O += P V,  l += sum P
//
// with m a running reference of the row's maximum.  All P, l and O of a row
// share one reference, so the result O / l does not depend on it; it is moved
// (and O, l rescaled) only when the maximum has grown by more than 2^8 over
// it, which keeps P in range of its 16-bit type and leaves O in TMEM alone in
// almost every step.
//
// sm_100a design, a persistent pair of CTAs (cluster of 2, cta_group::2) per two
// SMs:
//  * tile: M = 256 query rows (128 TMEM lanes in each CTA) x N = 128 keys (two
//    pages).  The rows are whole tokens: all G = Hq / Hkv query heads of a KV
//    head, so a key or value read once serves 256 / G tokens x G heads.
//  * each CTA stages half of the B operands: one page of keys (64 of the 128
//    columns of S) and half of the head's value columns.  A single CTA per tile
//    would pull 128 KB from L2 for 2,048 cycles of products at D = 256 and read
//    320 KB of shared memory (2,560 cycles) for them; the pair halves the
//    first and needs 1,500 cycles for the second.
//  * TMEM (512 columns): O in columns 0 .. D-1, two S tiles of 128 columns; P
//    overwrites its S tile (16-bit, half the columns) and is the A operand of
//    P V straight from TMEM.
//  * keys and values stream through one ring of stages (a K or V half tile
//    each; 32 KB at D = 256), in the order K0, K1, V0, K2, V1, ...: S of the
//    next tile is computed while the softmax of this one runs.  V is the
//    MN-major B operand, D columns in one product: products of 64 columns take
//    52 cycles instead of 32 (measured), those of 256 columns 131 of 128.
//  * warp 0 issues the CTA's TMA loads (boxes of one page x 64 columns, pages
//    looked up 32 at a time), warp 1 of the first CTA the MMAs of both; warps
//    4..11 do the softmax of the CTA's rows (two warps per TMEM lane quarter,
//    64 keys each), and warps 2 and 3 bring the next item's queries by cp.async.
//  * FP8 cache: boxes of codes land in a second ring, and warps 12..15 turn
//    them into FP16 stages (e4m3 is a subset of FP16, the product P V then
//    takes P in FP16).  The query is FP16 too: each row is scaled by a power
//    of two that puts its largest value at 2^10 .. 2^11, which keeps all bits
//    of every BF16 value down to 2^-24 of the row's largest; the scale is
//    undone in FP32 with the softmax scale.
//  * tiles that hold keys some row must not see ("edge" tiles: the causal
//    diagonal, the last page): masked P is 0, but 0 x NaN is NaN in the matrix
//    product, so the softmax warps first clear the value rows past the last
//    token and any non-finite value of the tile from its V stage.  Non-finite
//    values that a row does see are added back to its output at the end (the
//    `poison` flag; the sum is then non-finite whatever its weight).
//  * few tiles: the (tile, key block) space is divided evenly over the pairs and
//    a combine kernel merges shared tiles; many tiles: one pair per tile.
//  * every wait is bounded (mbarrier.cuh); after a time-out the warps finish
//    their loops without waiting, in-flight copies and MMAs are drained, and
//    TMEM is released.
//
// Measured (24/2 heads of D 256, BF16, 8,192 tokens behind 57,344): 9.3 ms,
// 1,330 TFLOP/s, 0.97 of what cuBLAS sustains under the power limit; 1,467
// TFLOP/s behind 24,576 tokens.  FP8 there: 1,267.  Bound by the tensor cores at
// D 256 (2,130 cycles a tile when fed, measured); at D 128 and 64 (858 and 437
// TFLOP/s, about 2,700 cycles a tile at both) by the chain of one tile's softmax:
// wait, TMEM load, maximum, exchange, exponentials, TMEM store, which all warps
// walk in step.  The 128 x 128 exponentials are 1,024 of those cycles, the
// products 1,065 (D 128) or 530, so neither unit is full.  Two groups of warps
// that take whole tiles in turn were 5 to 9% faster there and 5% slower at
// D 256.  Short items cost what surrounds them: about 8 us from the launch to
// the first product (schedule, page lookups, queries, first keys), 3 us for an
// item's output.  The compiler spills in every form (BF16 272 to 316 bytes
// stored, FP8 340 to 448): it allots the launch's 168 or 128 registers to all
// roles, whatever setmaxnreg gives the softmax warps later.
#include <cuda.h>

#include "chunk_common.cuh"
#include "umma.cuh"

namespace qsa {
namespace {

using namespace mbar;

constexpr int kRows = 128;               // rows of a CTA, half of a tile
constexpr int kKeys = 128;               // keys of a tile: two pages
constexpr uint32_t kSCol = 256;          // first TMEM column of the S tiles
constexpr uint32_t kTmemCols = 512;
constexpr int kSoftWarps = 8;
constexpr int kLead = 4;                 // what a tile costs beside its blocks, in blocks
constexpr float kGrow = 8.f;             // log2 of how far P may grow before O is rescaled
constexpr float kLn2 = 0.69314718055994530942f;

template <int D, bool FP8>
struct Cfg {
  static constexpr int DB = D / 64;                    // 64-column blocks of a key half: 64 rows of 128 bytes each
  static constexpr int VB = D >= 128 ? D / 128 : 1;    // column blocks of a value half: 128 rows of VR bytes each
  static constexpr int VR = D >= 128 ? 128 : 64;
  static constexpr int kStage = 64 * D * 2;            // a key half or a value half, 16-bit
  static constexpr int kRaw = 64 * D;                  // the same in codes
  static constexpr int kQBytes = DB * kRows * 128;
  // Q and the rings take up to 208 KB
  static constexpr int kStages = FP8 ? (D == 256 ? 3 : 6) : (D == 256 ? 4 : 8);
  static constexpr int kRaws = FP8 ? (D == 256 ? 2 : 6) : 0;
  static constexpr int kThreads = FP8 ? 512 : 384;
  // registers after the split: loads and MMA, softmax, conversion (their sum is within the launch's 3 x 168 or 4 x 128)
  static constexpr int kRegLow = FP8 ? 64 : 72, kRegSoft = FP8 ? 184 : 216, kRegConv = 80;
};

template <int D, bool FP8>
struct TcSmem {
  using C = Cfg<D, FP8>;
  alignas(1024) unsigned char q[C::kQBytes];
  alignas(1024) unsigned char stage[C::kStages][C::kStage];
  alignas(1024) unsigned char raw[C::kRaws ? C::kRaws : 1][C::kRaws ? C::kRaw : 16];
  // Waited for by the first CTA's MMA warp, arrived at from both CTAs: full,
  // q_full, p_full, o_free.  Signalled in both CTAs by the MMA warp: the others
  // but raw_*, which are the CTA's own.
  // s_full, p_full and pv_done count tiles, one of each two: a waiter is never
  // more than one phase ahead of a barrier, so a phase's parity names it.
  alignas(8) uint64_t full[C::kStages], empty[C::kStages];
  uint64_t raw_full[C::kRaws ? C::kRaws : 1], raw_empty[C::kRaws ? C::kRaws : 1];
  uint64_t q_full, q_empty, s_full[2], p_full[2], pv_done[2], o_free, v_ready, drain;
  float mx[2][2][kRows];                 // [tile parity][half][row] maxima
  float lx[2][2][kRows];                 // [item parity][half][row] sums
  float q_scale[2][kRows];               // FP8, by item parity: what undoes the row's power of two
  alignas(16) unsigned char out[kSoftWarps][32 * 64];   // 64 bytes of a warp's 32 output rows
  int poison[4];                         // by item, modulo 4
  uint32_t tmem_base;
  int abort_flag;
  ChunkSched sched;
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(saddr(dst)), "l"(map), "r"(saddr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// The same, signalling the barrier at the same place of the pair's first CTA.
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(saddr(dst)), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Addresses in the pair's CTAs, arrivals there.  (The arrivals release at CTA
// scope: what they publish lies in TMEM, ordered by tcgen05 fences, or in the
// CTA's own shared memory; a release at cluster scope waits some 1,000 cycles.)
__device__ __forceinline__ uint32_t map_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A and B in shared memory / A in TMEM
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
// Arrives on the barrier at this place in both CTAs once the MMAs issued before are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(saddr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// MN-major operand of rows of VR bytes: 8-row atoms, column blocks 128 rows apart
template <int VR>
__device__ __forceinline__ uint64_t v_desc(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFF);
  d |= (uint64_t)((128 * VR) >> 4) << 16;        // to the next column block
  d |= (uint64_t)((8 * VR) >> 4) << 32;          // to the next 8 keys
  d |= (uint64_t)1 << 46;                        // version
  d |= (uint64_t)(VR == 128 ? 2 : 4) << 61;      // swizzle over 128 or 64 bytes
  return d;
}
// kind::f16 instruction descriptor: F32 accumulators, M = 256; f16 or bf16
// operands; B K-major (keys of S) or MN-major (values)
constexpr uint32_t idesc(bool f16, int N, bool b_mn) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(2 * kRows >> 4) << 24);
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]),
      "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]),
      "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]),
      "r"(u[27]), "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// two FP32 operations an instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t x, y, z, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t x, y, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool FP8>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (FP8) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A bounded wait that gives up at once when the CTA is stopping.  The first
// look is the cheap one: a wait with a time limit costs some 200 cycles more.
__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
  if (mbar_test(b, parity)) return true;
  if (*abort_flag) return false;
  return mbar_wait(b, parity, abort_flag, status);
}
// A wait by a whole warp, which is converged on return (the TMEM loads and
// stores that follow need it).
__device__ __forceinline__ bool wait_warp(uint64_t* b, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
  return __all_sync(0xffffffffu, wait(b, parity, abort_flag, status));
}

// The physical token row of logical page lp of a request, or the first row
// past the cache (TMA then fills zeros) when no token needs it or it is bad.
__device__ __forceinline__ int page_row(const ChunkArgs& a, const int32_t* pt, int lp, int n_pages, bool report) {
  if (lp >= n_pages) return a.num_pages * kPageTokens;
  const int page = __ldg(pt + lp);
  if (page < 0 || page >= a.num_pages) {
    if (report) flag(a.status, QSA_DEV_BAD_PAGE);
    return a.num_pages * kPageTokens;
  }
  return page * kPageTokens;
}

template <bool FP8>
__device__ __forceinline__ uint32_t nonfinite16(uint32_t w) {  // mask of the non-finite halves of w
  constexpr uint32_t e = FP8 ? 0x7c00u : 0x7f80u;
  return ((w & e) == e ? 0xffffu : 0u) | ((w & (e << 16)) == (e << 16) ? 0xffff0000u : 0u);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads, 1)
    chunk_tc_kernel(ChunkArgs a, ChunkWs ws, float qk_scale_log2, float vmul, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D, FP8>;
  constexpr int DB = C::DB;
  // FP16 P is kept 2^7 larger, so that small probabilities stay in the type's
  // normal range down to 2^-21 of the largest
  constexpr float kShift = FP8 ? 7.f : 0.f;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  TcSmem<D, FP8>& sm = *reinterpret_cast<TcSmem<D, FP8>*>(smem_raw + ((1024 - ((uintptr_t)smem_raw & 1023)) & 1023));
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: uniform
  volatile int* abort_flag = &sm.abort_flag;
  const int G = a.Hq / a.Hkv, TPT = 2 * kRows / G;
  const uint32_t rank = cluster_rank();
  const int worker = blockIdx.x >> 1, workers = gridDim.x >> 1;
  const uint32_t g_inv = 65536u / G + 1;   // x / G = x * g_inv >> 16 for a tile's rows x < 256

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sm.full[s], FP8 ? 8 : 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < C::kRaws; ++s) {
      mbar_init(&sm.raw_full[s], 1);
      mbar_init(&sm.raw_empty[s], 4);
    }
    mbar_init(&sm.q_full, 4);
    mbar_init(&sm.q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.p_full[s], 2 * kSoftWarps);
      mbar_init(&sm.pv_done[s], 1);
    }
    mbar_init(&sm.o_free, 2 * kSoftWarps);
    mbar_init(&sm.v_ready, 1);
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    sm.poison[0] = sm.poison[1] = sm.poison[2] = sm.poison[3] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&sm.tmem_base)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0 && rank == 0) ws.desc[worker].n_parts = 0;
  chunk_sched_build(a, sm.sched, TPT, kKeys, worker, workers, false, kLead);
  tc_fence_before();
  __syncthreads();
  cluster_sync();          // the pair's barriers are initialised, its TMEM allocated
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  ChunkWalk walk;
  walk.begin(a, sm.sched, worker, workers);
  ChunkItem it;
  uint32_t s = 0, phase = 0;   // ring position of the loading, issuing and converting warps
  bool ok = true, issued = false;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegLow));
    if (warp == 0) {
      // ---------------- TMA producer: this CTA's halves ----------------
      constexpr int kRing = FP8 ? C::kRaws : C::kStages;
      constexpr uint32_t kBytes = FP8 ? C::kRaw : C::kStage;
      uint64_t* const empties = FP8 ? sm.raw_empty : sm.empty;
      // the cache rows of 32 pages of a piece, from its window w on
      auto pages = [&](const ChunkItem& x, int w) {
        const int lp0 = 2 * x.blk_lo;
        const int n_pages = min((x.kv + kPageTokens - 1) / kPageTokens, 2 * x.blk_hi);
        return page_row(a, a.page_table + (size_t)x.b * a.pt_stride, lp0 + 32 * w + lane, n_pages, rank == 0);
      };
      ChunkItem nx;
      bool have = walk.next(a, sm.sched, TPT, kKeys, it);
      int first = have ? pages(it, 0) : 0;
      for (; ok && have && !*abort_flag; it = nx) {
        const int n = it.blk_hi - it.blk_lo;
        int win = 0, cur = first, nxt = n > 16 ? pages(it, 1) : 0;
        // the next piece is found, and its pages, while this one streams
        have = walk.next(a, sm.sched, TPT, kKeys, nx);
        first = have ? pages(nx, 0) : 0;
        auto load = [&](bool key, int j) {
          const int x = 2 * j, from = (x >> 5) == win ? cur : nxt;
          const int y0 = __shfl_sync(0xffffffffu, from, x & 31), y1 = __shfl_sync(0xffffffffu, from, (x + 1) & 31);
          ok = wait_warp(&empties[s], phase ^ 1, abort_flag, a.status);
          if (!ok) return;
          if (elect_one()) {
            uint64_t* const own = &sm.raw_full[FP8 ? s : 0];
            const uint32_t bar = map_cta(saddr(&sm.full[FP8 ? 0 : s]), 0);
            unsigned char* dst = FP8 ? sm.raw[s] : sm.stage[s];
            if (FP8) mbar_arrive_tx(own, kBytes);
            else if (rank == 0) mbar_arrive_tx(&sm.full[s], 2 * kBytes);   // both CTAs' bytes
            auto box = [&](uint32_t off, const CUtensorMap* map, int col, int y) {
              if constexpr (FP8) tma_load_3d(dst + off, map, own, col, it.kvh, y);
              else tma_load_3d_pair(dst + off, map, bar, col, it.kvh, y);
            };
            if (key) {        // page `rank` of the two, all columns
#pragma unroll
              for (int db = 0; db < DB; ++db) box(db * (kBytes / DB), &map_k, db * 64, rank ? y1 : y0);
            } else {          // half of the columns, both pages
#pragma unroll
              for (int vb = 0; vb < C::VB; ++vb) {
                const int col = (int)rank * (D / 2) + vb * 64;
                box(vb * (kBytes / C::VB), &map_v, col, y0);
                box(vb * (kBytes / C::VB) + kBytes / C::VB / 2, &map_v, col, y1);
              }
            }
          }
          __syncwarp();
          if (++s == kRing) s = 0, phase ^= 1;
        };
        load(true, 0);
        for (int j = 0; ok && j < n; ++j) {
          if (j + 1 < n) load(true, j + 1);
          if (ok) load(false, j);
          if (((2 * j + 2) >> 5) != win) {   // the next V tile lies in the next window
            ++win;
            cur = nxt;
            nxt = pages(it, win + 1);
          }
        }
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMA issuer of the pair ----------------
      constexpr uint32_t kIdS = idesc(FP8, kKeys, false), kIdO = idesc(FP8, D, true);
      const uint64_t qd = umma::smem_desc(saddr(sm.q));
      const uint32_t ready0 = map_cta(saddr(&sm.v_ready), 0), ready1 = map_cta(saddr(&sm.v_ready), 1);
      uint32_t g = 0, item = 0;
      auto step = [&]() { if (++s == C::kStages) s = 0, phase ^= 1; };
      auto qk = [&](uint32_t buf) {
        ok = ok && wait_warp(&sm.full[s], phase, abort_flag, a.status);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t kd = umma::smem_desc(saddr(sm.stage[s]));
#pragma unroll
          for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ss(tmem + kSCol + buf * kKeys, qd + (db * (kRows * 128) >> 4) + ks * 2,
                     kd + (db * (64 * 128) >> 4) + ks * 2, kIdS, (db | ks) != 0);
          commit_pair(&sm.s_full[buf]);
          commit_pair(&sm.empty[s]);
        }
        __syncwarp();
        issued = true;
        step();
      };
      ChunkItem nx;
      bool have = walk.next(a, sm.sched, TPT, kKeys, it);
      for (; ok && have && !*abort_flag; it = nx) {
        const int n = it.blk_hi - it.blk_lo;
        const int lim0 = min(it.p0 + 1, it.kv);
        ok = wait_warp(&sm.q_full, item & 1, abort_flag, a.status);
        if (ok) qk(g & 1);
        have = walk.next(a, sm.sched, TPT, kKeys, nx);
        for (int j = 0; ok && j < n; ++j) {
          const uint32_t buf = (g + j) & 1;
          if (j + 1 < n) qk(buf ^ 1);
          if (!ok) break;
          if (j + 2 >= n && (j + 1 < n || n == 1)) {   // after the last Q K^T
            if (elect_one()) commit_pair(&sm.q_empty);
            __syncwarp();
          }
          // the previous item's O has been read out before the first P V
          if (j == 0) ok = wait_warp(&sm.o_free, (item & 1) ^ 1, abort_flag, a.status);
          ok = ok && wait_warp(&sm.full[s], phase, abort_flag, a.status);
          if (ok && (it.blk_lo + j + 1) * kKeys > lim0) {   // edge tile: the softmax warps clear V first
            if (elect_one()) {
              arrive_at(ready0);
              arrive_at(ready1);
            }
            __syncwarp();
          }
          ok = ok && wait_warp(&sm.p_full[buf], ((g + j) >> 1) & 1, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t vd = v_desc<C::VR>(saddr(sm.stage[s]));
            const uint32_t p = tmem + kSCol + buf * kKeys;
            // 16 keys a step: 8 columns of P, 16 rows of V; keys 64.. of P start 64 columns on
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_ts(tmem, p + (ks >> 2) * 64 + (ks & 3) * 8, vd + ks * (16 * C::VR >> 4), kIdO, j != 0 || ks != 0);
            commit_pair(&sm.pv_done[buf]);
            commit_pair(&sm.empty[s]);
          }
          __syncwarp();
          issued = true;
          step();
        }
        g += n;
        ++item;
      }
    } else if (warp >= 2) {
      // ---------------- Q of the next item: this CTA's rows into shared memory ----------------
      // (128-byte swizzle, K-major; rows past the item's tokens keep what they
      // held, which reaches nothing but those rows)
      constexpr int CH = D / 8, RP = 64 / CH;          // 16-byte chunks of a row, rows of a pass of 64 threads
      const int lt = threadIdx.x - 64, c = lt % CH;
      const uint32_t q_full0 = map_cta(saddr(&sm.q_full), 0);
      const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q);
      unsigned char* const dst = sm.q + (c >> 3) * (kRows * 128);
      auto at = [&](int r) { return reinterpret_cast<uint4*>(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4)); };
      for (uint32_t item = 0; !*abort_flag && walk.next(a, sm.sched, TPT, kKeys, it); ++item) {
        const int rows = min(it.ntok * G - (int)rank * kRows, kRows);   // this CTA's
        const __nv_bfloat16* qi = q + ((size_t)it.t0 * a.Hq + it.kvh * G) * D + c * 8;
        if (!wait_warp(&sm.q_empty, (item & 1) ^ 1, abort_flag, a.status)) break;
        // all of it in flight at once
#pragma unroll 4
        for (int r = lt / CH; r < rows; r += RP) {
          const int tr = (int)rank * kRows + r, tok = (int)((uint32_t)tr * g_inv >> 16);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(saddr(at(r))),
                       "l"(qi + ((size_t)tok * a.Hq + (tr - tok * G)) * D)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if constexpr (FP8) {                           // to FP16 in place, each thread what it brought
          constexpr int NB = 4;                        // rows at a time
          for (int r0 = lt / CH; r0 < rows + lt / CH; r0 += NB * RP) {
            uint4 v[NB];
            __nv_bfloat162 top[NB];                    // the row's largest magnitude, of odd and even columns
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              const int r = r0 + k * RP;
              v[k] = r < rows ? *at(r) : make_uint4(0, 0, 0, 0);
              const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&v[k]);
              top[k] = __hmax2(__hmax2(__habs2(x[0]), __habs2(x[1])), __hmax2(__habs2(x[2]), __habs2(x[3])));
            }
#pragma unroll
            for (int x = 1; x < CH; x <<= 1)
#pragma unroll
              for (int k = 0; k < NB; ++k) top[k] = __hmax2(top[k], __shfl_xor_sync(0xffffffffu, top[k], x));
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              const int r = r0 + k * RP;
              const uint32_t t = *reinterpret_cast<const uint32_t*>(&top[k]);
              const uint32_t E = min(max(max((t >> 7) & 0xffu, (t >> 23) & 0xffu), 11u), 254u);
              const float up = __uint_as_float((264u - E) << 23);    // 2^(137 - E): the largest lands in 2^10 .. 2^11
              auto to16 = [&](uint32_t w) {
                return pack16<true>(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
              };
              if (r < rows) {
                *at(r) = make_uint4(to16(v[k].x), to16(v[k].y), to16(v[k].z), to16(v[k].w));
                if (c == 0) sm.q_scale[item & 1][r] = __uint_as_float((E - 10u) << 23);  // 2^(E - 137)
              }
            }
          }
        }
        async_fence();
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_at(q_full0);
      }
    }
  } else if (warp < 4 + kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegSoft));
    // ---------------- softmax, correction, epilogue ----------------
    const int st = threadIdx.x - 128;                  // 0 .. 255
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int row = 32 * quarter + lane;
    const uint32_t tlane = tmem + ((uint32_t)(32 * quarter) << 16);
    constexpr int OC = D / 2;                          // columns of O per thread
    const uint32_t o_free0 = map_cta(saddr(&sm.o_free), 0);
    const uint32_t p_full0 = map_cta(saddr(&sm.p_full[0]), 0);
    uint32_t g = 0, item = 0;                          // tiles, items so far
    uint32_t pos = 0, edges = 0;                       // ring stage of the item's first K; edge tiles so far

    const int trow = (int)rank * kRows + row, tok = (int)((uint32_t)trow * g_inv >> 16);
    ChunkItem nx;
    bool have = walk.next(a, sm.sched, TPT, kKeys, it);
    while (have) {
      const bool have_next = walk.next(a, sm.sched, TPT, kKeys, nx);   // before the first wait
      const int n = it.blk_hi - it.blk_lo, rows = it.ntok * G;
      float sc = qk_scale_log2;
      const bool live = trow < rows;                   // this thread's row is a query
      const bool warp_live = (int)rank * kRows + 32 * quarter < rows;
      const int lim = live ? min(it.p0 + tok + 1, it.kv) : 0;   // keys the row sees
      const int lim0 = min(it.p0 + 1, it.kv);          // keys the tile's first row sees (the fewest)
      const int n_pages = (it.kv + kPageTokens - 1) / kPageTokens;
      const int32_t* pt = a.page_table + (size_t)it.b * a.pt_stride;
      float m = -INFINITY, l = 0.f;
      // this half's page of the tile, and the next one's (looked at a tile later)
      auto page_of = [&](int lp) { return lp < n_pages ? __ldg(pt + lp) : -1; };
      int page = page_of(2 * it.blk_lo + half);
      for (int j = 0; j < n; ++j) {
        const uint32_t buf = (g + j) & 1;
        const int key0 = (it.blk_lo + j) * kKeys + half * 64;
        const int page_next = j + 1 < n ? page_of(2 * (it.blk_lo + j + 1) + half) : -1;
        wait_warp(&sm.s_full[buf], ((g + j) >> 1) & 1, abort_flag, a.status);
        tc_fence_after();
        // never 0: 0 x -inf would be NaN where the logit is 0
        if (FP8 && j == 0 && live) sc = fmaxf(qk_scale_log2 * sm.q_scale[item & 1][row], 1.2e-38f);
        if (warp_live) {
          float s[64];
          const uint32_t ta = tlane + kSCol + buf * kKeys + half * 64;
          tmem_ld32(ta, s);
          tmem_ld32(ta + 32, s + 32);
          tmem_wait_ld();
          const int seen = page >= 0 && page < a.num_pages ? lim - key0 : 0;
          if (__any_sync(0xffffffffu, seen < 64)) {
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = i < seen ? s[i] : -INFINITY;
          }
          float mc[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i < 64; ++i) mc[i & 3] = fmaxf(mc[i & 3], s[i]);
          float mx = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
          sm.mx[buf][half][row] = mx;
          bar_sync(1 + quarter, 64);
          mx = fmaxf(mx, sm.mx[buf][half ^ 1][row]) * sc;
          // move the reference where the maximum has outgrown it
          const bool grow = mx > m + (kGrow + kShift) || (m == -INFINITY && mx > m);
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = fmaxf(m, mx - kShift);
            const float alpha = m == mn ? 1.f : ex2(m - mn);
            m = mn;
            l *= alpha;
            if (j > 0) {
              wait_warp(&sm.pv_done[buf ^ 1], ((g + j - 1) >> 1) & 1, abort_flag, a.status);
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < OC; c += 32) {
                float o[32];
                tmem_ld32(tlane + half * OC + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= alpha;
                tmem_st32(tlane + half * OC + c, reinterpret_cast<uint32_t*>(o));
              }
            }
          }
          const float neg = m == -INFINITY ? 0.f : -m;
          uint32_t p[32];
          const float2 sc2 = make_float2(sc, sc), neg2 = make_float2(neg, neg);
          float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float2 x = fma2(make_float2(s[2 * i], s[2 * i + 1]), sc2, neg2);
            float2 y = fma2(make_float2(s[2 * i + 2], s[2 * i + 3]), sc2, neg2);
            x.x = ex2(x.x), x.y = ex2(x.y), y.x = ex2(y.x), y.y = ex2(y.y);
            sum0 = add2(sum0, x);
            sum1 = add2(sum1, y);
            p[i] = pack16<FP8>(x.x, x.y);
            p[i + 1] = pack16<FP8>(y.x, y.y);
          }
          l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
          tmem_st32(ta, p);
          tmem_wait_st();
        }
        if ((it.blk_lo + j + 1) * kKeys > lim0) {
          // edge tile: clear from V what a zero probability would not silence
          wait_warp(&sm.v_ready, edges & 1, abort_flag, a.status);
          ++edges;
          const uint32_t vs = (pos + (j + 1 < n ? 2 * j + 2 : 2 * j + 1)) % C::kStages;   // K of the next tile goes first
          const int r = st >> 1;
          const bool past = (it.blk_lo + j) * kKeys + r >= it.kv;
          bool odd = false;
          for (int vb = 0; vb < C::VB; ++vb) {
            uint4* v = reinterpret_cast<uint4*>(sm.stage[vs] + vb * (kKeys * C::VR) + r * C::VR + (st & 1) * (C::VR / 2));
#pragma unroll
            for (int c = 0; c < C::VR / 32; ++c) {
              uint4 x = v[c];
              const uint32_t b0 = nonfinite16<FP8>(x.x), b1 = nonfinite16<FP8>(x.y), b2 = nonfinite16<FP8>(x.z),
                             b3 = nonfinite16<FP8>(x.w);
              if (past) {
                v[c] = make_uint4(0, 0, 0, 0);
              } else if (b0 | b1 | b2 | b3) {
                v[c] = make_uint4(x.x & ~b0, x.y & ~b1, x.z & ~b2, x.w & ~b3);
                odd = true;
              }
            }
          }
          if (odd) {   // both CTAs' rows may see it
#pragma unroll
            for (uint32_t cta = 0; cta < 2; ++cta)
              asm volatile("st.relaxed.cluster.shared::cluster.b32 [%0], %1;" ::"r"(map_cta(saddr(&sm.poison[item & 3]), cta)),
                           "r"(1)
                           : "memory");
          }
          asm volatile("fence.acq_rel.cluster;" ::: "memory");
          async_fence();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(p_full0 + buf * 8);
        page = page_next;
      }
      // ---- output
      g += n;
      pos = (pos + 2 * n) % C::kStages;
      // The flag of the item after next: its last readers are past the barrier of
      // the item before this one, its writers behind the P of the next one.
      if (st == 0) sm.poison[(item + 2) & 3] = 0;
      // By item parity: a warp without rows in the next item may be through with it
      // before its partner has read this one's sum.
      sm.lx[item & 1][half][row] = l;
      bar_sync(5, 256);
      l += sm.lx[item & 1][half ^ 1][row];
      wait_warp(&sm.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag, a.status);
      tc_fence_after();
      // The other CTA clears its half of V's columns and sets the flag here before
      // it hands over the tile's P: the item's last product is what orders both
      // with this read (bar_sync joins the warps of one CTA only).
      const bool poison = *reinterpret_cast<volatile int*>(&sm.poison[item & 3]) != 0;
      if (warp_live) {
        const size_t orow = (size_t)(it.t0 + tok) * a.Hq + it.kvh * G + (trow - tok * G);
        const size_t prow_out = (size_t)max(it.part, 0) * (2 * kRows) + trow;
        const float inv = l == 0.f ? 0.f : vmul / l;
        // 64 bytes of each of the warp's rows go through shared memory, so that
        // four lanes store a row's: 8 rows x 64 bytes an instruction, not 32 x 16
        unsigned char* const so = sm.out[warp - 4];
        size_t drow[4];                                // rows 8 k + lane / 4 of the warp
        bool dlive[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tr = (int)rank * kRows + 32 * quarter + 8 * k + (lane >> 2);
          const int tk = (int)((uint32_t)tr * g_inv >> 16);
          dlive[k] = tr < rows;
          drow[k] = it.part < 0 ? (size_t)(it.t0 + tk) * a.Hq + it.kvh * G + (tr - tk * G)
                                : (size_t)it.part * (2 * kRows) + tr;
        }
        auto put = [&](int ch, uint4 v) {              // this thread's row, 16-byte chunk ch
          *reinterpret_cast<uint4*>(so + lane * 64 + ((ch ^ ((lane >> 1) & 3)) << 4)) = v;
        };
        auto flush = [&](void* base, int row_bytes, int byte0) {
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rr = 8 * k + (lane >> 2), ch = lane & 3;
            const uint4 v = *reinterpret_cast<const uint4*>(so + rr * 64 + ((ch ^ ((rr >> 1) & 3)) << 4));
            if (dlive[k])
              *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(base) + drow[k] * row_bytes + byte0 + ch * 16) = v;
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int c = 0; c < OC; c += 32) {
          float o[32];
          tmem_ld32(tlane + half * OC + c, o);
          tmem_wait_ld();
          const int col = half * OC + c;
          if (l == 0.f) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
          }
          if (poison && live) {  // non-finite values of the edge tiles that this row sees
            const int from = max(it.blk_lo, max(lim0, 0) / kKeys) * kKeys, to = min(lim, it.blk_hi * kKeys);
            for (int t = from; t < to; ++t) {
              const int pr = page_row(a, pt, t / kPageTokens, n_pages, false);
              if (pr >= a.num_pages * kPageTokens) continue;
              const size_t src = ((size_t)(pr + t % kPageTokens) * a.Hkv + it.kvh) * D + col;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float v;
                if constexpr (FP8) v = Elem<__nv_fp8_e4m3>::get(reinterpret_cast<const __nv_fp8_e4m3*>(a.v_pages), src + i);
                else v = Elem<__nv_bfloat16>::get(reinterpret_cast<const __nv_bfloat16*>(a.v_pages), src + i);
                if (!isfinite(v)) o[i] += v;
              }
            }
          }
          if (it.part < 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              put(i, make_uint4(pack16<false>(o[8 * i] * inv, o[8 * i + 1] * inv),
                                pack16<false>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                pack16<false>(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                pack16<false>(o[8 * i + 6] * inv, o[8 * i + 7] * inv)));
            flush(a.out, D * 2, col * 2);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                put(i, make_uint4(__float_as_uint(o[16 * h + 4 * i]), __float_as_uint(o[16 * h + 4 * i + 1]),
                                  __float_as_uint(o[16 * h + 4 * i + 2]), __float_as_uint(o[16 * h + 4 * i + 3])));
              flush(ws.o, D * 4, (col + 16 * h) * 4);
            }
          }
        }
        if (live && half == 0) {
          if (it.part >= 0) ws.ml[prow_out] = make_float2(m, l);
          else if (a.lse) a.lse[orow] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
        }
      }
      if (it.n_parts > 0 && st == 0 && rank == 0) ws.desc[worker] = ChunkDesc{it.n_parts, it.t0, it.ntok, it.kvh};
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(o_free0);
      ++item;
      it = nx;
      have = have_next;
    }
  } else if constexpr (FP8) {
    // ---------------- codes to FP16 ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegConv));
    const int ct = threadIdx.x - 384;                  // 0 .. 127
    uint32_t r = 0, rphase = 0;
    while (ok && !*abort_flag && walk.next(a, sm.sched, TPT, kKeys, it)) {
      const int n = it.blk_hi - it.blk_lo;
      for (int i = 0; ok && i < 2 * n; ++i) {
        const bool key = i == 0 || (i != 2 * n - 1 && (i & 1));   // K0, K1, V0, K2, V1, ..., V of the last tile
        ok = wait_warp(&sm.raw_full[r], rphase, abort_flag, a.status) &&
             wait_warp(&sm.empty[s], phase ^ 1, abort_flag, a.status);
        if (!ok) break;
        const unsigned char* src = sm.raw[C::kRaws ? r : 0];
        unsigned char* dst = sm.stage[s];
        constexpr int N = C::kRaw / 16 / 128;          // 16-byte vectors of a thread
        constexpr int NB = N < 4 ? N : 4;              // loaded ahead
#pragma unroll
        for (int k0 = 0; k0 < N; k0 += NB) {
          uint4 x[NB];
#pragma unroll
          for (int k = 0; k < NB; ++k) x[k] = *reinterpret_cast<const uint4*>(src + ((k0 + k) * 128 + ct) * 16);
#pragma unroll
          for (int k = 0; k < NB; ++k) {
            const int idx = (k0 + k) * 128 + ct;
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[e] & 0xffffu), __NV_E4M3);
              const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[e] >> 16), __NV_E4M3);
              h[2 * e] = (uint32_t)lo.x | ((uint32_t)lo.y << 16);
              h[2 * e + 1] = (uint32_t)hi.x | ((uint32_t)hi.y << 16);
            }
            // rows of 64 codes (32 in a value half at D = 64) become rows of 128 (64) bytes, swizzled
            uint32_t o0, o1;
            if (D >= 128 || key) {
              const int tr = idx >> 2, c = 2 * (idx & 3);
              o0 = tr * 128 + ((c ^ (tr & 7)) << 4), o1 = tr * 128 + (((c + 1) ^ (tr & 7)) << 4);
            } else {
              const int tr = idx >> 1, c = 2 * (idx & 1);
              o0 = tr * 64 + ((c ^ ((tr >> 1) & 3)) << 4), o1 = tr * 64 + (((c + 1) ^ ((tr >> 1) & 3)) << 4);
            }
            *reinterpret_cast<uint4*>(dst + o0) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(dst + o1) = make_uint4(h[4], h[5], h[6], h[7]);
          }
        }
        async_fence();
        __syncwarp();
        if (lane == 0) {
          arrive_at(map_cta(saddr(&sm.full[s]), 0));
          mbar_arrive(&sm.raw_empty[r]);
        }
        if (++s == C::kStages) s = 0, phase ^= 1;
        if (++r == (uint32_t)C::kRaws) r = 0, rphase ^= 1;
      }
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (*abort_flag) {   // nothing may still be in flight when a CTA of the pair leaves
    if (threadIdx.x == 0 && (FP8 || rank == 0)) {
      // stages below s were last armed in this round, the others in the one before
      for (int i = 0; i < (FP8 ? C::kRaws : C::kStages); ++i)
        mbar_drain(FP8 ? &sm.raw_full[FP8 ? i : 0] : &sm.full[FP8 ? 0 : i], i < (int)s ? phase : phase ^ 1);
    } else if (warp == 1 && issued) {
      if (elect_one()) commit_pair(&sm.drain);
      __syncwarp();
      mbar_drain(&sm.drain, 0);
    }
    __syncthreads();
  }
  cluster_sync();      // the other CTA's operands, TMEM and barriers are used up to here
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

template <int D, bool FP8>
cudaError_t launch(const ChunkArgs& a, const ChunkWs& ws, int grid, float qk, float vmul, cudaStream_t s) {
  CUtensorMap mk, mv;
  if (!chunk_cache_map(&mk, a.k_pages, a, FP8, 64, kPageTokens, FP8 ? 0 : 128) ||
      !chunk_cache_map(&mv, a.v_pages, a, FP8, D >= 128 ? 64 : 32, kPageTokens, FP8 ? 0 : Cfg<D, FP8>::VR))
    return cudaErrorInvalidValue;
  auto kern = chunk_tc_kernel<D, FP8>;
  constexpr size_t smem = sizeof(TcSmem<D, FP8>) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(grid & ~1), dim3(Cfg<D, FP8>::kThreads), smem, s, 2, a, ws, qk, vmul, mk, mv);
}
template <int D>
cudaError_t launch_kv(const ChunkArgs& a, const ChunkWs& ws, int grid, float qk, float vmul, cudaStream_t s) {
  return a.kv_dt == QSA_FP8_E4M3 ? launch<D, true>(a, ws, grid, qk, vmul, s) : launch<D, false>(a, ws, grid, qk, vmul, s);
}

}  // namespace

bool chunk_tc_supported(const ChunkArgs& a) {
  return a.q_dt == QSA_BF16 && (a.kv_dt == QSA_BF16 || a.kv_dt == QSA_FP8_E4M3);
}
int chunk_tc_rows() { return 2 * kRows; }
cudaError_t launch_chunk_attn_tc(const ChunkArgs& a, const ChunkWs& ws, int grid, float qk, float vmul, cudaStream_t s) {
  switch (a.D) {
    case 64: return launch_kv<64>(a, ws, grid, qk, vmul, s);
    case 128: return launch_kv<128>(a, ws, grid, qk, vmul, s);
    default: return launch_kv<256>(a, ws, grid, qk, vmul, s);
  }
}

}  // namespace qsa
