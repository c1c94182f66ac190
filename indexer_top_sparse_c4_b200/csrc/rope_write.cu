// rope_write.cu -- rotary positions with one to three axes on a step's queries
// and keys, and the write of its keys and values into the paged cache ("QSA
// HiSparse" README, entry-point table: the backend's prefill writes; page size
// 64, FP8 E4M3 KV).
//
// For token t and frequency i < rot_dim / 2:
//   angle = pos[axis(i)][t] * inv_freq[i]
//   (a, b) -> rot_scale * (a cos - b sin, b cos + a sin)
// on the pair (a, b) = (x[i], x[i + rot_dim/2]) or (x[2i], x[2i+1]) of every
// query and key head; the values behind rot_dim stay as they are.  axis(i):
//   chunked      0 for i < sec0, 1 for the next sec1, 2 for the rest
//   interleaved  1 where i % 3 == 1 and i < 3 sec1, 2 where i % 3 == 2 and
//                i < 3 sec2, otherwise 0
//
// Angles: at position 262,144 a 32-bit product is off by up to 2^-7 radians.  A
// position of 31 bits times a frequency of 24 does not fit the 53 bits of a
// double either, and 1 / (2 pi) is known to no finite number of them, so both
// the product and the quotient are carried as two doubles (angle_turns): the
// fraction of a turn is good to 2^-53 of a turn at every position, and what
// remains is its rounding to FP32 and the sine's and cosine's own, a few units
// of 2^-24 of each, small sines near whole turns included.
//
// Bound: HBM for a prefill chunk (each value is read and written once), the
// launch for a decode step.  A warp takes a token, or with few tokens a part
// of its heads, and waits for no other: it forms the token's angles once
// (shared memory, then registers) and walks over the heads, D / 16 lanes to a
// head and two 16-byte vectors of a rotated pair to a lane, the next heads'
// loads in flight.  Measured (8,192 tokens, 24/2 heads of D 256, BF16): 44 us,
// 5.3 TB/s; one CTA per four tokens with the angles read from shared memory
// for every head took 60 us (eight lanes to a bank), and four heads in flight
// at twice the registers 57 us.  Six CTAs an SM allow 80 registers, for which
// all forms but BF16 to F32 spill a little (BF16 to BF16 and FP8 24 bytes
// stored, with adjacent pairs 4 and 28; F32 56 to 68).  A rotated pair is read
// and written by the same lane, so the queries may be rotated in place.
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxHalf = 128;
constexpr int kWarps = 4736;   // warps a call is spread over, if its heads are enough (32 an SM; 24 are resident)

struct Vec8 {
  float v[8];
};
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(float* p, const Vec8& x, float) {
  *reinterpret_cast<float4*>(p) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x.v[4], x.v[5], x.v[6], x.v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Vec8& x, float) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x.v[0], x.v[1]), pack_bf16(x.v[2], x.v[3]),
                                            pack_bf16(x.v[4], x.v[5]), pack_bf16(x.v[6], x.v[7]));
}
// code = e4m3(x / scale), to nearest even, values past +-448 to +-448
__device__ __forceinline__ void store8(__nv_fp8_e4m3* p, const Vec8& x, float scale) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const __nv_fp8x2_storage_t lo =
        __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x.v[4 * j], scale), __fdiv_rn(x.v[4 * j + 1], scale)),
                                 __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi =
        __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x.v[4 * j + 2], scale), __fdiv_rn(x.v[4 * j + 3], scale)),
                                 __NV_SATFINITE, __NV_E4M3);
    w[j] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// pos * freq / (2 pi) less the nearest whole turns, in -1/2 .. 1/2.
__device__ __forceinline__ float angle_turns(int pos, float freq) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;   // 1 / (2 pi)
  const double p = pos, f = freq;
  const double a = __dmul_rn(p, f), a_lo = fma(p, f, -a);                      // p f, exactly
  const double t = __dmul_rn(a, kHi);
  const double t_lo = fma(a, kHi, -t) + fma(a, kLo, a_lo * kHi);
  return (float)((t - rint(t)) + t_lo);
}

__device__ __forceinline__ int axis_of(const RopeArgs& a, int i) {
  if (a.interleaved_axes) {
    const int m = i % 3;
    return m == 1 && i < 3 * a.sec1 ? 1 : m == 2 && i < 3 * a.sec2 ? 2 : 0;
  }
  return i < a.sec0 ? 0 : i < a.sec0 + a.sec1 ? 1 : 2;
}

__device__ __forceinline__ void turn_adjacent(Vec8& x, const float2* cs) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float p = x.v[2 * e], r = x.v[2 * e + 1];
    x.v[2 * e] = p * cs[e].x - r * cs[e].y;
    x.v[2 * e + 1] = r * cs[e].x + p * cs[e].y;
  }
}

// What a lane holds of one head of one token: two vectors of 8.
template <typename XT>
struct Raw;
template <>
struct Raw<float> {
  float4 a[2], b[2];
  __device__ __forceinline__ void load(const float* p, const float* q) {
    a[0] = *reinterpret_cast<const float4*>(p), a[1] = *(reinterpret_cast<const float4*>(p) + 1);
    b[0] = *reinterpret_cast<const float4*>(q), b[1] = *(reinterpret_cast<const float4*>(q) + 1);
  }
  static __device__ __forceinline__ Vec8 vec(const float4 (&v)[2]) {
    return Vec8{{v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w}};
  }
};
template <>
struct Raw<__nv_bfloat16> {
  uint4 a[1], b[1];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* q) {
    a[0] = *reinterpret_cast<const uint4*>(p);
    b[0] = *reinterpret_cast<const uint4*>(q);
  }
  static __device__ __forceinline__ Vec8 vec(const uint4 (&v)[1]) {
    const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
    Vec8 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.v[2 * j] = __uint_as_float(w[j] << 16);
      r.v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
    return r;
  }
};

template <bool ADJ, typename XT, typename KVT>
__global__ void __launch_bounds__(kThreads, 6) rope_write_kernel(RopeArgs a, int parts, int part_heads, int lanes_log2) {
  constexpr int kAhead = sizeof(XT) == 2 ? 3 : 2;   // heads whose loads a lane has in flight
  __shared__ float2 cs_smem[kThreads / 32][kMaxHalf];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = a.rot_dim >> 1;
  const int w = blockIdx.x * (kThreads / 32) + warp, t = w / parts, part = w - t * parts;
  pdl_wait();
  pdl_launch_dependents();
  if (t >= a.T) return;                // whole warps; none waits for another
  int slot = a.slot[t];
  if (slot < -1 || slot >= a.num_pages * (long long)kPageTokens) {
    if (lane == 0) flag(a.status, QSA_DEV_BAD_PAGE);
    slot = -1;
  }
  if (slot < 0) return;
  // D / 16 lanes to a head, two vectors of 8 to a lane: the two of a pair, or
  // two of those behind rot_dim; with adjacent pairs, and for values, vector
  // `unit` of either half
  const int lanes = a.D >> 4, unit = lane & (lanes - 1), groups = 32 >> lanes_log2;
  const int h_end = min(a.Hq + 2 * a.Hkv, (part + 1) * part_heads);
  const int pairs = half >> 3, voff0 = unit * 8, voff1 = voff0 + (a.D >> 1);
  int off0 = voff0, off1 = voff1;
  if (!ADJ) {
    if (unit < pairs) off1 = half + unit * 8;
    else off0 = a.rot_dim + (unit - pairs) * 8, off1 = off0 + ((a.D - a.rot_dim) >> 1);
  }

  // a group of 2^lanes_log2 lanes per head, query heads first, then keys, then
  // values; the loads of kAhead heads are in flight at a time
  const XT* q = reinterpret_cast<const XT*>(a.q) + (size_t)t * a.q_stride;
  const XT* k = reinterpret_cast<const XT*>(a.k) + (size_t)t * a.k_stride;
  const XT* v = reinterpret_cast<const XT*>(a.v) + (size_t)t * a.v_stride;
  XT* q_out = reinterpret_cast<XT*>(a.q_out) + (size_t)t * a.Hq * a.D;
  KVT* kc = reinterpret_cast<KVT*>(a.k_pages) + (size_t)slot * a.Hkv * a.D;
  KVT* vc = reinterpret_cast<KVT*>(a.v_pages) + (size_t)slot * a.Hkv * a.D;
  auto fetch = [&](int h, Raw<XT>& x) {
    if (h >= h_end) return;
    if (h < a.Hq + a.Hkv) {
      const XT* src = h < a.Hq ? q + h * a.D : k + (h - a.Hq) * a.D;
      x.load(src + off0, src + off1);
    } else {
      const XT* src = v + (h - a.Hq - a.Hkv) * a.D;
      x.load(src + voff0, src + voff1);
    }
  };
  int hb = part * part_heads + (lane >> lanes_log2);
  Raw<XT> x[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) fetch(hb + j * groups, x[j]);   // in flight while the angles are formed

  // (cos, sin) of frequency f at [f % NF][f / NF], NF of them a thread: read
  // back without bank conflicts, and kept in registers for all heads
  constexpr int NF = ADJ ? 4 : 8;
  const int fu = half / NF;
  for (int f = lane; f < half; f += 32) {
    float s, c;
    sincospif(2.f * angle_turns(a.pos[(size_t)axis_of(a, f) * a.pos_stride + t], a.inv_freq[f]), &s, &c);
    cs_smem[warp][(f % NF) * fu + f / NF] = make_float2(c * a.rot_scale, s * a.rot_scale);
  }
  __syncwarp();
  float2 cs[8];                        // adjacent pairs: four of each vector
  const bool turn0 = unit < fu, turn1 = ADJ && unit + lanes < fu;
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    if (turn0) cs[j] = cs_smem[warp][j * fu + unit];
    if (turn1) cs[4 + j % 4] = cs_smem[warp][j * fu + unit + lanes];
  }
  for (;;) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {   // slot j is refilled as soon as its head has been taken from it
      const int h = hb + j * groups;
      if (h >= h_end) return;
      Vec8 y = Raw<XT>::vec(x[j].a), z = Raw<XT>::vec(x[j].b);
      fetch(h + kAhead * groups, x[j]);
      if (h < a.Hq + a.Hkv) {
        if constexpr (ADJ) {
          if (turn0) turn_adjacent(y, cs);
          if (turn1) turn_adjacent(z, cs + 4);
        } else if (turn0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float p = y.v[e], r = z.v[e];
            y.v[e] = p * cs[e].x - r * cs[e].y;
            z.v[e] = r * cs[e].x + p * cs[e].y;
          }
        }
        if (h < a.Hq) {
          store8(q_out + h * a.D + off0, y, 1.f);
          store8(q_out + h * a.D + off1, z, 1.f);
        } else {
          KVT* dst = kc + (h - a.Hq) * a.D;
          store8(dst + off0, y, a.k_scale);
          store8(dst + off1, z, a.k_scale);
        }
      } else {
        KVT* dst = vc + (h - a.Hq - a.Hkv) * a.D;
        store8(dst + voff0, y, a.v_scale);
        store8(dst + voff1, z, a.v_scale);
      }
    }
    hb += kAhead * groups;
  }
}

template <bool ADJ, typename XT, typename KVT>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  const int lg = a.D == 64 ? 2 : a.D == 128 ? 3 : 4;
  // a warp per token, or, with few tokens, per part of a token's heads: a whole
  // pass of the warp's groups at least, and up to about kWarps of them.  (A few
  // thousand tokens are cut finer than they need to be: 2,360 of 28 heads make
  // 7,080 warps, two rounds of the 3,552 that are resident.)
  const int heads = a.Hq + 2 * a.Hkv, groups = 32 >> lg;
  const int want = (kWarps + a.T - 1) / a.T;
  const int part_heads = (heads + want - 1) / want > groups ? ((heads + want - 1) / want + groups - 1) / groups * groups : groups;
  const int parts = (heads + part_heads - 1) / part_heads;
  const long long warps = (long long)a.T * parts;
  const int per = kThreads / 32;
  return launch_k(rope_write_kernel<ADJ, XT, KVT>, dim3((unsigned)((warps + per - 1) / per)), dim3(kThreads), 0, s, 1, a,
                  parts, part_heads, lg);
}
template <bool ADJ, typename XT>
cudaError_t launch_kv(const RopeArgs& a, cudaStream_t s) {
  switch (a.kv_dt) {
    case QSA_F32: return launch<ADJ, XT, float>(a, s);
    case QSA_BF16: return launch<ADJ, XT, __nv_bfloat16>(a, s);
    default: return launch<ADJ, XT, __nv_fp8_e4m3>(a, s);
  }
}

}  // namespace

cudaError_t launch_rope_write(const RopeArgs& a, cudaStream_t s) {
  static_assert(kMaxHalf * 2 <= 256, "rot_dim is at most 256");
  if (a.x_dt == QSA_F32) return a.adjacent_pairs ? launch_kv<true, float>(a, s) : launch_kv<false, float>(a, s);
  return a.adjacent_pairs ? launch_kv<true, __nv_bfloat16>(a, s) : launch_kv<false, __nv_bfloat16>(a, s);
}

}  // namespace qsa
