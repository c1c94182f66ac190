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
// Angles: at position 262,144 a 32-bit product is off by up to 2^-7 radians, so
// the product is formed in 64 bits (exact: 31 + 24 bits), divided by 2 pi and
// reduced to a fraction of a turn there; sine and cosine of the fraction (at
// most half a turn, in 32 bits) are then good to a few units of 2^-24.
// One thread per (token, frequency) computes them once for all heads.
//
// Bound: HBM for a prefill chunk (each value is read and written once), the
// launch for a decode step.  A thread moves 16-byte vectors of 8 BF16 values
// (two of them for F32), a warp whole heads; a rotated pair of vectors is
// read and written by the same thread, so the queries may be rotated in place.
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 128;

struct Vec8 {
  float v[8];
};
__device__ __forceinline__ Vec8 load8(const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ Vec8 load8(const __nv_bfloat16* p) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  Vec8 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r.v[2 * j] = __uint_as_float(w[j] << 16);
    r.v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
  return r;
}
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

__device__ __forceinline__ int axis_of(const RopeArgs& a, int i) {
  if (a.interleaved_axes) {
    const int m = i % 3;
    return m == 1 && i < 3 * a.sec1 ? 1 : m == 2 && i < 3 * a.sec2 ? 2 : 0;
  }
  return i < a.sec0 ? 0 : i < a.sec0 + a.sec1 ? 1 : 2;
}

// One head of one token: `unit` is the thread's piece of it.  Units of a head
// with pairs in halves: half/8 pairs of vectors, then the vectors behind
// rot_dim; with adjacent pairs: every vector.
template <bool ADJ, typename XT, typename OT>
__device__ __forceinline__ void head_unit(const XT* src, OT* dst, int unit, int rot, const float2* cs, float scale) {
  if constexpr (ADJ) {
    Vec8 x = load8(src + unit * 8);
    if (unit * 8 < rot) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = cs[unit * 4 + j];
        const float p = x.v[2 * j], q = x.v[2 * j + 1];
        x.v[2 * j] = p * c.x - q * c.y;
        x.v[2 * j + 1] = q * c.x + p * c.y;
      }
    }
    store8(dst + unit * 8, x, scale);
  } else {
    const int half = rot >> 1, pairs = half >> 3;
    if (unit < pairs) {
      Vec8 x = load8(src + unit * 8), y = load8(src + half + unit * 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 c = cs[unit * 8 + j];
        const float p = x.v[j], q = y.v[j];
        x.v[j] = p * c.x - q * c.y;
        y.v[j] = q * c.x + p * c.y;
      }
      store8(dst + unit * 8, x, scale);
      store8(dst + half + unit * 8, y, scale);
    } else {
      const int off = rot + (unit - pairs) * 8;
      store8(dst + off, load8(src + off), scale);
    }
  }
}

template <bool ADJ, typename XT, typename KVT>
__global__ void __launch_bounds__(kThreads) rope_write_kernel(RopeArgs a, int tok_per_cta, int lanes_log2) {
  extern __shared__ float2 cs_smem[];  // [tok_per_cta][half] (cos, sin)
  __shared__ int slots[32];
  const int tid = threadIdx.x, half = a.rot_dim >> 1;
  const int t0 = blockIdx.x * tok_per_cta;
  const int ntok = min(tok_per_cta, a.T - t0);
  pdl_wait();
  pdl_launch_dependents();
  if (tid < ntok) {
    int s = a.slot[t0 + tid];
    if (s < -1 || s >= a.num_pages * (long long)kPageTokens) {
      flag(a.status, QSA_DEV_BAD_PAGE);
      s = -1;
    }
    slots[tid] = s;
  }
  for (int i = tid; i < ntok * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    const double angle = (double)a.pos[(size_t)axis_of(a, f) * a.pos_stride + t0 + t] * (double)a.inv_freq[f];
    const double turns = angle * 0.15915494309189533577;  // 1 / (2 pi)
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs_smem[i] = make_float2(c * a.rot_scale, s * a.rot_scale);
  }
  __syncthreads();

  // a group of 2^lanes_log2 threads per head, query heads first, then keys, then values
  const int units = ADJ ? a.D >> 3 : (half >> 3) + ((a.D - a.rot_dim) >> 3);
  const int lanes = 1 << lanes_log2, unit = tid & (lanes - 1);
  const int heads = a.Hq + 2 * a.Hkv;
  const int groups = kThreads >> lanes_log2;
  const XT* q = reinterpret_cast<const XT*>(a.q);
  const XT* k = reinterpret_cast<const XT*>(a.k);
  const XT* v = reinterpret_cast<const XT*>(a.v);
  XT* q_out = reinterpret_cast<XT*>(a.q_out);
  KVT* kc = reinterpret_cast<KVT*>(a.k_pages);
  KVT* vc = reinterpret_cast<KVT*>(a.v_pages);
  for (int i = tid >> lanes_log2; i < ntok * heads; i += groups) {
    const int t = i / heads, h = i - t * heads;
    const int slot = slots[t];
    if (slot < 0) continue;
    const size_t tt = (size_t)(t0 + t);
    const float2* cs = cs_smem + t * half;
    if (h < a.Hq) {
      if (unit < units)
        head_unit<ADJ>(q + tt * a.q_stride + (size_t)h * a.D, q_out + (tt * a.Hq + h) * a.D, unit, a.rot_dim, cs, 1.f);
    } else if (h < a.Hq + a.Hkv) {
      const int kh = h - a.Hq;
      if (unit < units)
        head_unit<ADJ>(k + tt * a.k_stride + (size_t)kh * a.D, kc + ((size_t)slot * a.Hkv + kh) * a.D, unit, a.rot_dim,
                       cs, a.k_scale);
    } else {
      const int vh = h - a.Hq - a.Hkv;
      const XT* src = v + tt * a.v_stride + (size_t)vh * a.D;
      KVT* dst = vc + ((size_t)slot * a.Hkv + vh) * a.D;
      for (int u = unit; u < (a.D >> 3); u += lanes) store8(dst + u * 8, load8(src + u * 8), a.v_scale);
    }
  }
}

template <bool ADJ, typename XT, typename KVT>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  const int half = a.rot_dim >> 1;
  const int units = ADJ ? a.D >> 3 : (half >> 3) + ((a.D - a.rot_dim) >> 3);
  int lg = 0;
  while ((1 << lg) < units) ++lg;
  // few tokens: one per CTA, so that a step spreads over the SMs; many: four
  // share a CTA's set-up
  const int per = a.T <= 148 * 8 ? 1 : 4;
  return launch_k(rope_write_kernel<ADJ, XT, KVT>, dim3((a.T + per - 1) / per), dim3(kThreads),
                  (size_t)per * half * sizeof(float2), s, 1, a, per, lg);
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
