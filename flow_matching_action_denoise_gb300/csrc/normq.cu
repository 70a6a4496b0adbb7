// Residual addition, RMS norm and E4M3 output with scales in one pass (fm_norm_quant).
//
//   s = x + r;  y = s / sqrt(mean(s^2) + eps) * gamma;  scale = max|y| / 448 over the row or over 128 columns;
//   code = E4M3(y * fp32(1 / scale))
//
// The reciprocal is rounded once a scale: a division an element is what it saves, and a code differs from E4M3(y / scale)
// only where y / scale lies within 2^-23 of itself from a tie.
//
// Bound by HBM: x, r, the sum and the codes cross it once, a row stays in registers between its two reductions.
// A row belongs to 8..512 threads with one to four 8-element vectors each, all loads issued before the first reduction,
// and a CTA of its own where it takes more than a warp, so that no row waits for another's reduction (CTAs of four rows in
// step took 38 us for 12000 rows of 2048, now 29.9 us: 5.8 TB/s). Sums and scales are fp32; s is rounded once to x's
// type when stored and the norm uses it unrounded.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace fm {

namespace {

struct NormParams {
  const void* x;
  const __nv_bfloat16* r;
  const float* gamma;
  void* x_out;
  uint8_t* codes;
  float* scales;
  int64_t xs, rs, os;   // elements between rows
  int T, d, block;
  float eps;
};

template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t at, float* f) {
  if constexpr (F32) {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = src[0], b = src[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t at, const float* f) {
  if constexpr (F32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    dst[0] = make_float4(f[0], f[1], f[2], f[3]);
    dst[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The larger of two, NaN if either is: a row with a NaN gives NaN codes, not silent zeros.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Sum or maximum over the TPR threads of a row (in a fixed order); red: one float per warp of the CTA.
template <int TPR, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* red) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? max_nan(v, w) : v + w;
  }
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const int first = warp / (TPR / 32) * (TPR / 32);
    v = red[first];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) v = kMax ? max_nan(v, red[first + i]) : v + red[first + i];
  }
  return v;
}

// A CTA: rows that fit a warp in groups of 256 threads, else one row, so that no row waits for another's barrier.
__host__ __device__ constexpr int threads_of(int tpr) { return tpr > 32 ? tpr : 256; }

// CTAs an SM with 32, 48 or 64 registers a thread: a few more for the rare path cost 1000 rows of 2048 a second wave (5.0
// -> 6.1 us). fp32 rows of 512 threads need 40 (held to 32, 100 rows of 4096 took 5.0 us, now 4.2).
__host__ __device__ constexpr int resident(int tpr, int nv, bool f32) {
  return (nv == 1 ? (f32 && tpr == 512 ? 1536 : 2048) : nv == 2 ? 1280 : 1024) / threads_of(tpr);
}

template <int TPR, int NV, bool F32>
__global__ void __launch_bounds__(threads_of(TPR), resident(TPR, NV, F32)) norm_quant_kernel(const NormParams p) {
  constexpr int kThreads = threads_of(TPR);
  __shared__ float red[3][kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  const int vecs = p.d / 8;
  const bool live = row < p.T;   // every thread of the CTA takes part in the reductions
  float x[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = lane + k * TPR;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[k][e] = 0.f;
    if (live && v < vecs) load8<F32>(p.x, row * p.xs + v * 8, x[k]);
  }
  if (p.r) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = lane + k * TPR;
      if (live && v < vecs) {
        float r[8];
        load8<false>(p.r, row * p.rs + v * 8, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] += r[e];
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = lane + k * TPR;
    if (p.x_out && live && v < vecs) store8<F32>(p.x_out, row * p.os + v * 8, x[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[k][e], x[k][e], ss);
  }
  const float ms = row_reduce<TPR, false>(ss, red[0]) / p.d + p.eps;
  float rr = 1.0f / sqrtf(ms);
  // Squares out of fp32's range, the same in all of a row's threads: the row is taken times the power of two that puts the
  // larger of its maximum and sqrt(eps) into [2, 4). Not finite rows are NaN throughout, whatever a block's own columns are.
  const bool out = !(ms >= 0x1p-100f && ms < INFINITY);
  if (TPR > 32 ? out : __any_sync(0xffffffffu, out)) {
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(x[k][e]));
    top = row_reduce<TPR, true>(top, red[1]);
    const uint32_t ex = __float_as_uint(fmaxf(top, sqrtf(p.eps))) >> 23;   // biased exponent
    const float f = out ? __uint_as_float((255 - min(max(ex, 1u), 254u)) << 23) : 1.0f;
    ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[k][e] *= f;
        ss = fmaf(x[k][e], x[k][e], ss);
      }
    const float scaled = row_reduce<TPR, false>(ss, red[2]) / p.d + p.eps * f * f;
    if (out) rr = top < INFINITY ? 1.0f / sqrtf(scaled) : NAN;
  }
  float top[NV];
  float row_top = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = lane + k * TPR;
    float g[8];
    const bool has = p.gamma && v < vecs;
    if (has) load8<true>(p.gamma, v * 8, g);
    top[k] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[k][e] *= has ? rr * g[e] : rr;
      top[k] = max_nan(top[k], fabsf(x[k][e]));
    }
    row_top = max_nan(row_top, top[k]);
  }
  if (p.block) {
    // 128 columns are 16 consecutive vectors: 16 aligned lanes (a row of 8 threads has at most 64 columns)
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int o = (TPR < 16 ? TPR : 16) / 2; o > 0; o >>= 1) top[k] = max_nan(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
  } else {
    row_top = row_reduce<TPR, true>(row_top, red[1]);
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = lane + k * TPR;
    if (!live || v >= vecs) continue;
    const float scale = __fdiv_rn(p.block ? top[k] : row_top, 448.0f);
    if (scale > 1e-30f || !(scale == scale)) {
      const float inv = __fdiv_rn(1.0f, scale);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] *= inv;
    } else {   // the reciprocal may overflow; a zero scale (all zeros) gives zero codes
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] = scale > 0.f ? __fdiv_rn(x[k][e], scale) : 0.f;
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      w[e >> 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(x[k][e], x[k][e + 1]), __NV_SATFINITE, __NV_E4M3))
                   << (8 * (e & 2));
    *reinterpret_cast<uint2*>(p.codes + row * p.d + v * 8) = make_uint2(w[0], w[1]);
    if (p.block) {
      if ((v & 15) == 0) p.scales[row * ((p.d + 127) / 128) + (v >> 4)] = scale;
    } else if (v == 0) {
      p.scales[row] = scale;
    }
  }
}

template <int TPR, int NV>
cudaError_t run(const NormParams& p, bool f32, const LaunchOpts& o) {
  constexpr int kThreads = threads_of(TPR);
  const dim3 grid(static_cast<unsigned>((p.T - 1) / (kThreads / TPR) + 1));
  return f32 ? launch(norm_quant_kernel<TPR, NV, true>, grid, dim3(kThreads), 0, o, p)
             : launch(norm_quant_kernel<TPR, NV, false>, grid, dim3(kThreads), 0, o, p);
}

template <int kRowVecs>
cudaError_t many(const NormParams& p, bool f32, const LaunchOpts& o) {
  return f32 ? run<kRowVecs / 2, 2>(p, true, o) : run<kRowVecs / 4, 4>(p, false, o);
}

// Threads of a row and vectors of a thread. Many rows: four 16-byte vectors of bf16, two 32-byte ones of fp32 (12000
// rows of 2048, bf16: 28.8 us with 64 x 4, 30.5 with 128 x 2, 34 with 256 x 1, 52 with 32 x 8; fp32: 43 with 64 x 4,
// 40.8 with 128 x 2). Fewer than fill the GPU that way: one vector (1000 rows of 2048: 3.8 us against 5.1).
cudaError_t pick(const NormParams& p, bool f32, const LaunchOpts& o) {
  const int vecs = p.d / 8;
  if (vecs <= 8) return run<8, 1>(p, f32, o);
  if (vecs <= 16) return run<16, 1>(p, f32, o);
  if (static_cast<int64_t>(p.T) * vecs < 152 * 4096) {
    if (vecs <= 32) return run<32, 1>(p, f32, o);
    if (vecs <= 64) return run<64, 1>(p, f32, o);
    if (vecs <= 128) return run<128, 1>(p, f32, o);
    if (vecs <= 256) return run<256, 1>(p, f32, o);
    if (vecs <= 512) return run<512, 1>(p, f32, o);
    if (vecs <= 1024) return run<512, 2>(p, f32, o);
    return run<512, 4>(p, f32, o);
  }
  if (vecs <= 32) return run<16, 2>(p, f32, o);
  if (vecs <= 64) return run<32, 2>(p, f32, o);
  if (vecs <= 128) return many<128>(p, f32, o);
  if (vecs <= 256) return many<256>(p, f32, o);
  if (vecs <= 512) return many<512>(p, f32, o);
  if (vecs <= 1024) return many<1024>(p, f32, o);
  return run<512, 4>(p, f32, o);
}

}  // namespace

}  // namespace fm

extern "C" int fm_norm_quant(const void* x, int64_t x_stride, int x_f32, const uint16_t* r, int64_t r_stride,
                             const float* gamma, int T, int d, float eps, void* x_out, int64_t x_out_stride,
                             uint8_t* codes, float* scales, int block, void* stream) {
  using namespace fm;
  if (T < 0 || d < 16 || d > 16384 || d % 16) return record_error(FM_ERR_SHAPE, "T >= 0 and d a multiple of 16 up to 16384");
  if (block != 0 && block != 128) return record_error(FM_ERR_INVALID_ARG, "block must be 0 (a scale per row) or 128");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return record_error(FM_ERR_INVALID_ARG, "eps must not be negative");
  if (T == 0) return FM_OK;
  if (!x || !codes || !scales) return record_error(FM_ERR_INVALID_ARG, "NULL argument");
  if (x_stride < d || x_stride % 8 || (r && (r_stride < d || r_stride % 8)) ||
      (x_out && (x_out_stride < d || x_out_stride % 8)))
    return record_error(FM_ERR_SHAPE, "row strides must be multiples of 8 elements and hold d");
  if (x == x_out && x_stride != x_out_stride && T > 1) return record_error(FM_ERR_SHAPE, "x_out in the place of x needs x's stride");
  for (const void* q : {x, static_cast<const void*>(r), static_cast<const void*>(gamma), static_cast<const void*>(x_out),
                        static_cast<const void*>(codes)})
    if (reinterpret_cast<uintptr_t>(q) % 16) return record_error(FM_ERR_ALIGN, "x, r, gamma, x_out and codes must be 16-byte aligned");
  const NormParams p{x, reinterpret_cast<const __nv_bfloat16*>(r), gamma, x_out, codes, scales, x_stride, r_stride,
                     x_out_stride, T, d, block, eps};
  LaunchOpts o;
  o.stream = static_cast<cudaStream_t>(stream);
  o.pdl = true;
  const cudaError_t e = pick(p, x_f32 != 0, o);
  return e == cudaSuccess ? FM_OK : record_error(FM_ERR_CUDA, cudaGetErrorString(e));
}
