// Root-mean-square norm with the residual's addition and an 8-bit output with one scale per row, and
// the plain 8-bit quantisation of rows.
//
//   h = round(x + residual)         (x itself without a residual; rounded to the type that is stored)
//   v = h * gain (fp32),  A = max |v|,  q = rint(v * (127 / A)),  scale = A * rsqrt(mean h^2 + eps) / 127
// The norm's factor is the same for the whole row, so it cancels in q and appears in the scale alone:
// q is exact arithmetic on fp32 products, whatever the order of the sum of squares (fp32).
//
// One CTA per row.  The row stays in registers between the pass that reads it (sum of squares and
// maximum in one block reduction) and the pass that writes q, so every byte moves once; rows too long
// or not aligned for that are read again from the stored h.  Bound by HBM.

#include <cuda_fp16.h>

#include <algorithm>
#include <string>

#include "common.cuh"
#include "internal.h"

namespace dspark {

namespace {

struct NqArgs {
  const void* x;
  const void* res;
  const void* gain;
  void* h;
  int8_t* q;
  float* scale;
  long long ldx, ldr, ldh, ldq;
  int d, norm, gain_f32;
  float eps;
};

template <int DT>
struct Io;
template <>
struct Io<DSPARK_F32> {
  using T = float;
  static constexpr int kVec = 4;
  __device__ static float get(T v) { return v; }
  __device__ static T put(float v) { return v; }
};
template <>
struct Io<DSPARK_BF16> {
  using T = __nv_bfloat16;
  static constexpr int kVec = 8;
  __device__ static float get(T v) { return __bfloat162float(v); }
  __device__ static T put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Io<DSPARK_F16> {
  using T = __half;
  static constexpr int kVec = 8;
  __device__ static float get(T v) { return __half2float(v); }
  __device__ static T put(float v) { return __float2half_rn(v); }
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

__device__ __forceinline__ float nq_max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Block-wide sum and NaN-propagating maximum; every thread gets both.  sh: 64 floats.
__device__ __forceinline__ float2 block_sum_max(float s, float m, float* sh) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
  s = warp_sum_f(s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = nq_max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (nw == 1) return make_float2(s, m);
  __syncthreads();  // sh may hold an earlier result
  if (lane == 0) {
    sh[w] = s;
    sh[32 + w] = m;
  }
  __syncthreads();
  s = lane < nw ? sh[lane] : 0.f;
  m = lane < nw ? sh[32 + lane] : 0.f;
  s = warp_sum_f(s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = nq_max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return make_float2(s, m);
}

// The row's scale and the factor that takes v to the 8-bit grid.  Rows whose maximum is below 2^-120
// count as zero (127 / A would overflow); NaN or infinite values give scale NaN and q = 0.
__device__ __forceinline__ float2 row_scale(const NqArgs& a, float ss, float A, float ss_unit) {
  if (!(A < INFINITY) || isnan(ss)) return make_float2(__int_as_float(0x7FC00000), 0.f);
  if (A < 0x1p-120f) return make_float2(0.f, 0.f);
  const float f = __fdiv_rn(127.f, A);
  if (!a.norm) return make_float2(__fdiv_rn(A, 127.f), f);
  // ss holds the squares of h * ss_unit (a power of two, 1 unless the squares overflow)
  const float inv = __frsqrt_rn(ss / (float)a.d + a.eps * ss_unit * ss_unit) * ss_unit;
  return make_float2(__fmul_rn(__fmul_rn(A, inv), 1.f / 127.f), f);
}

__device__ __forceinline__ int8_t to_q8(float v, float f) { return (int8_t)__float2int_rn(__fmul_rn(v, f)); }

constexpr float kTiny = 0x1p-70f;

template <int DT, bool GF32, int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_q8_reg(NqArgs a) {
  using I = Io<DT>;
  using T = typename I::T;
  constexpr int kVec = I::kVec;
  using P = Pack<T, kVec>;
  using Q = Pack<int8_t, kVec>;
  using G = Pack<float, 4>;
  __shared__ float sh[64];
  const long long row = blockIdx.x;
  const int nv = a.d / kVec;
  const P* x = reinterpret_cast<const P*>(static_cast<const T*>(a.x) + row * a.ldx);
  const P* res = a.res ? reinterpret_cast<const P*>(static_cast<const T*>(a.res) + row * a.ldr) : nullptr;
  P xv[VPT], rv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i < nv) xv[j] = x[i];
    if (res && i < nv) rv[j] = res[i];
  }
  float v[VPT][kVec];
  float ss = 0.f, m = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i >= nv) continue;
    if (res) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) xv[j].v[e] = I::put(I::get(xv[j].v[e]) + I::get(rv[j].v[e]));
      reinterpret_cast<P*>(static_cast<T*>(a.h) + row * a.ldh)[i] = xv[j];
    }
    float g[kVec];
    if (!a.gain) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) g[e] = 1.f;
    } else if (GF32) {
#pragma unroll
      for (int k = 0; k < kVec / 4; ++k) {
        const G t = reinterpret_cast<const G*>(a.gain)[i * (kVec / 4) + k];
#pragma unroll
        for (int e = 0; e < 4; ++e) g[4 * k + e] = t.v[e];
      }
    } else {
      const P t = reinterpret_cast<const P*>(a.gain)[i];
#pragma unroll
      for (int e = 0; e < kVec; ++e) g[e] = I::get(t.v[e]);
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const float h = I::get(xv[j].v[e]);
      ss = fmaf(h, h, ss);
      v[j][e] = __fmul_rn(h, g[e]);
      m = nq_max_nan(m, fabsf(v[j][e]));
    }
  }
  float2 sm = block_sum_max(ss, m, sh);
  float unit = 1.f;
  if (a.norm && sm.x == INFINITY && sm.y < INFINITY) {  // the squares overflow: sum them scaled
    unit = kTiny;
    ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (j * blockDim.x + threadIdx.x < nv)
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float h = I::get(xv[j].v[e]) * kTiny;
          ss = fmaf(h, h, ss);
        }
    sm.x = block_sum_max(ss, 0.f, sh).x;
  }
  const float2 sf = row_scale(a, sm.x, sm.y, unit);
  if (threadIdx.x == 0) a.scale[row] = sf.x;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i >= nv) continue;
    Q o;
#pragma unroll
    for (int e = 0; e < kVec; ++e) o.v[e] = isnan(sf.x) ? (int8_t)0 : to_q8(v[j][e], sf.y);
    reinterpret_cast<Q*>(a.q + row * a.ldq)[i] = o;
  }
}

// Any length, stride and alignment: the row is read again from h (or x).
template <int DT, bool GF32>
__global__ void __launch_bounds__(512) rmsnorm_q8_any(NqArgs a) {
  using I = Io<DT>;
  using T = typename I::T;
  __shared__ float sh[64];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = a.res ? static_cast<const T*>(a.res) + row * a.ldr : nullptr;
  T* hs = res ? static_cast<T*>(a.h) + row * a.ldh : nullptr;
  const T* src = res ? hs : x;
  auto gain = [&](int i) {
    return !a.gain ? 1.f : GF32 ? static_cast<const float*>(a.gain)[i] : I::get(static_cast<const T*>(a.gain)[i]);
  };
  float ss = 0.f, m = 0.f;
  for (int i = threadIdx.x; i < a.d; i += blockDim.x) {
    float h = I::get(x[i]);
    if (res) {
      const T t = I::put(h + I::get(res[i]));
      hs[i] = t;
      h = I::get(t);
    }
    ss = fmaf(h, h, ss);
    m = nq_max_nan(m, fabsf(__fmul_rn(h, gain(i))));
  }
  float2 sm = block_sum_max(ss, m, sh);
  float unit = 1.f;
  if (a.norm && sm.x == INFINITY && sm.y < INFINITY) {
    unit = kTiny;
    ss = 0.f;
    for (int i = threadIdx.x; i < a.d; i += blockDim.x) {
      const float h = I::get(src[i]) * kTiny;
      ss = fmaf(h, h, ss);
    }
    sm.x = block_sum_max(ss, 0.f, sh).x;
  }
  const float2 sf = row_scale(a, sm.x, sm.y, unit);
  if (threadIdx.x == 0) a.scale[row] = sf.x;
  // every thread reads back the elements of h that it wrote itself
  for (int i = threadIdx.x; i < a.d; i += blockDim.x)
    a.q[row * a.ldq + i] = isnan(sf.x) ? (int8_t)0 : to_q8(__fmul_rn(I::get(src[i]), gain(i)), sf.y);
}

template <int DT, bool GF32>
static cudaError_t launch_nq(const NormQ8Call& c, const NqArgs& a) {
  using T = typename Io<DT>::T;
  constexpr int kVec = Io<DT>::kVec;
  auto ok = [](const void* p, long long ld, size_t es, size_t al) {
    return (uintptr_t)p % al == 0 && (ld * (long long)es) % (long long)al == 0;
  };
  const int nv = c.d / kVec;
  bool vec = c.d % kVec == 0 && ok(c.x, c.M > 1 ? c.ldx : 0, sizeof(T), 16) && ok(c.q, c.M > 1 ? c.ldq : 0, 1, kVec) &&
             (uintptr_t)c.gain % 16 == 0 && nv <= 4 * 1024;
  if (c.residual) vec = vec && ok(c.residual, c.M > 1 ? c.ldr : 0, sizeof(T), 16) && ok(c.h, c.M > 1 ? c.ldh : 0, sizeof(T), 16);
  if (!vec) {
    const int nt = std::min(512, (c.d + 31) / 32 * 32);
    rmsnorm_q8_any<DT, GF32><<<(unsigned)c.M, nt, 0, c.stream>>>(a);
    return cudaGetLastError();
  }
  auto threads = [&](int vpt) { return ((nv + vpt - 1) / vpt + 31) / 32 * 32; };
  if (threads(1) <= 256) rmsnorm_q8_reg<DT, GF32, 1><<<(unsigned)c.M, threads(1), 0, c.stream>>>(a);
  else if (threads(2) <= 512) rmsnorm_q8_reg<DT, GF32, 2><<<(unsigned)c.M, threads(2), 0, c.stream>>>(a);
  else rmsnorm_q8_reg<DT, GF32, 4><<<(unsigned)c.M, threads(4), 0, c.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

dspark_status launch_norm_q8(const NormQ8Call& c) {
  if (c.M == 0) return DSPARK_OK;
  NqArgs a{c.x, c.residual, c.gain, c.h, c.q, c.scale, c.ldx, c.ldr, c.ldh, c.ldq, c.d, c.norm, c.gain_f32, c.eps};
  cudaError_t rc;
  switch (c.dtype) {
    case DSPARK_F32: rc = launch_nq<DSPARK_F32, true>(c, a); break;
    case DSPARK_BF16: rc = c.gain_f32 ? launch_nq<DSPARK_BF16, true>(c, a) : launch_nq<DSPARK_BF16, false>(c, a); break;
    default: rc = c.gain_f32 ? launch_nq<DSPARK_F16, true>(c, a) : launch_nq<DSPARK_F16, false>(c, a); break;
  }
  if (rc != cudaSuccess) {
    set_error(std::string("rmsnorm_q8 launch: ") + cudaGetErrorString(rc));
    return DSPARK_ECUDA;
  }
  return DSPARK_OK;
}

}  // namespace dspark
