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
// or not aligned for that are read again from the stored h.  Bound by HBM: 16384 rows of 5120 bf16 with a
// residual take 89 us (6.6 TB/s; the call alone, in a row of calls on rotating inputs).  What it took to get
// there is few instructions: with one value at a time the same launch shape measured 127 us, three quarters
// of its issue slots busy.  A persistent grid that loads a row ahead measured 207 us (the registers of two
// rows leave too few warps).  Rows of odd length have a form of their own: 5000 x 4095 bf16 43 us, value by
// value 67 (5000 x 4096: 25).

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

// 16 bytes of a row: kPairs pairs of values.  add() is x + r rounded to the type: the 16-bit sums are
// the fp32 sums rounded (a sum that fp32 cannot hold is nowhere near a tie of the 16-bit type).
template <int DT>
struct Io;
template <>
struct Io<DSPARK_F32> {
  using T = float;
  static constexpr int kPairs = 2;
  __device__ static float get(T v) { return v; }
  __device__ static T put(float v) { return v; }
  __device__ static float2 pair(const uint4& u, int i) {
    return i == 0 ? make_float2(__uint_as_float(u.x), __uint_as_float(u.y))
                  : make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  __device__ static uint4 add(const uint4& x, const uint4& r) {
    const float2 a = p_add(pair(x, 0), pair(r, 0)), b = p_add(pair(x, 1), pair(r, 1));
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
};
__device__ __forceinline__ uint32_t word(const uint4& u, int i) { return i == 0 ? u.x : (i == 1 ? u.y : (i == 2 ? u.z : u.w)); }
template <>
struct Io<DSPARK_BF16> {
  using T = __nv_bfloat16;
  static constexpr int kPairs = 4;
  __device__ static float get(T v) { return __bfloat162float(v); }
  __device__ static T put(float v) { return __float2bfloat16_rn(v); }
  __device__ static float2 pair(const uint4& u, int i) {
    return make_float2(__uint_as_float(word(u, i) << 16), __uint_as_float(word(u, i) & 0xFFFF0000u));
  }
  __device__ static uint32_t add2(uint32_t x, uint32_t r) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(r));
    return d;
  }
  __device__ static uint4 add(const uint4& x, const uint4& r) {
    return make_uint4(add2(x.x, r.x), add2(x.y, r.y), add2(x.z, r.z), add2(x.w, r.w));
  }
};
template <>
struct Io<DSPARK_F16> {
  using T = __half;
  static constexpr int kPairs = 4;
  __device__ static float get(T v) { return __half2float(v); }
  __device__ static T put(float v) { return __float2half_rn(v); }
  __device__ static float2 pair(const uint4& u, int i) {
    const uint32_t w = word(u, i);
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  __device__ static uint32_t add2(uint32_t x, uint32_t r) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(r));
    return d;
  }
  __device__ static uint4 add(const uint4& x, const uint4& r) {
    return make_uint4(add2(x.x, r.x), add2(x.y, r.y), add2(x.z, r.z), add2(x.w, r.w));
  }
};

// Gains of a 16-byte vector's values, as loaded: fp32, or the row's type.
template <int DT, bool GF32>
struct Gain {
  static constexpr int kWords = GF32 ? Io<DT>::kPairs / 2 : 1;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const void* gain, int i) {
    if (!gain) return;
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = static_cast<const uint4*>(gain)[i * kWords + k];
  }
  __device__ __forceinline__ float2 pair(bool have, int i) const {
    if (!have) return make_float2(1.f, 1.f);
    return GF32 ? Io<DSPARK_F32>::pair(w[i / 2], i % 2) : Io<DT>::pair(w[0], i);
  }
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
  m = warp_max_nan(m);
  if (nw == 1) return make_float2(s, m);
  __syncthreads();  // sh may hold an earlier result
  if (lane == 0) {
    sh[w] = s;
    sh[32 + w] = m;
  }
  __syncthreads();
  s = lane < nw ? sh[lane] : 0.f;
  m = lane < nw ? sh[32 + lane] : 0.f;
  return make_float2(warp_sum_f(s), warp_max_nan(m));
}

// The row's scale and the factor that takes v to the 8-bit grid.  Rows whose maximum is below 2^-120
// count as zero (127 / A would overflow); NaN or infinite values give scale NaN and q = 0.
__device__ __forceinline__ float2 row_scale(const NqArgs& a, float ss, float A, float ss_unit) {
  if (!(A < INFINITY) || isnan(ss)) return make_float2(__int_as_float(0x7FC00000), 0.f);
  if (A < 0x1p-120f) return make_float2(0.f, 0.f);
  const float f = __fdiv_rn(127.f, A);
  if (!a.norm) return make_float2(__fdiv_rn(A, 127.f), f);
  // ss holds the squares of h * ss_unit (a power of two, 1 unless the squares overflow).  The unit goes to
  // the larger factor: 2^-128, the inverse for the largest rows, is a denormal.
  const float inv = __frsqrt_rn(ss / (float)a.d + a.eps * ss_unit * ss_unit);
  const float y = A > 1.f ? __fmul_rn(__fmul_rn(A, ss_unit), inv) : __fmul_rn(A, __fmul_rn(inv, ss_unit));
  return make_float2(__fmul_rn(y, 1.f / 127.f), f);
}

__device__ __forceinline__ int8_t to_q8(float v, float f) { return (int8_t)__float2int_rn(__fmul_rn(v, f)); }

// The unit of rows whose squares overflow.  Such a row holds |h| >= 2^48 (d < 2^31): (2^48 kTiny)^2 is 2^-84,
// and the squares of 2^31 values below 2^128 sum to less than 2^107.
constexpr float kTiny = 0x1p-90f;

// Two products v f (each rounded) to the nearest integers, ties to even: adding 1.5 * 2^23 leaves the
// integer in the low bits of the sum.  (Scalar instructions: a packed product followed by a packed
// addition was seen to round once, and the grid is defined on the rounded product.)
__device__ __forceinline__ float2 to_grid(float2 v, float f) {
  const float2 t = make_float2(__fmul_rn(v.x, f), __fmul_rn(v.y, f));
  return make_float2(__fadd_rn(t.x, 12582912.f), __fadd_rn(t.y, 12582912.f));
}
__device__ __forceinline__ uint32_t low_bytes(float2 a, float2 b) {
  const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// VPT vectors of 16 bytes a thread.  The row waits in its stored type and v is formed again for its
// second use: fewer registers, more CTAs, more loads in flight.
template <int DT, bool GF32, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 256 : VPT == 2 ? 512 : 1024) rmsnorm_q8_reg(NqArgs a) {
  using I = Io<DT>;
  using T = typename I::T;
  __shared__ float sh[64];
  const long long row = blockIdx.x;
  const int nv = a.d / (2 * I::kPairs);
  const bool have_g = a.gain != nullptr;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + row * a.ldx);
  pdl_wait();
  pdl_trigger();
  uint4 hv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i < nv) hv[j] = x[i];
  }
  if (a.res) {
    const uint4* res = reinterpret_cast<const uint4*>(static_cast<const T*>(a.res) + row * a.ldr);
    uint4* hs = reinterpret_cast<uint4*>(static_cast<T*>(a.h) + row * a.ldh);
    uint4 rv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = j * blockDim.x + threadIdx.x;
      if (i < nv) rv[j] = res[i];
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = j * blockDim.x + threadIdx.x;
      if (i < nv) hs[i] = hv[j] = I::add(hv[j], rv[j]);
    }
  }
  float2 s2 = make_float2(0.f, 0.f);
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i >= nv) continue;
    Gain<DT, GF32> g;
    g.load(a.gain, i);
#pragma unroll
    for (int e = 0; e < I::kPairs; ++e) {
      const float2 h = I::pair(hv[j], e), v = p_mul(h, g.pair(have_g, e));
      s2 = p_fma(h, h, s2);
      m = max3_nan(m, fabsf(v.x), fabsf(v.y));
    }
  }
  float2 sm = block_sum_max(s2.x + s2.y, m, sh);
  float unit = 1.f;
  if (a.norm && sm.x == INFINITY && sm.y < INFINITY) {  // the squares overflow: sum them scaled
    unit = kTiny;
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (j * blockDim.x + threadIdx.x < nv)
#pragma unroll
        for (int e = 0; e < I::kPairs; ++e) {
          const float2 h = p_mul(I::pair(hv[j], e), make_float2(kTiny, kTiny));
          ss = fmaf(h.x, h.x, fmaf(h.y, h.y, ss));
        }
    sm.x = block_sum_max(ss, 0.f, sh).x;
  }
  const float2 sf = row_scale(a, sm.x, sm.y, unit);
  if (threadIdx.x == 0) a.scale[row] = sf.x;
  const uint32_t keep = isnan(sf.x) ? 0u : ~0u;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i >= nv) continue;
    Gain<DT, GF32> g;
    g.load(a.gain, i);
    uint32_t o[I::kPairs / 2];
#pragma unroll
    for (int e = 0; e < I::kPairs; e += 2)
      o[e / 2] = keep & low_bytes(to_grid(p_mul(I::pair(hv[j], e), g.pair(have_g, e)), sf.y),
                                  to_grid(p_mul(I::pair(hv[j], e + 1), g.pair(have_g, e + 1)), sf.y));
    if (I::kPairs == 4) reinterpret_cast<uint2*>(a.q + row * a.ldq)[i] = make_uint2(o[0], o[I::kPairs / 2 - 1]);
    else reinterpret_cast<uint32_t*>(a.q + row * a.ldq)[i] = o[0];
  }
}

// Gains of the kN values from element i on, i anything: the 16-byte vectors they lie in, shifted (what
// of them lies past the d gains is not read).
template <int DT, bool GF32>
struct GainAt {
  static constexpr int kN = 2 * Io<DT>::kPairs;           // values
  static constexpr int kPer = GF32 ? 4 : kN;              // gains in a vector
  static constexpr int kVecs = kN / kPer + 1;
  static constexpr int kWords = GF32 ? kN : kN * (int)sizeof(typename Io<DT>::T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* gain, int i, int d) {
    if (!gain) return;
    const uint4* g = static_cast<const uint4*>(gain) + i / kPer;
    const int off = i % kPer;
    uint32_t in[kVecs * 4];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      uint4 t = make_uint4(0, 0, 0, 0);
      if (k < kVecs - 1 || off) {
        const int end = (i / kPer + k + 1) * kPer;  // past the vector's last gain
        if (end <= d) t = g[k];
        else t = partial(gain, end - kPer, d);
      }
      in[4 * k] = t.x;
      in[4 * k + 1] = t.y;
      in[4 * k + 2] = t.z;
      in[4 * k + 3] = t.w;
    }
    // off is the same for all threads of a row: a shift by words, then by half a word
    constexpr bool kHalves = !GF32 && sizeof(typename Io<DT>::T) == 2;
    const int words = kHalves ? off >> 1 : off;
    const int n_in = kWords + (kHalves ? 1 : 0);
    uint32_t a[kWords + 1];
#pragma unroll
    for (int k = 0; k < n_in; ++k) {
      uint32_t t = in[k];
#pragma unroll
      for (int o = 1; o < 4; ++o)
        if (words == o && k + o < kVecs * 4) t = in[k + o];
      a[k] = t;
    }
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = kHalves && (off & 1) ? __funnelshift_r(a[k], a[k + 1], 16) : a[k];
  }
  // the gains from element i to d - 1, one at a time
  static __device__ __forceinline__ uint4 partial(const void* gain, int i, int d) {
    uint32_t w[4] = {0, 0, 0, 0};
    for (int e = 0; i + e < d; ++e) {
      if (GF32 || DT == DSPARK_F32) w[e & 3] = static_cast<const uint32_t*>(gain)[i + e];
      else w[(e >> 1) & 3] |= (uint32_t)static_cast<const uint16_t*>(gain)[i + e] << (16 * (e & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ float2 pair(bool have, int e) const {
    if (!have) return make_float2(1.f, 1.f);
    if (GF32 || DT == DSPARK_F32) return make_float2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
    return Io<DT>::pair(make_uint4(w[e], 0, 0, 0), 0);
  }
};

// Rows that start anywhere within 16 bytes (odd lengths), x, residual and h alike: the vectors of
// rmsnorm_q8_reg from the first 16-byte boundary on, the few values before and behind them one to a
// thread, and q assembled in shared memory, since its rows are aligned where x's are not.
template <int DT, bool GF32, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 256 : VPT == 2 ? 512 : 1024) rmsnorm_q8_shift(NqArgs a) {
  using I = Io<DT>;
  using T = typename I::T;
  constexpr int kVec = 2 * I::kPairs;
  extern __shared__ __align__(16) uint8_t s_q[];  // value e of the row at byte e - head + 8
  __shared__ float sh[64];
  const long long row = blockIdx.x;
  const bool have_g = a.gain != nullptr;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = a.res ? static_cast<const T*>(a.res) + row * a.ldr : nullptr;
  T* hs = a.res ? static_cast<T*>(a.h) + row * a.ldh : nullptr;
  const int head = min(a.d, (int)(((16u - ((uint32_t)reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / sizeof(T)));
  const int nv = (a.d - head) / kVec, tail = a.d - head - nv * kVec;
  // the value this thread has beside its vectors, or none
  const int edge = (int)threadIdx.x < head            ? (int)threadIdx.x
                   : (int)threadIdx.x < head + tail ? nv * kVec + (int)threadIdx.x
                                                    : -1;
  pdl_wait();
  pdl_trigger();
  uint4 hv[VPT];
  float he = 0.f, ge = 1.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i < nv) hv[j] = reinterpret_cast<const uint4*>(x + head)[i];
  }
  if (edge >= 0) {
    he = I::get(x[edge]);
    if (have_g) ge = GF32 ? static_cast<const float*>(a.gain)[edge] : I::get(static_cast<const T*>(a.gain)[edge]);
  }
  if (res) {
    uint4 rv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = j * blockDim.x + threadIdx.x;
      if (i < nv) rv[j] = reinterpret_cast<const uint4*>(res + head)[i];
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = j * blockDim.x + threadIdx.x;
      if (i < nv) reinterpret_cast<uint4*>(hs + head)[i] = hv[j] = I::add(hv[j], rv[j]);
    }
    if (edge >= 0) {
      const T t = I::put(he + I::get(res[edge]));
      hs[edge] = t;
      he = I::get(t);
    }
  }
  constexpr bool kKeep = VPT <= 2;  // v stays in registers: the shifted gains cost more than they
  float2 v[kKeep ? VPT : 1][I::kPairs];
  float2 s2 = make_float2(0.f, 0.f);
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i >= nv) continue;
    GainAt<DT, GF32> g;
    g.load(a.gain, head + i * kVec, a.d);
#pragma unroll
    for (int e = 0; e < I::kPairs; ++e) {
      const float2 h = I::pair(hv[j], e), t = p_mul(h, g.pair(have_g, e));
      if (kKeep) v[kKeep ? j : 0][e] = t;
      s2 = p_fma(h, h, s2);
      m = max3_nan(m, fabsf(t.x), fabsf(t.y));
    }
  }
  s2.x = fmaf(he, he, s2.x);
  m = nq_max_nan(m, fabsf(__fmul_rn(he, ge)));
  float2 sm = block_sum_max(s2.x + s2.y, m, sh);
  float unit = 1.f;
  if (a.norm && sm.x == INFINITY && sm.y < INFINITY) {  // the squares overflow: sum them scaled
    unit = kTiny;
    float ss = he * kTiny * (he * kTiny);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (j * blockDim.x + threadIdx.x < nv)
#pragma unroll
        for (int e = 0; e < I::kPairs; ++e) {
          const float2 h = p_mul(I::pair(hv[j], e), make_float2(kTiny, kTiny));
          ss = fmaf(h.x, h.x, fmaf(h.y, h.y, ss));
        }
    sm.x = block_sum_max(ss, 0.f, sh).x;
  }
  const float2 sf = row_scale(a, sm.x, sm.y, unit);
  if (threadIdx.x == 0) a.scale[row] = sf.x;
  const uint32_t keep = isnan(sf.x) ? 0u : ~0u;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i >= nv) continue;
    GainAt<DT, GF32> g;
    if (!kKeep) g.load(a.gain, head + i * kVec, a.d);
    auto again = [&](int e) { return kKeep ? v[kKeep ? j : 0][e] : p_mul(I::pair(hv[j], e), g.pair(have_g, e)); };
    uint32_t o[I::kPairs / 2];
#pragma unroll
    for (int e = 0; e < I::kPairs; e += 2)
      o[e / 2] = keep & low_bytes(to_grid(again(e), sf.y), to_grid(again(e + 1), sf.y));
    if (I::kPairs == 4) *reinterpret_cast<uint2*>(s_q + 8 + i * kVec) = make_uint2(o[0], o[I::kPairs / 2 - 1]);
    else *reinterpret_cast<uint32_t*>(s_q + 8 + i * kVec) = o[0];
  }
  if (edge >= 0) s_q[edge - head + 8] = keep ? (uint8_t)to_q8(__fmul_rn(he, ge), sf.y) : (uint8_t)0;
  __syncthreads();
  int8_t* q = a.q + row * a.ldq;
  for (int c = threadIdx.x * 16; c < a.d; c += blockDim.x * 16) {
    const int p = c - head + 8;
    if (c + 16 <= a.d) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(s_q + (p & ~3));
      const int sft = 8 * (p & 3);
      uint32_t t[5];
#pragma unroll
      for (int k = 0; k < 5; ++k) t[k] = w[k];
      *reinterpret_cast<uint4*>(q + c) = make_uint4(__funnelshift_r(t[0], t[1], sft), __funnelshift_r(t[1], t[2], sft),
                                                    __funnelshift_r(t[2], t[3], sft), __funnelshift_r(t[3], t[4], sft));
    } else {
      for (int k = 0; c + k < a.d; ++k) q[c + k] = (int8_t)s_q[p + k];
    }
  }
}

// Any stride and alignment, EPT values a thread one by one, the row in registers.
template <int DT, bool GF32, int EPT>
__global__ void __launch_bounds__(1024) rmsnorm_q8_scalar(NqArgs a) {
  using I = Io<DT>;
  using T = typename I::T;
  __shared__ float sh[64];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  pdl_wait();
  pdl_trigger();
  T h[EPT];
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    h[j] = i < a.d ? x[i] : I::put(0.f);
  }
  if (a.res) {
    const T* res = static_cast<const T*>(a.res) + row * a.ldr;
    T* hs = static_cast<T*>(a.h) + row * a.ldh;
    T r[EPT];
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      const int i = j * blockDim.x + threadIdx.x;
      r[j] = i < a.d ? res[i] : I::put(0.f);
    }
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      const int i = j * blockDim.x + threadIdx.x;
      h[j] = I::put(I::get(h[j]) + I::get(r[j]));
      if (i < a.d) hs[i] = h[j];
    }
  }
  auto gain = [&](int i) {
    return !a.gain || i >= a.d ? 1.f : GF32 ? static_cast<const float*>(a.gain)[i] : I::get(static_cast<const T*>(a.gain)[i]);
  };
  float ss = 0.f, m = 0.f;
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const float f = I::get(h[j]);
    ss = fmaf(f, f, ss);
    m = nq_max_nan(m, fabsf(__fmul_rn(f, gain(j * blockDim.x + threadIdx.x))));
  }
  float2 sm = block_sum_max(ss, m, sh);
  float unit = 1.f;
  if (a.norm && sm.x == INFINITY && sm.y < INFINITY) {  // the squares overflow: sum them scaled
    unit = kTiny;
    ss = 0.f;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      const float f = I::get(h[j]) * kTiny;
      ss = fmaf(f, f, ss);
    }
    sm.x = block_sum_max(ss, 0.f, sh).x;
  }
  const float2 sf = row_scale(a, sm.x, sm.y, unit);
  if (threadIdx.x == 0) a.scale[row] = sf.x;
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i < a.d) a.q[row * a.ldq + i] = isnan(sf.x) ? (int8_t)0 : to_q8(__fmul_rn(I::get(h[j]), gain(i)), sf.y);
  }
}

// Longer rows: read again from h (or x).
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
  pdl_wait();
  pdl_trigger();
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
  constexpr int kVec = 2 * Io<DT>::kPairs;
  auto ok = [](const void* p, long long ld, size_t es, size_t al) {
    return (uintptr_t)p % al == 0 && (ld * (long long)es) % (long long)al == 0;
  };
  const int nv = c.d / kVec;
  bool vec = c.d % kVec == 0 && ok(c.x, c.M > 1 ? c.ldx : 0, sizeof(T), 16) && ok(c.q, c.M > 1 ? c.ldq : 0, 1, kVec) &&
             (uintptr_t)c.gain % 16 == 0 && nv <= 4 * 1024;
  if (c.residual) vec = vec && ok(c.residual, c.M > 1 ? c.ldr : 0, sizeof(T), 16) && ok(c.h, c.M > 1 ? c.ldh : 0, sizeof(T), 16);
  auto threads = [&](int vpt) { return ((nv + vpt - 1) / vpt + 31) / 32 * 32; };
  if (!vec) {
    // x, residual and h start every row at the same offset within 16 bytes, q and the gains on 16
    const size_t es = sizeof(T);
    auto alike = [&](const void* p, long long ld) {
      return ((uintptr_t)p - (uintptr_t)c.x) % 16 == 0 && (c.M == 1 || (ld - c.ldx) * (long long)es % 16 == 0);
    };
    const bool shift = nv >= 16 && nv <= 4 * 1024 && ok(c.q, c.M > 1 ? c.ldq : 0, 1, 16) && (uintptr_t)c.gain % 16 == 0 &&
                       (!c.residual || (alike(c.residual, c.ldr) && alike(c.h, c.ldh)));
    if (shift) {
      const size_t smem = (size_t)c.d + 64;
      if (threads(1) <= 256 && c.M <= device_sm_count()) return launch_dependent(rmsnorm_q8_shift<DT, GF32, 1>, c.M, threads(1), smem, c.stream, 1, a);
      if (threads(2) <= 512) return launch_dependent(rmsnorm_q8_shift<DT, GF32, 2>, c.M, threads(2), smem, c.stream, 1, a);
      return launch_dependent(rmsnorm_q8_shift<DT, GF32, 4>, c.M, threads(4), smem, c.stream, 1, a);
    }
    const int nt8 = ((c.d + 7) / 8 + 31) / 32 * 32;
    if (nt8 <= 1024) return launch_dependent(rmsnorm_q8_scalar<DT, GF32, 8>, c.M, nt8, 0, c.stream, 1, a);
    return launch_dependent(rmsnorm_q8_any<DT, GF32>, c.M, 512, 0, c.stream, 1, a);
  }
  // vectors a thread: one where there are few rows, two where there are many (1 x 2048 bf16 2.3 and 2.5 us,
  // 16384 x 2048 43.4 and 37.8, with four 3.2 and 38.6)
  if (threads(1) <= 256 && c.M <= device_sm_count()) return launch_dependent(rmsnorm_q8_reg<DT, GF32, 1>, c.M, threads(1), 0, c.stream, 1, a);
  if (threads(2) <= 512) return launch_dependent(rmsnorm_q8_reg<DT, GF32, 2>, c.M, threads(2), 0, c.stream, 1, a);
  return launch_dependent(rmsnorm_q8_reg<DT, GF32, 4>, c.M, threads(4), 0, c.stream, 1, a);
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
