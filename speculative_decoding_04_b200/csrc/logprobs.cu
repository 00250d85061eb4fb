// Log probabilities of given tokens with entropy and top alternatives, and their gradient.
//
// For a row of logits l and a temperature T, with m = max l and d = (l - m) / T:
//   S = sum exp(d),   logp = d_tok - ln S,   H = ln S - (sum exp(d) d) / S,
//   top = the `top` largest logits (ties: lowest index) with their log probabilities.
// Both terms of H are non-negative, so nothing cancels.
//
// Forward.  One cluster of C CTAs per row (C = 1 when the rows alone fill the GPU), the row cut into
// tiles of 2 KB that are contiguous in the vocabulary; the warps of a CTA take its tiles in turn.  One
// pass: a warp loads a tile (four 16-byte loads a lane, the next tile's loads in flight meanwhile),
// reduces its maximum, keeps it in shared memory as the tile's record and adds the tile to the warp's
// running (R, S, E) = (reference, sum 2^x, sum 2^x x), x = (l - R) log2(e)/T, rescaled when R grows.
// The sums are fp32 per lane (some 300 terms), joined over warps and CTAs in fp64.
//
// Alternatives.  The main pass spends nothing on them beyond the tiles' maxima.  The k best elements
// (value descending, index ascending) lie in the k best tiles ordered by (maximum descending, tile
// ascending): an element outside them is beaten by each of those tiles' maxima, on a tie by its lower
// index, because a tile is a contiguous range.  So the k tiles are read again (from L2), each yields
// at most k candidates at or above the k-th tile's maximum, and the candidates are ranked by counting.
//
// Backward.  One pass over the row: with G = g_logp + sum_j g_top,j and p, log p from (m, ln S),
//   dl = ( g_logp 1_tok + sum_j g_top,j 1_idx_j - p (G + g_H (log p + H)) ) / T,
// the few elements with an indicator written again after the rest, from the unrounded value.
// Both passes are bound by HBM.

#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <string>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace dspark {

namespace {

constexpr int kLpWarps = 16;
constexpr int kLpThreads = kLpWarps * 32;
constexpr int kLpMaxTiles = 4096;   // tiles of one CTA (2 KB each): 16 KB of maxima
constexpr int kLpMaxCluster = 16;
constexpr int kLpCand = DSPARK_TOP_MAX * DSPARK_TOP_MAX;

constexpr double kLog2eD = 1.4426950408889634074;
constexpr double kLn2D = 0.69314718055994530942;

struct LpArgs {
  const void* logits;
  long long ld;           // elements between rows
  const int64_t* rows;    // row of each entry, or null: entry n reads row n
  long long n_rows;
  const int32_t* tokens;
  int V, top;
  double inv_T;
  float c;                // log2(e) / T
  float* logp;
  float* entropy;
  int32_t* top_idx;
  float* top_logp;
  float2* stats;
  uint32_t* flags;
};

// One 16-byte vector of logits: VEC elements, as fp32 pairs.
template <int DT>
struct Elem;
template <>
struct Elem<DSPARK_F32> {
  using T = float;
  static constexpr int kVec = 4;
  __device__ static float get(T v) { return v; }
  __device__ static T neg_inf() { return -INFINITY; }
  __device__ static float2 pair(const uint4& u, int i) {
    return i == 0 ? make_float2(__uint_as_float(u.x), __uint_as_float(u.y))
                  : make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
};
template <>
struct Elem<DSPARK_BF16> {
  using T = __nv_bfloat16;
  static constexpr int kVec = 8;
  __device__ static float get(T v) { return __bfloat162float(v); }
  __device__ static T neg_inf() { return __ushort_as_bfloat16(0xFF80); }
  __device__ static float2 pair(const uint4& u, int i) {
    const uint32_t w = i == 0 ? u.x : (i == 1 ? u.y : (i == 2 ? u.z : u.w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
};
template <>
struct Elem<DSPARK_F16> {
  using T = __half;
  static constexpr int kVec = 8;
  __device__ static float get(T v) { return __half2float(v); }
  __device__ static T neg_inf() { return __ushort_as_half(0xFC00); }
  __device__ static float2 pair(const uint4& u, int i) {
    const uint32_t w = i == 0 ? u.x : (i == 1 ? u.y : (i == 2 ? u.z : u.w));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// max of three, NaN if any is (sm_100)
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// maximum over the warp, NaN if any lane's is (sm_100a)
__device__ __forceinline__ float warp_max_nan(float v) {
  float d;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}

// Unsigned key with the order (value descending, index ascending) = keys descending; -0 counts as +0.
__device__ __forceinline__ uint64_t cand_key(float x, uint32_t idx) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t o = b ^ ((b & 0x80000000u) ? 0xFFFFFFFFu : 0x80000000u);
  return ((uint64_t)o << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o ^ ((o & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}

// The tiles of a row: [0, head) first where the row does not start on 16 bytes, then tiles of kTile
// elements from there; contiguous and in vocabulary order.
template <int DT>
struct RowTiles {
  using E = Elem<DT>;
  using T = typename E::T;
  static constexpr int kTile = 32 * 4 * E::kVec;
  const T* p;
  int V, head, n;
  __device__ RowTiles(const T* p_, int V_) : p(p_), V(V_) {
    head = (int)(((16u - ((uint32_t)reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / sizeof(T));
    if (head > V) head = V;
    n = (head > 0 ? 1 : 0) + (V - head + kTile - 1) / kTile;
  }
  __device__ int start(int t) const { return head > 0 ? (t == 0 ? 0 : head + (t - 1) * kTile) : t * kTile; }
  __device__ int end(int t) const { return head > 0 && t == 0 ? head : min(V, start(t) + kTile); }
  // lane's 4 vectors of tile t: vector j covers elements start + (j*32 + lane)*VEC ..; elements past
  // the tile's end read as -inf
  __device__ __forceinline__ void load(int t, int lane, uint4 (&v)[4]) const {
    const int s = start(t), len = end(t) - s;
    if (len == kTile) {
      const uint4* q = reinterpret_cast<const uint4*>(p + s) + lane;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __ldg(q + j * 32);
    } else {
      load_edge(s, len, lane, v);
    }
  }
  __device__ __forceinline__ void load_edge(int s, int len, int lane, uint4 (&v)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      T e[E::kVec];
#pragma unroll
      for (int i = 0; i < E::kVec; ++i) {
        const int k = (j * 32 + lane) * E::kVec + i;
        e[i] = k < len ? p[s + k] : E::neg_inf();
      }
      v[j] = *reinterpret_cast<const uint4*>(e);
    }
  }
};

struct CtaPart {  // a CTA's sums: maximum, sum 2^x and sum 2^x x against it
  double S, E;
  float R;
  int bad;
};

template <int DT>
__global__ void __launch_bounds__(kLpThreads, 2) token_logprobs_kernel(LpArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int kPairs = E::kVec / 2;
  __shared__ float s_max[kLpMaxTiles];
  __shared__ uint64_t s_cand[kLpCand];
  __shared__ uint64_t s_top[DSPARK_TOP_MAX];
  __shared__ uint64_t s_all[kLpMaxCluster * DSPARK_TOP_MAX];
  __shared__ float s_R[kLpWarps], s_S[kLpWarps], s_E[kLpWarps];
  __shared__ int s_bad[kLpWarps];
  __shared__ int s_sel[DSPARK_TOP_MAX];
  __shared__ CtaPart s_part;
  __shared__ float s_thr;
  __shared__ int s_nsel, s_ncand, s_ntop, s_nall;
  __shared__ double s_m, s_logS;

  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long n = blockIdx.x / C;
  const int tok = __ldg(a.tokens + n);
  const long long row = a.rows ? __ldg(a.rows + n) : n;

  if (tok == -1 || row < 0 || row >= a.n_rows) {  // the whole cluster leaves
    if (rank == 0) {
      const bool pad = tok == -1;
      const float x = pad ? 0.f : __int_as_float(0x7FC00000);
      if (tid == 0) {
        a.logp[n] = x;
        if (a.entropy) a.entropy[n] = x;
        if (a.stats) a.stats[n] = make_float2(x, x);
        if (!pad && a.flags) atomicOr(a.flags + n, DSPARK_FLAG_RAGGED_OFFSETS);
      }
      for (int j = tid; j < a.top; j += kLpThreads) {
        a.top_idx[n * a.top + j] = -1;
        a.top_logp[n * a.top + j] = pad ? -INFINITY : x;
      }
    }
    return;
  }

  const RowTiles<DT> tiles(static_cast<const T*>(a.logits) + row * a.ld, a.V);
  const int t0 = (int)((long long)tiles.n * rank / C), t1 = (int)((long long)tiles.n * (rank + 1) / C);

  // ---------------------------------------------------------------- one pass over the CTA's tiles
  float R = -INFINITY;
  float2 S2 = make_float2(0.f, 0.f), E2 = make_float2(0.f, 0.f);
  int bad = 0;
  uint4 cur[4], nxt[4];
  if (t0 + warp < t1) tiles.load(t0 + warp, lane, cur);
  for (int t = t0 + warp; t < t1; t += kLpWarps) {
    if (t + kLpWarps < t1) tiles.load(t + kLpWarps, lane, nxt);
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 x = E::pair(cur[j], i);
        m = max3_nan(m, x.x, x.y);
      }
    m = warp_max_nan(m);
    if (lane == 0) s_max[t - t0] = m;
    if (!(m < INFINITY)) bad = 1;  // NaN or +inf
    if (m > R) {  // the same for all lanes
      if (R > -INFINITY) {
        const float dr = (R - m) * a.c, f = ex2(fmaxf(dr, -200.f));
        E2.x = (E2.x + S2.x * fmaxf(dr, -200.f)) * f;
        E2.y = (E2.y + S2.y * fmaxf(dr, -200.f)) * f;
        S2.x *= f;
        S2.y *= f;
      }
      R = m;
    }
    if (m > -INFINITY) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 x = E::pair(cur[j], i);
          // below 2^-200 nothing is added; the clamp also keeps 0 * inf out of E
          const float dx = fmaxf((x.x - R) * a.c, -200.f), dy = fmaxf((x.y - R) * a.c, -200.f);
          const float ex = ex2(dx), ey = ex2(dy);
          S2.x += ex;
          S2.y += ey;
          E2.x = fmaf(ex, dx, E2.x);
          E2.y = fmaf(ey, dy, E2.y);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) cur[j] = nxt[j];
  }
  {
    const float S = warp_sum_f(S2.x + S2.y), Es = warp_sum_f(E2.x + E2.y);
    if (lane == 0) {
      s_R[warp] = R;
      s_S[warp] = S;
      s_E[warp] = Es;
      s_bad[warp] = bad;
    }
  }
  if (tid == 0) s_ncand = 0;
  __syncthreads();

  // ---------------------------------------------------------------- the CTA's sums; its best tiles
  const double cd = a.inv_T * kLog2eD;
  if (warp == 1) {
    const float r = lane < kLpWarps ? s_R[lane] : -INFINITY;
    const float M = warp_max(r);
    const int b = __any_sync(0xffffffffu, lane < kLpWarps && s_bad[lane]);
    double S = 0.0, Es = 0.0;
    if (lane < kLpWarps && r > -INFINITY) {
      const double dr = fmax(((double)r - (double)M) * cd, -1000.0), f = exp2(dr);
      S = (double)s_S[lane] * f;
      Es = ((double)s_E[lane] + (double)s_S[lane] * dr) * f;
    }
    S = warp_sum_d(S);
    Es = warp_sum_d(Es);
    if (lane == 0) s_part = CtaPart{S, Es, M, b};
  }
  if (warp == 0 && a.top > 0) {
    const int nt = t1 - t0;
    int nsel = 0;
    float last = -INFINITY, best = -INFINITY;
    int bi = 0x7FFFFFFF;
    auto scan = [&] {
      best = -INFINITY;
      bi = 0x7FFFFFFF;
      for (int i = lane; i < nt; i += 32)
        if (s_max[i] > best) {
          best = s_max[i];
          bi = i;
        }
    };
    scan();
    while (nsel < a.top) {
      const float M = warp_max(best);
      if (!(M > -INFINITY)) break;
      const int w = (int)__reduce_min_sync(0xffffffffu, best == M ? (unsigned)bi : 0x7FFFFFFFu);
      if (lane == 0) s_sel[nsel] = w;
      ++nsel;
      last = M;
      if ((w & 31) == lane) {
        s_max[w] = -INFINITY;
        scan();
      }
      __syncwarp();
    }
    if (lane == 0) {
      s_nsel = nsel;
      s_thr = nsel == a.top ? last : -INFINITY;  // every element to come is at or above it
    }
  }
  __syncthreads();

  if (a.top > 0) {
    // -------------------------------------------------------------- candidates of the best tiles
    const int nsel = s_nsel;
    const float thr = s_thr;
    for (int j = warp; j < nsel; j += kLpWarps) {
      const int t = t0 + s_sel[j];
      const int ts = tiles.start(t);
      uint4 v[4];
      tiles.load(t, lane, v);
      float x[4 * E::kVec];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 f = E::pair(v[q], i);
          x[q * E::kVec + 2 * i] = f.x;
          x[q * E::kVec + 2 * i + 1] = f.y;
        }
      for (int round = 0; round < a.top; ++round) {
        float best = -INFINITY;
        int bi = 0x7FFFFFFF;
#pragma unroll
        for (int q = 0; q < 4 * E::kVec; ++q)
          if (x[q] > best) {  // in index order: the first of equal values stays
            best = x[q];
            bi = ((q / E::kVec) * 32 + lane) * E::kVec + q % E::kVec;
          }
        const float M = warp_max(best);
        if (!(M > -INFINITY) || M < thr) break;
        const int w = (int)__reduce_min_sync(0xffffffffu, best == M ? (unsigned)bi : 0x7FFFFFFFu);
        if (lane == 0) s_cand[atomicAdd(&s_ncand, 1)] = cand_key(M, (uint32_t)(ts + w));
        if (best == M && bi == w) {
#pragma unroll
          for (int q = 0; q < 4 * E::kVec; ++q)
            if (((q / E::kVec) * 32 + lane) * E::kVec + q % E::kVec == w) x[q] = -INFINITY;
        }
      }
    }
    __syncthreads();
    // rank by counting (the keys are distinct): key i goes to place #{j : key j > key i}
    const int nc = s_ncand;
    for (int i = tid; i < nc; i += kLpThreads) {
      const uint64_t k = s_cand[i];
      int place = 0;
      for (int j = 0; j < nc; ++j) place += s_cand[j] > k;
      if (place < a.top) s_top[place] = k;
    }
    if (tid == 0) s_ntop = min(nc, a.top);
  }

  // ---------------------------------------------------------------- join the cluster, write the row
  if (C > 1) cluster.sync();
  else __syncthreads();
  if (rank == 0) {
    if (warp == 0) {
      CtaPart p{0.0, 0.0, -INFINITY, 0};
      if (lane < C) p = C > 1 ? *cluster.map_shared_rank(&s_part, lane) : s_part;
      const float M = warp_max(p.R);
      const int b = __any_sync(0xffffffffu, p.bad);
      double S = 0.0, Es = 0.0;
      if (p.R > -INFINITY) {
        const double dr = fmax(((double)p.R - (double)M) * cd, -1000.0), f = exp2(dr);
        S = p.S * f;
        Es = (p.E + p.S * dr) * f;
      }
      S = warp_sum_d(S);
      Es = warp_sum_d(Es);
      if (lane == 0) {
        const float nan = __int_as_float(0x7FC00000);
        double logS = log(S);
        float lp, H, m = M;
        uint32_t fl = 0;
        if (b) {
          fl |= DSPARK_FLAG_NONFINITE;
          m = nan;
          logS = (double)nan;
          lp = H = nan;
        } else if (!(M > -INFINITY)) {  // nothing in the row is unmasked
          logS = -INFINITY;
          lp = -INFINITY;
          H = 0.f;
        } else {
          H = (float)(logS - Es / S * kLn2D);
          lp = 0.f;
        }
        if ((unsigned)tok >= (unsigned)a.V) {
          fl |= DSPARK_FLAG_TOKEN_RANGE;
          lp = nan;
        } else if (!b && M > -INFINITY) {
          lp = (float)(((double)E::get(tiles.p[tok]) - (double)M) * a.inv_T - logS);
        }
        a.logp[n] = lp;
        if (a.entropy) a.entropy[n] = H;
        if (a.stats) a.stats[n] = make_float2(m, (float)logS);
        if (fl && a.flags) atomicOr(a.flags + n, fl);
        s_m = (double)m;
        s_logS = logS;
      }
    }
    if (a.top > 0) {
      const uint64_t* from = s_top;
      int nc = s_ntop;
      if (C > 1) {  // the CTAs' lists, ranked again
        if (tid == 0) s_nall = 0;
        __syncthreads();
        for (int r = warp; r < C; r += kLpWarps) {
          const int k = *cluster.map_shared_rank(&s_ntop, r);
          const uint64_t* src = cluster.map_shared_rank(s_top, r);
          int at = 0;
          if (lane == 0) at = atomicAdd(&s_nall, k);
          at = __shfl_sync(0xffffffffu, at, 0);
          if (lane < k) s_all[at + lane] = src[lane];
        }
        __syncthreads();
        const int na = s_nall;
        for (int i = tid; i < na; i += kLpThreads) {
          const uint64_t k = s_all[i];
          int place = 0;
          for (int j = 0; j < na; ++j) place += s_all[j] > k;
          if (place < a.top) s_cand[place] = k;
        }
        from = s_cand;
        nc = min(na, a.top);
      }
      __syncthreads();
      const bool nan_row = isnan(s_m);
      if (tid < a.top) {
        const bool have = tid < nc && !nan_row;
        const uint64_t k = have ? from[tid] : 0;
        a.top_idx[n * a.top + tid] = have ? (int32_t)~(uint32_t)k : -1;
        a.top_logp[n * a.top + tid] = have      ? (float)(((double)key_value(k) - s_m) * a.inv_T - s_logS)
                                      : nan_row ? __int_as_float(0x7FC00000)
                                                : -INFINITY;
      }
    }
  }
  if (C > 1) cluster.sync();  // no CTA leaves while rank 0 may still read its shared memory
}

// ============================================================================ backward

constexpr int kLbThreads = 256;
constexpr int kLbVecs = 4;

struct LbArgs {
  const void* logits;
  void* grad;
  long long ld, ldg;
  const int32_t* tokens;
  const float2* stats;
  const float* entropy;
  const float* g_logp;
  const float* g_entropy;
  const int32_t* top_idx;
  const float* g_top;
  int V, top, chunks;
  float inv_T;
  int vec;  // every row of logits and grad starts at the same offset within 16 bytes
};

template <int DT>
__device__ __forceinline__ typename Elem<DT>::T to_elem(float x);
template <>
__device__ __forceinline__ float to_elem<DSPARK_F32>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_elem<DSPARK_BF16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half to_elem<DSPARK_F16>(float x) { return __float2half_rn(x); }

// A row's coefficients: dl = (indicators) / T + p (k1 log p + k0)
struct LbRow {
  float m, logS, inv_T, k1, k0;
  __device__ __forceinline__ float dense(float x) const {
    const float lp = fmaxf(fmaf(x - m, inv_T, -logS), -1e4f);  // exp(-1e4) is 0; keeps 0 * inf out
    return ex2(lp * kLog2e) * fmaf(lp, k1, k0);
  }
};

template <int DT>
__global__ void __launch_bounds__(kLbThreads) token_logprobs_bwd_kernel(LbArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int kChunk = kLbThreads * kLbVecs * E::kVec;
  const long long n = blockIdx.x / a.chunks;
  const int ch = (int)(blockIdx.x - n * a.chunks);
  const int tid = threadIdx.x;
  const T* p = static_cast<const T*>(a.logits) + n * a.ld;
  T* g = static_cast<T*>(a.grad) + n * a.ldg;
  // chunk 0 also takes the elements before the first 16-byte boundary
  int head = (int)(((16u - ((uint32_t)reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / sizeof(T));
  head = min(head, a.V);
  const int lo = ch == 0 ? 0 : head + ch * kChunk;
  const int hi = (int)min((long long)a.V, (long long)head + (long long)(ch + 1) * kChunk);
  if (lo >= hi) return;
  const int body = ch == 0 ? head : lo;

  const int tok = __ldg(a.tokens + n);
  const float2 st = __ldg(a.stats + n);
  if (tok < 0 || tok >= a.V || st.x == -INFINITY) {  // a row without a token or without any unmasked logit
    if (a.vec) {
      const uint4 z = make_uint4(0, 0, 0, 0);
      for (int i = lo + tid; i < body; i += kLbThreads) g[i] = to_elem<DT>(0.f);
      const int nv = (hi - body) / E::kVec;
      for (int i = tid; i < nv; i += kLbThreads) reinterpret_cast<uint4*>(g + body)[i] = z;
      for (int i = body + nv * E::kVec + tid; i < hi; i += kLbThreads) g[i] = to_elem<DT>(0.f);
    } else {
      for (int i = lo + tid; i < hi; i += kLbThreads) g[i] = to_elem<DT>(0.f);
    }
    return;
  }
  const float gl = a.g_logp ? __ldg(a.g_logp + n) : 0.f;
  const float gH = a.g_entropy ? __ldg(a.g_entropy + n) : 0.f;
  float G = gl;
  const int32_t* ti = a.top ? a.top_idx + n * a.top : nullptr;
  const float* gt = a.top ? a.g_top + n * a.top : nullptr;
  for (int j = 0; j < a.top; ++j)
    if (__ldg(ti + j) >= 0) G += __ldg(gt + j);
  LbRow r;
  r.m = st.x;
  r.logS = st.y;
  r.inv_T = a.inv_T;
  r.k1 = -a.inv_T * gH;
  r.k0 = -a.inv_T * (gH != 0.f ? fmaf(gH, __ldg(a.entropy + n), G) : G);
  if (!(st.x < INFINITY)) r.k0 = __int_as_float(0x7FC00000);  // a row with NaN or +inf: its gradient is NaN

  // elements with an indicator: thread j < top + 1 owns index j if it is its first occurrence.  The
  // value is formed before the dense pass overwrites the logit (grad may be the logits themselves).
  int own = -1;
  float fix = 0.f;
  if (tid <= a.top) {
    const int idx = tid == 0 ? tok : __ldg(ti + tid - 1);
    bool first = idx >= lo && idx < hi;
    if (first && tid > 0) {
      first = idx != tok;
      for (int j = 0; first && j < tid - 1; ++j) first = __ldg(ti + j) != idx;
    }
    if (first) {
      float add = tid == 0 ? gl : 0.f;
      for (int j = 0; j < a.top; ++j)
        if (__ldg(ti + j) == idx) add += __ldg(gt + j);
      own = idx;
      fix = r.dense(E::get(p[idx])) + add * a.inv_T;
    }
  }
  __syncthreads();

  if (a.vec) {
    for (int i = lo + tid; i < body; i += kLbThreads) g[i] = to_elem<DT>(r.dense(E::get(p[i])));
    const int nv = (hi - body) / E::kVec;
    const uint4* q = reinterpret_cast<const uint4*>(p + body);
    uint4* o = reinterpret_cast<uint4*>(g + body);
    uint4 v[kLbVecs];
#pragma unroll
    for (int j = 0; j < kLbVecs; ++j)
      if (j * kLbThreads + tid < nv) v[j] = q[j * kLbThreads + tid];
#pragma unroll
    for (int j = 0; j < kLbVecs; ++j)
      if (j * kLbThreads + tid < nv) {
        T e[E::kVec];
#pragma unroll
        for (int i = 0; i < E::kVec / 2; ++i) {
          const float2 x = E::pair(v[j], i);
          e[2 * i] = to_elem<DT>(r.dense(x.x));
          e[2 * i + 1] = to_elem<DT>(r.dense(x.y));
        }
        o[j * kLbThreads + tid] = *reinterpret_cast<const uint4*>(e);
      }
    for (int i = body + nv * E::kVec + tid; i < hi; i += kLbThreads) g[i] = to_elem<DT>(r.dense(E::get(p[i])));
  } else {
    for (int i = lo + tid; i < hi; i += kLbThreads) g[i] = to_elem<DT>(r.dense(E::get(p[i])));
  }
  __syncthreads();
  if (own >= 0) g[own] = to_elem<DT>(fix);
}

}  // namespace

// ============================================================================ host

template <int DT>
static dspark_status launch_lp(const LogprobsCall& c) {
  constexpr int kTile = RowTiles<DT>::kTile;
  const long long nt = ((long long)c.V + kTile - 1) / kTile + 1;
  // CTAs per row: while the rows alone leave SMs idle (two CTAs of 16 warps per SM), split each row,
  // down to one tile a warp; more where a CTA could not hold the tiles' records
  const long long slots = 2ll * device_sm_count();
  int C = 1;
  while (C < kLpMaxCluster && ((long long)c.N * 2 * C <= slots && nt / (2 * C) >= kLpWarps)) C *= 2;
  while (C < kLpMaxCluster && (nt + C - 1) / C > kLpMaxTiles) C *= 2;
  LpArgs a{c.logits, c.ld, c.rows, c.n_rows, c.tokens, c.V, c.top, 1.0 / (double)c.T, (float)(kLog2eD / (double)c.T),
           c.logp, c.entropy, c.top_idx, c.top_logp, reinterpret_cast<float2*>(c.stats), c.flags};
  auto kern = token_logprobs_kernel<DT>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = c.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t rc = cudaSuccess;
  if (C > 8 && ensure_nonportable_cluster((const void*)kern) != cudaSuccess) {
    cudaGetLastError();
    C = 8;
  }
  if ((nt + C - 1) / C > kLpMaxTiles) {
    set_error("dspark_token_logprobs: V too large for the clusters this device allows");
    return DSPARK_ENOTIMPL;
  }
  at[0].val.clusterDim.x = C;
  cfg.gridDim = dim3((unsigned)((long long)c.N * C));
  rc = cudaLaunchKernelEx(&cfg, kern, a);
  if (rc != cudaSuccess) {
    cudaGetLastError();
    set_error(std::string("token_logprobs launch: ") + cudaGetErrorString(rc));
    return DSPARK_ECUDA;
  }
  return DSPARK_OK;
}

dspark_status launch_token_logprobs(const LogprobsCall& c) {
  if (c.N == 0) return DSPARK_OK;
  switch (c.dtype) {
    case DSPARK_F32: return launch_lp<DSPARK_F32>(c);
    case DSPARK_BF16: return launch_lp<DSPARK_BF16>(c);
    default: return launch_lp<DSPARK_F16>(c);
  }
}

template <int DT>
static dspark_status launch_lb(const LogprobsBwdCall& c) {
  using T = typename Elem<DT>::T;
  constexpr int kChunk = kLbThreads * kLbVecs * Elem<DT>::kVec;
  const int chunks = (c.V + kChunk - 1) / kChunk;  // chunk 0 is longer by the unaligned head
  const long long grid = (long long)c.N * chunks;
  if (grid > 0x7FFFFFFFll) {
    set_error("dspark_token_logprobs_backward: too many rows");
    return DSPARK_ENOTIMPL;
  }
  const bool vec = ((uintptr_t)c.logits - (uintptr_t)c.grad) % 16 == 0 &&
                   (c.N == 1 || ((c.ld - c.ldg) * (long long)sizeof(T)) % 16 == 0);
  LbArgs a{c.logits, c.grad, c.ld, c.ldg, c.tokens, reinterpret_cast<const float2*>(c.stats), c.entropy, c.g_logp,
           c.g_entropy, c.top_idx, c.g_top, c.V, c.top, chunks, 1.f / c.T, vec ? 1 : 0};
  token_logprobs_bwd_kernel<DT><<<(unsigned)grid, kLbThreads, 0, c.stream>>>(a);
  const cudaError_t rc = cudaGetLastError();
  if (rc != cudaSuccess) {
    set_error(std::string("token_logprobs_backward launch: ") + cudaGetErrorString(rc));
    return DSPARK_ECUDA;
  }
  return DSPARK_OK;
}

dspark_status launch_token_logprobs_backward(const LogprobsBwdCall& c) {
  if (c.N == 0) return DSPARK_OK;
  switch (c.dtype) {
    case DSPARK_F32: return launch_lb<DSPARK_F32>(c);
    case DSPARK_BF16: return launch_lb<DSPARK_BF16>(c);
    default: return launch_lb<DSPARK_F16>(c);
  }
}

}  // namespace dspark
