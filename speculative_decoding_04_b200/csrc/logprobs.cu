// Log probabilities of given tokens with entropy and top alternatives, and their gradient.
//
// For a row of logits l and a temperature T, with m = max l and d = (l - m) / T:
//   S = sum exp(d),   logp = d_tok - ln S,   H = ln S - (sum exp(d) d) / S,
//   top = the `top` largest logits (ties: lowest index) with their log probabilities.
// Both terms of H are non-negative, so nothing cancels.
//
// Forward.  One cluster of C CTAs per row (C = 1 when the rows alone fill the GPU), the row cut into
// tiles of 512 values that are contiguous in the vocabulary; the warps of a CTA take its tiles in turn.
// One pass: a warp loads a tile (two or four 16-byte loads a lane, the next tile's loads in flight
// meanwhile), reduces its maximum, keeps it in shared memory as the tile's record and adds the tile to
// the warp's running (R, S, E) = (reference, sum 2^x, sum 2^x x), x = (l - R) log2(e)/T, rescaled when R
// grows (in a branch of its own: 47 against 49 us at 944 x 77028 bf16).  The sums are fp32 per lane (per
// tile, then over the tiles), joined pairwise over lanes, warps and CTAs, and leave one maximum out of S,
// so that the log probability and the entropy of a row with one dominant token keep their digits; the
// logarithm and what follows are fp64.  The maxima are taken past NaN; the sums keep every NaN, and a row
// whose sums are NaN is NaN.
// The roundings of a term of S, in half steps of fp32: 3 |d| for its exponent (what a rising reference adds
// to it included), 4 for ex2, 7 additions in its tile and one for each tile of its warp, 5 for each rise of the
// warp's reference, 6 to join the pairs and lanes, 14 to join the warps and 14 to join a cluster's CTAs (the
// factor 5, products 2, additions 5, and 2 for the value that was left out).  Measured errors of the log
// probabilities of language-model rows are 4e-8 to 8e-8.
// A value costs 8.5 instructions in fp32 and 7.2 in bf16 (packed fp32 pairs; one ex2), which at 16 bits a
// value keeps the SM about as busy as HBM: 1088 x 151936 fp32 takes 102 us among other calls (6.5
// TB/s), 2048 x 262144 bf16 183 us.  One row of 151936 takes 4.7 us without and 7.6 with 20 alternatives:
// a cluster of 16 CTAs, two cluster barriers, the choice of tiles and the candidates between them.
// After a flush of L2, on 1088 x 151936 fp32 unless stated, while this was built: CTAs of 8 warps, four to
// an SM, hide each other's row ends better than two of 16 (131 against 141 us; five with 48 registers,
// among other calls, 116 against 102); a ring filled by 16-byte asynchronous copies measured 139 us (its
// shared-memory traffic competes with the exponentials), two or three tiles ahead 133 and 143 (fewer warps
// fit), and values clamped one by one against -inf in every tile 204 us at 2048 x 262144 bf16 (hence the
// two forms of the loop).
//
// Alternatives.  The main pass spends nothing on them beyond the tiles' maxima.  The k best elements
// (value descending, index ascending) lie in the k best tiles ordered by (maximum descending, tile
// ascending): an element outside them is beaten by each of those tiles' maxima, on a tie by its lower
// index, because a tile is a contiguous range.  So the k tiles are read again (from L2, spread over the
// cluster), each yields at most k candidates at or above the k-th tile's maximum, and the candidates
// are ranked by counting.
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

constexpr int kLpMaxCluster = 16;

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

// How many of n distinct keys (from a 16-byte boundary on) are larger.
__device__ __forceinline__ int rank_of(uint64_t k, const uint64_t* keys, int n) {
  int r = 0;
  const ulonglong2* two = reinterpret_cast<const ulonglong2*>(keys);
#pragma unroll 4
  for (int j = 0; j < n / 2; ++j) {
    const ulonglong2 o = two[j];
    r += (o.x > k) + (o.y > k);
  }
  if (n & 1) r += keys[n - 1] > k;
  return r;
}

// The tiles of a row: [0, head) first where the row does not start on 16 bytes, then tiles of kTile
// elements from there; contiguous and in vocabulary order.
template <int DT>
struct RowTiles {
  using E = Elem<DT>;
  using T = typename E::T;
  static constexpr int kLoads = sizeof(T);  // 16-byte vectors of a tile a lane holds
  static constexpr int kTile = 32 * kLoads * E::kVec;
  const T* p;
  int V, head, n;
  __device__ RowTiles(const T* p_, int V_) : p(p_), V(V_) {
    head = (int)(((16u - ((uint32_t)reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / sizeof(T));
    if (head > V) head = V;
    n = (head > 0 ? 1 : 0) + (V - head + kTile - 1) / kTile;
  }
  __device__ int start(int t) const { return head > 0 ? (t == 0 ? 0 : head + (t - 1) * kTile) : t * kTile; }
  __device__ int end(int t) const { return head > 0 && t == 0 ? head : min(V, start(t) + kTile); }
  // lane's vectors of tile t: vector j covers elements start + (j*32 + lane)*VEC ..; elements past
  // the tile's end read as -inf
  __device__ __forceinline__ void load(int t, int lane, uint4 (&v)[kLoads]) const {
    const int s = start(t), len = end(t) - s;
    if (len == kTile) {
      const uint4* q = reinterpret_cast<const uint4*>(p + s) + lane;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) v[j] = q[j * 32];
    } else {
      load_edge(s, len, lane, v);
    }
  }
  // the tile after the last full one
  __device__ int full_end() const { return (head > 0 ? 1 : 0) + (V - head) / kTile; }
  __device__ __forceinline__ void load_edge(int s, int len, int lane, uint4 (&v)[kLoads]) const {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
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

// Sums against their maximum R: sum 2^x over all values but one that equals R (its 2^0 = 1 is left out, so
// that small sums beside it keep their digits), and sum 2^x x.
struct CtaPart {
  float S, E, R;
  int bad;
};

__device__ __forceinline__ float redux_max(float v) {
  float d;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
  return d;
}

// Nothing below 2^kFloor of the maximum is added; the clamp also keeps 0 * inf out of E.
constexpr float kFloor = -200.f;

// Sums against different maxima joined over the lanes of a warp.
__device__ __forceinline__ CtaPart join_parts(CtaPart p, float c) {
  const float M = redux_max(p.R);
  const unsigned who = __ballot_sync(0xffffffffu, p.R == M);
  float S = 0.f, E = 0.f;
  if (p.R > -INFINITY) {
    if ((int)(threadIdx.x & 31) == __ffs(who) - 1) {  // the one value left out of the joined sum is this one's
      S = p.S;
      E = p.E;
    } else {
      const float dr = fmaxf((p.R - M) * c, kFloor), f = exp2f(dr);
      S = fmaf(p.S, f, f);
      E = (fmaf(p.S, dr, p.E) + dr) * f;
    }
  }
  return CtaPart{warp_sum_f(S), warp_sum_f(E), M, __any_sync(0xffffffffu, p.bad)};
}

__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}

// Where a tile's maximum goes: this CTA's record, or (clusters) the record of every CTA, lane r writing
// to CTA r.
template <bool CLUSTER>
struct MaxOut {
  float* own;
  uint32_t at;
  bool mine;
  __device__ MaxOut(float* s_max, int C, int lane) : own(s_max), at(0), mine(lane < (CLUSTER ? C : 1)) {
    if (CLUSTER && mine) at = cluster_addr(s_max, lane);
  }
  __device__ __forceinline__ void put(int t, float m) const {
    if (!mine) return;
    if (CLUSTER) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4u * t), "f"(m) : "memory");
    else own[t] = m;
  }
};

// A warp's running sums over the tiles it takes.
template <int DT, bool CLUSTER>
struct WarpSums {
  using E = Elem<DT>;
  static constexpr int kPairs = E::kVec / 2, kLoads = RowTiles<DT>::kLoads;
  static constexpr int kAhead = 1;  // (two in 16 bits: 208 against 183 us for 2048 x 262144 bf16, registers spill)
  float c, R;
  float2 S2, E2;
  bool clamp;
  __device__ explicit WarpSums(float c_)
      : c(c_), R(-INFINITY), S2(make_float2(0.f, 0.f)), E2(make_float2(0.f, 0.f)), clamp(false) {}

  // One tile into the sums.  Masked values would make 0 * -inf in E, so they are clamped; that costs two
  // instructions a pair, which rows without them, most, go without until a tile's sum shows one.  A tile
  // that brings a new maximum takes that form too, with the maximum itself left out of S.  NaN stays in
  // the sums.
  __device__ __forceinline__ void tile(const uint4 (&v)[kLoads], int lane, int t, const MaxOut<CLUSTER>& out, bool edge) {
    float lm = -INFINITY;
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 x = E::pair(v[j], i);
        lm = max3(lm, x.x, x.y);
      }
    const float m = redux_max(lm);
    out.put(t, m);
    if (m > R) {  // the same for all lanes
      const float dr = fmaxf((R - m) * c, kFloor), f = ex2(dr);  // R = -inf: S = E = 0 stay
      E2 = p_mul(p_fma(S2, make_float2(dr, dr), E2), make_float2(f, f));
      S2 = p_mul(S2, make_float2(f, f));
      if (lane == 0 && R > -INFINITY) {  // the value left out so far
        S2.x += f;
        E2.x = fmaf(dr, f, E2.x);
      }
      R = m;
      bool leave = lane == __ffs(__ballot_sync(0xffffffffu, lm == m)) - 1;  // this lane's first value m is left out
      const float2 nR = make_float2(-R, -R), c2 = make_float2(c, c);
      float2 ts, te;
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 x = E::pair(v[j], i);
          float2 d = p_mul(p_add(x, nR), c2);
          d = make_float2(max_nan(d.x, kFloor), max_nan(d.y, kFloor));
          if (leave && x.x == m) {
            d.x = kFloor;
            leave = false;
          }
          if (leave && x.y == m) {
            d.y = kFloor;
            leave = false;
          }
          const float2 e = make_float2(ex2(d.x), ex2(d.y));
          const bool first = j == 0 && i == 0;
          ts = first ? e : p_add(ts, e);
          te = first ? p_mul(e, d) : p_fma(e, d, te);
        }
      S2 = p_add(S2, ts);
      E2 = p_add(E2, te);
      return;
    }
    const float2 nR = make_float2(-R, -R), c2 = make_float2(c, c);
    if (!clamp && !edge) {
      float2 ts, te;  // the tile's own sums: shorter chains of additions
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 d = p_mul(p_add(E::pair(v[j], i), nR), c2);
          const float2 e = make_float2(ex2(d.x), ex2(d.y));
          const bool first = j == 0 && i == 0;
          ts = first ? e : p_add(ts, e);
          te = first ? p_mul(e, d) : p_fma(e, d, te);
        }
      const float x = te.x + te.y;
      if (!__any_sync(0xffffffffu, x != x)) {
        S2 = p_add(S2, ts);
        E2 = p_add(E2, te);
        return;
      }
      clamp = true;
    }
    if (R == -INFINITY && m == -INFINITY) {  // nothing unmasked so far: -inf adds nothing, NaN stays
      float x = -INFINITY;
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 p = E::pair(v[j], i);
          x = max3_nan(x, p.x, p.y);
        }
      if (x != x) S2.x = x;  // (the maxima m and R are taken past NaN)
      return;
    }
    float2 ts, te;
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        float2 d = p_mul(p_add(E::pair(v[j], i), nR), c2);
        d = make_float2(max_nan(d.x, kFloor), max_nan(d.y, kFloor));
        const float2 e = make_float2(ex2(d.x), ex2(d.y));
        const bool first = j == 0 && i == 0;
        ts = first ? e : p_add(ts, e);
        te = first ? p_mul(e, d) : p_fma(e, d, te);
      }
    S2 = p_add(S2, ts);
    E2 = p_add(E2, te);
  }

  // Full tiles t, t + W, ... below end, the next kAhead tiles' loads in flight.
  template <int W>
  __device__ __forceinline__ void pass(const RowTiles<DT>& tiles, int t, int end, int lane, const MaxOut<CLUSTER>& out) {
    const uint4* src = reinterpret_cast<const uint4*>(tiles.p + tiles.start(t)) + lane;
    uint4 buf[kAhead + 1][kLoads];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch<W>(src, i, t, end, buf[i]);
    while (t < end) {
#pragma unroll
      for (int u = 0; u <= kAhead; ++u)
        if (t + u * W < end) {
          fetch<W>(src, u + kAhead, t, end, buf[(u + kAhead) % (kAhead + 1)]);
          tile(buf[u], lane, t + u * W, out, false);
        }
      t += (kAhead + 1) * W;
      src += (kAhead + 1) * (W * 32 * kLoads);
    }
  }
  template <int W>
  static __device__ __forceinline__ void fetch(const uint4* src, int i, int t, int end, uint4 (&v)[kLoads]) {
    if (t + i * W < end) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) v[j] = __ldcs(src + i * (W * 32 * kLoads) + j * 32);
    }
  }
};

template <int DT, int W, bool CLUSTER>
__global__ void __launch_bounds__(W * 32, 32 / W) token_logprobs_kernel(LpArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int kLoads = RowTiles<DT>::kLoads;
  constexpr int kLpWarps = W, kLpThreads = W * 32, kList = W < 8 ? W * 32 : 256;
  // [top^2] candidates (rank 0 of a cluster: the whole cluster's), the maxima of the row's tiles
  extern __shared__ __align__(16) uint8_t s_dyn[];
  uint64_t* s_cand = reinterpret_cast<uint64_t*>(s_dyn);
  float* s_max = reinterpret_cast<float*>(s_cand + a.top * a.top);
  __shared__ uint64_t s_top[DSPARK_TOP_MAX];
  __shared__ CtaPart s_warp[kLpWarps];
  __shared__ CtaPart s_part[kLpMaxCluster];  // (rank 0) the CTAs' sums
  __shared__ int s_sel[DSPARK_TOP_MAX];
  __shared__ int s_nsel, s_nlist, s_ncand;
  __shared__ __align__(16) uint64_t s_lane[32], s_list[kList];  // keys of tiles: the lanes' best, those to rank
  __shared__ uint64_t s_from;  // the top-th best tile, or a bound on it
  __shared__ double s_m, s_logS;

  cg::cluster_group cluster = cg::this_cluster();
  const int C = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long n = blockIdx.x / C;
  pdl_wait();
  pdl_trigger();
  const int tok = a.tokens[n];
  const long long row = a.rows ? a.rows[n] : n;

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
  const int nt = tiles.n;
  if (tid == 0) {
    s_ncand = s_nlist = 0;
    s_from = 0;
  }
  // the peers have started before anything is written to them (waited for below)
  __syncwarp();
  if (CLUSTER) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const bool in_range = (unsigned)tok < (unsigned)a.V;
  float x_tok = 0.f;
  if (rank == 0 && tid == 0 && in_range) x_tok = E::get(tiles.p[tok]);
  const int t0 = (int)((long long)nt * rank / C), t1 = (int)((long long)nt * (rank + 1) / C);

  // ---------------------------------------------------------------- one pass over the CTA's tiles
  // full tiles [b0, b1) of the CTA first, then what the row begins or ends with
  const int b0 = max(t0, tiles.head > 0 ? 1 : 0), b1 = min(t1, tiles.full_end());
  __syncwarp();
  if (CLUSTER) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const MaxOut<CLUSTER> out(s_max, C, lane);
  WarpSums<DT, CLUSTER> sums(a.c);
  sums.template pass<W>(tiles, b0 + warp, b1, lane, out);
  if (warp == W - 1) {
    for (int e = 0; e < 2; ++e) {
      const int t = e == 0 ? 0 : nt - 1;
      if (t < t0 || t >= t1 || (t >= b0 && t < b1) || (e == 1 && nt == 1)) continue;
      uint4 v[kLoads];
      tiles.load_edge(tiles.start(t), tiles.end(t) - tiles.start(t), lane, v);
      sums.tile(v, lane, t, out, true);
    }
  }
  {
    const float S = warp_sum_f(sums.S2.x + sums.S2.y), Es = warp_sum_f(sums.E2.x + sums.E2.y);
    if (lane == 0) s_warp[warp] = CtaPart{S, Es, sums.R, !(sums.R < INFINITY) || S != S || Es != Es};  // +inf or NaN
  }
  __syncwarp();
  // the tiles' maxima are everywhere, and the CTA's partial sums here
  if (CLUSTER) cluster.sync();
  else __syncthreads();
  if (warp == 1) {
    const CtaPart p = join_parts(lane < kLpWarps ? s_warp[lane] : CtaPart{0.f, 0.f, -INFINITY, 0}, a.c);
    if (lane == 0) *(CLUSTER ? cluster.map_shared_rank(&s_part[rank], 0) : &s_part[0]) = p;
  }

  if (a.top > 0) {
    // -------------------------------------------------------------- the row's best tiles
    // (every CTA of a cluster makes the same choice)  One or two are taken one after the other, 480 cycles
    // each.  For more, the top-th largest of 32 lanes' best tiles bounds the top-th best tile from below,
    // and the tiles from there on, mostly few, are ranked by counting (1 x 151936 fp32 with 1, 5, 20 and 32
    // alternatives: 7.0, 7.3, 7.6 and 8.3 us, one after the other 6.4, 7.6, 11.4 and 14.4).
    bool in_turn = a.top <= 2;
    if (!in_turn) {
      if (warp == 0) {
        float best = -INFINITY;
        int bi = 0;
#pragma unroll 4
        for (int i = lane; i < nt; i += 32)
          if (s_max[i] > best) {
            best = s_max[i];
            bi = i;
          }
        const uint64_t k = best > -INFINITY ? cand_key(best, (uint32_t)bi) : 0;
        s_lane[lane] = k;
        __syncwarp();
        const int place = rank_of(k, s_lane, 32);
        if (k && place == a.top - 1) s_from = k;
        if (nt <= 32) {  // a tile a lane: these are the tiles' places
          if (k && place < a.top) s_sel[place] = lane;
          const int have = __popc(__ballot_sync(0xffffffffu, k != 0));
          if (lane == 0) s_nsel = min(have, a.top);
        }
      }
      if (nt > 32) {
        __syncthreads();
        const uint64_t from = s_from;  // 0: fewer lanes than that have an unmasked tile
        for (int i0 = warp * 32; i0 < nt; i0 += kLpThreads) {
          const float x = i0 + lane < nt ? s_max[i0 + lane] : -INFINITY;
          const uint64_t k = cand_key(x, (uint32_t)(i0 + lane));
          const bool in = x > -INFINITY && k >= from;
          const unsigned who = __ballot_sync(0xffffffffu, in);
          if (!who) continue;
          int at = 0;
          if (lane == 0) at = atomicAdd(&s_nlist, __popc(who));
          at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
          if (in && at < kList) s_list[at] = k;
        }
        __syncthreads();
        const int listed = s_nlist;
        in_turn = listed > kList;  // a few lanes hold nearly all the large tiles
        if (!in_turn) {
          for (int i = tid; i < listed; i += kLpThreads) {
            const uint64_t k = s_list[i];
            const int place = rank_of(k, s_list, listed);
            if (place < a.top) s_sel[place] = (int)~(uint32_t)k;
            if (place == a.top - 1) s_from = k;
          }
          if (tid == 0) s_nsel = min(listed, a.top);
        }
      }
    }
    if (in_turn && warp == 0) {
      int nsel = 0;
      float best, last = -INFINITY;
      int bi;
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
        const float M = redux_max(best);
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
        s_from = cand_key(last, 0);
      }
    }
    __syncthreads();

    // -------------------------------------------------------------- their candidates
    const int nsel = s_nsel, room = nsel > 0 ? a.top * a.top / nsel : 0;
    const float thr = nsel == a.top ? key_value(s_from) : -INFINITY;  // every element to come is at or above it
    uint64_t* cand = CLUSTER ? cluster.map_shared_rank(s_cand, 0) : s_cand;
    int* ncand = CLUSTER ? cluster.map_shared_rank(&s_ncand, 0) : &s_ncand;
    for (int j = warp * C + rank; j < nsel; j += kLpWarps * C) {
      const int t = s_sel[j], ts = tiles.start(t);
      uint4 v[kLoads];
      tiles.load(t, lane, v);
      auto value = [&](int q) {
        const float2 f = E::pair(v[q / E::kVec], (q % E::kVec) / 2);
        return (q & 1) ? f.y : f.x;
      };
      auto index = [&](int q) { return ((q / E::kVec) * 32 + lane) * E::kVec + q % E::kVec; };
      auto at_least = [&](float t) {  // this lane's unmasked values at or above t, as bits
        uint32_t in = 0;
#pragma unroll
        for (int q = 0; q < kLoads * E::kVec; ++q)
          if (value(q) >= t && value(q) > -INFINITY) in |= 1u << q;
        return in;
      };
      // (nsel tiles share room for top^2 candidates)
      uint32_t in = at_least(thr);
      int all = __reduce_add_sync(0xffffffffu, __popc(in));
      if (all > room) {
        // too many: `top` lanes hold a value at or above the top-th largest lane maximum
        float lane_max = -INFINITY, t = -INFINITY;
#pragma unroll
        for (int q = 0; q < kLoads * E::kVec; ++q) lane_max = fmaxf(lane_max, value(q));
        for (int k = 0; k < a.top; ++k) {
          t = redux_max(lane_max);
          const unsigned who = __ballot_sync(0xffffffffu, lane_max == t);
          if (lane == __ffs(who) - 1) lane_max = -INFINITY;
        }
        if (t > thr) {
          in = at_least(t);
          all = __reduce_add_sync(0xffffffffu, __popc(in));
        }
      }
      if (all <= room) {
        if (in) {
          int at = atomicAdd(ncand, __popc(in));
#pragma unroll
          for (int q = 0; q < kLoads * E::kVec; ++q)
            if (in >> q & 1) cand[at++] = cand_key(value(q), (uint32_t)(ts + index(q)));
        }
      } else {  // many equal values: take the best ones in turn
        for (int round = 0; round < a.top; ++round) {
          float best = -INFINITY;
          int bq = -1;
#pragma unroll
          for (int q = 0; q < kLoads * E::kVec; ++q)
            if ((in >> q & 1) && value(q) > best) {  // in index order: the first of equal values stays
              best = value(q);
              bq = q;
            }
          const float M = redux_max(best);
          const int bi = bq < 0 ? 0x7FFFFFFF : index(bq);
          const int w = (int)__reduce_min_sync(0xffffffffu, best == M ? (unsigned)bi : 0x7FFFFFFFu);
          if (lane == 0) cand[atomicAdd(ncand, 1)] = cand_key(M, (uint32_t)(ts + w));
          if (bi == w) in &= ~(1u << bq);
        }
      }
    }
  }

  // ---------------------------------------------------------------- join the cluster, write the row
  __syncwarp();
  if (CLUSTER) cluster.sync();  // the last access to another CTA's memory was before it
  else __syncthreads();
  if (rank == 0) {
    if (warp == 0) {
      CtaPart p = s_part[0];
      if (CLUSTER) p = join_parts(lane < C ? s_part[lane] : CtaPart{0.f, 0.f, -INFINITY, 0}, a.c);
      if (lane == 0) {
        const float nan = __int_as_float(0x7FC00000);
        double logS = log1p((double)p.S);
        float lp, H, m = p.R;
        uint32_t fl = 0;
        if (p.bad) {
          fl |= DSPARK_FLAG_NONFINITE;
          m = nan;
          logS = (double)nan;
          lp = H = nan;
        } else if (!(p.R > -INFINITY)) {  // nothing in the row is unmasked
          logS = -INFINITY;
          lp = -INFINITY;
          H = 0.f;
        } else {
          H = (float)(logS - (double)p.E / (1.0 + (double)p.S) * kLn2D);
          lp = 0.f;
        }
        if (!in_range) {
          fl |= DSPARK_FLAG_TOKEN_RANGE;
          lp = nan;
        } else if (!p.bad && p.R > -INFINITY) {
          lp = (float)(((double)x_tok - (double)p.R) * a.inv_T - logS);
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
      const int nc = s_ncand;
      for (int i = tid; i < nc; i += kLpThreads) {
        const uint64_t k = s_cand[i];
        const int place = rank_of(k, s_cand, nc);
        if (place < a.top) s_top[place] = k;
      }
      __syncthreads();
      const bool nan_row = isnan(s_m);
      if (tid < a.top) {
        const bool have = tid < nc && !nan_row;
        const uint64_t k = have ? s_top[tid] : 0;
        a.top_idx[n * a.top + tid] = have ? (int32_t)~(uint32_t)k : -1;
        a.top_logp[n * a.top + tid] = have      ? (float)(((double)key_value(k) - s_m) * a.inv_T - s_logS)
                                      : nan_row ? __int_as_float(0x7FC00000)
                                                : -INFINITY;
      }
    }
  }
}

// ============================================================================ backward

// 16 KB of a row per CTA, eight vectors a thread in flight.  2048 x 151936 bf16 takes 182 us (6.5 TB/s);
// 256 threads with 2, 4, 8 or 16 vectors 237, 205, 192 and 211, 128 with 16 186.
constexpr int kLbThreads = 128;
constexpr int kLbVecs = 8;

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
  float inv_T, c;  // 1 / T, log2(e) / T
  int vec;  // every row of logits and grad starts at the same offset within 16 bytes
};

// Rounding to the logits' type, one value or a 16-byte vector of pairs.
template <int DT>
__device__ __forceinline__ typename Elem<DT>::T to_elem(float x);
template <>
__device__ __forceinline__ float to_elem<DSPARK_F32>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_elem<DSPARK_BF16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half to_elem<DSPARK_F16>(float x) { return __float2half_rn(x); }
template <int DT>
__device__ __forceinline__ void put_pair(uint4& o, int i, float2 v) {
  if (DT == DSPARK_F32) {
    (i == 0 ? o.x : o.z) = __float_as_uint(v.x);
    (i == 0 ? o.y : o.w) = __float_as_uint(v.y);
    return;
  }
  uint32_t w;
  if (DT == DSPARK_BF16) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v.x, v.y);
    w = *reinterpret_cast<const uint32_t*>(&t);
  } else {
    const __half2 t = __floats2half2_rn(v.x, v.y);
    w = *reinterpret_cast<const uint32_t*>(&t);
  }
  (i == 0 ? o.x : i == 1 ? o.y : i == 2 ? o.z : o.w) = w;
}

// A row's coefficients: dl = (indicators) / T + p (k1 log2 p + k0), log2 p = (l - m) c - s
struct LbRow {
  float m, s, c, k1, k0;
  __device__ __forceinline__ float2 dense(float2 x) const {
    float2 lp = p_fma(p_add(x, make_float2(-m, -m)), make_float2(c, c), make_float2(-s, -s));
    lp = make_float2(fmaxf(lp.x, -1e4f), fmaxf(lp.y, -1e4f));  // 2^-1e4 is 0; keeps 0 * inf out
    return p_mul(make_float2(ex2(lp.x), ex2(lp.y)), p_fma(lp, make_float2(k1, k1), make_float2(k0, k0)));
  }
  __device__ __forceinline__ float dense(float x) const { return dense(make_float2(x, x)).x; }
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

  pdl_wait();
  pdl_trigger();
  const int tok = a.tokens[n];
  const float2 st = a.stats[n];
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
  const int nv = a.vec ? (hi - body) / E::kVec : 0;
  const uint4* q = reinterpret_cast<const uint4*>(p + body);
  uint4 v[kLbVecs];
#pragma unroll
  for (int j = 0; j < kLbVecs; ++j)
    if (j * kLbThreads + tid < nv) v[j] = q[j * kLbThreads + tid];
  const float gl = a.g_logp ? a.g_logp[n] : 0.f;
  const float gH = a.g_entropy ? a.g_entropy[n] : 0.f;
  float G = gl;
  const int32_t* ti = a.top ? a.top_idx + n * a.top : nullptr;
  const float* gt = a.top ? a.g_top + n * a.top : nullptr;
  for (int j = 0; j < a.top; ++j)
    if ((unsigned)ti[j] < (unsigned)a.V) G += gt[j];
  LbRow r;
  r.m = st.x;
  r.s = st.y * kLog2e;
  r.c = a.c;
  r.k1 = -a.inv_T * gH * (float)kLn2D;
  r.k0 = -a.inv_T * (gH != 0.f ? fmaf(gH, a.entropy[n], G) : G);
  if (!(st.x < INFINITY)) r.k0 = __int_as_float(0x7FC00000);  // a row with NaN or +inf: its gradient is NaN

  // elements with an indicator: thread j < top + 1 owns index j if it is its first occurrence.  The
  // value is formed before the dense pass overwrites the logit (grad may be the logits themselves).
  int own = -1;
  float fix = 0.f;
  if (tid <= a.top) {
    const int idx = tid == 0 ? tok : ti[tid - 1];
    bool first = idx >= lo && idx < hi;
    if (first && tid > 0) {
      first = idx != tok;
      for (int j = 0; first && j < tid - 1; ++j) first = ti[j] != idx;
    }
    if (first) {
      float add = tid == 0 ? gl : 0.f;
      for (int j = 0; j < a.top; ++j)
        if (ti[j] == idx) add += gt[j];
      own = idx;
      const float x = E::get(p[idx]), lp2 = fmaf(x - r.m, r.c, -r.s), pr = ex2(lp2);
      if (pr > 0.5f)  // 1 - p from log p, so that a dominant token's gradient keeps its digits
        fix = a.inv_T * ((add - G) - G * expm1f(lp2 * (float)kLn2D) -
                         (gH != 0.f ? pr * gH * fmaf(lp2, (float)kLn2D, a.entropy[n]) : 0.f));
      else
        fix = r.dense(x) + add * a.inv_T;
    }
  }
  __syncthreads();

  if (a.vec) {
    for (int i = lo + tid; i < body; i += kLbThreads) g[i] = to_elem<DT>(r.dense(E::get(p[i])));
    uint4* o = reinterpret_cast<uint4*>(g + body);
#pragma unroll
    for (int j = 0; j < kLbVecs; ++j)
      if (j * kLbThreads + tid < nv) {
        uint4 e;
#pragma unroll
        for (int i = 0; i < E::kVec / 2; ++i) put_pair<DT>(e, i, r.dense(E::pair(v[j], i)));
        o[j * kLbThreads + tid] = e;
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

template <int DT, int W, bool CLUSTER>
static cudaError_t launch_lp(const LpArgs& a, int N, int C, int nt, cudaStream_t st) {
  auto kern = token_logprobs_kernel<DT, W, CLUSTER>;
  const size_t smem = (size_t)a.top * a.top * 8 + (size_t)nt * 4;
  cudaError_t rc = ensure_smem_attr((const void*)kern, smem);
  if (rc == cudaSuccess && C > 8) rc = ensure_nonportable_cluster((const void*)kern);
  if (rc != cudaSuccess) return rc;
  return launch_dependent(kern, (long long)N * C, W * 32, smem, st, C, a);
}

template <int DT>
static dspark_status launch_lp(const LogprobsCall& c) {
  constexpr int kTile = RowTiles<DT>::kTile;
  const long long nt = ((long long)c.V + kTile - 1) / kTile + 1;
  // CTAs per row: while the rows alone leave SMs idle (two CTAs of 16 warps per SM), split rows of at
  // least 8 tiles a warp, down to one tile a warp (at most 1, 2, 4, 8 and 16 CTAs: one row of 151936 fp32
  // with 20 alternatives 13.9, 10.4, 8.7, 7.8 and 7.6 us; 64 rows with 8 16.6, 13.5 and 12.8; 77 rows of
  // 50001 fp16, 6 tiles a warp, 8.4 by one CTA each and 10.1 by two)
  const long long slots = 2ll * device_sm_count();
  int C = 1;
  while (C < kLpMaxCluster && (long long)c.N * 2 * C <= slots && nt >= 128 && nt / (2 * C) >= 16) C *= 2;
  LpArgs a{c.logits, c.ld, c.rows, c.n_rows, c.tokens, c.V, c.top, 1.0 / (double)c.T, (float)(1.0 / (kLn2D * (double)c.T)),
           c.logp, c.entropy, c.top_idx, c.top_logp, reinterpret_cast<float2*>(c.stats), c.flags};
  // warps per CTA by the row's tiles, so that a warp has enough of them for the row's end to cost little
  // (2, 4 and 8 warps: 2000 x 12000 fp32 21.3, 23.3 and 28.7 us; 700 x 50000 fp32 38, 28.8 and 34 us;
  // 1000 x 100001 bf16 63, 51 and 46 us)
  int W = nt <= 32 ? 2 : nt <= 128 ? 4 : 8;
  // and more of them while the rows leave the SMs half empty (32 warps each)
  while (W < 16 && 2ll * W * c.N <= 16 * slots && nt >= 4 * W) W *= 2;
  auto one = W == 2   ? launch_lp<DT, 2, false>
             : W == 4 ? launch_lp<DT, 4, false>
             : W == 8 ? launch_lp<DT, 8, false>
                      : launch_lp<DT, 16, false>;
  cudaError_t rc = C > 1 ? launch_lp<DT, 16, true>(a, c.N, C, (int)nt, c.stream) : one(a, c.N, 1, (int)nt, c.stream);
  if (rc != cudaSuccess && C > 8) {  // no clusters of 16 here
    cudaGetLastError();
    rc = launch_lp<DT, 16, true>(a, c.N, 8, (int)nt, c.stream);
  }
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
           c.g_entropy, c.top_idx, c.g_top, c.V, c.top, chunks, 1.f / c.T, (float)(1.0 / (kLn2D * (double)c.T)), vec ? 1 : 0};
  const cudaError_t rc = launch_dependent(token_logprobs_bwd_kernel<DT>, grid, kLbThreads, 0, c.stream, 1, a);
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
