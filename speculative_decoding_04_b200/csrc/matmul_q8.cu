// Integer matrix product with scales: out[m, n] = q_scale[m] * w_scale[n] * sum_k q[m, k] w[n, k].
//
// The product is computed transposed on the tensor cores (tcgen05.mma kind::i8, int32 accumulators in
// tensor memory): the weights' rows n are the MMA's M dimension (the 128 TMEM lanes) and the tokens m
// its N dimension (TMEM columns), so that a few tokens waste no MMA rows and a warp's store covers 32
// consecutive outputs of one token.  Both operands are K-major as they lie in memory: TMA boxes of 128
// bytes of K (128-byte swizzle) by BV weight rows or BN tokens; K and rows past the end read as zero.
//   warp 0      TMA producer, a ring of stages [BV x 128 B of weights | BN x 128 B of tokens]
//   warp 1      MMA issuer: per stage 4 steps of K = 32, for one or two blocks of 128 weight rows
//   warp 2      TMEM allocation
//   warps 4-19  epilogue: TMEM -> registers, the two scales, stores
// Persistent: one CTA per SM takes tiles in turn, the token tiles of one weight tile next to each
// other, so that a weight tile comes from HBM once.
//
// The sum is exact (int32: K <= 131071 keeps |sum| below 2^31 even for -128 * -128); it is rounded to
// fp32 once, multiplied by the two scales in fp32 and rounded once to the output's type.

#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>
#include <string>

#include "common.cuh"
#include "internal.h"

namespace dspark {

namespace {

constexpr int kMqThreads = 640;
constexpr int kMqEpiWarps = 16;
constexpr int kMqKB = 128;    // bytes (= values) of a block of K: one swizzled row
constexpr int kMqBlocks = 2;  // blocks of K per stage
constexpr int kMqMaxStages = 8;
constexpr uint32_t kMqSmem = 227u * 1024u;
// Tokens of one single-CTA call; more than this: CTA pairs.  (One CTA a tile against pairs, in a row of calls,
// measured at two large vocabularies only: 151936 x 4096, fp32 out, 40 tokens 101 and 107 us, 80 108 and 113,
// 84 116 and 112, 100 124 and 117, 128 131 and 122; 129280 x 2048, bf16 out, 64 48 and 49, 84 57 and 50, 128 59
// and 55.)
constexpr int kMqMaxTokens = 80;

struct MqArgs {
  const float* q_scale;
  const float* w_scale;
  void* out;
  long long ldo;
  uint32_t* flags;
  int M, N, K;
  int bv, bn;          // tile: weight rows (multiple of 16, <= 256), tokens (multiple of 16, <= 256)
  int ntok, ntiles;    // token tiles; tiles in all
  int stages, blocks, tmem_cols;
  uint32_t w_bytes, x_bytes;            // one block of K: bytes of the tile's weights and tokens
  uint32_t x_off, stage_bytes, bars;    // tokens within a stage; a stage; barriers after the stages
  uint32_t out_off;                     // (CTA pairs) staging of the output
  int out_tma;                          // (CTA pairs) the output takes TMA stores
  uint32_t spin_limit;                  // polls before a bounded wait gives up
  int barrier_extra;                    // test-only: arrivals the accumulators' barriers expect beyond the commit
  int lost_warp;                        // test-only: an epilogue warp whose waits count as given up, or -1
};

// Tensor maps of the weights and the tokens: [rows, K] with boxes of 128 bytes of K by the tile's rows,
// and the same matrix as [K / 128][rows][128 bytes] with boxes of two blocks.  One copy of two blocks
// streams faster than two of one (single calls behind a flush of L2, when it was chosen: 1088 x 151936 x 4096
// 485 against 530 us, one token 115 against 121; in a row of calls they take 580-615 and 94); the last odd or
// partial block comes by the first map, which ends at K.
struct MqMaps {
  CUtensorMap w, x, w3, x3;
  CUtensorMap out;  // [M, N] of the output's type in boxes of kOutTokens x 128 (CTA pairs, out_tma)
};

struct MqParams {
  MqMaps tm;
  MqArgs a;
};

// A position in the ring of stages, advanced without divisions: the loops that issue copies and MMAs
// have a few hundred cycles a stage.
struct MqRing {
  int s;
  uint32_t phase;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
  }
};

struct MqSync {
  volatile int* abort;
  uint32_t limit;
};

// Bounded wait shared by all roles; after any timeout every later wait that has to wait returns at once.
__device__ __forceinline__ bool mq_wait(const MqSync& s, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*s.abort) return false;
  for (uint32_t i = 0; i < s.limit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023u) == 1023u && *s.abort) return false;
  }
  *s.abort = 1;
  return false;
}

__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns (no wait).
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Waits for the loads issued so far.  It names the registers of the load, so that nothing uses or copies
// them between the two.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

template <int DT>
__device__ __forceinline__ void store_out(void* out, long long i, float v) {
  if (DT == DSPARK_F32) static_cast<float*>(out)[i] = v;
  else if (DT == DSPARK_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[i] = __float2half_rn(v);
}

template <int DT>
__global__ void __launch_bounds__(kMqThreads, 1)
    matmul_q8_kernel(const __grid_constant__ MqParams p) {
  const MqMaps& tm = p.tm;
  const MqArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + a.bars);
  uint64_t* empty = full + kMqMaxStages;
  uint64_t* t_full = empty + kMqMaxStages;
  uint64_t* t_empty = t_full + 2;
  uint64_t* drain = t_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const MqSync sy{s_abort, a.spin_limit};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nkb = (a.K + kMqKB - 1) / kMqKB;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&t_full[i], 1 + a.barrier_extra);
      mbar_init(&t_empty[i], kMqEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tm.w3);
    prefetch_tmap(&tm.x3);
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, a.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // barriers and tensor memory are set up while the previous kernel ends
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      MqRing r{0, 0};
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < a.ntiles; t += gridDim.x) {
        const int v0 = (t / a.ntok) * a.bv, m0 = (t % a.ntok) * a.bn;
        for (int k = 0; k < nkb; k += kMqBlocks, ++it, r.next(a.stages)) {
          const int s = r.s;
          if (!mq_wait(sy, &empty[s], r.phase ^ 1u)) {
            ok = false;
            break;
          }
          uint8_t* st = sm + s * a.stage_bytes;
          const int nb = min(kMqBlocks, nkb - k);
          mbar_arrive_expect_tx(&full[s], (uint32_t)(a.bv + a.bn) * kMqKB * nb);
          if ((k + kMqBlocks) * kMqKB <= a.K) {
            tma_load_3d(st, &tm.w3, 0, v0, k, &full[s]);
            tma_load_3d(st + a.x_off, &tm.x3, 0, m0, k, &full[s]);
          } else {
            for (int i = 0; i < nb; ++i) {
              tma_load_2d(st + i * a.w_bytes, &tm.w, (k + i) * kMqKB, v0, &full[s]);
              tma_load_2d(st + a.x_off + i * a.x_bytes, &tm.x, (k + i) * kMqKB, m0, &full[s]);
            }
          }
        }
      }
      // the copies already issued land (bounded) before the CTA exits, whoever was to wait for them
      for (int i = max(0, it - a.stages); i < it; ++i)
        for (uint32_t n = 0; n < kSpinLimit && !mbar_try_wait(&full[i % a.stages], (i / a.stages) & 1); ++n) {
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = (2u << 4)                          // D int32
                             | (1u << 7) | (1u << 10)           // A, B signed 8-bit
                             | ((uint32_t)(a.bn >> 3) << 17)    // N
                             | ((uint32_t)(128 >> 4) << 24);    // M
      MqRing r{0, 0}, acc_r{0, 0};
      const uint64_t desc0 = smem_desc(smem_u32(sm), 16u, 1024u, 2u);  // + bytes / 16 for any stage and block
      bool ok = true;
      for (int t = blockIdx.x; ok && t < a.ntiles; t += gridDim.x, acc_r.next(2)) {
        const int buf = acc_r.s;
        if (!mq_wait(sy, &t_empty[buf], acc_r.phase ^ 1u)) break;
        tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)(buf * a.blocks * a.bn);
        for (int k = 0; k < nkb; k += kMqBlocks, r.next(a.stages)) {
          const int s = r.s;
          if (!mq_wait(sy, &full[s], r.phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t st = desc0 + ((uint32_t)s * a.stage_bytes >> 4);
          for (int i = 0; i < kMqBlocks && k + i < nkb; ++i) {
            const uint64_t w = st + (i * a.w_bytes >> 4), x = st + ((a.x_off + i * a.x_bytes) >> 4);
            for (int b = 0; b < a.blocks; ++b)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc_mma_i8(acc + (uint32_t)(b * a.bn), w + (b * 1024u + kk * 2u), x + kk * 2u, idesc,
                          (k | i | kk) != 0 ? 1u : 0u);
          }
          tc_commit(&empty[s]);
        }
        if (ok) tc_commit(&t_full[buf]);
      }
      tc_commit(drain);  // tensor memory and the stages stay until the MMAs already issued are done (bounded)
      mbar_wait(drain, 0);
    }
  } else if (warp >= 4) {
    // lane quadrant, block of 128 weight rows, and which of the alternating chunks of 16 tokens: the last
    // tile's epilogue runs alone (128 x 50000 x 1024 took 29 us with half as many warps and 25 with these)
    const int q = warp & 3, b = ((warp - 4) >> 2) & 1, h = (warp - 4) >> 3;
    // A warp whose wait gave up is done with the barriers: a parity does not tell a phase from the one two
    // later, and an arrival more would hand an accumulator on that other warps still read.  It writes NaN
    // from there on; the issuer, without its arrivals, gives up too.
    bool ok = warp != a.lost_warp;
    MqRing acc_r{0, 0};
    for (int t = blockIdx.x; t < a.ntiles; t += gridDim.x, acc_r.next(2)) {
      const int buf = acc_r.s;
      const int v = (t / a.ntok) * a.bv + b * 128 + q * 32 + lane, m0 = (t % a.ntok) * a.bn;
      const bool mine = b < a.blocks && b * 128 + q * 32 + lane < a.bv && v < a.N;
      const int nm = min(a.bn, a.M - m0);
      // both scales before the wait: lane i holds the tokens' i, i + 32, ...
      const float sw = mine ? a.w_scale[v] : 0.f;
      float sq[3];
      static_assert(kMqMaxTokens <= 3 * 32, "three scales a lane");
#pragma unroll
      for (int i = 0; i < 3; ++i) sq[i] = i * 32 + lane < nm ? a.q_scale[m0 + i * 32 + lane] : 0.f;
      ok = __all_sync(0xffffffffu, ok && mq_wait(sy, &t_full[buf], acc_r.phase));
      tc_fence_after();
      if (b < a.blocks) {
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)((buf * a.blocks + b) * a.bn);
#pragma unroll 1
        for (int c = h * 16; c < nm; c += 32) {
          const float sc = c < 32 ? sq[0] : c < 64 ? sq[1] : sq[2];
          uint32_t r[16];
          if (ok) {
            tmem_ld_x16(acc + c, r);
            tmem_wait_ld(r);
          }
          // all values before the first store: one branch a value cost 0.8 us a chunk
          float o[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float s = __shfl_sync(0xffffffffu, sc, (c + j) & 31);
            o[j] = ok ? (float)(int32_t)r[j] * s * sw : __int_as_float(0x7FC00000);
          }
          long long at = (long long)(m0 + c) * a.ldo + v;
          if (mine && c + 16 <= nm) {
#pragma unroll
            for (int j = 0; j < 16; ++j, at += a.ldo) store_out<DT>(a.out, at, o[j]);
          } else if (mine) {
#pragma unroll
            for (int j = 0; j < 15; ++j, at += a.ldo)
              if (c + j < nm) store_out<DT>(a.out, at, o[j]);
          }
          __syncwarp();
        }
        if (!ok && a.flags && __any_sync(0xffffffffu, mine)) {  // each warp for the tokens it wrote as NaN
          for (int c = h * 16 + lane; lane < 16 && c < nm; c += 32) atomicOr(a.flags + m0 + c, DSPARK_FLAG_DEVICE_TIMEOUT);
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&t_empty[buf]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, a.tmem_cols);
}

// ---------------------------------------------------------------------------- CTA pairs
//
// The same product for many tokens: a cluster of two CTAs shares one tile of 256 weight rows by bn
// tokens (tcgen05.mma.cta_group::2, M = 256).  Each CTA loads its 128 weight rows and half of the
// tokens, so a tile's operands cross from L2 to shared memory once per pair, and holds the accumulators
// of its rows: bn columns of tensor memory, twice, so that the epilogue of one tile runs beside the
// products of the next.  Rank 0 issues the MMAs; both CTAs' loads complete on rank 0's full barriers,
// and the commits arrive on both CTAs' empty and accumulator barriers.

constexpr int kPairGroups = 4;  // of four epilogue warps
constexpr int kPairEpiWarps = 4 * kPairGroups;
constexpr int kPairThreads = 128 + 32 * kPairEpiWarps;
static_assert(kPairThreads == kMqThreads, "the last warp of either form");
constexpr int kPairMaxStages = 8;
constexpr int kOutTokens = 16;  // tokens of one staged store

__device__ __forceinline__ uint32_t mapa_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Load into this CTA's shared memory, completing on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_mma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

template <int DT>
__global__ void __launch_bounds__(kPairThreads, 1)
    matmul_q8_pair(const __grid_constant__ MqParams p) {
  const MqMaps& tm = p.tm;
  const MqArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + a.bars);  // (rank 0) both CTAs' loads of a stage
  uint64_t* empty = full + kPairMaxStages;                    // the stage's MMAs are done
  uint64_t* t_full = empty + kPairMaxStages;                  // [2] an accumulator is complete
  uint64_t* t_empty = t_full + 2;                             // [2] (rank 0) both CTAs have read it
  uint64_t* drain = t_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const MqSync sy{s_abort, a.spin_limit};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int nkb = (a.K + kMqKB - 1) / kMqKB;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int half = a.bn >> 1;  // tokens this CTA loads

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&t_full[i], 1 + a.barrier_extra);
      mbar_init(&t_empty[i], 2 * kPairEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tm.w3);
    prefetch_tmap(&tm.x3);
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"((uint32_t)a.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's barriers are initialised before anything arrives on them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // barriers and tensor memory are set up while the previous kernel ends
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      MqRing r{0, 0};
      int it = 0;
      bool ok = true;
      const uint32_t full0 = mapa_rank(smem_u32(full), 0);
      for (int t = pair; ok && t < a.ntiles; t += npairs) {
        const int v0 = (t / a.ntok) * 256 + (int)rank * 128, m0 = (t % a.ntok) * a.bn + (int)rank * half;
        for (int k = 0; k < nkb; k += kMqBlocks, ++it, r.next(a.stages)) {
          const int s = r.s;
          if (!mq_wait(sy, &empty[s], r.phase ^ 1u)) {
            ok = false;
            break;
          }
          uint8_t* st = sm + s * a.stage_bytes;
          const int nb = min(kMqBlocks, nkb - k);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(256 + a.bn) * kMqKB * nb);
          const uint32_t bar = full0 + 8u * s;
          if ((k + kMqBlocks) * kMqKB <= a.K) {
            tma_load_3d_pair(st, &tm.w3, 0, v0, k, bar);
            tma_load_3d_pair(st + a.x_off, &tm.x3, 0, m0, k, bar);
          } else {
            for (int i = 0; i < nb; ++i) {
              tma_load_2d_pair(st + i * a.w_bytes, &tm.w, (k + i) * kMqKB, v0, bar);
              tma_load_2d_pair(st + a.x_off + i * a.x_bytes, &tm.x, (k + i) * kMqKB, m0, bar);
            }
          }
        }
      }
      // rank 0 lets the copies of both CTAs land (bounded), whoever was to wait for them; rank 1 waits for
      // it at the last cluster barrier.  Where rank 1 gave up it may have issued copies that rank 0 does
      // not count: they land within microseconds
      if (rank == 0) {
        for (int i = max(0, it - a.stages); i < it; ++i)
          for (uint32_t n = 0; n < kSpinLimit && !mbar_try_wait(&full[i % a.stages], (i / a.stages) & 1); ++n) {
          }
      } else if (!ok) {
        __nanosleep(1000000);
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      const uint32_t idesc = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(a.bn >> 3) << 17) |
                             ((uint32_t)(256 >> 4) << 24);
      MqRing r{0, 0}, acc_r{0, 0};
      const uint64_t desc0 = smem_desc(smem_u32(sm), 16u, 1024u, 2u);
      bool ok = true;
      for (int t = pair; ok && t < a.ntiles; t += npairs, acc_r.next(2)) {
        const int buf = acc_r.s;
        if (!mq_wait(sy, &t_empty[buf], acc_r.phase ^ 1u)) break;
        tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)(buf * a.bn);
        for (int k = 0; k < nkb; k += kMqBlocks, r.next(a.stages)) {
          const int s = r.s;
          if (!mq_wait(sy, &full[s], r.phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t st = desc0 + ((uint32_t)s * a.stage_bytes >> 4);
#pragma unroll
          for (int i = 0; i < kMqBlocks; ++i) {
            if (k + i >= nkb) break;
            const uint64_t w = st + (i * a.w_bytes >> 4), x = st + ((a.x_off + i * a.x_bytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_i8_pair(acc, w + kk * 2u, x + kk * 2u, idesc, (k | i | kk) != 0 ? 1u : 0u);
          }
          tc_commit_pair(&empty[s]);
        }
        if (ok) tc_commit_pair(&t_full[buf]);
      }
      tc_commit_pair(drain);  // tensor memory and the stages stay until the MMAs already issued are done (bounded)
      mbar_wait(drain, 0);
    } else if (lane == 0) {
      mbar_wait(drain, 0);  // the last of rank 0's arrivals at this CTA's barriers (bounded)
    }
  } else if (warp >= 4) {
    // The four warps of a group h hold 128 consecutive outputs of a token on their lanes.  Chunks of 16
    // tokens go to the groups in turn; a chunk is scaled and staged in the group's part of shared memory
    // while the next one's accumulators are read.  Where rows take TMA stores (16-byte rows) it is staged
    // as [16][128] and written by one, which also clips it to the matrix.  Other rows are staged at the
    // offset within 16 bytes that they have in memory, so that aligned 16-byte pieces go from one to the
    // other, and what is left at either end value by value.
    constexpr uint32_t kEs = DT == DSPARK_F32 ? 4u : 2u;
    constexpr uint32_t kPitch = 128u * kEs + 16u;  // a row staged at its offset
    constexpr int kPieces = (int)kPitch / 16;      // 16-byte pieces it can touch
    constexpr int kEdge = 16 / (int)kEs;           // values in a piece
    const int q = warp & 3, h = (warp - 4) >> 2, gt = q * 32 + lane;
    const bool issuer = q == 0 && lane == 0;
    uint8_t* stage = sm + a.out_off + (uint32_t)h * (kOutTokens * (a.out_tma ? 128u * kEs : kPitch));
    bool ok = warp != a.lost_warp;  // (as in the form of one CTA)
    MqRing acc_r{0, 0};
    for (int t = pair; t < a.ntiles; t += npairs, acc_r.next(2)) {
      const int buf = acc_r.s;
      const int v0 = (t / a.ntok) * 256 + (int)rank * 128, v = v0 + gt, m0 = (t % a.ntok) * a.bn;
      const float sw = v < a.N ? a.w_scale[v] : 0.f;
      const int nm = min(a.bn, a.M - m0);
      auto scale_of = [&](int c) {  // lanes 0-15: the tokens' scales of the chunk at c
        return c + lane < nm && lane < kOutTokens ? a.q_scale[m0 + c + lane] : 0.f;
      };
      float sq = scale_of(h * kOutTokens);
      ok = __all_sync(0xffffffffu, ok && mq_wait(sy, &t_full[buf], acc_r.phase));
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * a.bn);
      uint32_t r[16];
      if (ok && h * kOutTokens < nm) tmem_ld_x16(acc + h * kOutTokens, r);
      for (int c = h * kOutTokens; c < nm; c += kPairGroups * kOutTokens) {
        if (ok) tmem_wait_ld(r);
        float o[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float s = __shfl_sync(0xffffffffu, sq, j);
          o[j] = ok ? (float)(int32_t)r[j] * s * sw : __int_as_float(0x7FC00000);
        }
        const int cn = c + kPairGroups * kOutTokens;
        if (ok && cn < nm) tmem_ld_x16(acc + cn, r);
        sq = scale_of(cn);
        if (a.out_tma) {
          if (issuer) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          named_bar(1 + h, 128);  // the earlier store has read the stage
#pragma unroll
          for (int j = 0; j < 16; ++j) store_out<DT>(stage, j * 128 + gt, o[j]);
          fence_proxy_async_smem();
          named_bar(1 + h, 128);
          if (issuer && v0 < a.N) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(&tm.out),
                         "r"(smem_u32(stage)), "r"(v0), "r"(m0 + c)
                         : "memory");
          }
          if (issuer) bulk_commit();
        } else {
          uint8_t* base = static_cast<uint8_t*>(a.out) + ((long long)(m0 + c) * a.ldo + v0) * kEs;
          const long long step = a.ldo * kEs;
          named_bar(1 + h, 128);  // the earlier chunk has left the stage
#pragma unroll
          for (int j = 0; j < 16; ++j)
            store_out<DT>(stage + j * kPitch + ((uint32_t)reinterpret_cast<uintptr_t>(base + j * step) & 15u), gt, o[j]);
          named_bar(1 + h, 128);
          const int rows = min(kOutTokens, nm - c), bytes = min(128, a.N - v0) * (int)kEs;
          for (int i = gt; i < rows * kPieces; i += 128) {
            const int row = i / kPieces, at = (i - row * kPieces) * 16;
            uint8_t* to = base + row * step;
            const int shift = (int)((uint32_t)reinterpret_cast<uintptr_t>(to) & 15u);
            if (at >= shift && at + 16 <= shift + bytes)
              *reinterpret_cast<uint4*>(to + at - shift) = *reinterpret_cast<const uint4*>(stage + row * kPitch + at);
          }
          for (int i = gt; i < rows * 2 * kEdge; i += 128) {  // values e of the first and of the last piece
            const int row = i / (2 * kEdge), e = i % kEdge;
            uint8_t* to = base + row * step;
            const int shift = (int)((uint32_t)reinterpret_cast<uintptr_t>(to) & 15u), end = shift + bytes;
            const bool last = (i / kEdge) & 1;
            const int piece = last ? (end - 1) & ~15 : 0, b = piece + e * (int)kEs;
            const bool whole = piece >= shift && piece + 16 <= end;  // then it was written above
            if (whole || b < shift || b >= end || (last && piece == 0)) continue;
            const uint8_t* from = stage + row * kPitch + b;
            if (kEs == 4) *reinterpret_cast<uint32_t*>(to + b - shift) = *reinterpret_cast<const uint32_t*>(from);
            else *reinterpret_cast<uint16_t*>(to + b - shift) = *reinterpret_cast<const uint16_t*>(from);
          }
        }
      }
      if (!ok && a.flags && v0 + q * 32 < a.N)  // each warp for the tokens it wrote as NaN
        for (int c = h * kOutTokens + lane; lane < kOutTokens && c < nm; c += kPairGroups * kOutTokens)
          atomicOr(a.flags + m0 + c, DSPARK_FLAG_DEVICE_TIMEOUT);
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive_cluster(mapa_rank(smem_u32(&t_empty[buf]), 0));
    }
    if (issuer) bulk_wait0();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other may still reach its memory
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)a.tmem_cols)
                 : "memory");
}

template <int DT>
static cudaError_t launch_mq(const MqParams& p, bool pair, int grid, size_t smem, cudaStream_t st) {
  auto kern = pair ? matmul_q8_pair<DT> : matmul_q8_kernel<DT>;
  const cudaError_t rc = ensure_smem_attr((const void*)kern, smem);
  if (rc != cudaSuccess) return rc;
  return launch_dependent(kern, grid, pair ? kPairThreads : kMqThreads, smem, st, pair ? 2 : 1, p);
}

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// The two tensor maps of a [rows, K] byte matrix (128-byte swizzle).
static bool byte_maps(CUtensorMap* m, CUtensorMap* m3, const int8_t* base, uint64_t K, uint64_t rows, uint64_t ld,
                      uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  auto enc = [&](CUtensorMap* to, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(to, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<int8_t*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t d2[2] = {K, rows}, s2[1] = {ld};
  const cuuint32_t b2[2] = {(cuuint32_t)kMqKB, box_rows};
  const bool whole = K % (kMqBlocks * kMqKB) == 0, any = K >= kMqBlocks * kMqKB;
  if (!whole && !enc(m, 2, d2, s2, b2)) return false;
  if (!any) {  // no stage has two whole blocks
    *m3 = *m;
    return true;
  }
  const cuuint64_t d3[3] = {(cuuint64_t)kMqKB, rows, K / kMqKB}, s3[2] = {ld, (cuuint64_t)kMqKB};
  const cuuint32_t b3[3] = {(cuuint32_t)kMqKB, box_rows, (cuuint32_t)kMqBlocks};
  if (!enc(m3, 3, d3, s3, b3)) return false;
  if (whole) *m = *m3;  // not used
  return true;
}

static bool out_map(CUtensorMap* m, void* out, int dtype, uint64_t N, uint64_t M, uint64_t ldo) {
  auto fn = encode_fn();
  if (!fn) return false;
  const CUtensorMapDataType dt = dtype == DSPARK_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : dtype == DSPARK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint64_t dims[2] = {N, M}, strides[1] = {ldo * (dtype == DSPARK_F32 ? 4 : 2)};
  const cuuint32_t box[2] = {128, (cuuint32_t)kOutTokens}, es[2] = {1, 1};
  return fn(m, dt, 2, out, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

dspark_status launch_matmul_q8(const MatmulQ8Call& c) {
  if (c.M == 0) return DSPARK_OK;
  const int sms = device_sm_count();
  MqParams p{};
  MqArgs& a = p.a;
  MqMaps& tm = p.tm;
  a.q_scale = c.q_scale;
  a.w_scale = c.w_scale;
  a.out = c.out;
  a.ldo = c.ldo;
  a.flags = c.flags;
  const Options opt = options();
  a.spin_limit = opt.debug_wait_limit > 0 ? (uint32_t)std::min<long>(opt.debug_wait_limit, kSpinLimit) : kSpinLimit;
  a.barrier_extra = opt.debug_unreachable_barrier == 3 ? 1 : 0;
  a.lost_warp = opt.debug_unreachable_barrier == 4 ? kMqThreads / 32 - 1 : -1;
  a.M = c.M;
  a.N = c.N;
  a.K = c.K;
  const bool pair = c.M > kMqMaxTokens;
  const uint32_t misc = 8 * (2 * kMqMaxStages + 5) + 16;
  const int step = pair ? 32 : 16;
  a.ntok = (c.M + 255) / 256;
  a.bn = ((c.M + a.ntok - 1) / a.ntok + step - 1) / step * step;
  int box_v, box_m, grid;
  if (pair) {
    a.bv = 256;
    a.ntiles = a.ntok * ((c.N + 255) / 256);
    a.tmem_cols = 32;
    while (a.tmem_cols < 2 * a.bn) a.tmem_cols *= 2;
    a.w_bytes = 128 * kMqKB;
    a.x_bytes = (uint32_t)(a.bn / 2 * kMqKB);
    a.x_off = kMqBlocks * a.w_bytes;
    a.stage_bytes = kMqBlocks * (a.w_bytes + a.x_bytes);
    const int es = c.out_dtype == DSPARK_F32 ? 4 : 2;
    const uint32_t staging = kPairGroups * kOutTokens * (128u * es + 16u);
    a.stages = (int)std::min<uint32_t>(kPairMaxStages, (kMqSmem - 1024 - misc - staging) / a.stage_bytes);
    a.out_off = a.stages * a.stage_bytes;
    a.bars = a.out_off + staging;
    // (rows that end within 16 bytes too: a TMA store writes the whole of the 16 bytes that N ends in, over
    // what lies beside the output)
    a.out_tma = (uintptr_t)c.out % 16 == 0 && c.ldo * es % 16 == 0 && (long long)c.N * es % 16 == 0 && c.ldo * es < (1ll << 40);
    box_v = 128;
    box_m = a.bn / 2;
    grid = 2 * std::min(std::max(1, sms / 2), a.ntiles);
  } else {
    // weight rows per tile: the largest tile that gives every CTA the same number of tiles
    // (one token, 151936 x 4096, a single call behind a flush of L2: 115 us; at most 128 rows of 2 or 4
    // blocks of K 123 and 119, 64 of 8 137)
    const int per = std::max(1, (int)((c.N + 256ll * sms - 1) / (256ll * sms)));
    const long long rows = (c.N + (long long)sms * per - 1) / ((long long)sms * per);
    a.bv = (int)std::min(256ll, std::max(16ll, (rows + 15) / 16 * 16));
    a.ntiles = a.ntok * ((c.N + a.bv - 1) / a.bv);
    a.blocks = a.bv > 128 ? 2 : 1;
    a.tmem_cols = 32;
    while (a.tmem_cols < 2 * a.blocks * a.bn) a.tmem_cols *= 2;
    a.w_bytes = (uint32_t)(a.bv * kMqKB);
    a.x_bytes = (uint32_t)(a.bn * kMqKB);
    a.x_off = kMqBlocks * a.w_bytes;
    a.stage_bytes = kMqBlocks * (a.w_bytes + a.x_bytes);
    // an MMA reads 128 weight rows whatever the tile holds: what follows the last stage is readable
    const uint32_t reach = (kMqBlocks - 1) * a.w_bytes + a.blocks * 16384;
    const uint32_t slack = reach > a.stage_bytes ? reach - a.stage_bytes : 0;
    a.stages = (int)std::min<uint32_t>(kMqMaxStages, (kMqSmem - 1024 - misc - slack) / a.stage_bytes);
    a.bars = a.stages * a.stage_bytes + slack;
    box_v = a.bv;
    box_m = a.bn;
    grid = std::min(sms, a.ntiles);
  }
  const size_t smem = 1024 + a.bars + misc;
  if (pair && a.out_tma && !out_map(&tm.out, c.out, c.out_dtype, c.N, c.M, c.ldo)) {
    set_error("dspark_matmul_q8: cuTensorMapEncodeTiled failed for the output");
    return DSPARK_ECUDA;
  }
  if (!byte_maps(&tm.w, &tm.w3, c.w, c.K, c.N, c.ldw, box_v) || !byte_maps(&tm.x, &tm.x3, c.q, c.K, c.M, c.ldq, box_m)) {
    set_error("dspark_matmul_q8: cuTensorMapEncodeTiled failed");
    return DSPARK_ECUDA;
  }
  cudaError_t rc;
  switch (c.out_dtype) {
    case DSPARK_F32: rc = launch_mq<DSPARK_F32>(p, pair, grid, smem, c.stream); break;
    case DSPARK_BF16: rc = launch_mq<DSPARK_BF16>(p, pair, grid, smem, c.stream); break;
    default: rc = launch_mq<DSPARK_F16>(p, pair, grid, smem, c.stream); break;
  }
  if (rc != cudaSuccess) {
    set_error(std::string("matmul_q8 launch: ") + cudaGetErrorString(rc));
    return DSPARK_ECUDA;
  }
  return DSPARK_OK;
}

}  // namespace dspark
