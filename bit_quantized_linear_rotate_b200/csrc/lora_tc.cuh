// The adapters of lora_add.cuh for prompts: tiles of up to 128 tokens of one adapter on
// the tcgen05 tensor cores.
//
//   shrink: v (128 x R)  = x A^T      M = 128 tokens, N = R, K in blocks of 64
//   expand: d (128 x N)  = v B^T      M = 128 tokens, N in blocks of 128, K = R for each number that v is split into
//   out = y + scale d
//
// A cluster of CTAs owns a tile: each CTA takes a share of K for the shrink,
// the partial v are added through distributed shared memory, and each CTA takes a share of N
// for the expand. Bytes bound both: x, y and out once each, so that a tile of 128
// tokens at K = N = 3840 moves 2.9 MB and reads 2 R (K + N) bytes of adapter from L2 (1 MB at
// R = 64; tiles of 64 tokens read it twice as often). The tensor cores
// read their operands from shared memory themselves, which leaves the load-store
// units to x, y and out; with mma.sync fragments straight from global
// memory the M = 8192, R = 64 case (K = N = 3840) took 190 us, so it takes 48.6, where its bytes
// take 29 at the measured copy bandwidth: of a tile's time the list of tiles is 3 us, the shrink
// 12, the exchange of v 5 and the expand 21, which alone is near that bandwidth.
//
// Prompts are mostly tiles of consecutive tokens: then x and y come by tensor copies, and a full
// tile's output leaves by tensor stores. Any other tile is moved by 16-byte asynchronous
// copies and stores of the work warps, or element by element where y's rows do not start on
// 16 bytes.
//
// Warps 0-15 move x of such tiles, later reduce v and finish the output; warp 16 brings in A, B
// and x by tensor copies (rows of another adapter and zeros past the end fill what R leaves of a
// block); warp 17 issues the MMAs; warp 18 brings in y and stores the output. (y by bulk copies of
// one row's 256 bytes was slowest of all: 62 us where 25 had been.)
//
// Shared memory, one area used twice (LoraTc): the shrink's stages, then the partial sums of v,
// v as operands, the ring of B and the ring of y, where the output forms in place. One CTA
// an SM. All barrier waits are bounded; after a timeout the CTA runs on without waiting,
// so that its cluster's barriers are met.
#pragma once

#include <cuda.h>

#include "lora_add.cuh"

namespace ck {
namespace lora {

constexpr int kTcTokens = 128;
constexpr int kWork = 16;                      // warps that move x, y and out
constexpr int kTcThreads = 32 * (kWork + 3);
constexpr int kOp = 128 * 128;                 // bytes of a 128 x 64 operand block, 128-byte swizzle
constexpr int kTcCols = 256;                   // TMEM columns
constexpr int kYStage = 2 * kOp;               // a 128 x 128 block of y: two boxes of 64 columns, 128-byte swizzle

// Offset of row r, 16-byte chunk c (0 .. 15) of a block of y.
__device__ __forceinline__ int y_at(int r, int c) { return (c >> 3) * kOp + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

// Offset of a partial v's 16-byte chunk c (four ranks) of row r, in rows of `width` bytes (a multiple of 256): no two
// lanes of eight that hold chunk c of eight rows meet in a bank.
__device__ __forceinline__ int part_at(int r, int c, int width) { return r * width + ((c ^ (r & 7)) << 4); }

// RB blocks of 64 ranks, v as P numbers.
template <int RB, int P>
struct LoraTc {
  static constexpr int kStageA = RB * 64 * 128;                        // A: up to 64 RB rows
  static constexpr int kStage = kOp + kStageA;
  static constexpr int kPartRow = 64 * RB * 4;                         // partial v: 128 rows
  static constexpr int kV = 128 * kPartRow;                            // offset of v: [RB][P]
  static constexpr int kB = kV + RB * P * kOp;                         // offset of B's ring
  static constexpr int kStagesB = RB == 1 ? 2 : 1;
  static constexpr int kY = kB + kStagesB * RB * kOp;                  // offset of y's ring
  static constexpr int kStagesY = RB == 1 ? 3 : 1;
  static constexpr int kArea = kY + kStagesY * kYStage;
  static constexpr int kStages = RB == 1 ? 8 : 5;
  static constexpr int kSearch = kStages * kStage;                     // offset of the tile search's counters
  static constexpr int kSmem = 1024 + (kArea > kSearch + kPickBytes ? kArea : kSearch + kPickBytes);
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool bf16) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// v is written by this CTA or by others of the cluster, and read by the tensor cores.
__device__ __forceinline__ void fence_proxy_async_cluster() {
  asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_b32x4(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// The halves of cluster_sync.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// a: (L R, K), b: (L N, R), x: (M, K), y and out: (M, N); the last two only where p.vec.
struct TcMaps {
  CUtensorMap a, b, x, y, out;
};

__device__ __forceinline__ void tma_store_2d(const void* tmap, const void* smem, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(smem_u32(smem)), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until at most N of this thread's groups still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 16 TMEM lanes x 32 columns as MMA accumulator fragments: r[4 j ..] holds columns 8 j + 2 (lane % 4)
// and + 1 of row lane / 4, then of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

template <typename T, typename TY, int RB>
__global__ void __launch_bounds__(kTcThreads, 1)
    lora_tc_kernel(const __grid_constant__ TcMaps maps, const Params p) {
  constexpr int P = VOperand<T>::kPlanes;
  using C = LoraTc<RB, P>;
  using Tr = awq::Traits<T>;
  using TrY = awq::Traits<TY>;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* area = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  // the shrink's stages (filled by tensor copies, or with the work warps' help), and its end
  __shared__ uint64_t full1[C::kStages], full2[C::kStages], empty[C::kStages], shrunk;
  __shared__ uint64_t bfull[C::kStagesB], bempty[C::kStagesB], dfull[2], dempty[2];
  __shared__ uint64_t yfull[C::kStagesY], ydone[C::kStagesY];
  __shared__ int abort_flag;
  __shared__ uint32_t tmem_base;
  __shared__ int token[kTcTokens];
  __shared__ float row_scale[kTcTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
  volatile int* abort = &abort_flag;

  if (warp == kWork + 1) {
    tmem_alloc(&tmem_base, kTcCols);
    tmem_relinquish();
  } else if (tid == 32 * kWork) {
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
    prefetch_tmap(&maps.x);
    if (p.vec) {
      prefetch_tmap(&maps.y);
      prefetch_tmap(&maps.out);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full1[s], 1);
      mbar_init(&full2[s], 32 * kWork + 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&shrunk, 1);
    for (int s = 0; s < C::kStagesB; ++s) {
      mbar_init(&bfull[s], 1);
      mbar_init(&bempty[s], 1);
    }
    for (int s = 0; s < C::kStagesY; ++s) {
      mbar_init(&yfull[s], 1);
      mbar_init(&ydone[s], kWork);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&dfull[s], 1);
      mbar_init(&dempty[s], kWork);
    }
    abort_flag = 0;
    fence_mbarrier_init();
  }
  int* search = reinterpret_cast<int*>(area + C::kSearch);
  for (int i = tid; i < kPickBytes / 4; i += kTcThreads) search[i] = 0;
  tc_fence_before();
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  int adapter, n;
  if (p.tiles != nullptr) {
    const int4 tile = __ldcg(reinterpret_cast<const int4*>(p.tiles) + blockIdx.x / ranks);
    adapter = tile.x, n = tile.z;
    if (tid < n) token[tid] = __ldcg(p.order + tile.y + tid);
  } else {
    pick_tile<kTcThreads, kTcTokens>(p, (int)(blockIdx.x / ranks), token, adapter, n, search);
  }
  fence_proxy_async_smem();                                             // tensor copies may come to `search` later
  __syncthreads();
  // consecutive tokens: x by tensor copies; whole 16-byte pieces too: y as well
  const bool seq = __syncthreads_and(tid >= n || token[tid] == token[0] + tid) != 0;
  const bool seq_y = seq && p.vec, dense = seq_y && n == kTcTokens;
  uint64_t* full = seq ? full1 : full2;
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const T* x = reinterpret_cast<const T*>(p.x);
  const TY* y = reinterpret_cast<const TY*>(p.y);
  TY* out = reinterpret_cast<TY*>(p.out);
  const int blocks = (p.N + 127) / 128;                                 // of output columns
  const int b0 = blocks * rank / ranks, b1 = blocks * (rank + 1) / ranks;

  if (n == 0 || adapter < 0) {                                          // the same for the whole cluster
    if (n > 0) copy_rows(y, out, p, token, n, 128 * b0, min(128 * b1, p.N), warp, kWork + 3);
    __syncthreads();
    if (warp == kWork + 1) tmem_dealloc(tmem, kTcCols);
    return;
  }

  const int kblocks = (p.K + 63) / 64;
  const int k0 = kblocks * rank / ranks, k1 = kblocks * (rank + 1) / ranks;
  const int npad = (p.R + 15) / 16 * 16;                                // the shrink's N
  const int steps = npad / 16;                                          // the expand's K steps

  // ------------------------------------------------------------- shrink
  if (warp < kWork && !seq) {
    const int c = tid & 7, r0 = tid >> 3;                               // 16-byte chunk, rows r0 and r0 + 64
    const T* src[2];
    uint32_t dst[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 64 * i;
      src[i] = r < n ? x + token[r] * p.ldx + 8 * c : nullptr;
      dst[i] = smem_u32(area) + r * 128 + ((c ^ (r & 7)) << 4);
    }
    // a stage is handed over kLag blocks after its copies began, and free again some blocks later: two
    // fewer than there are stages, else every block waits for the MMAs of the one just handed over
    constexpr int kLag = C::kStages - 3;
    auto hand_over = [&](int s) {                                       // this thread's copies into stage s are done
      fence_proxy_async_smem();
      mbar_arrive(&full[s]);
    };
    for (int kb = k0; kb < k1; ++kb) {
      const int i = kb - k0, s = i % C::kStages;
      mbar_wait(&empty[s], ((i / C::kStages) & 1) ^ 1, abort, 60);
      const bool in = 64 * kb + 8 * c < p.K;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        cp_async_16(dst[j] + s * C::kStage, in && src[j] != nullptr ? src[j] + 64 * (int64_t)kb : x, in && src[j] != nullptr);
      cp_async_commit();
      if (i >= kLag) {
        cp_async_wait<kLag>();
        hand_over((i - kLag) % C::kStages);
      }
    }
    cp_async_wait<0>();
    for (int i = max(k1 - k0 - kLag, 0); i < k1 - k0; ++i) hand_over(i % C::kStages);
  } else if (warp == kWork) {
    if (lane == 0) {
      int issued = 0;
      for (int kb = k0; kb < k1; ++kb, ++issued) {
        const int i = kb - k0, s = i % C::kStages;
        if (!mbar_wait(&empty[s], ((i / C::kStages) & 1) ^ 1, abort, 61)) break;
        mbar_arrive_expect_tx(&full[s], npad * 128 + (seq ? kOp : 0));
        if (seq) tma_load_2d(area + s * C::kStage, &maps.x, &full[s], 64 * kb, token[0]);   // rows past n: nobody reads them
        tma_load_2d(area + s * C::kStage + kOp, &maps.a, &full[s], 64 * kb, adapter * p.R);
      }
      if (*abort)
        for (int i = issued - 1; i >= 0 && i >= issued - C::kStages; --i)
          mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1, nullptr, 62, 100000000ull);
    }
  } else if (warp == kWork + 1 && lane == 0) {
    const uint32_t id = idesc_f16(128, npad, !VOperand<T>::kScaled);
    for (int kb = k0; kb < k1; ++kb) {
      const int i = kb - k0, s = i % C::kStages;
      if (!mbar_wait(&full[s], (i / C::kStages) & 1, abort, 63)) break;
      tc_fence_after();
      const uint8_t* st = area + s * C::kStage;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_f16(tmem, desc_kmajor_sw128(st, 32 * k), desc_kmajor_sw128(st + kOp, 32 * k), id, i > 0 || k > 0);
      mma_commit(&empty[s]);
    }
    mma_commit(&shrunk);
  }
  __syncwarp();
  const bool any_k = k1 > k0;                                           // few K blocks: some CTAs have none

  // every role waits for the shrink's products: the area changes hands
  mbar_wait(&shrunk, 0, abort, 64);
  __syncwarp();
  auto fetch_b = [&](int i) {                                           // output block b0 + i of B
    const int s = i % C::kStagesB;
    mbar_arrive_expect_tx(&bfull[s], RB * kOp);
    for (int rb = 0; rb < RB; ++rb)
      tma_load_2d(area + C::kB + (s * RB + rb) * kOp, &maps.b, &bfull[s], 64 * rb, adapter * p.N + 128 * (b0 + i));
  };
  const int nb = b1 - b0;
  // A work warp's piece of an output block: rows 32 q .. of the tile (its TMEM lanes), columns 32 cq ..
  const int q = warp & 3, cq = warp >> 2;
  // Block i of y into its ring stage by tensor copies (one thread of warp 18) ...
  auto copy_y = [&](int i) {
    const int s = i % C::kStagesY, c0 = 128 * (b0 + i), boxes = c0 + 64 < p.N ? 2 : 1;
    mbar_arrive_expect_tx(&yfull[s], boxes * kOp);
    for (int h = 0; h < boxes; ++h)
      tma_load_2d(area + C::kY + s * kYStage + h * kOp, &maps.y, &yfull[s], c0 + 64 * h, token[0]);
  };
  // ... or a work warp's piece of it: 4 lanes a row, 8 rows at a time; rows that do not start on 16 bytes
  // element by element, a column a lane.
  auto fetch_y = [&](int i) {
    uint8_t* to = area + C::kY + (i % C::kStagesY) * kYStage;
    const int c0 = 128 * (b0 + i) + 32 * cq;
    if (p.vec) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 32 * q + 8 * j + (lane >> 2), col = c0 + 8 * (lane & 3);
        const bool in = r < n && col < p.N;
        cp_async_16(smem_u32(to + y_at(r, 4 * cq + (lane & 3))), in ? y + token[r] * p.ldy + col : y, in);
      }
    } else if (c0 + lane < p.N) {
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 8) {
        TY e[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) e[r] = y[token[min(32 * q + r0 + r, n - 1)] * p.ldy + c0 + lane];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          reinterpret_cast<TY*>(to + y_at(32 * q + r0 + r, 4 * cq + (lane >> 3)))[lane & 7] = e[r];
      }
    }
  };
  if (warp < kWork) {
    tc_fence_after();
    for (int c0 = 16 * cq; c0 < p.R; c0 += 64) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(tmem + ((uint32_t)(32 * q) << 16) + c0, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        if (c0 + i < p.R)
          *reinterpret_cast<float4*>(area + part_at(32 * q + lane, (c0 + i) >> 2, C::kPartRow)) =
              any_k ? make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]),
                                  __uint_as_float(v[i + 3]))
                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    tc_fence_before();
    __syncwarp();
    cluster_arrive();
    if (!seq_y) {                                                       // while v is exchanged
      if (nb > 0) fetch_y(0);
      cp_async_commit();                                                // a group a block, empty ones too
    }
  } else {                                                              // the first copies take 3 us to issue: arrive before
    __syncwarp();
    cluster_arrive();
    if (warp == kWork && lane == 0)
      for (int i = 0; i < min(nb, C::kStagesB); ++i) fetch_b(i);
    if (warp == kWork + 2 && lane == 0 && seq_y)
      for (int i = 0; i < min(nb, C::kStagesY); ++i) copy_y(i);
  }
  __syncwarp();
  cluster_wait();
  // The partial v of all ranks, added: in a cluster of two every CTA does all rows for itself, in a larger
  // one a share of them for all (reading everything from everybody took 9 us in a cluster of 8, this 3).
  // A power of two of lanes a row, 8 entries a lane.
  if (warp < kWork) {
    const float as = p.scales != nullptr ? __ldg(p.scales + adapter) : 1.0f;
    int lw = 1;
    while (1 << lw < 2 * steps) ++lw;
    const int l = lane & ((1 << lw) - 1), per = 32 >> lw;
    const bool alone = ranks <= 2;
    const int rows = alone ? kTcTokens : (kTcTokens + ranks - 1) / ranks, r0 = alone ? 0 : rank * rows;
    const int d0 = alone ? rank : 0, d1 = alone ? rank + 1 : ranks;     // the CTAs that get the sums
    for (int i = per * warp + (lane >> lw); i < (rows + per - 1) / per * per; i += per * kWork) {   // whole warps
      const int r = r0 + i;
      const bool mine = i < rows && r < kTcTokens;
      float v[8] = {};
      if (mine && 8 * l < p.R) {
        const uint32_t at0 = smem_u32(area) + part_at(r, 2 * l, C::kPartRow);
        const uint32_t at1 = smem_u32(area) + part_at(r, 2 * l + 1, C::kPartRow);
        float4 a[8], b[8];                                              // all ranks' loads before the first use
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < ranks) {
            a[k] = ld_cluster_f32x4(mapa_shared(at0, k));
            b[k] = ld_cluster_f32x4(mapa_shared(at1, k));
          }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < ranks) {
            v[0] += a[k].x, v[1] += a[k].y, v[2] += a[k].z, v[3] += a[k].w;
            v[4] += b[k].x, v[5] += b[k].y, v[6] += b[k].z, v[7] += b[k].w;
          }
      }
      int ex = 0;
      if constexpr (VOperand<T>::kScaled) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1)
          if (o >> lw == 0) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        ex = scale_exponent(top);
      }
      const float up = exp2_int(ex);
      alignas(16) T planes[P][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        T part[P];
        split(v[j] * up, part);
#pragma unroll
        for (int k = 0; k < P; ++k) planes[k][j] = part[k];
      }
      if (mine && l < 2 * steps) {
        const uint32_t at = smem_u32(area) + C::kV + (l >> 3) * P * kOp + r * 128 + (((l & 7) ^ (r & 7)) << 4);
        for (int k = d0; k < d1; ++k) {
          const uint32_t to = mapa_shared(at, k);
#pragma unroll
          for (int i = 0; i < P; ++i) st_cluster_b32x4(to + i * kOp, *reinterpret_cast<const uint4*>(planes[i]));
        }
      }
      if (mine && l == 0)
        for (int k = d0; k < d1; ++k) st_cluster_f32(mapa_shared(smem_u32(row_scale) + 4 * r, k), as * exp2_int(-ex));
    }
    fence_proxy_async_cluster();                                        // v is read by the tensor cores
  }
  __syncwarp();
  cluster_sync();
  fence_proxy_async_cluster();

  // ------------------------------------------------------------- expand
  if (warp < kWork) {
    if (!seq_y) {
#pragma unroll
      for (int i = 1; i < C::kStagesY; ++i) {
        if (i < nb) fetch_y(i);
        cp_async_commit();
      }
    }
    const int g = lane >> 2, t = lane & 3;
    float f[4];                                                         // scales of rows g + 8 k
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = row_scale[32 * q + g + 8 * k];
    for (int i = 0; i < nb; ++i) {
      const int ys = i % C::kStagesY;
      uint8_t* yb = area + C::kY + ys * kYStage;
      const int c0 = 128 * (b0 + i) + 32 * cq;
      if (seq_y) mbar_wait(&yfull[ys], (i / C::kStagesY) & 1, abort, 70);
      else cp_async_wait<C::kStagesY - 1>();                            // block i of y is here
      mbar_wait(&dfull[i & 1], (i >> 1) & 1, abort, 65);
      __syncwarp();
      tc_fence_after();
      uint32_t d[2][16];
      const uint32_t ta = tmem + ((uint32_t)(32 * q) << 16) + 128 * (i & 1) + 32 * cq;
      tmem_ld_16x256b_x4(ta, d[0]);
      tmem_ld_16x256b_x4(ta + (16u << 16), d[1]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&dempty[i & 1]);
      // rows g + 8 k, columns 8 j + 2 t: all loads before the first store, which they might otherwise wait for
      // (0.95 us a block like that, 0.7 so)
      uint32_t u[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          u[k][j] = reinterpret_cast<const uint32_t*>(yb + y_at(32 * q + g + 8 * k, 4 * cq + j))[t];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          TY* v = reinterpret_cast<TY*>(&u[k][j]);
          v[0] = TrY::fromf(fmaf(f[k], __uint_as_float(d[k >> 1][4 * j + 2 * (k & 1)]), TrY::tof(v[0])));
          v[1] = TrY::fromf(fmaf(f[k], __uint_as_float(d[k >> 1][4 * j + 2 * (k & 1) + 1]), TrY::tof(v[1])));
        }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          reinterpret_cast<uint32_t*>(yb + y_at(32 * q + g + 8 * k, 4 * cq + j))[t] = u[k][j];
      if (!dense) {
        __syncwarp();
        if (p.vec) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 32 * q + 8 * j + g, col = c0 + 8 * t;
            if (r < n && col < p.N)
              *reinterpret_cast<uint4*>(out + token[r] * p.ldo + col) =
                  *reinterpret_cast<const uint4*>(yb + y_at(r, 4 * cq + t));
          }
        } else if (c0 + lane < p.N) {
#pragma unroll 8
          for (int r = 32 * q; r < 32 * q + 32; ++r)
            if (r < n)
              out[token[r] * p.ldo + c0 + lane] =
                  reinterpret_cast<const TY*>(yb + y_at(r, 4 * cq + (lane >> 3)))[lane & 7];
        }
      }
      if (seq_y) {
        fence_proxy_async_smem();                                       // a tensor store or copy comes next
        __syncwarp();
        if (lane == 0) mbar_arrive(&ydone[ys]);
      } else {
        __syncwarp();                                                   // the stage is free
        if (i + C::kStagesY < nb) fetch_y(i + C::kStagesY);
        cp_async_commit();
      }
    }
  } else if (warp == kWork + 2) {
    if (lane == 0 && seq_y) {
      int issued = min(nb, C::kStagesY), i = 0;
      for (; i < nb; ++i) {
        const int s = i % C::kStagesY, c0 = 128 * (b0 + i);
        if (!mbar_wait(&ydone[s], (i / C::kStagesY) & 1, abort, 71)) break;
        if (dense) {
          for (int h = 0; h < 2 && c0 + 64 * h < p.N; ++h)
            tma_store_2d(&maps.out, area + C::kY + s * kYStage + h * kOp, c0 + 64 * h, token[0]);
          bulk_commit();
        }
        // the stage of block i - kBack has been read: fetch into it
        constexpr int kBack = C::kStagesY > 1 ? 1 : 0;
        if (dense) bulk_wait_read<kBack>();
        if (i >= kBack && issued < nb) copy_y(issued++);
      }
      bulk_wait_all();
      if (i < nb)                                                       // gave up: the copies in flight
        for (int k = issued - 1; k >= 0 && k >= issued - C::kStagesY; --k)
          mbar_wait(&yfull[k % C::kStagesY], (k / C::kStagesY) & 1, nullptr, 72, 100000000ull);
    }
  } else if (warp == kWork) {
    if (lane == 0) {
      int issued = min(nb, C::kStagesB);
      for (; issued < nb; ++issued) {
        if (!mbar_wait(&bempty[issued % C::kStagesB], ((issued / C::kStagesB) & 1) ^ 1, abort, 66)) break;
        fetch_b(issued);
      }
      if (*abort)
        for (int i = issued - 1; i >= 0 && i >= issued - C::kStagesB; --i)
          mbar_wait(&bfull[i % C::kStagesB], (i / C::kStagesB) & 1, nullptr, 67, 100000000ull);
    }
  } else if (lane == 0) {                                               // warp 17
    const uint32_t id = idesc_f16(128, 128, !VOperand<T>::kScaled);
    for (int i = 0; i < nb; ++i) {
      const int s = i % C::kStagesB;
      if (!mbar_wait(&bfull[s], (i / C::kStagesB) & 1, abort, 68)) break;
      if (!mbar_wait(&dempty[i & 1], ((i >> 1) & 1) ^ 1, abort, 69)) break;
      tc_fence_after();
      for (int k = 0; k < P; ++k)
        for (int st = 0; st < steps; ++st)
          mma_f16(tmem + 128 * (i & 1), desc_kmajor_sw128(area + C::kV + (P * (st >> 2) + k) * kOp, 32 * (st & 3)),
                  desc_kmajor_sw128(area + C::kB + (s * RB + (st >> 2)) * kOp, 32 * (st & 3)), id, k > 0 || st > 0);
      mma_commit(&bempty[s]);
      mma_commit(&dfull[i & 1]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kWork + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTcCols);
  }
}

}  // namespace lora
}  // namespace ck
