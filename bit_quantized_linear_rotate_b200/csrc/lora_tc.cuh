// The adapters of lora_add.cuh for prompts: tiles of up to 128 tokens of one adapter on
// the tcgen05 tensor cores.
//
//   shrink: v (128 x R)  = x A^T      M = 128 tokens, N = R, K in blocks of 64
//   expand: d (128 x N)  = v B^T      M = 128 tokens, N in blocks of 128, K = R, as hi + lo
//   out = y + scale d
//
// A cluster of CTAs owns a tile: each CTA takes a share of K for the shrink,
// the partial v are added through distributed shared memory, and each CTA takes a share of N
// for the expand. Bytes bound both: x, y and out once each, so that a tile of 128
// tokens at K = N = 3840 moves 2.9 MB and reads 2 R (K + N) bytes of adapter from L2 (1 MB at
// R = 64; tiles of 64 tokens read it twice as often). The tensor cores
// read their operands from shared memory themselves, which leaves the load-store
// units to x, y and out; with mma.sync fragments straight from global
// memory the M = 8192, R = 64 case took 190 us.
//
// Warps 0-7 bring x in (16-byte asynchronous copies: a tile's tokens may be any rows), later
// reduce v and write the output; warp 8 brings in A and B by tensor copies (rows of
// another adapter and zeros past the end fill what R leaves of a block); warp 9 issues
// the MMAs. Accumulators: 256 TMEM columns, so that two CTAs share an SM.
//
// Shared memory, one area used twice (LoraTc): the shrink's stages, then the partial sums of v,
// v as operands and the ring of B. All barrier waits are bounded; after a timeout the CTA
// runs on without waiting, so that its cluster's barriers are met.
#pragma once

#include <cuda.h>

#include "lora_add.cuh"

namespace ck {
namespace lora {

constexpr int kTcTokens = 128;
constexpr int kTcWarps = 10;
constexpr int kTcThreads = 32 * kTcWarps;
constexpr int kOp = 128 * 128;                 // bytes of a 128 x 64 operand block, 128-byte swizzle
constexpr int kTcCols = 256;                   // TMEM columns
constexpr int kStaging = 32 * 33 * 4;          // a warp's 32 x 32 floats, rows one bank apart

// RB blocks of 64 ranks.
template <int RB>
struct LoraTc {
  static constexpr int kStageA = RB * 64 * 128;                        // A: up to 64 RB rows
  static constexpr int kStage = kOp + kStageA;
  static constexpr int kStages = 4;
  static constexpr int kPart = (128 * (64 * RB + 4) * 4 + 1023) / 1024 * 1024;   // partial v; then the warps' staging
  static constexpr int kV = kPart;                                     // offset of v: [RB][hi, lo]
  static constexpr int kB = kV + RB * 2 * kOp;                         // offset of B's ring
  static constexpr int kStagesB = 2;
  static constexpr int kArea = kB + kStagesB * RB * kOp;
  static_assert(kArea >= kStages * kStage, "the shrink's stages lie in the same area");
  static_assert(kPart >= 8 * kStaging, "the staging lies in the partial sums' place");
  static constexpr int kSmem = 1024 + kArea;
  static constexpr int kCtas = kSmem <= 112 * 1024 ? 2 : 1;
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
__device__ __forceinline__ void fence_proxy_async_any() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_b32x4(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

template <typename T, typename TY, int RB>
__global__ void __launch_bounds__(kTcThreads, LoraTc<RB>::kCtas)
    lora_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const Params p) {
  using C = LoraTc<RB>;
  using Tr = awq::Traits<T>;
  using TrY = awq::Traits<TY>;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* area = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  __shared__ uint64_t full[C::kStages], empty[C::kStages], shrunk;      // the shrink's stages, its end
  __shared__ uint64_t bfull[C::kStagesB], bempty[C::kStagesB], dfull[2], dempty[2];
  __shared__ int abort_flag;
  __shared__ uint32_t tmem_base;
  __shared__ int token[kTcTokens];
  __shared__ float row_scale[kTcTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
  volatile int* abort = &abort_flag;

  if (warp == 9) {
    tmem_alloc(&tmem_base, kTcCols);
    tmem_relinquish();
  } else if (tid == 8 * 32) {
    prefetch_tmap(&map_a);
    prefetch_tmap(&map_b);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 8 * 32 + 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&shrunk, 1);
    for (int s = 0; s < C::kStagesB; ++s) {
      mbar_init(&bfull[s], 1);
      mbar_init(&bempty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&dfull[s], 1);
      mbar_init(&dempty[s], 8);
    }
    abort_flag = 0;
    fence_mbarrier_init();
  }
  tc_fence_before();
  grid_dep_wait();
  grid_dep_launch();
  const int4 tile = __ldcg(reinterpret_cast<const int4*>(p.tiles) + blockIdx.x / ranks);
  const int adapter = tile.x, n = tile.z;
  if (tid < n) token[tid] = __ldcg(p.order + tile.y + tid);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const T* x = reinterpret_cast<const T*>(p.x);
  const TY* y = reinterpret_cast<const TY*>(p.y);
  TY* out = reinterpret_cast<TY*>(p.out);
  const int blocks = (p.N + 127) / 128;                                 // of output columns
  const int b0 = blocks * rank / ranks, b1 = blocks * (rank + 1) / ranks;

  if (n == 0 || adapter < 0) {                                          // the same for the whole cluster
    if (n > 0) copy_rows(y, out, p, token, n, 128 * b0, min(128 * b1, p.N), warp, kTcWarps, lane);
    __syncthreads();
    if (warp == 9) tmem_dealloc(tmem, kTcCols);
    return;
  }

  const int kblocks = (p.K + 63) / 64;
  const int k0 = kblocks * rank / ranks, k1 = kblocks * (rank + 1) / ranks;
  const int npad = (p.R + 15) / 16 * 16;                                // the shrink's N
  const int steps = npad / 16;                                          // the expand's K steps

  // ------------------------------------------------------------- shrink
  if (warp < 8) {
    const int c = tid & 7, r0 = tid >> 3;                               // 16-byte chunk, rows r0 + 32 i
    const T* src[4];
    uint32_t dst[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 32 * i;
      src[i] = r < n ? x + token[r] * p.ldx + 8 * c : nullptr;
      dst[i] = smem_u32(area) + r * 128 + ((c ^ (r & 7)) << 4);
    }
    constexpr int kLag = C::kStages - 1;
    auto hand_over = [&](int s) {                                       // this thread's copies into stage s are done
      fence_proxy_async_smem();
      mbar_arrive(&full[s]);
    };
    for (int kb = k0; kb < k1; ++kb) {
      const int i = kb - k0, s = i % C::kStages;
      mbar_wait(&empty[s], ((i / C::kStages) & 1) ^ 1, abort, 60);
      const bool in = 64 * kb + 8 * c < p.K;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        cp_async_16(dst[j] + s * C::kStage, in && src[j] != nullptr ? src[j] + 64 * (int64_t)kb : x, in && src[j] != nullptr);
      cp_async_commit();
      if (i >= kLag) {
        cp_async_wait<kLag>();
        hand_over((i - kLag) % C::kStages);
      }
    }
    cp_async_wait<0>();
    for (int i = max(k1 - k0 - kLag, 0); i < k1 - k0; ++i) hand_over(i % C::kStages);
  } else if (warp == 8) {
    if (lane == 0) {
      int issued = 0;
      for (int kb = k0; kb < k1; ++kb, ++issued) {
        const int i = kb - k0, s = i % C::kStages;
        if (!mbar_wait(&empty[s], ((i / C::kStages) & 1) ^ 1, abort, 61)) break;
        mbar_arrive_expect_tx(&full[s], npad * 128);
        tma_load_2d(area + s * C::kStage + kOp, &map_a, &full[s], 64 * kb, adapter * p.R);
      }
      if (*abort)
        for (int i = issued - 1; i >= 0 && i >= issued - C::kStages; --i)
          mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1, nullptr, 62, 100000000ull);
    }
  } else if (lane == 0) {
    const uint32_t id = idesc_f16(128, npad, sizeof(T) == 2 && !Half2Of<T>::kScaled);
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
      tma_load_2d(area + C::kB + (s * RB + rb) * kOp, &map_b, &bfull[s], 64 * rb, adapter * p.N + 128 * (b0 + i));
  };
  const int nb = b1 - b0;
  if (warp == 8 && lane == 0)
    for (int i = 0; i < min(nb, C::kStagesB); ++i) fetch_b(i);
  __syncwarp();
  const int q = warp & 3, hc = warp >> 2;                               // TMEM lane quarter, half of the columns
  if (warp < 8) {
    tc_fence_after();
    float* part = reinterpret_cast<float*>(area) + (32 * q + lane) * (p.R + 4);
    for (int c0 = 16 * hc; c0 < p.R; c0 += 32) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(tmem + ((uint32_t)(32 * q) << 16) + c0, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        if (c0 + i < p.R)
          *reinterpret_cast<float4*>(part + c0 + i) =
              any_k ? make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]),
                                  __uint_as_float(v[i + 3]))
                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    tc_fence_before();
  }
  cluster_sync();
  // half a warp sums a row over the ranks, 8 entries a lane, and hands hi and lo to every CTA
  if (warp < 8) {
    const float as = p.scales != nullptr ? __ldg(p.scales + adapter) : 1.0f;
    const int l = lane & 15, rows = kTcTokens / ranks;
    for (int i = 2 * warp + (lane >> 4); i < (rows + 15) / 16 * 16; i += 16) {   // whole warps, for the shuffles
      const int r = rank * rows + i;
      const bool mine = i < rows;
      float v[8] = {};
      if (mine && 8 * l < p.R)
        for (int k = 0; k < ranks; ++k) {
          const uint32_t at = mapa_shared(smem_u32(area) + (r * (p.R + 4) + 8 * l) * 4, k);
          const float4 a = ld_cluster_f32x4(at), b = ld_cluster_f32x4(at + 16);
          v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
          v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
        }
      int ex = 0;
      if constexpr (Half2Of<T>::kScaled) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        ex = scale_exponent(top);
      }
      const float up = exp2_int(ex);
      T h[8], lo[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) split(v[j] * up, h[j], lo[j]);
      if (mine && l < 2 * steps) {
        const uint32_t at = smem_u32(area) + C::kV + (l >> 3) * 2 * kOp + r * 128 + (((l & 7) ^ (r & 7)) << 4);
        for (int k = 0; k < ranks; ++k) {
          const uint32_t to = mapa_shared(at, k);
          st_cluster_b32x4(to, *reinterpret_cast<const uint4*>(h));
          st_cluster_b32x4(to + kOp, *reinterpret_cast<const uint4*>(lo));
        }
      }
      if (mine && l == 0)
        for (int k = 0; k < ranks; ++k) st_cluster_f32(mapa_shared(smem_u32(row_scale) + 4 * r, k), as * exp2_int(-ex));
    }
    fence_proxy_async_any();                                            // v is read by the tensor cores
  }
  cluster_sync();
  fence_proxy_async_any();

  // ------------------------------------------------------------- expand
  if (warp < 8) {
    float* stage = reinterpret_cast<float*>(area + warp * kStaging);
    const int rr = 32 * q + (lane >> 2), cc = 8 * (lane & 3);           // rows rr + 8 i of the tile, column of the chunk
    const TY* yr[4];
    TY* orow[4];
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = rr + 8 * i;
      yr[i] = r < n ? y + token[r] * p.ldy : nullptr;
      orow[i] = r < n ? out + token[r] * p.ldo : nullptr;
      f[i] = row_scale[r];
    }
    auto load_y = [&](int col, uint4 (&v)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (yr[i] == nullptr || col >= p.N) continue;
        if (p.vec) {
          v[i] = *reinterpret_cast<const uint4*>(yr[i] + col);
        } else {
          TY e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = yr[i][min(col + j, p.N - 1)];
          v[i] = *reinterpret_cast<const uint4*>(e);
        }
      }
    };
    uint4 yv[4], yn[4];
    if (nb > 0) load_y(128 * b0 + 64 * hc + cc, yv);
    for (int i = 0; i < nb; ++i) {
      mbar_wait(&dfull[i & 1], (i >> 1) & 1, abort, 65);
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        const int col = 128 * (b0 + i) + 64 * hc + 32 * ch + cc;
        // the next chunk's y, while this one is finished
        load_y(ch == 0 ? col + 32 : i + 1 < nb ? col + 96 : p.N, yn);
        uint32_t d[32];
        tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * q) << 16) + 128 * (i & 1) + 64 * hc + 32 * ch, d);
        tmem_ld_wait();
        if (ch == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&dempty[i & 1]);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) stage[lane * 33 + j] = __uint_as_float(d[j]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* s = stage + ((lane >> 2) + 8 * k) * 33 + cc;
          if (orow[k] != nullptr && col < p.N) {
            TY e[8];
            *reinterpret_cast<uint4*>(e) = yv[k];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = TrY::fromf(fmaf(f[k], s[j], TrY::tof(e[j])));
            if (p.vec) {
              *reinterpret_cast<uint4*>(orow[k] + col) = *reinterpret_cast<const uint4*>(e);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (col + j < p.N) orow[k][col + j] = e[j];
            }
          }
          yv[k] = yn[k];
        }
        __syncwarp();
      }
    }
  } else if (warp == 8) {
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
  } else if (lane == 0) {
    const uint32_t id = idesc_f16(128, 128, sizeof(T) == 2 && !Half2Of<T>::kScaled);
    for (int i = 0; i < nb; ++i) {
      const int s = i % C::kStagesB;
      if (!mbar_wait(&bfull[s], (i / C::kStagesB) & 1, abort, 68)) break;
      if (!mbar_wait(&dempty[i & 1], ((i >> 1) & 1) ^ 1, abort, 69)) break;
      tc_fence_after();
      for (int k = 0; k < 2 * steps; ++k) {                             // hi, then lo
        const int st = k < steps ? k : k - steps, rb = st >> 2;
        mma_f16(tmem + 128 * (i & 1), desc_kmajor_sw128(area + C::kV + (2 * rb + (k < steps ? 0 : 1)) * kOp, 32 * (st & 3)),
                desc_kmajor_sw128(area + C::kB + (s * RB + rb) * kOp, 32 * (st & 3)), id, k > 0);
      }
      mma_commit(&bempty[s]);
      mma_commit(&dfull[i & 1]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTcCols);
  }
}

}  // namespace lora
}  // namespace ck
