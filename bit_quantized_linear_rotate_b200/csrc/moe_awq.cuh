// A mixture-of-experts layer for a few tokens on AWQ W4A16 experts, in two kernels.
//
//   W[n, c] = (u[n, c] - 8) s[c / G, n] + z[c / G, n]         (each expert's, as gemv_awq.cuh)
//   h[t, e] = silu(x_t Wg_e^T) * (x_t Wu_e^T),  silu(v) = v / (1 + exp(-v))
//   out_t   = sum over t's experts of w[t, e] (h[t, e] Wd_e^T)
//
// gate_up_kernel chooses (or takes) the experts and computes h; down_kernel
// computes the weighted sum. Each weight that some token needs is read from HBM
// once, which bounds both kernels: a sub-block of 64 columns of 16 weight
// rows (512 packed bytes) takes an SM 22 clocks of its share of the measured
// copy bandwidth.
//
// Products. The 16 weight rows are the A operand of mma.sync.m16n8k16, up to
// eight tokens the B operand, and a sub-block lies within one quantization
// group (G % 64 == 0). With P' = sum (offset + u) x from nibbles that one shift
// and one logical op turn into exact bf16 or fp16 numbers, and X = sum x from
// the same B operand against ones,
//   sum over the sub-block of W x = s P' + (z - (offset + 8) s) X
// in 32 bits. Row g of the fragment is physical row 2 g and row g + 8 is
// 2 g + 1, so that one 4-byte load brings a lane its two scales.
//
// h is kept as a pair of bf16 numbers, hi = bf16(h) and lo = bf16(h - hi):
// 2^-17 of h or less is lost. The two are neighbouring columns of the B operand
// in down_kernel, so up to four tokens of an expert cost no more products
// than h rounded to bf16 alone would.
//
// Sums run in a fixed order: the output does not depend on timing.
#pragma once

#include "cluster_mem.cuh"
#include "gemv_awq.cuh"
#include "moe_route.cuh"

namespace ck {
namespace moe {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kColsItem = 32;          // columns of h in one item of gate_up_kernel
constexpr int kRowsTile = 32;          // output columns of one cluster of down_kernel
constexpr int kChunk = 64 * kWarps;    // columns of h in one step of down_kernel

struct Params {
  Choice choice;
  const void* x;                       // (T, K) T, row stride ldx
  int64_t ldx;
  int K, I, gsh;                       // quantization group of sub-block sb: sb >> gsh
  const uint8_t* gate_up_q;            // (E, 2 I, K / 2): gate rows, then up rows
  const void *gate_up_s, *gate_up_z;   // (E, K / G, 2 I) T
  const uint8_t* down_q;               // (E, K, I / 2)
  const void *down_s, *down_z;         // (E, I / G, K) T
  __nv_bfloat16* h;                    // (slots, 2, I): hi, lo
  void* out;                           // (T, K) T
};

// Two neighbouring scales (or zeros) of type T as floats.
template <typename T>
__device__ __forceinline__ float2 load_pair(const T* p) {
  const uint32_t u = __ldg(reinterpret_cast<const unsigned int*>(p));
  const T* v = reinterpret_cast<const T*>(&u);
  return make_float2(awq::Traits<T>::tof(v[0]), awq::Traits<T>::tof(v[1]));
}

// 64 columns of two weight rows, as the four A operands of the sub-block. D is
// the type whose magic number the nibbles take.
template <typename D>
__device__ __forceinline__ void decode(const uint2 r0, const uint2 r1, uint32_t (&a)[4][4]) {
  const uint32_t w0[2] = {r0.x, r0.y}, w1[2] = {r1.x, r1.y};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int wd = j >> 1, s0 = (2 * j) & 3, s1 = (2 * j + 1) & 3;
    a[j][0] = awq::nib_pair_raw<D>(w0[wd], s0);
    a[j][1] = awq::nib_pair_raw<D>(w1[wd], s0);
    a[j][2] = awq::nib_pair_raw<D>(w0[wd], s1);
    a[j][3] = awq::nib_pair_raw<D>(w1[wd], s1);
  }
}

// 16 consecutive values of a token as the pairs (k, k + 4) that decode() makes of the weights.
__device__ __forceinline__ void regroup(const uint4 xa, const uint4 xb, uint32_t (&bp)[8]) {
  bp[0] = __byte_perm(xa.x, xa.z, 0x5410);
  bp[1] = __byte_perm(xa.x, xa.z, 0x7632);
  bp[2] = __byte_perm(xa.y, xa.w, 0x5410);
  bp[3] = __byte_perm(xa.y, xa.w, 0x7632);
  bp[4] = __byte_perm(xb.x, xb.z, 0x5410);
  bp[5] = __byte_perm(xb.x, xb.z, 0x7632);
  bp[6] = __byte_perm(xb.y, xb.w, 0x5410);
  bp[7] = __byte_perm(xb.y, xb.w, 0x7632);
}

// tot += s P' + (z - (offset + 8) s) X for the lane's rows 2 g (elements 0, 1) and 2 g + 1.
template <typename D>
__device__ __forceinline__ void add_block(float (&tot)[4], const uint32_t (&a)[4][4], const uint32_t (&bp)[8],
                                          const float (&X)[4], const float2 s, const float2 zo) {
  float P[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 4; ++j) awq::Traits<D>::mma(P, a[j], bp[2 * j], bp[2 * j + 1]);
  tot[0] += s.x * P[0] + zo.x * X[0];
  tot[1] += s.x * P[1] + zo.x * X[1];
  tot[2] += s.y * P[2] + zo.y * X[0];
  tot[3] += s.y * P[3] + zo.y * X[1];
}

template <typename D>
__device__ __forceinline__ float2 fold_zero(const float2 s, const float2 z) {
  constexpr float kOff = awq::RawOffset<D>::v;
  return make_float2(fmaf(-kOff, s.x, z.x), fmaf(-kOff, s.y, z.y));
}

template <typename D>
__device__ __forceinline__ void sum_tokens(const uint32_t (&bp)[8], float (&X)[4]) {
  const uint32_t ones[4] = {awq::Traits<D>::kOnes, awq::Traits<D>::kOnes, awq::Traits<D>::kOnes,
                            awq::Traits<D>::kOnes};
  X[0] = X[1] = X[2] = X[3] = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) awq::Traits<D>::mma(X, ones, bp[2 * j], bp[2 * j + 1]);
}

// -------------------------------------------------------------- gate and up

// An item is 32 columns of h of one unit (an expert's tokens, at most 8 NT):
// 32 gate rows and the 32 up rows that belong to them. A CTA takes a contiguous
// share of the items. Warp (kw, hf) multiplies the 16 gate and the 16 up rows of
// half hf with every fourth sub-block; the four partial sums meet in shared memory.
template <int NT>
struct GateUpSmem {
  Lists L;
  float4 red[2][4][2][2][NT][32];      // [buffer][kw][half][gate, up][token tile][lane]
};

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, 2) gate_up_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t sm[];
  GateUpSmem<NT>& S = *reinterpret_cast<GateUpSmem<NT>*>(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3, kw = warp >> 1, hf = warp & 1;
  grid_dep_wait();
  grid_dep_launch();   // after the wait: the next kernel may read the choice before its own wait
  build_lists<kThreads>(p.choice, S.L, 8 * NT);

  const int per_unit = p.I / kColsItem, nsub = p.K >> 6;
  const int64_t items = (int64_t)S.L.n_units * per_unit;
  const int i0 = (int)(items * blockIdx.x / gridDim.x), i1 = (int)(items * (blockIdx.x + 1) / gridDim.x);
  const int64_t half = p.K >> 1, rows = 2 * (int64_t)p.I;
  const int ngrp = nsub >> p.gsh;
  const T* x = reinterpret_cast<const T*>(p.x);

  for (int item = i0; item < i1; ++item) {
    const int u = item / per_unit, c0 = (item % per_unit) * kColsItem;
    const int e = S.L.unit_expert[u], start = S.L.unit_start[u], n = S.L.unit_n[u];
    const int row = c0 + 16 * hf + 2 * g;
    const uint8_t* wg = p.gate_up_q + (e * rows + row) * half + 8 * t;
    const uint8_t* wu = wg + p.I * half;
    const T* sp = reinterpret_cast<const T*>(p.gate_up_s) + (int64_t)e * ngrp * rows + row;
    const T* zp = reinterpret_cast<const T*>(p.gate_up_z) + (int64_t)e * ngrp * rows + row;
    const T* xr[NT];
#pragma unroll
    for (int tt = 0; tt < NT; ++tt)
      xr[tt] = 8 * tt + g < n ? x + (int64_t)S.L.slot_token[start + 8 * tt + g] * p.ldx + 16 * t : nullptr;

    float tg[NT][4] = {}, tu[NT][4] = {};
#pragma unroll 2
    for (int sb = kw; sb < nsub; sb += 4) {
      const uint2 g0 = __ldcs(reinterpret_cast<const uint2*>(wg + sb * 32));
      const uint2 g1 = __ldcs(reinterpret_cast<const uint2*>(wg + half + sb * 32));
      const uint2 u0 = __ldcs(reinterpret_cast<const uint2*>(wu + sb * 32));
      const uint2 u1 = __ldcs(reinterpret_cast<const uint2*>(wu + half + sb * 32));
      const int64_t so = (int64_t)(sb >> p.gsh) * rows;
      const float2 sg = load_pair(sp + so), zg = fold_zero<T>(sg, load_pair(zp + so));
      const float2 su = load_pair(sp + so + p.I), zu = fold_zero<T>(su, load_pair(zp + so + p.I));
      uint32_t ag[4][4], au[4][4];
      decode<T>(g0, g1, ag);
      decode<T>(u0, u1, au);
#pragma unroll
      for (int tt = 0; tt < NT; ++tt) {
        if (8 * tt >= n) break;
        uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
        if (xr[tt] != nullptr) {
          xa = __ldg(reinterpret_cast<const uint4*>(xr[tt] + sb * 64));
          xb = __ldg(reinterpret_cast<const uint4*>(xr[tt] + sb * 64 + 8));
        }
        uint32_t bp[8];
        regroup(xa, xb, bp);
        float X[4];
        sum_tokens<T>(bp, X);
        add_block<T>(tg[tt], ag, bp, X, sg, zg);
        add_block<T>(tu[tt], au, bp, X, su, zu);
      }
    }
    auto& red = S.red[item & 1];         // two buffers: one barrier an item is enough
#pragma unroll
    for (int tt = 0; tt < NT; ++tt) {
      red[kw][hf][0][tt][lane] = make_float4(tg[tt][0], tg[tt][1], tg[tt][2], tg[tt][3]);
      red[kw][hf][1][tt][lane] = make_float4(tu[tt][0], tu[tt][1], tu[tt][2], tu[tt][3]);
    }
    __syncthreads();
    for (int i = tid; i < 32 * n; i += kThreads) {
      const int c = i >> 5, r = i & 31;   // token of the unit, column of the item
      const int ln = ((r & 15) >> 1) * 4 + ((c & 7) >> 1), el = (r & 1) * 2 + (c & 1);
      float gate = 0.0f, up = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        gate += reinterpret_cast<const float*>(&red[w][r >> 4][0][c >> 3][ln])[el];
        up += reinterpret_cast<const float*>(&red[w][r >> 4][1][c >> 3][ln])[el];
      }
      const float h = gate / (1.0f + expf(-gate)) * up;
      const __nv_bfloat16 hi = __float2bfloat16_rn(h);
      const float hf32 = __bfloat162float(hi);
      const float lo = isfinite(hf32) ? h - hf32 : 0.0f;   // an infinity stays one
      __nv_bfloat16* hp = p.h + (int64_t)2 * (start + c) * p.I + c0 + r;
      hp[0] = hi;
      hp[p.I] = __float2bfloat16_rn(lo);
    }
  }
}

// --------------------------------------------------------------------- down

// A cluster of CTAs owns 32 output columns and walks (unit, 512 columns of h)
// steps, each CTA a contiguous share of them; warp w takes sub-block w of a
// step. A unit is at most 4 NT tokens: column 2 i of the B operand is token i's
// hi, column 2 i + 1 its lo. When the unit changes, each warp adds its sums, times
// the tokens' weights, to its own (T, 32) accumulator in shared memory; at the
// end the warps' accumulators and then the CTAs' are added in order.
struct DownSmem {
  Lists L;
  float acc[1];                          // [kWarps][T][32]
};

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, 2) down_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t sm[];
  DownSmem& S = *reinterpret_cast<DownSmem*>(sm);
  using D = __nv_bfloat16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_ctarank(), ranks = cluster_nctarank();
  const int tokens = p.choice.T, n0 = (int)(blockIdx.x / ranks) * kRowsTile;
  // The choice was complete before gate_up_kernel let this kernel start.
  build_lists<kThreads>(p.choice, S.L, 4 * NT);
  for (int i = tid; i < kWarps * tokens * kRowsTile; i += kThreads) S.acc[i] = 0.0f;
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();

  const int nsub = p.I >> 6, nchunk = (nsub + kWarps - 1) / kWarps;
  const int64_t steps = (int64_t)S.L.n_units * nchunk;
  const int s0 = (int)(steps * rank / ranks), s1 = (int)(steps * (rank + 1) / ranks);
  const int64_t half = p.I >> 1;
  const int ngrp = nsub >> p.gsh;
  float* acc = S.acc + warp * tokens * kRowsTile;
  float tot[2][NT][4] = {};
  for (int s = s0; s < s1; ++s) {
    const int u = s / nchunk, sb = (s % nchunk) * kWarps + warp;
    const int e = S.L.unit_expert[u], start = S.L.unit_start[u], n = S.L.unit_n[u];
    if (sb < nsub) {
      const int row = n0 + 2 * g;
      const uint8_t* wp = p.down_q + ((int64_t)e * p.K + row) * half + sb * 32 + 8 * t;
      const int64_t so = ((int64_t)e * ngrp + (sb >> p.gsh)) * p.K + row;
      const T* sp = reinterpret_cast<const T*>(p.down_s) + so;
      const T* zp = reinterpret_cast<const T*>(p.down_z) + so;
      uint32_t a[2][4][4];
      float2 sc[2], zo[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint2 r0 = __ldcs(reinterpret_cast<const uint2*>(wp + 16 * m * half));
        const uint2 r1 = __ldcs(reinterpret_cast<const uint2*>(wp + (16 * m + 1) * half));
        sc[m] = load_pair(sp + 16 * m);
        zo[m] = fold_zero<D>(sc[m], load_pair(zp + 16 * m));
        decode<D>(r0, r1, a[m]);
      }
#pragma unroll
      for (int tt = 0; tt < NT; ++tt) {
        if (4 * tt >= n) break;
        uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
        if (8 * tt + g < 2 * n) {
          const __nv_bfloat16* hp = p.h + (int64_t)(2 * start + 8 * tt + g) * p.I + sb * 64 + 16 * t;
          xa = __ldg(reinterpret_cast<const uint4*>(hp));
          xb = __ldg(reinterpret_cast<const uint4*>(hp + 8));
        }
        uint32_t bp[8];
        regroup(xa, xb, bp);
        float X[4];
        sum_tokens<D>(bp, X);
        add_block<D>(tot[0][tt], a[0], bp, X, sc[0], zo[0]);
        add_block<D>(tot[1][tt], a[1], bp, X, sc[1], zo[1]);
      }
    }
    if (s + 1 == s1 || (s + 1) / nchunk != u) {   // the unit's last step here
#pragma unroll
      for (int tt = 0; tt < NT; ++tt) {
        const int i = 4 * tt + t;                 // the lane's token: hi + lo are its two columns
        if (i < n) {
          const float w = S.L.slot_w[start + i];
          float* ap = acc + S.L.slot_token[start + i] * kRowsTile + 2 * g;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            ap[16 * m] += w * (tot[m][tt][0] + tot[m][tt][1]);
            ap[16 * m + 1] += w * (tot[m][tt][2] + tot[m][tt][3]);
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) tot[m][tt][0] = tot[m][tt][1] = tot[m][tt][2] = tot[m][tt][3] = 0.0f;
      }
      __syncwarp();                               // another lane may hold this token in the next unit
    }
  }
  __syncthreads();
  const int cells = tokens * kRowsTile;
  for (int i = tid; i < cells; i += kThreads) {
    float v = S.acc[i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += S.acc[w * cells + i];
    S.acc[i] = v;
  }
  cluster_sync();
  const uint32_t base = smem_u32(S.acc);
  for (int i = rank * kThreads + tid; i < cells; i += ranks * kThreads) {
    float v = 0.0f;
    for (uint32_t r = 0; r < ranks; ++r) v += ld_cluster_f32(mapa_shared(base + 4 * i, r));
    reinterpret_cast<T*>(p.out)[(int64_t)(i / kRowsTile) * p.K + n0 + i % kRowsTile] = awq::Traits<T>::fromf(v);
  }
  cluster_sync();                                 // no CTA leaves while another reads its sums
}

}  // namespace moe
}  // namespace ck
