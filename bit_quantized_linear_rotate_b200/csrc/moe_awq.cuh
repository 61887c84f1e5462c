// A mixture-of-experts layer for a few tokens on AWQ W4A16 experts.
//
//   W[n, c] = (u[n, c] - 8) s[c / G, n] + z[c / G, n]         (each expert's, as gemv_awq.cuh)
//   h[t, e] = silu(x_t Wg_e^T) * (x_t Wu_e^T),  silu(v) = v / (1 + exp(-v))
//   out_t   = sum over t's experts of w[t, e] (h[t, e] Wd_e^T)
//
// gate_up_kernel computes h, down_kernel the weighted sum. Both choose the
// experts (or take the choice) in every CTA; larger batches have that and the
// conversion of x done once, by prepare_kernel. Each weight that some token
// needs is read from HBM once, and that bounds the layer: a tile of 16 weight rows x 64
// columns (512 packed bytes) takes one of an SM's four schedulers 89 clocks at
// the measured copy bandwidth, so a tile must cost well under 89 issue slots.
//
// Products. Activations enter as 15-bit block fixed point: the 64 columns of a
// sub-block (which lies in one quantization group, G % 64 == 0) share a scale
// d = max |x| / 16256, and x ~ d q with q = 128 hi + lo, hi and lo in int8. Then
//   sum of W x over the sub-block = s d (128 sum u hi + sum u lo) + (z - 8 s) X,  X = d sum q.
// The sums are exact int32 products of mma.sync.m16n8k32 (16 weight rows, unsigned
// nibbles; 8 columns of B: hi and lo of four tokens), below 2^24 and so exact as
// floats, and the rest is 32-bit floating point. The rounding to 15 bits moves x
// by at most 2^-15 of its block's largest entry, 2^-16 on average against the
// 2^-9 (bf16) or 2^-12 (fp16) that rounding the result once costs. Nibbles as
// bf16 numbers in m16n8k16 took 136 instructions a tile, this 50: a packed word is three
// logical ops, a tile two MMAs, X needs no product.
//
// A block with an entry that is not finite gets d = NaN: the token's output is NaN.
//
// Sums run in a fixed order: the output does not depend on timing.
#pragma once

#include <cuda.h>

#include "cluster_mem.cuh"
#include "gemv_awq.cuh"
#include "moe_route.cuh"

namespace ck {
namespace moe {

constexpr int kCons = 8;               // consumer warps; one more warp feeds the ring
constexpr int kThreads = 32 * (kCons + 1);
constexpr int kColsItem = 64;          // columns of h in one item of gate_up_kernel: one block of the fixed point
constexpr int kRowsTile = 32;          // output columns of one cluster of down_kernel
constexpr int kMaxStages = 4;

// A stage of either ring: 16 KB of weights in boxes of 256 columns (128 bytes a row,
// 128-byte swizzle), then scales and zeros. In gate_up_kernel 256 columns of 64 gate
// and 64 up rows, in down_kernel 1024 columns of 32 rows.
constexpr int kStageW = 128 * 128;
constexpr int kStageS = 2048;
constexpr int kStage = kStageW + kStageS;

// Rows of activations as fixed point. Sub-block sb of row r: 128 bytes at q + r *
// q_stride + 128 sb, the hi bytes of its 64 columns, then the lo bytes, each in
// four runs of 16 columns in the order 0 2 4 6 1 3 5 7 8 10 12 14 9 11 13 15 (low
// nibbles of a packed word, then its high nibbles), and {d, X} at scale[r * s_stride + sb].
struct Fixed {
  uint8_t* q;
  float2* scale;
  int64_t q_stride;                    // bytes: 2 x columns
  int s_stride;                        // columns / 64
};

struct Params {
  Choice choice;
  const void* x;                       // (T, K) T, row stride ldx
  int64_t ldx;
  int K, I, gsh;                       // quantization group of sub-block sb: sb >> gsh
  Fixed xq;                            // (T) rows by prepare_kernel; unused where a CTA converts x itself
  Fixed hq;                            // (slots) rows of h
  void* out;                           // (T, K) T
};

// Tensor maps of one weight matrix of all experts and of its scales and zeros.
struct Maps {
  CUtensorMap w, s, z;
};

// ------------------------------------------------------- block fixed point

constexpr float kQMax = 16256.0f;      // 128 * 127

// {scale d, 1 / d} of a block whose largest magnitude is m. Below 2^-100 it counts as zero (1 / d
// must stay finite); not finite: NaN.
__device__ __forceinline__ float2 block_scale(float m) {
  if (!(m < INFINITY)) return make_float2(__int_as_float(0x7fffffff), 0.0f);
  if (m < 7.9e-31f) return make_float2(0.0f, 0.0f);
  return make_float2(m * (1.0f / kQMax), kQMax / m);
}

// |v| for a maximum that a NaN must not get lost in: as unsigned bits, where NaN is above infinity.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// hi and lo bytes of v / d.
__device__ __forceinline__ int fixed_point(float v, float inv) {
  return inv == 0.0f ? 0 : __float2int_rn(v * inv);
}

// Converts row `row` of x (K values) by a group of THREADS threads (a multiple of 8), 8 columns
// a thread at a time; lane groups of eight hold a sub-block.
template <typename T, int THREADS>
__device__ __forceinline__ void convert_row(const T* x, int K, uint8_t* q, float2* scale, int tid) {
  const int blocks = K >> 6;
  for (int b0 = 0; b0 < blocks; b0 += THREADS / 8) {   // the whole warp stays for the shuffles
    const int sb = b0 + tid / 8, part = tid & 7;
    const bool in = sb < blocks;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (in) raw = *reinterpret_cast<const uint4*>(x + sb * 64 + part * 8);
    const T* v = reinterpret_cast<const T*>(&raw);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, magnitude(awq::Traits<T>::tof(v[i])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float2 d = block_scale(__uint_as_float(m));
    uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};            // even columns, odd columns
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int f = fixed_point(awq::Traits<T>::tof(v[i]), d.y);
      const int h = (f + 64) >> 7, l = f - 128 * h;
      sum += f;
      hi[i & 1] |= (uint32_t)(h & 0xff) << (8 * (i >> 1));
      lo[i & 1] |= (uint32_t)(l & 0xff) << (8 * (i >> 1));
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (in) {
      *reinterpret_cast<uint2*>(q + sb * 128 + part * 8) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(q + sb * 128 + 64 + part * 8) = make_uint2(lo[0], lo[1]);
      if (part == 0) scale[sb] = make_float2(d.x, d.x * (float)sum);
    }
  }
}

// ----------------------------------------------------------- prepare (T > 4)

constexpr int kPrepThreads = 256;

// One CTA a token: its row of x as fixed point, and (logits given) its choice.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads)
    prepare_kernel(const Params p, int32_t* __restrict__ ids, float* __restrict__ weights) {
  grid_dep_wait();
  grid_dep_launch();
  const int t = blockIdx.x;
  convert_row<T, kPrepThreads>(reinterpret_cast<const T*>(p.x) + t * p.ldx, p.K, p.xq.q + t * p.xq.q_stride,
                               p.xq.scale + (int64_t)t * p.xq.s_stride, threadIdx.x);
  if (ids != nullptr && threadIdx.x < 32) {
    int id;
    float w;
    choose_any(p.choice.logits, p.choice.ldt, t, p.choice.E, p.choice.k, p.choice.renorm != 0, id, w);
    if ((int)threadIdx.x < p.choice.k) {
      ids[t * p.choice.k + threadIdx.x] = id;
      weights[t * p.choice.k + threadIdx.x] = w;
    }
  }
}

// ------------------------------------------------------------- weight tiles

// Two neighbouring scales (or zeros) of type T as floats.
template <typename T>
__device__ __forceinline__ float2 load_pair(const uint8_t* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  const T* v = reinterpret_cast<const T*>(&u);
  return make_float2(awq::Traits<T>::tof(v[0]), awq::Traits<T>::tof(v[1]));
}

// A tile of 16 weight rows x 64 columns as the A operands of two MMAs, from a
// box of 256 columns: 16-byte chunk c of row r is at c ^ (r % 8). Row g of the
// fragment is row r = r0 + 2 g, row g + 8 is r + 1, so that a lane's two
// scales are neighbours and a half-warp's reads hit each bank once.
__device__ __forceinline__ void load_tile(const uint8_t* box, int r, int sb, int t, uint32_t (&a)[2][4]) {
  const int c = 2 * (sb & 3) + (t >> 1), b = 8 * (t & 1);
  const uint2 w0 = *reinterpret_cast<const uint2*>(box + r * 128 + ((c ^ (r & 7)) << 4) + b);
  const uint2 w1 = *reinterpret_cast<const uint2*>(box + (r + 1) * 128 + ((c ^ ((r + 1) & 7)) << 4) + b);
  a[0][0] = w0.x & 0x0F0F0F0Fu;
  a[0][1] = w1.x & 0x0F0F0F0Fu;
  a[0][2] = (w0.x >> 4) & 0x0F0F0F0Fu;
  a[0][3] = (w1.x >> 4) & 0x0F0F0F0Fu;
  a[1][0] = w0.y & 0x0F0F0F0Fu;
  a[1][1] = w1.y & 0x0F0F0F0Fu;
  a[1][2] = (w0.y >> 4) & 0x0F0F0F0Fu;
  a[1][3] = (w1.y >> 4) & 0x0F0F0F0Fu;
}

__device__ __forceinline__ void mma_u8s8(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// tot += the sub-block's sum of W x, for the tile's rows r and r + 1 and token t of the four in b.
// s, z8: the rows' scales and z - 8 s; dx: {d, X} of that token's block.
__device__ __forceinline__ void add_block(float (&tot)[2], const uint32_t (&a)[2][4], const uint4 b, const float2 s,
                                          const float2 z8, const float2 dx) {
  int c[4] = {0, 0, 0, 0};
  mma_u8s8(c, a[0], b.x, b.y);
  mma_u8s8(c, a[1], b.z, b.w);
  tot[0] += (s.x * dx.x) * (float)(c[0] * 128 + c[1]);
  tot[1] += (s.y * dx.x) * (float)(c[2] * 128 + c[3]);
  tot[0] = fmaf(z8.x, dx.y, tot[0]);
  tot[1] = fmaf(z8.y, dx.y, tot[1]);
}

__device__ __forceinline__ float2 fold_zero(const float2 s, const float2 z) {
  return make_float2(fmaf(-8.0f, s.x, z.x), fmaf(-8.0f, s.y, z.y));
}

// ------------------------------------------------------------------ the ring

// full: the stage's bytes have arrived; empty: every consumer warp has taken
// them into registers. A wait that gives up sets `abort`; from then on the CTA runs
// to its end without waiting, on whatever the stages hold, so that no barrier
// is missed (the host learns of it from the device error word).
struct Ring {
  uint64_t full[kMaxStages], empty[kMaxStages];
  int abort;
};

__device__ __forceinline__ void ring_init(Ring& R, int stages) {
  for (int s = 0; s < stages; ++s) {
    mbar_init(&R.full[s], 1);
    mbar_init(&R.empty[s], kCons);
  }
  R.abort = 0;
  fence_mbarrier_init();
}

// Producer (one thread): waits until fill i may overwrite its stage.
__device__ __forceinline__ bool ring_claim(Ring& R, int stages, int i) {
  return i < stages || mbar_wait(&R.empty[i % stages], (i / stages - 1) & 1, &R.abort, 50);
}

// Producer: after giving up, waits (with a limit) for the copies in flight.
__device__ __forceinline__ void ring_drain(Ring& R, int stages, int issued) {
  for (int i = issued - 1; i >= 0 && i >= issued - stages; --i)
    mbar_wait(&R.full[i % stages], (i / stages) & 1, nullptr, 51, 100000000ull);
}

__device__ __forceinline__ void ring_await(Ring& R, int stages, int i) {
  warp_wait(&R.full[i % stages], (i / stages) & 1, &R.abort, 52);
}

__device__ __forceinline__ void ring_release(Ring& R, int stages, int i) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&R.empty[i % stages]);
}

// The consumer warps' own barrier.
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kCons) : "memory"); }

// Shared memory: the lists, what each kernel sums in, and the ring, whose memory the
// building of the lists uses first.
struct SmemHead {
  Lists L;
  Ring R;
};
constexpr int kHead = (sizeof(SmemHead) + 127) / 128 * 128;
static_assert(sizeof(ListsTemp) <= kStage, "the lists are built in the ring's first stage");

// Offset of the ring behind `sums` bytes: 1024-byte aligned boxes.
__host__ __device__ constexpr int ring_offset(int sums) { return (kHead + sums + 1023) / 1024 * 1024; }

// Up to kMaxStages stages that leave room for two CTAs on an SM (max_smem each, with
// 1024 bytes for aligning the base).
__host__ __device__ constexpr int ring_stages(int sums, int max_smem) {
  const int n = (max_smem - 1024 - ring_offset(sums)) / kStage;
  return n < kMaxStages ? n : kMaxStages;
}

// -------------------------------------------------------------- gate and up

// An item is 64 columns of h of one unit (an expert's tokens, at most 4 NT): 64
// gate rows and the 64 up rows that belong to them. A CTA takes a contiguous
// share of the items and streams their weights, 256 columns a stage. Consumer
// warp (kw, hf) multiplies 32 gate and 32 up rows with sub-block kw of each stage; the
// four partial sums meet in shared memory, where one warp a token forms h and
// converts it to fixed point.
//
// SELF: x is converted by every CTA, into shared memory (T <= 4 and T K <=
// kSelfX): the launch of prepare_kernel and the wait for it cost more.
constexpr int kSelfTokens = 4, kSelfX = 16384;

template <int NT>
__host__ __device__ constexpr int gate_up_sums() { return 4 * 2 * 4 * NT * 32 * 8; }   // float2 [kw][hf][tile][token tile][lane]

// Bytes of T rows of fixed point in shared memory.
__host__ __device__ constexpr int self_bytes(int T, int K) { return T * (2 * K + (K >> 6) * 8); }

template <typename T, int NT, bool SELF>
__global__ void __launch_bounds__(kThreads, 2)
    gate_up_kernel(const __grid_constant__ Maps maps, const Params p, int stages) {
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  SmemHead& S = *reinterpret_cast<SmemHead*>(sm);
  float2* red = reinterpret_cast<float2*>(sm + kHead);
  const int tokens = p.choice.T;
  uint8_t* own = sm + kHead + gate_up_sums<NT>();
  uint8_t* ring = sm + ring_offset(gate_up_sums<NT>() + (SELF ? self_bytes(tokens, p.K) : 0));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  if (tid == kThreads - 32) {
    prefetch_tmap(&maps.w);
    prefetch_tmap(&maps.s);
    prefetch_tmap(&maps.z);
    ring_init(S.R, stages);
  }
  grid_dep_wait();
  grid_dep_launch();   // after the wait: the next kernel may read the choice before its own wait
  build_lists<kThreads>(p.choice, S.L, *reinterpret_cast<ListsTemp*>(ring), 4 * NT);

  const int per_unit = p.I / kColsItem, nsub = p.K >> 6, nchunk = (nsub + 3) >> 2;
  const int64_t items = (int64_t)S.L.n_units * per_unit;
  const int i0 = (int)(items * blockIdx.x / gridDim.x), i1 = (int)(items * (blockIdx.x + 1) / gridDim.x);
  const int srows = 4 >> p.gsh;        // rows of scales a stage: its 256 columns' groups

  if (warp == kCons) {
    if (lane == 0) {
      const int ngrp = nsub >> p.gsh;
      int f = 0;
      for (int item = i0; item < i1; ++item) {
        const int u = item / per_unit, c0 = (item % per_unit) * kColsItem;
        const int e = S.L.unit_expert[u];
        for (int ch = 0; ch < nchunk; ++ch, ++f) {
          if (!ring_claim(S.R, stages, f)) break;
          uint8_t* st = ring + (f % stages) * kStage;
          uint64_t* bar = &S.R.full[f % stages];
          mbar_arrive_expect_tx(bar, kStageW + 4 * 128 * srows);
          tma_load_2d(st, &maps.w, bar, 128 * ch, e * 2 * p.I + c0);
          tma_load_2d(st + kStageW / 2, &maps.w, bar, 128 * ch, e * 2 * p.I + p.I + c0);
          const int sr = e * ngrp + ch * srows;
          tma_load_2d(st + kStageW, &maps.s, bar, c0, sr);
          tma_load_2d(st + kStageW + 512, &maps.z, bar, c0, sr);
          tma_load_2d(st + kStageW + 1024, &maps.s, bar, p.I + c0, sr);
          tma_load_2d(st + kStageW + 1536, &maps.z, bar, p.I + c0, sr);
        }
        if (S.R.abort) break;
      }
      if (S.R.abort) ring_drain(S.R, stages, f);
    }
    return;
  }

  Fixed xq = p.xq;
  if constexpr (SELF) {
    xq.q = own;
    xq.q_stride = 2 * p.K;
    xq.s_stride = nsub;
    xq.scale = reinterpret_cast<float2*>(own + tokens * 2 * p.K);
    for (int i = 0; i < tokens; ++i)
      convert_row<T, 32 * kCons>(reinterpret_cast<const T*>(p.x) + i * p.ldx, p.K, xq.q + i * xq.q_stride,
                                 xq.scale + i * xq.s_stride, tid);
    consumers_sync();
  }

  const int kw = warp >> 1, hf = warp & 1;
  int f = 0;
  for (int item = i0; item < i1; ++item) {
    const int u = item / per_unit, cb = item % per_unit;
    const int start = S.L.unit_start[u], n = S.L.unit_n[u];
    const uint8_t* bq[NT];             // the lane's column of B: hi or lo of token g / 2
    const float2* bs[NT];              // scales of token t
#pragma unroll
    for (int tt = 0; tt < NT; ++tt) {
      const int c = min(4 * tt + (g >> 1), n - 1), d = min(4 * tt + t, n - 1);   // past the last: its copies, unused
      bq[tt] = xq.q + S.L.slot_token[start + c] * xq.q_stride + kw * 128 + (g & 1) * 64 + t * 16;
      bs[tt] = xq.scale + (int64_t)S.L.slot_token[start + d] * xq.s_stride + kw;
    }
    float tot[4][NT][2] = {};
    for (int ch = 0; ch < nchunk; ++ch, ++f) {
      const uint8_t* st = ring + (f % stages) * kStage;
      const bool in = 4 * ch + kw < nsub;
      uint4 b[NT];
      float2 dx[NT];
      if (in) {
#pragma unroll
        for (int tt = 0; tt < NT; ++tt) {
          if (4 * tt >= n) break;
          b[tt] = *reinterpret_cast<const uint4*>(bq[tt] + ch * 512);
          dx[tt] = bs[tt][4 * ch];
        }
      }
      ring_await(S.R, stages, f);
      if (in) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {   // two gate tiles, two up tiles
          const int r = 32 * hf + 16 * (m & 1) + 2 * g;
          uint32_t a[2][4];
          load_tile(st + (m >> 1) * (kStageW / 2), r, kw, t, a);
          const uint8_t* sp = st + kStageW + (m >> 1) * 1024 + (kw >> p.gsh) * 128 + 2 * r;
          const float2 s = load_pair<T>(sp), z8 = fold_zero(s, load_pair<T>(sp + 512));
#pragma unroll
          for (int tt = 0; tt < NT; ++tt) {
            if (4 * tt >= n) break;
            add_block(tot[m][tt], a, b[tt], s, z8, dx[tt]);
          }
        }
      }
      ring_release(S.R, stages, f);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int tt = 0; tt < NT; ++tt)
        red[((warp * 4 + m) * NT + tt) * 32 + lane] = make_float2(tot[m][tt][0], tot[m][tt][1]);
    consumers_sync();
    for (int c = warp; c < n; c += kCons) {   // token c of the unit: a lane forms columns 2 lane and 2 lane + 1
      const int m = (lane >> 3) & 1, ln = (lane & 7) * 4 + (c & 3);
      float2 gate = make_float2(0.0f, 0.0f), up = gate;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2* q = red + (((2 * w + (lane >> 4)) * 4 + m) * NT + (c >> 2)) * 32 + ln;
        const float2 a = q[0], b = q[2 * NT * 32];
        gate.x += a.x, gate.y += a.y, up.x += b.x, up.y += b.y;
      }
      const float h0 = gate.x / (1.0f + expf(-gate.x)) * up.x, h1 = gate.y / (1.0f + expf(-gate.y)) * up.y;
      const uint32_t most = __reduce_max_sync(0xffffffffu, max(magnitude(h0), magnitude(h1)));
      const float2 d = block_scale(__uint_as_float(most));
      const int f0 = fixed_point(h0, d.y), f1 = fixed_point(h1, d.y);
      const int a0 = (f0 + 64) >> 7, a1 = (f1 + 64) >> 7;
      const int sum = __reduce_add_sync(0xffffffffu, f0 + f1);
      // columns 8 i + 2 j and + 1 (i = lane / 4, j = lane % 4): byte j of the run's even and odd words
      uint8_t* q = p.hq.q + (start + c) * p.hq.q_stride + cb * 128 + (lane >> 2) * 8 + (lane & 3);
      q[0] = (uint8_t)a0;
      q[4] = (uint8_t)a1;
      q[64] = (uint8_t)(f0 - 128 * a0);
      q[68] = (uint8_t)(f1 - 128 * a1);
      if (lane == 0) p.hq.scale[(int64_t)(start + c) * p.hq.s_stride + cb] = make_float2(d.x, d.x * (float)sum);
    }
    consumers_sync();                   // red is free again
  }
}

// --------------------------------------------------------------------- down

// A cluster of CTAs owns 32 output columns and walks (unit, 1024 columns of h)
// steps, each CTA a contiguous share of them; consumer warp w takes sub-blocks w
// and w + 8 of a step. When the unit changes, each warp adds its sums, times the
// tokens' weights, to its own (T, 32) accumulator in shared memory; at the end
// the warps' accumulators and then the CTAs' are added in order. The weights' ring
// starts before the dependency wait.
__host__ __device__ constexpr int down_sums(int T) { return kCons * T * kRowsTile * 4; }

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    down_kernel(const __grid_constant__ Maps maps, const Params p, int stages) {
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  SmemHead& S = *reinterpret_cast<SmemHead*>(sm);
  const int tokens = p.choice.T;
  float* sums = reinterpret_cast<float*>(sm + kHead);
  uint8_t* ring = sm + ring_offset(down_sums(tokens));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_ctarank(), ranks = cluster_nctarank();
  const int n0 = (int)(blockIdx.x / ranks) * kRowsTile, cells = tokens * kRowsTile;
  if (tid == kThreads - 32) {
    prefetch_tmap(&maps.w);
    prefetch_tmap(&maps.s);
    prefetch_tmap(&maps.z);
    ring_init(S.R, stages);
  }
  for (int i = tid; i < kCons * cells; i += kThreads) sums[i] = 0.0f;
  // The choice was complete before gate_up_kernel let this kernel start.
  build_lists<kThreads>(p.choice, S.L, *reinterpret_cast<ListsTemp*>(ring), 4 * NT);

  const int nsub = p.I >> 6, nchunk = (nsub + 15) >> 4;
  const int64_t steps = (int64_t)S.L.n_units * nchunk;
  const int s0 = (int)(steps * rank / ranks), s1 = (int)(steps * (rank + 1) / ranks);
  const int srows = 16 >> p.gsh;

  if (warp == kCons) {
    if (lane == 0) {
      const int ngrp = nsub >> p.gsh;
      int f = 0;
      for (int s = s0; s < s1; ++s, ++f) {
        if (!ring_claim(S.R, stages, f)) break;
        const int e = S.L.unit_expert[s / nchunk], ch = s % nchunk;
        uint8_t* st = ring + (f % stages) * kStage;
        uint64_t* bar = &S.R.full[f % stages];
        const int boxes = min(4, (nsub - 16 * ch + 3) >> 2);          // of 256 columns
        mbar_arrive_expect_tx(bar, boxes * (kStageW / 4) + 2 * 64 * srows);
        for (int i = 0; i < boxes; ++i)
          tma_load_2d(st + i * (kStageW / 4), &maps.w, bar, 512 * ch + 128 * i, e * p.K + n0);
        tma_load_2d(st + kStageW, &maps.s, bar, n0, e * ngrp + ch * srows);
        tma_load_2d(st + kStageW + 1024, &maps.z, bar, n0, e * ngrp + ch * srows);
      }
      if (S.R.abort) ring_drain(S.R, stages, f);
    }
    __syncwarp();
    grid_dep_wait();
    grid_dep_launch();
  } else {
    grid_dep_wait();
    grid_dep_launch();
    float* acc = sums + warp * cells;
    float tot[2][NT][2] = {};
    for (int s = s0, f = 0; s < s1; ++s, ++f) {
      const int u = s / nchunk, ch = s % nchunk;
      const int start = S.L.unit_start[u], n = S.L.unit_n[u];
      const uint8_t* st = ring + (f % stages) * kStage;
      uint4 b[2][NT];
      float2 dx[2][NT];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int sb = 16 * ch + warp + 8 * i;
        if (sb >= nsub) break;
#pragma unroll
        for (int tt = 0; tt < NT; ++tt) {
          if (4 * tt >= n) break;
          const int c = start + min(4 * tt + (g >> 1), n - 1), d = start + min(4 * tt + t, n - 1);
          b[i][tt] = *reinterpret_cast<const uint4*>(p.hq.q + c * p.hq.q_stride + sb * 128 + (g & 1) * 64 + t * 16);
          dx[i][tt] = p.hq.scale[(int64_t)d * p.hq.s_stride + sb];
        }
      }
      ring_await(S.R, stages, f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int sb = warp + 8 * i;
        if (16 * ch + sb >= nsub) break;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int r = 16 * m + 2 * g;
          uint32_t a[2][4];
          load_tile(st + (sb >> 2) * (kStageW / 4), r, sb, t, a);
          const uint8_t* sp = st + kStageW + (sb >> p.gsh) * 64 + 2 * r;
          const float2 sc = load_pair<T>(sp), z8 = fold_zero(sc, load_pair<T>(sp + 1024));
#pragma unroll
          for (int tt = 0; tt < NT; ++tt) {
            if (4 * tt >= n) break;
            add_block(tot[m][tt], a, b[i][tt], sc, z8, dx[i][tt]);
          }
        }
      }
      ring_release(S.R, stages, f);
      if (s + 1 == s1 || (s + 1) / nchunk != u) {   // the unit's last step here
#pragma unroll
        for (int tt = 0; tt < NT; ++tt) {
          const int i = 4 * tt + t;                 // the lane's token
          if (i < n) {
            const float w = S.L.slot_w[start + i];
            float* ap = acc + S.L.slot_token[start + i] * kRowsTile + 2 * g;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              ap[16 * m] = fmaf(w, tot[m][tt][0], ap[16 * m]);
              ap[16 * m + 1] = fmaf(w, tot[m][tt][1], ap[16 * m + 1]);
            }
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) tot[m][tt][0] = tot[m][tt][1] = 0.0f;
        }
        __syncwarp();                               // another lane may hold this token in the next unit
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < cells; i += kThreads) {
    float v = sums[i];
#pragma unroll
    for (int w = 1; w < kCons; ++w) v += sums[w * cells + i];
    sums[i] = v;
  }
  cluster_sync();
  const uint32_t base = smem_u32(sums);
  for (int i = rank * kThreads + tid; i < cells; i += ranks * kThreads) {
    float v = 0.0f;
    for (uint32_t r = 0; r < ranks; ++r) v += ld_cluster_f32(mapa_shared(base + 4 * i, r));
    reinterpret_cast<T*>(p.out)[(int64_t)(i / kRowsTile) * p.K + n0 + i % kRowsTile] = awq::Traits<T>::fromf(v);
  }
  cluster_sync();                                   // no CTA leaves while another reads its sums
}

}  // namespace moe
}  // namespace ck
