// A mixture-of-experts layer for a few tokens on AWQ W4A16 experts.
//
//   W[n, c] = (u[n, c] - 8) s[c / G, n] + z[c / G, n]         (each expert's, as gemv_awq.cuh)
//   h[t, e] = silu(x_t Wg_e^T) * (x_t Wu_e^T),  silu(v) = v / (1 + exp(-v))
//   out_t   = sum over t's experts of w[t, e] (h[t, e] Wd_e^T)
//
// gate_up_kernel computes h, down_kernel the weighted sum. For one or two tokens both choose
// the experts (or take the choice) in every CTA and gate_up orders x; otherwise
// prepare_kernel does that once for all. Each weight that some token
// needs is read from HBM once (again for each 16 tokens, or fewer, that share an expert), and that
// bounds the layer: a tile of 16 weight rows x 64 columns (512 packed bytes) takes one of
// an SM's four schedulers 89 clocks at the measured copy bandwidth, so a tile must cost well
// under 89 issue slots. Measured, device time and the bytes' time at the copy bandwidth: 16 tokens, top-8
// of 64 experts, K = 2048, I = 1024 60 us (31.0); 32 tokens, top-2 of 8, K = 3840, I = 10240
// 192 (77.8; the same loads without the products 124); one token 16.7 (4.4).
//
// Products. The nibbles become exact 16-bit numbers u - 8 in registers, the A operands of
// mma.sync.m16n8k16 (16 weight rows); the tokens are the columns of B. For a sub-block of 64
// columns, which lies in one quantization group (G % 64 == 0),
//   sum of W x = s P + z X,   P = sum of (u - 8) x,   X = sum of x,
// with P and X in 32 bits. A weight of zero adds an exact zero to P, however large its x is.
// * x enters as it is: eight tokens are the columns of B.
// * h, computed in 32 bits, enters as hi + lo, two fp16 numbers (four tokens' hi and lo are the columns
//   of B), for both types of x: u - 8 is exact in fp16 too. A power of two for each sub-block
//   brings its largest magnitude to [2^13, 2^14), so that h may be of any size. hi + lo has
//   22 bits and two signs: h moves by at most 2^-23 of itself, or where that is more by 2^-25, half of fp16's
//   smallest step, which is 2^-38 of the sub-block's largest h. Two bf16 numbers would lose 2^-18.
// (Activations as 15-bit fixed point with a scale for each 64 columns, int8 MMAs, took 46, 138 and 14.8 us for
// the three cases above, but an entry far above the others of its block cost those their bits:
// one of 1000 times their size moved them by 3 % of themselves.)
//
// A token with an entry of x that is not finite gets h and outputs that are not.
//
// Sums run in a fixed order: the output does not depend on timing.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "cluster_mem.cuh"
#include "gemv_awq.cuh"
#include "moe_route.cuh"

namespace ck {
namespace moe {

constexpr int kColsItem = 64;          // columns of h in one item of gate_up_kernel: one sub-block of down_kernel
constexpr int kRowsTile = 64;          // output columns of one cluster of down_kernel
constexpr int kMaxStages = 6;

// Rows of activations, in records. Eight columns (a packed word's nibbles) are a piece of 16 bytes in the
// order 0 4 1 5 2 6 3 7, in which decode() gives that word's nibbles.
// x: a record is four sub-blocks, each 128 bytes in the order of the pieces; behind them X of each.
// h: a record is two sub-blocks, each 256 bytes: the even pieces (columns 0-7, 16-23, ...) of hi, those of
//    lo, the odd ones of hi, those of lo; behind them {d, d, X, X} of each (operands of packed instructions).
constexpr int kRecord = 512 + 64;
constexpr int kRowPad = 16;            // between tokens in shared memory: what lanes read at once is in different banks
__host__ __device__ constexpr int x_row_bytes(int columns) { return (columns + 255) / 256 * kRecord; }
__host__ __device__ constexpr int h_row_bytes(int columns) { return (columns + 127) / 128 * kRecord; }

struct Params {
  Choice choice;
  const void* x;                       // (T, K) T, row stride ldx
  int64_t ldx;
  int K, I, gsh;                       // quantization group of sub-block sb: sb >> gsh
  uint8_t* xr;                         // (T) rows of x by prepare_kernel; unused where a CTA orders x itself
  uint8_t* hr;                         // (slots) rows of h
  uint8_t* lists;                      // by prepare_kernel (lists_at)
  void* out;                           // (T, K) T
};

// Tensor maps of one weight matrix of all experts and of its scales and zeros.
struct Maps {
  CUtensorMap w, s, z;
};

// ------------------------------------------------------- rows of activations

// |v| for a maximum that a NaN must not get lost in: as unsigned bits, where NaN is above infinity.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The power of two that brings a block's largest magnitude (its bits) to [2^13, 2^14), as far as it is a
// normal number, and its inverse, which scales the block's products. Not finite: {0, NaN}.
__device__ __forceinline__ float2 block_scale(uint32_t top) {
  const int e = (int)(top >> 23);
  if (e == 255) return make_float2(0.0f, __int_as_float(0x7fffffff));
  const int up = min(126, 140 - e);                  // 13 - (e - 127)
  return make_float2(__int_as_float((127 + up) << 23), __int_as_float((127 - up) << 23));
}

// Orders row `row` of x (K values) by a group of THREADS threads (a multiple of 8), a piece
// a thread at a time; lane groups of eight hold a sub-block.
template <typename T, int THREADS>
__device__ __forceinline__ void order_row(const T* x, int K, uint8_t* row, int tid) {
  const int blocks = K >> 6;
  for (int b0 = 0; b0 < blocks; b0 += THREADS / 8) {   // the whole warp stays for the shuffles
    const int sb = b0 + tid / 8, part = tid & 7;
    const bool in = sb < blocks;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (in) raw = *reinterpret_cast<const uint4*>(x + sb * 64 + part * 8);
    const T* v = reinterpret_cast<const T*>(&raw);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += awq::Traits<T>::tof(v[i]);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (in) {
      uint8_t* rec = row + (sb >> 2) * kRecord;
      *reinterpret_cast<uint4*>(rec + (sb & 3) * 128 + part * 16) =
          make_uint4(__byte_perm(raw.x, raw.z, 0x5410), __byte_perm(raw.x, raw.z, 0x7632),
                     __byte_perm(raw.y, raw.w, 0x5410), __byte_perm(raw.y, raw.w, 0x7632));
      if (part == 0) reinterpret_cast<float*>(rec + 512)[sb & 3] = sum;
    }
  }
}

// ----------------------------------------------------------- prepare

// CTA t < T: token t's row of x in the products' order. CTA T: the choice and its lists.
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) prepare_kernel(const Params p, int cap) {
  __shared__ ListsTemp tmp;
  __shared__ __align__(16) uint8_t block[lists_bytes(kMaxSlots)];
  grid_dep_wait();
  grid_dep_launch();
  const int t = blockIdx.x, slots = p.choice.T * p.choice.k;
  if (t < p.choice.T) {
    order_row<T, THREADS>(reinterpret_cast<const T*>(p.x) + t * p.ldx, p.K, p.xr + (int64_t)t * x_row_bytes(p.K),
                          threadIdx.x);
    return;
  }
  build_lists<THREADS>(p.choice, lists_at(block, slots), tmp, cap);
  for (int i = threadIdx.x; i < lists_bytes(slots) / 16; i += THREADS)
    reinterpret_cast<uint4*>(p.lists)[i] = reinterpret_cast<const uint4*>(block)[i];
}

// ------------------------------------------------------------- weight tiles

// Two neighbouring scales (or zeros) of type T as floats.
template <typename T>
__device__ __forceinline__ float2 load_pair(const uint8_t* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  const T* v = reinterpret_cast<const T*>(&u);
  return make_float2(awq::Traits<T>::tof(v[0]), awq::Traits<T>::tof(v[1]));
}

// Where a lane finds its 8 packed bytes of row r (even) and sub-block sb (0 .. 3) in a box of 256
// columns: 16-byte chunk c of row r is at c ^ (r % 8). Row r + 1's are at (that ^ 16) + 128, and those of
// sub-block sb ^ 2 at that ^ 64. Row g of an MMA's fragment is row r = r0 + 2 g, row g + 8 is r + 1: a lane's
// two scales are neighbours, and a half-warp's reads hit each bank once.
__device__ __forceinline__ int tile_offset(int r, int sb, int t) {
  return r * 128 + (((2 * sb + (t >> 1)) ^ (r & 7)) << 4) + 8 * (t & 1);
}

// (w & mask) | magic in one operation. `magic` must not be known to the compiler: an instruction holds one
// immediate, and with two constants it takes two (the logical operations of a tile bound the layer then:
// 16 tokens of 64 experts 70 us, 60 so).
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));
  return r;
}

// A packed word's nibbles as u - 8, exact, in four pairs of 16-bit numbers: columns (0, 4), (1, 5), (2, 6), (3, 7).
template <typename T>
__device__ __forceinline__ void decode(uint32_t w, uint32_t magic, uint32_t (&p)[4]) {
  if constexpr (std::is_same<T, __half>::value) {
    // 0x6400 | u is 1024 + u, 0x6400 | 16 u is 1024 + 16 u: one shift a word in place of three
    const __half2 bias = __float2half2_rn(-1032.0f), part = __float2half2_rn(0.0625f), rest = __float2half2_rn(-72.0f);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint32_t v = w >> (4 * i), a = and_or(v, 0x000F000Fu, magic), b = and_or(v, 0x00F000F0u, magic);
      const __half2 x = __hadd2(*reinterpret_cast<const __half2*>(&a), bias);
      const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&b), part, rest);
      p[i] = *reinterpret_cast<const uint32_t*>(&x);
      p[i + 1] = *reinterpret_cast<const uint32_t*>(&y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = awq::Traits<T>::sub2(and_or(w >> (4 * i), 0x000F000Fu, magic), awq::Traits<T>::kBias);
  }
}

// A tile of 16 weight rows x 64 columns as the A operands of four MMAs: the lane's 16 columns of rows r and r + 1.
template <typename T>
__device__ __forceinline__ void load_tile(const uint8_t* row0, const uint8_t* row1, uint32_t magic, uint32_t (&a)[4][4]) {
  const uint2 w0 = *reinterpret_cast<const uint2*>(row0), w1 = *reinterpret_cast<const uint2*>(row1);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t p[4], q[4];
    decode<T>(i == 0 ? w0.x : w0.y, magic, p);
    decode<T>(i == 0 ? w1.x : w1.y, magic, q);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      a[2 * i + j][0] = p[2 * j], a[2 * i + j][1] = q[2 * j];
      a[2 * i + j][2] = p[2 * j + 1], a[2 * i + j][3] = q[2 * j + 1];
    }
  }
}

// c = the sub-block's sums of (u - 8) times the columns of B, whose 16 columns of this lane are the pieces b0, b1.
template <typename T>
__device__ __forceinline__ void multiply(float (&c)[4], const uint32_t (&a)[4][4], const uint4 b0, const uint4 b1) {
  c[0] = c[1] = c[2] = c[3] = 0.0f;
  awq::Traits<T>::mma(c, a[0], b0.x, b0.y);
  awq::Traits<T>::mma(c, a[1], b0.z, b0.w);
  awq::Traits<T>::mma(c, a[2], b1.x, b1.y);
  awq::Traits<T>::mma(c, a[3], b1.z, b1.w);
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

__device__ __forceinline__ void ring_init(Ring& R, int stages, int consumers) {
  for (int s = 0; s < stages; ++s) {
    mbar_init(&R.full[s], 1);
    mbar_init(&R.empty[s], consumers);
  }
  R.abort = 0;
  fence_mbarrier_init();
}

// Where a thread is in the ring: its stage, and the parity of that stage's round.
struct Cursor {
  int stage = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) stage = 0, parity ^= 1;
  }
};

// Producer (one thread): waits until the stage may be overwritten (at once in the first round).
__device__ __forceinline__ bool ring_claim(Ring& R, const Cursor& c) {
  return mbar_wait(&R.empty[c.stage], c.parity ^ 1, &R.abort, 50);
}

// Producer: after giving up, waits (with a limit) for the copies in flight: every stage's last fill.
__device__ __forceinline__ void ring_drain(Ring& R, Cursor c, int stages, int issued) {
  for (int i = 0; i < issued && i < stages; ++i) {
    if (c.stage == 0) c.stage = stages, c.parity ^= 1;
    --c.stage;
    mbar_wait(&R.full[c.stage], c.parity, nullptr, 51, 100000000ull);
  }
}

__device__ __forceinline__ void ring_await(Ring& R, const Cursor& c) {
  warp_wait(&R.full[c.stage], c.parity, &R.abort, 52);
}

__device__ __forceinline__ void ring_release(Ring& R, const Cursor& c) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&R.empty[c.stage]);
}

// The consumer warps' own barrier.
template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Global memory that earlier kernels wrote may be read by bulk copies from here on.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Shared memory of both kernels: the ring's barriers, the lists, what the kernel sums in, and
// the ring (1024-byte aligned stages).
constexpr int kHead = (sizeof(Ring) + 127) / 128 * 128;
__host__ __device__ constexpr int ring_offset(int slots, int sums) {
  return (kHead + (lists_bytes(slots) + 127) / 128 * 128 + sums + 1023) / 1024 * 1024;
}

__device__ __forceinline__ uint8_t* align_1024(uint8_t* p) { return p + ((1024 - (smem_u32(p) & 1023)) & 1023); }

// -------------------------------------------------------------- gate and up

// An item is 64 columns of h of one unit (an expert's tokens, at most 4 NT): 64
// gate rows and the 64 up rows that belong to them. A CTA takes every gridDim.x-th
// item, so that units of many and of few tokens mix (in contiguous shares some CTAs
// ran for 45 us and others for 128), and streams its weights, with the unit's rows of x,
// 128 KW columns a stage. Consumer warp (kw, rq) multiplies 16 gate and 16 up rows with sub-blocks kw
// and kw + KW of each stage; the KW partial sums meet in shared memory, where
// one warp a token forms h, as hi + lo.
//
// SELF: every CTA routes and converts x itself, into shared memory (T <= kFewTokens): the
// launch of prepare_kernel and the wait for it cost more.
constexpr int kSelfBytes = 32 * 1024;

template <int NT, int KW, bool SELF>
struct GateUp {
  static constexpr int kCons = 4 * KW, kThreads = 32 * (kCons + 1);
  static constexpr int kCtas = KW == 4 ? 1 : 2;     // on an SM (three with shallower rings: 63.5 against 60.2 us at 16 tokens)
  static constexpr int kSubs = 2 * KW;                          // sub-blocks a stage
  static constexpr int kW = kSubs * 64 * 32;                    // its bytes of gate (or up) weights
  static constexpr int kS = kSubs * 128;                        // bytes of each kind of scales
  static constexpr int kRow = (kSubs / 4) * kRecord + kRowPad;  // of a token's columns of x in a stage
  static constexpr int kRows = SELF ? 0 : 4 * NT * kRow;
  static constexpr int kStage = (2 * kW + 4 * kS + kRows + 1023) / 1024 * 1024;
  static constexpr int kRed = KW * 4 * 2 * NT * 32 * 8;         // float2 [kw][rq][gate, up][token tile][lane]
  static_assert(sizeof(FewTemp) <= kRed, "the choice is handed on in it");
  __host__ __device__ static constexpr int sums(int T, int K) { return kRed + (SELF ? T * x_row_bytes(K) : 0); }
};

template <typename T, int NT, int KW, bool SELF>
__device__ __forceinline__ void gate_up(const Maps& maps, const Params& p, int stages) {
  using C = GateUp<NT, KW, SELF>;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = align_1024(sm_raw);
  Ring& R = *reinterpret_cast<Ring*>(sm);
  const int tokens = p.choice.T, slots = tokens * p.choice.k;
  const Lists L = lists_at(sm + kHead, slots);
  float2* red = reinterpret_cast<float2*>(sm + kHead + (lists_bytes(slots) + 127) / 128 * 128);
  uint8_t* own = reinterpret_cast<uint8_t*>(red) + C::kRed;
  uint8_t* ring = sm + ring_offset(slots, C::sums(tokens, p.K));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  if (tid == C::kThreads - 32) {
    prefetch_tmap(&maps.w);
    prefetch_tmap(&maps.s);
    prefetch_tmap(&maps.z);
    ring_init(R, stages, C::kCons);
  }
  grid_dep_wait();
  grid_dep_launch();   // after the wait: the next kernel may read the choice before its own wait
  const int xrow = x_row_bytes(p.K);
  if constexpr (SELF) {                // warps 0 and 1 choose (a token each) while the others order x
    FewTemp& few = *reinterpret_cast<FewTemp*>(red);
    constexpr int kOrder = C::kThreads - 32 * kFewTokens;
    if (warp < kFewTokens) {
      choose_few(p.choice, few);
    } else {
      for (int i = 0; i < tokens; ++i)
        order_row<T, kOrder>(reinterpret_cast<const T*>(p.x) + i * p.ldx, p.K, own + i * xrow, tid - 32 * kFewTokens);
    }
    __syncthreads();
    list_few(p.choice, L, few);
    __syncthreads();
  } else {
    copy_lists<C::kThreads>(sm + kHead, p.lists, slots);
  }

  const int per_unit = p.I / kColsItem, nsub = p.K >> 6, nchunk = (nsub + C::kSubs - 1) / C::kSubs;
  const int items = L.units() * per_unit;
  const int srows = C::kSubs >> p.gsh;   // rows of scales a stage: its columns' groups

  if (warp == C::kCons) {
    fence_proxy_async_all();
    const int ngrp = nsub >> p.gsh;
    Cursor at;
    int issued = 0;
    bool live = true;
    for (int item = blockIdx.x; item < items && live; item += gridDim.x) {
      const int u = item / per_unit, c0 = (item % per_unit) * kColsItem;
      const int e = L.unit_expert[u], row = e * 2 * p.I + c0, n = L.unit_n[u];
      const uint8_t* xr = nullptr;
      if (!SELF && lane < n) xr = p.xr + (int64_t)L.slot_token[L.unit_start[u] + lane] * xrow;
      for (int ch = 0; ch < nchunk; ++ch, at.next(stages)) {
        live = __all_sync(0xffffffffu, ring_claim(R, at));
        if (!live) break;
        ++issued;
        uint8_t* st = ring + at.stage * C::kStage;
        uint64_t* bar = &R.full[at.stage];
        const int boxes = min(C::kSubs / 4, (nsub - C::kSubs * ch + 3) >> 2);   // of 256 columns
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, boxes * (2 * 64 * 128 + (SELF ? 0 : n * kRecord)) + 4 * 128 * srows);
          for (int i = 0; i < boxes; ++i) {
            tma_load_2d(st + i * 64 * 128, &maps.w, bar, (C::kSubs * ch + 4 * i) * 32, row);
            tma_load_2d(st + C::kW + i * 64 * 128, &maps.w, bar, (C::kSubs * ch + 4 * i) * 32, row + p.I);
          }
          const int sr = e * ngrp + ch * srows;
          uint8_t* sc = st + 2 * C::kW;
          tma_load_2d(sc, &maps.s, bar, c0, sr);
          tma_load_2d(sc + C::kS, &maps.z, bar, c0, sr);
          tma_load_2d(sc + 2 * C::kS, &maps.s, bar, p.I + c0, sr);
          tma_load_2d(sc + 3 * C::kS, &maps.z, bar, p.I + c0, sr);
        }
        __syncwarp();
        if (!SELF && lane < n)
          bulk_load(st + 2 * C::kW + 4 * C::kS + lane * C::kRow, xr + ch * (C::kSubs / 4) * kRecord,
                    boxes * kRecord, bar);
      }
    }
    if (!live && lane == 0) ring_drain(R, at, stages, issued);
    return;
  }

  const int kw = warp >> 2, rq = warp & 3;
  const int tile = tile_offset(16 * rq + 2 * g, kw, t);
  const int sc0 = (kw >> p.gsh) * 128 + 32 * rq + 4 * g, sc1 = ((kw + KW) >> p.gsh) * 128 + 32 * rq + 4 * g;
  Cursor at;
  const uint32_t magic = awq::Traits<T>::kMagic | (uint32_t)(p.gsh >> 8);   // (gsh < 8)
  constexpr int N8 = (NT + 1) / 2;       // tiles of eight tokens
  float2 tot[2][N8][2];                  // gate and up: rows r and r + 1 for tokens 2 t and 2 t + 1 of a tile
  // One item's products with N tiles; sums in tot.
  auto products = [&](auto tiles, int start, int n) {
    constexpr int N = decltype(tiles)::value;
    // the lane's column of B (token g) and where the X of tokens 2 t and 2 t + 1 are; past the last
    // token its copies, whose results nobody reads
    int bq[N], bx[N][2];
    auto row_of = [&](int c) {
      c = min(c, n - 1);
      return SELF ? L.slot_token[start + c] * xrow : c * C::kRow;
    };
#pragma unroll
    for (int tt = 0; tt < N; ++tt) {
      bq[tt] = row_of(8 * tt + g) + kw * 128 + t * 32;
      bx[tt][0] = row_of(8 * tt + 2 * t) + 512 + kw * 4;
      bx[tt][1] = row_of(8 * tt + 2 * t + 1) + 512 + kw * 4;
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int tt = 0; tt < N; ++tt) tot[m][tt][0] = tot[m][tt][1] = make_float2(0.0f, 0.0f);
    for (int ch = 0; ch < nchunk; ++ch, at.next(stages)) {
      const uint8_t* st = ring + at.stage * C::kStage;
      const uint8_t* rec = SELF ? own + ch * (C::kSubs / 4) * kRecord : st + 2 * C::kW + 4 * C::kS;
      ring_await(R, at);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int sb = kw + KW * i;      // of the stage
        if (C::kSubs * ch + sb >= nsub) break;
        // KW = 2: sub-blocks kw and kw + 2 of one box; KW = 4: sub-block kw of two boxes
        const uint8_t* row0 = st + (KW == 2 && i == 1 ? tile ^ 64 : tile) + (KW == 4 ? i * 64 * 128 : 0);
        const uint8_t* row1 = st + 128 + (KW == 2 && i == 1 ? tile ^ 80 : tile ^ 16) + (KW == 4 ? i * 64 * 128 : 0);
        const uint8_t* sp = st + 2 * C::kW + (i == 0 ? sc0 : sc1);
        uint4 b[N][2];
        float2 X[N];
#pragma unroll
        for (int tt = 0; tt < N; ++tt) {
          const uint8_t* bp = rec + bq[tt] + (KW == 4 ? i * kRecord : i * 256);
          b[tt][0] = *reinterpret_cast<const uint4*>(bp);
          b[tt][1] = *reinterpret_cast<const uint4*>(bp + 16);
          const int at_x = KW == 4 ? i * kRecord : i * 8;
          X[tt] = make_float2(*reinterpret_cast<const float*>(rec + bx[tt][0] + at_x),
                              *reinterpret_cast<const float*>(rec + bx[tt][1] + at_x));
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {    // gate, up
          uint32_t a[4][4];
          load_tile<T>(row0 + m * C::kW, row1 + m * C::kW, magic, a);
          const float2 s = load_pair<T>(sp + 2 * m * C::kS), z = load_pair<T>(sp + 2 * m * C::kS + C::kS);
#pragma unroll
          for (int tt = 0; tt < N; ++tt) {
            float c[4];
            multiply<T>(c, a, b[tt][0], b[tt][1]);
            tot[m][tt][0] = __ffma2_rn(make_float2(s.x, s.x), make_float2(c[0], c[1]), tot[m][tt][0]);
            tot[m][tt][1] = __ffma2_rn(make_float2(s.y, s.y), make_float2(c[2], c[3]), tot[m][tt][1]);
            tot[m][tt][0] = __ffma2_rn(make_float2(z.x, z.x), X[tt], tot[m][tt][0]);
            tot[m][tt][1] = __ffma2_rn(make_float2(z.y, z.y), X[tt], tot[m][tt][1]);
          }
        }
      }
      ring_release(R, at);
    }
  };

  for (int item = blockIdx.x, turn = 0; item < items; item += gridDim.x, ++turn) {
    const int u = item / per_unit, cb = item % per_unit;
    const int start = L.unit_start[u], n = L.unit_n[u], nt = (n + 3) >> 2;
    if (N8 == 1 || n <= 8) products(std::integral_constant<int, 1>(), start, n);
    else products(std::integral_constant<int, N8>(), start, n);
    if (turn != 0) consumers_sync<32 * C::kCons>();   // the previous item's sums have been read
    // in red's tiles of four tokens lane 4 g' + t' holds rows 2 g' and 2 g' + 1 for token t'
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int tt = 0; tt < N8; ++tt) {
        const int four = 2 * tt + (t >> 1);
        const float2 u = tot[m][tt][0], v = tot[m][tt][1];
        if (four < nt)
          *reinterpret_cast<float4*>(&red[((warp * 2 + m) * NT + four) * 32 + 4 * g + 2 * (t & 1)]) =
              make_float4(u.x, v.x, u.y, v.y);
      }
    consumers_sync<32 * C::kCons>();
    // Token c of the unit: a lane forms columns 2 lane and 2 lane + 1. The other warps go on.
    for (int c = (warp + turn) & (C::kCons - 1); c < n; c += C::kCons) {
      const int ln = (lane & 7) * 4 + (c & 3);
      float2 gate = make_float2(0.0f, 0.0f), up = gate;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const float2* q = red + (((w * 4 + (lane >> 3)) * 2) * NT + (c >> 2)) * 32 + ln;
        const float2 a = q[0], b = q[NT * 32];
        gate.x += a.x, gate.y += a.y, up.x += b.x, up.y += b.y;
      }
      // with the token's weight: down_kernel only adds
      const float w = L.slot_w[start + c];
      const float h0 = w * (gate.x / (1.0f + expf(-gate.x)) * up.x), h1 = w * (gate.y / (1.0f + expf(-gate.y)) * up.y);
      const float2 d = block_scale(__reduce_max_sync(0xffffffffu, max(magnitude(h0), magnitude(h1))));
      float sum = h0 + h1;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      // hi and lo of h d.x; zeros where the block is not finite (its products get d.y = NaN)
      const float v0 = d.x == 0.0f ? 0.0f : h0 * d.x, v1 = d.x == 0.0f ? 0.0f : h1 * d.x;
      const __half hi0 = __float2half_rn(v0), hi1 = __float2half_rn(v1);
      const __half lo0 = __float2half_rn(v0 - __half2float(hi0)), lo1 = __float2half_rn(v1 - __half2float(hi1));
      // columns 8 i + 2 j and + 1 (i = lane / 4, j = lane % 4): of piece i, places 0 2, 4 6, 1 3, 5 7 by j
      uint8_t* rec = p.hr + (int64_t)(start + c) * h_row_bytes(p.I) + (cb >> 1) * kRecord;
      __half* q = reinterpret_cast<__half*>(rec + (cb & 1) * 256 + ((lane >> 2) & 1) * 128 + (lane >> 3) * 16) +
                  4 * (lane & 1) + ((lane >> 1) & 1);
      q[0] = hi0;
      q[2] = hi1;
      q[32] = lo0;
      q[34] = lo1;
      if (lane == 0) reinterpret_cast<float4*>(rec + 512)[cb & 1] = make_float4(d.y, d.y, sum, sum);
    }
  }
}

template <typename T, int NT>
__global__ void __launch_bounds__(GateUp<NT, 2, false>::kThreads, GateUp<NT, 2, false>::kCtas)
    gate_up_kernel(const __grid_constant__ Maps maps, const Params p, int stages) {
  gate_up<T, NT, 2, false>(maps, p, stages);
}

// 64 registers: a CTA of down_kernel fits beside this one's, and builds its lists and fetches its first weights
// while this kernel runs.
template <typename T>
__global__ void __maxnreg__(64)
    gate_up_few_kernel(const __grid_constant__ Maps maps, const Params p, int stages) {
  gate_up<T, 1, 4, true>(maps, p, stages);
}

// --------------------------------------------------------------------- down

// A cluster of CTAs owns 64 output columns and walks (unit, 512 columns of h)
// steps, each CTA a share of them; consumer warp (kw, rh) takes sub-blocks
// kw and kw + 4 of a step and 32 of the output columns. When the unit changes, each warp
// adds its sums to the accumulator (T, 64) that it shares with the other rh; at the
// end the four accumulators and then the CTAs' are added in order. The weights of
// the first stages are fetched before the dependency wait, the rows of h after it.
template <int NT>
struct Down {
  // CTAs on an SM. With rows of h for 16 tokens a second one finds no room; the registers that it would
  // need keep more products in flight instead (64 tokens, top-2 of 8, K = I = 4096: 154 us with half of them, 142 so).
  static constexpr int kCtas = NT == 4 ? 1 : 2;
  static constexpr int SUB = 2;                  // sub-blocks a warp and step (1: 64.3 against 60.2 us at 16 tokens of 64 experts)
  static constexpr int kCons = 8, kThreads = 32 * (kCons + 1);
  static constexpr int kSubs = 4 * SUB;
  static constexpr int kW = kSubs * 64 * 32;
  static constexpr int kS = kSubs * 128;
  static constexpr int kRecs = kSubs / 2;        // records of h a step
  static constexpr int kRow = kRecs * kRecord + kRowPad;
  static constexpr int kStage = (kW + 2 * kS + 4 * NT * kRow + 1023) / 1024 * 1024;
  __host__ __device__ static constexpr int sums(int T) { return 4 * T * kRowsTile * 4; }
};

template <typename T, int NT>
__global__ void __launch_bounds__(Down<NT>::kThreads, Down<NT>::kCtas)
    down_kernel(const __grid_constant__ Maps maps, const Params p, int stages) {
  using C = Down<NT>;
  constexpr int SUB = C::SUB;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = align_1024(sm_raw);
  Ring& R = *reinterpret_cast<Ring*>(sm);
  const int tokens = p.choice.T, slots = tokens * p.choice.k;
  const Lists L = lists_at(sm + kHead, slots);
  float* sums = reinterpret_cast<float*>(sm + kHead + (lists_bytes(slots) + 127) / 128 * 128);
  uint8_t* ring = sm + ring_offset(slots, C::sums(tokens));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_ctarank(), ranks = cluster_nctarank();
  const int n0 = (int)(blockIdx.x / ranks) * kRowsTile, cells = tokens * kRowsTile;
  if (tid == C::kThreads - 32) {
    prefetch_tmap(&maps.w);
    prefetch_tmap(&maps.s);
    prefetch_tmap(&maps.z);
    ring_init(R, stages, C::kCons);
  }
  // The choice and the lists were complete before gate_up_kernel let this kernel start.
  if (p.lists == nullptr) {
    FewTemp& few = *reinterpret_cast<FewTemp*>(sums);   // (cleared below)
    choose_few(p.choice, few);
    __syncthreads();
    list_few(p.choice, L, few);
    __syncthreads();
  } else {
    copy_lists<C::kThreads>(sm + kHead, p.lists, slots);
  }
  for (int i = tid; i < 4 * cells; i += C::kThreads) sums[i] = 0.0f;
  __syncthreads();

  const int nsub = p.I >> 6, nchunk = (nsub + C::kSubs - 1) / C::kSubs;
  const int srows = C::kSubs >> p.gsh;
  const int hrow = h_row_bytes(p.I), nrec = (nsub + 1) >> 1;
  // This CTA's steps: with many chunks a unit, every ranks-th chunk of each unit (units of many
  // and of few tokens mix); else a contiguous share.
  const int units = L.units();
  int u0 = 0, ch0 = (int)rank, stride = (int)ranks, left;
  if (nchunk >= 2 * (int)ranks) {
    left = units * ((nchunk - (int)rank + (int)ranks - 1) / (int)ranks);
  } else {
    const int steps = units * nchunk, s0 = (int)((int64_t)steps * rank / ranks);
    left = (int)((int64_t)steps * (rank + 1) / ranks) - s0;
    u0 = s0 / nchunk;
    ch0 = s0 - u0 * nchunk;
    stride = 1;
  }
  const int again = stride == 1 ? 0 : ch0;           // the first chunk of the next unit

  if (warp == C::kCons) {
    const int ngrp = nsub >> p.gsh;
    // Weights and scales of a step, and the bytes of its rows of h announced.
    auto fetch_weights = [&](int u, int ch, const Cursor& at) {
      const int e = L.unit_expert[u];
      uint8_t* st = ring + at.stage * C::kStage;
      uint64_t* bar = &R.full[at.stage];
      const int boxes = min(SUB, (nsub - C::kSubs * ch + 3) >> 2);
      const int recs = min(C::kRecs, nrec - C::kRecs * ch);
      mbar_arrive_expect_tx(bar, boxes * 64 * 128 + L.unit_n[u] * recs * kRecord + 2 * 128 * srows);
      for (int i = 0; i < boxes; ++i)
        tma_load_2d(st + i * 64 * 128, &maps.w, bar, (C::kSubs * ch + 4 * i) * 32, e * p.K + n0);
      tma_load_2d(st + C::kW, &maps.s, bar, n0, e * ngrp + ch * srows);
      tma_load_2d(st + C::kW + C::kS, &maps.z, bar, n0, e * ngrp + ch * srows);
    };
    auto fetch_rows = [&](int u, int ch, const Cursor& at) {
      const int recs = min(C::kRecs, nrec - C::kRecs * ch);
      if (lane < L.unit_n[u])
        bulk_load(ring + at.stage * C::kStage + C::kW + 2 * C::kS + lane * C::kRow,
                  p.hr + (int64_t)(L.unit_start[u] + lane) * hrow + ch * C::kRecs * kRecord, recs * kRecord,
                  &R.full[at.stage]);
    };
    const int ahead = min(stages, left);
    Cursor at;
    int u = u0, ch = ch0;
    auto step = [&] {
      at.next(stages);
      if ((ch += stride) >= nchunk) ch = again, ++u;
    };
    if (lane == 0)
      for (int i = 0; i < ahead; ++i, step()) fetch_weights(u, ch, at);
    __syncwarp();
    grid_dep_wait();
    grid_dep_launch();
    fence_proxy_async_all();
    at = Cursor();
    u = u0, ch = ch0;
    for (int i = 0; i < ahead; ++i, step()) fetch_rows(u, ch, at);
    int issued = ahead;
    bool live = true;
    for (; issued < left; ++issued, step()) {
      live = __all_sync(0xffffffffu, ring_claim(R, at));
      if (!live) break;
      if (lane == 0) fetch_weights(u, ch, at);
      __syncwarp();
      fetch_rows(u, ch, at);
    }
    if (!live && lane == 0) ring_drain(R, at, stages, issued);
  } else {
    grid_dep_wait();
    grid_dep_launch();
    const int kw = warp >> 1, rh = warp & 1;
    const uint32_t magic = awq::Traits<__half>::kMagic | (uint32_t)(p.gsh >> 8);   // (gsh < 8)
    float* acc = sums + kw * cells + 32 * rh + 2 * g;
    const int tile = tile_offset(32 * rh + 2 * g, kw, t);
    const int sc0 = (kw >> p.gsh) * 128 + 64 * rh + 4 * g, sc1 = ((kw + 4) >> p.gsh) * 128 + 64 * rh + 4 * g;
    Cursor at;
    // `chunks` steps of unit u from chunk ch on, with N token tiles.
    auto products = [&](auto tiles, int u, int ch, int chunks) {
      constexpr int N = decltype(tiles)::value;
      const int start = L.unit_start[u], n = L.unit_n[u];
      int bq[N], bs[N];
#pragma unroll
      for (int tt = 0; tt < N; ++tt) {
        // the lane's column of B is hi or lo of token g / 2; the scales are those of token t
        bq[tt] = min(4 * tt + (g >> 1), n - 1) * C::kRow + (kw >> 1) * kRecord + (kw & 1) * 256 + (g & 1) * 64 + t * 16;
        bs[tt] = min(4 * tt + t, n - 1) * C::kRow + (kw >> 1) * kRecord + 512 + (kw & 1) * 16;
      }
      float2 tot[2][N];
#pragma unroll
      for (int tt = 0; tt < N; ++tt) tot[0][tt] = tot[1][tt] = make_float2(0.0f, 0.0f);
      for (; chunks > 0; ch += stride, --chunks, at.next(stages)) {
        const uint8_t* st = ring + at.stage * C::kStage;
        const uint8_t* rec = st + C::kW + 2 * C::kS;
        ring_await(R, at);
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
          if (C::kSubs * ch + kw + 4 * i >= nsub) break;
          const uint8_t* row0 = st + tile + i * 64 * 128;
          const uint8_t* row1 = st + 128 + (tile ^ 16) + i * 64 * 128;
          const uint8_t* sp = st + C::kW + (i == 0 ? sc0 : sc1);
          uint32_t a[2][4][4];
          float2 sc[2], z[2];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            load_tile<__half>(row0 + m * 16 * 128, row1 + m * 16 * 128, magic, a[m]);
            sc[m] = load_pair<T>(sp + 32 * m), z[m] = load_pair<T>(sp + 32 * m + C::kS);
          }
#pragma unroll
          for (int tt = 0; tt < N; ++tt) {
            const uint8_t* bp = rec + bq[tt] + i * 2 * kRecord;
            const uint4 b0 = *reinterpret_cast<const uint4*>(bp), b1 = *reinterpret_cast<const uint4*>(bp + 128);
            const float4 dx = *reinterpret_cast<const float4*>(rec + bs[tt] + i * 2 * kRecord);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              float c[4];
              multiply<__half>(c, a[m], b0, b1);
              const float2 v = __fmul2_rn(make_float2(dx.x, dx.y), make_float2(c[0] + c[1], c[2] + c[3]));
              tot[m][tt] = __ffma2_rn(sc[m], v, tot[m][tt]);
              tot[m][tt] = __ffma2_rn(z[m], make_float2(dx.z, dx.w), tot[m][tt]);
            }
          }
        }
        ring_release(R, at);
      }
#pragma unroll
      for (int tt = 0; tt < N; ++tt) {
        const int i = 4 * tt + t;                   // the lane's token
        if (i < n) {
          float2* ap = reinterpret_cast<float2*>(acc + L.slot_token[start + i] * kRowsTile);
          const float2 v = ap[0], w = ap[8];
          ap[0] = make_float2(v.x + tot[0][tt].x, v.y + tot[0][tt].y);
          ap[8] = make_float2(w.x + tot[1][tt].x, w.y + tot[1][tt].y);
        }
      }
      __syncwarp();                                 // another lane may hold this token in the next unit
    };
    for (int u = u0, ch = ch0; left > 0; ++u, ch = again) {
      const int chunks = min((nchunk - ch + stride - 1) / stride, left);
      const int n = L.unit_n[u];
      if (NT == 1 || n <= 4) products(std::integral_constant<int, 1>(), u, ch, chunks);
      else if (NT == 2 || n <= 8) products(std::integral_constant<int, NT < 2 ? 1 : 2>(), u, ch, chunks);
      else if (n <= 12) products(std::integral_constant<int, NT < 3 ? 1 : 3>(), u, ch, chunks);
      else products(std::integral_constant<int, NT>(), u, ch, chunks);
      left -= chunks;
    }
  }
  __syncthreads();
  for (int i = tid; i < cells; i += C::kThreads) {
    float v = sums[i];
#pragma unroll
    for (int w = 1; w < 4; ++w) v += sums[w * cells + i];
    sums[i] = v;
  }
  cluster_sync();
  const uint32_t base = smem_u32(sums);
  for (int i = rank * C::kThreads + tid; i < cells; i += ranks * C::kThreads) {
    float part[8], v = 0.0f;                        // all loads before the first sum
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r) part[r] = r < ranks ? ld_cluster_f32(mapa_shared(base + 4 * i, r)) : 0.0f;
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r) v += part[r];
    reinterpret_cast<T*>(p.out)[(int64_t)(i / kRowsTile) * p.K + n0 + i % kRowsTile] = awq::Traits<T>::fromf(v);
  }
  cluster_sync();                                   // no CTA leaves while another reads its sums
}

}  // namespace moe
}  // namespace ck
