// Low-rank adapters of many requests beside a projection that all of them share.
//
//   out[m, :] = y[m, :] + scale[a] * ((x[m, :] A[a]^T) B[a]^T),   a = ids[m]
//   out[m, :] = y[m, :]                                           where a is no adapter
//
// A tile is at most 16 tokens of one adapter. A cluster of CTAs computes it in
// one launch: each CTA multiplies its share of K (v = x A^T, the "shrink"), the
// partial v are added through distributed shared memory in rank order, and
// each CTA then multiplies all of v with its share of B's N rows and adds y (the
// "expand"). v never goes to global memory. Both products are bound by bytes: x,
// y and out once for each token, an adapter once for each of its tiles.
//
// Products are mma.sync.m16n8k16 with the tokens as the 16 rows of A. Their
// operands come straight from global memory: a lane's 16 bytes are eight
// consecutive k of one row, which serve as the k pairs of two MMAs (a sum over
// k does not depend on how k is numbered). The columns of the expand's four
// neighbouring MMAs are numbered so that a lane's results are eight consecutive
// n of y: 16-byte loads and stores.
//
// v, a sum in 32 bits, enters the expand as a sum of numbers of the inputs' 16-bit type, each
// the rounding of what those before it leave (B's type is also the operand's). Three bf16 numbers hold all
// 24 bits of v (two lose up to 2^-18 of it, which shows where ranks cancel); two fp16 numbers hold
// it to 2^-23. For fp16 each row of v is first scaled by a power of two, which brings its
// largest entry to [2^13, 2^14): v itself may lie outside fp16's range.
//
// A token's arithmetic does not depend on which tile it is in or which tokens
// share that tile, so the order in which a batch is grouped does not show.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ck_common.cuh"
#include "cluster_mem.cuh"
#include "gemv_awq.cuh"

namespace ck {
namespace lora {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSelfGroup = 256;        // up to this many tokens a cluster of few tokens finds its tile itself,
constexpr int kSelfPick = 4096;        // or this many of at most kPickAdapters adapters (pick_tile)
constexpr int kMaxAdapters = 8192;     // group_kernel counts them in shared memory
constexpr int kGroupThreads = 1024;

struct Params {
  const void *x, *y, *a, *b;           // (M, K) T, (M, N) TY, (L, R, K) T, (L, N, R) T
  const int32_t* ids;                  // (M)
  const float* scales;                 // (L) or null
  void* out;                           // (M, N) TY
  int64_t ldx, ldy, ldo;
  int M, K, N, R, L;
  int vec;                             // y and out take 16-byte accesses
  const int32_t* tiles;                // group_kernel's {adapter, start, count, 0} per tile, or null
  const int32_t* order;                // its tokens in tile order
};

// Tiles of M tokens are at most this many, whatever the ids: full tiles, and one more for each
// adapter (and for the tokens without one).
__host__ __device__ inline int64_t max_tiles(int64_t M, int64_t L, int tm) {
  const int64_t n = M / tm + L + 1;
  return n < M ? n : M;
}

// Sorts the tokens of a large batch by adapter: tile list and token order, by one CTA. Bucket L
// holds the tokens without an adapter. A thread takes eight consecutive tokens at a time, read
// before any is counted (one at a time the two passes over 8192 ids took 7.6 us): prompts are
// runs of one id, so a warp mostly counts 256 tokens with one atomic.
constexpr int kGroupEach = 8;

// The buckets of tokens i0 .. i0 + E - 1; -1 past the last.
template <int E>
__device__ __forceinline__ void load_buckets(const int32_t* ids, int64_t i0, int M, int L, int (&a)[E]) {
  const bool wide = (reinterpret_cast<uintptr_t>(ids) & 15) == 0 && i0 + E <= M;
#pragma unroll
  for (int j = 0; j < E; j += 4) {
    if (wide) {
      const int4 v = *reinterpret_cast<const int4*>(ids + i0 + j);
      a[j] = v.x, a[j + 1] = v.y, a[j + 2] = v.z, a[j + 3] = v.w;
    } else {
#pragma unroll
      for (int i = j; i < j + 4; ++i) a[i] = i0 + i < M ? ids[i0 + i] : 0;
    }
  }
#pragma unroll
  for (int j = 0; j < E; ++j) a[j] = i0 + j >= M ? -1 : a[j] >= 0 && a[j] < L ? a[j] : L;
}

// The bucket that all tokens of a warp are in, or -1.
template <int E>
__device__ __forceinline__ int common_bucket(const int (&a)[E]) {
  const int a0 = __shfl_sync(0xffffffffu, a[0], 0);  // (not in a condition that only some lanes evaluate)
  bool one = a0 >= 0;
#pragma unroll
  for (int j = 0; j < E; ++j) one = one && a[j] == a0;
  return __all_sync(0xffffffffu, one) ? a0 : -1;
}

// Counts a warp's tokens: one atomic where they are of one bucket, else one for each run of a thread.
template <int E>
__device__ __forceinline__ void count_tokens(int* count, const int (&a)[E]) {
  const int all = common_bucket(a);
  if (all >= 0) {
    if ((threadIdx.x & 31) == 0) atomicAdd(&count[all], 32 * E);
    return;
  }
  int run = 1;
#pragma unroll
  for (int j = 1; j <= E; ++j) {
    if (j < E && a[j] == a[j - 1]) {
      ++run;
    } else {
      if (a[j - 1] >= 0) atomicAdd(&count[a[j - 1]], run);
      run = 1;
    }
  }
}

__global__ void __launch_bounds__(kGroupThreads) group_kernel(const int32_t* __restrict__ ids, int M, int L, int tm,
                                                              int max_tiles, int32_t* __restrict__ tiles,
                                                              int32_t* __restrict__ order) {
  extern __shared__ int32_t count[];                 // L + 1 counters, then each bucket's cursor
  __shared__ int warp_sum[2][kGroupThreads / 32];
  __shared__ int carry[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kRound = kGroupThreads * kGroupEach;
  const int rounds = (M + kRound - 1) / kRound;
  for (int i = tid; i <= L; i += kGroupThreads) count[i] = 0;
  if (tid == 0) carry[0] = carry[1] = 0;
  grid_dep_wait();
  grid_dep_launch();
  int a[kGroupEach];
  load_buckets(ids, kGroupEach * tid, M, L, a);
  __syncthreads();
  for (int r = 0; r < rounds; ++r) {
    if (r > 0) load_buckets(ids, (int64_t)kRound * r + kGroupEach * tid, M, L, a);
    count_tokens(count, a);
  }
  __syncthreads();
  for (int b0 = 0; b0 <= L; b0 += kGroupThreads) {   // running sums of tokens and of tiles
    const int b = b0 + tid;
    const int n = b <= L ? count[b] : 0, nt = (n + tm - 1) / tm;
    int in = n, it = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int un = __shfl_up_sync(0xffffffffu, in, o), ut = __shfl_up_sync(0xffffffffu, it, o);
      if (lane >= o) in += un, it += ut;
    }
    if (lane == 31) warp_sum[0][warp] = in, warp_sum[1][warp] = it;
    __syncthreads();
    int bn = carry[0], bt = carry[1];
    if (b0 + 32 * warp <= L)                         // warps without a bucket need no sums
      for (int w = 0; w < warp; ++w) bn += warp_sum[0][w], bt += warp_sum[1][w];
    const int start = bn + in - n;
    int tile = bt + it - nt;
    if (b <= L) {
      count[b] = start;
      for (int s = 0; s < n; s += tm, ++tile)
        reinterpret_cast<int4*>(tiles)[tile] = make_int4(b < L ? b : -1, start + s, min(tm, n - s), 0);
    }
    __syncthreads();
    if (b == min(L, b0 + kGroupThreads - 1)) carry[0] = bn + in, carry[1] = bt + it;
    __syncthreads();
  }
  for (int i = carry[1] + tid; i < max_tiles; i += kGroupThreads)   // tiles that this batch has not
    reinterpret_cast<int4*>(tiles)[i] = make_int4(-1, 0, 0, 0);
  for (int r = 0; r < rounds; ++r) {
    const int64_t i0 = (int64_t)kRound * r + kGroupEach * tid;
    if (rounds > 1) load_buckets(ids, i0, M, L, a);
    const int all = common_bucket(a);
    int base = 0;
    if (all >= 0 && lane == 0) base = atomicAdd(&count[all], 32 * kGroupEach);
    base = __shfl_sync(0xffffffffu, base, 0) + kGroupEach * lane;
#pragma unroll
    for (int j = 0; j < kGroupEach; ++j)
      if (a[j] >= 0) order[all >= 0 ? base + j : atomicAdd(&count[a[j]], 1)] = (int)i0 + j;
  }
}

// Tile number `tile` of a batch in one CTA: its adapter (-1: none), its tokens in ascending
// order and their number (0: there is no such tile). Tiles are numbered by adapter, the tokens
// without one last. The counts do not depend on the order of the atomics, and only the
// bucket that holds the tile is ranked, so all CTAs of a cluster find the same. `scratch`
// (kPickBytes) must be zero, before a barrier; token[] may be read after the next one. Reading all
// ids in every CTA costs less than a launch of group_kernel before it (5 us at M = 8192).
constexpr int kPickTokens = 32768;     // at most; larger batches use group_kernel
constexpr int kPickAdapters = kPickTokens / 32;
constexpr int kPickBytes = (kPickAdapters + 1 + 32) * 4;
template <int THREADS, int TM>
__device__ __forceinline__ void pick_tile(const Params& p, int tile, int* token, int& adapter, int& n, int* scratch) {
  constexpr int E = 16;                              // ids a thread and round
  constexpr int kRound = THREADS * E, warps = THREADS / 32;
  static_assert(warps <= 32, "a warp sums the warps");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* sums = scratch;                               // [32]
  int* count = scratch + 32;                         // [L + 1]
  int a[E];
  const int rounds = (p.M + kRound - 1) / kRound;
  for (int r = 0; r < rounds; ++r) {
    load_buckets(p.ids, kRound * r + E * tid, p.M, p.L, a);
    if (__any_sync(0xffffffffu, a[0] >= 0)) count_tokens(count, a);
  }
  __syncthreads();
  // every warp for itself: the bucket that holds the tile
  int bucket = -1, first = 0, before = 0;
  for (int b0 = 0; b0 <= p.L && bucket < 0; b0 += 32) {
    const int c = b0 + lane <= p.L ? count[b0 + lane] : 0, nt = (c + TM - 1) / TM;
    int it = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, it, o);
      if (lane >= o) it += u;
    }
    const int last = before + it;
    const unsigned here = __ballot_sync(0xffffffffu, tile >= last - nt && tile < last);
    if (here != 0) {
      const int l = __ffs(here) - 1;
      bucket = b0 + l;
      first = (tile - __shfl_sync(0xffffffffu, last - nt, l)) * TM;   // rank of the tile's first token
      n = min(TM, __shfl_sync(0xffffffffu, c, l) - first);
    }
    before = __shfl_sync(0xffffffffu, last, 31);
  }
  adapter = bucket < p.L ? bucket : -1;
  if (bucket < 0) {
    n = 0;
    return;
  }
  int rank0 = 0;                                     // tokens of the bucket in earlier rounds
  for (int r = 0; r < rounds; ++r) {
    const int i0 = kRound * r + E * tid;
    if (rounds > 1) load_buckets(p.ids, i0, p.M, p.L, a);
    int c = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) c += a[j] == bucket;
    int in = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += u;
    }
    if (r > 0) __syncthreads();                      // sums has been read
    if (lane == 31) sums[warp] = in;
    __syncthreads();
    const int w = lane < warps ? sums[lane] : 0;
    int at0 = rank0 + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + in - c - first;
    if (at0 < TM && at0 + c > 0) {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (a[j] == bucket) {
          if (at0 >= 0 && at0 < TM) token[at0] = i0 + j;
          ++at0;
        }
    }
    rank0 += __reduce_add_sync(0xffffffffu, w);
  }
}

// This cluster's tile: adapter (-1: none) and tokens; returns their number (0: no such tile).
template <int TM>
__device__ __forceinline__ int find_tile(const Params& p, int tile, int (&token)[TM], int& adapter, int* scratch) {
  const int tid = threadIdx.x;
  if (p.tiles != nullptr) {
    const int4 v = __ldcg(reinterpret_cast<const int4*>(p.tiles) + tile);
    if (tid < v.z) token[tid] = __ldcg(p.order + v.y + tid);
    adapter = v.x;
    __syncthreads();
    return v.z;
  }
  if (p.M > kSelfGroup) {                             // (pick_tile from 64 tokens on: 1 us slower at 128)
    int n = 0;
    for (int i = tid; i < p.L + 1 + 32; i += kThreads) scratch[i] = 0;
    __syncthreads();
    pick_tile<kThreads, TM>(p, tile, token, adapter, n, scratch);
    __syncthreads();
    return n;
  }
  // M <= 256 = kThreads: token i's rank among the tokens of its adapter; every TM-th begins a
  // tile, and tiles are numbered by their first tokens.
  int* id = scratch;                                  // [kSelfGroup]
  int* found = scratch + kSelfGroup;                  // adapter, rank of the tile's first token, count
  int a = -2;
  if (tid < p.M) {
    a = p.ids[tid];
    if (a < 0 || a >= p.L) a = -1;
  }
  id[tid] = a;
  if (tid == 0) found[0] = -1, found[1] = 0, found[2] = 0;
  __syncthreads();
  int rank = 0;
  if (tid < p.M)
    for (int j = 0; j < tid; ++j) rank += id[j] == a;
  const bool first = tid < p.M && rank % TM == 0;
  const int before = __popc(__ballot_sync(0xffffffffu, first) & ((1u << (tid & 31)) - 1));
  int* warp_n = found + 4;
  if ((tid & 31) == 31) warp_n[tid >> 5] = before + (first ? 1 : 0);
  __syncthreads();
  int number = before;
  for (int w = 0; w < (tid >> 5); ++w) number += warp_n[w];
  if (first && number == tile) found[0] = a, found[1] = rank, found[2] = 1;
  __syncthreads();
  const bool any = found[2] != 0;
  const int fa = found[0], fr = found[1];
  const bool mine = any && tid < p.M && a == fa && rank >= fr && rank < fr + TM;
  if (mine) token[rank - fr] = tid;
  adapter = fa;
  return __syncthreads_count(mine);
}

static_assert(kSelfGroup + 16 <= kPickBytes / 4, "find_tile's scratch");

// How v enters the expand: as kPlanes numbers of type T, with or without a power of two for each row.
template <typename T> struct VOperand;
template <> struct VOperand<__nv_bfloat16> {
  static constexpr int kPlanes = 3;
  static constexpr bool kScaled = false;
};
template <> struct VOperand<__half> {
  static constexpr int kPlanes = 2;
  static constexpr bool kScaled = true;
};

// The power of two that brings a row's largest magnitude (its bits) to [2^13, 2^14); 0 where it is zero,
// subnormal or not finite.
__device__ __forceinline__ int scale_exponent(uint32_t top) {
  const int e = (int)(top >> 23);
  return e > 0 && e < 255 ? max(-100, min(100, 13 - (e - 127))) : 0;
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// v as a sum of P numbers, the largest first; an infinity stays one.
template <typename T, int P>
__device__ __forceinline__ void split(float v, T (&part)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    part[i] = awq::Traits<T>::fromf(v);
    const float f = awq::Traits<T>::tof(part[i]);
    v = isfinite(f) ? v - f : 0.0f;
  }
}

// Columns [c0, c1) of y's rows token[0 .. n) into out (nothing where out is y): a row a warp, eight
// pieces a lane in flight (c0 % 8 == 0 and c1 % 8 == 0 where p.vec).
template <typename TY>
__device__ __forceinline__ void copy_rows(const TY* y, TY* out, const Params& p, const int* token, int n, int c0, int c1,
                                          int warp, int warps) {
  if (y == out) return;
  const int lane = threadIdx.x & 31, per = p.vec ? (c1 - c0) / 8 : c1 - c0;   // pieces a row
  for (int m = warp; m < n; m += warps) {
    const TY* from = y + token[m] * p.ldy + c0;
    TY* to = out + token[m] * p.ldo + c0;
    for (int k = lane; k < per; k += 256) {
      uint4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k + 32 * j < per) {
          if (p.vec) v[j] = reinterpret_cast<const uint4*>(from)[k + 32 * j];
          else v[j].x = reinterpret_cast<const uint16_t*>(from)[k + 32 * j];
        }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k + 32 * j < per) {
          if (p.vec) reinterpret_cast<uint4*>(to)[k + 32 * j] = v[j];
          else reinterpret_cast<uint16_t*>(to)[k + 32 * j] = (uint16_t)v[j].x;
        }
    }
  }
}

// Shared memory of a CTA: RC 32-wide chunks of rank, v as P numbers.
constexpr int kFewTile = 16;                          // tokens of a tile
template <int RC, int P>
struct alignas(16) Smem {
  static constexpr int kR = 32 * RC;
  static constexpr int kVStride = kR + 8;             // 16-bit elements: rows 16 bytes apart in the banks
  float part[kWarps][kFewTile][kR];                         // the warps' sums; [0]: this CTA's
  float v[kFewTile][kR];                                    // the cluster's
  uint16_t planes[P][kFewTile][kVStride];                   // v as the expand's operand
  float row_scale[kFewTile];
  int token[kFewTile];
  int scratch[kPickBytes / 4];
};

// Many small CTAs hide each other's latencies (ranks up to 32: three an SM, else two; 64 tokens with adapters of
// rank 128, K = N = 4096: 28.8 us; with v as two numbers 27.4, and 32.5 with one CTA). Latency bounds them: several loads of a step are
// issued before its first product, those of y before those of B (a decode step of 64 tokens, K = 4096,
// N = 12288, R = 32, 48 adapters 18.1 us, 16.5 with v as two bf16 numbers; with those 20.0 with a load for each
// product; its bytes take 6.3 at the measured copy bandwidth). Bringing B into shared memory from the start took the place
// of CTAs on the SMs: 29 us for that decode step.
template <typename T, typename TY, int RC>
__global__ void __launch_bounds__(kThreads, RC == 1 ? 3 : 2) lora_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t sm[];
  constexpr int P = VOperand<T>::kPlanes;
  using SM = Smem<RC, P>;
  using Tr = awq::Traits<T>;
  SM& S = *reinterpret_cast<SM*>(sm);
  constexpr int RT = 4 * RC;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
  grid_dep_wait();
  grid_dep_launch();
  int adapter;
  const int n = find_tile<kFewTile>(p, (int)(blockIdx.x / ranks), S.token, adapter, S.scratch);
  if (n == 0) return;                                 // the same for all CTAs of the cluster
  const T* x = reinterpret_cast<const T*>(p.x);
  const TY* y = reinterpret_cast<const TY*>(p.y);
  TY* out = reinterpret_cast<TY*>(p.out);
  const int nb = (p.N + 31) / 32;                     // blocks of 32 columns
  const int nb0 = (int)((int64_t)nb * rank / ranks), nb1 = (int)((int64_t)nb * (rank + 1) / ranks);

  if (adapter < 0) {                                  // tokens without an adapter
    copy_rows(y, out, p, S.token, n, 32 * nb0, min(32 * nb1, p.N), warp, kWarps);
    return;
  }
  const T* b = reinterpret_cast<const T*>(p.b) + ((int64_t)adapter * p.N + 32 * nb0) * p.R;   // this CTA's share

  // ---- shrink: part = x A^T over this warp's share of k
  {
    const int nk = (p.K + 31) / 32;
    const int kc0 = (int)((int64_t)nk * (rank * kWarps + warp) / (ranks * kWarps));
    const int kc1 = (int)((int64_t)nk * (rank * kWarps + warp + 1) / (ranks * kWarps));
    const T* x0 = g < n ? x + S.token[g] * p.ldx + 8 * t : nullptr;
    const T* x1 = g + 8 < n ? x + S.token[g + 8] * p.ldx + 8 * t : nullptr;
    const T* ap = reinterpret_cast<const T*>(p.a) + ((int64_t)adapter * p.R + g) * p.K + 8 * t;
    float c[RT][4] = {};
    constexpr int kBatch = RC == 2 ? 8 : 4;           // loads of A at once (RC = 4: 8 leave registers for one CTA an SM)
#pragma unroll 1
    for (int kc = kc0; kc < kc1; ++kc) {
      const int k = 32 * kc;
      const bool in = k + 8 * t < p.K;                // K % 8 == 0: all eight or none
      uint4 q0 = make_uint4(0, 0, 0, 0), q1 = q0;
      if (in && x0 != nullptr) q0 = *reinterpret_cast<const uint4*>(x0 + k);
      if (in && x1 != nullptr) q1 = *reinterpret_cast<const uint4*>(x1 + k);
      const uint32_t fa[4] = {q0.x, q1.x, q0.y, q1.y}, fb[4] = {q0.z, q1.z, q0.w, q1.w};
#pragma unroll
      for (int j0 = 0; j0 < RT; j0 += kBatch) {
        if (8 * j0 >= p.R) break;
        uint4 w[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          w[j] = make_uint4(0, 0, 0, 0);
          if (in && 8 * (j0 + j) < p.R)
            w[j] = __ldg(reinterpret_cast<const uint4*>(ap + (int64_t)8 * (j0 + j) * p.K + k));
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          Tr::mma(c[j0 + j], fa, w[j].x, w[j].y);
          Tr::mma(c[j0 + j], fb, w[j].z, w[j].w);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      *reinterpret_cast<float2*>(&S.part[warp][g][8 * j + 2 * t]) = make_float2(c[j][0], c[j][1]);
      *reinterpret_cast<float2*>(&S.part[warp][g + 8][8 * j + 2 * t]) = make_float2(c[j][2], c[j][3]);
    }
  }
  __syncthreads();
  constexpr int kCells = kFewTile * SM::kR / 4;             // of four floats
  const int cells = n * SM::kR / 4;                         // of this tile's tokens: other rows of v are not used
  float4* part = reinterpret_cast<float4*>(&S.part[0][0][0]);
  for (int i = tid; i < cells; i += kThreads) {
    float4 s = part[i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 u = part[w * kCells + i];
      s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
    }
    part[i] = s;
  }
  // each CTA adds its share of the cells over the ranks and hands the sums to all
  cluster_sync();
  const uint32_t part_at = smem_u32(part), v_at = smem_u32(&S.v[0][0]);
  for (int i = tid * ranks + rank; i < cells; i += ranks * kThreads) {
    float4 u[8], s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (r < ranks) u[r] = ld_cluster_f32x4(mapa_shared(part_at + 16 * i, r));
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (r < ranks) s.x += u[r].x, s.y += u[r].y, s.z += u[r].z, s.w += u[r].w;
    for (int r = 0; r < ranks; ++r) st_cluster_f32x4(mapa_shared(v_at + 16 * i, r), s);
  }
  cluster_sync();

  // ---- v as the expand's operand; zeros past the rank (where an infinity in x has made NaN of A's zeros)
  const float as = p.scales != nullptr ? __ldg(p.scales + adapter) : 1.0f;
  for (int m = warp; m < n; m += kWarps) {
    float v[RC];
    int ex = 0;
#pragma unroll
    for (int i = 0; i < RC; ++i) v[i] = 32 * i + lane < p.R ? S.v[m][32 * i + lane] : 0.0f;
    if constexpr (VOperand<T>::kScaled) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < RC; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
      ex = scale_exponent(__reduce_max_sync(0xffffffffu, top));
    }
    const float up = exp2_int(ex);
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      T part[P];
      split(v[i] * up, part);
#pragma unroll
      for (int k = 0; k < P; ++k) S.planes[k][m][32 * i + lane] = *reinterpret_cast<const uint16_t*>(&part[k]);
    }
    if (lane == 0) S.row_scale[m] = as * exp2_int(-ex);
  }
  __syncthreads();

  // ---- expand: out = y + row_scale * (v B^T), 32 columns at a time
  using TrY = awq::Traits<TY>;
  for (int blk = warp; blk < nb1 - nb0; blk += kWarps) {
    const int c0 = 32 * (nb0 + blk), col = c0 + 8 * t;   // the lane's eight columns: col ..
    float c[4][4] = {};
    uint4 yq[2] = {};
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
      if (p.vec && col < p.N && g + 8 * hf < n)
        yq[hf] = *reinterpret_cast<const uint4*>(y + S.token[g + 8 * hf] * p.ldy + col);
    constexpr int kBatch = RC < 2 ? RC : 2;
#pragma unroll
    for (int r0 = 0; r0 < RC; r0 += kBatch) {
      if (32 * r0 >= p.R) break;
      uint4 w[kBatch][4];
#pragma unroll
      for (int rc = 0; rc < kBatch; ++rc)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 32 * blk + 8 * (g >> 1) + 2 * j + (g & 1);      // of this CTA's share
          const int at = 32 * (r0 + rc) + 8 * t;
          w[rc][j] = make_uint4(0, 0, 0, 0);
          if (32 * nb0 + row < p.N && at < p.R)
            w[rc][j] = __ldg(reinterpret_cast<const uint4*>(b + (int64_t)row * p.R + at));
        }
#pragma unroll
      for (int rc = 0; rc < kBatch; ++rc) {
        if (32 * (r0 + rc) >= p.R) break;
        const int at = 32 * (r0 + rc) + 8 * t;
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const uint4 v0 = *reinterpret_cast<const uint4*>(&S.planes[k][g][at]);
          const uint4 v1 = *reinterpret_cast<const uint4*>(&S.planes[k][g + 8][at]);
          const uint32_t fa[4] = {v0.x, v1.x, v0.y, v1.y}, fb[4] = {v0.z, v1.z, v0.w, v1.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            Tr::mma(c[j], fa, w[rc][j].x, w[rc][j].y);
            Tr::mma(c[j], fb, w[rc][j].z, w[rc][j].w);
          }
        }
      }
    }
    if (col >= p.N) continue;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int m = g + 8 * hf;
      if (m >= n) continue;
      const float f = S.row_scale[m];
      const TY* yp = y + S.token[m] * p.ldy + col;
      TY* op = out + S.token[m] * p.ldo + col;
      if (p.vec) {
        uint4 u = yq[hf];
        TY* e = reinterpret_cast<TY*>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = TrY::fromf(fmaf(f, c[i >> 1][2 * hf + (i & 1)], TrY::tof(e[i])));
        *reinterpret_cast<uint4*>(op) = u;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < p.N) op[i] = TrY::fromf(fmaf(f, c[i >> 1][2 * hf + (i & 1)], TrY::tof(yp[i])));
      }
    }
  }
}

}  // namespace lora
}  // namespace ck
