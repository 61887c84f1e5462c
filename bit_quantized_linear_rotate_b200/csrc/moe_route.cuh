// Expert routing: the k largest of each token's logits, their softmax weights,
// and, inside one CTA, the lists of tokens that each expert gets.
//
//   chosen_t = the k live entries of l[t, :] that come first in (value
//              descending, index ascending); live means l > -inf (a NaN is not)
//   w[t, j]  = exp(l[t, c_j] - m_t) / S_t,  m_t = max_e l[t, e],
//              S_t = the sum of those exponentials over the chosen entries
//              (renormalised) or over all live ones
//
// A slot without a live entry gets the id -1 and the weight 0. Where m_t is
// +inf the limit is taken: the +inf entries share the weight equally.
//
// One warp handles one token. Every logit becomes an unsigned key that sorts as
// the value does (0 for entries that are not live), so a round of the choice
// is one redux.max over the keys and one redux.min over the indices of those
// that hold it: ties go to the lowest index, and no value is rounded.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ck_common.cuh"

namespace ck {
namespace moe {

constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 16;
constexpr int kMaxTokens = 64;                       // of the experts' kernels; ck_moe_route takes any number
constexpr int kMaxSlots = kMaxTokens * kMaxTopK;
constexpr int kLogitBf16 = 0, kLogitFp16 = 1, kLogitFp32 = 2;   // = ck_dtype

// Read past L1: a dependent kernel may read the logits before its own
// dependency wait (down_kernel), when this SM's L1 need not hold them yet.
__device__ __forceinline__ float load_logit(const void* p, int dt, int64_t i) {
  if (dt == kLogitFp32) return __ldcg(reinterpret_cast<const float*>(p) + i);
  const unsigned short u = __ldcg(reinterpret_cast<const unsigned short*>(p) + i);
  if (dt == kLogitBf16) return __uint_as_float((uint32_t)u << 16);
  return __half2float(__ushort_as_half(u));
}

// Unsigned key in the order of the values; 0 for an entry that is not live.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);      // -0 counts as +0
  const uint32_t key = (u >> 31) ? ~u : (u | 0x80000000u);
  return v > -INFINITY ? key : 0u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key >> 31) ? (key & 0x7fffffffu) : ~key);
}

// exp(v - m) with the limit at m = +inf.
__device__ __forceinline__ float exp_below(float v, float m) { return v == m ? 1.0f : expf(v - m); }

// The choice for one token by one warp, V logits a lane (E <= 32 V; lane l
// holds the entries l, l + 32, ...). Lane j < k returns slot j's id and weight.
template <int V>
__device__ __forceinline__ void choose(const void* logits, int ldt, int64_t row, int E, int k, bool renorm, int& id,
                                       float& w) {
  const int lane = threadIdx.x & 31;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < E ? order_key(load_logit(logits, ldt, row * E + e)) : 0u;
  }
  uint32_t all[V];
#pragma unroll
  for (int i = 0; i < V; ++i) all[i] = key[i];
  int my_id = -1;
  uint32_t my_key = 0u, top = 0u;
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = max(best, key[i]);
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    if (m == 0u) break;                              // no live entry is left
    uint32_t at = 0xffffffffu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] == m) at = (uint32_t)(lane + 32 * i);
    at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((uint32_t)(lane + 32 * i) == at) key[i] = 0u;
    if (j == 0) top = m;
    if (lane == j) {
      my_id = (int)at;
      my_key = m;
    }
  }
  const float mv = key_value(top);
  const float p = my_id >= 0 ? exp_below(key_value(my_key), mv) : 0.0f;
  float s = 0.0f;
  if (renorm) {
    s = p;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (all[i] != 0u) s += exp_below(key_value(all[i]), mv);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  id = my_id;
  w = my_id >= 0 ? p / s : 0.0f;
}

__device__ __forceinline__ void choose_any(const void* logits, int ldt, int64_t row, int E, int k, bool renorm,
                                           int& id, float& w) {
  if (E <= 128) choose<4>(logits, ldt, row, E, k, renorm, id, w);
  else choose<16>(logits, ldt, row, E, k, renorm, id, w);
}

constexpr int kRouteWarps = 4;

// One warp per token.
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_kernel(const void* logits, int ldt, int64_t T, int E, int k, int renorm, float* __restrict__ weights,
                 int32_t* __restrict__ ids) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  int id;
  float w;
  choose_any(logits, ldt, t, E, k, renorm != 0, id, w);
  const int lane = threadIdx.x & 31;
  if (lane < k) {
    weights[t * k + lane] = w;
    ids[t * k + lane] = id;
  }
}

// Where a layer's choice comes from: logits (ids == nullptr), or given ids and
// weights of shape (T, k).
struct Choice {
  const void* logits;
  const int32_t* ids;
  const float* weights;
  int ldt, T, E, k, renorm;
};

// The experts' token lists of a batch of at most kMaxTokens tokens, in shared
// memory. The slots that some token fills are numbered by (expert, token); a
// unit is at most `cap` consecutive slots of one expert.
struct Lists {
  float* slot_w;
  uint16_t *unit_expert, *unit_start;
  uint8_t *unit_n, *slot_token;
  int* scratch;                                      // [32], then the number of units
  __device__ __forceinline__ int units() const { return scratch[32]; }
};
__host__ __device__ constexpr int lists_bytes(int slots) { return (144 + slots * 10 + 15) / 16 * 16; }
__device__ __forceinline__ Lists lists_at(uint8_t* p, int slots) {
  Lists L;
  L.scratch = reinterpret_cast<int*>(p);
  L.slot_w = reinterpret_cast<float*>(p + 144);
  L.unit_expert = reinterpret_cast<uint16_t*>(L.slot_w + slots);
  L.unit_start = L.unit_expert + slots;
  L.unit_n = reinterpret_cast<uint8_t*>(L.unit_start + slots);
  L.slot_token = L.unit_n + slots;
  return L;
}
// What only the building of the lists needs; its memory may be used again afterwards.
struct ListsTemp {
  unsigned long long mask[kMaxExperts];              // tokens of each expert
  float w[kMaxSlots];                                // the choice as given
  int16_t id[kMaxSlots];
  uint16_t start[kMaxExperts];                       // the experts' first slots
};

// Fills L from the choice, by all THREADS threads of the CTA, closing with a
// barrier. An expert that a token names twice gets it once, with the sum of
// the two weights. Units are in the order of the experts.
template <int THREADS>
__device__ __forceinline__ void build_lists(const Choice& c, const Lists& L, ListsTemp& tmp, int cap) {
  constexpr int PER = (kMaxExperts + THREADS - 1) / THREADS;      // experts a thread
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < c.E; e += THREADS) tmp.mask[e] = 0ull;
  const int slots = c.T * c.k;
  if (c.ids == nullptr) {
    for (int t = warp; t < c.T; t += THREADS / 32) {
      int id;
      float w;
      choose_any(c.logits, c.ldt, t, c.E, c.k, c.renorm != 0, id, w);
      if (lane < c.k) {
        tmp.id[t * c.k + lane] = (int16_t)id;
        tmp.w[t * c.k + lane] = w;
      }
    }
  } else {
    for (int s = tid; s < slots; s += THREADS) {
      const int id = __ldcg(c.ids + s);
      tmp.id[s] = (int16_t)(id >= 0 && id < c.E ? id : -1);
      tmp.w[s] = __ldcg(c.weights + s);
    }
  }
  __syncthreads();
  for (int s = tid; s < slots; s += THREADS)
    if (tmp.id[s] >= 0) atomicOr(&tmp.mask[tmp.id[s]], 1ull << (s / c.k));
  __syncthreads();
  int n[PER], v = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = PER * tid + i;
    n[i] = e < c.E ? __popcll(tmp.mask[e]) : 0;
    v += ((n[i] + cap - 1) / cap) << 16 | n[i];      // units and slots in one word: both at most kMaxSlots
  }
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) L.scratch[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < warp; ++i) before += L.scratch[i];
  int unit = (before + incl - v) >> 16, slot = (before + incl - v) & 0xffff;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (n[i] == 0) continue;
    const int e = PER * tid + i;
    for (int s = 0; s < n[i]; s += cap, ++unit) {
      L.unit_expert[unit] = (uint16_t)e;
      L.unit_start[unit] = (uint16_t)(slot + s);
      L.unit_n[unit] = (uint8_t)min(cap, n[i] - s);
    }
    tmp.start[e] = (uint16_t)slot;
    slot += n[i];
  }
  __syncthreads();
  // a thread an entry of the choice (an expert's thread for all its tokens took 8 us more where 64 tokens share
  // 8 experts): the first that names the expert for its token fills the slot
  for (int s = tid; s < slots; s += THREADS) {
    const int e = tmp.id[s], t = s / c.k;
    if (e < 0) continue;
    float w = tmp.w[s];
    bool first = true;
    if (c.ids != nullptr) {
      w = 0.0f;
      for (int j = t * c.k; j < (t + 1) * c.k; ++j)
        if (tmp.id[j] == e) {
          w += tmp.w[j];
          if (j < s) first = false;
        }
    }
    if (!first) continue;
    const int at = tmp.start[e] + __popcll(tmp.mask[e] & ((1ull << t) - 1));
    L.slot_token[at] = (uint8_t)t;
    L.slot_w[at] = w;
  }
  if (tid == THREADS - 1) L.scratch[32] = (before + incl) >> 16;
  __syncthreads();
}

// The same for at most 32 slots of at most two tokens, by warp 0, a slot a lane, from the choice in
// tmp (choose_few and a barrier before it). An expert is one unit (cap >= 4), in the order in
// which the slots first name them. Every CTA of both kernels of a small batch builds them
// (3.3 us by build_lists, most of it barriers and waits on shared memory; 0.3 so).
constexpr int kFewTokens = 2, kFewSlots = 32;
struct FewTemp {
  float w[kFewSlots];
  int id[kFewSlots];
};

// Warp t < T: token t's choice into tmp.
__device__ __forceinline__ void choose_few(const Choice& c, FewTemp& tmp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp >= c.T) return;
  int id = -1;
  float w = 0.0f;
  if (c.ids == nullptr) {
    choose_any(c.logits, c.ldt, warp, c.E, c.k, c.renorm != 0, id, w);
  } else if (lane < c.k) {
    id = __ldcg(c.ids + warp * c.k + lane);
    if (id < 0 || id >= c.E) id = -1;
    w = __ldcg(c.weights + warp * c.k + lane);
  }
  if (lane < c.k) {
    tmp.id[warp * c.k + lane] = id;
    tmp.w[warp * c.k + lane] = w;
  }
}

__device__ __forceinline__ void list_few(const Choice& c, const Lists& L, const FewTemp& tmp) {
  if (threadIdx.x >= 32) return;
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x;
  const unsigned below = (1u << lane) - 1;
  const bool in = lane < c.T * c.k;
  const int e = in ? tmp.id[lane] : -1, t = in ? lane / c.k : 0;
  const float w = in ? tmp.w[lane] : 0.0f;
  const bool live = e >= 0;
  const unsigned same = __match_any_sync(kAll, live ? e : -1 - lane);            // slots of this expert
  const unsigned twin = __match_any_sync(kAll, live ? kFewTokens * e + t : -1 - lane);    // of this expert and token
  float sum = 0.0f;                                  // the twins' weights, in order
  for (unsigned left = __reduce_or_sync(kAll, __popc(twin) > 1 ? twin : 0u); left != 0; left &= left - 1) {
    const int j = __ffs(left) - 1;
    const float v = __shfl_sync(kAll, w, j);
    if (twin >> j & 1) sum += v;
  }
  if (__popc(twin) == 1) sum = w;
  const bool first = live && (same & below) == 0, first_twin = live && (twin & below) == 0;
  unsigned tokens = 0;                               // of this expert
#pragma unroll
  for (int i = 0; i < kFewTokens; ++i)
    if (__ballot_sync(kAll, live && t == i) & same) tokens |= 1u << i;
  const int n = __popc(tokens);
  int start = first ? n : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kAll, start, o);
    if (lane >= o) start += u;
  }
  start = __shfl_sync(kAll, start - n, __ffs(same) - 1);      // the leader's: slots before this expert's
  const unsigned leaders = __ballot_sync(kAll, first);
  if (first) {
    const int unit = __popc(leaders & below);
    L.unit_expert[unit] = (uint16_t)e;
    L.unit_start[unit] = (uint16_t)start;
    L.unit_n[unit] = (uint8_t)n;
  }
  if (first_twin) {
    const int slot = start + __popc(tokens & ((1u << t) - 1));
    L.slot_token[slot] = (uint8_t)t;
    L.slot_w[slot] = sum;
  }
  if (lane == 0) L.scratch[32] = __popc(leaders);
}

// Lists that another kernel has built, as the bytes of lists_at's block; closes with a barrier.
template <int THREADS>
__device__ __forceinline__ void copy_lists(uint8_t* to, const uint8_t* from, int slots) {
  for (int i = threadIdx.x; i < lists_bytes(slots) / 16; i += THREADS)
    reinterpret_cast<uint4*>(to)[i] = __ldcg(reinterpret_cast<const uint4*>(from) + i);
  __syncthreads();
}

}  // namespace moe
}  // namespace ck
