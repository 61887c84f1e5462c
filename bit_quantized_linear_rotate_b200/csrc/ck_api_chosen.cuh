// Host side of the operators whose weights are chosen for each token: expert
// routing, the mixture-of-experts layer and the low-rank adapters. Included by
// ck_api.cu, whose helpers (fail, launch_status, aligned, S, sm_count) it uses.

namespace {

// Launches `kern` as a programmatic dependent (see launch_pdl) with clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), unsigned grid, unsigned cluster, unsigned block, size_t smem,
                           cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

bool known_float(ck_dtype t) { return t == CK_BF16 || t == CK_FP16; }

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// ------------------------------------------------------------------ routing

ck_status check_choice(const char* who, int64_t E, int top_k) {
  using namespace ck::moe;
  if (E <= 0 || top_k <= 0) return fail(CK_ERR_INVALID_ARG, "%s: E and top_k must be > 0", who);
  if (E > kMaxExperts) return fail(CK_ERR_UNSUPPORTED, "%s: E=%lld > %d", who, (long long)E, kMaxExperts);
  if (top_k > kMaxTopK) return fail(CK_ERR_UNSUPPORTED, "%s: top_k=%d > %d", who, top_k, kMaxTopK);
  if (top_k > E) return fail(CK_ERR_INVALID_ARG, "%s: top_k=%d > E=%lld", who, top_k, (long long)E);
  return CK_OK;
}

ck_status check_logits(const char* who, const void* logits, ck_dtype lt) {
  if (!known_float(lt) && lt != CK_FP32) return fail(CK_ERR_INVALID_ARG, "%s: unknown logits dtype", who);
  if (!logits) return fail(CK_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned(logits, lt == CK_FP32 ? 4 : 2)) return fail(CK_ERR_INVALID_ARG, "%s: misaligned logits", who);
  return CK_OK;
}

// -------------------------------------------------------- mixture of experts

// Stages of `stage` bytes that fit beside what precedes the ring, for `ctas` CTAs on an SM (0: fewer
// than two do).
int moe_stages(int offset, int stage, int ctas) {
  const int room = (228 * 1024) / ctas - 1024;       // 1 KB of an SM's 228 is reserved for each CTA
  const int n = (std::min(room, 227 * 1024) - 1024 - offset) / stage;   // 1 KB: the base's alignment
  return n < 2 ? 0 : std::min(n, ck::moe::kMaxStages);
}

// Once a device: the kernel may take all of an SM's shared memory, and the SM is set up for that (a CTA
// of the next kernel can then join one that needs less).
template <typename Tag, typename KernelT>
cudaError_t set_smem_all(KernelT kern) {
  static std::atomic<bool> done[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

// How many clusters of `cs` CTAs with `smem` bytes run at once (0: none). Remembered for each kernel and
// device in a small table; an entry holds its key and the answer.
template <typename Tag, typename KernelT>
int clusters_at_once(KernelT kern, int threads, int smem, int cs) {
  static std::atomic<uint64_t> table[kMaxDevices][128];
  const int dev = current_device(), kb = (smem + 1023) / 1024;
  if (dev < 0) return 0;
  const uint32_t key = (uint32_t)(kb * 16 + cs);
  std::atomic<uint64_t>& entry = table[dev][(kb * 8 + cs - 1) & 127];
  const uint64_t known = entry.load(std::memory_order_relaxed);
  if ((uint32_t)(known >> 32) == key) return (int)(uint32_t)known;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)cs);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 0) {
    cudaGetLastError();
    n = 0;
  }
  entry.store((uint64_t)key << 32 | (uint32_t)n, std::memory_order_relaxed);
  return n;
}

template <typename T, int NT, int KW, bool SELF>
cudaError_t launch_gate_up(const ck::moe::Maps& maps, const ck::moe::Params& p, cudaStream_t st) {
  using namespace ck::moe;
  using C = GateUp<NT, KW, SELF>;
  void (*kern)(const Maps, const Params, int);
  if constexpr (SELF) kern = gate_up_few_kernel<T>;
  else kern = gate_up_kernel<T, NT>;
  struct Tag {};
  const int offset = ring_offset(p.choice.T * p.choice.k, C::sums(p.choice.T, p.K));
  int ctas = C::kCtas;
  while (ctas > 1 && moe_stages(offset, C::kStage, ctas) == 0) --ctas;
  int stages = moe_stages(offset, C::kStage, ctas);
  if (stages == 0) return cudaErrorInvalidValue;
  if (SELF) stages = std::min(stages, 3);   // leaves room for a CTA of down_kernel beside it
  const int smem = 1024 + offset + stages * C::kStage;
  const cudaError_t e = set_smem_all<Tag>(kern);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)p.choice.T * p.choice.k * (p.I / kColsItem);   // a unit has a slot at least
  const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)ctas * sm_count());
  return launch_pdl(kern, dim3(grid), dim3(C::kThreads), smem, st, maps, p, stages);
}

template <typename T, int NT>
cudaError_t launch_down(const ck::moe::Maps& maps, const ck::moe::Params& p, cudaStream_t st) {
  using namespace ck::moe;
  using C = Down<NT>;
  auto kern = down_kernel<T, NT>;
  struct Tag {};
  const int offset = ring_offset(p.choice.T * p.choice.k, C::sums(p.choice.T));
  cudaError_t e = set_smem_all<Tag>(kern);
  if (e != cudaSuccess) return e;
  // C::kCtas CTAs an SM (one where the sums leave no room for two). The cluster size by the time expected: rounds of
  // clusters (33 of 8 run at once, 71 of 4), each some 0.5 us a step and 0.35 us a CTA of the cluster for
  // meeting and adding up (fitted to 1 to 110 steps: 16 tokens of 64 experts, K = 2048, are fastest in
  // clusters of 8, 59 against 72 us in clusters of 4; 32 tokens of 16 experts, K = 5120, of 3, 101
  // against 119 in clusters of 2). Behind gate_up_few_kernel, beside which there is room for one CTA an
  // SM, every CTA costs (K = I = 3840, one token: 22.3 us in clusters of 2, 27.2 of 8).
  const int tiles = p.K / kRowsTile;
  const double units = p.choice.E * (1 - std::pow(1 - std::min(1.0, (double)p.choice.k / p.choice.E), p.choice.T));
  const double steps = std::max(1.0, units) * ((p.I + 64 * C::kSubs - 1) / (64 * C::kSubs));
  int ctas = C::kCtas, cs = 0;
  int stages = moe_stages(offset, C::kStage, ctas);
  if (stages == 0) stages = moe_stages(offset, C::kStage, ctas = 1);
  const int smem = 1024 + offset + stages * C::kStage;
  double best = 1e30;
  const double each = p.lists == nullptr ? 0.012 : 0.0;
  for (int s = 1; s <= 8; ++s) {
    const int fit = clusters_at_once<Tag>(kern, C::kThreads, smem, s);
    if (stages == 0 || fit <= 0) continue;
    const double t = ((tiles + fit - 1) / fit) * (std::ceil(steps / s) * 0.5 + 0.35 * s) + each * tiles * s;
    if (t < best) best = t, cs = s;
  }
  if (cs == 0) return cudaErrorInvalidValue;
  return launch_cluster(kern, (unsigned)(tiles * cs), (unsigned)cs, C::kThreads, smem, st, maps, p, stages);
}

// Workspace: rows of x, rows of h, the lists.
struct MoeWorkspace {
  size_t xr, hr, lists, total;
  MoeWorkspace(int64_t T, int k, int64_t K, int64_t I) {
    size_t at = 0;
    auto take = [&at](int64_t bytes) {
      const size_t a = at;
      at = (at + (size_t)bytes + 255) / 256 * 256;
      return a;
    };
    xr = take(T * ck::moe::x_row_bytes((int)K));
    hr = take(T * k * ck::moe::h_row_bytes((int)I));
    lists = take(ck::moe::lists_bytes((int)(T * k)));
    total = at;
  }
};

// Which kernels a call runs. One or two tokens whose items (64 columns of h of an expert) each get
// an SM of their own: 16 consumer warps, one CTA an SM, which routes and orders x itself (K = 2048,
// I = 1024: one token, top-8 of 64, 16.2 us, 17.2 with prepare_kernel; two, top-4, 16.2 and 17.8). With a second
// round of items it gains nothing or loses: two tokens, top-8, 26.2 us either way, and K = 4096, I = 4096,
// top-4 at one 39.9 against 37.7.
// Else two CTAs an SM, and token tiles (of four) a unit by how many
// tokens an expert is likely to get, the mean and three standard deviations: an expert with
// more is read again for the rest, while room for 16 tokens in every stage costs depth of the ring.
bool moe_self(const ck::moe::Params& p) {
  const int64_t items = (int64_t)p.choice.T * p.choice.k * (p.I / ck::moe::kColsItem);
  return p.choice.T <= ck::moe::kFewTokens && items <= sm_count() &&
         p.choice.T * p.choice.k <= ck::moe::kFewSlots && p.choice.T * ck::moe::x_row_bytes(p.K) <= ck::moe::kSelfBytes;
}
int moe_token_tiles(const ck::moe::Params& p) {
  const double mean = (double)p.choice.T * p.choice.k / p.choice.E;
  const double likely = std::min<double>(p.choice.T, mean + 3 * std::sqrt(mean));
  return likely <= 4 ? 1 : likely <= 8 ? 2 : 4;
}
int gate_up_stage_cols(const ck::moe::Params& p) { return moe_self(p) ? 512 : 256; }

template <typename T>
cudaError_t launch_moe(const ck::moe::Maps& gate_up, const ck::moe::Maps& down, ck::moe::Params& p, uint8_t* ws,
                       const MoeWorkspace& w, cudaStream_t st) {
  using namespace ck::moe;
  const int tiles = moe_token_tiles(p);
  cudaError_t e;
  if (moe_self(p)) {
    p.lists = nullptr;
    e = launch_gate_up<T, 1, 4, true>(gate_up, p, st);
  } else {
    p.lists = ws + w.lists;
    // 1024 threads from 17 tokens on: their warps choose for one token at a time (64 tokens of 256 experts, K =
    // I = 512: 72 us for the layer against 80; for fewer tokens 0.3 us slower)
    const bool many = p.choice.T > 16;
    e = launch_pdl(many ? prepare_kernel<T, 1024> : prepare_kernel<T, 512>, dim3((unsigned)p.choice.T + 1),
                   dim3(many ? 1024 : 512), 0, st, p, 4 * tiles);
    if (e != cudaSuccess) return e;
    e = tiles == 1 ? launch_gate_up<T, 1, 2, false>(gate_up, p, st)
      : tiles == 2 ? launch_gate_up<T, 2, 2, false>(gate_up, p, st)
                   : launch_gate_up<T, 4, 2, false>(gate_up, p, st);
  }
  if (e != cudaSuccess) return e;
  return tiles == 1 ? launch_down<T, 1>(down, p, st)
       : tiles == 2 ? launch_down<T, 2>(down, p, st)
                    : launch_down<T, 4>(down, p, st);
}

// Maps of `rows` weight rows of `cols` columns for each expert: boxes of 64
// rows x 256 columns, and of their scales for the groups of `stage_cols` columns.
ck_status make_expert_maps(ck::moe::Maps* m, const uint8_t* q, const void* s, const void* z, int64_t E, int64_t rows,
                           int64_t cols, int G, int stage_cols) {
  ck_status r = make_tmap(&m->w, q, (uint64_t)cols / 2, (uint64_t)(E * rows), (uint64_t)cols / 2, 128, 64,
                          CU_TENSOR_MAP_SWIZZLE_128B);
  if (r != CK_OK) return r;
  const uint64_t groups = (uint64_t)(E * (cols / G));
  r = make_tmap(&m->s, s, (uint64_t)rows, groups, (uint64_t)rows * 2, 64, (uint32_t)(stage_cols / G),
                CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_DATA_TYPE_UINT16);
  if (r != CK_OK) return r;
  return make_tmap(&m->z, z, (uint64_t)rows, groups, (uint64_t)rows * 2, 64, (uint32_t)(stage_cols / G),
                   CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_DATA_TYPE_UINT16);
}

struct MoeArgs {
  const void* x;
  ck_dtype dt;
  int64_t T, K, I, E, ldx;
  int G;
  const uint8_t* gq;
  const void *gs, *gz;
  const uint8_t* dq;
  const void *ds, *dz;
  void *out, *ws;
  size_t ws_bytes;
};

ck_status moe_impl(const char* who, const MoeArgs& a, const ck::moe::Choice& choice, cudaStream_t st) {
  using namespace ck::moe;
  if (a.T < 0 || a.K <= 0 || a.I <= 0) return fail(CK_ERR_INVALID_ARG, "%s: T must be >= 0, K and I > 0", who);
  if (!known_float(a.dt)) return fail(CK_ERR_INVALID_ARG, "%s: unknown dtype", who);
  if (a.T > kMaxTokens) return fail(CK_ERR_UNSUPPORTED, "%s: T=%lld > %d", who, (long long)a.T, kMaxTokens);
  if (a.G != 64 && a.G != 128 && a.G != 256)
    return fail(CK_ERR_UNSUPPORTED, "%s: group_size=%d must be 64, 128 or 256", who, a.G);
  if (a.K % a.G != 0 || a.I % a.G != 0)
    return fail(CK_ERR_INVALID_ARG, "%s: K and I must be multiples of group_size", who);
  if (a.K > (1 << 20) || a.I > (1 << 20)) return fail(CK_ERR_UNSUPPORTED, "%s: dimension too large", who);
  if (a.T == 0) return ok();
  if (a.ldx < a.K || a.ldx % 8 != 0)
    return fail(CK_ERR_INVALID_ARG, "%s: ldx=%lld must be >= K and a multiple of 8", who, (long long)a.ldx);
  if (!a.x || !a.gq || !a.gs || !a.gz || !a.dq || !a.ds || !a.dz || !a.out || !a.ws)
    return fail(CK_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned(a.x, 16) || !aligned(a.gq, 16) || !aligned(a.dq, 16) || !aligned(a.gs, 16) || !aligned(a.gz, 16) ||
      !aligned(a.ds, 16) || !aligned(a.dz, 16))
    return fail(CK_ERR_INVALID_ARG, "%s: x, the weights, scales and zeros must be 16-byte aligned", who);
  if (!aligned(a.out, 2)) return fail(CK_ERR_INVALID_ARG, "%s: misaligned output", who);
  if (!aligned(a.ws, 256)) return fail(CK_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  const MoeWorkspace w(a.T, choice.k, a.K, a.I);
  if (a.ws_bytes < w.total)
    return fail(CK_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", who, a.ws_bytes, w.total);
  Params p;
  p.choice = choice;
  p.x = a.x; p.ldx = a.ldx; p.K = (int)a.K; p.I = (int)a.I;
  p.gsh = a.G == 64 ? 0 : a.G == 128 ? 1 : 2;
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.ws);
  p.xr = ws + w.xr;
  p.hr = ws + w.hr;
  p.out = a.out;
  Maps gate_up, down;
  ck_status r = make_expert_maps(&gate_up, a.gq, a.gs, a.gz, a.E, 2 * a.I, a.K, a.G, gate_up_stage_cols(p));
  if (r != CK_OK) return r;
  r = make_expert_maps(&down, a.dq, a.ds, a.dz, a.E, a.K, a.I, a.G, 512);
  if (r != CK_OK) return r;
  const cudaError_t e = a.dt == CK_BF16 ? launch_moe<__nv_bfloat16>(gate_up, down, p, ws, w, st)
                                        : launch_moe<__half>(gate_up, down, p, ws, w, st);
  if (e != cudaSuccess) return fail(CK_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
  return launch_status(who);
}

// ----------------------------------------------------------------- adapters

template <typename T, typename TY, int RC>
cudaError_t launch_lora_few(const ck::lora::Params& p, int64_t tiles, cudaStream_t st) {
  using namespace ck::lora;
  auto kern = lora_kernel<T, TY, RC>;
  struct Tag {};
  const int smem = (int)sizeof(Smem<RC, VOperand<T>::kPlanes>);
  const cudaError_t e = set_smem_max<Tag>(kern, smem, smem);
  if (e != cudaSuccess) return e;
  // The cluster size by the time expected: rounds of as many clusters as run at once, each a share of a tile's
  // adapter (at 14 GB/s a CTA) and some 4 us for finding the tile and exchanging v; the number of
  // tiles, known on the device only, as that of the different ids that M draws make. (K = N = 4096, R = 16, 64
  // adapters, 100 tokens: 11.7 us, 14.1 in clusters of 4, 17.0 of 8, which need two rounds.)
  const double work = 2.0 * p.R * ((double)p.K + p.N) / 14e3;
  const double likely = std::max(1.0, (p.L + 1) * (1 - std::pow(1 - 1.0 / (p.L + 1), p.M)) + (double)p.M / kFewTile / 2);
  int cs = 1;
  double best = 1e30;
  for (int s = 8; s >= 1; --s) {
    const int fit = clusters_at_once<Tag>(kern, kThreads, smem, s);
    if (fit <= 0) continue;
    const double t = std::ceil(std::min(likely, (double)tiles) / fit) * (work / s + 4);
    if (t < best) best = t, cs = s;
  }
  return launch_cluster(kern, (unsigned)(tiles * cs), (unsigned)cs, kThreads, smem, st, p);
}

template <typename T, typename TY, int RB>
cudaError_t launch_lora_tc(const ck::lora::Params& p, int64_t tiles, cudaStream_t st) {
  using namespace ck::lora;
  using C = LoraTc<RB, VOperand<T>::kPlanes>;
  auto kern = lora_tc_kernel<T, TY, RB>;
  struct Tag {};
  const cudaError_t e = set_smem_max<Tag>(kern, C::kSmem, C::kSmem);
  if (e != cudaSuccess) return e;
  const CUtensorMapDataType dt = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapDataType dy = std::is_same<TY, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  constexpr CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  TcMaps m;           // boxes of 64 columns x: A's R rows (rounded up), 128 rows of B, x, y and out
  if (make_tmap(&m.a, p.a, p.K, (uint64_t)p.L * p.R, (uint64_t)p.K * 2, 64, (uint32_t)((p.R + 15) / 16 * 16), sw, dt) ||
      make_tmap(&m.b, p.b, p.R, (uint64_t)p.L * p.N, (uint64_t)p.R * 2, 64, 128, sw, dt) ||
      make_tmap(&m.x, p.x, p.K, p.M, (uint64_t)p.ldx * 2, 64, 128, sw, dt))
    return cudaErrorInvalidValue;
  m.y = m.out = m.x;  // not used unless p.vec
  if (p.vec && (make_tmap(&m.y, p.y, p.N, p.M, (uint64_t)p.ldy * 2, 64, 128, sw, dy) ||
                make_tmap(&m.out, p.out, p.N, p.M, (uint64_t)p.ldo * 2, 64, 128, sw, dy)))
    return cudaErrorInvalidValue;
  // The cluster size by the time it is expected to take: rounds of as many clusters as run at once (15 of
  // 8 CTAs, 22 of 6), each 1 / cs of a tile's bytes (at an SM's 43 GB/s) and 6 us for the stages that
  // wait for one another (M = 2048, K = N = 4096, R = 16, 4 adapters: 23.2 us with clusters of 6, 37.5 with
  // clusters of 8, the best if all SMs took part). The number of tiles, known on the device only, is taken
  // between that of requests of 128 tokens, each with any adapter or none, and that of all adapters in turn.
  const double work = 128.0 * (p.K + 2.0 * p.N) * 2 / 43e3, fixed = 6.0;
  const double full = (double)p.M / kTcTokens, ids = p.L + 1.0;
  auto tiles_of = [&](double adapters) { return adapters * std::max(1.0, full / adapters + 0.5); };
  const double likely = (tiles_of(ids) + tiles_of(ids * (1 - std::pow(1 - 1 / ids, full)))) / 2;
  int cs = 0;
  double best = 1e30;
  for (int c = 1; c <= 8; ++c) {
    const int fit = clusters_at_once<Tag>(kern, kTcThreads, C::kSmem, c);
    if (fit <= 0) continue;
    const double t = std::ceil(std::min(likely, (double)tiles) / fit) * (work / c + fixed);
    if (t < best) best = t, cs = c;
  }
  if (cs == 0) return cudaErrorInvalidValue;
  return launch_cluster(kern, (unsigned)(tiles * cs), (unsigned)cs, kTcThreads, C::kSmem, st, m, p);
}

template <typename T, typename TY>
cudaError_t launch_lora(const ck::lora::Params& p, int tm, int64_t tiles, cudaStream_t st) {
  using ck::lora::kFewTile;
  if (tm == kFewTile) {
    if (p.R <= 32) return launch_lora_few<T, TY, 1>(p, tiles, st);
    if (p.R <= 64) return launch_lora_few<T, TY, 2>(p, tiles, st);
    return launch_lora_few<T, TY, 4>(p, tiles, st);
  }
  return p.R <= 64 ? launch_lora_tc<T, TY, 1>(p, tiles, st) : launch_lora_tc<T, TY, 2>(p, tiles, st);
}

// Tokens of a tile, by how many tokens there are and an adapter has on average: 128 from 513 tokens on
// (K = N = 4096, R = 16, one adapter: 512 tokens 12.4 us in tiles of 16, 17.3 of 128; 1024 tokens 22.9 and 18.2).
// With more adapters in memory than tokens / 32 small tiles win even where all tokens name one of them, whose weights
// then come from L2 for each tile (2000 tokens, 64 adapters: 21.8 us, 32.3 in tiles of 128).
int lora_tile(int64_t M, int64_t L) {
  return M > 512 && M >= 32 * L ? ck::lora::kTcTokens : ck::lora::kFewTile;
}

// Whether the CTAs find their tiles themselves; else group_kernel lists them.
bool lora_finds_tiles(int64_t M, int64_t L) {
  using namespace ck::lora;
  if (lora_tile(M, L) == kTcTokens) return M <= kPickTokens;
  return M <= kSelfGroup || (M <= kSelfPick && L <= kPickAdapters);
}

}  // namespace

extern "C" {

ck_status ck_moe_route(const void* logits, ck_dtype lt, int64_t T, int64_t E, int top_k, int renormalize,
                       float* weights, int32_t* ids, void* stream) {
  const char* who = "moe_route";
  if (T < 0) return fail(CK_ERR_INVALID_ARG, "%s: T must be >= 0", who);
  ck_status r = check_choice(who, E, top_k);
  if (r != CK_OK) return r;
  if (T == 0) return ok();
  r = check_logits(who, logits, lt);
  if (r != CK_OK) return r;
  if (!weights || !ids) return fail(CK_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned(weights, 4) || !aligned(ids, 4)) return fail(CK_ERR_INVALID_ARG, "%s: misaligned output", who);
  const int64_t grid = (T + ck::moe::kRouteWarps - 1) / ck::moe::kRouteWarps;
  if (grid > INT32_MAX) return fail(CK_ERR_UNSUPPORTED, "%s: T=%lld too large", who, (long long)T);
  const cudaError_t e = launch_pdl(ck::moe::route_kernel, dim3((unsigned)grid), dim3(32 * ck::moe::kRouteWarps), 0,
                                   S(stream), logits, (int)lt, T, (int)E, top_k, renormalize, weights, ids);
  if (e != cudaSuccess) return fail(CK_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
  return launch_status(who);
}

size_t ck_moe_awq_w4a16_workspace_bytes(int64_t T, int top_k, int64_t K, int64_t I) {
  return T <= 0 || top_k <= 0 || K <= 0 || I <= 0 ? 0 : MoeWorkspace(T, top_k, K, I).total;
}

ck_status ck_moe_awq_w4a16(const void* x, ck_dtype dt, int64_t T, int64_t K, int64_t I, int64_t E, int64_t ldx,
                           int group_size, const void* logits, ck_dtype lt, int top_k, int renormalize,
                           const uint8_t* gate_up_q, const void* gate_up_s, const void* gate_up_z,
                           const uint8_t* down_q, const void* down_s, const void* down_z, void* out,
                           void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "moe_awq_w4a16";
  ck_status r = check_choice(who, E, top_k);
  if (r != CK_OK) return r;
  if (T != 0) {
    r = check_logits(who, logits, lt);
    if (r != CK_OK) return r;
  }
  const ck::moe::Choice c = {logits, nullptr, nullptr, (int)lt, (int)T, (int)E, top_k, renormalize};
  const MoeArgs a = {x, dt, T, K, I, E, ldx, group_size, gate_up_q, gate_up_s, gate_up_z,
                     down_q, down_s, down_z, out, workspace, workspace_bytes};
  return moe_impl(who, a, c, S(stream));
}

ck_status ck_moe_experts_awq_w4a16(const void* x, ck_dtype dt, int64_t T, int64_t K, int64_t I, int64_t E,
                                   int64_t ldx, int group_size, const int32_t* ids, const float* weights, int top_k,
                                   const uint8_t* gate_up_q, const void* gate_up_s, const void* gate_up_z,
                                   const uint8_t* down_q, const void* down_s, const void* down_z, void* out,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "moe_experts_awq_w4a16";
  if (E <= 0 || top_k <= 0) return fail(CK_ERR_INVALID_ARG, "%s: E and top_k must be > 0", who);
  if (E > ck::moe::kMaxExperts)
    return fail(CK_ERR_UNSUPPORTED, "%s: E=%lld > %d", who, (long long)E, ck::moe::kMaxExperts);
  if (top_k > ck::moe::kMaxTopK)
    return fail(CK_ERR_UNSUPPORTED, "%s: top_k=%d > %d", who, top_k, ck::moe::kMaxTopK);
  if (T != 0) {
    if (!ids || !weights) return fail(CK_ERR_INVALID_ARG, "%s: null pointer", who);
    if (!aligned(ids, 4) || !aligned(weights, 4))
      return fail(CK_ERR_INVALID_ARG, "%s: misaligned ids or weights", who);
  }
  const ck::moe::Choice c = {nullptr, ids, weights, 0, (int)T, (int)E, top_k, 0};
  const MoeArgs a = {x, dt, T, K, I, E, ldx, group_size, gate_up_q, gate_up_s, gate_up_z,
                     down_q, down_s, down_z, out, workspace, workspace_bytes};
  return moe_impl(who, a, c, S(stream));
}

size_t ck_lora_add_workspace_bytes(int64_t M, int64_t L) {
  if (M <= 0 || L <= 0 || lora_finds_tiles(M, L)) return 0;
  return (size_t)ck::lora::max_tiles(M, L, lora_tile(M, L)) * 16 + (size_t)M * 4;   // tile list, token order
}

ck_status ck_lora_add(const void* y, ck_dtype yt, const void* x, ck_dtype xt, int64_t M, int64_t K, int64_t N,
                      int64_t R, int64_t L, int64_t ldx, int64_t ldy, int64_t ldo, const void* lora_a,
                      const void* lora_b, const int32_t* ids, const float* scales, void* out, void* workspace,
                      size_t workspace_bytes, void* stream) {
  const char* who = "lora_add";
  if (M < 0 || K <= 0 || N <= 0 || R <= 0 || L <= 0)
    return fail(CK_ERR_INVALID_ARG, "%s: M must be >= 0, K, N, R and L > 0", who);
  if (!known_float(xt) || !known_float(yt)) return fail(CK_ERR_INVALID_ARG, "%s: unknown dtype", who);
  if (yt != CK_BF16 && yt != xt)
    return fail(CK_ERR_UNSUPPORTED, "%s: y must be bf16 or of x's dtype", who);
  if (R % 8 != 0 || R > 128) return fail(CK_ERR_UNSUPPORTED, "%s: R=%lld must be a multiple of 8, at most 128", who, (long long)R);
  if (K % 8 != 0) return fail(CK_ERR_UNSUPPORTED, "%s: K=%lld must be a multiple of 8", who, (long long)K);
  if (L > ck::lora::kMaxAdapters)
    return fail(CK_ERR_UNSUPPORTED, "%s: L=%lld > %d", who, (long long)L, ck::lora::kMaxAdapters);
  if (K > INT32_MAX / 2 || N > INT32_MAX / 2 || L * N > INT32_MAX || M > (int64_t)1 << 26)
    return fail(CK_ERR_UNSUPPORTED, "%s: dimension too large", who);
  if (M == 0) return ok();
  if (ldx < K || ldx % 8 != 0)
    return fail(CK_ERR_INVALID_ARG, "%s: ldx=%lld must be >= K and a multiple of 8", who, (long long)ldx);
  if (ldy < N || ldo < N) return fail(CK_ERR_INVALID_ARG, "%s: ldy and ldo must be >= N", who);
  if (!y || !x || !lora_a || !lora_b || !ids || !out) return fail(CK_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned(x, 16) || !aligned(lora_a, 16) || !aligned(lora_b, 16))
    return fail(CK_ERR_INVALID_ARG, "%s: x and the adapters must be 16-byte aligned", who);
  if (!aligned(y, 2) || !aligned(out, 2) || !aligned(ids, 4) || (scales && !aligned(scales, 4)))
    return fail(CK_ERR_INVALID_ARG, "%s: misaligned y, output, ids or scales", who);
  const int64_t out_bytes = 2 * ((M - 1) * ldo + N);
  if (!(out == y && ldo == ldy) && overlap(out, out_bytes, y, 2 * ((M - 1) * ldy + N)))
    return fail(CK_ERR_INVALID_ARG, "%s: the output overlaps y without being y", who);
  if (overlap(out, out_bytes, x, 2 * ((M - 1) * ldx + K)))
    return fail(CK_ERR_INVALID_ARG, "%s: the output overlaps x", who);
  using namespace ck::lora;
  const int tm = lora_tile(M, L);
  const int64_t tiles = max_tiles(M, L, tm);
  ck::lora::Params p;
  p.x = x; p.y = y; p.a = lora_a; p.b = lora_b; p.ids = ids; p.scales = scales; p.out = out;
  p.ldx = ldx; p.ldy = ldy; p.ldo = ldo;
  p.M = (int)M; p.K = (int)K; p.N = (int)N; p.R = (int)R; p.L = (int)L;
  p.vec = N % 8 == 0 && ldy % 8 == 0 && ldo % 8 == 0 && aligned(y, 16) && aligned(out, 16);
  p.tiles = nullptr;
  p.order = nullptr;
  cudaError_t e = cudaSuccess;
  if (!lora_finds_tiles(M, L)) {
    const size_t need = ck_lora_add_workspace_bytes(M, L);
    if (!workspace) return fail(CK_ERR_INVALID_ARG, "%s: null workspace", who);
    if (!aligned(workspace, 256)) return fail(CK_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
    if (workspace_bytes < need)
      return fail(CK_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes, need);
    int32_t* tl = reinterpret_cast<int32_t*>(workspace);
    int32_t* order = tl + 4 * tiles;
    p.tiles = tl;
    p.order = order;
    e = launch_pdl(group_kernel, dim3(1), dim3(kGroupThreads), (size_t)(L + 1) * 4, S(stream), ids, (int)M, (int)L, tm,
                   (int)tiles, tl, order);
    if (e != cudaSuccess) return fail(CK_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
  }
  if (xt == CK_BF16) e = launch_lora<__nv_bfloat16, __nv_bfloat16>(p, tm, tiles, S(stream));
  else if (yt == CK_FP16) e = launch_lora<__half, __half>(p, tm, tiles, S(stream));
  else e = launch_lora<__half, __nv_bfloat16>(p, tm, tiles, S(stream));
  if (e != cudaSuccess) return fail(CK_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
  return launch_status(who);
}

}  // extern "C"
