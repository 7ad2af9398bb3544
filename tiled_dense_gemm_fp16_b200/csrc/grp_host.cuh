// grp_host.cuh -- argument checks, kernel choice and launches of the grouped
// products, their gradients and the low-rank adapters.  Included by tg_gemm.cu
// after ff_host.cuh, whose helpers it uses.
#pragma once

#include "gemm_grp_narrow.cuh"
#include "gemm_grp_pair.cuh"
#include "gemm_grp_wgrad.cuh"
#include "lora_shrink.cuh"

namespace tg {
namespace {

constexpr int64_t kLoraMaxRank = 512;
constexpr int64_t kLoraMaxAdapters = int64_t(1) << 20;

// current_device, with the device's context bound to this host thread.  Encoding a
// tensor map needs one, and a thread that has made no runtime call yet has none
// (autograd's, whose memory comes out of torch's cache, when a backward pass
// starts with a product).
tg_status grp_device(DeviceInfo*& info) {
  int dev = 0;
  const tg_status st = current_device(dev, info);
  static thread_local int bound = -1;
  if (st == TG_OK && bound != dev) {
    if (cudaSetDevice(dev) != cudaSuccess) {
      cudaGetLastError();
      return TG_ERR_LAUNCH;
    }
    bound = dev;
  }
  return st;
}

// `mats` matrices of 16-bit values, `stride` elements apart.
struct GrpStack {
  FfMat m;  // the first
  int64_t mats, stride;

  bool empty() const { return mats == 0 || m.empty(); }
  // First to last byte, of a valid stack.
  FfMat span() const {
    if (empty()) return FfMat{m.p, 0, 0, 1, 2};
    const int64_t n = (mats - 1) * stride + (m.rows - 1) * m.ld + m.cols;
    return FfMat{m.p, 1, n, n, 2};
  }
  bool valid(bool written) const {
    if (empty()) return true;
    if (!m.valid() || m.rows > kFfMaxSpan / m.ld) return false;
    if (mats == 1) return true;
    const int64_t least = written ? (m.rows - 1) * m.ld + m.cols : m.cols;
    return stride >= least && stride <= kFfMaxStride && mats <= kFfMaxSpan / stride;
  }
  bool on16() const { return m.rows_on(16) && (mats == 1 || (stride * 2) % 16 == 0); }
  bool even_rows() const { return mats <= 1 || stride == m.rows * m.ld; }
  // All rows as one matrix, for a stack of evenly spaced rows.
  FfMat rows() const { return FfMat{m.p, mats * m.rows, m.cols, m.ld, 2}; }
};

GrpStack grp_stack(const void* p, int64_t mats, int64_t rows, int64_t cols, int64_t ld, int64_t stride) {
  GrpStack s;
  s.m = FfMat{p, rows, cols, ld ? ld : cols, 2};
  s.mats = mats;
  s.stride = stride;
  if (stride == 0) s.stride = rows <= kFfMaxSize && s.m.ld <= kFfMaxSpan / (rows + 1) ? rows * s.m.ld : 0;
  if (rows == 1 && mats > 1 && s.stride >= cols) s.m.ld = s.stride;  // matrices of one row: the stack's rows
  return s;
}

// Bytes of the padded copy of a stack that TMA cannot describe, 0 where it can, -1 where it
// cannot be copied: rows that are not evenly spaced, or so many that the kernel's steps over them would pass 32 bits.
int64_t grp_copy_bytes(const GrpStack& s) {
  if (s.empty() || s.on16()) return 0;
  if (!s.even_rows() || s.mats * s.m.rows > INT_MAX - 65536) return -1;
  return up256(2 * s.mats * s.m.rows * round_up(s.m.cols, 8));
}

// Padded copies, those of the weights of groups with rows only.
struct GrpPadParams {
  PadSetParams set;
  const int* ends;
  int M, weights, rows_each;  // which of the set are the weights, and rows of one
};
__global__ void __launch_bounds__(256) grp_pad_kernel(const __grid_constant__ GrpPadParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const RepackParams& m = p.set.m[blockIdx.y];
  for (int row = blockIdx.x * 8 + (threadIdx.x >> 5); row < m.rows; row += gridDim.x * 8) {
    if (static_cast<int>(blockIdx.y) == p.weights) {
      const int g = row / p.rows_each;
      if (grp_end(p.ends, g, p.M) <= grp_end(p.ends, g - 1, p.M)) continue;
    }
    pad_row(m, row, threadIdx.x & 31);
  }
}

// The copies of those of x, y and w (which may be null) that TMA cannot describe, in one launch; advances `ws`.
tg_status grp_make_copies(FfMat* x, FfMat* y, GrpStack* w, const int32_t* ends, int64_t M, uint8_t*& ws, cudaStream_t stream,
                          DeviceInfo* info) {
  if (w == nullptr || w->empty() || w->on16()) {
    FfMat* mats[2];
    int n = 0;
    if (x) mats[n++] = x;
    if (y) mats[n++] = y;
    return ff_make_copies(mats, n, ws, stream, info);
  }
  GrpPadParams p;
  std::memset(&p, 0, sizeof p);
  FfMat rows = w->rows();
  FfMat* mats[3] = {x, y, &rows};
  int n = 0;
  int64_t most = 0;
  for (FfMat* m : mats) {
    if (m == nullptr || (m != &rows && ff_copy_bytes(*m) == 0)) continue;
    if (m == &rows) p.weights = n;
    most = m->rows > most ? m->rows : most;
    ff_copy_plan(*m, p.set.m[n++], ws);
  }
  w->m.p = rows.p;
  w->m.ld = rows.ld;
  w->stride = w->m.rows * rows.ld;
  p.ends = ends;
  p.M = static_cast<int>(M);
  p.rows_each = static_cast<int>(w->m.rows);
  int64_t blocks = (most + 7) / 8;  // eight warps, a row each
  const int64_t cap = static_cast<int64_t>(info->sm_count) * 8;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(blocks > cap ? cap : blocks), static_cast<unsigned>(n), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  LaunchAttrs la;
  la.fill(cfg, 1);
  if (cudaLaunchKernelEx(&cfg, grp_pad_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return TG_ERR_LAUNCH;
  }
  return TG_OK;
}

bool grp_encode3(CUtensorMap* map, const GrpStack& s, int box_cols, int box_rows,
                 CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto fn = encode_fn();
  if (!fn) return false;
  const int64_t stride = s.mats == 1 ? round_up(s.m.rows * s.m.ld, 8) : s.stride;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(s.m.cols), static_cast<cuuint64_t>(s.m.rows),
                        static_cast<cuuint64_t>(s.mats)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(s.m.ld) * 2, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estride[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(s.m.p), dims, strides, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One product whose rows pick their weight: c[r] = w_g a[r], or w_g^T a[r].
struct GrpProduct {
  FfMat a, c;
  GrpStack w;
  const int32_t* ends = nullptr;  // nullptr: one group of all rows
  int groups = 1;
  int64_t out = 0, red = 0;
  bool transposed = false, rest = false, bf16 = false;
  bool beside = false;  // see GrpParams
  bool lora = false;
  LoraParams l;
  GrpStack lb;  // with adapters
  FfMat t;
};

bool grp_fill(const GrpProduct& f, GrpMaps& maps, GrpParams& p, int weight_rows, int tokens) {
  std::memset(&maps, 0, sizeof maps);
  std::memset(&p, 0, sizeof p);
  if (!grp_encode3(&maps.w, f.w, 64, f.transposed ? 64 : 128)) return false;
  for (int i = 0; i < 4 && 16 << i <= tokens; ++i)
    if (!ff_encode(&maps.x[i], f.a, 64, 16 << i, CU_TENSOR_MAP_SWIZZLE_128B)) return false;
  if (f.lora) {
    p.lora = f.l;
    if (f.l.adapters > 0 && (!grp_encode3(&maps.lb, f.lb, 64, 128) ||
                             !ff_encode(&maps.lt, f.t, 64, 16, CU_TENSOR_MAP_SWIZZLE_128B)))
      return false;
  }
  p.c = const_cast<void*>(f.c.p);
  p.ldc = f.c.ld;
  p.ends = f.ends;
  p.M = static_cast<int>(f.a.rows);
  p.groups = f.groups;
  p.out = static_cast<int>(f.out);
  p.red = static_cast<int>(f.red);
  p.col_tiles = static_cast<int>((f.out + weight_rows - 1) / weight_rows);
  p.k_blocks = static_cast<int>((f.red + 63) / 64);
  p.w_mn = f.transposed ? 1 : 0;
  p.rest = f.rest ? 1 : 0;
  p.bf16 = f.bf16 ? 1 : 0;
  p.beside = f.beside ? 1 : 0;
  p.wait_budget_ns = wait_budget(p.k_blocks);
  return true;
}

// Whether the walk's numbers of tiles, and its groups of `super` tiles, stay in 32 bits.
bool grp_countable(const GrpParams& p, int64_t most) {
  const int64_t tiles = (static_cast<int64_t>(p.M) + most - 1) / most + p.groups + 1;
  return tiles * p.col_tiles <= INT_MAX - 65536 && static_cast<int64_t>(p.super) * p.col_tiles <= INT_MAX;
}

tg_status launch_grp_pair(const GrpProduct& f, cudaStream_t stream, DeviceInfo* info) {
  using Cfg = GrpPairCfg;
  const int kind = f.lora ? (f.bf16 ? 2 : 1) : 0;
  auto kernel = kind == 0 ? grp_pair_kernel<0> : kind == 1 ? grp_pair_kernel<1> : grp_pair_kernel<2>;
  if (!ff_set_smem(reinterpret_cast<const void*>(kernel), info->grp_attr, 1u << kind,
                   Cfg::smem_bytes(f.lora ? 1 : kGrpMaxGroups, f.lora)))
    return TG_ERR_LAUNCH;
  GrpMaps maps;
  GrpParams p;
  if (!grp_fill(f, maps, p, Cfg::PAIR_M, Cfg::TOKENS / 2)) return TG_ERR_LAUNCH;
  p.vec = f.c.rows_on(16) ? 1 : 0;
  p.idesc = make_idesc_ff(kFfF16, f.bf16, Cfg::PAIR_M, 0, f.transposed, false);
  p.super = tune_int("TG_TUNE_GRP_SUPER", 8);
  if (!grp_countable(p, Cfg::TOKENS)) return TG_ERR_INVALID_ARG;
  const int64_t most = ((f.a.rows + 95) / 96 + f.groups) * p.col_tiles;  // tiles of the least width
  const int64_t pairs = info->sm_count / 2, clusters = most < pairs ? most : pairs;
  p.adapt = tune_int("TG_TUNE_GRP_ADAPT", (f.a.rows + 255) / 256 * p.col_tiles < 8 * pairs ? 1 : 0);
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters), 1, 1);
  cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(Cfg::smem_bytes(f.groups, f.lora));
  cfg.stream = stream;
  LaunchAttrs la;
  la.fill(cfg, 2);
  if (cudaLaunchKernelEx(&cfg, kernel, maps, p) != cudaSuccess) {
    cudaGetLastError();
    return TG_ERR_LAUNCH;
  }
  return TG_OK;
}

// Clusters of `splits` CTAs, one an SM, that fit on the device (see ff_resident_clusters).
int grp_resident_clusters(int splits, DeviceInfo* info) {
  std::lock_guard<std::mutex> lock(g_mutex);
  short& known = info->grp_clusters[splits];
  if (known == 0) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(splits) * 1024, 1, 1);
    cfg.blockDim = dim3(GrpNarrowCfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(GrpNarrowCfg::smem_bytes(128, 4, 1));
    LaunchAttrs la;
    la.fill(cfg, static_cast<unsigned>(splits));
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, grp_narrow_kernel<0>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = info->sm_count / splits > 0 ? info->sm_count / splits : 1;
    }
    known = static_cast<short>(n > 32767 ? 32767 : n);
  }
  return known;
}

// Estimated times in us.  The pair kernel: a wave of tiles takes 0.222 a k-block, 5.2
// before and after.  The rate of the weights flatters it: it reads them at 4.5 TB/s (64
// groups of 128 rows) or 3.3 (16 of 256, cold), which shifts the choice by some groups'
// worth towards it where the weights bound both.
double grp_pair_us(const GrpProduct& f, int64_t live, int k_blocks, DeviceInfo* info) {
  const int64_t rows = f.a.rows, pairs = info->sm_count / 2;
  const int64_t tiles = ((rows + 255) / 256 > live ? (rows + 255) / 256 : live) * ((f.out + 255) / 256);
  const double work = static_cast<double>((tiles + pairs - 1) / pairs) * k_blocks * 0.222;
  const double stream = static_cast<double>(live) * f.out * f.red * 2.0 / 5.6e6;  // of the weights from memory
  return 5.2 + (work > stream ? work : stream);
}

// The narrow kernel: a k-block takes 0.26 (up to 0.56 of 128 tokens); finishing a tile 1 + 0.03 a token alone,
// 2.2 + 0.045 with the exchange, while the next one's sums are under way.  Measured,
// us, narrow / pair, for g groups of n rows: 16 x 8 through 4096 x 512 (two splits)
// 23.4 / 14.7, 4 x 32 through 256 x 4096 10.6 / 19.4, 16 x 128 through 1024 x 1024 29 /
// 12, 16 x 8 through 2048 x 4096 44.5 / 48.2, 1 x 8 through 1024 x 1024 6.7 / 8.9.
double grp_narrow_us(const GrpProduct& f, int64_t live, int k_blocks, int tokens, int splits, DeviceInfo* info) {
  const int64_t rows = f.a.rows;
  const int64_t tiles = ((rows + tokens - 1) / tokens > live ? (rows + tokens - 1) / tokens : live) * ((f.out + 127) / 128);
  const int64_t fit = info->sm_count / splits - (splits > 2 ? 4 : 0);  // clusters of four leave some SMs out
  const double rounds = static_cast<double>((tiles + fit - 1) / fit);
  // Of 128 tokens the ring is short: felt where most SMs have a CTA.
  const double main = (k_blocks + splits - 1) / splits * (tokens < 128 || tiles * splits <= info->sm_count / 2 ? 0.26 : 0.56);
  const double finish = splits == 1 ? 1.0 + 0.03 * tokens : 2.2 + 0.045 * tokens;
  const double work = (splits < 4 ? 2.9 : 3.5) + main + (rounds - 1.0) * (main > finish ? main : finish) + finish;
  const double stream = 5.0 + static_cast<double>(live) * f.out * f.red * 2.0 / 6.3e6;
  return work > stream ? work : stream;
}

tg_status launch_grp_narrow(const GrpProduct& f, int tokens, int splits, cudaStream_t stream, DeviceInfo* info) {
  using Cfg = GrpNarrowCfg;
  const int kind = f.lora ? (f.bf16 ? 2 : 1) : 0;
  auto kernel = kind == 0 ? grp_narrow_kernel<0> : kind == 1 ? grp_narrow_kernel<1> : grp_narrow_kernel<2>;
  if (!ff_set_smem(reinterpret_cast<const void*>(kernel), info->grp_attr, 8u << kind, 232448)) return TG_ERR_LAUNCH;
  if (f.lora && !ff_set_smem(reinterpret_cast<const void*>(grp_narrow_kernel<0>), info->grp_attr, 8u, 232448))
    return TG_ERR_LAUNCH;  // the one that grp_resident_clusters asks about
  GrpMaps maps;
  GrpNarrowParams p;
  std::memset(&p, 0, sizeof p);
  if (!grp_fill(f, maps, p.g, Cfg::PANEL, tokens)) return TG_ERR_LAUNCH;
  p.g.idesc = make_idesc_ff(kFfF16, f.bf16, Cfg::PANEL, 0, f.transposed, false);
  p.g.super = 8;
  if (!grp_countable(p.g, tokens)) return TG_ERR_INVALID_ARG;
  p.tokens = tokens;
  p.own_t = f.lora && f.l.adapters > 0 && f.l.t == nullptr ? 1 : 0;
  splits = tune_int("TG_TUNE_GRP_SPLITS", splits);
  while (splits > p.g.k_blocks) splits >>= 1;
  p.splits = splits;
  // As deep as fits a CTA an SM, less a little for the kernel that makes T, which is still at work beside it.
  const bool adapted = f.lora && f.l.adapters > 0;
  const int fixed = Cfg::smem_bytes(tokens, 0, f.groups) + (adapted ? Cfg::lora_bytes(tokens, splits, p.own_t != 0) : 0);
  const int stage_bytes = Cfg::W_BYTES + tokens * 128;
  const int deepest = (232448 - (adapted && !p.own_t ? 4096 : 0) - fixed) / stage_bytes;
  p.per_stage = tune_int("TG_TUNE_GRP_PER", 2);
  while (p.per_stage > 1 && deepest < 3 * p.per_stage) p.per_stage >>= 1;
  p.stages = deepest / p.per_stage;
  if (p.stages > Cfg::MAX_STAGES) p.stages = Cfg::MAX_STAGES;
  p.tmem_cols = static_cast<uint32_t>(2 * tokens);
  const int64_t most = ((f.a.rows + tokens - 1) / tokens + f.groups) * p.g.col_tiles;
  const int64_t fit = grp_resident_clusters(splits, info), clusters = most < fit ? most : fit;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(splits * clusters), 1, 1);
  cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(fixed + p.stages * p.per_stage * stage_bytes);
  cfg.stream = stream;
  LaunchAttrs la;
  la.fill(cfg, static_cast<unsigned>(splits));
  if (cudaLaunchKernelEx(&cfg, kernel, maps, p) != cudaSuccess) {
    cudaGetLastError();
    return TG_ERR_LAUNCH;
  }
  return TG_OK;
}

// With adapters the host does not know how many there are among the rows: where
// each row has its own, both kernels compute their part outside the large tensor
// cores; where runs share one, the pair kernel has it on them.  So up to 96 rows, and
// 128 with long sums, take the narrow kernel, whose CTAs share that part as well (us,
// narrow / pair: 64 rows through 4096 x 4096, rank 64, 64 adapters 36 / 60, one 23 / 24;
// 128 rows 67 / 88 and 24 / 24; 96 rows through 512 x 512, rank 16, 32 / 43 and 18 / 13;
// 128 rows 38 / 37 and 22 / 12).  Where rows share one adapter that is the slower choice
// from about 96 rows on, which only the device could know.
bool grp_lora_narrow(const GrpProduct& f) { return f.a.rows <= 96 || (f.a.rows <= 128 && f.red > 31 * 64); }

// Splits of its sums then, of which there are at least two where it makes T itself.
int grp_lora_splits(const GrpProduct& f) { return f.red > 7 * 64 && f.out <= 40 * 128 ? 4 : 2; }

// Whether that kernel makes T itself, without a kernel before it: where that is a value
// at most for each warp that waits for the sums anyway, of which a cluster of two CTAs has
// 8 and one of four 16 (us, so / with the kernel before: one
// token through 4096 x 4096, rank 16, 12.6 / 13.5; with two values a warp 13.9 / 12.6,
// four 15 / 12.8).
bool grp_lora_own_t(const GrpProduct& f) {
  return grp_lora_narrow(f) && f.red > 64 && f.a.rows * f.l.rank <= GrpNarrowCfg::own_t(grp_lora_splits(f));
}

// Which kernel, by estimated time.
tg_status launch_grp(const GrpProduct& f, cudaStream_t stream, DeviceInfo* info) {
  const int64_t rows = f.a.rows, live = rows < f.groups ? rows : f.groups;  // groups that can have rows
  const int64_t each = (rows + live - 1) / live;
  const int k_blocks = static_cast<int>((f.red + 63) / 64);
  // Twice the even share, so that a group with more is one tile as a rule.
  int tokens = 16, splits = 1;
  while (tokens < 128 && tokens < (live > 1 ? 2 * each : each)) tokens <<= 1;
  bool narrow;
  if (f.lora && f.l.adapters > 0) {
    narrow = grp_lora_narrow(f);
    splits = grp_lora_splits(f);
  } else {
    double best = grp_narrow_us(f, live, k_blocks, tokens, 1, info);
    for (int s = 2; s <= 4 && s <= k_blocks; s *= 2) {
      const double us = grp_narrow_us(f, live, k_blocks, tokens, s, info);
      if (us < best) {
        best = us;
        splits = s;
      }
    }
    narrow = best < grp_pair_us(f, live, k_blocks, info);
  }
  if (tune_int("TG_TUNE_GRP_NARROW", narrow ? 1 : 0) == 0) return launch_grp_pair(f, stream, info);
  return launch_grp_narrow(f, tokens, splits, stream, info);
}

// A result that is a sum over nothing: +0 in the rows of the groups, or in all with `rest`.
struct GrpZeroParams {
  unsigned short* c;
  int64_t ldc;
  const int* ends;
  int groups, M, cols, rest;
};

__global__ void __launch_bounds__(256) grp_zero_kernel(const GrpZeroParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  int rows = p.rest ? p.M : 0;  // the greatest end
  for (int g = threadIdx.x & 31; !p.rest && g < p.groups; g += 32) rows = max(rows, grp_end(p.ends, g, p.M));
  rows = __reduce_max_sync(0xffffffffu, rows);
  const int64_t items = static_cast<int64_t>(rows) * p.cols;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < items;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t m = i / p.cols;
    p.c[m * p.ldc + (i - m * p.cols)] = 0;
  }
}

tg_status grp_zero(const FfMat& c, const int32_t* ends, int groups, bool rest, cudaStream_t stream, DeviceInfo* info) {
  if (c.empty() || (groups == 0 && !rest)) return TG_OK;
  if (rest) return ff_zero(c, stream);
  const GrpZeroParams p{static_cast<unsigned short*>(const_cast<void*>(c.p)), c.ld, ends, groups,
                        static_cast<int>(c.rows), static_cast<int>(c.cols), rest ? 1 : 0};
  return launch_simple(grp_zero_kernel, p, c.rows * c.cols, 1, stream, info);
}

// ---------------------------------------------------------------------------
// Grouped products
// ---------------------------------------------------------------------------
struct GroupedArgs {
  FfMat x, y, dx;  // y is dY in the backward pass
  GrpStack w, dw;
  int groups;
  int64_t M, N, K;
  bool bf16, rest;
};

bool grouped_args(GroupedArgs& a, const void* X, const void* W, const void* Y, const void* dX, const void* dW, int32_t G,
                  int64_t M, int64_t N, int64_t K, const tg_grouped_options* opt) {
  tg_grouped_options o;
  std::memset(&o, 0, sizeof o);
  if (opt) o = *opt;
  if (o.reserved != 0 || !ff_type_valid(o.type) || (o.rest != 0 && o.rest != 1) || !ff_sizes_valid(M, N, K) || G < 0 ||
      G > kGrpMaxGroups || G * N > kFfMaxSpan / (K > 0 ? K : 1))
    return false;
  if (o.ldx < 0 || o.ldw < 0 || o.ldy < 0 || o.stride_w < 0 || o.lddx < 0 || o.lddw < 0 || o.stride_dw < 0) return false;
  a.x = mat16(X, M, K, o.ldx);
  a.y = mat16(Y, M, N, o.ldy);
  a.dx = mat16(dX, M, K, o.lddx);
  a.w = grp_stack(W, G, N, K, o.ldw, o.stride_w);
  a.dw = grp_stack(dW, G, N, K, o.lddw, o.stride_dw);
  a.groups = G;
  a.M = M;
  a.N = N;
  a.K = K;
  a.bf16 = o.type == TG_TYPE_BF16;
  a.rest = o.rest != 0;
  return true;
}

int64_t grouped_workspace(const GroupedArgs& a) {
  if (a.M == 0 || a.N == 0 || a.K == 0 || a.groups == 0) return 0;
  const int64_t w = grp_copy_bytes(a.w);
  return w < 0 ? -1 : ff_copy_bytes(a.x) + w;
}

tg_status run_grouped(GroupedArgs& a, const int32_t* ends, void* stream_ptr, void* ws_ptr, int64_t ws_bytes) {
  if (a.M == 0 || a.N == 0) return TG_OK;
  const FfMat e = vec32(ends, a.groups);
  const int64_t need = grouped_workspace(a);
  if (!a.x.valid() || !a.w.valid(false) || !a.y.valid() || !e.valid() || need < 0) return TG_ERR_INVALID_ARG;
  const FfMat in[4] = {a.x, a.w.span(), e, a.y};
  if (!ff_disjoint(in, 3, &a.y, 1) || !ff_workspace_valid(ws_ptr, ws_bytes, need, in, 4)) return TG_ERR_INVALID_ARG;
  DeviceInfo* info = nullptr;
  tg_status st = grp_device(info);
  if (st != TG_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (a.K == 0 || a.groups == 0) return grp_zero(a.y, ends, a.groups, a.rest, stream, info);
  uint8_t* ws = static_cast<uint8_t*>(ws_ptr);
  if ((st = grp_make_copies(&a.x, nullptr, &a.w, ends, a.M, ws, stream, info)) != TG_OK) return st;
  GrpProduct f;
  f.a = a.x;
  f.c = a.y;
  f.w = a.w;
  f.ends = ends;
  f.groups = a.groups;
  f.out = a.N;
  f.red = a.K;
  f.rest = a.rest;
  f.bf16 = a.bf16;
  return launch_grp(f, stream, info);
}

int64_t grouped_grad_workspace(const GroupedArgs& a) {
  if (a.M == 0 || a.N == 0 || a.K == 0 || a.groups == 0) return 0;
  int64_t need = ff_copy_bytes(a.y);
  if (a.dx.p) {
    const int64_t w = grp_copy_bytes(a.w);
    if (w < 0) return -1;
    need += w;
  }
  return a.dw.m.p ? need + ff_copy_bytes(a.x) : need;
}

tg_status launch_grp_wgrad(const GroupedArgs& a, const int32_t* ends, cudaStream_t stream, DeviceInfo* info) {
  using Cfg = GrpWgradCfg;
  if (!ff_set_smem(reinterpret_cast<const void*>(grp_wgrad_kernel), info->grp_attr, 64u, Cfg::smem_bytes(kGrpMaxGroups)))
    return TG_ERR_LAUNCH;
  GrpWgradMaps maps;
  std::memset(&maps, 0, sizeof maps);
  if (!ff_encode(&maps.d, a.y, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !ff_encode(&maps.x, a.x, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return TG_ERR_LAUNCH;
  GrpWgradParams p;
  std::memset(&p, 0, sizeof p);
  p.c = const_cast<void*>(a.dw.m.p);
  p.ldc = a.dw.m.ld;
  p.stride_c = a.dw.stride;
  p.ends = ends;
  p.M = static_cast<int>(a.M);
  p.groups = a.groups;
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.n_tiles = (p.N + Cfg::TILE - 1) / Cfg::TILE;
  p.k_tiles = (p.K + Cfg::TILE - 1) / Cfg::TILE;
  const int64_t tiles = static_cast<int64_t>(p.n_tiles) * p.k_tiles * a.groups;
  if (tiles > INT_MAX - 65536) return TG_ERR_INVALID_ARG;
  p.num_tiles = static_cast<int>(tiles);
  p.vec = a.dw.on16() ? 1 : 0;
  if (p.vec && !grp_encode3(&maps.c, a.dw, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)) return TG_ERR_LAUNCH;
  p.bf16 = a.bf16 ? 1 : 0;
  p.idesc = make_idesc_ff(kFfF16, a.bf16, Cfg::TILE, Cfg::TILE, true, true);
  p.wait_budget_ns = wait_budget((a.M + 63) / 64);
  const int64_t pairs = info->sm_count / 2, clusters = tiles < pairs ? tiles : pairs;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters), 1, 1);
  cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(Cfg::smem_bytes(a.groups));
  cfg.stream = stream;
  LaunchAttrs la;
  la.fill(cfg, 2);
  if (cudaLaunchKernelEx(&cfg, grp_wgrad_kernel, maps, p) != cudaSuccess) {
    cudaGetLastError();
    return TG_ERR_LAUNCH;
  }
  return TG_OK;
}

// Every row of a stack's matrices set to +0.
tg_status grp_zero_stack(const GrpStack& s, cudaStream_t stream) {
  if (s.empty()) return TG_OK;
  if (s.even_rows()) return ff_zero(s.rows(), stream);
  for (int64_t g = 0; g < s.mats; ++g) {
    FfMat m = s.m;
    m.p = static_cast<const uint8_t*>(m.p) + 2 * g * s.stride;
    const tg_status st = ff_zero(m, stream);
    if (st != TG_OK) return st;
  }
  return TG_OK;
}

tg_status run_grouped_grad(GroupedArgs& a, const int32_t* ends, void* stream_ptr, void* ws_ptr, int64_t ws_bytes) {
  const bool want_x = a.dx.p != nullptr && !a.dx.empty(), want_w = a.dw.m.p != nullptr && !a.dw.empty();
  if (!want_x && !want_w) return TG_OK;
  const FfMat e = vec32(ends, a.groups);
  const int64_t need = grouped_grad_workspace(a);
  if (!a.x.valid() || !a.w.valid(false) || !a.y.valid() || !e.valid() || need < 0) return TG_ERR_INVALID_ARG;
  FfMat all[6] = {a.x, a.w.span(), e, a.y};
  int n = 4;
  if (want_x) {
    if (!a.dx.valid()) return TG_ERR_INVALID_ARG;
    all[n++] = a.dx;
  }
  if (want_w) {
    if (!a.dw.valid(true)) return TG_ERR_INVALID_ARG;
    all[n++] = a.dw.span();
  }
  if (!ff_disjoint(all, 4, all + 4, n - 4) || !ff_workspace_valid(ws_ptr, ws_bytes, need, all, n)) return TG_ERR_INVALID_ARG;
  DeviceInfo* info = nullptr;
  tg_status st = grp_device(info);
  if (st != TG_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (a.M == 0 || a.N == 0 || a.groups == 0) {  // sums over nothing
    if (want_w && (st = grp_zero_stack(a.dw, stream)) != TG_OK) return st;
    return want_x ? grp_zero(a.dx, ends, a.groups, a.rest, stream, info) : TG_OK;
  }
  uint8_t* ws = static_cast<uint8_t*>(ws_ptr);
  if ((st = grp_make_copies(&a.y, want_w ? &a.x : nullptr, want_x ? &a.w : nullptr, ends, a.M, ws, stream, info)) != TG_OK) return st;
  if (want_w && (st = launch_grp_wgrad(a, ends, stream, info)) != TG_OK) return st;
  if (!want_x) return TG_OK;
  GrpProduct f;
  f.a = a.y;
  f.c = a.dx;
  f.w = a.w;
  f.ends = ends;
  f.groups = a.groups;
  f.out = a.K;
  f.red = a.N;
  f.transposed = true;
  f.beside = want_w && tune_int("TG_TUNE_GRP_BESIDE", 1) != 0;
  f.rest = a.rest;
  f.bf16 = a.bf16;
  return launch_grp(f, stream, info);
}

// ---------------------------------------------------------------------------
// Adapters
// ---------------------------------------------------------------------------
struct LoraArgs {
  FfMat x, w, y;
  GrpStack a, b;
  int64_t M, N, K, rank, adapters;
  bool bf16;
};

bool lora_args(LoraArgs& l, const void* X, const void* W, const void* A, const void* B, const void* Y, int64_t M, int64_t N,
               int64_t K, int64_t rank, int64_t adapters, const tg_lora_options* opt) {
  tg_lora_options o;
  std::memset(&o, 0, sizeof o);
  if (opt) o = *opt;
  if (o.reserved != 0 || !ff_type_valid(o.type) || !ff_sizes_valid(M, N, K) || rank < 0 || rank > kLoraMaxRank ||
      rank % 8 != 0 || adapters < 0 || adapters > kLoraMaxAdapters)
    return false;
  if (o.ldx < 0 || o.ldw < 0 || o.ldy < 0 || o.lda < 0 || o.stride_a < 0 || o.ldb < 0 || o.stride_b < 0) return false;
  if (rank == 0) adapters = 0;
  l.x = mat16(X, M, K, o.ldx);
  l.w = mat16(W, N, K, o.ldw);
  l.y = mat16(Y, M, N, o.ldy);
  l.a = grp_stack(A, adapters, rank, K, o.lda, o.stride_a);
  l.b = grp_stack(B, adapters, N, rank, o.ldb, o.stride_b);
  l.M = M;
  l.N = N;
  l.K = K;
  l.rank = rank;
  l.adapters = adapters;
  l.bf16 = o.type == TG_TYPE_BF16;
  return true;
}

// T, and behind it what stands beside it: the kinds of 32 rows and, in fp16, a byte
// of power for each row and eight ranks and, before those, the misfits of 32 rows.
struct LoraInner {
  int64_t kind, misfits, exps, bytes;  // from T's start
};
LoraInner lora_inner(const LoraArgs& l) {
  LoraInner n{0, 0, 0, 0};
  if (l.adapters == 0) return n;
  const int64_t blocks = (l.M + 31) / 32;
  n.kind = up256(2 * l.M * l.rank);
  n.misfits = n.kind + round_up(4 * blocks, 8);
  n.exps = n.misfits + 8 * blocks * ((l.rank + 127) / 128);
  n.bytes = n.kind + up256(l.bf16 ? 4 * blocks : n.exps + l.M * (l.rank / 8) - n.kind);
  return n;
}

int64_t lora_workspace(const LoraArgs& l) {
  if (l.M == 0 || l.N == 0 || l.K == 0) return 0;
  return lora_inner(l).bytes + ff_copy_bytes(l.x) + ff_copy_bytes(l.w);
}

// T of few tokens.
tg_status launch_lora_rows(const LoraArgs& l, const GrpProduct& f, const float* scale, cudaStream_t stream) {
  LoraRowsParams p;
  std::memset(&p, 0, sizeof p);
  p.x = l.x.p;
  p.a = l.a.m.p;
  p.index = f.l.index;
  p.scale = scale;
  p.t = const_cast<void*>(f.l.t);
  p.exps = const_cast<signed char*>(f.l.exps);
  p.ldx = l.x.ld;
  p.lda = l.a.m.ld;
  p.stride_a = l.a.stride;
  p.K = static_cast<int>(l.K);
  p.rank = static_cast<int>(l.rank);
  p.adapters = static_cast<int>(l.adapters);
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(l.M), static_cast<unsigned>((l.rank + kLoraRowsWarps - 1) / kLoraRowsWarps), 1);
  cfg.blockDim = dim3(kLoraRowsWarps * 32, 1, 1);
  cfg.stream = stream;
  LaunchAttrs la;
  la.fill(cfg, 1);
  if (cudaLaunchKernelEx(&cfg, l.bf16 ? lora_rows_kernel<true> : lora_rows_kernel<false>, p) != cudaSuccess) {
    cudaGetLastError();
    return TG_ERR_LAUNCH;
  }
  return TG_OK;
}

// T and the kinds of 32 tokens.
tg_status launch_lora_shrink(const LoraArgs& l, const GrpProduct& f, const float* scale, cudaStream_t stream, DeviceInfo* info) {
  using Cfg = LoraShrinkCfg;
  auto kernel = l.bf16 ? lora_shrink_kernel<true> : lora_shrink_kernel<false>;
  if (!ff_set_smem(reinterpret_cast<const void*>(kernel), info->grp_attr, l.bf16 ? 128u : 256u, 210 * 1024)) return TG_ERR_LAUNCH;
  LoraShrinkMaps maps;
  std::memset(&maps, 0, sizeof maps);
  LoraShrinkParams p;
  std::memset(&p, 0, sizeof p);
  p.a_rows = static_cast<int>(l.rank < 128 ? l.rank : 128);
  if (!grp_encode3(&maps.a, l.a, 64, p.a_rows)) return TG_ERR_LAUNCH;
  p.index = f.l.index;
  p.scale = scale;
  p.t = const_cast<void*>(f.l.t);
  p.kind = const_cast<int*>(f.l.kind);
  p.exps = const_cast<signed char*>(f.l.exps);
  p.misfits = reinterpret_cast<uint8_t*>(const_cast<uint2*>(f.l.misfits));
  p.M = static_cast<int>(l.M);
  p.rank = static_cast<int>(l.rank);
  p.adapters = static_cast<int>(l.adapters);
  p.k_blocks = static_cast<int>((l.K + 63) / 64);
  // Small blocks where large ones would leave SMs without one.
  p.tokens = l.M <= 32 * info->sm_count / 4 ? 32 : l.M <= 64 * info->sm_count ? 64 : 128;
  for (int i = 0; i < 4 && 16 << i <= p.tokens; ++i)
    if (!ff_encode(&maps.x[i], l.x, 64, 16 << i, CU_TENSOR_MAP_SWIZZLE_128B)) return TG_ERR_LAUNCH;
  const int64_t blocks = (l.M + p.tokens - 1) / p.tokens;
  const int64_t deep = (l.rank + 127) / 128;
  // Two splits where that leaves SMs for both; four made the exchange between them dearer
  // than what they saved (1049 rows of 40 requests, K = 2048, rank 32: 53.7 us against
  // 58.2; 200 rows of one, K = 8192, rank 64: 42.5 / 46.9; no split 54.4 and 44.2).
  p.splits = p.k_blocks >= 4 && blocks * deep * 2 <= info->sm_count ? 2 : 1;
  // Clusters for the items of a block, as many as it may have, for four times the SMs at
  // most: a batch of 60 adapters behind a prompt needs them (2048 rows: 195 us with
  // half as many, 127 so), and one without an item costs a little (512 rows of 4
  // requests through 4096 x 1024: 31.2 us, 28.9 with half as many, 33.9 with more).
  int64_t y = 4 * info->sm_count / (blocks * deep * p.splits);
  y = y < 1 ? 1 : y > p.tokens ? p.tokens : y;
  y = y > l.adapters ? l.adapters : y;
  const int deepest = (96 * 1024 - 1024 - Cfg::BAR_BYTES - Cfg::recv_bytes(p.tokens, p.splits, p.a_rows)) / ((p.a_rows + p.tokens) * 128);
  p.per_stage = tune_int("TG_TUNE_SHRINK_PER", 2);
  while (p.per_stage > 1 && deepest < 4 * p.per_stage) p.per_stage >>= 1;
  p.stages = deepest / p.per_stage;
  if (p.stages > Cfg::MAX_STAGES) p.stages = Cfg::MAX_STAGES;
  if (p.stages < 2) p.stages = 2;
  p.tmem_cols = p.tokens;
  p.idesc = make_idesc_ff(kFfF16, l.bf16, 128, 0, false, false);
  p.wait_budget_ns = wait_budget(p.k_blocks);
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * p.splits), static_cast<unsigned>(y), static_cast<unsigned>(deep));
  cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(Cfg::smem_bytes(p.tokens, p.splits, p.a_rows, p.stages * p.per_stage));
  cfg.stream = stream;
  LaunchAttrs la;
  la.fill(cfg, static_cast<unsigned>(p.splits));
  if (cudaLaunchKernelEx(&cfg, kernel, maps, p) != cudaSuccess) {
    cudaGetLastError();
    return TG_ERR_LAUNCH;
  }
  return TG_OK;
}

tg_status run_lora(LoraArgs& l, const float* scale, const int32_t* index, const void* bias, void* stream_ptr, void* ws_ptr,
                   int64_t ws_bytes) {
  if (l.M == 0 || l.N == 0) return TG_OK;
  const bool adapted = l.adapters > 0 && l.K > 0;
  const int64_t need = lora_workspace(l);
  const FfMat s = vec32(scale, scale ? l.adapters : 0), i = vec32(index, adapted ? l.M : 0);
  const FfMat bv = mat16(bias, bias ? 1 : 0, l.N, l.N);
  if (!l.x.valid() || !l.w.valid() || !l.y.valid() || !s.valid() || !i.valid() || !bv.valid()) return TG_ERR_INVALID_ARG;
  if (adapted && (!l.a.valid(false) || !l.b.valid(false) || !l.a.on16() || !l.b.on16())) return TG_ERR_INVALID_ARG;
  FfMat all[8] = {l.x, l.w, s, i, bv, l.y, l.a.span(), l.b.span()};
  if (!adapted) all[6] = all[7] = FfMat{nullptr, 0, 0, 1, 2};
  for (int q = 0; q < 8; ++q)
    if (q != 5 && l.y.overlaps(all[q])) return TG_ERR_INVALID_ARG;
  if (!ff_workspace_valid(ws_ptr, ws_bytes, need, all, 8)) return TG_ERR_INVALID_ARG;
  DeviceInfo* info = nullptr;
  tg_status st = grp_device(info);
  if (st != TG_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (l.K == 0) {
    const BiasFillParams b{const_cast<void*>(l.y.p), bias, l.y.ld, static_cast<int>(l.M), static_cast<int>(l.N), 0, l.bf16 ? 1 : 0};
    return launch_simple(bias_fill_kernel, b, l.M * l.N, 1, stream, info);
  }
  uint8_t* ws = static_cast<uint8_t*>(ws_ptr);
  GrpProduct f;
  std::memset(&f.l, 0, sizeof f.l);
  f.lora = true;
  f.l.bias = bias;
  if (adapted) {
    f.l.index = index;
    f.l.t = ws;
    const LoraInner inner = lora_inner(l);
    f.l.kind = reinterpret_cast<const int*>(ws + inner.kind);
    f.l.misfits = reinterpret_cast<const uint2*>(ws + inner.misfits);
    f.l.exps = reinterpret_cast<const signed char*>(ws + inner.exps);
    f.l.deep = static_cast<int>((l.rank + 127) / 128);
    f.l.b = l.b.m.p;
    f.l.ldb = l.b.m.ld;
    f.l.stride_b = l.b.stride;
    f.l.rank = static_cast<int>(l.rank);
    f.l.adapters = static_cast<int>(l.adapters);
    f.lb = l.b;
    f.t = FfMat{ws, l.M, l.rank, l.rank, 2};
    ws += inner.bytes;
  }
  FfMat* const operands[2] = {&l.x, &l.w};
  if ((st = ff_make_copies(operands, 2, ws, stream, info)) != TG_OK) return st;
  f.a = l.x;
  f.c = l.y;
  f.w = GrpStack{l.w, 1, 0};
  f.out = l.N;
  f.red = l.K;
  f.bf16 = l.bf16;
  if (adapted) {
    if (grp_lora_own_t(f)) {
      f.l.t = nullptr;
      f.l.x = l.x.p;
      f.l.ldx = l.x.ld;
      f.l.a = l.a.m.p;
      f.l.lda = l.a.m.ld;
      f.l.stride_a = l.a.stride;
      f.l.scale = scale;
    } else {
      st = grp_lora_narrow(f) ? launch_lora_rows(l, f, scale, stream) : launch_lora_shrink(l, f, scale, stream, info);
      if (st != TG_OK) return st;
    }
  }
  return launch_grp(f, stream, info);
}

}  // namespace
}  // namespace tg

extern "C" {

tg_status tg_grouped(const void* X, const void* W, const int32_t* ends, void* Y, int32_t groups, int64_t M, int64_t N,
                     int64_t K, const tg_grouped_options* options, void* stream, void* workspace,
                     int64_t workspace_bytes) {
  tg::GroupedArgs a;
  if (!tg::grouped_args(a, X, W, Y, nullptr, nullptr, groups, M, N, K, options)) return TG_ERR_INVALID_ARG;
  return tg::run_grouped(a, ends, stream, workspace, workspace_bytes);
}

int64_t tg_grouped_workspace_size(const void* X, const void* W, int32_t groups, int64_t M, int64_t N, int64_t K,
                                  const tg_grouped_options* options) {
  tg::GroupedArgs a;
  if (!tg::grouped_args(a, X, W, nullptr, nullptr, nullptr, groups, M, N, K, options)) return -1;
  return tg::grouped_workspace(a);
}

tg_status tg_grouped_backward(const void* dY, const void* X, const void* W, const int32_t* ends, void* dX, void* dW,
                              int32_t groups, int64_t M, int64_t N, int64_t K, const tg_grouped_options* options,
                              void* stream, void* workspace, int64_t workspace_bytes) {
  tg::GroupedArgs a;
  if (!tg::grouped_args(a, X, W, dY, dX, dW, groups, M, N, K, options)) return TG_ERR_INVALID_ARG;
  return tg::run_grouped_grad(a, ends, stream, workspace, workspace_bytes);
}

int64_t tg_grouped_backward_workspace_size(const void* dY, const void* X, const void* W, const void* dX, const void* dW,
                                           int32_t groups, int64_t M, int64_t N, int64_t K,
                                           const tg_grouped_options* options) {
  tg::GroupedArgs a;
  if (!tg::grouped_args(a, X, W, dY, dX, dW, groups, M, N, K, options)) return -1;
  return tg::grouped_grad_workspace(a);
}

tg_status tg_lora(const void* X, const void* W, const void* A, const void* B, const float* scale, const int32_t* index,
                  const void* bias, void* Y, int64_t M, int64_t N, int64_t K, int64_t rank, int64_t adapters,
                  const tg_lora_options* options, void* stream, void* workspace, int64_t workspace_bytes) {
  tg::LoraArgs l;
  if (!tg::lora_args(l, X, W, A, B, Y, M, N, K, rank, adapters, options)) return TG_ERR_INVALID_ARG;
  return tg::run_lora(l, scale, index, bias, stream, workspace, workspace_bytes);
}

int64_t tg_lora_workspace_size(const void* X, const void* W, int64_t M, int64_t N, int64_t K, int64_t rank, int64_t adapters,
                               const tg_lora_options* options) {
  tg::LoraArgs l;
  if (!tg::lora_args(l, X, W, nullptr, nullptr, nullptr, M, N, K, rank, adapters, options)) return -1;
  return tg::lora_workspace(l);
}

}  // extern "C"
