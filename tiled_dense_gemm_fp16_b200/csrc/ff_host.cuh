// ff_host.cuh -- argument checks, kernel choice and launches of the
// feed-forward operators: the gated block and its gradients, row quantization
// and the 8-bit products.  Included by tg_gemm.cu after its shared helpers.
#pragma once

#include "ff_rows.cuh"
#include "gemm_ff_pair.cuh"
#include "gemm_ff_skinny.cuh"

namespace tg {
namespace {

constexpr int64_t kFfMaxSize = int64_t(1) << 30;    // M, N, K: tile coordinates stay in 32 bits
constexpr int64_t kFfMaxSpan = int64_t(1) << 50;    // elements of a matrix, gaps included: byte counts stay in 64 bits
constexpr int64_t kFfMaxStride = int64_t(1) << 38;  // elements: byte strides stay below TMA's 2^40
constexpr int64_t kFfMaxKI8 = 131071;               // 2^31 / 128^2: a sum of products of two codes stays in 32 bits

// A row-major matrix of the caller (or of the workspace): elements of `elem` bytes.
struct FfMat {
  const void* p;
  int64_t rows, cols, ld;
  int elem;

  bool empty() const { return rows == 0 || cols == 0; }
  int64_t bytes() const { return empty() ? 0 : elem * ((rows - 1) * ld + cols); }  // of a valid matrix
  bool rows_on(int align) const {  // every row starts on a multiple of `align` bytes
    return (reinterpret_cast<uintptr_t>(p) % align) == 0 && (ld * elem) % align == 0;
  }
  // Pointer, alignment and stride of a matrix that is read or written.
  bool valid() const {
    if (empty()) return true;
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) % elem) == 0 && ld >= cols && ld <= kFfMaxStride &&
           rows <= kFfMaxSpan / ld;
  }
  // Any byte of both.  Where their ranges meet, rows of one may still lie in the
  // gaps between the other's (column ranges of one wider buffer): both repeat
  // with the same pitch, and their columns are disjoint within it.
  bool overlaps(const FfMat& o) const {
    if (!ranges_overlap(p, bytes(), o.p, o.bytes())) return false;
    const int64_t mine = ld * elem, other = o.ld * o.elem, pitch = rows > 1 ? mine : other;
    if ((rows > 1 && o.rows > 1 && mine != other) || (rows <= 1 && o.rows <= 1)) return true;
    int64_t at = (reinterpret_cast<intptr_t>(o.p) - reinterpret_cast<intptr_t>(p)) % pitch;
    at = at < 0 ? at + pitch : at;
    return at < cols * elem || at + o.cols * o.elem > pitch;
  }
};

// The caller's matrix; ld 0 means dense rows.  A single row has no stride, so
// it gets one that any tensor map takes.
FfMat ff_mat(const void* p, int64_t rows, int64_t cols, int64_t ld, int elem) {
  if (rows == 1 && cols <= kFfMaxSize && (ld == 0 || ld >= cols)) ld = (cols + 15) / 16 * 16;
  return FfMat{p, rows, cols, ld ? ld : cols, elem};
}
FfMat mat16(const void* p, int64_t rows, int64_t cols, int64_t ld) { return ff_mat(p, rows, cols, ld, 2); }
FfMat mat8(const void* p, int64_t rows, int64_t cols, int64_t ld) { return ff_mat(p, rows, cols, ld, 1); }
FfMat vec32(const void* p, int64_t n) { return FfMat{p, n > 0 ? 1 : 0, n, n, 4}; }

bool ff_sizes_valid(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && K >= 0 && M <= kFfMaxSize && N <= kFfMaxSize && K <= kFfMaxSize &&
         M * N <= kFfMaxSpan && N * K <= kFfMaxSpan && M * K <= kFfMaxSpan;
}
bool ff_type_valid(int32_t t) { return t == TG_TYPE_F16 || t == TG_TYPE_BF16; }
bool ff_act_valid(int32_t a) { return a == TG_ACT_RELU || a == TG_ACT_SILU || a == TG_ACT_GELU; }

// No result overlaps an input or another result.
bool ff_disjoint(const FfMat* in, int n_in, const FfMat* out, int n_out) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (out[i].overlaps(in[j])) return false;
    for (int j = 0; j < i; ++j)
      if (out[i].overlaps(out[j])) return false;
  }
  return true;
}

// Tensor map of a matrix: boxes of box_cols x box_rows elements, rows and
// columns past the matrix read as zero and are not written.
bool ff_encode(CUtensorMap* map, const FfMat& m, int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(m.cols), static_cast<cuuint64_t>(m.rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(m.ld) * m.elem};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estride[2] = {1, 1};
  return fn(map, m.elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(m.p), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One product of the feed-forward kernels.
//   gated:        c[0] (and c[1], c[2] when saved) = act(a[0] b[0]^T) * (a[0] b[1]^T)
//   k_sources 2:  c[0] = a[0] b[0] + a[1] b[1]
//   row_sources 2: c[i] = a[i] . b[0]
// A is M x K (or K x M with a_km), B is N x K (or K x N with b_kn).
struct FfProduct {
  int kind = kFfF16;
  bool gated = false, save = false;
  FfMat a[2], b[2], c[3];
  bool a_km = false, b_kn = false;
  int k_sources = 1, row_sources = 1;
  int64_t M = 0, N = 0, K = 0;  // of one source
  const float* row_scale = nullptr;
  const float* col_scale[2] = {nullptr, nullptr};
  const void* bias = nullptr;
  bool bf16 = false;
  int act = 0, relu = 0;

  int results() const { return gated ? (save ? 3 : 1) : row_sources; }
  int weights() const { return gated ? 2 : k_sources; }
  int k_elems() const { return kind == kFfI8 ? 128 : 64; }
};

bool ff_set_smem(const void* kernel, unsigned& done, unsigned bit, int bytes) {
  std::lock_guard<std::mutex> lock(g_mutex);
  if (done & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done |= bit;
  return true;
}

template <int STAGES, int BN, int EPI_WARPS, int KIND, bool GATED>
tg_status launch_ff_pair_cfg(const FfProduct& f, cudaStream_t stream, DeviceInfo* info) {
  using Cfg = FfPairCfg<STAGES, BN, EPI_WARPS>;
  auto kernel = ff_pair_kernel<STAGES, BN, EPI_WARPS, KIND, GATED>;
  constexpr unsigned kBit = 1u << (BN / 256 + (KIND == kFfI8 ? 3 : 0) + (GATED ? 6 : 0));
  if (!ff_set_smem(reinterpret_cast<const void*>(kernel), info->ff_attr, kBit, Cfg::SMEM_BYTES)) return TG_ERR_LAUNCH;
  FfMaps maps;
  std::memset(&maps, 0, sizeof maps);
  FfParams p;
  std::memset(&p, 0, sizeof p);
  const int ke = f.k_elems();
  const int a_sources = f.k_sources > f.row_sources ? f.k_sources : f.row_sources;
  for (int i = 0; i < a_sources; ++i)
    if (!ff_encode(&maps.a[i], f.a[i], f.a_km ? 64 : ke, f.a_km ? 64 : Cfg::BM, CU_TENSOR_MAP_SWIZZLE_128B))
      return TG_ERR_LAUNCH;
  for (int i = 0; i < f.weights(); ++i)
    if (!ff_encode(&maps.b[i], f.b[i], f.b_kn ? 64 : ke, f.b_kn ? 64 : (GATED ? Cfg::B_ROWS / 2 : Cfg::B_ROWS), CU_TENSOR_MAP_SWIZZLE_128B))
      return TG_ERR_LAUNCH;
  for (int i = 0; i < f.results(); ++i) {
    p.c[i] = const_cast<void*>(f.c[i].p);
    p.ldc[i] = f.c[i].ld;
    p.c_aligned[i] = f.c[i].rows_on(16) ? 1 : 0;
    if (p.c_aligned[i] && !ff_encode(&maps.c[i], f.c[i], 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)) return TG_ERR_LAUNCH;
  }
  const int tile_n = GATED ? BN / 2 : BN;
  p.row_scale = f.row_scale;
  p.col_scale[0] = f.col_scale[0];
  p.col_scale[1] = f.col_scale[1];
  p.bias = f.bias;
  p.M = static_cast<int>(f.M);
  p.N = static_cast<int>(f.N);
  p.m_tiles_src = static_cast<int>((f.M + Cfg::PAIR_M - 1) / Cfg::PAIR_M);
  p.m_tiles = p.m_tiles_src * f.row_sources;
  p.n_tiles = static_cast<int>((f.N + tile_n - 1) / tile_n);
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  p.k_blocks_src = static_cast<int>((f.K + ke - 1) / ke);
  p.k_blocks = p.k_blocks_src * f.k_sources;
  p.group_m = BN == 512 ? 16 : 12;
  if (tiles > INT_MAX - 65536 || static_cast<int64_t>(p.group_m) * p.n_tiles > INT_MAX) return TG_ERR_INVALID_ARG;
  const int pairs = info->sm_count / 2;
  // Whole waves of whole tiles; what is left over, if it fits in one wave of
  // half tiles, runs as those (half the time of a last wave of whole tiles).
  const int rest = static_cast<int>(tiles % pairs);
  const bool halves = Cfg::SLABS == 2 && 2 * rest <= pairs;
  p.whole_tiles = static_cast<int>(halves ? tiles - rest : tiles);
  p.num_tiles = static_cast<int>(halves ? tiles + rest : tiles);
  p.a_mnmajor = f.a_km ? 1 : 0;
  p.b_kmajor = f.b_kn ? 0 : 1;
  p.bf16 = f.bf16 ? 1 : 0;
  p.act = f.act;
  p.relu = f.relu;
  p.save = f.save ? 1 : 0;
  p.l2_hints = BN == 512 ? 2 : 5;
  p.idesc = make_idesc_ff(KIND, f.bf16, Cfg::PAIR_M, Cfg::SLAB, f.a_km, f.b_kn);
  p.wait_budget_ns = wait_budget(p.k_blocks);
  const int clusters = p.num_tiles < pairs ? p.num_tiles : pairs;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters), 1, 1);
  cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(Cfg::SMEM_BYTES);
  cfg.stream = stream;
  LaunchAttrs la;
  la.fill(cfg, 2);
  if (cudaLaunchKernelEx(&cfg, kernel, maps, p) != cudaSuccess) {
    cudaGetLastError();
    return TG_ERR_LAUNCH;
  }
  return TG_OK;
}

template <int KIND, bool GATED>
tg_status launch_ff_pair(const FfProduct& f, int bn, cudaStream_t stream, DeviceInfo* info) {
  switch (bn) {
    case 512: return launch_ff_pair_cfg<4, 512, 16, KIND, GATED>(f, stream, info);
    case 256: return launch_ff_pair_cfg<6, 256, 16, KIND, GATED>(f, stream, info);
    default: return launch_ff_pair_cfg<8, 128, 8, KIND, GATED>(f, stream, info);
  }
}

// ---------------------------------------------------------------------------
// Small-M kernel
// ---------------------------------------------------------------------------
using FfSkinnyKernel = void (*)(FfMaps, FfSkinnyParams);

int ff_skinny_index(const FfProduct& f) { return (f.kind == kFfI8 ? 1 : 0) + (f.gated ? 2 : 0); }

FfSkinnyKernel ff_skinny_kernel_of(const FfProduct& f) {
  if (f.kind == kFfI8) return f.gated ? ff_skinny_kernel<kFfI8, true> : ff_skinny_kernel<kFfI8, false>;
  return f.gated ? ff_skinny_kernel<kFfF16, true> : ff_skinny_kernel<kFfF16, false>;
}

struct FfSkinnyPlan {
  int m_pad, m_blocks, a_bytes, stages, smem, k_blocks, splits;
  int64_t panels, waves;
  double us;  // estimated time
};

// Clusters of `splits` CTAs that fit on the device with one CTA per SM, asked
// of the runtime once per number of splits (for the largest launch, whose
// shared memory allows one): GPCs hold different numbers of SMs, so there is no
// formula (a B200 gave 148, 74, 45, 33, 26, 22, 15, 15 for 1 .. 8).
int ff_resident_clusters(const FfProduct& f, int splits, DeviceInfo* info) {
  std::lock_guard<std::mutex> lock(g_mutex);
  short& known = info->ff_clusters[splits];
  if (known == 0) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(splits), 1024, 1);
    cfg.blockDim = dim3(FfSkinnyCfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(FfSkinnyCfg::MAX_SMEM);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(splits);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, ff_skinny_kernel_of(f), &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = info->sm_count / splits > 0 ? info->sm_count / splits : 1;
    }
    known = static_cast<short>(n > 32767 ? 32767 : n);
  }
  return known;
}

// The plan of a product in blocks of at most `block_rows` rows, or false if the
// kernel cannot take it.  Splits of K, by estimated time in us: at most as many
// as give every SM two CTAs (one where two do not fit).  One block of rows: a
// k-block takes 0.59 with one CTA per SM and 0.72 with two (the weight's stream
// from memory), a wave 1.5 for its start, a second CTA per SM 1.5 + M / 40 more
// for the partials both have to move and add.  Measured, us, gated fp16 N = K =
// 2048 with 4 / 8 splits: M = 128 9.4 / 12.2, M = 1 6.0 / 6.0; 4096 with 2 / 4: M
// = 128 19.4 / 16.8; 8-bit 5120 at M = 128 with 4 in one wave / 7 that do not
// quite fit: 13 / 21.  Several blocks read the operands from L2: 0.31 with one
// CTA per SM, 0.44 with two, for blocks of 128 rows (a CTA takes in 32 KiB), 0.11
// more with rows stored K x M, and 2 for a second CTA; in between where some SMs
// have two (dX of 152 x 3344 x 896: 16 clusters of 8, one more than fit alone,
// 12.7, of 6 14.2).  Measured, gated fp16
// 1024 x 1024 x 8192 with 1 / 2 splits 44 / 35, 512 x 1024 x 2048 11.7 with 2.
bool ff_skinny_plan(const FfProduct& f, int block_rows, DeviceInfo* info, FfSkinnyPlan* out) {
  using Cfg = FfSkinnyCfg;
  if (!ff_set_smem(reinterpret_cast<const void*>(ff_skinny_kernel_of(f)), info->ff_attr, 1u << (12 + ff_skinny_index(f)),
                   Cfg::MAX_SMEM))
    return false;
  FfSkinnyPlan pl;
  const int64_t m_blocks = (f.M + block_rows - 1) / block_rows;
  if (m_blocks * f.row_sources > 65535) return false;
  pl.m_blocks = static_cast<int>(m_blocks);
  const int unit = f.a_km ? 64 : 16;  // rows stored K x M come in whole panels
  pl.m_pad = static_cast<int>(((f.M + m_blocks - 1) / m_blocks + unit - 1) / unit * unit);
  pl.a_bytes = Cfg::a_bytes(pl.m_pad, f.a_km);
  const int64_t kb = (f.K + f.k_elems() - 1) / f.k_elems() * f.k_sources;
  const int cols = f.gated ? 64 : 128;
  pl.panels = (f.N + cols - 1) / cols;
  if (kb > INT_MAX || pl.panels > 65535) return false;
  pl.k_blocks = static_cast<int>(kb);
  const int stage_bytes = Cfg::W_STAGE_BYTES + pl.a_bytes;
  pl.stages = Cfg::stages(pl.m_pad, f.a_km);
  // The partial [m_pad][128] reuses the ring after the main loop.
  if (pl.stages < 2 || pl.stages * stage_bytes < pl.m_pad * Cfg::PANEL * 4) return false;
  pl.smem = Cfg::smem_bytes(pl.a_bytes, pl.stages);
  double best = 0.0;
  pl.splits = 0;
  const int per_sm = Cfg::ctas_per_sm(pl.m_pad);
  const int64_t slots = per_sm * info->sm_count;
  const int64_t tiles = pl.panels * pl.m_blocks * f.row_sources;
  const int64_t most = tiles >= slots ? 1 : slots / tiles;
  const bool from_l2 = f.a_km || pl.m_blocks > 1;
  for (int s = 1; s <= 8 && s <= most && s <= pl.k_blocks; ++s) {
    const int64_t resident = per_sm * ff_resident_clusters(f, s, info);
    const int64_t waves = (tiles + resident - 1) / resident;
    const double alone = static_cast<double>(ff_resident_clusters(f, s, info));
    const bool second = static_cast<double>(tiles) > alone;
    double per_block = second ? 0.72 : 0.59, share = second ? 1.5 + pl.m_pad / 40.0 : 0.0;
    if (from_l2) {
      const double part = !second ? 0.0 : tiles < 2 * alone ? tiles / alone - 1.0 : 1.0;  // SMs with two
      per_block = (0.31 + 0.13 * part + (f.a_km ? 0.11 : 0.0)) * (128 + pl.m_pad) / 256.0;
      share = 2.0 * part;
    }
    const double cost = static_cast<double>(waves) * ((pl.k_blocks + s - 1) / s * per_block + 1.5) + share + 0.05 * s;
    if (pl.splits == 0 || cost < best) {
      best = cost;
      pl.splits = s;
      pl.waves = waves;
    }
  }
  const double rows = static_cast<double>(f.M);
  pl.us = from_l2 ? best + 5.0
                  : 6.0 + rows / 64.0 + static_cast<double>(pl.waves) * ((pl.k_blocks + pl.splits - 1) / pl.splits) *
                                            (0.2 + 0.3 * rows / 256.0);
  *out = pl;
  return true;
}

tg_status launch_ff_skinny(const FfProduct& f, const FfSkinnyPlan& pl, cudaStream_t stream) {
  using Cfg = FfSkinnyCfg;
  const int ke = f.k_elems();
  FfSkinnyParams p;
  std::memset(&p, 0, sizeof p);
  for (int i = 0; i < f.results(); ++i) {
    p.c[i] = const_cast<void*>(f.c[i].p);
    p.ldc[i] = f.c[i].ld;
    p.c_aligned[i] = f.c[i].rows_on(8) ? 1 : 0;
  }
  p.row_scale = f.row_scale;
  p.col_scale[0] = f.col_scale[0];
  p.col_scale[1] = f.col_scale[1];
  p.bias = f.bias;
  p.M = static_cast<int>(f.M);
  p.N = static_cast<int>(f.N);
  p.m_pad = pl.m_pad;
  p.m_blocks = pl.m_blocks;
  p.k_blocks_src = pl.k_blocks / f.k_sources;
  p.k_blocks = pl.k_blocks;
  p.stages = pl.stages;
  p.splits = pl.splits;
  p.a_stage_bytes = static_cast<uint32_t>(pl.a_bytes);
  uint32_t cols = 32;
  while (cols < static_cast<uint32_t>(p.m_pad)) cols <<= 1;
  p.tmem_cols = cols;
  p.idesc = make_idesc_ff(f.kind, f.bf16, Cfg::PANEL, p.m_pad, f.b_kn, f.a_km);
  p.a_mnmajor = f.a_km ? 1 : 0;
  p.b_kmajor = f.b_kn ? 0 : 1;
  p.bf16 = f.bf16 ? 1 : 0;
  p.act = f.act;
  p.relu = f.relu;
  p.save = f.save ? 1 : 0;
  // Four k-blocks ahead where a CTA streams 16 or more of two weights (32 of
  // one).  Measured back to back, us, without / with: gated 64 x 8192 x 8192 49.2
  // / 46.7, 8-bit gated 64 x 8192 x 4096 17.1 / 15.9; 8-bit 16 x 8192 x 8192 (16
  // of one weight) 14.7 / 15.2.
  p.prefetch_kb = p.k_blocks / p.splits >= (f.gated ? 16 : 32) ? 4 : 0;
  p.wait_budget_ns = wait_budget(p.k_blocks);
  FfMaps maps;
  std::memset(&maps, 0, sizeof maps);
  const int a_sources = f.k_sources > f.row_sources ? f.k_sources : f.row_sources;
  for (int i = 0; i < a_sources; ++i)
    if (!ff_encode(&maps.a[i], f.a[i], f.a_km ? 64 : ke, f.a_km ? 64 : p.m_pad, CU_TENSOR_MAP_SWIZZLE_128B))
      return TG_ERR_LAUNCH;
  for (int i = 0; i < f.weights(); ++i)
    if (!ff_encode(&maps.b[i], f.b[i], f.b_kn ? 64 : ke, f.b_kn || f.gated ? 64 : Cfg::PANEL,
                   CU_TENSOR_MAP_SWIZZLE_128B))
      return TG_ERR_LAUNCH;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(pl.splits), static_cast<unsigned>(pl.panels),
                     static_cast<unsigned>(pl.m_blocks * f.row_sources));
  cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(pl.smem);
  cfg.stream = stream;
  LaunchAttrs la;
  la.fill(cfg, static_cast<unsigned>(pl.splits));
  if (cudaLaunchKernelEx(&cfg, ff_skinny_kernel_of(f), maps, p) != cudaSuccess) {
    cudaGetLastError();
    return TG_ERR_LAUNCH;
  }
  return TG_OK;
}

// Few rows take the split-K kernel: M <= 128 always (two CTAs share an SM), where
// it loses at most 2 us to the pair kernel, with short K (gated 8-bit 4096 x 1024,
// M = 128: 8.7 / 7.3).  So do products with few tiles and long K, in blocks of at
// most 128 rows: where the pair kernel would take 128-wide tiles it leaves SMs
// idle, and each of those that work is held up by its own loads.  Up to 256 rows
// of a weight of 64 panels or more are one block (its second reading costs more
// than the longer reduction: dX of 160 x 8192 x 8192 56 in one block, 62 in two;
// gated 256 x 1024 x 4096, 16 panels, 13.3 and 11.5).  Both by estimated time: a
// k-block takes the pair kernel 0.28 us with 128-wide tiles, 0.27 with 8-bit
// operands, 0.33 with one stored K-first, after 3.7 (8-bit 5), and 0.344 after 5
// with wider ones.  Measured, us, split-K / pair: gated fp16 512 x 512 with K =
// 512, 1024, 2048 7.0 / 6.0, 7.6 / 8.4, 9.0 / 13.3; 1024 x 1024 with K = 8192 35 /
// 44; dX of 1024 x 4096 x 256 19.5 / 49; dWg and dWu (with dG and dU before) of
// 8192 x 512 x 512 26 / 51, of 512 x 512 x 512 8.9 / 7.7; 8-bit 512 x 512 x 2048
// 7.5 / 9.1, 256 x 8192 x 8192 26 / 28.
bool ff_skinny_route(const FfProduct& f, DeviceInfo* info, FfSkinnyPlan* plan) {
  const int64_t pairs = info->sm_count / 2, cols = f.N * (f.gated ? 2 : 1);
  const int64_t tiles = (f.M + 255) / 256 * f.row_sources * ((cols + 255) / 256);
  const bool few_rows = f.M <= 128 && !f.a_km, narrow = 2 * tiles <= pairs;
  const bool one_block = f.M <= kSkinnyMaxM && !f.a_km && cols > 63 * FfSkinnyCfg::PANEL;
  if (!few_rows && !one_block && !narrow) return false;
  if (!ff_skinny_plan(f, one_block ? kSkinnyMaxM : 128, info, plan)) return false;
  if (few_rows) return true;
  const double kb = static_cast<double>(plan->k_blocks);
  const double pair = !narrow                ? 5.0 + static_cast<double>((tiles + pairs - 1) / pairs) * kb * 0.344
                      : f.kind == kFfI8      ? 5.0 + kb * 0.27
                                             : 3.7 + kb * (f.b_kn ? 0.33 : 0.28);
  return plan->us < pair;
}

// Accumulator width of the pair kernel, by estimated time in units of one
// accumulator column and 16-bit element of K on one of `pairs` SM pairs.  The
// 256-wide tile hides its epilogue behind the next tile (two accumulators), but
// fetches a third more operand bytes per product, which L2 cannot quite feed:
// 0.93 of the rate.  The 512-wide tile's epilogue hides about half; the rest is
// worth 160 elements of K (gated: half the results) or 256.  Its last wave may
// be of half tiles.  Measured, us, 512 / 256: gated fp16 4096 x 8192 with K =
// 4096 357 / 371, 2048 219 / 220, 1024 130 / 124; 8-bit product 4096 x 8192 with
// K = 4096 119 / 109, 8192^3 375 / 390; dX of 8192 x 8192 x 4096 825 / 935.
// Where all 128-wide tiles find a pair at once, they take half the time of
// 256-wide ones a k-block (us, 128 / 256: gated fp16 500 x 700 x 600 8.3 / 10, 129
// x 1000 x 264 stored 6.4 / 8.1; 8-bit 1000^3 7.3 / 10); in several waves they
// gain nothing (3001 x 5003 x 1021 with a last wave of them 59.7 / 58.3).
int ff_tile_width(const FfProduct& f, int64_t pairs) {
  const int64_t m_tiles = (f.M + 255) / 256 * f.row_sources;
  const int64_t cols = f.N * (f.gated ? 2 : 1);
  const double k = static_cast<double>(f.K * f.k_sources) * (f.kind == kFfI8 ? 0.5 : 1.0);
  const double drain = f.gated ? 160.0 : 256.0;
  const int64_t tiles256 = m_tiles * ((cols + 255) / 256), tiles512 = m_tiles * ((cols + 511) / 512);
  if (2 * tiles256 <= pairs) return 128;
  const double t256 = static_cast<double>((tiles256 + pairs - 1) / pairs) * k / 0.93 + drain;
  const int64_t rest = tiles512 % pairs;
  const double waves512 = 2.0 * static_cast<double>(tiles512 / pairs) + (rest == 0 ? 0.0 : 2 * rest <= pairs ? 1.0 : 2.0);
  return waves512 * (k + drain) <= t256 ? 512 : 256;
}

tg_status launch_ff(const FfProduct& f, cudaStream_t stream, DeviceInfo* info) {
  FfSkinnyPlan plan;
  if (ff_skinny_route(f, info, &plan)) return launch_ff_skinny(f, plan, stream);
  const int bn = ff_tile_width(f, info->sm_count / 2);
  if (f.kind == kFfI8)
    return f.gated ? launch_ff_pair<kFfI8, true>(f, bn, stream, info) : launch_ff_pair<kFfI8, false>(f, bn, stream, info);
  return f.gated ? launch_ff_pair<kFfF16, true>(f, bn, stream, info) : launch_ff_pair<kFfF16, false>(f, bn, stream, info);
}

// Columns [0, cols) of every row of a result set to +0.
tg_status ff_zero(const FfMat& m, cudaStream_t stream) {
  if (m.bytes() == 0) return TG_OK;
  void* p = const_cast<void*>(m.p);
  const cudaError_t e =
      m.ld == m.cols || m.rows == 1
          ? cudaMemsetAsync(p, 0, static_cast<size_t>(m.bytes()), stream)
          : cudaMemset2DAsync(p, static_cast<size_t>(m.ld * m.elem), 0, static_cast<size_t>(m.cols * m.elem),
                              static_cast<size_t>(m.rows), stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return TG_ERR_LAUNCH;
  }
  return TG_OK;
}

// Workspace layout: each piece 256-byte aligned, in order.
int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

// Bytes of the padded copy of a 16-bit operand that TMA cannot describe (rows
// rounded up to 8 elements), or 0.
int64_t ff_copy_bytes(const FfMat& m) {
  return (m.empty() || m.rows_on(16)) ? 0 : up256(2 * m.rows * round_up(m.cols, 8));
}

// m's padded copy at `ws`, which takes m's place; advances `ws`.
void ff_copy_plan(FfMat& m, RepackParams& r, uint8_t*& ws) {
  const int64_t ld = round_up(m.cols, 8);
  r.src = static_cast<const __half*>(m.p);
  r.dst = reinterpret_cast<__half*>(ws);
  r.src_ld = m.ld;
  r.rows = static_cast<int>(m.rows);
  r.cols = static_cast<int>(m.cols);
  r.cols_pad = static_cast<int>(ld);
  r.chunks = m.rows * (ld / 8);
  m.p = ws;
  m.ld = ld;
  ws += up256(2 * m.rows * ld);
}

// Replace those of `mats` that need one by their padded copies at `ws`, made by
// one launch; advances `ws`.
tg_status ff_make_copies(FfMat* const* mats, int count, uint8_t*& ws, cudaStream_t stream, DeviceInfo* info) {
  PadSetParams p;
  std::memset(&p, 0, sizeof p);
  int n = 0;
  int64_t most = 0;
  for (int i = 0; i < count; ++i) {
    FfMat& m = *mats[i];
    if (ff_copy_bytes(m) == 0) continue;
    most = m.rows > most ? m.rows : most;
    ff_copy_plan(m, p.m[n++], ws);
  }
  if (n == 0) return TG_OK;
  int64_t blocks = (most + 7) / 8;  // eight warps, a row each
  const int64_t cap = static_cast<int64_t>(info->sm_count) * 8;
  blocks = blocks > cap ? cap : blocks;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(n), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  LaunchAttrs la;
  la.fill(cfg, 1);
  if (cudaLaunchKernelEx(&cfg, pad_set_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return TG_ERR_LAUNCH;
  }
  return TG_OK;
}

bool ff_workspace_valid(const void* ws, int64_t ws_bytes, int64_t need, const FfMat* mats, int n) {
  if (ws_bytes < 0 || (ws_bytes > 0 && ws == nullptr) || ws_bytes < need) return false;
  if (need == 0) return true;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return false;
  for (int i = 0; i < n; ++i)
    if (ranges_overlap(ws, need, mats[i].p, mats[i].bytes())) return false;
  return true;
}

// ---------------------------------------------------------------------------
// The gated block, 16-bit operands
// ---------------------------------------------------------------------------
struct GatedArgs {
  FfMat x, wg, wu, h, g, u;
  int64_t M, N, K;
  int type, act;
};

bool gated_args(GatedArgs& a, const void* X, const void* Wg, const void* Wu, const void* H, const void* G,
                const void* U, int64_t M, int64_t N, int64_t K, const tg_gated_options* opt) {
  tg_gated_options o;
  std::memset(&o, 0, sizeof o);
  if (opt) o = *opt;
  if (o.reserved != 0 || !ff_type_valid(o.type) || !ff_act_valid(o.act) || !ff_sizes_valid(M, N, K)) return false;
  if (o.ldx < 0 || o.ldwg < 0 || o.ldwu < 0 || o.ldh < 0 || o.ldg < 0 || o.ldu < 0) return false;
  a.x = mat16(X, M, K, o.ldx);
  a.wg = mat16(Wg, N, K, o.ldwg);
  a.wu = mat16(Wu, N, K, o.ldwu);
  a.h = mat16(H, M, N, o.ldh);
  a.g = mat16(G, M, N, o.ldg);
  a.u = mat16(U, M, N, o.ldu);
  a.M = M;
  a.N = N;
  a.K = K;
  a.type = o.type;
  a.act = o.act;
  return true;
}

int64_t gated_workspace(const GatedArgs& a) {
  if (a.M == 0 || a.N == 0 || a.K == 0) return 0;
  return ff_copy_bytes(a.x) + ff_copy_bytes(a.wg) + ff_copy_bytes(a.wu);
}

tg_status run_gated(GatedArgs& a, void* stream_ptr, void* ws_ptr, int64_t ws_bytes) {
  const bool save = a.g.p != nullptr || a.u.p != nullptr;
  if (a.M == 0 || a.N == 0) return TG_OK;
  const FfMat in[3] = {a.x, a.wg, a.wu};
  const FfMat out[3] = {a.h, a.g, a.u};
  const int n_out = save ? 3 : 1;
  for (const FfMat& m : in)
    if (!m.valid()) return TG_ERR_INVALID_ARG;
  for (int i = 0; i < n_out; ++i)
    if (!out[i].valid()) return TG_ERR_INVALID_ARG;
  if (!ff_disjoint(in, 3, out, n_out)) return TG_ERR_INVALID_ARG;
  const FfMat all[6] = {a.x, a.wg, a.wu, a.h, a.g, a.u};
  if (!ff_workspace_valid(ws_ptr, ws_bytes, gated_workspace(a), all, save ? 6 : 4)) return TG_ERR_INVALID_ARG;
  int dev = 0;
  DeviceInfo* info = nullptr;
  tg_status st = current_device(dev, info);
  if (st != TG_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (a.K == 0) {  // both projections are empty sums: act(0) * 0
    for (int i = 0; i < n_out; ++i)
      if ((st = ff_zero(out[i], stream)) != TG_OK) return st;
    return TG_OK;
  }
  uint8_t* ws = static_cast<uint8_t*>(ws_ptr);
  FfMat* const operands[3] = {&a.x, &a.wg, &a.wu};
  if ((st = ff_make_copies(operands, 3, ws, stream, info)) != TG_OK) return st;
  FfProduct f;
  f.gated = true;
  f.save = save;
  f.a[0] = a.x;
  f.b[0] = a.wg;
  f.b[1] = a.wu;
  f.c[0] = a.h;
  f.c[1] = a.g;
  f.c[2] = a.u;
  f.M = a.M;
  f.N = a.N;
  f.K = a.K;
  f.bf16 = a.type == TG_TYPE_BF16;
  f.act = a.act;
  return launch_ff(f, stream, info);
}

// Gradients.  Workspace: dG and dU (M rows of N rounded up to 8), then padded
// copies of the operands that TMA cannot describe.
struct GatedGradArgs {
  GatedArgs f;  // h is dH
  FfMat dx, dwg, dwu;
};

bool gated_grad_args(GatedGradArgs& a, const void* dH, const void* X, const void* Wg, const void* Wu, const void* G,
                     const void* U, const void* dX, const void* dWg, const void* dWu, int64_t M, int64_t N, int64_t K,
                     const tg_gated_options* opt) {
  if (!gated_args(a.f, X, Wg, Wu, dH, G, U, M, N, K, opt)) return false;
  if (opt && (opt->lddx < 0 || opt->lddwg < 0 || opt->lddwu < 0)) return false;
  a.dx = mat16(dX, M, K, opt ? opt->lddx : 0);
  a.dwg = mat16(dWg, N, K, opt ? opt->lddwg : 0);
  a.dwu = mat16(dWu, N, K, opt ? opt->lddwu : 0);
  return true;
}

int64_t gated_grad_half(const GatedGradArgs& a) { return up256(2 * a.f.M * round_up(a.f.N, 8)); }

int64_t gated_grad_workspace(const GatedGradArgs& a) {
  if (a.f.M == 0 || a.f.N == 0 || a.f.K == 0) return 0;
  int64_t need = 2 * gated_grad_half(a);
  if (a.dwg.p || a.dwu.p) need += ff_copy_bytes(a.f.x);
  if (a.dx.p) need += ff_copy_bytes(a.f.wg) + ff_copy_bytes(a.f.wu);
  return need;
}

tg_status run_gated_grad(GatedGradArgs& a, void* stream_ptr, void* ws_ptr, int64_t ws_bytes) {
  const int64_t M = a.f.M, N = a.f.N, K = a.f.K;
  const FfMat in[6] = {a.f.h, a.f.x, a.f.wg, a.f.wu, a.f.g, a.f.u};
  FfMat out[3];
  int n_out = 0;
  for (const FfMat& m : {a.dx, a.dwg, a.dwu})
    if (m.p != nullptr) out[n_out++] = m;
  if (n_out == 0) return TG_OK;
  for (const FfMat& m : in)
    if (!m.valid()) return TG_ERR_INVALID_ARG;
  for (int i = 0; i < n_out; ++i)
    if (!out[i].valid()) return TG_ERR_INVALID_ARG;
  if (!ff_disjoint(in, 6, out, n_out)) return TG_ERR_INVALID_ARG;
  FfMat all[9];
  int n_all = 0;
  for (const FfMat& m : in) all[n_all++] = m;
  for (int i = 0; i < n_out; ++i) all[n_all++] = out[i];
  if (!ff_workspace_valid(ws_ptr, ws_bytes, gated_grad_workspace(a), all, n_all)) return TG_ERR_INVALID_ARG;
  int64_t written = 0;
  for (int i = 0; i < n_out; ++i) written += out[i].bytes();
  if (written == 0) return TG_OK;
  int dev = 0;
  DeviceInfo* info = nullptr;
  tg_status st = current_device(dev, info);
  if (st != TG_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (M == 0 || N == 0 || K == 0) {  // sums over nothing
    for (int i = 0; i < n_out; ++i)
      if ((st = ff_zero(out[i], stream)) != TG_OK) return st;
    return TG_OK;
  }
  uint8_t* ws = static_cast<uint8_t*>(ws_ptr);
  const int64_t ld = round_up(N, 8);
  FfMat dg{ws, M, N, ld, 2}, du{ws + gated_grad_half(a), M, N, ld, 2};
  ws += 2 * gated_grad_half(a);

  GatedGradParams gp;
  std::memset(&gp, 0, sizeof gp);
  gp.dH = a.f.h.p;
  gp.G = a.f.g.p;
  gp.U = a.f.u.p;
  gp.dG = const_cast<void*>(dg.p);
  gp.dU = const_cast<void*>(du.p);
  gp.ld_dh = a.f.h.ld;
  gp.ld_g = a.f.g.ld;
  gp.ld_u = a.f.u.ld;
  gp.ld_out = ld;
  gp.M = static_cast<int>(M);
  gp.N = static_cast<int>(N);
  gp.vec = (a.f.h.rows_on(16) && a.f.g.rows_on(16) && a.f.u.rows_on(16)) ? 1 : 0;
  gp.bf16 = a.f.type == TG_TYPE_BF16 ? 1 : 0;
  gp.act = a.f.act;
  {
    // A block takes several rows where they are short: dG and dU of 4442 x 89
    // take 11.3 us with a row a block, 6.9 so.
    using Kernel = void (*)(GatedGradParams);
    static const Kernel kernels[] = {gated_grad_kernel<1>, gated_grad_kernel<2>,  gated_grad_kernel<4>,
                                     gated_grad_kernel<8>, gated_grad_kernel<16>, gated_grad_kernel<32>};
    const int64_t chunks = (N + 7) / 8;
    int log_rows = 0;
    while (log_rows < 5 && chunks <= (kGatedGradThreads >> (log_rows + 1))) ++log_rows;
    const int tx = kGatedGradThreads >> log_rows;
    const int64_t bx = (chunks + tx - 1) / tx, row_blocks = (M + (1 << log_rows) - 1) >> log_rows;
    int64_t by = (static_cast<int64_t>(info->sm_count) * 8 * 4 + bx - 1) / bx;
    by = by < 1 ? 1 : (by > row_blocks ? row_blocks : by);
    if (by > 65535) by = 65535;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(bx), static_cast<unsigned>(by), 1);
    cfg.blockDim = dim3(kGatedGradThreads, 1, 1);
    cfg.stream = stream;
    LaunchAttrs la;
    la.fill(cfg, 1);
    if (cudaLaunchKernelEx(&cfg, kernels[log_rows], gp) != cudaSuccess) {
      cudaGetLastError();
      return TG_ERR_LAUNCH;
    }
  }
  FfMat* operands[3];
  int n_operands = 0;
  if (a.dwg.p || a.dwu.p) operands[n_operands++] = &a.f.x;
  if (a.dx.p) {
    operands[n_operands++] = &a.f.wg;
    operands[n_operands++] = &a.f.wu;
  }
  if ((st = ff_make_copies(operands, n_operands, ws, stream, info)) != TG_OK) return st;
  if (a.dwg.p || a.dwu.p) {
    FfProduct f;  // dW = dG^T X: rows of the result are columns of dG
    f.a_km = true;
    f.b_kn = true;
    f.bf16 = gp.bf16 != 0;
    f.M = N;
    f.N = K;
    f.K = M;
    f.b[0] = a.f.x;
    f.row_sources = 0;
    if (a.dwg.p) {
      f.a[f.row_sources] = dg;
      f.c[f.row_sources++] = a.dwg;
    }
    if (a.dwu.p) {
      f.a[f.row_sources] = du;
      f.c[f.row_sources++] = a.dwu;
    }
    if ((st = launch_ff(f, stream, info)) != TG_OK) return st;
  }
  if (a.dx.p) {
    FfProduct f;  // dX = dG Wg + dU Wu
    f.b_kn = true;
    f.bf16 = gp.bf16 != 0;
    f.M = M;
    f.N = K;
    f.K = N;
    f.k_sources = 2;
    f.a[0] = dg;
    f.a[1] = du;
    f.b[0] = a.f.wg;
    f.b[1] = a.f.wu;
    f.c[0] = a.dx;
    if ((st = launch_ff(f, stream, info)) != TG_OK) return st;
  }
  return TG_OK;
}

// ---------------------------------------------------------------------------
// 8-bit operands
// ---------------------------------------------------------------------------
template <int THREADS, int HELD>
tg_status launch_quantize(const QuantizeParams& p, bool bf16, bool vec, cudaStream_t stream, DeviceInfo* info) {
  using Cfg = QuantizeCfg<THREADS, HELD>;
  const int64_t blocks = (static_cast<int64_t>(p.M) + Cfg::ROWS - 1) / Cfg::ROWS;
  const int64_t cap = static_cast<int64_t>(info->sm_count) * Cfg::BLOCKS_PER_SM;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < cap ? blocks : cap), 1, 1);
  cfg.blockDim = dim3(Cfg::BLOCK, 1, 1);
  cfg.stream = stream;
  LaunchAttrs la;
  la.fill(cfg, 1);
  auto kernel = bf16 ? (vec ? quantize_rows_kernel<THREADS, HELD, true, true> : quantize_rows_kernel<THREADS, HELD, true, false>)
                     : (vec ? quantize_rows_kernel<THREADS, HELD, false, true> : quantize_rows_kernel<THREADS, HELD, false, false>);
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return TG_ERR_LAUNCH;
  }
  return TG_OK;
}

tg_status run_quantize(const void* X, void* Q, float* scales, int64_t M, int64_t K, int64_t ldx, int64_t ldq,
                       int32_t type, void* stream_ptr) {
  if (!ff_sizes_valid(M, 1, K) || !ff_type_valid(type) || ldx < 0 || ldq < 0) return TG_ERR_INVALID_ARG;
  if (M == 0) return TG_OK;
  const FfMat x = mat16(X, M, K, ldx), q = mat8(Q, M, K, ldq), s = vec32(scales, M);
  if (!x.valid() || !q.valid() || !s.valid() || q.overlaps(x) || s.overlaps(x) || s.overlaps(q))
    return TG_ERR_INVALID_ARG;
  int dev = 0;
  DeviceInfo* info = nullptr;
  tg_status st = current_device(dev, info);
  if (st != TG_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (K == 0) return ff_zero(s, stream);  // the maximum of nothing
  QuantizeParams p;
  std::memset(&p, 0, sizeof p);
  p.X = X;
  p.Q = static_cast<int8_t*>(Q);
  p.scale = scales;
  p.ldx = x.ld;
  p.ldq = q.ld;
  p.M = static_cast<int>(M);
  p.K = static_cast<int>(K);
  p.vec_out = q.rows_on(8) ? 1 : 0;
  const bool vec = x.rows_on(16);
  const bool bf16 = type == TG_TYPE_BF16;
  // Threads per row: the fewest that hold the row, at four chunks each, so that
  // many rows are in flight per SM.  Measured at 8192 rows, us: K = 2048 with 64
  // / 256 threads 12.1 / 21.8, K = 4096 with 128 / 256 21.0 / 27.9.  With fewer
  // rows than SMs a block of 1024, one chunk each, shortens a long row's path
  // (16 x 8192: 2.2 us).
  if (K <= QuantizeCfg<32, 4>::HELD_VALUES) return launch_quantize<32, 4>(p, bf16, vec, stream, info);
  if (M <= info->sm_count) return launch_quantize<1024, 1>(p, bf16, vec, stream, info);
  if (K <= QuantizeCfg<64, 4>::HELD_VALUES) return launch_quantize<64, 4>(p, bf16, vec, stream, info);
  if (K <= QuantizeCfg<128, 4>::HELD_VALUES) return launch_quantize<128, 4>(p, bf16, vec, stream, info);
  if (K <= QuantizeCfg<256, 4>::HELD_VALUES) return launch_quantize<256, 4>(p, bf16, vec, stream, info);
  return launch_quantize<512, 4>(p, bf16, vec, stream, info);
}

// The 8-bit operands of a product: rows on 16-byte boundaries (TMA).
bool ff_i8_operand(const FfMat& m) { return m.valid() && (m.empty() || m.rows_on(16)); }

tg_status run_gemm_i8(const void* A, const float* a_scale, const void* W, const float* w_scale, const void* bias,
                      void* C, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldw, int64_t ldc, int32_t relu,
                      int32_t type, void* stream_ptr) {
  if (!ff_sizes_valid(M, N, K) || K > kFfMaxKI8 || !ff_type_valid(type) || (relu != 0 && relu != 1) || lda < 0 ||
      ldw < 0 || ldc < 0)
    return TG_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return TG_OK;
  const FfMat in[5] = {mat8(A, M, K, lda), mat8(W, N, K, ldw), vec32(a_scale, M), vec32(w_scale, N),
                       mat16(bias, bias ? 1 : 0, N, N)};
  const FfMat c = mat16(C, M, N, ldc);
  if (!ff_i8_operand(in[0]) || !ff_i8_operand(in[1]) || !in[2].valid() || !in[3].valid() || !in[4].valid() ||
      !c.valid() || !ff_disjoint(in, 5, &c, 1))
    return TG_ERR_INVALID_ARG;
  int dev = 0;
  DeviceInfo* info = nullptr;
  tg_status st = current_device(dev, info);
  if (st != TG_OK) return st;
  if (K == 0) {
    const BiasFillParams b{C, bias, c.ld, static_cast<int>(M), static_cast<int>(N), relu, type == TG_TYPE_BF16 ? 1 : 0};
    return launch_simple(bias_fill_kernel, b, M * N, 1, static_cast<cudaStream_t>(stream_ptr), info);
  }
  FfProduct f;
  f.kind = kFfI8;
  f.a[0] = in[0];
  f.b[0] = in[1];
  f.c[0] = c;
  f.M = M;
  f.N = N;
  f.K = K;
  f.row_scale = a_scale;
  f.col_scale[0] = w_scale;
  f.bias = bias;
  f.relu = relu;
  f.bf16 = type == TG_TYPE_BF16;
  return launch_ff(f, static_cast<cudaStream_t>(stream_ptr), info);
}

tg_status run_gated_i8(const void* A, const float* a_scale, const void* Wg, const float* g_scale, const void* Wu,
                       const float* u_scale, void* H, int64_t M, int64_t N, int64_t K, const tg_gated_options* opt,
                       void* stream_ptr) {
  tg_gated_options o;
  std::memset(&o, 0, sizeof o);
  if (opt) o = *opt;
  if (!ff_sizes_valid(M, N, K) || K > kFfMaxKI8 || o.reserved != 0 || !ff_type_valid(o.type) || !ff_act_valid(o.act) ||
      o.ldx < 0 || o.ldwg < 0 || o.ldwu < 0 || o.ldh < 0)
    return TG_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return TG_OK;
  const FfMat in[6] = {mat8(A, M, K, o.ldx),  mat8(Wg, N, K, o.ldwg), mat8(Wu, N, K, o.ldwu),
                       vec32(a_scale, M), vec32(g_scale, N),      vec32(u_scale, N)};
  const FfMat h = mat16(H, M, N, o.ldh);
  for (int i = 0; i < 6; ++i)
    if (i < 3 ? !ff_i8_operand(in[i]) : !in[i].valid()) return TG_ERR_INVALID_ARG;
  if (!h.valid() || !ff_disjoint(in, 6, &h, 1)) return TG_ERR_INVALID_ARG;
  int dev = 0;
  DeviceInfo* info = nullptr;
  tg_status st = current_device(dev, info);
  if (st != TG_OK) return st;
  if (K == 0) return ff_zero(h, static_cast<cudaStream_t>(stream_ptr));
  FfProduct f;
  f.kind = kFfI8;
  f.gated = true;
  f.a[0] = in[0];
  f.b[0] = in[1];
  f.b[1] = in[2];
  f.c[0] = h;
  f.M = M;
  f.N = N;
  f.K = K;
  f.row_scale = a_scale;
  f.col_scale[0] = g_scale;
  f.col_scale[1] = u_scale;
  f.act = o.act;
  f.bf16 = o.type == TG_TYPE_BF16;
  return launch_ff(f, static_cast<cudaStream_t>(stream_ptr), info);
}

}  // namespace
}  // namespace tg

extern "C" {

tg_status tg_gated(const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U, int64_t M, int64_t N,
                   int64_t K, const tg_gated_options* options, void* stream, void* workspace,
                   int64_t workspace_bytes) {
  tg::GatedArgs a;
  if (!tg::gated_args(a, X, Wg, Wu, H, G, U, M, N, K, options) || ((G == nullptr) != (U == nullptr)))
    return TG_ERR_INVALID_ARG;
  return tg::run_gated(a, stream, workspace, workspace_bytes);
}

int64_t tg_gated_workspace_size(const void* X, const void* Wg, const void* Wu, int64_t M, int64_t N, int64_t K,
                                const tg_gated_options* options) {
  tg::GatedArgs a;
  if (!tg::gated_args(a, X, Wg, Wu, nullptr, nullptr, nullptr, M, N, K, options)) return -1;
  return tg::gated_workspace(a);
}

tg_status tg_gated_backward(const void* dH, const void* X, const void* Wg, const void* Wu, const void* G,
                            const void* U, void* dX, void* dWg, void* dWu, int64_t M, int64_t N, int64_t K,
                            const tg_gated_options* options, void* stream, void* workspace, int64_t workspace_bytes) {
  tg::GatedGradArgs a;
  if (!tg::gated_grad_args(a, dH, X, Wg, Wu, G, U, dX, dWg, dWu, M, N, K, options)) return TG_ERR_INVALID_ARG;
  return tg::run_gated_grad(a, stream, workspace, workspace_bytes);
}

int64_t tg_gated_backward_workspace_size(const void* X, const void* Wg, const void* Wu, const void* dX,
                                         const void* dWg, const void* dWu, int64_t M, int64_t N, int64_t K,
                                         const tg_gated_options* options) {
  tg::GatedGradArgs a;
  if (!tg::gated_grad_args(a, nullptr, X, Wg, Wu, nullptr, nullptr, dX, dWg, dWu, M, N, K, options)) return -1;
  return tg::gated_grad_workspace(a);
}

tg_status tg_quantize_rows_i8(const void* X, void* Q, float* scales, int64_t M, int64_t K, int64_t ldx, int64_t ldq,
                              int32_t type, void* stream) {
  return tg::run_quantize(X, Q, scales, M, K, ldx, ldq, type, stream);
}

tg_status tg_gemm_i8(const void* A, const float* a_scale, const void* W, const float* w_scale, const void* bias,
                     void* C, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldw, int64_t ldc, int32_t relu,
                     int32_t type, void* stream) {
  return tg::run_gemm_i8(A, a_scale, W, w_scale, bias, C, M, N, K, lda, ldw, ldc, relu, type, stream);
}

tg_status tg_gated_i8(const void* A, const float* a_scale, const void* Wg, const float* g_scale, const void* Wu,
                      const float* u_scale, void* H, int64_t M, int64_t N, int64_t K, const tg_gated_options* options,
                      void* stream) {
  return tg::run_gated_i8(A, a_scale, Wg, g_scale, Wu, u_scale, H, M, N, K, options, stream);
}

}  // extern "C"
