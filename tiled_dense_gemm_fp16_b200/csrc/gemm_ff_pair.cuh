// gemm_ff_pair.cuh -- the products of a feed-forward block on CTA pairs
// (cta_group::2): one persistent tcgen05 kernel for
//   * the gated forward  H = act(X Wg^T) * (X Wu^T), 16-bit or 8-bit operands,
//     both projections, the activation and the product in one pass, G and U
//     stored too on request (for the backward pass);
//   * its gradients: dX = dG Wg + dU Wu as one K loop over both sources, and
//     dWg = dG^T X, dWu = dU^T X as one grid over both results;
//   * the 8-bit product C = (A W^T) sa sw + bias with an optional ReLU.
//
// The pipeline is that of the fp16 pair kernel: both CTAs load their half of a
// 256 x BN tile by TMA into an mbarrier ring (128-byte swizzle, 128 bytes of K
// per k-block), the even CTA's MMA thread issues 256 x 256 MMAs over both SMs'
// shared memory, the epilogue warps of both CTAs drain TMEM.
//
// Gated tiles: of every 256 accumulator columns each CTA supplies the B rows
// of 128, and these are 64 rows of Wg followed by the same 64 rows of Wu.  So
// one MMA computes both projections of 128 block columns, the same thread of
// an epilogue warp reads G and U of an element, and neither leaves the SM.  A
// 256 x BN accumulator gives 256 x BN / 2 values of H; per SM and k-block it
// moves what the plain product moves.
//
// An epilogue warp first turns all its accumulator columns into packed 16-bit
// results in registers, then frees the accumulator, then stores: TMA boxes
// where rows of the result start on 16-byte boundaries, else through the same
// staging boxes row by row, 64 bytes per store instruction.  Stored G and U
// (twice the registers) leave during the drain.
#pragma once

#include "ff_ops.cuh"
#include "gemm_tc_pair.cuh"

namespace tg {

struct FfMaps {
  CUtensorMap a[2];  // sources along K (dX) or along the rows of the result (dWg, dWu)
  CUtensorMap b[2];  // gate and up weights, or sources along K
  CUtensorMap c[3];  // H, G, U; or the results of the two row sources
};

struct FfParams {
  void* c[3];
  int64_t ldc[3];
  const float* row_scale;     // 8-bit: one per row of A
  const float* col_scale[2];  // 8-bit: one per row of the (gate, up) weight
  const void* bias;           // 16-bit values of the result's type, or nullptr
  int M, N;                   // rows and columns of one result
  int m_tiles, n_tiles;       // m_tiles over all row sources
  int num_tiles;              // tiles to walk: `whole_tiles` whole ones, then halves of the rest
  int whole_tiles;
  int m_tiles_src;            // row tiles of one row source
  int k_blocks, k_blocks_src; // k-blocks over all K sources, and of one
  int group_m;
  int a_mnmajor, b_kmajor;
  int bf16;                   // type of the 16-bit results (and operands)
  int act, relu;
  int save;                   // gated: store G and U
  int c_aligned[3];           // rows of the result start on 16-byte boundaries (they may end inside 16 bytes)
  int l2_hints;               // as TcParams
  uint32_t idesc;
  uint64_t wait_budget_ns;
};

template <int STAGES_, int BN_, int EPI_WARPS_>
struct FfPairCfg {
  static constexpr int BM = 128;
  static constexpr int PAIR_M = 256;
  static constexpr int BN = BN_;                       // accumulator columns per tile
  static constexpr int SLAB = BN < 256 ? BN : 256;     // of one MMA
  static constexpr int SLABS = BN / SLAB;
  static constexpr int B_ROWS = SLAB / 2;              // rows of B a CTA loads per slab
  static constexpr int STAGES = STAGES_;
  static constexpr int MMA_WARP = 1;
  static constexpr int EPI_WARP0 = 2;
  static constexpr int EPI_WARPS = EPI_WARPS_;
  static constexpr int EPI_COLS = SLAB * 4 / EPI_WARPS;  // accumulator columns of a slab per epilogue warp
  static constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
  static constexpr int K_BYTES = 128;                  // bytes of K per k-block
  static constexpr int A_BYTES = BM * K_BYTES;
  static constexpr int B_SLAB_BYTES = B_ROWS * K_BYTES;
  static constexpr int B_BYTES = SLABS * B_SLAB_BYTES;
  static constexpr int PANEL_BYTES = 64 * K_BYTES;     // one 64-column panel of an MN-major operand
  static constexpr int NUM_ACC = SLABS == 1 ? 2 : 1;
  static constexpr int TMEM_COLS = 512;
  static constexpr int BAR_BYTES = 256;
  static constexpr int C_BUF_BYTES = 32 * 64;          // one 32 x 32 box of 16-bit values
  static constexpr int C_BUFS = 16 / EPI_WARPS;        // staging boxes per epilogue warp
  static constexpr int C_STAGE_BYTES = EPI_WARPS * C_BUFS * C_BUF_BYTES;
  static constexpr int SMEM_BYTES = 1024 + STAGES * (A_BYTES + B_BYTES) + C_STAGE_BYTES + BAR_BYTES;
  static_assert(SMEM_BYTES <= 232448, "dynamic shared memory per CTA");
  static_assert((2 * STAGES + 5) * 8 + 8 <= BAR_BYTES, "barriers");
  static_assert(NUM_ACC * BN <= TMEM_COLS, "TMEM columns");
  static_assert(EPI_COLS % 64 == 0, "a warp finishes whole boxes of 32 result columns");
  // Every address that TMA, the MMAs and the barriers get is the base (on 1024)
  // plus a sum of these.
  static_assert(A_BYTES % 1024 == 0 && PANEL_BYTES % 1024 == 0 && B_SLAB_BYTES % 2048 == 0,
                "operand tiles, and the gate and up halves of a slab, start on the swizzle's 1024 bytes");
  static_assert(C_BUF_BYTES % 512 == 0, "staging boxes start on their swizzle's 512 bytes");
  static_assert((STAGES * (A_BYTES + B_BYTES) + C_STAGE_BYTES) % 512 == 0, "barriers on 8 bytes");
};

// Tile t of the walk: its place, and for a half tile (one slab of 256
// accumulator columns) which half.
struct FfTile {
  int m_blk, n_blk;
  int row_src;   // which source of rows, m_blk counted inside it
  int half;      // 0 or 1 of a half tile
  bool whole;
};

__device__ __forceinline__ FfTile ff_tile(const FfParams& p, int t) {
  FfTile f;
  f.whole = t < p.whole_tiles;
  f.half = 0;
  if (!f.whole) {
    const int r = t - p.whole_tiles;
    f.half = r & 1;
    t = p.whole_tiles + (r >> 1);
  }
  const int group_tiles = p.group_m * p.n_tiles;
  const int g = t / group_tiles;
  const int first_m = g * p.group_m;
  const int gm = min(p.m_tiles - first_m, p.group_m);
  const int local = t - g * group_tiles;
  f.m_blk = first_m + local % gm;
  f.n_blk = local / gm;
  f.row_src = f.m_blk >= p.m_tiles_src ? 1 : 0;
  f.m_blk -= f.row_src * p.m_tiles_src;
  return f;
}

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// Scales of 16 consecutive columns (0 past N).
__device__ __forceinline__ void load_scale16(const float* scale, int col, int N, float (&s)[16]) {
  const float* src = scale + col;
  if (col + 16 <= N && (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(src) + q);
      s[4 * q] = v.x;
      s[4 * q + 1] = v.y;
      s[4 * q + 2] = v.z;
      s[4 * q + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = col + e < N ? __ldg(src + e) : 0.0f;
  }
}

// 16 consecutive 16-bit values from `src` on, for columns from `col` on (0 past N).
__device__ __forceinline__ void load_bias16(const unsigned short* src, int col, int N, bool bf16, float (&v)[16]) {
  if (col + 16 <= N && (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(src) + q);
      const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = unpack_16(h[e], bf16);
        v[8 * q + 2 * e] = x.x;
        v[8 * q + 2 * e + 1] = x.y;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = col + e < N ? load_16(src + e, bf16) : 0.0f;
  }
}

// Scales (and bias) of tile t's rows and columns into L1: `row` is this lane's row inside
// the tile, `col` its first column inside a slab.
template <bool GATED, int TILE_N, int SLAB_N, int OUT>
__device__ __forceinline__ void ff_prefetch_scales(const FfParams& p, int t, int row, int col) {
  if (t >= p.num_tiles) return;
  const FfTile f = ff_tile(p, t);
  if (f.m_blk * 256 + row < p.M) prefetch_l1(p.row_scale + f.m_blk * 256 + row);
#pragma unroll
  for (int c = 0; c < TILE_N; c += SLAB_N) {
    if (c > 0 && !f.whole) break;
#pragma unroll
    for (int q = 0; q < OUT; q += 32) {
      const int n = f.n_blk * TILE_N + f.half * SLAB_N + c + col + q;
      if (n < p.N) {
        prefetch_l1(p.col_scale[0] + n);
        if (GATED) prefetch_l1(p.col_scale[1] + n);
        if (!GATED && p.bias != nullptr) prefetch_l1(static_cast<const unsigned short*>(p.bias) + n);
      }
    }
  }
}

// 16 accumulator words as fp32: the fp32 sums themselves, or the 32-bit
// integer sums (one rounding to fp32) times the row's and column's scale.
template <int KIND>
__device__ __forceinline__ void ff_values(const uint32_t (&r)[16], float row_scale, const float* col_scale, int col,
                                          int N, float (&v)[16]) {
  if (KIND == kFfF16) {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(r[e]);
  } else {
    float s[16];
    load_scale16(col_scale, col, N, s);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float2 x = make_float2(__int2float_rn(static_cast<int>(r[e])), __int2float_rn(static_cast<int>(r[e + 1])));
      const float2 y = mul2(mul2(x, same2(row_scale)), make_float2(s[e], s[e + 1]));
      v[e] = y.x;
      v[e + 1] = y.y;
    }
  }
}

template <int ACT>
__device__ __forceinline__ void gate_row(float (&g)[16], const float (&u)[16]) {
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const float2 h = mul2(act_value2<ACT>(make_float2(g[e], g[e + 1])), make_float2(u[e], u[e + 1]));
    g[e] = h.x;
    g[e + 1] = h.y;
  }
}

// One 32 x 32 box of a result: lane = row, h = its 32 packed values, `buf` one
// of the warp's BUFS staging boxes (64-byte swizzle), which take turns.  Rows
// that start on 16-byte boundaries leave as one TMA box, but for a box in which
// they end inside 16 bytes: TMA clips a store to whole 16-byte pieces (measured:
// N = 41 in rows of 48 writes zeros up to column 47).  Else two rows leave
// per store instruction, 4 bytes a lane: the rows are staged shifted so that
// words start on 4-byte boundaries, which leaves the first and last value of a
// row on an odd 2-byte boundary to single stores by the row's lane.
template <int BUFS>
__device__ __forceinline__ void ff_store_box(const CUtensorMap* map, void* c, int64_t ldc, bool aligned, int M, int N,
                                             int y0, int col0, const uint32_t* h, uint8_t* buf, int lane,
                                             uint64_t policy) {
  if (lane == 0) bulk_wait_group_read<BUFS - 1>();  // the last box stored from `buf` has been read
  __syncwarp();
  const uint32_t row_addr = smem_u32(buf) + lane * 64;
  if (aligned && (col0 + 32 <= N || (N & 7) == 0)) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      st_shared_v4(row_addr + ((q ^ ((lane >> 1) & 3)) << 4), h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d_hint(map, buf, col0, y0, policy);
      bulk_commit_group();
    }
    return;
  }
  unsigned short* box = static_cast<unsigned short*>(c) + static_cast<int64_t>(y0) * ldc + col0;
  const int rows = min(32, M - y0);
  const bool whole = col0 + 32 <= N;
  const uint32_t odd0 = (reinterpret_cast<uintptr_t>(box) >> 1) & 1u;  // row 0 starts on an odd 2-byte boundary
  const uint32_t odd = whole ? (odd0 ^ (lane & static_cast<uint32_t>(ldc) & 1u)) : 0u;  // this lane's row
  uint32_t w[17];
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = h[e];
  w[16] = 0u;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    st_shared_v4(row_addr + ((q ^ ((lane >> 1) & 3)) << 4), __funnelshift_r(w[4 * q], w[4 * q + 1], odd * 16),
                 __funnelshift_r(w[4 * q + 1], w[4 * q + 2], odd * 16),
                 __funnelshift_r(w[4 * q + 2], w[4 * q + 3], odd * 16),
                 __funnelshift_r(w[4 * q + 3], w[4 * q + 4], odd * 16));
  __syncwarp();
  if (whole) {
    const int half = lane >> 4, j = lane & 15;  // row 2 i + half, word j
    const uint32_t odd_r = odd0 ^ (static_cast<uint32_t>(half) & static_cast<uint32_t>(ldc) & 1u);
    const bool word_ok = j + static_cast<int>(odd_r) < 16;
    uint32_t* dst = reinterpret_cast<uint32_t*>(box + half * ldc + 2 * j + odd_r);
    const uint32_t src = smem_u32(buf) + half * 64 + (j & 3) * 4;
    const int turns = rows == 32 ? 16 : (rows - half + 1) / 2;
    if (word_ok) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i < turns) {
          uint32_t v;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(src + i * 128 + (((j >> 2) ^ (i & 3)) << 4)));
          *dst = v;
        }
        dst += ldc;  // two rows of 2-byte values
      }
    }
    if (odd && lane < rows) {
      unsigned short* r = box + lane * ldc;
      r[0] = static_cast<unsigned short>(h[0] & 0xffffu);
      r[31] = static_cast<unsigned short>(h[15] >> 16);
    }
  } else {  // the last columns: lane = column, one row per store
    unsigned short* dst = box + lane;
    const bool col_ok = col0 + lane < N;
#pragma unroll 4
    for (int r = 0; r < 32; ++r) {
      const unsigned short v = *reinterpret_cast<const unsigned short*>(
          buf + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2);
      if (r < rows && col_ok) dst[r * ldc] = v;
    }
  }
  if (lane == 0) bulk_commit_group();  // an empty group, so that the wait above counts boxes
  __syncwarp();
}

template <int STAGES, int BN, int EPI_WARPS, int KIND, bool GATED>
__global__ void __launch_bounds__(FfPairCfg<STAGES, BN, EPI_WARPS>::THREADS, 1)
    ff_pair_kernel(const __grid_constant__ FfMaps maps, const FfParams p) {
  using Cfg = FfPairCfg<STAGES, BN, EPI_WARPS>;
  constexpr int K_ELEMS = KIND == kFfI8 ? 128 : 64;   // elements of K per k-block
  constexpr int SLAB_N = GATED ? Cfg::SLAB / 2 : Cfg::SLAB;  // result columns per slab
  constexpr int TILE_N = Cfg::SLABS * SLAB_N;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* a_smem = smem;
  uint8_t* b_smem = smem + Cfg::STAGES * Cfg::A_BYTES;
  uint8_t* c_stage = smem + Cfg::STAGES * (Cfg::A_BYTES + Cfg::B_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(c_stage + Cfg::C_STAGE_BYTES);
  uint64_t* full_bar = bars;                              // used in the even CTA
  uint64_t* empty_bar = bars + Cfg::STAGES;               // per CTA
  uint64_t* acc_full_bar = bars + 2 * Cfg::STAGES;        // per CTA
  uint64_t* acc_empty_bar = acc_full_bar + 2;             // used in the even CTA: one per slab of TMEM
  uint64_t* mma_done_bar = acc_empty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1;
  const int num_clusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full_bar[b], 1);
      mbar_init(&acc_empty_bar[b], 2 * Cfg::EPI_WARPS);
    }
    mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
    if (GATED) tma_prefetch_desc(&maps.b[1]);
    if (p.c_aligned[0]) tma_prefetch_desc(&maps.c[0]);
  }
  if (warp == Cfg::MMA_WARP) {
    tmem_alloc_pair(tmem_slot, Cfg::TMEM_COLS);
    tmem_relinquish_alloc_permit_pair();
  }
  tcgen05_fence_before_sync();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised before any remote use
  tcgen05_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    // Producer (both CTAs): this CTA's half of the A and B tiles.
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int last_parity[Cfg::STAGES];
#pragma unroll
      for (int s = 0; s < Cfg::STAGES; ++s) last_parity[s] = -1;
      bool ok = true;
      const uint64_t pol_a = (p.l2_hints & 1) ? l2_policy_evict_last() : l2_policy_evict_normal();
      const uint64_t pol_b = (p.l2_hints & 2)   ? l2_policy_evict_last()
                             : (p.l2_hints & 4) ? l2_policy_evict_first()
                                                : l2_policy_evict_normal();
      const uint32_t full_even0 = mapa_shared(smem_u32(full_bar), 0);
      for (int t = cluster_id; t < p.num_tiles && ok; t += num_clusters) {
        const FfTile f = ff_tile(p, t);
        const int row_src = f.row_src;
        const int slabs = f.whole ? Cfg::SLABS : 1;
        const int m0 = f.m_blk * Cfg::PAIR_M + static_cast<int>(rank) * Cfg::BM;
        const int n0 = f.n_blk * TILE_N + f.half * SLAB_N + static_cast<int>(rank) * (GATED ? Cfg::B_ROWS / 2 : Cfg::B_ROWS);
        const uint32_t tx = 2 * (Cfg::A_BYTES + slabs * Cfg::B_SLAB_BYTES);
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, p.wait_budget_ns, 0x81)) {
            ok = false;
            break;
          }
          const uint32_t full_even = full_even0 + stage * 8;
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], tx);
          const int k_src = kb >= p.k_blocks_src ? 1 : 0;
          const int k0 = (kb - k_src * p.k_blocks_src) * K_ELEMS;
          const CUtensorMap* ma = &maps.a[row_src | k_src];
          uint8_t* adst = a_smem + stage * Cfg::A_BYTES;
          uint8_t* bdst = b_smem + stage * Cfg::B_BYTES;
          if (KIND == kFfF16 && p.a_mnmajor) {
            // A stored K x M: this CTA's 128 rows as two 64 m x 64 k boxes.
            tma_load_2d_pair_hint(adst, ma, full_even, m0, k0, pol_a);
            tma_load_2d_pair_hint(adst + Cfg::PANEL_BYTES, ma, full_even, m0 + 64, k0, pol_a);
          } else {
            tma_load_2d_pair_hint(adst, ma, full_even, k0, m0, pol_a);
          }
#pragma unroll
          for (int j = 0; j < Cfg::SLABS; ++j) {
            if (j >= slabs) break;
            uint8_t* slab = bdst + j * Cfg::B_SLAB_BYTES;
            const int n = n0 + SLAB_N * j;
            if (GATED) {
              // Half of the slab's rows of Wg, then the same rows of Wu.
              tma_load_2d_pair_hint(slab, &maps.b[0], full_even, k0, n, pol_b);
              tma_load_2d_pair_hint(slab + Cfg::B_SLAB_BYTES / 2, &maps.b[1], full_even, k0, n, pol_b);
            } else if (KIND == kFfI8 || p.b_kmajor) {
              tma_load_2d_pair_hint(slab, &maps.b[k_src], full_even, k0, n, pol_b);
            } else {
#pragma unroll
              for (int q = 0; q < Cfg::B_ROWS / 64; ++q)
                tma_load_2d_pair_hint(slab + q * Cfg::PANEL_BYTES, &maps.b[k_src], full_even, n + 64 * q, k0, pol_b);
            }
          }
          last_parity[stage] = static_cast<int>(phase);
          if (++stage == Cfg::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // The even CTA's full barriers count both CTAs' bytes: once they have
      // completed, every load of the pair has landed.
      if (leader) {
#pragma unroll 1
        for (int s = 0; s < Cfg::STAGES; ++s) {
          if (last_parity[s] >= 0) {
            volatile int no_abort = 0;
            mbar_wait(&full_bar[s], static_cast<uint32_t>(last_parity[s]), &no_abort, p.wait_budget_ns, 0x82);
          }
        }
      }
    }
  } else if (warp == Cfg::MMA_WARP) {
    // MMA issuer (even CTA only).
    if (leader && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;
      bool ok = true;
      const bool a_mn = KIND == kFfF16 && p.a_mnmajor != 0;
      const bool b_mn = KIND == kFfF16 && !GATED && p.b_kmajor == 0;
      // Descriptors of stage 0 and their steps in units of 16 bytes: one
      // addition per descriptor and MMA (shared memory ends below 2^18, so the
      // address field takes no carry).  This thread's instructions bound the
      // 128-wide tile: a k-block takes 0.28 us (0.30 with descriptors built
      // anew for each MMA), of which the loads of a stage are not felt.
      const uint64_t a_desc0 = make_sw128_desc(smem_u32(a_smem), a_mn ? Cfg::PANEL_BYTES : 16, 1024);
      const uint64_t b_desc0 = make_sw128_desc(smem_u32(b_smem), b_mn ? Cfg::PANEL_BYTES : 16, 1024);
      const uint32_t a_step = a_mn ? 2048 / 16 : 32 / 16, b_step = b_mn ? 2048 / 16 : 32 / 16;
      // The four MMAs of one k-block and one slab, 32 bytes of K each.
      auto issue = [&](int st, int j, uint32_t d_tmem, bool first) {
        const uint64_t a_desc = a_desc0 + st * (Cfg::A_BYTES / 16);
        const uint64_t b_desc = b_desc0 + st * (Cfg::B_BYTES / 16) + j * (Cfg::B_SLAB_BYTES / 16);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_ff_pair<KIND>(d_tmem + Cfg::SLAB * j, a_desc + k * a_step, b_desc + k * b_step, p.idesc,
                             (first && k == 0) ? 0u : 1u);
      };
      auto advance = [&](int& st, uint32_t& ph) {
        if (++st == Cfg::STAGES) {
          st = 0;
          ph ^= 1u;
        }
      };
      for (int t = cluster_id; t < p.num_tiles && ok; t += num_clusters, ++local) {
        const bool whole = t < p.whole_tiles;
        const int acc = local % Cfg::NUM_ACC;
        const uint32_t acc_phase = (local / Cfg::NUM_ACC) & 1;
        if (!mbar_wait(&acc_empty_bar[acc], acc_phase ^ 1u, abort_flag, p.wait_budget_ns, 0x83)) break;
        tcgen05_fence_after_sync();
        const uint32_t d_tmem = tmem_base + acc * Cfg::BN;
        int kb = 0;
        if (Cfg::SLABS == 2) {
          // The epilogue frees slab 0 while it still drains slab 1: until that
          // is free too, the k-blocks in the ring go into slab 0 alone, and
          // catch up in slab 1 after.
          const uint32_t second = smem_u32(&acc_empty_bar[1]);
          int ahead = 0, st = stage;
          uint32_t ph = phase;
          while (whole && ahead < Cfg::STAGES && ahead < p.k_blocks && !mbar_test_wait(second, acc_phase ^ 1u)) {
            if (!mbar_wait(&full_bar[st], ph, abort_flag, p.wait_budget_ns, 0x87)) {
              ok = false;
              break;
            }
            tcgen05_fence_after_sync();
            issue(st, 0, d_tmem, ahead == 0);
            ++ahead;
            advance(st, ph);
          }
          if (!ok || !mbar_wait(&acc_empty_bar[1], acc_phase ^ 1u, abort_flag, p.wait_budget_ns, 0x88)) break;
          tcgen05_fence_after_sync();
          for (; kb < ahead; ++kb) {
            issue(stage, 1, d_tmem, kb == 0);
            umma_commit_pair_mc(&empty_bar[stage], 0x3);
            advance(stage, phase);
          }
        }
        for (; kb < p.k_blocks; ++kb) {
          if (!mbar_wait(&full_bar[stage], phase, abort_flag, p.wait_budget_ns, 0x84)) {
            ok = false;
            break;
          }
          tcgen05_fence_after_sync();
          issue(stage, 0, d_tmem, kb == 0);
          if (Cfg::SLABS == 2 && whole) issue(stage, 1, d_tmem, kb == 0);
          umma_commit_pair_mc(&empty_bar[stage], 0x3);  // both CTAs may refill this stage
          advance(stage, phase);
        }
        if (!ok) break;
        umma_commit_pair_mc(&acc_full_bar[acc], 0x3);
      }
      umma_commit_pair_mc(mma_done_bar, 0x1);
      volatile int no_abort = 0;
      mbar_wait(mma_done_bar, 0, &no_abort, p.wait_budget_ns, 0x85);
    }
    __syncwarp();
  } else {
    // Epilogue (both CTAs): warp w takes TMEM lanes 32 (w mod 4) .. + 31 and
    // part `part` of every slab's columns.
    const int quad = warp & 3;
    const int part = (warp - Cfg::EPI_WARP0) >> 2;
    constexpr int OUT = GATED ? Cfg::EPI_COLS / 2 : Cfg::EPI_COLS;  // result columns of this warp per slab
    uint8_t* wbuf = c_stage + (warp - Cfg::EPI_WARP0) * Cfg::C_BUFS * Cfg::C_BUF_BYTES;
    const uint64_t pol = l2_policy_evict_first();
    const int row_in_tile = static_cast<int>(rank) * Cfg::BM + quad * 32;
    int local = 0;
    int turn = 0;  // which staging box comes next
    if (KIND == kFfI8)
      ff_prefetch_scales<GATED, TILE_N, SLAB_N, OUT>(p, cluster_id, row_in_tile + lane, part * OUT + lane);
    for (int t = cluster_id; t < p.num_tiles; t += num_clusters, ++local) {
      const FfTile f = ff_tile(p, t);
      const int acc = local % Cfg::NUM_ACC;
      const uint32_t acc_phase = (local / Cfg::NUM_ACC) & 1;
      const int y0 = f.m_blk * Cfg::PAIR_M + row_in_tile;
      const int out0 = f.n_blk * TILE_N + f.half * SLAB_N + part * OUT;
      float row_scale = 0.0f;
      if (KIND == kFfI8) {
        if (y0 + lane < p.M) row_scale = __ldg(p.row_scale + y0 + lane);
        // The next tile's scales come into L1 while this tile is finished.
        ff_prefetch_scales<GATED, TILE_N, SLAB_N, OUT>(p, t + num_clusters, row_in_tile + lane, part * OUT + lane);
      }
      const bool ready = mbar_wait(&acc_full_bar[acc], acc_phase, abort_flag, p.wait_budget_ns, 0x86);
      if (!__all_sync(0xffffffffu, ready)) break;
      tcgen05_fence_after_sync();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * Cfg::BN;
      const bool rows_live = y0 < p.M;
      uint32_t h[Cfg::SLABS][OUT / 2];
#pragma unroll
      for (int s = 0; s < Cfg::SLABS; ++s) {
        if (s == 0 || f.whole) {
#pragma unroll
          for (int c = 0; c < OUT / 32; ++c) {
            const int col0 = out0 + s * SLAB_N + c * 32;
            if (GATED) {
              // Result column o of the slab: with W = B_ROWS / 2 (64, or 32 in
              // the narrow tile) its gate is accumulator column 2 W (o / W) +
              // o mod W, its up value W columns further.
              constexpr int W = Cfg::B_ROWS / 2;
              const int o = part * OUT + c * 32;
              const uint32_t gaddr = taddr + s * Cfg::SLAB + (o / W) * (2 * W) + o % W;
              const bool save = KIND == kFfF16 && p.save && rows_live && col0 < p.N;
              uint32_t hg[16], hu[16];
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                uint32_t rg[16], ru[16];
                tmem_ld_32x32b_x16(gaddr + b * 16, rg);
                tmem_ld_32x32b_x16(gaddr + W + b * 16, ru);
                tmem_ld_wait();
                float g[16], u[16];
                ff_values<KIND>(rg, row_scale, p.col_scale[0], col0 + b * 16, p.N, g);
                ff_values<KIND>(ru, row_scale, p.col_scale[1], col0 + b * 16, p.N, u);
                if (save) {
                  pack_row<16>(g, hg + b * 8, p.bf16 != 0);
                  pack_row<16>(u, hu + b * 8, p.bf16 != 0);
                }
                if (p.act == kActSilu)
                  gate_row<kActSilu>(g, u);
                else if (p.act == kActGelu)
                  gate_row<kActGelu>(g, u);
                else
                  gate_row<kActRelu>(g, u);
                pack_row<16>(g, h[s] + c * 16 + b * 8, p.bf16 != 0);
              }
              if (save) {
                ff_store_box<Cfg::C_BUFS>(&maps.c[1], p.c[1], p.ldc[1], p.c_aligned[1] != 0, p.M, p.N, y0, col0, hg,
                                          wbuf + (turn % Cfg::C_BUFS) * Cfg::C_BUF_BYTES, lane, pol);
                ff_store_box<Cfg::C_BUFS>(&maps.c[2], p.c[2], p.ldc[2], p.c_aligned[2] != 0, p.M, p.N, y0, col0, hu,
                                          wbuf + ((turn + 1) % Cfg::C_BUFS) * Cfg::C_BUF_BYTES, lane, pol);
                turn += 2;
              }
            } else {
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(taddr + s * Cfg::SLAB + part * OUT + c * 32 + b * 16, r);
                tmem_ld_wait();
                const int col = col0 + b * 16;
                float v[16];
                ff_values<KIND>(r, row_scale, p.col_scale[0], col, p.N, v);
                if (KIND == kFfI8) {
                  if (p.bias != nullptr) {
                    float bias[16];
                    load_bias16(static_cast<const unsigned short*>(p.bias) + col, col, p.N, p.bf16 != 0, bias);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] += bias[e];
                  }
                  if (p.relu) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = v[e] > 0.0f ? v[e] : 0.0f;
                  }
                }
                pack_row<16>(v, h[s] + c * 16 + b * 8, p.bf16 != 0);
              }
            }
          }
        }
        tcgen05_fence_before_sync();
        __syncwarp();
        // Relaxed: the arrival orders only the TMEM reads, which are complete
        // (wait::ld) and fenced; a release would also wait for the stores of
        // the tile before.
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acc_empty_bar[acc + s]), 0));
      }
      if (rows_live) {
        const int ci = GATED ? 0 : f.row_src;
#pragma unroll
        for (int s = 0; s < Cfg::SLABS; ++s) {
          if (s > 0 && !f.whole) break;
#pragma unroll
          for (int c = 0; c < OUT / 32; ++c) {
            const int col0 = out0 + s * SLAB_N + c * 32;
            if (col0 < p.N) {
              ff_store_box<Cfg::C_BUFS>(&maps.c[ci], p.c[ci], p.ldc[ci], p.c_aligned[ci] != 0, p.M, p.N, y0, col0,
                                        h[s] + c * 16, wbuf + (turn % Cfg::C_BUFS) * Cfg::C_BUF_BYTES, lane, pol);
              ++turn;
            }
          }
        }
      }
    }
  }

  if (warp >= Cfg::EPI_WARP0 && lane == 0) bulk_wait_group<0>();  // the results are written
  tcgen05_fence_before_sync();
  __syncthreads();
  cluster_sync();  // the pair is done with each other's shared memory and barriers
  if (warp == Cfg::MMA_WARP) {
    tcgen05_fence_after_sync();
    tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
  }
}

}  // namespace tg
