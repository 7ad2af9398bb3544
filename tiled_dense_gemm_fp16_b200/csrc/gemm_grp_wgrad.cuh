// gemm_grp_wgrad.cuh -- weight gradients of the grouped products:
// dW_g = sum over the rows r of group g of dY[r] X[r]^T, on CTA pairs, persistent.
//
// The sum runs over a ragged range of rows, so both operands are stored with the
// sum's index outermost (MN-major), in k-blocks of 64 rows.  A tile is 256 x 256 of one
// dW_g, with two accumulators.  Where a group ends inside 16 rows (an MMA's
// depth), the rows behind it belong to another group, or to nobody: a warp of
// each CTA overwrites them with zeros in shared memory, in both operands (zeros
// in one would still meet the other's infinities), before that block's MMAs; its
// further 16-row steps are left out.  Groups without rows get zeros.
//
// Measured alone: 16384 rows in 8 groups, 4096 x 4096, 377 us, 1.46 PFLOP/s, tensor
// pipe 81 % busy, which bounds it (and the power cap, in a row of calls).  8192 rows in 63 of 64 groups, 1024 x 2048: 83 us
// for sums of two k-blocks a tile and 268 MB of results; bound by writing them (a plain
// fill of as much memory takes 70 us here, 3.8 TB/s: writes have little more than half
// of the rate of reads).  Not split over the rows: few tiles of long sums (one group of
// 1992 rows, 128 x 104: 16 us) leave most pairs idle.
#pragma once

#include "grp_ops.cuh"

namespace tg {

struct GrpWgradMaps {
  CUtensorMap d;  // dY, boxes of 64 columns and 64 rows
  CUtensorMap x;  // X, the same
  CUtensorMap c;  // dW, boxes of 32 x 32 of one matrix
};

// One box of results to matrix z of a stack.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

struct GrpWgradParams {
  void* c;
  int64_t ldc, stride_c;  // rows of one dW_g, and from one to the next
  const int* ends;
  int M, groups;
  int N, K;               // dW_g is N x K
  int n_tiles, k_tiles, num_tiles;
  int vec;
  int bf16;
  uint32_t idesc;
  uint64_t wait_budget_ns;
};

struct GrpWgradCfg {
  static constexpr int STAGES = 5;
  static constexpr int BM = 128;
  static constexpr int TILE = 256;
  static constexpr int PANEL_BYTES = 64 * 128;
  static constexpr int A_BYTES = 2 * PANEL_BYTES;  // 128 columns of dY
  static constexpr int B_BYTES = 2 * PANEL_BYTES;  // 128 columns of X
  static constexpr int MMA_WARP = 1;
  static constexpr int ZERO_WARP = 2;
  static constexpr int EPI_WARP0 = 3;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
  static constexpr int TMEM_COLS = 512;
  static constexpr int BOX_BYTES = 2 * kGrpBoxBytes;  // a warp's two staging boxes
  static constexpr int STAGING = EPI_WARPS * BOX_BYTES;
  static constexpr int BAR_BYTES = 256;
  static constexpr int FIXED_SMEM = 1024 + STAGES * (A_BYTES + B_BYTES) + STAGING + BAR_BYTES;
  static constexpr int smem_bytes(int groups) { return FIXED_SMEM + (groups + 1) * 4; }
  static_assert(FIXED_SMEM + (kGrpMaxGroups + 1) * 4 <= 232448, "dynamic shared memory per CTA");
  static_assert((3 * STAGES + 5) * 8 + 8 <= BAR_BYTES, "barriers");
};

// The tiles of one cluster, in turn: group, place, rows of the sum.
struct GrpWgradTile {
  int g, n_blk, k_blk;
  int lo, rows;
};
struct GrpWgradWalk {
  int g, local;  // tile of the group; from one tile to the next by subtraction
  float inv_last;  // of the last, narrower strip

  __device__ __forceinline__ GrpWgradWalk(const GrpWgradParams& p, int first) {
    g = first / (p.n_tiles * p.k_tiles);
    local = first - g * p.n_tiles * p.k_tiles;
    inv_last = 1.0f / static_cast<float>(max(1, p.n_tiles % 8));
  }
  __device__ __forceinline__ void skip(const GrpWgradParams& p, int tiles) {
    local += tiles;
    for (const int per = p.n_tiles * p.k_tiles; local >= per; ++g) local -= per;
  }
  // By a whole warp.
  __device__ __forceinline__ GrpWgradTile tile(const GrpWgradParams& p, const int* ends) const {
    GrpWgradTile f;
    f.g = g;
    // Eight tiles of dY's columns next to each other for one of X's.
    int s = 0, in = local;
    while (in >= 8 * p.k_tiles && 8 * (s + 1) < p.n_tiles) {
      in -= 8 * p.k_tiles;
      ++s;
    }
    const int wide = min(8, p.n_tiles - 8 * s);
    f.k_blk = wide == 8 ? in >> 3 : quick_div(in, wide, inv_last);
    f.n_blk = 8 * s + in - f.k_blk * wide;
    f.lo = uniform(ends[g]);
    f.rows = uniform(ends[g + 1]) - f.lo;
    return f;
  }
};

__global__ void __launch_bounds__(GrpWgradCfg::THREADS, 1)
    grp_wgrad_kernel(const __grid_constant__ GrpWgradMaps maps, const GrpWgradParams p) {
  using Cfg = GrpWgradCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* a_smem = smem;
  uint8_t* b_smem = smem + Cfg::STAGES * Cfg::A_BYTES;
  uint8_t* staging = smem + Cfg::STAGES * (Cfg::A_BYTES + Cfg::B_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + Cfg::STAGING);
  uint64_t* full_bar = bars;                        // used in the even CTA
  uint64_t* empty_bar = bars + Cfg::STAGES;         // per CTA
  uint64_t* tail_bar = bars + 2 * Cfg::STAGES;      // per CTA: a group's last block has landed
  uint64_t* acc_full_bar = bars + 3 * Cfg::STAGES;  // per CTA
  uint64_t* acc_empty_bar = acc_full_bar + 2;       // used in the even CTA
  uint64_t* mma_done_bar = acc_empty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* ends = reinterpret_cast<int*>(staging + Cfg::STAGING + Cfg::BAR_BYTES);  // from 0 on

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1;
  const int num_clusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(&full_bar[s], 2);  // two of the leader's producer, or one of each CTA's zeroing warp
      mbar_init(&empty_bar[s], 1);
      mbar_init(&tail_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full_bar[b], 1);
      mbar_init(&acc_empty_bar[b], 2 * Cfg::EPI_WARPS);
    }
    mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&maps.d);
    tma_prefetch_desc(&maps.x);
  }
  if (warp == Cfg::MMA_WARP) {
    tmem_alloc_pair(tmem_slot, Cfg::TMEM_COLS);
    tmem_relinquish_alloc_permit_pair();
  }
  tcgen05_fence_before_sync();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised before any remote use
  tcgen05_fence_after_sync();
  grid_dependency_wait();
  grid_launch_dependents();
  bool rising = true;
  for (int g = threadIdx.x; g <= p.groups; g += Cfg::THREADS) {
    ends[g] = grp_end(p.ends, g - 1, p.M);
    rising = rising && ends[g] >= grp_end(p.ends, g - 2, p.M);
  }
  if (!__syncthreads_and(rising)) {
    if (warp == Cfg::ZERO_WARP)
      for (int g = lane, top = 0; g - lane <= p.groups; g += 32) {
        const int lo = grp_raise(g <= p.groups ? ends[g] : p.M, top, lane);
        if (g <= p.groups) ends[g] = lo;
      }
    __syncthreads();
  }
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // As in gemm_grp_pair.cuh: the warp loops, one lane issues.
    const bool one = elect_one();
    int stage = 0;
    uint32_t phase = 0, used = 0, parities = 0;
    bool ok = true;
    const uint64_t pol = l2_policy_evict_normal();
    const uint32_t full_even0 = mapa_shared(smem_u32(full_bar), 0);
    GrpWgradWalk walk(p, cluster_id);
    for (int t = cluster_id; t < p.num_tiles && ok; t += num_clusters, walk.skip(p, num_clusters)) {
      const GrpWgradTile f = walk.tile(p, ends);
      const int n0 = f.n_blk * Cfg::TILE + static_cast<int>(rank) * Cfg::BM;
      const int k0 = f.k_blk * Cfg::TILE + static_cast<int>(rank) * Cfg::BM;
      for (int r = 0; r < f.rows; r += 64) {
        if (!mbar_wait_warp(&empty_bar[stage], phase ^ 1u, abort_flag, p.wait_budget_ns, 0xc1)) {
          ok = false;
          break;
        }
        if (one) {
          uint8_t* adst = a_smem + stage * Cfg::A_BYTES;
          uint8_t* bdst = b_smem + stage * Cfg::B_BYTES;
          const int y = f.lo + r;
          if ((min(64, f.rows - r) & 15) == 0) {
            const uint32_t full = full_even0 + stage * 8;
            if (leader) {
              mbar_arrive(&full_bar[stage]);
              mbar_arrive_expect_tx(&full_bar[stage], 2 * (Cfg::A_BYTES + Cfg::B_BYTES));
            }
            tma_load_2d_pair_hint(adst, &maps.d, full, n0, y, pol);
            tma_load_2d_pair_hint(adst + Cfg::PANEL_BYTES, &maps.d, full, n0 + 64, y, pol);
            tma_load_2d_pair_hint(bdst, &maps.x, full, k0, y, pol);
            tma_load_2d_pair_hint(bdst + Cfg::PANEL_BYTES, &maps.x, full, k0 + 64, y, pol);
          } else {  // to this CTA's zeroing warp first
            mbar_arrive_expect_tx(&tail_bar[stage], Cfg::A_BYTES + Cfg::B_BYTES);
            tma_load_2d_hint(adst, &maps.d, &tail_bar[stage], n0, y, pol);
            tma_load_2d_hint(adst + Cfg::PANEL_BYTES, &maps.d, &tail_bar[stage], n0 + 64, y, pol);
            tma_load_2d_hint(bdst, &maps.x, &tail_bar[stage], k0, y, pol);
            tma_load_2d_hint(bdst + Cfg::PANEL_BYTES, &maps.x, &tail_bar[stage], k0 + 64, y, pol);
          }
        }
        used |= 1u << stage;
        parities = (parities & ~(1u << stage)) | phase << stage;
        if (++stage == Cfg::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // The even CTA's full barriers count both CTAs' bytes, or both zeroing warps.
    if (leader) {
      for (int s = 0; s < Cfg::STAGES; ++s) {
        if (used >> s & 1u) {
          volatile int no_abort = 0;
          mbar_wait(&full_bar[s], parities >> s & 1u, &no_abort, p.wait_budget_ns, 0xc2);
        }
      }
    }
  } else if (warp == Cfg::MMA_WARP) {
    if (leader) {
      const bool one = elect_one();
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;
      bool ok = true;
      const uint64_t a_desc0 = make_sw128_desc(smem_u32(a_smem), Cfg::PANEL_BYTES, 1024);
      const uint64_t b_desc0 = make_sw128_desc(smem_u32(b_smem), Cfg::PANEL_BYTES, 1024);
      const uint32_t tmem = uniform(tmem_base);
      GrpWgradWalk walk(p, cluster_id);
      for (int t = cluster_id; t < p.num_tiles && ok; t += num_clusters, walk.skip(p, num_clusters)) {
        const GrpWgradTile f = walk.tile(p, ends);
        if (f.rows == 0) continue;
        const int acc = local & 1;
        if (!mbar_wait_warp(&acc_empty_bar[acc], ((local >> 1) & 1) ^ 1u, abort_flag, p.wait_budget_ns, 0xc3)) break;
        tcgen05_fence_after_sync();
        const uint32_t d_tmem = tmem + acc * Cfg::TILE;
        for (int r = 0; r < f.rows; r += 64) {
          // Acquire at cluster scope: the other CTA's zeroing warp may have arrived.
          if (!__all_sync(0xffffffffu, mbar_wait_cluster(&full_bar[stage], phase, abort_flag, p.wait_budget_ns, 0xc4))) {
            ok = false;
            break;
          }
          tcgen05_fence_after_sync();
          const uint64_t a_desc = a_desc0 + stage * (Cfg::A_BYTES / 16), b_desc = b_desc0 + stage * (Cfg::B_BYTES / 16);
          const int steps = (min(64, f.rows - r) + 15) / 16;
          if (one) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < steps)
                umma_f16_ss_pair(d_tmem, a_desc + k * (2048 / 16), b_desc + k * (2048 / 16), p.idesc, (r | k) != 0 ? 1u : 0u);
            umma_commit_pair_mc(&empty_bar[stage], 0x3);
          }
          if (++stage == Cfg::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (one) umma_commit_pair_mc(&acc_full_bar[acc], 0x3);
        ++local;
      }
      if (one) umma_commit_pair_mc(mma_done_bar, 0x1);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(mma_done_bar, 0, &no_abort, p.wait_budget_ns, 0xc5);
    }
    __syncwarp();
  } else if (warp == Cfg::ZERO_WARP) {
    // Rows behind a group's end, up to the next 16, in this CTA's operands.
    const uint32_t full_even0 = mapa_shared(smem_u32(full_bar), 0);
    int stage = 0;
    uint32_t tail_phase = 0;  // a bit a stage
    GrpWgradWalk walk(p, cluster_id);
    for (int t = cluster_id; t < p.num_tiles; t += num_clusters, walk.skip(p, num_clusters)) {
      const GrpWgradTile f = walk.tile(p, ends);
      const int blocks = (f.rows + 63) / 64;
      if (blocks == 0) continue;
      const int last = (stage + blocks - 1) % Cfg::STAGES;
      const int have = f.rows - (blocks - 1) * 64;
      if ((have & 15) != 0) {
        const bool landed = mbar_wait(&tail_bar[last], (tail_phase >> last) & 1u, abort_flag, p.wait_budget_ns, 0xc7);
        if (!__all_sync(0xffffffffu, landed)) break;
        tail_phase ^= 1u << last;
        const int pieces = (16 - (have & 15)) * 8;  // of 16 bytes in a panel
        for (int i = lane; i < 4 * pieces; i += 32) {
          const int panel = i / pieces, at = i - panel * pieces;
          uint8_t* base = (panel < 2 ? a_smem + last * Cfg::A_BYTES : b_smem + last * Cfg::B_BYTES) + (panel & 1) * Cfg::PANEL_BYTES;
          *reinterpret_cast<uint4*>(base + have * 128 + at * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(full_even0 + last * 8);
      }
      stage = (last + 1) % Cfg::STAGES;
    }
  } else {
    const int quad = warp & 3;
    const int part = (warp - Cfg::EPI_WARP0) >> 2;
    uint8_t* boxes = staging + (warp - Cfg::EPI_WARP0) * Cfg::BOX_BYTES;
    int turn = 0;
    const bool bf16 = p.bf16 != 0;
    int local = 0;
    GrpWgradWalk walk(p, cluster_id);
    for (int t = cluster_id; t < p.num_tiles; t += num_clusters, walk.skip(p, num_clusters)) {
      const GrpWgradTile f = walk.tile(p, ends);
      const int n0 = f.n_blk * Cfg::TILE + static_cast<int>(rank) * Cfg::BM + quad * 32;
      const bool zero = f.rows == 0;
      const int acc = local & 1;
      if (!zero) {
        const bool ready = mbar_wait(&acc_full_bar[acc], (local >> 1) & 1, abort_flag, p.wait_budget_ns, 0xc6);
        if (!__all_sync(0xffffffffu, ready)) break;
        tcgen05_fence_after_sync();
      }
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * Cfg::TILE;
      unsigned short* dst = static_cast<unsigned short*>(p.c) + f.g * p.stride_c + n0 * p.ldc;
      for (int b = part; b < Cfg::TILE / 32; b += Cfg::EPI_WARPS / 4) {
        const int k0 = f.k_blk * Cfg::TILE + b * 32;
        if (n0 >= p.N || k0 >= p.K) break;
        uint32_t h[16];
        if (!zero) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(taddr + b * 32, r);
          tmem_ld_wait();
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
          pack_row<32>(v, h, bf16);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) h[e] = 0u;
        }
        // As ff_store_box, with TMA boxes of one matrix of the stack.
        uint8_t* box = boxes + (turn++ & 1) * kGrpBoxBytes;
        if (p.vec && (k0 + 32 <= p.K || (p.K & 7) == 0)) {
          if (lane == 0) bulk_wait_group_read<1>();  // the last but one has left
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(box + grp_box_at(lane, q)) = make_uint4(h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&maps.c, box, k0, n0, f.g);
            bulk_commit_group();
          }
        } else {
          ff_store_box<2>(nullptr, dst - n0 * p.ldc, p.ldc, false, p.N, p.K, n0, k0, h, box, lane, 0);
        }
      }
      if (!zero) {
        tcgen05_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acc_empty_bar[acc]), 0));
        ++local;
      }
    }
  }

  if (warp >= Cfg::EPI_WARP0 && lane == 0) bulk_wait_group<0>();  // the results are written
  tcgen05_fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == Cfg::MMA_WARP) {
    tcgen05_fence_after_sync();
    tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
  }
}

}  // namespace tg
