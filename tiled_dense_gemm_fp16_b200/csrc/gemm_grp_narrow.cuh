// gemm_grp_narrow.cuh -- the products of gemm_grp_pair.cuh where whole tiles
// would leave most SMs idle: decoding batches (a few rows per group, bound by
// streaming the weights that have rows once) and small results.
//
// A cluster of S CTAs takes a panel of 128 weight rows and up to `tokens` rows of
// one group, splits the sum over its CTAs, and adds the S partials out of each
// other's shared memory in rank order (so results do not depend on timing).  The
// kernel is persistent: which groups have rows is known on the device only, so
// each cluster walks the tiles there are, its loads running ahead into the next
// tile while the partials of the last one are added.
#pragma once

#include "gemm_ff_skinny.cuh"
#include "gemm_grp_pair.cuh"

namespace tg {

struct GrpNarrowParams {
  GrpParams g;         // col_tiles: panels of 128 columns; idesc without N
  int tokens;          // most of a tile: 16, 32, 64 or 128
  int splits, stages;
  uint32_t tmem_cols;  // two accumulators
};

struct GrpNarrowCfg {
  static constexpr int PANEL = 128;
  static constexpr int W_BYTES = PANEL * 128;
  static constexpr int HALF_BYTES = W_BYTES / 2;
  static constexpr int UNIT = 16;
  static constexpr int EPI_WARP0 = 2;
  static constexpr int THREADS = 192;
  static constexpr int MAX_STAGES = 10;
  static constexpr int BAR_BYTES = 256;
  static constexpr int smem_bytes(int tokens, int stages, int groups) {
    return 1024 + stages * (W_BYTES + tokens * 128) + tokens * PANEL * 4 + BAR_BYTES + grp_plan_bytes(groups);
  }
  // As deep as fits a CTA an SM.
  static constexpr int stages(int tokens, int groups) {
    const int n = (232448 - smem_bytes(tokens, 0, groups)) / (W_BYTES + tokens * 128);
    return n > MAX_STAGES ? MAX_STAGES : n;
  }
  static_assert((2 * MAX_STAGES + 7) * 8 + 8 <= BAR_BYTES, "barriers");
  static_assert(HALF_BYTES % 1024 == 0 && UNIT * 128 % 1024 == 0, "operands start on the swizzle's 1024 bytes");
};

// Four results of a token from its partials on, with the adapter's part.
template <bool LORA>
__device__ __forceinline__ void grp_narrow_finish(const GrpNarrowParams& p, float (&v)[4], int m, int n, bool early) {
  const bool bf16 = p.g.bf16 != 0;
  if (LORA) {
    const LoraParams& l = p.g.lora;
    if (early) {
      const int a = __ldg(l.index + m);
      if (a >= 0 && a < l.adapters) {
        const unsigned short* trow = static_cast<const unsigned short*>(l.t) + static_cast<int64_t>(m) * l.rank;
        const unsigned short* brow = static_cast<const unsigned short*>(l.b) + a * l.stride_b + n * l.ldb;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (n + q < p.g.out) v[q] += lora_dot(brow + q * l.ldb, trow, l.rank, bf16);
      }
    }
    if (l.bias != nullptr) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (n + q < p.g.out) v[q] += load_16(static_cast<const unsigned short*>(l.bias) + n + q, bf16);
    }
  }
  ff_store4(p.g.c, p.g.ldc, p.g.vec != 0, m, n, p.g.out, v, bf16);
}

template <bool LORA>
__global__ void __launch_bounds__(GrpNarrowCfg::THREADS, 1)
    grp_narrow_kernel(const __grid_constant__ GrpMaps maps, const GrpNarrowParams p) {
  using Cfg = GrpNarrowCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t x_bytes = p.tokens * 128;
  uint8_t* w_smem = smem;
  uint8_t* x_smem = smem + p.stages * Cfg::W_BYTES;
  float* partial = reinterpret_cast<float*>(smem + p.stages * (Cfg::W_BYTES + x_bytes));  // [tokens][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(partial) + p.tokens * Cfg::PANEL * 4);
  uint64_t* full_bar = bars;
  uint64_t* empty_bar = bars + Cfg::MAX_STAGES;
  uint64_t* acc_full_bar = bars + 2 * Cfg::MAX_STAGES;
  uint64_t* acc_empty_bar = acc_full_bar + 2;
  uint64_t* part_full_bar = acc_empty_bar + 2;   // every CTA's partial is written
  uint64_t* part_empty_bar = part_full_bar + 1;  // every CTA has read this one's
  uint64_t* mma_done_bar = part_empty_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  GrpPlan plan;
  plan.lo = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + Cfg::BAR_BYTES);
  plan.first = plan.lo + p.g.groups + 2;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cluster_id = blockIdx.x / p.splits;
  const int num_clusters = gridDim.x / p.splits;
  const int kb_lo = static_cast<int>(static_cast<int64_t>(p.g.k_blocks) * rank / p.splits);
  const int kb_hi = static_cast<int>(static_cast<int64_t>(p.g.k_blocks) * (rank + 1) / p.splits);  // > kb_lo: splits <= k_blocks

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full_bar[b], 1);
      mbar_init(&acc_empty_bar[b], 4);
    }
    mbar_init(part_full_bar, 4 * p.splits);
    mbar_init(part_empty_bar, 4 * p.splits);
    mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.x[0]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish_alloc_permit();
  }
  const bool early = LORA && p.g.lora.adapters > 0;  // as in the pair kernel
  if (!early) {
    grid_dependency_wait();
    grid_launch_dependents();
  }
  if (warp == Cfg::EPI_WARP0)
    grp_make_plan(plan, p.g.ends, p.g.groups, p.g.M, p.tokens, p.g.col_tiles, p.g.rest != 0, lane);
  tcgen05_fence_before_sync();
  __syncthreads();
  cluster_sync();  // every CTA's barriers are initialised before any remote use
  tcgen05_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const int num_tiles = plan.first[p.g.groups + 1];

  if (warp == 0) {
    // Producer: this CTA's slice of the sum.
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int last_parity[Cfg::MAX_STAGES];
#pragma unroll
      for (int s = 0; s < Cfg::MAX_STAGES; ++s) last_parity[s] = -1;
      bool ok = true;
      const uint64_t pol_w = l2_policy_evict_first();
      const uint64_t pol_x = l2_policy_evict_last();
      GrpWalk walk;
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
        const GrpTile f = walk.at(plan, t, p.g.col_tiles, p.g.super, p.tokens, Cfg::UNIT);
        if (f.g == p.g.groups) break;
        const int width = (f.cnt + Cfg::UNIT - 1) / Cfg::UNIT * Cfg::UNIT;
        const int n0 = f.col_blk * Cfg::PANEL;
        const uint32_t tx = Cfg::W_BYTES + width * 128;
        for (int kb = kb_lo; kb < kb_hi; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, p.g.wait_budget_ns, 0xb1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full_bar[stage], tx);
          const int k0 = kb * 64;
          uint8_t* wdst = w_smem + stage * Cfg::W_BYTES;
          uint8_t* xdst = x_smem + stage * x_bytes;
          if (p.g.w_mn) {
            tma_load_3d_hint(wdst, &maps.w, &full_bar[stage], n0, k0, f.g, pol_w);
            tma_load_3d_hint(wdst + Cfg::HALF_BYTES, &maps.w, &full_bar[stage], n0 + 64, k0, f.g, pol_w);
          } else {
            tma_load_3d_hint(wdst, &maps.w, &full_bar[stage], k0, n0, f.g, pol_w);
          }
          grp_token_boxes(width, [&](int b, int at) {
            tma_load_2d_hint(xdst + at * 128, &maps.x[b], &full_bar[stage], k0, f.tok0 + at, pol_x);
          });
          last_parity[stage] = static_cast<int>(phase);
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
#pragma unroll
      for (int s = 0; s < Cfg::MAX_STAGES; ++s) {
        if (last_parity[s] >= 0) {
          volatile int no_abort = 0;
          mbar_wait(&full_bar[s], static_cast<uint32_t>(last_parity[s]), &no_abort, p.g.wait_budget_ns, 0xb2);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;
      bool ok = true;
      const uint64_t w_desc0 = make_sw128_desc(smem_u32(w_smem), p.g.w_mn ? Cfg::HALF_BYTES : 16, 1024);
      const uint64_t x_desc0 = make_sw128_desc(smem_u32(x_smem), 16, 1024);
      const uint32_t w_step = p.g.w_mn ? 2048 / 16 : 32 / 16;
      GrpWalk walk;
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters, ++local) {
        const GrpTile f = walk.at(plan, t, p.g.col_tiles, p.g.super, p.tokens, Cfg::UNIT);
        if (f.g == p.g.groups) break;
        const int width = (f.cnt + Cfg::UNIT - 1) / Cfg::UNIT * Cfg::UNIT;
        const uint32_t idesc = p.g.idesc | static_cast<uint32_t>(width >> 3) << 17;
        const int acc = local & 1;
        if (!mbar_wait(&acc_empty_bar[acc], ((local >> 1) & 1) ^ 1u, abort_flag, p.g.wait_budget_ns, 0xb3)) break;
        tcgen05_fence_after_sync();
        const uint32_t d_tmem = tmem_base + acc * p.tokens;
        for (int kb = kb_lo; kb < kb_hi; ++kb) {
          if (!mbar_wait(&full_bar[stage], phase, abort_flag, p.g.wait_budget_ns, 0xb4)) {
            ok = false;
            break;
          }
          tcgen05_fence_after_sync();
          const uint64_t w_desc = w_desc0 + stage * (Cfg::W_BYTES / 16), x_desc = x_desc0 + stage * (x_bytes / 16);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_f16_ss(d_tmem, w_desc + k * w_step, x_desc + k * 2, idesc, (kb - kb_lo) | k ? 1u : 0u);
          umma_commit(&empty_bar[stage]);
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit(&acc_full_bar[acc]);
      }
      umma_commit(mma_done_bar);
      volatile int no_abort = 0;
      mbar_wait(mma_done_bar, 0, &no_abort, p.g.wait_budget_ns, 0xb5);
    }
    __syncwarp();
  } else {
    const int quad = warp & 3;
    const int e = threadIdx.x - Cfg::EPI_WARP0 * 32;
    const int step = p.splits * 128;
    GrpWalk walk;
    int local = 0;
    bool waited = false;
    for (int t = cluster_id; t < num_tiles; t += num_clusters) {
      const GrpTile f = walk.at(plan, t, p.g.col_tiles, p.g.super, p.tokens, Cfg::UNIT);
      const int n0 = f.col_blk * Cfg::PANEL;
      const int items = f.cnt * 32;  // (token, four columns)
      if (f.g == p.g.groups) {
        for (int it = rank * 128 + e; it < items; it += step) {
          const int n = n0 + (it & 31) * 4;
          const float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if (n < p.g.out) ff_store4(p.g.c, p.g.ldc, p.g.vec != 0, f.tok0 + (it >> 5), n, p.g.out, v, p.g.bf16 != 0);
        }
        continue;
      }
      if (early && !waited) {
        // The adapters' rows that this tile's results need come into L2 meanwhile.
        for (int it = rank * 128 + e; it < items; it += step) {
          const int n = n0 + (it & 31) * 4;
          const int a = __ldg(p.g.lora.index + f.tok0 + (it >> 5));
          if (a < 0 || a >= p.g.lora.adapters || n >= p.g.out) continue;
          const char* row = reinterpret_cast<const char*>(static_cast<const unsigned short*>(p.g.lora.b) + a * p.g.lora.stride_b +
                                                          n * p.g.lora.ldb);
          const int64_t pitch = p.g.lora.ldb * 2;
          for (int q = 0; q < 4 && n + q < p.g.out; ++q)
            for (int at = 0; at < p.g.lora.rank * 2; at += 128)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(row + q * pitch + at));
        }
      }
      const int acc = local & 1;
      bool ready = mbar_wait(&acc_full_bar[acc], (local >> 1) & 1, abort_flag, p.g.wait_budget_ns, 0xb6);
      // Every CTA has read the partial before.
      if (ready) ready = mbar_wait_cluster(part_empty_bar, (local & 1) ^ 1u, abort_flag, p.g.wait_budget_ns, 0xb7);
      if (!__all_sync(0xffffffffu, ready)) break;
      tcgen05_fence_after_sync();
      for (int c = 0; c < (f.cnt + 15) / 16; ++c) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * p.tokens + c * 16, r);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 16; ++q) partial[(c * 16 + q) * Cfg::PANEL + quad * 32 + lane] = __uint_as_float(r[q]);
      }
      tcgen05_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&acc_empty_bar[acc]);
        for (int s = 0; s < p.splits; ++s) mbar_arrive_cluster(mapa_shared(smem_u32(part_full_bar), s));
      }
      ready = mbar_wait_cluster(part_full_bar, local & 1, abort_flag, p.g.wait_budget_ns, 0xb8);
      if (!__all_sync(0xffffffffu, ready)) break;
      if (early && !waited) {
        grid_dependency_wait();  // T
        grid_launch_dependents();
        waited = true;
      }
      for (int it = rank * 128 + e; it < items; it += step) {
        const int n = n0 + (it & 31) * 4;
        if (n >= p.g.out) continue;
        float4 x[8];
        ff_cluster_read(smem_u32(partial) + ((it >> 5) * Cfg::PANEL + (it & 31) * 4) * 4, p.splits, x);
        float v[4];
        ff_cluster_sum<kFfF16>(x, p.splits, v);
        grp_narrow_finish<LORA>(p, v, f.tok0 + (it >> 5), n, early);
      }
      __syncwarp();
      if (lane == 0)
        for (int s = 0; s < p.splits; ++s) mbar_arrive_cluster(mapa_shared(smem_u32(part_empty_bar), s));
      ++local;
    }
    if (early && !waited) {  // nothing to do: the grid still ends after the one before
      grid_dependency_wait();
      grid_launch_dependents();
    }
  }

  tcgen05_fence_before_sync();
  __syncthreads();
  cluster_sync();  // peers are done reading this CTA's partial
  if (warp == 1) {
    tcgen05_fence_after_sync();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

}  // namespace tg
