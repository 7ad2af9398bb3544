// gemm_grp_narrow.cuh -- the products of gemm_grp_pair.cuh where whole tiles
// would leave most SMs idle: decoding batches (a few rows per group, bound by
// streaming the weights that have rows once) and small results.
//
// A cluster of S CTAs takes a panel of 128 weight rows and up to `tokens` rows of
// one group and splits the sum over its CTAs.  Each CTA finishes 128 / S of the
// panel's columns: the others write their partials into its shared memory, and
// it adds them in rank order, so results do not depend on timing.  The kernel is
// persistent: which groups have rows is known on the device only, so each cluster
// walks the tiles there are, its loads running ahead into the next tile while the
// partials of the last one are added.  Adapters' T is made here too where it is a
// value a warp: one or two tokens, 8 values with clusters of two CTAs, 16 with four
// (grp_lora_own_t).
//
// Bound by reading the weights that have rows: 512 rows in 60 of 64 groups of 2048 x
// 4096 (1.01 GB) 155 us, 6.5 TB/s, the rate of a plain copy; 8 rows in 8 groups (134
// MB) 26.7 us, 5.0 TB/s, of which 5 us are the launch and the first loads.
#pragma once

#include "gemm_ff_skinny.cuh"
#include "gemm_grp_pair.cuh"

namespace tg {

struct GrpNarrowParams {
  GrpParams g;         // col_tiles: panels of 128 columns; idesc without N
  int tokens;          // most of a tile: 16, 32, 64 or 128
  int splits, stages;  // 1, 2 or 4 splits
  int per_stage;       // k-blocks of a stage of the ring
  int own_t;           // adapters: T is made here
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
  // Partials of a tile: [source][column][tokens + 4], the 4 to spread the columns over the banks.
  __host__ __device__ static constexpr int recv_bytes(int tokens) { return PANEL * (tokens + 4) * 4; }
  // The adapters' part of this CTA's columns: [column][tokens + 4].
  static constexpr int delta_bytes(int tokens, int splits) { return PANEL / splits * (tokens + 4) * 4; }
  static constexpr int smem_bytes(int tokens, int stages, int groups) {
    return 1024 + stages * (W_BYTES + tokens * 128) + recv_bytes(tokens) + BAR_BYTES + grp_plan_align(groups);
  }
  // And T where it is made here, a value by each warp that finishes results: up to 16
  // of 16 bits in bf16, in fp16 of 32 bits, from which each warp makes its own of 16
  // bits and their powers (48 bytes apart).
  static constexpr int own_t(int splits) { return 4 * splits; }
  static constexpr int OWN_T_BYTES = 64 + 4 * 48;
  static constexpr int lora_bytes(int tokens, int splits, bool with_t) {
    return delta_bytes(tokens, splits) + (with_t ? OWN_T_BYTES : 0);
  }
  static_assert((2 * MAX_STAGES + 8) * 8 + 8 <= BAR_BYTES, "barriers");
  static_assert(HALF_BYTES % 1024 == 0 && UNIT * 128 % 1024 == 0, "operands start on the swizzle's 1024 bytes");
};

// The adapters of a tile's tokens: a warp's lane holds those of lane + 32 i.
struct GrpTileAdapters {
  int a[4];
  __device__ __forceinline__ void load(const LoraParams& l, int tok0, int cnt, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = 32 * i + lane < cnt ? lora_adapter(l, tok0 + 32 * i + lane) : -1;
  }
  // Of token t + lane, for 16 lanes and t a multiple of 16.
  __device__ __forceinline__ int from(int t) const {
    const int i = t >> 5, lane = threadIdx.x & 31;
    return __shfl_sync(0xffffffffu, i == 0 ? a[0] : i == 1 ? a[1] : i == 2 ? a[2] : a[3], (t & 31) + (lane & 15));
  }
  // Of token t, the same in the whole warp.
  __device__ __forceinline__ int of(int t) const {
    const int i = t >> 5;
    return __shfl_sync(0xffffffffu, i == 0 ? a[0] : i == 1 ? a[1] : i == 2 ? a[2] : a[3], t & 31);
  }
};

// Results of column n and up to eight tokens from `tok` of the tile on; `delta` holds the adapters' part, if there is one.
__device__ __forceinline__ void grp_narrow_store(const GrpParams& p, float (&v)[8], const GrpTile& f, int tok, int n,
                                                 const float* delta, float bias) {
  if (n >= p.out) return;
  const bool bf16 = p.bf16 != 0;
  unsigned short* c = static_cast<unsigned short*>(p.c) + (f.tok0 + tok) * p.ldc + n;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    if (delta != nullptr) v[q] += delta[q];
    if (q < f.cnt - tok) c[q * p.ldc] = round_16(v[q] + bias, bf16);
  }
}

// 8 values from p (on 16 bytes) on, of which n are in the row.
__device__ __forceinline__ uint4 lora_row8(const unsigned short* p, int n) {
  if (n >= 8) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) w[e >> 1] |= static_cast<uint32_t>(__ldg(p + e)) << ((e & 1) * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The inner product of two rows of K values, by a warp; DEEP times 256 values of each are in flight.
template <bool BF16, int DEEP>
__device__ __forceinline__ float lora_dot(const unsigned short* a, const unsigned short* x, int K, int lane) {
  float2 s = make_float2(0.0f, 0.0f);
  for (int k = lane * 8; k - lane * 8 < K; k += DEEP * 256) {
    uint4 u[DEEP], v[DEEP];
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      u[i] = lora_row8(a + k + 256 * i, K - k - 256 * i);
      v[i] = lora_row8(x + k + 256 * i, K - k - 256 * i);
    }
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      s = fma2(unpack_16(u[i].x, BF16), unpack_16(v[i].x, BF16), s);
      s = fma2(unpack_16(u[i].y, BF16), unpack_16(v[i].y, BF16), s);
      s = fma2(unpack_16(u[i].z, BF16), unpack_16(v[i].z, BF16), s);
      s = fma2(unpack_16(u[i].w, BF16), unpack_16(v[i].w, BF16), s);
    }
  }
  float sum = s.x + s.y;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

// T of all tokens, of which there are no more values than warps, into every CTA of
// the cluster: value v by this warp.  In fp16 still of 32 bits: the eight ranks
// that share a power come from two CTAs.
template <bool BF16>
__device__ __forceinline__ void lora_own_t(const LoraParams& l, void* t, int M, int K, int v, int ctas, int lane) {
  if (v >= M * l.rank) return;
  const int m = v / l.rank, a = lora_adapter(l, m);
  if (a < 0) return;
  const float sum = lora_dot<BF16, 8>(static_cast<const unsigned short*>(l.a) + a * l.stride_a + (v - m * l.rank) * l.lda,
                                      static_cast<const unsigned short*>(l.x) + m * l.ldx, K, lane);
  const float scale = l.scale != nullptr ? __ldg(l.scale + a) : 1.0f;
  if (lane < ctas) {
    if (BF16)
      st_cluster_u16(mapa_shared(smem_u32(static_cast<unsigned short*>(t) + v), lane), round_16(sum * scale, true));
    else
      st_cluster_f32(mapa_shared(smem_u32(static_cast<float*>(t) + v), lane), sum * scale);
  }
}
// The 16-bit form of those n values and the powers of eight each, by a warp for itself.
__device__ __forceinline__ void lora_own_round(const float* t, int n, unsigned short* to, signed char* exps, int lane) {
  const float v = lane < n ? t[lane] : 0.0f;
  const LoraRounded r = lora_round(v);
  if (lane < n) to[lane] = r.y;
  if (lane < n && (lane & 7) == 0) exps[lane >> 3] = static_cast<signed char>(r.e);
  __syncwarp();
}

// LORA as in the pair kernel.
template <int LORA>
__global__ void __maxnreg__(240)  // of 192 threads, so that the kernel that makes T finds registers beside it
    grp_narrow_kernel(const __grid_constant__ GrpMaps maps, const GrpNarrowParams p) {
  using Cfg = GrpNarrowCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t x_bytes = p.tokens * 128;
  uint8_t* w_smem = smem;
  uint8_t* x_smem = smem + p.stages * p.per_stage * Cfg::W_BYTES;
  float* recv = reinterpret_cast<float*>(smem + p.stages * p.per_stage * (Cfg::W_BYTES + x_bytes));
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(recv) + Cfg::recv_bytes(p.tokens));
  uint64_t* full_bar = bars;
  uint64_t* empty_bar = bars + Cfg::MAX_STAGES;
  uint64_t* acc_full_bar = bars + 2 * Cfg::MAX_STAGES;
  uint64_t* acc_empty_bar = acc_full_bar + 2;
  uint64_t* part_full_bar = acc_empty_bar + 2;   // every CTA's partials of this one's columns are here
  uint64_t* part_empty_bar = part_full_bar + 1;  // every CTA has added what this one sent
  uint64_t* mma_done_bar = part_empty_bar + 1;
  uint64_t* t_bar = mma_done_bar + 1;            // adapters: every CTA's values of T are here
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(t_bar + 1);
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
    mbar_init(part_full_bar, 4);  // S sources, of each the 4 / S warps that hold this CTA's columns
    mbar_init(part_empty_bar, 4 * p.splits);
    mbar_init(mma_done_bar, 1);
    mbar_init(t_bar, 4 * p.splits);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&maps.w);
    for (int b = 0; b < 4 && 16 << b <= p.tokens; ++b) tma_prefetch_desc(&maps.x[b]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish_alloc_permit();
  }
  tcgen05_fence_before_sync();
  __syncthreads();
  cluster_sync();  // every CTA's barriers are initialised before any remote use
  tcgen05_fence_after_sync();
  const bool adapted = LORA != 0 && p.g.lora.adapters > 0;
  const bool early = adapted && !p.own_t;  // as in the pair kernel
  const bool beside = LORA == 0 && p.g.beside != 0;
  if (!early) {
    if (!beside) grid_dependency_wait();
    grid_launch_dependents();
  }
  if (warp == Cfg::EPI_WARP0)
    grp_make_plan(plan, p.g.ends, p.g.groups, p.g.M, p.tokens, p.g.col_tiles, p.g.rest != 0, lane);
  __syncthreads();
  const uint32_t tmem_base = *tmem_slot;
  const int num_tiles = plan.first[p.g.groups + 1];

  if (warp == 0) {
    // Producer: this CTA's slice of the sum.  The loop is the warp's, so that
    // addresses and coordinates are in uniform registers where the TMA and MMA
    // instructions want them; one lane issues.
    const bool one = elect_one();
    int stage = 0;
    uint32_t phase = 0, used = 0, parities = 0;
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
      for (int kb = kb_lo; kb < kb_hi; kb += p.per_stage) {
        if (!mbar_wait_warp(&empty_bar[stage], phase ^ 1u, abort_flag, p.g.wait_budget_ns, 0xb1)) {
          ok = false;
          break;
        }
        if (one) {
          const int n = min(p.per_stage, kb_hi - kb);
          mbar_arrive_expect_tx(&full_bar[stage], n * tx);
          for (int i = 0; i < n; ++i) {
            const int k0 = (kb + i) * 64;
            uint8_t* wdst = w_smem + (stage * p.per_stage + i) * Cfg::W_BYTES;
            uint8_t* xdst = x_smem + (stage * p.per_stage + i) * x_bytes;
            if (p.g.w_mn) {
              tma_load_3d_hint(wdst, &maps.w, &full_bar[stage], n0, k0, f.g, pol_w);
              tma_load_3d_hint(wdst + Cfg::HALF_BYTES, &maps.w, &full_bar[stage], n0 + 64, k0, f.g, pol_w);
            } else {
              tma_load_3d_hint(wdst, &maps.w, &full_bar[stage], k0, n0, f.g, pol_w);
            }
            grp_token_boxes(width, [&](int b, int at) {
              tma_load_2d_hint(xdst + at * 128, &maps.x[b], &full_bar[stage], k0, f.tok0 + at, pol_x);
            });
          }
        }
        used |= 1u << stage;
        parities = (parities & ~(1u << stage)) | phase << stage;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    for (int s = 0; s < p.stages; ++s) {
      if (used >> s & 1u) {
        volatile int no_abort = 0;
        mbar_wait(&full_bar[s], parities >> s & 1u, &no_abort, p.g.wait_budget_ns, 0xb2);
      }
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    int local = 0;
    bool ok = true;
    const uint64_t w_desc0 = make_sw128_desc(smem_u32(w_smem), p.g.w_mn ? Cfg::HALF_BYTES : 16, 1024);
    const uint64_t x_desc0 = make_sw128_desc(smem_u32(x_smem), 16, 1024);
    const uint32_t w_step = p.g.w_mn ? 2048 / 16 : 32 / 16;
    const uint32_t tmem = uniform(tmem_base);
    GrpWalk walk;
    for (int t = cluster_id; t < num_tiles && ok; t += num_clusters, ++local) {
      const GrpTile f = walk.at(plan, t, p.g.col_tiles, p.g.super, p.tokens, Cfg::UNIT);
      if (f.g == p.g.groups) break;
      const int width = (f.cnt + Cfg::UNIT - 1) / Cfg::UNIT * Cfg::UNIT;
      const uint32_t idesc = p.g.idesc | static_cast<uint32_t>(width >> 3) << 17;
      const int acc = local & 1;
      if (!mbar_wait_warp(&acc_empty_bar[acc], ((local >> 1) & 1) ^ 1u, abort_flag, p.g.wait_budget_ns, 0xb3)) break;
      tcgen05_fence_after_sync();
      const uint32_t d_tmem = tmem + acc * p.tokens;
      for (int kb = kb_lo; kb < kb_hi; kb += p.per_stage) {
        if (!mbar_wait_warp(&full_bar[stage], phase, abort_flag, p.g.wait_budget_ns, 0xb4)) {
          ok = false;
          break;
        }
        tcgen05_fence_after_sync();
        const int n = min(p.per_stage, kb_hi - kb);
        const uint64_t w_desc = w_desc0 + stage * p.per_stage * (Cfg::W_BYTES / 16);
        const uint64_t x_desc = x_desc0 + stage * p.per_stage * (x_bytes / 16);
        if (one) {
          for (int i = 0; i < n; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f16_ss(d_tmem, w_desc + i * (Cfg::W_BYTES / 16) + k * w_step, x_desc + i * (x_bytes / 16) + k * 2, idesc,
                          kb > kb_lo || i > 0 || k > 0 ? 1u : 0u);
          umma_commit(&empty_bar[stage]);
        }
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (one) umma_commit(&acc_full_bar[acc]);
    }
    if (one) umma_commit(mma_done_bar);
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait(mma_done_bar, 0, &no_abort, p.g.wait_budget_ns, 0xb5);
    __syncwarp();
  } else {
    const int quad = warp & 3;
    float* delta = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(plan.lo) + grp_plan_align(p.g.groups));  // adapters only
    const int e = quad * 32 + lane;  // also the column of the panel that this thread sends
    const int own = Cfg::PANEL / p.splits;  // columns that this CTA finishes
    const int pitch = p.tokens + 4;
    uint8_t* own_t = reinterpret_cast<uint8_t*>(delta + own * pitch);
    uint8_t* own_16 = LORA == 2 ? own_t : own_t + 64 + quad * 48;
    const void* const T = LORA && p.own_t ? own_16 : p.g.lora.t;
    const signed char* const exps = LORA && p.own_t ? reinterpret_cast<signed char*>(own_16 + 32) : p.g.lora.exps;
    const int sent = e;
    const uint32_t owner = sent / own;
    const uint32_t to = mapa_shared(smem_u32(recv) + (rank * own + sent % own) * pitch * 4, owner);
    const uint32_t to_bar = mapa_shared(smem_u32(part_full_bar), owner);
    GrpWalk walk;
    int local = 0;
    bool waited = false;
    for (int t = cluster_id; t < num_tiles; t += num_clusters) {
      const GrpTile f = walk.at(plan, t, p.g.col_tiles, p.g.super, p.tokens, Cfg::UNIT);
      const int n0 = f.col_blk * Cfg::PANEL + rank * own;
      // Units of 32 columns and TOK tokens, the warps in turn.
      constexpr int TOK = LORA ? kLoraTokens : 8;
      const int col_blocks = own / 32, units = col_blocks * ((f.cnt + TOK - 1) / TOK);
      if (f.g == p.g.groups) {
        const unsigned short zero = 0;
        for (int it = e; it < own * f.cnt; it += 128)
          if (n0 + it % own < p.g.out)
            static_cast<unsigned short*>(p.g.c)[(f.tok0 + it / own) * p.g.ldc + n0 + it % own] = zero;
        continue;
      }
      const int width = (f.cnt + Cfg::UNIT - 1) / Cfg::UNIT * Cfg::UNIT;
      if (LORA && adapted) {
        // The adapters' part, while the tile is computed: it is this warp's own
        // until the sums are there.  The first tile's rows of B come into L2 before
        // T is waited for.
        GrpTileAdapters adapters;
        adapters.load(p.g.lora, f.tok0, f.cnt, lane);
        if (!waited) {
          for (int it = e; it < own * f.cnt; it += 128) {
            const int n = n0 + it % own, a = adapters.of(it / own);
            if (a < 0 || n >= p.g.out) continue;
            const unsigned short* row = static_cast<const unsigned short*>(p.g.lora.b) + a * p.g.lora.stride_b + n * p.g.lora.ldb;
            for (int at = 0; at < p.g.lora.rank; at += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + at));
          }
          __syncwarp();
          if (!p.own_t) {
            grid_dependency_wait();
            grid_launch_dependents();
          } else {
            lora_own_t<LORA == 2>(p.g.lora, own_t, p.g.M, p.g.red, rank * 4 + quad, p.splits, lane);
            __syncwarp();
            if (lane == 0) {
              fence_cluster();
              for (int q = 0; q < p.splits; ++q) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(t_bar), q));
            }
            const bool here = mbar_wait_cluster(t_bar, 0, abort_flag, p.g.wait_budget_ns, 0xb9);
            if (!__all_sync(0xffffffffu, here)) break;
            if (LORA == 1)
              lora_own_round(reinterpret_cast<const float*>(own_t), p.g.M * p.g.lora.rank, reinterpret_cast<unsigned short*>(own_16),
                             reinterpret_cast<signed char*>(own_16 + 32), lane);
          }
          waited = true;
        }
        for (int u = quad; u < units; u += 4) {
          const int col = u % col_blocks * 32, tok = u / col_blocks * TOK;
          const int mine = adapters.from(tok);
          lora_part<LORA == 2, 4>(p.g.lora, T, exps, mine, f.tok0 + tok, n0 + col, p.g.out, delta + col * pitch + tok, pitch, lane);
        }
      }
      const int acc = local & 1;
      bool ready = mbar_wait(&acc_full_bar[acc], (local >> 1) & 1, abort_flag, p.g.wait_budget_ns, 0xb6);
      // Every CTA has added the partials before.
      if (ready && p.splits > 1) ready = mbar_wait_cluster(part_empty_bar, (local & 1) ^ 1u, abort_flag, p.g.wait_budget_ns, 0xb7);
      if (!__all_sync(0xffffffffu, ready)) break;
      tcgen05_fence_after_sync();
      for (int c = 0; c < width; c += 16) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * p.tokens + c, r);
        tmem_ld_wait();
        if (p.splits > 1) {
#pragma unroll
          for (int q = 0; q < 16; q += 4) st_cluster_v4(to + (c + q) * 4, r[q], r[q + 1], r[q + 2], r[q + 3]);
        } else {
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(r[h + q]);
            grp_narrow_store(p.g, v, f, c + h, n0 + sent, LORA && adapted ? delta + sent * pitch + c + h : nullptr,
                             LORA && p.g.lora.bias != nullptr && n0 + sent < p.g.out
                                 ? load_16(static_cast<const unsigned short*>(p.g.lora.bias) + n0 + sent, p.g.bf16 != 0)
                                 : 0.0f);
          }
        }
      }
      tcgen05_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&acc_empty_bar[acc]);
        if (p.splits > 1) mbar_arrive_cluster(to_bar);
      }
      ++local;
      if (p.splits == 1) continue;
      ready = mbar_wait_cluster(part_full_bar, (local - 1) & 1, abort_flag, p.g.wait_budget_ns, 0xb8);
      if (!__all_sync(0xffffffffu, ready)) break;
      for (int u = quad; u < units; u += 4) {
        const int col = u % col_blocks * 32 + lane;
#pragma unroll
        for (int tok = u / col_blocks * TOK, i = 0; i < TOK; i += 8, tok += 8) {
          if (tok >= f.cnt) break;
          const float* at = recv + col * pitch + tok;
          float v[8];
          for (int q = 0; q < p.splits; ++q) {
#pragma unroll
            for (int h = 0; h < 8; h += 4) {
              const float4 x = *reinterpret_cast<const float4*>(at + q * own * pitch + h);
              v[h] = q == 0 ? x.x : v[h] + x.x;
              v[h + 1] = q == 0 ? x.y : v[h + 1] + x.y;
              v[h + 2] = q == 0 ? x.z : v[h + 2] + x.z;
              v[h + 3] = q == 0 ? x.w : v[h + 3] + x.w;
            }
          }
          grp_narrow_store(p.g, v, f, tok, n0 + col, LORA && adapted ? delta + col * pitch + tok : nullptr,
                           LORA && p.g.lora.bias != nullptr && n0 + col < p.g.out
                               ? load_16(static_cast<const unsigned short*>(p.g.lora.bias) + n0 + col, p.g.bf16 != 0)
                               : 0.0f);
        }
      }
      __syncwarp();
      // Relaxed: the values read have been used, and nothing else is ordered.
      if (lane == 0)
        for (int q = 0; q < p.splits; ++q) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(part_empty_bar), q));
    }
    if (LORA && early && !waited) {  // nothing to do: the grid still ends after the one before
      grid_dependency_wait();
      grid_launch_dependents();
    }
  }

  if (beside) grid_dependency_wait();
  tcgen05_fence_before_sync();
  __syncthreads();
  cluster_sync();  // nobody writes to a CTA that has left
  if (warp == 1) {
    tcgen05_fence_after_sync();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

}  // namespace tg
