// gemm_ff_skinny.cuh -- the same products where whole tiles would leave most SMs
// idle: few rows (M <= 256), bound by streaming the weights from HBM once, or
// few tiles and a long K (dWg and dWu of a narrow block: K is the tokens).  The
// kernel computes the transposed result (the weight's rows fill the 128-row MMA
// side, a block of up to 256 rows is the MMA's N) and splits K over a cluster
// of S CTAs, as the fp16 small-M kernel does.  With few tiles a kernel is held
// up by what one SM can load, about 50 bytes a clock, so its time goes down with
// the number of SMs until the cluster's reduction (about 3 us) is what is left:
// dWg and dWu of 8192 x 256 x 256 (with dG and dU before) take 50 us on 8 CTA
// pairs, 19 on 64 CTAs.
//   * Gated: a panel is 64 rows of Wg and the same 64 rows of Wu, so both
//     projections of 64 block columns meet in one accumulator.
//   * Plain: a panel is 128 rows of W (K-major), or, for dX = dG Wg + dU Wu,
//     128 columns of Wg and then of Wu (stored K x N, MN-major) with the K
//     loop over both sources.
//   * dWg and dWu: a panel is 128 columns of X, the rows are columns of dG and
//     then of dU (both stored K x M, MN-major, in panels of 64 rows).
// Each CTA moves its partial (fp32, or 32-bit integers) to shared memory; after
// a cluster barrier every CTA adds a share of the panel's outputs over the S
// partials in rank order, so results do not depend on timing.
#pragma once

#include "ff_ops.cuh"
#include "gemm_ff_pair.cuh"

namespace tg {

struct FfSkinnyParams {
  void* c[3];                 // H, G, U; or the results of the row sources
  int64_t ldc[3];
  int c_aligned[3];           // rows of the result start on 8-byte boundaries
  const float* row_scale;
  const float* col_scale[2];
  const void* bias;
  int M, N;
  int m_pad;                  // rows of a block, a multiple of 16
  int m_blocks;               // blocks of rows of one row source
  int k_blocks, k_blocks_src;
  int splits, stages;
  uint32_t a_stage_bytes;     // of the activations: m_pad * 128, or whole 64-row panels if stored K x M
  uint32_t tmem_cols;
  uint32_t idesc;
  int a_mnmajor, b_kmajor;
  int bf16, act, relu, save;
  int prefetch_kb;            // k-blocks of the weight brought into L2 ahead of the previous kernel's end
  uint64_t wait_budget_ns;
};

struct FfSkinnyCfg {
  static constexpr int PANEL = 128;                    // weight rows per panel
  static constexpr int W_STAGE_BYTES = PANEL * 128;    // 16 KiB
  static constexpr int HALF_BYTES = W_STAGE_BYTES / 2;
  static constexpr int EPI_WARP0 = 2;
  static constexpr int THREADS = 192;
  static constexpr int MAX_STAGES = 8;
  static constexpr int BAR_BYTES = 256;
  static constexpr int MAX_SMEM = 1024 + 220 * 1024 + BAR_BYTES;
  static constexpr int SM_SMEM = 228 * 1024;           // of one SM
  static constexpr int CTA_RESERVED = 1024;            // of it, taken by the system for each resident CTA
  static constexpr int a_bytes(int m_pad, bool a_km) { return a_km ? (m_pad + 63) / 64 * HALF_BYTES : m_pad * 128; }
  static constexpr int smem_bytes(int a_bytes, int stages) {
    return 1024 + stages * (W_STAGE_BYTES + a_bytes) + BAR_BYTES;
  }
  static_assert(HALF_BYTES % 1024 == 0 && (16 * 128) % 1024 == 0, "halves and blocks start on the swizzle's 1024 bytes");
  // CTAs that share an SM with blocks of m_pad rows, and the most stages a CTA's
  // ring can have so that they do: at m_pad = 96 three, since two rings of four
  // pass the SM's shared memory by 512 bytes (with four, one CTA an SM, gated
  // fp16 96 x 8192 x 8192 takes 64 us; so 51).  At m_pad <= 32 three stages
  // of up to 20 KiB stream best.
  static constexpr int ctas_per_sm(int m_pad) { return m_pad <= 128 ? 2 : 1; }
  static constexpr int stages(int m_pad, bool a_km) {
    const int share = SM_SMEM / ctas_per_sm(m_pad) - CTA_RESERVED;
    const int most = share < MAX_SMEM ? share : MAX_SMEM;
    const int budget = m_pad <= 32 ? 64 * 1024 : most - smem_bytes(0, 0);
    const int n = budget / (W_STAGE_BYTES + a_bytes(m_pad, a_km));
    return n > MAX_STAGES ? MAX_STAGES : n;
  }
};

// Four results of one row, from column n on.
__device__ __forceinline__ void ff_store4(void* c, int64_t ldc, bool aligned, int m, int n, int N, const float (&v)[4],
                                          bool bf16) {
  uint32_t w[2];
  pack_row<4>(v, w, bf16);
  unsigned short* dst = static_cast<unsigned short*>(c) + static_cast<int64_t>(m) * ldc + n;
  if (aligned && n + 4 <= N) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < N) dst[e] = static_cast<unsigned short>(w[e >> 1] >> ((e & 1) * 16));
  }
}

// The cluster's partials of four words at `addr`: every remote read is issued
// before the first sum (read one after the other, 8 of them cost 4 us at M =
// 128).
__device__ __forceinline__ void ff_cluster_read(uint32_t addr, int splits, float4 (&x)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (q < splits) x[q] = ld_shared_cluster_f4(mapa_shared(addr, static_cast<uint32_t>(q)));
}

// Their sum in rank order, as fp32 (8-bit operands: the exact integer sum,
// then one rounding).
template <int KIND>
__device__ __forceinline__ void ff_cluster_sum(const float4 (&x)[8], int splits, float (&v)[4]) {
  if (KIND == kFfF16) {
    float4 s = x[0];
#pragma unroll
    for (int q = 1; q < 8; ++q) {
      if (q < splits) {
        s.x += x[q].x;
        s.y += x[q].y;
        s.z += x[q].z;
        s.w += x[q].w;
      }
    }
    v[0] = s.x;
    v[1] = s.y;
    v[2] = s.z;
    v[3] = s.w;
  } else {
    int i[4] = {__float_as_int(x[0].x), __float_as_int(x[0].y), __float_as_int(x[0].z), __float_as_int(x[0].w)};
#pragma unroll
    for (int q = 1; q < 8; ++q) {
      if (q < splits) {
        i[0] += __float_as_int(x[q].x);
        i[1] += __float_as_int(x[q].y);
        i[2] += __float_as_int(x[q].z);
        i[3] += __float_as_int(x[q].w);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __int2float_rn(i[e]);
  }
}

__device__ __forceinline__ void ff_scale4(float (&v)[4], float row_scale, const float* col_scale, int n, int N) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = v[e] * row_scale * (n + e < N ? __ldg(col_scale + n + e) : 0.0f);
}

template <int KIND, bool GATED>
__global__ void __launch_bounds__(FfSkinnyCfg::THREADS, 1)
    ff_skinny_kernel(const __grid_constant__ FfMaps maps, const FfSkinnyParams p) {
  using Cfg = FfSkinnyCfg;
  constexpr int K_ELEMS = KIND == kFfI8 ? 128 : 64;
  constexpr int OUT = GATED ? 64 : 128;  // result columns per panel
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* w_smem = smem;
  uint8_t* a_smem = smem + p.stages * Cfg::W_STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.stages * (Cfg::W_STAGE_BYTES + p.a_stage_bytes));
  uint64_t* full_bar = bars;
  uint64_t* empty_bar = bars + Cfg::MAX_STAGES;
  uint64_t* acc_full_bar = bars + 2 * Cfg::MAX_STAGES;
  uint64_t* mma_done_bar = acc_full_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* partial = reinterpret_cast<uint32_t*>(smem);  // [m_pad][128] words, reuses the ring

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int n0 = blockIdx.y * OUT;
  const int row_src = KIND == kFfF16 && !GATED && static_cast<int>(blockIdx.z) >= p.m_blocks ? 1 : 0;
  const int m0 = (static_cast<int>(blockIdx.z) - row_src * p.m_blocks) * p.m_pad;
  const int kb_lo = static_cast<int>((static_cast<int64_t>(p.k_blocks) * rank) / p.splits);
  const int kb_hi = static_cast<int>((static_cast<int64_t>(p.k_blocks) * (rank + 1)) / p.splits);
  const int my_blocks = kb_hi - kb_lo;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(acc_full_bar, 1);
    mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
    if (GATED) tma_prefetch_desc(&maps.b[1]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish_alloc_permit();
  }
  if (threadIdx.x == 0) {
    // The weight's first boxes come into L2 while the previous kernel on the
    // stream still drains.  That is a hint, which reads nothing into this
    // kernel: should that kernel write the weight, its stores update the same
    // L2 lines before the loads below, which wait for it.
    const int ahead = min(kb_hi, kb_lo + p.prefetch_kb);
    for (int kb = kb_lo; kb < ahead; ++kb) {
      const int k_src = kb >= p.k_blocks_src ? 1 : 0;
      const int k0 = (kb - k_src * p.k_blocks_src) * K_ELEMS;
      if (GATED) {
        tma_prefetch_l2_2d(&maps.b[0], k0, n0);
        tma_prefetch_l2_2d(&maps.b[1], k0, n0);
      } else if (KIND == kFfI8 || p.b_kmajor) {
        tma_prefetch_l2_2d(&maps.b[k_src], k0, n0);
      } else {
        tma_prefetch_l2_2d(&maps.b[k_src], n0, k0);
        tma_prefetch_l2_2d(&maps.b[k_src], n0 + 64, k0);
      }
    }
  }
  tcgen05_fence_before_sync();
  __syncthreads();
  tcgen05_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    // Producer: this CTA's K slice of the panel and of the activations.
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int last_parity[Cfg::MAX_STAGES];
#pragma unroll
      for (int s = 0; s < Cfg::MAX_STAGES; ++s) last_parity[s] = -1;
      const uint32_t tx = Cfg::W_STAGE_BYTES + p.a_stage_bytes;
      const uint64_t pol_w = l2_policy_evict_first();
      const uint64_t pol_a = l2_policy_evict_last();
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, p.wait_budget_ns, 0x91)) break;
        mbar_arrive_expect_tx(&full_bar[stage], tx);
        const int k_src = kb >= p.k_blocks_src ? 1 : 0;
        const int k0 = (kb - k_src * p.k_blocks_src) * K_ELEMS;
        uint8_t* wdst = w_smem + stage * Cfg::W_STAGE_BYTES;
        if (GATED) {
          tma_load_2d_hint(wdst, &maps.b[0], &full_bar[stage], k0, n0, pol_w);
          tma_load_2d_hint(wdst + Cfg::HALF_BYTES, &maps.b[1], &full_bar[stage], k0, n0, pol_w);
        } else if (KIND == kFfI8 || p.b_kmajor) {
          tma_load_2d_hint(wdst, &maps.b[k_src], &full_bar[stage], k0, n0, pol_w);
        } else {
          tma_load_2d_hint(wdst, &maps.b[k_src], &full_bar[stage], n0, k0, pol_w);
          tma_load_2d_hint(wdst + Cfg::HALF_BYTES, &maps.b[k_src], &full_bar[stage], n0 + 64, k0, pol_w);
        }
        uint8_t* adst = a_smem + stage * p.a_stage_bytes;
        if (KIND == kFfF16 && !GATED && p.a_mnmajor) {
          for (uint32_t b = 0; b < p.a_stage_bytes; b += Cfg::HALF_BYTES)  // panels of 64 rows
            tma_load_2d_hint(adst + b, &maps.a[row_src], &full_bar[stage], m0 + static_cast<int>(b >> 7), k0, pol_a);
        } else {
          tma_load_2d_hint(adst, &maps.a[k_src], &full_bar[stage], k0, m0, pol_a);
        }
        last_parity[stage] = static_cast<int>(phase);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      for (int s = 0; s < p.stages; ++s) {
        if (last_parity[s] >= 0) {
          volatile int no_abort = 0;
          mbar_wait(&full_bar[s], static_cast<uint32_t>(last_parity[s]), &no_abort, p.wait_budget_ns, 0x92);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const bool w_mn = KIND == kFfF16 && !GATED && p.b_kmajor == 0;
      const bool a_mn = KIND == kFfF16 && !GATED && p.a_mnmajor != 0;
      // As in the pair kernel: one addition per descriptor and MMA.
      const uint64_t w_desc0 = make_sw128_desc(smem_u32(w_smem), w_mn ? Cfg::HALF_BYTES : 16, 1024);
      const uint64_t a_desc0 = make_sw128_desc(smem_u32(a_smem), a_mn ? Cfg::HALF_BYTES : 16, 1024);
      const uint32_t w_step = w_mn ? 2048 / 16 : 32 / 16, a_step = a_mn ? 2048 / 16 : 32 / 16;
      for (int i = 0; i < my_blocks; ++i) {
        if (!mbar_wait(&full_bar[stage], phase, abort_flag, p.wait_budget_ns, 0x93)) {
          ok = false;
          break;
        }
        tcgen05_fence_after_sync();
        const uint64_t w_desc = w_desc0 + stage * (Cfg::W_STAGE_BYTES / 16);
        const uint64_t a_desc = a_desc0 + stage * (p.a_stage_bytes / 16);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_ff<KIND>(tmem_base, w_desc + k * w_step, a_desc + k * a_step, p.idesc, (i | k) != 0 ? 1u : 0u);
        umma_commit(&empty_bar[stage]);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok && my_blocks > 0) umma_commit(acc_full_bar);
      umma_commit(mma_done_bar);
      volatile int no_abort = 0;
      mbar_wait(mma_done_bar, 0, &no_abort, p.wait_budget_ns, 0x94);
    }
    __syncwarp();
  } else {
    // TMEM partial -> shared memory [m][panel row].
    const int quad = warp & 3;
    const int n_local = quad * 32 + lane;
    bool ready = true;
    if (my_blocks > 0) ready = mbar_wait(acc_full_bar, 0, abort_flag, p.wait_budget_ns, 0x95);
    ready = __all_sync(0xffffffffu, ready);
    if (ready) {
      tcgen05_fence_after_sync();
      for (int c = 0; c < p.m_pad / 16; ++c) {
        uint32_t r[16];
        if (my_blocks > 0) {
          tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + c * 16, r);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) r[e] = 0u;  // empty K slice
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) partial[(c * 16 + e) * Cfg::PANEL + n_local] = r[e];
      }
    }
    tcgen05_fence_before_sync();
  }

  __syncthreads();
  cluster_sync();  // every partial of the cluster is in shared memory

  if (!*abort_flag) {
    // Items are (m, 4-column group); CTA `rank` finishes its share.
    const int e = threadIdx.x;
    constexpr int GROUPS = OUT / 4;
    const int rows = min(p.m_pad, p.M - m0);
    const int items = rows * GROUPS;
    const int lo = static_cast<int>((static_cast<int64_t>(items) * rank) / p.splits);
    const int hi = static_cast<int>((static_cast<int64_t>(items) * (rank + 1)) / p.splits);
    const uint32_t part_addr = smem_u32(partial);
    const bool bf16 = p.bf16 != 0;
    void* const c0 = row_src ? p.c[1] : p.c[0];
    const int64_t ldc0 = row_src ? p.ldc[1] : p.ldc[0];
    const bool aligned0 = (row_src ? p.c_aligned[1] : p.c_aligned[0]) != 0;
    for (int it = lo + e; it < hi; it += Cfg::THREADS) {
      const int y = it / GROUPS;
      const int j = it - y * GROUPS;
      const int m = m0 + y;
      const int n = n0 + 4 * j;
      if (n >= p.N) continue;
      const uint32_t off = part_addr + static_cast<uint32_t>((y * Cfg::PANEL + 4 * j) * 4);
      float4 xv[8], xu[8];
      ff_cluster_read(off, p.splits, xv);
      if (GATED) ff_cluster_read(off + 64 * 4, p.splits, xu);
      float v[4];
      ff_cluster_sum<KIND>(xv, p.splits, v);
      const float row_scale = KIND == kFfI8 ? __ldg(p.row_scale + m) : 1.0f;
      if (KIND == kFfI8) ff_scale4(v, row_scale, p.col_scale[0], n, p.N);
      if (GATED) {
        float u[4];
        ff_cluster_sum<KIND>(xu, p.splits, u);
        if (KIND == kFfI8) ff_scale4(u, row_scale, p.col_scale[1], n, p.N);
        if (KIND == kFfF16 && p.save) {
          ff_store4(p.c[1], p.ldc[1], p.c_aligned[1] != 0, m, n, p.N, v, bf16);
          ff_store4(p.c[2], p.ldc[2], p.c_aligned[2] != 0, m, n, p.N, u, bf16);
        }
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const float2 g = make_float2(v[q], v[q + 1]);
          const float2 a = p.act == kActSilu   ? act_value2<kActSilu>(g)
                           : p.act == kActGelu ? act_value2<kActGelu>(g)
                                               : act_value2<kActRelu>(g);
          v[q] = a.x * u[q];
          v[q + 1] = a.y * u[q + 1];
        }
      } else if (KIND == kFfI8) {
        if (p.bias != nullptr) {
          const unsigned short* b16 = static_cast<const unsigned short*>(p.bias) + n;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + q < p.N) v[q] += load_16(b16 + q, bf16);
        }
        if (p.relu) {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = v[q] > 0.0f ? v[q] : 0.0f;
        }
      }
      ff_store4(c0, ldc0, aligned0, m, n, p.N, v, bf16);
    }
  }

  cluster_sync();  // peers are done reading this CTA's partial
  if (warp == 1) {
    tcgen05_fence_after_sync();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

}  // namespace tg
