// lora_shrink.cuh -- the first half of the low-rank adapters:
// T[m][j] = scale_a sum_k A_a[j][k] X[m][k] with a = index[m].
//
// Bound by reading X and the used adapters' A.  An item is one adapter among a
// block of up to 128 tokens, and up to 128 rows of its A: these are the MMA's M side
// (rows behind the rank are whatever lies in shared memory behind them, in lanes
// that nobody reads), the tokens from the adapter's first to its last in the block the N side.
// Columns of D are independent, so tokens of other adapters in between cost
// nothing but their loads, and are not written.  A cluster of S CTAs splits the
// sum over K; each finishes every S-th four tokens from the partials that the
// others write into its shared memory, in rank order.  Blocks of a prompt have one item, those of a
// decoding batch up to 128, spread over blockIdx.y.  T is rounded once to the
// 16-bit type, as the tensor cores read it (and as two linear layers in a row would),
// in fp16 with a power of two where its range needs one (gemm_grp_pair.cuh).
//
// A decoding batch takes the second kernel: a warp a value of T.  Its tokens rarely
// share an adapter, so there is nothing to multiply by tiles, and without tiles
// there is no list, ring or exchange on the way from the index to T (whole call, one
// token through 4096 x 4096, rank 16: 14.5 us with tiles, 13.4 so; 64 tokens of 64
// adapters 29 and 24).  The main product runs meanwhile on the same SMs (it waits for
// T only when its own sums are under way).  One token
// or two with 8 or 16 values of T in all (grp_lora_own_t) go without either: the narrow
// kernel's warps make a value each.
//
// Measured: 8192 rows of 8 requests, K = 4096, rank 64, 29.5 us alone, 2.3 TB/s:
// bound by the latency of a block's loads.  The main product hides most of it.  fp16's
// powers (looked for, none found) cost 2-4 us there and 2 of 30 with split sums: the
// votes come after the stores, and full warps take part in them (votes among eight lanes
// took 6 us more).
#pragma once

#include "gemm_grp_narrow.cuh"

namespace tg {

struct LoraShrinkMaps {
  CUtensorMap a;     // adapters' A: boxes of 64 x min(128, rank)
  CUtensorMap x[4];  // X: boxes of 64 columns and 16, 32, 64, 128 rows
};

struct LoraShrinkParams {
  const int* index;
  const float* scale;  // of each adapter, or nullptr
  void* t;
  int* kind;
  signed char* exps;   // fp16: T's powers, of each row and eight ranks
  uint8_t* misfits;    // fp16: of each 32 tokens and 128 ranks, a byte of each warp of up to two CTAs: 1 where a power is not 0
  int M, rank, adapters;
  int k_blocks, splits, stages;
  int per_stage;       // k-blocks of a stage of the ring
  int tokens;          // most of an item, and rows of a block: 32, 64 or 128
  int a_rows;          // of a box: min(128, rank)
  uint32_t tmem_cols;
  uint32_t idesc;      // without N
  uint64_t wait_budget_ns;
};

struct LoraShrinkCfg {
  static constexpr int EPI_WARP0 = 2;
  static constexpr int THREADS = 192;
  static constexpr int MAX_STAGES = 16;
  static constexpr int BAR_BYTES = 512;
  // Partials: [source][four tokens][row of A] of 16 bytes, for this CTA's share of the tokens; none without a split.
  __host__ __device__ static constexpr int recv_bytes(int tokens, int splits, int a_rows) {
    return splits == 1 ? 0 : splits * ((tokens / 4 + splits - 1) / splits) * a_rows * 16;
  }
  // The MMAs read 128 rows from each stage's A on, the last ones of other stages and of X.
  static constexpr int smem_bytes(int tokens, int splits, int a_rows, int stages) {
    const int n = stages * (a_rows + tokens) * 128 + recv_bytes(tokens, splits, a_rows) + BAR_BYTES;
    const int least = (stages * a_rows + 128) * 128;
    return 1024 + (n < least ? least : n);
  }
  static_assert((2 * MAX_STAGES + 5) * 8 + 8 <= BAR_BYTES, "barriers");
};

// The adapters among a block's tokens, in order of their first.
struct LoraItems {
  int count;
  int adapter[128], first[128], last[128];
};

// Two CTAs an SM: their 6 warps take the registers of 8, so 128 a thread (with 150 of them the
// split sums of 1049 rows took 35 us in the whole call instead of 30).
template <bool BF16>
__global__ void __launch_bounds__(256, 2)
    lora_shrink_kernel(const __grid_constant__ LoraShrinkMaps maps, const LoraShrinkParams p) {
  using Cfg = LoraShrinkCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t a_bytes = p.a_rows * 128, x_bytes = p.tokens * 128;
  uint8_t* a_smem = smem;
  uint8_t* x_smem = smem + p.stages * p.per_stage * a_bytes;
  float4* recv = reinterpret_cast<float4*>(smem + p.stages * p.per_stage * (a_bytes + x_bytes));
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(recv) + Cfg::recv_bytes(p.tokens, p.splits, p.a_rows));
  uint64_t* full_bar = bars;
  uint64_t* empty_bar = bars + Cfg::MAX_STAGES;
  uint64_t* acc_full_bar = bars + 2 * Cfg::MAX_STAGES;
  uint64_t* acc_empty_bar = acc_full_bar + 1;
  uint64_t* part_full_bar = acc_empty_bar + 1;
  uint64_t* part_empty_bar = part_full_bar + 1;
  uint64_t* mma_done_bar = part_empty_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Barriers and tensor memory.  The first cluster of a block sets them up while the
  // kernel before this one ends; the others are there for blocks of many adapters,
  // look at the list first and leave at once where it is short.
  auto set_up = [&]() {
    if (threadIdx.x == 0) {
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(&full_bar[s], 1);
        mbar_init(&empty_bar[s], 1);
      }
      mbar_init(acc_full_bar, 1);
      mbar_init(acc_empty_bar, 4);
      mbar_init(part_full_bar, 4 * p.splits);
      mbar_init(part_empty_bar, 4 * p.splits);
      mbar_init(mma_done_bar, 1);
      *abort_flag = 0;
      fence_mbarrier_init();
      tma_prefetch_desc(&maps.a);
      for (int b = 0; b < 4 && 16 << b <= p.tokens; ++b) tma_prefetch_desc(&maps.x[b]);
    }
    if (warp == 1) {
      tmem_alloc(tmem_slot, p.tmem_cols);
      tmem_relinquish_alloc_permit();
    }
    tcgen05_fence_before_sync();
    __syncthreads();
    cluster_sync();
    tcgen05_fence_after_sync();
  };
  if (blockIdx.y == 0) set_up();
  grid_dependency_wait();
  grid_launch_dependents();
  const int rank = static_cast<int>(cluster_ctarank());
  const int m0 = static_cast<int>(blockIdx.x / p.splits) * p.tokens;
  const int j0 = static_cast<int>(blockIdx.z) * 128;
  const int rows = min(128, p.rank - j0);  // of A
  __shared__ __align__(16) int owner_of[128];
  __shared__ int firsts[4];
  __shared__ int kinds[4];  // of each 32 tokens
  __shared__ LoraItems items;
  if (p.tokens <= 32) {  // each warp by itself finds what it needs; one keeps the list
    const bool valid = lane < p.tokens && m0 + lane < p.M;
    const int a = valid ? __ldg(p.index + m0 + lane) : -1;
    const int mine = a >= 0 && a < p.adapters ? a : -1;
    const unsigned peers = __match_any_sync(0xffffffffu, mine);
    const bool opens = mine >= 0 && __ffs(peers) - 1 == lane;
    const unsigned all = __ballot_sync(0xffffffffu, opens);
    if (warp == 0) {
      if (opens) {
        const int d = __popc(all & ((1u << lane) - 1));
        items.adapter[d] = mine;
        items.first[d] = lane;
        items.last[d] = 31 - __clz(peers);
      }
      const int r0 = __shfl_sync(0xffffffffu, mine, 0);
      const bool same = __all_sync(0xffffffffu, !valid || mine == r0);
      if (lane == 0) {
        items.count = __popc(all);
        kinds[0] = !same ? kLoraMixed : r0 < 0 ? kLoraNone : r0;
        if (blockIdx.y == 0 && blockIdx.z == 0 && rank == 0) p.kind[m0 / 32] = kinds[0];
      }
    }
    __syncthreads();
  } else {  // each of 128 threads looks for its token's adapter among the tokens before
    int mine = -1;
    const int tok = threadIdx.x;
    if (tok < 128) {
      const bool valid = tok < p.tokens && m0 + tok < p.M;
      const int a = valid ? __ldg(p.index + m0 + tok) : -1;
      mine = a >= 0 && a < p.adapters ? a : -1;
      owner_of[tok] = mine;
      const int r0 = __shfl_sync(0xffffffffu, mine, 0);
      const bool same = __all_sync(0xffffffffu, !valid || mine == r0);
      // What each 32 tokens are to the main product.
      if (lane == 0) kinds[warp] = !same ? kLoraMixed : r0 < 0 ? kLoraNone : r0;
      if (lane == 0 && valid && blockIdx.y == 0 && blockIdx.z == 0 && rank == 0) p.kind[(m0 + tok) / 32] = kinds[warp];
    }
    __syncthreads();
    int before = 128;  // the first token of this one's adapter, from the end of the search on
    if (tok < 128) {
      for (int s = (tok & ~31) + 28; s >= 0; s -= 4) {
        const int4 o = *reinterpret_cast<const int4*>(owner_of + s);
        if (o.w == mine) before = s + 3;
        if (o.z == mine) before = s + 2;
        if (o.y == mine) before = s + 1;
        if (o.x == mine) before = s;
      }
      const unsigned opens = __ballot_sync(0xffffffffu, mine >= 0 && before == tok);
      if (lane == 0) firsts[warp] = __popc(opens);
      if (mine >= 0 && before == tok) items.last[tok] = tok;  // by the first token for now
      before = mine < 0 ? -1 : before;
      mine = __popc(opens & ((1u << lane) - 1));  // its number in this warp
    }
    __syncthreads();
    if (tok < 128 && before >= 0 && before != tok) atomicMax(&items.last[before], tok);
    __syncthreads();
    int last = 0;
    if (tok < 128 && before == tok) last = items.last[tok];
    __syncthreads();
    if (tok < 128) {
      for (int w = 0; w < warp; ++w) mine += firsts[w];
      if (before == tok) {
        items.adapter[mine] = owner_of[tok];
        items.first[mine] = tok;
        items.last[mine] = last;
      }
      if (tok == 0) items.count = firsts[0] + firsts[1] + firsts[2] + firsts[3];
    }
    __syncthreads();
  }
  const int count = items.count, step = static_cast<int>(gridDim.y);
  if (blockIdx.y != 0) {
    if (static_cast<int>(blockIdx.y) >= count) return;  // the whole cluster
    set_up();
  }
  const uint32_t tmem_base = *tmem_slot;
  const int kb_lo = static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / p.splits);
  const int kb_hi = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / p.splits);

  if (warp == 0) {
    // As in the narrow kernel: the warp loops, one lane issues.
    const bool one = elect_one();
    int stage = 0;
    uint32_t phase = 0, used = 0, parities = 0;
    bool ok = true;
    const uint64_t pol_a = l2_policy_evict_first(), pol_x = l2_policy_evict_normal();
    for (int d = blockIdx.y; ok && d < count; d += step) {
      const int adapter = uniform(items.adapter[d]), t0 = uniform(items.first[d] & ~15);
      const int width = uniform((items.last[d] & ~15) + 16) - t0;
      for (int kb = kb_lo; kb < kb_hi; kb += p.per_stage) {
        if (!mbar_wait_warp(&empty_bar[stage], phase ^ 1u, abort_flag, p.wait_budget_ns, 0xd1)) {
          ok = false;
          break;
        }
        if (one) {
          const int n = min(p.per_stage, kb_hi - kb);
          mbar_arrive_expect_tx(&full_bar[stage], n * (p.a_rows + width) * 128);
          for (int i = 0; i < n; ++i) {
            const int at_k = (kb + i) * 64, slot = stage * p.per_stage + i;
            tma_load_3d_hint(a_smem + slot * a_bytes, &maps.a, &full_bar[stage], at_k, j0, adapter, pol_a);
            grp_token_boxes(width, [&](int b, int at) {
              tma_load_2d_hint(x_smem + slot * x_bytes + at * 128, &maps.x[b], &full_bar[stage], at_k, m0 + t0 + at, pol_x);
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
        mbar_wait(&full_bar[s], parities >> s & 1u, &no_abort, p.wait_budget_ns, 0xd2);
      }
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    int stage = 0, local = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint64_t a_desc0 = make_sw128_desc(smem_u32(a_smem), 16, 1024);
    const uint64_t x_desc0 = make_sw128_desc(smem_u32(x_smem), 16, 1024);
    const uint32_t d_tmem = uniform(tmem_base);
    for (int d = blockIdx.y; ok && d < count; d += step, ++local) {
      const int width = uniform(((items.last[d] & ~15) + 16) - (items.first[d] & ~15));
      const uint32_t idesc = p.idesc | static_cast<uint32_t>(width >> 3) << 17;
      if (!mbar_wait_warp(acc_empty_bar, (local & 1) ^ 1u, abort_flag, p.wait_budget_ns, 0xd3)) break;
      tcgen05_fence_after_sync();
      for (int kb = kb_lo; kb < kb_hi; kb += p.per_stage) {
        if (!mbar_wait_warp(&full_bar[stage], phase, abort_flag, p.wait_budget_ns, 0xd4)) {
          ok = false;
          break;
        }
        tcgen05_fence_after_sync();
        const int n = min(p.per_stage, kb_hi - kb);
        const uint64_t a_desc = a_desc0 + stage * p.per_stage * (a_bytes / 16);
        const uint64_t x_desc = x_desc0 + stage * p.per_stage * (x_bytes / 16);
        if (one) {
          for (int i = 0; i < n; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f16_ss(d_tmem, a_desc + i * (a_bytes / 16) + k * 2, x_desc + i * (x_bytes / 16) + k * 2, idesc,
                          kb > kb_lo || i > 0 || k > 0 ? 1u : 0u);
          umma_commit(&empty_bar[stage]);
        }
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok && one) umma_commit(acc_full_bar);
    }
    if (one) umma_commit(mma_done_bar);
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait(mma_done_bar, 0, &no_abort, p.wait_budget_ns, 0xd5);
    __syncwarp();
  } else {
    const int quad = warp & 3;
    const int j = quad * 32 + lane;  // row of A
    const int e = threadIdx.x - Cfg::EPI_WARP0 * 32;
    const int share = (p.tokens / 4 + p.splits - 1) / p.splits;  // four tokens each, of a source
    int local = 0;
    constexpr bool powers = !BF16;
    const int groups = p.rank >> 3;  // of eight ranks
    // Whether the 32-token blocks that are the adapter's alone (bit i: tokens 32 i and
    // on) hold what needs a power, as far as this warp has seen.
    auto note = [&](int adapter, unsigned misfit) {
      misfit = __reduce_or_sync(0xffffffffu, misfit);
      for (int b = 0; b * 32 < p.tokens; ++b) {
        if (kinds[b] != adapter || lane != 0) continue;
        uint8_t* at = p.misfits + (static_cast<int64_t>((m0 >> 5) + b) * gridDim.z + blockIdx.z) * 8 + quad * 2;
        const unsigned bit = misfit >> b & 1u;
        if (p.splits == 1)
          *reinterpret_cast<unsigned short*>(at) = static_cast<unsigned short>(bit);
        else
          at[rank] = static_cast<uint8_t>(bit);
      }
      __syncwarp();
    };
    for (int d = blockIdx.y; d < count; d += step) {
      const int adapter = items.adapter[d], t0 = items.first[d] & ~15, width = ((items.last[d] & ~15) + 16) - t0;
      unsigned misfit = 0;
      const int fours = width / 4, mine = (fours - rank + p.splits - 1) / p.splits;  // those of this CTA: rank, rank + splits, ...
      const float scale = p.scale != nullptr ? __ldg(p.scale + adapter) : 1.0f;
      bool ready = mbar_wait(acc_full_bar, local & 1, abort_flag, p.wait_budget_ns, 0xd6);
      if (p.splits == 1) {  // nothing to exchange
        if (!__all_sync(0xffffffffu, ready)) break;
        tcgen05_fence_after_sync();
        for (int c = 0; c < width && quad * 32 < rows; c += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + c, r);
          const int m = m0 + t0 + c;
          const int owner = lane < 16 && m + lane < p.M ? __ldg(p.index + m + lane) : -1;
          const unsigned mine_of = __ballot_sync(0xffffffffu, owner == adapter);
          tmem_ld_wait();
          unsigned short* dst = static_cast<unsigned short*>(p.t) + static_cast<int64_t>(m) * p.rank + j0 + j;
#pragma unroll
          for (int q = 0; q < 16; ++q)
            if (j < rows && (mine_of >> q & 1u)) dst[q * p.rank] = round_16(__uint_as_float(r[q]) * scale, BF16);
          if (powers) {
            if (lane < 16 && (mine_of >> lane & 1u)) {
              const int here = min(4, (rows - quad * 32) >> 3);
              signed char* at = p.exps + static_cast<int64_t>(m + lane) * groups + (j0 >> 3) + quad * 4;
              if (here == 4 && (groups & 3) == 0)
                *reinterpret_cast<uint32_t*>(at) = 0u;
              else
                for (int g = 0; g < here; ++g) at[g] = 0;
            }
            // As a rule that was it: each eight ranks have a normal number, none passes the range.
            unsigned lost = 0;
            bool past = false;
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float v = fabsf(__uint_as_float(r[q]) * scale);
              const unsigned normal = __ballot_sync(0xffffffffu, v >= kLoraLeast || j >= rows);
              const unsigned none = (normal - 0x01010101u) & ~normal & 0x80808080u;  // a byte of zeros
              lost |= mine_of >> q & 1u ? none : 0u;
              past = past || ((mine_of >> q & 1u) && j < rows && v >= kLoraMost);
            }
            if (lost != 0 || __any_sync(0xffffffffu, past)) {
              __syncwarp();
#pragma unroll 1
              for (int q = 0; q < 16; ++q) {  // short: it is read from memory when it is first needed
                uint32_t one;
                tmem_ld_32x32b_x1(tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + c + q, one);
                tmem_ld_wait();
                const LoraRounded t = lora_round(__uint_as_float(one) * scale);
                if (j < rows && (mine_of >> q & 1u)) {
                  if (t.e != 0) misfit |= 1u << ((t0 + c) >> 5);
                  if ((lane & 7) == 0) p.exps[static_cast<int64_t>(m + q) * groups + ((j0 + j) >> 3)] = static_cast<signed char>(t.e);
                  dst[q * p.rank] = t.y;
                }
                __syncwarp();  // the next load wants the whole warp
              }
            }
          }
        }
        if (powers) note(adapter, misfit);
        tcgen05_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty_bar);
        ++local;
        continue;
      }
      if (ready) ready = mbar_wait_cluster(part_empty_bar, (local & 1) ^ 1u, abort_flag, p.wait_budget_ns, 0xd7);
      if (!__all_sync(0xffffffffu, ready)) break;
      tcgen05_fence_after_sync();
      if (quad * 32 < rows) {
        for (int c = 0; c < width; c += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + c, r);
          tmem_ld_wait();
          if (j < rows) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int four = c / 4 + q;
              const uint32_t owner = four % p.splits;
              st_cluster_v4(mapa_shared(smem_u32(recv + (rank * share + four / p.splits) * p.a_rows + j), owner), r[4 * q],
                            r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
            }
          }
        }
      }
      tcgen05_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(acc_empty_bar);
        fence_cluster();
        for (int q = 0; q < p.splits; ++q) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(part_full_bar), q));
      }
      ready = mbar_wait_cluster(part_full_bar, local & 1, abort_flag, p.wait_budget_ns, 0xd8);
      if (!__all_sync(0xffffffffu, ready)) break;
      for (int it = e; it - lane < mine * rows; it += 128) {
        const bool in = it < mine * rows;
        const int four = in ? it / rows : 0, row = it - four * rows;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int q = 0; in && q < p.splits; ++q) {
          const float4 x = recv[(q * share + four) * p.a_rows + row];
          s.x = q == 0 ? x.x : s.x + x.x;
          s.y = q == 0 ? x.y : s.y + x.y;
          s.z = q == 0 ? x.z : s.z + x.z;
          s.w = q == 0 ? x.w : s.w + x.w;
        }
        const float v[4] = {s.x * scale, s.y * scale, s.z * scale, s.w * scale};
        const int m = m0 + t0 + (four * p.splits + rank) * 4;
        unsigned short* dst = static_cast<unsigned short*>(p.t) + static_cast<int64_t>(m) * p.rank + j0 + row;
        signed char* at = p.exps + static_cast<int64_t>(m) * groups + ((j0 + row) >> 3);
        unsigned own = 0, odd = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bool mine_q = in && m + q < p.M && __ldg(p.index + m + q) == adapter;
          own |= mine_q ? 1u << q : 0u;
          if (mine_q) dst[q * p.rank] = round_16(v[q], BF16);
          if (!powers) continue;
          if (mine_q && (lane & 7) == 0) at[q * groups] = 0;
          // Rows of A come in eights: eight lanes have the same token.
          const unsigned normal = __ballot_sync(0xffffffffu, !mine_q || fabsf(v[q]) >= kLoraLeast);
          odd |= (normal - 0x01010101u) & ~normal & 0x80808080u;
          odd |= mine_q && fabsf(v[q]) >= kLoraMost ? 1u : 0u;
        }
        if (powers && __any_sync(0xffffffffu, odd != 0)) {
          __syncwarp();
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            const LoraRounded t = lora_round(q == 0 ? v[0] : q == 1 ? v[1] : q == 2 ? v[2] : v[3]);
            if (own >> q & 1u) {
              if (t.e != 0) misfit |= 1u << ((m - m0) >> 5);
              if ((lane & 7) == 0) at[q * groups] = static_cast<signed char>(t.e);
              dst[q * p.rank] = t.y;
            }
            __syncwarp();
          }
        }
      }
      __syncwarp();
      if (powers) note(adapter, misfit);
      if (lane == 0)
        for (int q = 0; q < p.splits; ++q) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(part_empty_bar), q));
      ++local;
    }
  }

  tcgen05_fence_before_sync();
  __syncthreads();
  cluster_sync();  // nobody writes to a CTA that has left
  if (warp == 1) {
    tcgen05_fence_after_sync();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

// ----------------------------------------------------------------------------
// Few tokens: T[m][j] by a warp
// ----------------------------------------------------------------------------
struct LoraRowsParams {
  const void* x;
  const void* a;
  const int* index;
  const float* scale;  // of each adapter, or nullptr
  void* t;
  signed char* exps;   // fp16: T's powers, of each row and eight ranks
  int64_t ldx, lda, stride_a;
  int K, rank, adapters;
};

constexpr int kLoraRowsWarps = 8;  // the ranks that share a power

template <bool BF16>
__global__ void __launch_bounds__(kLoraRowsWarps * 32) lora_rows_kernel(const LoraRowsParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, m = blockIdx.x;
  const int j = blockIdx.y * kLoraRowsWarps + (threadIdx.x >> 5);
  const int adapter = __ldg(p.index + m);
  if (adapter < 0 || adapter >= p.adapters || j >= p.rank) return;  // the whole block: ranks come in eights
  const unsigned short* x = static_cast<const unsigned short*>(p.x) + m * p.ldx;
  const unsigned short* a = static_cast<const unsigned short*>(p.a) + adapter * p.stride_a + j * p.lda;
  const float scale = p.scale != nullptr ? __ldg(p.scale + adapter) : 1.0f;
  const float sum = lora_dot<BF16, 4>(a, x, p.K, lane);
  const float v = sum * scale;
  unsigned short y;
  if (!BF16) {
    __shared__ float values[kLoraRowsWarps];
    if (lane == 0) values[threadIdx.x >> 5] = v;
    __syncthreads();
    const LoraRounded r = lora_round(values[lane & 7]);
    y = __shfl_sync(0xffffffffu, r.y, threadIdx.x >> 5);  // this warp's value's
    if (threadIdx.x == 0) p.exps[static_cast<int64_t>(m) * (p.rank >> 3) + blockIdx.y] = static_cast<signed char>(r.e);
  } else {
    y = round_16(v, true);
  }
  if (lane == 0) static_cast<unsigned short*>(p.t)[static_cast<int64_t>(m) * p.rank + j] = y;
}

}  // namespace tg
