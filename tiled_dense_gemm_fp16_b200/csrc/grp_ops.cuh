// grp_ops.cuh -- what the kernels of the grouped products and of the low-rank
// adapters share: the walk over ragged groups, loads of one matrix of several,
// staged 16-bit results.
//
// Both operators are products in which a row of X meets a weight that an index
// on the device picks, so tiles put the weight's rows on the MMA's M side (128
// lanes of TMEM a CTA) and the tokens on its N side, whose width an instruction
// chooses: a group of 40 rows costs 64 columns of N, where tokens on the M side
// would cost 256 rows.
#pragma once

#include "ff_ops.cuh"
#include "gemm_ff_pair.cuh"

namespace tg {

constexpr int kGrpMaxGroups = 1024;

// One matrix of a stack: box at (x, y, z), counted on the pair's even CTA.
__device__ __forceinline__ void tma_load_3d_pair_hint(void* smem_dst, const CUtensorMap* map, uint32_t bar_cluster_addr,
                                                      int x, int y, int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_hint(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y,
                                                 int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0u;
}
// A value that is the same in all lanes, as one that the compiler knows to be.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
// mbar_wait by a whole warp, with one answer.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t budget_ns,
                                               unsigned int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, budget_ns, site));
}

// 16 bytes into the shared memory of a CTA of the cluster.
__device__ __forceinline__ void st_cluster_v4(uint32_t cluster_addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void st_cluster_u16(uint32_t cluster_addr, unsigned short v) {
  asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(cluster_addr), "h"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}
// This lane's value of one column.
__device__ __forceinline__ void tmem_ld_32x32b_x1(uint32_t tmem, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(tmem));
}
// What this thread (and, after __syncwarp, its warp) has written is seen by a
// CTA of the cluster that acquires a later relaxed arrival.  One fence for several
// arrivals: each release at cluster scope measured about 1 us.
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

// ----------------------------------------------------------------------------
// Groups
// ----------------------------------------------------------------------------
// n / d for n >= 0, d > 0 with inv = 1 / d: every warp of a kernel places its tiles
// by divisions, and the compiler's takes 150 cycles or more one after the other.
// The product is off by one where n / d < 2^22, and by little beyond.
__device__ __forceinline__ int quick_div(int n, int d, float inv) {
  int q = __float2int_rz(__int2float_rn(n) * inv);
  int64_t r = n - static_cast<int64_t>(q) * d;
  while (r < 0) {
    --q;
    r += d;
  }
  while (r >= d) {
    ++q;
    r -= d;
  }
  return q;
}

// Group g owns rows [ends[g - 1], ends[g]) of X (from 0 for g = 0).  The ends
// are data on the device, so nothing on the host depends on them and a captured
// graph may be replayed with others.  They are clamped to [0, M] and raised to the
// greatest before them (grp_raise): whatever they hold, no access leaves a matrix,
// each row has one group, and the tiles of all groups are no more than the
// host has counted in 32 bits.  Without ends (one weight for all rows) there is one group.
__device__ __forceinline__ int grp_end(const int* ends, int g, int M) {
  if (g < 0) return 0;
  return ends == nullptr ? M : max(0, min(__ldg(ends + g), M));
}

// The starts of 32 groups in turn, a lane each, raised: `top` is that of the group
// before.  As a rule none has to be.
__device__ __forceinline__ int grp_raise(int lo, int& top, int lane) {
  const int before = __shfl_up_sync(0xffffffffu, lo, 1);
  if (!__all_sync(0xffffffffu, lo >= (lane == 0 ? top : before))) {
    lo = max(lo, top);
    for (int d = 1; d < 32; d <<= 1) lo = max(lo, __shfl_up_sync(0xffffffffu, lo, d));  // of lane < d: its own
  }
  top = __shfl_sync(0xffffffffu, lo, 31);
  return lo;
}

// A group's rows as tiles of `most`, whose last two share what a short last one
// would leave between them (a tile of few tokens still loads its whole weight
// tile).  All but the group's last width are multiples of `unit`.
struct GrpCut {
  int tiles, whole, width;  // `whole` tiles of `most`, one of `width` rows, and the rest in the last
};
__host__ __device__ __forceinline__ GrpCut grp_cut(int rows, int most, int unit) {
  GrpCut c;
  c.tiles = rows <= most ? 1 : (rows + most - 1) / most;
  c.whole = c.tiles - 1;
  c.width = 0;
  const int last = rows - c.whole * most;
  if (c.tiles >= 2 && 2 * last < most) {
    --c.whole;
    c.width = ((most + last + 1) / 2 + unit - 1) / unit * unit;
  }
  return c;
}
// First row and number of rows of tile i.
__host__ __device__ __forceinline__ void grp_cut_tile(const GrpCut& c, int rows, int most, int i, int& first, int& count) {
  first = (i < c.whole ? i : c.whole) * most + (i > c.whole ? c.width : 0);
  count = i < c.whole ? most : (i == c.whole && c.width != 0 ? c.width : rows - first);
}

// Starts and running numbers of tiles, in shared memory: group G stands for the
// rows behind the last group, which get zeros where `rest` is set.
struct GrpPlan {
  int* lo;     // G + 2 row starts; the rows of g end at lo[g + 1]
  int* first;  // G + 2 numbers of tiles before the group, in tiles of the whole result
};

__host__ __device__ constexpr int grp_plan_bytes(int groups) { return (groups + 2) * 8; }
__host__ __device__ constexpr int grp_plan_align(int groups) { return (grp_plan_bytes(groups) + 15) / 16 * 16; }

// By one warp; the others wait for it.
__device__ __forceinline__ void grp_make_plan(GrpPlan plan, const int* ends, int G, int M, int most, int col_tiles,
                                              bool rest, int lane) {
  int before = 0, top = 0;
  for (int base = 0; base <= G; base += 32) {
    const int g = base + lane;
    const int lo = grp_raise(g <= G ? grp_end(ends, g - 1, M) : M, top, lane);
    int tiles = 0;
    if (g <= G) {
      const int hi = g < G ? grp_end(ends, g, M) : (rest ? M : lo);
      tiles = hi > lo ? (hi - lo + most - 1) / most * col_tiles : 0;
    }
    int sum = tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int other = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += other;
    }
    if (g <= G) {
      plan.lo[g] = lo;
      plan.first[g] = before + sum - tiles;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (lane == 0) {
    plan.lo[G + 1] = M;
    plan.first[G + 1] = before;
  }
}

// Tile t of the walk, which goes up: group by group, in each the tokens' tiles
// of up to `super` next to each other for one tile of columns, so that the tiles
// in flight at one time share both operands in L2.
struct GrpTile {
  int g;          // group; G: rows behind the last one
  int tok0, cnt;  // rows of X and Y
  int col_blk;    // tile of result columns
};

// The walk of a whole warp.
struct GrpWalk {
  int g = 0;
  __device__ __forceinline__ GrpTile at(const GrpPlan& plan, int t, int col_tiles, int super, int most, int unit) {
    while (t >= plan.first[g + 1]) ++g;  // t < first[G + 1]
    GrpTile f;
    f.g = g;
    const int lo = plan.lo[g], rows = plan.lo[g + 1] - lo;
    const GrpCut cut = grp_cut(rows, most, unit);
    const int local = t - plan.first[g];
    int i = 0;
    f.col_blk = local;
    if (cut.tiles > 1) {  // divisions only where there is something to divide
      const int s = cut.tiles > super ? local / (super * col_tiles) : 0;
      const int wide = min(super, cut.tiles - s * super);
      const int in = local - s * super * col_tiles;
      f.col_blk = quick_div(in, wide, 1.0f / static_cast<float>(wide));
      i = s * super + in - f.col_blk * wide;
    }
    grp_cut_tile(cut, rows, most, i, f.tok0, f.cnt);
    f.tok0 += lo;
    f.g = uniform(f.g);
    f.tok0 = uniform(f.tok0);
    f.cnt = uniform(f.cnt);
    f.col_blk = uniform(f.col_blk);
    return f;
  }
};

// ----------------------------------------------------------------------------
// Results
// ----------------------------------------------------------------------------
// A warp's staging box: 32 rows of 32 values of 16 bits, 16-byte pieces swapped
// within a row so that neither side meets a bank twice.
constexpr int kGrpBoxBytes = 32 * 64;
__device__ __forceinline__ uint32_t grp_box_at(int row, int piece) {
  return static_cast<uint32_t>(row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
}

// The box's first `rows` rows and `cols` columns to `c`, whose rows start on
// 16-byte boundaries (and c's column is a multiple of 8): 16 bytes a lane, 8 rows a
// store.
__device__ __forceinline__ void grp_store_box(unsigned short* c, int64_t ld, int rows, int cols, const uint8_t* box, int lane) {
  const int piece = lane & 3;
  const int n = cols - piece * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    if (r >= rows || n <= 0) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(box + grp_box_at(r, piece));
    unsigned short* dst = c + r * ld + piece * 8;
    if (n >= 8) {
      *reinterpret_cast<uint4*>(dst) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < n) dst[e] = static_cast<unsigned short>(w[e >> 1] >> ((e & 1) * 16));
    }
  }
}

// Rows that start anywhere on 2 bytes, by the 128 threads whose warps have staged
// 32 rows of 128 columns (256 bytes a row).  Four threads a row: the whole 16-byte
// blocks of the result out of two staged pieces each, then the columns before the
// first block and behind the last one.
__device__ __forceinline__ void grp_store_rows(unsigned short* c, int64_t ld, int rows, int cols, const uint8_t* staged, int thread) {
  const int r = thread >> 2, q = thread & 3;
  if (r >= rows) return;
  unsigned short* row = c + r * ld;
  const uint8_t* from = staged + r * 256;
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1) & 7;  // columns from a boundary to the row's start
  const int head = (8 - skew) & 7;                                               // columns before the first block
  const int blocks = (cols - head) >> 3;                                         // negative: cols < head
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int g = q + 4 * i;
    if (g < blocks) {
      const uint4* piece = reinterpret_cast<const uint4*>(from) + g;
      // With head > 0 at most 15 blocks fit, so the piece behind is there.
      const uint4 v = head == 0 ? piece[0] : edge_realign(piece[0], piece[1], 2 * head);
      *reinterpret_cast<uint4*>(row + head + 8 * g) = v;
    }
  }
  const unsigned short* values = reinterpret_cast<const unsigned short*>(from);
  const int tail = blocks > 0 ? head + 8 * blocks : min(head, cols);  // columns from here on are left
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = q + 4 * i;
    if (e < min(head, cols)) row[e] = values[e];
    if (tail + e < cols) row[tail + e] = values[tail + e];
  }
}

// The 128 threads of a named barrier; whether `all` holds for each of them.
__device__ __forceinline__ bool bar_all_128(int id, bool all) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %2, 0;\n\t"
      "barrier.cta.red.and.pred p, %1, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(all))
      : "memory");
  return r != 0u;
}
__device__ __forceinline__ void bar_128(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }

}  // namespace tg
