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

// ----------------------------------------------------------------------------
// Groups
// ----------------------------------------------------------------------------
// Group g owns rows [ends[g - 1], ends[g]) of X (from 0 for g = 0).  The ends
// are data on the device, so nothing on the host depends on them and a captured
// graph may be replayed with others.  They are clamped to [0, M], and a group
// whose end lies before its start is empty: whatever they hold, no access leaves
// a matrix.  Without ends (one weight for all rows) there is one group.
__device__ __forceinline__ int grp_end(const int* ends, int g, int M) {
  if (g < 0) return 0;
  return ends == nullptr ? M : max(0, min(__ldg(ends + g), M));
}

// A group's rows in tiles of at most `most`: as many as are needed, of equal
// width up to `unit`, so that no tile is a sliver.  The last one starts before
// the group's end, since tiles - 1 of the widest would not hold the group.
__device__ __forceinline__ int grp_tile_width(int rows, int most, int unit) {
  const int tiles = (rows + most - 1) / most;
  const int even = (rows + tiles - 1) / tiles;
  return (even + unit - 1) / unit * unit;
}

// Starts and running numbers of tiles, in shared memory: group G stands for the
// rows behind the last group, which get zeros where `rest` is set.
struct GrpPlan {
  int* lo;     // G + 2 row starts; the rows of g end at lo[g + 1]
  int* first;  // G + 2 numbers of tiles before the group, in tiles of the whole result
};

constexpr int grp_plan_bytes(int groups) { return (groups + 2) * 8; }

// By one warp; the others wait for it.
__device__ __forceinline__ void grp_make_plan(GrpPlan plan, const int* ends, int G, int M, int most, int col_tiles,
                                              bool rest, int lane) {
  int before = 0;
  for (int base = 0; base <= G; base += 32) {
    const int g = base + lane;
    int lo = 0, tiles = 0;
    if (g <= G) {
      lo = grp_end(ends, g - 1, M);
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

struct GrpWalk {
  int g = 0;
  __device__ __forceinline__ GrpTile at(const GrpPlan& plan, int t, int col_tiles, int super, int most, int unit) {
    while (t >= plan.first[g + 1]) ++g;  // t < first[G + 1]
    GrpTile f;
    f.g = g;
    const int lo = plan.lo[g], rows = plan.lo[g + 1] - lo;
    const int tiles = (rows + most - 1) / most, width = grp_tile_width(rows, most, unit);
    const int local = t - plan.first[g];
    const int s = local / (super * col_tiles);
    const int wide = min(super, tiles - s * super);
    const int in = local - s * super * col_tiles;
    f.col_blk = in / wide;
    const int i = s * super + in - f.col_blk * wide;
    f.tok0 = lo + i * width;
    f.cnt = min(width, rows - i * width);
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

// The box's first `rows` rows and `cols` columns to `c`.  vec: rows of the result
// start on 16-byte boundaries (and c's column is a multiple of 8): 16 bytes a
// lane, 8 rows a store.  Else value by value, a row a store.
__device__ __forceinline__ void grp_store_box(unsigned short* c, int64_t ld, int rows, int cols, bool vec,
                                              const uint8_t* box, int lane) {
  if (vec) {
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
  } else if (lane < cols) {
    unsigned short* dst = c + lane;
#pragma unroll 4
    for (int r = 0; r < 32; ++r) {
      if (r >= rows) break;
      dst[r * ld] = *reinterpret_cast<const unsigned short*>(box + grp_box_at(r, lane >> 3) + (lane & 7) * 2);
    }
  }
}

}  // namespace tg
