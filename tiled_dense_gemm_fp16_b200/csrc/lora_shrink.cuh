// lora_shrink.cuh -- the first half of the low-rank adapters:
// T[m][j] = scale_a sum_k A_a[j][k] X[m][k] with a = index[m].
//
// A block takes 32 tokens and one of the adapters among them (most blocks of a
// prompt find one, decoding requests up to 32, over blockIdx.y), up to 64 rows
// of A.  Its 8 warps split K; each multiplies 32 x 16 by 16 x 8 on the warp-level
// tensor cores, whose rows are independent: tokens of other adapters are read as
// zeros and not written.  Within 32 values of K a thread's fragments are 8
// adjacent ones (the sum's order is free), so every load is 16 bytes, straight
// into registers.  Bound by reading X and the adapters' A.  T is rounded once to the 16-bit
// type, as the tensor cores read it (and as two linear layers in a row would).
#pragma once

#include "grp_ops.cuh"
#include "gemm_grp_pair.cuh"

namespace tg {

struct LoraShrinkParams {
  const void* x;
  const void* a;
  const int* index;
  const float* scale;        // of each adapter, or nullptr
  void* t;
  int* kind;
  int64_t ldx, lda, stride_a;
  int M, K, rank, adapters;
  int bf16;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, bool bf16) {
  if (bf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 values from p on, of which n (any number) are in the row; p on 16 bytes.
__device__ __forceinline__ uint4 row8(const unsigned short* p, int n) {
  if (n >= 8) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) w[e >> 1] |= static_cast<uint32_t>(__ldg(p + e)) << ((e & 1) * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kShrinkWarps = 8;

// NT: tiles of 8 rows of A.
template <int NT, bool BF16>
__global__ void __launch_bounds__(kShrinkWarps * 32) lora_shrink_kernel(const LoraShrinkParams p) {
  __shared__ float sums[4][32 * NT * 8];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m0 = blockIdx.x * 32, j0 = blockIdx.z * NT * 8;
  const int a_of = m0 + lane < p.M ? __ldg(p.index + m0 + lane) : -1;
  const int mine = a_of >= 0 && a_of < p.adapters ? a_of : -1;
  const unsigned valid = __ballot_sync(0xffffffffu, m0 + lane < p.M);
  unsigned left = __ballot_sync(0xffffffffu, mine >= 0);
  if (blockIdx.y == 0 && blockIdx.z == 0 && warp == 0) {
    const int r0 = __shfl_sync(0xffffffffu, mine, 0);
    const unsigned same = __ballot_sync(0xffffffffu, mine == r0) & valid;
    if (lane == 0) p.kind[blockIdx.x] = left == 0 ? kLoraNone : same == valid ? r0 : kLoraMixed;
  }
  for (int d = 0; left != 0; ++d) {
    const int r = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
    const unsigned rows = __ballot_sync(0xffffffffu, mine == r);
    left &= ~rows;
    if (d % gridDim.y != blockIdx.y) continue;
    float acc[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.0f;
    const int row = lane >> 2, q = lane & 3;
    const unsigned short* x = static_cast<const unsigned short*>(p.x) + static_cast<int64_t>(m0 + row) * p.ldx;
    const unsigned short* a = static_cast<const unsigned short*>(p.a) + r * p.stride_a + static_cast<int64_t>(j0 + row) * p.lda;
    for (int k = warp * 32 + q * 8; k - q * 8 < p.K; k += kShrinkWarps * 32) {
      uint4 xv[4], av[NT];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xv[i] = (rows >> (row + 8 * i)) & 1u ? row8(x + 8 * i * p.ldx + k, p.K - k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        av[n] = j0 + n * 8 + row < p.rank ? row8(a + n * 8 * p.lda + k, p.K - k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma_16816(acc[i][n], xv[2 * i].x, xv[2 * i + 1].x, xv[2 * i].y, xv[2 * i + 1].y, av[n].x, av[n].y, BF16);
          mma_16816(acc[i][n], xv[2 * i].z, xv[2 * i + 1].z, xv[2 * i].w, xv[2 * i + 1].w, av[n].z, av[n].w, BF16);
        }
    }
    // The warps' sums, pairwise in a fixed order: 4 to 7 onto 0 to 3, 2 and 3 onto 0 and 1, 1 onto 0.
#pragma unroll
    for (int half = kShrinkWarps / 2; half > 0; half >>= 1) {
      __syncthreads();
      if (warp >= half && warp < 2 * half) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[warp - half][((i * NT + n) * 4 + e) * 32 + lane] = acc[i][n][e];
      }
      __syncthreads();
      if (warp < half) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][n][e] += sums[warp][((i * NT + n) * 4 + e) * 32 + lane];
      }
    }
    if (warp == 0) {
      const float s = p.scale != nullptr ? __ldg(p.scale + r) : 1.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int m = 16 * i + 8 * h + row;
          if (!((rows >> m) & 1u)) continue;
          uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<unsigned short*>(p.t) + static_cast<int64_t>(m0 + m) * p.rank + j0) + q;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (j0 + n * 8 >= p.rank) break;  // rank is a multiple of 8
            const float u = acc[i][n][2 * h] * s, v = acc[i][n][2 * h + 1] * s;
            dst[n * 4] = BF16 ? pack_bf16(u, v) : pack_f16(u, v);
          }
        }
    }
  }
}

}  // namespace tg
