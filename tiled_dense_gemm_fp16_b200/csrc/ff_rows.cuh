// ff_rows.cuh -- the feed-forward block's passes over rows, both bound by
// memory: the gradients of the gate and up values, and row quantization to
// 8-bit integers.
#pragma once

#include "ff_ops.cuh"

namespace tg {

// ----------------------------------------------------------------------------
// dG = dH * U * act'(G), dU = dH * act(G)
// ----------------------------------------------------------------------------
// Reads dH, G and U once and writes dG and dU once (10 bytes an element).
// Rows of the results are padded to 8 elements (16 bytes) for the products
// that read them by TMA; rows of the inputs may start anywhere.  fp32
// arithmetic, one rounding to the operands' type, which is what the tensor
// cores read.
struct GatedGradParams {
  const void* dH;
  const void* G;
  const void* U;
  void* dG;
  void* dU;
  int64_t ld_dh, ld_g, ld_u, ld_out;
  int M, N;
  int vec;  // rows of dH, G and U start on 16-byte boundaries
  int bf16, act;
};

constexpr int kGatedGradThreads = 256;

__device__ __forceinline__ uint4 load8_16(const unsigned short* p, int n, bool vec) {
  if (vec && n >= 8) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) w[e >> 1] |= static_cast<uint32_t>(__ldg(p + e)) << ((e & 1) * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int ACT>
__device__ __forceinline__ void gated_grad_rows(const GatedGradParams& p) {
  const bool bf16 = p.bf16 != 0, vec = p.vec != 0;
  const int col = (blockIdx.x * kGatedGradThreads + threadIdx.x) * 8;
  if (col >= p.N) return;
  const int n = p.N - col;
  for (int row = blockIdx.y; row < p.M; row += gridDim.y) {
    const int64_t r = row;
    const uint4 d4 = load8_16(static_cast<const unsigned short*>(p.dH) + r * p.ld_dh + col, n, vec);
    const uint4 g4 = load8_16(static_cast<const unsigned short*>(p.G) + r * p.ld_g + col, n, vec);
    const uint4 u4 = load8_16(static_cast<const unsigned short*>(p.U) + r * p.ld_u + col, n, vec);
    const uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w}, gw[4] = {g4.x, g4.y, g4.z, g4.w},
                   uw[4] = {u4.x, u4.y, u4.z, u4.w};
    float dg[8], du[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 d = unpack_16(dw[q], bf16), g = unpack_16(gw[q], bf16), u = unpack_16(uw[q], bf16);
      float2 a, s;
      act_value_slope2<ACT>(g, a, s);
      const float2 vg = mul2(mul2(d, u), s), vu = mul2(d, a);
      dg[2 * q] = vg.x;
      dg[2 * q + 1] = vg.y;
      du[2 * q] = vu.x;
      du[2 * q + 1] = vu.y;
    }
    uint32_t h[4];
    pack_row<8>(dg, h, bf16);
    *reinterpret_cast<uint4*>(static_cast<unsigned short*>(p.dG) + r * p.ld_out + col) =
        make_uint4(h[0], h[1], h[2], h[3]);
    pack_row<8>(du, h, bf16);
    *reinterpret_cast<uint4*>(static_cast<unsigned short*>(p.dU) + r * p.ld_out + col) =
        make_uint4(h[0], h[1], h[2], h[3]);
  }
}

__global__ void __launch_bounds__(kGatedGradThreads) gated_grad_kernel(const GatedGradParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (p.act == kActSilu)
    gated_grad_rows<kActSilu>(p);
  else if (p.act == kActGelu)
    gated_grad_rows<kActGelu>(p);
  else
    gated_grad_rows<kActRelu>(p);
}

// ----------------------------------------------------------------------------
// Row quantization
// ----------------------------------------------------------------------------
// scale = max |x| / 127 (one IEEE fp32 division), q = x / scale rounded to the
// nearest integer, ties to even, exactly.  Two steps:
//   * t = x * (1 / scale), off from the quotient by at most 127 * 2^-23; one
//     fused multiply-add onto 1.5 * 2^23 leaves its nearest integer in the low
//     mantissa bits, a second gives the distance of t from that integer;
//   * where a distance comes within 2^-14 of a half (a few values in ten
//     thousand), the chunk is settled by remainders: r = x - q scale, which
//     one fused multiply-add gives without error (|r| stays below 2 scale and
//     is a multiple of scale's last place).
// So codes do not depend on how a division rounds.  |q| <= 127.
//
// Bound by memory: 2 bytes in and 1 out an element, each read once.  A row is
// held in registers between its maximum and its codes (up to THREADS * 8 HELD
// values; what a longer row has more is read again, from L2), and the next
// row's loads are in flight meanwhile.
struct QuantizeParams {
  const void* X;
  int8_t* Q;
  float* scale;
  int64_t ldx, ldq;
  int M, K;
  int vec;  // rows of X start on 16-byte boundaries, rows of Q on 8-byte ones
  int bf16;
};

constexpr float kTwo64 = 18446744073709551616.0f;

__device__ __forceinline__ int quantize_settled(float x, float scale, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, scale, x);
  const float half = 0.5f * scale;
  const bool odd = (static_cast<int>(q) & 1) != 0;
  // Past the half (or on it with an odd q) the neighbour on r's side is right.
  if (r > half || (r == half && odd)) q += 1.0f;
  if (-r > half || (-r == half && odd)) q -= 1.0f;
  return static_cast<int>(q);
}

// Eight codes of one chunk, packed.  `tiny`: scale is below 2^-64, where 1 /
// scale could overflow; values and scale are multiplied by 2^64 first (exact),
// and `inv` belongs to the product.
__device__ __forceinline__ uint2 quantize8(const uint4& v, float scale, float inv, bool tiny, bool bf16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack_16(w[e], bf16);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
  if (!tiny) {
    uint32_t q[8];
    float worst = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f = fmaf(x[e], inv, kMagic);
      worst = fmaxf(worst, fabsf(fmaf(x[e], inv, kMagic - f)));
      q[e] = __float_as_uint(f);
    }
    if (worst < 0.5f - 6.103515625e-5f)
      return make_uint2(__byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410),
                        __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410));
  }
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int q = quantize_settled(tiny ? x[e] * kTwo64 : x[e], tiny ? scale * kTwo64 : scale, inv);
    out[e >> 2] |= static_cast<uint32_t>(q & 0xff) << ((e & 3) * 8);
  }
  return make_uint2(out[0], out[1]);
}

// THREADS threads per row: a warp (several rows a block) or a whole block of
// them.  HELD: 16-byte chunks a thread keeps.
template <int THREADS, int HELD>
struct QuantizeCfg {
  static constexpr int BLOCK = THREADS < 256 ? 256 : THREADS;
  static constexpr int ROWS = BLOCK / THREADS;
  static constexpr int HELD_VALUES = THREADS * HELD * 8;
};

template <int THREADS, int HELD>
__global__ void __launch_bounds__(QuantizeCfg<THREADS, HELD>::BLOCK) quantize_rows_kernel(const QuantizeParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  using Cfg = QuantizeCfg<THREADS, HELD>;
  constexpr int WARPS = Cfg::BLOCK / 32;
  __shared__ uint32_t warp_max[2][WARPS];
  const int t = threadIdx.x % THREADS;
  const bool bf16 = p.bf16 != 0, vec = p.vec != 0;
  const int chunks = (p.K + 7) / 8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * Cfg::ROWS;
  int64_t row = static_cast<int64_t>(blockIdx.x) * Cfg::ROWS + threadIdx.x / THREADS;
  auto row_of = [&](int64_t r) { return static_cast<const unsigned short*>(p.X) + r * p.ldx; };
  auto load = [&](int64_t r, uint4 (&held)[HELD]) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int c = t + i * THREADS;
      held[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < p.M && c < chunks) held[i] = load8_16(row_of(r) + c * 8, p.K - c * 8, vec);
    }
  };
  uint4 held[HELD], next[HELD];
  load(row, held);
  int parity = 0;
  for (; row < p.M; row += stride, parity ^= 1) {
    load(row + stride, next);
    // The maximum of the magnitudes' bits: fp16 and bf16 order as integers,
    // and infinities and NaN come out above every finite value.
    uint32_t best = 0u;
    auto take = [&](const uint4& v) {
      best = __vmaxu2(best, v.x & 0x7fff7fffu);
      best = __vmaxu2(best, v.y & 0x7fff7fffu);
      best = __vmaxu2(best, v.z & 0x7fff7fffu);
      best = __vmaxu2(best, v.w & 0x7fff7fffu);
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i) take(held[i]);
    for (int c = t + HELD * THREADS; c < chunks; c += THREADS) take(load8_16(row_of(row) + c * 8, p.K - c * 8, vec));
    best = max(best & 0xffffu, best >> 16);
    best = __reduce_max_sync(0xffffffffu, best);
    if (THREADS > 32) {
      if ((threadIdx.x & 31) == 0) warp_max[parity][threadIdx.x >> 5] = best;
      __syncthreads();  // the other half of warp_max serves the next row, so one barrier a row is enough
      best = __reduce_max_sync(0xffffffffu, warp_max[parity][threadIdx.x & (WARPS - 1)]);
    }
    const float amax =
        bf16 ? __uint_as_float(best << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(best)));
    const bool finite = best < (bf16 ? 0x7f80u : 0x7c00u);
    const float scale = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7fffffffu);
    const bool live = finite && scale > 0.0f;
    const bool tiny = scale < 5.421010862427522e-20f;  // 2^-64
    const float inv = live ? __fdiv_rn(1.0f, tiny ? scale * kTwo64 : scale) : 0.0f;
    if (t == 0) p.scale[row] = scale;
    int8_t* dst = p.Q + row * p.ldq;
    auto put = [&](int c, const uint4& v) {
      const uint2 q = live ? quantize8(v, scale, inv, tiny, bf16) : make_uint2(0u, 0u);
      const int n = p.K - c * 8;
      if (vec && n >= 8) {
        *reinterpret_cast<uint2*>(dst + c * 8) = q;
      } else {
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < n) dst[c * 8 + e] = static_cast<int8_t>(w[e >> 2] >> ((e & 3) * 8));
      }
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int c = t + i * THREADS;
      if (c < chunks) put(c, held[i]);
    }
    for (int c = t + HELD * THREADS; c < chunks; c += THREADS) put(c, load8_16(row_of(row) + c * 8, p.K - c * 8, vec));
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = next[i];
  }
}

// ----------------------------------------------------------------------------
// An 8-bit product without any K: every row is bias, or +0 (with ReLU on it)
// ----------------------------------------------------------------------------
struct BiasFillParams {
  void* C;
  const void* bias;  // or nullptr
  int64_t ldc;
  int M, N;
  int relu, bf16;
};

__global__ void __launch_bounds__(256) bias_fill_kernel(const BiasFillParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t items = static_cast<int64_t>(p.M) * p.N;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < items;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t m = i / p.N, n = i - m * p.N;
    float v = p.bias ? load_16(static_cast<const unsigned short*>(p.bias) + n, p.bf16 != 0) : 0.0f;
    if (p.relu) v = v > 0.0f ? v : 0.0f;
    static_cast<unsigned short*>(p.C)[m * p.ldc + n] = round_16(v, p.bf16 != 0);
  }
}

}  // namespace tg
