// ff_rows.cuh -- the feed-forward block's passes over rows, both bound by
// memory: the gradients of the gate and up values, and row quantization to
// 8-bit integers.
#pragma once

#include "ff_ops.cuh"
#include "gemm_tc.cuh"
#include "repack.cuh"

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

// The first n (up to 8) 16-bit values at p, zeros after them.  vec: p is on a
// 16-byte boundary.  Else two aligned 16-byte loads cover 8 values on any
// 2-byte boundary and are shifted into place, if both lie inside the matrix
// [lo, hi); what is left is read value by value.
__device__ __forceinline__ uint4 load8_16(const unsigned short* p, int n, bool vec, const void* lo, const void* hi) {
  if (n >= 8) {
    if (vec) return __ldg(reinterpret_cast<const uint4*>(p));
    const uintptr_t at = reinterpret_cast<uintptr_t>(p), block = at & ~uintptr_t(15);
    if (block >= reinterpret_cast<uintptr_t>(lo) && block + 32 <= reinterpret_cast<uintptr_t>(hi)) {
      const uint4* q = reinterpret_cast<const uint4*>(block);
      return edge_realign(__ldg(q), __ldg(q + 1), static_cast<uint32_t>(at - block));
    }
  }
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) w[e >> 1] |= static_cast<uint32_t>(__ldg(p + e)) << ((e & 1) * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// End of a matrix of `rows` rows of `cols` 16-bit values.
__device__ __forceinline__ const unsigned short* end_16(const void* p, int64_t rows, int64_t ld, int cols) {
  return static_cast<const unsigned short*>(p) + (rows - 1) * ld + cols;
}

// d * v for a v that may be an infinity because the stored 16-bit value
// overflowed: the value was finite, so a gradient of 0 (a padded token's) stays
// 0.  NaN in either carries over.
__device__ __forceinline__ float times_stored(float d, float v) {
  return d == 0.0f && fabsf(v) == __uint_as_float(0x7f800000u) ? 0.0f : d * v;
}

// dG of one element.  A closed gate gives 0 whatever U is, but does not hide a
// gradient that is not finite.
__device__ __forceinline__ float gate_grad(float d, float u, float slope) {
  return slope == 0.0f ? d * 0.0f : times_stored(d, u) * slope;
}

template <int ACT, int ROWS>
__device__ __forceinline__ void gated_grad_rows(const GatedGradParams& p) {
  constexpr int TX = kGatedGradThreads / ROWS;  // threads per row, 8 columns each
  const bool bf16 = p.bf16 != 0, vec = p.vec != 0;
  const int col = (blockIdx.x * TX + threadIdx.x % TX) * 8;
  if (col >= p.N) return;
  const int n = p.N - col;
  const void* end_d = end_16(p.dH, p.M, p.ld_dh, p.N);
  const void* end_g = end_16(p.G, p.M, p.ld_g, p.N);
  const void* end_u = end_16(p.U, p.M, p.ld_u, p.N);
  for (int row = blockIdx.y * ROWS + threadIdx.x / TX; row < p.M; row += gridDim.y * ROWS) {
    const int64_t r = row;
    const uint4 d4 = load8_16(static_cast<const unsigned short*>(p.dH) + r * p.ld_dh + col, n, vec, p.dH, end_d);
    const uint4 g4 = load8_16(static_cast<const unsigned short*>(p.G) + r * p.ld_g + col, n, vec, p.G, end_g);
    const uint4 u4 = load8_16(static_cast<const unsigned short*>(p.U) + r * p.ld_u + col, n, vec, p.U, end_u);
    const uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w}, gw[4] = {g4.x, g4.y, g4.z, g4.w},
                   uw[4] = {u4.x, u4.y, u4.z, u4.w};
    float dg[8], du[8];
    float2 check = same2(0.0f);  // 0 while every result is finite
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 d = unpack_16(dw[q], bf16), g = unpack_16(gw[q], bf16), u = unpack_16(uw[q], bf16);
      float2 a, s;
      act_value_slope2<ACT>(g, a, s);
      const float2 vg = mul2(mul2(d, u), s), vu = mul2(d, a);
      check = fma2(vg, same2(0.0f), fma2(vu, same2(0.0f), check));
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
    if (!(check.x + check.y == 0.0f)) {
      // Rare, so tested once for eight columns and gone through value by value
      // (98 us at 8192 x 8192; 102 with these rules in every element).
#pragma unroll 1
      for (int c = col; c < p.N && c < col + 8; ++c) {
        const float d = load_16(static_cast<const unsigned short*>(p.dH) + r * p.ld_dh + c, bf16);
        const float g = load_16(static_cast<const unsigned short*>(p.G) + r * p.ld_g + c, bf16);
        const float u = load_16(static_cast<const unsigned short*>(p.U) + r * p.ld_u + c, bf16);
        float2 a, s;
        act_value_slope2<ACT>(same2(g), a, s);
        static_cast<unsigned short*>(p.dG)[r * p.ld_out + c] = round_16(gate_grad(d, u, s.x), bf16);
        static_cast<unsigned short*>(p.dU)[r * p.ld_out + c] = round_16(times_stored(d, a.x), bf16);
      }
    }
  }
}

// ROWS rows a block at a time, so that short rows leave no thread idle.
template <int ROWS>
__global__ void __launch_bounds__(kGatedGradThreads) gated_grad_kernel(const GatedGradParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (p.act == kActSilu)
    gated_grad_rows<kActSilu, ROWS>(p);
  else if (p.act == kActGelu)
    gated_grad_rows<kActGelu, ROWS>(p);
  else
    gated_grad_rows<kActRelu, ROWS>(p);
}

// ----------------------------------------------------------------------------
// Row quantization
// ----------------------------------------------------------------------------
// scale = max |x| / 127 (one IEEE fp32 division), q = x / scale rounded to the
// nearest integer, ties to even, exactly.  One fused multiply-add of x * inv
// onto 1.5 * 2^23 leaves the nearest integer in the low mantissa bits; what
// makes it exact is inv, 1 / scale rounded in the direction that ties need:
//   * x and max |x| = A are integers below 2^11 times powers of two, so 127 x /
//     A either is a half-integer exactly (a rational tie) or stays away from
//     every half-integer by 1 / (2 * 127 * 2047) of itself or more, 1.9e-6.
//     Scale and inv are off by 2^-24 and 2^-23, 1.8e-7: only rational ties
//     are in doubt;
//   * at a rational tie x / scale is off the tie to the side that scale's
//     rounding sends it: away from zero where scale < A / 127, so inv is
//     rounded up there, and down where scale > A / 127;
//   * where scale = A / 127 exactly, ties are true ones: inv is exact if scale
//     is a power of two, and the row is settled by remainders otherwise (8 of
//     1024 fp16 maxima; no bf16 one), as are rows with scale below 2^-64, whose
//     rounding may be coarser.
// |q| <= 127.
//
// Bound by memory: 2 bytes in and 1 out an element, each read once.  A row is
// held in registers between its maximum and its codes (up to THREADS * 8 HELD
// values; what a longer row has more is read again, from L2).  Enough rows are
// in flight per SM to cover the memory's latency.
struct QuantizeParams {
  const void* X;
  int8_t* Q;
  float* scale;
  int64_t ldx, ldq;
  int M, K;
  int vec_out;  // rows of Q start on 8-byte boundaries
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

// Eight codes of one chunk, packed, each settled by its remainder.  `tiny`:
// scale is below 2^-64, where 1 / scale could overflow; values and scale are
// multiplied by 2^64 first (exact), and `inv` belongs to the product.  Out of
// line: it is rarely called, and its registers would cost the others warps.
template <bool BF16>
__device__ __noinline__ uint2 quantize8_settled(uint4 v, float scale, float inv, bool tiny) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[2] = {0u, 0u};
  const float up = tiny ? kTwo64 : 1.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = unpack_16(w[e], BF16);
    const int q0 = quantize_settled(x.x * up, scale * up, inv), q1 = quantize_settled(x.y * up, scale * up, inv);
    out[e >> 1] |= (static_cast<uint32_t>(q0 & 0xff) | (static_cast<uint32_t>(q1 & 0xff) << 8)) << ((e & 1) * 16);
  }
  return make_uint2(out[0], out[1]);
}

// Eight codes of one chunk, packed.
template <bool BF16>
__device__ __forceinline__ uint2 quantize8(const uint4& v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  uint32_t half[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = fma2(unpack_16(w[e], BF16), same2(inv), same2(kMagic));
    half[e] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x0040);
  }
  return make_uint2(__byte_perm(half[0], half[1], 0x5410), __byte_perm(half[2], half[3], 0x5410));
}

// THREADS threads per row: a warp (several rows a block) or a whole block of
// them.  HELD: 16-byte chunks a thread keeps.  VEC: rows of X start on 16-byte
// boundaries.
template <int THREADS, int HELD>
struct QuantizeCfg {
  static constexpr int BLOCK = THREADS == 32 ? 256 : THREADS;
  static constexpr int ROWS = BLOCK / THREADS;
  static constexpr int HELD_VALUES = THREADS * HELD * 8;
  static constexpr int BLOCKS_PER_SM = 1536 / BLOCK;
};

template <int THREADS, int HELD, bool BF16, bool VEC>
__global__ void __launch_bounds__(QuantizeCfg<THREADS, HELD>::BLOCK,
                                  QuantizeCfg<THREADS, HELD>::BLOCKS_PER_SM) quantize_rows_kernel(const QuantizeParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  using Cfg = QuantizeCfg<THREADS, HELD>;
  constexpr int WARPS = Cfg::BLOCK / 32;
  constexpr int STEP = THREADS * 8;  // values between a thread's chunks
  __shared__ uint32_t warp_max[2][WARPS];
  const int first = (threadIdx.x % THREADS) * 8;  // this thread's chunks start at first + i STEP
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * Cfg::ROWS + threadIdx.x / THREADS;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * Cfg::ROWS;
  const unsigned short* src = static_cast<const unsigned short*>(p.X) + row0 * p.ldx + first;
  int8_t* dst = p.Q + row0 * p.ldq + first;
  const void* end = end_16(p.X, p.M, p.ldx, p.K);
  const bool vec_out = p.vec_out != 0;
  int parity = 0;
  for (int64_t row = row0; row < p.M; row += stride, parity ^= 1) {
    uint4 held[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int n = p.K - first - i * STEP;
      held[i] = make_uint4(0u, 0u, 0u, 0u);
      if (n > 0) held[i] = load8_16(src + i * STEP, n, VEC, p.X, end);
    }
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
    for (int c = HELD * STEP; c < p.K - first; c += STEP) take(load8_16(src + c, p.K - first - c, VEC, p.X, end));
    best = max(best & 0xffffu, best >> 16);
    best = __reduce_max_sync(0xffffffffu, best);
    if (THREADS > 32) {
      if ((threadIdx.x & 31) == 0) warp_max[parity][threadIdx.x >> 5] = best;
      __syncthreads();  // the other half of warp_max serves the next row, so one barrier a row is enough
      best = __reduce_max_sync(0xffffffffu, warp_max[parity][threadIdx.x & (WARPS - 1)]);
    }
    const float amax =
        BF16 ? __uint_as_float(best << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(best)));
    const bool finite = best < (BF16 ? 0x7f80u : 0x7c00u);
    const float scale = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7fffffffu);
    const bool live = finite && scale > 0.0f;
    const bool tiny = scale < 5.421010862427522e-20f;  // 2^-64
    const float off = fmaf(-scale, 127.0f, amax);      // exact: the sign of A / 127 - scale
    const bool settle = tiny || (off == 0.0f && (__float_as_uint(scale) & 0x7fffffu) != 0u);
    const float base = tiny ? scale * kTwo64 : scale;
    const float inv = !live ? 0.0f : off > 0.0f ? __fdiv_ru(1.0f, base) : __fdiv_rd(1.0f, base);
    if (first == 0) p.scale[row] = scale;
    auto put = [&](int c, const uint4& v) {
      const uint2 q = !live ? make_uint2(0u, 0u)
                      : settle ? quantize8_settled<BF16>(v, scale, inv, tiny)
                               : quantize8<BF16>(v, inv);
      const int n = p.K - first - c;
      if (vec_out && n >= 8) {
        *reinterpret_cast<uint2*>(dst + c) = q;
      } else {
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < n) dst[c + e] = static_cast<int8_t>(w[e >> 2] >> ((e & 3) * 8));
      }
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (p.K - first > i * STEP) put(i * STEP, held[i]);
    for (int c = HELD * STEP; c < p.K - first; c += STEP) put(c, load8_16(src + c, p.K - first - c, VEC, p.X, end));
    src += stride * p.ldx;
    dst += stride * p.ldq;
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

// ----------------------------------------------------------------------------
// Padded copies of up to three operands that TMA cannot describe, in one launch
// ----------------------------------------------------------------------------
// A warp copies a row: its lanes read the row's aligned 16-byte blocks, each
// once, take the block after theirs from the next lane, and shift by the row's
// offset, the same for all of them.  (3001 + 2 x 5003 rows of 1021 values: 15.6
// us when every lane read both of its blocks and worked out its own place.)
struct PadSetParams {
  RepackParams m[3];  // blockIdx.y picks one
};

// The aligned 16-byte block at `at`; what lies outside [lo, hi) is not read.
__device__ __forceinline__ uint4 load_block(uintptr_t at, uintptr_t lo, uintptr_t hi) {
  if (at >= lo && at + 16 <= hi) return __ldg(reinterpret_cast<const uint4*>(at));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (at + 2 * e >= lo && at + 2 * e < hi)
      w[e >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(at) + e)) << ((e & 1) * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(256) pad_set_kernel(const __grid_constant__ PadSetParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const RepackParams& m = p.m[blockIdx.y];
  const int lane = threadIdx.x & 31;
  const int chunks = m.cols_pad >> 3;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(m.src);
  const uintptr_t hi = lo + 2 * static_cast<uintptr_t>((m.rows - 1) * m.src_ld + m.cols);
  for (int row = blockIdx.x * 8 + (threadIdx.x >> 5); row < m.rows; row += gridDim.x * 8) {
    const uintptr_t start = lo + 2 * static_cast<uintptr_t>(row * m.src_ld);
    const uintptr_t first = start & ~uintptr_t(15);
    const uint32_t shift = static_cast<uint32_t>(start - first);
    uint4* dst = reinterpret_cast<uint4*>(m.dst + static_cast<int64_t>(row) * m.cols_pad);
    // Four blocks of a lane in flight.
    for (int c0 = lane; c0 - lane < chunks; c0 += 128) {
      uint4 v[4], last[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 32 * i;
        v[i] = last[i] = make_uint4(0u, 0u, 0u, 0u);
        if (c - lane < chunks) {
          v[i] = load_block(first + 16 * static_cast<uintptr_t>(c), lo, hi);
          if (lane == 31) last[i] = load_block(first + 16 * static_cast<uintptr_t>(c + 1), lo, hi);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 32 * i;
        if (c - lane >= chunks) break;
        uint4 b = make_uint4(__shfl_down_sync(0xffffffffu, v[i].x, 1), __shfl_down_sync(0xffffffffu, v[i].y, 1),
                             __shfl_down_sync(0xffffffffu, v[i].z, 1), __shfl_down_sync(0xffffffffu, v[i].w, 1));
        if (lane == 31) b = last[i];
        uint4 o = edge_realign(v[i], b, shift);
        const int n = m.cols - c * 8;
        if (n < 8) {  // the row's last values, then zeros
          uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) w[q] = n >= 2 * q + 2 ? w[q] : n == 2 * q + 1 ? w[q] & 0xffffu : 0u;
          o = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (c < chunks) dst[c] = o;
      }
    }
  }
}

}  // namespace tg
