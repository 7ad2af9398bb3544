// gemm_grp_pair.cuh -- products whose rows pick their weight, on CTA pairs
// (cta_group::2), persistent:
//   * grouped:  Y[r] = W_g X[r] (W_g stored N x K, read K-major), or its gradient
//     dX[r] = W_g^T dY[r] (the same weight read MN-major);
//   * adapters: Y[r] = W X[r] + B_a T[r] + bias with T[r] = s_a A_a X[r] of the row's
//     adapter a (made by the kernel of lora_shrink.cuh).
//
// A tile is 256 rows of a weight (128 a CTA) by up to 256 tokens: the even
// CTA's MMA thread issues 256 x width instructions over both SMs' shared memory,
// with the width of the tile at hand (a multiple of 32).  Two accumulators of
// 256 columns, so that the epilogue of a tile hides behind the next one.  The
// result leaves transposed: a lane of TMEM is a column of Y, so a warp stages
// 32 x 32 boxes with a row per token.
//
// Adapters: each 32 tokens that share one get its product as further k-blocks into
// their own 32 columns of the accumulator, so that no adapter's values meet
// another request's rows, not even times zero.  Tokens of several adapters within
// 32 (decoding requests beside each other, the ends of prompts) get theirs from the
// epilogue's warps (lora_part).
//
// Weights on the MMA's M side and tokens on its N side, since N may be any multiple
// of 32: a group of 40 rows costs 64, not 256.
//
// Measured alone: 8192 rows, 8 groups, 4096 x 7168, 321 us, 1.50 PFLOP/s, tensor pipe
// 83 % busy (one call after another the power cap holds it at 355-420).  Large tiles are
// bound by the tensor pipe, narrower ones by their operands' way from L2 (about 50
// bytes a cycle and SM), many groups of ~128 rows by reading the weights (64 of 1024 x
// 2048, 268 MB, 60 us, 4.5 TB/s).  Adapters, 8192 rows of 8, 8192 x 4096, rank 64: 383
// us, tensor pipe 77 % busy.
#pragma once

#include "grp_ops.cuh"

namespace tg {

struct GrpMaps {
  CUtensorMap w;     // the weights: boxes of 64 x 128, or 64 x 64 where read MN-major
  CUtensorMap x[4];  // tokens: boxes of 64 columns and 16, 32, 64, 128 rows
  CUtensorMap lb;    // adapters' B: boxes of 64 x 128
  CUtensorMap lt;    // T: boxes of 64 columns and 16 rows
};

// The adapters' part of a call.
struct LoraParams {
  const int* index;           // adapter of each token; outside [0, adapters): none
  const int* kind;            // of each 32 tokens: their adapter, kLoraNone or kLoraMixed
  const void* t;              // T: M x rank, 16-bit
  const signed char* exps;    // fp16: powers of two that T was divided by, of each row and eight ranks
  const uint2* misfits;       // fp16: of each 32 tokens, eight bytes per 128 ranks, all 0 if no value was divided
  int deep;                   // ranks in 128s
  const void* b;              // adapters' B
  const void* bias;           // N values, or nullptr
  int64_t ldb, stride_b;      // elements between rows and between adapters
  int rank, adapters;         // no adapters: only W's product and the bias
  // Where the main product makes T itself:
  const void* x;
  const void* a;              // adapters' A
  const float* scale;         // of each adapter, or nullptr
  int64_t ldx, lda, stride_a;
};
enum { kLoraNone = -1, kLoraMixed = -2 };

struct GrpParams {
  void* c;
  int64_t ldc;
  const int* ends;            // device; nullptr: one group of all rows
  int M, groups;
  int out, red;               // columns of the result, length of the sums
  int col_tiles, super;
  int k_blocks;
  int w_mn;                   // the weight is read MN-major (dX)
  int rest;                   // rows behind the last group get zeros
  int adapt;                  // few tiles: their width is chosen in the kernel
  int vec;                    // rows of the result start on 16-byte boundaries
  int bf16;
  int beside;                 // the kernel before this one writes nothing that it reads, and reads nothing that it writes
  uint32_t idesc;             // without N
  uint64_t wait_budget_ns;
  LoraParams lora;
};

__device__ __forceinline__ uint4 ld_v4(const void* p) {  // of any memory
  uint4 v;
  asm volatile("ld.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ int ld_global_s32(const int* p) {
  int v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// T's range.  bf16 has that of fp32; fp16 has not: s A X of 1e5 would be infinite, of
// 1e-7 lose its digits, where B T is an ordinary number.  So eight ranks of a row
// whose largest finite value is outside fp16's normal numbers below 2^15 are divided
// by the power of two that brings it to [2^15, 2^16), and its exponent stands beside
// T: values from 2^15 on say that there may be one.  lora_part then multiplies its fp32
// sums by it; 32 tokens of one adapter of which one has a power do not go through
// the main accumulator, whose other terms know none.  All others keep their bits.  A
// value of T is off by half a step, 2^-11 relative to it or to the largest of the 32
// ranks that are summed with it.  (A power for every row would close the accumulator's way to
// all: 8192 rows of 8 requests through 8192 x 4096, rank 64, 425 us, where all have one 957.)
constexpr float kLoraLeast = 6.103515625e-05f, kLoraMost = 32752.0f;  // below: still below 2^15 once rounded
constexpr float kLoraNothing = 3.85185988877447e-34f;                 // 2^-111: below, B T is far below fp16, and T is 0
__device__ __forceinline__ bool lora_fits(float v) { return fabsf(v) >= kLoraLeast && fabsf(v) < kLoraMost; }
// Of eight ranks with the largest finite magnitude m: the power's exponent, -126 .. 112, 0 for none.
__device__ __forceinline__ int lora_exponent(float m) {
  return m < kLoraNothing || lora_fits(m) ? 0 : (__float_as_int(m) >> 23) - 127 - 15;
}
__device__ __forceinline__ float lora_power(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127
// v of eight adjacent lanes, in a whole warp, as it stands in T, and its group's
// exponent.  What is finite stays so (65504 for up to 65536: 2^-11 of it).
struct LoraRounded {
  unsigned short y;
  int e;
};
__device__ __forceinline__ LoraRounded lora_round(float v) {
  const float inf = __int_as_float(0x7f800000);
  const bool finite = fabsf(v) < inf;
  float m = finite ? fabsf(v) : 0.0f;
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  LoraRounded r;
  r.e = lora_exponent(m);
  if (finite) v = m < kLoraNothing ? 0.0f : fminf(fmaxf(v * lora_power(-r.e), -65504.0f), 65504.0f);
  r.y = round_16(v, false);
  return r;
}
// Whether one of eight values of fp16 is 2^15 or more, or not finite.
__device__ __forceinline__ bool lora_powered(const uint4& w) {
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
  return m >= 0x78000000u || (m & 0xffffu) >= 0x7800u;
}

__device__ __forceinline__ int ld_s8(const signed char* p) {  // of any memory
  int v;
  asm volatile("ld.s8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
// Eight values of fp16 times 2^e, e <= 0.
__device__ __forceinline__ void lora_scale(uint4& w, int e) {
  const float f = lora_power(max(e, -126));
  uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = unpack_16(v[k], false);
    v[k] = pack_f16(x.x * f, x.y * f);
  }
  w = make_uint4(v[0], v[1], v[2], v[3]);
}
// The kind of 32 tokens, as the main product takes them: in one run only what fits the accumulator.
template <bool BF16>
__device__ __forceinline__ int lora_kind(const LoraParams& l, int block) {
  const int kind = ld_global_s32(l.kind + block);
  if (BF16) return kind;
  uint32_t any = 0u;
  for (int z = 0; z < l.deep; ++z) {
    uint2 u;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(u.x), "=r"(u.y) : "l"(l.misfits + static_cast<int64_t>(block) * l.deep + z));
    any |= u.x | u.y;
  }
  return kind >= 0 && any != 0u ? kLoraMixed : kind;
}

// Runs of 32-token groups of a tile that share an adapter, in order; for a whole
// warp, whose lanes hold the groups' kinds.
struct LoraRun {
  int first, count, adapter;
};
__device__ __forceinline__ bool lora_next_run(int kinds, int groups, LoraRun& run) {
  int i = run.first + run.count;
  int r = kLoraNone;
  while (i < groups && (r = __shfl_sync(0xffffffffu, kinds, i)) < 0) ++i;
  if (i >= groups) return false;
  run.first = i;
  run.adapter = r;
  while (++i < groups && __shfl_sync(0xffffffffu, kinds, i) == r) {
  }
  run.count = i - run.first;
  return true;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8) on the warp-level tensor cores.
template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if (BF16)
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

constexpr int kLoraTokens = 16;
// lora_part where T carries powers (fp16): of 32 ranks a token's four groups are brought
// to the largest power among them (those without a value have no say), and the fp32
// product of these ranks takes it.  Such values are rare, so this form goes over 16 columns
// and 8 tokens at a time and leaves the other's registers alone: all at once the two made
// the pair kernel spill (1049 rows of 40 requests 60-66 us, so 58).
__device__ __forceinline__ void lora_part_powers(const LoraParams& l, const void* T, const signed char* exps, int mine, int m0, int n0,
                                                 int N, float* out, int pitch, int lane) {
  const int row = lane >> 2, q = lane & 3;
#pragma unroll 1
  for (int part = 0; part < 4; ++part) {
    const int col = (part & 1) * 16, tok = (part >> 1) * 8;
    const int own = __shfl_sync(0xffffffffu, mine, tok + row);  // of this thread's row of T
    const int64_t m = m0 + tok + row;
    const unsigned short* t = static_cast<const unsigned short*>(T) + m * l.rank;
    const signed char* ex = exps + m * (l.rank >> 3);
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    unsigned left = __ballot_sync(0xffffffffu, lane >= tok && lane < tok + 8 && mine >= 0);
    while (left != 0) {
      const int adapter = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
      const unsigned mask = __ballot_sync(0xffffffffu, mine == adapter) & left;
      left &= ~mask;
      const unsigned short* b = static_cast<const unsigned short*>(l.b) + adapter * l.stride_b + (n0 + col + row) * l.ldb;
      float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
      for (int at = q * 8; at - q * 8 < l.rank; at += 32) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u, w = u;
        int top = -126;
        if (at < l.rank && n0 + col + row < N) u = __ldg(reinterpret_cast<const uint4*>(b + at));
        if (at < l.rank && n0 + col + row + 8 < N) v = __ldg(reinterpret_cast<const uint4*>(b + 8 * l.ldb + at));
        if (at < l.rank && own >= 0) {
          w = ld_v4(t + at);
          top = ld_s8(ex + (at >> 3));
        }
        if (((w.x | w.y | w.z | w.w) & 0x7fff7fffu) == 0u) top = -126;
        const int power = top;
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        lora_scale(w, power - top);
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma_16816<false>(s, u.x, v.x, u.y, v.y, w.x, w.y);
        mma_16816<false>(s, u.z, v.z, u.w, v.w, w.z, w.w);
        // Columns of the product are tokens 2 q and 2 q + 1.
        const float up0 = lora_power(__shfl_sync(0xffffffffu, top, 8 * q)), up1 = lora_power(__shfl_sync(0xffffffffu, top, 8 * q + 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = fmaf(s[e], e & 1 ? up1 : up0, p[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (mask >> (tok + 2 * q + (e & 1)) & 1u) d[e] = p[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) out[(col + 8 * (e >> 1) + row) * pitch + tok + 2 * q + (e & 1)] = d[e];
  }
  __syncwarp();
}

// The adapters' part of 32 columns from n0 on and 16 tokens from m0 on, by a warp
// whose lane t < 16 holds token t's adapter (negative: none): sum_j B_a[n][j] T[m][j]
// in fp32 to out[column * pitch + token].
//
// For each adapter among the tokens the warp multiplies its 32 rows of B by all 16
// rows of T and keeps the columns of its own tokens: columns of a product do not
// depend on each other, so nothing of one adapter reaches another's tokens.
// Within 32 ranks a thread's fragments are 8 adjacent ones (the order of the sum
// is free), so all loads are 16 bytes, and rows are read 64 bytes at a time; 32 ranks
// of ITEMS adapters, or 32 ITEMS of one, are in flight together.  As many as the
// registers hold: beside 220 KiB of shared memory a spill goes to L2 and back.  The
// pair kernel takes 3 (7414 mixed rows, 1110 x 880, rank 112: 81 us, 2 take 79, 4
// take 90; 8192 rows of 8 requests, 8192 x 4096, rank 64: 422, 436, 450), the narrow one 4.  (A
// thread a column, with fused multiply-adds, read each row in pieces of its own: 3000
// cycles for 16 ranks of 8 tokens.)
template <bool BF16, int ITEMS>
__device__ __forceinline__ void lora_part(const LoraParams& l, const void* T, const signed char* exps, int mine, int m0, int n0, int N,
                                          float* out, int pitch, int lane) {
  const int row = lane >> 2, q = lane & 3;
  const unsigned tokens = __ballot_sync(0xffffffffu, lane < kLoraTokens && mine >= 0);
  const int steps = (l.rank + 31) >> 5;
  const unsigned short* t = static_cast<const unsigned short*>(T) + static_cast<int64_t>(m0 + row) * l.rank + q * 8;
  const unsigned short* b = static_cast<const unsigned short*>(l.b) + (n0 + row) * l.ldb + q * 8;
  float d[2][2][4], p[2][2][4];  // [16 columns][8 tokens]: the results, and the adapter's at hand
#pragma unroll
  for (int i = 0; i < 16; ++i) d[i >> 3][i >> 2 & 1][i & 3] = 0.0f;
  unsigned left = tokens, mask = 0;
  int adapter = -1, step = steps;
  while (left != 0 || step < steps) {
    int at[ITEMS];         // first rank, negative: nothing
    unsigned done[ITEMS];  // the tokens that take the sum after it
    uint4 x[ITEMS][4], y[ITEMS][2];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (step == steps && left != 0) {
        adapter = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
        mask = __ballot_sync(0xffffffffu, mine == adapter) & tokens;
        left &= ~mask;
        step = 0;
      }
      at[i] = step < steps ? step * 32 : -1;
      step = min(step + 1, steps);
      done[i] = step == steps ? mask : 0u;
      const bool in = at[i] >= 0 && at[i] + q * 8 < l.rank;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[i][r] = make_uint4(0u, 0u, 0u, 0u);
        if (in && n0 + row + 8 * r < N)
          x[i][r] = __ldg(reinterpret_cast<const uint4*>(b + adapter * l.stride_b + 8 * r * l.ldb + at[i]));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        y[i][h] = make_uint4(0u, 0u, 0u, 0u);
        if (in && (tokens >> (row + 8 * h) & 1u)) y[i][h] = ld_v4(t + 8 * h * l.rank + at[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (at[i] < 0) break;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (at[i] == 0)
#pragma unroll
            for (int e = 0; e < 4; ++e) p[c][h][e] = 0.0f;
          const uint4 &u = x[i][2 * c], &v = x[i][2 * c + 1], &w = y[i][h];
          mma_16816<BF16>(p[c][h], u.x, v.x, u.y, v.y, w.x, w.y);
          mma_16816<BF16>(p[c][h], u.z, v.z, u.w, v.w, w.z, w.w);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (done[i] >> (8 * h + 2 * q + (e & 1)) & 1u) d[c][h][e] = p[c][h][e];
        }
    }
  }
  if (!BF16) {  // T's rows again, which L1 holds by now (looked at in the loop: 64 rows of 64 requests 45.8 us, so 44.2)
    bool powered = false;
    for (int at = q * 8; at < l.rank; at += 32) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (tokens >> (row + 8 * h) & 1u) powered |= lora_powered(ld_v4(t + 8 * h * l.rank + at - q * 8));
    }
    if (__any_sync(0xffffffffu, powered)) {
      lora_part_powers(l, T, exps, mine, m0, n0, N, out, pitch, lane);
      return;
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) out[(16 * c + 8 * (e >> 1) + row) * pitch + 8 * h + 2 * q + (e & 1)] = d[c][h][e];
  __syncwarp();
}

// A token's adapter, or -1.
__device__ __forceinline__ int lora_adapter(const LoraParams& l, int m) {
  const int a = __ldg(l.index + m);
  return a >= 0 && a < l.adapters ? a : -1;
}

// A warp's adapters' part: [32 columns][16 tokens + 1].
constexpr int kPartPitch = kLoraTokens + 1;
constexpr int kPartBytes = 32 * kPartPitch * 4;

struct GrpPairCfg {
  static constexpr int STAGES = 6;                 // of the widest tiles; more of narrower ones
  static constexpr int MAX_STAGES = 8;
  static constexpr int BM = 128;                   // weight rows of a CTA
  static constexpr int PAIR_M = 256;
  static constexpr int TOKENS = 256;               // most of a tile
  static constexpr int UNIT = 32;                  // its width is a multiple of
  static constexpr int WIDTHS = 6;                 // 256, 224, .. 96 tokens to choose from
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = TOKENS / 2 * 128;
  static constexpr int PANEL_BYTES = 64 * 128;
  static constexpr int MMA_WARP = 1;
  static constexpr int EPI_WARP0 = 2;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
  static constexpr int TMEM_COLS = 512;
  static constexpr int STAGING = EPI_WARPS * kGrpBoxBytes;
  static constexpr int BAR_BYTES = 256;
  static constexpr int FIXED_SMEM = 1024 + STAGES * (A_BYTES + B_BYTES) + STAGING + BAR_BYTES;
  static constexpr int smem_bytes(int groups, bool lora) {
    return FIXED_SMEM + (lora ? grp_plan_align(1) + EPI_WARPS * kPartBytes : grp_plan_align(groups));
  }
  static_assert(FIXED_SMEM + (kGrpMaxGroups + 4) * 8 + WIDTHS * 4 <= 232448 &&
                    FIXED_SMEM + 32 + EPI_WARPS * kPartBytes + WIDTHS * 4 <= 232448, "dynamic shared memory per CTA");
  static_assert((2 * MAX_STAGES + 5) * 8 + 8 <= BAR_BYTES, "barriers");
  static_assert(A_BYTES % 1024 == 0 && PANEL_BYTES % 1024 == 0 && B_BYTES % 1024 == 0 && UNIT / 2 * 128 % 1024 == 0,
                "operand tiles, and the pieces of rows they are loaded in, start on the swizzle's 1024 bytes");
};

// `rows` rows of tokens (a multiple of 16, at most 128) as the boxes of its binary digits.
template <typename Load>
__device__ __forceinline__ void grp_token_boxes(int rows, Load&& load) {
  int at = 0;
#pragma unroll
  for (int b = 3; b >= 0; --b) {
    const int box = 16 << b;
    if (rows & box) {
      load(b, at);
      at += box;
    }
  }
}

// LORA: 0 for groups, else the adapters' type: 1 fp16, 2 bf16.
template <int LORA>
__global__ void __launch_bounds__(GrpPairCfg::THREADS, 1)
    grp_pair_kernel(const __grid_constant__ GrpMaps maps, const GrpParams p) {
  using Cfg = GrpPairCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + Cfg::STAGES * (Cfg::A_BYTES + Cfg::B_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + Cfg::STAGING);
  uint64_t* full_bar = bars;                            // used in the even CTA
  uint64_t* empty_bar = bars + Cfg::MAX_STAGES;         // per CTA
  uint64_t* acc_full_bar = bars + 2 * Cfg::MAX_STAGES;  // per CTA
  uint64_t* acc_empty_bar = acc_full_bar + 2;       // used in the even CTA
  uint64_t* mma_done_bar = acc_empty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ int costs[Cfg::WIDTHS];
  GrpPlan plan;
  plan.lo = reinterpret_cast<int*>(staging + Cfg::STAGING + Cfg::BAR_BYTES);
  plan.first = plan.lo + p.groups + 2;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1;
  const int num_clusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::MAX_STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full_bar[b], 1);
      mbar_init(&acc_empty_bar[b], 2 * Cfg::EPI_WARPS);
    }
    mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&maps.w);
    for (int b = 0; b < 4; ++b) tma_prefetch_desc(&maps.x[b]);
  }
  if (warp == Cfg::MMA_WARP) {
    tmem_alloc_pair(tmem_slot, Cfg::TMEM_COLS);
    tmem_relinquish_alloc_permit_pair();
  }
  tcgen05_fence_before_sync();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised before any remote use
  tcgen05_fence_after_sync();
  // Adapters: the kernel before this one on the stream makes T.  It waited for
  // what came before it and then let this one start, so X, W, index and the
  // workspace's copies are there already; only T and kind are waited for, by
  // the threads that read them.
  const bool early = LORA != 0 && p.lora.adapters > 0;
  // Gradients: the kernel before this one makes dW from the same dY.  It too waited
  // for what came before it, so dX is computed beside its last tiles; only the end of
  // this kernel waits for it, for those who wait for this one (see the end).
  const bool beside = LORA == 0 && p.beside != 0;
  if (!early) {
    if (!beside) grid_dependency_wait();
    grid_launch_dependents();
  }
  // Tokens of a tile.  Few tiles leave pairs idle in the last wave, so the width is
  // chosen by the number of waves that it gives, at a tile's time of (256 + width):
  // its MMAs take 2 width cycles a k-block, its loads 128 (128 + width / 2) bytes at
  // about 50 a cycle.
  if (p.adapt && warp >= Cfg::EPI_WARP0 && warp < Cfg::EPI_WARP0 + Cfg::WIDTHS) {
    const int width = Cfg::TOKENS - 32 * (warp - Cfg::EPI_WARP0);
    int tiles = 0;
    for (int g = lane; g < p.groups; g += 32) {
      const int rows = grp_end(p.ends, g, p.M) - grp_end(p.ends, g - 1, p.M);
      if (rows > 0) tiles += (rows + width - 1) / width;
    }
    tiles = __reduce_add_sync(0xffffffffu, tiles) * p.col_tiles;
    if (lane == 0) costs[warp - Cfg::EPI_WARP0] = (tiles + num_clusters - 1) / num_clusters * (Cfg::TOKENS + width);
  }
  if (p.adapt) __syncthreads();
  int most = Cfg::TOKENS;
  if (p.adapt) {
    int best = costs[0];
#pragma unroll
    for (int i = 1; i < Cfg::WIDTHS; ++i)
      if (costs[i] < best) {
        best = costs[i];
        most = Cfg::TOKENS - 32 * i;
      }
    most = uniform(most);
  }
  // The ring: as many stages of `most` tokens as there is room for.  (Adapters' k-blocks fit too: 16 rows of 32 tokens each.)
  const int b_bytes = most / 2 * 128;
  const int stages = min(Cfg::MAX_STAGES, Cfg::STAGES * (Cfg::A_BYTES + Cfg::B_BYTES) / (Cfg::A_BYTES + b_bytes));
  uint8_t* a_smem = smem;
  uint8_t* b_smem = smem + stages * Cfg::A_BYTES;
  if (warp == Cfg::EPI_WARP0)
    grp_make_plan(plan, p.ends, p.groups, p.M, most, p.col_tiles, p.rest != 0, lane);
  __syncthreads();
  const uint32_t tmem_base = *tmem_slot;
  const int num_tiles = plan.first[p.groups + 1];

  if (warp == 0) {
    // Producer (both CTAs): this CTA's half of the weight's rows and of the
    // tokens.  The loop is the warp's, so that addresses and coordinates are in
    // uniform registers where the TMA and MMA instructions want them; one lane
    // issues.
    const bool one = elect_one();
    int stage = 0;
    uint32_t phase = 0, used = 0, parities = 0;
    bool ok = true, waited = false;
    const uint64_t pol = l2_policy_evict_normal();
    const uint32_t full_even0 = mapa_shared(smem_u32(full_bar), 0);
    GrpWalk walk;
    auto next = [&]() {
      used |= 1u << stage;
      parities = (parities & ~(1u << stage)) | phase << stage;
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    };
    for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
      const GrpTile f = walk.at(plan, t, p.col_tiles, p.super, most, Cfg::UNIT);
      if (f.g == p.groups) break;  // zeros from here on
      const int width = (f.cnt + Cfg::UNIT - 1) / Cfg::UNIT * Cfg::UNIT;
      const int rows = width / 2;
      const int tok = f.tok0 + static_cast<int>(rank) * rows;
      const int n0 = f.col_blk * Cfg::PAIR_M + static_cast<int>(rank) * Cfg::BM;
      const uint32_t tx = 2 * (Cfg::A_BYTES + rows * 128);
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        if (!mbar_wait_warp(&empty_bar[stage], phase ^ 1u, abort_flag, p.wait_budget_ns, 0xa1)) {
          ok = false;
          break;
        }
        if (one) {
          const uint32_t full = full_even0 + stage * 8;
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], tx);
          const int k0 = kb * 64;
          uint8_t* adst = a_smem + stage * Cfg::A_BYTES;
          uint8_t* bdst = b_smem + stage * b_bytes;
          if (p.w_mn) {
            tma_load_3d_pair_hint(adst, &maps.w, full, n0, k0, f.g, pol);
            tma_load_3d_pair_hint(adst + Cfg::PANEL_BYTES, &maps.w, full, n0 + 64, k0, f.g, pol);
          } else {
            tma_load_3d_pair_hint(adst, &maps.w, full, k0, n0, f.g, pol);
          }
          grp_token_boxes(rows, [&](int b, int at) {
            tma_load_2d_pair_hint(bdst + at * 128, &maps.x[b], full, k0, tok + at, pol);
          });
        }
        next();
      }
      if (early && ok) {
        if (!waited) grid_dependency_wait();
        waited = true;
        LoraRun run{0, 0, 0};
        const int kinds = lane < width / 32 ? lora_kind<LORA == 2>(p.lora, f.tok0 / 32 + lane) : kLoraNone;
        while (ok && lora_next_run(kinds, width / 32, run)) {
          for (int j0 = 0; j0 < p.lora.rank; j0 += 64) {
            if (!mbar_wait_warp(&empty_bar[stage], phase ^ 1u, abort_flag, p.wait_budget_ns, 0xa1)) {
              ok = false;
              break;
            }
            if (one) {
              const uint32_t full = full_even0 + stage * 8;
              if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * (Cfg::A_BYTES + run.count * 2048));
              tma_load_3d_pair_hint(a_smem + stage * Cfg::A_BYTES, &maps.lb, full, j0, n0, run.adapter, pol);
              // 16 of each 32 tokens, where an MMA of 32 columns wants them.
              for (int i = 0; i < run.count; ++i)
                tma_load_2d_pair_hint(b_smem + stage * b_bytes + i * 2048, &maps.lt, full, j0,
                                      f.tok0 + (run.first + i) * 32 + static_cast<int>(rank) * 16, pol);
            }
            next();
          }
        }
      }
    }
    // The even CTA's full barriers count both CTAs' bytes: once they have
    // completed, every load of the pair has landed.
    if (leader) {
      for (int s = 0; s < stages; ++s) {
        if (used >> s & 1u) {
          volatile int no_abort = 0;
          mbar_wait(&full_bar[s], parities >> s & 1u, &no_abort, p.wait_budget_ns, 0xa2);
        }
      }
    }
  } else if (warp == Cfg::MMA_WARP) {
    // MMA issuer (even CTA only).
    if (leader) {
      const bool one = elect_one();
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;
      bool ok = true, waited = false;
      // Descriptors of stage 0 and their steps in units of 16 bytes.
      const uint64_t a_desc0 = make_sw128_desc(smem_u32(a_smem), p.w_mn ? Cfg::PANEL_BYTES : 16, 1024);
      const uint64_t lb_desc0 = make_sw128_desc(smem_u32(a_smem), 16, 1024);
      const uint64_t b_desc0 = make_sw128_desc(smem_u32(b_smem), 16, 1024);
      const uint32_t a_step = p.w_mn ? 2048 / 16 : 32 / 16;
      const uint32_t tmem = uniform(tmem_base);
      GrpWalk walk;
      auto next = [&]() {
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      };
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters, ++local) {
        const GrpTile f = walk.at(plan, t, p.col_tiles, p.super, most, Cfg::UNIT);
        if (f.g == p.groups) break;
        const int width = (f.cnt + Cfg::UNIT - 1) / Cfg::UNIT * Cfg::UNIT;
        const uint32_t idesc = p.idesc | static_cast<uint32_t>(width >> 3) << 17;
        const int acc = local & 1;
        if (!mbar_wait_warp(&acc_empty_bar[acc], ((local >> 1) & 1) ^ 1u, abort_flag, p.wait_budget_ns, 0xa3)) break;
        tcgen05_fence_after_sync();
        const uint32_t d_tmem = tmem + acc * Cfg::TOKENS;
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait_warp(&full_bar[stage], phase, abort_flag, p.wait_budget_ns, 0xa4)) {
            ok = false;
            break;
          }
          tcgen05_fence_after_sync();
          const uint64_t a_desc = a_desc0 + stage * (Cfg::A_BYTES / 16), b_desc = b_desc0 + stage * (b_bytes / 16);
          if (one) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f16_ss_pair(d_tmem, a_desc + k * a_step, b_desc + k * 2, idesc, (kb | k) != 0 ? 1u : 0u);
            umma_commit_pair_mc(&empty_bar[stage], 0x3);  // both CTAs may refill this stage
          }
          next();
        }
        if (early && ok) {
          if (!waited) grid_dependency_wait();
          waited = true;
          const uint32_t idesc32 = p.idesc | (32u >> 3) << 17;
          LoraRun run{0, 0, 0};
          const int kinds = lane < width / 32 ? lora_kind<LORA == 2>(p.lora, f.tok0 / 32 + lane) : kLoraNone;
          while (ok && lora_next_run(kinds, width / 32, run)) {
            for (int j0 = 0; j0 < p.lora.rank; j0 += 64) {
              if (!mbar_wait_warp(&full_bar[stage], phase, abort_flag, p.wait_budget_ns, 0xa4)) {
                ok = false;
                break;
              }
              tcgen05_fence_after_sync();
              const int steps = (min(p.lora.rank - j0, 64) + 15) / 16;
              const uint64_t a_desc = lb_desc0 + stage * (Cfg::A_BYTES / 16);
              if (one) {
                for (int i = 0; i < run.count; ++i) {
                  const uint64_t b_desc = b_desc0 + stage * (b_bytes / 16) + i * (2048 / 16);
                  for (int k = 0; k < steps; ++k)
                    umma_f16_ss_pair(d_tmem + (run.first + i) * 32, a_desc + k * 2, b_desc + k * 2, idesc32, 1u);
                }
                umma_commit_pair_mc(&empty_bar[stage], 0x3);
              }
              next();
            }
          }
        }
        if (!ok) break;
        if (one) umma_commit_pair_mc(&acc_full_bar[acc], 0x3);
      }
      if (one) umma_commit_pair_mc(mma_done_bar, 0x1);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(mma_done_bar, 0, &no_abort, p.wait_budget_ns, 0xa5);
    }
    __syncwarp();
  } else {
    // Epilogue (both CTAs): warp w takes TMEM lanes 32 (w mod 4) .. + 31, which
    // are columns of the result, and every other 32 tokens.
    if (early) {
      grid_dependency_wait();
      grid_launch_dependents();
    }
    const int quad = warp & 3;
    constexpr int PARTS = Cfg::EPI_WARPS / 4;
    const int part = (warp - Cfg::EPI_WARP0) >> 2;
    uint8_t* box = staging + (warp - Cfg::EPI_WARP0) * kGrpBoxBytes;
    float* part_buf = reinterpret_cast<float*>(staging + Cfg::STAGING + Cfg::BAR_BYTES + grp_plan_align(p.groups) +
                                               (warp - Cfg::EPI_WARP0) * kPartBytes);  // adapters only
    constexpr bool BF16 = LORA == 2;
    const bool bf16 = LORA ? BF16 : p.bf16 != 0;
    GrpWalk walk;
    int local = 0;
    for (int t = cluster_id; t < num_tiles; t += num_clusters) {
      const GrpTile f = walk.at(plan, t, p.col_tiles, p.super, most, Cfg::UNIT);
      const int n0 = f.col_blk * Cfg::PAIR_M + static_cast<int>(rank) * Cfg::BM + quad * 32;
      const bool zero = f.g == p.groups;
      const int acc = local & 1;
      if (early) {
        // The rows of B that the epilogue will read come into L2 while the tile is computed.
        for (int b = 0; b * 32 < f.cnt && n0 < p.out; ++b) {
          const int mine = b * 32 + lane < f.cnt ? lora_adapter(p.lora, f.tok0 + b * 32 + lane) : -1;
          const int first = __shfl_sync(0xffffffffu, mine, 0);
          if (__all_sync(0xffffffffu, mine == first || b * 32 + lane >= f.cnt)) continue;
          for (int e = part * (32 / PARTS); e < (part + 1) * (32 / PARTS); ++e) {
            const int a = __shfl_sync(0xffffffffu, mine, e);
            if (a < 0 || n0 + lane >= p.out) continue;
            const unsigned short* row = static_cast<const unsigned short*>(p.lora.b) + a * p.lora.stride_b + (n0 + lane) * p.lora.ldb;
            for (int at = 0; at < p.lora.rank; at += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + at));
          }
        }
        __syncwarp();
      }
      if (!zero) {
        bool ready = mbar_wait_warp(&acc_full_bar[acc], (local >> 1) & 1, abort_flag, p.wait_budget_ns, 0xa6);
        // The four warps that stage rows together go on or give up together.
        if (!p.vec) ready = bar_all_128(1 + part, ready);
        if (!ready) break;
        tcgen05_fence_after_sync();
      }
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * Cfg::TOKENS;
      const int boxes = (f.cnt + 31) / 32;
      const int cta_n0 = f.col_blk * Cfg::PAIR_M + static_cast<int>(rank) * Cfg::BM;
      const int n = n0 + lane, cols = p.vec ? min(32, p.out - n0) : min(Cfg::BM, p.out - cta_n0);  // of a warp, or of four
      const float bias = LORA && p.lora.bias != nullptr && n < p.out
                             ? load_16(static_cast<const unsigned short*>(p.lora.bias) + n, bf16) : 0.0f;
      unsigned mixed_boxes = 0;
      if (early)
        mixed_boxes = __ballot_sync(
            0xffffffffu, (lane < boxes ? lora_kind<BF16>(p.lora, f.tok0 / 32 + lane) : kLoraNone) == kLoraMixed);
      for (int b = 0; b < boxes && cols > 0; ++b) {
        const bool mixed = mixed_boxes >> b & 1u;
        if (!mixed && b % PARTS != part) continue;
        // A mixed box is shared: 16 tokens for each of the two warps that have these columns.
        const int e0 = mixed ? part * (32 / PARTS) : 0;
        const int rows = min(mixed ? 32 / PARTS : 32, f.cnt - b * 32 - e0);
        unsigned short* c = static_cast<unsigned short*>(p.c) + static_cast<int64_t>(f.tok0 + b * 32 + e0) * p.ldc;
        // This lane's column of row e into staging: a box of the warp's own, or (rows
        // off 16 bytes) a row of four warps.
        uint8_t* mine_at = p.vec ? box + (lane & 7) * 2 : staging + part * 4 * kGrpBoxBytes + quad * 64 + lane * 2;
        auto put = [&](int e, float y) {
          *reinterpret_cast<unsigned short*>(mine_at + (p.vec ? grp_box_at(e, lane >> 3) : e * 256)) =
              round_16(LORA ? y + bias : y, bf16);
        };
        if (p.vec)
          __syncwarp();  // the box before has left
        else
          bar_128(1 + part);
        if (mixed) {
          const int mine = lane < rows ? lora_adapter(p.lora, f.tok0 + b * 32 + e0 + lane) : -1;
          lora_part<BF16, 3>(p.lora, p.lora.t, p.lora.exps, mine, f.tok0 + b * 32 + e0, n0, p.out, part_buf, kPartPitch, lane);
          uint32_t r[16];
          tmem_ld_32x32b_x16(taddr + b * 32 + e0, r);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < kLoraTokens; ++e) put(e, __uint_as_float(r[e]) + part_buf[lane * kPartPitch + e]);
          __syncwarp();  // read, before the next box's
        } else {
          uint32_t r[32];
          if (!zero) {
            tmem_ld_32x32b_x32(taddr + b * 32, r);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0u;
          }
          if (p.vec) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              *reinterpret_cast<unsigned short*>(mine_at + grp_box_at(e, lane >> 3)) =
                  round_16(LORA ? __uint_as_float(r[e]) + bias : __uint_as_float(r[e]), bf16);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              *reinterpret_cast<unsigned short*>(mine_at + e * 256) =
                  round_16(LORA ? __uint_as_float(r[e]) + bias : __uint_as_float(r[e]), bf16);
          }
        }
        if (p.vec) {
          __syncwarp();
          grp_store_box(c + n0, p.ldc, rows, cols, box, lane);
        } else {
          bar_128(1 + part);
          grp_store_rows(c + cta_n0, p.ldc, rows, cols, staging + part * 4 * kGrpBoxBytes, quad * 32 + lane);
        }
      }
      if (!zero) {
        tcgen05_fence_before_sync();
        __syncwarp();
        // Relaxed, as in the feed-forward pair kernel: it orders only TMEM reads.
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acc_empty_bar[acc]), 0));
        ++local;
      }
    }
  }

  if (beside) grid_dependency_wait();
  tcgen05_fence_before_sync();
  __syncthreads();
  cluster_sync();  // the pair is done with each other's shared memory and barriers
  if (warp == Cfg::MMA_WARP) {
    tcgen05_fence_after_sync();
    tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
  }
}

}  // namespace tg
