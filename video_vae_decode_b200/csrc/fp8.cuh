// fp8.cuh -- linear layers in 8-bit floating point (e4m3) with one scale for
// each block of 128, single or grouped by expert, on the sm_100a tensor cores
// (tcgen05 kind::mxf8f6f4 with E8M0 block scales, fp32 accumulators in TMEM).
//
// Scheme.  A group is 128 consecutive input channels of one row (activations)
// or 128 output x 128 input channels (weights).  With amax the largest |v| of
// the group,
//   e = the least integer >= -126 with amax <= 448 * 2^e,
//   code = e4m3_rne(v * 2^-e),  scale byte (E8M0) = e + 127,
//   out[m,n] = bf16_rne( sum_kb 2^(ex[m,kb] + ew[n/128,kb]) sum_{k in kb} cx[m,k] cw[n,k] + bias[n] ).
// e4m3 is a floating-point format, so its relative precision does not depend
// on the scale; a power of two keeps the scaling exact and is what the tensor
// cores apply by themselves while they accumulate: no partial sum is rescaled
// outside them.  A group with an infinity or a NaN gets scale byte 255 (NaN)
// and NaN codes, so that the outputs it reaches are NaN.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "conv.cuh"
#include "ptx.cuh"

namespace qvae {

constexpr int kFp8Block = 128;  // channels (and, for weights, rows) of a scale block

// ------------------------------------------------------------------ scales

// E8M0 byte of the least power of two 2^e, e >= -126, with amax <= 448 * 2^e,
// from the bits of amax >= 0: 448 = 1.75 * 2^8, so e is the exponent of amax
// less 8, and one more where its mantissa is above 1.75.  255 (NaN) for an
// infinity or a NaN.
__device__ __forceinline__ uint32_t e8m0_of_amax(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const int p = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(p, 1));
}

// 2^-e of a scale byte e + 127 (e in -126..120: a normal number); NaN for 255.
__device__ __forceinline__ float e8m0_reciprocal(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - byte) << 23);
}

// Two values -> two e4m3 codes (the first in the low byte), round half to even; NaN -> 0x7F.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

// Eight values times a power of two -> eight codes.
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float inv) {
  return make_uint2(e4m3x2(v[0] * inv, v[1] * inv) | (e4m3x2(v[2] * inv, v[3] * inv) << 16),
                    e4m3x2(v[4] * inv, v[5] * inv) | (e4m3x2(v[6] * inv, v[7] * inv) << 16));
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Eight bf16 values x[k .. k+8) of a row of K, zeros beyond K.  kVec: the row
// starts on a 16-byte boundary and k is a multiple of 8.
template <bool kVec>
__device__ __forceinline__ uint4 load_bf16x8(const uint16_t* row, int64_t k, int64_t K) {
  if (kVec && k + 8 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = k + 2 * i < K ? __ldg(row + k + 2 * i) : 0u;
    const uint32_t hi = k + 2 * i + 1 < K ? __ldg(row + k + 2 * i + 1) : 0u;
    u[i] = lo | (hi << 16);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Sixteen of them, of rows that start anywhere: the three aligned 16-byte
// pieces around them, shifted into place.  Where one of the pieces reaches out
// of the tensor [first, end), or the values end, one by one.  (One by one
// throughout, 8192 rows of 4095 took 42 us instead of 22.)
__device__ __forceinline__ void load_bf16x16_anywhere(const uint16_t* row, int64_t k, int64_t K, const uint16_t* first,
                                                      const uint16_t* end, uint4 (&w)[2]) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + k), base = at & ~uintptr_t{15};
  if (k + 16 <= K && base >= reinterpret_cast<uintptr_t>(first) && base + 48 <= reinterpret_cast<uintptr_t>(end)) {
    const uint4* const p = reinterpret_cast<const uint4*>(base);
    const uint4 a = __ldg(p), b = __ldg(p + 1), c = __ldg(p + 2);
    uint32_t u[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
    const uint32_t shift = static_cast<uint32_t>(at - base) >> 1;  // values
    if (shift & 2) {
#pragma unroll
      for (int i = 0; i < 11; ++i) u[i] = u[i + 1];
    }
    if (shift & 4) {
#pragma unroll
      for (int i = 0; i < 9; ++i) u[i] = u[i + 2];
    }
    if (shift & 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = __funnelshift_r(u[i], u[i + 1], 16);
    }
    w[0] = make_uint4(u[0], u[1], u[2], u[3]);
    w[1] = make_uint4(u[4], u[5], u[6], u[7]);
  } else {
    w[0] = load_bf16x8<false>(row, k, K);
    w[1] = load_bf16x8<false>(row, k + 8, K);
  }
}

__device__ __forceinline__ void widen_bf16x8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// Bits (as fp32) of the largest magnitude of eight bf16 values.
__device__ __forceinline__ uint32_t abs_max_bf16x8(const uint4& w) {
  const uint32_t m = abs_bits_max2x(abs_bits_max2x(abs_bits_max2x(abs_bits_max2x(0u, w.x), w.y), w.z), w.w);
  return max(m << 16, m & 0xFFFF0000u);
}

// silu(g) * u = g / (1 + exp(-g)) * u in fp32 with the hardware's exponential
// and reciprocal: off by about |g| * 2^-23 of its value, far below the 2^-4 of
// the code it ends in (an IEEE divide made the quantiser issue-bound: 39 us
// instead of 29 for 8192 rows of 4096).  Computed as g / 4 over a quarter of
// 1 + exp(-g), both exact: the reciprocal of the whole sum would be below
// fp32's normal numbers, and flushed to 0, from g = -87.3 on down to -88.7,
// where exp(-g) leaves fp32 and the formula gives 0.  (Flushing a quarter of
// exp(-g) itself changes nothing beside 1 / 4, and saves the instructions that
// an exponential with subnormal results takes.)
__device__ __forceinline__ float silu_mul(float g, float u) {
  float t, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(g, -1.44269504f, -2.0f)));  // 2^(-g log2(e) - 2)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t + 0.25f));
  return 0.25f * g * r * u;
}

// --------------------------------------------------------------- quantiser

constexpr int kFp8QuantThreads = 256;
// Rows of a warp: 64 bytes of loads in flight a lane (silu takes two values an
// element).  Twice as many measured 17.4 instead of 16.1 us for 8192 rows of
// 4096, and 2.0 instead of 1.6 us for one row.
template <bool kSilu>
constexpr int kFp8RowsPerWarp = kSilu ? 1 : 2;
template <bool kSilu>
constexpr int kFp8RowsPerBlock = kFp8QuantThreads / 32 * kFp8RowsPerWarp<kSilu>;

// Activations: codes [Kb][M][128] (zeros beyond K) and scale words
// [ceil(Kb / 4)][M], byte j of word (g, m) being the scale of row m's block
// 4 g + j.  Blocks beyond Kb get byte 1.  kSilu: rows are [gate | up], K each,
// and what is quantised is silu(gate) * up.
//
// A warp takes a few rows of one group of four blocks (512 channels), 16
// channels to a lane: eight lanes hold a block and the maximum takes three
// shuffles.  Blocks of the grid walk along the rows first, so that what runs at
// one time reads whole rows.  One pass over x, bound by its bytes.
template <bool kSilu, bool kVec>
__global__ void __launch_bounds__(kFp8QuantThreads)
    fp8_quant_act_kernel(const uint16_t* __restrict__ x, int64_t ldx, int M, int K, int Kb, uint8_t* __restrict__ xq,
                         uint32_t* __restrict__ x_scale) {
  const uint16_t* const x_end = x + (M - 1) * ldx + (kSilu ? 2 : 1) * static_cast<int64_t>(K);
  constexpr int kRows = kFp8RowsPerWarp<kSilu>;
  grid_dependency_wait();
  // only now: a kernel behind this one may rely on all that came before this one
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kgroups = (Kb + 3) / 4;
  const int kg = blockIdx.x % kgroups;
  const int kb = kg * 4 + (lane >> 3), col = (lane & 7) * 16;
  const int64_t k = static_cast<int64_t>(kb) * kFp8Block + col;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / kgroups) * kFp8RowsPerBlock<kSilu> + warp * kRows;
  uint4 w[kRows][2], u[kSilu ? kRows : 1][2];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const uint16_t* row = x + (row0 + r) * ldx;
    if (kVec) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool in = row0 + r < M && k + 8 * i < K;
        w[r][i] = in ? load_bf16x8<kVec>(row, k + 8 * i, K) : make_uint4(0u, 0u, 0u, 0u);
        if (kSilu) u[r][i] = in ? load_bf16x8<kVec>(row + K, k + 8 * i, K) : make_uint4(0u, 0u, 0u, 0u);
      }
    } else {
      w[r][0] = w[r][1] = make_uint4(0u, 0u, 0u, 0u);
      if (kSilu) u[r][0] = u[r][1] = make_uint4(0u, 0u, 0u, 0u);
      if (row0 + r < M && k < K) {
        load_bf16x16_anywhere(row, k, K, x, x_end, w[r]);
        if (kSilu) load_bf16x16_anywhere(row + K, k, K, x, x_end, u[r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float v[2][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      widen_bf16x8(w[r][i], v[i]);
      if (kSilu) {  // (zeros beyond K stay zeros)
        float up[8];
        widen_bf16x8(u[r][i], up);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] = silu_mul(v[i][j], up[j]);
          m = max(m, abs_bits(v[i][j]));
        }
      } else {
        m = max(m, abs_max_bf16x8(w[r][i]));
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const uint32_t byte = e8m0_of_amax(m);
    const float inv = e8m0_reciprocal(byte);
    const uint2 lo = e4m3x8(v[0], inv), hi = e4m3x8(v[1], inv);
    if (row0 + r < M && kb < Kb)
      *reinterpret_cast<uint4*>(xq + (static_cast<int64_t>(kb) * M + row0 + r) * kFp8Block + col) =
          make_uint4(lo.x, lo.y, hi.x, hi.y);
    const uint32_t two = byte | (__shfl_down_sync(0xFFFFFFFFu, byte, 8) << 8);
    const uint32_t four = two | (__shfl_down_sync(0xFFFFFFFFu, two, 16) << 16);
    if (lane == 0 && row0 + r < M) x_scale[static_cast<int64_t>(kg) * M + row0 + r] = four;
  }
}

// ----------------------------------------------------------------- weights

constexpr int kFp8PackThreads = 256;

// One block per 128 x 128 weight block of w [E][N][K]: its scale byte and its
// codes in the product's order, [e][n / 128][k / 128] tiles of 128 rows x 128
// bytes in the tensor cores' 128-byte swizzle (16-byte group g of row r at
// position g ^ (r % 8)), zeros beyond N and K.  Scale bytes [e][n / 128][4
// ceil(Kb / 4)], bytes beyond Kb set to 1.
template <bool kVec>
__global__ void __launch_bounds__(kFp8PackThreads)
    fp8_pack_weights_kernel(const uint16_t* __restrict__ w, int N, int K, int nblk, int Kb,
                            uint8_t* __restrict__ packed, uint8_t* __restrict__ w_scale) {
  __shared__ uint32_t red[kFp8PackThreads / 32];
  const int64_t tile = blockIdx.x;
  const int kb = static_cast<int>(tile % Kb);
  const int64_t enb = tile / Kb;
  const int nb = static_cast<int>(enb % nblk);
  const int64_t e = enb / nblk;
  const int col = (threadIdx.x & 15) * 8, r0 = threadIdx.x >> 4;
  const int64_t k = static_cast<int64_t>(kb) * kFp8Block + col;
  uint4 v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = static_cast<int64_t>(nb) * kFp8Block + r0 + 16 * i;
    v[i] = n < N && k < K ? load_bf16x8<kVec>(w + (e * N + n) * K, k, K) : make_uint4(0u, 0u, 0u, 0u);
    m = max(m, abs_max_bf16x8(v[i]));
  }
  m = block_max_u32<kFp8PackThreads>(m, red);
  const uint32_t byte = e8m0_of_amax(m);
  const float inv = e8m0_reciprocal(byte);
  uint8_t* const dst = packed + tile * (kFp8Block * kFp8Block);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    float f[8];
    widen_bf16x8(v[i], f);
    *reinterpret_cast<uint2*>(dst + r * kFp8Block + (((col >> 4) ^ (r & 7)) << 4) + (col & 8)) = e4m3x8(f, inv);
  }
  const int kpad = (Kb + 3) / 4 * 4;
  if (threadIdx.x == 0) w_scale[enb * kpad + kb] = static_cast<uint8_t>(byte);
  if (kb == Kb - 1 && kb + 1 + static_cast<int>(threadIdx.x) < kpad) w_scale[enb * kpad + kb + 1 + threadIdx.x] = 1;
}

// ------------------------------------------------------------- tensor cores

// D[tmem] (+)= sum over 32 k of 2^(sfa + sfb) A[smem] * B[smem]^T, e4m3 x e4m3 -> fp32, one
// E8M0 scale per row of A and of B taken from TMEM (a byte of the scale words, by the
// instruction descriptor).  kPair: by a CTA pair, as in mma_i8_pair; each CTA's TMEM holds the
// scales of its own 128 rows of A and of all rows of B.
template <bool kPair>
__device__ __forceinline__ void mma_mxf8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (kPair) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  }
}

// 3-D tiled tensor load into shared memory; kPair: counted on a barrier of the pair's leader (see tma_load_2d_pair).
template <bool kPair>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1, int c2) {
  if (kPair) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  }
}

// A whole warp's wait for a phase.  Mostly the phase is there, or comes within
// the time that one try waits by itself: the warp then goes on without
// diverging (one lane waiting and telling the others cost about 280 cycles
// each time).  Else lane 0 waits within the time limit.  kTmem: a signal from either CTA of a pair behind which only
// TMEM is touched (see mbar_try_wait_cluster_relaxed).
template <bool kTmem = false>
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns,
                                               int err_code) {
  if (__all_sync(0xFFFFFFFFu, kTmem ? mbar_try_wait_cluster_relaxed(bar, parity) : mbar_try_wait(bar, parity))) return true;
  int ok = 1;
  if ((threadIdx.x & 31) == 0)
    ok = kTmem ? mbar_wait_cluster<true>(bar, parity, abort_flag, limit_ns, err_code)
               : mbar_wait(bar, parity, abort_flag, limit_ns, err_code);
  ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
  __syncwarp();
  return ok != 0;
}

// Eight bf16 values, or the first `left` of them, to a 16-byte boundary.
__device__ __forceinline__ void store_bf16x8(__nv_bfloat16* dst, const uint4& w, int left) {
  if (left >= 8) {
    *reinterpret_cast<uint4*>(dst) = w;
  } else {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) reinterpret_cast<uint16_t*>(dst)[i] = static_cast<uint16_t>(u[i >> 1] >> ((i & 1) * 16));
  }
}

// Instruction descriptor of kind::mxf8f6f4: e4m3 x e4m3, both operands K-major, E8M0 scales,
// byte `sf` of the scale words of both operands.
__device__ __forceinline__ uint32_t idesc_mxf8(uint32_t M, uint32_t N, uint32_t sf) {
  return (sf << 4)            // B's scale byte
         | ((N >> 3) << 17)   // N / 8
         | (1u << 23)         // scale format: E8M0
         | ((M >> 4) << 24)   // M / 16
         | (sf << 29);        // A's scale byte
}

// This warp's 32 lanes of four TMEM columns: lane l gets the words of thread l.
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, const uint32_t* w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3])
               : "memory");
}
// 16 lanes x 32 columns of TMEM as 2 x 4 pieces of 8 lanes x 8 columns: register pair (2 i, 2 i + 1) of piece
// i = 2 c + h holds lane 8 h + l / 4, columns 8 c + 2 (l % 4) and the next.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 32 lanes x 16 columns (thread i: lane i), loaded when it returns.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed, to the rows whose addresses the lanes give (lane 8 i + j: row j of
// matrix i): thread l's word i goes to rows 2 (l % 4) and the next, column l / 4, of matrix i.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ----------------------------------------------------------------- product

struct LinArgs {
  int E, M, N, K;
  int Kb, last_ksteps;   // 128-channel blocks; 32-channel steps in the last one
  int nblk, kgroups;     // 128-channel output blocks; groups of four 128-channel blocks (one scale word)
  int tiles_n;           // output tiles: blocks, or pairs of them
  int NT;                // most rows of a tile (a multiple of 16)
  int spans;             // spans of a single layer's rows
  int span_group;        // spans walked under each output tile (see LinTiles)
  int box_rows;          // most rows of a CTA's part of a tile, rounded up to a box
  int stages;
  uint32_t stage_bytes;  // of a stage's blocks: 16 KB of weights + box_rows rows of codes each
  uint32_t acc_cols, sf_col, tmem_cols;
  int split;             // CTAs or pairs of a cluster that share a tile along K (above 1: one tile to a cluster)
  const __nv_bfloat16* x;  // (quantising variant) the rows, ldx apart
  int64_t ldx;
  int vec_x;             // (quantising variant) rows of x (and their second halves) start on 16 bytes
  int silu;              // (quantising variant) rows are [gate | up]
  uint32_t codes_bytes;  // (quantising variant) codes of a CTA's part of K
  int early;             // weights and offsets are final before the kernel before this one ends
  int vec_out;           // rows of out start on 16 bytes
  const int32_t* offsets;    // [E + 1] row offsets of the experts, or null (one span of M rows)
  const uint32_t* x_scale;   // [kgroups][M]
  const uint32_t* w_scale;   // [E][nblk][kgroups]
  const __nv_bfloat16* bias;  // [E][N] or null
  __nv_bfloat16* out;
  int64_t ldo;
  uint64_t wait_limit_ns;
};

constexpr int kLinScaleWarps = 4, kLinEpiWarps = 4;
constexpr int kLinOutWarps = kLinScaleWarps + kLinEpiWarps;  // that write a CTA's only tile
constexpr int kLinThreads = 32 * (2 + kLinOutWarps);
constexpr int kLinMaxStages = 12;
constexpr int kLinMaxExperts = 1024;
constexpr int kLinMaxSplit = 8;                        // CTAs of a cluster that share a tile
constexpr int kLinStageBlocks = 2;                     // 128-channel blocks of a pipeline stage
constexpr int kLinBoxRows = 16;                        // TMA boxes of codes hold a multiple of these rows,
constexpr int kLinBoxes = 8;                           // up to so many times as many

// Tensor maps: the codes in boxes of 16, 32 .. 128 rows of a stage's blocks, and the weights' tiles.
struct LinMaps {
  CUtensorMap x[kLinBoxes], w;
};

constexpr uint32_t kLinATile = kFp8Block * kFp8Block;  // bytes of one weight tile
constexpr uint32_t kLinBars = 8 * (2 * kLinMaxStages + 4 + 4 + 1);
// The variant that quantises its rows itself: rows of its tile and 128-channel blocks of its part of K, at most.
constexpr int kLinFuseRows = 16, kLinFuseBlocks = 32;
constexpr int kLinFuseItems = 64;  // rows times blocks: one pass of its warps
constexpr uint32_t kLinFuseScales = (kLinFuseBlocks / 4 + 1) * kLinFuseRows * 4;  // its scale words (a part may start inside a group)
constexpr uint32_t kLinEpiBuf = 2048;                  // an epilogue warp's 32 rows x 32 channels of bf16
// Most rows of a tile: two accumulators and two sets of scale words (4 columns of weights', 1 per 32 rows) fit the 512
// columns of TMEM.
template <bool kPair>
constexpr int kLinMaxNT = kPair ? 240 : 128;
template <bool kPair>
constexpr int kLinSfCols = kPair ? 12 : 8;  // columns of one set of scale words

struct LinTile {
  int e, nb, row0, rows;
  int n;  // rows of the product: `rows` rounded up to the 16 that an MMA takes
};

// Tile `local` of an expert's `count` rows from `start` in `spans` spans.
__device__ __forceinline__ LinTile lin_tile(int local, int spans, int group, int tiles_n, int e, int start, int count) {
  const int full = group * tiles_n;
  const int g0 = local / full * group, in = local % full;
  const int gs = min(group, spans - g0);
  LinTile t;
  t.e = e;
  t.nb = in / gs;
  const int per = ((count + spans - 1) / spans + 15) & ~15;
  const int s = g0 + in % gs;
  t.row0 = start + s * per;
  t.rows = min(per, count - s * per);
  t.n = (t.rows + 15) & ~15;
  return t;
}

// The tiles of a launch: for each expert, its rows in spans of at most NT (as
// even as multiples of 16 allow), and for each span every output tile.
// `first` [E + 1]: spans before expert e; `start` [E]: its first row; `count`
// [E]: its rows.  Tiles are walked in increasing order, so the expert is found
// by moving on from the last one.  Inside an expert the order is: groups of
// `group` spans; output tiles; spans of the group -- what runs at one time then
// shares its weights, and the group's codes stay in L2.
struct LinTiles {
  const int *first, *start, *count;
  int E, tiles_n, group;
  int e = 0;
  __device__ __forceinline__ int total() const { return first[E] * tiles_n; }
  __device__ __forceinline__ LinTile at(int tile) {
    while (tile >= first[e + 1] * tiles_n) ++e;
    return lin_tile(tile - first[e] * tiles_n, first[e + 1] - first[e], group, tiles_n, e, start[e], count[e]);
  }
};

// Swapped product: the weights are the MMA's 128-row operand and the rows of x
// its N, so that a tile takes any multiple of 16 rows and few rows cost few
// MMA cycles.  Accumulators: lane = output channel, column = row of x.
//
// Pipeline stages hold two 128-channel blocks: what the issuing warp does for a
// stage besides the MMAs themselves (waits, descriptors, commits) takes some
// hundred cycles, the four MMAs of a block 290 (16 rows) to 500 (a pair's 240).
// Stages of one block, although more of them fit, took 16.0 us instead of 13.4
// for 300 x 4096 x 4096 and 226 instead of 215 for 8192 x 8192 x 4096.
//
// Warp roles: warp 0 loads (a stage's weights as one 32 KB box that is already
// in the MMA's order, its rows' codes as one box of the height that holds them:
// a load takes the issuing thread about 100 cycles whatever its size), warp 1
// owns TMEM and issues the MMAs, warps 2-5 write the scale words of each group
// of four 128-channel blocks into TMEM (every lane quarter holds a copy: warp %
// 4 is the quarter a warp can reach), warps 6-9 write the outputs.
//
// Measured, product alone (without its quantiser): 8192 x 8192 x 4096 in 197 us
// in short bursts (2.8 PFLOP/s; tensor pipe 89 % active) and 228 us in a loop of
// seconds, at the power cap and 1.2 GHz; 16384 rows over 64 experts of
// 2048 x 2048 in 81 and 97 us; 64 rows over 24 of 32 such experts in 20.5 us
// (4.9 TB/s).
//
// kPair: a CTA pair runs the tensor cores' cta_group::2 path.  A tile is then
// 256 output channels; each CTA loads its own 128 rows of weights and half of
// the rows' codes, and writes the outputs of its own channels.  The leader
// issues the MMAs; loads and scale words of both are counted on its barriers,
// and its commits arrive on the barriers of both.
//
// Split along K: where few rows leave too few tiles for the SMs, a cluster of
// `split` CTAs (or pairs) takes one tile, each a part of its K.  The sums of
// each are put in its shared memory, added in the order of the ranks over
// distributed shared memory (no atomics: the same bits every time, and no
// workspace), and written.  (Pushing them into the adding CTA's memory with
// asynchronous stores counted on a barrier there was no faster for one row and
// took 12.0 us instead of 10.3 for 16 rows, 8192 x 4096.)
//
// kFuse (single CTAs, one tile each): the rows are bf16 and eight warps quantise
// the CTA's part of them -- the codes, scales and outputs of the quantiser and
// the product, in one launch.  Every CTA of a row does it again, so it is for
// few rows: one pass of the warps (1 x 2048 x 2048 5.1 us, the two launches
// 5.9; 4 x 4096 x 4096 6.8 and 7.2; with two passes, 16 x 4096 x 4096, 8.3 and
// 7.4).  It is done once, in front of the MMAs, while the ring fills with
// weights: a stage at a time beside the MMAs its chain of barriers took 2200
// cycles a stage.
//
// Launched as a programmatic dependent.  With `early` (the quantiser of the
// same call in front) the first weights are loaded before its end is waited
// for; codes, scales and everything written wait for it.
template <bool kPair, bool kFuse>
__global__ void __launch_bounds__(kLinThreads, kPair ? 1 : 2)
    linear_fp8_kernel(const __grid_constant__ LinMaps maps, const LinArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const uint32_t codes = base + static_cast<uint32_t>(a.stages) * a.stage_bytes;  // (kFuse) codes, then scale words
  const uint32_t scale_words = codes + a.codes_bytes;
  const uint32_t epi_stage = codes + (kFuse ? a.codes_bytes + kLinFuseScales : 0u);
  const uint32_t bars = epi_stage + kLinOutWarps * kLinEpiBuf;
  const uint32_t full = bars, empty = full + 8 * kLinMaxStages;
  const uint32_t sf_full = empty + 8 * kLinMaxStages, sf_empty = sf_full + 16;
  const uint32_t acc_full = sf_empty + 16, acc_empty = acc_full + 16;
  const uint32_t drain_bar = acc_empty + 16;
  uint8_t* const misc = base_ptr + (bars - base) + kLinBars;
  volatile uint32_t* const tmem_slot = reinterpret_cast<volatile uint32_t*>(misc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  int* const first = reinterpret_cast<int*>(misc + 8);
  int* const start = first + a.E + 1;
  int* const count = start + a.E;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = a.wait_limit_ns;
  constexpr int kCtas = kPair ? 2 : 1;
  const bool split = a.split > 1;
  const uint32_t cta = kPair || split ? cluster_ctarank() : 0u;  // in the cluster
  const uint32_t rank = cta % kCtas;                             // in the pair: 0 = its leader
  const uint32_t lead_cta = cta - rank;
  const bool leader = rank == 0;
  const int first_tile = kPair || split ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int tile_step = kPair || split ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  // this CTA's blocks of K: whole stages
  int kb0 = 0, kb1 = a.Kb;
  if (split) {
    const int r = static_cast<int>(cta) / kCtas, stages = (a.Kb + kLinStageBlocks - 1) / kLinStageBlocks;
    kb0 = stages * r / a.split * kLinStageBlocks;
    kb1 = min(stages * (r + 1) / a.split * kLinStageBlocks, a.Kb);
  }

  if (warp == 0) {
    if (lane == 0) prefetch_tmap(&maps.w);
    if (lane == 1 && !kFuse) prefetch_tmap(&maps.x[a.box_rows / kLinBoxRows - 1]);
    if (lane < a.stages) {
      mbar_init(full + 8 * lane, 1);
      mbar_init(empty + 8 * lane, 1);
    }
    if (lane < 2) {
      mbar_init(sf_full + 8 * lane, kCtas * kLinScaleWarps);
      mbar_init(sf_empty + 8 * lane, 1);
      mbar_init(acc_full + 8 * lane, 1);
      mbar_init(acc_empty + 8 * lane, kCtas * kLinEpiWarps);
    }
    if (lane == 2) {
      mbar_init(drain_bar, 1);
      *abort_flag = 0;
    }
    fence_barrier_init();
    __syncwarp();
  }
  // Weights of the stage at ring position `at`.  A last stage of one block loads what follows its weights, or the zeros
  // behind the tensor: no MMA reads it.
  auto load_w = [&](uint32_t at, int wrow, uint32_t bytes) {
    const uint32_t dst = base + at * a.stage_bytes, bar = full + 8 * at;
    if (leader) mbar_arrive_expect_tx(bar, bytes * kCtas);
    if (!check_bounds(bytes <= a.stage_bytes && wrow >= 0 && wrow < a.E * a.nblk * a.Kb && at < static_cast<uint32_t>(a.stages)))
      return;
    if (kPair) {
      tma_load_2d_pair(dst, &maps.w, map_to_cta(bar, lead_cta), 0, wrow * kFp8Block);
    } else {
      tma_load_2d(dst, &maps.w, bar, 0, wrow * kFp8Block);
    }
  };
  // Bytes of a stage of tile t: the weights and the boxes of codes.
  auto stage_boxes = [&](const LinTile& t) { return (t.n / kCtas + kLinBoxRows - 1) / kLinBoxRows; };
  auto stage_bytes = [&](const LinTile& t) {
    return kLinStageBlocks * (kLinATile + (kFuse ? 0u : static_cast<uint32_t>(stage_boxes(t)) * (kLinBoxRows * 128u)));
  };
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(tmem_slot)), a.tmem_cols);
    } else {
      tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), a.tmem_cols);
    }
  }
  if (!a.early) grid_dependency_wait();
  if (!a.offsets) {
    if (threadIdx.x == 64) {
      first[0] = start[0] = 0;
      first[1] = a.spans;
      count[0] = a.M;
    }
  } else if (warp == 2) {
    // spans of each expert; an offset outside 0..M is clipped, one below an earlier one counts as that one
    int sum = 0, top = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      int lo = min(max(__ldcg(a.offsets + min(e, a.E)), top), a.M);
      for (int o = 1; o < 32; o <<= 1) lo = max(lo, __shfl_up_sync(0xFFFFFFFFu, lo, o));
      const int hi = max(lo, min(__ldcg(a.offsets + min(e + 1, a.E)), a.M));
      top = __shfl_sync(0xFFFFFFFFu, hi, 31);
      const int c = e < a.E ? hi - lo : 0;
      int p = (c + a.NT - 1) / a.NT;
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, p, o);
        if (lane >= o) p += up;
      }
      if (e < a.E) {
        start[e] = lo;
        count[e] = c;
        first[e + 1] = sum + p;
      }
      sum += __shfl_sync(0xFFFFFFFFu, p, 31);
    }
    if (lane == 0) first[0] = 0;
  }
  __syncwarp();
  tc_fence_before();
  if (kPair) {
    cluster_sync();  // both CTAs' barriers exist before either signals the other
  } else {
    __syncthreads();
  }
  tc_fence_after();
  // Only now: a kernel behind this one may rely on all that came before this one, and must not take TMEM that a CTA
  // of this grid still waits for.
  if (!a.early) grid_dependents_launch();
  const uint32_t tmem_base = *tmem_slot;
  LinTiles tiles{first, start, count, a.E, a.tiles_n, a.span_group};
  const int total = tiles.total();
  // Where no CTA has a second tile, the scale warps, which have nothing left to do by then, write half of the outputs.
  const bool solo = a.NT > 32 && (split || total <= tile_step);

  if (kFuse && warp >= 2 && first_tile < total) {
    // ----------------------------------------------------------- quantisers
    // The tile's rows, this CTA's part of K: 16 channels to a lane and eight
    // lanes to a block, as in the quantiser; codes [block][16 rows][128] in the
    // MMA's swizzled order and scale bytes in shared memory.  Then four of the
    // warps put the scale words into TMEM: row l's at lane l.
    const LinTile t = tiles.at(first_tile);
    const int sub = lane >> 3, col = lane & 7;
    const int blocks = kb1 - kb0, items = t.rows * blocks;  // at most kLinFuseItems
    constexpr int kWarps = kLinOutWarps, kItems = kLinFuseItems / (kWarps * 4);
    uint4 w[kItems][2], u[kItems][2];
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
      const int item = (r * kWarps + warp - 2) * 4 + sub;
      const int row = item / blocks, b = item - row * blocks;
      const int64_t k = static_cast<int64_t>(kb0 + b) * kFp8Block + col * 16;
      const uint16_t* const x = reinterpret_cast<const uint16_t*>(a.x);
      const uint16_t* const src = x + (t.row0 + row) * a.ldx;
      w[r][0] = w[r][1] = u[r][0] = u[r][1] = make_uint4(0u, 0u, 0u, 0u);
      if (item < items && k < a.K && check_bounds(t.row0 + row < a.M)) {
        if (a.vec_x) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (k + 8 * h >= a.K) continue;
            w[r][h] = load_bf16x8<true>(src, k + 8 * h, a.K);
            if (a.silu) u[r][h] = load_bf16x8<true>(src + a.K, k + 8 * h, a.K);
          }
        } else {
          const uint16_t* const x_end = x + (a.M - 1) * a.ldx + (a.silu ? 2 : 1) * static_cast<int64_t>(a.K);
          load_bf16x16_anywhere(src, k, a.K, x, x_end, w[r]);
          if (a.silu) load_bf16x16_anywhere(src + a.K, k, a.K, x, x_end, u[r]);
        }
      }
    }
    // the weights' words: lane g holds group g's
    uint32_t wword = 0;
    const int kg0 = kb0 >> 2, kg1 = (kb1 + 3) >> 2;
    if (kg0 + lane < kg1) wword = __ldcg(a.w_scale + static_cast<int64_t>(t.e * a.nblk + t.nb) * a.kgroups + kg0 + lane);
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
      const int item = (r * kWarps + warp - 2) * 4 + sub;
      const int row = item / blocks, b = item - row * blocks;
      float v[2][8];
      uint32_t m = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        widen_bf16x8(w[r][h], v[h]);
        if (a.silu) {  // (zeros beyond K stay zeros)
          float up[8];
          widen_bf16x8(u[r][h], up);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[h][j] = silu_mul(v[h][j], up[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[h][j]));
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      if (item < items) {
        const uint32_t byte = e8m0_of_amax(m);
        const float inv = e8m0_reciprocal(byte);
        const uint2 lo = e4m3x8(v[0], inv), hi = e4m3x8(v[1], inv);
        const uint32_t line = static_cast<uint32_t>(b * kLinFuseRows + row);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(codes + line * 128u + static_cast<uint32_t>((col ^ (row & 7)) << 4)),
                     "r"(lo.x), "r"(lo.y), "r"(hi.x), "r"(hi.y)
                     : "memory");
        // byte (kb & 3) of word [group][row]
        const int kb = kb0 + b;
        if (col == 0)
          asm volatile("st.shared.u8 [%0], %1;" ::"r"(scale_words + static_cast<uint32_t>((((kb >> 2) - kg0) * kLinFuseRows + row) * 4 + (kb & 3))),
                       "r"(byte)
                       : "memory");
      }
    }
    fence_proxy_async_smem();  // the codes are read by the tensor cores
    named_barrier_sync(1, 32 * kWarps);
    if (warp < 2 + kLinScaleWarps) {
      const uint32_t dst = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + a.sf_col;
      for (int g = 0; g < kg1 - kg0; ++g) {
        uint32_t sf[8] = {};
        sf[0] = sf[1] = sf[2] = sf[3] = __shfl_sync(0xFFFFFFFFu, wword, g);
        asm volatile("ld.shared.u32 %0, [%1];"
                     : "=r"(sf[4])
                     : "r"(scale_words + static_cast<uint32_t>(g * kLinFuseRows + (lane & (kLinFuseRows - 1))) * 4u));
        tmem_st_x4(dst + static_cast<uint32_t>(g) * kLinSfCols<kPair>, sf);
        tmem_st_x4(dst + static_cast<uint32_t>(g) * kLinSfCols<kPair> + 4, sf + 4);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sf_full);
    }
  }

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer
    uint32_t s = 0, p = 0, armed = 0, par = 0;
    bool waited = !a.early;
    int ahead = kb0;  // blocks of the first tile whose weights have been asked for
    for (int tile = first_tile; tile < total; tile += tile_step) {
      const LinTile t = tiles.at(tile);
      const int mine = t.n / kCtas;  // this CTA's rows of the codes
      const CUtensorMap* const map_x = &maps.x[stage_boxes(t) - 1];
      const uint32_t bytes = stage_bytes(t);
      // the second CTA of the last pair may have no output block of its own: it reads the last one again
      const int nb = min(t.nb * kCtas + static_cast<int>(rank), a.nblk - 1);
      const int wrow = (t.e * a.nblk + nb) * a.Kb;
      const int row = t.row0 + static_cast<int>(rank) * mine;
      if (!waited) {  // the ring is empty: fill it with weights, then wait for the rows' codes
        for (uint32_t i = 0; i < static_cast<uint32_t>(a.stages) && ahead < kb1; ++i, ahead += kLinStageBlocks)
          load_w(i, wrow + ahead, bytes);
        grid_dependency_wait();
        waited = true;
      }
      if (tile != first_tile) ahead = kb0;
      for (int kb = kb0; kb < kb1; kb += kLinStageBlocks) {
        const uint32_t dst_x = base + s * a.stage_bytes + kLinStageBlocks * kLinATile;
        const uint32_t bar = full + 8 * s;
        if (kb >= ahead) {
          if (!mbar_wait(empty + 8 * s, p ^ 1, abort_flag, limit, kErrTimeoutProducer)) goto producer_done;
          load_w(s, wrow + kb, bytes);
        }
        if (check_bounds(t.row0 >= 0 && t.row0 < a.M)) {
          if (!kFuse) tma_load_3d<kPair>(dst_x, map_x, kPair ? map_to_cta(bar, lead_cta) : bar, 0, row, kb);
        }
        armed |= 1u << s;
        par = (par & ~(1u << s)) | (p << s);
        if (++s == static_cast<uint32_t>(a.stages)) { s = 0; p ^= 1; }
      }
    }
  producer_done:
    if (*abort_flag && leader) {
      // let every copy counted on this CTA's barriers land before it exits
      int dummy = 0;
      for (int i = 0; i < a.stages; ++i)
        if (armed >> i & 1) mbar_wait(full + 8 * i, par >> i & 1, &dummy, limit, kErrTimeoutDrain);
    }
  } else if (warp == 1 && leader) {
    // ---------------------------------------------------------- MMA issuer
    // The whole warp runs the loop; one elected lane issues a stage's MMAs and
    // commits as straight-line code.
    auto wait = [&](uint32_t bar, uint32_t parity) {
      return mbar_wait_warp(bar, parity, abort_flag, limit, kErrTimeoutMma);
    };
    // scale words written, accumulator read: signals from both CTAs of a pair (kFuse: with the codes in shared memory)
    auto wait_tmem = [&](uint32_t bar, uint32_t parity) {
      return mbar_wait_warp<kPair>(bar, parity, abort_flag, limit, kErrTimeoutMma);
    };
    auto commit = [&](uint32_t bar) {
      if (kPair) {
        mma_commit_pair_multicast(bar, static_cast<uint16_t>(0x3u << lead_cta));
      } else {
        mma_commit(bar);
      }
    };
    const uint64_t ad0 = sw128_kmajor_desc(base, 1024u);
    const uint64_t bd0 = sw128_kmajor_desc(kFuse ? codes : base + kLinStageBlocks * kLinATile, 1024u);
    const uint32_t stage16 = a.stage_bytes >> 4;
    // 32-channel steps of the tile's last stage
    const int last_steps = kb1 < a.Kb ? 4 * kLinStageBlocks : (a.Kb - 1) % kLinStageBlocks * 4 + a.last_ksteps;
    uint32_t s = 0, p = 0, g = 0, gp = 0, c = 0, cp = 0;
    bool issued = false, ok = true;
    for (int tile = first_tile; tile < total && ok; tile += tile_step) {
      const LinTile t = tiles.at(tile);
      const uint32_t d = tmem_base + c * a.acc_cols;
      if (!check_bounds(static_cast<uint32_t>(t.n) <= a.acc_cols) || !(ok = wait_tmem(acc_empty + 8 * c, cp ^ 1))) {
        ok = false;
        break;
      }
      uint32_t acc = 0;  // the tile's first MMA overwrites the accumulator
      // from the first block's codes to the second's
      const uint32_t rows16 = static_cast<uint32_t>(kFuse ? kLinFuseRows : stage_boxes(t) * kLinBoxRows) * 8u;
      for (int kb = kb0; kb < kb1; kb += kLinStageBlocks) {
        // a scale word serves two stages (kFuse: all are there, and stay, from the first on)
        const bool last = kb + kLinStageBlocks >= kb1, first_half = (kb & 3) == 0;
        const bool group_end = !kFuse && (!first_half || last);
        if ((kb == kb0 || (!kFuse && first_half)) && !(ok = wait_tmem(sf_full + 8 * g, gp))) break;
        if (!(ok = wait(full + 8 * s, p))) break;
        tc_fence_after();
        const uint64_t ad = ad0 + s * stage16;
        const uint64_t bd = kFuse ? bd0 + static_cast<uint32_t>(kb - kb0) * rows16 : bd0 + s * stage16;
        const uint32_t sf = tmem_base + a.sf_col +
                            (kFuse ? static_cast<uint32_t>((kb >> 2) - (kb0 >> 2)) : g) * kLinSfCols<kPair>;
        const uint32_t idesc = idesc_mxf8(128 * kCtas, static_cast<uint32_t>(t.n), first_half ? 0u : 2u);
        constexpr uint32_t kNextByte = (1u << 4) | (1u << 29);  // the second block's byte of the scale words
        const int steps = last ? last_steps : 4 * kLinStageBlocks;
        if (elect_one()) {
          // 32 bytes of K = 2 units of the descriptors
          auto step = [&](int j) {
            mma_mxf8<kPair>(d, ad + (j >> 2) * (kLinATile >> 4) + 2 * (j & 3), bd + (j >> 2) * rows16 + 2 * (j & 3),
                            j < 4 ? idesc : idesc + kNextByte, sf, sf + 4, j == 0 ? acc : 1u);
          };
          if (steps == 4 * kLinStageBlocks) {
#pragma unroll
            for (int j = 0; j < 4 * kLinStageBlocks; ++j) step(j);
          } else {
            for (int j = 0; j < steps; ++j) step(j);
          }
          commit(empty + 8 * s);
          if (group_end) commit(sf_empty + 8 * g);
          if (last) commit(acc_full + 8 * c);
        }
        __syncwarp();
        issued = true;
        acc = 1;
        if (++s == static_cast<uint32_t>(a.stages)) { s = 0; p ^= 1; }
        if (group_end) {
          g ^= 1;
          gp ^= g == 0;
        }
      }
      c ^= 1;
      cp ^= c == 0;
    }
    if (!ok && issued && lane == 0) {
      // the tensor cores finish what was issued before TMEM is freed
      int dummy = 0;
      if (kPair) {
        mma_commit_pair(drain_bar);
      } else {
        mma_commit(drain_bar);
      }
      mbar_wait(drain_bar, 0, &dummy, limit, kErrTimeoutDrain);
    }
    __syncwarp();
  } else if (!kFuse && warp >= 2 && warp < 2 + kLinScaleWarps) {
    // -------------------------------------------------------------- scales
    // Group of four blocks: the weights' word (the same for all 128 channels)
    // into four columns, the rows' words into the next: row 32 j + l at lane l
    // of column j.
    const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
    constexpr int kRowCols = kLinSfCols<kPair> - 4;
    const int kg0 = kb0 >> 2, kg1 = (kb1 + 3) >> 2;
    uint32_t next[1 + kRowCols];  // the next group's words, in flight while this group's are waited for
    if (a.early) {
      grid_dependency_wait();
      grid_dependents_launch();
    }
    uint32_t g = 0, gp = 0;
    bool ok = true;
    for (int tile = first_tile; tile < total && ok; tile += tile_step) {
      const LinTile t = tiles.at(tile);
      const int nb = min(t.nb * kCtas + static_cast<int>(rank), a.nblk - 1);
      const uint32_t* const ws = a.w_scale + static_cast<int64_t>(t.e * a.nblk + nb) * a.kgroups;
      auto load = [&](int kg) {
        next[0] = __ldcg(ws + kg);
#pragma unroll
        for (int j = 0; j < kRowCols; ++j) {
          const int row = t.row0 + 32 * j + lane;
          next[1 + j] =
              32 * j < t.n && row < a.M ? __ldcg(a.x_scale + static_cast<int64_t>(kg) * a.M + row) : 0x7F7F7F7Fu;
        }
      };
      load(kg0);
      for (int kg = kg0; kg < kg1; ++kg) {
        uint32_t w[4 + kRowCols];
        w[0] = w[1] = w[2] = w[3] = next[0];
#pragma unroll
        for (int j = 0; j < kRowCols; ++j) w[4 + j] = next[1 + j];
        if (kg + 1 < kg1) load(kg + 1);
        if (!(ok = mbar_wait_warp(sf_empty + 8 * g, gp ^ 1, abort_flag, limit, kErrTimeoutConvert))) break;
        tc_fence_after();
        const uint32_t dst = tmem_base + quarter + a.sf_col + g * kLinSfCols<kPair>;
#pragma unroll
        for (int j = 0; j < 4 + kRowCols; j += 4) tmem_st_x4(dst + j, w + j);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          // what the issuer's MMAs read of this are TMEM stores that tcgen05.wait::st has seen complete and the fence
          // orders: no release at cluster scope, which also waits for the next words' loads and for everything else
          // this warp has in flight (it cost 15 % of the whole product: 237 against 205 us at 8192 x 8192 x 4096)
          if (kPair) {
            mbar_arrive_cluster_relaxed(map_to_cta(sf_full + 8 * g, lead_cta));
          } else {
            mbar_arrive(sf_full + 8 * g);
          }
        }
        g ^= 1;
        gp ^= g == 0;
      }
    }
  }
  if (warp >= (solo ? 2 : 2 + kLinScaleWarps)) {
    // ------------------------------------------------------------ epilogue
    // 32 rows of x (columns) by this warp's 32 channels (lanes) at a time:
    // sums + bias, rounded to bf16, transposed through shared memory (64-byte
    // lines of 32 channels, 16-byte groups permuted by the line against bank
    // conflicts) and written as 16-byte groups of 8 channels.
    const int q = warp & 3;
    // blocks of 32 rows: all, or every other one (the scale warps': the odd ones)
    const int r_first = solo && warp < 2 + kLinScaleWarps ? 32 : 0, r_step = solo ? 64 : 32;
    const uint32_t buf = epi_stage + static_cast<uint32_t>(warp - 2) * kLinEpiBuf;
    const uint32_t empty_leader = kPair ? map_to_cta(acc_empty, lead_cta) : acc_empty;
    // stmatrix: lane 8 i + j gives line 8 * step + j, group i
    const uint32_t st_line = static_cast<uint32_t>(lane & 7), st_grp = static_cast<uint32_t>(lane >> 3);
    const uint32_t st_addr = buf + st_line * 64u + ((st_grp ^ (st_line >> 1)) << 4);
    // reading back: lane 4 j + i reads line 8 * step + j, group i
    const uint32_t ld_line = static_cast<uint32_t>(lane >> 2), ld_grp = static_cast<uint32_t>(lane & 3);
    const uint32_t ld_addr = buf + ld_line * 64u + ((ld_grp ^ ((ld_line >> 1) & 3u)) << 4);
    uint32_t c = 0, cp = 0;
    if (a.early) grid_dependency_wait();
    if (split && first_tile < total) {
      // this CTA's sums into its ring (every stage has been read): [row][128 channels] of fp32.  The tile's groups of 4
      // channels are then added CTA by CTA (see below)
      const LinTile t = tiles.at(first_tile);
      if (mbar_wait_warp(acc_full, 0, abort_flag, limit, kErrTimeoutEpilogue)) {
        tc_fence_after();
#pragma unroll 1
        for (int r0 = r_first / 2; r0 < t.n; r0 += r_step / 2) {  // (the ring holds NT rows, a multiple of 16)
          uint32_t v[16];
          tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(r0), v);
          const uint32_t dst = base + static_cast<uint32_t>(r0 * kFp8Block + q * 32 + lane) * 4u;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + static_cast<uint32_t>(j * kFp8Block * 4)), "r"(v[j]) : "memory");
        }
        tc_fence_before();
      }
    }
    for (int tile = split ? total : first_tile; tile < total; tile += tile_step) {
      const LinTile t = tiles.at(tile);
      const int ch0 = (t.nb * kCtas + static_cast<int>(rank)) * kFp8Block + q * 32;  // this warp's first channel
      float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // bias of channels ch0 + 8 i + lane / 4
      if (a.bias) {
        const __nv_bfloat16* const be = a.bias + static_cast<int64_t>(t.e) * a.N;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (ch0 + 8 * i + (lane >> 2) < a.N) b[i] = __bfloat162float(be[ch0 + 8 * i + (lane >> 2)]);
      }
      if (!mbar_wait_warp(acc_full + 8 * c, cp, abort_flag, limit, kErrTimeoutEpilogue)) break;
      tc_fence_after();
      const uint32_t src = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + c * a.acc_cols;
      const int ch = ch0 + 8 * static_cast<int>(ld_grp);  // the group of channels this lane writes
      auto issue = [&](int r0, uint32_t(&v)[32]) {
        tmem_ld_16x256b_x4(src + static_cast<uint32_t>(r0), v);
        tmem_ld_16x256b_x4(src + (16u << 16) + static_cast<uint32_t>(r0), v + 16);
      };
      auto process = [&](int r0, const uint32_t(&v)[32]) {
        __syncwarp();  // the last block's lines have been read
#pragma unroll
        for (int step = 0; step < 4; ++step) {  // 8 rows of x: matrices of channels 0-7, 8-15, 16-23, 24-31
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = (i >> 1) * 16 + step * 4 + (i & 1) * 2;
            const __nv_bfloat162 p2 =
                __floats2bfloat162_rn(__uint_as_float(v[at]) + b[i], __uint_as_float(v[at + 1]) + b[i]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p2);
          }
          stmatrix_x4_trans(st_addr + static_cast<uint32_t>(step) * 512u, w);
        }
        __syncwarp();
        if (!a.vec_out) {  // rows of out that start anywhere: 32 adjacent values at a time
          const int mine = ch0 + lane;
          __nv_bfloat16* const dst = a.out + (t.row0 + r0) * a.ldo + mine;
#pragma unroll 4
          for (int r = 0; r < 32; ++r) {
            uint16_t v16;
            asm volatile("ld.shared.u16 %0, [%1];"
                         : "=h"(v16)
                         : "r"(buf + static_cast<uint32_t>(r * 64 + ((((lane >> 3) ^ (r >> 1)) & 3) << 4) + (lane & 7) * 2)));
            if (r0 + r < t.rows && mine < a.N && check_bounds(t.row0 + r0 + r < a.M))
              *reinterpret_cast<uint16_t*>(dst + r * a.ldo) = v16;
          }
          return;
        }
#pragma unroll
        for (int step = 0; step < 4; ++step) {
          const int r = r0 + step * 8 + static_cast<int>(ld_line);
          if (r < t.rows && ch < a.N && check_bounds(t.row0 + r < a.M)) {
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(ld_addr + static_cast<uint32_t>(step) * 512u));
            store_bf16x8(a.out + (t.row0 + r) * a.ldo + ch, w, a.N - ch);
          }
        }
      };
      for (int r0 = r_first; r0 < t.rows; r0 += r_step) {
        uint32_t v[32];
        issue(r0, v);
        tmem_ld_wait(v);
        process(r0, v);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair) {
          mbar_arrive_cluster_relaxed(empty_leader + 8 * c);
        } else {
          mbar_arrive(acc_empty + 8 * c);
        }
      }
      c ^= 1;
      cp ^= c == 0;
    }
  }

  __syncwarp();
  if (split) {
    // Each CTA adds and writes its share of the tile's groups of 4 channels (sums of a CTA that gave up are whatever its
    // ring holds: the error word says that the call's results are invalid).
    const bool have = first_tile < total;
    LinTile t = {};
    if (have) t = tiles.at(first_tile);
    const int r = static_cast<int>(cta) / kCtas, items = t.rows * (kFp8Block / 4);
    const int end = items * (r + 1) / a.split, c0 = (t.nb * kCtas + static_cast<int>(rank)) * kFp8Block;
    const int begin = items * r / a.split + static_cast<int>(threadIdx.x);
    const __nv_bfloat16* const be = a.bias ? a.bias + static_cast<int64_t>(t.e) * a.N : nullptr;
    // kS: the split, rounded up to a power of two; eight loads of four sums in flight a thread
    auto add = [&](auto KS) {
      constexpr int kS = decltype(KS)::value, kU = kLinMaxSplit / kS;
      for (int i0 = begin; i0 < end; i0 += kU * kLinThreads) {
        float w[kU][kS][4], b[kU][4];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int i = min(i0 + u * kLinThreads, end - 1), ch = c0 + i % (kFp8Block / 4) * 4;
#pragma unroll
          for (int k = 0; k < kS; ++k)  // (beyond the split: the last one again, not used)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(w[u][k][0]), "=f"(w[u][k][1]), "=f"(w[u][k][2]), "=f"(w[u][k][3])
                         : "r"(map_to_cta(base + static_cast<uint32_t>(i) * 16u,
                                          static_cast<uint32_t>(min(k, a.split - 1) * kCtas) + rank)));
#pragma unroll
          for (int j = 0; j < 4; ++j) b[u][j] = be && ch + j < a.N ? __bfloat162float(be[ch + j]) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int i = i0 + u * kLinThreads;
          const int row = i / (kFp8Block / 4), ch = c0 + i % (kFp8Block / 4) * 4;
          float v[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            v[h] = w[u][0][h];
#pragma unroll
            for (int k = 1; k < kS; ++k)
              if (k < a.split) v[h] += w[u][k][h];
            v[h] += b[u][h];
          }
          if (i < end && ch < a.N && check_bounds(t.row0 + row < a.M)) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
            const uint2 out = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            __nv_bfloat16* const dst = a.out + (t.row0 + row) * a.ldo + ch;
            if (a.vec_out && ch + 4 <= a.N) {
              *reinterpret_cast<uint2*>(dst) = out;
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (ch + j < a.N)
                  reinterpret_cast<uint16_t*>(dst)[j] = static_cast<uint16_t>((j < 2 ? out.x : out.y) >> ((j & 1) * 16));
            }
          }
        }
      }
    };
    cluster_sync();  // every CTA's sums are in its shared memory
    if (a.split <= 2) {
      add(IntC<2>{});
    } else if (a.split <= 4) {
      add(IntC<4>{});
    } else {
      add(IntC<8>{});
    }
    // no CTA leaves while another may still read its sums: waited for at the very end
    tc_fence_before();
    __syncwarp();
    cluster_arrive();
  }
  tc_fence_before();
  if (kPair) {
    // neither CTA leaves, or frees the pair's TMEM, while its partner may still touch its memory.  (A split pair has
    // arrived above, with its last reads of TMEM behind it: this wait is that arrive's, and the end's.)
    if (!split) cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if (kPair) {
      tmem_dealloc_pair(tmem_base, a.tmem_cols);
    } else {
      tmem_dealloc(tmem_base, a.tmem_cols);
    }
  }
  if (split && !kPair) {
    __syncwarp();
    cluster_wait();
  }
}

// Stands for linear_fp8_kernel where CUDA is asked how many clusters the device holds (never launched): the occupancy
// functions count one CTA to an SM for any kernel that allocates TMEM, however few columns, but the hardware runs as many
// as fit (two of 100 KB and 32 columns on every SM, in clusters of 1 to 8, measured).
__global__ void __launch_bounds__(kLinThreads, 2) linear_room_kernel() {}

}  // namespace qvae
