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

// Eight bf16 values x[k .. k+8) of a row of K as fp32, zeros beyond K.  kVec:
// the row starts on a 16-byte boundary and k is a multiple of 8.
template <bool kVec>
__device__ __forceinline__ void load_bf16x8(const uint16_t* row, int64_t k, int64_t K, float (&v)[8]) {
  if (kVec && k + 8 <= K) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + k));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < K ? bf16_bits_to_f32(__ldg(row + k + i)) : 0.0f;
  }
}

// silu(g) * u = g / (1 + exp(-g)) * u in fp32.  __expf is off by about
// |g| * 2^-23 of its value, far below the 2^-4 of the code it ends in; the
// divide is the IEEE one (the fast one gives 0 for denominators above 2^126).
__device__ __forceinline__ float silu_mul(float g, float u) { return __fdiv_rn(g, 1.0f + __expf(-g)) * u; }

// --------------------------------------------------------------- quantiser

constexpr int kFp8QuantThreads = 256;
constexpr int kFp8RowsPerWarp = 4;
constexpr int kFp8RowsPerBlock = kFp8QuantThreads / 32 * kFp8RowsPerWarp;

// Activations: codes [M][Kb * 128] (zeros beyond K) and scale words
// [ceil(Kb / 4)][M], byte j of word (g, m) being the scale of row m's block
// 4 g + j.  Blocks beyond Kb get byte 1.  kSilu: rows are [gate | up], K each,
// and what is quantised is silu(gate) * up.
//
// A warp takes four rows of one group of four blocks (512 channels): a half
// warp holds a block, 8 channels to a lane, and the maximum takes four
// shuffles.  One pass over x, bound by its bytes.
template <bool kSilu, bool kVec>
__global__ void __launch_bounds__(kFp8QuantThreads)
    fp8_quant_act_kernel(const uint16_t* __restrict__ x, int64_t ldx, int M, int K, int Kb, uint8_t* __restrict__ xq,
                         uint32_t* __restrict__ x_scale) {
  grid_dependency_wait();
  // only now: a kernel behind this one may rely on all that came before this one
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = lane >> 4, col = (lane & 15) * 8;
  const int kg = blockIdx.y;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kFp8RowsPerBlock + warp * kFp8RowsPerWarp;
  float v[kFp8RowsPerWarp][2][8];
#pragma unroll
  for (int r = 0; r < kFp8RowsPerWarp; ++r) {
    const uint16_t* row = x + (row0 + r) * ldx;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t k = static_cast<int64_t>(kg * 4 + i * 2 + half) * kFp8Block + col;
      if (row0 + r < M && k < K) {
        load_bf16x8<kVec>(row, k, K, v[r][i]);
        if (kSilu) {
          float u[8];
          load_bf16x8<kVec>(row + K, k, K, u);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[r][i][j] = k + j < K ? silu_mul(v[r][i][j], u[j]) : 0.0f;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[r][i][j] = 0.0f;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kFp8RowsPerWarp; ++r) {
    uint32_t byte[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[r][i][j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      byte[i] = e8m0_of_amax(m);
      const int kb = kg * 4 + i * 2 + half;
      if (row0 + r < M && kb < Kb)
        *reinterpret_cast<uint2*>(xq + ((row0 + r) * Kb + kb) * kFp8Block + col) =
            e4m3x8(v[r][i], e8m0_reciprocal(byte[i]));
    }
    const uint32_t hi0 = __shfl_down_sync(0xFFFFFFFFu, byte[0], 16), hi1 = __shfl_down_sync(0xFFFFFFFFu, byte[1], 16);
    if (lane == 0 && row0 + r < M)
      x_scale[static_cast<int64_t>(kg) * M + row0 + r] = byte[0] | (hi0 << 8) | (byte[1] << 16) | (hi1 << 24);
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
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = static_cast<int64_t>(nb) * kFp8Block + r0 + 16 * i;
    if (n < N && k < K) {
      load_bf16x8<kVec>(w + (e * N + n) * K, k, K, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
  }
  m = block_max_u32<kFp8PackThreads>(m, red);
  const uint32_t byte = e8m0_of_amax(m);
  const float inv = e8m0_reciprocal(byte);
  uint8_t* const dst = packed + tile * (kFp8Block * kFp8Block);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    *reinterpret_cast<uint2*>(dst + r * kFp8Block + (((col >> 4) ^ (r & 7)) << 4) + (col & 8)) = e4m3x8(v[i], inv);
  }
  const int kpad = (Kb + 3) / 4 * 4;
  if (threadIdx.x == 0) w_scale[enb * kpad + kb] = static_cast<uint8_t>(byte);
  if (kb == Kb - 1 && kb + 1 + static_cast<int>(threadIdx.x) < kpad) w_scale[enb * kpad + kb + 1 + threadIdx.x] = 1;
}

// ------------------------------------------------------------- tensor cores

// D[tmem] (+)= sum over 32 k of 2^(sfa + sfb) A[smem] * B[smem]^T, e4m3 x e4m3 -> fp32, one
// E8M0 scale per row of A and of B taken from TMEM (byte a_sf / b_sf of the scale word).
__device__ __forceinline__ void mma_mxf8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
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

// This warp's 32 lanes of four or eight TMEM columns: lane l gets the words of thread l.
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, const uint32_t* w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ----------------------------------------------------------------- product

struct LinArgs {
  int E, M, N, K;
  int Kb, last_ksteps;   // 128-channel blocks; 32-channel steps in the last one
  int nblk, kgroups;     // 128-channel output blocks; groups of four 128-channel blocks (one scale word)
  int NT;                // most rows of a tile (a multiple of 16)
  int stages;
  uint32_t stage_bytes;  // 16 KB of weights + the rows' codes
  uint32_t acc_cols, sf_col, tmem_cols;
  const int32_t* offsets;    // [E + 1] row offsets of the experts, or null (one span of M rows)
  const uint32_t* x_scale;   // [kgroups][M]
  const uint32_t* w_scale;   // [E][nblk][kgroups]
  const __nv_bfloat16* bias;  // [E][N] or null
  __nv_bfloat16* out;
  int64_t ldo;
  uint64_t wait_limit_ns;
};

constexpr int kLinScaleWarps = 4, kLinEpiWarps = 4;
constexpr int kLinThreads = 32 * (2 + kLinScaleWarps + kLinEpiWarps);
constexpr int kLinMaxStages = 12;
constexpr int kLinMaxNT = 128;
constexpr int kLinMaxExperts = 1024;
constexpr int kLinBoxRows = 32;                        // rows of one TMA box of codes
constexpr uint32_t kLinATile = kFp8Block * kFp8Block;  // bytes of one weight tile
constexpr uint32_t kLinBars = 8 * (2 * kLinMaxStages + 4 + 4 + 1);

struct LinTile {
  int e, nb, row0, rows;
  int n;  // rows of the product: `rows` rounded up to the 16 that an MMA takes
};

// The tiles of a launch: for each expert, its rows in spans of at most NT (as
// even as multiples of 16 allow), and for each span every output block.
// `first` [E + 1]: spans before expert e; `start` [E]: its first row; `count`
// [E]: its rows.  Tiles are walked in increasing order, so the expert is found
// by moving on from the last one.
struct LinTiles {
  const int *first, *start, *count;
  int E, nblk;
  int e = 0;
  __device__ __forceinline__ int total() const { return first[E] * nblk; }
  __device__ __forceinline__ LinTile at(int tile) {
    while (tile >= first[e + 1] * nblk) ++e;
    const int spans = first[e + 1] - first[e];
    const int local = tile - first[e] * nblk;
    LinTile t;
    t.e = e;
    t.nb = local / spans;
    const int per = ((count[e] + spans - 1) / spans + 15) & ~15;
    const int s = local % spans;
    t.row0 = start[e] + s * per;
    t.rows = min(per, count[e] - s * per);
    t.n = (t.rows + 15) & ~15;
    return t;
  }
};

// Swapped product: the weights are the MMA's 128-row operand and the rows of x
// its N, so that a tile takes any multiple of 16 rows and few rows cost few
// MMA cycles.  Accumulators: lane = output channel, column = row of x.
//
// Warp roles: warp 0 loads (weights as one 128 x 128-byte box that is already
// in the MMA's order, rows as boxes of 32 x 128 bytes), warp 1 owns TMEM and
// issues the MMAs, warps 2-5 write the scale words of each group of four
// 128-channel blocks into TMEM (every lane quarter holds a copy: warp % 4 is
// the quarter a warp can reach), warps 6-9 write the outputs.
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_fp8_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                      const LinArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const uint32_t bars = base + static_cast<uint32_t>(a.stages) * a.stage_bytes;
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

  if (threadIdx.x == 0) {
    prefetch_tmap(&tmap_x);
    prefetch_tmap(&tmap_w);
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sf_full + 8 * i, kLinScaleWarps);
      mbar_init(sf_empty + 8 * i, 1);
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, kLinEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), a.tmem_cols);
  grid_dependency_wait();
  grid_dependents_launch();  // only now: a kernel behind this one may rely on all that came before this one
  if (warp == 2) {
    // spans of each expert; offsets outside 0..M or decreasing are taken as empty or clipped
    int sum = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      int s = 0, c = 0;
      if (e < a.E) {
        s = a.offsets ? min(max(__ldcg(a.offsets + e), 0), a.M) : 0;
        c = a.offsets ? max(min(__ldcg(a.offsets + e + 1), a.M) - s, 0) : a.M;
        start[e] = s;
        count[e] = c;
      }
      int p = (c + a.NT - 1) / a.NT;
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, p, o);
        if (lane >= o) p += up;
      }
      if (e < a.E) first[e + 1] = sum + p;
      sum += __shfl_sync(0xFFFFFFFFu, p, 31);
    }
    if (lane == 0) first[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  LinTiles tiles{first, start, count, a.E, a.nblk};
  const int total = tiles.total();

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer
    uint32_t s = 0, p = 0, armed = 0, par = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const LinTile t = tiles.at(tile);
      const int boxes = (t.n + kLinBoxRows - 1) / kLinBoxRows;
      const uint32_t bytes = kLinATile + static_cast<uint32_t>(boxes) * (kLinBoxRows * 128u);
      const int wrow = (t.e * a.nblk + t.nb) * a.Kb;
      for (int kb = 0; kb < a.Kb; ++kb) {
        if (!mbar_wait(empty + 8 * s, p ^ 1, abort_flag, limit, kErrTimeoutProducer)) goto producer_done;
        const uint32_t dst = base + s * a.stage_bytes;
        mbar_arrive_expect_tx(full + 8 * s, bytes);
        if (check_bounds(bytes <= a.stage_bytes && wrow + kb < a.E * a.nblk * a.Kb && s < static_cast<uint32_t>(a.stages) &&
                         t.row0 >= 0 && t.row0 < a.M)) {
          tma_load_2d(dst, &tmap_w, full + 8 * s, 0, (wrow + kb) * kFp8Block);
          for (int i = 0; i < boxes; ++i)
            tma_load_2d(dst + kLinATile + i * (kLinBoxRows * 128), &tmap_x, full + 8 * s, kb * kFp8Block,
                        t.row0 + i * kLinBoxRows);
        }
        armed |= 1u << s;
        par = (par & ~(1u << s)) | (p << s);
        if (++s == static_cast<uint32_t>(a.stages)) { s = 0; p ^= 1; }
      }
    }
  producer_done:
    if (*abort_flag) {
      // let every copy counted on this CTA's barriers land before it exits
      int dummy = 0;
      for (int i = 0; i < a.stages; ++i)
        if (armed >> i & 1) mbar_wait(full + 8 * i, par >> i & 1, &dummy, limit, kErrTimeoutDrain);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // The whole warp runs the loop; lane 0 waits, one elected lane issues.
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
      int ok = 1;
      if (lane == 0) ok = mbar_wait(bar, parity, abort_flag, limit, kErrTimeoutMma);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      __syncwarp();
      tc_fence_after();
      return ok != 0;
    };
    uint32_t s = 0, p = 0, g = 0, gp = 0, c = 0, cp = 0;
    bool issued = false, ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const LinTile t = tiles.at(tile);
      const uint32_t d = tmem_base + c * a.acc_cols;
      if (!check_bounds(static_cast<uint32_t>(t.n) <= a.acc_cols) || !(ok = wait(acc_empty + 8 * c, cp ^ 1))) {
        ok = false;
        break;
      }
      for (int kb = 0; kb < a.Kb; ++kb) {
        if ((kb & 3) == 0 && !(ok = wait(sf_full + 8 * g, gp))) break;
        if (!(ok = wait(full + 8 * s, p))) break;
        const uint32_t st = base + s * a.stage_bytes;
        const uint64_t ad = sw128_kmajor_desc(st, 1024u), bd = sw128_kmajor_desc(st + kLinATile, 1024u);
        const uint32_t sf = tmem_base + a.sf_col + g * 8;
        const uint32_t idesc = idesc_mxf8(128, static_cast<uint32_t>(t.n), static_cast<uint32_t>(kb & 3));
        const int ks = kb == a.Kb - 1 ? a.last_ksteps : 4;
        if (elect_one()) {
          for (int j = 0; j < ks; ++j)  // 32 bytes of K = 2 units of the descriptors
            mma_mxf8(d, ad + 2 * j, bd + 2 * j, idesc, sf, sf + 4, (kb | j) != 0);
          mma_commit(empty + 8 * s);
          if ((kb & 3) == 3 || kb == a.Kb - 1) mma_commit(sf_empty + 8 * g);
          if (kb == a.Kb - 1) mma_commit(acc_full + 8 * c);
        }
        __syncwarp();
        issued = true;
        if (++s == static_cast<uint32_t>(a.stages)) { s = 0; p ^= 1; }
        if ((kb & 3) == 3 || kb == a.Kb - 1) {
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
      mma_commit(drain_bar);
      mbar_wait(drain_bar, 0, &dummy, limit, kErrTimeoutDrain);
    }
    __syncwarp();
  } else if (warp >= 2 && warp < 2 + kLinScaleWarps) {
    // -------------------------------------------------------------- scales
    // Group of four blocks: the weights' word (the same for all 128 channels)
    // into four columns, the rows' words into four: row 32 j + l at lane l of
    // column j.
    const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t g = 0, gp = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const LinTile t = tiles.at(tile);
      const uint32_t* const ws = a.w_scale + static_cast<int64_t>(t.e * a.nblk + t.nb) * a.kgroups;
      for (int kg = 0; kg < a.kgroups; ++kg) {
        uint32_t w[8];
        w[0] = w[1] = w[2] = w[3] = __ldcg(ws + kg);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = t.row0 + 32 * j + lane;
          w[4 + j] = 32 * j < t.n && row < a.M ? __ldcg(a.x_scale + static_cast<int64_t>(kg) * a.M + row) : 0x7F7F7F7Fu;
        }
        int got = 1;
        if (lane == 0) got = mbar_wait(sf_empty + 8 * g, gp ^ 1, abort_flag, limit, kErrTimeoutConvert);
        if (!(ok = __shfl_sync(0xFFFFFFFFu, got, 0) != 0)) break;
        __syncwarp();
        tc_fence_after();
        const uint32_t dst = tmem_base + quarter + a.sf_col + g * 8;
        tmem_st_x4(dst, w);
        tmem_st_x4(dst + 4, w + 4);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sf_full + 8 * g);
        g ^= 1;
        gp ^= g == 0;
      }
    }
  } else if (warp >= 2 + kLinScaleWarps) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    uint32_t c = 0, cp = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const LinTile t = tiles.at(tile);
      int got = 1;
      if (lane == 0) got = mbar_wait(acc_full + 8 * c, cp, abort_flag, limit, kErrTimeoutEpilogue);
      if (!__shfl_sync(0xFFFFFFFFu, got, 0)) break;
      __syncwarp();
      tc_fence_after();
      const int ch = t.nb * kFp8Block + q * 32 + lane;
      const float b = a.bias && ch < a.N ? __bfloat162float(a.bias[static_cast<int64_t>(t.e) * a.N + ch]) : 0.0f;
      const uint32_t src = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + c * a.acc_cols;
      for (int r0 = 0; r0 < t.rows; r0 += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(src + static_cast<uint32_t>(r0), v);
        tmem_ld_wait(v);
        if (ch < a.N) {
          __nv_bfloat16* dst = a.out + (t.row0 + r0) * a.ldo + ch;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (r0 + j < t.rows && check_bounds(t.row0 + r0 + j < a.M)) dst[j * a.ldo] = __float2bfloat16_rn(__uint_as_float(v[j]) + b);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + 8 * c);
      c ^= 1;
      cp ^= c == 0;
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem_base, a.tmem_cols);
  }
}

}  // namespace qvae
