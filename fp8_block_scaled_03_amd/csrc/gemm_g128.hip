// E4M3 GEMM with one fp32 scale per row and 128 K of A and one per 128x128
// block of the K-major weight, for one matrix and for ragged row groups.
//
//   C[i,j] = sum_kb sa[i,kb] sb[j/128,kb] P,  P = sum_{k in kb} A[i,k] Bt[j,k]
//
// A K-block of 128 is exactly the depth of v_mfma_f32_16x16x128_f8f6f4, the
// instruction with the full FP8 rate (its 32-deep relatives run at half of
// it), so P is one MFMA with a zero accumulator and the promotion is four fp32
// fmas per lane and 16x16x128 products: 16 VALU cycles beside 32 matrix
// cycles.  The instruction cuts small products (2^-13 below the largest of
// their group of eight); the cut is below the bf16 rounding of C and is not
// carried along K, because the sum over K-blocks is the fp32 accumulator's.
//
// Every kernel here runs the same sequence per element - the same MFMA operands,
// s = RN(sa * sb), acc = fma(P, s, acc), kb ascending - so a row's result does
// not depend on M, on its place or on the kernel.
//
// Operand layout of the instruction (lane l, g = l >> 4): lane l holds row
// (l & 15) of the 16-row operand, bytes 0-15 = K [16g, 16g+16) and bytes
// 16-31 = K [64+16g, 64+16g+16).  The first operand is the weight, so a lane's
// four results are four columns of one row of C.
#include "common.hpp"
#include "launch_g128.hpp"
#include "ragged.hpp"

namespace fp8bs {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float v2f_t __attribute__((ext_vector_type(2)));

constexpr int GK = 128;        // K-block = K step = bytes of one staged row
constexpr int SCH = 8;         // K-blocks per staged chunk of A's scales

// 16 zero bytes that stand for K past the end of a row
__device__ const uint4 g128_zeros = {0, 0, 0, 0};

// P of one K-block for a 16x16 output sub-tile (w: weight rows, x: A rows).
__device__ __forceinline__ v4f mfma_block(v8i_t w, v8i_t x) {
  const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, z, 0, 0, 0, 0, 0, 0);
}

// Two accumulators -> two bf16 (nearest even, NaN kept), a zero stored as +0.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const v2f_t v = {lo + 0.0f, hi + 0.0f};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2bf));
}

// Direct global->LDS load of 16 bytes per lane from a uniform base plus a
// 32-bit offset per lane.
__device__ __forceinline__ void dma16_at(const uint8_t* base, uint32_t off, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds_base), "v"(off), "s"(base)
               : "memory");
}

// A tile of BM = 16*MI*WM rows by BN = 16*NJ*WN columns per workgroup of
// WM x WN waves; wave (wm, wn) owns MI x NJ sub-tiles of 16x16.  A and Bt are
// streamed as bytes into a ring of two 128-deep steps in LDS with direct loads,
// a step ahead; row r of a stage holds its 128 bytes with 16-byte piece p at
// position p ^ (r & 7), which spreads a fragment read over all banks.  A's
// scales of eight K-blocks at a time are loaded to registers, then placed in LDS
// in the order in which a lane needs them (its MI sub-tile rows side by side).
// A weight scale is one value per wave and step: lane l holds the one of step
// 64c + l.
template <int MI, int NJ, int WM, int WN, bool GROUPED>
__global__ void __launch_bounds__(64 * WM * WN) gemm_g128_tile_kernel(
    const uint8_t* __restrict__ a, const float* __restrict__ sa, const uint8_t* __restrict__ bt,
    const float* __restrict__ sbt, const int32_t* __restrict__ offsets, int G, uint16_t* __restrict__ c, int64_t M,
    int64_t N, int64_t K, uint32_t tiles_n) {
  constexpr int BM = 16 * MI * WM, BN = 16 * NJ * WN, WAVES = WM * WN, THREADS = 64 * WAVES;
  constexpr int STAGE = (BM + BN) * GK;
  constexpr int A_PIECES = BM / 8 / WAVES, B_PIECES = BN / 8 / WAVES;  // 1 KB loads per wave and step
  constexpr int S_ITEMS = (2 * BM + THREADS - 1) / THREADS;            // half chunks of one row per thread
  static_assert(A_PIECES * 8 * WAVES == BM && B_PIECES * 8 * WAVES == BN, "tile is a whole number of loads");
  static_assert(NJ * 16 <= 128 && 128 % (NJ * 16) == 0, "a wave's columns lie in one weight block");
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  float* const s_lds = reinterpret_cast<float*>(smem + 2 * STAGE);     // [2][SCH][BM]

  const int lane = threadIdx.x & 63;
  const int w = wave_id_uniform();
  // the waves of one SIMD (w, w + 4) lie in different row bands, so a tile with
  // few rows still uses every SIMD
  const int wm = w / WN, wn = w % WN;
  const int g = lane >> 4, lo = lane & 15;

  TileAt t;
  if constexpr (GROUPED) {
    if (!find_tile<BM>(offsets, G, M, tiles_n, blockIdx.x, t)) return;
    bt += (int64_t)t.group * N * K;
    sbt += (int64_t)t.group * ((N + 127) >> 7) * ((K + 127) >> 7);
  } else {
    dense_tile<BM>(M, tiles_n, blockIdx.x, gridDim.x, t);
  }
  const int64_t row0 = t.row0, col0 = (int64_t)t.tn * BN;
  const int m_valid = (int)(t.row_end - row0 < BM ? t.row_end - row0 : BM);
  const int n_valid = (int)(N - col0 < BN ? N - col0 : BN);
  const int KB = (int)((K + 127) >> 7);
  const bool wave_live = wm * 16 * MI < m_valid && wn * 16 * NJ < n_valid;

  // ---- direct loads: piece i of a wave is rows 8p .. 8p+7, p = w*PIECES + i;
  // lane l loads row 8p + (l >> 3), 16-byte piece (l & 7) ^ (row & 7).  Rows past
  // the range read its last row (never stored).
  const int piece = (lane & 7) ^ (lane >> 3);
  uint32_t a_off[A_PIECES], b_off[B_PIECES];
#pragma unroll
  for (int i = 0; i < A_PIECES; ++i) {
    int r = 8 * (w * A_PIECES + i) + (lane >> 3);
    r = r < m_valid ? r : m_valid - 1;
    a_off[i] = (uint32_t)r * (uint32_t)K + piece * 16;
  }
#pragma unroll
  for (int i = 0; i < B_PIECES; ++i) {
    int r = 8 * (w * B_PIECES + i) + (lane >> 3);
    r = r < n_valid ? r : n_valid - 1;
    b_off[i] = (uint32_t)r * (uint32_t)K + piece * 16;
  }
  const uint8_t* const a0 = uniform_ptr(a + row0 * K);
  const uint8_t* const b0 = uniform_ptr(bt + col0 * K);
  typedef __attribute__((address_space(3))) unsigned char lds_u8;
  const uint32_t ring = (uint32_t)(uintptr_t)((lds_u8*)smem);

  auto issue = [&](int ks) __attribute__((always_inline)) {
    const uint32_t slot = ring + (ks & 1) * STAGE;
    const uint8_t* const ak = a0 + (int64_t)ks * GK;
    const uint8_t* const bk = b0 + (int64_t)ks * GK;
    if ((int64_t)(ks + 1) * GK <= K) {
#pragma unroll
      for (int i = 0; i < A_PIECES; ++i) dma16_at(ak, a_off[i], slot + (w * A_PIECES + i) * 1024);
#pragma unroll
      for (int i = 0; i < B_PIECES; ++i) dma16_at(bk, b_off[i], slot + BM * GK + (w * B_PIECES + i) * 1024);
    } else {
      // the partial last K-block: pieces past K are zeros
      const bool in = (int64_t)ks * GK + piece * 16 < K;
      const uint8_t* const zero = reinterpret_cast<const uint8_t*>(&g128_zeros);
#pragma unroll
      for (int i = 0; i < A_PIECES; ++i) dma16(in ? ak + a_off[i] : zero, slot + (w * A_PIECES + i) * 1024);
#pragma unroll
      for (int i = 0; i < B_PIECES; ++i)
        dma16(in ? bk + b_off[i] : zero, slot + BM * GK + (w * B_PIECES + i) * 1024);
    }
  };

  // ---- A's scales: item = (row, half of the chunk), four K-blocks each
  float s_reg[S_ITEMS][4];
  auto load_scales = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < S_ITEMS; ++n) {
      const int item = n * THREADS + threadIdx.x;
      int r = (item >> 1) < m_valid ? item >> 1 : m_valid - 1;
      const float* const p = sa + (row0 + r) * KB;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int kb = chunk * SCH + (item & 1) * 4 + x;
        s_reg[n][x] = p[kb < KB ? kb : KB - 1];
      }
    }
  };
  auto place_scales = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < S_ITEMS; ++n) {
      const int item = n * THREADS + threadIdx.x;
      const int r = item >> 1;
      if (S_ITEMS * THREADS == 2 * BM || r < BM) {
        // row r = 16*MI*band + 16*i + lane -> [band][lane][i]
        const int at = r / (16 * MI) * (16 * MI) + (r & 15) * MI + (r % (16 * MI)) / 16;
        float* const p = s_lds + ((chunk & 1) * SCH + (item & 1) * 4) * BM + at;
#pragma unroll
        for (int x = 0; x < 4; ++x) p[x * BM] = s_reg[n][x];
      }
    }
  };
  const int64_t nb = (col0 + wn * 16 * NJ) >> 7;
  const float* const sb_row = sbt + (nb < ((N + 127) >> 7) ? nb : 0) * KB;
  auto load_sb = [&](int ks) __attribute__((always_inline)) {
    return sb_row[ks + lane < KB ? ks + lane : KB - 1];
  };

  v4f acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  auto frag = [&](const unsigned char* base, int r) __attribute__((always_inline)) -> v8i_t {
    const v4i p0 = *reinterpret_cast<const v4i*>(base + r * GK + 16 * (g ^ (lo & 7)));
    const v4i p1 = *reinterpret_cast<const v4i*>(base + r * GK + 16 * ((4 + g) ^ (lo & 7)));
    return v8i_t{p0[0], p0[1], p0[2], p0[3], p1[0], p1[1], p1[2], p1[3]};
  };

  float sb_now = 0.0f, sb_next = 0.0f;
  if (KB > 0) {
    load_scales(0);
    sb_now = load_sb(0);
    place_scales(0);
    issue(0);
  }
  for (int ks = 0; ks < KB; ++ks) {
    wait_vmcnt<0>();  // step ks has landed
    if ((ks & 7) == 4 && ks + 4 < KB) place_scales((ks >> 3) + 1);
    lds_barrier();    // ... for every wave; step ks-1's slot is free
    if ((ks & 7) == 0) {
      if ((ks & 63) == 0 && ks > 0) sb_now = sb_next;
      if (ks + 8 < KB) load_scales((ks >> 3) + 1);
      if ((ks & 63) == 56) sb_next = load_sb(ks + 8);
    }
    if (ks + 1 < KB) issue(ks + 1);
    if (wave_live) {
      const unsigned char* const slot = smem + (ks & 1) * STAGE;
      const float* const sp = s_lds + (((ks >> 3) & 1) * SCH + (ks & 7)) * BM + wm * 16 * MI + lo * MI;
      const float sb = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sb_now), ks & 63));
      float sc[MI];
#pragma unroll
      for (int i = 0; i < MI; ++i) sc[i] = sp[i] * sb;
      v8i_t bf[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) bf[j] = frag(slot + BM * GK, wn * 16 * NJ + 16 * j + lo);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const v8i_t af = frag(slot, wm * 16 * MI + 16 * i + lo);
        v4f p[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) p[j] = mfma_block(bf[j], af);
#pragma unroll
        for (int j = 0; j < NJ; ++j) promote(acc[i][j], p[j], sc[i]);
      }
    }
  }

  // ---- epilogue: lane holds row 16i + lo, columns 16j + 4g .. +3 of its wave
  if (!wave_live) return;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int r = wm * 16 * MI + 16 * i + lo;
    if (r < m_valid) {
      uint16_t* const cr = c + (row0 + r) * N + col0;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int col = wn * 16 * NJ + 16 * j + 4 * g;
        if (col < n_valid)
          *reinterpret_cast<uint2*>(cr + col) =
              make_uint2(bf16_pair(acc[i][j][0], acc[i][j][1]), bf16_pair(acc[i][j][2], acc[i][j][3]));
      }
    }
  }
}

template <int MI, int NJ, int WM, int WN>
constexpr int tile_lds() {
  return 2 * (16 * MI * WM + 16 * NJ * WN) * GK + 2 * SCH * 16 * MI * WM * 4;
}

template <int MI, int NJ, int WM, int WN>
static hipError_t set_tile_attributes() {
  hipError_t e = hipFuncSetAttribute((const void*)gemm_g128_tile_kernel<MI, NJ, WM, WN, false>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, tile_lds<MI, NJ, WM, WN>());
  if (e != hipSuccess) return e;
  return hipFuncSetAttribute((const void*)gemm_g128_tile_kernel<MI, NJ, WM, WN, true>,
                             hipFuncAttributeMaxDynamicSharedMemorySize, tile_lds<MI, NJ, WM, WN>());
}

template <int MI, int NJ, int WM, int WN>
static hipError_t launch_tile(const void* a, const float* sa, const void* bt, const float* sbt,
                              const int32_t* offsets, int G, void* c, int64_t M, int64_t N, int64_t K,
                              hipStream_t stream) {
  constexpr int BM = 16 * MI * WM, BN = 16 * NJ * WN, THREADS = 64 * WM * WN;
  const int64_t tiles_n = (N + BN - 1) / BN;
  // each range adds at most one partial tile
  const int64_t tiles_m = offsets ? (M + BM - 1) / BM + (G < M ? G : M) : (M + BM - 1) / BM;
  if (tiles_m * tiles_n > (int64_t)0xFFFFFFFF / THREADS) return hipErrorNotSupported;
  const dim3 grid((unsigned)(tiles_m * tiles_n));
  if (offsets)
    hipLaunchKernelGGL((gemm_g128_tile_kernel<MI, NJ, WM, WN, true>), grid, dim3(THREADS),
                       (tile_lds<MI, NJ, WM, WN>()), stream, (const uint8_t*)a, sa, (const uint8_t*)bt, sbt, offsets,
                       G, (uint16_t*)c, M, N, K, (uint32_t)tiles_n);
  else
    hipLaunchKernelGGL((gemm_g128_tile_kernel<MI, NJ, WM, WN, false>), grid, dim3(THREADS),
                       (tile_lds<MI, NJ, WM, WN>()), stream, (const uint8_t*)a, sa, (const uint8_t*)bt, sbt, offsets,
                       G, (uint16_t*)c, M, N, K, (uint32_t)tiles_n);
  return hipGetLastError();
}

hipError_t set_gemm_g128_attributes() {
  hipError_t e = set_tile_attributes<8, 4, 2, 4>();
  if (e == hipSuccess) e = set_tile_attributes<4, 4, 2, 2>();
  if (e == hipSuccess) e = set_tile_attributes<2, 2, 2, 2>();
  return e;
}

hipError_t launch_gemm_g128(const void* a, const float* sa, const void* bt, const float* sbt, const int32_t* offsets,
                            int G, void* c, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  const int64_t avg = (M + G - 1) / G;  // rows per range
  auto tiles = [&](int64_t b) { return G * ((avg + b - 1) / b) * ((N + b - 1) / b); };
  if (tiles(256) >= 256) return launch_tile<8, 4, 2, 4>(a, sa, bt, sbt, offsets, G, c, M, N, K, stream);
  if (tiles(128) >= 256) return launch_tile<4, 4, 2, 2>(a, sa, bt, sbt, offsets, G, c, M, N, K, stream);
  return launch_tile<2, 2, 2, 2>(a, sa, bt, sbt, offsets, G, c, M, N, K, stream);
}

}  // namespace fp8bs
