// Weight gradients of a grouped product: dW_g[n,k] (+)= sum over the rows m of
// range g of dY[m,n] X[m,k], bf16 operands, fp32 accumulation and result.
//
// Both operands are walked along their slow axis, so a fragment (eight rows of
// one column per lane) comes from the LDS transpose read ds_read_b64_tr_b16.
// The first MFMA operand is X, so a lane's four results are four neighbouring k
// of one n and dW is written 16 bytes at a time.
//
// Bound: with R rows per range, 2RNK flops at the bf16 MFMA rate against 4NK bytes
// written (8NK moved when accumulating); below about 1000 rows per range the
// writes of dW are the larger part.
#include "common.hpp"
#include "launch_g128.hpp"
#include "ragged.hpp"

namespace fp8bs {

constexpr int WT = 32;  // rows (of dY and X) per step: the depth of one bf16 MFMA

__device__ const uint4 wgrad_zeros = {0, 0, 0, 0};

// LDS stage of one operand: WT rows of COLS bf16; the 32-byte chunk J of row r
// lies at chunk J ^ sw(r).  A transpose read takes 32 bytes of four rows per
// 16 lanes and of rows eight apart per neighbouring 16 lanes; sw puts these
// eight on different banks.
__device__ __forceinline__ int wg_sw(int r) { return (r & 3) | ((r >> 3) & 1) << 2; }

// A tile of BK = 16*MI*WK columns of X by BN = 16*NJ*WN columns of dY per
// workgroup of WK x WN waves; ring of S stages of WT rows.
template <int MI, int NJ, int WK, int WN, int S>
__global__ void __launch_bounds__(64 * WK * WN) wgrad_kernel(const uint16_t* __restrict__ dy,
                                                             const uint16_t* __restrict__ x,
                                                             const int32_t* __restrict__ offsets,
                                                             float* __restrict__ dw, int accumulate, int64_t M,
                                                             int64_t N, int64_t K, uint32_t tiles_n,
                                                             uint32_t tiles_k) {
  constexpr int BK = 16 * MI * WK, BN = 16 * NJ * WN, WAVES = WK * WN;
  constexpr int X_BYTES = WT * BK * 2, STAGE = WT * (BK + BN) * 2;
  constexpr int X_PIECES = X_BYTES / 1024 / WAVES, Y_PIECES = WT * BN * 2 / 1024 / WAVES;
  static_assert(X_PIECES * WAVES * 1024 == X_BYTES && Y_PIECES * WAVES * 1024 == WT * BN * 2, "whole loads");
  constexpr int PIECES = X_PIECES + Y_PIECES;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];

  const int lane = threadIdx.x & 63;
  const int w = wave_id_uniform();
  const int wk = w / WN, wn = w % WN;
  const uint32_t per_group = tiles_n * tiles_k;
  const uint32_t lin = xcd_run(blockIdx.x, gridDim.x);
  const int gi = __builtin_amdgcn_readfirstlane(lin / per_group);
  uint32_t tk, tn;
  band_walk(lin - gi * per_group, tiles_k, tiles_n, tk, tn);
  int64_t begin, end;
  range_of(offsets, gi, M, begin, end);
  begin = uniform64(begin);
  end = uniform64(end);
  const int64_t k0 = (int64_t)__builtin_amdgcn_readfirstlane(tk) * BK;
  const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(tn) * BN;
  const int k_valid = (int)(K - k0 < BK ? K - k0 : BK), n_valid = (int)(N - n0 < BN ? N - n0 : BN);
  const int rows = (int)(end - begin);
  const int steps = (rows + WT - 1) / WT;
  dw += (int64_t)gi * N * K;

  // ---- direct loads: 16 bytes (eight columns) per lane; lane l of piece p fills
  // LDS bytes 1024 p + 16 l of the operand's stage, that is row R, chunk
  // position J; it loads chunk J ^ sw(R).  Columns past the matrix read its
  // last eight (never stored).
  auto source = [&](int p, int cols, int valid, int64_t ld, uint32_t& off, int& row) __attribute__((always_inline)) {
    const int byte = p * 1024 + lane * 16;
    row = byte / (cols * 2);
    const int chunk = (byte % (cols * 2)) / 32 ^ wg_sw(row);
    int col = chunk * 16 + (lane & 1) * 8;
    col = col < valid ? col : valid - 8;
    off = (uint32_t)row * (uint32_t)(ld * 2) + col * 2;
  };
  uint32_t x_off[X_PIECES], y_off[Y_PIECES];
  int x_row[X_PIECES], y_row[Y_PIECES];
#pragma unroll
  for (int i = 0; i < X_PIECES; ++i) source(w * X_PIECES + i, BK, k_valid, K, x_off[i], x_row[i]);
#pragma unroll
  for (int i = 0; i < Y_PIECES; ++i) source(w * Y_PIECES + i, BN, n_valid, N, y_off[i], y_row[i]);
  const uint8_t* const x0 = uniform_ptr(reinterpret_cast<const uint8_t*>(x + begin * K + k0));
  const uint8_t* const y0 = uniform_ptr(reinterpret_cast<const uint8_t*>(dy + begin * N + n0));
  typedef __attribute__((address_space(3))) unsigned char lds_u8;
  const uint32_t ring = (uint32_t)(uintptr_t)((lds_u8*)smem);

  auto dma_at = [](const uint8_t* base, uint32_t off, uint32_t lds_base) __attribute__((always_inline)) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds_base), "v"(off), "s"(base)
                 : "memory");
  };
  // Steps past the last one load zeros into a slot that is never read, so that
  // every wave always has the same number of loads in flight.
  auto issue = [&](int t) __attribute__((always_inline)) {
    const uint32_t slot = ring + (t % S) * STAGE;
    const uint8_t* const xt = x0 + (int64_t)t * WT * K * 2;
    const uint8_t* const yt = y0 + (int64_t)t * WT * N * 2;
    const int left = rows - t * WT;
    if (left >= WT) {
#pragma unroll
      for (int i = 0; i < X_PIECES; ++i) dma_at(xt, x_off[i], slot + (w * X_PIECES + i) * 1024);
#pragma unroll
      for (int i = 0; i < Y_PIECES; ++i) dma_at(yt, y_off[i], slot + X_BYTES + (w * Y_PIECES + i) * 1024);
    } else {
      // rows past the range are zeros
      const uint8_t* const zero = reinterpret_cast<const uint8_t*>(&wgrad_zeros);
#pragma unroll
      for (int i = 0; i < X_PIECES; ++i)
        dma16(x_row[i] < left ? xt + x_off[i] : zero, slot + (w * X_PIECES + i) * 1024);
#pragma unroll
      for (int i = 0; i < Y_PIECES; ++i)
        dma16(y_row[i] < left ? yt + y_off[i] : zero, slot + X_BYTES + (w * Y_PIECES + i) * 1024);
    }
  };

  // ---- fragments.  Lane (g, r, c) = (lane >> 4, (lane >> 2) & 3, lane & 3) reads 8
  // bytes of row 8g + 4h + r (h = 0, 1), columns 4c.. of the sub-tile's 16; it
  // receives rows 8g + 4h .. + 3 of column lane & 15.  The row's swizzle is
  // r | (g & 1) << 2 for both h, so sub-tile J is at chunk J ^ that.
  const int tg = lane >> 4, tr = (lane >> 2) & 3, tc = lane & 3;
  const int sw = tr | (tg & 1) << 2;
  auto frag = [&](const unsigned char* base, int cols, int J) __attribute__((always_inline)) -> v8bf {
    const unsigned char* const p = base + (8 * tg + tr) * cols * 2 + ((J ^ sw) << 5) + tc * 8;
    const v4s h0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)(p));
    const v4s h1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)(p + 4 * cols * 2));
    const v2i a = __builtin_bit_cast(v2i, h0), b = __builtin_bit_cast(v2i, h1);
    return __builtin_bit_cast(v8bf, v4i{a[0], a[1], b[0], b[1]});
  };

  v4f acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  if (steps > 0) {
#pragma unroll
    for (int t = 0; t < S - 1; ++t) issue(t);
  }
  for (int t = 0; t < steps; ++t) {
    wait_vmcnt<PIECES*(S - 2)>();  // step t has landed
    lds_barrier();                 // ... for every wave; step t-1's slot is free
    issue(t + S - 1);
    const unsigned char* const slot = smem + (t % S) * STAGE;
    v8bf yf[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) yf[j] = frag(slot + X_BYTES, BN, wn * NJ + j);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const v8bf xf = frag(slot, BK, wk * MI + i);
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, yf[j], acc[i][j], 0, 0, 0);
    }
  }
  wait_vmcnt<0>();

  // ---- lane holds n = 16j + (lane & 15), k = 16i + 4g .. +3 of its wave's part
  if (accumulate && rows == 0) return;
  const int lo = lane & 15;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int n = (wn * NJ + j) * 16 + lo;
    if (n < n_valid) {
      float* const row = dw + (n0 + n) * K + k0;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int k = (wk * MI + i) * 16 + 4 * tg;
        if (k < k_valid) {
          v4f* const p = reinterpret_cast<v4f*>(row + k);
          v4f v = acc[i][j];
          if (accumulate) {
            const v4f old = *p;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = old[e] + v[e];
          }
          *p = v;
        }
      }
    }
  }
}

template <int MI, int NJ, int WK, int WN, int S>
constexpr int wgrad_lds() {
  return S * WT * (16 * MI * WK + 16 * NJ * WN) * 2;
}

template <int MI, int NJ, int WK, int WN, int S>
static hipError_t launch_wgrad_t(const void* dy, const void* x, const int32_t* offsets, int G, float* dw,
                                 bool accumulate, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  constexpr int BK = 16 * MI * WK, BN = 16 * NJ * WN, THREADS = 64 * WK * WN;
  const int64_t tiles_n = (N + BN - 1) / BN, tiles_k = (K + BK - 1) / BK;
  if (G * tiles_n * tiles_k > (int64_t)0xFFFFFFFF / THREADS) return hipErrorNotSupported;
  hipLaunchKernelGGL((wgrad_kernel<MI, NJ, WK, WN, S>), dim3((unsigned)(G * tiles_n * tiles_k)), dim3(THREADS),
                     (wgrad_lds<MI, NJ, WK, WN, S>()), stream, (const uint16_t*)dy, (const uint16_t*)x, offsets, dw,
                     accumulate ? 1 : 0, M, N, K, (uint32_t)tiles_n, (uint32_t)tiles_k);
  return hipGetLastError();
}

hipError_t set_wgrad_attributes() {
  hipError_t e = hipFuncSetAttribute((const void*)wgrad_kernel<8, 4, 2, 4, 4>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, wgrad_lds<8, 4, 2, 4, 4>());
  if (e != hipSuccess) return e;
  return hipFuncSetAttribute((const void*)wgrad_kernel<4, 4, 2, 2, 4>, hipFuncAttributeMaxDynamicSharedMemorySize,
                             wgrad_lds<4, 4, 2, 2, 4>());
}

hipError_t launch_grouped_wgrad(const void* dy, const void* x, const int32_t* offsets, int G, float* dw,
                                bool accumulate, int64_t M_total, int64_t N, int64_t K, hipStream_t stream) {
  const int64_t big = G * ((N + 255) / 256) * ((K + 255) / 256);
  if (big >= 512) return launch_wgrad_t<8, 4, 2, 4, 4>(dy, x, offsets, G, dw, accumulate, M_total, N, K, stream);
  return launch_wgrad_t<4, 4, 2, 2, 4>(dy, x, offsets, G, dw, accumulate, M_total, N, K, stream);
}

}  // namespace fp8bs
