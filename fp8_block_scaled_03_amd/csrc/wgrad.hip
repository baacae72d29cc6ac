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

#include <type_traits>

namespace fp8bs {

constexpr int WT = 32;  // rows (of dY and X): the depth of one bf16 MFMA

// LDS stage of one operand: WT rows of COLS bf16; the 32-byte chunk J of row r
// lies at chunk J ^ sw(r).  A transpose read takes 32 bytes of four rows per
// 16 lanes and of rows eight apart per neighbouring 16 lanes; sw puts these
// eight on different banks (a row of 64 columns has only four chunks: there the
// four rows lie on different banks).
__device__ __forceinline__ constexpr int wg_sw(int r, int cols) {
  return (r & 3) | (cols >= 128 ? ((r >> 3) & 1) << 2 : 0);
}

// A tile of BK = 16*MI*WK columns of X by BN = 16*NJ*WN columns of dY per
// workgroup of WK x WN waves; ring of S stages of R*WT rows.  The steps that load
// another whole stage have no branch between them: with few small tiles the loop's
// own instructions were most of the time (1 x 16384 x 1024 x 1024 with 64x64 128 us,
// 78 so, 68 with two times WT rows between the barriers).
template <int MI, int NJ, int WK, int WN, int S, int R>
__global__ void __launch_bounds__(64 * WK * WN) wgrad_kernel(const uint16_t* __restrict__ dy,
                                                             const uint16_t* __restrict__ x,
                                                             const int32_t* __restrict__ offsets,
                                                             float* __restrict__ dw, int accumulate, int64_t M,
                                                             int64_t N, int64_t K, uint32_t tiles_n,
                                                             uint32_t tiles_k) {
  constexpr int BK = 16 * MI * WK, BN = 16 * NJ * WN, WAVES = WK * WN;
  constexpr int RT = R * WT, X_BYTES = RT * BK * 2, STAGE = RT * (BK + BN) * 2;
  constexpr int X_PIECES = X_BYTES / 1024 / WAVES, Y_PIECES = RT * BN * 2 / 1024 / WAVES;
  static_assert(X_PIECES * WAVES * 1024 == X_BYTES && Y_PIECES * WAVES * 1024 == RT * BN * 2, "whole loads");
  static_assert(MI % 2 == 0 && BK >= 64 && BN >= 64, "the swizzle and the epilogue's pairs");
  constexpr int PIECES = X_PIECES + Y_PIECES;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];

  const int lane = threadIdx.x & 63;
  const int w = wave_id_uniform();
  const int wk = w / WN, wn = w % WN;
  const uint32_t per_group = tiles_n * tiles_k;
  // Range by range, each one's tiles over all XCDs: ranges differ in rows, and an
  // XCD with a run of long ones would finish last (16 uneven ranges of 32768 rows,
  // 4096 x 2048: 707 us with runs over all tiles, 519 so).
  const int gi = __builtin_amdgcn_readfirstlane(blockIdx.x / per_group);
  uint32_t tk, tn;
  band_walk(xcd_run(blockIdx.x - gi * per_group, per_group), tiles_k, tiles_n, tk, tn);
  int64_t begin, end;
  range_of(offsets, gi, M, begin, end);
  begin = uniform64(begin);
  end = uniform64(end);
  const int64_t k0 = (int64_t)__builtin_amdgcn_readfirstlane(tk) * BK;
  const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(tn) * BN;
  const int k_valid = (int)(K - k0 < BK ? K - k0 : BK), n_valid = (int)(N - n0 < BN ? N - n0 : BN);
  const int rows = (int)(end - begin);
  const int steps = (rows + RT - 1) / RT;
  dw += (int64_t)gi * N * K;

  // ---- direct loads: 16 bytes (eight columns) per lane; lane l of piece p fills
  // LDS bytes 1024 p + 16 l of the operand's stage, that is row R, chunk
  // position J; it loads chunk J ^ sw(R).  Columns past the matrix read its
  // last eight (never stored).
  auto source = [&](int p, int cols, int valid, int64_t ld, uint32_t& off, int& row) __attribute__((always_inline)) {
    const int byte = p * 1024 + lane * 16;
    row = byte / (cols * 2);
    const int chunk = (byte % (cols * 2)) / 32 ^ wg_sw(row, cols);
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

  // The load of step t into the slot at `at`.  LAST: it may be the last one, where rows
  // past the range read its last row; their LDS bytes are cleared before they are used.
  auto issue = [&](int t, uint32_t at, auto last) __attribute__((always_inline)) {
    const uint8_t* const xt = x0 + (int64_t)t * RT * K * 2;
    const uint8_t* const yt = y0 + (int64_t)t * RT * N * 2;
    const int left = rows - t * RT;
#pragma unroll
    for (int i = 0; i < X_PIECES; ++i) {
      uint32_t back = 0;
      if constexpr (decltype(last)::value) back = x_row[i] < left ? 0 : x_row[i] - left + 1;
      dma16_at(xt, x_off[i] - back * (uint32_t)(K * 2), ring + at + (w * X_PIECES + i) * 1024);
    }
#pragma unroll
    for (int i = 0; i < Y_PIECES; ++i) {
      uint32_t back = 0;
      if constexpr (decltype(last)::value) back = y_row[i] < left ? 0 : y_row[i] - left + 1;
      dma16_at(yt, y_off[i] - back * (uint32_t)(N * 2), ring + at + X_BYTES + (w * Y_PIECES + i) * 1024);
    }
  };
  auto clear_rows = [&](int t, uint32_t at) __attribute__((always_inline)) {
    const int left = rows - t * RT;
    unsigned char* const slot = smem + at;
    for (int b = left * BK * 2 + (int)threadIdx.x * 16; b < X_BYTES; b += 64 * WAVES * 16)
      *reinterpret_cast<v4i*>(slot + b) = v4i{0, 0, 0, 0};
    for (int b = left * BN * 2 + (int)threadIdx.x * 16; b < RT * BN * 2; b += 64 * WAVES * 16)
      *reinterpret_cast<v4i*>(slot + X_BYTES + b) = v4i{0, 0, 0, 0};
  };

  // ---- fragments.  Lane (g, r, c) = (lane >> 4, (lane >> 2) & 3, lane & 3) reads 8
  // bytes of row 8g + 4h + r (h = 0, 1), columns 4c.. of the sub-tile's 16; it
  // receives rows 8g + 4h .. + 3 of column lane & 15.  Both rows have the swizzle
  // of row 8g + r, so sub-tile J is at chunk J ^ that.
  const int tg = lane >> 4, tr = (lane >> 2) & 3, tc = lane & 3;
  auto frag = [&](const unsigned char* base, int cols, int J) __attribute__((always_inline)) -> v8bf {
    const unsigned char* const p = base + (8 * tg + tr) * cols * 2 + ((J ^ wg_sw(8 * tg + tr, cols)) << 5) + tc * 8;
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

  // All of a step's fragments are asked for before its first MFMA (4096 rows, 4096 x
  // 4096: 122 us, 134 in the compiler's order).
  auto multiply = [&](uint32_t at) __attribute__((always_inline)) {
    const unsigned char* const slot = smem + at;
    v8bf xf[R][MI], yf[R][NJ];
#pragma unroll
    for (int h = 0; h < R; ++h) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) yf[h][j] = frag(slot + X_BYTES + h * WT * BN * 2, BN, wn * NJ + j);
#pragma unroll
      for (int i = 0; i < MI; ++i) xf[h][i] = frag(slot + h * WT * BK * 2, BK, wk * MI + i);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < R; ++h)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[h][i], yf[h][j], acc[i][j], 0, 0, 0);
  };
  for (int t = 0; t < S - 1 && t < steps; ++t) issue(t, t * STAGE, std::true_type());
  uint32_t at = 0, before = (S - 1) * STAGE;
  int t = 0;
  auto step = [&](auto rest) __attribute__((always_inline)) {
    constexpr bool REST = decltype(rest)::value;
    if constexpr (REST) wait_steps<S - 2, PIECES>(steps - 1 - t);
    else wait_vmcnt<(S - 2) * PIECES>();  // step t has landed
    lds_barrier();                        // ... for every wave; step t-1's slot is free
    if (!REST || t + S - 1 < steps) issue(t + S - 1, before, rest);
    if (REST && t == steps - 1 && rows % RT) {
      clear_rows(t, at);
      lds_barrier();
    }
    multiply(at);
    before = at;
    at = at == (S - 1) * STAGE ? 0 : at + STAGE;
    ++t;
  };
  // the steps that load another whole one, then the rest
  const int whole = steps - (S - 1) - (rows % RT ? 1 : 0);
#pragma unroll 1
  while (t < whole) step(std::false_type());
#pragma unroll 1
  while (t < steps) step(std::true_type());

  // ---- lane (tg, lo) holds n = 16j + lo, k = 16i + 4 tg .. +3 of its wave's part: 64
  // bytes of 16 rows per store.  Lanes lo and lo ^ 8 exchange one of two
  // neighbouring sub-tiles i, so that a store covers 128 bytes of eight rows,
  // and whole lines leave with a non-temporal hint (nothing here reads them
  // again): 16 ranges of 512 rows, 4096 x 2048, 316 -> 228 us (the hint alone 251,
  // the exchange alone 310).
  if (accumulate && rows == 0) return;
  const int lo = lane & 15;
  const bool low = lo < 8;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
#pragma unroll
    for (int i = 0; i < MI; i += 2) {
      v4f mine[2];  // rows lo & 7 and 8 + (lo & 7) of sub-tile i (low lanes) or i + 1
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int give = __builtin_bit_cast(int, low ? acc[i + 1][j][e] : acc[i][j][e]);
        const float got = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, give, 0x128, 0xF, 0xF, true));
        mine[0][e] = low ? acc[i][j][e] : got;
        mine[1][e] = low ? got : acc[i + 1][j][e];
      }
      const int k = (wk * MI + i + (low ? 0 : 1)) * 16 + 4 * tg;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = (wn * NJ + j) * 16 + h * 8 + (lo & 7);
        if (n < n_valid && k < k_valid) {
          v4f* const p = reinterpret_cast<v4f*>(dw + (n0 + n) * K + k0 + k);
          v4f v = mine[h];
          if (accumulate) {
            const v4f old = *p;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = old[e] + v[e];
          }
          __builtin_nontemporal_store(v, p);
        }
      }
    }
  }
}

template <int MI, int NJ, int WK, int WN, int S, int R>
constexpr int wgrad_lds() {
  return S * R * WT * (16 * MI * WK + 16 * NJ * WN) * 2;
}

template <int MI, int NJ, int WK, int WN, int S, int R>
static hipError_t launch_wgrad_t(const void* dy, const void* x, const int32_t* offsets, int G, float* dw,
                                 bool accumulate, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  constexpr int BK = 16 * MI * WK, BN = 16 * NJ * WN, THREADS = 64 * WK * WN;
  const int64_t tiles_n = (N + BN - 1) / BN, tiles_k = (K + BK - 1) / BK;
  if (G * tiles_n * tiles_k > (int64_t)0xFFFFFFFF / THREADS) return hipErrorNotSupported;
  hipLaunchKernelGGL((wgrad_kernel<MI, NJ, WK, WN, S, R>), dim3((unsigned)(G * tiles_n * tiles_k)), dim3(THREADS),
                     (wgrad_lds<MI, NJ, WK, WN, S, R>()), stream, (const uint16_t*)dy, (const uint16_t*)x, offsets, dw,
                     accumulate ? 1 : 0, M, N, K, (uint32_t)tiles_n, (uint32_t)tiles_k);
  return hipGetLastError();
}

template <int MI, int NJ, int WK, int WN, int S, int R>
static hipError_t set_wgrad_t() {
  return hipFuncSetAttribute((const void*)wgrad_kernel<MI, NJ, WK, WN, S, R>,
                             hipFuncAttributeMaxDynamicSharedMemorySize, wgrad_lds<MI, NJ, WK, WN, S, R>());
}

hipError_t set_wgrad_attributes() {
  hipError_t e = set_wgrad_t<8, 4, 2, 2, 3, 1>();
  if (e == hipSuccess) e = set_wgrad_t<4, 4, 2, 4, 3, 1>();
  if (e == hipSuccess) e = set_wgrad_t<4, 4, 2, 2, 3, 1>();
  if (e == hipSuccess) e = set_wgrad_t<4, 4, 2, 2, 2, 1>();
  if (e == hipSuccess) e = set_wgrad_t<4, 2, 2, 2, 4, 1>();
  if (e == hipSuccess) e = set_wgrad_t<2, 2, 2, 2, 3, 2>();
  return e;
}

// The tile (columns of X x columns of dY) and the ring's depth.  Two or more
// workgroups per CU let one write its tile while others compute; long ranges gain
// from larger tiles and deeper rings, few tiles from smaller ones (ranges x rows
// each, N x K, us):
//   16 x 512, 4096 x 2048    256x128 (3 steps) 208   128x256 (3) 209   128x128 (2) 222
//   64 x 512, 2048 x 1024    256x128 (3) 232   128x256 (3) 239   128x128 (2) 242
//   64 x 128, 2048 x 1024    128x128 (2) 99    128x128 (3) 108   128x256 (3) 110
//   1 x 4096, 4096 x 4096    128x256 (3) 113   256x128 (3) 118   128x128 (3) 122
//   4 x 4096, 2048 x 2048    128x256 (3) 143   128x128 (3) 148   256x128 (3) 152
//   1 x 8192, 2048 x 2048    128x128 (3) 71    128x64 (4) 80
//   3 x 2300, 1200 x 896     128x128 (3) 31    128x64 (4) 32     64x64 34
//   1 x 16384, 1024 x 1024   64x64 66          128x64 (4) 118
hipError_t launch_grouped_wgrad(const void* dy, const void* x, const int32_t* offsets, int G, float* dw,
                                bool accumulate, int64_t M_total, int64_t N, int64_t K, hipStream_t stream) {
  const int64_t avg = M_total / G;  // rows per range
  auto tiles = [&](int64_t bk, int64_t bn) { return G * ((N + bn - 1) / bn) * ((K + bk - 1) / bk); };
  if (avg >= 400 && tiles(256, 128) >= 1024)
    return launch_wgrad_t<8, 4, 2, 2, 3, 1>(dy, x, offsets, G, dw, accumulate, M_total, N, K, stream);
  if (avg >= 400 && tiles(128, 256) >= 512)
    return launch_wgrad_t<4, 4, 2, 4, 3, 1>(dy, x, offsets, G, dw, accumulate, M_total, N, K, stream);
  if (tiles(128, 128) > (avg >= 400 ? 200 : 400)) {
    if (avg >= 400) return launch_wgrad_t<4, 4, 2, 2, 3, 1>(dy, x, offsets, G, dw, accumulate, M_total, N, K, stream);
    return launch_wgrad_t<4, 4, 2, 2, 2, 1>(dy, x, offsets, G, dw, accumulate, M_total, N, K, stream);
  }
  if (tiles(128, 64) > 256)
    return launch_wgrad_t<4, 2, 2, 2, 4, 1>(dy, x, offsets, G, dw, accumulate, M_total, N, K, stream);
  return launch_wgrad_t<2, 2, 2, 2, 3, 2>(dy, x, offsets, G, dw, accumulate, M_total, N, K, stream);
}

}  // namespace fp8bs
