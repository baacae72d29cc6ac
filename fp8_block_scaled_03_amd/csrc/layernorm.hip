// Residual add + layer norm + the row quantizer of 128 values, and the backward pass.
//
//   h = bf16(x + r),  mu = sum h / d,  var = sum (h - mu)^2 / d,  rstd = 1 / sqrt(var + eps)
//   y = (h - mu) rstd gamma + beta;  codes and scales of the fp32 y, 128 columns each
//
// A row stays in registers between the sums (packed bf16), so x and the residual are
// read once.  mu is summed in 64 bits over the lanes (a lane's 8 to 32 values of eight bits in 32 bits,
// which lose next to nothing) and held as m, mu rounded to fp32, and the rest delta, so that a row
// far from zero (|mu| >> sigma) keeps its digits: the deviation is (h - m) - delta, var =
// sum (h - m)^2 / d - delta^2.  (delta as the fp32 sum of h - m is no better than m alone: the differences
// of a binade are all rounded by the same bits of m, and the mean was off by 0.3 to 0.5 x 2^-24
// sigma on ordinary rows.)
//
//   backward, with xh = (h - mean) rstd and g = dy gamma:
//   dx = rstd (g - sum g / d - xh sum (g xh) / d) [+ the residual stream's gradient]
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Row mapping: WPR waves hold a row, lane l of wave k the columns
// 512 (WPR i + k) + 8 l .. +7, i < NL <= 4: 16 lanes hold a group of 128.  Sums run
// over a lane's columns in order, over lanes by a butterfly, over waves in order: a
// row's results depend on that row and on d only, so the mapping goes by d.  Forward a row
// has up to eight waves before a lane has a second piece: few rows are latency (us with
// twice to four times the pieces, and so: 8 x 8192 6.5 and 4.9, 8 x 2048 5.7 and 3.8, 512 x 4096 7.4
// and 5.6; but 32768 x 1024 40.2 and 41.3).  Sixteen waves are slower (8192 x 8192 95, not 83).
//
// dgamma and dbeta: a workgroup walks every gridDim.x-th set of rows and keeps
// its columns' sums in registers, joins its rows' sums in LDS and writes them once
// to the workspace; a second launch adds the workgroups' sums in order.  The
// grid depends on the sizes only, so results are the same bits every time.
//
// Bound by HBM traffic: forward 7 bytes a value (9 with y; 8192 x 8192 93 us, 6.5 TB/s), backward
// 6 (8; 97 us, 5.6 TB/s); few rows by a launch and one chain of loads and sums (8 x 8192 4.3 us in a graph).
#include "column_sum.hpp"
#include "launch_layer.hpp"
#include "quant_g128.hpp"
#include "stream.hpp"

#include <type_traits>

namespace fp8bs {

constexpr int LN_NL = 4, LN_MAX_WPR = 8;

// Sum over the lanes of a wave, in every lane: turns within 16 lanes, then the two exchanges
// of rows of 16 and of halves (through LDS, as __shfl_xor goes, 8 x 8192 takes 0.4 us more).
__device__ __forceinline__ float wave_sum(float v) {
  auto turned = [](float x, auto by) __attribute__((always_inline)) {
    constexpr int ROW_ROR = 0x120 + decltype(by)::value;
    return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ROW_ROR, 0xF, 0xF,
                                                                     true));
  };
  v = turned(v, std::integral_constant<int, 8>());
  v = turned(v, std::integral_constant<int, 4>());
  v = turned(v, std::integral_constant<int, 2>());
  v = turned(v, std::integral_constant<int, 1>());
  auto both = [](auto pair) __attribute__((always_inline)) {
    const uint32_t a = pair[0], b = pair[1];
    return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
  };
  uint32_t x = __builtin_bit_cast(uint32_t, v);
  v = both(__builtin_amdgcn_permlane16_swap(x, x, false, false));
  x = __builtin_bit_cast(uint32_t, v);
  return both(__builtin_amdgcn_permlane32_swap(x, x, false, false));
}

// The same of 64-bit values: 32 bits at a time through the exchanges.
__device__ __forceinline__ double wave_sum(double v) {
  typedef uint32_t v2u __attribute__((ext_vector_type(2)));
  auto turned = [](double x, auto by) __attribute__((always_inline)) {
    constexpr int ROW_ROR = 0x120 + decltype(by)::value;
    const v2u w = __builtin_bit_cast(v2u, x);
    const v2u t = {(uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[0], ROW_ROR, 0xF, 0xF, true),
                   (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[1], ROW_ROR, 0xF, 0xF, true)};
    return x + __builtin_bit_cast(double, t);
  };
  v = turned(v, std::integral_constant<int, 8>());
  v = turned(v, std::integral_constant<int, 4>());
  v = turned(v, std::integral_constant<int, 2>());
  v = turned(v, std::integral_constant<int, 1>());
  auto both = [](auto low, auto high) __attribute__((always_inline)) {
    const v2u a = {low[0], high[0]}, b = {low[1], high[1]};
    return __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b);
  };
  v2u w = __builtin_bit_cast(v2u, v);
  v = both(__builtin_amdgcn_permlane16_swap(w[0], w[0], false, false),
           __builtin_amdgcn_permlane16_swap(w[1], w[1], false, false));
  w = __builtin_bit_cast(v2u, v);
  return both(__builtin_amdgcn_permlane32_swap(w[0], w[0], false, false),
              __builtin_amdgcn_permlane32_swap(w[1], w[1], false, false));
}

// A sum over a row's WPR waves, of which this is one, wave w of the workgroup; `lds` is not in
// use by another sum since the last barrier but one.
template <int WPR, typename T>
__device__ __forceinline__ T row_sum(T a, int w, T* lds) {
  a = wave_sum(a);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) lds[w] = a;
    __syncthreads();
    const int first = w & ~(WPR - 1);
    a = lds[first];
#pragma unroll
    for (int k = 1; k < WPR; ++k) a += lds[first + k];
  }
  return a;
}

// Two sums.
template <int WPR>
__device__ __forceinline__ void row_sums(float& a, float& b, int w, float (*lds)[2]) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) {
      lds[w][0] = a;
      lds[w][1] = b;
    }
    __syncthreads();
    const int first = w & ~(WPR - 1);
    a = lds[first][0];
    b = lds[first][1];
#pragma unroll
    for (int k = 1; k < WPR; ++k) {
      a += lds[first + k][0];
      b += lds[first + k][1];
    }
  }
}

struct LayerNorm {
  const uint16_t *x, *res, *gamma, *beta;
  uint16_t *h, *y;
  uint8_t* q;
  float *scales, *mean, *rstd;
  int64_t rows, d;
  double inv_d;
  float eps;
};

template <int NL, int WPR, bool LINES, bool PAST>
__global__ void __launch_bounds__(WPR == 8 ? 512 : 256) layernorm_kernel(LayerNorm p, uint32_t sets) {
  constexpr int WAVES = WPR == 8 ? 8 : 4, RPW = WAVES / WPR;  // waves and rows of a workgroup
  __shared__ double totals[WAVES];
  __shared__ float squares[WAVES];
  const int lane = threadIdx.x & 63, w = wave_id_uniform(), wk = w & (WPR - 1);
  const int d = (int)p.d, nb = (d + 127) >> 7;
  const float inv_d = (float)p.inv_d;
  uint4 gv[NL], bv[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int col = (WPR * i + wk) * 512 + lane * 8;
    gv[i] = col < d ? *reinterpret_cast<const uint4*>(p.gamma + col) : make_uint4(0, 0, 0, 0);
    bv[i] = p.beta != nullptr && col < d ? *reinterpret_cast<const uint4*>(p.beta + col) : make_uint4(0, 0, 0, 0);
  }
  for (uint32_t id = blockIdx.x; id < sets; id += gridDim.x) {
    const int64_t row = (int64_t)region_at<LINES>(id, sets) * RPW + w / WPR;
    const bool row_ok = row < p.rows;
    const int64_t at = (row_ok ? row : p.rows - 1) * p.d;
    uint4 hv[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int col = (WPR * i + wk) * 512 + lane * 8;
      hv[i] = col < d ? load_once<PAST>(p.x + at + col) : make_uint4(0, 0, 0, 0);
    }
    if (p.res != nullptr) {
      uint4 rv[NL];
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int col = (WPR * i + wk) * 512 + lane * 8;
        rv[i] = col < d ? load_once<PAST>(p.res + at + col) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int col = (WPR * i + wk) * 512 + lane * 8;
        float a[8], b[8];
        unpack8(hv[i], a);
        unpack8(rv[i], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] += b[j];  // rounds to bf16 as the exact sum does
        hv[i] = bf16_round8(a);
        if (p.h != nullptr && row_ok && col < d) store_once<PAST>(p.h + at + col, hv[i]);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      float a[8];
      unpack8(hv[i], a);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += a[j];
    }
    const double total = row_sum<WPR>((double)s, w, totals);
    double mu = total * p.inv_d;
    mu = __builtin_fma(__builtin_fma(-mu, (double)d, total), p.inv_d, mu);  // equal values are their mean; inf: NaN
    const float m = (float)mu, delta = (float)(mu - (double)m);
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int col = (WPR * i + wk) * 512 + lane * 8;
      float a[8];
      unpack8(hv[i], a);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float c = col < d ? a[j] - m : 0.0f;
        sq = __builtin_fmaf(c, c, sq);
      }
    }
    sq = row_sum<WPR>(sq, w, squares) * inv_d;
    const float var = __builtin_elementwise_maximum(__builtin_fmaf(-delta, delta, sq), 0.0f);  // a NaN stays
    const float rstd = 1.0f / __builtin_sqrtf(var + p.eps);
    if (p.mean != nullptr && row_ok && lane == 0 && wk == 0) {
      p.mean[row] = m + delta;
      p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int col = (WPR * i + wk) * 512 + lane * 8;
      const bool ok = row_ok && col < d;
      // unpacked again: the floats of the row are not kept over the sums
      asm volatile("" : "+v"(hv[i].x), "+v"(hv[i].y), "+v"(hv[i].z), "+v"(hv[i].w));
      asm volatile("" : "+v"(gv[i].x), "+v"(gv[i].y), "+v"(gv[i].z), "+v"(gv[i].w));
      asm volatile("" : "+v"(bv[i].x), "+v"(bv[i].y), "+v"(bv[i].z), "+v"(bv[i].w));
      float v[8], g[8], b[8];
      unpack8(hv[i], v);
      unpack8(gv[i], g);
      unpack8(bv[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = col < d ? __builtin_fmaf(((v[j] - m) - delta) * rstd, g[j], b[j]) : 0.0f;
      if (p.y != nullptr && ok) *reinterpret_cast<uint4*>(p.y + at + col) = bf16_round8(v);
      if (p.q != nullptr) {
        const Scale sc = scale_of(row16_max(amax8(v)));
        const uint2 codes = __all(sc.r != 0.0f || !ok) ? codes8<true>(v, sc) : codes8<false>(v, sc);
        if (ok) {
          put_codes8<LINES>(p.q + at + col, codes);
          if ((lane & 15) == 0) p.scales[row * nb + (col >> 7)] = sc.s;
        }
      }
    }
  }
}

// ---- backward ---------------------------------------------------------------------------
constexpr int LNB_WAVES = 16, LNB_NL = 2;  // waves of a workgroup, pieces of a lane at most

struct LayerNormBackward {
  const uint16_t *dy, *h, *gamma, *dres;
  const float *mean, *rstd;
  uint16_t* dx;
  float* partial;  // [gridDim.x, 2, d]
  int64_t rows, d;
};

template <int NL, int WPR, bool STREAM, bool PAST>
__global__ void __launch_bounds__(64 * LNB_WAVES) layernorm_backward_kernel(LayerNormBackward p, uint32_t sets) {
  constexpr int RPW = LNB_WAVES / WPR;  // rows of a workgroup
  __shared__ float sums[2][LNB_WAVES][2];
  extern __shared__ __attribute__((aligned(16))) float joined[];  // [RPW][2][512 NL WPR] if RPW > 1
  const int lane = threadIdx.x & 63, w = wave_id_uniform(), wk = w & (WPR - 1), sub = w / WPR;
  const int d = (int)p.d;
  const float inv_d = 1.0f / (float)d;
  int at_col[NL];  // columns past d read column 0 (which may be infinite: they are left out of the row's sums)
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int col = (WPR * i + wk) * 512 + lane * 8;
    at_col[i] = col < d ? col : 0;
  }
  // Rows past the end read the last row (not added, not stored).
  auto row_of = [&](uint32_t id) __attribute__((always_inline)) -> int64_t {
    const int64_t row = (int64_t)(id < sets ? id : sets - 1) * RPW + sub;
    return row < p.rows ? row : p.rows - 1;
  };
  auto load = [&](uint32_t id, uint4 (&dy)[NL], uint4 (&h)[NL], float& mean, float& rstd)
      __attribute__((always_inline)) {
    const int64_t from = row_of(id);
    const uint16_t *const a = p.dy + from * p.d, *const b = p.h + from * p.d;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      dy[i] = load_once<PAST>(a + at_col[i]);
      h[i] = load_once<PAST>(b + at_col[i]);
    }
    mean = p.mean[from];
    rstd = p.rstd[from];
  };
  uint4 gv[NL];
  float dg[NL][8], db[NL][8];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int col = (WPR * i + wk) * 512 + lane * 8;
    gv[i] = col < d ? *reinterpret_cast<const uint4*>(p.gamma + col) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = 0.0f;
  }
  // The residual stream's gradient is needed last: it is asked for before the next
  // set's rows, which stay in flight when it is waited for.
  uint4 rv[STREAM ? NL : 1];
  auto load_stream = [&](uint32_t id) __attribute__((always_inline)) {
    if constexpr (STREAM) {
      const uint16_t* const a = p.dres + row_of(id) * p.d;
#pragma unroll
      for (int i = 0; i < NL; ++i) rv[i] = load_once<PAST>(a + at_col[i]);
    }
  };
  // One set of rows; the next set's loads are in flight meanwhile.
  auto work = [&](uint32_t id, uint4 (&dyv)[NL], uint4 (&hv)[NL], float mean, float rstd, int turn)
      __attribute__((always_inline)) {
    const int64_t row = (int64_t)id * RPW + sub;
    const bool row_ok = row < p.rows;  // (the same for the whole wave)
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      if (!row_ok) break;
      const float before1 = s1, before2 = s2;
      float dy[8], h[8], g[8];
      unpack8(dyv[i], dy);
      unpack8(hv[i], h);
      unpack8(gv[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (h[j] - mean) * rstd, gy = dy[j] * g[j];
        s1 += gy;
        s2 = __builtin_fmaf(gy, xh, s2);
        db[i][j] += dy[j];
        dg[i][j] = __builtin_fmaf(dy[j], xh, dg[i][j]);
      }
      const bool in = (WPR * i + wk) * 512 + lane * 8 < d;
      s1 = in ? s1 : before1;
      s2 = in ? s2 : before2;
    }
    row_sums<WPR>(s1, s2, w, sums[turn]);
    const float c1 = s1 * inv_d, c2 = s2 * inv_d;
    uint16_t* const out = p.dx + row * p.d;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      // unpacked a second time: 24 values for each of the row's pieces are not kept over the sums
      asm volatile("" : "+v"(dyv[i].x), "+v"(dyv[i].y), "+v"(dyv[i].z), "+v"(dyv[i].w));
      asm volatile("" : "+v"(hv[i].x), "+v"(hv[i].y), "+v"(hv[i].z), "+v"(hv[i].w));
      asm volatile("" : "+v"(gv[i].x), "+v"(gv[i].y), "+v"(gv[i].z), "+v"(gv[i].w));
      const int col = (WPR * i + wk) * 512 + lane * 8;
      float dy[8], h[8], g[8], r[8];
      unpack8(dyv[i], dy);
      unpack8(hv[i], h);
      unpack8(gv[i], g);
      if constexpr (STREAM) unpack8(rv[i], r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (h[j] - mean) * rstd;
        const float v = __builtin_fmaf(-xh, c2, __builtin_fmaf(dy[j], g[j], -c1));
        if constexpr (STREAM) dy[j] = __builtin_fmaf(v, rstd, r[j]);
        else dy[j] = v * rstd;
      }
      if (row_ok && col < d) store_once<PAST>(out + col, bf16_round8(dy));
    }
  };
  uint4 dy0[NL], h0[NL], dy1[NL], h1[NL];
  float mean0, rstd0, mean1, rstd1;
  const uint32_t step = gridDim.x;
  load(blockIdx.x, dy0, h0, mean0, rstd0);
  for (uint32_t id = blockIdx.x; id < sets; id += 2 * step) {
    load_stream(id);
    load(id + step, dy1, h1, mean1, rstd1);
    work(id, dy0, h0, mean0, rstd0, 0);
    if (id + step >= sets) break;  // (the same for the whole workgroup)
    load_stream(id + step);
    load(id + 2 * step, dy0, h0, mean0, rstd0);
    work(id + step, dy1, h1, mean1, rstd1, 1);
  }
  // The workgroup's rows in order: every wave leaves its sums in LDS, 16 x 8 KB in all.
  float* const out = p.partial + (int64_t)blockIdx.x * 2 * p.d;
  constexpr int COLS = 512 * NL * WPR;
  float* const to = RPW > 1 ? joined + sub * 2 * COLS : out;
  const int64_t second = RPW > 1 ? COLS : p.d;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int col = (WPR * i + wk) * 512 + lane * 8;
    if (col < d) {
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        *reinterpret_cast<float4*>(to + col + j) = make_float4(dg[i][j], dg[i][j + 1], dg[i][j + 2], dg[i][j + 3]);
        *reinterpret_cast<float4*>(to + second + col + j) =
            make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
      }
    }
  }
  if constexpr (RPW > 1) {
    __syncthreads();
    for (int e = threadIdx.x * 4; e < 2 * COLS; e += 64 * LNB_WAVES * 4) {
      const int half = e >= COLS ? 1 : 0, col = e - half * COLS;
      if (col >= d) continue;
      v4f sum = *reinterpret_cast<const v4f*>(joined + e);
#pragma unroll
      for (int k = 1; k < RPW; ++k) sum = sum + *reinterpret_cast<const v4f*>(joined + k * 2 * COLS + e);
      *reinterpret_cast<v4f*>(out + half * p.d + col) = sum;
    }
  }
}

int layernorm_max_cols() { return 512 * LN_NL * LN_MAX_WPR; }

template <int NL, int WPR>
static void launch_ln(const LayerNorm& p, hipStream_t stream) {
  constexpr int THREADS = WPR == 8 ? 512 : 256, RPW = THREADS / 64 / WPR;
  const int64_t sets = (p.rows + RPW - 1) / RPW;
  const dim3 grid((unsigned)(sets < 2048 ? sets : 2048));
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(THREADS), 0, stream, p, (uint32_t)sets);
  };
  const bool past = p.rows * p.d * (p.res ? 4 : 2) > INPUTS_PAST;
  if (p.d % 128 == 0)
    past ? launch(layernorm_kernel<NL, WPR, true, true>) : launch(layernorm_kernel<NL, WPR, true, false>);
  else
    past ? launch(layernorm_kernel<NL, WPR, false, true>) : launch(layernorm_kernel<NL, WPR, false, false>);
}

hipError_t launch_layernorm(const void* x, const void* residual, const void* gamma, const void* beta, float eps,
                            int64_t rows, int64_t d, void* h, void* q, float* scales, void* y, float* mean,
                            float* rstd, hipStream_t stream) {
  const LayerNorm p = {(const uint16_t*)x, (const uint16_t*)residual, (const uint16_t*)gamma, (const uint16_t*)beta,
                       (uint16_t*)h,       (uint16_t*)y,              (uint8_t*)q,            scales,
                       mean,               rstd,                      rows,                   d, 1.0 / (double)d, eps};
  if (d <= 512) launch_ln<1, 1>(p, stream);
  else if (d <= 1024) launch_ln<1, 2>(p, stream);
  else if (d <= 2048) launch_ln<1, 4>(p, stream);
  else if (d <= 4096) launch_ln<1, 8>(p, stream);
  else if (d <= 8192) launch_ln<2, 8>(p, stream);
  else launch_ln<4, 8>(p, stream);
  return hipGetLastError();
}

// Sets of rows (what a workgroup takes at once: up to eight waves hold a row before a lane has a
// second piece) and workgroups of the backward pass.  A workgroup takes four rows at
// least, as long as that leaves 128 of them, since its partial sums are as much traffic as
// two to three rows (us with one set each, and so: 500 x 4096 11.4 and 9.7, 500 x 8192 15.5 and
// 14.6, 300 x 12288 19.5 and 17.4).
static int64_t ln_sets(int64_t rows, int64_t d) {
  const int wpr = d <= 512 ? 1 : d <= 1024 ? 2 : d <= 2048 ? 4 : d <= 8192 ? 8 : 16, rpw = LNB_WAVES / wpr;
  return (rows + rpw - 1) / rpw;
}
static int64_t ln_backward_grid(int64_t rows, int64_t d) {
  const int64_t sets = ln_sets(rows, d), fours = (rows + 3) / 4;
  const int64_t want = fours < 128 ? 128 : fours < 256 ? fours : 256;
  const int64_t turns = (sets + want - 1) / want;
  return turns ? (sets + turns - 1) / turns : 0;  // the same number of sets to each but the last
}

int64_t layernorm_backward_workspace(int64_t rows, int64_t d) { return ln_backward_grid(rows, d) * 2 * d * 4; }

template <int NL, int WPR>
constexpr int ln_backward_lds() { return WPR < LNB_WAVES ? LNB_WAVES * 2 * 512 * NL * 4 : 0; }

template <int NL, int WPR>
static void launch_ln_backward(const LayerNormBackward& p, unsigned grid, uint32_t sets, hipStream_t stream) {
  constexpr int LDS = ln_backward_lds<NL, WPR>(), THREADS = 64 * LNB_WAVES;
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(THREADS), LDS, stream, p, sets);
  };
  const bool past = p.rows * p.d * (p.dres ? 6 : 4) > INPUTS_PAST;
  if (p.dres)
    past ? launch(layernorm_backward_kernel<NL, WPR, true, true>)
         : launch(layernorm_backward_kernel<NL, WPR, true, false>);
  else
    past ? launch(layernorm_backward_kernel<NL, WPR, false, true>)
         : launch(layernorm_backward_kernel<NL, WPR, false, false>);
}

hipError_t set_layernorm_attributes() {
  hipError_t e = hipSuccess;
  auto allow = [&](const void* kernel, int lds) {
    if (e == hipSuccess) e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  };
  auto allow_all = [&](auto nl, auto wpr) {
    constexpr int NL = decltype(nl)::value, WPR = decltype(wpr)::value, LDS = ln_backward_lds<NL, WPR>();
    allow((const void*)layernorm_backward_kernel<NL, WPR, true, true>, LDS);
    allow((const void*)layernorm_backward_kernel<NL, WPR, true, false>, LDS);
    allow((const void*)layernorm_backward_kernel<NL, WPR, false, true>, LDS);
    allow((const void*)layernorm_backward_kernel<NL, WPR, false, false>, LDS);
  };
  using std::integral_constant;
  allow_all(integral_constant<int, 1>(), integral_constant<int, 1>());
  allow_all(integral_constant<int, 1>(), integral_constant<int, 2>());
  allow_all(integral_constant<int, 1>(), integral_constant<int, 4>());
  allow_all(integral_constant<int, 1>(), integral_constant<int, 8>());
  allow_all(integral_constant<int, LNB_NL>(), integral_constant<int, 8>());
  return e;
}

hipError_t launch_layernorm_backward(const void* dy, const void* h, const void* gamma, const float* mean,
                                     const float* rstd, const void* dresidual, int64_t rows, int64_t d, void* dx,
                                     float* dgamma, float* dbeta, bool accumulate, float* workspace,
                                     hipStream_t stream) {
  const LayerNormBackward p = {(const uint16_t*)dy, (const uint16_t*)h, (const uint16_t*)gamma,
                               (const uint16_t*)dresidual, mean, rstd, (uint16_t*)dx, workspace, rows, d};
  const uint32_t sets = (uint32_t)ln_sets(rows, d);
  const unsigned grid = (unsigned)ln_backward_grid(rows, d);
  if (grid > 0) {
    if (d <= 512) launch_ln_backward<1, 1>(p, grid, sets, stream);
    else if (d <= 1024) launch_ln_backward<1, 2>(p, grid, sets, stream);
    else if (d <= 2048) launch_ln_backward<1, 4>(p, grid, sets, stream);
    else if (d <= 4096) launch_ln_backward<1, 8>(p, grid, sets, stream);
    else if (d <= 8192) launch_ln_backward<LNB_NL, 8>(p, grid, sets, stream);
    else launch_ln_backward<LNB_NL, 16>(p, grid, sets, stream);
  }
  launch_column_sum(workspace, grid, 2 * d, d, dgamma, dbeta, accumulate, stream);
  return hipGetLastError();
}

}  // namespace fp8bs
