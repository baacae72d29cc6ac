// E4M3 GEMM with one fp32 scale per row and 128 K of A and one per 128x128
// block of the K-major weight, for one matrix and for ragged row groups.
//
//   C[i,j] = sum_kb sa[i,kb] sb[j/128,kb] P,  P = sum_{k in kb} A[i,k] Bt[j,k]
//
// A K-block of 128 is exactly the depth of v_mfma_f32_16x16x128_f8f6f4, the
// instruction with the full FP8 rate (its 32-deep relatives run at half of
// it), so P is one MFMA with a zero accumulator and the promotion is four fp32
// fmas per lane and 16x16x128 products: 16 VALU cycles beside 32 matrix
// cycles.
//
// Precision: the instruction cuts each product toward zero to 2^-13 of the largest
// exponent sum of its group of eight K, before it sums in fp32 (the header states
// the bound).  That is the price of the rate: the exact bf16 MFMA of the 32-value
// forms has half of it.  The cut is relative to the products and not to
// C: on quantized normal rows with a few strong channels (64 x 128 x 1024) it is
// 2.6e-5 of C, rms, and it exceeds half a bf16 step of C in 0.5% of the elements, by
// up to 200 times, where products cancel.  It is not carried along K, because the
// sum over K-blocks is the fp32 accumulator's.
//
// Every kernel here runs the same sequence per element - the same MFMA operands,
// s = RN(sa * sb), acc = fma(P, s, acc), kb ascending - so a row's result does
// not depend on M, on its place or on the kernel.
//
// Operand layout of the instruction (lane l, g = l >> 4): lane l holds row
// (l & 15) of the 16-row operand, bytes 0-15 = K [16g, 16g+16) and bytes
// 16-31 = K [64+16g, 64+16g+16).  The first operand is the weight, so a lane's
// four results are four columns of one row of C.
#include "activation.hpp"
#include "common.hpp"
#include "launch_g128.hpp"
#include "launch_layer.hpp"
#include "ragged.hpp"

#include <algorithm>
#include <type_traits>

namespace fp8bs {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float v2f_t __attribute__((ext_vector_type(2)));

constexpr int GK = 128;        // K-block = K step = bytes of one staged row
constexpr int SCH = 8;         // K-blocks per staged chunk of A's scales

// P of one K-block for a 16x16 output sub-tile (w: weight rows, x: A rows).
__device__ __forceinline__ v4f mfma_block(v8i_t w, v8i_t x) {
  const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, z, 0, 0, 0, 0, 0, 0);
}

// The lane's number, anew: what is computed from it is not kept, and spilled, from one
// tile of a persistent workgroup to the next.  (Spilled row addresses put a memory
// wait between the stores of the large tile: 8 ranges of 8192 rows, 4096 x 2048, 92 us,
// 84 so; 2048 x 8192 x 512 19.5 and 16.5.)
__device__ __forceinline__ int fresh_lane() {
  int l = threadIdx.x & 63;
  asm volatile("" : "+v"(l));
  return l;
}

// Two accumulators -> two bf16 (nearest even, NaN kept), a zero stored as +0.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const v2f_t v = {lo + 0.0f, hi + 0.0f};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2bf));
}

// Two accumulators of one lane (sub-tiles j and j + 1, four columns each) -> eight
// neighbouring columns: lanes 16 apart swap, so that those of even g = lane >> 4 hold
// columns 4g .. 4g+7 of sub-tile j and those of odd g columns 4g-4 .. 4g+3 of j + 1.
__device__ __forceinline__ uint4 bf16_octet(v4f x, v4f y) {
  const auto lo = __builtin_amdgcn_permlane16_swap(bf16_pair(x[0], x[1]), bf16_pair(y[0], y[1]), false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(bf16_pair(x[2], x[3]), bf16_pair(y[2], y[3]), false, false);
  return make_uint4(lo[0], hi[0], lo[1], hi[1]);
}

// The MI x NJ sub-tiles of a wave, from row and column `r0`, `c0` of the tile at `c`:
// a lane holds row 16i + lo, columns 16j + 4g .. +3.
template <int MI, int NJ>
__device__ __forceinline__ void store_wave(uint16_t* c, int64_t N, const v4f (&acc)[MI][NJ], int r0, int c0,
                                           int m_valid, int n_valid) {
  const int lane = fresh_lane(), g = lane >> 4, lo = lane & 15;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int r = r0 + 16 * i + lo;
    uint16_t* const cr = c + r * N;
    if constexpr (NJ % 2 == 0) {
#pragma unroll
      for (int j = 0; j < NJ; j += 2) {
        const uint4 v = bf16_octet(acc[i][j], acc[i][j + 1]);
        const int col = c0 + 16 * (j + (g & 1)) + 4 * (g & 2);
        if (r < m_valid && col < n_valid) *reinterpret_cast<uint4*>(cr + col) = v;
      }
    } else {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int col = c0 + 16 * j + 4 * g;
        if (r < m_valid && col < n_valid)
          *reinterpret_cast<uint2*>(cr + col) =
              make_uint2(bf16_pair(acc[i][j][0], acc[i][j][1]), bf16_pair(acc[i][j][2], acc[i][j][3]));
      }
    }
  }
}

// 16 bytes, past the caches if LINES.
template <bool LINES>
__device__ __forceinline__ void put16(uint16_t* p, uint4 v) {
  typedef unsigned v4u __attribute__((ext_vector_type(4)));
  if constexpr (LINES) __builtin_nontemporal_store(v4u{v.x, v.y, v.z, v.w}, reinterpret_cast<v4u*>(p));
  else *reinterpret_cast<uint4*>(p) = v;
}

// 64 columns of a row from a multiple of 64 are one line of C.
__device__ __forceinline__ bool whole_lines(const uint16_t* c, int64_t N) {
  return N % 64 == 0 && (uintptr_t)c % 128 == 0;
}

// The same for NJ = 4, 128 bytes of a row of C per wave: lanes lo and lo ^ 8 exchange
// half a row, so that a store covers eight whole rows' 128 bytes.  LINES: they are
// lines of C and leave past the caches (8192 x 8192 x 1024 79 us, as 16 half rows
// through the L2 87, whole rows through it 84; 8192 x 14336 x 2048 214, 229, 229;
// with the 128x128 tile 8192 x 1024 x 1024 12.8 and 14.3).
template <bool LINES, int MI>
__device__ __forceinline__ void store_wave_rows(uint16_t* c, int64_t N, const v4f (&acc)[MI][4], int r0, int c0,
                                                int m_valid, int n_valid) {
  const int ln = fresh_lane(), g = ln >> 4, lo = ln & 15;
  const bool low = lo < 8;
  const int col = c0 + 16 * (g & 1) + 4 * (g & 2) + (low ? 0 : 32);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const uint4 v0 = bf16_octet(acc[i][0], acc[i][1]), v1 = bf16_octet(acc[i][2], acc[i][3]);
    auto ror8 = [](uint32_t x) __attribute__((always_inline)) -> uint32_t {
      return __builtin_amdgcn_update_dpp(0, x, 0x128, 0xF, 0xF, true);
    };
    const uint4 got = make_uint4(ror8(low ? v1.x : v0.x), ror8(low ? v1.y : v0.y), ror8(low ? v1.z : v0.z),
                                 ror8(low ? v1.w : v0.w));
    const int r = r0 + 16 * i + (lo & 7);
    const uint4 a = low ? v0 : got, b = low ? got : v1;
    if (r < m_valid && col < n_valid) put16<LINES>(c + r * N + col, a);
    if (r + 8 < m_valid && col < n_valid) put16<LINES>(c + (r + 8) * N + col, b);
  }
}

// ---- epilogue: z = acc + bias, C = act(z) + residual, pre = z (include/fp8bs_layer.h), in
// the accumulators' layout: lane l holds row lo, columns 16j + 4g .. +3 of a row
// sub-tile.  The residual is read, and results are written, as C is without an
// epilogue (16 bytes a lane, whole lines where there are); the exchanges between
// lanes that lead there are their own inverse.
//
// Nothing overlaps it but the next tile's first loads, so it costs its instructions and its
// traffic.  In one run: 8192 x 16384 x 4096 454 us, with bias 465, silu 484, gelu 503 (21 issue
// slots a value), gelu and pre 540 (268 MB more), bias and residual 530; 1017 x 2064 x 1552
// 12.9, with bias 14.0, gelu and pre 16.3, silu and residual 15.6; 8 x 8192 x 8192 13.9, with
// bias and residual 14.7.  All residual rows asked for before the bias (small tiles) gained nothing.
struct NoEpilogue {};

// The result's pointer.  With an epilogue the residual may be the result itself, so that no
// promise of an only access can be given; without one nothing else is there.
template <typename E>
struct ResultPointer {
  typedef uint16_t* type;
};
template <>
struct ResultPointer<NoEpilogue> {
  typedef uint16_t* __restrict__ type;
};
template <typename E>
using result_t = typename ResultPointer<E>::type;

enum ActivationCode { CODE_CLAMP, CODE_GATED, CODE_GELU };  // what the loops over a tile are compiled for

// What does not depend on the element: none and relu are max(z, low) with low = -inf and 0
// (a NaN stays), gelu_tanh and silu z sigma(z (c0 + c1 z^2)).
template <int CODE>
struct Activate {
  float low, c0, c1;
  __device__ __forceinline__ explicit Activate(int act)
      : low(act == ACT_RELU ? 0.0f : -__builtin_inff()),
        c0(act == ACT_SILU ? 1.0f : GT_C0),
        c1(act == ACT_SILU ? 0.0f : GT_C1) {}
  __device__ __forceinline__ float operator()(float z) const {
    if constexpr (CODE == CODE_CLAMP) return z < low ? low : z;
    // (an infinite square times silu's c1 = 0 would be a NaN)
    if constexpr (CODE == CODE_GATED) return gated(z, z * __builtin_fmaf(c1, fminf(z * z, 0x1p100f), c0));
    return gelu(z);
  }
};

template <typename F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  if (act == ACT_GELU) f(Activate<CODE_GELU>(act));
  else if (act == ACT_GELU_TANH || act == ACT_SILU) f(Activate<CODE_GATED>(act));
  else f(Activate<CODE_CLAMP>(act));
}

__device__ __forceinline__ v4f add_bf16x4(v4f v, uint32_t lo, uint32_t hi) {
  return v4f{v[0] + bf16_lo(lo), v[1] + bf16_hi(lo), v[2] + bf16_lo(hi), v[3] + bf16_hi(hi)};
}
// The inverse of bf16_octet's exchange, added to both accumulators.
__device__ __forceinline__ void add_octet(v4f& x, v4f& y, uint4 v) {
  const auto lo = __builtin_amdgcn_permlane16_swap(v.x, v.z, false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(v.y, v.w, false, false);
  x = add_bf16x4(x, lo[0], hi[0]);
  y = add_bf16x4(y, lo[1], hi[1]);
}

// Row sub-tile at row `r0`, column `c0` of the tile at offset `at` of C, the residual and pre.
// ROWS: as store_wave_rows (NJ = 4), else as store_wave.
template <int NJ, bool ROWS>
struct EpilogueRow {
  uint4 res[NJ / 2 > 0 ? NJ / 2 : 1];

  __device__ __forceinline__ static int64_t place(int part, int64_t N, int r0, int c0, int& r, int& col) {
    const int ln = fresh_lane(), g = ln >> 4, lo = ln & 15;
    if constexpr (ROWS) {
      r = r0 + (lo & 7) + 8 * part;
      col = c0 + 16 * (g & 1) + 4 * (g & 2) + (lo < 8 ? 0 : 32);
    } else if constexpr (NJ % 2 == 0) {
      r = r0 + lo;
      col = c0 + 16 * (2 * part + (g & 1)) + 4 * (g & 2);
    } else {
      r = r0 + lo;
      col = c0 + 4 * g;
    }
    return r * N + col;
  }
  static constexpr int PARTS = NJ % 2 == 0 ? NJ / 2 : 1;

  __device__ __forceinline__ void load(const uint16_t* p, int64_t N, int r0, int c0, int m_valid, int n_valid) {
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      int r, col;
      const int64_t off = place(k, N, r0, c0, r, col);
      res[k] = make_uint4(0, 0, 0, 0);
      if (r < m_valid && col < n_valid) {
        if constexpr (NJ % 2 == 0) {
          res[k] = *reinterpret_cast<const uint4*>(p + off);
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(p + off);
          res[k].x = v.x;
          res[k].y = v.y;
        }
      }
    }
  }
  __device__ __forceinline__ static uint32_t ror8(uint32_t x) {
    return __builtin_amdgcn_update_dpp(0, x, 0x128, 0xF, 0xF, true);
  }
  __device__ __forceinline__ void add(v4f (&acc)[NJ]) const {
    if constexpr (ROWS) {
      const bool low = (fresh_lane() & 15) < 8;
      auto side = [&](uint32_t a, uint32_t b) __attribute__((always_inline)) { return ror8(low ? b : a); };
      const uint4 a = res[0], b = res[1];
      const uint4 x = make_uint4(side(a.x, b.x), side(a.y, b.y), side(a.z, b.z), side(a.w, b.w));
      add_octet(acc[0], acc[1], low ? a : x);
      add_octet(acc[2], acc[3], low ? x : b);
    } else if constexpr (NJ % 2 == 0) {
#pragma unroll
      for (int j = 0; j < NJ; j += 2) add_octet(acc[j], acc[j + 1], res[j / 2]);
    } else {
      acc[0] = add_bf16x4(acc[0], res[0].x, res[0].y);
    }
  }
};

template <int MI, int NJ>
__device__ __forceinline__ void epilogue_wave(const Epilogue& e, uint16_t* c, int64_t at, int64_t N,
                                              v4f (&acc)[MI][NJ], int64_t col0, int r0, int c0, int m_valid,
                                              int n_valid) {
  constexpr bool ROWS = NJ == 4;
  const bool lines = ROWS && whole_lines(c, N);
  static_assert(NJ == 1 || NJ % 2 == 0, "pairs of sub-tiles");
  if (e.bias != nullptr) {
    const int g = fresh_lane() >> 4;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int col = c0 + 16 * j + 4 * g;
      uint2 b = make_uint2(0, 0);
      if (col < n_valid) b = *reinterpret_cast<const uint2*>(e.bias + col0 + col);
#pragma unroll
      for (int i = 0; i < MI; ++i) acc[i][j] = add_bf16x4(acc[i][j], b.x, b.y);
    }
  }
  auto store = [&](uint16_t* p, const v4f (&v)[1][NJ], int r) __attribute__((always_inline)) {
    if constexpr (ROWS) {
      if (lines) store_wave_rows<true, 1>(p, N, v, r, c0, m_valid, n_valid);
      else store_wave_rows<false, 1>(p, N, v, r, c0, m_valid, n_valid);
    } else {
      store_wave<1, NJ>(p, N, v, r, c0, m_valid, n_valid);
    }
  };
  with_activation(e.act, [&](auto activate) __attribute__((always_inline)) {
    EpilogueRow<NJ, ROWS> next;
    if (e.residual != nullptr) next.load(e.residual + at, N, r0, c0, m_valid, n_valid);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const EpilogueRow<NJ, ROWS> now = next;
      if (e.residual != nullptr && i + 1 < MI) next.load(e.residual + at, N, r0 + 16 * (i + 1), c0, m_valid, n_valid);
      v4f v[1][NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) v[0][j] = acc[i][j];
      if (e.pre != nullptr) store(e.pre + at, v, r0 + 16 * i);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[0][j][k] = activate(v[0][j][k]);
      if (e.residual != nullptr) now.add(v[0]);
      store(c + at, v, r0 + 16 * i);
      __builtin_amdgcn_sched_barrier(0);  // one row sub-tile's values at a time
    }
  });
}

// ---- small and middle tiles: BM = 16*MI*WM rows by BN = 16*NJ*WN columns per
// workgroup of WM x WN waves; wave (wm, wn) owns MI x NJ sub-tiles of 16x16.
//
// A and Bt are streamed as bytes with direct loads into a ring of S steps in
// LDS, S - 1 steps ahead: few workgroups (a decode step's tiles) then still keep
// enough bytes in flight.  Row r of a stage holds its 128 bytes with 16-byte
// piece p at position p ^ (r & 7), which spreads a fragment read over all
// banks.  A's scales come eight K-blocks at a time, a chunk ahead; a weight scale is
// one value per wave and step, held by lane l for step 64c + l.  A wave's MFMAs,
// promotions and fragment reads are in the large tile's order (below); left to the
// compiler's order 512 x 8192 x 8192 took 7% longer.
template <int MI, int NJ, int WM, int WN, int S, bool GROUPED, typename E>
__global__ void __launch_bounds__(64 * WM * WN) gemm_g128_tile_kernel(
    const uint8_t* __restrict__ a, const float* __restrict__ sa, const uint8_t* __restrict__ bt,
    const float* __restrict__ sbt, const int32_t* __restrict__ offsets, int G, result_t<E> c, int64_t M,
    int64_t N, int64_t K, uint32_t tiles_n, E epilogue) {
  constexpr int BM = 16 * MI * WM, BN = 16 * NJ * WN, WAVES = WM * WN;
  constexpr int STAGE = (BM + BN) * GK;
  constexpr int PIECES = (BM + BN) / 8 / WAVES;            // 1 KB loads per wave and step
  constexpr int S_PIECES = BM / 8;                         // 256-byte scale loads per chunk
  constexpr int S_STEPS = (S_PIECES + WAVES - 1) / WAVES;  // steps of a chunk that issue one per wave
  constexpr int SSUB = 576, SBUF = BM / 16 * SSUB;
  constexpr int A_PIECES = BM / 8 / WAVES;                 // of these A's
  static_assert(PIECES * 8 * WAVES == BM + BN && A_PIECES * 8 * WAVES == BM, "tile is a whole number of loads");
  static_assert(S_STEPS == 1 || S_STEPS * WAVES == S_PIECES, "every wave has a scale load in such a step");
  static_assert(NJ * 16 <= 128 && 128 % (NJ * 16) == 0, "a wave's columns lie in one weight block");
  static_assert(S_STEPS + S <= SCH, "a chunk of scales has landed before its first step");
  static_assert(PIECES * (S - 1) < 64, "vmcnt range");
  // A small tile's wave holds the next step's fragments while it multiplies this
  // one's, so that reading them is not waited for; a larger tile has no registers
  // for that and two waves a SIMD to fill the time (64 x 8192 x 8192 20.6 -> 17.9 us,
  // 300 x 1040 x 4096 11.8 -> 10.3; 512 x 8192 x 8192 with it 45, without 43).
  constexpr int AHEAD = MI * NJ <= 4 ? 1 : 0;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  typedef __attribute__((address_space(3))) unsigned char lds_u8;
  typedef __attribute__((address_space(3))) const v4i lds_v4i;
  typedef __attribute__((address_space(3))) const float lds_f32;
  lds_u8* const lds = (lds_u8*)smem;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  const int lane = threadIdx.x & 63;
  const int w = wave_id_uniform();
  const int wm = w / WN, wn = w % WN;
  const int g = lane >> 4, lo = lane & 15;

  TileAt t;
  if constexpr (GROUPED) {
    if (!find_tile<BM>(offsets, G, M, tiles_n, blockIdx.x, gridDim.x, t)) return;
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

  // ---- direct loads: piece p = w + i*WAVES is rows 8p .. 8p+7 of the stage (A's rows,
  // then the weight's); lane l loads row l >> 3, 16-byte piece (l & 7) ^ (row & 7).
  // Rows past the range read its last row (never stored); in the partial last
  // K-block the pieces past K read the last whole piece (see frag_a).
  const int piece = (lane & 7) ^ (lane >> 3);
  uint32_t off[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int p = w + i * WAVES;
    const int valid = i < A_PIECES ? m_valid : n_valid;
    const int r = (i < A_PIECES ? p : p - BM / 8) * 8 + (lane >> 3);
    off[i] = (uint32_t)(r < valid ? r : valid - 1) * (uint32_t)K + piece * 16;
  }
  const uint8_t* const a0 = uniform_ptr(a + row0 * K);
  const uint8_t* const b0 = uniform_ptr(bt + col0 * K);
  const uint8_t* const sa0 = uniform_ptr(reinterpret_cast<const uint8_t*>(sa + row0 * KB));
  const bool partial = (K & 127) != 0;
  const uint32_t dst = lds0 + w * 1024;  // (scalar)

  // The load of step ks into the slot at `at`; LAST: it may be the partial one.
  auto issue = [&](int ks, uint32_t at, auto last) __attribute__((always_inline)) {
    uint32_t back = 0;
    if constexpr (decltype(last)::value) {
      const int over = (KB - 1) * GK + piece * 16 + 16 - (int)K;
      if (ks == KB - 1 && over > 0) back = over;
    }
    const int64_t k = (int64_t)ks * GK;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      dma16_at((i < A_PIECES ? a0 : b0) + k, off[i] - back, dst + at + i * WAVES * 1024);
  };
  // Scales of chunk `chunk`, the wave's share number q.  The chunk behind the last one
  // is the last scale again, and is not used.
  uint32_t s_off[S_STEPS];
#pragma unroll
  for (int q = 0; q < S_STEPS; ++q) {
    const int r = (q * WAVES + w) * 8 + (lane & 7);
    s_off[q] = (uint32_t)(r < m_valid ? r : m_valid - 1) * (uint32_t)KB;
  }
  auto issue_s = [&](int chunk, int q) __attribute__((always_inline)) {
    const int p = q * WAVES + w, kb = chunk * SCH + (lane >> 3);
    dma4_at(sa0, (s_off[q] + (kb < KB ? kb : KB - 1)) * 4,
            lds0 + S * STAGE + (chunk & 1) * SBUF + (p >> 1) * SSUB + (p & 1) * 288);
  };
  const int64_t nb = (col0 + wn * 16 * NJ) >> 7;
  const float* const sb_row = sbt + (nb < ((N + 127) >> 7) ? nb : 0) * KB;
  auto load_sb = [&](int ks) __attribute__((always_inline)) -> int {
    int v = __builtin_bit_cast(int, sb_row[ks + lane < KB ? ks + lane : KB - 1]);
    asm volatile("" : "+v"(v));
    return v;
  };

  v4f acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  if (KB > 0) {
    int sb_lanes = load_sb(0);
#pragma unroll
    for (int q = 0; q < S_STEPS; ++q)
      if (q * WAVES + w < S_PIECES) issue_s(0, q);
    for (int ks = 0; ks < S - 1 + AHEAD && ks < KB; ++ks) issue(ks, ks * STAGE, std::true_type());

    const int sw0 = 16 * (g ^ (lo & 7)), sw1 = 16 * ((4 + g) ^ (lo & 7));
    const lds_u8* const ra = lds + (wm * 16 * MI + lo) * GK;
    const lds_u8* const rb = lds + (BM + wn * 16 * NJ + lo) * GK;
    const lds_u8* const rs = lds + S * STAGE + wm * MI * SSUB + (lo >> 3) * 288 + (lo & 7) * 4;
    auto frag = [&](const lds_u8* base) __attribute__((always_inline)) -> v8i_t {
      const v4i x = *(lds_v4i*)(base + sw0), y = *(lds_v4i*)(base + sw1);
      return v8i_t{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    };
    // A's fragment.  LAST: zeros behind K, where the loads left the row's last piece
    // again; the weight's keeps it, which is no NaN that its column has not.
    auto frag_a = [&](const lds_u8* base, int ks, auto last) __attribute__((always_inline)) -> v8i_t {
      v8i_t f = frag(base);
      if constexpr (decltype(last)::value) {
        const int rest = (int)K - ks * GK;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[e] = 16 * g < rest ? f[e] : 0;
          f[4 + e] = 64 + 16 * g < rest ? f[4 + e] : 0;
        }
      }
      return f;
    };
    struct Block {  // one K-block of the wave's part
      v8i_t a[MI], b[NJ];
      float sc[MI];
    };
    auto read = [&](Block& f, int ks, uint32_t at, auto last) __attribute__((always_inline)) {
      const lds_u8* const q = rs + ((ks >> 3) & 1) * SBUF + (ks & 7) * 32;
#pragma unroll
      for (int j = 0; j < NJ; ++j) f.b[j] = frag(rb + at + 16 * j * GK);
#pragma unroll
      for (int i = 0; i < MI; ++i) f.sc[i] = *(lds_f32*)(q + i * SSUB);
#pragma unroll
      for (int i = 0; i < (AHEAD ? MI : 1); ++i) f.a[i] = frag_a(ra + at + 16 * i * GK, ks, last);
      __builtin_amdgcn_sched_barrier(0);
    };
    auto multiply = [&](Block& f, int ks, uint32_t at, auto last) __attribute__((always_inline)) {
      const float sb =
          __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sb_lanes), ks & 63));
      v4f p[NJ];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (!AHEAD && i + 1 < MI) f.a[i + 1] = frag_a(ra + at + 16 * (i + 1) * GK, ks, last);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          if (i > 0) {
            promote(acc[i - 1][j], p[j], f.sc[i - 1] * sb);
            asm volatile("" : "+v"(acc[i - 1][j]));  // here, not where it is next needed
            __builtin_amdgcn_sched_barrier(0);
          }
          p[j] = mfma_block(f.b[j], f.a[i]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) promote(acc[MI - 1][j], p[j], f.sc[MI - 1] * sb);
    };
    // One step.  REST: one of the last, whose own or next loads may be the partial
    // K-block or lie behind the last one; without it the only branch is the scales'.
    int ks = 0;
    uint32_t at = 0, before = (S - 1) * STAGE;
    auto step = [&](Block& now, Block& then, auto rest) __attribute__((always_inline)) {
      constexpr bool REST = decltype(rest)::value;
      if ((ks & 63) == 0 && ks > 0) sb_lanes = load_sb(ks);
      const uint32_t after = at == (S - 1) * STAGE ? 0 : at + STAGE;
      if (!REST || ks + AHEAD < KB) {
        if constexpr (REST) wait_steps<S - 2, PIECES>(KB - 1 - AHEAD - ks);
        else wait_vmcnt<(S - 2) * PIECES>();  // step ks + AHEAD has landed (scale loads only make it stricter)
        lds_barrier();                        // ... for every wave; step ks + AHEAD - 1's slot is free
#pragma unroll
        for (int q = 0; q < S_STEPS; ++q)
          if ((ks & 7) == q && (!REST || (ks >> 3) < (KB - 1) >> 3) && (S_STEPS > 1 || w < S_PIECES))
            issue_s((ks >> 3) + 1, q);
        if (!REST || ks + S - 1 + AHEAD < KB) issue(ks + S - 1 + AHEAD, AHEAD ? at : before, rest);
        if constexpr (AHEAD) {
          if (wave_live) read(then, ks + 1, after, rest);
        }
      }
      if (wave_live) {
        if constexpr (!AHEAD) read(now, ks, at, rest);
        multiply(now, ks, at, rest);
      }
      before = at;
      at = after;
      ++ks;
    };
    Block f0, f1;
    if constexpr (AHEAD) {
      wait_steps<S - 1, PIECES>(KB - 1);
      lds_barrier();
      if (wave_live) read(f0, 0, 0, std::true_type());
    }
    const int whole = KB - (S - 1) - AHEAD - (partial ? 1 : 0);
    if constexpr (AHEAD) {
#pragma unroll 1
      while (ks + 2 <= whole) {
        step(f0, f1, std::false_type());
        step(f1, f0, std::false_type());
      }
#pragma unroll 1
      while (ks < KB) {
        step(f0, f1, std::true_type());
        if (ks < KB) step(f1, f0, std::true_type());
      }
    } else {
#pragma unroll 1
      while (ks < whole) step(f0, f0, std::false_type());
#pragma unroll 1
      while (ks < KB) step(f0, f0, std::true_type());
    }
  }

  if (!wave_live) return;
  if constexpr (!std::is_same_v<E, NoEpilogue>) {
    const int64_t at = row0 * N + col0;
    const int r0 = wm * 16 * MI, c0 = wn * 16 * NJ;
    epilogue_wave(epilogue, c, at, N, acc, col0, r0, c0, m_valid, n_valid);
    return;
  }
  uint16_t* const ct = c + row0 * N + col0;
  if constexpr (NJ == 4) {
    if (whole_lines(c, N)) {
      store_wave_rows<true>(ct, N, acc, wm * 16 * MI, wn * 16 * NJ, m_valid, n_valid);
      return;
    }
  }
  store_wave<MI, NJ>(ct, N, acc, wm * 16 * MI, wn * 16 * NJ, m_valid, n_valid);
}

// ---- the large tile: 256 x 256 per workgroup, eight waves of 128 x 64 (2 row bands by
// 4 column bands), MFMAs fed without a pause.
//
// In a wave every MFMA of row sub-tile i is preceded by the four promotion fmas of
// the product that the same column sub-tile had for row sub-tile i - 1, so the
// fmas run under the matrix pipe and no product is waited for (a register-only
// loop in this order reaches 4.84 PFLOP/s on constants, the MFMAs alone 4.92; 4.1 to
// 4.3 on random data, whose power lowers the clock).  Fragments of row sub-tile
// i + 1 are read from LDS one sub-tile ahead; the weight fragments of the next step
// replace the current ones as the last row sub-tile's MFMAs issue.
//
// A step's data arrive in three parts with two barriers per step:
//   middle (before row sub-tile 3): rows of sub-tiles 0-3 of A's slot and the
//     weight's slot have been read by every wave; the loads of step ks + 2 into them
//     are issued;
//   end (before row sub-tile 7): the rest of A's slot has been read, its loads
//     for ks + 2 are issued; the next step's first fragments may be read.
// Each load has about one and a half steps to land.  The waits count a wave's own
// loads (they return in order); the barrier makes them everybody's.
//
// A workgroup takes every gridDim.x-th tile.  The next tile's first two steps are loaded
// before the current one's results are written, so neither the writes nor the first
// loads' way through memory leave the CU idle.
constexpr int XBM = 256, XBN = 256, XTHREADS = 512;
constexpr int X_A = 0, X_B = 2 * XBM * GK, X_S = X_B + 2 * XBN * GK;  // LDS: A slots, weight slots, scales
constexpr int X_SLOT = XBM * GK;
// Scales of 256 rows x 8 K-blocks: eight rows as [K-block][row], 256 bytes, two such
// pieces per row sub-tile at 0 and 288 of its 768 bytes: the 16 rows that a
// read takes for one K-block lie on 16 banks.
constexpr int X_SSUB = 768, X_SBUF = XBM / 16 * X_SSUB;
constexpr int X_LDS = X_S + 2 * X_SBUF;

template <bool GROUPED, typename E>
__global__ void __launch_bounds__(XTHREADS) gemm_g128_big_kernel(
    const uint8_t* __restrict__ a, const float* __restrict__ sa, const uint8_t* __restrict__ bt,
    const float* __restrict__ sbt, const int32_t* __restrict__ offsets, int G, result_t<E> c, int64_t M,
    int64_t N, int64_t K, uint32_t tiles_n, uint32_t tiles, E epilogue) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  typedef __attribute__((address_space(3))) unsigned char lds_u8;
  typedef __attribute__((address_space(3))) const v4i lds_v4i;
  typedef __attribute__((address_space(3))) const float lds_f32;
  typedef __attribute__((address_space(3))) v4i lds_v4i_w;
  lds_u8* const lds = (lds_u8*)smem;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  const int lane = threadIdx.x & 63;
  const int w = wave_id_uniform();
  const int wm = w >> 2, wn = w & 3;  // the waves of one SIMD (w, w + 4) are in different row bands
  const int g = lane >> 4, lo = lane & 15;

  const int KB = (int)((K + 127) >> 7);
  const bool lines = whole_lines(c, N);
  auto tile_at = [&](uint32_t id, TileAt& t) __attribute__((always_inline)) -> bool {
    if (id >= tiles) return false;
    if constexpr (GROUPED) return find_tile<XBM>(offsets, G, M, tiles_n, id, tiles, t);
    dense_tile<XBM>(M, tiles_n, id, tiles, t);
    return true;
  };
  TileAt t;
  uint32_t id = blockIdx.x;
  if (!tile_at(id, t)) return;

  // ---- direct loads of 8 rows each; lane l loads row l >> 3, 16-byte piece
  // (l & 7) ^ (row & 7).  Rows past the range read its last row.
  auto row_off = [&](int l, int row, int valid) __attribute__((always_inline)) -> uint32_t {
    const int r = row + (l >> 3);
    return (uint32_t)(r < valid ? r : valid - 1) * (uint32_t)K + ((l & 7) ^ (l >> 3)) * 16;
  };
  const int a_first = (w >> 2) * 128 + (w & 3) * 16;  // rows of sub-tiles 0-3; those of 4-7 lie 64 further
  // what the loads of the current tile need
  int m_valid = 0, n_valid = 0, sb_lanes = 0;
  uint32_t a_off[4] = {}, b_off[4] = {};
  const uint8_t *a0 = nullptr, *b0 = nullptr, *sa0 = nullptr;
  const float* sb_row = nullptr;
  auto load_sb = [&](int ks) __attribute__((always_inline)) -> int {
    return __builtin_bit_cast(int, sb_row[ks + lane < KB ? ks + lane : KB - 1]);
  };
  auto begin_tile = [&]() __attribute__((always_inline)) {
    const int64_t col0 = (int64_t)t.tn * XBN;
    m_valid = (int)(t.row_end - t.row0 < XBM ? t.row_end - t.row0 : XBM);
    n_valid = (int)(N - col0 < XBN ? N - col0 : XBN);
    const int l = fresh_lane();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a_off[i] = row_off(l, a_first + (i >> 1) * 64 + (i & 1) * 8, m_valid);
      b_off[i] = row_off(l, (w * 4 + i) * 8, n_valid);
    }
    a0 = uniform_ptr(a + t.row0 * K);
    b0 = uniform_ptr(bt + ((int64_t)t.group * N + col0) * K);
    sa0 = uniform_ptr(reinterpret_cast<const uint8_t*>(sa + t.row0 * KB));
    const int64_t nbs = (N + 127) >> 7, nb = (col0 + wn * 64) >> 7;
    sb_row = sbt + (t.group * nbs + (nb < nbs ? nb : 0)) * KB;
  };
  // In the partial last K-block the pieces past K read the last whole piece (the
  // LDS bytes are cleared afterwards).  It is loaded by the last steps only (P =
  // -1 below), whose loads ask for it.
  const bool partial = (K & 127) != 0;
  auto tail_back = [&](int ks) __attribute__((always_inline)) -> uint32_t {
    if (!partial || ks != KB - 1) return 0u;
    const int over = ((lane & 7) ^ (lane >> 3)) * 16 + 16 - (int)(K & 127);
    return over > 0 ? over : 0;
  };

  // i 0, 1: row sub-tiles 0-3; 2, 3: 4-7
  auto issue_a = [&](int ks, int i, uint32_t back = 0) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + X_A + (ks & 1) * X_SLOT + (a_first + (i >> 1) * 64 + (i & 1) * 8) * GK;
    dma16_at(a0 + (int64_t)ks * GK, a_off[i] - back, dst);
  };
  auto issue_b = [&](int ks, int i, uint32_t back = 0) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + X_B + (ks & 1) * X_SLOT + (w * 32 + i * 8) * GK;
    dma16_at(b0 + (int64_t)ks * GK, b_off[i] - back, dst);
  };
  // Scales of eight rows x eight K-blocks, one per lane: part q (0..3) of this
  // wave's 32 rows of chunk `chunk`.
  auto issue_s = [&](int chunk, int q, int l) __attribute__((always_inline)) {
    const int r = w * 32 + q * 8 + (l & 7), kb = chunk * SCH + (l >> 3);
    const uint32_t off = (uint32_t)(r < m_valid ? r : m_valid - 1) * (uint32_t)KB + (kb < KB ? kb : KB - 1);
    dma4_at(sa0, off * 4, lds0 + X_S + (chunk & 1) * X_SBUF + (w * 2 + (q >> 1)) * X_SSUB + (q & 1) * 288);
  };
  // Zeros behind K in the last K-block's slots, once its data are there for every wave.
  auto clear_tail = [&]() __attribute__((always_inline)) {
    const int first = (int)(K & 127) >> 4;  // first piece past K
    const int r = (w & 3) * 64 + fresh_lane();
    lds_u8* const base = lds + (w < 4 ? X_A : X_B) + ((KB - 1) & 1) * X_SLOT + r * GK;
    for (int p = first; p < 8; ++p) *(lds_v4i_w*)(base + 16 * (p ^ (r & 7))) = v4i{0, 0, 0, 0};
  };

  // The loads of step ks + 2, one at a time: after the middle barrier the scales
  // (even steps), sub-tiles 0-3 of A and the weight, after the end barrier
  // sub-tiles 4-7 of A.
  auto issue_mid = [&](int ks, int n, bool last) __attribute__((always_inline)) {
    const uint32_t back = last ? tail_back(ks + 2) : 0u;
    if (n == 0) {
      if ((ks & 1) == 0) issue_s((ks >> 3) + 1, (ks & 7) >> 1, lane);
    } else if (n < 3) {
      issue_a(ks + 2, n - 1, back);
    } else {
      issue_b(ks + 2, n - 3, back);
    }
  };
  auto issue_end = [&](int ks, int n, bool last) __attribute__((always_inline)) {
    issue_a(ks + 2, 2 + n, last ? tail_back(ks + 2) : 0u);
  };

  // The waits and barriers of one step, between which `work` runs its parts: 0
  // before the middle, 1 to the end, 2 after it; part 1 issues the seven loads of
  // issue_mid and part 2 the two of issue_end if `loads`.  P is ks & 1 while steps
  // ks + 2 are loaded (waits leave the younger loads in flight); with P = -1 (the
  // last steps) every load has been waited for.
  auto step = [&](int ks, auto P_, auto&& work) __attribute__((always_inline)) {
    constexpr int P = decltype(P_)::value;
    const bool loads = P >= 0 || ks + 2 < KB;
    if constexpr (P >= 0) __builtin_assume((ks & 1) == P);
    constexpr auto LAST = std::integral_constant<bool, (P < 0)>{};
    work(std::integral_constant<int, 0>{}, loads, LAST);
    if constexpr (P >= 0) wait_vmcnt<(P == 1 ? 9 : 8)>();
    else wait_vmcnt<0>();
    lds_barrier();
    work(std::integral_constant<int, 1>{}, loads, LAST);
    if constexpr (P >= 0) wait_vmcnt<(P == 0 ? 9 : 8)>();
    else wait_vmcnt<0>();
    lds_barrier();
    if (P < 0 && partial && ks + 2 == KB) {
      clear_tail();
      lds_barrier();
    }
    work(std::integral_constant<int, 2>{}, loads, LAST);
  };
  auto run = [&](auto&& work) __attribute__((always_inline)) {
    int ks = 0;
    const int steady = KB - (partial ? 4 : 3);
#pragma unroll 1
    for (; ks < steady; ks += 2) {
      step(ks, std::integral_constant<int, 0>{},
           [&](auto part, bool loads, auto last) __attribute__((always_inline)) { work(ks, part, loads, last); });
      step(ks + 1, std::integral_constant<int, 1>{},
           [&](auto part, bool loads, auto last) __attribute__((always_inline)) { work(ks + 1, part, loads, last); });
    }
#pragma unroll 1
    for (; ks < KB; ++ks)
      step(ks, std::integral_constant<int, -1>{},
           [&](auto part, bool loads, auto last) __attribute__((always_inline)) { work(ks, part, loads, last); });
  };

  // The first two steps' loads of a tile, in the loop's order: sub-tiles 0-3 and the
  // weight, then sub-tiles 4-7.
  auto first_loads = [&]() __attribute__((always_inline)) {
    auto mid = [&](int ks) __attribute__((always_inline)) {
      const uint32_t back = tail_back(ks);
      issue_a(ks, 0, back);
      issue_a(ks, 1, back);
#pragma unroll
      for (int n = 0; n < 4; ++n) issue_b(ks, n, back);
    };
    const int l = fresh_lane();
#pragma unroll
    for (int q = 0; q < 4; ++q) issue_s(0, q, l);
    mid(0);
    issue_a(0, 2, tail_back(0));
    issue_a(0, 3, tail_back(0));
    if (KB > 1) mid(1);
    // The weight's scales, one per wave and step: lane l holds step 64c + l's.
    sb_lanes = load_sb(0);
  };

  const int sw0 = 16 * (g ^ (lo & 7)), sw1 = 16 * ((4 + g) ^ (lo & 7));
  const lds_u8* const ra0 = lds + X_A + (wm * 128 + lo) * GK + sw0;
  const lds_u8* const ra1 = lds + X_A + (wm * 128 + lo) * GK + sw1;
  const lds_u8* const rb0 = lds + X_B + (wn * 64 + lo) * GK + sw0;
  const lds_u8* const rb1 = lds + X_B + (wn * 64 + lo) * GK + sw1;
  const lds_u8* const rs = lds + X_S + wm * 8 * X_SSUB + (lo >> 3) * 288 + (lo & 7) * 4;
  auto read = [&](const lds_u8* p0, const lds_u8* p1, int off) __attribute__((always_inline)) -> v8i_t {
    const v4i x = *(lds_v4i*)(p0 + off), y = *(lds_v4i*)(p1 + off);
    return v8i_t{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  };

  begin_tile();
  if (KB > 0) first_loads();
#pragma unroll 1
  for (;;) {
    const int64_t at_here = t.row0 * N + (int64_t)t.tn * XBN, col0_here = (int64_t)t.tn * XBN;
    uint16_t* const ct = c + at_here;
    const int m_here = m_valid, n_here = n_valid;
    const bool wave_live = wm * 128 < m_here && wn * 64 < n_here;
    id += gridDim.x;
    const bool more = tile_at(id, t);  // looked up while the first loads land

    v4f acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (KB > 0) {
      // everything before this, a last tile's stores among it: they are not counted
      // among the loads
      wait_vmcnt<0>();
      asm volatile("" : "+v"(sb_lanes));
      lds_barrier();
      if (KB > 1) {
        issue_a(1, 2, tail_back(1));
        issue_a(1, 3, tail_back(1));
      }
      if (partial && KB == 1) {
        clear_tail();
        lds_barrier();
      }
      if (wave_live) {
        v8i_t bf[4], af[2];
        v4f p[4];
        float sc[8];
        // the first step's fragments; products of "row sub-tile 7 of the step before" are zeros
        af[0] = read(ra0, ra1, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf[j] = read(rb0, rb1, j * 2048);
          p[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sc[i] = 0.0f;

        run([&](int ks, auto part_, bool loads, auto last) __attribute__((always_inline)) {
          constexpr int part = decltype(part_)::value;
          const int slot = (ks & 1) * X_SLOT;
          if (part == 0 && (ks & 63) == 0 && ks > 0) {
            sb_lanes = load_sb(ks);
            asm volatile("" : "+v"(sb_lanes));  // waited for here, not in every step
          }
          constexpr int first = part == 0 ? 0 : part == 1 ? 3 : 7, past = part == 0 ? 3 : part == 1 ? 7 : 8;
#pragma unroll
          for (int i = first; i < past; ++i) {
            if (i < 7) af[(i + 1) & 1] = read(ra0, ra1, slot + (i + 1) * 2048);
            else af[0] = read(ra0, ra1, (X_SLOT - slot));  // after the last step: in bounds, never used
            float s_raw[8];
            if (i == 0) {
              const lds_u8* const q = rs + ((ks >> 3) & 1) * X_SBUF + (ks & 7) * 32;
#pragma unroll
              for (int x = 0; x < 8; ++x) s_raw[x] = *(lds_f32*)(q + x * X_SSUB);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              promote(acc[(i + 7) & 7][j], p[j], sc[(i + 7) & 7]);
              asm volatile("" : "+v"(acc[(i + 7) & 7][j]));  // here, not where it is next needed
              __builtin_amdgcn_sched_barrier(0);
              p[j] = mfma_block(bf[j], af[i & 1]);
              __builtin_amdgcn_sched_barrier(0);
              if (i == 7) bf[j] = read(rb0, rb1, (X_SLOT - slot) + j * 2048);
              // one load per two MFMAs: a burst would hold up the wave's issue
              if (j & 1) {
                const int n = (i - first) * 2 + (j >> 1);
                if (part == 1 && n < 7 && loads) issue_mid(ks, n, last);
                if (part == 2 && loads) issue_end(ks, n, last);
              }
            }
            if (i == 0) {
              const float sb = __builtin_bit_cast(float, __builtin_amdgcn_readlane(sb_lanes, ks & 63));
#pragma unroll
              for (int x = 0; x < 8; ++x) sc[x] = s_raw[x] * sb;
              __builtin_amdgcn_sched_barrier(0);
            }
          }
        });
#pragma unroll
        for (int j = 0; j < 4; ++j) promote(acc[7][j], p[j], sc[7]);
      } else {
        run([&](int ks, auto part_, bool loads, auto last) __attribute__((always_inline)) {
          constexpr int part = decltype(part_)::value;
          if (part == 1 && loads)
#pragma unroll
            for (int n = 0; n < 7; ++n) issue_mid(ks, n, last);
          if (part == 2 && loads) {
            issue_end(ks, 0, last);
            issue_end(ks, 1, last);
          }
        });
      }
      wait_vmcnt<0>();
      if (more) {
        lds_barrier();  // every wave has read the last step's fragments
        begin_tile();
        first_loads();
      }
    } else if (more) {
      begin_tile();
    }
    if constexpr (!std::is_same_v<E, NoEpilogue>) {
      if (wave_live) epilogue_wave(epilogue, c, at_here, N, acc, col0_here, wm * 128, wn * 64, m_here, n_here);
    } else if (wave_live) {
      if (lines) store_wave_rows<true>(ct, N, acc, wm * 128, wn * 64, m_here, n_here);
      else store_wave_rows<false>(ct, N, acc, wm * 128, wn * 64, m_here, n_here);
    }
    if (!more) return;
  }
}

static hipError_t launch_big(const void* a, const float* sa, const void* bt, const float* sbt, const int32_t* offsets,
                             int G, void* c, int64_t M, int64_t N, int64_t K, const Epilogue* e, hipStream_t stream) {
  const int64_t tiles_n = (N + XBN - 1) / XBN;
  // each range adds at most one partial tile
  const int64_t tiles_m = offsets ? (M + XBM - 1) / XBM + (G < M ? G : M) : (M + XBM - 1) / XBM;
  const int64_t tiles = tiles_m * tiles_n;
  if (tiles > 0x7FFFFFFF) return hipErrorNotSupported;
  // one workgroup per CU (their LDS allows no second one)
  const dim3 grid((unsigned)(tiles < 256 ? tiles : 256));
  auto launch = [&](auto kernel, auto epilogue) {
    hipLaunchKernelGGL(kernel, grid, dim3(XTHREADS), X_LDS, stream, (const uint8_t*)a, sa, (const uint8_t*)bt, sbt,
                       offsets, G, (uint16_t*)c, M, N, K, (uint32_t)tiles_n, (uint32_t)tiles, epilogue);
  };
  if (e) launch(gemm_g128_big_kernel<false, Epilogue>, *e);
  else if (offsets) launch(gemm_g128_big_kernel<true, NoEpilogue>, NoEpilogue());
  else launch(gemm_g128_big_kernel<false, NoEpilogue>, NoEpilogue());
  return hipGetLastError();
}

template <int MI, int NJ, int WM, int WN, int S>
constexpr int tile_lds() {
  return S * (16 * MI * WM + 16 * NJ * WN) * GK + 2 * MI * WM * 576;
}

static hipError_t allow_lds(const void* kernel, int bytes) {
  return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int MI, int NJ, int WM, int WN, int S>
static hipError_t set_tile_attributes() {
  constexpr int LDS = tile_lds<MI, NJ, WM, WN, S>();
  hipError_t e = allow_lds((const void*)gemm_g128_tile_kernel<MI, NJ, WM, WN, S, false, NoEpilogue>, LDS);
  if (e == hipSuccess) e = allow_lds((const void*)gemm_g128_tile_kernel<MI, NJ, WM, WN, S, true, NoEpilogue>, LDS);
  if (e == hipSuccess) e = allow_lds((const void*)gemm_g128_tile_kernel<MI, NJ, WM, WN, S, false, Epilogue>, LDS);
  return e;
}

template <int MI, int NJ, int WM, int WN, int S>
static hipError_t launch_tile(const void* a, const float* sa, const void* bt, const float* sbt,
                              const int32_t* offsets, int G, void* c, int64_t M, int64_t N, int64_t K,
                              const Epilogue* e, hipStream_t stream) {
  constexpr int BM = 16 * MI * WM, BN = 16 * NJ * WN, THREADS = 64 * WM * WN;
  const int64_t tiles_n = (N + BN - 1) / BN;
  // each range adds at most one partial tile
  const int64_t tiles_m = offsets ? (M + BM - 1) / BM + (G < M ? G : M) : (M + BM - 1) / BM;
  if (tiles_m * tiles_n > (int64_t)0xFFFFFFFF / THREADS) return hipErrorNotSupported;
  const dim3 grid((unsigned)(tiles_m * tiles_n));
  auto launch = [&](auto kernel, auto epilogue) {
    hipLaunchKernelGGL(kernel, grid, dim3(THREADS), (tile_lds<MI, NJ, WM, WN, S>()), stream, (const uint8_t*)a, sa,
                       (const uint8_t*)bt, sbt, offsets, G, (uint16_t*)c, M, N, K, (uint32_t)tiles_n, epilogue);
  };
  if (e) launch(gemm_g128_tile_kernel<MI, NJ, WM, WN, S, false, Epilogue>, *e);
  else if (offsets) launch(gemm_g128_tile_kernel<MI, NJ, WM, WN, S, true, NoEpilogue>, NoEpilogue());
  else launch(gemm_g128_tile_kernel<MI, NJ, WM, WN, S, false, NoEpilogue>, NoEpilogue());
  return hipGetLastError();
}

// ---- up to 16 rows of a narrow weight: it is streamed once, straight to registers,
// by workgroups of four waves that own 16 columns of C and all K, so that the few
// columns still occupy every CU.
//
// The waves share K: wave w forms the products of K-blocks 8r + 2w and 8r + 2w + 1
// of round r and puts them into LDS beside their scale products; after one barrier
// the same threads add the round's eight products to their accumulators in
// ascending order.  So many K-blocks are in flight at once, yet an element's
// sequence of operations is that of the tiles, whatever M is.  The next round's
// loads are issued before the round's products are formed.
constexpr int RU = 2, RKC = 4 * RU;  // K-blocks of a wave and of a round

template <typename E>
__global__ void __launch_bounds__(256) gemm_g128_rows_kernel(const uint8_t* __restrict__ a,
                                                             const float* __restrict__ sa,
                                                             const uint8_t* __restrict__ bt,
                                                             const float* __restrict__ sbt,
                                                             result_t<E> c, int64_t M, int64_t N, int64_t K,
                                                             E epilogue) {
  __shared__ __attribute__((aligned(16))) float part[2][RKC][256];
  __shared__ float sprod[2][RKC][16];
  const int lane = threadIdx.x & 63;
  const int w = wave_id_uniform();
  const int g = lane >> 4, lo = lane & 15;
  const int KB = (int)((K + 127) >> 7);
  const bool partial = (K & 127) != 0;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int rounds = (KB + RKC - 1) / RKC;
  const int last = (int)K - 16;  // K offset of the last whole piece
  const int64_t a_row = lo < M ? lo : M - 1;
  const uint8_t* const ap = a + a_row * K;
  const uint8_t* const bp = bt + (n0 + lo) * K;
  const float* const sap = sa + a_row * KB;
  const float* const sbp = sbt + (n0 >> 7) * KB;

  struct Set {
    v4i b[RU][2], a[RU][2];
    float sa, sb;  // of K-block g of the wave's, lanes g < RU
  };
  // Loads past the last K-block repeat it and are not used; pieces past K read the
  // last whole piece and are replaced by zeros.
  auto load = [&](Set& s, int r) __attribute__((always_inline)) {
    const int kb0 = r * RKC + w * RU;
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const int kb = kb0 + u < KB ? kb0 + u : KB - 1;
      int o0 = kb * GK + 16 * g, o1 = o0 + 64;
      o0 = o0 < last ? o0 : last;
      o1 = o1 < last ? o1 : last;
      s.b[u][0] = *reinterpret_cast<const v4i*>(bp + o0);
      s.b[u][1] = *reinterpret_cast<const v4i*>(bp + o1);
      s.a[u][0] = *reinterpret_cast<const v4i*>(ap + o0);
      s.a[u][1] = *reinterpret_cast<const v4i*>(ap + o1);
    }
    const int u = g < RU ? g : RU - 1, kb = kb0 + u < KB ? kb0 + u : KB - 1;
    s.sa = sap[kb];
    s.sb = sbp[kb];
  };
  auto products = [&](Set& s, int r) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const int kb = r * RKC + w * RU + u;
      if (partial && kb == KB - 1) {
        const v4i z = {0, 0, 0, 0};
        const bool in0 = kb * GK + 16 * g < K, in1 = kb * GK + 64 + 16 * g < K;
        s.b[u][0] = in0 ? s.b[u][0] : z;
        s.b[u][1] = in1 ? s.b[u][1] : z;
        s.a[u][0] = in0 ? s.a[u][0] : z;
        s.a[u][1] = in1 ? s.a[u][1] : z;
      }
      auto join = [](v4i x, v4i y) __attribute__((always_inline)) {
        return v8i_t{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
      };
      *reinterpret_cast<v4f*>(&part[r & 1][w * RU + u][lane * 4]) =
          mfma_block(join(s.b[u][0], s.b[u][1]), join(s.a[u][0], s.a[u][1]));
    }
    if (g < RU) sprod[r & 1][w * RU + g][lo] = s.sa * s.sb;
  };

  // thread t owns result t & 3 of lane t >> 2
  const int row = (threadIdx.x >> 2) & 15, col = (threadIdx.x >> 6) * 4 + (threadIdx.x & 3);
  float acc = 0.0f;
  auto chain = [&](int r) __attribute__((always_inline)) {
    const int n = KB - r * RKC < RKC ? KB - r * RKC : RKC;
    auto add = [&](int k) __attribute__((always_inline)) {
      acc = __builtin_fmaf(part[r & 1][k][threadIdx.x], sprod[r & 1][k][row], acc);
    };
    if (n == RKC) {
#pragma unroll
      for (int k = 0; k < RKC; ++k) add(k);
    } else {
      for (int k = 0; k < n; ++k) add(k);
    }
  };

  // A round writes the LDS half that the round before the last one was read from:
  // every thread has passed the barrier between them.
  Set s0, s1;
  load(s0, 0);
  for (int r = 0; r < rounds; r += 2) {
    load(s1, r + 1);
    products(s0, r);
    __syncthreads();
    chain(r);
    if (r + 1 < rounds) {
      load(s0, r + 2);
      products(s1, r + 1);
      __syncthreads();
      chain(r + 1);
    }
  }
  if (row >= M) return;
  const int64_t at = row * N + n0 + col;
  if constexpr (!std::is_same_v<E, NoEpilogue>) {
    auto value = [](const uint16_t* p) __attribute__((always_inline)) { return bf16_lo(*p); };
    if (epilogue.bias != nullptr) acc += value(epilogue.bias + n0 + col);
    if (epilogue.pre != nullptr) epilogue.pre[at] = (uint16_t)bf16_pair(acc, 0.0f);
    with_activation(epilogue.act, [&](auto activate) __attribute__((always_inline)) { acc = activate(acc); });
    if (epilogue.residual != nullptr) acc += value(epilogue.residual + at);
  }
  c[at] = (uint16_t)bf16_pair(acc, 0.0f);
}

hipError_t set_gemm_g128_attributes() {
  hipError_t e = allow_lds((const void*)gemm_g128_big_kernel<false, NoEpilogue>, X_LDS);
  if (e == hipSuccess) e = allow_lds((const void*)gemm_g128_big_kernel<true, NoEpilogue>, X_LDS);
  if (e == hipSuccess) e = allow_lds((const void*)gemm_g128_big_kernel<false, Epilogue>, X_LDS);
  if (e == hipSuccess) e = set_tile_attributes<4, 4, 2, 4, 3>();
  if (e == hipSuccess) e = set_tile_attributes<4, 4, 2, 2, 2>();
  if (e == hipSuccess) e = set_tile_attributes<2, 4, 4, 2, 3>();
  if (e == hipSuccess) e = set_tile_attributes<2, 4, 2, 2, 2>();
  if (e == hipSuccess) e = set_tile_attributes<2, 2, 2, 4, 3>();
  if (e == hipSuccess) e = set_tile_attributes<2, 2, 2, 2, 4>();
  if (e == hipSuccess) e = set_tile_attributes<1, 2, 2, 2, 3>();
  if (e == hipSuccess) e = set_tile_attributes<1, 1, 2, 2, 4>();
  return e;
}

// The kernel is the largest tile that still gives the 256 CUs enough workgroups: a
// larger tile moves fewer bytes per flop, but tiles that do not fill the chip
// leave CUs idle.  Time per K-block, ns, by the number of tiles (8w: eight waves
// and three K-blocks in the ring, one or two workgroups a CU; else four waves and
// two to four; the last column is the whole call's overhead at 256 tiles, us):
//              128   256   288   512   768   1024
//   256x256   1045  1506        3092                9
//   128x256 8w 848  1024  1742  1977  2980  3825     5
//   128x128 8w 554   591  1105  1258  1866  2390     4
//   128x128    664   703   809   994  1655  1992     4
//   64x128 8w  389   408   539   628  1001  1257     4
//   64x128     556   572   560   611   965  1428     3
//   64x64      262   295   365   427   635   777     4
//   32x64      226   240   284   304   445   568     3
//   32x32      189   206   230   237   313   410     3
// (1536 x 7168 x 4096: 256x256 [168 tiles] 47 us, 128x128 59; 256 x 28672 x 8192:
// 128x256 8w [224] 75, 128x128 [448] 87; 1540 x 832 x 7648: 64x128 8w [175] 30, 32x64
// 41.)  One row tile of a wide weight is bound by the weight's stream, which needs
// bytes in flight: the ring of 64x64 is four K-blocks deep (8 x 28672 x 8192: 45,
// 32x64 with three 48).  Up to 16 rows of a narrow weight: 16 x 4096 x 4096 rows 6.9,
// 32x32 [128] 8.5; 8 x 8192 x 8192 32x32 [256] 13.8, rows 16.6.
// A range has half a tile too much on average, which the count includes, and a tile
// is not chosen much taller than the ranges: rows past a range's end are work for
// nothing (ranges x average rows, N x K: 64 x 8, 4096 x 2048: 32x64 94, 64x128 94;
// 16 x 25, 4096 x 7168: 64x128 74, 128x128 82; 16 x 56: 128x256 8w 84, 64x128 95;
// 16 x 125, 4096 x 2048: 256x256 35, 128x256 8w 41, 64x128 44; 16 x 250, 2048 x 4096:
// 256x256 55, 128x128 70).  Over 90 dense and 90 ragged sizes drawn from 17 to 8192
// rows the choice is 1.5% and 3% slower than the best of these tiles on average; what
// none of them reaches this does not see (32 x 576 x 7168 is 18 workgroups of 56
// K-blocks one after another: 13.7 us).
static hipError_t launch(const void* a, const float* sa, const void* bt, const float* sbt, const int32_t* offsets,
                         int G, void* c, int64_t M, int64_t N, int64_t K, const Epilogue* e, hipStream_t stream) {
  const int64_t live = G < M ? G : M;           // ranges that can have rows
  const int64_t avg = (M + live - 1) / live;    // rows of one
  auto tiles = [&](int64_t bm, int64_t bn) {
    const int64_t rows = offsets ? std::max(live, (M + live * (bm / 2)) / bm) : (M + bm - 1) / bm;
    return rows * ((N + bn - 1) / bn);
  };
  if (!offsets && K > 0 && M <= 16 && tiles(32, 32) < 200) {
    auto rows = [&](auto kernel, auto epilogue) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)(N / 16)), dim3(256), 0, stream, (const uint8_t*)a, sa,
                         (const uint8_t*)bt, sbt, (uint16_t*)c, M, N, K, epilogue);
    };
    if (e) rows(gemm_g128_rows_kernel<Epilogue>, *e);
    else rows(gemm_g128_rows_kernel<NoEpilogue>, NoEpilogue());
    return hipGetLastError();
  }
  const int64_t big = tiles(256, 256), wide = tiles(128, 256), square = tiles(128, 128), low = tiles(64, 128);
  const int64_t small = tiles(64, 64);
  if (avg >= (offsets ? 112 : 160) && big >= 160)
    return launch_big(a, sa, bt, sbt, offsets, G, c, M, N, K, e, stream);
  if (avg >= (offsets ? 48 : 65) && wide >= 150 && wide <= 256)
    return launch_tile<4, 4, 2, 4, 3>(a, sa, bt, sbt, offsets, G, c, M, N, K, e, stream);
  if (avg > 64 && square >= 200 && square <= 256)
    return launch_tile<2, 4, 4, 2, 3>(a, sa, bt, sbt, offsets, G, c, M, N, K, e, stream);
  if (avg >= 128 && square > 256)
    return launch_tile<4, 4, 2, 2, 2>(a, sa, bt, sbt, offsets, G, c, M, N, K, e, stream);
  if (!offsets && M <= 64 && small > 256)
    return launch_tile<2, 2, 2, 2, 4>(a, sa, bt, sbt, offsets, G, c, M, N, K, e, stream);
  if (avg >= 20 && low > 256)
    return launch_tile<2, 4, 2, 2, 2>(a, sa, bt, sbt, offsets, G, c, M, N, K, e, stream);
  if (avg >= 20 && low > 128)
    return launch_tile<2, 2, 2, 4, 3>(a, sa, bt, sbt, offsets, G, c, M, N, K, e, stream);
  if (avg > 32 && small > 128 && small <= 256)
    return launch_tile<2, 2, 2, 2, 4>(a, sa, bt, sbt, offsets, G, c, M, N, K, e, stream);
  if (tiles(32, 64) >= 150) return launch_tile<1, 2, 2, 2, 3>(a, sa, bt, sbt, offsets, G, c, M, N, K, e, stream);
  return launch_tile<1, 1, 2, 2, 4>(a, sa, bt, sbt, offsets, G, c, M, N, K, e, stream);
}

hipError_t launch_gemm_g128(const void* a, const float* sa, const void* bt, const float* sbt, const int32_t* offsets,
                            int G, void* c, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  return launch(a, sa, bt, sbt, offsets, G, c, M, N, K, nullptr, stream);
}

hipError_t launch_gemm_g128_epilogue(const void* a, const float* sa, const void* bt, const float* sbt,
                                     const Epilogue& e, void* c, int64_t M, int64_t N, int64_t K,
                                     hipStream_t stream) {
  return launch(a, sa, bt, sbt, nullptr, 1, c, M, N, K, &e, stream);
}

}  // namespace fp8bs
