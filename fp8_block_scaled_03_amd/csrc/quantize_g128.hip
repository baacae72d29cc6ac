// bf16 -> E4M3 quantizers with one scale per row and 128 columns, and per
// 128x128 block (with the transposed codes on request).
//
// Per group: amax = max |x|, s = amax / 448 in fp32, q = E4M3(x / s); the
// quotient is formed from the scale's reciprocal and one correction (see
// quantize.hip), the same bits as a division.  Both kernels are bound by HBM
// traffic: two bytes read, one written (two with the transpose) per value.
//
// Sixteen lanes hold a group's 128 columns of one row, eight (16 bytes) each, so
// a wave's load covers four rows of 256 bytes and a group's maximum is found
// by DPP exchanges inside a row of lanes.
#include "launch_g128.hpp"
#include "quant_g128.hpp"
#include "ragged.hpp"

#include <type_traits>

namespace fp8bs {

// A region is 4U rows x 512 columns, 128 columns (a group) per wave; all U loads of
// a lane are in flight before any arithmetic.  LINES as in put_codes8 (32768 x 2048
// with it 35 us, without 40; 32768 x 2064 45 and 43, 3000 x 4112 9.8 and 8.1).
template <int U, bool LINES>
__global__ void __launch_bounds__(256) quantize_tg128_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                             int64_t cols, uint8_t* __restrict__ q,
                                                             float* __restrict__ scales, uint32_t n_regions) {
  const int lane = threadIdx.x & 63;
  const int piece = lane & 15, rsub = lane >> 4;
  const uint32_t nb = (uint32_t)((cols + 127) >> 7), quads = (nb + 3) >> 2;
  for (uint32_t id = blockIdx.x; id < n_regions; id += gridDim.x) {
    const uint32_t reg = region_at<LINES>(id, n_regions);
    const uint32_t rb = reg / quads, cb = (reg - rb * quads) * 4 + (threadIdx.x >> 6);
    const int64_t row0 = (int64_t)rb * (4 * U) + rsub;
    const int64_t col = (int64_t)cb * 128 + piece * 8;
    uint4 w[U];
    bool ok[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t row = row0 + 4 * k;
      ok[k] = row < rows && col < cols;
      w[k] = ok[k] ? *reinterpret_cast<const uint4*>(x + row * cols + col) : make_uint4(0, 0, 0, 0);
    }
    Scale sc[U];
    bool all_recip = true;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      sc[k] = scale_of(row16_max(amax_bf16x8(w[k])));
      all_recip = all_recip && (sc[k].r != 0.0f || !ok[k]);
    }
    auto store = [&](auto RECIP_) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int64_t row = row0 + 4 * k;
        float v[8];
        unpack8(w[k], v);
        const uint2 p = codes8<decltype(RECIP_)::value>(v, sc[k]);
        if (ok[k]) {
          put_codes8<LINES>(q + row * cols + col, p);
          if (piece == 0) scales[row * nb + cb] = sc[k].s;
        }
      }
    };
    // every group of the wave on the reciprocal path (the common case): no
    // per-element branches
    if (__all(all_recip)) store(std::true_type{});
    else store(std::false_type{});
  }
}

// Four bytes of four rows, transposed: dword c of the result holds byte c of
// r0, r1, r2, r3.
__device__ __forceinline__ void transpose4x4(uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3, uint32_t (&o)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(r1, r0, 0x05010400u);  // r0.0 r1.0 r0.1 r1.1
  const uint32_t b = __builtin_amdgcn_perm(r1, r0, 0x07030602u);  // r0.2 r1.2 r0.3 r1.3
  const uint32_t c = __builtin_amdgcn_perm(r3, r2, 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(r3, r2, 0x07030602u);
  o[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// 16 bytes, past the caches if PAST.
template <bool PAST>
__device__ __forceinline__ uint4 load16(const uint16_t* p) {
  if constexpr (PAST) {
    typedef unsigned v4u __attribute__((ext_vector_type(4)));
    const v4u v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
    return make_uint4(v[0], v[1], v[2], v[3]);
  } else {
    return *reinterpret_cast<const uint4*>(p);
  }
}

// One 256-thread workgroup per 128x128 block.  Lane (piece, rsub) of wave w holds
// rows 32w + 8 rsub .. +7 of columns 8 piece .. +7, an 8x8 square that it transposes
// by byte permutes; the transposed codes go through LDS so that whole
// 128-byte rows of qt are written.
constexpr int TPAD = 128 + 16;  // LDS row of 128 codes, 16-byte aligned, rows 4 banks apart

// LINES: columns are multiples of 128, so the lines of a block's rows belong to it
// alone: they are read and written past the caches (8 x 4096 x 2048 with the
// transpose 51 us, 61 through the L2).  Otherwise, or if the transposed rows are no
// multiples of 128, neighbouring blocks share lines: they are walked in runs per
// XCD and the shared lines go through its L2, which joins them (8 x 4112 x 2064 with
// the transpose 76 us, past the caches 93; 8 x 4112 x 2048 63 us).
template <bool TRANSPOSED, bool LINES>
__global__ void __launch_bounds__(256) quantize_b128_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                            int64_t cols, uint8_t* __restrict__ q,
                                                            float* __restrict__ scales, uint8_t* __restrict__ qt,
                                                            float* __restrict__ scales_t, uint32_t rb_count,
                                                            uint32_t cb_count, bool runs) {
  __shared__ uint32_t wave_max[4];
  __shared__ __attribute__((aligned(16))) uint8_t tile[TRANSPOSED ? 128 * TPAD : 16];
  const int lane = threadIdx.x & 63;
  const int w = threadIdx.x >> 6;
  const int piece = lane & 15, rsub = lane >> 4;
  const uint32_t id = runs ? xcd_run(blockIdx.x, gridDim.x) : blockIdx.x;
  const uint32_t cb = id % cb_count, rest = id / cb_count;
  const uint32_t rb = rest % rb_count;
  const int64_t gi = rest / rb_count;
  x += gi * rows * cols;
  q += gi * rows * cols;
  const int64_t col = (int64_t)cb * 128 + piece * 8;
  const int r0 = 32 * w + 8 * rsub;
  uint4 v[8];
  bool ok[8];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t row = (int64_t)rb * 128 + r0 + k;
    ok[k] = row < rows && col < cols;
    v[k] = ok[k] ? load16<LINES>(x + row * cols + col) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t mk = amax_bf16x8(v[k]);
    m = m > mk ? m : mk;
  }
  m = row16_max(m);
#pragma unroll
  for (int d = 16; d <= 32; d <<= 1) {
    const uint32_t o = __shfl_xor(m, d, 64);
    m = m > o ? m : o;
  }
  if (lane == 0) wave_max[w] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) m = m > wave_max[i] ? m : wave_max[i];
  const Scale sc = scale_of(m);
  uint2 p[8];
  if (sc.r != 0.0f) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float f[8];
      unpack8(v[k], f);
      p[k] = codes8<true>(f, sc);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float f[8];
      unpack8(v[k], f);
      p[k] = codes8<false>(f, sc);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t row = (int64_t)rb * 128 + r0 + k;
    if (ok[k]) {
      put_codes8<LINES>(q + row * cols + col, p[k]);
    }
  }
  if (threadIdx.x == 0) {
    scales[(gi * rb_count + rb) * cb_count + cb] = sc.s;
    if constexpr (TRANSPOSED) scales_t[(gi * cb_count + cb) * rb_count + rb] = sc.s;
  }
  if constexpr (TRANSPOSED) {
    qt += gi * rows * cols;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // columns 4h .. 4h + 3 of the lane's eight
      uint32_t lo[4], hi[4];
      auto word = [&](int k) __attribute__((always_inline)) { return h == 0 ? p[k].x : p[k].y; };
      transpose4x4(word(0), word(1), word(2), word(3), lo);
      transpose4x4(word(4), word(5), word(6), word(7), hi);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint2*>(tile + (piece * 8 + 4 * h + c) * TPAD + r0) = make_uint2(lo[c], hi[c]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 32 columns of the block per pass, eight lanes of 16 bytes each
      const int c = i * 32 + (threadIdx.x >> 3), r = (threadIdx.x & 7) * 16;
      const int64_t qc = (int64_t)cb * 128 + c, qr = (int64_t)rb * 128 + r;
      if (qc < cols && qr < rows)
        *reinterpret_cast<uint4*>(qt + qc * rows + qr) = *reinterpret_cast<const uint4*>(tile + c * TPAD + r);
    }
  }
}

hipError_t launch_quantize_tg128(const void* x, int64_t rows, int64_t cols, void* q, float* scales,
                                 hipStream_t stream) {
  const int64_t quads = (cols + 511) / 512;
  // few rows: one load per lane, more waves
  const int u = (rows + 7) / 8 * quads >= 512 ? 2 : 1;
  const int64_t n_regions = (rows + 4 * u - 1) / (4 * u) * quads;
  if (n_regions > MAX_REGIONS) return hipErrorNotSupported;
  auto go = [&](auto U_, auto LINES_) {
    hipLaunchKernelGGL((quantize_tg128_kernel<decltype(U_)::value, decltype(LINES_)::value>),
                       dim3((unsigned)(n_regions < MAX_GRID ? n_regions : MAX_GRID)), dim3(256), 0, stream,
                       (const uint16_t*)x, rows, cols, (uint8_t*)q, scales, (uint32_t)n_regions);
  };
  const bool lines = cols % 128 == 0;
  using std::integral_constant;
  if (u == 2 && lines) go(integral_constant<int, 2>{}, std::true_type{});
  else if (u == 2) go(integral_constant<int, 2>{}, std::false_type{});
  else if (lines) go(integral_constant<int, 1>{}, std::true_type{});
  else go(integral_constant<int, 1>{}, std::false_type{});
  return hipGetLastError();
}

hipError_t launch_quantize_b128(const void* x, int64_t G, int64_t rows, int64_t cols, void* q, float* scales,
                                void* qt, float* scales_t, hipStream_t stream) {
  const int64_t rb = (rows + 127) / 128, cb = (cols + 127) / 128;
  const bool runs = cols % 128 != 0 || (qt && rows % 128 != 0);
  auto go = [&](auto TRANSPOSED_, auto LINES_) {
    hipLaunchKernelGGL((quantize_b128_kernel<decltype(TRANSPOSED_)::value, decltype(LINES_)::value>),
                       dim3((unsigned)(G * rb * cb)), dim3(256), 0, stream, (const uint16_t*)x, rows, cols,
                       (uint8_t*)q, scales, (uint8_t*)qt, scales_t, (uint32_t)rb, (uint32_t)cb, runs);
  };
  const bool lines = cols % 128 == 0;
  if (qt && lines) go(std::true_type{}, std::true_type{});
  else if (qt) go(std::true_type{}, std::false_type{});
  else if (lines) go(std::false_type{}, std::true_type{});
  else go(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

}  // namespace fp8bs
