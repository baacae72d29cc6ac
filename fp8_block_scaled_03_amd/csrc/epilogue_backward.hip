// The backward pass of a product's epilogue C = act(z) + residual, z = A B + bias:
//
//   dz = dC act'(z), rounded to bf16 for the weight gradient, and as codes with a scale
//   per row and 128 columns of the fp32 values for the input gradient's product;
//   dbias = sum over the rows of the fp32 dz.
//
// A wave takes 128 columns (16 lanes of eight) of four rows at a time and walks every
// `slabs`-th such set of rows; its columns' sums stay in registers, are joined over
// the four rows by two lane exchanges and written once to the workspace, and a second
// launch adds the slabs' sums in order.  Slabs depend on the sizes only.  The next
// set's loads are in flight while one is worked on.
//
// Bound by HBM traffic (7 bytes a value, 5 without z; 8192 x 16384, gelu, 168 us, 5.6 TB/s), for
// gelu nearly as much by the VALU: about 45 issue slots a value.  Few rows are latency (the slabs below).
#include "activation.hpp"
#include "column_sum.hpp"
#include "launch_layer.hpp"
#include "quant_g128.hpp"
#include "stream.hpp"

#include <type_traits>

namespace fp8bs {

template <int ACT, bool LINES, bool PAST>
__global__ void __launch_bounds__(256) epilogue_backward_kernel(const uint16_t* __restrict__ dout,
                                                                const uint16_t* __restrict__ z, int64_t rows,
                                                                int64_t n, uint16_t* __restrict__ dz,
                                                                uint8_t* __restrict__ q, float* __restrict__ scales,
                                                                float* __restrict__ partial, uint32_t slabs) {
  const int lane = threadIdx.x & 63, piece = lane & 15, rsub = lane >> 4;
  const uint32_t nb = (uint32_t)((n + 127) >> 7);
  const uint32_t task = region_at<LINES>(blockIdx.x, gridDim.x) * 4 + wave_id_uniform();
  const uint32_t slab = task / nb, cb = task - slab * nb;
  if (slab >= slabs) return;
  const int64_t col = (int64_t)cb * 128 + piece * 8;
  const bool in = col < n;
  const int64_t from = in ? col : 0;  // lanes past n read column 0 and count as zeros
  auto load = [&](int64_t set, uint4& d, uint4& x) __attribute__((always_inline)) {
    const int64_t row = set * 4 + rsub < rows ? set * 4 + rsub : rows - 1;
    d = load_once<PAST>(dout + row * n + from);
    if constexpr (ACT != ACT_NONE) x = load_once<PAST>(z + row * n + from);
  };
  const int64_t sets = (rows + 3) >> 2;
  float sums[8] = {};
  uint4 d_next, z_next = make_uint4(0, 0, 0, 0);
  load(slab, d_next, z_next);
  for (int64_t set = slab; set < sets; set += slabs) {
    const uint4 dw = d_next, zw = z_next;
    load(set + slabs < sets ? set + slabs : set, d_next, z_next);
    const int64_t row = set * 4 + rsub;
    const bool ok = in && row < rows;
    float v[8], x[8];
    unpack8(dw, v);
    unpack8(zw, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (ACT != ACT_NONE) v[i] *= slope<ACT>(x[i]);
      v[i] = ok ? v[i] : 0.0f;
      sums[i] += v[i];
    }
    const Scale sc = scale_of(row16_max(amax8(v)));
    const uint2 codes = __all(sc.r != 0.0f || !ok) ? codes8<true>(v, sc) : codes8<false>(v, sc);
    if (ok) {
      if (dz != nullptr) store_once<PAST>(dz + row * n + col, bf16_round8(v));
      put_codes8<LINES && !PAST>(q + row * n + col, codes);
      if (piece == 0) scales[row * nb + cb] = sc.s;
    }
  }
  if (partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sums[i] += __shfl_xor(sums[i], 16, 64);
    sums[i] += __shfl_xor(sums[i], 32, 64);
  }
  if (rsub == 0 && in) {
    float4* const out = reinterpret_cast<float4*>(partial + (int64_t)slab * n + col);
    out[0] = make_float4(sums[0], sums[1], sums[2], sums[3]);
    out[1] = make_float4(sums[4], sums[5], sums[6], sums[7]);
  }
}

// At least eight sets of four rows to a slab, so that the partial sums are few beside
// the rows, and at most 8192 waves in all, which fill the chip.  With few rows the sets are walked one
// after another by few waves (in a graph, gelu: 8 x 8192 6.0 us, 256 x 4096 12.3, 1017 x 2064 13.5, of
// which two launches are 4.8).
static int64_t epilogue_slabs(int64_t rows, int64_t n) {
  const int64_t sets = (rows + 3) / 4, nb = (n + 127) / 128;
  const int64_t most = nb < 8192 ? 8192 / nb : 1, want = (sets + 7) / 8;
  return want < most ? want : most;
}

int64_t epilogue_backward_workspace(int64_t rows, int64_t n) { return epilogue_slabs(rows, n) * n * 4; }

hipError_t launch_epilogue_backward(const void* dout, const void* z, int act, int64_t rows, int64_t n, void* dz,
                                    void* q, float* scales, float* dbias, bool accumulate, float* workspace,
                                    hipStream_t stream) {
  const int64_t slabs = epilogue_slabs(rows, n), tasks = slabs * ((n + 127) / 128);
  if (rows > 0) {
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)((tasks + 3) / 4)), dim3(256), 0, stream, (const uint16_t*)dout,
                         (const uint16_t*)z, rows, n, (uint16_t*)dz, (uint8_t*)q, scales,
                         dbias ? workspace : nullptr, (uint32_t)slabs);
    };
    const bool past = rows * n * (act == ACT_NONE ? 2 : 4) > INPUTS_PAST;
    auto choose = [&](auto act_) {
      constexpr int ACT = decltype(act_)::value;
      if (n % 128 == 0)
        past ? launch(epilogue_backward_kernel<ACT, true, true>) : launch(epilogue_backward_kernel<ACT, true, false>);
      else
        past ? launch(epilogue_backward_kernel<ACT, false, true>) : launch(epilogue_backward_kernel<ACT, false, false>);
    };
    switch (act) {
      case ACT_RELU: choose(std::integral_constant<int, ACT_RELU>()); break;
      case ACT_GELU: choose(std::integral_constant<int, ACT_GELU>()); break;
      case ACT_GELU_TANH: choose(std::integral_constant<int, ACT_GELU_TANH>()); break;
      case ACT_SILU: choose(std::integral_constant<int, ACT_SILU>()); break;
      default: choose(std::integral_constant<int, ACT_NONE>());
    }
  }
  if (dbias) launch_column_sum(workspace, rows > 0 ? (unsigned)slabs : 0, n, n, dbias, nullptr, accumulate, stream);
  return hipGetLastError();
}

}  // namespace fp8bs
