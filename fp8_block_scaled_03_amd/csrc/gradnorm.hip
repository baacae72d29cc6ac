// The norm over the gradients of many tensors, and their clipping.
//
//   total = sum g^2,  norm = sqrt(total),  out = g * min(1, max_norm / (norm + eps))
//
// Squares and sums are 64-bit: a bf16 or fp32 square neither overflows nor
// vanishes there, and the sum of 2^30 values is right to fp32's last bit.
//
// A tensor is cut into chunks of 8 or 32 KB from the 16-byte boundary at or before
// its first value, so that every 16-byte piece but a tensor's first and last is whole
// and aligned.  A launch takes up to TABLE tensors, whose addresses and first
// chunks are kernel arguments (nothing is copied to the device, so a captured graph
// holds them); a workgroup takes every gridDim.x-th chunk, finds its tensor with one
// comparison per lane, and leaves one partial sum.  The clipping kernel's workgroups
// each add up the partial sums, in the same order, so two launches do the whole.
#include "common.hpp"
#include "launch_layer.hpp"
#include "stream.hpp"

namespace fp8bs {

constexpr int TABLE = 96;
constexpr int GRAD_GRID = 1024;
// Pieces of 16 bytes that a thread has of a chunk.  While 8 KB a workgroup are enough for all, more
// workgroups share the latency; above, larger chunks have more loads in flight (us in a graph, norm and
// clipping into other tensors, one list again and again, 32 KB and 8 KB: 61 x 4096 values 9.2 and 6.4, 61 x 20000
// 9.7 and 7.9, 61 x 50000 11.4 and 11.5, 403 M 842 and 969; in place 61 x 20000 11.4 and 10.2).
constexpr int FEW = 2, MANY = 8;
constexpr int64_t chunk_bytes(int pieces) { return int64_t(256) * 16 * pieces; }
constexpr int64_t SMALL_LIST = GRAD_GRID * chunk_bytes(FEW);  // bytes of all gradients
constexpr int64_t JOIN_MAX = 4096;  // partial sums that every workgroup of the clipping kernel adds up by itself

struct GradTable {
  const uint8_t* src[TABLE];
  uint8_t* dst[TABLE];
  int64_t n[TABLE];
  uint32_t first[TABLE + 1];  // first chunk; entries behind the last tensor hold the end
  uint8_t bf16[TABLE];
};

// Gradients beyond what the caches keep are read past them.  Of 256 MB of Infinity Cache a
// norm that fits leaves the clipping its gradients; above that, lines that are
// not kept cost nothing to replace (403 M values: norm 285 us through the caches, 209 past
// them; clipping 531 and 519; but 32 M values, 112 MB, 66 us in place through the caches and 73).
constexpr int64_t NORM_PAST = int64_t(512) << 20, CLIP_PAST = int64_t(192) << 20;  // bytes of all gradients

typedef uint4 piece_t;
template <bool PAST>
__device__ __forceinline__ piece_t load_piece(const piece_t* p) {
  return load_once<PAST>(reinterpret_cast<const uint16_t*>(p));
}
__device__ __forceinline__ void store_piece(uint8_t* p, piece_t v) {  // (it is read in another step of the program)
  store_once<true>(reinterpret_cast<uint16_t*>(p), v);
}
struct __attribute__((packed, aligned(2))) loose_piece_t {
  uint32_t v[4];
};

// The sum of one double per thread of a workgroup of 256, in every thread.
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) lds[w] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// Tensor that holds `chunk`.
__device__ __forceinline__ int tensor_of(const GradTable& t, uint32_t chunk) {
  const int lane = threadIdx.x & 63;
  const uint32_t a = t.first[lane + 1], b = t.first[lane + 65 < TABLE ? lane + 65 : TABLE];
  const int below = __popcll(__ballot(a <= chunk)) + __popcll(__ballot(lane + 65 <= TABLE && b <= chunk));
  return __builtin_amdgcn_readfirstlane(below);
}

__device__ __forceinline__ void add_squares(piece_t v, bool bf16, double (&acc)[2]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      const double lo = bf16_lo(w[i]), hi = bf16_hi(w[i]);
      acc[0] = __builtin_fma(lo, lo, acc[0]);
      acc[1] = __builtin_fma(hi, hi, acc[1]);
    } else {
      const double x = __builtin_bit_cast(float, w[i]);
      acc[i & 1] = __builtin_fma(x, x, acc[i & 1]);
    }
  }
}

template <bool PAST, int P>
__global__ void __launch_bounds__(256) grad_sumsq_kernel(GradTable t, uint32_t chunks, double* __restrict__ partial) {
  __shared__ double lds[4];
  constexpr int64_t CHUNK = chunk_bytes(P);
  double acc[2] = {0.0, 0.0};
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int k = tensor_of(t, c);
    const bool bf16 = t.bf16[k];
    const uint8_t* const p = t.src[k];
    const int lead = (int)((uintptr_t)p & 15);
    const int64_t end = lead + (t.n[k] << (bf16 ? 1 : 2));   // from the boundary before p
    const int64_t at = (int64_t)(c - t.first[k]) * CHUNK;
    const uint8_t* const q = p - lead + at;
    if (at >= lead && at + CHUNK <= end) {
      piece_t v[P];
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = load_piece<PAST>(reinterpret_cast<const piece_t*>(q) + i * 256 + threadIdx.x);
#pragma unroll
      for (int i = 0; i < P; ++i) add_squares(v[i], bf16, acc);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int off = (i * 256 + threadIdx.x) * 16;
        if (at + off >= lead && at + off + 16 <= end) {
          add_squares(*reinterpret_cast<const piece_t*>(q + off), bf16, acc);
        } else {
          const int step = bf16 ? 2 : 4;
          for (int e = 0; e < 16; e += step) {
            if (at + off + e < lead || at + off + e >= end) continue;
            const double x = bf16 ? bf16_lo(*reinterpret_cast<const uint16_t*>(q + off + e))
                                  : *reinterpret_cast<const float*>(q + off + e);
            acc[0] = __builtin_fma(x, x, acc[0]);
          }
        }
      }
    }
  }
  const double sum = block_sum(acc[0] + acc[1], lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__device__ __forceinline__ double join(const double* __restrict__ partial, int64_t n, double* lds) {
  double v = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 256) v += partial[i];
  return block_sum(v, lds);
}

// total (if given) and norm (if given) from n partial sums; one workgroup.
__global__ void __launch_bounds__(256) grad_join_kernel(const double* __restrict__ partial, int64_t n,
                                                        double* __restrict__ total, float* __restrict__ norm) {
  __shared__ double lds[4];
  const double sum = join(partial, n, lds);
  if (threadIdx.x == 0) {
    if (total) *total = sum;
    if (norm) *norm = (float)__builtin_sqrt(sum);
  }
}

__device__ __forceinline__ piece_t scaled(piece_t v, bool bf16, float f) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      typedef float v2f __attribute__((ext_vector_type(2)));
      const v2f x = {bf16_lo(w[i]) * f, bf16_hi(w[i]) * f};
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2bf));
    } else {
      w[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, w[i]) * f);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// n partial sums, or (partial null) the norm at norm_in.
template <bool PAST, int P>
__global__ void __launch_bounds__(256) clip_kernel(GradTable t, uint32_t chunks, const double* __restrict__ partial,
                                                   int n, const float* __restrict__ norm_in, double max_norm,
                                                   double eps, float* __restrict__ norm_out) {
  __shared__ double lds[4];
  constexpr int64_t CHUNK = chunk_bytes(P);
  const double norm = partial ? __builtin_sqrt(join(partial, n, lds)) : (double)*norm_in;
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const double wanted = max_norm / (norm + eps);
  const float f = (float)(wanted >= 1.0 ? 1.0 : wanted);  // a NaN stays
  for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const uint32_t c = chunks - 1 - i;  // backwards: the last chunks that the norm read are still in the caches
    const int k = tensor_of(t, c);
    const uint8_t* const p = t.src[k];
    uint8_t* const d = t.dst[k];
    if (f == 1.0f && d == p) continue;
    const bool bf16 = t.bf16[k];
    const int lead = (int)((uintptr_t)p & 15);
    const int64_t end = lead + (t.n[k] << (bf16 ? 1 : 2));
    const int64_t at = (int64_t)(c - t.first[k]) * CHUNK;
    const uint8_t* const q = p - lead + at;
    uint8_t* const o = d - lead + at;
    const bool even = ((uintptr_t)o & 15) == 0;
    if (at >= lead && at + CHUNK <= end) {
      piece_t v[P];
#pragma unroll
      for (int j = 0; j < P; ++j) v[j] = load_piece<PAST>(reinterpret_cast<const piece_t*>(q) + j * 256 + threadIdx.x);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const piece_t r = scaled(v[j], bf16, f);
        const int64_t off = (j * 256 + threadIdx.x) * 16;
        if (even) store_piece(o + off, r);
        else *reinterpret_cast<loose_piece_t*>(o + off) = loose_piece_t{{r.x, r.y, r.z, r.w}};
      }
    } else {
      for (int j = 0; j < P; ++j) {
        const int off = (j * 256 + threadIdx.x) * 16;
        const int step = bf16 ? 2 : 4;
        if (even && at + off >= lead && at + off + 16 <= end) {
          *reinterpret_cast<piece_t*>(o + off) = scaled(*reinterpret_cast<const piece_t*>(q + off), bf16, f);
          continue;
        }
        for (int e = 0; e < 16; e += step) {
          if (at + off + e < lead || at + off + e >= end) continue;
          if (bf16) {
            const uint32_t x = *reinterpret_cast<const uint16_t*>(q + off + e);
            *reinterpret_cast<uint16_t*>(o + off + e) = (uint16_t)scaled(make_uint4(x, 0, 0, 0), true, f).x;
          } else {
            *reinterpret_cast<float*>(o + off + e) = *reinterpret_cast<const float*>(q + off + e) * f;
          }
        }
      }
    }
  }
}

// The workspace: the joined total, one unused, then GRAD_GRID partial sums for each launch.
int64_t grad_norm_workspace(int n) { return 8 * (2 + (int64_t)((n + TABLE - 1) / TABLE) * GRAD_GRID); }

static uint32_t fill_table(const Grads& g, int first, int64_t chunk, GradTable& t) {
  uint32_t chunks = 0;
  for (int i = 0; i < TABLE; ++i) {
    const int k = first + i;
    const int64_t count = k < g.n ? g.counts[k] : 0;
    t.src[i] = (const uint8_t*)(k < g.n ? g.src[k] : nullptr);
    t.dst[i] = (uint8_t*)(k < g.n && g.dst ? g.dst[k] : nullptr);
    t.n[i] = count;
    t.bf16[i] = k < g.n && g.types[k] == 1;
    t.first[i] = chunks;
    if (count > 0) chunks += (uint32_t)((((uintptr_t)t.src[i] & 15) + count * (t.bf16[i] ? 2 : 4) + chunk - 1) / chunk);
  }
  t.first[TABLE] = chunks;
  return chunks;
}

static unsigned grad_grid(uint32_t chunks) { return chunks < GRAD_GRID ? chunks : GRAD_GRID; }

static int64_t grad_bytes(const Grads& g) {
  int64_t bytes = 0;
  for (int i = 0; i < g.n; ++i) bytes += g.counts[i] * (g.types[i] == 1 ? 2 : 4);
  return bytes;
}

// Partial sums of all tensors at workspace + 2; their number.
static int64_t launch_sumsq(const Grads& g, double* workspace, hipStream_t stream) {
  const int64_t bytes = grad_bytes(g);
  const bool few = bytes <= SMALL_LIST;
  const auto kernel = few ? grad_sumsq_kernel<false, FEW>
                          : bytes > NORM_PAST ? grad_sumsq_kernel<true, MANY> : grad_sumsq_kernel<false, MANY>;
  int64_t used = 0;
  for (int first = 0; first < g.n; first += TABLE) {
    GradTable t;
    const uint32_t chunks = fill_table(g, first, chunk_bytes(few ? FEW : MANY), t);
    if (chunks == 0) continue;
    const unsigned grid = grad_grid(chunks);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, stream, t, chunks, workspace + 2 + used);
    used += grid;
  }
  return used;
}

hipError_t launch_grad_norm(const Grads& g, float* norm, double* workspace, hipStream_t stream) {
  const int64_t used = launch_sumsq(g, workspace, stream);
  hipLaunchKernelGGL(grad_join_kernel, dim3(1), dim3(256), 0, stream, workspace + 2, used, (double*)nullptr, norm);
  return hipGetLastError();
}

hipError_t launch_clip_grads(const Grads& g, double max_norm, double eps, float* norm, double* workspace,
                             hipStream_t stream) {
  const double* partial = nullptr;
  float* norm_out = nullptr;
  int64_t used = 0;
  if (workspace) {
    used = launch_sumsq(g, workspace, stream);
    partial = workspace + 2;
    norm_out = norm;
    if (used > JOIN_MAX || used == 0) {
      hipLaunchKernelGGL(grad_join_kernel, dim3(1), dim3(256), 0, stream, partial, used, workspace, norm);
      partial = workspace;
      used = 1;
      norm_out = nullptr;
    }
  }
  const int64_t bytes = grad_bytes(g);
  const bool few = bytes <= SMALL_LIST;
  const auto kernel =
      few ? clip_kernel<false, FEW> : bytes > CLIP_PAST ? clip_kernel<true, MANY> : clip_kernel<false, MANY>;
  for (int first = (g.n - 1) / TABLE * TABLE; first >= 0 && g.n > 0; first -= TABLE) {
    GradTable t;
    const uint32_t chunks = fill_table(g, first, chunk_bytes(few ? FEW : MANY), t);
    if (chunks == 0) continue;
    hipLaunchKernelGGL(kernel, dim3(grad_grid(chunks)), dim3(256), 0, stream, t, chunks, partial, (int)used,
                       (const float*)norm, max_norm, eps, norm_out);
    norm_out = nullptr;
  }
  return hipGetLastError();
}

}  // namespace fp8bs
