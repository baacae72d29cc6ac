// A whole mixture-of-experts layer for a few tokens, in two kernels:
//
//   out[t] = sum_j weights[t,j] W2[e] (silu(g) u) (+ residual[t]),  [g | u] = W1[e] x[t],  e = ids[t,j]
//
// Few tokens leave the weights' stream as what it costs, so activations stay as they
// are: bf16 x, fp32 h and y.  An E4M3 code is a bf16 value, so the products run on the
// bf16 MFMA, which forms the 32-deep sums with exact products; y enters as two bf16
// parts (y rounded, and the rest rounded: 2^-17 of it is lost).  A K-block of 128 is
// four MFMAs into one sum P, then acc = fma(P, scale, acc).
//
// A slot is one choice (t, j) of an expert.  A candidate y of the first kernel is an expert,
// or, if there are fewer slots than experts, a slot: it stands for its expert if no
// earlier slot has the same.  What a candidate stands for every wave finds by
// comparing all ids, one ballot for 64 of them.  MFMA columns are a candidate's slots,
// 16 at a time; rows are 16 rows of the weight.
//
//   kernel 1: a workgroup of four waves takes 16 gates and the 16 ups that belong to them;
//     the waves share K and are joined in order in LDS; y goes to the workspace.
//     The first workgroup of a candidate also leaves its expert and slots there.
//   kernel 2: a workgroup of 16 waves takes 16 columns of out; a wave takes an expert and a
//     chunk of K at a time and leaves each slot's 16 sums in LDS; in the end every token
//     adds its slots' sums, chunks and choices in order.
//
// Neither order depends on the other tokens: results are batch invariant.
#include "activation.hpp"
#include "common.hpp"
#include "launch_layer.hpp"
#include "quant_g128.hpp"

namespace fp8bs {

constexpr int MOE_SLOTS = 512;     // most choices of a call
constexpr int MOE_WAVES1 = 4, MOE_WAVES2 = 16;
constexpr int MOE_CHUNKS = 4;      // most chunks of K in the second kernel

struct Moe {
  const uint16_t* x;
  const int32_t* ids;
  const float* weights;
  const uint8_t* w1;
  const float* s1;
  const uint8_t* w2;
  const float* s2;
  const uint16_t* residual;
  uint16_t* out;
  int tokens, top, experts, hidden, inner;
  int slots, candidates;
  // workspace
  int32_t* count;    // [candidates] slots of its expert, 0: it stands for none
  int32_t* expert;   // [candidates]
  uint16_t* list;    // [candidates, slots]
  uint16_t *y_hi, *y_lo;  // [slots, inner]
};

__device__ __forceinline__ v4f mfma_bf16(v8bf w, v8bf x, v4f acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, acc, 0, 0, 0);
}

// A lane's pieces of one K-block: 16 codes each of a weight row from 16g and 64 + 16g, and
// for its column the values at the same K.
struct Codes {
  v4i c[2];
};
struct Values {
  v4i v[4];
};

__device__ __forceinline__ Codes load_codes(const uint8_t* row, int kb, int g, int last) {
  int o0 = kb * 128 + 16 * g, o1 = o0 + 64;
  o0 = o0 < last ? o0 : last;  // pieces past K read the last whole one; their values are zeros
  o1 = o1 < last ? o1 : last;
  return {{*reinterpret_cast<const v4i*>(row + o0), *reinterpret_cast<const v4i*>(row + o1)}};
}
__device__ __forceinline__ Values load_values(const uint16_t* row, int kb, int g, int k, bool live) {
  const v4i z = {0, 0, 0, 0};
  const int o0 = kb * 128 + 16 * g, o1 = o0 + 64;
  Values r = {{z, z, z, z}};
  if (live && o0 < k) {
    r.v[0] = *reinterpret_cast<const v4i*>(row + o0);
    r.v[1] = *reinterpret_cast<const v4i*>(row + o0 + 8);
  }
  if (live && o1 < k) {
    r.v[2] = *reinterpret_cast<const v4i*>(row + o1);
    r.v[3] = *reinterpret_cast<const v4i*>(row + o1 + 8);
  }
  return r;
}
// P of one K-block for 16 weight rows x 16 columns.
__device__ __forceinline__ v4f block_product(const Codes& c, const Values& x, v4f p) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const v8bf lo = e4m3x8_to_bf16x8(v2i{c.c[h][0], c.c[h][1]}), hi = e4m3x8_to_bf16x8(v2i{c.c[h][2], c.c[h][3]});
    p = mfma_bf16(lo, __builtin_bit_cast(v8bf, x.v[2 * h]), p);
    p = mfma_bf16(hi, __builtin_bit_cast(v8bf, x.v[2 * h + 1]), p);
  }
  return p;
}

// The expert that candidate `y` stands for, or -1, and its slots in order: their
// number, and list[0 ..] for this wave.
__device__ __forceinline__ int slots_of(const Moe& m, int y, int& count, uint16_t* list) {
  const int lane = threadIdx.x & 63;
  const bool by_slot = m.slots < m.experts;
  const int e = by_slot ? m.ids[y] : y;
  count = 0;
  if (e < 0 || e >= m.experts) return -1;
  int first = -1;
  for (int base = 0; base < m.slots; base += 64) {
    const int i = base + lane;
    const uint64_t same = __ballot(i < m.slots && m.ids[i < m.slots ? i : 0] == e);
    if (same == 0) continue;
    if (first < 0) first = base + __ffsll((unsigned long long)same) - 1;
    const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
    if ((same >> lane) & 1) list[count + before] = (uint16_t)i;
    count += __popcll(same);
  }
  __builtin_amdgcn_wave_barrier();  // the lanes' entries are there for every lane
  if (by_slot && first != y) count = 0;
  return count > 0 ? e : -1;
}

__global__ void __launch_bounds__(64 * MOE_WAVES1) moe_up_kernel(Moe m) {
  __shared__ uint16_t lists[MOE_WAVES1][MOE_SLOTS];
  __shared__ __attribute__((aligned(16))) float part[MOE_WAVES1][2][64][4];
  const int lane = threadIdx.x & 63, w = wave_id_uniform(), g = lane >> 4, lo = lane & 15;
  const int tile = blockIdx.x, y = blockIdx.y;
  int count;
  const int e = slots_of(m, y, count, lists[w]);
  if (tile == 0 && w == 0) {
    if (lane == 0) {
      m.count[y] = e < 0 ? 0 : count;
      m.expert[y] = e;
    }
    for (int i = lane; e >= 0 && i < count; i += 64) m.list[(int64_t)y * m.slots + i] = lists[w][i];
  }
  if (e < 0) return;
  const int H = m.hidden, I = m.inner, KB = (H + 127) >> 7;
  const int per = (KB + MOE_WAVES1 - 1) / MOE_WAVES1, kb0 = w * per, kb1 = kb0 + per < KB ? kb0 + per : KB;
  const int64_t gate = (int64_t)e * 2 * I + tile * 16, up = gate + I;  // first rows
  const uint8_t *const wg = m.w1 + (gate + lo) * H, *const wu = m.w1 + (up + lo) * H;
  const int nb = (2 * I + 127) >> 7;
  const float* const sg = m.s1 + ((int64_t)e * nb + (tile * 16 >> 7)) * KB;
  const float* const su = m.s1 + ((int64_t)e * nb + ((I + tile * 16) >> 7)) * KB;
  for (int c0 = 0; c0 < count; c0 += 16) {
    const bool live = c0 + lo < count;
    const int slot = live ? lists[w][c0 + lo] : 0;
    const uint16_t* const x = m.x + (int64_t)(slot / m.top) * H;
    v4f ag = {0.0f, 0.0f, 0.0f, 0.0f}, au = ag;
    const v4f zero = ag;
    struct Set {
      Codes g, u;
      Values x;
    };
    auto load = [&](Set& s, int kb) __attribute__((always_inline)) {
      kb = kb < kb1 ? kb : kb1 - 1;
      s.g = load_codes(wg, kb, g, H - 16);
      s.u = load_codes(wu, kb, g, H - 16);
      s.x = load_values(x, kb, g, H, live);
    };
    auto multiply = [&](const Set& s, int kb) __attribute__((always_inline)) {
      promote(ag, block_product(s.g, s.x, zero), sg[kb]);
      promote(au, block_product(s.u, s.x, zero), su[kb]);
    };
    Set a, b;
    load(a, kb0);
    for (int kb = kb0; kb < kb1; kb += 2) {
      load(b, kb + 1);
      multiply(a, kb);
      load(a, kb + 2);
      if (kb + 1 < kb1) multiply(b, kb + 1);
    }
    __syncthreads();  // the last pass' sums have been read
    *reinterpret_cast<v4f*>(part[w][0][lane]) = ag;
    *reinterpret_cast<v4f*>(part[w][1][lane]) = au;
    __syncthreads();
    // thread 4l + i: result i of lane l, that is row 4 (l >> 4) + i of the tile, column l & 15
    const int l = threadIdx.x >> 2, i = threadIdx.x & 3;
    if (c0 + (l & 15) < count) {
      float hg = part[0][0][l][i], hu = part[0][1][l][i];
#pragma unroll
      for (int k = 1; k < MOE_WAVES1; ++k) {
        hg += part[k][0][l][i];
        hu += part[k][1][l][i];
      }
      const float v = hg * sigmoid(hg).s * hu;
      const uint32_t hi = bf16_round_pair(v, 0.0f);
      const float rest = v - bf16_lo(hi);
      const int64_t at = (int64_t)lists[w][c0 + (l & 15)] * I + tile * 16 + (l >> 4) * 4 + i;
      m.y_hi[at] = (uint16_t)hi;
      m.y_lo[at] = (uint16_t)bf16_round_pair(rest - rest == 0.0f ? rest : 0.0f, 0.0f);  // (none of an infinity)
    }
  }
}

__global__ void __launch_bounds__(64 * MOE_WAVES2) moe_down_kernel(Moe m, int chunks) {
  extern __shared__ __attribute__((aligned(16))) float sums[];  // [chunks][slots][16]
  const int lane = threadIdx.x & 63, w = wave_id_uniform(), g = lane >> 4, lo = lane & 15;
  const int I = m.inner, KB = (I + 127) >> 7, per = (KB + chunks - 1) / chunks;
  const int n0 = blockIdx.x * 16;
  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int item = w; item < m.candidates * chunks; item += MOE_WAVES2) {
    const int y = item / chunks, chunk = item - y * chunks;
    const int count = m.count[y], e = m.expert[y];
    if (count == 0) continue;
    const int kb0 = chunk * per, kb1 = kb0 + per < KB ? kb0 + per : KB;
    const uint8_t* const row = m.w2 + ((int64_t)e * m.hidden + n0 + lo) * I;
    const float* const s = m.s2 + ((int64_t)e * ((m.hidden + 127) >> 7) + (n0 >> 7)) * KB;
    for (int c0 = 0; c0 < count; c0 += 16) {
      const bool live = c0 + lo < count;
      const int slot = live ? m.list[(int64_t)y * m.slots + c0 + lo] : 0;
      const uint16_t *const hi = m.y_hi + (int64_t)slot * I, *const low = m.y_lo + (int64_t)slot * I;
      v4f acc = zero;
      struct Set {
        Codes c;
        Values hi, lo;
      };
      auto load = [&](Set& t, int kb) __attribute__((always_inline)) {
        kb = kb < kb1 ? kb : kb1 - 1;
        t.c = load_codes(row, kb, g, I - 16);
        t.hi = load_values(hi, kb, g, I, live);
        t.lo = load_values(low, kb, g, I, live);
      };
      auto multiply = [&](const Set& t, int kb) __attribute__((always_inline)) {
        promote(acc, block_product(t.c, t.hi, block_product(t.c, t.lo, zero)), s[kb]);
      };
      Set a, b;
      load(a, kb0);
      for (int kb = kb0; kb < kb1; kb += 2) {
        load(b, kb + 1);
        multiply(a, kb);
        load(a, kb + 2);
        if (kb + 1 < kb1) multiply(b, kb + 1);
      }
      if (live) *reinterpret_cast<v4f*>(sums + ((int64_t)chunk * m.slots + slot) * 16 + 4 * g) = acc;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < m.tokens * 16; i += 64 * MOE_WAVES2) {
    const int t = i >> 4, n = i & 15;
    float acc = 0.0f;
    for (int j = 0; j < m.top; ++j) {
      const int slot = t * m.top + j, e = m.ids[slot];
      if (e < 0 || e >= m.experts) continue;
      float v = sums[slot * 16 + n];
      for (int c = 1; c < chunks; ++c) v += sums[(c * m.slots + slot) * 16 + n];
      acc = __builtin_fmaf(m.weights[slot], v, acc);
    }
    const int64_t at = (int64_t)t * m.hidden + n0 + n;
    if (m.residual != nullptr) acc += bf16_lo(m.residual[at]);
    m.out[at] = (uint16_t)bf16_round_pair(acc + 0.0f, 0.0f);
  }
}

static int moe_candidates(int slots, int experts) { return slots < experts ? slots : experts; }
static int moe_chunks(int inner) {
  const int wanted = (inner + 511) / 512;  // (a function of inner alone: sums of a token are the same in every batch)
  return wanted < MOE_CHUNKS ? (wanted > 0 ? wanted : 1) : MOE_CHUNKS;
}

int moe_max_slots() { return MOE_SLOTS; }

int64_t moe_decode_workspace(int tokens, int top, int experts, int64_t inner) {
  const int64_t slots = (int64_t)tokens * top, candidates = moe_candidates((int)slots, experts);
  auto pad = [](int64_t n) { return (n + 15) / 16 * 16; };
  return 2 * pad(4 * candidates) + pad(2 * candidates * slots) + 2 * pad(2 * slots * inner);
}

hipError_t set_moe_attributes() {
  return hipFuncSetAttribute((const void*)moe_down_kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                             MOE_CHUNKS * MOE_SLOTS * 64);
}

hipError_t launch_moe_decode(const void* x, const int32_t* ids, const float* weights, const void* w1,
                             const float* s1, const void* w2, const float* s2, const void* residual, void* out,
                             int tokens, int top, int experts, int64_t hidden, int64_t inner, void* workspace,
                             hipStream_t stream) {
  Moe m = {(const uint16_t*)x, ids, weights, (const uint8_t*)w1, s1, (const uint8_t*)w2, s2,
           (const uint16_t*)residual, (uint16_t*)out, tokens, top, experts, (int)hidden, (int)inner,
           tokens * top, moe_candidates(tokens * top, experts), nullptr, nullptr, nullptr, nullptr, nullptr};
  uint8_t* at = (uint8_t*)workspace;
  auto take = [&](int64_t bytes) {
    uint8_t* const p = at;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  m.count = (int32_t*)take(4 * m.candidates);
  m.expert = (int32_t*)take(4 * m.candidates);
  m.list = (uint16_t*)take(2 * (int64_t)m.candidates * m.slots);
  m.y_hi = (uint16_t*)take(2 * (int64_t)m.slots * inner);
  m.y_lo = (uint16_t*)take(2 * (int64_t)m.slots * inner);
  const int chunks = moe_chunks((int)inner);
  if (m.slots > 0 && inner > 0)
    hipLaunchKernelGGL(moe_up_kernel, dim3((unsigned)(inner / 16), (unsigned)m.candidates), dim3(64 * MOE_WAVES1), 0,
                       stream, m);
  hipLaunchKernelGGL(moe_down_kernel, dim3((unsigned)(hidden / 16)), dim3(64 * MOE_WAVES2),
                     chunks * m.slots * 64, stream, m, chunks);
  return hipGetLastError();
}

}  // namespace fp8bs
