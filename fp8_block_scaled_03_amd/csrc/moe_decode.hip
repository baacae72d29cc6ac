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

// An expert with choices, as the first kernel leaves it for the second.
struct Live {
  int32_t expert, count, start;  // count 0: the candidate stands for none; its slots are list[start ..]
  int32_t unused;
};

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
  Live* live;       // [candidates]
  uint16_t* list;   // [slots], by expert
  uint16_t* y;      // [2, slots, inner]: y rounded, and the rest rounded
};

__device__ __forceinline__ v4f mfma_bf16(v8bf w, v8bf x, v4f acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, acc, 0, 0, 0);
}

// A lane's pieces of one K-block: 16 codes each of a weight row from 16g and 64 + 16g, and
// for its column the values at the same K.  Loads have no conditions, so that the
// compiler can count them: pieces past K read the row's last whole one (values are then
// replaced by zeros, in the last K-block only), columns without a slot read the
// first one's and are not stored.
struct Codes {
  v4i c[2];
};
struct Values {
  v4i v[4];
};

__device__ __forceinline__ Codes load_codes(const uint8_t* row, int kb, int g, int k) {
  int o0 = kb * 128 + 16 * g, o1 = o0 + 64;
  o0 = o0 < k ? o0 : k - 16;
  o1 = o1 < k ? o1 : k - 16;
  return {{*reinterpret_cast<const v4i*>(row + o0), *reinterpret_cast<const v4i*>(row + o1)}};
}
__device__ __forceinline__ Values load_values(const uint16_t* row, int kb, int g, int k) {
  int o0 = kb * 128 + 16 * g, o1 = o0 + 64;
  o0 = o0 < k ? o0 : k - 16;
  o1 = o1 < k ? o1 : k - 16;
  const v4i *const a = reinterpret_cast<const v4i*>(row + o0), *const b = reinterpret_cast<const v4i*>(row + o1);
  return {{a[0], a[1], b[0], b[1]}};
}
__device__ __forceinline__ void clear_past(Values& x, int kb, int g, int k) {
  if (kb * 128 + 128 <= k) return;
  const v4i z = {0, 0, 0, 0};
  const bool in0 = kb * 128 + 16 * g < k, in1 = kb * 128 + 64 + 16 * g < k;
  x.v[0] = in0 ? x.v[0] : z;
  x.v[1] = in0 ? x.v[1] : z;
  x.v[2] = in1 ? x.v[2] : z;
  x.v[3] = in1 ? x.v[3] : z;
}
// P of one K-block for 16 weight rows x 16 columns, for N sets of rows or of columns.
__device__ __forceinline__ v4f block_product(const Codes& c, const Values& x) {
  v4f p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const v8bf lo = e4m3x8_to_bf16x8(v2i{c.c[h][0], c.c[h][1]}), hi = e4m3x8_to_bf16x8(v2i{c.c[h][2], c.c[h][3]});
    p = mfma_bf16(lo, __builtin_bit_cast(v8bf, x.v[2 * h]), p);
    p = mfma_bf16(hi, __builtin_bit_cast(v8bf, x.v[2 * h + 1]), p);
  }
  return p;
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// What candidate `y` stands for; its slots in order at list[0 ..] for this wave.
__device__ __forceinline__ Live slots_of(const Moe& m, int y, uint16_t* list) {
  const int lane = threadIdx.x & 63;
  const bool by_slot = m.slots < m.experts;
  const int e = by_slot ? m.ids[y] : y;
  Live r = {e, 0, 0, 0};
  if (e < 0 || e >= m.experts) return r;
  int id[MOE_SLOTS / 64];
#pragma unroll
  for (int i = 0; i < MOE_SLOTS / 64; ++i)
    if (i * 64 < m.slots) id[i] = m.ids[i * 64 + lane < m.slots ? i * 64 + lane : m.slots - 1];
  int first = -1;
#pragma unroll
  for (int i = 0; i < MOE_SLOTS / 64; ++i) {
    if (i * 64 >= m.slots) break;
    const bool in = i * 64 + lane < m.slots;
    const uint64_t same = __ballot(in && id[i] == e);
    r.start += __popcll(__ballot(in && id[i] >= 0 && id[i] < e));
    if (same == 0) continue;
    if (first < 0) first = i * 64 + __ffsll((unsigned long long)same) - 1;
    if ((same >> lane) & 1)
      list[r.count + __popcll(same & ((uint64_t(1) << lane) - 1))] = (uint16_t)(i * 64 + lane);
    r.count += __popcll(same);
  }
  __builtin_amdgcn_wave_barrier();  // the lanes' entries are there for every lane
  if (by_slot && first != y) r.count = 0;
  return r;
}

__global__ void __launch_bounds__(64 * MOE_WAVES1) moe_up_kernel(Moe m) {
  constexpr int D = 3;  // K-blocks that a wave loads at a time
  __shared__ uint16_t lists[MOE_WAVES1][MOE_SLOTS];
  __shared__ __attribute__((aligned(16))) float part[MOE_WAVES1][2][64][4];
  const int lane = threadIdx.x & 63, w = wave_id_uniform(), g = lane >> 4, lo = lane & 15;
  const int tile = blockIdx.x, y = blockIdx.y;
  const Live v = slots_of(m, y, lists[w]);
  if (tile == 0 && w == 0) {
    if (lane == 0) m.live[y] = v;
    for (int i = lane; i < v.count; i += 64) m.list[v.start + i] = lists[w][i];
  }
  if (v.count == 0) return;
  const int H = m.hidden, I = m.inner, KB = (H + 127) >> 7;
  const int per = (KB + MOE_WAVES1 - 1) / MOE_WAVES1, kb0 = w * per, kb1 = kb0 + per < KB ? kb0 + per : KB;
  const int64_t gate = (int64_t)v.expert * 2 * I + tile * 16, up = gate + I;  // first rows
  const uint8_t *const wg = m.w1 + (gate + lo) * H, *const wu = m.w1 + (up + lo) * H;
  // the wave's scales, one for each K-block (at most 64), in the lanes
  const int nb = (2 * I + 127) >> 7, mine = kb0 + lane < KB ? kb0 + lane : KB - 1;
  const float sg = m.s1[((int64_t)v.expert * nb + (tile * 16 >> 7)) * KB + mine];
  const float su = m.s1[((int64_t)v.expert * nb + ((I + tile * 16) >> 7)) * KB + mine];
  for (int c0 = 0; c0 < v.count; c0 += 16) {
    const int slot = lists[w][c0 + lo < v.count ? c0 + lo : c0];
    const uint16_t* const x = m.x + (int64_t)(slot / m.top) * H;
    v4f ag = {0.0f, 0.0f, 0.0f, 0.0f}, au = ag;
    for (int kb = kb0; kb < kb1; kb += D) {
      Codes cg[D], cu[D];
      Values xv[D];
#pragma unroll
      for (int i = 0; i < D; ++i) {
        const int at = kb + i < kb1 ? kb + i : kb1 - 1;
        cg[i] = load_codes(wg, at, g, H);
        cu[i] = load_codes(wu, at, g, H);
        xv[i] = load_values(x, at, g, H);
      }
#pragma unroll
      for (int i = 0; i < D; ++i) {
        if (kb + i >= kb1) break;
        clear_past(xv[i], kb + i, g, H);
        promote(ag, block_product(cg[i], xv[i]), lane_value(sg, kb + i - kb0));
        promote(au, block_product(cu[i], xv[i]), lane_value(su, kb + i - kb0));
      }
    }
    __syncthreads();  // the last pass' sums have been read
    *reinterpret_cast<v4f*>(part[w][0][lane]) = ag;
    *reinterpret_cast<v4f*>(part[w][1][lane]) = au;
    __syncthreads();
    // thread 4l + i: result i of lane l, that is row 4 (l >> 4) + i of the tile, column l & 15
    const int l = threadIdx.x >> 2, i = threadIdx.x & 3;
    if (c0 + (l & 15) < v.count) {
      float hg = part[0][0][l][i], hu = part[0][1][l][i];
#pragma unroll
      for (int k = 1; k < MOE_WAVES1; ++k) {
        hg += part[k][0][l][i];
        hu += part[k][1][l][i];
      }
      const float val = hg * sigmoid(hg).s * hu;
      const uint32_t hi = bf16_round_pair(val, 0.0f);
      const float rest = val - bf16_lo(hi);
      const int64_t at = (int64_t)lists[w][c0 + (l & 15)] * I + tile * 16 + (l >> 4) * 4 + i;
      m.y[at] = (uint16_t)hi;
      // (no rest of an infinity)
      m.y[(int64_t)m.slots * I + at] = (uint16_t)bf16_round_pair(rest - rest == 0.0f ? rest : 0.0f, 0.0f);
    }
  }
}

// One expert's slots c0 .. c0 + 8 NT - 1, K-blocks kb0 .. kb1 - 1: columns 0-7 of an MFMA are
// the slots' rounded y, columns 8-15 the rests, whose sums join in the end.
template <int NT, int D>
__device__ __forceinline__ void moe_down_part(const Moe& m, const uint8_t* row, float scales, int kb0, int kb1, int g,
                                              int lo, const uint16_t* list, int count, float* sums) {
  const uint16_t* y[NT];
  v4f acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = 8 * t + (lo & 7);
    const int slot = list[c < count ? c : 0];
    y[t] = m.y + ((int64_t)(lo >> 3) * m.slots + slot) * m.inner;
    acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  for (int kb = kb0; kb < kb1; kb += D) {
    Codes c[D];
    Values v[D][NT];
#pragma unroll
    for (int i = 0; i < D; ++i) {
      const int at = kb + i < kb1 ? kb + i : kb1 - 1;
      c[i] = load_codes(row, at, g, m.inner);
#pragma unroll
      for (int t = 0; t < NT; ++t) v[i][t] = load_values(y[t], at, g, m.inner);
    }
#pragma unroll
    for (int i = 0; i < D; ++i) {
      if (kb + i >= kb1) break;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        clear_past(v[i][t], kb + i, g, m.inner);
        promote(acc[t], block_product(c[i], v[i][t]), lane_value(scales, kb + i - kb0));
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float own = acc[t][i];
      const int other = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, own), 0x128, 0xF, 0xF, true);  // lane ^ 8
      acc[t][i] = own + __builtin_bit_cast(float, other);
    }
    const int c = 8 * t + lo;
    if (lo < 8 && c < count) *reinterpret_cast<v4f*>(sums + list[c] * 16 + 4 * g) = acc[t];
  }
}

__global__ void __launch_bounds__(64 * MOE_WAVES2) moe_down_kernel(Moe m, int chunks) {
  extern __shared__ __attribute__((aligned(16))) float sums[];  // [chunks][slots][16]
  __shared__ Live live[MOE_SLOTS];
  __shared__ uint16_t list[MOE_SLOTS];
  __shared__ int found[MOE_SLOTS / 64];
  const int lane = threadIdx.x & 63, w = wave_id_uniform(), g = lane >> 4, lo = lane & 15;
  const int n0 = blockIdx.x * 16;
  // the experts with choices, without gaps
  Live v = {0, 0, 0, 0};
  if ((int)threadIdx.x < m.candidates) v = m.live[threadIdx.x];
  if ((int)threadIdx.x < m.slots) list[threadIdx.x] = m.list[threadIdx.x];
  const uint64_t there = __ballot(v.count > 0);
  if (w < MOE_SLOTS / 64 && lane == 0) found[w] = __popcll(there);
  __syncthreads();
  int total = 0, before = 0;
#pragma unroll
  for (int i = 0; i < MOE_SLOTS / 64; ++i) {
    before += i < w ? found[i] : 0;
    total += found[i];
  }
  if (v.count > 0) live[before + __popcll(there & ((uint64_t(1) << lane) - 1))] = v;
  __syncthreads();

  const int I = m.inner, KB = (I + 127) >> 7, per = (KB + chunks - 1) / chunks;
  const int items = __builtin_amdgcn_readfirstlane(total) * chunks;
  for (int item = w; item < items; item += MOE_WAVES2) {
    const int at = item / chunks, chunk = item - at * chunks;
    const int e = __builtin_amdgcn_readfirstlane(live[at].expert);
    const int count = __builtin_amdgcn_readfirstlane(live[at].count);
    const int start = __builtin_amdgcn_readfirstlane(live[at].start);
    const int kb0 = chunk * per, kb1 = kb0 + per < KB ? kb0 + per : KB;
    const uint8_t* const row = m.w2 + ((int64_t)e * m.hidden + n0 + lo) * I;
    const int mine = kb0 + lane < KB ? kb0 + lane : KB - 1;
    const float scales = m.s2[((int64_t)e * ((m.hidden + 127) >> 7) + (n0 >> 7)) * KB + mine];
    float* const to = sums + (int64_t)chunk * m.slots * 16;
    for (int c0 = 0; c0 < count; c0 += 16) {
      if (count - c0 <= 8) moe_down_part<1, 4>(m, row, scales, kb0, kb1, g, lo, list + start + c0, count - c0, to);
      else moe_down_part<2, 2>(m, row, scales, kb0, kb1, g, lo, list + start + c0, count - c0, to);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < m.tokens * 16; i += 64 * MOE_WAVES2) {
    const int t = i >> 4, n = i & 15;
    float acc = 0.0f;
    for (int j = 0; j < m.top; ++j) {
      const int slot = t * m.top + j, e = m.ids[slot];
      if (e < 0 || e >= m.experts) continue;
      float s = sums[slot * 16 + n];
      for (int c = 1; c < chunks; ++c) s += sums[(c * m.slots + slot) * 16 + n];
      acc = __builtin_fmaf(m.weights[slot], s, acc);
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
  return (int64_t)sizeof(Live) * candidates + pad(2 * slots) + pad(4 * slots * inner);
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
           tokens * top, moe_candidates(tokens * top, experts), nullptr, nullptr, nullptr};
  uint8_t* at = (uint8_t*)workspace;
  auto take = [&](int64_t bytes) {
    uint8_t* const p = at;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  m.live = (Live*)take((int64_t)sizeof(Live) * m.candidates);
  m.list = (uint16_t*)take(2 * (int64_t)m.slots);
  m.y = (uint16_t*)take(4 * (int64_t)m.slots * inner);
  const int chunks = moe_chunks((int)inner);
  hipLaunchKernelGGL(moe_up_kernel, dim3((unsigned)(inner / 16), (unsigned)m.candidates), dim3(64 * MOE_WAVES1), 0,
                     stream, m);
  hipLaunchKernelGGL(moe_down_kernel, dim3((unsigned)(hidden / 16)), dim3(64 * MOE_WAVES2),
                     chunks * m.slots * 64, stream, m, chunks);
  return hipGetLastError();
}

}  // namespace fp8bs
