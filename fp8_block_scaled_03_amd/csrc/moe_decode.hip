// A whole mixture-of-experts layer for a few tokens:
//
//   out[t] = sum_j weights[t,j] W2[e] (silu(g) u) (+ residual[t]),  [g | u] = W1[e] x[t],  e = ids[t,j]
//
// Few tokens leave the weights' stream as what it costs, so activations stay as they
// are: bf16 x, fp32 h and y.  An E4M3 code is a bf16 value, so the products run on the
// bf16 MFMA, which forms the 32-deep sums with exact products; y enters as two bf16
// parts (y rounded, and the rest rounded: 2^-17 of it is lost).  A K-block of 128 is
// four MFMAs into one sum P, then acc = fma(P, scale, acc).
//
// A slot is one choice (t, j) of an expert.  A candidate is an expert,
// or, if there are fewer slots than experts, a slot: it stands for its expert if no
// earlier slot has the same.  What a candidate stands for every wave finds by
// comparing all ids, one ballot for 64 of them.  MFMA columns are a candidate's slots,
// 16 at a time; rows are 16 rows of the weight.
//
//   up: a workgroup of four waves takes 16, 32 or 64 gates and the ups that belong to them; y goes to the
//     workspace.  The first workgroup of a candidate also leaves its expert and slots there.
//   down: a workgroup takes 32, 64 or 128 columns of out for one candidate; its slots' sums go to the workspace.
//   join: every token adds its slots' sums, choices in order.
// In the first two the waves share K (always a quarter each) and are joined in order in LDS.  For one
// token of few choices a workgroup has all of them for its columns, down and join in one.
//
// What bounds it is the weights' stream (6.0 to 6.2 TB/s from 8 tokens to 32 with 64 experts of
// 4096 x 2048, top 8: 174 and 262 us), and beside it what every workgroup reads of x and y through its
// L2, which costs as much a byte, as if the lines that a CU has asked for were the limit.  The
// two products alone, 61 tokens, trial copies: 16 gates to a workgroup: up 250 us, 190 without x,
// 200 with an x that the L1 holds; 16 columns: down 210, 88, 120; with 64 weight rows to a
// K-block of values 190 and 160, 138 and 97; with 128 173 and 128.  So many slots of an expert
// take large tiles; few read little, and smaller tiles give more workgroups.  Waves that share
// rows of y instead of K did not help (down 190): their reads do not meet in the L1; nor did y by
// eight K of all slots, two lines to a load (141; one token 16.7, not 14.7).  From about 15 slots
// of an expert on the products of quantized activations take less time (the header has figures).
//
// No order depends on the other tokens: results are batch invariant.
#include "activation.hpp"
#include "common.hpp"
#include "fp8bs_layer.h"
#include "launch_layer.hpp"
#include "quant_g128.hpp"

#include <type_traits>

namespace fp8bs {

constexpr int MOE_SLOTS = FP8BS_MAX_MOE_CHOICES;  // what a call may have, so what lists and lanes hold
static_assert(MOE_SLOTS % 64 == 0 && MOE_SLOTS <= 65536, "whole waves of ids, slots of 16 bits");
constexpr int MOE_WAVES = 4;       // of a workgroup; they share K

// What a candidate stands for, as the first kernel leaves it for the second.
struct Live {
  int32_t expert, count, start;  // count 0: it stands for none; its slots are list[start ..]
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
  float* z;         // [slots, hidden]: the experts' results
};

__device__ __forceinline__ v4f mfma_bf16(v8bf w, v8bf x, v4f acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, acc, 0, 0, 0);
}

// A K-block's loads.  A load of codes covers eight rows' 128 bytes, whole lines (a line read in
// halves past the caches comes twice: up 290 us, not 250): lane (g, lo) loads row lo & 7, or 8
// + that, from 32g + 2 (lo & 8).  Lanes lo and lo ^ 8 then exchange one of their two pieces, and
// lane (g, lo) has row lo from 32g and from 32g + 16, as the MFMA takes it; and for its
// column the values at the same K.  Loads have no conditions, so that the compiler
// can count them: pieces past K read the row's last whole one (values are then
// replaced by zeros, in the last K-block only), columns without a slot read another
// one's and are not stored.
struct Codes {
  v4i c[2];
};
struct Values {
  v4i v[4];
};

struct Pieces {
  uint32_t code, o0, o1;  // first K of this lane's load of codes, and of its two pieces of values
  __device__ __forceinline__ Pieces(int kb, int g, int lo, int k) {
    const int a = kb * 128 + 32 * g, b = a + 16, c = a + 2 * (lo & 8);
    o0 = a < k ? a : k - 16;
    o1 = b < k ? b : k - 16;
    code = c < k ? c : k - 16;
  }
};
// The weights are read once: past the caches, which x and y share (a call of 1 to 32 tokens 4 to 9%
// less).
__device__ __forceinline__ v4i stream(const uint8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const v4i*>(p));
}
// row: of the tile's first eight rows
__device__ __forceinline__ Codes load_codes(const uint8_t* base, uint32_t row, uint32_t eight, Pieces p) {
  return {{stream(base + (row + p.code)), stream(base + (row + eight + p.code))}};
}
__device__ __forceinline__ Values load_values(const uint8_t* base, uint32_t row, Pieces p) {
  const uint32_t a = row + 2 * p.o0, b = row + 2 * p.o1;  // (bytes)
  return {{*reinterpret_cast<const v4i*>(base + a), *reinterpret_cast<const v4i*>(base + (a + 16)),
           *reinterpret_cast<const v4i*>(base + b), *reinterpret_cast<const v4i*>(base + (b + 16))}};
}
__device__ __forceinline__ void clear_past(Values& x, int kb, int g, int k) {
  if (kb * 128 + 128 <= k) return;
  const v4i z = {0, 0, 0, 0};
  const bool in0 = kb * 128 + 32 * g < k, in1 = kb * 128 + 32 * g + 16 < k;
  x.v[0] = in0 ? x.v[0] : z;
  x.v[1] = in0 ? x.v[1] : z;
  x.v[2] = in1 ? x.v[2] : z;
  x.v[3] = in1 ? x.v[3] : z;
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// RT row tiles x NT column tiles over K-blocks kb0 .. kb1 - 1 (at most 64): acc += sum of scale * P.
// rows: the tiles' first rows; scales: a tile's, K-block kb0 + l in lane l; column t's values
// begin at base + col[t].
template <int RT, int NT, int D>
__device__ __forceinline__ void products(const uint8_t* const (&rows)[RT], const float (&scales)[RT],
                                         const uint8_t* base, const uint32_t (&col)[NT], int kb0, int kb1, int k,
                                         v4f (&acc)[RT][NT]) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const uint32_t row = (uint32_t)(lane & 7) * (uint32_t)k, eight = 8 * (uint32_t)k;
  const bool low = (lane & 8) == 0;
  struct Set {
    Codes c[RT];
    Values v[NT];
  };
  auto load = [&](Set& s, int kb) __attribute__((always_inline)) {
    const Pieces p(kb < kb1 ? kb : kb1 - 1, g, lane & 15, k);
#pragma unroll
    for (int r = 0; r < RT; ++r) s.c[r] = load_codes(rows[r], row, eight, p);
#pragma unroll
    for (int t = 0; t < NT; ++t) s.v[t] = load_values(base, col[t], p);
  };
  auto multiply = [&](Set& s, int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < NT; ++t) clear_past(s.v[t], kb, g, k);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float scale = lane_value(scales[r], kb - kb0);
      v8bf w[4];
      v4i both[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int a = s.c[r].c[0][i], b = s.c[r].c[1][i], send = low ? b : a;
        const int got = __builtin_amdgcn_update_dpp(0, send, 0x128, 0xF, 0xF, true);  // from lane ^ 8
        both[0][i] = low ? a : got;
        both[1][i] = low ? got : b;
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const v4i q = both[h >> 1];
        w[h] = e4m3x8_to_bf16x8(v2i{q[2 * (h & 1)], q[2 * (h & 1) + 1]});
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        v4f p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 4; ++h) p = mfma_bf16(w[h], __builtin_bit_cast(v8bf, s.v[t].v[h]), p);
        promote(acc[r][t], p, scale);
      }
    }
  };
#pragma unroll 1
  for (int kb = kb0; kb < kb1; kb += D) {
    Set s[D];
#pragma unroll
    for (int i = 0; i < D; ++i) load(s[i], kb + i);
#pragma unroll
    for (int i = 0; i < D; ++i)
      if (kb + i < kb1) multiply(s[i], kb + i);
  }
}

// What candidate `y` stands for; its slots in order at list[0 ..] for this wave.
__device__ __forceinline__ Live slots_of(const Moe& m, int y, uint16_t* list) {
  const int lane = threadIdx.x & 63;
  const bool by_slot = m.slots < m.experts;
  int id[MOE_SLOTS / 64];
#pragma unroll
  for (int i = 0; i < MOE_SLOTS / 64; ++i)
    if (i * 64 < m.slots) id[i] = m.ids[i * 64 + lane < m.slots ? i * 64 + lane : m.slots - 1];
  const int e = by_slot ? m.ids[y] : y;
  Live r = {e, 0, 0, 0};
  if (e < 0 || e >= m.experts) return r;
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

__device__ __forceinline__ Live uniform(const Live& v) {
  return {__builtin_amdgcn_readfirstlane(v.expert), __builtin_amdgcn_readfirstlane(v.count),
          __builtin_amdgcn_readfirstlane(v.start), 0};
}

// The waves' shares of K, and their sums in LDS: part[wave][row tile][lane][row].
struct Share {
  int kb0, kb1, mine;  // K-blocks, and the one whose scales this lane holds
  __device__ __forceinline__ Share(int w, int KB) {
    const int per = (KB + MOE_WAVES - 1) / MOE_WAVES;
    kb0 = w * per;
    kb1 = kb0 + per < KB ? kb0 + per : KB;
    mine = kb0 + (int)(threadIdx.x & 63);
    mine = mine < KB ? mine : KB - 1;
  }
};
template <int RT>
using Part = float[MOE_WAVES][RT][64][4];

template <int RT, int NT>
__device__ __forceinline__ void leave(Part<RT>& part, int w, const v4f (&acc)[RT][NT], int t) {
  __syncthreads();  // the sums before these have been read
#pragma unroll
  for (int r = 0; r < RT; ++r) *reinterpret_cast<v4f*>(part[w][r][threadIdx.x & 63]) = acc[r][t];
  __syncthreads();
}

// RT / 2 tiles of 16 gates and their ups; a pass has one column tile of 16 slots, or MOST of them;
// WAVES share a SIMD.  Two K-blocks are loaded at a time, with several column tiles one
// (more would cost waves).
template <int RT, int MOST, int WAVES>
__global__ void __launch_bounds__(64 * MOE_WAVES, WAVES) moe_up_kernel(Moe m) {
  constexpr int G = RT / 2, ROWS = 16 * G;  // row tiles, and rows, of gates
  __shared__ uint16_t lists[MOE_WAVES][MOE_SLOTS];
  __shared__ __attribute__((aligned(16))) Part<RT> part;
  const int lane = threadIdx.x & 63, w = wave_id_uniform(), lo = lane & 15;
  const int tile = blockIdx.x, y = blockIdx.y;
  const Live v = uniform(slots_of(m, y, lists[w]));
  if (tile == 0 && w == 0) {
    if (lane == 0) m.live[y] = v;
    for (int i = lane; i < v.count; i += 64) m.list[v.start + i] = lists[w][i];
  }
  if (v.count == 0) return;
  const int H = m.hidden, I = m.inner, KB = (H + 127) >> 7, nb = (2 * I + 127) >> 7;
  const Share share(w, KB);
  // the first half of the row tiles are gates from tile * ROWS, the second their ups; behind
  // inner the first tile again
  const uint8_t* rows[RT];
  float scales[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int n = tile * ROWS + (r % G) * 16, row = (r / G) * I + (n < I ? n : tile * ROWS);
    rows[r] = uniform_ptr(m.w1 + ((int64_t)v.expert * 2 * I + row) * H);
    scales[r] = m.s1[((int64_t)v.expert * nb + (row >> 7)) * KB + share.mine];
  }
  auto pass = [&](int c0, auto nt) __attribute__((always_inline)) {
    constexpr int NT = decltype(nt)::value;
    uint32_t col[NT];
    v4f acc[RT][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = c0 + 16 * t + lo;
      const int slot = lists[w][c < v.count ? c : c0];
      col[t] = (uint32_t)(slot / m.top) * (uint32_t)H * 2;
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    products<RT, NT, (NT == 1 ? 2 : 1)>(rows, scales, (const uint8_t*)m.x, col, share.kb0, share.kb1, H, acc);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (c0 + 16 * t >= v.count) break;
      leave<RT, NT>(part, w, acc, t);
      // a thread has a slot and two gates of a row tile
      for (int i = threadIdx.x; i < G * 128; i += 64 * MOE_WAVES) {
        const int c = c0 + 16 * t + (i & 15), l = i & 63, pair = (i >> 6) & 1, r = i >> 7;
        const int n = tile * ROWS + r * 16 + (l >> 4) * 4 + 2 * pair;
        if (c >= v.count || n >= I) continue;
        uint32_t hi[2], rest[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float g = part[0][r][l][2 * pair + e], u = part[0][r + G][l][2 * pair + e];
#pragma unroll
          for (int k = 1; k < MOE_WAVES; ++k) {
            g += part[k][r][l][2 * pair + e];
            u += part[k][r + G][l][2 * pair + e];
          }
          const float val = g * sigmoid(g).s * u;
          hi[e] = bf16_round_pair(val, 0.0f);
          const float left = val - bf16_lo(hi[e]);
          rest[e] = bf16_round_pair(left - left == 0.0f ? left : 0.0f, 0.0f);  // (none of an infinity)
        }
        uint16_t* const to = m.y + (int64_t)lists[w][c] * I + n;
        *reinterpret_cast<uint32_t*>(to) = hi[0] | (hi[1] << 16);
        *reinterpret_cast<uint32_t*>(to + (int64_t)m.slots * I) = rest[0] | (rest[1] << 16);
      }
    }
  };
  for (int c0 = 0; c0 < v.count;) {
    if (MOST == 1 || v.count - c0 <= 16) {
      pass(c0, std::integral_constant<int, 1>());
      c0 += 16;
    } else {
      pass(c0, std::integral_constant<int, MOST>());
      c0 += 16 * MOST;
    }
  }
}

// RT tiles of 16 columns of out; a pass has one column tile of 8 slots, or MOST of them: MFMA
// columns 0-7 are the slots' rounded y, columns 8-15 the rests, whose sums join in
// the end.
template <int RT, int MOST, int WAVES>
__global__ void __launch_bounds__(64 * MOE_WAVES, WAVES) moe_down_kernel(Moe m) {
  __shared__ __attribute__((aligned(16))) Part<RT> part;
  const int lane = threadIdx.x & 63, w = wave_id_uniform(), lo = lane & 15;
  const Live v = uniform(m.live[blockIdx.y]);
  if (v.count == 0) return;
  const int I = m.inner, KB = (I + 127) >> 7, nb = (m.hidden + 127) >> 7, n0 = blockIdx.x * 16 * RT;
  const Share share(w, KB);
  const uint8_t* rows[RT];
  float scales[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {  // behind hidden: the first tile again
    const int row = n0 + (n0 + 16 * r < m.hidden ? 16 * r : 0);
    rows[r] = uniform_ptr(m.w2 + ((int64_t)v.expert * m.hidden + row) * I);
    scales[r] = m.s2[((int64_t)v.expert * nb + (row >> 7)) * KB + share.mine];
  }
  const uint16_t* const list = m.list + v.start;
  auto pass = [&](int c0, auto nt) __attribute__((always_inline)) {
    constexpr int NT = decltype(nt)::value;
    uint32_t col[NT];
    v4f acc[RT][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = c0 + 8 * t + (lo & 7);
      const int slot = list[c < v.count ? c : c0];
      col[t] = (uint32_t)((lo >> 3) * m.slots + slot) * (uint32_t)I * 2;
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    products<RT, NT, (NT == 1 ? 2 : 1)>(rows, scales, (const uint8_t*)m.y, col, share.kb0, share.kb1, I, acc);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (c0 + 8 * t >= v.count) break;
      leave<RT, NT>(part, w, acc, t);
      // a thread has a slot and four rows of a row tile
      for (int i = threadIdx.x; i < RT * 32; i += 64 * MOE_WAVES) {
        const int c = c0 + 8 * t + (i & 7), q = (i >> 3) & 3, r = i >> 5, at = 16 * q + (i & 7);
        if (c >= v.count || n0 + 16 * r >= m.hidden) continue;
        v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < MOE_WAVES; ++k) {
          const v4f one = *reinterpret_cast<const v4f*>(part[k][r][at]) +
                          *reinterpret_cast<const v4f*>(part[k][r][at + 8]);
          sum = k == 0 ? one : sum + one;
        }
        *reinterpret_cast<v4f*>(m.z + (int64_t)list[c] * m.hidden + n0 + 16 * r + 4 * q) = sum;
      }
    }
  };
  for (int c0 = 0; c0 < v.count;) {
    if (MOST == 1 || v.count - c0 <= 8) {
      pass(c0, std::integral_constant<int, 1>());
      c0 += 8;
    } else {
      pass(c0, std::integral_constant<int, MOST>());
      c0 += 8 * MOST;
    }
  }
}

// Four columns of a token's sum, the residual added.
__device__ __forceinline__ void store_token(const Moe& m, int t, int col, v4f acc) {
  const int64_t at = (int64_t)t * m.hidden + col;
  if (m.residual != nullptr) {
    const uint2 r = *reinterpret_cast<const uint2*>(m.residual + at);
    acc = acc + v4f{bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y)};
  }
  *reinterpret_cast<uint2*>(m.out + at) =
      make_uint2(bf16_round_pair(acc[0] + 0.0f, acc[1] + 0.0f), bf16_round_pair(acc[2] + 0.0f, acc[3] + 0.0f));
}

// Down and join for one token of at most S choices, 16 RT columns of out: four waves to a choice, each
// a quarter of K (MFMA columns 0-7 the slot's rounded y, 8-15 its rests).  The same sums in the
// same order as in the two kernels that it stands for: quarters, then choices.
template <int S, int RT>
__global__ void __launch_bounds__(64 * S * MOE_WAVES) moe_token_kernel(Moe m) {
  constexpr int QUADS = 4 * RT;  // of columns
  __shared__ __attribute__((aligned(16))) float part[S][MOE_WAVES][2][QUADS][4];  // y and its rests apart
  __shared__ __attribute__((aligned(16))) float sums[S][QUADS][4];
  const int lane = threadIdx.x & 63, w = wave_id_uniform(), g = lane >> 4, lo = lane & 15;
  const int n0 = blockIdx.x * 16 * RT, s = w / MOE_WAVES, quarter = w % MOE_WAVES;
  const int I = m.inner, KB = (I + 127) >> 7, nb = (m.hidden + 127) >> 7;
  const int mine = lane < m.top ? lane : m.top - 1;  // lane c has choice c
  const int id = lane < m.top ? m.ids[mine] : -1;
  const float weight = m.weights[mine];
  const int e = __builtin_amdgcn_readlane(id, s);
  if (e >= 0 && e < m.experts) {
    const Share share(quarter, KB);
    const uint32_t col[1] = {(uint32_t)((lo >> 3) * m.slots + s) * (uint32_t)I * 2};
    const uint8_t* rows[RT];
    float scales[RT];
    v4f acc[RT][1];
#pragma unroll
    for (int r = 0; r < RT; ++r) {  // behind hidden: the first tile again
      const int row = n0 + (n0 + 16 * r < m.hidden ? 16 * r : 0);
      rows[r] = uniform_ptr(m.w2 + ((int64_t)e * m.hidden + row) * I);
      scales[r] = m.s2[((int64_t)e * nb + (row >> 7)) * KB + share.mine];
      acc[r][0] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    products<RT, 1, 2>(rows, scales, (const uint8_t*)m.y, col, share.kb0, share.kb1, I, acc);
#pragma unroll
    for (int r = 0; r < RT; ++r)
      if ((lo & 7) == 0) *reinterpret_cast<v4f*>(part[s][quarter][lo >> 3][4 * r + g]) = acc[r][0];
  }
  __syncthreads();
  if (w > 0) return;
  if (lane < QUADS * S) {  // (of a choice that is skipped the sums mean nothing, and are not used)
    const int c = lane / QUADS, q = lane % QUADS;
    v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < MOE_WAVES; ++k) {
      const v4f one = *reinterpret_cast<const v4f*>(part[c][k][0][q]) + *reinterpret_cast<const v4f*>(part[c][k][1][q]);
      sum = k == 0 ? one : sum + one;
    }
    *reinterpret_cast<v4f*>(sums[c][q]) = sum;
  }
  __builtin_amdgcn_wave_barrier();  // the lanes' sums are there for every lane
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < S; ++c) {
    const int of = __builtin_amdgcn_readlane(id, c);
    const float by = lane_value(weight, c);
    if (of >= 0 && of < m.experts) promote(acc, *reinterpret_cast<const v4f*>(sums[c][lane % QUADS]), by);
  }
  if (lane < QUADS && n0 + 4 * lane < m.hidden) store_token(m, 0, n0 + 4 * lane, acc);
}

// Four columns of a token to a thread.
__global__ void __launch_bounds__(256) moe_join_kernel(Moe m) {
  const int quads = m.hidden / 4, q = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (q >= quads) return;
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int J = 8;  // choices that are loaded at a time; a skipped one reads its own z, which is not used
  for (int j0 = 0; j0 < m.top; j0 += J) {
    int id[J];
    float w[J];
    v4f z[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int slot = t * m.top + (j0 + j < m.top ? j0 + j : m.top - 1);
      id[j] = m.ids[slot];
      w[j] = m.weights[slot];
      z[j] = *reinterpret_cast<const v4f*>(m.z + (int64_t)slot * m.hidden + 4 * q);
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (j0 + j < m.top && id[j] >= 0 && id[j] < m.experts) promote(acc, z[j], w[j]);
  }
  store_token(m, t, 4 * q, acc);
}

static int moe_candidates(int slots, int experts) { return slots < experts ? slots : experts; }

int64_t moe_decode_workspace(int tokens, int top, int experts, int64_t hidden, int64_t inner) {
  const int64_t slots = (int64_t)tokens * top, candidates = moe_candidates((int)slots, experts);
  auto pad = [](int64_t n) { return (n + 15) / 16 * 16; };
  return (int64_t)sizeof(Live) * candidates + pad(2 * slots) + pad(4 * slots * inner) + pad(4 * slots * hidden);
}

hipError_t launch_moe_decode(const void* x, const int32_t* ids, const float* weights, const void* w1,
                             const float* s1, const void* w2, const float* s2, const void* residual, void* out,
                             int tokens, int top, int experts, int64_t hidden, int64_t inner, void* workspace,
                             hipStream_t stream) {
  Moe m = {(const uint16_t*)x, ids, weights, (const uint8_t*)w1, s1, (const uint8_t*)w2, s2,
           (const uint16_t*)residual, (uint16_t*)out, tokens, top, experts, (int)hidden, (int)inner,
           tokens * top, moe_candidates(tokens * top, experts), nullptr, nullptr, nullptr, nullptr};
  uint8_t* at = (uint8_t*)workspace;
  auto take = [&](int64_t bytes) {
    uint8_t* const p = at;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  m.live = (Live*)take((int64_t)sizeof(Live) * m.candidates);
  m.list = (uint16_t*)take(2 * (int64_t)m.slots);
  m.y = (uint16_t*)take(4 * (int64_t)m.slots * inner);
  m.z = (float*)take(4 * (int64_t)m.slots * hidden);
  const dim3 threads(64 * MOE_WAVES);
  auto tiles = [&](int64_t n, int rows) { return dim3((unsigned)((n + rows - 1) / rows), (unsigned)m.candidates); };
  auto up = [&](auto kernel, int rows) { hipLaunchKernelGGL(kernel, tiles(inner, rows), threads, 0, stream, m); };
  auto down = [&](auto kernel, int rows) { hipLaunchKernelGGL(kernel, tiles(hidden, rows), threads, 0, stream, m); };
  // By the slots of an expert, on average if every one is taken.  One run, us a call in a graph, three sets of
  // weights and choices in turn, every expert as likely; tiles of 32 weight rows (down: 32 columns), of 64 with up to
  // two column tiles a pass, of 64 with up to four, and of 128; by tokens:
  //   64 experts of 4096 x 2048, top 8: 1 43, 47, 48, 50; 4 115, 124, 129, 127; 8 175, 182, 189, 186; 12 202, 207,
  //     216, 219; 16 225, 222, 233, 231; 32 284, 263, 279, 262; 48 335, 284, 306, 277; 61 405, 318, 338, 297
  //   32, top 8: 16 148, 141, 151, 143; 40 230, 167, 188, 160; 61 351, 229, 230, 203
  //   16, top 8: 8 81, 79, 85, 80; 16 106, 90, 98, 83; 32 181, 120, 126, 113; 61 317, 204, 172, 182 (with 128 the
  //     weights come twice)
  //   8, top 2: 16 48, 48, 50, 51; 32 61, 50, 56, 53; 61 86, 64, 68, 70; 128 168, 105, 92, 109
  //   8, top 4: 61 160, 106, 92, 107; 128 299, 177, 141, 172
  //   8 of 4096 x 14336, top 2: 16 264, 233, 245, 233; 61 544, 347, 357, 323; 128 1051, 631, 533, 538
  // 128 weight rows halve what is read of x and y, but take registers for two waves a SIMD, and with fewer than
  // two workgroups to a CU (8 experts of 4096 x 2048) they are slower.
  const bool few = 2 * m.slots < 3 * m.candidates, many = m.slots >= 12 * m.candidates;
  auto large = [&](int64_t tiles) {
    return m.slots >= 5 * m.candidates && m.slots < 20 * m.candidates && tiles * m.candidates >= 512;
  };
  if (few) up(moe_up_kernel<2, 1, 4>, 16);
  else if (large(inner / 64)) up(moe_up_kernel<8, 2, 2>, 64);
  else if (many) up(moe_up_kernel<4, 4, 2>, 32);
  else up(moe_up_kernel<4, 2, 3>, 32);
  // One token with few choices: down and join in one, 32 columns from hidden 5120 on (us in a graph, three
  // kernels and two: 8 experts of 4096 x 14336, top 2, 74.4 and 63.9; of 4096 x 2048, top 1 19.6 and 16.5, top 2 21.7
  // and 18.6; of 512 x 256, top 2 9.3 and 7.5; 64 of 4096 x 2048, top 4 26.9 and 25.2; 8 of 8192 x 2048, top 2 31.2
  // and 28.7, with 16 columns 29.8; 16 of 7168 x 2048, top 4 37.0 and 34.8, 38.3).  More choices, or three and
  // four of few columns, gain nothing or lose: a workgroup reads y for fewer columns, and workgroups
  // are few (64 of 4096 x 2048, top 8 42.2 and 41.6, two tokens 70 and 73; 2048 x 4096, top 8 43 and 52; 8 of
  // 1024 x 4096, top 4 22 and 24).
  if (few && tokens == 1 && (top <= 2 || (top <= 4 && hidden >= 4096))) {
    auto token = [&](auto kernel, int choices, int columns) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)((hidden + columns - 1) / columns)), dim3(64 * MOE_WAVES * choices), 0,
                         stream, m);
    };
    const bool wide = hidden >= 5120;
    if (top <= 2) wide ? token(moe_token_kernel<2, 2>, 2, 32) : token(moe_token_kernel<2, 1>, 2, 16);
    else wide ? token(moe_token_kernel<4, 2>, 4, 32) : token(moe_token_kernel<4, 1>, 4, 16);
    return hipGetLastError();
  }
  if (few) down(moe_down_kernel<2, 1, 4>, 32);
  else if (large(hidden / 128)) down(moe_down_kernel<8, 2, 2>, 128);
  else if (many) down(moe_down_kernel<4, 4, 2>, 64);
  else down(moe_down_kernel<4, 2, 3>, 64);
  const dim3 join((unsigned)((hidden / 4 + 255) / 256), (unsigned)tokens);
  hipLaunchKernelGGL(moe_join_kernel, join, dim3(256), 0, stream, m);
  return hipGetLastError();
}

}  // namespace fp8bs
