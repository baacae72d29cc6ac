// Ragged row ranges: which rows and columns a workgroup's tile covers; and the loads and
// waits of LDS rings.
#pragma once
#include "common.hpp"

namespace fp8bs {

struct TileAt {
  int group;
  uint32_t tn;      // column tile
  int64_t row0;     // first row, and the end of the range that holds it
  int64_t row_end;
};

// A 64-bit value that is the same in every lane, in scalar registers.
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
template <typename T>
__device__ __forceinline__ T* uniform_ptr(T* p) {
  return reinterpret_cast<T*>(uniform64(reinterpret_cast<int64_t>(p)));
}

// Consecutive workgroup ids are dealt round-robin to the 8 XCDs.  Position of
// workgroup `id` when each XCD is given a contiguous run of the `total` tiles:
// neighbouring tiles, which share rows or weights, then meet in one L2.
__device__ __forceinline__ uint32_t xcd_run(uint32_t id, uint32_t total) {
  const uint32_t x = id & 7, per = total >> 3, rest = total & 7;
  return x * per + (x < rest ? x : rest) + (id >> 3);
}

// Tile r of a range with tiles_m x tiles_n tiles, walked in bands of four row
// tiles so that a run shares weight columns and rows.
__device__ __forceinline__ void band_walk(uint32_t r, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
  const uint32_t band = r / (4 * tiles_n);
  const uint32_t rows = tiles_m - band * 4 < 4 ? tiles_m - band * 4 : 4;
  const uint32_t at = r - band * 4 * tiles_n;
  tn = at / rows;
  tm = band * 4 + (at - tn * rows);
}

template <int BM>
__device__ __forceinline__ void dense_tile(int64_t M, uint32_t tiles_n, uint32_t id, uint32_t total, TileAt& t) {
  uint32_t tm;
  band_walk(xcd_run(id, total), total / tiles_n, tiles_n, tm, t.tn);
  t.group = 0;
  t.row0 = (int64_t)tm * BM;
  t.row_end = M;
}

// Range g of the offsets table, clamped into [0, M]; a range that runs
// backwards is empty.
__device__ __forceinline__ void range_of(const int32_t* offsets, int g, int64_t M, int64_t& begin, int64_t& end) {
  int64_t b = offsets[g], e = offsets[g + 1];
  b = b < 0 ? 0 : (b > M ? M : b);
  e = e < b ? b : (e > M ? M : e);
  begin = b;
  end = e;
}

// Tile `id` of all ranges' tiles (range by range), of which at most `most` are
// given out; false past the last one.  Every wave finds it for itself: lane l
// looks at range 64c + l, a prefix sum over the lanes counts the row tiles.
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ offsets, int G, int64_t M, uint32_t tiles_n,
                                          uint32_t id, uint32_t most, TileAt& t) {
  const int lane = threadIdx.x & 63;
  auto count = [&](int c, int64_t& begin, int64_t& end) __attribute__((always_inline)) -> uint32_t {
    const int gi = c * 64 + lane;
    begin = end = 0;
    if (gi < G) range_of(offsets, gi, M, begin, end);
    return (uint32_t)((end - begin + BM - 1) / BM);
  };
  auto prefix = [&](uint32_t n) __attribute__((always_inline)) -> uint32_t {  // inclusive, over the lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t up = __shfl_up(n, d, 64);
      n += lane >= d ? up : 0u;
    }
    return n;
  };
  const int chunks = (G + 63) >> 6;
  int64_t begin, end;
  uint32_t row_tiles = 0;
  for (int c = 0; c < chunks; ++c) row_tiles += __shfl(prefix(count(c, begin, end)), 63, 64);
  row_tiles = __builtin_amdgcn_readfirstlane(row_tiles);
  // a bad table may count more tiles than the launch was sized for: every tile is
  // still inside [0, M]
  const uint64_t total64 = (uint64_t)row_tiles * tiles_n;
  const uint32_t total = total64 < most ? (uint32_t)total64 : most;
  if (id >= total) return false;
  const uint32_t lin = xcd_run(id, total);
  const uint32_t want = lin / tiles_n;
  uint32_t before = 0;
  for (int c = 0; c < chunks; ++c) {
    const uint32_t n = count(c, begin, end);
    const uint32_t upto = before + prefix(n);
    const uint64_t hit = __ballot(upto > want);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const uint32_t n_l = __shfl(n, l, 64), first = __shfl(upto, l, 64) - n_l;
      uint32_t tm;
      band_walk(lin - first * tiles_n, n_l, tiles_n, tm, t.tn);
      const int64_t b = __shfl((long long)begin, l, 64);
      t.group = c * 64 + l;
      t.row0 = b + (int64_t)tm * BM;
      t.row_end = __shfl((long long)end, l, 64);
      // one value per wave: keep the addresses built from them scalar
      t.group = __builtin_amdgcn_readfirstlane(t.group);
      t.tn = __builtin_amdgcn_readfirstlane(t.tn);
      t.row0 = uniform64(t.row0);
      t.row_end = uniform64(t.row_end);
      return true;
    }
    before = __shfl(upto, 63, 64);
  }
  return false;
}

// ---- rings of direct loads -------------------------------------------------------
// Direct global->LDS load of 16 bytes per lane from a uniform base plus a
// 32-bit offset per lane.
__device__ __forceinline__ void dma16_at(const uint8_t* base, uint32_t off, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds_base), "v"(off), "s"(base)
               : "memory");
}

// Waits until at most min(ahead, MOST) steps of P loads are in flight.
template <int MOST, int P>
__device__ __forceinline__ void wait_steps(int ahead) {
  if constexpr (MOST == 0) {
    wait_vmcnt<0>();
  } else {
    if (ahead >= MOST) wait_vmcnt<MOST * P>();
    else wait_steps<MOST - 1, P>(ahead);
  }
}

}  // namespace fp8bs
