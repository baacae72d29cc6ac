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

// Tile `id` of all ranges' tiles, of which at most `most` are given out; false past
// the last one.  First come the tiles with more than BM/2 rows, range by range,
// then each range's last tile if it has fewer: the light ones, whose upper row
// bands are idle, fill the last round (16 uneven ranges, 8192 rows, 4096 x 7168:
// 280 us in one order, 273 so).  Every wave finds the tile for itself:
// lane l looks at range 64c + l, a prefix sum over the lanes counts row tiles.
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ offsets, int G, int64_t M, uint32_t tiles_n,
                                          uint32_t id, uint32_t most, TileAt& t) {
  const int lane = threadIdx.x & 63;
  struct Count {
    uint32_t heavy, light;
  };
  auto count = [&](int c, int64_t& begin, int64_t& end) __attribute__((always_inline)) -> Count {
    const int gi = c * 64 + lane;
    begin = end = 0;
    if (gi < G) range_of(offsets, gi, M, begin, end);
    const uint32_t rows = (uint32_t)(end - begin), rest = rows % BM;
    return {rows / BM + (rest > BM / 2 ? 1u : 0u), rest > 0 && rest <= BM / 2 ? 1u : 0u};
  };
  auto prefix = [&](uint32_t n) __attribute__((always_inline)) -> uint32_t {  // inclusive, over the lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t up = __shfl_up(n, d, 64);
      n += lane >= d ? up : 0u;
    }
    return n;
  };
  auto total_of = [&](uint32_t n) __attribute__((always_inline)) -> uint32_t {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d, 64);
    return __builtin_amdgcn_readfirstlane(n);
  };
  const int chunks = (G + 63) >> 6;
  int64_t begin, end;
  uint64_t heavy_rows = 0, light_rows = 0;
  for (int c = 0; c < chunks; ++c) {
    const Count n = count(c, begin, end);
    heavy_rows += total_of(n.heavy);
    light_rows += total_of(n.light);
  }
  // a bad table may count more tiles than the launch was sized for: every tile is
  // still inside [0, M]
  const uint64_t heavy64 = heavy_rows * tiles_n, all64 = (heavy_rows + light_rows) * tiles_n;
  const uint32_t heavy = heavy64 < most ? (uint32_t)heavy64 : most, all = all64 < most ? (uint32_t)all64 : most;
  if (id >= all) return false;
  const bool light = id >= heavy;
  const uint32_t lin = light ? xcd_run(id - heavy, all - heavy) : xcd_run(id, heavy);
  const uint32_t want = lin / tiles_n;
  uint32_t before = 0;
  for (int c = 0; c < chunks; ++c) {
    const Count both = count(c, begin, end);
    const uint32_t n = light ? both.light : both.heavy;
    const uint32_t upto = before + prefix(n);
    const uint64_t hit = __ballot(upto > want);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const uint32_t n_l = __shfl(n, l, 64), first = __shfl(upto, l, 64) - n_l;
      const int64_t b = __shfl((long long)begin, l, 64), e = __shfl((long long)end, l, 64);
      uint32_t tm;
      band_walk(lin - first * tiles_n, n_l, tiles_n, tm, t.tn);
      if (light) tm = (uint32_t)((e - b) / BM);
      // one value per wave: keep the addresses built from them scalar
      t.group = __builtin_amdgcn_readfirstlane(c * 64 + l);
      t.tn = __builtin_amdgcn_readfirstlane(t.tn);
      t.row0 = uniform64(b + (int64_t)tm * BM);
      t.row_end = uniform64(e);
      return true;
    }
    before = __builtin_amdgcn_readfirstlane(__shfl(upto, 63, 64));
  }
  return false;
}

// ---- rings of direct loads -------------------------------------------------------
// Direct global->LDS loads of 16 (4) bytes per lane from a uniform base plus a 32-bit
// offset per lane, to a uniform LDS address.
__device__ __forceinline__ void dma16_at(const uint8_t* base, uint32_t off, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(
                   __builtin_amdgcn_readfirstlane(lds_base)),
               "v"(off), "s"(base)
               : "memory");
}
__device__ __forceinline__ void dma4_at(const uint8_t* base, uint32_t off, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(
                   __builtin_amdgcn_readfirstlane(lds_base)),
               "v"(off), "s"(base)
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
