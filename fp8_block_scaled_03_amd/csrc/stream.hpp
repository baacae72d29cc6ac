// Loads and stores of rows that are read and written once, past the caches or through them.
#pragma once
#include "common.hpp"

namespace fp8bs {

// Inputs that together are beyond what the 256 MB of Infinity Cache keep come faster past it;
// smaller ones may still be there from the kernel that wrote them (us through the caches
// and past them: layer norm 8192 x 8192 117 and 97, its gradient 109 and 98, an
// epilogue's gradient 8192 x 16384, gelu, 195 and 174; gradients of 2048 x 4096 20.9 and 22.6, of
// 2048 x 8192 27.8 and 34.4).  What is written then leaves past them too, all but one
// of the results (all past them: 108, 98, 184; with loads past them and all
// writes through them 115, 101, 203).
constexpr int64_t INPUTS_PAST = int64_t(192) << 20;  // bytes of a call's inputs

template <bool PAST>
__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
  typedef unsigned v4u __attribute__((ext_vector_type(4)));
  if constexpr (!PAST) return *reinterpret_cast<const uint4*>(p);
  const v4u v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

template <bool PAST>
__device__ __forceinline__ void store_once(uint16_t* p, uint4 v) {
  typedef unsigned v4u __attribute__((ext_vector_type(4)));
  if constexpr (PAST) __builtin_nontemporal_store(v4u{v.x, v.y, v.z, v.w}, reinterpret_cast<v4u*>(p));
  else *reinterpret_cast<uint4*>(p) = v;
}

}  // namespace fp8bs
