// Shared parts of the kernels around the experts' products.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gemm_experts.h"
#include "lp_common.h"

namespace gemmlp {

// Reductions over groups of 16 neighbouring lanes, by rotations on the vector unit, and from there
// over the wave.  Every lane gets the result, and the same one: sums of FP32 are the same tree
// from every lane, as a + b = b + a.
template <class X, class F>
__device__ __forceinline__ X over_16(X v, F f) {
  auto turn = [&](auto ctrl) {
    const int i = __builtin_bit_cast(int, v);
    v = f(v, __builtin_bit_cast(
                 X, __builtin_amdgcn_update_dpp(i, i, decltype(ctrl)::value, 0xf, 0xf, false)));
  };
  turn(std::integral_constant<int, 0x128>{});  // row_ror:8
  turn(std::integral_constant<int, 0x124>{});
  turn(std::integral_constant<int, 0x122>{});
  turn(std::integral_constant<int, 0x121>{});
  return v;
}
// L: lanes of a group, 16 or 64.
template <int L, class X, class F>
__device__ __forceinline__ X over_lanes(X v, F f) {
  v = over_16(v, f);
  if constexpr (L == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}

struct Add {
  template <class X>
  __device__ __forceinline__ X operator()(X a, X b) const { return a + b; }
};
struct Least {
  template <class X>
  __device__ __forceinline__ X operator()(X a, X b) const { return min(a, b); }
};
struct Most {
  template <class X>
  __device__ __forceinline__ X operator()(X a, X b) const { return max(a, b); }
};

// Inclusive sums over the lanes of a wave, on the vector unit.
__device__ __forceinline__ int wave_scan(int v) {
  auto step = [&](auto ctrl, auto rows) {
    v += __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, decltype(rows)::value, 0xf, false);
  };
  using std::integral_constant;
  step(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});  // row_shr:1
  step(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});  // row_bcast:15
  step(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});  // row_bcast:31
  return v;
}

// COUNT neighbouring values as they are, from p on, of any alignment.
template <class T, int COUNT>
using Raw = typename T::type __attribute__((ext_vector_type(COUNT)));
template <class T, int COUNT>
__device__ __forceinline__ Raw<T, COUNT> load_raw(const typename T::type* p) {
  typedef typename T::type any __attribute__((ext_vector_type(COUNT), aligned(sizeof(typename T::type))));
  return *(const any*)p;
}

}  // namespace gemmlp
