// The MMA's descriptor, shared by the tensor-core weight-gradient kernels.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace lat {
namespace wtc {

template <typename T> constexpr bool is_bf16() { return !std::is_same<T, __half>::value; }

// kind::f16, fp32 D, A and B MN-major, M x N
template <typename T, int M, int N>
__host__ __device__ constexpr uint32_t make_idesc() {
    return (1u << 4) | ((is_bf16<T>() ? 1u : 0u) << 7) | ((is_bf16<T>() ? 1u : 0u) << 10) | (1u << 15) |
           (1u << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

}  // namespace wtc
}  // namespace lat
