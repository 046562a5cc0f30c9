// What the tensor-core weight-gradient kernels share: the MMA's descriptor and the cut of
// the pair list into shares (W of them at most) and segments.
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

// Clamped pair offsets of the k3 offsets (off[k3] = P) into shared memory; one warp.
__device__ __forceinline__ void load_offsets(const int64_t *pair_off, int64_t capacity, int k3, int64_t *off) {
    for (int e = threadIdx.x & 31; e <= k3; e += 32) off[e] = min(pair_off[e], capacity);
}

// Shares of a list of P pairs: min(W, P), so that no share is empty
// (every share then writes the partials its slots stand for).
template <int W>
__device__ __forceinline__ int share_count(int64_t P) { return int(min(int64_t(W), P)); }

// Share v of the pair list: pairs [P v / S, P (v+1) / S), S = share_count(P).
template <int W>
__device__ __forceinline__ int64_t share_lo(int64_t P, int v) { return P * v / share_count<W>(P); }

// The share holding pair `pair` (largest v with share_lo<W>(P, v) <= pair); a binary search.
template <int W>
__device__ __forceinline__ int share_of(int64_t P, int64_t pair) {
    int lo = 0, hi = share_count<W>(P) - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (share_lo<W>(P, mid) <= pair) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The segments of this CTA's shares, in order: share v = blockIdx.x, +gridDim.x,
// ..., and within a share the offsets its range meets.  Every role walks the
// same sequence.
template <int W>
struct Segments {
    const int64_t *off;
    int k3;
    int64_t P;
    int v, k;
    int64_t hv;
    __device__ Segments(const int64_t *o, int k3_) : off(o), k3(k3_), P(o[k3_]), v(int(blockIdx.x) - int(gridDim.x)),
                                                   k(k3_), hv(0) {}
    // next segment: offset ko, pairs [lo, hi), partial slot
    __device__ bool next(int &ko, int64_t &lo, int64_t &hi, int &slot) {
        for (;;) {
            while (k < k3 && off[k] < hv) {
                const int64_t a = max(share_lo<W>(P, v), off[k]), b = min(hv, off[k + 1]);
                const int kk = k++;
                if (a < b) {
                    ko = kk;
                    lo = a;
                    hi = b;
                    slot = v + kk;
                    return true;
                }
            }
            v += gridDim.x;
            if (v >= share_count<W>(P)) return false;
            const int64_t wl = share_lo<W>(P, v);
            hv = share_lo<W>(P, v + 1);
            k = 0;
            while (k < k3 && off[k + 1] <= wl) ++k;
        }
    }
};

}  // namespace wtc
}  // namespace lat
