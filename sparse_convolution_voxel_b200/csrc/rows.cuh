// Feature rows in 8-channel slices: the loads, stores and the 8-bit form shared by the
// row-wise kernels (norm.cu, embed.cu, q8.cu).
#pragma once

#include <cuda_fp8.h>
#include <float.h>

#include <type_traits>

#include "common.cuh"

namespace lat {
namespace rows {

// 8 consecutive channels of one row: 16 bytes (fp16 / bf16) or 32 (fp32), moved by one
// instruction per lane.  (fp32 as two 16-byte halves, each 32 bytes from its neighbour's,
// costs twice the L1 wavefronts: 69% of L1's rate at 3.2 TB/s in the lookup gradient.)
template <typename T> struct Slice8 {
    uint32_t v[2 * sizeof(T)];
};

// An ordinary load, in order with the stores: several entry points may write a row over the
// one they read.
template <typename T>
__device__ __forceinline__ Slice8<T> ld(const T *p) {
    Slice8<T> s;
    if constexpr (sizeof(T) == 4) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(s.v[0]), "=r"(s.v[1]), "=r"(s.v[2]), "=r"(s.v[3]), "=r"(s.v[4]), "=r"(s.v[5]), "=r"(s.v[6]),
                       "=r"(s.v[7])
                     : "l"(p)
                     : "memory");
    } else {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        s.v[0] = q.x;
        s.v[1] = q.y;
        s.v[2] = q.z;
        s.v[3] = q.w;
    }
    return s;
}
template <typename T>
__device__ __forceinline__ Slice8<T> zero_slice() {
    Slice8<T> s;
#pragma unroll
    for (int h = 0; h < int(2 * sizeof(T)); ++h) s.v[h] = 0u;
    return s;
}
template <typename T>
__device__ __forceinline__ void to_f(const Slice8<T> &s, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = __uint_as_float(s.v[c]);
    } else if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&s.v[c]));
            v[2 * c] = f.x;
            v[2 * c + 1] = f.y;
        }
    } else {  // a bf16 is the upper half of its fp32
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[2 * c] = __uint_as_float(s.v[c] << 16);
            v[2 * c + 1] = __uint_as_float(s.v[c] & 0xFFFF0000u);
        }
    }
}
// Two values of T (16 bits) in a word, rounded to nearest even.
template <typename T>
__device__ __forceinline__ uint32_t two(float a, float b) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <typename T>
__device__ __forceinline__ void st(T *p, const float (&v)[8]) {
    Slice8<T> s;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int c = 0; c < 8; ++c) s.v[c] = __float_as_uint(v[c]);
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) s.v[c] = two<T>(v[2 * c], v[2 * c + 1]);
    }
    if constexpr (sizeof(T) == 4)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(s.v[0]), "r"(s.v[1]),
                     "r"(s.v[2]), "r"(s.v[3]), "r"(s.v[4]), "r"(s.v[5]), "r"(s.v[6]), "r"(s.v[7])
                     : "memory");
    else
        *reinterpret_cast<uint4 *>(p) = make_uint4(s.v[0], s.v[1], s.v[2], s.v[3]);
}

// 16 channels at a 32-byte aligned address: one 256-bit access (fp16 / bf16) or two (fp32).
__device__ __forceinline__ Slice8<float> ld32(const void *p) { return ld(static_cast<const float *>(p)); }
template <typename T>
__device__ __forceinline__ void ld16(const T *p, float (&v)[2][8]) {
    if constexpr (sizeof(T) == 4) {
        to_f(ld(p), v[0]);
        to_f(ld(p + 8), v[1]);
    } else {
        const Slice8<float> r = ld32(p);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Slice8<T> s;
#pragma unroll
            for (int c = 0; c < 4; ++c) s.v[c] = r.v[4 * h + c];
            to_f(s, v[h]);
        }
    }
}
template <typename T>
__device__ __forceinline__ void st16(T *p, const float (&v)[2][8]) {
    if constexpr (sizeof(T) == 4) {
        st(p, v[0]);
        st(p + 8, v[1]);
    } else {
        float w[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = __uint_as_float(two<T>(v[c / 4][2 * (c % 4)], v[c / 4][2 * (c % 4) + 1]));
        st(reinterpret_cast<float *>(p), w);
    }
}

// Two fp32 operations in one instruction (sm_100).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)),
          "l"(*reinterpret_cast<uint64_t *>(&c)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// ------------------------------------------------------------------- 8-bit rows
// A group of 32 channels of one row shares the scale 2^(E - 127), E >= 1 the smallest
// exponent byte with amax <= 448 * scale (448: the largest e4m3 value), amax over the
// finite values; a value is stored as e4m3(v / scale), rounded to nearest even.  The
// division by a power of two is exact, so the one rounding is e4m3's (at most 2^-4 of
// the value, or 2^-10 scale below 2^-6 scale), and scale * e4m3 has 4 significant bits:
// bf16 holds it exactly.
constexpr int kQ8Group = 32;

__host__ __device__ __forceinline__ int q8_groups(int c) { return (c + kQ8Group - 1) / kQ8Group; }

// amax = m 2^x with 1 <= m < 2: the scale is 2^(x - 8) while m <= 1.75, else 2^(x - 7).
// Adding 0x1FFFFF carries into the exponent exactly for mantissas above 1.75.
__device__ __forceinline__ int q8_exponent(float amax) {
    return max(1, int((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8);
}
__device__ __forceinline__ float q8_scale(int e) { return __uint_as_float(uint32_t(e) << 23); }
__device__ __forceinline__ float q8_inverse(int e) { return __uint_as_float(uint32_t(254 - e) << 23); }

// Largest finite magnitude of 8 channels (0 if none is finite).
__device__ __forceinline__ float finite_amax(const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const float a = fabsf(v[c]);
        m = fmaxf(m, a <= FLT_MAX ? a : 0.f);
    }
    return m;
}

__device__ __forceinline__ uint32_t q8_pair(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// 8 channels to e4m3; what is not finite becomes NaN (the format has no infinity).
__device__ __forceinline__ uint2 q8_from_f(const float (&v)[8], int e) {
    const float inv = q8_inverse(e);
    float u[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) u[c] = fabsf(v[c]) <= FLT_MAX ? v[c] * inv : __int_as_float(0x7FFFFFFF);
    return make_uint2(q8_pair(u[0], u[1]) | (q8_pair(u[2], u[3]) << 16),
                      q8_pair(u[4], u[5]) | (q8_pair(u[6], u[7]) << 16));
}
template <typename T>
__device__ __forceinline__ void to_f2(const Slice8<T> &s, float2 (&v)[4]) {
    float f[8];
    to_f(s, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = make_float2(f[2 * e], f[2 * e + 1]);
}
__device__ __forceinline__ void q8_to_f2(uint2 q, int e, float2 (&v)[4]) {
    const uint32_t w[4] = {q.x, q.x >> 16, q.y, q.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w[i] & 0xFFFFu), __NV_E4M3);
        v[i] = mul2(__half22float2(__half2(r)), both(q8_scale(e)));
    }
}

__device__ __forceinline__ void q8_to_f(uint2 q, int e, float (&v)[8]) {
    float2 f[4];
    q8_to_f2(q, e, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = f[i].x;
        v[2 * i + 1] = f[i].y;
    }
}

// Stores slice `vi` of row `row` in 8 bits.  Called by every lane of the warp: the four
// lanes of a 4-aligned run hold the four slices of one group (slices past the row's end
// hold zeros and are not stored).
__device__ __forceinline__ void q8_store(const float (&v)[8], bool in, uint8_t *q, uint8_t *scale, int64_t row, int c,
                                         int vi) {
    float m = in ? finite_amax(v) : 0.f;
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (!in) return;
    const int e = q8_exponent(m);
    *reinterpret_cast<uint2 *>(q + row * c + vi * 8) = q8_from_f(v, e);
    if ((vi & 3) == 0) scale[row * q8_groups(c) + (vi >> 2)] = uint8_t(e);
}

// Slice `vi` of row `row` of 8-bit rows.
__device__ __forceinline__ void q8_load(const uint8_t *q, const uint8_t *scale, int64_t row, int c, int vi, uint2 &bits,
                                        int &e) {
    bits = __ldg(reinterpret_cast<const uint2 *>(q + row * c + vi * 8));
    e = __ldg(scale + row * q8_groups(c) + (vi >> 2));
}

// A value in T: fp16 ends at 65504, which a group's largest value can round past, so it
// is held there; bf16 and fp32 have the range of the scales.
template <typename T> __device__ __forceinline__ float in_range(float v) { return v; }
template <> __device__ __forceinline__ float in_range<__half>(float v) {
    return fabsf(v) > 65504.f ? copysignf(65504.f, v) : v;  // NaN stays NaN
}

// Values of a group with scale byte e as T holds them, back in fp32: only fp16 changes one (bf16 does below 2^-133,
// which is left), and none of a group with 2^-9 scale, e4m3's smallest step, at least 2^-24 and 448 scale below 65504.
template <typename T>
__device__ __forceinline__ void as_held(float (&v)[8], int e) {
    if constexpr (std::is_same<T, __half>::value) {
        if (uint32_t(e - 112) <= 134u - 112u) return;
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = __half2float(__float2half_rn(in_range<T>(v[c])));
    }
}

// Host checks of the row-wise entry points.
constexpr int kMaxChannels = 16384;
inline bool chan_ok(int c) { return c >= 8 && c % 8 == 0 && c <= kMaxChannels; }
inline bool rows_ok(int64_t n) { return n >= 0 && n < (int64_t(1) << 31); }
// Rows are read and written in slices of 8 channels.
inline size_t slice_bytes(lat_dtype dtype) { return dtype == LAT_F32 ? 32 : 16; }
inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace rows
}  // namespace lat
