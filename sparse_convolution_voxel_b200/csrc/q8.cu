// Activation checkpoints in 8 bits (lat_q8_pack, lat_q8_unpack): rows to e4m3 with one
// power-of-two scale per 32 channels, and back.  The format is in rows.cuh.
//
// Both are one pass over the rows, bound by memory: pack moves (e + 33/32) bytes per
// value, unpack the same.  Rows of whole groups (c a multiple of 32) are one run of
// groups: a lane takes 16 channels, 16 bytes of e4m3 and 32 (fp16 / bf16) or 2 x 32 (fp32)
// of values, and two lanes make a group.  Other rows: a lane takes 8 channels, the four
// lanes of a group exchange their largest magnitudes, L lanes take a row (a power of two, 4
// to 32) and a warp takes wider rows in steps of 32 slices.
#include "rows.cuh"

namespace lat {
namespace q8 {

constexpr int kThreads = 256;

template <typename T, int L>
__global__ void __launch_bounds__(kThreads)
pack_kernel(const T *__restrict__ x, int64_t n, int c, uint8_t *__restrict__ q, uint8_t *__restrict__ scale) {
    pdl_enter();
    const int64_t row = blockIdx.x * int64_t(kThreads / L) + threadIdx.x / L;
    const int slices = c / 8;
    for (int v0 = 0; v0 < slices; v0 += L) {
        const int vi = v0 + threadIdx.x % L;
        const bool in = row < n && vi < slices;
        float v[8] = {};
        if (in) rows::to_f(rows::ld(x + row * c + vi * 8), v);
        rows::q8_store(v, in, q, scale, row, c, vi);
    }
}

template <typename T, int L>
__global__ void __launch_bounds__(kThreads)
unpack_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale, int64_t n, int c, T *__restrict__ x) {
    pdl_enter();
    const int64_t row = blockIdx.x * int64_t(kThreads / L) + threadIdx.x / L;
    if (row >= n) return;
    for (int vi = threadIdx.x % L; vi < c / 8; vi += L) {
        uint2 bits;
        int e;
        rows::q8_load(q, scale, row, c, vi, bits, e);
        float v[8];
        rows::q8_to_f(bits, e, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = rows::in_range<T>(v[i]);
        rows::st(x + row * c + vi * 8, v);
    }
}

// Whole groups: thread t takes channels 16 t .. 16 t + 15 of the run of n * c.
template <typename T>
__global__ void __launch_bounds__(kThreads)
pack_run_kernel(const T *__restrict__ x, int64_t halves, uint8_t *__restrict__ q, uint8_t *__restrict__ scale) {
    pdl_enter();
    const int64_t t = blockIdx.x * int64_t(kThreads) + threadIdx.x;
    const bool in = t < halves;
    float v[2][8] = {};
    if (in) rows::ld16(x + t * 16, v);
    float m = fmaxf(rows::finite_amax(v[0]), rows::finite_amax(v[1]));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    if (!in) return;
    const int e = rows::q8_exponent(m);
    const uint2 a = rows::q8_from_f(v[0], e), b = rows::q8_from_f(v[1], e);
    reinterpret_cast<uint4 *>(q)[t] = make_uint4(a.x, a.y, b.x, b.y);
    if ((t & 1) == 0) scale[t >> 1] = uint8_t(e);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
unpack_run_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale, int64_t halves, T *__restrict__ x) {
    pdl_enter();
    const int64_t t = blockIdx.x * int64_t(kThreads) + threadIdx.x;
    if (t >= halves) return;
    const uint4 r = __ldg(reinterpret_cast<const uint4 *>(q) + t);
    const int e = __ldg(scale + (t >> 1));
    float v[2][8];
    rows::q8_to_f(make_uint2(r.x, r.y), e, v[0]);
    rows::q8_to_f(make_uint2(r.z, r.w), e, v[1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[0][i] = rows::in_range<T>(v[0][i]);
        v[1][i] = rows::in_range<T>(v[1][i]);
    }
    rows::st16(x + t * 16, v);
}

static unsigned run_blocks(int64_t halves) { return unsigned((halves + kThreads - 1) / kThreads); }

template <typename F>
static lat_status by_lanes(int c, F &&f) {
    const int slices = c / 8;
    if (slices <= 4) return f(std::integral_constant<int, 4>{});
    if (slices <= 8) return f(std::integral_constant<int, 8>{});
    if (slices <= 16) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

template <typename T>
lat_status pack(const void *x, int64_t n, int c, uint8_t *q, uint8_t *scale, cudaStream_t s) {
    if (c % rows::kQ8Group == 0 && rows::aligned(x, 32)) {
        LAT_CUDA_TRY(launch_pdl(pack_run_kernel<T>, dim3(run_blocks(n * c / 16)), dim3(kThreads), 0, s,
                                static_cast<const T *>(x), n * c / 16, q, scale));
        return LAT_OK;
    }
    return by_lanes(c, [&](auto l) -> lat_status {
        constexpr int L = decltype(l)::value;
        const int64_t per = kThreads / L;
        LAT_CUDA_TRY(launch_pdl(pack_kernel<T, L>, dim3(unsigned((n + per - 1) / per)), dim3(kThreads), 0, s,
                                static_cast<const T *>(x), n, c, q, scale));
        return LAT_OK;
    });
}

template <typename T>
lat_status unpack(const uint8_t *q, const uint8_t *scale, int64_t n, int c, void *x, cudaStream_t s) {
    if (c % rows::kQ8Group == 0 && rows::aligned(x, 32)) {
        LAT_CUDA_TRY(launch_pdl(unpack_run_kernel<T>, dim3(run_blocks(n * c / 16)), dim3(kThreads), 0, s, q, scale,
                                n * c / 16, static_cast<T *>(x)));
        return LAT_OK;
    }
    return by_lanes(c, [&](auto l) -> lat_status {
        constexpr int L = decltype(l)::value;
        const int64_t per = kThreads / L;
        LAT_CUDA_TRY(launch_pdl(unpack_kernel<T, L>, dim3(unsigned((n + per - 1) / per)), dim3(kThreads), 0, s, q, scale,
                                n, c, static_cast<T *>(x)));
        return LAT_OK;
    });
}

}  // namespace q8
}  // namespace lat

extern "C" lat_status lat_q8_pack(const void *x, int64_t n, int32_t c, void *q, void *scale, lat_dtype dtype,
                                  lat_stream stream) {
    using namespace lat;
    if (!rows::rows_ok(n) || !rows::chan_ok(c)) return LAT_ERR_ARG;
    if (dtype != LAT_F32 && dtype != LAT_F16 && dtype != LAT_BF16) return LAT_ERR_ARG;
    if (n > 0 && (!x || !q || !scale)) return LAT_ERR_ARG;
    if (!rows::aligned(x, rows::slice_bytes(dtype)) || !rows::aligned(q, 16)) return LAT_ERR_ARG;
    if (n == 0) return LAT_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *qb = static_cast<uint8_t *>(q), *sb = static_cast<uint8_t *>(scale);
    switch (dtype) {
        case LAT_F32: return q8::pack<float>(x, n, c, qb, sb, s);
        case LAT_F16: return q8::pack<__half>(x, n, c, qb, sb, s);
        case LAT_BF16: return q8::pack<__nv_bfloat16>(x, n, c, qb, sb, s);
    }
    return LAT_ERR_ARG;
}

extern "C" lat_status lat_q8_unpack(const void *q, const void *scale, int64_t n, int32_t c, void *x, lat_dtype dtype,
                                    lat_stream stream) {
    using namespace lat;
    if (!rows::rows_ok(n) || !rows::chan_ok(c)) return LAT_ERR_ARG;
    if (dtype != LAT_F32 && dtype != LAT_F16 && dtype != LAT_BF16) return LAT_ERR_ARG;
    if (n > 0 && (!x || !q || !scale)) return LAT_ERR_ARG;
    if (!rows::aligned(x, rows::slice_bytes(dtype)) || !rows::aligned(q, 16)) return LAT_ERR_ARG;
    if (n == 0) return LAT_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const uint8_t *qb = static_cast<const uint8_t *>(q), *sb = static_cast<const uint8_t *>(scale);
    switch (dtype) {
        case LAT_F32: return q8::unpack<float>(qb, sb, n, c, x, s);
        case LAT_F16: return q8::unpack<__half>(qb, sb, n, c, x, s);
        case LAT_BF16: return q8::unpack<__nv_bfloat16>(qb, sb, n, c, x, s);
    }
    return LAT_ERR_ARG;
}
