// Root-mean-square norm of feature rows with the residual's addition, and its backward
// pass (lat_rms_norm_fwd, lat_rms_norm_bwd).
//
//   h = x + res      rstd = (mean_c h^2 + eps)^(-1/2)      y = h rstd w
//   g = dy w         xh = h rstd
//   dx = rstd (g - xh mean_c(g xh)) + dh                   dw = sum over rows of dy xh
//
// Everything between the loads and the one rounding of each output is fp32.  Both passes
// read each input once and write each output once; what bounds them is memory.
//
// A row lies in the registers of its lanes, 8 channels (16 bytes of fp16 / bf16) each:
// up to 256 channels a group of 4 to 32 lanes takes a row (K = 1), up to 512 a warp
// (K = 2 slices per lane), wider rows a block of as many warps as the row needs
// (K = 1 up to 4096 channels, else 2), whose sums meet in shared memory once per row.
//
// dw: a fixed number of blocks (never more than there are row groups) walks the rows in
// fixed steps with the sums of its rows in registers, adds its groups' sums in order in
// shared memory and stores one fp32 partial; a second kernel adds the partials in a fixed
// order.  No atomics: the bits depend neither on timing nor on the GPU.
#include <algorithm>

#include "rows.cuh"

namespace lat {
namespace norm {

using rows::Slice8;

constexpr int kThreads = 256;      // of the kernels that take several rows per block
constexpr int kShares = 592;       // blocks of the backward pass: four per B200 SM
constexpr int kMaxWarps = 32;

// Sum over the L lanes of a row's group (L <= 32), or over the block (L == 0).
template <int L>
__device__ __forceinline__ float row_sum(float v, float *s_sum, int &turn) {
    constexpr int W = L == 0 ? 32 : L;
#pragma unroll
    for (int m = W / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
    if constexpr (L == 0) {
        // two alternating sets: a set is written again only after a barrier that follows its reads
        float *s = s_sum + turn * kMaxWarps;
        turn ^= 1;
        const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        if ((threadIdx.x & 31) == 0) s[warp] = v;
        __syncthreads();
        float t = 0.f;
        for (int w = 0; w < warps; ++w) t += s[w];
        v = t;
    }
    return v;
}

template <typename T> struct Fwd {
    const T *x, *res, *w;
    T *h, *y;
    uint8_t *y8, *y8s, *h8, *h8s;
    float *rstd;
    int64_t n;
    int c;
    float eps;
};

template <typename T, int L, int K>
__global__ void __launch_bounds__(L == 0 ? 1024 : kThreads) norm_fwd_kernel(Fwd<T> a) {
    pdl_enter();
    __shared__ float s_sum[2 * kMaxWarps];
    const int lanes = L == 0 ? int(blockDim.x) : L;
    const int64_t row = L == 0 ? int64_t(blockIdx.x) : blockIdx.x * int64_t(kThreads / (L == 0 ? 1 : L)) + threadIdx.x / lanes;
    const int lane = L == 0 ? int(threadIdx.x) : int(threadIdx.x) % lanes;
    const int slices = a.c / 8;
    Slice8<T> xs[K], rs[K], ws[K];
    bool in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int vi = lane + k * lanes;
        in[k] = row < a.n && vi < slices;
        const int64_t at = row * a.c + vi * 8;
        xs[k] = in[k] ? rows::ld(a.x + at) : rows::zero_slice<T>();
        if (a.res) rs[k] = in[k] ? rows::ld(a.res + at) : rows::zero_slice<T>();
        if (a.w) ws[k] = vi < slices ? rows::ld(a.w + vi * 8) : rows::zero_slice<T>();
    }
    float v[K][8];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        rows::to_f(xs[k], v[k]);
        if (a.res) {
            float r[8];
            rows::to_f(rs[k], r);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] += r[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[k][e], v[k][e], ss);
    }
    int turn = 0;
    ss = row_sum<L>(ss, s_sum, turn);
    const float rstd = 1.f / sqrtf(ss / float(a.c) + a.eps);
    if (lane == 0 && row < a.n && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int vi = lane + k * lanes;
        const int64_t at = row * a.c + vi * 8;
        if (a.h && in[k]) rows::st(a.h + at, v[k]);
        if (a.h8) rows::q8_store(v[k], in[k], a.h8, a.h8s, row, a.c, vi);
        if (a.w) {
            float w[8];
            rows::to_f(ws[k], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] = v[k][e] * rstd * w[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] *= rstd;
        }
        if (a.y && in[k]) rows::st(a.y + at, v[k]);
        if (a.y8) rows::q8_store(v[k], in[k], a.y8, a.y8s, row, a.c, vi);
    }
}

template <typename T> struct Bwd {
    const T *dy, *h, *w, *dh;
    const uint8_t *h8, *h8s;
    const float *rstd;
    T *dx;
    float *partial;  // [gridDim.x][c], or null: no dw
    int64_t n;
    int c;
};

template <typename T, int L, int K, bool Q8>
__global__ void __launch_bounds__(L == 0 ? 1024 : kThreads) norm_bwd_kernel(Bwd<T> a) {
    pdl_enter();
    __shared__ float s_sum[2 * kMaxWarps];
    extern __shared__ float s_dw[];  // L > 0: [kThreads / L][c], the groups' sums
    constexpr int G = L == 0 ? 1 : kThreads / (L == 0 ? 1 : L);  // rows the block takes at a time
    const int lanes = L == 0 ? int(blockDim.x) : L;
    const int group = L == 0 ? 0 : int(threadIdx.x) / lanes;
    const int lane = L == 0 ? int(threadIdx.x) : int(threadIdx.x) % lanes;
    const int slices = a.c / 8;
    float w[K][8], dw[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int vi = lane + k * lanes;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[k][e] = 1.f;
            dw[k][e] = 0.f;
        }
        if (a.w && vi < slices) rows::to_f(rows::ld(a.w + vi * 8), w[k]);
    }
    const float inv_c = 1.f / float(a.c);
    int turn = 0;
    for (int64_t row0 = blockIdx.x * int64_t(G); row0 < a.n; row0 += gridDim.x * int64_t(G)) {
        const int64_t row = row0 + group;
        const float rstd = row < a.n ? __ldg(a.rstd + row) : 0.f;
        Slice8<T> ds[K], hs[K], ps[K];
        uint2 hb[K];
        int he[K];
        bool in[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int vi = lane + k * lanes;
            in[k] = row < a.n && vi < slices;
            const int64_t at = row * a.c + vi * 8;
            ds[k] = in[k] ? rows::ld(a.dy + at) : rows::zero_slice<T>();
            if constexpr (Q8) {
                hb[k] = make_uint2(0u, 0u);
                he[k] = 1;
                if (in[k]) rows::q8_load(a.h8, a.h8s, row, a.c, vi, hb[k], he[k]);
            } else {
                hs[k] = in[k] ? rows::ld(a.h + at) : rows::zero_slice<T>();
            }
            if (a.dh) ps[k] = in[k] ? rows::ld(a.dh + at) : rows::zero_slice<T>();
        }
        float xh[K][8], g[K][8];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            rows::to_f(ds[k], g[k]);
            if constexpr (Q8) rows::q8_to_f(hb[k], he[k], xh[k]);
            else rows::to_f(hs[k], xh[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[k][e] *= rstd;
                dw[k][e] = fmaf(g[k][e], xh[k][e], dw[k][e]);
                g[k][e] *= w[k][e];
                sum = fmaf(g[k][e], xh[k][e], sum);
            }
        }
        const float mean = row_sum<L>(sum, s_sum, turn) * inv_c;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!in[k]) continue;
            float p[8] = {};
            if (a.dh) rows::to_f(ps[k], p);
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = fmaf(rstd, g[k][e] - xh[k][e] * mean, p[e]);
            rows::st(a.dx + row * a.c + (lane + k * lanes) * 8, p);
        }
    }
    if (!a.partial) return;
    float *out = a.partial + blockIdx.x * int64_t(a.c);
    if constexpr (L == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (lane + k * lanes < slices) rows::st(out + (lane + k * lanes) * 8, dw[k]);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (lane + k * lanes < slices) {
                float4 *d = reinterpret_cast<float4 *>(s_dw + group * a.c + (lane + k * lanes) * 8);
                d[0] = make_float4(dw[k][0], dw[k][1], dw[k][2], dw[k][3]);
                d[1] = make_float4(dw[k][4], dw[k][5], dw[k][6], dw[k][7]);
            }
        __syncthreads();
        for (int c = threadIdx.x; c < a.c; c += kThreads) {
            float t = 0.f;
            for (int i = 0; i < G; ++i) t += s_dw[i * a.c + c];
            out[c] = t;
        }
    }
}

// dw[c] = sum over the blocks' partials: 32 channels per block, row p of 32 takes the
// partials p, p + 32, ... in order, then the 32 sums are added in order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *__restrict__ partial, int shares, int c,
                                                       float *__restrict__ dw) {
    pdl_enter();
    __shared__ float s[32][33];
    const int ch = blockIdx.x * 32 + threadIdx.x;
    float t = 0.f;
    if (ch < c) {
#pragma unroll 4
        for (int p = threadIdx.y; p < shares; p += 32) t += partial[int64_t(p) * c + ch];
    }
    s[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y == 0 && ch < c) {
        t = 0.f;
#pragma unroll
        for (int p = 0; p < 32; ++p) t += s[p][threadIdx.x];
        dw[ch] = t;
    }
}

// Calls f with the row layout for c channels: lanes per row (0: a block), slices per
// lane, and the threads of a block.
template <typename F>
static lat_status by_layout(int c, F &&f) {
    const int slices = c / 8;
    if (slices <= 4) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{}, kThreads);
    if (slices <= 8) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{}, kThreads);
    if (slices <= 16) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{}, kThreads);
    if (slices <= 32) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{}, kThreads);
    if (slices <= 64) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{}, kThreads);
    if (slices <= 512)
        return f(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{}, (slices + 31) / 32 * 32);
    return f(std::integral_constant<int, 0>{}, std::integral_constant<int, 2>{}, (slices + 63) / 64 * 32);
}

// Rows a block takes at a time.
static int rows_per_block(int c) {
    const int slices = c / 8;
    int l = 4;
    while (l < 32 && l < slices) l *= 2;
    return slices <= 64 ? kThreads / l : 1;
}

static int64_t shares(int64_t n, int c) {
    const int per = rows_per_block(c);
    return std::max<int64_t>(1, std::min<int64_t>(kShares, (n + per - 1) / per));
}

template <typename T>
lat_status fwd(const void *x, const void *res, const void *w, int64_t n, int c, float eps, void *h, void *y, void *y8,
               void *y8s, void *h8, void *h8s, float *rstd, cudaStream_t s) {
    Fwd<T> a{static_cast<const T *>(x), static_cast<const T *>(res), static_cast<const T *>(w), static_cast<T *>(h),
             static_cast<T *>(y), static_cast<uint8_t *>(y8), static_cast<uint8_t *>(y8s), static_cast<uint8_t *>(h8),
             static_cast<uint8_t *>(h8s), rstd, n, c, eps};
    const int64_t per = rows_per_block(c);
    return by_layout(c, [&](auto l, auto k, int threads) -> lat_status {
        LAT_CUDA_TRY(launch_pdl(norm_fwd_kernel<T, decltype(l)::value, decltype(k)::value>,
                                dim3(unsigned((n + per - 1) / per)), dim3(threads), 0, s, a));
        return LAT_OK;
    });
}

template <typename T>
lat_status bwd(const void *dy, const void *dh, const void *h, const void *h8, const void *h8s, const float *rstd,
               const void *w, int64_t n, int c, void *dx, float *dw, float *partial, cudaStream_t s) {
    Bwd<T> a{static_cast<const T *>(dy), static_cast<const T *>(h), static_cast<const T *>(w),
             static_cast<const T *>(dh), static_cast<const uint8_t *>(h8), static_cast<const uint8_t *>(h8s), rstd,
             static_cast<T *>(dx), dw ? partial : nullptr, n, c};
    const int64_t blocks = shares(n, c);
    const lat_status st = by_layout(c, [&](auto l, auto k, int threads) -> lat_status {
        constexpr int L = decltype(l)::value, K = decltype(k)::value;
        const size_t smem = L == 0 ? 0 : sizeof(float) * size_t(kThreads / (L == 0 ? 1 : L)) * size_t(c);
        if (h8)
            LAT_CUDA_TRY(launch_pdl(norm_bwd_kernel<T, L, K, true>, dim3(unsigned(blocks)), dim3(threads), smem, s, a));
        else
            LAT_CUDA_TRY(launch_pdl(norm_bwd_kernel<T, L, K, false>, dim3(unsigned(blocks)), dim3(threads), smem, s, a));
        return LAT_OK;
    });
    if (st != LAT_OK || !dw) return st;
    LAT_CUDA_TRY(launch_pdl(norm_dw_kernel, dim3(unsigned((c + 31) / 32)), dim3(32, 32), 0, s, partial, int(blocks), c,
                            dw));
    return LAT_OK;
}

}  // namespace norm
}  // namespace lat

extern "C" lat_status lat_rms_norm_fwd(const void *x, const void *res, const void *w, int64_t n, int32_t c, float eps,
                                       void *h, void *y, void *y8, void *y8_scale, void *h8, void *h8_scale,
                                       float *rstd, lat_dtype dtype, lat_stream stream) {
    using namespace lat;
    if (!rows::rows_ok(n) || !rows::chan_ok(c) || !(eps > 0.f) || !(eps <= FLT_MAX)) return LAT_ERR_ARG;
    if (dtype != LAT_F32 && dtype != LAT_F16 && dtype != LAT_BF16) return LAT_ERR_ARG;
    if (!y8 != !y8_scale || !h8 != !h8_scale) return LAT_ERR_ARG;
    if (n > 0 && !x) return LAT_ERR_ARG;
    for (const void *p : {x, res, w, static_cast<const void *>(h), static_cast<const void *>(y)})
        if (!rows::aligned(p, rows::slice_bytes(dtype))) return LAT_ERR_ARG;
    if (!rows::aligned(y8, 16) || !rows::aligned(h8, 16)) return LAT_ERR_ARG;
    if (n == 0) return LAT_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (dtype) {
        case LAT_F32: return norm::fwd<float>(x, res, w, n, c, eps, h, y, y8, y8_scale, h8, h8_scale, rstd, s);
        case LAT_F16: return norm::fwd<__half>(x, res, w, n, c, eps, h, y, y8, y8_scale, h8, h8_scale, rstd, s);
        case LAT_BF16:
            return norm::fwd<__nv_bfloat16>(x, res, w, n, c, eps, h, y, y8, y8_scale, h8, h8_scale, rstd, s);
    }
    return LAT_ERR_ARG;
}

extern "C" size_t lat_rms_norm_bwd_ws_bytes(int64_t n, int32_t c) {
    using namespace lat;
    if (!rows::rows_ok(n) || !rows::chan_ok(c)) return 0;
    return align_up(sizeof(float) * size_t(norm::shares(n, c)) * size_t(c), 256);
}

extern "C" lat_status lat_rms_norm_bwd(const void *dy, const void *dh, const void *h, const void *h8,
                                       const void *h8_scale, const float *rstd, const void *w, int64_t n, int32_t c,
                                       void *dx, float *dw, lat_dtype dtype, void *ws, size_t ws_bytes,
                                       lat_stream stream) {
    using namespace lat;
    if (!rows::rows_ok(n) || !rows::chan_ok(c)) return LAT_ERR_ARG;
    if (dtype != LAT_F32 && dtype != LAT_F16 && dtype != LAT_BF16) return LAT_ERR_ARG;
    if (!h8 != !h8_scale || (h && h8)) return LAT_ERR_ARG;
    if (n > 0 && (!dy || !rstd || !dx || (!h && !h8))) return LAT_ERR_ARG;
    for (const void *p : {dy, dh, h, w, static_cast<const void *>(dx)})
        if (!rows::aligned(p, rows::slice_bytes(dtype))) return LAT_ERR_ARG;
    if (!rows::aligned(h8, 16) || !rows::aligned(dw, 4)) return LAT_ERR_ARG;
    if (dw && (!ws || !rows::aligned(ws, 32) || ws_bytes < lat_rms_norm_bwd_ws_bytes(n, c))) return LAT_ERR_WORKSPACE;
    if (n == 0 && !dw) return LAT_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    float *partial = static_cast<float *>(ws);
    switch (dtype) {
        case LAT_F32: return norm::bwd<float>(dy, dh, h, h8, h8_scale, rstd, w, n, c, dx, dw, partial, s);
        case LAT_F16: return norm::bwd<__half>(dy, dh, h, h8, h8_scale, rstd, w, n, c, dx, dw, partial, s);
        case LAT_BF16: return norm::bwd<__nv_bfloat16>(dy, dh, h, h8, h8_scale, rstd, w, n, c, dx, dw, partial, s);
    }
    return LAT_ERR_ARG;
}
