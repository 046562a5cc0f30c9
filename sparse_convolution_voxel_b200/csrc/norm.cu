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
// A row lies in the registers of its lanes, 8 channels each: up to 256 channels a group of 4
// to 32 lanes takes a row (K = 1 slice per lane), up to 512 a warp (K = 2), wider rows a
// block with K = 1 (to 1024 channels), 2 (to 8192) or 4 slices per lane, whose sums meet in
// shared memory once per row.
//
// The backward pass walks several rows per group.  A lane copies its slices of the rows ahead
// with cp.async into a ring of its own in shared memory -- it alone reads them, so its own
// copies are all it waits for -- which keeps them in flight without the registers that loads
// ahead would take: 160 KB per SM at 500k x 128 bf16 from 8-bit rows with dh (450 MB; back to back
// on the same rows 98 us with a row's loads in front of its work, 106 us with the next row in
// registers, 89 us so; 81 with offsets that advance and two fp32 operations per instruction, of
// which 6 are dw's second kernel).  It is 28 KB at the least, at 1,032 channels of 16 bits from 8-bit
// rows without dh, and above 8,192 channels of fp32 it holds no row ahead.
//
// dw: a fixed number of blocks (never more than there are row groups) walks the rows in
// fixed steps with the sums of its rows in registers, adds its groups' sums in order in
// shared memory and stores one fp32 partial; a second kernel adds the partials in a fixed
// order.  No atomics: the bits depend neither on timing nor on the GPU.
#include <algorithm>

#include "rows.cuh"
#include "tc_ptx.cuh"

namespace lat {
namespace norm {

using rows::Slice8;

constexpr int kThreads = 256;      // of the kernels that take several rows per block
constexpr int kWideThreads = 512;  // at most, where a block takes a row
constexpr int kMaxWarps = kWideThreads / 32;

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
__global__ void __launch_bounds__(L == 0 ? kWideThreads : kThreads) norm_fwd_kernel(Fwd<T> a) {
    pdl_enter();
    __shared__ float s_sum[2 * kMaxWarps];
    const int lanes = L == 0 ? int(blockDim.x) : L;
    const int64_t row = L == 0 ? int64_t(blockIdx.x)
                               : blockIdx.x * int64_t(kThreads / (L == 0 ? 1 : L)) + threadIdx.x / lanes;
    const int lane = L == 0 ? int(threadIdx.x) : int(threadIdx.x) % lanes;
    const int slices = a.c / 8;
    Slice8<T> xs[K], rs[K];
    bool in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int vi = lane + k * lanes;
        in[k] = row < a.n && vi < slices;
        const int64_t at = row * a.c + vi * 8;
        xs[k] = in[k] ? rows::ld(a.x + at) : rows::zero_slice<T>();
        if (a.res) rs[k] = in[k] ? rows::ld(a.res + at) : rows::zero_slice<T>();
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
            rows::to_f(vi < slices ? rows::ld(a.w + vi * 8) : rows::zero_slice<T>(), w);
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

// Rows in the ring (the one at work included): within 200 KB of shared memory per SM for the widest rows of a form.
template <typename T, int L, int K>
constexpr int ring_rows() {
    return K == 4 && sizeof(T) == 4 ? 1 : K == 4 || sizeof(T) == 4 || (K == 2 && L == 0) ? 2 : 4;
}
// Bytes of a thread's slices of one row.
template <typename T, int K, bool Q8>
constexpr int ring_bytes(bool dh) {
    return K * (int(8 * sizeof(T)) * (1 + (Q8 ? 0 : 1) + (dh ? 1 : 0)) + (Q8 ? 8 : 0));
}

// Shared memory of a call: the ring, and in its place at the end the groups' sums of dw.
template <typename T, int L, int K, bool Q8>
constexpr size_t bwd_smem(bool dh, int threads, int c) {
    const size_t ring = size_t(ring_bytes<T, K, Q8>(dh)) * size_t(threads) * ring_rows<T, L, K>();
    const size_t sums = L == 0 ? 0 : sizeof(float) * size_t(kThreads / (L == 0 ? 1 : L)) * size_t(c);
    return ring > sums ? ring : sums;
}
// Most that any call of the kernel takes: its limit is the same in every call, since another host thread may be about
// to launch it with more than this one.
template <typename T, int L, int K, bool Q8>
constexpr size_t bwd_smem_limit() {
    return bwd_smem<T, L, K, Q8>(true, L == 0 ? kWideThreads : kThreads, 8 * L * K);
}

template <typename T, int L, int K>
constexpr int min_blocks() {  // per SM, for the registers
    return L > 0 && K == 1 ? 4 : L == 0 && K == 2 && sizeof(T) == 2 ? 2 : 1;
}

template <typename T, int L, int K, bool Q8>
__global__ void __launch_bounds__(L == 0 ? kWideThreads : kThreads, min_blocks<T, L, K>())
norm_bwd_kernel(Bwd<T> a) {
    pdl_enter();
    __shared__ float s_sum[2 * kMaxWarps];
    extern __shared__ __align__(16) uint8_t s_ring[];  // and, at the end, the groups' sums of dw: [kThreads / L][c]
    constexpr int G = L == 0 ? 1 : kThreads / (L == 0 ? 1 : L);  // rows the block takes at a time
    constexpr int D = ring_rows<T, L, K>(), CH = int(sizeof(T)) / 2;  // 16-byte chunks per slice
    const int threads = L == 0 ? int(blockDim.x) : kThreads;
    const int lanes = L == 0 ? int(blockDim.x) : L;
    const int group = L == 0 ? 0 : int(threadIdx.x) / lanes;
    const int lane = L == 0 ? int(threadIdx.x) : int(threadIdx.x) % lanes;
    const int slices = a.c / 8;
    const bool with_dh = a.dh != nullptr;
    // a row of the ring: 16-byte chunks of dy, h (or 8-byte chunks of h8, last) and dh, each one
    // chunk after the other for all threads
    const uint32_t row_bytes = ring_bytes<T, K, Q8>(with_dh) * threads;
    const uint32_t array_bytes = K * CH * threads * 16;
    const uint32_t dh_at = (Q8 ? 1 : 2) * array_bytes, h8_at = (with_dh ? 2 : 1) * array_bytes;
    uint8_t *mine = s_ring + threadIdx.x * 16;
    auto chunk = [&](uint32_t at, int k, int half) { return mine + at + (k * CH + half) * threads * 16; };
    auto chunk8 = [&](uint32_t slot, int k) { return s_ring + slot + h8_at + (k * threads + int(threadIdx.x)) * 8; };
    bool has[K];
#pragma unroll
    for (int k = 0; k < K; ++k) has[k] = lane + k * lanes < slices;
    // offsets of this lane's first slice: of the row at work and of the row that is copied next;
    // of its scale byte, one row ahead
    const uint32_t rows_n = uint32_t(a.n), stride = gridDim.x * G;
    const int64_t step = int64_t(stride) * a.c, scale_step = int64_t(stride) * rows::q8_groups(a.c);
    uint32_t row = blockIdx.x * G + group, copy_row = row;
    int64_t at = int64_t(row) * a.c + lane * 8, copy_at = at;
    int64_t scale_at = int64_t(row) * rows::q8_groups(a.c) + (lane >> 2);
    auto copy = [&](uint32_t slot) {
        if (copy_row < rows_n) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!has[k]) continue;
                const int64_t o = copy_at + k * lanes * 8;
#pragma unroll
                for (int half = 0; half < CH; ++half) {
                    ptx::cp_async16(chunk(slot, k, half), a.dy + o + half * 4, 16u);
                    if constexpr (!Q8) ptx::cp_async16(chunk(slot + array_bytes, k, half), a.h + o + half * 4, 16u);
                    if (with_dh) ptx::cp_async16(chunk(slot + dh_at, k, half), a.dh + o + half * 4, 16u);
                }
                if constexpr (Q8) ptx::cp_async8(chunk8(slot, k), a.h8 + o);
            }
        }
        ptx::cp_async_commit();
        copy_row += stride;
        copy_at += step;
    };
    auto slice = [&](uint32_t at_, int k) {
        Slice8<T> r;
#pragma unroll
        for (int half = 0; half < CH; ++half) {
            const uint4 q = *reinterpret_cast<const uint4 *>(chunk(at_, k, half));
            r.v[4 * half] = q.x;
            r.v[4 * half + 1] = q.y;
            r.v[4 * half + 2] = q.z;
            r.v[4 * half + 3] = q.w;
        }
        return r;
    };
    using rows::add2;
    using rows::both;
    using rows::fma2;
    using rows::mul2;
    float2 dw[K][4] = {};
    // one slice per lane: a row's g and h stay in registers; more: they are computed again, which
    // leaves room for two blocks per SM.  The weights stay but for four slices (from L1 then).
    constexpr bool kKeep = K == 1, kKeepW = K < 4;
    float2 ws[kKeepW ? K : 1][4];
    auto weight = [&](int k, float2 (&v)[4]) {
        const int vi = lane + k * lanes;
        if (a.w && vi < slices) {
            rows::to_f2(rows::ld(a.w + vi * 8), v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = both(1.f);
        }
    };
    if constexpr (kKeepW) {
#pragma unroll
        for (int k = 0; k < K; ++k) weight(k, ws[k]);
    }
    const float inv_c = 1.f / float(a.c);
    struct Small {  // the row's rstd and scale bytes, read one row ahead
        float rstd;
        int e[K];
    };
    auto small = [&](uint32_t r) {
        Small m;
        m.rstd = r < rows_n ? __ldg(a.rstd + r) : 0.f;
        if constexpr (Q8) {
#pragma unroll
            for (int k = 0; k < K; ++k) m.e[k] = r < rows_n && has[k] ? __ldg(a.h8s + scale_at + (k * lanes >> 2)) : 1;
            scale_at += scale_step;
        }
        return m;
    };
    uint32_t slot = 0, ahead = (D - 1) * row_bytes;  // byte offsets in the ring
    // slice k of d = rstd dy, of h, and of g = rstd dy w
    auto terms = [&](const Small &m, int k, float2 (&d)[4], float2 (&h)[4], float2 (&g)[4]) {
        rows::to_f2(slice(slot, k), d);
        if constexpr (Q8) rows::q8_to_f2(*reinterpret_cast<const uint2 *>(chunk8(slot, k)), m.e[k], h);
        else rows::to_f2(slice(slot + array_bytes, k), h);
        float2 w[4];
        if constexpr (!kKeepW) weight(k, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            d[e] = mul2(d[e], both(m.rstd));
            g[e] = mul2(d[e], kKeepW ? ws[k][e] : w[e]);
        }
    };
    int turn = 0;
#pragma unroll
    for (int d = 0; d < D - 1; ++d) copy(d * row_bytes);
    Small cur = small(row);
    // every group of a block takes as many turns as the first one: they meet in row_sum
    for (uint32_t row0 = blockIdx.x * G; row0 < rows_n; row0 += stride) {
        copy(ahead);
        const Small next = small(row + stride);
        ptx::cp_async_wait<D - 1>();
        const bool in = row < rows_n;
        float2 sum = both(0.f), h[kKeep ? K : 1][4], g[kKeep ? K : 1][4];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!in || !has[k]) continue;
            constexpr int S = kKeep ? 1 : 0;
            float2 d[4];
            terms(cur, k, d, h[S * k], g[S * k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dw[k][e] = fma2(d[e], h[S * k][e], dw[k][e]);
                sum = fma2(g[S * k][e], h[S * k][e], sum);
            }
        }
        // dx = g - h rstd^2 mean(g h) + dh
        const float2 back = both(-row_sum<L>(sum.x + sum.y, s_sum, turn) * inv_c * cur.rstd * cur.rstd);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!in || !has[k]) continue;
            constexpr int S = kKeep ? 1 : 0;
            float2 d[4];
            if constexpr (!kKeep) terms(cur, k, d, h[0], g[0]);
            if (with_dh) {
                float2 p[4];
                rows::to_f2(slice(slot + dh_at, k), p);
#pragma unroll
                for (int e = 0; e < 4; ++e) g[S * k][e] = add2(g[S * k][e], p[e]);
            }
            float out[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 o = fma2(h[S * k][e], back, g[S * k][e]);
                out[2 * e] = o.x;
                out[2 * e + 1] = o.y;
            }
            rows::st(a.dx + at + k * lanes * 8, out);
        }
        cur = next;
        row += stride;
        at += step;
        slot = slot + row_bytes == D * row_bytes ? 0 : slot + row_bytes;
        ahead = ahead + row_bytes == D * row_bytes ? 0 : ahead + row_bytes;
    }
    ptx::cp_async_wait<0>();
    if (!a.partial) return;
    float *out = a.partial + blockIdx.x * int64_t(a.c);
    if constexpr (L == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (lane + k * lanes < slices) {
                const float v[8] = {dw[k][0].x, dw[k][0].y, dw[k][1].x, dw[k][1].y,
                                    dw[k][2].x, dw[k][2].y, dw[k][3].x, dw[k][3].y};
                rows::st(out + (lane + k * lanes) * 8, v);
            }
    } else {
        float *s_dw = reinterpret_cast<float *>(s_ring);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (lane + k * lanes < slices) {
                float4 *d = reinterpret_cast<float4 *>(s_dw + group * a.c + (lane + k * lanes) * 8);
                d[0] = make_float4(dw[k][0].x, dw[k][0].y, dw[k][1].x, dw[k][1].y);
                d[1] = make_float4(dw[k][2].x, dw[k][2].y, dw[k][3].x, dw[k][3].y);
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
// few: fewer rows than SMs, where a row's latency counts (4 x 4096: 3.5 us with one slice per
// lane, 5.0 with two).
template <typename F>
static lat_status by_layout(int c, bool few, F &&f) {
    const int slices = c / 8;
    auto threads = [&](int k) { return (slices + 32 * k - 1) / (32 * k) * 32; };
    using std::integral_constant;
    if (slices <= 4) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{}, kThreads);
    if (slices <= 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{}, kThreads);
    if (slices <= 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{}, kThreads);
    if (slices <= 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{}, kThreads);
    if (slices <= 64) return f(integral_constant<int, 32>{}, integral_constant<int, 2>{}, kThreads);
    if (slices <= 128 || (few && slices <= kWideThreads))
        return f(integral_constant<int, 0>{}, integral_constant<int, 1>{}, threads(1));
    if (slices <= 1024) return f(integral_constant<int, 0>{}, integral_constant<int, 2>{}, threads(2));
    return f(integral_constant<int, 0>{}, integral_constant<int, 4>{}, threads(4));
}

// Rows a block takes at a time.
static int rows_per_block(int c) {
    const int slices = c / 8;
    int l = 4;
    while (l < 32 && l < slices) l *= 2;
    return slices <= 64 ? kThreads / l : 1;
}

// Blocks of the backward pass, constants, so that the sums of dw depend on n and c alone: four on each of a B200's 148
// SMs up to 256 channels and from 520 to 1,024, two up to 512, one above 8,192, which fit at once.  From 1,032 to 8,192
// channels three, which fit up to 5,120 channels of 16 bits and 3,584 of fp32 (fewer with dh); wider rows take one and a
// half to three waves.  With two instead (84 MB each of dy, h and dx, us): fp16 1,536 channels 109 -> 149, 2,048
// 90 -> 122, 4,096 64 -> 78, 5,120 57 -> 74, but 8,192 67 -> 55; fp32 1,536 87 -> 89, but 2,048 89 -> 83, 4,096
// 77 -> 66, 5,120 78 -> 67, 8,192 71 -> 69.
static int64_t shares(int64_t n, int c) {
    const int64_t per = rows_per_block(c), most = c <= 256 ? 592 : c <= 512 ? 296 : c <= 1024 ? 592 : c <= 8192 ? 444 : 148;
    return std::max<int64_t>(1, std::min<int64_t>(most, (n + per - 1) / per));
}

template <typename T>
lat_status fwd(const void *x, const void *res, const void *w, int64_t n, int c, float eps, void *h, void *y, void *y8,
               void *y8s, void *h8, void *h8s, float *rstd, cudaStream_t s) {
    Fwd<T> a{static_cast<const T *>(x), static_cast<const T *>(res), static_cast<const T *>(w), static_cast<T *>(h),
             static_cast<T *>(y), static_cast<uint8_t *>(y8), static_cast<uint8_t *>(y8s), static_cast<uint8_t *>(h8),
             static_cast<uint8_t *>(h8s), rstd, n, c, eps};
    const int64_t per = rows_per_block(c);
    return by_layout(c, n < num_sms(), [&](auto l, auto k, int threads) -> lat_status {
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
    const lat_status st = by_layout(c, false, [&](auto l, auto k, int threads) -> lat_status {
        constexpr int L = decltype(l)::value, K = decltype(k)::value;
        auto go = [&](auto q8) -> lat_status {
            constexpr bool Q8 = decltype(q8)::value;
            auto kern = norm_bwd_kernel<T, L, K, Q8>;
            LAT_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              int(bwd_smem_limit<T, L, K, Q8>())));
            LAT_CUDA_TRY(launch_pdl(kern, dim3(unsigned(blocks)), dim3(threads),
                                    bwd_smem<T, L, K, Q8>(dh != nullptr, threads, c), s, a));
            return LAT_OK;
        };
        return h8 ? go(std::true_type{}) : go(std::false_type{});
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
