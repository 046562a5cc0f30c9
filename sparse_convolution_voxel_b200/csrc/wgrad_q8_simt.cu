// Per-offset weight gradient from 8-bit input rows on CUDA cores, for fp32 and the channel
// counts that wgrad_q8.cu's tensor-core tiles do not take: dW[k] = sum over pairs (i, j) of
// offset k of x[i]^T dy[j], all products and sums in fp32 (FFMA, no TF32).  In fp16, x is rounded
// to fp16 as on the tensor cores, so that the channel counts do not change what is multiplied.
//
// The pair list is cut into shares of at least kSharePairs pairs, at most as many as the
// shape's grid has; their number depends on the pair count and the shape alone.  A block takes
// a share and a 64 x 64 piece of dW[k] (input channels x output channels).  For every 64 pairs
// of a segment (the share's pairs of one offset) it widens the piece's x and dy into shared
// memory, and each thread adds 8 x 4 products of the pairs of its group: a piece has at most 128
// such tiles, so that the block has two groups and more, which take the pairs in turn and are
// added in group order at the segment's end.  One fp32 partial per segment; wgrad_q8.cu's reduction
// adds the partials in share order.
//
// A small map is bound by the chain of dependent reads (offsets, pairs, rows): few long
// shares, one block each, where the kernels for rows of 16 and 32 bits walk four short ones
// (2,000 voxels, 16 -> 16, the whole call: 14 us; unpacking the rows and running those
// kernels took 27).
#include <algorithm>

#include "conv_common.cuh"
#include "rows.cuh"

namespace lat {
namespace wq8s {

constexpr int kThreads = 256;
constexpr int kBatch = 64;       // pairs in shared memory
constexpr int kPiece = 64;       // channels of a piece, each way
constexpr int kSharePairs = 32;  // at least
constexpr int kTileM = 8;        // a thread's products: 8 input channels x 4 output channels

__host__ __device__ inline int pieces(int c) { return (c + kPiece - 1) / kPiece; }
// Shares at most: the two blocks that each of a B200's 148 SMs holds (60,000 voxels, 305,000 pairs, 64 -> 64 fp32:
// 91 us, with twice as many 96, with half 114 and more).
inline int most_shares(int cin, int cout) { return std::max(148, 296 / (pieces(cin) * pieces(cout))); }

__device__ __forceinline__ int share_count(int64_t P, int most) {
    return int(max(int64_t(P > 0), min(int64_t(most), P / kSharePairs)));
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
wgrad_q8_simt_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale, int cin,
                     const T *__restrict__ dy, int cout, const int64_t *__restrict__ pair_off,
                     const int32_t *__restrict__ pair_in, const int32_t *__restrict__ pair_out, int64_t capacity, int k3,
                     int64_t n_in, int64_t n_out, int most, float *__restrict__ partial, int32_t *__restrict__ ranges,
                     int32_t *d_status) {
    pdl_enter();
    __shared__ int64_t s_off[33];
    __shared__ int s_in[2][kBatch], s_out[2][kBatch];
    __shared__ __align__(16) float s_x[2 * kBatch * kPiece];  // x, then dy
    float *s_dy = s_x + kBatch * kPiece;
    const int tid = threadIdx.x;
    if (tid <= k3) s_off[tid] = min(pair_off[tid], capacity);
    __syncthreads();
    const int64_t P = s_off[k3];
    const int S = share_count(P, most), v = blockIdx.x;
    if (v == 0 && blockIdx.y == 0 && tid < k3) {
        // for the reduction, the partials (slot share + offset) of the shares meeting offset tid's pairs [a, b):
        // share v has the pairs from P v / S, so pair p is in share floor((S (p + 1) - 1) / P)
        const int64_t a = max(int64_t(0), s_off[tid]), b = min(s_off[tid + 1], P);
        ranges[2 * tid] = a < b ? int((S * (a + 1) - 1) / P) + tid : 0;
        ranges[2 * tid + 1] = a < b ? int((S * b - 1) / P) + tid : -1;
    }
    if (v >= S) return;
    const int ci0 = int(blockIdx.y) / pieces(cout) * kPiece, co0 = int(blockIdx.y) % pieces(cout) * kPiece;
    const int M = min(kPiece, cin - ci0), N = min(kPiece, cout - co0);
    const int tiles = (M / kTileM) * (N / 4);
    int lanes = 2;  // threads of a group
    while (lanes < tiles) lanes *= 2;
    static_assert(2 * (kPiece / kTileM) * (kPiece / 4) <= kThreads, "two groups at least");
    const int groups = kThreads / lanes, group = tid / lanes, tile = tid % lanes;
    const bool has_tile = tile < tiles;
    const int ti = has_tile ? tile / (N / 4) * kTileM : 0, tj = has_tile ? tile % (N / 4) * 4 : 0;
    const int xg = M / 8, yg = N / 8;  // 8-channel slices of a row
    int64_t lo = P * v / S;
    const int64_t hi = P * (v + 1) / S;
    int k = 0;
    while (k < k3 && s_off[k + 1] <= lo) ++k;
    int32_t bad = 0;
    // A batch's slices on their way: thread t has the slices t and t + kThreads of x and of dy.
    constexpr int kMine = kBatch * kPiece / 8 / kThreads;
    uint2 xq[kMine];
    int xe[kMine];
    rows::Slice8<T> yv[kMine];
    auto pairs = [&](int64_t p0, int64_t end, int to) {  // the batch's rows, -1 for none
        if (tid >= kBatch) return;
        int i = -1, j = -1;
        if (p0 + tid < end) {
            i = __ldg(pair_in + p0 + tid);
            j = __ldg(pair_out + p0 + tid);
            if (i < 0 || i >= n_in || j < 0 || j >= n_out) {
                bad |= LAT_ERR_BAD_MAP;
                i = j = -1;
            }
        }
        s_in[to][tid] = i;
        s_out[to][tid] = j;
    };
    auto read = [&](int from) {
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int o = tid + m * kThreads, px = o / xg, py = o / yg;
            const int i = px < kBatch ? s_in[from][px] : -1, j = py < kBatch ? s_out[from][py] : -1;
            xq[m] = make_uint2(0u, 0u);
            xe[m] = 1;
            if (i >= 0) rows::q8_load(q, scale, i, cin, ci0 / 8 + o % xg, xq[m], xe[m]);
            yv[m] = j >= 0 ? rows::ld(dy + int64_t(j) * cout + co0 + o % yg * 8) : rows::zero_slice<T>();
        }
    };
    auto widen = [&]() {
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int o = tid + m * kThreads;
            float f[8];
            if (o < kBatch * xg) {
                rows::q8_to_f(xq[m], xe[m], f);
                rows::as_held<T>(f, xe[m]);
                float4 *d = reinterpret_cast<float4 *>(s_x + o * 8);
                d[0] = make_float4(f[0], f[1], f[2], f[3]);
                d[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
            if (o < kBatch * yg) {
                rows::to_f(yv[m], f);
                float4 *d = reinterpret_cast<float4 *>(s_dy + o * 8);
                d[0] = make_float4(f[0], f[1], f[2], f[3]);
                d[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
        }
    };
    while (lo < hi) {
        const int64_t end = min(hi, s_off[k + 1]);
        float2 acc[kTileM / 2][4] = {};  // two input channels each: one instruction multiplies and adds both
        int from = 0;
        pairs(lo, end, 0);
        pairs(lo + kBatch, end, 1);
        __syncthreads();
        read(0);
        for (int64_t p0 = lo; p0 < end; p0 += kBatch, from ^= 1) {
            const int count = int(min(int64_t(kBatch), end - p0));
            widen();
            __syncthreads();
            // the next batch's rows and the pairs of the one after it, while this one is added
            if (p0 + kBatch < end) {
                read(from ^ 1);
                pairs(p0 + 2 * kBatch, end, from);
            }
            if (has_tile) {
#pragma unroll 4
                for (int p = group; p < count; p += groups) {
                    const float4 x0 = *reinterpret_cast<const float4 *>(s_x + p * M + ti);
                    const float4 x1 = *reinterpret_cast<const float4 *>(s_x + p * M + ti + 4);
                    const float4 y = *reinterpret_cast<const float4 *>(s_dy + p * N + tj);
                    const float2 xv[kTileM / 2] = {make_float2(x0.x, x0.y), make_float2(x0.z, x0.w),
                                                   make_float2(x1.x, x1.y), make_float2(x1.z, x1.w)};
                    const float2 yy[4] = {rows::both(y.x), rows::both(y.y), rows::both(y.z), rows::both(y.w)};
#pragma unroll
                    for (int a = 0; a < kTileM / 2; ++a)
#pragma unroll
                        for (int b = 0; b < 4; ++b) acc[a][b] = rows::fma2(xv[a], yy[b], acc[a][b]);
                }
            }
            __syncthreads();
        }
        // the groups' sums meet in shared memory, in the rows' place: [group][M][N], at most kThreads * 32 floats
        if (has_tile) {
#pragma unroll
            for (int a = 0; a < kTileM; ++a) {
                float4 *d = reinterpret_cast<float4 *>(s_x + (group * M + ti + a) * N + tj);
                const float2 *r = acc[a / 2];
                *d = a & 1 ? make_float4(r[0].y, r[1].y, r[2].y, r[3].y) : make_float4(r[0].x, r[1].x, r[2].x, r[3].x);
            }
        }
        __syncthreads();
        float *out = partial + int64_t(v + k) * cin * cout + (ci0 * cout + co0);
        for (int e = tid; e < M * N; e += kThreads) {
            float t = 0.f;
#pragma unroll 4
            for (int g = 0; g < groups; ++g) t += s_x[g * M * N + e];
            out[e / N * cout + e % N] = t;
        }
        __syncthreads();
        lo = end;
        ++k;
        while (k < k3 && s_off[k + 1] <= lo) ++k;
    }
    if (bad) flag(d_status, bad);
}

}  // namespace wq8s

size_t wgrad_q8_simt_ws_bytes(int cin, int cout, const lat_kmap *map) {
    Carver cv(nullptr);
    cv.take<float>(size_t(wq8s::most_shares(cin, cout) + map->k3) * cin * cout);
    cv.take<int32_t>(64);
    return align_up(cv.used, 256);
}

template <typename T>
lat_status launch_wgrad_q8_simt(const void *q, const void *scale, int cin, const void *dy, int cout,
                                const lat_kmap *map, float *dw, void *ws, int32_t *d_status, cudaStream_t s) {
    const int most = wq8s::most_shares(cin, cout);
    Carver cv(ws);
    float *partial = cv.take<float>(size_t(most + map->k3) * cin * cout);
    int32_t *ranges = cv.take<int32_t>(64);
    LAT_CUDA_TRY(launch_pdl(wq8s::wgrad_q8_simt_kernel<T>,
                            dim3(unsigned(most), unsigned(wq8s::pieces(cin) * wq8s::pieces(cout))), dim3(wq8s::kThreads),
                            0, s, static_cast<const uint8_t *>(q), static_cast<const uint8_t *>(scale), cin,
                            static_cast<const T *>(dy), cout, map->pair_off, map->pair_in, map->pair_out,
                            map->pair_capacity, map->k3, map->n_in, map->n_out, most, partial, ranges, d_status));
    return launch_wgrad_q8_reduce(partial, ranges, cin * cout, map->k3, dw, s);
}

template lat_status launch_wgrad_q8_simt<float>(const void *, const void *, int, const void *, int, const lat_kmap *,
                                                float *, void *, int32_t *, cudaStream_t);
template lat_status launch_wgrad_q8_simt<__half>(const void *, const void *, int, const void *, int, const lat_kmap *,
                                                 float *, void *, int32_t *, cudaStream_t);
template lat_status launch_wgrad_q8_simt<__nv_bfloat16>(const void *, const void *, int, const void *, int,
                                                        const lat_kmap *, float *, void *, int32_t *, cudaStream_t);

}  // namespace lat
