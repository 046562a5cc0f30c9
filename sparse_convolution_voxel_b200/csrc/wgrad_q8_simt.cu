// Per-offset weight gradient from 8-bit input rows on CUDA cores, for fp32 and the channel
// counts that wgrad_q8.cu's tensor-core tiles do not take: dW[k] = sum over pairs (i, j) of
// offset k of x[i]^T dy[j], all products and sums in fp32 (FFMA, no TF32).
//
// The pair list is cut into shares of at least kSharePairs pairs, at most as many as the
// shape's grid has; their number depends on the pair count and the shape alone.  A block takes
// a share and a 64 x 64 piece of dW[k] (input channels x output channels).  For every 64 pairs
// of a segment (the share's pairs of one offset) it widens the piece's x and dy into shared
// memory, and each thread adds 4 x 4 products of the pairs of its group: a piece of fewer than
// 256 such tiles leaves threads for several groups, which take the pairs in turn and are added
// in group order at the segment's end.  One fp32 partial per segment; wgrad_q8.cu's reduction
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

__host__ __device__ inline int pieces(int c) { return (c + kPiece - 1) / kPiece; }
// Shares at most: about four blocks per B200 SM.
inline int most_shares(int cin, int cout) { return std::max(148, 592 / (pieces(cin) * pieces(cout))); }

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
    __shared__ int s_in[kBatch], s_out[kBatch];
    __shared__ __align__(16) float s_x[kBatch * kPiece], s_dy[kBatch * kPiece];
    const int tid = threadIdx.x;
    if (tid <= k3) s_off[tid] = min(pair_off[tid], capacity);
    __syncthreads();
    const int64_t P = s_off[k3];
    const int S = share_count(P, most), v = blockIdx.x;
    if (v == 0 && blockIdx.y == 0 && tid < k3) {
        // for the reduction, the partials (slot share + offset) of the shares meeting offset tid's pairs [a, b): share v has the pairs
        // from P v / S, so pair p is in share floor((S (p + 1) - 1) / P)
        const int64_t a = s_off[tid], b = s_off[tid + 1];
        ranges[2 * tid] = a < b ? int((S * (a + 1) - 1) / P) + tid : 0;
        ranges[2 * tid + 1] = a < b ? int((S * b - 1) / P) + tid : -1;
    }
    if (v >= S) return;
    const int ci0 = int(blockIdx.y) / pieces(cout) * kPiece, co0 = int(blockIdx.y) % pieces(cout) * kPiece;
    const int M = min(kPiece, cin - ci0), N = min(kPiece, cout - co0);
    const int tiles = (M / 4) * (N / 4);
    int lanes = 4;  // threads of a group
    while (lanes < tiles) lanes *= 2;
    const int groups = kThreads / lanes, group = tid / lanes, tile = tid % lanes;
    const bool has_tile = tile < tiles;
    const int ti = has_tile ? tile / (N / 4) * 4 : 0, tj = has_tile ? tile % (N / 4) * 4 : 0;
    const int xg = M / 8, yg = N / 8;  // 8-channel slices of a row
    int64_t lo = P * v / S;
    const int64_t hi = P * (v + 1) / S;
    int k = 0;
    while (k < k3 && s_off[k + 1] <= lo) ++k;
    int32_t bad = 0;
    while (lo < hi) {
        const int64_t end = min(hi, s_off[k + 1]);
        float acc[4][4] = {};
        for (int64_t p0 = lo; p0 < end; p0 += kBatch) {
            const int count = int(min(int64_t(kBatch), end - p0));
            if (tid < kBatch) {
                int i = -1, j = -1;
                if (tid < count) {
                    i = __ldg(pair_in + p0 + tid);
                    j = __ldg(pair_out + p0 + tid);
                    if (i < 0 || i >= n_in || j < 0 || j >= n_out) {
                        bad |= LAT_ERR_BAD_MAP;
                        i = j = -1;
                    }
                }
                s_in[tid] = i;
                s_out[tid] = j;
            }
            __syncthreads();
            for (int o = tid; o < count * xg; o += kThreads) {
                const int p = o / xg, c = (o % xg) * 8, i = s_in[p];
                float f[8] = {};
                if (i >= 0) {
                    uint2 bits;
                    int e;
                    rows::q8_load(q, scale, i, cin, (ci0 + c) / 8, bits, e);
                    rows::q8_to_f(bits, e, f);
                }
                float4 *d = reinterpret_cast<float4 *>(s_x + p * M + c);
                d[0] = make_float4(f[0], f[1], f[2], f[3]);
                d[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
            for (int o = tid; o < count * yg; o += kThreads) {
                const int p = o / yg, c = (o % yg) * 8, j = s_out[p];
                float f[8];
                rows::to_f(j >= 0 ? rows::ld(dy + int64_t(j) * cout + co0 + c) : rows::zero_slice<T>(), f);
                float4 *d = reinterpret_cast<float4 *>(s_dy + p * N + c);
                d[0] = make_float4(f[0], f[1], f[2], f[3]);
                d[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
            __syncthreads();
            if (has_tile) {
#pragma unroll 4
                for (int p = group; p < count; p += groups) {
                    const float4 x = *reinterpret_cast<const float4 *>(s_x + p * M + ti);
                    const float4 y = *reinterpret_cast<const float4 *>(s_dy + p * N + tj);
                    const float xv[4] = {x.x, x.y, x.z, x.w}, yv[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int a = 0; a < 4; ++a)
#pragma unroll
                        for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(xv[a], yv[b], acc[a][b]);
                }
            }
            __syncthreads();
        }
        // the groups' sums meet in shared memory: [group][M][N], in the rows' place
        float *sums = groups > 1 ? s_x : nullptr;  // groups * M * N <= kThreads * 16 floats
        float *out = partial + int64_t(v + k) * cin * cout + int64_t(ci0) * cout + co0;
        if (has_tile) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                float4 *d = reinterpret_cast<float4 *>(sums ? sums + (group * M + ti + a) * N + tj
                                                            : out + int64_t(ti + a) * cout + tj);
                *d = make_float4(acc[a][0], acc[a][1], acc[a][2], acc[a][3]);
            }
        }
        if (sums) {
            __syncthreads();
            for (int e = tid; e < M * N; e += kThreads) {
                float t = 0.f;
#pragma unroll 8
                for (int g = 0; g < groups; ++g) t += sums[g * M * N + e];
                out[int64_t(e / N) * cout + e % N] = t;
            }
            __syncthreads();
        }
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
