// tcgen05 per-offset weight gradient from 8-bit input rows: dW[k] = sum over pairs (i, j)
// of offset k of x[i]^T dy[j], x in e4m3 with a power-of-two scale per 32 channels, dy in
// fp16 / bf16, fp32 accumulate in TMEM, fp32 out.
//
// The GEMM, its tiles, the shares of the pair list and the partials are those of
// wgrad_tc.cu.  What differs is the way of x: tcgen05 multiplies 8-bit rows only with
// 8-bit rows, so the rows are fetched in 8 bits (half the bytes of the pair's x, which
// is what the kernel waits for) and widened on the way into the MMA's tile.  A value has
// 4 significant bits and a power of two: bf16 holds it exactly.  fp16 rounds values below
// 2^-14 to its subnormals' steps and is held at 65504.
//
// One CTA per SM.  Two groups of eight warps take the blocks of 64 pairs in turn, each with
// an A tile, a ring of kDy dy tiles and a ring of kRaw raw x blocks of its own.  A group
// copies raw x chunks, scale bytes and dy rows (dy straight into its swizzled tile) with
// cp.async three of its blocks ahead; each thread widens the chunks that it copied itself
// -- only its own cp.async groups to wait for, no barrier -- into the A tile and arrives at
// the tile's barrier, on which the MMA warp waits.  The commit of a block's MMAs frees the
// A tile and the dy tile.  (One group of eight warps with two A tiles took 95 us at 500k
// rows, 128 -> 128: a chain of latencies in two warps per scheduler.)
//
// A segment's sum leaves TMEM every kFlush blocks: the tensor cores cut bits off when they
// add, and over a share of thousands of pairs in one accumulator that would be the largest
// error of the result.  Four warps add it in fp32 to the segment's partial, which the same
// thread wrote.
#include <algorithm>

#include "conv_common.cuh"
#include "rows.cuh"
#include "tc_ptx.cuh"
#include "wgrad_tc.cuh"

namespace lat {
namespace wq8 {

constexpr int kKP = 64;        // pairs per block (GEMM K block)
constexpr int kWorkers = 148;  // shares of the pair list: one per B200 SM
constexpr int kGroups = 2, kGroupWarps = 8;
constexpr int kProdWarps = kGroups * kGroupWarps, kEpiWarps = 4;
constexpr int kGroupThreads = kGroupWarps * 32;
constexpr int kAhead = 3;                   // blocks that a group copies ahead
constexpr int kDy = kAhead + 1, kRaw = kAhead;  // slots of its rings
constexpr int kMmaWarp = kProdWarps + kEpiWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kPairs = kKP / kGroupWarps;  // pairs of a block that one warp copies
constexpr int kFlush = 32;                // blocks per TMEM sum
constexpr uint64_t kDrainNs = 1000000000ull;  // limit of the waits that drain a CTA that gave up

template <int M, int N>
struct Cfg {
    static constexpr uint32_t kABytes = uint32_t(M) * 128;  // 64 pairs x M channels x 2 bytes
    static constexpr uint32_t kBBytes = uint32_t(N) * 128;
    static constexpr uint32_t kXBytes = uint32_t(M) * 64;   // raw
    static constexpr uint32_t kDyAt = kGroups * kABytes;        // the A tiles, then the dy tiles, raw x, scales
    static constexpr uint32_t kRawAt = kDyAt + kGroups * kDy * kBBytes;
    static constexpr uint32_t kScaleAt = kRawAt + kGroups * kRaw * kXBytes;  // 4 bytes per pair
    static constexpr uint32_t kBars = kScaleAt + kGroups * kRaw * kKP * 4;
    static constexpr uint32_t kSmem = kBars + 256 + 1024;
    static constexpr uint32_t kTmemCols = 2 * N;
    static constexpr int kChunks = M / 64;  // 16-byte raw chunks per thread and block
};
template <typename T, int M, int N> struct KernelTag {};  // one launch-config cache per kernel

// Walks the blocks of this CTA's segments.
struct Blocks {
    wtc::Segments<kWorkers> seg;
    int64_t p0 = 0, hi = 0;
    __device__ Blocks(const int64_t *off, int k3) : seg(off, k3) {}
    __device__ bool next() {  // pairs [p0, min(p0 + kKP, hi))
        p0 += kKP;
        if (p0 < hi) return true;
        int k, slot;
        return seg.next(k, p0, hi, slot);
    }
};

template <typename T>
__device__ __forceinline__ uint4 widen(uint2 q, int e) {
    float v[8];
    rows::q8_to_f(q, e, v);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = rows::in_range<T>(v[c]);
    return make_uint4(rows::two<T>(v[0], v[1]), rows::two<T>(v[2], v[3]), rows::two<T>(v[4], v[5]),
                      rows::two<T>(v[6], v[7]));
}

template <typename T, int M, int N>
__global__ void __launch_bounds__(kThreads, 1)
wgrad_q8_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale, const T *__restrict__ dy,
                const int64_t *__restrict__ pair_off, const int32_t *__restrict__ pair_in,
                const int32_t *__restrict__ pair_out, int64_t capacity, int k3, int64_t n_in, int64_t n_out,
                float *__restrict__ partial, int32_t *__restrict__ ranges, uint64_t wait_ns, int32_t *d_status) {
    pdl_enter();
    using C = Cfg<M, N>;
    constexpr uint32_t idesc = wtc::make_idesc<T, M, N>();

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBars);
    uint64_t *empty = full + kGroups;
    uint64_t *accfull = empty + kGroups;
    uint64_t *accempty = accfull + 2;
    uint64_t *drain = accempty + 2;  // tracks the MMAs still in flight when a CTA gives up
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    __shared__ int s_abort;
    __shared__ int64_t s_off[33];
    __shared__ uint8_t s_odd[kGroups * kRaw][kKP];  // M = 64: the pair's scale bytes are the upper half of their word

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == 1) {
        wtc::load_offsets(pair_off, capacity, k3, s_off);
        __syncwarp();
        if (blockIdx.x == 0 && lane < k3) {
            // for the reduce: the shares meeting offset lane's pairs [a, b)
            const int64_t P = s_off[k3], a = s_off[lane], b = s_off[lane + 1];
            ranges[2 * lane] = a < b ? wtc::share_of<kWorkers>(P, a) : 0;
            ranges[2 * lane + 1] = a < b ? wtc::share_of<kWorkers>(P, b - 1) : -1;
        }
    }
    if (tid == 0) {
        for (int s = 0; s < kGroups; ++s) {
            ptx::mbar_init(&full[s], kGroupThreads);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(&accfull[s], 1);
            ptx::mbar_init(&accempty[s], kEpiWarps * 32);
        }
        ptx::mbar_init(drain, 1);
        s_abort = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 0) {
        ptx::tmem_alloc(tmem_slot, C::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    int32_t bad = 0;

    if (warp < kProdWarps) {
        // ------------------------------------------------------------ copy ahead, widen x
        constexpr int XL = M / 16;       // lanes per raw x row
        constexpr int XP = 32 / XL;      // rows per warp and chunk
        const int grp = warp / kGroupWarps, gw = warp % kGroupWarps, gt = tid % kGroupThreads;
        const int xc = lane % XL, xg = lane / XL;
        const int g = lane >> 3, c = lane & 7;
        Blocks blk(s_off, k3);
        bool have = blk.next();
        for (int i = 0; i < grp; ++i) have = have && blk.next();
        int si = -1, sj = -1;
        auto fetch = [&]() {  // lanes 0..7: the indices of this warp's pairs of the group's next block
            const int64_t mp = blk.p0 + gw * kPairs + lane;
            si = sj = -1;
            if (have && lane < kPairs && mp < blk.hi) {
                si = __ldg(pair_in + mp);
                sj = __ldg(pair_out + mp);
            }
        };
        fetch();
        uint32_t issued = 0;
        auto issue = [&]() {  // copies of the group's next block, one cp.async group (empty past the last block)
            if (have) {
                if (si >= n_in || sj >= n_out || (si < 0) != (sj < 0)) {
                    bad |= LAT_ERR_BAD_MAP;
                    si = sj = -1;
                }
                const uint32_t r = grp * kRaw + issued % kRaw;
                uint8_t *xs = smem + C::kRawAt + r * C::kXBytes;
                uint8_t *Bs = smem + C::kDyAt + (grp * kDy + issued % kDy) * C::kBBytes;
                if (lane < kPairs) {
                    const int p = gw * kPairs + lane;
                    const int64_t at = si < 0 ? 0 : int64_t(si) * (M / 32), word = at & ~int64_t(3);
                    const int64_t left = n_in * (M / 32) - word;
                    ptx::cp_async4(smem + C::kScaleAt + (r * kKP + p) * 4, scale + word,
                                   si < 0 ? 0u : uint32_t(left < 4 ? left : 4));
                    if (M == 64) s_odd[r][p] = uint8_t(at & 2);
                }
#pragma unroll
                for (int i = 0; i < C::kChunks; ++i) {
                    const int ii = __shfl_sync(0xFFFFFFFFu, si, i * XP + xg);
                    const uint8_t *src = ii >= 0 ? q + int64_t(ii) * M + xc * 16 : q;
                    ptx::cp_async16(xs + (i * kGroupThreads + gt) * 16, src, ii >= 0 ? 16u : 0u);
                }
#pragma unroll
                for (int i = 0; i < kPairs / 4; ++i) {
                    const int pl = 4 * i + g, p = gw * kPairs + pl;
                    const int jj = __shfl_sync(0xFFFFFFFFu, sj, pl);
                    const uint32_t off = (p >> 3) * 1024 + (p & 7) * 128 + ((c ^ (p & 7)) << 4);
#pragma unroll
                    for (int nb = 0; nb < N / 64; ++nb) {
                        const T *src = jj >= 0 ? dy + int64_t(jj) * N + nb * 64 + c * 8 : dy;
                        ptx::cp_async16(Bs + nb * 8192 + off, src, jj >= 0 ? 16u : 0u);
                    }
                }
                ++issued;
                for (int i = 0; i < kGroups; ++i) have = have && blk.next();
                fetch();
            }
            ptx::cp_async_commit();
        };
#pragma unroll 1
        for (int d = 0; d < kAhead; ++d) issue();
        uint8_t *As = smem + grp * C::kABytes;
        bool ok = true;
#pragma unroll 1
        for (uint32_t it = 0; it < issued; ++it) {
            // the MMAs of the group's previous block: they read the A tile and the dy tile that issue() refills
            if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&empty[grp], (it & 1) ^ 1, wait_ns))) {
                ok = false;
                break;
            }
            ptx::cp_async_wait<kAhead - 1>();
            __syncwarp();
            const uint32_t r = grp * kRaw + it % kRaw;
            const uint8_t *xs = smem + C::kRawAt + r * C::kXBytes;
            const uint32_t *ss = reinterpret_cast<const uint32_t *>(smem + C::kScaleAt) + r * kKP;
#pragma unroll
            for (int i = 0; i < C::kChunks; ++i) {
                const int p = gw * kPairs + i * XP + xg;
                const uint4 raw = *reinterpret_cast<const uint4 *>(xs + (i * kGroupThreads + gt) * 16);
                const int shift = 8 * (xc >> 1) + (M == 64 ? 8 * s_odd[r][p] : 0);  // channels 16 xc ..
                const int e = (ss[p] >> shift) & 0xFF;
                const uint4 lo = widen<T>(make_uint2(raw.x, raw.y), e), hi = widen<T>(make_uint2(raw.z, raw.w), e);
                // 16-byte chunks 2 xc and 2 xc + 1 of the pair's row; the upper half of the lanes stores them the
                // other way round, so that eight lanes meet eight different banks
                const int mb = xc >> 2, cc = (2 * xc) & 7, sw = p & 7;
                uint8_t *row = As + mb * 8192 + (p >> 3) * 1024 + sw * 128;
                const bool turn = mb & 1;
                *reinterpret_cast<uint4 *>(row + (((cc + (turn ? 1 : 0)) ^ sw) << 4)) = turn ? hi : lo;
                *reinterpret_cast<uint4 *>(row + (((cc + (turn ? 0 : 1)) ^ sw) << 4)) = turn ? lo : hi;
            }
            // the tile and this thread's dy chunks, written through the generic proxy, before the tensor cores' reads
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&full[grp]);
            __syncwarp();  // the raw block and the scales are read: issue() refills them
            issue();
        }
        ptx::cp_async_wait<0>();
        if (!ok) s_abort = 1;
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ epilogue: partial of each segment
        const int quad = warp & 3;
        // M = 128: lane l of quadrant w holds row 32w + l; M = 64: lanes 0..15 hold rows 16w + l
        const int row = M == 128 ? quad * 32 + lane : quad * 16 + lane;
        const bool has_row = M == 128 || lane < 16;
        uint32_t ta = 0;
        bool ok = true;
        wtc::Segments<kWorkers> seg(s_off, k3);
        int k, slot;
        int64_t lo, hi;
        while (ok && seg.next(k, lo, hi, slot)) {
            float *dst = partial + int64_t(slot) * M * N + int64_t(row) * N;
            for (int64_t p = lo; p < hi; p += kFlush * kKP) {
                const uint32_t a = ta & 1;
                if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&accfull[a], (ta >> 1) & 1, wait_ns))) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t taddr = tmem_base + (uint32_t(quad * 32) << 16) + a * N;
#pragma unroll
                for (int c0 = 0; c0 < N; c0 += 16) {
                    uint32_t v[16];
                    ptx::tmem_ld16(taddr + c0, v);
                    ptx::tmem_wait_ld();
                    if (has_row) {
                        float4 *d4 = reinterpret_cast<float4 *>(dst + c0);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float4 o = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                                   __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
                            if (p != lo) {
                                const float4 was = d4[e];
                                o = make_float4(o.x + was.x, o.y + was.y, o.z + was.z, o.w + was.w);
                            }
                            d4[e] = o;
                        }
                    }
                }
                ptx::tc_fence_before();
                ptx::mbar_arrive(&accempty[a]);
                ++ta;
            }
        }
        if (!ok) s_abort = 1;
    } else if (lane == 0) {
        // ------------------------------------------------------------ MMA issue
        uint32_t it = 0, ta = 0;
        bool ok = true;
        wtc::Segments<kWorkers> seg(s_off, k3);
        int k, slot;
        int64_t lo, hi;
        while (ok && seg.next(k, lo, hi, slot)) {
            for (int64_t p = lo; ok && p < hi; p += kFlush * kKP) {
                const uint32_t a = ta & 1;
                if (!ptx::mbar_wait(&accempty[a], ((ta >> 1) & 1) ^ 1, wait_ns)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t dcol = tmem_base + a * N;
                const int64_t end = min(hi, p + kFlush * kKP);
                uint32_t acc = 0;
                for (int64_t p0 = p; p0 < end; p0 += kKP) {
                    const uint32_t grp = it % kGroups, n = it / kGroups;  // block n of its group
                    if (!ptx::mbar_wait(&full[grp], n & 1, wait_ns)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t as = ptx::smem_u32(smem + grp * C::kABytes);
                    const uint32_t bs = ptx::smem_u32(smem + C::kDyAt + (grp * kDy + n % kDy) * C::kBBytes);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t ad = ptx::desc_sw128(as + ks * 2048, 8192, 1024);
                        const uint64_t bd = ptx::desc_sw128(bs + ks * 2048, 8192, 1024);
                        ptx::umma_f16(dcol, ad, bd, idesc, acc);
                        acc = 1;
                    }
                    ptx::umma_commit(&empty[grp]);
                    ++it;
                }
                if (!ok) break;
                ptx::umma_commit(&accfull[a]);
                ++ta;
            }
        }
        if (!ok) s_abort = 1;
    }

    __syncthreads();
    if (s_abort) {
        // A role gave up: the copies are complete (cp.async.wait_all above); the MMA thread
        // commits every MMA it issued to `drain` and waits for it (with its own limit) before
        // the TMEM and shared memory are released.
        bad |= (tid == 0) ? LAT_ERR_TIMEOUT : 0;
        if (warp == kMmaWarp && lane == 0) {
            ptx::umma_commit(drain);
            ptx::mbar_wait(drain, 0, kDrainNs);
        }
        __syncthreads();
    }
    if (bad) flag(d_status, bad);
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_base, C::kTmemCols);
    }
}

// dW[k] = sum of offset k's partials (slots share + k, shares v0..v1 from the main kernel).
// A block takes 32 float4 columns of dW[k]; row r of kRedRows adds the shares v0 + r,
// v0 + r + kRedRows, ... in order, then the rows' sums are added in order.  Offsets
// without pairs get 0.
constexpr int kRedRows = 8;
__global__ void __launch_bounds__(32 * kRedRows)
wgrad_q8_reduce_kernel(const float *__restrict__ partial, const int32_t *__restrict__ ranges, int nelem,
                       float *__restrict__ dw) {
    pdl_enter();
    __shared__ float4 s[kRedRows][32];
    const int k = blockIdx.y;
    const int v0 = __ldg(ranges + 2 * k), v1 = __ldg(ranges + 2 * k + 1);
    const int el = (blockIdx.x * 32 + threadIdx.x) * 4;
    const bool in = el < nelem;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4 &x) {
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
    };
#pragma unroll 8
    for (int v = v0 + int(threadIdx.y); in && v <= v1; v += kRedRows)
        add(__ldg(reinterpret_cast<const float4 *>(partial + int64_t(v + k) * nelem + el)));
    s[threadIdx.y][threadIdx.x] = acc;
    __syncthreads();
    if (threadIdx.y == 0 && in) {
#pragma unroll
        for (int r = 1; r < kRedRows; ++r) add(s[r][threadIdx.x]);
        *reinterpret_cast<float4 *>(dw + int64_t(k) * nelem + el) = acc;
    }
}

template <typename T, int M, int N>
static lat_status launch(const uint8_t *q, const uint8_t *scale, const void *dy, const lat_kmap *map, float *dw,
                         void *ws, int32_t *d_status, cudaStream_t s) {
    using C = Cfg<M, N>;
    Carver cv(ws);
    float *partial = cv.take<float>(size_t(kWorkers + map->k3) * M * N);
    int32_t *ranges = cv.take<int32_t>(64);
    auto kern = wgrad_q8_kernel<T, M, N>;
    const int64_t grid =
        std::min<int64_t>(kWorkers, GridCache<KernelTag<T, M, N>>::get(kern, C::kSmem, int(C::kTmemCols), 1));
    if (grid <= 0) return LAT_ERR_CUDA;
    LAT_CUDA_TRY(launch_pdl(kern, dim3(unsigned(grid)), dim3(kThreads), C::kSmem, s, q, scale,
                            static_cast<const T *>(dy), map->pair_off, map->pair_in, map->pair_out, map->pair_capacity,
                            map->k3, map->n_in, map->n_out, partial, ranges, wait_limit_ns(), d_status));
    return launch_wgrad_q8_reduce(partial, ranges, M * N, map->k3, dw, s);
}

}  // namespace wq8

// dw[k] from the partials of nelem floats (a multiple of 4) at slots share + k; ranges[k]: the
// first and the last share that meets offset k.
lat_status launch_wgrad_q8_reduce(const float *partial, const int32_t *ranges, int nelem, int k3, float *dw,
                                  cudaStream_t s) {
    LAT_CUDA_TRY(launch_pdl(wq8::wgrad_q8_reduce_kernel, dim3(unsigned((nelem + 127) / 128), unsigned(k3)),
                            dim3(32, wq8::kRedRows), 0, s, partial, ranges, nelem, dw));
    return LAT_OK;
}

size_t wgrad_q8_tc_ws_bytes(int cin, int cout, const lat_kmap *map) {
    Carver cv(nullptr);
    cv.take<float>(size_t(wq8::kWorkers + map->k3) * cin * cout);
    cv.take<int32_t>(64);
    return align_up(cv.used, 256);
}

lat_status launch_wgrad_q8_tc(bool bf16, const void *q, const void *scale, int cin, const void *dy, int cout,
                              const lat_kmap *map, float *dw, void *ws, int32_t *d_status, cudaStream_t s) {
    const uint8_t *qb = static_cast<const uint8_t *>(q), *sb = static_cast<const uint8_t *>(scale);
#define LAT_WQ8(T, M, N) \
    if (cin == M && cout == N) return wq8::launch<T, M, N>(qb, sb, dy, map, dw, ws, d_status, s);
    if (bf16) {
        LAT_WQ8(__nv_bfloat16, 64, 64) LAT_WQ8(__nv_bfloat16, 64, 128) LAT_WQ8(__nv_bfloat16, 128, 64)
        LAT_WQ8(__nv_bfloat16, 128, 128)
    } else {
        LAT_WQ8(__half, 64, 64) LAT_WQ8(__half, 64, 128) LAT_WQ8(__half, 128, 64) LAT_WQ8(__half, 128, 128)
    }
#undef LAT_WQ8
    return LAT_ERR_UNSUPPORTED;
}

}  // namespace lat
