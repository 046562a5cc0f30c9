// tcgen05 per-offset weight gradient from 8-bit input rows: dW[k] = sum over pairs (i, j)
// of offset k of x[i]^T dy[j], x in e4m3 with a power-of-two scale per 32 channels, dy in
// fp16 / bf16, fp32 accumulate in TMEM, fp32 out.
//
// The GEMM and its tiles are those of wgrad_tc.cu; the cut of the pair list is its own (kWorkers,
// Work).  What differs most is the way of x: tcgen05 multiplies 8-bit rows only with
// 8-bit rows, so the rows are fetched in 8 bits (half the bytes of the pair's x, which
// is what the kernel waits for) and widened on the way into the MMA's tile.  A value has
// 4 significant bits and a power of two: bf16 holds it exactly.  fp16 rounds values below
// 2^-14 to its subnormals' steps and is held at 65504, as lat_q8_unpack writes it.
//
// One CTA per SM, every role of its own:
//   * two groups of eight warps widen the blocks of 64 pairs in turn, each with two A tiles
//     and a ring of kRing blocks (raw x rows, scale bytes, dy tile) of its own: wait for the
//     block's copies, widen x into an A tile, arrive at the tile's barrier.  (One group took
//     95 us at 500k rows, 128 -> 128: a chain of latencies in two warps per scheduler.)
//   * four warps per group gather the blocks' rows with cp.async, dy straight into its
//     swizzled tile.
//   * one thread fetches the blocks that are a run: three quarters of a scan's pairs are
//     (j, j), the centre of a submanifold map, in row order, so that 64 pairs are 64
//     consecutive rows: bulk copies of x and the scales, a tensor copy per 64 channels of dy.
//   * a thread per group issues its MMAs, into an accumulator of its own; their commits free
//     the A tile and the ring slot.  (It takes some 1,000 cycles a block: with one thread for
//     both, that bounded maps whose rows lie in L2.)  Four warps store each segment's sum.
// With the gathers in the widening warps, which then wait for one another's latencies, and
// in shares of one piece, it took 76 us; now 64 back to back on the same rows, of which the kernel's
// some 55 move 240 MB.
//
// The tensor cores cut bits off when they add: over thousands of pairs in one accumulator
// that would be the largest error of the result (1.0e-6 of the norm at the size above, 5.5e-7
// for fp32 matrix products).  So an accumulator takes a segment's next kFlush blocks at most,
// and the epilogue adds it in fp32 to a total, in TMEM too, which is stored when the sum ends.
#include <algorithm>

#include "conv_common.cuh"
#include "rows.cuh"
#include "tc_ptx.cuh"
#include "wgrad_tc.cuh"

namespace lat {
namespace wq8 {

constexpr int kKP = 64;        // pairs per block (GEMM K block)
// The pair list is cut into equal contiguous shares of at least a block, at most kTurns for
// each of kWorkers workers (one per B200 SM); worker w takes the shares w, w + kWorkers, ....
// So the gathers, which a scan's map has at both ends of its list, are spread over all
// workers: in one share each, the CTAs with gathers alone took 77 us and the others 53.
constexpr int kWorkers = 148, kTurns = 4;
constexpr int kGroups = 2, kGroupWarps = 8;
constexpr int kWideWarps = kGroups * kGroupWarps, kEpiWarps = 4, kGatherWarps = 4;  // gathering: per group
constexpr int kGroupThreads = kGroupWarps * 32, kGatherThreads = kGatherWarps * 32;
constexpr int kTiles = 2;     // A tiles of a group
constexpr int kMaxRing = 8;
constexpr int kFlush = 32;    // blocks of a group per accumulator
constexpr int kLook = 3;      // blocks of a group whose pairs are read ahead
constexpr int kScaleBytes = kKP * 4 + 32;  // of a ring slot: a word per pair, or a run's bytes from a 16-byte boundary
constexpr int kGatherAt = kWideWarps + kEpiWarps;  // first gathering warp
constexpr int kMmaWarp = kGatherAt + kGroups * kGatherWarps, kLoadWarp = kMmaWarp + kGroups;
constexpr int kThreads = (kLoadWarp + 1) * 32;
constexpr int kWidePairs = kKP / kGroupWarps, kGatherPairs = kKP / kGatherWarps;  // of a block, per warp
constexpr uint32_t kMaxSmem = 232448, kBarBytes = 512, kAlign = 1024;  // of a CTA; its barriers; the tiles' alignment
constexpr uint64_t kDrainNs = 1000000000ull;  // limit of the waits that drain a CTA that gave up

// A worker's pairs of one offset in one of its shares, in the order in which it takes them.
// Segments of one offset that follow one another are one sum: one partial.
struct Segment {
    int64_t lo, hi;  // pairs
    int k, slot;     // offset, partial
    bool begins, ends;  // the sum
};
constexpr int kMaxSegments = kTurns + 32;  // every segment ends a share or an offset

// The worker's segments, made by one warp: lane k looks at offset k.
struct Work {
    int64_t off[33];  // offset k has pairs [off[k], off[k + 1])
    int64_t cut[kTurns][2];
    int count;
    Segment seg[kMaxSegments];
    __device__ void make(const int64_t *pair_off, int64_t capacity, int k3, int worker, int32_t *ranges) {
        const int lane = threadIdx.x & 31;
        // whatever the offsets hold, they rise from 0 here to at most the capacity, which bounds the segments and slots
        auto read = [&](int e) { return e <= k3 ? max(int64_t(0), min(pair_off[e], capacity)) : int64_t(0); };
        int64_t upper = read(lane);
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) upper = max(upper, int64_t(__shfl_up_sync(0xFFFFFFFFu, (long long)upper, m)));
        off[lane] = upper;
        if (lane == 31) off[32] = max(upper, read(32));
        __syncwarp();
        const int64_t P = off[k3];
        const int S = int(max(int64_t(P > 0), min(int64_t(kWorkers * kTurns), P / kKP)));
        if (lane < 2 * kTurns) {  // share v has pairs [P v / S, P (v + 1) / S)
            const int v = worker + lane / 2 * kWorkers;
            cut[lane / 2][lane & 1] = v < S ? P * (v + (lane & 1)) / S : 0;
        }
        // the shares and the workers that meet this lane's offset: pair p is in share floor((S (p + 1) - 1) / P)
        const int64_t a = lane < k3 ? off[lane] : 0, b = lane < k3 ? off[lane + 1] : 0;
        int parts = 0, first = 0;
        if (a < b) {
            const int v0 = int((S * (a + 1) - 1) / P), v1 = int((S * b - 1) / P);
            parts = min(v1 - v0 + 1, kWorkers);
            first = parts < kWorkers ? v0 % kWorkers : 0;
        }
        int upto = parts;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, upto, m);
            if (lane >= m) upto += u;
        }
        if (ranges && lane < k3) {
            ranges[2 * lane] = upto - parts;
            ranges[2 * lane + 1] = upto - 1;
        }
        const int slot = upto - parts + (worker - first + kWorkers) % kWorkers;
        __syncwarp();
        int n = 0;
        for (int t = 0; t < kTurns; ++t) {
            const int64_t lo = max(a, cut[t][0]), hi = min(b, cut[t][1]);
            const uint32_t some = __ballot_sync(0xFFFFFFFFu, lo < hi);
            if (lo < hi) seg[n + __popc(some & ((1u << lane) - 1u))] = Segment{lo, hi, lane, slot, true, true};
            n += __popc(some);
        }
        __syncwarp();
        for (int i = lane; i < n; i += 32) {
            seg[i].begins = i == 0 || seg[i - 1].k != seg[i].k;
            seg[i].ends = i == n - 1 || seg[i + 1].k != seg[i].k;
        }
        if (lane == 0) count = n;
    }
};

// A CTA's static shared memory.
struct Static {
    Work work;
    uint8_t odd[kGroups * kMaxRing][kKP];  // M = 64: the pair's scale bytes are the upper half of their word
    int last[kGroups * kMaxRing];          // parity of the slot's phase if its last block is a run, else -1
    int run[kGroups * kMaxRing];           // the block is a run: where its scale bytes begin, else -1
    int abort;
};

template <int M, int N>
struct Cfg {
    static constexpr uint32_t kABytes = uint32_t(M) * 128;  // 64 pairs x M channels x 2 bytes
    static constexpr uint32_t kBBytes = uint32_t(N) * 128;
    static constexpr uint32_t kXBytes = uint32_t(M) * 64;   // raw
    // Blocks in a group's ring: what shared memory admits.  (A block takes some 3,000 cycles from its gather to its
    // MMAs' end: where the rows lie in L2, the ring's length bounds the rate.)
    static constexpr uint32_t kSlot = kBBytes + kXBytes + kScaleBytes;
    static constexpr uint32_t kRoom = kMaxSmem - uint32_t(sizeof(Static)) - kBarBytes - kAlign - kGroups * kTiles * kABytes;
    static constexpr int kRing = kRoom / (kGroups * kSlot) < kMaxRing ? kRoom / (kGroups * kSlot) : kMaxRing;
    static_assert(kRing > kTiles, "a group's ring is longer than its A tiles are many");
    static constexpr uint32_t kDyAt = kGroups * kTiles * kABytes;        // the A tiles, then the dy tiles, raw x, scales
    static constexpr uint32_t kRawAt = kDyAt + kGroups * kRing * kBBytes;
    static constexpr uint32_t kScaleAt = kRawAt + kGroups * kRing * kXBytes;
    static constexpr uint32_t kBars = kScaleAt + kGroups * kRing * kScaleBytes;
    static constexpr uint32_t kSmem = kBars + kBarBytes + kAlign;
    static_assert(kSmem + sizeof(Static) <= kMaxSmem, "a CTA's shared memory");
    static_assert(8 * (kGroups * (kTiles + 2 + 2 * kRing) + 1) + 4 <= kBarBytes, "the barriers and the TMEM address");
    static constexpr uint32_t kTmemCols = 4 * N;  // the groups' accumulators and the total; a power of two
    static constexpr int kChunks = M / 64;  // 16-byte raw chunks per thread and block
    // arrivals that a slot's copies take: the load thread, the gathering threads' copies and, where they store st.odd,
    // their warps
    static constexpr uint32_t kLandings = 1 + kGatherThreads + (M == 64 ? kGatherWarps : 0);
};
template <typename T, int M, int N> struct KernelTag {};  // one launch-config cache per kernel

// Walks the blocks of the segments.  A block is a run if its pairs are 64 consecutive rows
// whose scale bytes (G per row) can be copied from a 16-byte boundary: the full blocks of the
// centre, but for the last rows' bytes.
template <int G>
struct Blocks {
    const Work &work;
    int64_t p0 = 0, hi = 0, run_end = 0, row0 = 0;  // pairs [p0, min(p0 + kKP, hi)); row0: p0's row in the centre
    int64_t rows;
    int s = 0, centre;
    bool run = false;
    __device__ Blocks(const Work &w, int centre_, int64_t rows_) : work(w), rows(rows_), centre(centre_) {}
    __device__ __forceinline__ bool next() {
        p0 += kKP;
        row0 += kKP;
        if (p0 >= hi) {
            if (s == work.count) return false;
            const Segment &g = work.seg[s++];
            p0 = g.lo;
            hi = g.hi;
            run_end = -1;
            if (g.k == centre) {
                row0 = p0 - work.off[g.k];
                // full blocks, inside the rows, and floor16(row G) + 64 G + 16 <= rows G
                run_end = min(hi - kKP, work.off[g.k] + min(rows - kKP, rows - kKP - (16 + G - 1) / G));
            }
        }
        run = p0 <= run_end;
        return true;
    }
};

// 16 values of a group with scale byte e, widened: lo and hi are their halves.
template <typename T>
__device__ __forceinline__ void widen(const uint4 &q, int e, uint4 &lo, uint4 &hi) {
    if constexpr (std::is_same<T, __half>::value) {
        // scales of 2^-14 .. 2^7 are fp16 numbers and 448 of them an fp16 value: one product, rounded once
        if (uint32_t(e - 113) < 22u) {
            const __half2 s = __half2half2(__ushort_as_half(uint16_t((e - 112) << 10)));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const __half2_raw r =
                    __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
                const __half2 v = __hmul2(__half2(r), s);
                o[i] = *reinterpret_cast<const uint32_t *>(&v);
            }
            lo = make_uint4(o[0], o[1], o[2], o[3]);
            hi = make_uint4(o[4], o[5], o[6], o[7]);
            return;
        }
    }
    auto half = [&](uint2 w) {
        float v[8];
        rows::q8_to_f(w, e, v);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = rows::in_range<T>(v[c]);
        return make_uint4(rows::two<T>(v[0], v[1]), rows::two<T>(v[2], v[3]), rows::two<T>(v[4], v[5]),
                          rows::two<T>(v[6], v[7]));
    };
    lo = half(make_uint2(q.x, q.y));
    hi = half(make_uint2(q.z, q.w));
}

template <typename T, int M, int N>
__global__ void __launch_bounds__(kThreads, 1)
wgrad_q8_kernel(const __grid_constant__ CUtensorMap dy_map, int centre, const uint8_t *__restrict__ q,
                const uint8_t *__restrict__ scale, const T *__restrict__ dy,
                const int64_t *__restrict__ pair_off, const int32_t *__restrict__ pair_in,
                const int32_t *__restrict__ pair_out, int64_t capacity, int k3, int64_t n_in, int64_t n_out,
                float *__restrict__ partial, int32_t *__restrict__ ranges, uint64_t wait_ns, int32_t *d_status) {
    pdl_enter();
    using C = Cfg<M, N>;
    constexpr int kRing = C::kRing;
    constexpr uint32_t idesc = wtc::make_idesc<T, M, N>();

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBars);
    uint64_t *freed = full + kGroups * kTiles;  // the MMAs of the slot's block are done: slot and A tile are free
    uint64_t *accfull = freed + kGroups * kRing;
    uint64_t *accempty = accfull + kGroups;
    uint64_t *landed = accempty + kGroups;  // bulk and tensor copies, [group][slot]
    uint64_t *drain = landed + kGroups * kRing;  // tracks the MMAs still in flight when a CTA gives up
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    __shared__ Static st;
    Work &s_work = st.work;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == 1) s_work.make(pair_off, capacity, k3, int(blockIdx.x), blockIdx.x == 0 ? ranges : nullptr);
    if (tid == 0) {
        for (int s = 0; s < kGroups * kTiles; ++s) ptx::mbar_init(&full[s], kGroupThreads);
        for (int s = 0; s < kGroups; ++s) {
            ptx::mbar_init(&accfull[s], 1);
            ptx::mbar_init(&accempty[s], kEpiWarps * 32);
        }
        for (int s = 0; s < kGroups * kRing; ++s) {
            ptx::mbar_init(&landed[s], C::kLandings);
            ptx::mbar_init(&freed[s], 1);
            st.last[s] = -1;
        }
        ptx::mbar_init(drain, kGroups);
        st.abort = 0;
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

    if (warp < kWideWarps) {
        // ------------------------------------------------------------ widen x
        constexpr int XL = M / 16, XP = 32 / XL;  // lanes per raw x row, rows per warp and chunk
        const int grp = warp / kGroupWarps, gw = warp % kGroupWarps, xc = lane % XL, xg = lane / XL;
        // 16-byte chunks 2 xc and 2 xc + 1 of a pair's row; the upper half of the lanes stores them the other way
        // round, so that eight lanes meet eight different banks
        const int mb = xc >> 2, cc = (2 * xc) & 7;
        const bool turn = mb & 1;
        const int first = cc + (turn ? 1 : 0), second = cc + (turn ? 0 : 1);
        uint32_t blocks = 0;  // of this group
        for (int i = 0; i < s_work.count; ++i)
            blocks += uint32_t((s_work.seg[i].hi - s_work.seg[i].lo + kKP - 1) / kKP);
        blocks = (blocks + kGroups - 1 - grp) / kGroups;
        uint32_t slot = 0, phase = 0;  // the block's ring slot, and the slot's phase
        bool ok = true;
#pragma unroll 1
        for (uint32_t it = 0; it < blocks; ++it) {
            const uint32_t r = grp * kRing + slot, t = grp * kTiles + it % kTiles;
            // this block's copies, and the MMAs that read the A tile last, of the block kTiles before
            const uint32_t was = slot >= kTiles ? slot - kTiles : slot + kRing - kTiles;
            const uint32_t was_phase = slot >= kTiles ? phase : phase ^ 1;
            if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&landed[r], phase, wait_ns) &&
                                             (it < kTiles || ptx::mbar_wait(&freed[grp * kRing + was], was_phase, wait_ns)))) {
                ok = false;
                break;
            }
            const uint8_t *xs = smem + C::kRawAt + r * C::kXBytes + (gw * kWidePairs + xg) * M + xc * 16;
            const uint8_t *ss = smem + C::kScaleAt + r * kScaleBytes;
            const int from = st.run[r];
            uint8_t *row = smem + t * C::kABytes + mb * 8192 + gw * 1024;  // kWidePairs == 8: one 8-pair atom per warp
#pragma unroll
            for (int i = 0; i < C::kChunks; ++i) {
                const int sw = i * XP + xg, p = gw * kWidePairs + sw;
                const uint4 raw = *reinterpret_cast<const uint4 *>(xs + i * XP * M);
                // channels 16 xc .. 16 xc + 15
                const int e = ss[(from >= 0 ? from + p * (M / 32) : p * 4 + (M == 64 ? st.odd[r][p] : 0)) + (xc >> 1)];
                uint4 lo, hi;
                widen<T>(raw, e, lo, hi);
                *reinterpret_cast<uint4 *>(row + sw * 128 + ((first ^ sw) << 4)) = turn ? hi : lo;
                *reinterpret_cast<uint4 *>(row + sw * 128 + ((second ^ sw) << 4)) = turn ? lo : hi;
            }
            // the tile, written through the generic proxy, before the tensor cores' reads
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&full[t]);
            if (++slot == kRing) {
                slot = 0;
                phase ^= 1;
            }
        }
        if (!ok) st.abort = 1;
    } else if (warp < kGatherAt) {
        // ------------------------------------------------------------ epilogue: partial of each segment
        const int quad = warp & 3;
        // M = 128: lane l of quadrant w holds row 32w + l; M = 64: lanes 0..15 hold rows 16w + l
        const int row = M == 128 ? quad * 32 + lane : quad * 16 + lane;
        const bool has_row = M == 128 || lane < 16;
        uint32_t phase[kGroups] = {}, it = 0;  // it: the segment's first block
        bool ok = true;
        for (int i = 0; ok && i < s_work.count; ++i) {
            const Segment sg = s_work.seg[i];
            float *dst = partial + int64_t(sg.slot) * M * N + int64_t(row) * N;
            const int blocks = int((sg.hi - sg.lo + kKP - 1) / kKP);
            for (int b0 = 0; b0 < blocks; b0 += kGroups * kFlush) {
                const int n = min(kGroups * kFlush, blocks - b0);
                const bool begins = sg.begins && b0 == 0, ends = sg.ends && b0 + n == blocks;
                // one block alone: the other group has none
                const bool has[kGroups] = {n > 1 || ((it + b0) & 1) == 0, n > 1 || ((it + b0) & 1) == 1};
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    if (!has[g]) continue;
                    ok = ok && __all_sync(0xFFFFFFFFu, ptx::mbar_wait(&accfull[g], phase[g], wait_ns));
                    phase[g] ^= 1;
                }
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t at = tmem_base + (uint32_t(quad * 32) << 16);
#pragma unroll
                for (int c0 = 0; c0 < N; c0 += 16) {
                    uint32_t v[16];
                    float sum[16] = {};
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        if (!has[g]) continue;
                        ptx::tmem_ld16(at + g * N + c0, v);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) sum[e] += __uint_as_float(v[e]);
                    }
                    if (!begins) {
                        ptx::tmem_ld16(at + kGroups * N + c0, v);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) sum[e] = __uint_as_float(v[e]) + sum[e];
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(sum[e]);
                    if (!ends) {
                        ptx::tmem_st16(at + kGroups * N + c0, v);
                    } else if (has_row) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t *w = v + 8 * e;
                            const uint32_t o[8] = {w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]};
                            ptx::st_global_v8(dst + c0 + 8 * e, o);
                        }
                    }
                }
                if (!ends) ptx::tmem_wait_st();
                ptx::tc_fence_before();
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
                    if (has[g]) ptx::mbar_arrive(&accempty[g]);
            }
            it += blocks;
        }
        if (!ok) st.abort = 1;
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ gather rows
        constexpr int XL = M / 16, XP = 32 / XL;
        const int grp = (warp - kGatherAt) / kGatherWarps, gw = (warp - kGatherAt) % kGatherWarps;
        const int xc = lane % XL, xg = lane / XL, g = lane >> 3, c = lane & 7;
        Blocks<M / 32> blk(s_work, centre, n_in);
        // lanes 0..15: the indices of this warp's pairs of the group's next kLook blocks (a run needs none), so that
        // their own latency, as long as a block's work, is not met once per block
        int si[kLook], sj[kLook];
        bool have[kLook], run[kLook];
        bool more = true;
        auto fetch = [&](int u, int skip) {
            si[u] = sj[u] = -1;
            for (int i = 0; i < skip; ++i) more = more && blk.next();
            have[u] = more;
            run[u] = blk.run;
            if (!more || run[u]) return;
            const int64_t mp = blk.p0 + gw * kGatherPairs + lane;
            if (lane < kGatherPairs && mp < blk.hi) {
                si[u] = __ldg(pair_in + mp);
                sj[u] = __ldg(pair_out + mp);
            }
        };
#pragma unroll
        for (int u = 0; u < kLook; ++u) fetch(u, u == 0 ? 1 + grp : kGroups);
        bool ok = true;
        uint32_t slot = 0, phase = 1;  // the wait for the slot's previous block; the first ones pass
        const uint8_t *q_lane = q + xc * 16;
        const T *dy_lane = dy + c * 8;
        auto gather = [&](int u) -> bool {
            const uint32_t r = grp * kRing + slot;
            if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&freed[r], phase, wait_ns))) return false;
            if (!run[u]) {
                int ri = si[u], rj = sj[u];
                if (ri >= n_in || rj >= n_out || (ri < 0) != (rj < 0)) {
                    bad |= LAT_ERR_BAD_MAP;
                    ri = rj = -1;
                }
                uint8_t *xs = smem + C::kRawAt + r * C::kXBytes + (gw * kGatherPairs + xg) * M + xc * 16;
                uint8_t *Bs = smem + C::kDyAt + r * C::kBBytes + gw * (kGatherPairs * 128);
                if (lane < kGatherPairs) {
                    const int p = gw * kGatherPairs + lane;
                    const int64_t at = ri < 0 ? 0 : int64_t(ri) * (M / 32), word = at & ~int64_t(3);
                    const int64_t left = n_in * (M / 32) - word;
                    ptx::cp_async4(smem + C::kScaleAt + r * kScaleBytes + p * 4, scale + word,
                                   ri < 0 ? 0u : uint32_t(left < 4 ? left : 4));
                    if (M == 64) st.odd[r][p] = uint8_t(at & 2);
                }
#pragma unroll
                for (int i = 0; i < kGatherPairs / XP; ++i) {
                    const int ii = __shfl_sync(0xFFFFFFFFu, ri, i * XP + xg);
                    ptx::cp_async16(xs + i * XP * M, q_lane + uint64_t(uint32_t(max(ii, 0))) * M, ii >= 0 ? 16u : 0u);
                }
#pragma unroll
                for (int i = 0; i < kGatherPairs / 4; ++i) {
                    const int pl = 4 * i + g;  // gw * 16 is a multiple of 8: the pair's place in its 8-pair atom is pl & 7
                    const int jj = __shfl_sync(0xFFFFFFFFu, rj, pl);
                    const uint32_t off = (pl >> 3) * 1024 + (pl & 7) * 128 + ((c ^ (pl & 7)) << 4);
                    const T *src = dy_lane + uint64_t(uint32_t(max(jj, 0))) * N;
#pragma unroll
                    for (int nb = 0; nb < N / 64; ++nb)
                        ptx::cp_async16(Bs + nb * 8192 + off, src + nb * 64, jj >= 0 ? 16u : 0u);
                }
            }
            ptx::cp_async_arrive_noinc(&landed[r]);  // when this thread's copies are there
            if (M == 64) {
                // that arrival stands for the copies alone: the warp's stores to st.odd are released by one of their own
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&landed[r]);
            }
            if (++slot == kRing) {
                slot = 0;
                phase ^= 1;
            }
            return true;
        };
#pragma unroll 1
        while (ok && have[0]) {
#pragma unroll
            for (int u = 0; u < kLook; ++u) {
                if (!have[u]) break;
                ok = gather(u);
                if (!ok) break;
                fetch(u, kGroups);
            }
        }
        ptx::cp_async_wait<0>();
        if (!ok) st.abort = 1;
    } else if (warp < kLoadWarp) {
        // ------------------------------------------------------------ MMA issue, a thread per group
        if (lane == 0) {
            const uint32_t grp = warp - kMmaWarp;
            const uint64_t a_desc = ptx::desc_sw128(ptx::smem_u32(smem + grp * kTiles * C::kABytes), 8192, 1024);
            const uint64_t b_desc = ptx::desc_sw128(ptx::smem_u32(smem + C::kDyAt + grp * kRing * C::kBBytes), 8192, 1024);
            uint32_t tile = 0, slot = 0, tile_phase = 0;  // of the block; phase of its tile's barrier
            uint32_t acc_phase = 1, it = 0;               // the first wait passes; it: the segment's first block
            const uint32_t dcol = tmem_base + grp * N;
            bool ok = true;
            for (int i = 0; ok && i < s_work.count; ++i) {
                const int blocks = int((s_work.seg[i].hi - s_work.seg[i].lo + kKP - 1) / kKP);
                // this group's blocks of the segment
                int left = (blocks + int((it + grp + 1) & 1)) / 2;
                it += blocks;
                while (ok && left > 0) {
                    if (!ptx::mbar_wait(&accempty[grp], acc_phase, wait_ns)) {
                        ok = false;
                        break;
                    }
                    acc_phase ^= 1;
                    ptx::tc_fence_after();
                    const int n = min(left, kFlush);
                    left -= n;
                    for (int b = 0; b < n; ++b) {
                        // the widened tile; its threads have seen the dy tile land
                        if (!ptx::mbar_wait(&full[grp * kTiles + tile], tile_phase, wait_ns)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        // the gathered dy rows were written by cp.async (generic proxy)
                        ptx::fence_proxy_async_smem();
                        const uint64_t ad = a_desc + tile * (C::kABytes >> 4), bd = b_desc + slot * (C::kBBytes >> 4);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            ptx::umma_f16(dcol, ad + ks * 128, bd + ks * 128, idesc, b > 0 || ks > 0);
                        ptx::umma_commit(&freed[grp * kRing + slot]);
                        slot = slot + 1 == kRing ? 0 : slot + 1;
                        tile ^= 1;
                        tile_phase ^= tile == 0;
                    }
                    if (ok) ptx::umma_commit(&accfull[grp]);
                }
            }
            if (!ok) st.abort = 1;
        }
    } else if (warp == kLoadWarp && lane == 0) {
        // ------------------------------------------------------------ runs of rows
        Blocks<M / 32> blk(s_work, centre, n_in);
        bool ok = true;
        uint32_t grp = 0, slot = 0, phase = 1;
        while (blk.next()) {
            const uint32_t r = grp * kRing + slot;
            // every block's slot is waited for, also a gathered one's: a wait knows a phase only by its
            // parity, so the one before it must have been seen
            if (!ptx::mbar_wait(&freed[r], phase, wait_ns)) {
                ok = false;
                break;
            }
            if (blk.run) {
                const int64_t row0 = blk.row0, at = row0 * (M / 32);
                constexpr uint32_t kBytes = kKP * (M / 32) + 16;
                st.run[r] = int(at & 15);
                st.last[r] = int(phase ^ 1);
                ptx::mbar_arrive_expect_tx(&landed[r], C::kXBytes + C::kBBytes + kBytes);
                ptx::bulk_load(smem + C::kRawAt + r * C::kXBytes, q + row0 * M, C::kXBytes, &landed[r]);
                ptx::bulk_load(smem + C::kScaleAt + r * kScaleBytes, scale + (at & ~int64_t(15)), kBytes, &landed[r]);
#pragma unroll
                for (int nb = 0; nb < N / 64; ++nb)
                    ptx::tma_load_2d(smem + C::kDyAt + r * C::kBBytes + nb * 8192, &dy_map, &landed[r], nb * 64,
                                     int(row0));
            } else {
                st.run[r] = -1;
                st.last[r] = -1;
                ptx::mbar_arrive(&landed[r]);
            }
            if (++grp == kGroups) {
                grp = 0;
                if (++slot == kRing) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) st.abort = 1;
    }

    __syncthreads();
    if (st.abort) {
        // A role gave up.  Before the CTA releases its TMEM and shared memory, everything still
        // writing into them must land: the gathers have (cp.async.wait_all above); the load
        // thread waits for the run that a slot was given last, and the MMA threads commit every MMA they
        // issued to `drain` and wait for it.  These waits have their own limit.
        bad |= (tid == 0) ? LAT_ERR_TIMEOUT : 0;
        if (warp == kLoadWarp && lane == 0)
            for (int r = 0; r < kGroups * kRing; ++r)  // (a phase whose gather warps gave up stays open: one limit for all)
                if (st.last[r] >= 0 && !ptx::mbar_wait(&landed[r], st.last[r], kDrainNs)) break;
        if (warp >= kMmaWarp && warp < kLoadWarp && lane == 0) {
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

// dW[k] = sum of offset k's partials, slots ranges[2 k] .. ranges[2 k + 1].  A block takes 64
// float4 columns of dW[k], two per thread; row r of kRedRows adds the slots first + r,
// first + r + kRedRows, ... in order, then the rows' sums are added in order.  Offsets
// without pairs get 0.
constexpr int kRedRows = 16;
__global__ void __launch_bounds__(32 * kRedRows)
wgrad_q8_reduce_kernel(const float *__restrict__ partial, const int32_t *__restrict__ ranges, int nelem,
                       float *__restrict__ dw) {
    pdl_enter();
    __shared__ float4 s[kRedRows][2][32];
    const int k = blockIdx.y;
    const int v0 = __ldg(ranges + 2 * k), v1 = __ldg(ranges + 2 * k + 1);
    const int el = (blockIdx.x * 64 + threadIdx.x) * 4;
    const bool in[2] = {el < nelem, el + 128 < nelem};
    float4 acc[2] = {};
    auto add = [](float4 &a, const float4 &x) {
        a.x += x.x;
        a.y += x.y;
        a.z += x.z;
        a.w += x.w;
    };
#pragma unroll 5
    for (int v = v0 + int(threadIdx.y); v <= v1; v += kRedRows) {
        const float *src = partial + int64_t(v) * nelem + el;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (in[h]) add(acc[h], __ldg(reinterpret_cast<const float4 *>(src + 128 * h)));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) s[threadIdx.y][h][threadIdx.x] = acc[h];
    __syncthreads();
    if (threadIdx.y < 2) {
        const int h = threadIdx.y;
        float4 t = s[0][h][threadIdx.x];
#pragma unroll
        for (int r = 1; r < kRedRows; ++r) add(t, s[r][h][threadIdx.x]);
        if (in[h]) *reinterpret_cast<float4 *>(dw + int64_t(k) * nelem + el + 128 * h) = t;
    }
}

template <typename T, int M, int N>
static lat_status launch(const uint8_t *q, const uint8_t *scale, const void *dy, const lat_kmap *map, float *dw,
                         void *ws, int32_t *d_status, cudaStream_t s) {
    using C = Cfg<M, N>;
    constexpr bool is_bf16 = wtc::is_bf16<T>();
    Carver cv(ws);
    float *partial = cv.take<float>(size_t(kWorkers * kTurns + map->k3) * M * N);
    int32_t *ranges = cv.take<int32_t>(64);
    auto kern = wgrad_q8_kernel<T, M, N>;
    if (GridCache<KernelTag<T, M, N>>::get(kern, C::kSmem, int(C::kTmemCols), 1) <= 0) return LAT_ERR_CUDA;
    // in a submanifold map pair m of the centre offset is (m, m)
    CUtensorMap dy_map = {};
    int centre = map->mode == LAT_SUBM && map->n_in == map->n_out && map->n_out >= kKP &&
                         reinterpret_cast<uintptr_t>(scale) % 16 == 0
                     ? map->k3 / 2
                     : -1;
    if (centre >= 0 && !tensor_map_2d(&dy_map, dy, is_bf16, map->n_out, N, 64, kKP)) return LAT_ERR_CUDA;
    LAT_CUDA_TRY(launch_pdl(kern, dim3(kWorkers), dim3(kThreads), C::kSmem, s, dy_map, centre, q, scale,
                            static_cast<const T *>(dy), map->pair_off, map->pair_in, map->pair_out, map->pair_capacity,
                            map->k3, map->n_in, map->n_out, partial, ranges, wait_limit_ns(), d_status));
    return launch_wgrad_q8_reduce(partial, ranges, M * N, map->k3, dw, s);
}

}  // namespace wq8

// dw[k] from the partials of nelem floats (a multiple of 4); ranges[2 k], ranges[2 k + 1]: its first
// and last one (first > last: none).
lat_status launch_wgrad_q8_reduce(const float *partial, const int32_t *ranges, int nelem, int k3, float *dw,
                                  cudaStream_t s) {
    LAT_CUDA_TRY(launch_pdl(wq8::wgrad_q8_reduce_kernel, dim3(unsigned((nelem + 255) / 256), unsigned(k3)),
                            dim3(32, wq8::kRedRows), 0, s, partial, ranges, nelem, dw));
    return LAT_OK;
}

size_t wgrad_q8_tc_ws_bytes(int cin, int cout, const lat_kmap *map) {
    Carver cv(nullptr);
    cv.take<float>(size_t(wq8::kWorkers * wq8::kTurns + map->k3) * cin * cout);
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
