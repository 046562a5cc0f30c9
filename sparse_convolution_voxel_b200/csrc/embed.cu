// Embedding lookup with scaling and its gradient by sorted tokens (lat_embed_fwd,
// lat_embed_wgrad).
//
//   y[i] = scale * table[id_i]          dtable[t] = scale * sum over i with id_i = t of dy[i]
//
// Lookup: a gather, bound by the bytes it copies.  L lanes take a row, 8 channels each.
//
// Gradient: the rows are sorted by token (a stable LSD radix sort of (token, row) pairs;
// rows without a token get the key `vocab`, behind every token), so that each token's
// rows are one run of the sorted list.  The table's rows and the sorted rows together are
// one path of vocab + n steps: "add the next row" while its token is the current one,
// else "store the current token's sum and go on to the next token".  The path is cut into
// equal shares (the cut is where sorted token + position passes the share's start, found
// by a search of the group's lanes), each walked by one group of lanes with the sum in
// registers.  So a token with a hundred thousand rows is spread over many shares, and
// tokens without rows, whose gradient is zero, cost the one store that they need.  A
// token whose run crosses a cut leaves one fp32 partial per share (head: the sum up to its
// end in a later share, tail: the sum from its begin), and a second kernel adds them in
// share order.  No atomics: the bits depend neither on timing nor on the GPU.
#include <algorithm>

#include "rows.cuh"

namespace lat {
namespace embed {

using rows::Slice8;

constexpr int kThreads = 256;

// Row i's token, or -1 for none (the padding id, or an id outside [0, vocab), which is flagged).
template <typename I>
__device__ __forceinline__ int64_t token(const I *ids, int64_t i, int64_t vocab, int64_t pad, int32_t &bad) {
    const int64_t t = int64_t(__ldg(ids + i));
    if (t == pad) return -1;
    if (t < 0 || t >= vocab) {
        bad |= LAT_ERR_BAD_ID;
        return -1;
    }
    return t;
}

template <typename T, typename I, int L>
__global__ void __launch_bounds__(kThreads)
lookup_kernel(const I *__restrict__ ids, int64_t n, const T *__restrict__ table, int64_t vocab, int c, float scale,
              int64_t pad, T *__restrict__ y, int32_t *d_status) {
    pdl_enter();
    const int64_t row = blockIdx.x * int64_t(kThreads / L) + threadIdx.x / L;
    if (row >= n) return;
    int32_t bad = 0;
    const int64_t t = token(ids, row, vocab, pad, bad);
    const int slices = c / 8;
    for (int vi = threadIdx.x % L + blockIdx.y * L; vi < slices; vi += L * gridDim.y) {
        float v[8] = {};
        if (t >= 0) rows::to_f(rows::ld(table + t * c + vi * 8), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= scale;
        rows::st(y + row * c + vi * 8, v);
    }
    if (bad && threadIdx.x % L == 0 && blockIdx.y == 0) flag(d_status, bad);
}

// ------------------------------------------------------------------------- the sort
// One stable counting pass by a digit of `bits` bits: counts per (tile, digit value),
// their scan over the tiles, and the scatter.  A tile is a run of rows; in the
// scatter a warp takes an eighth of them, 32 at a time, and ranks the rows of equal digit
// by ballots, so equal keys keep their order.  A tile has kThreads * R rows.
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBits = 10;
constexpr int kMaxBins = 1 << kMaxBits;

struct Pass {
    const uint32_t *key_in, *row_in;  // null: the ids themselves (first pass)
    uint32_t *key_out, *row_out;
    uint32_t *counts;   // [tiles][bins]: rows of the tile with the digit, then (scan) those of earlier tiles
    uint32_t *totals;   // [bins]
    int64_t n;
    int tiles, shift, bits;
};
template <typename I> struct Ids {
    const I *ids;
    int64_t vocab, pad;
};

template <typename I>
__device__ __forceinline__ uint32_t sort_key(const Pass &p, const Ids<I> &d, int64_t i, int32_t &bad) {
    if (p.key_in) return p.key_in[i];
    const int64_t t = token(d.ids, i, d.vocab, d.pad, bad);
    return uint32_t(t < 0 ? d.vocab : t);
}

template <typename I, int R>
__global__ void __launch_bounds__(kThreads) count_kernel(Pass p, Ids<I> d, int32_t *d_status) {
    pdl_enter();
    __shared__ uint32_t s_cnt[kMaxBins];
    const int bins = 1 << p.bits;
    for (int b = threadIdx.x; b < bins; b += kThreads) s_cnt[b] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * int64_t(kThreads * R), hi = min(p.n, lo + kThreads * R);
    int32_t bad = 0;
#pragma unroll R
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads)
        atomicAdd(&s_cnt[(sort_key(p, d, i, bad) >> p.shift) & (bins - 1)], 1u);
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kThreads) p.counts[int64_t(blockIdx.x) * bins + b] = s_cnt[b];
    if (bad) flag(d_status, bad);
}

// 32 digit values per block: lane row t of 32 takes a run of the tiles.
// (Also clears the count of open runs for the sums.)
__global__ void __launch_bounds__(1024) tile_scan_kernel(uint32_t *__restrict__ counts, uint32_t *__restrict__ totals,
                                                         int tiles, int bins, int32_t *__restrict__ open_count) {
    pdl_enter();
    if (blockIdx.x == 0 && threadIdx.x == 0 && threadIdx.y == 0) *open_count = 0;
    __shared__ uint32_t s[32][33];
    const int b = blockIdx.x * 32 + threadIdx.x;
    const int per = (tiles + 31) / 32, lo = min(tiles, int(threadIdx.y) * per), hi = min(tiles, lo + per);
    uint32_t sum = 0;
    if (b < bins) {
#pragma unroll 8
        for (int t = lo; t < hi; ++t) sum += counts[int64_t(t) * bins + b];
    }
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    uint32_t run = 0, all = 0;
#pragma unroll
    for (int t = 0; t < 32; ++t) {
        const uint32_t v = s[t][threadIdx.x];
        if (t < int(threadIdx.y)) run += v;
        all += v;
    }
    if (b >= bins) return;
    if (threadIdx.y == 0) totals[b] = all;
    for (int t = lo; t < hi; ++t) {
        const uint32_t v = counts[int64_t(t) * bins + b];
        counts[int64_t(t) * bins + b] = run;
        run += v;
    }
}

// Inclusive sum over the lanes of a warp.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, m);
        if (lane >= m) v += u;
    }
    return v;
}

// The lanes whose digit (`bits` bits; false `in`: none) equals this lane's, by one ballot per
// bit.  (A warp match takes a turn per distinct value: 44 us instead of 17 for the one-block
// sort of 16,383 rows.)
template <int kMax>
__device__ __forceinline__ uint32_t same_digit(uint32_t digit, int bits, bool in) {
    uint32_t peers = __ballot_sync(0xFFFFFFFFu, in);
#pragma unroll
    for (int b = 0; b < kMax; ++b) {
        if (b >= bits) break;
        const bool one = (digit >> b) & 1u;
        const uint32_t ones = __ballot_sync(0xFFFFFFFFu, one);
        peers &= one ? ones : ~ones;
    }
    return peers;
}

template <typename I, int R>
__global__ void __launch_bounds__(kThreads) scatter_kernel(Pass p, Ids<I> d) {
    pdl_enter();
    static_assert(kMaxBins == 4 * kThreads, "four digits per thread in the scan");
    __shared__ uint4 s_cnt4[kWarps][kMaxBins / 4];
    __shared__ uint32_t s_scan[kWarps];
    uint32_t(*s_cnt)[kMaxBins] = reinterpret_cast<uint32_t(*)[kMaxBins]>(s_cnt4);
    const int bins = 1 << p.bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t lo = (blockIdx.x * int64_t(kWarps) + warp) * (32 * R);
    uint32_t key[R], rank[R], row[R];
    int32_t bad = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t i = lo + r * 32 + lane;
        key[r] = i < p.n ? sort_key(p, d, i, bad) : 0u;
        row[r] = i < p.n ? (p.row_in ? p.row_in[i] : uint32_t(i)) : 0u;
    }
    const bool own = int(threadIdx.x) * 4 < bins;  // this thread's digits 4 t .. 4 t + 3
    uint4 total = make_uint4(0u, 0u, 0u, 0u), start = total;
    if (own) {
        total = reinterpret_cast<const uint4 *>(p.totals)[threadIdx.x];
        start = reinterpret_cast<const uint4 *>(p.counts + int64_t(blockIdx.x) * bins)[threadIdx.x];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s_cnt4[w][threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    }
    // first position of each digit: an exclusive scan of the totals
    const uint32_t sum = total.x + total.y + total.z + total.w;
    const uint32_t upto = warp_scan(sum, lane);
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    uint32_t at = upto - sum;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) at += w < warp ? s_scan[w] : 0u;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = lo + r * 32 + lane < p.n;
        const uint32_t digit = (key[r] >> p.shift) & (bins - 1);
        const uint32_t peers = same_digit<kMaxBits>(digit, p.bits, in);
        const uint32_t before = __popc(peers & ((1u << lane) - 1u));
        if (in) rank[r] = s_cnt[warp][digit] + before;
        __syncwarp();
        if (in && before == 0) s_cnt[warp][digit] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    if (own) {
        uint4 run = make_uint4(at + start.x, at + total.x + start.y, at + total.x + total.y + start.z,
                               at + total.x + total.y + total.z + start.w);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint4 v = s_cnt4[w][threadIdx.x];
            s_cnt4[w][threadIdx.x] = run;
            run = make_uint4(run.x + v.x, run.y + v.y, run.z + v.z, run.w + v.w);
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (lo + r * 32 + lane < p.n) {
            const uint32_t pos = s_cnt[warp][(key[r] >> p.shift) & (bins - 1)] + rank[r];
            p.key_out[pos] = key[r];
            p.row_out[pos] = row[r];
        }
    }
}

// All passes of up to kSmall rows by one block, in shared memory: the same ranks, with the
// counts of (digit value, warp) scanned in that order.  (One SM's issue slots bound it: at
// 16,383 rows it took 38 us, more than the passes above.)
constexpr int kSmall = 4096, kSmallThreads = 1024, kSmallWarps = kSmallThreads / 32;
constexpr int kSmallRounds = kSmall / kSmallThreads, kSmallBits = 8, kSmallBins = 1 << kSmallBits;
constexpr int kCntStride = kSmallWarps + 1;
constexpr size_t kSmallSmem = kSmall * 4 + kSmall * 2 + kSmallBins * kCntStride * 2 + 16;
template <typename I>
__global__ void __launch_bounds__(kSmallThreads)
sort_small_kernel(Ids<I> d, int n, int bits, uint32_t *__restrict__ key_out, uint32_t *__restrict__ row_out,
                  int32_t *__restrict__ open_count, int32_t *d_status) {
    pdl_enter();
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t *s_key = reinterpret_cast<uint32_t *>(smem);
    uint16_t *s_row = reinterpret_cast<uint16_t *>(smem + kSmall * 4);
    uint16_t *s_cnt = s_row + kSmall;
    __shared__ uint32_t s_scan[kSmallWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rounds = (n + kSmallThreads - 1) / kSmallThreads, lo = warp * rounds * 32;
    if (threadIdx.x == 0) *open_count = 0;
    uint32_t key[kSmallRounds], row[kSmallRounds];  // row: and the rank, in the upper half
    int32_t bad = 0;
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r) {
        const int i = lo + r * 32 + lane;
        if (r < rounds && i < n) {
            const int64_t t = token(d.ids, i, d.vocab, d.pad, bad);
            key[r] = uint32_t(t < 0 ? d.vocab : t);
            row[r] = uint32_t(i);
        }
    }
    for (int shift = 0; shift < bits; shift += kSmallBits) {
        for (int b = threadIdx.x; b < kSmallBins * kCntStride / 2; b += kSmallThreads)
            reinterpret_cast<uint32_t *>(s_cnt)[b] = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kSmallRounds; ++r) {
            if (r >= rounds) break;
            const bool in = lo + r * 32 + lane < n;
            const uint32_t digit = in ? (key[r] >> shift) & (kSmallBins - 1) : 0u;
            const uint32_t peers = same_digit<kSmallBits>(digit, kSmallBits, in);
            const uint32_t before = __popc(peers & ((1u << lane) - 1u));
            uint16_t *cnt = s_cnt + digit * kCntStride + warp;
            if (in) row[r] = (row[r] & 0xFFFFu) | ((*cnt + before) << 16);
            __syncwarp();
            if (in && before == 0) *cnt += uint16_t(__popc(peers));
            __syncwarp();
        }
        __syncthreads();
        constexpr int kOwn = kSmallBins * kSmallWarps / kSmallThreads;  // a thread's counts, in (digit, warp) order
        uint16_t *own = s_cnt + threadIdx.x * kOwn / kSmallWarps * kCntStride + threadIdx.x * kOwn % kSmallWarps;
        uint32_t sum = 0, c[kOwn];
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            c[o] = own[o];
            sum += c[o];
        }
        const uint32_t upto = warp_scan(sum, lane);
        if (lane == 31) s_scan[warp] = upto;
        __syncthreads();
        const uint32_t base = lane < warp ? s_scan[lane] : 0u;
        uint32_t at = upto - sum + __reduce_add_sync(0xFFFFFFFFu, base);
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            own[o] = uint16_t(at);
            at += c[o];
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kSmallRounds; ++r) {
            if (r < rounds && lo + r * 32 + lane < n) {
                const uint32_t pos =
                    s_cnt[((key[r] >> shift) & (kSmallBins - 1)) * kCntStride + warp] + (row[r] >> 16);
                s_key[pos] = key[r];
                s_row[pos] = uint16_t(row[r]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kSmallRounds; ++r) {
            const int i = lo + r * 32 + lane;
            if (r < rounds && i < n) {
                key[r] = s_key[i];
                row[r] = s_row[i];
            }
        }
        // the next pass writes s_key again only after its own barriers
    }
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r) {
        const int i = lo + r * 32 + lane;
        if (r < rounds && i < n) {
            key_out[i] = key[r];
            row_out[i] = row[r];
        }
    }
    if (bad) flag(d_status, bad);
}

// ------------------------------------------------------------------------ the sums
struct Path {
    const uint32_t *key, *row;  // sorted
    uint32_t n, vocab;          // steps: n + vocab < 2^32
    uint32_t share;             // steps per share
    int shares;
    int c;
    float scale;
    float *head, *tail;         // [shares][c]
    // shares in which a run begins that goes on behind them, in any order: the share, the token,
    // the sorted rows up to the share's end
    int4 *open;
    int32_t *open_count;
    float *dtable;
};

// One range of a search: the first index in [lo, hi) at which `before` no longer holds (hi if it
// holds everywhere).  W lanes of a group search together: a round splits the range into W + 1
// parts, so 500,000 rows take four dependent reads with 32 lanes.
template <int W>
struct Range {
    uint32_t lo, hi;
    __device__ __forceinline__ uint32_t part(uint32_t k) const {
        return lo + uint32_t(uint64_t(hi - lo) * k / (W + 1));
    }
    // votes of the group's lanes for their probes part(lane + 1): the probes are in order, so the votes are a prefix
    __device__ __forceinline__ void narrow(uint32_t votes) {
        if (lo >= hi) return;
        const int k = __popc(votes);
        const uint32_t nlo = k == 0 ? lo : part(k) + 1, nhi = k == W ? hi : part(k + 1);
        lo = nlo;
        hi = nhi;
    }
};

// Sorted rows among the first a and the first b steps of the path: the first i with
// key[i] + i >= a (b); key[i] + i increases strictly.  The two searches share their rounds.
// mask, first: the group's lanes in its warp.
template <int W>
__device__ __forceinline__ void path_rows(const Path &p, uint32_t a, uint32_t b, int lane, uint32_t mask, int first,
                                          uint32_t &ia, uint32_t &ib) {
    Range<W> ra{a > p.vocab ? a - p.vocab : 0u, min(a, p.n)}, rb{b > p.vocab ? b - p.vocab : 0u, min(b, p.n)};
    auto before = [&](const Range<W> &r, uint32_t step) {
        if (r.lo >= r.hi) return false;
        const uint32_t at = r.part(lane + 1);
        return uint64_t(__ldg(p.key + at)) + at < step;
    };
    while (ra.lo < ra.hi || rb.lo < rb.hi) {
        const bool ba = before(ra, a), bb = before(rb, b);
        ra.narrow((__ballot_sync(mask, ba) & mask) >> first);
        rb.narrow((__ballot_sync(mask, bb) & mask) >> first);
    }
    ia = ra.lo;
    ib = rb.lo;
}

// A group's lanes read the tokens and rows of L steps at a time, one step each, and the next
// ones before they add; kFlight rows of dy are in flight while kFlight are added.  A row of
// more than 256 channels takes several groups (slabs), up to eight of them side by side in a
// block, so that a block reads and writes long pieces.  A block takes `per_block` consecutive
// shares; if a token's run covers them all, their sums meet in shared memory and the first
// share's head stands for the block.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads, 3) sums_kernel(Path p, const T *__restrict__ dy, int per_block) {
    pdl_enter();
    constexpr int kFlight = sizeof(T) == 4 || L == 4 ? 2 : 4;  // an even number of times per batch
    __shared__ float s_acc[8][kThreads];
    const int group = threadIdx.x / L, lane = threadIdx.x % L, first = (threadIdx.x & 31) / L * L;
    const uint32_t mask = (L == 32 ? 0xFFFFFFFFu : ((1u << (L & 31)) - 1u) << first);
    const int slabs = L < 32 ? 1 : int(blockDim.x) / L / per_block;  // of a block
    const int v = blockIdx.x * per_block + group / slabs;
    const uint32_t steps = p.vocab + p.n;
    const uint32_t s0 = uint32_t(min(uint64_t(v) * p.share, uint64_t(steps)));
    const uint32_t s1 = uint32_t(min(uint64_t(s0) + p.share, uint64_t(steps)));
    uint32_t i0, i1;
    path_rows<L>(p, s0, s1, lane, mask, first, i0, i1);
    const uint32_t r0 = s0 - i0, r1 = s1 - i1;
    const int vi = (int(blockIdx.y) * slabs + group % slabs) * L + lane;
    const bool own = vi < p.c / 8;
    const uint32_t col = vi * 8;
    // the first token's run began in an earlier share; the last token's run goes on in the next one
    const bool cut = i0 > 0 && __ldg(p.key + i0 - 1) == r0;
    const bool goes_on = r1 < p.vocab && i1 > 0 && __ldg(p.key + i1 - 1) == r1;
    float acc[8] = {};
    uint32_t r = r0;
    auto store = [&]() {
        if (own) {
            if (cut && r == r0) {
                rows::st(p.head + v * int64_t(p.c) + col, acc);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] *= p.scale;
                rows::st(p.dtable + int64_t(r) * p.c + col, acc);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        ++r;
    };
    auto go_to = [&](uint32_t t) {  // the path's stores up to token t
        if (r >= t) return;
        store();
        if (r >= t) return;
        float *at = p.dtable + int64_t(r) * p.c + col;
        for (; r < t; ++r, at += p.c)
            if (own) rows::st(at, acc);  // tokens without rows: zeros
    };
    // a step past the share's end, and a row without a token, adds nothing
    auto step_key = [&](uint32_t i) { return i < i1 ? __ldg(p.key + i) : p.vocab; };
    auto step_row = [&](uint32_t i) { return i < i1 ? __ldg(p.row + i) : 0u; };
    uint32_t key = step_key(i0 + lane), row = step_row(i0 + lane), next_key = 0, next_row = 0;
    Slice8<T> x[2][kFlight];
    auto load = [&](Slice8<T> (&to)[kFlight], uint32_t keys, uint32_t rows_, int q) {
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const uint32_t t = __shfl_sync(mask, keys, (q + u) % L, L), at = __shfl_sync(mask, rows_, (q + u) % L, L);
            to[u] = own && t < p.vocab ? rows::ld(dy + int64_t(at) * p.c + col) : rows::zero_slice<T>();
        }
    };
    load(x[0], key, row, 0);
    for (uint32_t b = i0; b < i1; b += L) {
        next_key = step_key(b + L + lane);
        next_row = step_row(b + L + lane);
        // steps of this batch that begin a new token (bit: the step)
        const uint32_t before = __shfl_up_sync(mask, key, 1, L);
        const uint32_t begins = (__ballot_sync(mask, (lane == 0 || key != before) && key < p.vocab) & mask) >> first;
#pragma unroll
        for (int q = 0; q < L; q += kFlight) {
            const int now = (q / kFlight) & 1;
            if (b + q >= i1) break;
            if (q + kFlight < L) load(x[now ^ 1], key, row, q + kFlight);
            else load(x[now ^ 1], next_key, next_row, 0);
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if ((begins >> (q + u)) & 1u) go_to(__shfl_sync(mask, key, q + u, L));
                float f[8];
                rows::to_f(x[now][u], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += f[e];
            }
        }
        key = next_key;
        row = next_row;
    }
    go_to(r1);
    const bool through = cut && goes_on && r == r0;  // the share lies inside one token's run
    if (per_block > 1 && __syncthreads_and(through)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s_acc[e][threadIdx.x] = acc[e];
        __syncthreads();
        if (group < slabs && own) {
            for (int g = 1; g < per_block; ++g)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += s_acc[e][g * slabs * L + threadIdx.x];
            rows::st(p.head + v * int64_t(p.c) + col, acc);
        }
    } else if (goes_on && own) {
        rows::st((through ? p.head : p.tail) + v * int64_t(p.c) + col, acc);
        if (!through && vi == 0) p.open[atomicAdd(p.open_count, 1)] = make_int4(v, int(r1), int(i1), 0);
    }
}

// Tokens whose run crosses a cut: for each listed share v the run is tail[v], then the heads
// of the shares up to the one that holds the run's end, where a sums block that lies between
// v's and the last one's has one head for all its shares.  Row t of kJoinRows adds the parts
// t, t + kJoinRows, ... in order, then the rows' sums are added in order.  The list's order
// does not matter: every token is the sum of one entry.
constexpr int kJoinRows = 8, kJoinBlocks = 1184;
__global__ void __launch_bounds__(32 * kJoinRows) join_kernel(Path p, int per_block) {
    pdl_enter();
    __shared__ int s_last;
    __shared__ float4 s[kJoinRows][32];
    const int count = *p.open_count;
    for (int o = blockIdx.x; o < count; o += gridDim.x) {
        const int4 run = p.open[o];
        const int v = run.x;
        const uint32_t token = uint32_t(run.y);
        if (threadIdx.y == 0) {
            // the first sorted row past the run
            Range<32> r{uint32_t(run.z), p.n};
            while (r.lo < r.hi)
                r.narrow(__ballot_sync(0xFFFFFFFFu, __ldg(p.key + r.part(threadIdx.x + 1)) <= token));
            if (threadIdx.x == 0) s_last = int((uint64_t(r.lo) + token) / p.share);  // the share that stores the token
        }
        __syncthreads();
        const int last = s_last;
        // shares v .. end of v's block, whole blocks, then the shares of the last block
        const int block = v / per_block, blocks = max(0, last / per_block - block - 1);
        const int lead = min(last, (block + 1) * per_block - 1) - v + 1;
        const int parts = blocks > 0 ? lead + blocks + last % per_block + 1 : last - v + 1;
        const int col = (blockIdx.y * 32 + threadIdx.x) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float4 &x) {
            acc.x += x.x;
            acc.y += x.y;
            acc.z += x.z;
            acc.w += x.w;
        };
        if (col < p.c) {
#pragma unroll 4
            for (int q = threadIdx.y; q < parts; q += kJoinRows) {
                int64_t at = v + q;
                if (blocks > 0 && q >= lead)
                    at = q < lead + blocks ? (block + 1 + q - lead) * per_block : last - (parts - 1 - q);
                add(*reinterpret_cast<const float4 *>((q == 0 ? p.tail : p.head) + at * p.c + col));
            }
        }
        s[threadIdx.y][threadIdx.x] = acc;
        __syncthreads();
        if (threadIdx.y == 0 && col < p.c) {
#pragma unroll
            for (int q = 1; q < kJoinRows; ++q) add(s[q][threadIdx.x]);
            *reinterpret_cast<float4 *>(p.dtable + int64_t(token) * p.c + col) =
                make_float4(acc.x * p.scale, acc.y * p.scale, acc.z * p.scale, acc.w * p.scale);
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------- host
// Lanes of a group for rows of c channels.
static int lanes_of(int c) {
    int l = 4;
    while (l < 32 && l < c / 8) l *= 2;
    return l;
}
template <typename F>
static lat_status by_lanes(int c, F &&f) {
    switch (lanes_of(c)) {
        case 4: return f(std::integral_constant<int, 4>{});
        case 8: return f(std::integral_constant<int, 8>{});
        case 16: return f(std::integral_constant<int, 16>{});
    }
    return f(std::integral_constant<int, 32>{});
}

// Shares of the path: one wave of groups (the sums' registers admit 24 warps on each of a
// B200's 148 SMs), but at least 16 steps each; the numbers depend on the sizes alone.
static int path_shares(int64_t n, int64_t vocab, int c) {
    const int64_t slabs = (c / 8 + 31) / 32, want = 148 * 24 * (32 / lanes_of(c)) / slabs;
    return int(std::max<int64_t>(1, std::min<int64_t>(want, (n + vocab + 15) / 16)));
}

static int key_bits(int64_t vocab) {
    int b = 1;
    while ((int64_t(1) << b) <= vocab) ++b;  // keys 0 .. vocab
    return b;
}

// Rows per thread of the sort's tiles: small tiles while there are few rows, so that enough
// SMs sort; large ones later, so that the counts stay few.
static int tile_rounds(int64_t n) { return n <= 65536 ? 2 : 4; }
static int64_t tiles_of(int64_t n) {
    const int64_t tile = kThreads * tile_rounds(n);
    return (n + tile - 1) / tile;
}

struct Ws {
    uint32_t *key[2], *row[2], *counts, *totals;
    float *head, *tail;
    int4 *open;
    int32_t *open_count;
    size_t bytes;
    Ws(void *base, int64_t n, int64_t vocab, int c) {
        Carver cv(base);
        for (int i = 0; i < 2; ++i) {
            key[i] = cv.take<uint32_t>(size_t(n));
            row[i] = cv.take<uint32_t>(size_t(n));
        }
        counts = cv.take<uint32_t>(size_t(tiles_of(n)) * kMaxBins);
        totals = cv.take<uint32_t>(kMaxBins);
        const size_t part = size_t(path_shares(n, vocab, c)) * size_t(c);
        head = cv.take<float>(part);
        tail = cv.take<float>(part);
        open = cv.take<int4>(size_t(path_shares(n, vocab, c)));
        open_count = cv.take<int32_t>(1);
        bytes = align_up(cv.used, 256);
    }
};

template <typename T, typename I>
lat_status wgrad(const I *ids, int64_t n, const T *dy, int64_t vocab, int c, float scale, int64_t pad, float *dtable,
                 void *ws, int32_t *d_status, cudaStream_t s) {
    Ws w(ws, n, vocab, c);
    int at = 0;
    if (n > 0 && n <= kSmall) {
        auto kern = sort_small_kernel<I>;
        LAT_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmallSmem)));
        LAT_CUDA_TRY(launch_pdl(kern, dim3(1), dim3(kSmallThreads), kSmallSmem, s, Ids<I>{ids, vocab, pad}, int(n),
                                key_bits(vocab), w.key[0], w.row[0], w.open_count, d_status));
    } else if (n > 0) {
        const int bits = key_bits(vocab), passes = (bits + kMaxBits - 1) / kMaxBits, digit = std::max(2, (bits + passes - 1) / passes);
        const int tiles = int(tiles_of(n)), bins = 1 << digit;
        const bool few = tile_rounds(n) == 2;
        auto count = few ? count_kernel<I, 2> : count_kernel<I, 4>;
        auto scatter = few ? scatter_kernel<I, 2> : scatter_kernel<I, 4>;
        const Ids<I> d{ids, vocab, pad};
        for (int i = 0; i < passes; ++i) {
            const int to = i & 1;
            Pass p{i ? w.key[1 - to] : nullptr, i ? w.row[1 - to] : nullptr, w.key[to], w.row[to], w.counts, w.totals, n,
                   tiles, i * digit, digit};
            LAT_CUDA_TRY(launch_pdl(count, dim3(tiles), dim3(kThreads), 0, s, p, d, i ? nullptr : d_status));
            LAT_CUDA_TRY(launch_pdl(tile_scan_kernel, dim3((bins + 31) / 32), dim3(32, 32), 0, s, w.counts, w.totals,
                                    tiles, bins, w.open_count));
            LAT_CUDA_TRY(launch_pdl(scatter, dim3(tiles), dim3(kThreads), 0, s, p, d));
            at = to;
        }
    }
    Path p{w.key[at], w.row[at], uint32_t(n), uint32_t(vocab), 0, path_shares(n, vocab, c), c, scale, w.head, w.tail,
           w.open, w.open_count, dtable};
    p.share = uint32_t((n + vocab + p.shares - 1) / p.shares);
    const int groups = kThreads / lanes_of(c), slabs = (c / 8 + 31) / 32, side = std::min(slabs, groups);
    const int per_block = groups / side;
    const lat_status st = by_lanes(c, [&](auto l) -> lat_status {
        constexpr int L = decltype(l)::value;
        const dim3 grid(unsigned((p.shares + per_block - 1) / per_block), unsigned((slabs + side - 1) / side));
        LAT_CUDA_TRY(launch_pdl(sums_kernel<T, L>, grid, dim3(unsigned(L * side * per_block)), 0, s, p, dy, per_block));
        return LAT_OK;
    });
    if (st != LAT_OK || n == 0) return st;
    const int cols = (c + 127) / 128;
    LAT_CUDA_TRY(launch_pdl(join_kernel, dim3(unsigned(std::min(p.shares, std::max(1, kJoinBlocks / cols))), unsigned(cols)),
                            dim3(32, kJoinRows), 0, s, p, per_block));
    return LAT_OK;
}

template <typename T, typename I>
lat_status lookup(const I *ids, int64_t n, const T *table, int64_t vocab, int c, float scale, int64_t pad, T *y,
                  int32_t *d_status, cudaStream_t s) {
    return by_lanes(c, [&](auto l) -> lat_status {
        constexpr int L = decltype(l)::value;
        const int64_t per = kThreads / L;
        const dim3 grid(unsigned((n + per - 1) / per), unsigned((c / 8 + 4 * L - 1) / (4 * L)));
        LAT_CUDA_TRY(launch_pdl(lookup_kernel<T, I, L>, grid, dim3(kThreads), 0, s, ids, n, table, vocab, c, scale, pad,
                                y, d_status));
        return LAT_OK;
    });
}

static bool args_ok(const void *ids, int32_t id_bytes, int64_t n, int64_t vocab, int32_t c, lat_dtype dtype) {
    if (!rows::rows_ok(n) || !rows::chan_ok(c) || vocab < 1 || vocab >= (int64_t(1) << 31) - 1) return false;
    if (dtype != LAT_F32 && dtype != LAT_F16 && dtype != LAT_BF16) return false;
    return (id_bytes == 4 || id_bytes == 8) && (n == 0 || ids) && rows::aligned(ids, size_t(id_bytes));
}

// Calls f(ids as int32* or int64*, element) for the id width and the dtype.
template <typename F>
static lat_status by_types(const void *ids, int32_t id_bytes, lat_dtype dtype, F &&f) {
    auto both = [&](auto e) {
        return id_bytes == 4 ? f(static_cast<const int32_t *>(ids), e) : f(static_cast<const int64_t *>(ids), e);
    };
    switch (dtype) {
        case LAT_F32: return both(float{});
        case LAT_F16: return both(__half{});
        case LAT_BF16: return both(__nv_bfloat16{});
    }
    return LAT_ERR_ARG;
}

}  // namespace embed
}  // namespace lat

extern "C" lat_status lat_embed_fwd(const void *ids, int32_t id_bytes, int64_t n, const void *table, int64_t vocab,
                                    int32_t c, float scale, int64_t pad_id, void *y, lat_dtype dtype,
                                    int32_t *d_status, lat_stream stream) {
    using namespace lat;
    if (!embed::args_ok(ids, id_bytes, n, vocab, c, dtype) || !table || (n > 0 && !y)) return LAT_ERR_ARG;
    if (!rows::aligned(table, rows::slice_bytes(dtype)) || !rows::aligned(y, rows::slice_bytes(dtype))) return LAT_ERR_ARG;
    if (n == 0) return LAT_OK;
    return embed::by_types(ids, id_bytes, dtype, [&](auto id, auto e) {
        using T = decltype(e);
        return embed::lookup(id, n, static_cast<const T *>(table), vocab, c, scale, pad_id, static_cast<T *>(y),
                             d_status, reinterpret_cast<cudaStream_t>(stream));
    });
}

extern "C" size_t lat_embed_wgrad_ws_bytes(int64_t n, int64_t vocab, int32_t c) {
    using namespace lat;
    if (!rows::rows_ok(n) || !rows::chan_ok(c) || vocab < 1 || vocab >= (int64_t(1) << 31) - 1) return 0;
    return embed::Ws(nullptr, n, vocab, c).bytes;
}

extern "C" lat_status lat_embed_wgrad(const void *ids, int32_t id_bytes, int64_t n, const void *dy, int64_t vocab,
                                      int32_t c, float scale, int64_t pad_id, float *dtable, lat_dtype dtype, void *ws,
                                      size_t ws_bytes, int32_t *d_status, lat_stream stream) {
    using namespace lat;
    if (!embed::args_ok(ids, id_bytes, n, vocab, c, dtype) || !dtable || (n > 0 && !dy)) return LAT_ERR_ARG;
    if (!rows::aligned(dy, rows::slice_bytes(dtype)) || !rows::aligned(dtable, 32)) return LAT_ERR_ARG;
    if (!ws || !rows::aligned(ws, 32) || ws_bytes < lat_embed_wgrad_ws_bytes(n, vocab, c)) return LAT_ERR_WORKSPACE;
    return embed::by_types(ids, id_bytes, dtype, [&](auto id, auto e) {
        using T = decltype(e);
        return embed::wgrad(id, n, static_cast<const T *>(dy), vocab, c, scale, pad_id, dtable, ws, d_status,
                            reinterpret_cast<cudaStream_t>(stream));
    });
}
