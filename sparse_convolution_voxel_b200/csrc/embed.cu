// Embedding lookup with scaling and its gradient by sorted tokens (lat_embed_fwd,
// lat_embed_wgrad).
//
//   y[i] = scale * table[id_i]          dtable[t] = scale * sum over i with id_i = t of dy[i]
//
// Lookup: a gather, bound by the bytes it copies.  L lanes take a row, 8 channels each.
//
// Gradient: the rows are sorted by token (a stable LSD radix sort of (token, row) pairs;
// rows without a token get the key `vocab`, behind every token), so that each token's rows
// are one run of the sorted list.  The list is cut into equal shares, each walked by one group
// of lanes with the sum in registers, which is stored when the token changes.  So a token with
// a hundred thousand rows is spread over many shares.  A token whose run crosses a cut leaves
// one fp32 partial per share (head: the sum up to its end or over a whole share, tail: the sum
// from its begin), and another kernel adds them in share order.  No atomics on sums: the bits
// depend neither on timing nor on the GPU.
//
// Tokens without rows have gradient zero, most of the table in a step of few tokens: the sort
// marks the tokens that it meets in a bitmap, and the kernel that adds the partials stores the
// other rows too.  Where these are many megabytes, a kernel of its own does, on a side stream,
// while the sort and the sums, which wait for latencies more than for bandwidth, go on.
//
// Launches: up to 4,096 rows (of 2^20 tokens at most) the sort, the sums and the join; beyond, the
// bitmap's clear, a count and a scatter for every 10 bits of the vocabulary, with a scan between
// them where the counts are many, the sums and the join; the zeros of a large table take one more.
// So three to sixteen, of 2 us and more each.  500k x 128 bf16 rows of 1,000 tokens take 56 us with
// six; the sums alone, one after the others, 33 (3.9 TB/s of random rows).
#include <algorithm>

#include "rows.cuh"
#include "tc_ptx.cuh"

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
        if (t >= 0) {
            rows::to_f(rows::ld(table + t * c + vi * 8), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= scale;
        }
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
    uint32_t *totals;   // [bins]; null: the counts are not scanned, the scatter's blocks do it
    int32_t *open_count;  // of the sums' list, cleared by the count
    int64_t n;
    int tiles, shift, bits;
};
template <typename I> struct Ids {
    const I *ids;
    int64_t vocab, pad;
    uint32_t *present;  // bitmap of the tokens with rows
};
__device__ __forceinline__ void mark(uint32_t *present, uint32_t word, uint32_t bits) {
    if (bits & ~__ldcg(present + word)) atomicOr(present + word, bits);
}

template <typename I>
__device__ __forceinline__ uint32_t sort_key(const Pass &p, const Ids<I> &d, int64_t i, int32_t &bad) {
    if (p.key_in) return p.key_in[i];
    const int64_t t = token(d.ids, i, d.vocab, d.pad, bad);
    return uint32_t(t < 0 ? d.vocab : t);
}

constexpr int kSeenWords = 8192, kSeenTokens = 1024;  // of a block's shared memory
static size_t seen_bytes(int64_t vocab) {
    return 4 * size_t(vocab <= 32 * kSeenWords ? (vocab + 31) / 32 : kSeenTokens);
}
template <typename I, int R>
__global__ void __launch_bounds__(kThreads) count_kernel(Pass p, Ids<I> d, int32_t *d_status) {
    pdl_enter();
    __shared__ uint32_t s_cnt[kMaxBins];
    // Tokens of this block that are marked: a bitmap while the vocabulary fits (lanes then mark neighbouring words
    // of the table's bitmap, each once per block: with one access per token 489 blocks of 1,000 tokens took 33 us,
    // now 7, and 42, now 17, among 100,000 tokens), else the last token by its low bits, which keeps the frequent
    // ones from the table's words.
    extern __shared__ uint32_t s_seen[];
    const bool first = !p.key_in, fits = d.vocab <= 32 * kSeenWords;
    const int seen = fits ? int((d.vocab + 31) / 32) : kSeenTokens;
    const int bins = 1 << p.bits;
    for (int b = threadIdx.x; b < bins; b += kThreads) s_cnt[b] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.open_count = 0;
    if (first)
        for (int b = threadIdx.x; b < seen; b += kThreads) s_seen[b] = fits ? 0u : ~0u;
    __syncthreads();
    const int64_t lo = blockIdx.x * int64_t(kThreads * R), hi = min(p.n, lo + kThreads * R);
    int32_t bad = 0;
#pragma unroll R
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
        const uint32_t key = sort_key(p, d, i, bad);
        atomicAdd(&s_cnt[(key >> p.shift) & (bins - 1)], 1u);
        if (!first || key >= d.vocab) continue;
        if (fits) {
            if (!(s_seen[key >> 5] >> (key & 31) & 1u)) atomicOr(&s_seen[key >> 5], 1u << (key & 31));
        } else if (s_seen[key % kSeenTokens] != key) {
            s_seen[key % kSeenTokens] = key;
            mark(d.present, key >> 5, 1u << (key & 31));
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kThreads) p.counts[int64_t(blockIdx.x) * bins + b] = s_cnt[b];
    if (first && fits)
        for (int b = threadIdx.x; b < seen; b += kThreads)
            if (s_seen[b]) mark(d.present, b, s_seen[b]);
    if (bad) flag(d_status, bad);
}

// 8 digit values per block, 128 threads each: thread row t takes a run of the tiles.
constexpr int kScanBins = 8, kScanRows = 128;
__global__ void __launch_bounds__(kScanBins * kScanRows)
tile_scan_kernel(uint32_t *__restrict__ counts, uint32_t *__restrict__ totals, int tiles, int bins) {
    pdl_enter();
    __shared__ uint32_t s[2][kScanRows][kScanBins];
    const int b = blockIdx.x * kScanBins + threadIdx.x, t = threadIdx.y;
    const int per = (tiles + kScanRows - 1) / kScanRows, lo = min(tiles, t * per), hi = min(tiles, lo + per);
    uint32_t sum = 0;
    if (b < bins) {
#pragma unroll 4
        for (int i = lo; i < hi; ++i) sum += counts[int64_t(i) * bins + b];
    }
    uint32_t upto = sum;
    int at = 0;
    s[0][t][threadIdx.x] = upto;
    __syncthreads();
#pragma unroll
    for (int m = 1; m < kScanRows; m <<= 1, at ^= 1) {
        if (t >= m) upto += s[at][t - m][threadIdx.x];
        s[at ^ 1][t][threadIdx.x] = upto;
        __syncthreads();
    }
    if (b >= bins) return;
    if (t == kScanRows - 1) totals[b] = upto;
    uint32_t run = upto - sum;
    for (int i = lo; i < hi; ++i) {
        const uint32_t v = counts[int64_t(i) * bins + b];
        counts[int64_t(i) * bins + b] = run;
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
    auto add4 = [](uint4 &a, const uint4 &v) { a = make_uint4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w); };
    if (!p.totals) {
        // thread row g of four digits per thread adds the tiles g, g + rows, ...; then the rows meet
        const int quads = bins / 4, tile_rows = kThreads / quads, g = threadIdx.x / quads;
#pragma unroll 16
        for (int t = g; t < p.tiles; t += tile_rows) {
            const uint4 v = reinterpret_cast<const uint4 *>(p.counts + int64_t(t) * bins)[threadIdx.x % quads];
            add4(total, v);
            if (t < int(blockIdx.x)) add4(start, v);
        }
        s_cnt4[0][threadIdx.x] = total;
        s_cnt4[1][threadIdx.x] = start;
        __syncthreads();
        if (own)
            for (int o = 1; o < min(tile_rows, p.tiles); ++o) {
                add4(total, s_cnt4[0][o * quads + threadIdx.x]);
                add4(start, s_cnt4[1][o * quads + threadIdx.x]);
            }
        else
            total = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
    } else if (own) {
        total = reinterpret_cast<const uint4 *>(p.totals)[threadIdx.x];
        start = reinterpret_cast<const uint4 *>(p.counts + int64_t(blockIdx.x) * bins)[threadIdx.x];
    }
    if (own) {
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
    for (int64_t i = threadIdx.x; i < (d.vocab + 31) / 32; i += kSmallThreads) d.present[i] = 0;
    __syncthreads();
    uint32_t key[kSmallRounds], row[kSmallRounds];  // row: and the rank, in the upper half
    int32_t bad = 0;
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r) {
        const int i = lo + r * 32 + lane;
        if (r < rounds && i < n) {
            const int64_t t = token(d.ids, i, d.vocab, d.pad, bad);
            key[r] = uint32_t(t < 0 ? d.vocab : t);
            row[r] = uint32_t(i);
            if (t >= 0) mark(d.present, key[r] >> 5, 1u << (key[r] & 31));
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
struct Runs {
    const uint32_t *key, *row;  // sorted
    uint32_t n, vocab;
    uint32_t share;             // sorted rows per share
    int shares;
    int c;
    float scale;
    float *head, *tail;         // [shares][c]
    int2 *open;                 // (share, token) where a run begins that goes on behind the share, in any order
    int32_t *open_count;
    int32_t *last;              // [vocab]: of a token whose run ends behind a cut, the share with its end
    float *dtable;
    const uint32_t *present;    // bitmap of the tokens with rows if the join stores the other rows' zeros, else null
};

// A group's lanes read the tokens and rows of L sorted rows at a time, one each, and the next
// ones before they add; kFlight rows of dy are in flight while kFlight are added.  A row of
// more than 256 channels takes several groups (slabs), up to eight of them side by side in a
// block, so that a block reads and writes long pieces.  A block takes `per_block` consecutive
// shares; if a token's run covers them all, their sums meet in shared memory and the first
// share's head stands for the block.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads, 3) sums_kernel(Runs p, const T *__restrict__ dy, int per_block) {
    pdl_enter();
    constexpr int kFlight = sizeof(T) == 4 || L == 4 ? 2 : 4;  // an even number of times per batch
    __shared__ float s_acc[8][kThreads];
    const int group = threadIdx.x / L, lane = threadIdx.x % L, first = (threadIdx.x & 31) / L * L;
    const uint32_t mask = (L == 32 ? 0xFFFFFFFFu : ((1u << (L & 31)) - 1u) << first);
    const int slabs = L < 32 ? 1 : int(blockDim.x) / L / per_block;  // of a block
    const int v = blockIdx.x * per_block + group / slabs;
    const uint32_t i0 = uint32_t(min(uint64_t(v) * p.share, uint64_t(p.n)));
    const uint32_t i1 = uint32_t(min(uint64_t(i0) + p.share, uint64_t(p.n)));
    const int vi = (int(blockIdx.y) * slabs + group % slabs) * L + lane;
    const bool own = vi < p.c / 8;
    const uint32_t col = vi * 8;
    // the first token, and whether its run began in an earlier share; the last token, and whether its run goes on
    const bool some = i0 < i1;
    const uint32_t r0 = some ? __ldg(p.key + i0) : p.vocab, r1 = some ? __ldg(p.key + i1 - 1) : p.vocab;
    const bool cut = some && i0 > 0 && __ldg(p.key + i0 - 1) == r0;
    const bool goes_on = r1 < p.vocab && i1 < p.n && __ldg(p.key + i1) == r1;
    float acc[8] = {};
    uint32_t r = r0;
    auto store = [&]() {  // the sum of token r
        if (own && r < p.vocab) {
            if (cut && r == r0) {
                rows::st(p.head + v * int64_t(p.c) + col, acc);
                if (vi == 0) p.last[r] = v;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] *= p.scale;
                rows::st(p.dtable + int64_t(r) * p.c + col, acc);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    };
    // behind the share's end, and for a row without a token, there is nothing to add
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
    uint32_t before_batch = r0;
    for (uint32_t b = i0; b < i1; b += L) {
        next_key = step_key(b + L + lane);
        next_row = step_row(b + L + lane);
        // rows of this batch (bit: the row) whose token is not the one before it
        uint32_t before = __shfl_up_sync(mask, key, 1, L);
        if (lane == 0) before = before_batch;
        const uint32_t begins = (__ballot_sync(mask, key != before) & mask) >> first;
        before_batch = __shfl_sync(mask, key, L - 1, L);
#pragma unroll
        for (int q = 0; q < L; q += kFlight) {
            const int now = (q / kFlight) & 1;
            if (b + q >= i1) break;
            if (q + kFlight < L) load(x[now ^ 1], key, row, q + kFlight);
            else load(x[now ^ 1], next_key, next_row, 0);
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if (((begins >> (q + u)) & 1u) && b + q + u < i1) {
                    store();
                    r = __shfl_sync(mask, key, q + u, L);
                }
                float f[8];
                rows::to_f(x[now][u], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += f[e];
            }
        }
        key = next_key;
        row = next_row;
    }
    if (some && !goes_on) store();
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
        if (!through && vi == 0) p.open[atomicAdd(p.open_count, 1)] = make_int2(v, int(r1));
    }
}

// Tokens whose run crosses a cut: for each listed share v the run is tail[v], then the heads
// of the shares up to the one that holds the run's end, where a sums block that lies between
// v's and the last one's has one head for all its shares.  A block takes a run: row t of
// kJoinRows adds the parts t, t + kJoinRows, ... in order, then the rows' sums are added in
// order.  Where there are more runs than blocks, a warp takes a run of up to kShort parts by
// itself and adds them in order (7,000 runs of 500k x 128 rows of 100,000 tokens: 10.5 us, with
// a block for each 16).  The list's order does not matter: every token is the sum of one entry.
// Stores the zeros too, see Runs::present: 2 us less than by a launch of their own.
constexpr int kJoinRows = 8, kJoinBlocks = 1184, kShort = 16;
__global__ void __launch_bounds__(32 * kJoinRows) join_kernel(Runs p, int per_block) {
    pdl_enter();
    __shared__ float4 s[kJoinRows][32];
    __shared__ int s_long[kJoinRows];
    const int count = *p.open_count, col = (blockIdx.y * 32 + threadIdx.x) * 4;
    const bool own = col < p.c;
    if (p.present && own)
        for (uint32_t r = blockIdx.x * kJoinRows + threadIdx.y; r < p.vocab; r += gridDim.x * kJoinRows)
            if (!((__ldg(p.present + (r >> 5)) >> (r & 31)) & 1u))
                *reinterpret_cast<float4 *>(p.dtable + int64_t(r) * p.c + col) = make_float4(0.f, 0.f, 0.f, 0.f);
    struct Run {
        int v, token, last, lead, blocks, parts;
    };
    auto run_of = [&](int o) {
        const int2 open = p.open[o];
        Run r{open.x, open.y, p.last[open.y], 0, 0, 0};
        // shares v .. end of v's block, whole blocks, then the shares of the last block
        const int block = r.v / per_block;
        r.blocks = max(0, r.last / per_block - block - 1);
        r.lead = min(r.last, (block + 1) * per_block - 1) - r.v + 1;
        r.parts = r.blocks > 0 ? r.lead + r.blocks + r.last % per_block + 1 : r.last - r.v + 1;
        return r;
    };
    auto part = [&](const Run &r, int q) {
        int64_t at = r.v + q;
        if (r.blocks > 0 && q >= r.lead)
            at = q < r.lead + r.blocks ? (r.v / per_block + 1 + q - r.lead) * per_block : r.last - (r.parts - 1 - q);
        return *reinterpret_cast<const float4 *>((q == 0 ? p.tail : p.head) + at * p.c + col);
    };
    auto add = [](float4 &a, const float4 &x) {
        a.x += x.x;
        a.y += x.y;
        a.z += x.z;
        a.w += x.w;
    };
    auto store = [&](const Run &r, const float4 &a) {
        *reinterpret_cast<float4 *>(p.dtable + int64_t(r.token) * p.c + col) =
            make_float4(a.x * p.scale, a.y * p.scale, a.z * p.scale, a.w * p.scale);
    };
    auto by_block = [&](int o) {
        const Run r = run_of(o);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (own) {
#pragma unroll 4
            for (int q = threadIdx.y; q < r.parts; q += kJoinRows) add(acc, part(r, q));
        }
        s[threadIdx.y][threadIdx.x] = acc;
        __syncthreads();
        if (threadIdx.y == 0 && own) {
#pragma unroll
            for (int q = 1; q < kJoinRows; ++q) add(acc, s[q][threadIdx.x]);
            store(r, acc);
        }
    };
    if (count <= int(gridDim.x)) {
        if (int(blockIdx.x) < count) by_block(blockIdx.x);
        return;
    }
    for (int o0 = blockIdx.x; o0 < count; o0 += gridDim.x * kJoinRows) {
        const int o = o0 + int(gridDim.x * threadIdx.y);
        bool long_run = false;
        if (o < count) {
            const Run r = run_of(o);
            long_run = r.parts > kShort;
            if (own && !long_run) {
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int q = 0; q < r.parts; ++q) add(acc, part(r, q));
                store(r, acc);
            }
        }
        if (!__syncthreads_or(long_run)) continue;
        if (threadIdx.x == 0) s_long[threadIdx.y] = long_run ? o : -1;
        __syncthreads();
        for (int w = 0; w < kJoinRows; ++w) {
            if (s_long[w] < 0) continue;
            by_block(s_long[w]);
            __syncthreads();
        }
    }
}

// Zeros for the tokens without rows, where the join does not store them.  A warp takes `tokens`
// of them at a time (a power of two up to 32): each run of absent ones is a piece of the table
// without a gap, written by bulk stores from a buffer of zeros.  (Stores from registers fill the
// load and store units: for 32,768 rows x 512, 131,072 tokens, the call took 45 us more with them.)
constexpr int kZeroThreads = 128, kZeroWarps = kZeroThreads / 32;
constexpr uint32_t kZeroBytes = 16384;  // of the buffer
__global__ void __launch_bounds__(kZeroThreads)
zeros_kernel(const uint32_t *__restrict__ present, uint32_t vocab, uint32_t tokens, uint32_t row_bytes,
             uint8_t *__restrict__ dtable) {
    pdl_enter();
    __shared__ uint4 s_zero[kZeroBytes / 16];
    for (int i = threadIdx.x; i < int(kZeroBytes / 16); i += kZeroThreads) s_zero[i] = make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
    __syncthreads();
    const uint32_t lane = threadIdx.x & 31, stride = gridDim.x * kZeroWarps * tokens;
    for (uint64_t t = (blockIdx.x * kZeroWarps + (threadIdx.x >> 5)) * tokens; t < vocab; t += stride) {
        uint32_t absent = ~__ldg(present + (t >> 5)) >> (t & 31);
        const uint32_t here = uint32_t(min(uint64_t(tokens), vocab - t));
        if (here < 32) absent &= (1u << here) - 1u;
        const uint32_t from = absent >> lane;  // this lane's token and those behind it
        if (!(from & 1u) || (lane > 0 && ((absent >> (lane - 1)) & 1u))) continue;  // no run begins here
        const uint32_t count = from == ~0u ? 32u : uint32_t(__ffs(int(~from))) - 1u;
        uint8_t *at = dtable + (t + lane) * row_bytes;
        for (uint32_t left = count * row_bytes; left > 0;) {
            const uint32_t bytes = min(left, kZeroBytes);
            ptx::bulk_store(at, s_zero, bytes);
            at += bytes;
            left -= bytes;
        }
    }
    ptx::bulk_store_commit();
    ptx::bulk_store_wait();
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

// Shares of the sorted rows: one wave of groups (the sums' registers admit 24 warps on each of a
// B200's 148 SMs), but at least 16 rows each; the numbers depend on the sizes alone.
static int run_shares(int64_t n, int c) {
    const int64_t slabs = (c / 8 + 31) / 32, want = 148 * 24 * (32 / lanes_of(c)) / slabs;
    return int(std::max<int64_t>(1, std::min<int64_t>(want, (n + 15) / 16)));
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
    return std::max<int64_t>(1, (n + tile - 1) / tile);
}

// Up to this many counts (tiles x digit values) every block of the scatter scans them itself, a
// launch less in every pass.  Where calls wait for their launches that is what counts: back to
// back, 24,000 rows x 64 of 50,000 tokens (two passes of 47 x 256) take 38 us, with the scan 43.
// Behind queued work, which hides the launches, the scatter's own scan costs a little: 40 us with
// the scan's launch, 42 without; 16,384 x 64 of 1,000 tokens (32 x 1024) 29 and 33.  Beside a large
// table's zeros, whose writes every read of a count waits behind, it costs more, so fewer there:
// 32,768 rows x 512, 131,072 tokens (64 x 512 counts) 87 us with the scan, 125 without; 16,383 x
// 1024, 50,257 tokens (32 x 256) 65 either way.
constexpr int64_t kFewCounts = 32768, kFewCountsBeside = 8192;

// Zeros of at least this many bytes have a kernel of their own: with the launches of a sort ahead
// on the side stream (a fork and a join cost a few microseconds, the zeros of 16 MB as many);
// behind a one-block sort in front of the sums, which are short.  (Beside those it came after the
// sums' and the join's blocks had taken every SM, and crowded on the first that came free: 443 us
// for 2,048 rows x 4096, 32,000 tokens, now 110.)
constexpr size_t kLargeBytes = size_t(16) << 20;
// (32,768 rows x 512, 131,072 tokens: 103 us with 74 blocks, 107 with 148, 93 with 296, 87 with 592; 2,048 x 4096,
// 32,000 tokens: 144, 134, 112 and 110)
constexpr int kZeroBlocks = 592;
constexpr int64_t kSmallWords = 32768;  // of the bitmap that the one-block sort clears itself

// The side stream, or null where there is none to be had: creating it is left to calls outside
// a capture, and one that takes part in another capture is not ours to use.
static SideStream *free_side_stream(cudaStream_t s) {
    cudaStreamCaptureStatus mine = cudaStreamCaptureStatusNone, its = cudaStreamCaptureStatusNone;
    unsigned long long my_id = 0, its_id = 0;
    if (cudaStreamGetCaptureInfo(s, &mine, &my_id) != cudaSuccess) return nullptr;
    SideStream *side = nullptr;
    if (side_stream_slot(side) != cudaSuccess || (mine != cudaStreamCaptureStatusNone && !side->side)) return nullptr;
    if (side_stream(side) != cudaSuccess || cudaStreamGetCaptureInfo(side->side, &its, &its_id) != cudaSuccess)
        return nullptr;
    return its == cudaStreamCaptureStatusNone || (mine == its && my_id == its_id) ? side : nullptr;
}

struct Ws {
    uint32_t *key[2], *row[2], *counts, *totals;
    float *head, *tail;
    int2 *open;
    int32_t *open_count;
    int32_t *last;
    uint32_t *present;
    size_t bytes;
    Ws(void *base, int64_t n, int64_t vocab, int c) {
        Carver cv(base);
        for (int i = 0; i < 2; ++i) {
            key[i] = cv.take<uint32_t>(size_t(n));
            row[i] = cv.take<uint32_t>(size_t(n));
        }
        counts = cv.take<uint32_t>(size_t(tiles_of(n)) * kMaxBins);
        totals = cv.take<uint32_t>(kMaxBins);
        const size_t part = size_t(run_shares(n, c)) * size_t(c);
        head = cv.take<float>(part);
        tail = cv.take<float>(part);
        open = cv.take<int2>(size_t(run_shares(n, c)));
        open_count = cv.take<int32_t>(1);
        last = cv.take<int32_t>(size_t(vocab));
        present = cv.take<uint32_t>(size_t(vocab + 31) / 32);
        bytes = align_up(cv.used, 256);
    }
};

template <typename T, typename I>
lat_status wgrad(const I *ids, int64_t n, const T *dy, int64_t vocab, int c, float scale, int64_t pad, float *dtable,
                 void *ws, int32_t *d_status, cudaStream_t s) {
    Ws w(ws, n, vocab, c);
    const int64_t words = (vocab + 31) / 32;
    const Ids<I> d{ids, vocab, pad, w.present};
    const bool one_block = n <= kSmall && words <= kSmallWords;  // of the sort
    SideScope beside(s);  // the zeros of a large table
    auto zeros = [&](cudaStream_t to) -> lat_status {
        uint32_t tokens = 32;  // of a warp at a time: some 64 KB of zeros
        while (tokens > 1 && tokens * uint32_t(c) * 4 > 65536) tokens /= 2;
        const int64_t blocks = std::min<int64_t>((vocab + tokens * kZeroWarps - 1) / (tokens * kZeroWarps), kZeroBlocks);
        LAT_CUDA_TRY(launch_pdl(zeros_kernel, dim3(unsigned(blocks)), dim3(kZeroThreads), 0, to, w.present,
                                uint32_t(vocab), tokens, uint32_t(c) * 4, reinterpret_cast<uint8_t *>(dtable)));
        return LAT_OK;
    };
    const bool joined = n > 0 && size_t(vocab) * size_t(c) * sizeof(float) < kLargeBytes;  // the zeros are the join's
    int at = 0;
    if (one_block) {
        auto kern = sort_small_kernel<I>;
        LAT_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmallSmem)));
        LAT_CUDA_TRY(launch_pdl(kern, dim3(1), dim3(kSmallThreads), kSmallSmem, s, d, int(n), key_bits(vocab), w.key[0],
                                w.row[0], w.open_count, d_status));
        if (!joined) {
            const lat_status st = zeros(s);
            if (st != LAT_OK) return st;
        }
    } else {
        LAT_CUDA_TRY(fill_u32(w.present, words, 0u, s));
        const int bits = key_bits(vocab), passes = (bits + kMaxBits - 1) / kMaxBits;
        const int digit = std::max(2, (bits + passes - 1) / passes), tiles = int(tiles_of(n));
        const int bins = 1 << digit;
        const bool few = tile_rounds(n) == 2;
        const bool scan = int64_t(tiles) * bins > (joined ? kFewCounts : kFewCountsBeside);
        auto count = few ? count_kernel<I, 2> : count_kernel<I, 4>;
        auto scatter = few ? scatter_kernel<I, 2> : scatter_kernel<I, 4>;
        for (int i = 0; i < passes; ++i) {
            const int to = i & 1;
            Pass p{i ? w.key[1 - to] : nullptr, i ? w.row[1 - to] : nullptr, w.key[to], w.row[to], w.counts,
                   scan ? w.totals : nullptr, w.open_count, n, tiles, i * digit, digit};
            LAT_CUDA_TRY(launch_pdl(count, dim3(tiles), dim3(kThreads), i ? 0 : seen_bytes(vocab), s, p, d,
                                    i ? nullptr : d_status));
            if (i == 0 && !joined) {  // the bitmap is complete on s
                SideStream *side = free_side_stream(s);
                if (side) LAT_CUDA_TRY(beside.fork(*side));
                const lat_status st = zeros(side ? side->side : s);
                if (st != LAT_OK) return st;
            }
            if (scan)
                LAT_CUDA_TRY(launch_pdl(tile_scan_kernel, dim3((bins + kScanBins - 1) / kScanBins),
                                        dim3(kScanBins, kScanRows), 0, s, w.counts, w.totals, tiles, bins));
            LAT_CUDA_TRY(launch_pdl(scatter, dim3(tiles), dim3(kThreads), 0, s, p, d));
            at = to;
        }
    }
    if (n > 0) {
        Runs p{w.key[at], w.row[at], uint32_t(n), uint32_t(vocab), 0, run_shares(n, c), c, scale, w.head, w.tail, w.open,
               w.open_count, w.last, dtable, joined ? w.present : nullptr};
        p.share = uint32_t((n + p.shares - 1) / p.shares);
        const int groups = kThreads / lanes_of(c), slabs = (c / 8 + 31) / 32, abreast = std::min(slabs, groups);
        const int per_block = groups / abreast;
        const lat_status st = by_lanes(c, [&](auto l) -> lat_status {
            constexpr int L = decltype(l)::value;
            const dim3 grid(unsigned((p.shares + per_block - 1) / per_block), unsigned((slabs + abreast - 1) / abreast));
            LAT_CUDA_TRY(launch_pdl(sums_kernel<T, L>, grid, dim3(unsigned(L * abreast * per_block)), 0, s, p, dy,
                                    per_block));
            return LAT_OK;
        });
        if (st != LAT_OK) return st;
        const int cols = (c + 127) / 128, most = std::max(1, kJoinBlocks / cols);
        LAT_CUDA_TRY(launch_pdl(join_kernel, dim3(unsigned(joined ? most : std::min(p.shares, most)), unsigned(cols)),
                                dim3(32, kJoinRows), 0, s, p, per_block));
    }
    LAT_CUDA_TRY(beside.join());
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
