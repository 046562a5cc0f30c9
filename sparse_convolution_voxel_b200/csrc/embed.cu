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
// their scan over the tiles, and the scatter.  A tile is kTile consecutive rows; in the
// scatter a warp takes kTile / 8 of them, 32 at a time, and ranks the rows of equal digit
// by a warp match, so equal keys keep their order.
constexpr int kTile = 2048;
constexpr int kWarps = kThreads / 32;
constexpr int kPerWarp = kTile / kWarps;
constexpr int kRounds = kPerWarp / 32;
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

template <typename I>
__global__ void __launch_bounds__(kThreads) count_kernel(Pass p, Ids<I> d, int32_t *d_status) {
    pdl_enter();
    __shared__ uint32_t s_cnt[kMaxBins];
    const int bins = 1 << p.bits;
    for (int b = threadIdx.x; b < bins; b += kThreads) s_cnt[b] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * int64_t(kTile), hi = min(p.n, lo + kTile);
    int32_t bad = 0;
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

template <typename I>
__global__ void __launch_bounds__(kThreads) scatter_kernel(Pass p, Ids<I> d) {
    pdl_enter();
    __shared__ uint32_t s_cnt[kWarps][kMaxBins];
    __shared__ uint32_t s_scan[kThreads];
    const int bins = 1 << p.bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int b = threadIdx.x; b < bins; b += kThreads)
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s_cnt[w][b] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * int64_t(kTile) + warp * kPerWarp;
    uint32_t key[kRounds], rank[kRounds], row[kRounds];
    int32_t bad = 0;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int64_t i = lo + r * 32 + lane;
        key[r] = i < p.n ? sort_key(p, d, i, bad) : 0u;
        row[r] = i < p.n ? (p.row_in ? p.row_in[i] : uint32_t(i)) : 0u;
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const bool in = lo + r * 32 + lane < p.n;
        const uint32_t digit = in ? (key[r] >> p.shift) & (bins - 1) : uint32_t(bins);
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, digit);
        const uint32_t before = __popc(peers & ((1u << lane) - 1u));
        if (in) rank[r] = s_cnt[warp][digit] + before;
        __syncwarp();
        if (in && before == 0) s_cnt[warp][digit] += __popc(peers);
        __syncwarp();
    }
    // first position of each digit: an exclusive scan of the totals, a run of digits per thread
    const int per = (bins + kThreads - 1) / kThreads;
    const int b0 = min(bins, int(threadIdx.x) * per), b1 = min(bins, b0 + per);
    uint32_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += p.totals[b];
    s_scan[threadIdx.x] = sum;
    __syncthreads();
    for (int m = 1; m < kThreads; m <<= 1) {
        const uint32_t v = int(threadIdx.x) >= m ? s_scan[threadIdx.x - m] : 0u;
        __syncthreads();
        s_scan[threadIdx.x] += v;
        __syncthreads();
    }
    uint32_t at = threadIdx.x ? s_scan[threadIdx.x - 1] : 0u;
    for (int b = b0; b < b1; ++b) {
        uint32_t run = at + p.counts[int64_t(blockIdx.x) * bins + b];
        at += p.totals[b];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t v = s_cnt[w][b];
            s_cnt[w][b] = run;
            run += v;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        if (lo + r * 32 + lane < p.n) {
            const uint32_t pos = s_cnt[warp][(key[r] >> p.shift) & (bins - 1)] + rank[r];
            p.key_out[pos] = key[r];
            p.row_out[pos] = row[r];
        }
    }
}

// ------------------------------------------------------------------------ the sums
struct Path {
    const uint32_t *key, *row;  // sorted
    int64_t n, vocab;
    int64_t share;              // steps per share
    int shares;
    int c;
    float scale;
    float *head, *tail;         // [shares][c]
    int32_t *open, *open_count; // shares in which a run begins that goes on behind them, in any order
    float *dtable;
};

// Sorted rows among the first `step` steps of the path: the first i with key[i] + i >= step
// (key[i] + i increases strictly).  W lanes search together: each round splits the range
// into W + 1 parts.
template <int W>
__device__ __forceinline__ int64_t path_rows(const Path &p, int64_t step, int lane, uint32_t mask, int first) {
    int64_t lo = max(int64_t(0), step - p.vocab), hi = min(step, p.n);  // the answer is in [lo, hi]
    while (lo < hi) {
        const int64_t span = hi - lo;
        const int64_t at = lo + span * (lane + 1) / (W + 1);  // in [lo, hi)
        const bool less = int64_t(p.key[at]) + at < step;
        const uint32_t votes = (__ballot_sync(mask, less) & mask) >> first;
        const int k = __popc(votes);  // the probes are in order, so the votes are a prefix
        const int64_t nlo = k == 0 ? lo : lo + span * k / (W + 1) + 1;
        const int64_t nhi = k == W ? hi : lo + span * (k + 1) / (W + 1);
        lo = nlo;
        hi = nhi;
    }
    return lo;
}

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) sums_kernel(Path p, const T *__restrict__ dy) {
    pdl_enter();
    constexpr int U = sizeof(T) == 2 ? 8 : 4;  // rows in flight
    const int group = threadIdx.x / L, lane = threadIdx.x % L, first = (threadIdx.x & 31) / L * L;
    const uint32_t mask = (L == 32 ? 0xFFFFFFFFu : ((1u << L) - 1u) << first);
    const int v = blockIdx.x * (kThreads / L) + group;
    if (v >= p.shares) return;
    const int64_t s0 = v * p.share, s1 = min(s0 + p.share, p.vocab + p.n);
    const int64_t i0 = path_rows<L>(p, s0, lane, mask, first), i1 = path_rows<L>(p, s1, lane, mask, first);
    const int64_t r0 = s0 - i0, r1 = s1 - i1;
    const int vi = blockIdx.y * L + lane;
    if (vi >= p.c / 8) return;
    const int64_t col = vi * 8;
    // the first token's run began in an earlier share
    const bool cut = i0 > 0 && int64_t(p.key[i0 - 1]) == r0;
    float acc[8] = {};
    int64_t r = r0;
    auto store = [&]() {
        if (cut && r == r0) {
            rows::st(p.head + v * int64_t(p.c) + col, acc);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] *= p.scale;
            rows::st(p.dtable + r * p.c + col, acc);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        ++r;
    };
    for (int64_t b = i0; b < i1; b += U) {
        int64_t key[U];
        Slice8<T> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            key[u] = b + u < i1 ? int64_t(p.key[b + u]) : p.vocab;
            x[u] = key[u] < p.vocab ? rows::ld(dy + int64_t(p.row[b + u]) * p.c + col) : rows::zero_slice<T>();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b + u >= i1) break;
            while (r < key[u] && r < p.vocab) store();
            float f[8];
            rows::to_f(x[u], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += f[e];
        }
    }
    while (r < r1) store();
    // the last token's run goes on in the next share
    if (r < p.vocab && i1 > 0 && int64_t(p.key[i1 - 1]) == r) {
        const bool begun_before = cut && r == r0;
        rows::st((begun_before ? p.head : p.tail) + v * int64_t(p.c) + col, acc);
        if (!begun_before && vi == 0) p.open[atomicAdd(p.open_count, 1)] = v;
    }
}

// Tokens whose run crosses a cut: for each listed share v a block adds tail[v], head[v + 1],
// ..., up to the share that holds the run's end: row t of kJoinRows takes the shares v + t,
// v + t + kJoinRows, ... in order, then the rows' sums are added in order.  The list's order
// does not matter: every token is the sum of one entry.
constexpr int kJoinRows = 16, kJoinBlocks = 592;
__global__ void __launch_bounds__(32 * kJoinRows) join_kernel(Path p) {
    pdl_enter();
    __shared__ int s_last;
    __shared__ int64_t s_row;
    __shared__ float4 s[kJoinRows][32];
    const int count = *p.open_count;
    for (int o = blockIdx.x; o < count; o += gridDim.x) {
        const int v = p.open[o];
        if (threadIdx.y == 0) {
            const int lane = threadIdx.x;
            const int64_t s1 = (v + 1) * p.share, i1 = path_rows<32>(p, s1, lane, 0xFFFFFFFFu, 0), r = s1 - i1;
            int64_t lo = i1, hi = p.n;  // the first sorted row past the run of token r
            while (lo < hi) {
                const int64_t span = hi - lo, at = lo + span * (lane + 1) / 33;
                const int k = __popc(__ballot_sync(0xFFFFFFFFu, int64_t(p.key[at]) <= r));
                const int64_t nlo = k == 0 ? lo : lo + span * k / 33 + 1, nhi = k == 32 ? hi : lo + span * (k + 1) / 33;
                lo = nlo;
                hi = nhi;
            }
            if (lane == 0) {
                s_last = int((lo + r) / p.share);  // the share of the step that stores the token
                s_row = r;
            }
        }
        __syncthreads();
        const int last = s_last;
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
            for (int q = v + threadIdx.y; q <= last; q += kJoinRows)
                add(*reinterpret_cast<const float4 *>((q == v ? p.tail : p.head) + q * int64_t(p.c) + col));
        }
        s[threadIdx.y][threadIdx.x] = acc;
        __syncthreads();
        if (threadIdx.y == 0 && col < p.c) {
#pragma unroll
            for (int q = 1; q < kJoinRows; ++q) add(s[q][threadIdx.x]);
            *reinterpret_cast<float4 *>(p.dtable + s_row * p.c + col) =
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

// Shares of the path: enough groups for every warp slot of a B200, but at least 16 steps
// each; the numbers depend on the sizes alone.
static int path_shares(int64_t n, int64_t vocab, int c) {
    const int64_t slabs = (c / 8 + 31) / 32, want = 148 * 32 * (32 / lanes_of(c)) / slabs;
    return int(std::max<int64_t>(1, std::min<int64_t>(want, (n + vocab + 15) / 16)));
}

static int key_bits(int64_t vocab) {
    int b = 1;
    while ((int64_t(1) << b) <= vocab) ++b;  // keys 0 .. vocab
    return b;
}

struct Ws {
    uint32_t *key[2], *row[2], *counts, *totals;
    float *head, *tail;
    int32_t *open;  // the count, then the list
    size_t bytes;
    Ws(void *base, int64_t n, int64_t vocab, int c) {
        Carver cv(base);
        for (int i = 0; i < 2; ++i) {
            key[i] = cv.take<uint32_t>(size_t(n));
            row[i] = cv.take<uint32_t>(size_t(n));
        }
        counts = cv.take<uint32_t>(size_t((n + kTile - 1) / kTile) * kMaxBins);
        totals = cv.take<uint32_t>(kMaxBins);
        const size_t part = size_t(path_shares(n, vocab, c)) * size_t(c);
        head = cv.take<float>(part);
        tail = cv.take<float>(part);
        open = cv.take<int32_t>(size_t(path_shares(n, vocab, c)) + 1);
        bytes = align_up(cv.used, 256);
    }
};

template <typename T, typename I>
lat_status wgrad(const I *ids, int64_t n, const T *dy, int64_t vocab, int c, float scale, int64_t pad, float *dtable,
                 void *ws, int32_t *d_status, cudaStream_t s) {
    Ws w(ws, n, vocab, c);
    int at = 0;
    if (n > 0) {
        const int bits = key_bits(vocab), passes = (bits + kMaxBits - 1) / kMaxBits, digit = (bits + passes - 1) / passes;
        const int tiles = int((n + kTile - 1) / kTile), bins = 1 << digit;
        const Ids<I> d{ids, vocab, pad};
        for (int i = 0; i < passes; ++i) {
            const int to = i & 1;
            Pass p{i ? w.key[1 - to] : nullptr, i ? w.row[1 - to] : nullptr, w.key[to], w.row[to], w.counts, w.totals, n,
                   tiles, i * digit, digit};
            LAT_CUDA_TRY(launch_pdl(count_kernel<I>, dim3(tiles), dim3(kThreads), 0, s, p, d, i ? nullptr : d_status));
            LAT_CUDA_TRY(launch_pdl(tile_scan_kernel, dim3((bins + 31) / 32), dim3(32, 32), 0, s, w.counts, w.totals,
                                    tiles, bins, w.open));
            LAT_CUDA_TRY(launch_pdl(scatter_kernel<I>, dim3(tiles), dim3(kThreads), 0, s, p, d));
            at = to;
        }
    }
    Path p{w.key[at], w.row[at], n, vocab, 0, path_shares(n, vocab, c), c, scale, w.head, w.tail,
           w.open + 1, w.open, dtable};
    p.share = (n + vocab + p.shares - 1) / p.shares;
    const lat_status st = by_lanes(c, [&](auto l) -> lat_status {
        constexpr int L = decltype(l)::value;
        const dim3 grid(unsigned((p.shares + kThreads / L - 1) / (kThreads / L)), unsigned((c / 8 + L - 1) / L));
        LAT_CUDA_TRY(launch_pdl(sums_kernel<T, L>, grid, dim3(kThreads), 0, s, p, dy));
        return LAT_OK;
    });
    if (st != LAT_OK || n == 0) return st;
    LAT_CUDA_TRY(launch_pdl(join_kernel, dim3(unsigned(std::min(p.shares, kJoinBlocks)), unsigned((c + 127) / 128)),
                            dim3(32, kJoinRows), 0, s, p));
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
    if (!rows::aligned(table, 16) || !rows::aligned(y, 16)) return LAT_ERR_ARG;
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
    if (!rows::aligned(dy, 16) || !rows::aligned(dtable, 16)) return LAT_ERR_ARG;
    if (!ws || !rows::aligned(ws, 16) || ws_bytes < lat_embed_wgrad_ws_bytes(n, vocab, c)) return LAT_ERR_WORKSPACE;
    return embed::by_types(ids, id_bytes, dtype, [&](auto id, auto e) {
        using T = decltype(e);
        return embed::wgrad(id, n, static_cast<const T *>(dy), vocab, c, scale, pad_id, dtable, ws, d_status,
                            reinterpret_cast<cudaStream_t>(stream));
    });
}
