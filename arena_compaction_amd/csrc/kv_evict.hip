// kv_evict.hip -- keeps `budget` tokens of every (sequence, head).
//
// Kept are first the safe tokens (position below `sink`, or among the last
// `recent`), then those of largest weight; equal weights go to the lowest
// place, a NaN counts as +infinity.  Kept tokens inside the first `budget`
// places stay where they are; the places of dropped ones (holes) take the
// kept tokens behind the budget, both in ascending order.
//
// The order is that of a 33-bit key: the safe bit above the weight's bits,
// turned so that they ascend.  Its budget-th largest value (the edge) is
// found in three digits of 12, 11 and 10 bits, each by a histogram in LDS;
// of the tokens at the edge the first few are kept.  Then prefix sums over
// flags number the holes and the moved tokens.
//
//   k_kv_select  rows of up to 16384 tokens: one workgroup a (sequence,
//                head), keys in registers, everything in one launch;
//   k_kv_digit, k_kv_list  longer rows: a workgroup a piece of the row, a
//                launch a digit and one for the lists.  Each piece stores its
//                histogram and every piece adds up all of them, so no counter
//                has to be cleared and none is shared;
//   k_kv_fold    one workgroup a (page, head): gathers the page's 64 tokens,
//                finds the new scale and writes new codes.  Pages without a
//                hole are left alone.
// The fold is what an eviction costs: 32 sequences of up to 8190 tokens x 8
// heads of 128 cut to 4096 take 20 us to choose and 115 to fold (408 MB through
// L2: every page with a hole is read for its largest code), two of 131,000 cut
// to 32,768 take 47 and 108.  What bounds it is the latency of the strips that
// follow one another through LDS, and of the lists before them.
//
// Tokens that move lie behind the budget, and a workgroup writes its own
// strip alone: none reads what another writes.
#include "kv_device.h"

namespace ac {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kBins1 = 4096, kBins2 = 2048, kBins3 = 1024;
constexpr int kFoldThreads = 256;

// Larger weight, larger key; -0 and +0 are one key, NaN that of +infinity.
__device__ inline uint32_t weight_key(float w) {
    uint32_t u = __builtin_bit_cast(uint32_t, w + 0.0f);
    if (w != w) u = 0x7F800000u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Row {
    const float *w;
    const int32_t *pos;
    int64_t sink, border;
    __device__ bool safe(int32_t at) const { return at < sink || at >= border; }
};

__device__ inline Row row_of(const KvEvict &a, uint32_t h, uint32_t b) {
    const uint64_t at = ((uint64_t)b * a.c.heads + h) * a.cap;
    return Row{a.weight + at, a.pos + at, a.sink, (int64_t)a.next_pos[b] - a.recent};
}

// Tokens of a sequence; -1 where its length is out of range.
__device__ inline int evict_len(const KvEvict &a, uint32_t b) {
    const int64_t n = a.c.lens[b];
    return n < 0 || n > (int64_t)a.max_len ? -1 : (int)n;
}

// Exclusive prefix of x over the workgroup and the total (two barriers).
__device__ inline int block_scan(int x, int *red, int *total) {
    const int incl = wave_incl_scan(x, [](int p, int q) { return p + q; });
    __syncthreads();
    if (threadIdx.x % 64 == 63) red[threadIdx.x / 64] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < kSelWaves; ++k) {
        const int v = red[k];
        if (k < (int)(threadIdx.x / 64)) before += v;
        all += v;
    }
    *total = all;
    return before + incl - x;
}

// The bin that holds the need-th largest of the counted keys, and how many of
// its own are needed.  c: this lane's counts of bins (from the top) PER * tid
// to PER * tid + PER - 1.
template <int PER>
__device__ inline void find_bin(const int (&c)[PER], int need, int *red, int *out) {
    int sum = 0, total;
#pragma unroll
    for (int k = 0; k < PER; ++k) sum += c[k];
    int before = block_scan(sum, red, &total);
    if (before < need && need <= before + sum) {
        bool found = false;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (!found && need <= before + c[k]) {
                found = true;
                out[0] = PER * kSelThreads - 1 - (PER * (int)threadIdx.x + k);
                out[1] = need - before;
            }
            before += c[k];
        }
    }
    __syncthreads();
}

template <int BINS>
__device__ inline void find_in_lds(const uint32_t *hist, int need, int *red, int *out) {
    constexpr int PER = BINS / kSelThreads;
    int c[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) c[k] = (int)hist[BINS - 1 - (PER * (int)threadIdx.x + k)];
    find_bin<PER>(c, need, red, out);
}

__device__ inline void clear_bins(uint32_t *hist, int n) {
    for (int i = threadIdx.x; i < n; i += kSelThreads) hist[i] = 0;
}

// Rank among the set flags of the workgroup's tokens, in order of place, for
// each of a lane's KPT flags; tokens lie as (wave * KPT + k) * 64 + lane.
template <int KPT>
__device__ inline int ordered_ranks(uint32_t flags, int (&rank)[KPT], int *red) {
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const uint64_t below = (1ull << lane) - 1;
    int n = 0;
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        const uint64_t m = __builtin_amdgcn_ballot_w64((flags >> k) & 1);
        rank[k] = n + __builtin_popcountll(m & below);
        n += __builtin_popcountll(m);
    }
    __syncthreads();
    if (lane == 0) red[wave] = n;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSelWaves; ++w) {
        const int v = red[w];
        if (w < wave) before += v;
        all += v;
    }
#pragma unroll
    for (int k = 0; k < KPT; ++k) rank[k] += before;
    return all;
}

// What an edge decides: keep the keys above it and the first `ties` at it.
struct Edge {
    uint32_t safe, key;
    int ties;
};

// The lists of one block of kSelThreads * KPT tokens from place `base` on:
// flags of the kept ones, then the numbers of holes and moved tokens.
// Running totals over earlier blocks go in and out.
template <int KPT>
__device__ inline void list_block(const KvEvict &a, uint64_t row, const Row &r, int base, int end,
                                  const uint32_t (&key)[KPT], uint32_t safe, const Edge &edge,
                                  int *red, int *tied, int *holes, int *moved) {
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, K = (int)a.budget;
    uint32_t keep = 0, tie = 0, hole = 0, move = 0;
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        const int i = base + (wave * KPT + k) * 64 + lane;
        const uint32_t s = (safe >> k) & 1;
        const bool above = s > edge.safe || (s == edge.safe && key[k] > edge.key);
        if (i < end) {
            keep |= (uint32_t)above << k;
            tie |= (uint32_t)(s == edge.safe && key[k] == edge.key) << k;
        }
    }
    int rank[KPT];
    const int t = ordered_ranks<KPT>(tie, rank, red);
#pragma unroll
    for (int k = 0; k < KPT; ++k)
        if (((tie >> k) & 1) && *tied + rank[k] < edge.ties) keep |= 1u << k;
    *tied += t;
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        const int i = base + (wave * KPT + k) * 64 + lane;
        if (i < end) {
            if (i < K)
                hole |= (~(keep >> k) & 1u) << k;
            else
                move |= ((keep >> k) & 1u) << k;
        }
    }
    const int nh = ordered_ranks<KPT>(hole, rank, red);
    int32_t *src = a.src + row * a.budget, *mv = a.moved + row * a.budget;
    const uint64_t to = row * a.cap_out;
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        const int i = base + (wave * KPT + k) * 64 + lane;
        if (i < K && i < end) {
            if ((hole >> k) & 1) {
                src[i] = ~(*holes + rank[k]);
            } else {
                src[i] = i;
                a.weight_out[to + i] = r.w[i];
                a.pos_out[to + i] = r.pos[i];
            }
        }
    }
    *holes += nh;
    const int nm = ordered_ranks<KPT>(move, rank, red);
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        const int i = base + (wave * KPT + k) * 64 + lane;
        if ((move >> k) & 1) mv[*moved + rank[k]] = i;
    }
    *moved += nm;
}

template <int KPT>
__device__ inline uint32_t load_keys_of(const Row &r, int base, int end, uint32_t (&key)[KPT]) {
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    uint32_t safe = 0;
    float w[KPT];
    int32_t p[KPT];
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        const int i = base + (wave * KPT + k) * 64 + lane;
        w[k] = i < end ? r.w[i] : 0.0f;
        p[k] = i < end ? r.pos[i] : 0;
    }
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
        key[k] = weight_key(w[k]);
        safe |= (uint32_t)r.safe(p[k]) << k;
    }
    return safe;
}

// Copies a row that keeps everything.
__device__ inline void copy_row(const KvEvict &a, uint64_t row, const Row &r, int from, int to, int step) {
    for (int i = from; i < to; i += step) {
        a.weight_out[row * a.cap_out + i] = r.w[i];
        a.pos_out[row * a.cap_out + i] = r.pos[i];
    }
}

template <int KPT>
__global__ __launch_bounds__(kSelThreads) void k_kv_select(KvEvict a) {
    __shared__ int red[kSelWaves], found[2];
    __shared__ uint32_t hist[kBins1];
    const uint32_t h = blockIdx.x, b = blockIdx.y;
    const uint64_t row = (uint64_t)b * a.c.heads + h;
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64, K = (int)a.budget;
    const int n = evict_len(a, b);
    int bad_pages = 0;
    if (n > K) {
        int bad = 0;
        for (int j = tid; j * kKvPage < n; j += kSelThreads) bad += page_at(a.c, b, j) == nullptr;
        block_scan(bad, red, &bad_pages);
    }
    if (tid == 0) {
        a.fold[row] = n > K && !bad_pages;
        if (h == 0) {
            if (n < 0 || bad_pages) {
                if (a.c.n_invalid) atomicAdd(a.c.n_invalid, (unsigned long long)(bad_pages ? bad_pages : 1));
            } else {
                a.lens_out[b] = n < K ? n : K;
            }
        }
    }
    if (n < 0 || bad_pages) return;
    const Row r = row_of(a, h, b);
    if (n <= K) {
        copy_row(a, row, r, tid, n, kSelThreads);
        return;
    }
    uint32_t key[KPT];
    const uint32_t safe = load_keys_of<KPT>(r, 0, n, key);
    clear_bins(hist, kBins1);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KPT; ++k)
        if ((wave * KPT + k) * 64 + lane < n) atomicAdd(&hist[(((safe >> k) & 1) << 11) | (key[k] >> 21)], 1u);
    __syncthreads();
    find_in_lds<kBins1>(hist, K, red, found);
    const uint32_t d1 = (uint32_t)found[0];
    int need = found[1];
    Edge edge{d1 >> 11, (d1 & 2047u) << 21, 0};
    clear_bins(hist, kBins2);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KPT; ++k)
        if ((wave * KPT + k) * 64 + lane < n && ((safe >> k) & 1) == edge.safe && ((key[k] ^ edge.key) >> 21) == 0)
            atomicAdd(&hist[(key[k] >> 10) & 2047u], 1u);
    __syncthreads();
    find_in_lds<kBins2>(hist, need, red, found);
    edge.key |= (uint32_t)found[0] << 10;
    need = found[1];
    clear_bins(hist, kBins3);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KPT; ++k)
        if ((wave * KPT + k) * 64 + lane < n && ((safe >> k) & 1) == edge.safe && ((key[k] ^ edge.key) >> 10) == 0)
            atomicAdd(&hist[key[k] & 1023u], 1u);
    __syncthreads();
    find_in_lds<kBins3>(hist, need, red, found);
    edge.key |= (uint32_t)found[0];
    edge.ties = found[1];
    int tied = 0, holes = 0, moved = 0;
    list_block<KPT>(a, row, r, 0, n, key, safe, edge, red, &tied, &holes, &moved);
}

// ---- long rows, in pieces ----

constexpr int kPieceKeys = 8;
constexpr uint32_t kOneBlock = kSelThreads * 16;  // tokens k_kv_select holds
constexpr uint32_t kMaxPieces = 1026;             // of at most 32768 tokens: counts fit 16 bits

// Places [begin, end) of piece c: the first pieces cover the budget, the
// others what lies behind it.
__device__ inline void piece_range(const KvEvict &a, int c, int n, int *begin, int *end) {
    const int K = (int)a.budget, front = (K + a.piece - 1) / a.piece;
    const int64_t lo = c < front ? (int64_t)c * a.piece : K + (int64_t)(c - front) * a.piece;
    const int64_t hi = lo + a.piece, stop = c < front ? K : n;
    *begin = (int)(lo < stop ? lo : stop);
    *end = (int)(hi < stop ? hi : stop);
}

// What the launches of a long row pass on.
struct PieceState {
    int32_t bad, above;  // pages that are none; keys above the edge so far
};
struct RowState {
    int32_t d1, need1, d2, need2;
};

struct EvictWs {
    PieceState *piece;
    RowState *row;
    uint16_t *h1, *h2, *h3;
};

__host__ __device__ inline EvictWs long_ws(const KvEvict &a) {
    const uint64_t rows = (uint64_t)a.c.batch * a.c.heads, np = rows * a.pieces;
    EvictWs w;
    w.row = reinterpret_cast<RowState *>(a.rest);
    w.piece = reinterpret_cast<PieceState *>(w.row + rows);
    w.h1 = reinterpret_cast<uint16_t *>(w.piece + np);
    w.h2 = w.h1 + np * kBins1;
    w.h3 = w.h2 + np * kBins2;
    return w;
}

// Adds up the pieces' counts of this lane's bins, from the top.
template <int BINS>
__device__ inline void sum_bins(const uint16_t *h, int pieces, int (&c)[BINS / kSelThreads]) {
    constexpr int PER = BINS / kSelThreads;
    const int first = BINS - PER * ((int)threadIdx.x + 1);
#pragma unroll
    for (int k = 0; k < PER; ++k) c[k] = 0;
#pragma unroll 4
    for (int p = 0; p < pieces; ++p) {
        uint16_t v[PER];
        __builtin_memcpy(v, __builtin_assume_aligned(h + (uint64_t)p * BINS + first, PER * 2), PER * 2);
#pragma unroll
        for (int k = 0; k < PER; ++k) c[PER - 1 - k] += v[k];
    }
}

__device__ inline bool row_is_bad(const KvEvict &a, const EvictWs &w, uint64_t row, int *red) {
    int bad = 0, total;
    for (int p = threadIdx.x; p < (int)a.pieces; p += kSelThreads) bad += w.piece[row * a.pieces + p].bad;
    block_scan(bad, red, &total);
    return total != 0;
}

// One digit of the edge: DIGIT 1 counts the first, 2 and 3 find the digit
// before from the pieces' counts and count the next.
template <int DIGIT>
__global__ __launch_bounds__(kSelThreads) void k_kv_digit(KvEvict a) {
    __shared__ int red[kSelWaves], found[2];
    __shared__ uint32_t hist[kBins1];
    const uint32_t c = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const uint64_t row = (uint64_t)b * a.c.heads + h, at = row * a.pieces;
    const int tid = threadIdx.x, K = (int)a.budget;
    const int n = evict_len(a, b);
    if (n <= K) return;
    const EvictWs w = long_ws(a);
    const Row r = row_of(a, h, b);
    int begin, end;
    piece_range(a, (int)c, n, &begin, &end);
    Edge edge{0, 0, 0};
    uint32_t key[kPieceKeys];  // of the piece's first block, under way while the digit before is found
    uint32_t safe = load_keys_of<kPieceKeys>(r, begin, end, key);
    if constexpr (DIGIT == 1) {
        int bad = 0, total;
        // pages that begin in the piece (pieces and the budget are whole pages)
        for (int j = begin / kKvPage + tid; j * kKvPage < end; j += kSelThreads)
            bad += page_at(a.c, b, j) == nullptr;
        block_scan(bad, red, &total);
        if (tid == 0) w.piece[at + c] = PieceState{total, 0};
    } else {
        if (row_is_bad(a, w, row, red)) return;
        int above = 0;
        if constexpr (DIGIT == 2) {
            int v[kBins1 / kSelThreads];
            sum_bins<kBins1>(w.h1 + at * kBins1, (int)a.pieces, v);
            find_bin(v, K, red, found);
            for (int i = found[0] + 1 + tid; i < kBins1; i += kSelThreads) above += w.h1[(at + c) * kBins1 + i];
            if (c == 0 && tid == 0) {
                w.row[row].d1 = found[0];
                w.row[row].need1 = found[1];
            }
            edge.safe = (uint32_t)found[0] >> 11;
            edge.key = ((uint32_t)found[0] & 2047u) << 21;
        } else {
            const RowState s = w.row[row];
            int v[kBins2 / kSelThreads];
            sum_bins<kBins2>(w.h2 + at * kBins2, (int)a.pieces, v);
            find_bin(v, s.need1, red, found);
            for (int i = found[0] + 1 + tid; i < kBins2; i += kSelThreads) above += w.h2[(at + c) * kBins2 + i];
            if (c == 0 && tid == 0) {
                w.row[row].d2 = found[0];
                w.row[row].need2 = found[1];
            }
            edge.safe = (uint32_t)s.d1 >> 11;
            edge.key = ((uint32_t)s.d1 & 2047u) << 21 | (uint32_t)found[0] << 10;
        }
        int total;
        block_scan(above, red, &total);
        if (tid == 0) w.piece[at + c].above += total;
    }
    constexpr int kBins = DIGIT == 1 ? kBins1 : DIGIT == 2 ? kBins2 : kBins3;
    clear_bins(hist, kBins);
    __syncthreads();
    for (int base = begin; base < end; base += kSelThreads * kPieceKeys) {
        if (base != begin) safe = load_keys_of<kPieceKeys>(r, base, end, key);
#pragma unroll
        for (int k = 0; k < kPieceKeys; ++k) {
            if (base + (tid / 64 * kPieceKeys + k) * 64 + tid % 64 >= end) continue;
            const uint32_t s = (safe >> k) & 1;
            if constexpr (DIGIT == 1) {
                atomicAdd(&hist[(s << 11) | (key[k] >> 21)], 1u);
            } else if constexpr (DIGIT == 2) {
                if (s == edge.safe && ((key[k] ^ edge.key) >> 21) == 0) atomicAdd(&hist[(key[k] >> 10) & 2047u], 1u);
            } else {
                if (s == edge.safe && ((key[k] ^ edge.key) >> 10) == 0) atomicAdd(&hist[key[k] & 1023u], 1u);
            }
        }
    }
    __syncthreads();
    uint16_t *out = DIGIT == 1 ? w.h1 : DIGIT == 2 ? w.h2 : w.h3;
    uint32_t *out2 = reinterpret_cast<uint32_t *>(out + (at + c) * kBins);
    for (int i = tid; i < kBins / 2; i += kSelThreads) out2[i] = hist[2 * i] | (hist[2 * i + 1] << 16);
}

// The last digit, then a piece's part of the lists.
__global__ __launch_bounds__(kSelThreads) void k_kv_list(KvEvict a) {
    __shared__ int red[kSelWaves], found[2];
    __shared__ int kept_before[2], ties_before, above_in[kMaxPieces];
    const uint32_t c = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const uint64_t row = (uint64_t)b * a.c.heads + h, at = row * a.pieces;
    const int tid = threadIdx.x, K = (int)a.budget;
    const int n = evict_len(a, b);
    const EvictWs w = long_ws(a);
    const bool bad = n > K && row_is_bad(a, w, row, red);
    if (c == 0) {
        if (tid == 0) {
            a.fold[row] = n > K && !bad;
            if (h == 0 && n >= 0 && !bad) a.lens_out[b] = n < K ? n : K;
        }
        if (h == 0 && a.c.n_invalid) {
            if (n < 0 && tid == 0) atomicAdd(a.c.n_invalid, 1ull);
            if (bad)
                for (int p = tid; p < (int)a.pieces; p += kSelThreads)
                    if (w.piece[at + p].bad) atomicAdd(a.c.n_invalid, (unsigned long long)w.piece[at + p].bad);
        }
    }
    if (n < 0 || bad) return;
    const Row r = row_of(a, h, b);
    if (n <= K) {
        copy_row(a, row, r, (int)c * kSelThreads + tid, n, (int)a.pieces * kSelThreads);
        return;
    }
    const RowState s = w.row[row];
    int v[1];
    sum_bins<kBins3>(w.h3 + at * kBins3, (int)a.pieces, v);
    find_bin(v, s.need2, red, found);
    const int d3 = found[0];
    const Edge edge{(uint32_t)s.d1 >> 11, ((uint32_t)s.d1 & 2047u) << 21 | (uint32_t)s.d2 << 10 | (uint32_t)d3, found[1]};
    // what earlier pieces keep: keys above the edge, and of the ties the
    // first; `front` pieces give holes, the others moved tokens
    const int front = (K + a.piece - 1) / a.piece;
    for (int p = tid / 64; p < (int)c; p += kSelWaves) {
        int above = 0;
        for (int i = d3 + 1 + tid % 64; i < kBins3; i += 64) above += w.h3[(at + p) * kBins3 + i];
        above = wave_reduce(above, [](int x, int y) { return x + y; });
        if (tid % 64 == 0) above_in[p] = w.piece[at + p].above + above;
    }
    __syncthreads();
    if (tid < 64) {
        int tied = 0, kept[2] = {0, 0};
        // one wave, a piece a lane; ties in order through a prefix
        for (int p0 = 0; p0 < (int)c; p0 += 64) {
            const int p = p0 + tid;
            int above = 0, ties = 0;
            if (p < (int)c) {
                above = above_in[p];
                ties = w.h3[(at + p) * kBins3 + d3];
            }
            const int incl = wave_incl_scan(ties, [](int x, int y) { return x + y; });
            const int before = tied + incl - ties, left = edge.ties > before ? edge.ties - before : 0;
            const int k = p < (int)c ? above + (ties < left ? ties : left) : 0;
            kept[0] += wave_reduce(p < front ? k : 0, [](int x, int y) { return x + y; });
            kept[1] += wave_reduce(p >= front ? k : 0, [](int x, int y) { return x + y; });
            tied += read_lane<63>(incl);
        }
        if (tid == 0) {
            ties_before = tied;
            kept_before[0] = kept[0];
            kept_before[1] = kept[1];
        }
    }
    __syncthreads();
    int begin, end, tied = ties_before;
    piece_range(a, (int)c, n, &begin, &end);
    int holes = (int)c < front ? begin - kept_before[0] : 0, moved = kept_before[1];
    for (int base = begin; base < end; base += kSelThreads * kPieceKeys) {
        uint32_t key[kPieceKeys];
        const uint32_t safe = load_keys_of<kPieceKeys>(r, base, end, key);
        list_block<kPieceKeys>(a, row, r, base, end, key, safe, edge, red, &tied, &holes, &moved);
    }
}

// Old scale over new one.  Every code but 0 and NaN fits the new scale, so its
// quotient is at most 448 / 2^-9; a kept token of zeros may come from a page
// whose scale is any number of powers larger, and has to stay zeros where the
// quotient would be infinite.
__device__ inline float scale_quotient(float was, float inv) { return fminf(was * inv, 0x1p18f); }

// A value code stands alone in its 64 bytes: a token's are D such rows apart.
// Read byte by byte from memory, every lane would cost L1 an access of its
// own (163 us for 32 x 8190 tokens cut to 4096, where this takes 115), so
// the strips that hold the page's tokens pass through LDS whole, one after the
// other -- few, since moved tokens lie in order -- and bytes are picked there.
// Keys and values of a page are two workgroups: each waits for little, and
// more of them are under way.
template <int D, int CODES>
__global__ __launch_bounds__(kFoldThreads) void k_kv_fold(KvEvict a) {
    __shared__ u32x2 sm_v[2][D * kKvPage / 8];
    __shared__ uint64_t strip_of[kKvPage];
    __shared__ int place[kKvPage];
    __shared__ float scale[kKvPage];
    __shared__ float red[kFoldThreads / 64];
    // neighbouring pages on one of the 8 XCDs: they take tokens from the same
    // strips, which its L2 then holds
    const uint32_t pages = gridDim.x / 2, x = blockIdx.x % pages, per_xcd = pages / 8;
    const bool values = blockIdx.x < pages;
    const uint32_t j = pages % 8 ? x : x % 8 * per_xcd + x / 8;
    const uint32_t h = blockIdx.y, b = blockIdx.z;
    const uint64_t row = (uint64_t)b * a.c.heads + h;
    const int tid = threadIdx.x, lane = tid % 64;
    // every wave: token `lane` of the page, where it comes from
    const int own = (int)(j * kKvPage) + lane;
    if (!a.fold[row]) return;
    int s = a.src[row * a.budget + own];
    if (__builtin_amdgcn_ballot_w64(s != own) == 0) return;
    if (s < 0) {
        s = a.moved[row * a.budget + ~s];
        if (!values && tid < kKvPage) {
            a.weight_out[row * a.cap_out + own] = a.weight[row * a.cap + s];
            a.pos_out[row * a.cap_out + own] = a.pos[row * a.cap + s];
        }
    }
    const int from = s / kKvPage;
    const uint64_t stay = __builtin_amdgcn_ballot_w64(s == own);
    const uint64_t page = page_offset(a.c, b, from), strip = page + (uint64_t)h * 2 * kKvPage * D;
    const uint64_t base = page_offset(a.c, b, j);
    float *sc = page_scales(a.c, a.c.arena + base, h);
    uint8_t *kc = a.c.arena + base + (uint64_t)h * 2 * kKvPage * D, *vc = kc + kKvPage * D;
    if (tid < kKvPage) {
        place[tid] = s % kKvPage;
        scale[tid] = page_scales(a.c, a.c.arena + page, h)[values];
        strip_of[tid] = strip;
    }
    constexpr int kK = D / 32, kV = D / 16, kPer = D / 8;
    float most = 0.0f;
    if (!values) {  // 8 dimensions of a token a lane
        const int e_was = exp_of_pow2(sc[0]);
        __syncthreads();
        u32x2 kw[kK];
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            const int item = tid + i * kFoldThreads, t = item / kPer, d = item % kPer * 8;
            kw[i] = *reinterpret_cast<const u32x2 *>(a.c.arena + strip_of[t] + place[t] * D + d);
        }
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            ByteMax m;
            byte_max<CODES>(m, kw[i][0]);
            byte_max<CODES>(m, kw[i][1]);
            const uint32_t two = max_u16x2(m.even, m.odd), top = two >> 16 > (two & 0xFFFFu) ? two >> 16 : two & 0xFFFFu;
            most = fmaxf(most, magnitude<CODES>(top) * scale[(tid + i * kFoldThreads) / kPer]);
        }
        most = wave_max0(most);
        if (lane == 0) red[tid / 64] = most;
        __syncthreads();  // all of the page's keys have been read, too
        most = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const int e = scale_exp<CODES>(most);
        const float inv = pow2(-e);
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            const int item = tid + i * kFoldThreads, t = item / kPer, d = item % kPer * 8;
            // at the page's old scale, tokens that stay keep their codes
            if (e == e_was && ((stay >> t) & 1)) continue;
            const float f = scale_quotient(scale[t], inv);
            u32x2 w = kw[i];
            if (f != 1.0f) {
                w[0] = requant4<CODES>(w[0], f);
                w[1] = requant4<CODES>(w[1], f);
            }
            *reinterpret_cast<u32x2 *>(kc + t * D + d) = w;
        }
        if (tid == 0) sc[0] = pow2(e);
        return;
    }
    // 4 tokens of a dimension a lane, its tokens the same for all of its dimensions
    u32x2 raw[kK];
    uint32_t vw[kV] = {};
    const int t0 = tid % 16 * 4, dv = tid / 16;
    uint64_t todo = ~0ull;
    auto load = [&](int at) __attribute__((always_inline)) {
        const uint8_t *p = a.c.arena + lane_u64(strip, at) + kKvPage * D;
#pragma unroll
        for (int i = 0; i < kK; ++i) raw[i] = reinterpret_cast<const u32x2 *>(p)[tid + i * kFoldThreads];
    };
    load(0);
    int cur = 0, at = 0;
    while (todo) {
        const uint64_t here = __builtin_amdgcn_ballot_w64(from == __builtin_amdgcn_readlane(from, at));
        todo &= ~here;
#pragma unroll
        for (int i = 0; i < kK; ++i) sm_v[cur][tid + i * kFoldThreads] = raw[i];
        at = todo ? __builtin_ctzll(todo) : at;
        load(at);  // the last one once more
        __syncthreads();
        const uint32_t mine = (uint32_t)(here >> t0) & 15u;
        const uint8_t *bytes = reinterpret_cast<const uint8_t *>(sm_v[cur]) + dv * kKvPage;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if ((mine >> e) & 1) {
                const uint8_t *p = bytes + place[t0 + e];
#pragma unroll
                for (int i = 0; i < kV; ++i) vw[i] |= (uint32_t)p[i * 16 * kKvPage] << (8 * e);
            }
        }
        cur ^= 1;  // filled again only behind the next barrier, which follows these reads
    }
    const float g[4] = {scale[t0], scale[t0 + 1], scale[t0 + 2], scale[t0 + 3]};
    ByteMax m;
#pragma unroll
    for (int i = 0; i < kV; ++i) byte_max<CODES>(m, vw[i]);
    most = fmaxf(fmaxf(magnitude<CODES>(m.even & 255u) * g[0], magnitude<CODES>(m.odd & 255u) * g[1]),
                 fmaxf(magnitude<CODES>(m.even >> 16) * g[2], magnitude<CODES>(m.odd >> 16) * g[3]));
    most = wave_max0(most);
    if (lane == 0) red[tid / 64] = most;
    __syncthreads();
    most = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const int e = scale_exp<CODES>(most);
    const float inv = pow2(-e);
    // codes of a scale that stays are the new ones as they are
    const float f[4] = {scale_quotient(g[0], inv), scale_quotient(g[1], inv), scale_quotient(g[2], inv),
                        scale_quotient(g[3], inv)};
    if (f[0] != 1.0f || f[1] != 1.0f || f[2] != 1.0f || f[3] != 1.0f) {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            vw[i] = to_codes4<CODES>(code_value<CODES, 0>(vw[i]) * f[0], code_value<CODES, 1>(vw[i]) * f[1],
                                     code_value<CODES, 2>(vw[i]) * f[2], code_value<CODES, 3>(vw[i]) * f[3]);
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) *reinterpret_cast<uint32_t *>(vc + (dv + i * 16) * kKvPage + t0) = vw[i];
    if (tid == 0) sc[1] = pow2(e);
}

template <int D>
void fold_go(const KvEvict &a, int codes, hipStream_t s) {
    const dim3 grid(2 * (a.budget / kKvPage), a.c.heads, a.c.batch);
    if (codes == kE4m3)
        hipLaunchKernelGGL((k_kv_fold<D, kE4m3>), grid, dim3(kFoldThreads), 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_fold<D, kInt8>), grid, dim3(kFoldThreads), 0, s, a);
}

}  // namespace

KvEvictPlan kv_evict_plan(uint32_t batch, uint32_t heads, uint32_t budget, uint32_t max_len) {
    KvEvictPlan p{};
    const uint64_t rows = (uint64_t)batch * heads;
    p.list_bytes = rows * budget * 4;
    p.fold_bytes = (rows * 4 + 255) / 256 * 256;
    if (max_len > kOneBlock) {
        const uint32_t behind = max_len > budget ? max_len - budget : 0;
        p.piece = kSelThreads * kPieceKeys;
        for (;;) {
            p.pieces = (budget + p.piece - 1) / p.piece + (behind + p.piece - 1) / p.piece;
            if (p.pieces <= kMaxPieces) break;
            p.piece *= 2;
        }
        p.rest_bytes = rows * sizeof(RowState) +
                       rows * p.pieces * (sizeof(PieceState) + 2 * (kBins1 + kBins2 + kBins3));
    }
    p.total = 2 * p.list_bytes + p.fold_bytes + p.rest_bytes;
    return p;
}

hipError_t launch_kv_evict(const KvEvict &a, int codes, hipStream_t s) {
    if (a.max_len <= kOneBlock) {
        const dim3 grid(a.c.heads, a.c.batch);
        if (a.max_len <= kOneBlock / 2)
            hipLaunchKernelGGL((k_kv_select<8>), grid, dim3(kSelThreads), 0, s, a);
        else
            hipLaunchKernelGGL((k_kv_select<16>), grid, dim3(kSelThreads), 0, s, a);
    } else {
        const dim3 grid(a.pieces, a.c.heads, a.c.batch);
        hipLaunchKernelGGL((k_kv_digit<1>), grid, dim3(kSelThreads), 0, s, a);
        hipLaunchKernelGGL((k_kv_digit<2>), grid, dim3(kSelThreads), 0, s, a);
        hipLaunchKernelGGL((k_kv_digit<3>), grid, dim3(kSelThreads), 0, s, a);
        hipLaunchKernelGGL(k_kv_list, grid, dim3(kSelThreads), 0, s, a);
    }
    if (a.max_len <= a.budget) return hipGetLastError();  // nothing can move
    switch (a.c.dim) {
        case 64: fold_go<64>(a, codes, s); break;
        case 96: fold_go<96>(a, codes, s); break;
        case 128: fold_go<128>(a, codes, s); break;
        case 192: fold_go<192>(a, codes, s); break;
        case 256: fold_go<256>(a, codes, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace ac
