// kv_attend.hip -- attention over the 8-bit cache: which kernel a call gets and
// how the cache is cut, and the launches.
#include "kv_few.h"

namespace ac {

// Rows up to which a wave takes all rows and its own pages; above, the rows of
// a workgroup share a page brought to 16 bits once, in LDS.
constexpr uint64_t kFewRows = 32;

namespace {

// Pieces of the cache for few rows.  Fewer (sequence, head)s than compute units
// are cut into 1024 workgroups with 16 rows, 512 with more, so that lengths
// that differ even out.  From a workgroup a unit on, a cut costs more than it
// evens out, unless the caches are long, which 3 pieces fit best (3 workgroups
// share a unit).  128 dimensions, 8 heads, lengths down to a tenth of:
//             4096 tokens                     16,000 tokens
//   units   whole   3   4 pieces            whole   3   4 pieces
//    256     33    39    44 us               123   135   131 us
//    384     52    48    55                  210   177   195
//    504     57    60    76                  223   222   255
//    512     60    61    77                  235   227   255
//    520     66    61    81
//    768     93    92   119                  342   319   383
// and of 1000 tokens, 504 units, whole 20 us, in 3 pieces 28; with 32 rows, 504
// units of 4096, 63 and 79; of 9000 whole and 3 pieces lie within a tenth.
// With a cap or a bias, up to 16 rows and 96 or 128 dimensions, 2 pieces even out
// the second round of workgroups where the caches are whole otherwise; 8000
// tokens, those with a bias with weights, in two pieces and whole:
//   units                            264       272       304       336       384       408
//   128, lengths to a third, bias  106 105   120 139   130 144   136 150   147 163   169 171 us
//   128, lengths alike, bias       159 186   162 188   168 192   179 197   200 211   226 222
//   128, lengths to a third, cap    80  73    92 105   101 110   106 115   113 119   130 125
//    96, lengths to a third, bias   87  73    95 102   103 114   111 122   120 133   140 139
//    96, lengths to a third, cap    63  48    69  72    78  81    83  87    90  94   107  99
//    96, lengths alike, cap         95 111    96 112    98 113   101 115   110 118   129 119
// (at 288 units, lengths to a third, a cap is 2% to 7% longer in pieces).  Of 64
// dimensions a cap is up to 20% longer in pieces, a bias with weights 7% shorter
// to 9% longer; 17 to 32 rows of 320 units and more are up to 14% longer.
uint64_t few_splits(uint64_t units, uint64_t pages, uint32_t rows, uint32_t dim, bool terms) {
    if (units == 0) return 1;
    if (terms && rows == 16 && (dim == 96 || dim == 128) && units >= 272 && units <= 384 && pages > 60 && pages <= 192) return 2;
    if (units >= 256) return pages <= 192 ? 1 : 3;
    return ((rows == 16 ? 1024 : 512) + units - 1) / units;
}

// Pieces for many rows: those that should end first.  A step is a page; beside
// another workgroup on its compute unit one takes 2 us for 128 dimensions,
// alone 1.5 (above 128 dimensions it always is); a cut costs 18 us, and 1 us for
// 40 workgroups, since each writes its sums for the join (one sequence, 16
// query heads a head, 8 heads of 128, 63 pages: 128 tokens whole 96 us, in 2
// pieces 75, in 4 64, in 8 74; 256 tokens whole 106, in 4 pieces 113).  For a few
// short caches that is too much.  Trees of drafts, 8 heads of 128 x 4, with the
// pieces that this gives, twice and three times as many:
//   4 x 1000, 30 drafts   37  29  23 us     48 x 2000, 16 drafts    52  62  62 us
//   8 x 4000, 32          40  49  49        32 x 4000, 32          104  96 113
//   16 x 10,000, 25      107 116 121        2 x 131,000, 25        184 193 203
uint64_t prompt_splits(uint64_t units, uint64_t pages, uint32_t max_new, uint32_t dim) {
    const uint64_t slots = dim <= 128 ? 512 : 256;
    uint64_t best = 1, least = ~0ull;
    if (units == 0 || units >= slots) return 1;
    const uint64_t own = max_new / (2 * kKvPage), seen = pages > own ? pages - own : 1;  // by a mean row
    for (uint64_t n = 1; n <= pages && units * n <= 2 * slots; n += n / 8 + 1) {
        const uint64_t per = (pages + n - 1) / n, jobs = units * ((seen + per - 1) / per), rounds = (jobs + slots - 1) / slots;
        const uint64_t step = dim <= 128 && jobs <= 256 ? 3 : 4;  // in half microseconds of 128 dimensions
        const uint64_t cost = rounds * per * step + (n > 1 ? 36 + jobs / 20 : 0);
        if (cost < least) {
            least = cost;
            best = n;
        }
    }
    return best;
}

}  // namespace

template hipError_t launch_kv_few<kPlain>(const KvAttend &a, int codes, int dtype, hipStream_t s);

namespace {

template <int MODE>
hipError_t launch_mode(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    constexpr int kOther = MODE == kCapped ? kTerms : MODE;
    hipError_t e = a.rows > kFewRows ? launch_kv_prompt<MODE>(a, codes, dtype, s) : launch_kv_few<kOther>(a, codes, dtype, s);
    if (e == hipSuccess) e = launch_kv_finish(a, dtype, s);
    if (e == hipSuccess && a.weight && !a.scores) e = launch_kv_weigh<kOther>(a, codes, dtype, s);
    return e;
}

}  // namespace

KvAttendPlan kv_attend_plan(uint32_t batch, uint32_t heads, uint32_t group, uint32_t dim,
                            uint64_t tokens, uint32_t max_new, uint32_t max_len, bool scored, int mode) {
    KvAttendPlan p{};
    const uint64_t rows = (uint64_t)max_new * group;
    // 32 rows a wave share the codes brought to 16 bits; above 128 dimensions
    // their sums would leave no registers to load ahead
    p.rows = rows > kFewRows ? kKvPromptRows : rows <= 16 || dim > 128 ? 16 : 32;
    // Small trees: half of 128 rows would be none.  8 heads of 128, 4 query
    // heads each, 16 sequences of 5000-10,000 tokens: 9 drafts 69 us with 64
    // rows and 93 with 128, 16 drafts 82 and 100; 64 sequences of 1200-4000, 16
    // drafts 103 and 138.  (A mask alone: the kernels with a cap or a bias have 128
    // rows, and take these calls 119, 123 and 168 under a cap, 121, 123 and 171
    // with a bias; they were not made for 64.)
    if (mode == kMasked && dim <= 128 && p.rows == kKvPromptRows && rows <= kKvTreeRows) p.rows = kKvTreeRows;
    p.row_blocks = (uint32_t)((rows + p.rows - 1) / p.rows);
    const uint64_t units = (uint64_t)batch * heads * p.row_blocks;
    const uint64_t pages = (max_len + kKvPage - 1) / kKvPage;
    const bool many = p.rows > kFewRows;
    const uint64_t splits = many ? prompt_splits(units, pages, max_new, dim) : few_splits(units, pages, p.rows, dim, mode >= kCapped);
    uint64_t per = splits ? (pages + splits - 1) / splits : pages;
    // With terms short caches are whole: the join is a launch, and a call 4 us
    // longer.  7 drafts, 8 heads of 128, 2 query heads each, a call (and out of a
    // captured graph) cut and whole: 500 tokens 18.6 (11.2) and 14.3 us (9.4),
    // 1000 18.2 (12.0) and 14.1 (12.3), 2000 18.5 (12.8) and 17.5 (17.5); of 256
    // dimensions 760 tokens 18.7 (18.3) and 21.0 (20.9).
    if (mode != kPlain && !many && dim <= 128 && pages <= 16) per = pages;
    if (per < kWaves) per = kWaves;
    // a lane keeps the offset of each page of its wave
    if (!many && per > 64 * kWaves) per = 64 * kWaves;
    p.per_split = (uint32_t)per;
    p.splits = (uint32_t)((pages + per - 1) / per);
    if (p.splits < 1) p.splits = 1;
    const uint64_t all = tokens * heads * group;
    p.part_bytes = p.splits > 1 ? (p.splits * all * (dim + 2) * 4 + 255) / 256 * 256 : 0;
    // one row block keeps its scores for the weights (a write and a read of 4
    // bytes a row and token) where that is less than reading the keys again
    if (scored && rows <= 16 && rows * 8 <= dim) {
        p.score_rows = (uint32_t)rows;
        p.score_bytes = (uint64_t)batch * heads * pages * rows * kKvPage * 4;
    }
    p.sum_bytes = scored ? (all * 8 + 255) / 256 * 256 : 0;
    if (scored && !p.score_rows) {
        // A workgroup a (page, head).  Where those are fewer than compute
        // units, each takes a piece of the rows, of at least 4 turns of its
        // waves, and another launch adds up (2 x 206 tokens x 3 heads of 256,
        // 16 query heads each, 24 (page, head)s: whole 36 us, in 7 pieces 21);
        // where they are more, pieces cost what their starts take (516: whole
        // 250 us, in 4 pieces 293).
        const uint64_t cells = (uint64_t)batch * heads * pages, waves = kv_weigh_waves(dim);
        const uint64_t turns = ((rows + 15) / 16 + waves - 1) / waves, most = (turns + 3) / 4;
        uint64_t pieces = cells == 0 || cells >= 256 ? 1 : (512 + cells - 1) / cells;
        if (pieces > most) pieces = most;
        if (pieces < 1) pieces = 1;
        const uint64_t each = (turns + pieces - 1) / pieces;
        p.weigh_tiles = (uint32_t)(each * waves);
        p.weigh_pieces = (uint32_t)(turns ? (turns + each - 1) / each : 1);
        if (p.weigh_pieces > 1) p.weigh_bytes = cells * p.weigh_pieces * kKvPage * 4;
    }
    p.total = p.part_bytes + p.score_bytes + p.sum_bytes + p.weigh_bytes;
    return p;
}

hipError_t launch_kv_attend(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    switch (kv_mode(a.score_cap, a.slopes, a.mask)) {
        case kPlain: return launch_mode<kPlain>(a, codes, dtype, s);
        case kMasked: return launch_mode<kMasked>(a, codes, dtype, s);
        case kCapped: return launch_mode<kCapped>(a, codes, dtype, s);
        default: return launch_mode<kTerms>(a, codes, dtype, s);
    }
}

}  // namespace ac
