// kv.h -- the 8-bit key/value cache: the layout of a page, its number
// formats and the launches of its operators (kv_api.cpp checks arguments;
// kv_store.h, kv_turn.h, kv_few.h, kv_prompt.h, kv_weigh.h, kv_finish.hip,
// kv_evict.hip and kv_accept.hip hold the kernels).
//
// A page is one block of the arena with 64 tokens of every head.  For head h
// a strip of 2 * 64 * D bytes: 64 x D key codes, token by token, and then
// D x 64 value codes, dimension by dimension.  Behind the strips, H pairs of
// float32 scales (key, value), each a power of two of at least 2^-64.
//
// Keys lie token by token and values dimension by dimension because a matrix
// instruction wants, in each lane, consecutive elements along the axis it
// sums over: dimensions for query x key, tokens for weight x value.  Both
// codes are then fed to it as loaded, with no transpose.
#ifndef ARENA_COMPACTION_KV_H
#define ARENA_COMPACTION_KV_H
#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

namespace ac {

constexpr int kKvPage = 64;       // tokens of a page
constexpr int kKvExpMin = -64;    // least exponent of a scale
constexpr uint32_t kKvPromptRows = 128;  // query rows of a workgroup over a prompt
constexpr uint32_t kKvTreeRows = 64;     // and of one over a small tree

// An axis of a grid holds fewer than 2^32 lanes, 2^22 workgroups of 1024.
// What may need more is numbered through x, row by row of y (block_number in
// kv_device.h); the last row is filled up with workgroups that leave at once.
constexpr uint64_t kGridRow = 1u << 21;
constexpr uint64_t kMaxBlocks = 0x7FFFFFFFu;
inline dim3 grid_of(uint64_t blocks) {
    return blocks <= kGridRow ? dim3((uint32_t)blocks) : dim3((uint32_t)kGridRow, (uint32_t)((blocks + kGridRow - 1) / kGridRow));
}

// Waves of a workgroup that makes weights from the keys again.
inline __host__ __device__ constexpr uint32_t kv_weigh_waves(uint32_t dim) { return dim <= 64 ? 16 : 8; }

inline __host__ __device__ uint64_t kv_page_bytes(uint32_t heads, uint32_t dim) {
    return (uint64_t)heads * (2ull * kKvPage * dim + 8);
}

// What every operator is given: the cache, checked on the host.
struct KvCache {
    uint8_t *arena;
    uint64_t arena_bytes;
    const int64_t *pages;  // [batch][stride] byte offsets
    uint64_t stride;
    const int32_t *lens;
    uint32_t batch, heads, dim;
    unsigned long long *n_invalid;
};

struct KvAppend {
    KvCache c;
    const uint16_t *k, *v;  // 16-bit elements
    int64_t k_row, k_head, v_row, v_head;  // strides in elements
    uint64_t tokens;
    const int32_t *starts;  // batch + 1, or null: one token a sequence
    uint32_t max_new;
    float *weight;          // [batch][heads][cap], or null
    int32_t *pos;
    const int32_t *first_pos;
    uint64_t cap;
};

// Appending with rotated keys, and queries rotated beside them.
struct KvRotary : KvAppend {
    const double *freq;        // radians a position of each pair
    uint32_t rotary;           // dimensions that are rotated, two a pair
    int32_t next;              // pairs of neighbours, else of the two halves
    const int32_t *token_pos;  // tokens, or null: first_pos and the number
    const uint16_t *q;
    int64_t q_row, q_head;
    uint16_t *q_out;
    int64_t o_row, o_head;
    uint32_t q_heads;
    uint32_t lanes;            // of a workgroup
};
constexpr uint32_t kRotaryHeads = 8;  // query heads of a workgroup

struct KvAttend {
    KvCache c;
    const uint16_t *q;
    int64_t q_row, q_head;
    uint64_t tokens;
    const int32_t *starts;
    uint32_t max_new, max_len, group;
    float scale;
    uint16_t *out;   // [tokens][heads * group][dim]
    float *lse;      // [tokens][heads * group], or null
    float *weight;   // [batch][heads][cap], or null
    uint64_t cap;
    // the plan (kv_attend_plan)
    uint32_t splits, per_split;  // pieces of the cache, pages of each
    uint32_t rows;               // query rows of a workgroup
    uint32_t row_blocks;
    float *part;     // [splits][tokens * heads * group][dim + 2]
    float *scores;   // [batch][heads][score_pages][tile 4][group 4][score_rows][4], or null
    uint32_t score_pages, score_rows;
    float2 *sums;    // [tokens * heads * group]: m and 1 / sum of 2^(t - m), or null
    // weights made from the keys again: pieces of the rows, tiles of 16 rows
    // in each, and what each piece adds to a token (where there is more than one)
    uint32_t weigh_pieces, weigh_tiles;
    float *weigh_part;  // [pieces][batch][heads][score_pages][64]
    // terms beside causal softmax (null and 0 where there are none)
    const uint64_t *mask;  // [tokens][mask_words] bits
    uint64_t mask_words;
    float score_cap;       // natural units
    float cap_by;          // 2 / score_cap
    const float *slopes;   // [heads * group]
    const int32_t *pos;    // [batch][heads][pos_cap]
    uint64_t pos_cap;
};

// Which terms a kernel knows: none, the mask, the mask and a cap up to kLowCap
// (prompts alone: few rows do not gain by it), or all of them.
constexpr int kPlain = 0, kMasked = 1, kCapped = 2, kTerms = 3;
constexpr float kLowCap = 128.0f;  // above, small scores go by a form of their own (cap_scores)
inline int kv_mode(float cap, const float *slopes, const uint64_t *mask) {
    return slopes || cap > kLowCap ? kTerms : cap != 0.0f ? kCapped : mask ? kMasked : kPlain;
}

struct KvAccept {
    KvCache c;
    const int32_t *starts;  // batch + 1, or null: one token a sequence
    uint64_t tokens;
    uint32_t max_new;
    const int32_t *path;    // [batch][path_stride]
    uint64_t path_stride;
    const int32_t *kept;
    float *weight;          // [batch][heads][cap], or null
    int32_t *pos;
    uint64_t cap;
    int32_t *lens_out;
};

struct KvEvict {
    KvCache c;
    uint32_t budget, max_len;
    int32_t sink, recent;
    const int32_t *next_pos;
    const float *weight;  // [batch][heads][cap]
    const int32_t *pos;
    uint64_t cap;
    float *weight_out;    // [batch][heads][cap_out]
    int32_t *pos_out;
    uint64_t cap_out;
    int32_t *lens_out;
    // workspace (kv_evict_plan)
    int32_t *src;    // [batch][heads][budget]: a kept place, or ~(number of the hole)
    int32_t *moved;  // [batch][heads][budget]: place of the token for each hole
    int32_t *fold;   // [batch][heads]: whether anything may move
    uint8_t *rest;   // histograms of long rows
    uint32_t piece, pieces;
};

struct KvEvictPlan {
    uint64_t list_bytes, fold_bytes, rest_bytes, total;
    uint32_t piece, pieces;
};

KvEvictPlan kv_evict_plan(uint32_t batch, uint32_t heads, uint32_t budget, uint32_t max_len);

struct KvAttendPlan {
    uint32_t rows, row_blocks, splits, per_split, score_rows, weigh_pieces, weigh_tiles;
    uint64_t part_bytes, score_bytes, sum_bytes, weigh_bytes, total;
};

KvAttendPlan kv_attend_plan(uint32_t batch, uint32_t heads, uint32_t group, uint32_t dim,
                            uint64_t tokens, uint32_t max_new, uint32_t max_len, bool scored, int mode);

// Workgroups of the launches that follow from the plan.
inline uint64_t kv_prompt_blocks(uint64_t splits, uint64_t row_blocks, uint64_t heads, uint64_t batch) {
    return splits * row_blocks * heads * batch;
}
inline uint64_t kv_weigh_blocks(uint64_t pages, uint64_t pieces, uint64_t heads, uint64_t batch) {
    return pages * pieces * heads * batch;
}
constexpr uint32_t kKeptTokens = 512;  // of a workgroup that adds up kept scores
inline uint64_t kv_kept_blocks(uint64_t max_len, uint64_t heads) { return (max_len + kKeptTokens - 1) / kKeptTokens * heads; }

// Pages of a sequence that max_new tokens can touch, wherever in a page they
// begin, of those that a table's row has (at least 1: it counts what is refused).
inline uint32_t kv_append_pages(uint32_t max_new, uint64_t stride) {
    const uint64_t n = ((uint64_t)max_new + kKvPage - 2) / kKvPage + 1;
    return (uint32_t)(n < stride ? n : stride > 1 ? stride : 1);
}

// codes: 0 e4m3, 1 int8; dtype: 0 bfloat16, 1 float16
hipError_t launch_kv_append(const KvAppend &a, int codes, int dtype, hipStream_t s);
hipError_t launch_kv_append_rotary(const KvRotary &a, int codes, int dtype, hipStream_t s);
hipError_t launch_kv_accept(const KvAccept &a, int codes, hipStream_t s);
hipError_t launch_kv_attend(const KvAttend &a, int codes, int dtype, hipStream_t s);
hipError_t launch_kv_finish(const KvAttend &a, int dtype, hipStream_t s);
// (instantiated for each mode where its kernels are compiled)
template <int MODE>
hipError_t launch_kv_few(const KvAttend &a, int codes, int dtype, hipStream_t s);
template <int MODE>
hipError_t launch_kv_prompt(const KvAttend &a, int codes, int dtype, hipStream_t s);
template <int MODE>
hipError_t launch_kv_weigh(const KvAttend &a, int codes, int dtype, hipStream_t s);
hipError_t launch_kv_evict(const KvEvict &a, int codes, hipStream_t s);
hipError_t launch_kv_zero(uint64_t *p, hipStream_t s);

}  // namespace ac

#endif
