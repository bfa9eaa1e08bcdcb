// kv_api.cpp -- the C-ABI entry points of the 8-bit key/value cache:
// argument checks, workspace layout, launches and error mapping.
#include "../../include/arena_compaction.h"
#include "kv.h"

using namespace ac;

namespace {

constexpr uint64_t kMaxTokens = 1u << 29;  // tokens of a call, places of a table's row
constexpr uint64_t kMaxGrid = (1u << 24) - 1;  // workgroups of 256 along one axis
constexpr uint64_t kMaxHeadRows = 0x7FFFFC00u;  // query rows of a (sequence, head): the kernels hold them in an int
constexpr uint64_t kMaxRows = 1ull << 36;       // query rows of a call: sizes in bytes stay below 2^64
constexpr uint64_t kMaxEvict = 1u << 25;  // tokens of an evicted sequence
constexpr uint64_t kMaxMaskWords = kMaxTokens / 64;
constexpr float kLeastCap = 0x1p-64f, kMostCap = 0x1p64f;  // so that its inverse is a number
constexpr uint64_t kMaxPath = 1ull << 32;  // entries of a row: sizes in bytes stay below 2^64
constexpr uint64_t kLeastWs = 1;  // none is needed: 0 means "refused"

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Bytes of memory; of no bytes or no address they overlap nothing.
struct Span {
    const void *p;
    unsigned __int128 bytes;
};

// The used part of rows x (stride of them apart) numbers of 4 bytes.
Span plane(const void *p, uint64_t rows, uint64_t stride, uint64_t used) {
    return Span{p, rows && used ? ((unsigned __int128)(rows - 1) * stride + used) * 4 : 0};
}

bool overlap(const Span &a, const Span &b) {
    const auto x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x && y && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

// From the first to the last of tokens x heads x dim numbers of 2 bytes.
Span strided(const void *p, uint64_t tokens, int64_t row, uint64_t heads, int64_t head, uint32_t dim) {
    if (!p || !tokens || !heads) return Span{nullptr, 0};
    const __int128 r = (__int128)(tokens - 1) * row, h = (__int128)(heads - 1) * head;
    const __int128 lo = (r < 0 ? r : 0) + (h < 0 ? h : 0), hi = (r > 0 ? r : 0) + (h > 0 ? h : 0) + dim;
    return Span{reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(p) + (intptr_t)(lo * 2)), (unsigned __int128)(hi - lo) * 2};
}

// Whether no two rows of tokens x heads x dim numbers share memory: one stride
// steps over all that the other reaches.
bool rows_apart(uint64_t tokens, int64_t row, uint64_t heads, int64_t head, uint32_t dim) {
    const __int128 r = row < 0 ? -(__int128)row : row, h = head < 0 ? -(__int128)head : head;
    const __int128 of_heads = (__int128)(heads - 1) * h + dim, of_tokens = (__int128)(tokens - 1) * r + dim;
    const bool token_by_token = (heads == 1 || h >= dim) && (tokens == 1 || r >= of_heads);
    const bool head_by_head = (tokens == 1 || r >= dim) && (heads == 1 || h >= of_tokens);
    return token_by_token || head_by_head;
}

// tokens x heads x dim numbers of 2 bytes.
struct Rows {
    const void *p;
    uint64_t tokens;
    int64_t row;
    uint64_t heads;
    int64_t head;
    uint32_t dim;
    Span span() const { return strided(p, tokens, row, heads, head, dim); }
};

// Whether intervals of x and y numbers, `apart` bytes from the one's start to
// the other's, share any when both are repeated every `step` numbers.
bool repeated_overlap(__int128 apart, __int128 x, __int128 y, int64_t stride) {
    const __int128 step = stride < 0 ? -(__int128)stride : stride;
    if (step == 0 || apart % 2) return true;
    const __int128 at = (apart / 2 % step + step) % step;
    return at < x || at + y > step;
}

// Whether two sets of rows share memory, or cannot be seen not to: slices of
// one fused projection lie between one another's rows, or heads, the same
// stride apart.
bool rows_overlap(const Rows &a, const Rows &b) {
    if (!overlap(a.span(), b.span())) return false;
    const auto at = [](const Span &s) { return (__int128)reinterpret_cast<uintptr_t>(s.p); };
    const bool same_row = a.tokens > 1 && b.tokens > 1 && (b.row == a.row || b.row == -a.row);
    const bool same_head = a.heads > 1 && b.heads > 1 && (b.head == a.head || b.head == -a.head);
    if (same_row) {
        const Span x = Rows{a.p, 1, 0, a.heads, a.head, a.dim}.span(), y = Rows{b.p, 1, 0, b.heads, b.head, b.dim}.span();
        if (!repeated_overlap(at(y) - at(x), (__int128)x.bytes / 2, (__int128)y.bytes / 2, a.row)) return false;
    }
    if (same_head && ((a.tokens == 1 && b.tokens == 1) || (same_row && a.head && a.row % a.head == 0)))
        return repeated_overlap((__int128)reinterpret_cast<uintptr_t>(b.p) - (__int128)reinterpret_cast<uintptr_t>(a.p), a.dim, b.dim, a.head);
    return true;
}

// Whether outputs overlap one another or an input.
template <size_t OUT, size_t IN>
bool any_overlap(const Span (&out)[OUT], const Span (&in)[IN]) {
    for (size_t i = 0; i < OUT; ++i) {
        for (size_t j = i + 1; j < OUT; ++j)
            if (overlap(out[i], out[j])) return true;
        for (const Span &x : in)
            if (overlap(out[i], x)) return true;
    }
    return false;
}

bool dim_ok(uint32_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

// The parts of a cache that every call needs; lens_dev and pages_dev may be
// null only where there is no sequence.
int check_cache(const defrag_kv_cache *c) {
    if (!c) return DEFRAG_EINVAL;
    if (c->batch > 65535 || c->heads < 1 || c->heads > 65535 || !dim_ok(c->dim)) return DEFRAG_EINVAL;
    if (c->codes != DEFRAG_KV_E4M3 && c->codes != DEFRAG_KV_INT8) return DEFRAG_EINVAL;
    if (c->page_stride * kKvPage > kMaxTokens || c->page_stride > kMaxTokens) return DEFRAG_EINVAL;
    if (!aligned(c->arena_dev, 32) || !aligned(c->pages_dev, 8) || !aligned(c->lens_dev, 4) ||
        !aligned(c->n_invalid_dev, 8))
        return DEFRAG_EINVAL;
    if (c->batch && (!c->lens_dev || (c->page_stride && !c->pages_dev))) return DEFRAG_EINVAL;
    if (c->arena_bytes && !c->arena_dev) return DEFRAG_EINVAL;
    return DEFRAG_OK;
}

KvCache cache_of(const defrag_kv_cache *c) {
    return KvCache{static_cast<uint8_t *>(c->arena_dev), c->arena_bytes, c->pages_dev, c->page_stride,
                   c->lens_dev, c->batch, c->heads, c->dim,
                   reinterpret_cast<unsigned long long *>(c->n_invalid_dev)};
}

int dtype_ok(int32_t t) { return t == DEFRAG_KV_BF16 || t == DEFRAG_KV_FP16; }

int check_new(const defrag_kv_cache *c, const int32_t *starts, uint64_t tokens, uint32_t max_new) {
    if (tokens > kMaxTokens || !aligned(starts, 4)) return DEFRAG_EINVAL;
    if (!starts && tokens != c->batch) return DEFRAG_EINVAL;
    if (tokens && (c->batch == 0 || max_new == 0)) return DEFRAG_EINVAL;
    if (max_new > tokens) return DEFRAG_EINVAL;
    return DEFRAG_OK;
}

int check_append(const defrag_kv_append_args *a) {
    if (!a) return DEFRAG_EINVAL;
    int rc = check_cache(a->cache);
    if (rc) return rc;
    const defrag_kv_cache *c = a->cache;
    rc = check_new(c, a->starts_dev, a->tokens, a->max_new);
    if (rc) return rc;
    if (!dtype_ok(a->dtype) || !aligned(a->k_dev, 2) || !aligned(a->v_dev, 2) ||
        !aligned(a->weight_dev, 4) || !aligned(a->pos_dev, 4) || !aligned(a->first_pos_dev, 4))
        return DEFRAG_EINVAL;
    if (a->tokens && (!a->k_dev || !a->v_dev)) return DEFRAG_EINVAL;
    if ((uint64_t)kv_append_pages(a->max_new, c->page_stride) * 2 * c->dim > 0xFFFFFFFFu) return DEFRAG_EINVAL;
    // (every head writes its own rows of the planes, and reads all of these)
    const uint64_t rows = (uint64_t)c->batch * c->heads;
    const Span out[] = {plane(a->weight_dev, rows, a->weight_stride, a->weight_stride),
                        plane(a->pos_dev, rows, a->weight_stride, a->weight_stride)};
    const Span in[] = {strided(a->k_dev, a->tokens, a->k_row, c->heads, a->k_head, c->dim),
                       strided(a->v_dev, a->tokens, a->v_row, c->heads, a->v_head, c->dim),
                       plane(a->first_pos_dev, 1, 0, c->batch), plane(a->starts_dev, 1, 0, c->batch + 1ull),
                       plane(c->lens_dev, 1, 0, c->batch), plane(c->pages_dev, 1, 0, 2 * c->batch * c->page_stride)};
    return any_overlap(out, in) ? DEFRAG_EINVAL : DEFRAG_OK;
}

KvAppend append_of(const defrag_kv_append_args *a) {
    return KvAppend{cache_of(a->cache),
                    static_cast<const uint16_t *>(a->k_dev), static_cast<const uint16_t *>(a->v_dev),
                    a->k_row, a->k_head, a->v_row, a->v_head, a->tokens, a->starts_dev, a->max_new,
                    a->weight_dev, a->pos_dev, a->first_pos_dev, a->weight_stride};
}

int check_rotary(const defrag_kv_rotary_args *r) {
    if (!r) return DEFRAG_EINVAL;
    const defrag_kv_append_args *a = r->append;
    const int rc = check_append(a);
    if (rc) return rc;
    const defrag_kv_cache *c = a->cache;
    if (r->rotary_dim < 8 || r->rotary_dim % 8 || r->rotary_dim > c->dim || (r->interleaved != 0 && r->interleaved != 1))
        return DEFRAG_EINVAL;
    if (!aligned(r->freq_dev, 8) || !aligned(r->token_pos_dev, 4) || !aligned(r->q_dev, 2) || !aligned(r->out_dev, 2))
        return DEFRAG_EINVAL;
    if (a->tokens && (!r->freq_dev || (r->q_heads && (!r->q_dev || !r->out_dev)))) return DEFRAG_EINVAL;
    if (c->heads + ((uint64_t)r->q_heads + kRotaryHeads - 1) / kRotaryHeads > 65535 || a->tokens * r->q_heads > kMaxRows)
        return DEFRAG_EINVAL;
    const uint64_t rows = (uint64_t)c->batch * c->heads;
    const Span planes[] = {plane(a->weight_dev, rows, a->weight_stride, a->weight_stride),
                           plane(a->pos_dev, rows, a->weight_stride, a->weight_stride)};
    const Span read[] = {plane(r->freq_dev, 1, 0, r->rotary_dim), plane(r->token_pos_dev, 1, 0, a->tokens),
                         strided(r->q_dev, a->tokens, r->q_row, r->q_heads, r->q_head, c->dim)};
    if (any_overlap(planes, read)) return DEFRAG_EINVAL;
    if (!a->tokens || !r->q_heads) return DEFRAG_OK;
    if (!rows_apart(a->tokens, r->out_row, r->q_heads, r->out_head, c->dim)) return DEFRAG_EINVAL;
    const Rows to{r->out_dev, a->tokens, r->out_row, r->q_heads, r->out_head, c->dim};
    const Rows q{r->q_dev, a->tokens, r->q_row, r->q_heads, r->q_head, c->dim};
    const Rows k{a->k_dev, a->tokens, a->k_row, c->heads, a->k_head, c->dim}, v{a->v_dev, a->tokens, a->v_row, c->heads, a->v_head, c->dim};
    const bool same = r->out_dev == r->q_dev && (a->tokens == 1 || r->out_row == r->q_row) && (r->q_heads == 1 || r->out_head == r->q_head);
    if ((!same && rows_overlap(to, q)) || rows_overlap(to, k) || rows_overlap(to, v)) return DEFRAG_EINVAL;
    const Span out[] = {to.span()};
    const Span in[] = {Span{c->arena_dev, c->arena_bytes}, planes[0], planes[1], read[0], read[1], plane(a->first_pos_dev, 1, 0, c->batch),
                       plane(a->starts_dev, 1, 0, c->batch + 1ull), plane(c->lens_dev, 1, 0, c->batch),
                       plane(c->pages_dev, 1, 0, 2 * c->batch * c->page_stride)};
    return any_overlap(out, in) ? DEFRAG_EINVAL : DEFRAG_OK;
}

int check_accept(const defrag_kv_accept_args *a) {
    if (!a) return DEFRAG_EINVAL;
    int rc = check_cache(a->cache);
    if (rc) return rc;
    const defrag_kv_cache *c = a->cache;
    rc = check_new(c, a->starts_dev, a->tokens, a->max_new);
    if (rc) return rc;
    if (a->path_stride > kMaxPath || !aligned(a->path_dev, 4) || !aligned(a->kept_dev, 4) || !aligned(a->weight_dev, 4) ||
        !aligned(a->pos_dev, 4) || !aligned(a->lens_out_dev, 4))
        return DEFRAG_EINVAL;
    if (c->batch && (!a->kept_dev || !a->lens_out_dev || (a->path_stride && !a->path_dev))) return DEFRAG_EINVAL;
    const uint64_t rows = (uint64_t)c->batch * c->heads;
    const Span out[] = {plane(a->lens_out_dev, 1, 0, c->batch), plane(a->weight_dev, rows, a->weight_stride, a->weight_stride),
                        plane(a->pos_dev, rows, a->weight_stride, a->weight_stride), Span{c->arena_dev, c->arena_bytes}};
    const Span in[] = {plane(c->lens_dev, 1, 0, c->batch), plane(a->starts_dev, 1, 0, c->batch + 1ull),
                       plane(a->path_dev, c->batch, a->path_stride, a->path_stride), plane(a->kept_dev, 1, 0, c->batch),
                       plane(c->pages_dev, 1, 0, 2 * c->batch * c->page_stride)};
    return any_overlap(out, in) ? DEFRAG_EINVAL : DEFRAG_OK;
}

KvAttendPlan plan_of(const defrag_kv_attend_args *a, int mode) {
    return kv_attend_plan(a->cache->batch, a->cache->heads, a->group, a->cache->dim, a->tokens,
                          a->max_new, a->max_len, a->weight_dev != nullptr, mode);
}

// The plan of a call, and whether its launches fit their grids.  (Rows are
// joined by a workgroup each at the most, where the cache is cut: fewer than
// 2^21 of them, as kv_attend_plan cuts few rows or few workgroups.)
int check_attend(const defrag_kv_attend_args *a, KvAttendPlan *p, int mode = kPlain) {
    if (!a) return DEFRAG_EINVAL;
    int rc = check_cache(a->cache);
    if (rc) return rc;
    const defrag_kv_cache *c = a->cache;
    rc = check_new(c, a->starts_dev, a->tokens, a->max_new);
    if (rc) return rc;
    if (!dtype_ok(a->dtype) || a->group < 1 || a->group > 256 ||
        (uint64_t)c->heads * a->group > 65535 || a->max_len > c->page_stride * kKvPage)
        return DEFRAG_EINVAL;
    if ((uint64_t)a->max_new * a->group > kMaxHeadRows || a->tokens * c->heads * a->group > kMaxRows)
        return DEFRAG_EINVAL;
    if (!(a->scale - a->scale == 0.0f)) return DEFRAG_EINVAL;  // not finite
    if (!aligned(a->q_dev, 2) || !aligned(a->out_dev, 16) || !aligned(a->lse_dev, 4) ||
        !aligned(a->weight_dev, 4))
        return DEFRAG_EINVAL;
    if (a->tokens && (!a->q_dev || !a->out_dev)) return DEFRAG_EINVAL;
    if (a->weight_dev && a->weight_stride < a->max_len) return DEFRAG_EINVAL;
    const uint64_t q_heads = (uint64_t)c->heads * a->group, rows = a->tokens * q_heads;
    const Span out[] = {plane(a->out_dev, 1, 0, rows * c->dim / 2), plane(a->lse_dev, 1, 0, rows),
                        plane(a->weight_dev, (uint64_t)c->batch * c->heads, a->weight_stride, a->max_len)};
    const Span in[] = {strided(a->q_dev, a->tokens, a->q_row, q_heads, a->q_head, c->dim),
                       plane(a->starts_dev, 1, 0, c->batch + 1ull), plane(c->lens_dev, 1, 0, c->batch),
                       plane(c->pages_dev, 1, 0, 2 * c->batch * c->page_stride)};
    if (any_overlap(out, in)) return DEFRAG_EINVAL;
    *p = KvAttendPlan{};
    if (!a->tokens) return DEFRAG_OK;
    *p = plan_of(a, mode);
    if (p->rows >= kKvTreeRows && kv_prompt_blocks(p->splits, p->row_blocks, c->heads, c->batch) > kMaxBlocks)
        return DEFRAG_EINVAL;
    const uint64_t pages = (a->max_len + (uint64_t)kKvPage - 1) / kKvPage;
    if (a->weight_dev && !p->score_bytes && kv_weigh_blocks(pages, p->weigh_pieces, c->heads, c->batch) > kMaxBlocks)
        return DEFRAG_EINVAL;
    if (p->score_bytes && kv_kept_blocks(a->max_len, c->heads) + (uint64_t)a->max_new * c->heads * a->group > kMaxGrid)
        return DEFRAG_EINVAL;
    return DEFRAG_OK;
}

// The same with terms; a call without any is defrag_kv_attend's.
int check_terms(const defrag_kv_attend_args *a, const defrag_kv_terms *t, KvAttendPlan *p) {
    if (!t) return DEFRAG_EINVAL;
    const int rc = check_attend(a, p, kv_mode(t->cap, t->slopes_dev, t->mask_dev));
    if (rc) return rc;
    const defrag_kv_cache *c = a->cache;
    if (t->cap != 0.0f && !(t->cap >= kLeastCap && t->cap <= kMostCap)) return DEFRAG_EINVAL;
    if (!aligned(t->mask_dev, 8) || !aligned(t->slopes_dev, 4) || !aligned(t->pos_dev, 4)) return DEFRAG_EINVAL;
    if (t->mask_dev && (t->mask_words > kMaxMaskWords || t->mask_words * 64 < a->max_new)) return DEFRAG_EINVAL;
    const uint64_t places = (a->max_len + (uint64_t)kKvPage - 1) / kKvPage * kKvPage;
    if (t->pos_dev && (t->pos_stride < places || t->pos_stride > kMaxTokens)) return DEFRAG_EINVAL;
    const uint64_t q_heads = (uint64_t)c->heads * a->group, rows = a->tokens * q_heads, units = (uint64_t)c->batch * c->heads;
    const Span out[] = {plane(a->out_dev, 1, 0, rows * c->dim / 2), plane(a->lse_dev, 1, 0, rows),
                        plane(a->weight_dev, units, a->weight_stride, a->max_len)};
    const Span in[] = {plane(t->mask_dev, 1, 0, 2 * a->tokens * t->mask_words), plane(t->slopes_dev, 1, 0, q_heads),
                       plane(t->pos_dev, units, t->pos_stride, places)};
    return any_overlap(out, in) ? DEFRAG_EINVAL : DEFRAG_OK;
}

int check_evict(const defrag_kv_evict_args *a) {
    if (!a) return DEFRAG_EINVAL;
    const int rc = check_cache(a->cache);
    if (rc) return rc;
    const defrag_kv_cache *c = a->cache;
    if (a->budget == 0 || a->budget % kKvPage || a->budget > kMaxEvict || a->max_len > kMaxEvict)
        return DEFRAG_EINVAL;
    if (a->max_len > c->page_stride * kKvPage ||
        a->max_len > a->weight_stride || a->recent < 0)
        return DEFRAG_EINVAL;
    const uint64_t kept = a->budget < a->max_len ? a->budget : a->max_len;
    if (a->weight_out_stride < kept) return DEFRAG_EINVAL;
    if (!aligned(a->weight_dev, 4) || !aligned(a->pos_dev, 4) || !aligned(a->next_pos_dev, 4) ||
        !aligned(a->weight_out_dev, 4) || !aligned(a->pos_out_dev, 4) || !aligned(a->lens_out_dev, 4))
        return DEFRAG_EINVAL;
    if (c->batch && (!a->weight_dev || !a->pos_dev || !a->next_pos_dev || !a->weight_out_dev ||
                     !a->pos_out_dev || !a->lens_out_dev))
        return DEFRAG_EINVAL;
    // (weights and positions may be replaced where they are: a place below the
    // budget is written by one lane, from itself or from behind the budget)
    const uint64_t rows = (uint64_t)c->batch * c->heads;
    const bool same = a->weight_out_stride == a->weight_stride;
    const Span out[] = {plane(a->lens_out_dev, 1, 0, c->batch), plane(a->weight_out_dev, rows, a->weight_out_stride, kept),
                        plane(a->pos_out_dev, rows, a->weight_out_stride, kept)};
    const Span in[] = {plane(a->weight_out_dev == a->weight_dev && same ? nullptr : a->weight_dev, rows, a->weight_stride, a->max_len),
                       plane(a->pos_out_dev == a->pos_dev && same ? nullptr : a->pos_dev, rows, a->weight_stride, a->max_len),
                       plane(c->lens_dev, 1, 0, c->batch), plane(a->next_pos_dev, 1, 0, c->batch),
                       plane(c->pages_dev, 1, 0, 2 * c->batch * c->page_stride)};
    if (any_overlap(out, in)) return DEFRAG_EINVAL;
    return DEFRAG_OK;
}

int clear_count(const defrag_kv_cache *c, hipStream_t s) {
    if (!c->n_invalid_dev) return DEFRAG_OK;
    return launch_kv_zero(c->n_invalid_dev, s) == hipSuccess ? DEFRAG_OK : DEFRAG_EHIP;
}

int check_ws(const void *ws, size_t have, uint64_t need) {
    if (!need) return DEFRAG_OK;
    if (!ws || !aligned(ws, 256) || have < need) return DEFRAG_EWORKSPACE;
    return DEFRAG_OK;
}

// The launches of an attention whose arguments have been checked.
int attend(const defrag_kv_attend_args *a, const defrag_kv_terms *t, const KvAttendPlan &p, void *ws_dev, size_t ws_bytes,
           hipStream_t stream) {
    const defrag_kv_cache *c = a->cache;
    int rc = check_ws(ws_dev, ws_bytes, p.total);
    if (rc) return rc;
    rc = clear_count(c, stream);
    if (rc || !a->tokens) return rc;
    uint8_t *ws = static_cast<uint8_t *>(ws_dev);
    KvAttend k{};
    k.c = cache_of(c);
    k.q = static_cast<const uint16_t *>(a->q_dev);
    k.q_row = a->q_row;
    k.q_head = a->q_head;
    k.tokens = a->tokens;
    k.starts = a->starts_dev;
    k.max_new = a->max_new;
    k.max_len = a->max_len;
    k.group = a->group;
    k.scale = a->scale;
    k.out = static_cast<uint16_t *>(a->out_dev);
    k.lse = a->lse_dev;
    k.weight = a->weight_dev;
    k.cap = a->weight_stride;
    k.splits = p.splits;
    k.per_split = p.per_split;
    k.rows = p.rows;
    k.row_blocks = p.row_blocks;
    k.part = reinterpret_cast<float *>(ws);
    k.scores = p.score_bytes ? reinterpret_cast<float *>(ws + p.part_bytes) : nullptr;
    k.score_pages = (a->max_len + kKvPage - 1) / kKvPage;
    k.score_rows = p.score_rows;
    k.sums = p.sum_bytes ? reinterpret_cast<float2 *>(ws + p.part_bytes + p.score_bytes) : nullptr;
    k.weigh_pieces = p.weigh_pieces;
    k.weigh_tiles = p.weigh_tiles;
    k.weigh_part = p.weigh_bytes ? reinterpret_cast<float *>(ws + p.part_bytes + p.score_bytes + p.sum_bytes) : nullptr;
    if (t) {
        k.mask = t->mask_dev;
        k.mask_words = t->mask_words;
        k.score_cap = t->cap;
        k.cap_by = t->cap != 0.0f ? 2.0f / t->cap : 0.0f;
        k.slopes = t->slopes_dev;
        k.pos = t->pos_dev;
        k.pos_cap = t->pos_stride;
    }
    return launch_kv_attend(k, c->codes, a->dtype, stream) == hipSuccess ? DEFRAG_OK : DEFRAG_EHIP;
}

}  // namespace

extern "C" {

size_t defrag_kv_page_bytes(uint32_t heads, uint32_t dim) {
    if (heads < 1 || heads > 65535 || !dim_ok(dim)) return 0;
    return (kv_page_bytes(heads, dim) + 31) / 32 * 32;
}

int defrag_kv_append(const defrag_kv_append_args *a, hipStream_t stream) {
    int rc = check_append(a);
    if (rc) return rc;
    const defrag_kv_cache *c = a->cache;
    rc = clear_count(c, stream);
    if (rc || !a->tokens) return rc;
    return launch_kv_append(append_of(a), c->codes, a->dtype, stream) == hipSuccess ? DEFRAG_OK : DEFRAG_EHIP;
}

int defrag_kv_append_rotary(const defrag_kv_rotary_args *r, hipStream_t stream) {
    int rc = check_rotary(r);
    if (rc) return rc;
    const defrag_kv_append_args *a = r->append;
    const defrag_kv_cache *c = a->cache;
    rc = clear_count(c, stream);
    if (rc || !a->tokens) return rc;
    KvRotary k{};
    static_cast<KvAppend &>(k) = append_of(a);
    k.freq = r->freq_dev;
    k.rotary = r->rotary_dim;
    k.next = r->interleaved;
    k.token_pos = r->token_pos_dev;
    k.q = static_cast<const uint16_t *>(r->q_dev);
    k.q_row = r->q_row;
    k.q_head = r->q_head;
    k.q_out = static_cast<uint16_t *>(r->out_dev);
    k.o_row = r->out_row;
    k.o_head = r->out_head;
    k.q_heads = r->q_heads;
    return launch_kv_append_rotary(k, c->codes, a->dtype, stream) == hipSuccess ? DEFRAG_OK : DEFRAG_EHIP;
}

int defrag_kv_accept(const defrag_kv_accept_args *a, hipStream_t stream) {
    int rc = check_accept(a);
    if (rc) return rc;
    const defrag_kv_cache *c = a->cache;
    rc = clear_count(c, stream);
    if (rc || !c->batch) return rc;
    const KvAccept k{cache_of(c), a->starts_dev, a->tokens, a->max_new, a->path_dev, a->path_stride, a->kept_dev,
                     a->weight_dev, a->pos_dev, a->weight_stride, a->lens_out_dev};
    return launch_kv_accept(k, c->codes, stream) == hipSuccess ? DEFRAG_OK : DEFRAG_EHIP;
}

size_t defrag_kv_attend_workspace_bytes(const defrag_kv_attend_args *a) {
    KvAttendPlan p;
    if (check_attend(a, &p)) return 0;
    return p.total > kLeastWs ? p.total : kLeastWs;
}

int defrag_kv_attend(const defrag_kv_attend_args *a, void *ws_dev, size_t ws_bytes,
                     hipStream_t stream) {
    KvAttendPlan p;
    const int rc = check_attend(a, &p);
    return rc ? rc : attend(a, nullptr, p, ws_dev, ws_bytes, stream);
}

size_t defrag_kv_attend_terms_workspace_bytes(const defrag_kv_attend_args *a, const defrag_kv_terms *t) {
    KvAttendPlan p;
    if (check_terms(a, t, &p)) return 0;
    return p.total > kLeastWs ? p.total : kLeastWs;
}

int defrag_kv_attend_terms(const defrag_kv_attend_args *a, const defrag_kv_terms *t, void *ws_dev, size_t ws_bytes,
                           hipStream_t stream) {
    KvAttendPlan p;
    const int rc = check_terms(a, t, &p);
    return rc ? rc : attend(a, t, p, ws_dev, ws_bytes, stream);
}

size_t defrag_kv_evict_workspace_bytes(const defrag_kv_evict_args *a) {
    if (check_evict(a)) return 0;
    const uint64_t need = kv_evict_plan(a->cache->batch, a->cache->heads, a->budget, a->max_len).total;
    return need > kLeastWs ? need : kLeastWs;
}

int defrag_kv_evict(const defrag_kv_evict_args *a, void *ws_dev, size_t ws_bytes,
                    hipStream_t stream) {
    int rc = check_evict(a);
    if (rc) return rc;
    const defrag_kv_cache *c = a->cache;
    const KvEvictPlan p = kv_evict_plan(c->batch, c->heads, a->budget, a->max_len);
    rc = check_ws(ws_dev, ws_bytes, p.total);
    if (rc) return rc;
    rc = clear_count(c, stream);
    if (rc || !c->batch) return rc;
    uint8_t *ws = static_cast<uint8_t *>(ws_dev);
    KvEvict k{};
    k.c = cache_of(c);
    k.budget = a->budget;
    k.max_len = a->max_len;
    k.sink = a->sink;
    k.recent = a->recent;
    k.next_pos = a->next_pos_dev;
    k.weight = a->weight_dev;
    k.pos = a->pos_dev;
    k.cap = a->weight_stride;
    k.weight_out = a->weight_out_dev;
    k.pos_out = a->pos_out_dev;
    k.cap_out = a->weight_out_stride;
    k.lens_out = a->lens_out_dev;
    k.src = reinterpret_cast<int32_t *>(ws);
    k.moved = reinterpret_cast<int32_t *>(ws + p.list_bytes);
    k.fold = reinterpret_cast<int32_t *>(ws + 2 * p.list_bytes);
    k.rest = ws + 2 * p.list_bytes + p.fold_bytes;
    k.piece = p.piece;
    k.pieces = p.pieces;
    return launch_kv_evict(k, c->codes, stream) == hipSuccess ? DEFRAG_OK : DEFRAG_EHIP;
}

}  // extern "C"
