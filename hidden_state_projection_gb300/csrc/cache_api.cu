// cache_api.cu -- the C entry points of the paged cache: checks of arguments, plans, launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "api_internal.h"
#include "cache_args.h"

namespace {

using hsp::api_fail;

constexpr int kSmemLimit = 232448;
constexpr int kSmemPerSm = 228 * 1024;
constexpr int kSmemReserved = 1024;  // per CTA, the system's own

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

proj_status check_index(const proj_page_index *ix, bool counts) {
    if (!ix) return api_fail(PROJ_ERR_INVALID_ARG, "index must not be NULL");
    if (ix->num_rows < 0 || ix->max_pages < 0 || ix->num_pages < 0)
        return api_fail(PROJ_ERR_INVALID_ARG, "negative size (num_rows=%d max_pages=%d num_pages=%d)", ix->num_rows,
                        ix->max_pages, ix->num_pages);
    if (ix->num_rows < 1 || ix->max_pages < 1 || ix->num_pages < 1)
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "num_rows, max_pages and num_pages must be at least 1");
    if (ix->page_size < 16 || ix->page_size > 1024 || (ix->page_size & (ix->page_size - 1)) != 0)
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "page_size=%d is not a power of two from 16 to 1024", ix->page_size);
    if (static_cast<int64_t>(ix->max_pages) * ix->page_size >= (int64_t(1) << 31) - 1024)
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "max_pages=%d of %d tokens exceed 2^31 - 1024", ix->max_pages, ix->page_size);
    if (ix->num_pages > (1 << 30) || ix->num_rows > (1 << 24))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "num_pages=%d or num_rows=%d too large", ix->num_pages, ix->num_rows);
    if (ix->table_stride < ix->max_pages) return api_fail(PROJ_ERR_INVALID_ARG, "table_stride is shorter than a table row");
    if (!ix->block_table || !ix->seq_lens || (counts && !ix->ref_counts))
        return api_fail(PROJ_ERR_INVALID_ARG, "block_table, seq_lens%s must not be NULL", counts ? " and ref_counts" : "");
    if (!aligned(ix->block_table, 4) || !aligned(ix->seq_lens, 4) || !aligned(ix->ref_counts, 4))
        return api_fail(PROJ_ERR_MISALIGNED, "block_table, seq_lens and ref_counts must be 4-byte aligned");
    return PROJ_OK;
}

// Heads and columns the attention kernel serves.
struct AttnShape {
    int KB, VB, shared, N, head_tiles, slots, per_sm, smem, weight;
};

proj_status attn_shape(int heads, int kv_heads, int k_dim, int v_dim, bool latent, AttnShape *s) {
    if (heads < 1 || kv_heads < 1) return api_fail(PROJ_ERR_INVALID_ARG, "heads=%d, kv_heads=%d (need at least 1)", heads, kv_heads);
    if (heads % kv_heads != 0) return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "%d query heads over %d kv heads", heads, kv_heads);
    if (heads > 65536) return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "heads=%d exceeds 65536", heads);
    if (latent ? !((k_dim == 576 || k_dim == 512) && v_dim == 512) : !((k_dim == 64 || k_dim == 128) && v_dim == k_dim))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE,
                        "k_dim=%d, v_dim=%d: a latent cache has 576 or 512 and 512 columns, a grouped one 64 or 128 of each",
                        k_dim, v_dim);
    const int group = heads / kv_heads;
    s->KB = k_dim / 64;
    s->VB = v_dim / 64;
    s->shared = latent ? 1 : 0;
    s->N = group <= 16 ? 16 : group <= 32 ? 32 : 64;
    s->head_tiles = (group + s->N - 1) / s->N;
    const int box = hsp::kAttnTile * 128, group_bytes = hsp::attn_group_boxes(s->VB) * box;
    const int fixed = hsp::attn_fixed_smem(s->KB, s->N) + (latent ? (s->KB - s->VB) * 2 * box : 0);
    s->per_sm = hsp::attn_ctas_per_sm(s->KB, latent, s->N);
    const int room = s->per_sm == 1 ? kSmemLimit : kSmemPerSm / s->per_sm - kSmemReserved;
    s->slots = (room - fixed) / group_bytes;
    if (s->slots > hsp::kAttnMaxSlots) s->slots = hsp::kAttnMaxSlots;
    if (!latent) s->slots &= ~1;  // keys and values take turns: each kind keeps its places (attn_kernel.cuh)
    s->smem = fixed + s->slots * group_bytes;
    // What a part's start and end cost, in tiles: its pipeline fills, and O^T finds its way out of tensor
    // memory.  Weights in turn, sequences of mixed lengths, us: 200 x 8 kv heads of 128 columns with 4 heads
    // each, up to 600 tokens 60.2 (0), 53.3 (1), 54.5 (3); 100 x 4 kv heads of 64 columns with 20 heads each
    // 49.3 (1), 47.0 (2), 48.0 (5); 64 x 4 with 64 each 40.3 (2), 37.4 (3), 39.6 (8); latent heads: 100 x 16
    // 23.7 (0), 22.9 (1), 24.5 (4); 64 x 128 72.2 (2), 70.4 (3), 75.0 (8).
    s->weight = 1 + s->N / 32;
    return PROJ_OK;
}

// The same of a cache in 8 bits: the same heads and columns, other tiles and places.
proj_status attn8_shape(int batch, int heads, int kv_heads, int k_dim, int v_dim, bool latent, int sms, AttnShape *s) {
    const proj_status st = attn_shape(heads, kv_heads, k_dim, v_dim, latent, s);
    if (st != PROJ_OK) return st;
    const int group_bytes = hsp::kAttn8Tile * (v_dim >= 128 ? 128 : 64);
    const int fixed = hsp::attn8_fixed_smem(k_dim, latent && k_dim > v_dim, s->N);
    s->per_sm = hsp::attn8_ctas_per_sm(latent, s->N, static_cast<int64_t>(batch) * kv_heads, sms);
    const int room = s->per_sm == 1 ? kSmemLimit : kSmemPerSm / s->per_sm - kSmemReserved;
    s->slots = (room - fixed) / group_bytes;
    if (s->slots > hsp::kAttnMaxSlots) s->slots = hsp::kAttnMaxSlots;
    if (!latent) s->slots &= ~1;  // (as above)
    s->smem = fixed + s->slots * group_bytes;
    // A part's start and end in tiles.  us with 1, 2 and 3 (sequences x kv heads x heads of each, up to so many tokens), latent: 8 x 16 heads, 2000
    // 17.0, 16.5, 16.3; 40 x 16, 3000 23.3, 22.2, 23.0; 100 x 64, 2000 45.9, 42.1, 43.3; 48 x 128, 6001 62.9, 59.7, 59.4; 100 x 128, 700 44.9, 44.9,
    // 42.1; 64 columns: 13 x 4 x 7, 2333 14.9, 15.7, 15.9; 16 x 8 x 4, 2000 19.0, 16.9, 17.3; 61 x 8 x 4, 4099 58.7, 55.4, 55.3; 60 x 2 x 24, 2000
    // 21.4, 20.2, 21.3; 60 x 2 x 64, 2000 29.6, 27.4, 25.9; 128 columns: 13 x 4 x 7, 2333 15.8, 16.4, 16.6; 18 x 8 x 8, 1000 16.8, 15.7, 16.7; 61 x 8 x 4,
    // 4099 67.5, 62.4, 61.9; 200 x 8 x 4, 600 72.4, 71.5, 72.3; 30 x 5 x 1, 6000 38.6, 35.0, 34.3.  Of 49 shapes 2 is the best or within 2 % of
    // it in 42, 3 in 37 and 1 in 19.
    s->weight = 2;
    return PROJ_OK;
}

int attn_ctas(const AttnShape &s, int sms) {
    int c = sms * s.per_sm / s.head_tiles;
    if (c < 1) c = 1;
    return c > hsp::kAttnMaxCtas ? hsp::kAttnMaxCtas : c;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

size_t attn_workspace(const AttnShape &s, int ctas) {
    return up256(static_cast<size_t>(ctas) * sizeof(hsp::AttnEntry)) +
           static_cast<size_t>(s.head_tiles) * ctas * 2 * hsp::attn_part(s.VB * 64, s.N) * 4;
}

// Of a cache in 8 bits, in front: the queries' images.
proj_status attn8_images(const AttnShape &s, int batch, int heads, int kv_heads, int k_dim, size_t *bytes) {
    *bytes = up256(static_cast<size_t>(batch) * kv_heads * s.head_tiles * hsp::attn8_image_bytes(k_dim, s.N));
    if (*bytes >= (size_t(1) << 40)) return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "batch=%d of %d heads is too large", batch, heads);
    return PROJ_OK;
}

proj_status check_kv(const proj_kv_pages *kv) {
    if (!kv || !kv->k) return api_fail(PROJ_ERR_INVALID_ARG, "kv and kv->k must not be NULL");
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return api_fail(PROJ_ERR_MISALIGNED, "k and v must be 16-byte aligned");
    const int64_t st[6] = {kv->k_page_stride, kv->k_token_stride, kv->k_head_stride,
                           kv->v ? kv->v_page_stride : 8, kv->v ? kv->v_token_stride : 8, kv->v ? kv->v_head_stride : 8};
    for (int64_t x : st) {
        if (x < 0 || x >= (int64_t(1) << 38)) return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "cache stride %lld out of range", (long long)x);
        if (x % 8 != 0) return api_fail(PROJ_ERR_MISALIGNED, "cache stride %lld is not a multiple of 8 elements", (long long)x);
    }
    return PROJ_OK;
}

// Steps through what a call writes: `extent` places, `stride` apart.
struct Dim {
    int64_t extent, stride;
};
// Whether places of `inner` units lie apart, as they do where every step (in the order of their strides) is at
// least as long as all that lies inside it.
template <size_t N>
bool nested(Dim (&dims)[N], int64_t inner) {
    std::sort(dims, dims + N, [](const Dim &x, const Dim &y) { return x.stride < y.stride; });
    __int128 reach = inner;
    for (const Dim &d : dims) {
        if (d.extent <= 1) continue;
        if (d.stride < reach) return false;
        reach += static_cast<__int128>(d.stride) * (d.extent - 1);
    }
    return true;
}

// The same of a cache that is written.
proj_status check_writable(const proj_kv_pages *kv, const proj_page_index *ix) {
    Dim k[3] = {{ix->num_pages, kv->k_page_stride}, {ix->page_size, kv->k_token_stride}, {kv->kv_heads, kv->k_head_stride}};
    Dim v[3] = {{ix->num_pages, kv->v_page_stride}, {ix->page_size, kv->v_token_stride}, {kv->kv_heads, kv->v_head_stride}};
    if (!nested(k, kv->k_dim) || (kv->v && !nested(v, kv->v_dim)))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "pages, tokens and heads of a cache that is written must not overlap");
    return PROJ_OK;
}

// Tokens, heads and pages that steps can reach lie apart.
proj_status check_apart(const proj_kv_pages *kv, const proj_page_index *ix) {
    if (kv->k_token_stride < 8 || (kv->v && kv->v_token_stride < 8))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "tokens of the cache must lie apart (token stride 0)");
    if ((kv->kv_heads > 1 && (kv->k_head_stride < 8 || (kv->v && kv->v_head_stride < 8))) ||
        (ix->num_pages > 1 && (kv->k_page_stride < 8 || (kv->v && kv->v_page_stride < 8))))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "heads and pages of the cache must lie apart (stride 0)");
    return PROJ_OK;
}

// The rotary turn of an append, and the queries that go with it.
proj_status check_turn(const proj_rotary *rotary, int k_dim, const void *q) {
    if (q && !rotary) return api_fail(PROJ_ERR_INVALID_ARG, "queries are only turned: q needs rotary");
    if (rotary) {
        if (!rotary->cos_sin || rotary->max_pos < 1) return api_fail(PROJ_ERR_INVALID_ARG, "rotary without a table");
        if (rotary->dim < 16 || rotary->dim % 16 || rotary->dim > k_dim)
            return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "rotary dim=%d is not a multiple of 16 up to k_dim=%d", rotary->dim, k_dim);
        if (!aligned(rotary->cos_sin, 16)) return api_fail(PROJ_ERR_MISALIGNED, "cos_sin must be 16-byte aligned");
    }
    return PROJ_OK;
}
proj_status check_q_out(const void *q, int64_t q_row, int64_t q_head, const void *q_out, int64_t qo_row, int64_t qo_head,
                        int tokens, int heads, int k_dim) {
    Dim dims[2] = {{tokens, qo_row}, {heads, qo_head}};
    if (!nested(dims, k_dim)) return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "tokens and heads of q_out must not overlap");
    if (q == q_out && ((tokens > 1 && q_row != qo_row) || (heads > 1 && q_head != qo_head)))
        return api_fail(PROJ_ERR_INVALID_ARG, "q_out may be q, with the same strides");
    return PROJ_OK;
}

// [pages][heads][64-column boxes][tokens][64]: token lines of 128 bytes as the products read them.
proj_status encode_pages(const void *p, const proj_page_index *ix, int heads, int dim, int64_t page, int64_t token,
                         int64_t head, int box_count, CUtensorMap *out) {
    const int boxes = dim / 64;
    const int tile = hsp::kAttnTile;
    const int tok = ix->page_size < tile ? ix->page_size : tile;
    const uint64_t dims[5] = {64, static_cast<uint64_t>(ix->page_size), static_cast<uint64_t>(boxes),
                              static_cast<uint64_t>(heads), static_cast<uint64_t>(ix->num_pages)};
    // a stride that no step takes (one head, one page) may be anything: give the map a plain one
    const uint64_t strides[4] = {static_cast<uint64_t>(token) * 2, 128, heads > 1 ? static_cast<uint64_t>(head) * 2 : 128,
                                 ix->num_pages > 1 ? static_cast<uint64_t>(page) * 2 : 128};
    const uint32_t box[5] = {64, static_cast<uint32_t>(tok), static_cast<uint32_t>(tok == tile ? box_count : 1), 1, 1};
    return hsp::api_encode_5d(p, dims, strides, box, out);
}

// [pages][heads][boxes of `width` columns][tokens][width]: the codes of `dim` columns, token lines of `width` bytes (joined: next to
// each other, or to the other boxes').
proj_status encode_codes(const void *p, const proj_page_index *ix, int heads, int dim, int width, int64_t page, int64_t token, int64_t head,
                         bool joined, CUtensorMap *out) {
    const int tok = ix->page_size < hsp::kAttn8Tile ? ix->page_size : hsp::kAttn8Tile;
    const uint64_t w = static_cast<uint64_t>(width);
    const uint64_t dims[5] = {w, static_cast<uint64_t>(ix->page_size), static_cast<uint64_t>(dim / width), static_cast<uint64_t>(heads),
                              static_cast<uint64_t>(ix->num_pages)};
    const uint64_t strides[4] = {static_cast<uint64_t>(token), w, heads > 1 ? static_cast<uint64_t>(head) : w,
                                 ix->num_pages > 1 ? static_cast<uint64_t>(page) : w};
    const uint32_t box[5] = {static_cast<uint32_t>(width), static_cast<uint32_t>(tok), 1, 1, 1};
    return hsp::api_encode_codes_5d(p, dims, strides, box, joined, out);
}

proj_status check_pools(const proj_page_pool *pools, int num_pools, hsp::PoolList *out) {
    if (!pools || num_pools < 1 || num_pools > PROJ_MAX_POOLS)
        return api_fail(PROJ_ERR_INVALID_ARG, "num_pools=%d (1..%d) or pools NULL", num_pools, PROJ_MAX_POOLS);
    memset(out, 0, sizeof *out);
    out->count = num_pools;
    int64_t total = 0;
    for (int i = 0; i < num_pools; ++i) {
        const proj_page_pool &p = pools[i];
        if (!p.base) return api_fail(PROJ_ERR_INVALID_ARG, "pools[%d].base is NULL", i);
        if (p.layers < 1 || p.page_bytes < 1 || p.layer_stride < 0 || p.page_stride < 0)
            return api_fail(PROJ_ERR_INVALID_ARG, "pools[%d]: layers, page_bytes at least 1, strides not negative", i);
        if (p.page_stride < p.page_bytes) return api_fail(PROJ_ERR_INVALID_ARG, "pools[%d]: pages overlap", i);
        if (!aligned(p.base, 16) || p.layer_stride % 16 || p.page_stride % 16 || p.page_bytes % 16)
            return api_fail(PROJ_ERR_MISALIGNED, "pools[%d]: base, strides and page_bytes must be multiples of 16 bytes", i);
        const int64_t pieces = (p.page_bytes + hsp::kCopyPiece - 1) / hsp::kCopyPiece;
        total += pieces * p.layers;
        if (total > (1 << 24)) return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "pages of the pools are too large");
        out->layers[i] = p.layers;
        out->pieces[i] = static_cast<int32_t>(pieces);
        out->base[i] = static_cast<char *>(p.base);
        out->layer_stride[i] = p.layer_stride;
        out->page_stride[i] = p.page_stride;
        out->page_bytes[i] = p.page_bytes;
    }
    out->pieces_total = static_cast<int32_t>(total);
    return PROJ_OK;
}

// Pages of different layers do not overlap either.
proj_status check_layers(const proj_page_pool *pools, int num_pools, int num_pages) {
    for (int i = 0; i < num_pools; ++i) {
        Dim dims[2] = {{pools[i].layers, pools[i].layer_stride}, {num_pages, pools[i].page_stride}};
        if (!nested(dims, pools[i].page_bytes)) return api_fail(PROJ_ERR_INVALID_ARG, "pools[%d]: layers overlap", i);
    }
    return PROJ_OK;
}

// ---- the cache in 8 bits ----

// Pointers, strides and block size; `heads` and columns are the callers' to check.
proj_status check_kv_q8(const proj_kv_pages_q8 *kv, const proj_page_index *ix) {
    if (!kv || !kv->k || !kv->k_scale) return api_fail(PROJ_ERR_INVALID_ARG, "kv, kv->k and kv->k_scale must not be NULL");
    if ((kv->v != nullptr) != (kv->v_scale != nullptr)) return api_fail(PROJ_ERR_INVALID_ARG, "v_scale goes with v");
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return api_fail(PROJ_ERR_MISALIGNED, "k and v must be 16-byte aligned");
    if (!aligned(kv->k_scale, 4) || !aligned(kv->v_scale, 4)) return api_fail(PROJ_ERR_MISALIGNED, "scales must be 4-byte aligned");
    if (kv->block < 1 || kv->block > ix->page_size || (kv->block & (kv->block - 1)) != 0)
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "block=%d is not a power of two up to the page size %d", kv->block, ix->page_size);
    const int64_t st[6] = {kv->k_page_stride, kv->k_token_stride, kv->k_head_stride,
                           kv->v ? kv->v_page_stride : 16, kv->v ? kv->v_token_stride : 16, kv->v ? kv->v_head_stride : 16};
    for (int64_t x : st) {
        if (x < 0 || x >= (int64_t(1) << 39)) return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "cache stride %lld out of range", (long long)x);
        if (x % 16 != 0) return api_fail(PROJ_ERR_MISALIGNED, "cache stride %lld is not a multiple of 16 bytes", (long long)x);
    }
    const int64_t ss[6] = {kv->k_scale_page_stride, kv->k_scale_block_stride, kv->k_scale_head_stride,
                           kv->v ? kv->v_scale_page_stride : 0, kv->v ? kv->v_scale_block_stride : 0, kv->v ? kv->v_scale_head_stride : 0};
    for (int64_t x : ss)
        if (x < 0 || x >= (int64_t(1) << 38)) return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "scale stride %lld out of range", (long long)x);
    return PROJ_OK;
}

// Tokens, heads and pages that steps can reach lie apart (the smallest step of a tensor copy is 16 bytes).
proj_status check_apart_q8(const proj_kv_pages_q8 *kv, const proj_page_index *ix) {
    if (kv->k_token_stride < 16 || (kv->v && kv->v_token_stride < 16))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "tokens of the cache must lie apart (token stride 0)");
    if ((kv->kv_heads > 1 && (kv->k_head_stride < 16 || (kv->v && kv->v_head_stride < 16))) ||
        (ix->num_pages > 1 && (kv->k_page_stride < 16 || (kv->v && kv->v_page_stride < 16))))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "heads and pages of the cache must lie apart (stride 0)");
    return PROJ_OK;
}

// Heads and columns that tokens are written to or read from by pieces of 16 codes.
proj_status check_columns_q8(const proj_kv_pages_q8 *kv, int64_t more) {
    if (kv->kv_heads < 1 || kv->kv_heads > 65536 || kv->k_dim < 16 || kv->k_dim % 16 || kv->k_dim > 65536 ||
        (kv->v && (kv->v_dim < 16 || kv->v_dim % 16 || kv->v_dim > 65536)))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "kv_heads=%d, k_dim=%d, v_dim=%d: columns in multiples of 16, heads at least 1",
                        kv->kv_heads, kv->k_dim, kv->v_dim);
    const int64_t columns = static_cast<int64_t>(kv->kv_heads) * (kv->k_dim + (kv->v ? kv->v_dim : 0)) + more;
    if (columns > (1 << 24)) return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "%lld columns of a token exceed 2^24", (long long)columns);
    return PROJ_OK;
}

// Places of codes and scales that are written lie apart.
proj_status check_writable_q8(const proj_kv_pages_q8 *kv, const proj_page_index *ix) {
    const int blocks = ix->page_size / kv->block;
    Dim k[3] = {{ix->num_pages, kv->k_page_stride}, {ix->page_size, kv->k_token_stride}, {kv->kv_heads, kv->k_head_stride}};
    Dim v[3] = {{ix->num_pages, kv->v_page_stride}, {ix->page_size, kv->v_token_stride}, {kv->kv_heads, kv->v_head_stride}};
    Dim ks[3] = {{ix->num_pages, kv->k_scale_page_stride}, {blocks, kv->k_scale_block_stride}, {kv->kv_heads, kv->k_scale_head_stride}};
    Dim vs[3] = {{ix->num_pages, kv->v_scale_page_stride}, {blocks, kv->v_scale_block_stride}, {kv->kv_heads, kv->v_scale_head_stride}};
    if (!nested(k, kv->k_dim) || !nested(ks, 1) || (kv->v && (!nested(v, kv->v_dim) || !nested(vs, 1))))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "pages, tokens (blocks) and heads of a cache that is written must not overlap");
    return PROJ_OK;
}

hsp::Q8Side k_side(const proj_kv_pages_q8 *kv) {
    return {static_cast<uint8_t *>(kv->k), kv->k_scale, kv->k_page_stride, kv->k_token_stride, kv->k_head_stride,
            kv->k_scale_page_stride, kv->k_scale_block_stride, kv->k_scale_head_stride, kv->k_dim};
}
hsp::Q8Side v_side(const proj_kv_pages_q8 *kv) {
    if (!kv->v) return {nullptr, nullptr, 0, 0, 0, 0, 0, 0, 0};
    return {static_cast<uint8_t *>(kv->v), kv->v_scale, kv->v_page_stride, kv->v_token_stride, kv->v_head_stride,
            kv->v_scale_page_stride, kv->v_scale_block_stride, kv->v_scale_head_stride, kv->v_dim};
}

hsp::IndexArgs index_args(const proj_page_index *ix, int *err_word) {
    hsp::IndexArgs a;
    a.table = ix->block_table;
    a.table_stride = ix->table_stride;
    a.lens = ix->seq_lens;
    a.refs = ix->ref_counts;
    a.num_rows = ix->num_rows;
    a.max_pages = ix->max_pages;
    a.num_pages = ix->num_pages;
    a.page_shift = log2_of(ix->page_size);
    a.err_word = err_word;
    return a;
}

// Workspace of resize and compact, in this order: head, claims, list, pairs, plan.
struct CacheWorkspace {
    size_t claims, list, pairs, plan, bytes;
};
CacheWorkspace cache_workspace(const proj_page_index *ix, int n) {
    CacheWorkspace w;
    const size_t pairs = static_cast<size_t>(n > ix->num_pages / 2 + 1 ? n : ix->num_pages / 2 + 1);
    w.claims = 256;
    w.list = w.claims + up256(static_cast<size_t>(ix->num_rows) * 4);
    w.pairs = w.list + up256(static_cast<size_t>(ix->num_pages) * 4);
    w.plan = w.pairs + up256(pairs * 8);
    w.bytes = w.plan + up256(static_cast<size_t>(n) * sizeof(hsp::RowPlan));
    return w;
}

// What both attention calls ask of their batch, scale and queries.
proj_status check_attention(const proj_page_index *index, const AttnShape &s, int batch, int kv_heads, int tile, float scale, float *scale_log2) {
    if (batch < 0) return api_fail(PROJ_ERR_INVALID_ARG, "batch=%d is negative", batch);
    *scale_log2 = scale * 1.4426950408889634f;  // log2(e)
    if (!std::isfinite(*scale_log2)) return api_fail(PROJ_ERR_INVALID_ARG, "scale (times log2 e) must be finite");
    // (units of the line fit 30 bits)
    const int64_t most_tiles = (static_cast<int64_t>(index->max_pages) * index->page_size + tile - 1) / tile;
    if (static_cast<int64_t>(batch) * kv_heads * (most_tiles + s.weight) >= (int64_t(1) << 30))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "batch=%d of up to %d pages is too large", batch, index->max_pages);
    return PROJ_OK;
}
proj_status check_queries(const void *q, int64_t q_row_stride, int64_t q_head_stride, const proj_page_index *index, const int32_t *rows,
                          int batch, int heads, const void *out, const float *lse) {
    if (!rows && batch > index->num_rows)
        return api_fail(PROJ_ERR_INVALID_ARG, "batch=%d exceeds the table's %d rows", batch, index->num_rows);
    if (!q || !out) return api_fail(PROJ_ERR_INVALID_ARG, "q and out must not be NULL");
    if (!aligned(q, 16) || !aligned(out, 16) || q_row_stride % 8 || q_head_stride % 8)
        return api_fail(PROJ_ERR_MISALIGNED, "q and out must be 16-byte aligned, q's strides multiples of 8 elements");
    if ((heads > 1 && (q_head_stride < 8 || q_head_stride >= (int64_t(1) << 38))) ||
        (batch > 1 && (q_row_stride < 8 || q_row_stride >= (int64_t(1) << 38))))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "queries must lie apart (strides %lld, %lld)", (long long)q_row_stride,
                        (long long)q_head_stride);
    if (!aligned(lse, 4) || !aligned(rows, 4)) return api_fail(PROJ_ERR_MISALIGNED, "lse and rows must be 4-byte aligned");
    return PROJ_OK;
}

// The launch arguments that both attention kernels walk their line of tiles by.
void attention_line(const proj_page_index *index, const int32_t *rows, int batch, int heads, int kv_heads, const AttnShape &s, int ctas,
                    bool split, float scale_log2, void *out, float *lse, void *workspace, const hsp::ApiOptions &opt,
                    const hsp::ApiDevice &dev, hsp::AttnArgs *args) {
    hsp::AttnArgs &a = *args;
    a.table = index->block_table;
    a.table_stride = index->table_stride;
    a.lens = index->seq_lens;
    a.rows = rows;
    a.num_rows = index->num_rows;
    a.max_pages = index->max_pages;
    a.num_pages = index->num_pages;
    a.page_shift = log2_of(index->page_size);
    a.batch = batch;
    a.kv_heads = kv_heads;
    a.group = heads / kv_heads;
    a.ctas = ctas;
    a.split = split ? 1 : 0;
    a.weight = s.weight;
    a.slots = s.slots;
    a.scale_log2 = scale_log2;
    a.out = out;
    a.lse = lse;
    if (split) {
        a.entries = static_cast<hsp::AttnEntry *>(workspace);
        a.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + up256(static_cast<size_t>(ctas) * sizeof(hsp::AttnEntry)));
    }
    a.skip_tile = opt.skip_stage;
    a.wait_limit_ns = opt.wait_limit_ns;
    a.err_word = dev.err_word;
}

proj_status check_workspace(const void *ws, size_t have, size_t need) {
    if (!ws) return api_fail(PROJ_ERR_INVALID_ARG, "workspace must not be NULL");
    if (!aligned(ws, 16)) return api_fail(PROJ_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    if (have < need) return api_fail(PROJ_ERR_INVALID_ARG, "workspace of %zu bytes, this call needs %zu", have, need);
    return PROJ_OK;
}

}  // namespace

extern "C" {

size_t proj_paged_attention_workspace_bytes(int32_t heads, int32_t kv_heads, int32_t k_dim, int32_t v_dim, int32_t latent) {
    AttnShape s;
    if (attn_shape(heads, kv_heads, k_dim, v_dim, latent != 0, &s) != PROJ_OK) return 0;
    return attn_workspace(s, attn_ctas(s, hsp::api_plan_sms()));
}

proj_status proj_paged_attention(const void *q, int64_t q_row_stride, int64_t q_head_stride, const proj_kv_pages *kv,
                                 const proj_page_index *index, const int32_t *rows, int32_t batch, int32_t heads,
                                 float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                 proj_stream_t stream) {
    proj_status st = check_index(index, false);
    if (st != PROJ_OK) return st;
    if ((st = check_kv(kv)) != PROJ_OK) return st;
    AttnShape s;
    if ((st = attn_shape(heads, kv->kv_heads, kv->k_dim, kv->v_dim, kv->v == nullptr, &s)) != PROJ_OK) return st;
    float scale_log2;
    if ((st = check_attention(index, s, batch, kv->kv_heads, hsp::kAttnTile, scale, &scale_log2)) != PROJ_OK) return st;
    if ((st = check_apart(kv, index)) != PROJ_OK) return st;
    if (batch == 0) return hsp::api_ok();
    if ((st = check_queries(q, q_row_stride, q_head_stride, index, rows, batch, heads, out, lse)) != PROJ_OK) return st;
    hsp::ApiDevice dev;
    if ((st = hsp::api_device(&dev)) != PROJ_OK) return st;
    const int ctas = attn_ctas(s, dev.sms);
    const bool split = static_cast<int64_t>(index->max_pages) * index->page_size > PROJ_UNCUT_TOKENS;
    if (split && (st = check_workspace(workspace, workspace_bytes, attn_workspace(s, ctas))) != PROJ_OK) return st;
    hsp::AttnLaunchReq r{};
    const int boxes = hsp::attn_group_boxes(s.VB);
    if ((st = encode_pages(kv->k, index, kv->kv_heads, kv->k_dim, kv->k_page_stride, kv->k_token_stride, kv->k_head_stride,
                           boxes, &r.tmap_k)) != PROJ_OK)
        return st;
    {
        const uint64_t dims[5] = {64, static_cast<uint64_t>(heads), static_cast<uint64_t>(s.KB), static_cast<uint64_t>(batch), 1};
        const uint64_t strides[4] = {heads > 1 ? static_cast<uint64_t>(q_head_stride) * 2 : 128, 128,
                                     batch > 1 ? static_cast<uint64_t>(q_row_stride) * 2 : 128, 128};
        const uint32_t box[5] = {64, static_cast<uint32_t>(s.N), static_cast<uint32_t>(s.KB), 1, 1};
        if ((st = hsp::api_encode_5d(q, dims, strides, box, &r.tmap_q)) != PROJ_OK) return st;
    }
    // the values' map; of a latent cache, the same pages one box at a time (the rotary box)
    st = PROJ_OK;
    if (kv->v)
        st = encode_pages(kv->v, index, kv->kv_heads, kv->v_dim, kv->v_page_stride, kv->v_token_stride, kv->v_head_stride, boxes,
                          &r.tmap_v);
    else if (s.KB > s.VB)
        st = encode_pages(kv->k, index, kv->kv_heads, kv->k_dim, kv->k_page_stride, kv->k_token_stride, kv->k_head_stride, 1,
                          &r.tmap_v);
    else
        r.tmap_v = r.tmap_k;
    if (st != PROJ_OK) return st;
    const hsp::ApiOptions opt = hsp::api_options();
    r.KB = s.KB;
    r.VB = s.VB;
    r.shared = s.shared;
    r.N = s.N;
    r.head_tiles = s.head_tiles;
    r.smem_bytes = s.smem;
    r.pdl = opt.pdl;
    r.sms = dev.sms;
    r.stream = reinterpret_cast<cudaStream_t>(stream);
    attention_line(index, rows, batch, heads, kv->kv_heads, s, ctas, split, scale_log2, out, lse, workspace, opt, dev, &r.args);
    const cudaError_t e = s.shared ? hsp::launch_attn_latent(r) : hsp::launch_attn_grouped(r);
    if (e != cudaSuccess) return hsp::api_cuda_fail(e, "kernel launch (paged attention)");
    hsp::api_count_launches(split ? 2 : 1);
    return hsp::api_ok();
}

proj_status proj_cache_append(const void *k_new, int64_t k_row_stride, const void *v_new, int64_t v_row_stride,
                              const proj_kv_pages *kv, const proj_page_index *index, const int32_t *rows,
                              const int32_t *positions, int32_t tokens, const proj_rotary *rotary, const void *q,
                              int64_t q_row_stride, int64_t q_head_stride, void *q_out, int64_t q_out_row_stride,
                              int64_t q_out_head_stride, int32_t heads, proj_stream_t stream) {
    proj_status st = check_index(index, false);
    if (st != PROJ_OK) return st;
    if ((st = check_kv(kv)) != PROJ_OK) return st;
    if (tokens < 0) return api_fail(PROJ_ERR_INVALID_ARG, "tokens=%d is negative", tokens);
    if (kv->kv_heads < 1 || kv->kv_heads > 65536 || kv->k_dim < 8 || kv->k_dim % 8 || kv->k_dim > 65536 ||
        (kv->v && (kv->v_dim < 8 || kv->v_dim % 8 || kv->v_dim > 65536)))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "kv_heads=%d, k_dim=%d, v_dim=%d: columns in multiples of 8, heads at least 1",
                        kv->kv_heads, kv->k_dim, kv->v_dim);
    if ((kv->v != nullptr) != (v_new != nullptr) && tokens > 0)
        return api_fail(PROJ_ERR_INVALID_ARG, "v_new goes with a cache that has values of its own");
    if (q && (heads < 1 || heads > 65536)) return api_fail(PROJ_ERR_INVALID_ARG, "heads=%d (1..65536)", heads);
    const int64_t columns = static_cast<int64_t>(kv->kv_heads) * (kv->k_dim + (kv->v ? kv->v_dim : 0)) +
                            (q ? static_cast<int64_t>(heads) * kv->k_dim : 0);
    if (columns > (1 << 24)) return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "%lld columns of a token exceed 2^24", (long long)columns);
    if ((st = check_writable(kv, index)) != PROJ_OK) return st;
    if ((st = check_turn(rotary, kv->k_dim, q)) != PROJ_OK) return st;
    if (tokens == 0) return hsp::api_ok();
    if (!rows && tokens > index->num_rows)
        return api_fail(PROJ_ERR_INVALID_ARG, "tokens=%d exceeds the table's %d rows", tokens, index->num_rows);
    if (!k_new || (q && !q_out)) return api_fail(PROJ_ERR_INVALID_ARG, "k_new (and q_out beside q) must not be NULL");
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q, 16) || !aligned(q_out, 16) || k_row_stride % 8 ||
        v_row_stride % 8 || q_row_stride % 8 || q_head_stride % 8 || q_out_row_stride % 8 || q_out_head_stride % 8)
        return api_fail(PROJ_ERR_MISALIGNED, "k_new, v_new, q and q_out: 16-byte aligned, strides multiples of 8 elements");
    if (!aligned(rows, 4) || !aligned(positions, 4))
        return api_fail(PROJ_ERR_MISALIGNED, "rows and positions must be 4-byte aligned");
    if (q && (st = check_q_out(q, q_row_stride, q_head_stride, q_out, q_out_row_stride, q_out_head_stride, tokens, heads, kv->k_dim)) != PROJ_OK)
        return st;
    hsp::ApiDevice dev;
    if ((st = hsp::api_device(&dev)) != PROJ_OK) return st;
    hsp::AppendArgs a;
    memset(&a, 0, sizeof a);
    a.k_new = k_new;
    a.v_new = v_new;
    a.k_row = k_row_stride;
    a.v_row = v_row_stride;
    a.k = kv->k;
    a.v = kv->v;
    a.k_page = kv->k_page_stride;
    a.k_token = kv->k_token_stride;
    a.k_head = kv->k_head_stride;
    a.v_page = kv->v_page_stride;
    a.v_token = kv->v_token_stride;
    a.v_head = kv->v_head_stride;
    a.table = index->block_table;
    a.table_stride = index->table_stride;
    a.lens = index->seq_lens;
    a.refs = index->ref_counts;
    a.rows = rows;
    a.positions = positions;
    a.cos_sin = rotary ? rotary->cos_sin : nullptr;
    a.rot = rotary ? rotary->dim : 0;
    a.max_pos = rotary ? rotary->max_pos : 0;
    a.interleaved = rotary ? (rotary->interleaved != 0) : 1;
    a.q = q;
    a.q_out = q_out;
    a.q_row = q_row_stride;
    a.q_head = q_head_stride;
    a.qo_row = q_out_row_stride;
    a.qo_head = q_out_head_stride;
    a.num_rows = index->num_rows;
    a.max_pages = index->max_pages;
    a.num_pages = index->num_pages;
    a.page_shift = log2_of(index->page_size);
    a.tokens = tokens;
    a.kv_heads = kv->kv_heads;
    a.heads = q ? heads : 0;
    a.k_dim = kv->k_dim;
    a.v_dim = kv->v_dim;
    a.err_word = dev.err_word;
    const cudaError_t e = hsp::launch_append(a, dev.sms, hsp::api_options().pdl, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return hsp::api_cuda_fail(e, "kernel launch (cache append)");
    hsp::api_count_launches(1);
    return hsp::api_ok();
}

proj_status proj_cache_append_q8(const void *k_new, int64_t k_row_stride, const void *v_new, int64_t v_row_stride,
                                 const proj_kv_pages_q8 *kv, const proj_page_index *index, const int32_t *rows,
                                 const int32_t *positions, int32_t tokens, const proj_rotary *rotary, const void *q,
                                 int64_t q_row_stride, int64_t q_head_stride, void *q_out, int64_t q_out_row_stride,
                                 int64_t q_out_head_stride, int32_t heads, proj_stream_t stream) {
    proj_status st = check_index(index, false);
    if (st != PROJ_OK) return st;
    if ((st = check_kv_q8(kv, index)) != PROJ_OK) return st;
    if (tokens < 0) return api_fail(PROJ_ERR_INVALID_ARG, "tokens=%d is negative", tokens);
    if ((kv->v != nullptr) != (v_new != nullptr) && tokens > 0)
        return api_fail(PROJ_ERR_INVALID_ARG, "v_new goes with a cache that has values of its own");
    if (q && (heads < 1 || heads > 65536)) return api_fail(PROJ_ERR_INVALID_ARG, "heads=%d (1..65536)", heads);
    if ((st = check_columns_q8(kv, q ? static_cast<int64_t>(heads) * kv->k_dim : 0)) != PROJ_OK) return st;
    if ((st = check_writable_q8(kv, index)) != PROJ_OK) return st;
    if ((st = check_turn(rotary, kv->k_dim, q)) != PROJ_OK) return st;
    if (tokens == 0) return hsp::api_ok();
    if (!rows && tokens > index->num_rows)
        return api_fail(PROJ_ERR_INVALID_ARG, "tokens=%d exceeds the table's %d rows", tokens, index->num_rows);
    if (!k_new || (q && !q_out)) return api_fail(PROJ_ERR_INVALID_ARG, "k_new (and q_out beside q) must not be NULL");
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q, 16) || !aligned(q_out, 16) || k_row_stride % 8 ||
        v_row_stride % 8 || q_row_stride % 8 || q_head_stride % 8 || q_out_row_stride % 8 || q_out_head_stride % 8)
        return api_fail(PROJ_ERR_MISALIGNED, "k_new, v_new, q and q_out: 16-byte aligned, strides multiples of 8 elements");
    if (!aligned(rows, 4) || !aligned(positions, 4))
        return api_fail(PROJ_ERR_MISALIGNED, "rows and positions must be 4-byte aligned");
    if (q && (st = check_q_out(q, q_row_stride, q_head_stride, q_out, q_out_row_stride, q_out_head_stride, tokens, heads, kv->k_dim)) != PROJ_OK)
        return st;
    hsp::ApiDevice dev;
    if ((st = hsp::api_device(&dev)) != PROJ_OK) return st;
    hsp::AppendQ8Args a;
    memset(&a, 0, sizeof a);
    a.k_new = k_new;
    a.v_new = v_new;
    a.k_row = k_row_stride;
    a.v_row = v_row_stride;
    a.k = k_side(kv);
    a.v = v_side(kv);
    a.table = index->block_table;
    a.table_stride = index->table_stride;
    a.lens = index->seq_lens;
    a.refs = index->ref_counts;
    a.rows = rows;
    a.positions = positions;
    a.cos_sin = rotary ? rotary->cos_sin : nullptr;
    a.rot = rotary ? rotary->dim : 0;
    a.max_pos = rotary ? rotary->max_pos : 0;
    a.interleaved = rotary ? (rotary->interleaved != 0) : 1;
    a.q = q;
    a.q_out = q_out;
    a.q_row = q_row_stride;
    a.q_head = q_head_stride;
    a.qo_row = q_out_row_stride;
    a.qo_head = q_out_head_stride;
    a.num_rows = index->num_rows;
    a.max_pages = index->max_pages;
    a.num_pages = index->num_pages;
    a.page_shift = log2_of(index->page_size);
    a.block_shift = log2_of(kv->block);
    a.tokens = tokens;
    a.kv_heads = kv->kv_heads;
    a.heads = q ? heads : 0;
    a.err_word = dev.err_word;
    const cudaError_t e = hsp::launch_append_q8(a, dev.sms, hsp::api_options().pdl, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return hsp::api_cuda_fail(e, "kernel launch (cache append, 8 bits)");
    hsp::api_count_launches(1);
    return hsp::api_ok();
}

proj_status proj_cache_read_q8(const proj_kv_pages_q8 *kv, const proj_page_index *index, const int32_t *rows,
                               const int32_t *positions, int32_t tokens, void *k_out, int64_t k_row_stride, void *v_out,
                               int64_t v_row_stride, proj_stream_t stream) {
    proj_status st = check_index(index, false);
    if (st != PROJ_OK) return st;
    if ((st = check_kv_q8(kv, index)) != PROJ_OK) return st;
    if (tokens < 0) return api_fail(PROJ_ERR_INVALID_ARG, "tokens=%d is negative", tokens);
    if ((kv->v != nullptr) != (v_out != nullptr) && tokens > 0)
        return api_fail(PROJ_ERR_INVALID_ARG, "v_out goes with a cache that has values of its own");
    if ((st = check_columns_q8(kv, 0)) != PROJ_OK) return st;
    if (tokens == 0) return hsp::api_ok();
    if (!rows && tokens > index->num_rows)
        return api_fail(PROJ_ERR_INVALID_ARG, "tokens=%d exceeds the table's %d rows", tokens, index->num_rows);
    if (!k_out) return api_fail(PROJ_ERR_INVALID_ARG, "k_out must not be NULL");
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || k_row_stride % 8 || v_row_stride % 8)
        return api_fail(PROJ_ERR_MISALIGNED, "k_out and v_out: 16-byte aligned, strides multiples of 8 elements");
    if (!aligned(rows, 4) || !aligned(positions, 4))
        return api_fail(PROJ_ERR_MISALIGNED, "rows and positions must be 4-byte aligned");
    Dim dk[1] = {{tokens, k_row_stride}}, dv[1] = {{tokens, v_row_stride}};
    if (!nested(dk, static_cast<int64_t>(kv->kv_heads) * kv->k_dim) || (v_out && !nested(dv, static_cast<int64_t>(kv->kv_heads) * kv->v_dim)))
        return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "tokens of k_out and v_out must not overlap");
    hsp::ApiDevice dev;
    if ((st = hsp::api_device(&dev)) != PROJ_OK) return st;
    hsp::ReadQ8Args a;
    memset(&a, 0, sizeof a);
    a.k = k_side(kv);
    a.v = v_side(kv);
    a.k_out = k_out;
    a.v_out = v_out;
    a.k_row = k_row_stride;
    a.v_row = v_row_stride;
    a.table = index->block_table;
    a.table_stride = index->table_stride;
    a.lens = index->seq_lens;
    a.rows = rows;
    a.positions = positions;
    a.num_rows = index->num_rows;
    a.max_pages = index->max_pages;
    a.num_pages = index->num_pages;
    a.page_shift = log2_of(index->page_size);
    a.block_shift = log2_of(kv->block);
    a.tokens = tokens;
    a.kv_heads = kv->kv_heads;
    a.err_word = dev.err_word;
    const cudaError_t e = hsp::launch_read_q8(a, dev.sms, hsp::api_options().pdl, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return hsp::api_cuda_fail(e, "kernel launch (cache read, 8 bits)");
    hsp::api_count_launches(1);
    return hsp::api_ok();
}

size_t proj_paged_attention_q8_workspace_bytes(int32_t batch, int32_t heads, int32_t kv_heads, int32_t k_dim, int32_t v_dim,
                                               int32_t latent) {
    AttnShape s;
    if (attn8_shape(batch, heads, kv_heads, k_dim, v_dim, latent != 0, hsp::api_plan_sms(), &s) != PROJ_OK) return 0;
    if (batch < 0) {
        api_fail(PROJ_ERR_INVALID_ARG, "batch=%d is negative", batch);
        return 0;
    }
    size_t images;
    if (attn8_images(s, batch, heads, kv_heads, k_dim, &images) != PROJ_OK) return 0;
    return images + attn_workspace(s, attn_ctas(s, hsp::api_plan_sms()));
}

proj_status proj_paged_attention_q8(const void *q, int64_t q_row_stride, int64_t q_head_stride, const proj_kv_pages_q8 *kv,
                                    const proj_page_index *index, const int32_t *rows, int32_t batch, int32_t heads,
                                    float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                    proj_stream_t stream) {
    proj_status st = check_index(index, false);
    if (st != PROJ_OK) return st;
    if ((st = check_kv_q8(kv, index)) != PROJ_OK) return st;
    AttnShape s;
    if ((st = attn8_shape(batch, heads, kv->kv_heads, kv->k_dim, kv->v_dim, kv->v == nullptr, hsp::api_plan_sms(), &s)) != PROJ_OK) return st;
    float scale_log2;
    if ((st = check_attention(index, s, batch, kv->kv_heads, hsp::kAttn8Tile, scale, &scale_log2)) != PROJ_OK) return st;
    if ((st = check_apart_q8(kv, index)) != PROJ_OK) return st;
    if (batch == 0) return hsp::api_ok();
    if ((st = check_queries(q, q_row_stride, q_head_stride, index, rows, batch, heads, out, lse)) != PROJ_OK) return st;
    hsp::ApiDevice dev;
    if ((st = hsp::api_device(&dev)) != PROJ_OK) return st;
    const int ctas = attn_ctas(s, dev.sms);
    const bool split = static_cast<int64_t>(index->max_pages) * index->page_size > PROJ_UNCUT_TOKENS;
    size_t images;
    if ((st = attn8_images(s, batch, heads, kv->kv_heads, kv->k_dim, &images)) != PROJ_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, images + (split ? attn_workspace(s, ctas) : 0))) != PROJ_OK) return st;
    hsp::Attn8LaunchReq r{};
    const int width = kv->v_dim >= 128 ? 128 : 64;
    if ((st = encode_codes(kv->k, index, kv->kv_heads, kv->v ? kv->k_dim : kv->v_dim, width, kv->k_page_stride, kv->k_token_stride,
                           kv->k_head_stride, !kv->v || kv->k_token_stride == kv->k_dim, &r.tmap_k)) != PROJ_OK)
        return st;
    // the values' map; of a latent cache, the rotary columns of the same pages
    st = PROJ_OK;
    if (kv->v)
        st = encode_codes(kv->v, index, kv->kv_heads, kv->v_dim, width, kv->v_page_stride, kv->v_token_stride, kv->v_head_stride,
                          kv->v_token_stride == kv->v_dim, &r.tmap_v);
    else if (kv->k_dim > kv->v_dim)
        st = encode_codes(static_cast<const char *>(kv->k) + kv->v_dim, index, kv->kv_heads, 64, 64, kv->k_page_stride, kv->k_token_stride,
                          kv->k_head_stride, true, &r.tmap_v);
    else
        r.tmap_v = r.tmap_k;
    if (st != PROJ_OK) return st;
    const hsp::ApiOptions opt = hsp::api_options();
    r.DK = kv->k_dim;
    r.DV = kv->v_dim;
    r.shared = s.shared;
    r.N = s.N;
    r.per_sm = s.per_sm;
    r.head_tiles = s.head_tiles;
    r.smem_bytes = s.smem;
    r.pdl = opt.pdl;
    r.sms = dev.sms;
    r.stream = reinterpret_cast<cudaStream_t>(stream);
    attention_line(index, rows, batch, heads, kv->kv_heads, s, ctas, split, scale_log2, out, lse, static_cast<char *>(workspace) + images, opt,
                   dev, &r.args.line);
    r.queries = {q, batch > 1 ? q_row_stride : 0, heads > 1 ? q_head_stride : 0, static_cast<uint8_t *>(workspace), batch, kv->kv_heads,
                 heads / kv->kv_heads, s.head_tiles, s.N};
    r.args.images = static_cast<const uint8_t *>(workspace);
    r.args.k_scales = kv->k_scale;
    r.args.v_scales = kv->v ? kv->v_scale : kv->k_scale;
    r.args.ks_page = kv->k_scale_page_stride;
    r.args.ks_block = kv->k_scale_block_stride;
    r.args.ks_head = kv->k_scale_head_stride;
    r.args.vs_page = kv->v_scale_page_stride;
    r.args.vs_block = kv->v_scale_block_stride;
    r.args.vs_head = kv->v_scale_head_stride;
    r.args.block_shift = log2_of(kv->block);
    const cudaError_t e = s.shared ? hsp::launch_attn8_latent(r) : hsp::launch_attn8_grouped(r);
    if (e != cudaSuccess) return hsp::api_cuda_fail(e, "kernel launch (paged attention, 8 bits)");
    hsp::api_count_launches(split ? 3 : 2);
    return hsp::api_ok();
}

size_t proj_cache_workspace_bytes(const proj_page_index *index, int32_t n) {
    if (check_index(index, false) != PROJ_OK) return 0;
    if (n < 0) {
        api_fail(PROJ_ERR_INVALID_ARG, "n=%d is negative", n);
        return 0;
    }
    return cache_workspace(index, n).bytes;
}

proj_status proj_cache_resize(const proj_page_index *index, const int32_t *rows, const int32_t *new_lens, int32_t n,
                              const proj_page_pool *pools, int32_t num_pools, int32_t *status, void *workspace,
                              size_t workspace_bytes, proj_stream_t stream) {
    proj_status st = check_index(index, true);
    if (st != PROJ_OK) return st;
    hsp::ResizeArgs a;
    memset(&a, 0, sizeof a);
    if ((st = check_pools(pools, num_pools, &a.pools)) != PROJ_OK) return st;
    if ((st = check_layers(pools, num_pools, index->num_pages)) != PROJ_OK) return st;
    if (n < 0) return api_fail(PROJ_ERR_INVALID_ARG, "n=%d is negative", n);
    if (n == 0) return hsp::api_ok();
    if (!rows || !new_lens || !status) return api_fail(PROJ_ERR_INVALID_ARG, "rows, new_lens and status must not be NULL");
    if (!aligned(rows, 4) || !aligned(new_lens, 4) || !aligned(status, 4))
        return api_fail(PROJ_ERR_MISALIGNED, "rows, new_lens and status must be 4-byte aligned");
    const CacheWorkspace w = cache_workspace(index, n);
    if ((st = check_workspace(workspace, workspace_bytes, w.bytes)) != PROJ_OK) return st;
    hsp::ApiDevice dev;
    if ((st = hsp::api_device(&dev)) != PROJ_OK) return st;
    a.ix = index_args(index, dev.err_word);
    a.rows = rows;
    a.new_lens = new_lens;
    a.status = status;
    a.n = n;
    char *ws = static_cast<char *>(workspace);
    a.head = reinterpret_cast<int32_t *>(ws);
    a.taken = reinterpret_cast<unsigned long long *>(ws + 16);
    a.claims = reinterpret_cast<int32_t *>(ws + w.claims);
    a.list = reinterpret_cast<int32_t *>(ws + w.list);
    a.pairs = reinterpret_cast<int2 *>(ws + w.pairs);
    a.plan = reinterpret_cast<hsp::RowPlan *>(ws + w.plan);
    const cudaError_t e = hsp::launch_resize(a, dev.sms, hsp::api_options().pdl, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return hsp::api_cuda_fail(e, "kernel launch (cache resize)");
    hsp::api_count_launches(hsp::team_resize(a) ? 1 : 2);
    return hsp::api_ok();
}

proj_status proj_cache_fork(const proj_page_index *index, const int32_t *parents, const int32_t *children, int32_t n,
                            int32_t *status, proj_stream_t stream) {
    proj_status st = check_index(index, true);
    if (st != PROJ_OK) return st;
    if (n < 0) return api_fail(PROJ_ERR_INVALID_ARG, "n=%d is negative", n);
    if (n == 0) return hsp::api_ok();
    if (!parents || !children || !status) return api_fail(PROJ_ERR_INVALID_ARG, "parents, children and status must not be NULL");
    if (!aligned(parents, 4) || !aligned(children, 4) || !aligned(status, 4))
        return api_fail(PROJ_ERR_MISALIGNED, "parents, children and status must be 4-byte aligned");
    hsp::ApiDevice dev;
    if ((st = hsp::api_device(&dev)) != PROJ_OK) return st;
    hsp::ForkArgs a;
    a.ix = index_args(index, dev.err_word);
    a.parents = parents;
    a.children = children;
    a.status = status;
    a.n = n;
    const cudaError_t e = hsp::launch_fork(a, hsp::api_options().pdl, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return hsp::api_cuda_fail(e, "kernel launch (cache fork)");
    hsp::api_count_launches(1);
    return hsp::api_ok();
}

proj_status proj_cache_compact(const proj_page_index *index, const proj_page_pool *pools, int32_t num_pools,
                               int32_t *live, void *workspace, size_t workspace_bytes, proj_stream_t stream) {
    proj_status st = check_index(index, true);
    if (st != PROJ_OK) return st;
    hsp::CompactArgs a;
    memset(&a, 0, sizeof a);
    if ((st = check_pools(pools, num_pools, &a.pools)) != PROJ_OK) return st;
    if ((st = check_layers(pools, num_pools, index->num_pages)) != PROJ_OK) return st;
    if (!live) return api_fail(PROJ_ERR_INVALID_ARG, "live must not be NULL");
    if (!aligned(live, 4)) return api_fail(PROJ_ERR_MISALIGNED, "live must be 4-byte aligned");
    const CacheWorkspace w = cache_workspace(index, 0);
    if ((st = check_workspace(workspace, workspace_bytes, w.bytes)) != PROJ_OK) return st;
    hsp::ApiDevice dev;
    if ((st = hsp::api_device(&dev)) != PROJ_OK) return st;
    a.ix = index_args(index, dev.err_word);
    a.live = live;
    char *ws = static_cast<char *>(workspace);
    a.head = reinterpret_cast<int32_t *>(ws);
    a.taken = reinterpret_cast<unsigned long long *>(ws + 16);
    a.list = reinterpret_cast<int32_t *>(ws + w.list);
    a.pairs = reinterpret_cast<int2 *>(ws + w.pairs);
    const cudaError_t e = hsp::launch_compact(a, dev.sms, hsp::api_options().pdl, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return hsp::api_cuda_fail(e, "kernel launch (cache compact)");
    hsp::api_count_launches(2);
    return hsp::api_ok();
}

proj_status proj_cache_copy_pages(const proj_page_pool *pools, int32_t num_pools, int32_t num_pages, const int32_t *src,
                                  const int32_t *dst, int32_t n, proj_stream_t stream) {
    hsp::PoolList pl;
    proj_status st = check_pools(pools, num_pools, &pl);
    if (st != PROJ_OK) return st;
    if (n < 0 || num_pages < 0) return api_fail(PROJ_ERR_INVALID_ARG, "negative size (n=%d num_pages=%d)", n, num_pages);
    if (n > PROJ_MAX_COPY_PAIRS) return api_fail(PROJ_ERR_UNSUPPORTED_SHAPE, "n=%d exceeds %d pairs", n, PROJ_MAX_COPY_PAIRS);
    if ((st = check_layers(pools, num_pools, num_pages)) != PROJ_OK) return st;
    if (n == 0) return hsp::api_ok();
    if (!src || !dst) return api_fail(PROJ_ERR_INVALID_ARG, "src and dst must not be NULL");
    // destinations in a table of their own: a second one, or a source among them, is refused
    constexpr int kSlots = 4 * PROJ_MAX_COPY_PAIRS;
    int32_t slots[kSlots];
    uint32_t mask = 63;
    while (mask + 1 < 4u * static_cast<uint32_t>(n)) mask = 2 * mask + 1;
    memset(slots, 0xff, sizeof(int32_t) * (mask + 1));
    auto find = [&](int32_t id) {
        uint32_t h = (static_cast<uint32_t>(id) * 2654435761u) >> 7;
        while (slots[h & mask] != -1 && slots[h & mask] != id) ++h;
        return h & mask;
    };
    for (int i = 0; i < n; ++i) {
        if (src[i] < 0 || src[i] >= num_pages || dst[i] < 0 || dst[i] >= num_pages)
            return api_fail(PROJ_ERR_INVALID_ARG, "pair %d (%d -> %d) outside the %d pages", i, src[i], dst[i], num_pages);
        const uint32_t at = find(dst[i]);
        if (slots[at] != -1) return api_fail(PROJ_ERR_INVALID_ARG, "page %d is a destination twice", dst[i]);
        slots[at] = dst[i];
    }
    for (int i = 0; i < n; ++i)
        if (slots[find(src[i])] != -1)
            return api_fail(PROJ_ERR_INVALID_ARG, "page %d is a source and a destination", src[i]);
    hsp::ApiDevice dev;
    if ((st = hsp::api_device(&dev)) != PROJ_OK) return st;
    const cudaError_t e = hsp::launch_copy_pages(pl, src, dst, n, hsp::api_options().pdl, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return hsp::api_cuda_fail(e, "kernel launch (cache copy)");
    hsp::api_count_launches(1);
    return hsp::api_ok();
}

}  // extern "C"
