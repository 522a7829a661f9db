// cache_args.h -- launch arguments of the paged-cache kernels (attention, append, pages).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace hsp {

constexpr int kDeviceErrIndex = 8;  // same value as PROJ_ERR_BAD_INDEX

constexpr int kAttnTile = 64;       // tokens per tile
constexpr int kAttnMaxCtas = 512;  // CTAs along the length (the join lists them in shared memory)
constexpr int kAttnThreads = 224;   // four softmax warps, the copy producer, the issuers of S^T and of O^T
// Floats of one partial: O^T, and per head the reference point m, the sums l and u.
__host__ __device__ constexpr int attn_part(int dv, int N) { return N * dv + 3 * N; }

// One sequence part that a CTA began and another one finishes: what the join adds up.
// Entry c belongs to CTA c of the length axis; batch < 0: CTA c began no such part.
struct AttnEntry {
    int32_t batch;   // sequence (row of q), -1: none
    int32_t kv_head;
    int32_t last;    // the CTA that finishes the sequence
    int32_t slot;    // CTA c's partial slot (the later CTAs use slot 0)
};

struct AttnArgs {
    const int32_t *table;        // [num_rows, max_pages] page ids, rows at table_stride
    int64_t table_stride;
    const int32_t *lens;         // [num_rows]
    const int32_t *rows;         // [batch] table rows, or null (row = batch index)
    int32_t num_rows, max_pages, num_pages;
    int32_t page_shift;          // log2(page size)
    int32_t batch, kv_heads, group;  // group: query heads per kv head
    int32_t ctas;                // CTAs along the length (grid.y)
    int32_t split;               // 0: no sequence is cut (and nothing is to join)
    int32_t weight;              // units of a part's start and end (one per tile besides)
    int32_t slots;               // group places in the ring
    float scale_log2;            // softmax scale * log2(e)
    void *out;                   // [batch, heads, VB * 64] bf16
    float *lse;                  // [batch, heads] or null
    AttnEntry *entries;          // [ctas]
    float *parts;                // [head tiles][ctas][2][attn_part]
    int32_t skip_tile;           // test hook: this tile of every CTA is never loaded (-1: off)
    uint64_t wait_limit_ns;
    int *err_word;
};

struct AttnLaunchReq {
    int KB, VB, shared, N;       // key boxes, value boxes (64 columns each), v = columns of k, head tile
    int head_tiles;              // grid.x
    int smem_bytes;
    int pdl;
    int sms;
    cudaStream_t stream;
    CUtensorMap tmap_q;          // [batch][boxes][heads][64], a box: the head tile's queries
    CUtensorMap tmap_k, tmap_v;  // boxes of a group (latent: tmap_v has the single rotary box)
    AttnArgs args;
};
// One translation unit per cache kind.
cudaError_t launch_attn_latent(const AttnLaunchReq &r);
cudaError_t launch_attn_grouped(const AttnLaunchReq &r);
// Shared memory of the attention kernel besides its stages: queries, probabilities, reduction
// buffers, barriers (of at most kAttnMaxSlots places) and the alignment slack.
constexpr int kAttnMaxSlots = 12;
inline int attn_fixed_smem(int KB, int N) { return KB * N * 128 + kAttnTile * 128 + 5 * N * 4 + 512 + 1024; }
// CTAs per SM.  A latent tile is 73.7 KB, one CTA takes the shared memory of an SM; grouped tiles
// are 32 or 16 KB, and the softmaxes and products of two or three CTAs overlap (32 sequences of
// up to 4096 tokens, 8 kv heads of 64 columns: 38.4 us with two, 33.0 with three; its bytes take 19
// to 20 at the copy rate).  64 heads: registers allow one.
constexpr int attn_ctas_per_sm(int KB, bool shared, int N) { return shared || N == 64 ? 1 : KB == 1 && N == 16 ? 3 : 2; }
inline int attn_group_boxes(int VB) { return VB >= 2 ? 2 : 1; }

// ---- append ---------------------------------------------------------------------------

struct AppendArgs {
    const void *k_new, *v_new;       // [tokens, kv_heads, k_dim / v_dim] bf16, tokens at *_row (elements)
    int64_t k_row, v_row;
    void *k, *v;                     // the cache (v null: latent)
    int64_t k_page, k_token, k_head; // strides in elements
    int64_t v_page, v_token, v_head;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens, *rows, *positions;  // rows, positions may be null
    const int32_t *refs;             // [num_pages] or null: pages are not checked to be the row's own
    const float *cos_sin;            // [max_pos, rot] or null
    const void *q;                   // [tokens, heads, k_dim] or null, tokens at q_row, heads at q_head
    void *q_out;
    int64_t q_row, q_head, qo_row, qo_head;
    int32_t num_rows, max_pages, num_pages, page_shift;
    int32_t tokens, kv_heads, heads, k_dim, v_dim, rot, max_pos, interleaved;
    int *err_word;
};
cudaError_t launch_append(const AppendArgs &a, int sms, int pdl, cudaStream_t stream);

// ---- the cache in 8 bits ------------------------------------------------------------------

// Where the codes and scales of one side (keys or values) lie: codes in bytes, scales in elements.
struct Q8Side {
    uint8_t *codes;                  // null: none (the values of a latent cache)
    float *scales;
    int64_t page, token, head;       // code strides
    int64_t s_page, s_block, s_head; // scale strides
    int32_t dim;
};

struct AppendQ8Args {
    const void *k_new, *v_new;       // as in AppendArgs
    int64_t k_row, v_row;
    Q8Side k, v;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens, *rows, *positions;  // rows, positions may be null
    const int32_t *refs;
    const float *cos_sin;
    const void *q;
    void *q_out;
    int64_t q_row, q_head, qo_row, qo_head;
    int32_t num_rows, max_pages, num_pages, page_shift;
    int32_t block_shift;             // log2(tokens per scale)
    int32_t tokens, kv_heads, heads, rot, max_pos, interleaved;
    int *err_word;
};
cudaError_t launch_append_q8(const AppendQ8Args &a, int sms, int pdl, cudaStream_t stream);

struct ReadQ8Args {
    Q8Side k, v;
    void *k_out, *v_out;             // [tokens, kv_heads, dim] bf16, tokens at *_row (elements)
    int64_t k_row, v_row;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens, *rows, *positions;
    int32_t num_rows, max_pages, num_pages, page_shift, block_shift;
    int32_t tokens, kv_heads;
    int *err_word;
};
cudaError_t launch_read_q8(const ReadQ8Args &a, int sms, int pdl, cudaStream_t stream);

constexpr int kAttn8Tile = 128;      // tokens per tile
constexpr int kAttn8ScaleSlots = 2;  // tiles whose scales lie ready
// The queries in two 8-bit pieces, as a kernel of its own writes them: for each sequence, kv head and head tile of N the
// image of shared memory that the attention's instructions read (2 N rows of DK bytes, swizzled), then N bytes of units.
struct Attn8QueryArgs {
    const void *q;                   // [batch, heads, k_dim] bf16
    int64_t q_row, q_head;
    uint8_t *images;
    int32_t batch, kv_heads, group, head_tiles, N;
};
__host__ __device__ constexpr int attn8_image_bytes(int DK, int N) { return 2 * N * DK + N; }
struct Attn8Args {
    AttnArgs line;
    const uint8_t *images;
    const float *k_scales, *v_scales;
    int64_t ks_page, ks_block, ks_head, vs_page, vs_block, vs_head;
    int32_t block_shift;
};
struct Attn8LaunchReq {
    int DK, DV, shared, N;           // columns, v = columns of k, head tile
    int per_sm;                      // CTAs
    int head_tiles;                  // grid.x
    int smem_bytes;
    int pdl;
    int sms;
    cudaStream_t stream;
    CUtensorMap tmap_k, tmap_v;      // boxes of 128 (64) columns; latent: tmap_v has the 64 rotary columns
    Attn8QueryArgs queries;
    Attn8Args args;
};
cudaError_t launch_attn8_queries(const Attn8LaunchReq &r);
cudaError_t launch_attn8_latent(const Attn8LaunchReq &r);
cudaError_t launch_attn8_grouped(const Attn8LaunchReq &r);
// Four softmax warps for every 16 heads, then the copies, the two issuers, the scales.
constexpr int attn8_threads(int N) { return 8 * N + 128; }
// CTAs per SM (see attn_ctas_per_sm; 64 heads fill tensor memory).  16 grouped heads: three where there is a part for every SM
// from the start, else two, with more registers and longer rings (sequences x kv heads x columns, up to so many tokens, us with
// two and three: 61 x 8 x 128, 4099 64.0 and 60.0; 40 x 8 x 64, 1000 25.2 and 23.6; 24 x 8 x 128, 1000 18.5 and 18.2; 12 x 8 x 128, 4000
// 23.5 and 24.6; 16 x 8 x 128, 2000 19.7 and 22.7; 13 x 4 x 64, 2333 15.4 and 16.7; 1 x 8 x 128, 60000 32.5 and 34.6).
inline int attn8_ctas_per_sm(bool shared, int N, int64_t sequence_heads, int sms) {
    return shared || N == 64 ? 1 : N == 16 && sequence_heads >= sms ? 3 : 2;
}
constexpr int kAttn8RopeBytes = kAttn8Tile * 64;
// Places of the rotary boxes: one where the queries of 64 heads leave no more beside two whole tiles.
constexpr int attn8_rope_slots(int N) { return N == 64 ? 1 : 2; }
// Shared memory besides the ring of groups: queries (two pieces), probabilities, rotary boxes, scales, the queries' units,
// barriers.  (Together with two tiles of 576 columns and 64 heads nearly all that a CTA can have.)
inline int attn8_fixed_smem(int DK, bool rope, int N) {
    return 2 * N * DK + kAttn8Tile * 2 * N + (rope ? attn8_rope_slots(N) * kAttn8RopeBytes : 0) + kAttn8ScaleSlots * kAttn8Tile * 8 + 4 * N + 768;
}

// ---- pages ------------------------------------------------------------------------------

constexpr int kMaxPools = 4;
constexpr int kCopyPiece = 16384;    // bytes of one copy unit
constexpr int kMaxCopyPairs = 2048;

struct PoolList {
    int32_t count;
    int32_t layers[kMaxPools];
    int32_t pieces[kMaxPools];       // copy units of one page
    char *base[kMaxPools];
    int64_t layer_stride[kMaxPools], page_stride[kMaxPools], page_bytes[kMaxPools];
    int32_t pieces_total;            // copy units of one page of all pools and layers
};

// The bookkeeping of a cache: which pages a sequence holds and how many sequences hold a page.
struct IndexArgs {
    int32_t *table;                  // [num_rows, max_pages]
    int64_t table_stride;
    int32_t *lens;                   // [num_rows]
    int32_t *refs;                   // [num_pages]
    int32_t num_rows, max_pages, num_pages, page_shift;
    int *err_word;
};

// One row of a resize (workspace).
struct RowPlan {
    int32_t row;                     // -1: nothing to do
    int32_t len;                     // its new length
    int32_t have, want;              // pages before and after
    int32_t first;                   // its first entry in the free list
    int32_t cow_src;                 // the shared last page to copy, -1: none
};

// Small resizes decide and move in one launch: a cluster of kTeam CTAs that all make the same plan.
// The bytes that it may have to copy bound it: a beam step with 0.6 MB to copy took 17.2 us where two launches
// for either resize take 19.1, one with 1.2 MB 19.1 and 19.2.
constexpr int kTeam = 8;             // (the portable limit)
constexpr int kTeamRows = 256;       // rows of a request: one per warp of the team
constexpr int kTeamPages = 4096;     // pages of the pool: four per lane, their list in shared memory
constexpr int64_t kTeamBytes = 1 << 20;
struct ResizeArgs {
    IndexArgs ix;
    const int32_t *rows, *new_lens;  // [n]
    int32_t *status;                 // [n]
    int32_t n;
    // workspace
    int32_t *head;                   // [0]: copy pairs, [1]: live pages (compaction)
    unsigned long long *taken;       // copy units taken so far
    RowPlan *plan;                   // [n]
    int32_t *claims;                 // [num_rows]
    int32_t *list;                   // [num_pages] free pages (resize) or new places (compaction)
    int2 *pairs;                     // (source, destination)
    PoolList pools;
};
inline bool team_resize(const ResizeArgs &a) {
    int64_t page = 0;
    for (int p = 0; p < a.pools.count; ++p) page += a.pools.layers[p] * a.pools.page_bytes[p];
    return a.n <= kTeamRows && a.ix.num_pages <= kTeamPages && a.n <= kTeamBytes / page;
}
cudaError_t launch_resize(const ResizeArgs &a, int sms, int pdl, cudaStream_t stream);

struct ForkArgs {
    IndexArgs ix;
    const int32_t *parents, *children;
    int32_t *status;
    int32_t n;
};
cudaError_t launch_fork(const ForkArgs &a, int pdl, cudaStream_t stream);

struct CompactArgs {
    IndexArgs ix;
    int32_t *live;                   // [1]
    int32_t *head, *list;            // workspace, as in ResizeArgs
    unsigned long long *taken;
    int2 *pairs;
    PoolList pools;
};
cudaError_t launch_compact(const CompactArgs &a, int sms, int pdl, cudaStream_t stream);

// n pairs of host arrays (n <= kMaxCopyPairs), passed by value.
cudaError_t launch_copy_pages(const PoolList &pools, const int32_t *src, const int32_t *dst, int n, int pdl, cudaStream_t stream);

}  // namespace hsp
