// attn8_kernel.cuh -- attention of one new token per sequence over a paged cache held in 8 bits.
//
//   o[b, h] = sum_t p_t vs_t vc_t,  p = softmax_t(scale ks_t q[b, h] . kc_t),  t < len_b
//
// kc, vc: e4m3 codes, ks, vs: the scales of their blocks.  The shape of the bf16 kernel (attn_kernel.cuh: tokens or
// value columns on the instruction's rows, query heads its columns, tiles in a ring, a line of tiles cut over the
// CTAs), with 8-bit instructions that read the codes as they lie in the cache, so that nothing is converted on the
// way and a byte of the cache passes shared memory three times (copy, scores, values):
//   S^T[128 tokens x 2N] = KC[128 x dk] . [Qh; Ql]^T       (both operands K-major)
//   O^T[dv x N]         += VC^T[dv x 128] . (Wh + Wl)^T    (both MN-major)
//
// Queries.  A bf16 number has 8 significant bits, e4m3 has 4: q 2^-e = Qh + Ql / 16, e the head's own exponent (the
// largest |q| of the head falls to 224 .. 448), is exact down to 2^-14, 2^-21.8 of the head's largest.  The two products
// lie side by side in tensor memory and are added in the softmax.
//
// Weights.  The scale of a token's values goes into its weight: w_t = p_t vs_t, in the softmax's own units
// 2^(s_t + log2 vs_t - m).  w = Wh + Wl of w in fp16 (2^-11), Wh rounded to e4m3, the rest to e5m2: at most 2^-7 of w while w is at least
// 2^-6 (the rest of a smaller one is half of 2^-9 or less, and e5m2 keeps an eighth of that), largest 448.  Two 8-bit
// pieces have not the range of a bf16 number, so the reference point m (a whole number) follows the tiles in both directions: a tile whose
// largest weight in some column is beyond 2^8.75, or below 2^-4, moves that column's m (largest weight to 2^3 .. 2^4) and
// rescales O^T; what a tile's rounding leaves out is small beside the largest weight of the tile and of the row,
// whatever weights other tiles have (a first token with nearly all the weight before a long tail).  Normal scores of
// variance 3 in 64 columns move a point in 2 tiles of 133 (in 54 with a window of 2^0.5 to 2^8.75).  Downwards m stops 30
// below its highest point.
//
// Sums.  A token whose weight is nothing beside the others' because its values are (a block of zeros has the scale 2^-60)
// still has its probability, and that counts in what O^T is divided by: l = u + sum over w_t >= 2^-6 of (Wh + Wl - w)_t / vs_t,
// u = sum w_t / vs_t of the unrounded weights.  So a large weight counts as it is rounded, and the rounding that all of a row's
// weight has in common cancels; a small one counts as it is, with the 2^-22 of fp32's exponential.  (Summed as rounded, small
// weights took their probabilities with them: of two tokens with equal scores, one with values of zero, the other came out
// whole.)  What is lost is what fp32 has no number for: weights below 2^-126 of the reference point, 2^-129 of the row's largest, which
// takes values' scales more than 2^90 apart.  (With those summed apart, and sums moved from point to point in two steps, the
// grouped batch below took 66.8 us, not 61.6 as then.)  The mask of the large weights takes 0.5 of the 128 heads' 59.  lse takes u.  Sums
// and statistics are fp32.
//
// Warps: four for the softmax of every 16 heads (they also carry O^T out), a copy producer, an issuer of the scores, an
// issuer of the products with the values, one that fetches the tiles' scales ahead.  All waits are at mbarriers and
// bounded.  The queries are split by a small kernel in front, into the images that the instructions read (split by every
// CTA for itself they took 4 to 10 us: all wait for it, and code that runs once comes from L2 at 100 cycles per 128 bytes).
//
// What bounds it (one GB300, cycles at 1.9 GHz).  64 latent heads: operands from shared memory.  A tile of 576 columns is
// 73 KB written by copies, 147 read for the scores (18 products of 128 x 128 x 32, 65 cycles each), 196 for the values (32 of
// 128 x 64 x 32, 48 cycles each) and 16 of weights: 3400 cycles at 128 bytes each, 3800 to 4300 measured; the softmax (2500)
// and the copies hide behind it.  Fewer heads: memory.  Beside the tiles stand 4.5 us from the launch to the first copy, 4 to
// 5 from there to the first weights (DRAM, and code that runs for the first time), 5 us for each further part (its queries,
// 128 KB of partial O^T at 28 bytes a cycle) and the join.  With the queries' kernel and the join: 48 sequences up to 6001
// tokens, 128 heads of 576 columns 59.3 us (bf16 cache 61.9); one of 131071 tokens, 64 heads of 512 columns 35.0 (41.0);
// 61 sequences up to 4099 tokens, 32 heads over 8 of 128 columns 61.0 to 63.4 (91.4; 253 MB, 53 % of the DRAM's rate); 13 sequences up to
// 2333 tokens, 28 heads over 4 of 64 columns 15.3; 1 sequence of 77 tokens, 16 heads, not cut 8.1.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "attn_common.cuh"
#include "q8.cuh"

namespace hsp {

// A product of 8-bit operands (32 elements of K per instruction), fp32 accumulator.
__device__ __forceinline__ void umma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// K-major operand in 64-byte lines (64-byte swizzle): eight rows in 512 bytes.
__device__ __forceinline__ uint64_t umma_desc_sw64(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(16u >> 4) << 16;
    d |= static_cast<uint64_t>(512u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(4u) << 61;
    return d;
}
// MN-major operand whose M (or N) extent lies in one line of LINE bytes, swizzled over that width; eight lines of K
// follow each other, groups of eight 8 * LINE bytes apart.  (K-major with LINE = 128 or 64: the same numbers.)
template <int LINE>
__device__ __forceinline__ uint64_t umma_desc_lines(uint32_t smem_addr) {
    static_assert(LINE == 128 || LINE == 64 || LINE == 32, "a swizzle width");
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((8u * LINE) >> 4) << 16;
    d |= static_cast<uint64_t>((8u * LINE) >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(LINE == 128 ? 2u : LINE == 64 ? 4u : 6u) << 61;
    return d;
}
// Where 16-byte piece `chunk` of line `row` lies in its line.
template <int LINE>
__device__ __forceinline__ int swizzled(int row, int chunk) {
    return LINE == 128 ? (chunk ^ (row & 7)) << 4 : LINE == 64 ? (chunk ^ ((row >> 1) & 3)) << 4 : (chunk ^ ((row >> 2) & 1)) << 4;
}

// Two fp16 numbers to e4m3 or e5m2 codes and e5m2 codes back (`lo` in bits 0-7).
__device__ __forceinline__ uint32_t half2_to_e4m3x2(__half2 v) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f16x2 c, %1;\n\tcvt.u32.u16 %0, c;\n\t}" : "=r"(r) : "r"(*reinterpret_cast<const uint32_t *>(&v)));
    return r;
}
__device__ __forceinline__ uint32_t half2_to_e5m2x2(__half2 v) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e5m2x2.f16x2 c, %1;\n\tcvt.u32.u16 %0, c;\n\t}" : "=r"(r) : "r"(*reinterpret_cast<const uint32_t *>(&v)));
    return r;
}
__device__ __forceinline__ __half2 e5m2x2_to_half2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e5m2x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
    return *reinterpret_cast<const __half2 *>(&r);
}

// Column c of pairs of columns.
template <int P>
__device__ __forceinline__ float col(const float2 (&v)[P], int c) {
    return (c & 1) ? v[c >> 1].y : v[c >> 1].x;
}

template <int DK, int DV, bool SHARED, int N>
struct Attn8Cfg {
    static constexpr int kW = DV >= 128 ? 128 : 64;           // columns of a box: its line in bytes
    static constexpr int kMV = kW;                            // rows of one O^T instruction
    static constexpr int kOT = DV / kMV;                      // O^T tiles
    static constexpr int kVG = DV / kW;                       // value groups of a tile
    static constexpr int kKG = SHARED ? 0 : 1;                // key groups of its own
    static constexpr int kGroups = kVG + kKG;
    static constexpr bool kRope = SHARED && DK > DV;          // 64 rotary columns
    static constexpr int kX = kRope ? attn8_rope_slots(N) : 0;  // places of the rotary boxes
    static constexpr int kGroupBytes = kAttn8Tile * kW;
    static constexpr int kQRows = 2 * N;
    static constexpr int kQBytes = kQRows * DK;
    static constexpr int kPLine = 2 * N;                      // bytes of a token's weights: Wh, then Wl
    static constexpr int kPBytes = kAttn8Tile * kPLine;
    static constexpr int kCols = kOT * N + 4 * N;             // O^T, then two S^T
    static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static_assert(kCols <= 512, "tensor memory");
    static constexpr int kThreads = attn8_threads(N);
    static constexpr int kSets = N / 16;                      // sets of four softmax warps, 16 heads each
    static constexpr int kSoft = 128 * kSets;                 // softmax threads
    static constexpr int kRoles = 4 * kSets;                  // the first warp behind the softmax
};

// The window of a column's largest weight in a tile, log2, and where it is put.
constexpr float kAttn8Up = 8.75f, kAttn8Low = -4.f, kAttn8Aim = 3.f, kAttn8Down = 30.f;
// Weights from here on count in the sum as they are rounded.
constexpr float kAttn8Large = 0x1p-6f;

template <int DK, int DV, bool SHARED, int N, int PER_SM>
__global__ void __launch_bounds__(attn8_threads(N), PER_SM)
    hsp_attn8_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ Attn8Args g) {
    using C = Attn8Cfg<DK, DV, SHARED, N>;
    constexpr int T = kAttn8Tile, kC = 4;  // (heads of a softmax thread)
    const AttnArgs &a = g.line;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t ring = smem_u32(smem);
    uint8_t *const x_smem = smem + a.slots * C::kGroupBytes;            // the rotary boxes' places
    uint8_t *const q_smem = x_smem + C::kX * kAttn8RopeBytes;
    uint8_t *const p_smem = q_smem + C::kQBytes;
    float *const red = reinterpret_cast<float *>(p_smem);               // [4 warps][N], where the weights are not under way
    float *const fac = red + 4 * N;                                     // [N], likewise
    float *const points = fac + N, *const bottom = points + N;          // [N], likewise
    float *const scales = reinterpret_cast<float *>(p_smem + C::kPBytes);  // [slots][2][T]: ks (times the scale), log2 vs
    uint32_t *const seen = reinterpret_cast<uint32_t *>(scales + kAttn8ScaleSlots * 2 * T);  // [2][16 warps], 16-byte aligned
    uint8_t *const q_unit = reinterpret_cast<uint8_t *>(seen + 32);     // [4][N] the unit of a part's queries, 2^(e - 127) of the head
    uint64_t *const full = reinterpret_cast<uint64_t *>(q_unit + 4 * N);
    uint64_t *const empty = full + a.slots;
    uint64_t *const x_full = empty + a.slots;                           // [2]
    uint64_t *const x_empty = x_full + 2;                               // [2]
    uint64_t *const s_full = x_empty + 2;                               // [2]
    uint64_t *const s_free = s_full + 2;                                // [2]
    uint64_t *const q_full = s_free + 2;
    uint64_t *const q_free = q_full + 1;
    uint64_t *const p_full = q_free + 1;
    uint64_t *const pv_done = p_full + 1;
    uint64_t *const drained = pv_done + 1;
    uint64_t *const unit_full = drained + 1;                            // [4] q_unit
    uint64_t *const sc_full = unit_full + 4;                            // [kAttn8ScaleSlots]
    uint64_t *const sc_empty = sc_full + kAttn8ScaleSlots;
    int *const ints = reinterpret_cast<int *>(sc_empty + kAttn8ScaleSlots);
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(ints);
    volatile int *const abort_flag = ints + 1;
    int *const issued = ints + 2;                                       // groups, rotary boxes, queries whose copies were issued
    int *const place = ints + 5;
    int *const warp_sum = ints + 8;                                     // [20]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ht = blockIdx.x, cta = blockIdx.y;

    if (tid == 0) {
        for (int s = 0; s < a.slots; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&x_full[s]), 1);
            mbar_init(smem_u32(&x_empty[s]), 1);
            mbar_init(smem_u32(&s_full[s]), 1);
            mbar_init(smem_u32(&s_free[s]), C::kSoft / 32);
        }
        for (int s = 0; s < 4; ++s) mbar_init(smem_u32(&unit_full[s]), 1);
        for (int s = 0; s < kAttn8ScaleSlots; ++s) {
            mbar_init(smem_u32(&sc_full[s]), 1);
            mbar_init(smem_u32(&sc_empty[s]), C::kSoft / 32);
        }
        mbar_init(smem_u32(q_full), 1);
        mbar_init(smem_u32(q_free), 1);
        mbar_init(smem_u32(p_full), C::kSoft / 32);
        mbar_init(smem_u32(pv_done), 1);
        mbar_init(smem_u32(drained), 2);
        *abort_flag = 0;
        issued[0] = issued[1] = issued[2] = 0;
        mbar_fence_init();
        tma_prefetch_map(&tmap_k);
        if (!SHARED || C::kRope) tma_prefetch_map(&tmap_v);
    }
    if (warp == C::kRoles + 1) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // What is read below comes from before the kernel that splits the queries, which has let this one start when all of
    // that was complete; only its own images are still to come, and the issuer of the scores waits for those.

    const AttnLine ln = attn_find_line<T, C::kThreads>(a, cta, place, warp_sum);
    const uint32_t tmem = *tmem_slot;
    const uint32_t tmem_s = tmem + C::kOT * N;
    auto await = [&](uint64_t *bar, uint32_t phase) { return attn_wait(smem_u32(bar), phase & 1u, a.wait_limit_ns, abort_flag); };

    auto warp_arrive = [&](uint64_t *bar) {  // once for the warp, when all of its lanes are there
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(bar));
    };

    if (warp == C::kRoles) {
        // ---------------- copy producer: one thread reads the table two tiles ahead and issues ----------------
        // A group's turn (a wait, the bytes, a copy for each page) is a chain of instructions on one thread beside busy softmax
        // warps: what can be is done once for a tile, and pages of 64 tokens or more have code of their own (two pages to a
        // tile, not eight).
        if (elect_one()) {
            auto copies = [&](auto pages_of_a_tile) {
                constexpr int E = decltype(pages_of_a_tile)::value;
                constexpr bool kAhead = SHARED && N == 64 && E == 2;  // (see `ahead`; the table is read two tiles ahead, else one)
                AttnWalk walk(ln);
                int i = 0;
                AttnSegment sg;
                RingPos rp, xp;
                int ng = 0, nx = 0;                          // groups and rotary boxes so far
                const int pbox = min(T, 1 << a.page_shift);  // tokens per box
                const int boxes = T / pbox;                  // pages that meet a tile (1 to E)
                const uint32_t line_bytes = static_cast<uint32_t>(pbox) * C::kW;
                const uint32_t full_at = smem_u32(full), empty_at = smem_u32(empty);
                bool alive = true;
                while (alive && attn_next_segment<T>(a, ln, walk, sg)) {
                    const int row = a.rows ? a.rows[sg.b] : sg.b;
                    const int32_t *tbl = a.table + row * a.table_stride;
                    const int pages = static_cast<int>((static_cast<int64_t>(sg.len) + (1 << a.page_shift) - 1) >> a.page_shift);
                    auto ids_of = [&](int k, int (&id)[E]) {  // (0: none)
                        const int p0 = static_cast<int>((static_cast<int64_t>(sg.t0 + k) * T) >> a.page_shift);
#pragma unroll
                        for (int e = 0; e < E; ++e) id[e] = (e < boxes && p0 + e < pages) ? tbl[p0 + e] : 0;
                    };
                    int next[E], then[E];
                    ids_of(0, next);
                    if (kAhead) ids_of(1, then);
                    for (int k = 0; k < sg.n && alive; ++k, ++i) {
                        int id[E];
                        bool out = false;
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            id[e] = next[e];
                            if (kAhead) next[e] = then[e];
                            out |= static_cast<uint32_t>(id[e]) >= static_cast<uint32_t>(a.num_pages);
                        }
                        if (__builtin_expect(out, false)) {
                            atomicCAS(a.err_word, 0, kDeviceErrIndex);
#pragma unroll
                            for (int e = 0; e < E; ++e)
                                if (static_cast<uint32_t>(id[e]) >= static_cast<uint32_t>(a.num_pages)) id[e] = 0;  // stays inside the pool; the call is reported
                        }
                        if (k + 1 + kAhead < sg.n) ids_of(k + 1 + kAhead, kAhead ? then : next);
                        const int64_t tok = static_cast<int64_t>(sg.t0 + k) * T;
                        const int np = min(boxes, pages - static_cast<int>(tok >> a.page_shift));
                        const int off = boxes == 1 ? static_cast<int>(tok & ((1 << a.page_shift) - 1)) : 0;
                        const uint32_t bytes = static_cast<uint32_t>(np) * line_bytes;
                        // A ring of two tiles is too short for DRAM's latency behind the products: with several head tiles one
                        // of them sends the next tile to L2 while this one waits for its places (the first: when it has them).
                        auto ahead = [&]() {
                            if (!kAhead || gridDim.x == 1 || k + 1 >= sg.n || (k + 1) % static_cast<int>(gridDim.x) != ht) return;
                            const int64_t after = tok + T;
                            const int to = boxes == 1 ? static_cast<int>(after & ((1 << a.page_shift) - 1)) : 0;
#pragma unroll 1
                            for (int e = 0; e < boxes; ++e) {
                                const int page = e == 0 ? next[0] : next[E > 1 ? 1 : 0];
                                if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages) || (after >> a.page_shift) + e >= pages) continue;
#pragma unroll 1
                                for (int gr = 0; gr < C::kGroups; ++gr) tma_prefetch_5d(&tmap_k, 0, to, gr, sg.kv, page);
                                if (C::kRope) tma_prefetch_5d(&tmap_v, 0, to, 0, sg.kv, page);
                            }
                        };
                        if (k > 0) ahead();
                        const bool skip = i == a.skip_tile;
#pragma unroll 1
                        for (int gr = 0; gr < C::kGroups; ++gr) {
                            // (a fresh barrier's phase before the first counts as complete)
                            alive = attn_wait(empty_at + rp.slot * 8, rp.phase ^ 1u, a.wait_limit_ns, abort_flag);
                            if (!alive) break;
                            ++ng;
                            if (!skip) {
                                const CUtensorMap *map = SHARED || gr < C::kKG ? &tmap_k : &tmap_v;
                                const uint32_t fb = full_at + rp.slot * 8, dst = ring + rp.slot * C::kGroupBytes;
                                mbar_arrive_expect_tx(fb, bytes);
#pragma unroll
                                for (int e = 0; e < E; ++e)
                                    if (e < np) tma_load_5d(dst + e * line_bytes, map, 0, off, SHARED ? gr : 0, sg.kv, id[e], fb);
                            }
                            rp.next(a.slots);
                        }
                        if (C::kRope && alive) {
                            alive = await(&x_empty[xp.slot], xp.phase ^ 1u);
                            if (!alive) break;
                            ++nx;
                            if (!skip) {
                                const uint32_t fb = smem_u32(&x_full[xp.slot]), dst = smem_u32(x_smem) + xp.slot * kAttn8RopeBytes;
                                mbar_arrive_expect_tx(fb, static_cast<uint32_t>(np * pbox) * 64);
#pragma unroll
                                for (int e = 0; e < E; ++e)
                                    if (e < np) tma_load_5d(dst + e * (pbox * 64), &tmap_v, 0, off, 0, sg.kv, id[e], fb);
                            }
                            xp.next(C::kX);
                        }
                        if (k == 0) ahead();
                    }
                }
                issued[0] = ng;
                issued[1] = nx;
            };
            if (SHARED && a.page_shift >= 6) copies(std::integral_constant<int, 2>());
            else copies(std::integral_constant<int, 8>());
        }
        __syncwarp();
    } else if (warp == C::kRoles + 1) {
        // ---------------- issuer of the scores ----------------
        if (elect_one()) {
            constexpr uint32_t kDesc = (1u << 4) | (static_cast<uint32_t>(C::kQRows >> 3) << 17) | (static_cast<uint32_t>(T >> 4) << 24);
            AttnWalk walk(ln);
            uint32_t seg = 0;
            AttnSegment sg;
            bool alive = true;
            const uint64_t qd = umma_desc_lines<C::kW>(smem_u32(q_smem));
            RingPos rp, xp, sp;
            griddep_wait();  // the images (in every CTA: the next kernel but one may write them anew)
            while (alive && attn_next_segment<T>(a, ln, walk, sg)) {
                // the part's queries, when the scores of the last part are done with theirs
                if (!await(q_free, seg ^ 1u)) break;
                const uint8_t *from = g.images + ((static_cast<int64_t>(sg.b) * a.kv_heads + sg.kv) * gridDim.x + ht) * attn8_image_bytes(DK, N);
                mbar_arrive_expect_tx(smem_u32(q_full), C::kQBytes);
                bulk_load(smem_u32(q_smem), from, C::kQBytes, smem_u32(q_full));
                mbar_arrive_expect_tx(smem_u32(&unit_full[seg & 3u]), N);
                bulk_load(smem_u32(q_unit) + (seg & 3u) * N, from + C::kQBytes, N, smem_u32(&unit_full[seg & 3u]));
                issued[2] = static_cast<int>(seg + 1);
                if (!await(q_full, seg)) break;
                ++seg;
                for (int k = 0; k < sg.n; ++k) {
                    // the scores of the tile before last have been read out of this accumulator
                    if (!(alive = await(&s_free[sp.slot], sp.phase ^ 1u))) break;
                    const uint32_t d = tmem_s + sp.slot * C::kQRows;
                    constexpr int kGroupsK = SHARED ? C::kVG : C::kKG;
#pragma unroll 1
                    for (int gr = 0; gr < kGroupsK; ++gr) {
                        if (alive) alive = await(&full[rp.slot], rp.phase);
                        if (!alive) break;
                        tc_fence_after_sync();
                        const uint64_t kd = umma_desc_lines<C::kW>(ring + rp.slot * C::kGroupBytes);
#pragma unroll
                        for (int e = 0; e < C::kW / 32; ++e)  // (descriptors count 16 bytes)
                            umma_f8(d, kd + e * 2, qd + gr * (C::kQRows * C::kW / 16) + e * 2, kDesc, (gr | e) != 0 ? 1u : 0u);
                        if (!SHARED) umma_commit(smem_u32(&empty[rp.slot]));
                        rp.next(a.slots);
                    }
                    if (!alive) break;
                    if (!SHARED) rp.next(a.slots);  // the value group
                    if (C::kRope) {
                        if (!(alive = await(&x_full[xp.slot], xp.phase))) break;
                        tc_fence_after_sync();
                        const uint64_t kd = umma_desc_lines<64>(smem_u32(x_smem) + xp.slot * kAttn8RopeBytes);
                        const uint64_t xd = umma_desc_lines<64>(smem_u32(q_smem) + C::kQRows * DV);
#pragma unroll
                        for (int e = 0; e < 2; ++e) umma_f8(d, kd + e * 2, xd + e * 2, kDesc, 1u);
                        umma_commit(smem_u32(&x_empty[xp.slot]));
                        xp.next(C::kX);
                    }
                    umma_commit(smem_u32(&s_full[sp.slot]));
                    sp.next(2);
                }
                umma_commit(smem_u32(q_free));
            }
            umma_commit(smem_u32(drained));
        }
        __syncwarp();
    } else if (warp == C::kRoles + 2) {
        // ---------------- issuer of the products with the values ----------------
        if (elect_one()) {
            constexpr uint32_t kDescH = (1u << 4) | (1u << 15) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(C::kMV >> 4) << 24);
            constexpr uint32_t kDescL = kDescH | (1u << 10);  // e5m2 weights
            AttnWalk walk(ln);
            int i = 0;
            AttnSegment sg;
            bool alive = true;
            const uint64_t pd = umma_desc_lines<C::kPLine>(smem_u32(p_smem));
            RingPos rp;
            while (alive && attn_next_segment<T>(a, ln, walk, sg)) {
                for (int k = 0; k < sg.n; ++k, ++i) {
                    const int valid = min(T, sg.len - (sg.t0 + k) * T);  // tokens of this tile
                    alive = await(p_full, static_cast<uint32_t>(i));
                    if (!alive) break;
                    tc_fence_after_sync();
                    if (!SHARED) {
                        rp.next(a.slots);  // the key group
                        alive = await(&full[rp.slot], rp.phase);
                        if (!alive) break;
                        tc_fence_after_sync();
                    }
#pragma unroll 1
                    for (int jt = 0; jt < C::kOT; ++jt) {
                        const uint64_t vd = umma_desc_lines<C::kW>(ring + rp.slot * C::kGroupBytes);
#pragma unroll
                        for (int e = 0; e < T / 32; ++e)
                            if (e * 32 < valid) {
                                umma_f8(tmem + jt * N, vd + e * (2 * C::kW), pd + e * (2 * C::kPLine), kDescH, (k | e) != 0 ? 1u : 0u);
                                umma_f8(tmem + jt * N, vd + e * (2 * C::kW), pd + e * (2 * C::kPLine) + N / 16, kDescL, 1u);
                            }
                        umma_commit(smem_u32(&empty[rp.slot]));
                        rp.next(a.slots);
                    }
                    umma_commit(smem_u32(pv_done));
                }
            }
            // always committed and awaited (both issuers'), so that no product is in flight when the memory goes
            umma_commit(smem_u32(drained));
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(smem_u32(drained), 0u) && global_timer_ns() - t0 < a.wait_limit_ns) {
            }
        }
        __syncwarp();
    } else if (warp == C::kRoles + 3) {
        // ---------------- the tiles' scales, up to kAttn8ScaleSlots tiles ahead ----------------
        AttnWalk walk(ln);
        int i = 0;
        AttnSegment sg;
        bool alive = true;
        while (alive && attn_next_segment<T>(a, ln, walk, sg)) {
            const int row = a.rows ? a.rows[sg.b] : sg.b;
            const int32_t *tbl = a.table + row * a.table_stride;
            const float *ks = g.k_scales + sg.kv * g.ks_head, *vs = g.v_scales + sg.kv * g.vs_head;
            // a tile's scales are requested while the ones before wait for their place
            auto fetch = [&](int tile, float (&kk)[4], float (&vv)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = tile * T + e * 32 + lane;
                    kk[e] = 0.f;
                    vv[e] = 1.f;
                    if (t < sg.len) {
                        int page = tbl[t >> a.page_shift];
                        if (page < 0 || page >= a.num_pages) page = 0;  // (reported by the copy producer)
                        const int blk = (t & ((1 << a.page_shift) - 1)) >> g.block_shift;
                        kk[e] = ks[page * g.ks_page + blk * g.ks_block];
                        vv[e] = SHARED ? kk[e] : vs[page * g.vs_page + blk * g.vs_block];
                    }
                }
            };
            float kk[2][4], vv[2][4];
            fetch(sg.t0, kk[0], vv[0]);
            if (sg.n > 1) fetch(sg.t0 + 1, kk[1], vv[1]);
#pragma unroll 1
            for (int k = 0; k < sg.n; ++k, ++i) {
                const int slot = i % kAttn8ScaleSlots;
                alive = await(&sc_empty[slot], static_cast<uint32_t>(i / kAttn8ScaleSlots) ^ 1u);
                alive = __all_sync(0xffffffffu, alive);
                if (!alive) break;
                float *to = scales + slot * 2 * T;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = fminf(fmaxf(vv[0][e], two_to(kQ8MinExp)), two_to(kQ8MaxExp));
                    to[e * 32 + lane] = kk[0][e] * a.scale_log2;
                    to[T + e * 32 + lane] = __log2f(v);
                    kk[0][e] = kk[1][e];
                    vv[0][e] = vv[1][e];
                }
                warp_arrive(&sc_full[slot]);
                if (k + 2 < sg.n) fetch(sg.t0 + k + 2, kk[1], vv[1]);
            }
        }
    } else {
        // ---------------- softmax warps ----------------
        AttnWalk walk(ln);
        int i = 0;
        AttnSegment sg;
        uint32_t seg = 0;
        const int head0 = ht * N;                              // of the group
        const int nheads = min(N, a.group - head0);            // real heads of this tile
        const int all_heads = a.kv_heads * a.group;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
        const int wq = warp & 3, set = warp >> 2;
        const int r0 = wq * 32 + (lane >> 2);                  // this thread's token rows: r0 + 0, 8, 16, 24
        const int c4 = lane & 3;
        const int h0 = set * 16 + c4 * kC;                     // its heads: h0 + 0 .. kC - 1
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        if (a.split && ht == 0 && tid == 96) {
            AttnEntry e;
            e.batch = -1;
            e.kv_head = e.last = e.slot = 0;
            a.entries[cta] = e;
        }
        // heads behind the last one: columns that nothing reads, which move nothing
        uint32_t unused = 0;
#pragma unroll
        for (int c = 0; c < kC; ++c)
            if (h0 + c >= nheads) unused |= 1u << c;
        while (attn_next_segment<T>(a, ln, walk, sg)) {
            const bool begins = sg.t0 == 0, ends = sg.t0 + sg.n == sg.tiles;
            float m[kC];             // reference points
            float2 u[kC / 2], d[kC / 2];  // sums of the unrounded weights, and of what the rounding of the large ones adds
            uint32_t lowest = unused;     // columns whose reference point goes no further down
            float mine = 0.f, peak = 0.f;  // column tid's point, and its highest
#pragma unroll
            for (int e = 0; e < kC; ++e) m[e] = 0.f;
#pragma unroll
            for (int j = 0; j < kC / 2; ++j) u[j] = d[j] = make_float2(0.f, 0.f);
            await(&unit_full[seg & 3u], seg >> 2);
            float2 unit[kC / 2];     // of the heads' queries
#pragma unroll
            for (int j = 0; j < kC / 2; ++j) {
                const uint32_t e = *reinterpret_cast<const uint16_t *>(q_unit + (seg & 3u) * N + h0 + 2 * j);
                unit[j] = make_float2(__uint_as_float((e & 0xffu) << 23), __uint_as_float(e >> 8 << 23));
            }
            ++seg;
            for (int k = 0; k < sg.n; ++k, ++i) {
                const int64_t tok0 = static_cast<int64_t>(sg.t0 + k) * T;
                const int valid = static_cast<int>(min(static_cast<int64_t>(T), sg.len - tok0));
                const float *const sc = scales + i % kAttn8ScaleSlots * 2 * T + r0;
                float ksc[4], vlog[4];
                await(&sc_full[i % kAttn8ScaleSlots], static_cast<uint32_t>(i / kAttn8ScaleSlots));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    ksc[r] = sc[8 * r];
                    vlog[r] = sc[T + 8 * r];
                }
                warp_arrive(&sc_empty[i % kAttn8ScaleSlots]);
                await(&s_full[i & 1], static_cast<uint32_t>(i >> 1));
                tc_fence_after_sync();
                // s[r][j]: row r0 + 8 r, heads h0 + 2 j and + 1, in log2 units with the values' scale
                float2 s[4][kC / 2];
                {
                    float hi[2][8], lo[2][8];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint32_t from = tmem_s + (i & 1) * C::kQRows + set * 16 + lane_base + (static_cast<uint32_t>(hf * 16) << 16);
                        tmem_ld_frag<2>(from, hi[hf]);
                        tmem_ld_frag<2>(from + N, lo[hf]);
                    }
                    tmem_wait_ld();
                    tc_fence_before_sync();
                    warp_arrive(&s_free[i & 1]);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int j = 0; j < kC / 2; ++j) {
                            const int at = 4 * j + 2 * (r & 1);
                            const float2 x = fma2(make_float2(lo[r >> 1][at], lo[r >> 1][at + 1]), make_float2(0.0625f, 0.0625f),
                                                  make_float2(hi[r >> 1][at], hi[r >> 1][at + 1]));
                            // (the unit, a power of two, goes to the scale: with the product of large queries it may pass fp32's range)
                            s[r][j] = fma2(x, mul2(unit[j], make_float2(ksc[r], ksc[r])), make_float2(vlog[r], vlog[r]));
                        }
                }
                if (__builtin_expect(valid < T, false)) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (r0 + 8 * r >= valid) {
#pragma unroll
                            for (int j = 0; j < kC / 2; ++j) s[r][j] = make_float2(-INFINITY, -INFINITY);
                        }
                }
                float mx[kC];
#pragma unroll
                for (int c = 0; c < kC; ++c) mx[c] = fmaxf(fmaxf(col(s[0], c), col(s[1], c)), fmaxf(col(s[2], c), col(s[3], c)));
                // columns that exceed the window, and those that some token reaches from below
                bool over = k == 0;
                uint32_t reached = lowest;
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const float most = mx[c] - m[c];
                    over |= most > kAttn8Up && !((unused >> c) & 1u);
                    if (most >= kAttn8Low) reached |= 1u << c;
                }
                {
                    // kC bits for each of the four places, the warps of a set together
                    const uint32_t all = __reduce_or_sync(0xffffffffu, reached << (c4 * kC));
                    if (lane == 0) seen[(i & 1) * 16 + warp] = all;
                }
                bool move = softmax_any<C::kSoft>(over);
#pragma unroll
                for (int w = 0; w < C::kSets; ++w) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(seen + (i & 1) * 16 + w * 4);
                    move |= (x.x | x.y | x.z | x.w) != 0xffffu;
                }
                if (__builtin_expect(move, false)) {
                    // column maxima over the tile's tokens, new reference points (a column per thread), O^T rescaled
                    if (i > 0) await(pv_done, static_cast<uint32_t>(i - 1));  // (red, fac and points lie where the weights did)
                    tc_fence_after_sync();
#pragma unroll
                    for (int c = 0; c < kC; ++c)
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], d));
                    if (lane < 4) {
#pragma unroll
                        for (int c = 0; c < kC; c += 4)
                            *reinterpret_cast<float4 *>(red + wq * N + h0 + c) = make_float4(mx[c], mx[c + 1], mx[c + 2], mx[c + 3]);
                    }
                    softmax_sync<C::kSoft>();
                    if (tid < N) {
                        const float t = fmaxf(fmaxf(red[tid], red[N + tid]), fmaxf(red[2 * N + tid], red[3 * N + tid]));
                        const float most = t - mine;
                        float n = mine;
                        if (k == 0) n = t > -INFINITY ? floorf(t - kAttn8Aim) : 0.f;  // (0: nothing but NaN or minus infinity)
                        else if (most > kAttn8Up || !(most >= kAttn8Low)) n = fmaxf(floorf(t - kAttn8Aim), peak - kAttn8Down);
                        peak = k == 0 ? n : fmaxf(peak, n);
                        fac[tid] = k == 0 ? 0.f : fast_exp2(mine - n);
                        points[tid] = n;
                        bottom[tid] = n == peak - kAttn8Down ? 1.f : 0.f;
                        mine = n;
                    }
                    softmax_sync<C::kSoft>();
                    lowest = unused;
#pragma unroll
                    for (int j = 0; j < kC / 2; ++j) {
                        const float2 f = *reinterpret_cast<const float2 *>(fac + h0 + 2 * j), n = *reinterpret_cast<const float2 *>(points + h0 + 2 * j);
                        const float2 low = *reinterpret_cast<const float2 *>(bottom + h0 + 2 * j);
                        d[j] = mul2(d[j], f);
                        u[j] = mul2(u[j], f);
                        m[2 * j] = n.x;
                        m[2 * j + 1] = n.y;
                        if (low.x != 0.f) lowest |= 1u << 2 * j;
                        if (low.y != 0.f) lowest |= 2u << 2 * j;
                    }
                    if (k > 0) {
#pragma unroll 1
                        for (int c0 = set * 16; c0 < C::kOT * N; c0 += C::kSets * 16) {
                            float o[16];
                            tmem_ld16(tmem + c0 + lane_base, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= fac[(c0 & (N - 1)) + e];
                            tmem_st16(tmem + c0 + lane_base, o);
                        }
                        tmem_wait_st();
                    }
                    softmax_sync<C::kSoft>();  // (before weights take their place)
                }
                if (__builtin_expect(valid < T, false)) {
                    // the last tile: what lies behind the sequence must not reach the product (0 x NaN).  Its last
                    // step of 32 tokens is filled up with zeros; the steps behind that are not taken.
                    const int first = i * C::kGroups + C::kKG;  // its first value group in the ring
                    if (!SHARED)                                // (a latent tile's scores have waited for it)
                        await(&full[first % a.slots], static_cast<uint32_t>(first / a.slots));
                    constexpr int kPieces = C::kW / 16;
                    int at = first % a.slots;
#pragma unroll
                    for (int gr = 0; gr < C::kVG; ++gr) {
                        for (int e = tid; e < (-valid & 31) * kPieces; e += C::kSoft)
                            *reinterpret_cast<uint4 *>(smem + at * C::kGroupBytes + valid * C::kW + e * 16) = make_uint4(0, 0, 0, 0);
                        at = at + 1 == a.slots ? 0 : at + 1;
                    }
                }
                // the weights in two pieces, and their sums
                uint32_t wh[4], wl[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float v = fast_exp2(-vlog[r]);  // 1 / vs
                    uint32_t h8[2], l8[2];
#pragma unroll
                    for (int j = 0; j < kC / 2; ++j) {
                        float2 p = s[r][j];
                        add2(p, make_float2(-m[2 * j], -m[2 * j + 1]));
                        p = make_float2(fast_exp2(p.x), fast_exp2(p.y));
                        const __half2 p16 = __floats2half2_rn(p.x, p.y);
                        h8[j] = half2_to_e4m3x2(p16);
                        const __half2 rest = __hsub2(p16, e4m3x2_to_half2(h8[j]));
                        l8[j] = half2_to_e5m2x2(rest);
                        // Wh + Wl - w (w as fp16: the 2^-11 between them does not cancel), exact
                        const __half2 off = __hsub2(e5m2x2_to_half2(l8[j]), rest);
                        const uint32_t large = __hge2_mask(p16, __float2half2_rn(kAttn8Large)) & *reinterpret_cast<const uint32_t *>(&off);
                        u[j] = fma2(p, make_float2(v, v), u[j]);
                        d[j] = fma2(__half22float2(*reinterpret_cast<const __half2 *>(&large)), make_float2(v, v), d[j]);
                    }
                    wh[r] = __byte_perm(h8[0], h8[1], 0x5410);
                    wl[r] = __byte_perm(l8[0], l8[1], 0x5410);
                }
                // the weights of tile i - 1 have been read before these replace them
                if (i > 0) await(pv_done, static_cast<uint32_t>(i - 1));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = r0 + 8 * r;
                    uint8_t *line = p_smem + row * C::kPLine + c4 * 4;
                    *reinterpret_cast<uint32_t *>(line + swizzled<C::kPLine>(row, set)) = wh[r];
                    *reinterpret_cast<uint32_t *>(line + swizzled<C::kPLine>(row, C::kSets + set)) = wl[r];
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                warp_arrive(p_full);
            }
            // ---- the part is done: its sums over the tokens, then O^T out of tensor memory ----
            await(pv_done, static_cast<uint32_t>(i - 1));  // (red and fac lie where the weights did)
            tc_fence_after_sync();
            auto over_tokens = [&](float2 (&v)[kC / 2]) {  // a warp's sums to `red`
#pragma unroll
                for (int j = 0; j < kC / 2; ++j)
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        v[j].x += __shfl_xor_sync(0xffffffffu, v[j].x, d);
                        v[j].y += __shfl_xor_sync(0xffffffffu, v[j].y, d);
                    }
                softmax_sync<C::kSoft>();  // the last tile's maxima and factors, the sums l (u) have been read
                if (lane < 4) {
#pragma unroll
                    for (int j = 0; j < kC / 2; ++j) *reinterpret_cast<float2 *>(red + wq * N + h0 + 2 * j) = v[j];
                }
            };
#pragma unroll
            for (int j = 0; j < kC / 2; ++j) add2(d[j], u[j]);
            over_tokens(d);
            if (wq == 0 && lane < 4) {
#pragma unroll
                for (int j = 0; j < kC / 2; ++j) *reinterpret_cast<float2 *>(fac + h0 + 2 * j) = make_float2(m[2 * j], m[2 * j + 1]);
            }
            softmax_sync<C::kSoft>();
            const bool whole = begins && ends;
            const int slot = sg.x0 == ln.x0 ? 0 : 1;
            float *part = a.parts + (static_cast<int64_t>(ht) * a.ctas + cta) * 2 * attn_part(DV, N) + slot * attn_part(DV, N);
            float ref = 0.f;
            if (tid < N) {  // a column per thread
                const float t = red[tid] + red[N + tid] + red[2 * N + tid] + red[3 * N + tid];
                ref = fac[tid];
                if (whole) {
                    fac[tid] = t == 0.f ? 0.f : 1.f / t;
                } else {
                    part[N * DV + tid] = ref;
                    part[N * DV + N + tid] = t;
                }
            }
            if (a.lse) {
                over_tokens(u);
                softmax_sync<C::kSoft>();
                if (tid < N) {
                    const float t = red[tid] + red[N + tid] + red[2 * N + tid] + red[3 * N + tid];
                    if (!whole)
                        part[N * DV + 2 * N + tid] = t;
                    else if (tid < nheads && *abort_flag == 0)
                        a.lse[static_cast<int64_t>(sg.b) * all_heads + sg.kv * a.group + head0 + tid] =
                            t == 0.f ? -INFINITY : (ref + log2f(t)) * 0.6931471805599453f;
                }
            }
            if (ht == 0 && tid == 96 && begins && !ends) {
                AttnEntry e;
                e.batch = sg.b;
                e.kv_head = sg.kv;
                e.last = line_owner(ln.total, sg.end - 1, ln.ctas);
                e.slot = slot;
                a.entries[cta] = e;
            }
            softmax_sync<C::kSoft>();
            const bool good = *abort_flag == 0;
            const int64_t obase = (static_cast<int64_t>(sg.b) * all_heads + sg.kv * a.group + head0) * DV;
            attn_store_part<N, DV, C::kMV, C::kOT, C::kSets>(tmem, wq, lane, good, whole, nheads, fac, out + obase, part, set);
            tc_fence_before_sync();
            softmax_sync<C::kSoft>();  // red and fac are free again
        }
        if (tid < 128) attn_store_empty<DV>(a, cta, head0, nheads);
    }
    tc_fence_before_sync();
    if (a.split) {  // the join waits for the end of this grid: no fence
        __syncthreads();
        griddep_launch_dependents();
    } else {
        cta_release_and_trigger();
    }
    if (*abort_flag != 0 && tid == 0) {
        atomicCAS(a.err_word, 0, kDeviceErrTimeout);
        // copies still in flight land before the shared memory goes
        const int n = issued[0], nx = issued[1];
        auto land = [&](uint64_t *bar, int phase) {
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(smem_u32(bar), static_cast<uint32_t>(phase) & 1u) && global_timer_ns() - t0 < a.wait_limit_ns / 16 + 1) {
            }
        };
        for (int j = max(0, n - a.slots); j < n; ++j)
            if (j / C::kGroups != a.skip_tile) land(&full[j % a.slots], j / a.slots);
        if (issued[2] > 0) land(q_full, issued[2] - 1);
        for (int j = max(0, issued[2] - 4); j < issued[2]; ++j) land(&unit_full[j & 3], j >> 2);
        if (C::kRope)
            for (int j = max(0, nx - C::kX); j < nx; ++j)
                if (j != a.skip_tile) land(&x_full[j % max(C::kX, 1)], j / max(C::kX, 1));
    }
    if (warp == C::kRoles + 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    __syncthreads();
}

}  // namespace hsp
