// attn_kernel.cuh -- attention of one new token per sequence over a paged cache.
//
//   o[b, h] = sum_t p_t v[t],  p = softmax_t(scale * q[b, h] . k[t]),  t < len_b
//
// One kernel for the latent cache (one key head of 576 or 512 columns whose first 512
// columns are the values: a key tile is read once and used twice) and for grouped heads
// (keys and values of 64 or 128 columns, `group` query heads per key head).
//
// Both products run on tcgen05 with the TOKENS (or the value columns) on the 128/64-row
// side and the query heads as the N columns, so a handful of heads still uses whole
// instructions:
//   S^T[64 tokens x N heads] = K[64 x dk] . Q[N x dk]^T       (M = 64, both operands K-major)
//   O^T[dv x N heads]       += V^T[dv x 64] . P^T[64 x N]     (M = 128 or 64, both operands
//                                                              MN-major: V as it lies in the
//                                                              tile, P stored token by token)
// O^T stays in tensor memory for a whole sequence part (dv/128 x N columns), S^T is double
// buffered next to it, so the scores of tile i + 1 are computed while tile i is in its softmax.
//
// Softmax over the length in one pass: the running maximum m is only a reference point,
// kept while no new score exceeds it by more than 8 in log2 units (p <= 2^8, the sums are
// fp32 and bf16 keeps its relative precision), so most tiles need no exchange between the
// threads but one barrier with an OR; a tile that exceeds it takes the column maxima over
// all warps and rescales O^T.  P is rounded to bf16 for the product (2^-9 relative per
// weight, the sum l adds the unrounded values), all sums and statistics are fp32.
//
// The tokens of all sequences, each a multiple of 64, form one line that is cut evenly over
// the CTAs (grid.y), so ragged batches balance; CTAs of one y and different x take the
// different head tiles of the same tokens at the same time (the second read hits L2).  A
// sequence cut over several CTAs leaves fp32 partials (O^T, m, l) in the workspace, and the
// join kernel adds them in CTA order; the cut depends on the lengths and the grid only.
//
// Bound by the cache's bytes: a latent tile is 73.7 KB per 64 tokens.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "cache_args.h"
#include "ptx.cuh"
#include "stream_args.h"

namespace hsp {

// ---- tcgen05 pieces used only here -------------------------------------------------

// MN-major operand in the 128-byte-swizzled layout of a tensor copy: 64 consecutive
// M (or N) elements per 128-byte line, lines one K apart; `lead` bytes between groups of
// 64 elements, 1024 bytes between groups of eight K.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t smem_addr, uint32_t lead) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(lead >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// 16 lanes x 8 columns per step: register 4j + e of lane l holds row l/4 + 8 (e/2), column
// 8j + 2 (l mod 4) + (e mod 2) -- the fragment layout of an m16n8 accumulator.
template <int STEPS>
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[STEPS * 4]);
template <>
__device__ __forceinline__ void tmem_ld_frag<2>(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
template <>
__device__ __forceinline__ void tmem_ld_frag<4>(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
template <>
__device__ __forceinline__ void tmem_ld_frag<8>(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
        "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
        "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
        "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
        "r"(__float_as_uint(v[15]))
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 5-D tensor copy (coordinates innermost first).
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2,
                                            int32_t c3, int32_t c4, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}

// Barrier 1 of the 128 softmax threads, and the same with an OR over their predicates.
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync.aligned 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred.aligned q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(p))
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bounded wait.  Once any thread of the CTA has given up, waits that are not yet satisfied
// return at once; the roles keep their barrier pattern and store nothing.
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int *abort_flag,
                                          int *err_word) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 7u) == 7u) {
            if (*abort_flag != 0) return false;
            if (global_timer_ns() - t0 > limit_ns) {
                atomicCAS(err_word, 0, kDeviceErrTimeout);
                *abort_flag = 1;
                return false;
            }
        }
    }
}

// ---- the line of tiles ---------------------------------------------------------------

// Length of sequence b, clamped to what its table row can hold; a row outside the table
// is an empty sequence.  Both are reported.
__device__ __forceinline__ int attn_len(const AttnArgs &a, int b) {
    const int row = a.rows ? a.rows[b] : b;
    if (row < 0 || row >= a.num_rows) {
        atomicCAS(a.err_word, 0, kDeviceErrIndex);
        return 0;
    }
    const int n = a.lens[row];
    const int64_t most = static_cast<int64_t>(a.max_pages) << a.page_shift;
    if (n < 0 || n > most) {
        atomicCAS(a.err_word, 0, kDeviceErrIndex);
        return n < 0 ? 0 : static_cast<int>(most);
    }
    return n;
}
__device__ __forceinline__ int attn_tiles(int len) { return static_cast<int>((static_cast<uint32_t>(len) + kAttnTile - 1) / kAttnTile); }

// First tile of CTA c of C over a line of T tiles, and the CTA that holds tile x.
__device__ __forceinline__ int64_t line_start(int64_t T, int c, int C) { return T * c / C; }
__device__ __forceinline__ int line_owner(int64_t T, int64_t x, int C) {
    return static_cast<int>(((x + 1) * C + T - 1) / T) - 1;
}

// Where a CTA's tiles lie: set up once, then walked by every role alike.
struct AttnLine {
    int64_t total;    // T
    int64_t x0, x1;   // this CTA's tiles
    int64_t base;     // tiles (of one kv head) before sequence b0
    int32_t b0;
    int32_t ctas;     // CTAs that hold tiles
};
struct AttnSegment {
    int b, kv, len, t0, n, tiles;  // n tiles from t0 of the sequence's `tiles`
};

__device__ __forceinline__ bool attn_next_segment(const AttnArgs &a, const AttnLine &ln, int64_t &x, int &b, int64_t &base,
                                                  AttnSegment &s) {
    if (x >= ln.x1) return false;
    int len, tiles;
    for (;;) {
        if (b >= a.batch) return false;  // (lengths that changed under the call)
        len = attn_len(a, b);
        tiles = attn_tiles(len);
        if (x < (base + tiles) * a.kv_heads) break;
        base += tiles;
        ++b;
    }
    const int64_t rel = x - base * a.kv_heads;
    s.b = b;
    s.kv = static_cast<int>(rel / tiles);
    s.t0 = static_cast<int>(rel - static_cast<int64_t>(s.kv) * tiles);
    s.len = len;
    s.tiles = tiles;
    const int64_t left = ln.x1 - x;
    s.n = static_cast<int>(min(static_cast<int64_t>(tiles - s.t0), left));
    x += s.n;
    return true;
}

template <int KB, int VB, bool SHARED, int N>
struct AttnCfg {
    static constexpr int kDV = VB * 64;
    static constexpr int kMV = kDV >= 128 ? 128 : 64;       // rows of one O^T instruction
    static constexpr int kOT = kDV / kMV;                   // O^T tiles
    static constexpr int kCols = kOT * N + 2 * N;           // O^T, then two S^T
    static constexpr uint32_t kTmemCols = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static_assert(kCols <= 512, "tensor memory");
    static constexpr int kStageBytes = (KB + (SHARED ? 0 : VB)) * kAttnTile * 128;
    static constexpr int kVOff = SHARED ? 0 : KB * kAttnTile * 128;  // value boxes in a stage
    static constexpr int kQBytes = KB * N * 128;
    static constexpr int kPBytes = kAttnTile * 128;
};

template <int KB, int VB, bool SHARED, int N>
__global__ void __launch_bounds__(kAttnThreads, 1)
    hsp_attn_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                    const __grid_constant__ AttnArgs a) {
    using C = AttnCfg<KB, VB, SHARED, N>;
    constexpr int kS = N / 8;          // 8-column steps of S^T
    constexpr int kDV = C::kDV;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t ring = smem_u32(smem);
    uint8_t *const q_smem = smem + a.stages * C::kStageBytes;
    uint8_t *const p_smem = q_smem + C::kQBytes;
    float *const red = reinterpret_cast<float *>(p_smem + C::kPBytes);  // [4 warps][N]
    float *const fac = red + 4 * N;                                     // [N]
    uint64_t *const full = reinterpret_cast<uint64_t *>(fac + N);       // [stages]
    uint64_t *const empty = full + a.stages;
    uint64_t *const s_full = empty + a.stages;                          // [2]
    uint64_t *const q_full = s_full + 2;
    uint64_t *const p_full = q_full + 1;
    uint64_t *const pv_done = p_full + 1;
    uint64_t *const drained = pv_done + 1;
    AttnLine *const line = reinterpret_cast<AttnLine *>(drained + 1);
    int *const ints = reinterpret_cast<int *>(line + 1);
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(ints);
    volatile int *const abort_flag = ints + 1;
    int *const issued = ints + 2;                                       // tiles whose copies were issued
    int *const warp_sum = ints + 4;                                     // [6]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ht = blockIdx.x, cta = blockIdx.y;

    if (tid == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(&s_full[0]), 1);
        mbar_init(smem_u32(&s_full[1]), 1);
        mbar_init(smem_u32(q_full), 128);
        mbar_init(smem_u32(p_full), 128);
        mbar_init(smem_u32(pv_done), 1);
        mbar_init(smem_u32(drained), 1);
        *abort_flag = 0;
        *issued = 0;
        mbar_fence_init();
        tma_prefetch_map(&tmap_k);
        if (!SHARED) tma_prefetch_map(&tmap_v);
    }
    if (warp == 5) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    griddep_wait();  // everything read below may come from the previous kernel

    // ---- the line: total tiles, and where this CTA's first tile lies ----
    const int per = (a.batch + kAttnThreads - 1) / kAttnThreads;
    const int bfirst = min(a.batch, tid * per), blast = min(a.batch, bfirst + per);
    int mine = 0;
    for (int b = bfirst; b < blast; ++b) mine += attn_tiles(attn_len(a, b));
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kAttnThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        all += warp_sum[w];
    }
    const int64_t T = static_cast<int64_t>(all) * a.kv_heads;
    const int64_t want = (T + a.min_tiles - 1) / a.min_tiles;
    const int nctas = static_cast<int>(min(want, static_cast<int64_t>(a.ctas)));
    const int64_t x0 = cta < nctas ? line_start(T, cta, nctas) : T, x1 = cta < nctas ? line_start(T, cta + 1, nctas) : T;
    {
        const int64_t first = static_cast<int64_t>(before + incl - mine) * a.kv_heads;
        if (tid == 0) {
            line->total = T;
            line->x0 = x0;
            line->x1 = x1;
            line->ctas = nctas;
            line->b0 = a.batch;
            line->base = 0;
        }
        __syncthreads();
        if (x0 < x1 && x0 >= first && x0 < first + static_cast<int64_t>(mine) * a.kv_heads) {
            line->b0 = bfirst;
            line->base = before + incl - mine;
        }
        __syncthreads();
    }
    const uint32_t tmem = *tmem_slot;
    const uint32_t tmem_s = tmem + C::kOT * N;
    const AttnLine ln = *line;

    if (warp == 4) {
        // ---------------- copy producer: the whole warp reads the table, lanes issue ----------------
        int64_t x = ln.x0, base = ln.base;
        int b = ln.b0, i = 0;
        AttnSegment sg;
        const int pbox = min(kAttnTile, 1 << a.page_shift);         // tokens per box
        const int boxes = kAttnTile / pbox;                         // pages that meet a tile
        bool alive = true;
        while (alive && attn_next_segment(a, ln, x, b, base, sg)) {
            const int row = a.rows ? a.rows[sg.b] : sg.b;
            const int32_t *tbl = a.table + row * a.table_stride;
            const int pages = static_cast<int>((static_cast<int64_t>(sg.len) + (1 << a.page_shift) - 1) >> a.page_shift);
            int win0 = -64, win = 0;
            for (int k = 0; k < sg.n && alive; ++k, ++i) {
                const int64_t tok = static_cast<int64_t>(sg.t0 + k) * kAttnTile;
                const int p0 = static_cast<int>(tok >> a.page_shift);
                if (p0 + boxes > win0 + 32) {  // the next 32 ids in one load
                    win0 = p0;
                    win = 0;
                    if (p0 + lane < pages) {
                        win = tbl[p0 + lane];
                        if (win < 0 || win >= a.num_pages) {
                            atomicCAS(a.err_word, 0, kDeviceErrIndex);
                            win = 0;  // stays inside the pool; the call is reported
                        }
                    }
                }
                const int slot = i % a.stages;
                const uint32_t fb = smem_u32(&full[slot]);
                if (i >= a.stages) {
                    int ok = 1;
                    if (lane == 0)
                        ok = attn_wait(smem_u32(&empty[slot]), static_cast<uint32_t>(i / a.stages - 1) & 1u, a.wait_limit_ns,
                                       abort_flag, a.err_word);
                    if (!__shfl_sync(0xffffffffu, ok, 0)) {
                        alive = false;
                        break;
                    }
                }
                if (i == a.skip_tile) continue;
                const int np = min(boxes, pages - p0);
                const uint32_t bytes = static_cast<uint32_t>(np * pbox * 128 * (KB + (SHARED ? 0 : VB)));
                const uint32_t dst = ring + slot * C::kStageBytes;
                const int id0 = __shfl_sync(0xffffffffu, win, p0 - win0);
                if (lane == 0) {
                    mbar_arrive_expect_tx(fb, bytes);
                    *issued = i + 1;
                    if (boxes == 1) {
                        const int off = static_cast<int>(tok & ((1 << a.page_shift) - 1));
                        tma_load_5d(dst, &tmap_k, 0, off, 0, sg.kv, id0, fb);
                        if (!SHARED) tma_load_5d(dst + C::kVOff, &tmap_v, 0, off, 0, sg.kv, id0, fb);
                    }
                }
                if (boxes > 1) {  // small pages: one copy per page and 64 columns, shared out over the lanes
                    __syncwarp();
                    for (int e0 = 0; e0 < np * KB; e0 += 32) {
                        const int e = e0 + lane, pg = e / KB, kb = e - pg * KB;
                        const int id = __shfl_sync(0xffffffffu, win, (p0 - win0 + pg) & 31);
                        if (e < np * KB)
                            tma_load_5d(dst + kb * (kAttnTile * 128) + pg * pbox * 128, &tmap_k, 0, 0, kb, sg.kv, id, fb);
                    }
                    if (!SHARED)
                        for (int e0 = 0; e0 < np * VB; e0 += 32) {
                            const int e = e0 + lane, pg = e / VB, vb = e - pg * VB;
                            const int id = __shfl_sync(0xffffffffu, win, (p0 - win0 + pg) & 31);
                            if (e < np * VB)
                                tma_load_5d(dst + C::kVOff + vb * (kAttnTile * 128) + pg * pbox * 128, &tmap_v, 0, 0, vb,
                                            sg.kv, id, fb);
                        }
                }
            }
        }
    } else if (warp == 5) {
        // ---------------- MMA issuer ----------------
        if (lane == 0) {
            constexpr uint32_t kBase = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17);
            constexpr uint32_t kDescS = kBase | (static_cast<uint32_t>(kAttnTile >> 4) << 24);
            constexpr uint32_t kDescO = kBase | (1u << 15) | (1u << 16) | (static_cast<uint32_t>(C::kMV >> 4) << 24);
            int64_t x = ln.x0, base = ln.base;
            int b = ln.b0, i = 0;
            uint32_t seg = 0;
            AttnSegment sg;
            bool alive = true;
            const uint32_t qa = smem_u32(q_smem), pa = smem_u32(p_smem);
            auto scores = [&](int j) {
                const int slot = j % a.stages;
                if (!attn_wait(smem_u32(&full[slot]), static_cast<uint32_t>(j / a.stages) & 1u, a.wait_limit_ns, abort_flag,
                               a.err_word))
                    return false;
                tc_fence_after_sync();
                const uint32_t ka = ring + slot * C::kStageBytes;
                const uint32_t d = tmem_s + (j & 1) * N;
#pragma unroll 1
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_f16(d, umma_desc_sw128(ka + kb * (kAttnTile * 128) + k * 32),
                                 umma_desc_sw128(qa + kb * (N * 128) + k * 32), kDescS, (kb | k) != 0 ? 1u : 0u);
                umma_commit(smem_u32(&s_full[j & 1]));
                return true;
            };
            while (alive && attn_next_segment(a, ln, x, b, base, sg)) {
                if (!attn_wait(smem_u32(q_full), seg & 1u, a.wait_limit_ns, abort_flag, a.err_word)) break;
                ++seg;
                alive = scores(i);
                for (int k = 0; k < sg.n && alive; ++k, ++i) {
                    if (k + 1 < sg.n && !(alive = scores(i + 1))) break;
                    if (!(alive = attn_wait(smem_u32(p_full), static_cast<uint32_t>(i) & 1u, a.wait_limit_ns, abort_flag,
                                            a.err_word)))
                        break;
                    tc_fence_after_sync();
                    const int slot = i % a.stages;
                    const uint32_t va = ring + slot * C::kStageBytes + C::kVOff;
#pragma unroll 1
                    for (int jt = 0; jt < C::kOT; ++jt)
#pragma unroll
                        for (int kk = 0; kk < kAttnTile / 16; ++kk)
                            umma_f16(tmem + jt * N,
                                     umma_desc_mn_sw128(va + jt * (C::kMV / 64) * (kAttnTile * 128) + kk * 2048, kAttnTile * 128),
                                     umma_desc_mn_sw128(pa + kk * 2048, kAttnTile * 128), kDescO, (k | kk) != 0 ? 1u : 0u);
                    umma_commit(smem_u32(&empty[slot]));
                    umma_commit(smem_u32(pv_done));
                }
            }
            // always committed and awaited, so that no product is in flight when the memory goes
            umma_commit(smem_u32(drained));
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(smem_u32(drained), 0u) && global_timer_ns() - t0 < a.wait_limit_ns) {
            }
        }
        __syncwarp();
    } else {
        // ---------------- softmax warps ----------------
        int64_t x = ln.x0, base = ln.base;
        int b = ln.b0, i = 0;
        AttnSegment sg;
        const int head0 = ht * N;                              // of the group
        const int nheads = min(N, a.group - head0);            // real heads of this tile
        const int all_heads = a.kv_heads * a.group;
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q);
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
        const int r0 = warp * 16 + (lane >> 2);                // this thread's token rows: r0 and r0 + 8
        const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
        constexpr float kFloor = -3.0e38f;
        if (ht == 0 && tid == 0) {
            AttnEntry e;
            e.batch = -1;
            e.kv_head = e.last = e.slot = 0;
            a.entries[cta] = e;
        }
        while (attn_next_segment(a, ln, x, b, base, sg)) {
            const int64_t seg_x0 = x - sg.n;
            const bool begins = sg.t0 == 0, ends = sg.t0 + sg.n == sg.tiles;
            const int64_t qrow = static_cast<int64_t>(sg.b);
            // queries of this head tile, K-major with the 128-byte swizzle; rows past the heads are zero
            {
                const __nv_bfloat16 *qb = q + qrow * a.q_row + static_cast<int64_t>(sg.kv * a.group + head0) * a.q_head;
#pragma unroll 4
                for (int e = tid; e < N * KB * 8; e += 128) {
                    const int r = e / (KB * 8), ch = e - r * (KB * 8);
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (r < nheads) v = *reinterpret_cast<const uint4 *>(qb + r * a.q_head + ch * 8);
                    *reinterpret_cast<uint4 *>(q_smem + (ch >> 3) * (N * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
                }
                fence_proxy_async_smem();
                mbar_arrive(smem_u32(q_full));
            }
            float m[kS * 2], l[kS * 2];
#pragma unroll
            for (int e = 0; e < kS * 2; ++e) {
                m[e] = kFloor;
                l[e] = 0.f;
            }
            for (int k = 0; k < sg.n; ++k, ++i) {
                const int64_t tok0 = static_cast<int64_t>(sg.t0 + k) * kAttnTile;
                const int valid = static_cast<int>(min(static_cast<int64_t>(kAttnTile), sg.len - tok0));
                attn_wait(smem_u32(&s_full[i & 1]), static_cast<uint32_t>(i >> 1) & 1u, a.wait_limit_ns, abort_flag, a.err_word);
                tc_fence_after_sync();
                float s[kS * 4];
                tmem_ld_frag<kS>(tmem_s + (i & 1) * N + lane_base, s);
                if (valid < kAttnTile) {
                    // the last tile: what lies behind the sequence must not reach the product (0 x NaN)
                    uint8_t *v = smem + (i % a.stages) * C::kStageBytes + C::kVOff;
                    const int lines = (kAttnTile - valid) * VB;
                    for (int e = tid; e < lines * 8; e += 128) {
                        const int ln2 = e >> 3, vb = ln2 / (kAttnTile - valid), r = valid + ln2 - vb * (kAttnTile - valid);
                        *reinterpret_cast<uint4 *>(v + vb * (kAttnTile * 128) + r * 128 + ((e & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                }
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < kS * 4; ++e) s[e] *= a.scale_log2;
                const bool ok0 = r0 < valid, ok1 = r0 + 8 < valid;
                bool over = (k == 0);
#pragma unroll
                for (int j = 0; j < kS; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (!ok0) s[4 * j + e] = -INFINITY;
                        if (!ok1) s[4 * j + 2 + e] = -INFINITY;
                        over = over || fmaxf(s[4 * j + e], s[4 * j + 2 + e]) > m[2 * j + e] + 8.f;
                    }
                if (softmax_any(over)) {
                    // column maxima over the tile's 64 tokens, a new reference point, O^T rescaled
                    float mx[kS * 2];
#pragma unroll
                    for (int j = 0; j < kS; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float t = fmaxf(s[4 * j + e], s[4 * j + 2 + e]);
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                            mx[2 * j + e] = t;
                        }
                    if (lane < 4) {
#pragma unroll
                        for (int j = 0; j < kS; ++j)
                            *reinterpret_cast<float2 *>(red + warp * N + 8 * j + 2 * lane) = make_float2(mx[2 * j], mx[2 * j + 1]);
                    }
                    softmax_sync();
#pragma unroll
                    for (int j = 0; j < kS; ++j) {
                        const int c = 8 * j + 2 * (lane & 3);
                        float2 t = *reinterpret_cast<const float2 *>(red + c);
#pragma unroll
                        for (int w = 1; w < 4; ++w) {
                            const float2 u = *reinterpret_cast<const float2 *>(red + w * N + c);
                            t.x = fmaxf(t.x, u.x);
                            t.y = fmaxf(t.y, u.y);
                        }
                        const float n0 = fmaxf(m[2 * j], t.x), n1 = fmaxf(m[2 * j + 1], t.y);
                        const float f0 = fast_exp2(m[2 * j] - n0), f1 = fast_exp2(m[2 * j + 1] - n1);
                        m[2 * j] = n0;
                        m[2 * j + 1] = n1;
                        l[2 * j] *= f0;
                        l[2 * j + 1] *= f1;
                        if (warp == 0 && lane < 4) *reinterpret_cast<float2 *>(fac + c) = make_float2(f0, f1);
                    }
                    if (k > 0) {
                        attn_wait(smem_u32(pv_done), static_cast<uint32_t>(i - 1) & 1u, a.wait_limit_ns, abort_flag, a.err_word);
                        tc_fence_after_sync();
                        softmax_sync();
#pragma unroll 1
                        for (int c0 = 0; c0 < C::kOT * N; c0 += 16) {
                            float o[16];
                            tmem_ld16(tmem + c0 + lane_base, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= fac[(c0 & (N - 1)) + e];
                            tmem_st16(tmem + c0 + lane_base, o);
                        }
                        tmem_wait_st();
                    }
                }
                // the probabilities of tile i - 1 have been read before these replace them
                if (i > 0)
                    attn_wait(smem_u32(pv_done), static_cast<uint32_t>(i - 1) & 1u, a.wait_limit_ns, abort_flag, a.err_word);
#pragma unroll
                for (int j = 0; j < kS; ++j) {
                    const float p00 = fast_exp2(s[4 * j] - m[2 * j]), p01 = fast_exp2(s[4 * j + 1] - m[2 * j + 1]);
                    const float p10 = fast_exp2(s[4 * j + 2] - m[2 * j]), p11 = fast_exp2(s[4 * j + 3] - m[2 * j + 1]);
                    l[2 * j] += p00 + p10;
                    l[2 * j + 1] += p01 + p11;
                    const __nv_bfloat162 u = __floats2bfloat162_rn(p00, p01), w = __floats2bfloat162_rn(p10, p11);
                    uint8_t *pr = p_smem + r0 * 128 + ((j ^ (r0 & 7)) << 4) + (lane & 3) * 4;
                    *reinterpret_cast<__nv_bfloat162 *>(pr) = u;
                    *reinterpret_cast<__nv_bfloat162 *>(pr + 8 * 128) = w;
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                mbar_arrive(smem_u32(p_full));
            }
            // ---- the part is done: l over the tokens, then O^T out of tensor memory ----
#pragma unroll
            for (int e = 0; e < kS * 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
            }
            softmax_sync();  // the last tile's maxima have been read
            if (lane < 4) {
#pragma unroll
                for (int j = 0; j < kS; ++j)
                    *reinterpret_cast<float2 *>(red + warp * N + 8 * j + 2 * lane) = make_float2(l[2 * j], l[2 * j + 1]);
            }
            softmax_sync();
            const bool whole = begins && ends;
            const int slot = seg_x0 == ln.x0 ? 0 : 1;
            float *part = a.parts + (static_cast<int64_t>(ht) * a.ctas + cta) * 2 * (N * kDV + 2 * N) + slot * (N * kDV + 2 * N);
            if (warp == 0 && lane < 4) {
#pragma unroll
                for (int j = 0; j < kS; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = 8 * j + 2 * lane + e;
                        const float t = red[c] + red[N + c] + red[2 * N + c] + red[3 * N + c];
                        if (whole) {
                            fac[c] = t == 0.f ? 0.f : 1.f / t;
                            if (a.lse && c < nheads && *abort_flag == 0)
                                a.lse[static_cast<int64_t>(sg.b) * all_heads + sg.kv * a.group + head0 + c] =
                                    t == 0.f ? -INFINITY : (m[2 * j + e] + log2f(t)) * 0.6931471805599453f;
                        } else {
                            part[N * kDV + c] = m[2 * j + e];
                            part[N * kDV + N + c] = t;
                        }
                    }
            }
            if (ht == 0 && tid == 0 && begins && !ends) {
                AttnEntry e;
                e.batch = sg.b;
                e.kv_head = sg.kv;
                e.last = line_owner(ln.total, seg_x0 + sg.tiles - 1, ln.ctas);
                e.slot = slot;
                a.entries[cta] = e;
            }
            attn_wait(smem_u32(pv_done), static_cast<uint32_t>(i - 1) & 1u, a.wait_limit_ns, abort_flag, a.err_word);
            tc_fence_after_sync();
            softmax_sync();
            const bool good = *abort_flag == 0;
            const int rpw = C::kMV / 4;
            const int64_t obase = (static_cast<int64_t>(sg.b) * all_heads + sg.kv * a.group + head0) * kDV;
#pragma unroll 1
            for (int c0 = 0; c0 < C::kOT * N; c0 += 16) {
                const int h0 = c0 & (N - 1);
                if (h0 >= nheads) continue;
                float o[16];
                tmem_ld16(tmem + c0 + lane_base, o);
                tmem_wait_ld();
                const int dv = (c0 / N) * C::kMV + warp * rpw + lane;
                if (lane < rpw && good) {
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (h0 + e < nheads)
                                out[obase + static_cast<int64_t>(h0 + e) * kDV + dv] = __float2bfloat16_rn(o[e] * fac[h0 + e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (h0 + e < nheads) part[(h0 + e) * kDV + dv] = o[e];
                    }
                }
            }
            tc_fence_before_sync();
            softmax_sync();  // red and fac are free again
        }
        // sequences without a token: zeros, and no weight at all
        for (int e = cta; e < a.batch; e += a.ctas) {
            if (attn_len(a, e) != 0) continue;
            for (int kv = 0; kv < a.kv_heads; ++kv) {
                const int64_t h = static_cast<int64_t>(e) * all_heads + kv * a.group + head0;
                for (int c = tid; c < nheads * kDV; c += 128) out[h * kDV + c] = __float2bfloat16_rn(0.f);
                if (a.lse)
                    for (int c = tid; c < nheads; c += 128) a.lse[h + c] = -INFINITY;
            }
        }
        fence_release_gpu();
    }
    tc_fence_before_sync();
    __syncthreads();
    griddep_launch_dependents();
    if (*abort_flag != 0 && tid == 0) {
        // copies still in flight land before the shared memory goes
        const int n = *issued;
        for (int j = max(0, n - a.stages); j < n; ++j) {
            if (j == a.skip_tile) continue;
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(smem_u32(&full[j % a.stages]), static_cast<uint32_t>(j / a.stages) & 1u) &&
                   global_timer_ns() - t0 < a.wait_limit_ns / 16 + 1) {
            }
        }
    }
    if (warp == 5) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    __syncthreads();
}

// ---- join ------------------------------------------------------------------------------
//
// Sequences cut over several CTAs: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i, the
// parts in CTA order.  A unit is one head and 128 value columns; eight warps take the parts
// in turn and add their sums in warp order.

constexpr int kJoinThreads = 256;

template <int DV, int N>
__global__ void __launch_bounds__(kJoinThreads) hsp_attn_join_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int kCols = DV < 128 ? DV : 128;  // columns of a unit
    constexpr int kParts = DV / kCols;
    constexpr int kPart = N * DV + 2 * N;       // floats of one partial
    __shared__ float4 acc_s[8][32];
    __shared__ int list[kAttnMaxCtas];
    __shared__ uint32_t begun[kAttnMaxCtas / 32];  // bit c: CTA c began a part
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_wait();
    // the parts to join, in CTA order in every CTA of this kernel: its units are shared out by their place
    for (int c = tid; c < kAttnMaxCtas; c += kJoinThreads) {
        const uint32_t m = __ballot_sync(0xffffffffu, c < a.ctas && a.entries[c].batch >= 0);
        if (lane == 0) begun[c >> 5] = m;
    }
    __syncthreads();
    int n = 0;
    for (int w = 0; w < kAttnMaxCtas / 32; ++w) {
        if (warp == (w & 7) && ((begun[w] >> lane) & 1u)) list[n + __popc(begun[w] & ((1u << lane) - 1u))] = w * 32 + lane;
        n += __popc(begun[w]);
    }
    __syncthreads();
    const int64_t units = static_cast<int64_t>(n) * a.group * kParts;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int item = static_cast<int>(u / (a.group * kParts));
        const int rem = static_cast<int>(u - static_cast<int64_t>(item) * (a.group * kParts));
        const int h = rem / kParts, dp = rem - h * kParts;
        const int c0 = list[item];
        const AttnEntry e = a.entries[c0];
        const int ht = h / N, col = h - ht * N;
        const float *first = a.parts + ((static_cast<int64_t>(ht) * a.ctas + c0) * 2 + e.slot) * kPart;
        const float *next = a.parts + (static_cast<int64_t>(ht) * a.ctas + c0 + 1) * 2 * kPart;  // slot 0 of CTA c0 + 1
        const int parts = min(e.last, a.ctas - 1) - c0 + 1;
        auto part = [&](int p) { return p == 0 ? first : next + static_cast<int64_t>(p - 1) * 2 * kPart; };
        float M = -3.0e38f;
        for (int p = lane; p < parts; p += 32) M = fmaxf(M, part(p)[N * DV + col]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        float L = 0.f;
        for (int p = lane; p < parts; p += 32) L += part(p)[N * DV + N + col] * fast_exp2(part(p)[N * DV + col] - M);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane * 4 < kCols) {
#pragma unroll 4
            for (int p = warp; p < parts; p += 8) {
                const float *pp = part(p);
                const float w = fast_exp2(pp[N * DV + col] - M);
                const float4 v = *reinterpret_cast<const float4 *>(pp + col * DV + dp * kCols + lane * 4);
                acc.x += w * v.x;
                acc.y += w * v.y;
                acc.z += w * v.z;
                acc.w += w * v.w;
            }
        }
        acc_s[warp][lane] = acc;
        __syncthreads();
        const int64_t oh = static_cast<int64_t>(e.batch) * a.kv_heads * a.group + e.kv_head * a.group + h;
        if (warp == 0 && lane * 4 < kCols) {
#pragma unroll
            for (int w = 1; w < 8; ++w) {
                const float4 v = acc_s[w][lane];
                acc.x += v.x;
                acc.y += v.y;
                acc.z += v.z;
                acc.w += v.w;
            }
            const float inv = L == 0.f ? 0.f : 1.f / L;
            __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
            uint2 o;
            o.x = *reinterpret_cast<uint32_t *>(&lo);
            o.y = *reinterpret_cast<uint32_t *>(&hi);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + oh * DV + dp * kCols + lane * 4) = o;
            if (a.lse && dp == 0 && lane == 0) a.lse[oh] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        }
        __syncthreads();
    }
    fence_release_gpu();
    __syncthreads();
    griddep_launch_dependents();
}

}  // namespace hsp
