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
// Measured cycles per instruction (one SM, operands in shared memory, products back to back):
// 64 x 64 x 16 33, 128 x 64 x 16 49, 128 x 16 x 16 40; a latent tile of 64 heads is 36 of the
// first and 16 of the second, 1970 cycles, against 3140 that its bytes take at 1/152 of the
// device's bandwidth, so up to 64 heads wait for memory and 128 (two CTAs sharing the bytes)
// for the chain of a tile's copy, products and softmax.
//
// Seven warps: a copy producer (one thread: page ids a tile ahead, one tensor copy per group of
// 128 columns, or per page and 64 columns where pages are smaller than a tile), an issuer of
// the scores, an issuer of the products with the values (each one elected thread), and four
// softmax warps that also carry O^T out.  They meet at mbarriers only; every wait is bounded.
//
// Softmax over the length in one pass: the running maximum m is only a reference point,
// kept while no new score exceeds it by more than 8 in log2 units (p <= 2^8, the sums are
// fp32 and bf16 keeps its relative precision), so most tiles need no exchange between the
// threads but one barrier with an OR; a tile that exceeds it takes the column maxima over
// all warps and rescales O^T.  P is rounded to bf16 for the product (at most 2^-8 relative per
// weight; the values are bf16, and one instruction takes one type).  O^T is divided by the sum l
// of the rounded weights, so the rounding that all of a row's weight has in common cancels and a
// token with nearly all the weight comes out as it is; lse takes the sum u of the unrounded
// ones.  All sums and statistics are fp32.
//
// The tiles of all sequences form one line that is cut over the CTAs (grid.y), so ragged
// batches balance; CTAs of one y and different x take the different head tiles of the same
// tokens at the same time (DRAM reads of 128 heads in two tiles: 158 MB for 157 MB of cache).  A
// sequence cut over several CTAs leaves fp32 partials (O^T, m, l, u) in the workspace, and the
// join kernel adds them; the cut depends on the lengths and the grid only.
//
// On a GB300 (graph replay): one sequence of 131071 tokens and 64 heads over 512 columns 41.0 us
// (134 MB, 19.8 us at the copy rate): 4 us until the first tile is there, 24 us at 5.6 TB/s, 3 us
// for 128 KB of partial per CTA (an SM stores 21 bytes per cycle), 7 us for the join with its
// launch.  48 sequences up to 6001 tokens, 128 heads: 61.4 us: 1.5 us per tile (two tiles, all that
// shared memory holds, take turns at copy, scores, softmax and values; the products alone are 0.95),
// 3.2 us per part, 7 us for the join.  61 sequences up to 4099, 32 heads over 8 of 128: 91.5 us
// (515 MB, 75.8): 70 us at the memory's limit, the rest start, the spread of the CTAs' ends and the
// join.  One sequence of 77 tokens, 16 heads: 7.1 us in a table of at most 256 tokens (one launch:
// dependent loads and two tiles in turn), 9.4 in one of 2048 pages (cut over three CTAs and joined).
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

// True in one thread of a converged warp.  The compiler knows that one thread runs what it
// guards, and keeps the operands of tcgen05.mma in uniform registers (issued under a plain
// lane test, a product of 64 x 64 x 16 took 74 cycles to issue, here 33, its time on the pipe).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
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

// a += b, both columns in one instruction.
__device__ __forceinline__ void add2(float2 &a, float2 b) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a.x), "+f"(a.y)
        : "f"(b.x), "f"(b.y));
}

// A box of a tensor on its way to L2.
__device__ __forceinline__ void tma_prefetch_5d(const CUtensorMap *map, int c0, int c1, int c2, int c3, int c4) {
    asm volatile("cp.async.bulk.prefetch.tensor.5d.L2.global.tile [%0, {%1, %2, %3, %4, %5}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
                 : "memory");
}

__device__ __forceinline__ void prefetch_l1(const void *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// Bounded wait.  Once any thread of the CTA has given up, waits that are not yet satisfied
// return at once; the roles keep their barrier pattern and store nothing, and the CTA reports it at its
// end.  (Inlined at every wait of every role: short, for the sake of the instruction cache.)
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int *abort_flag) {
    uint64_t t0 = 0;
    for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
        if ((it & 7u) != 0) continue;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > limit_ns) *abort_flag = 1;
        if (*abort_flag != 0) return false;
    }
    return true;
}

// ---- the line of tiles ---------------------------------------------------------------

// Length of sequence b, clamped to what its table row can hold; a row outside the table
// is an empty sequence.  Both are reported where the CTA looks for empty sequences (REPORT),
// which meets each of them once.
template <bool REPORT = false>
__device__ __forceinline__ int attn_len(const AttnArgs &a, int b) {
    const int row = a.rows ? a.rows[b] : b;
    const bool in = row >= 0 && row < a.num_rows;
    const int n = in ? a.lens[row] : 0;
    const int most = a.max_pages << a.page_shift;  // (the host checks that it fits)
    if (REPORT && (!in || n < 0 || n > most)) atomicCAS(a.err_word, 0, kDeviceErrIndex);
    return min(max(n, 0), most);
}
__device__ __forceinline__ int attn_tiles(int len) { return static_cast<int>((static_cast<uint32_t>(len) + kAttnTile - 1) / kAttnTile); }

// The work of all sequences and kv heads forms a line: `weight` units for the start and the
// end of a sequence part (its queries, the way out of tensor memory), one unit per tile.  CTA c
// of C takes units [T c / C, T (c + 1) / C); a range that ends inside a sequence's first
// `weight` units holds none of its tiles.
// (T and the products of C stay below 2^31: the host checks T, C is at most kAttnMaxCtas.)
__device__ __forceinline__ uint32_t line_start(uint32_t T, uint32_t c, uint32_t C) {
    const uint32_t q = T / C, r = T - q * C;
    return q * c + r * c / C;
}
__device__ __forceinline__ int line_owner(uint32_t T, uint32_t x, uint32_t C) {
    return static_cast<int>((static_cast<uint64_t>(x + 1) * C + T - 1) / T) - 1;
}

// Where a CTA's units lie, and a walk over them; every role walks alike.
struct AttnLine {
    uint32_t total;    // T
    uint32_t x0, x1;   // this CTA's units (uncut: its first sequence and head, the number of them)
    uint32_t base;     // units of all kv heads before sequence b0
    int32_t b0, len0;  // the sequence that holds x0, its length
    uint32_t ctas;     // CTAs that hold units
};
struct AttnWalk {
    uint32_t x, base;
    int b, len;
    __device__ __forceinline__ explicit AttnWalk(const AttnLine &ln) : x(ln.x0), base(ln.base), b(ln.b0), len(ln.len0) {}
};
struct AttnSegment {
    int b, kv, len, t0, n, tiles;  // n tiles from t0 of the sequence's `tiles`
    uint32_t x0, end;              // its first unit on the line, and the end of the sequence's (of one kv head)
};

__device__ __forceinline__ bool attn_next_segment(const AttnArgs &a, const AttnLine &ln, AttnWalk &w, AttnSegment &s) {
    while (w.x < ln.x1) {
        if (!a.split) {  // whole sequences, taken in turn
            const int item = static_cast<int>(w.x);
            w.x += a.ctas;
            s.b = item / a.kv_heads;
            s.kv = item - s.b * a.kv_heads;
            s.len = attn_len(a, s.b);
            s.n = s.tiles = attn_tiles(s.len);
            s.t0 = 0;
            s.x0 = item;
            s.end = item + 1;
            if (s.n > 0) return true;
            continue;
        }
        uint32_t units;
        for (;;) {
            units = w.len > 0 ? attn_tiles(w.len) + a.weight : 0;
            if (w.x < w.base + units * a.kv_heads) break;
            w.base += units * a.kv_heads;
            if (++w.b >= a.batch) return false;  // (lengths that changed under the call)
            w.len = attn_len(a, w.b);
        }
        const uint32_t rel = w.x - w.base;
        s.kv = a.kv_heads == 1 ? 0 : static_cast<int>(rel / units);
        const int p = static_cast<int>(rel - static_cast<uint32_t>(s.kv) * units);
        const int n = static_cast<int>(min(units - p, ln.x1 - w.x));
        s.b = w.b;
        s.len = w.len;
        s.tiles = static_cast<int>(units) - a.weight;
        s.t0 = max(0, p - a.weight);
        s.n = max(0, p + n - a.weight) - s.t0;
        s.x0 = w.x;
        s.end = w.x + (units - p);
        w.x += n;
        if (s.n > 0) return true;
    }
    return false;
}

// Instruction descriptor: bf16 operands, fp32 accumulator, N columns.
template <int N>
constexpr uint32_t kIdescBase = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17);

// A tile is loaded in groups of two 64-column boxes (one where a head has only one), each with
// its own place in a ring: the scores start on the first group that is there, and a group's
// place is free as soon as the product that reads it last is done.
//   latent:  the value groups 0 .. 3 (read by the scores and by one O^T tile each), and for 576
//            columns the rotary box in a small ring of its own (read by the scores only)
//   grouped: the key group (scores only), then the value group.  The number of places is even and at least four:
//            the issuer of the scores waits for key groups only, and a barrier's parity tells it
//            one use of a place from the next, not from the one after; with an odd number a
//            place would hold keys and values in turn, and a wait for keys could pass on the
//            phase before the values that are still to come.
template <int KB, int VB, bool SHARED, int N>
struct AttnCfg {
    static constexpr int kDV = VB * 64;
    static constexpr int kMV = kDV >= 128 ? 128 : 64;       // rows of one O^T instruction
    static constexpr int kOT = kDV / kMV;                   // O^T tiles
    static constexpr int kCols = kOT * N + 2 * N;           // O^T, then two S^T
    static constexpr uint32_t kTmemCols = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static_assert(kCols <= 512, "tensor memory");
    static constexpr int kGB = kMV / 64;                    // boxes per group
    static constexpr int kVG = VB / kGB;                    // value groups of a tile
    static constexpr int kKG = SHARED ? 0 : KB / kGB;       // key groups of its own
    static_assert(SHARED || (kKG == 1 && kVG == 1), "one key and one value group");
    static constexpr int kGroups = kVG + kKG;
    static constexpr int kExtra = SHARED ? KB - VB : 0;     // rotary boxes
    static_assert(kExtra <= 1, "one rotary box");
    static constexpr int kGroupBytes = kGB * kAttnTile * 128;
    static constexpr int kBoxBytes = kAttnTile * 128;
    static constexpr int kQBytes = KB * N * 128;
    static constexpr int kPBytes = kAttnTile * 128;
};
// A place in a ring, walked by producer and consumers alike.
struct RingPos {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

template <int KB, int VB, bool SHARED, int N>
__global__ void __launch_bounds__(kAttnThreads, attn_ctas_per_sm(KB, SHARED, N))
    hsp_attn_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ AttnArgs a) {
    using C = AttnCfg<KB, VB, SHARED, N>;
    constexpr int kS = N / 8;          // 8-column steps of S^T
    constexpr int kDV = C::kDV;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t ring = smem_u32(smem);
    const uint32_t extra = ring + a.slots * C::kGroupBytes;             // the rotary boxes' two places
    uint8_t *const q_smem = smem + a.slots * C::kGroupBytes + C::kExtra * 2 * C::kBoxBytes;
    uint8_t *const p_smem = q_smem + C::kQBytes;
    float *const red = reinterpret_cast<float *>(p_smem + C::kPBytes);  // [4 warps][N]
    float *const fac = red + 4 * N;                                     // [N]
    uint64_t *const full = reinterpret_cast<uint64_t *>(fac + N);       // [slots]
    uint64_t *const empty = full + a.slots;
    uint64_t *const x_full = empty + a.slots;                           // [2] the rotary boxes
    uint64_t *const x_empty = x_full + 2;                               // [2]
    uint64_t *const s_full = x_empty + 2;                               // [2]
    uint64_t *const s_free = s_full + 2;                                // [2]
    uint64_t *const q_full = s_free + 2;
    uint64_t *const q_free = q_full + 1;
    uint64_t *const p_full = q_free + 1;
    uint64_t *const pv_done = p_full + 1;
    uint64_t *const drained = pv_done + 1;
    int *const ints = reinterpret_cast<int *>(drained + 1);
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(ints);
    volatile int *const abort_flag = ints + 1;
    int *const issued = ints + 2;                                       // groups, rotary boxes, queries whose copies were issued
    int *const place = ints + 5;                                        // the first sequence of this CTA, units before it, its length
    int *const warp_sum = ints + 8;                                     // [7]

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
        }
        mbar_init(smem_u32(&s_full[0]), 1);
        mbar_init(smem_u32(&s_full[1]), 1);
        mbar_init(smem_u32(&s_free[0]), 128);
        mbar_init(smem_u32(&s_free[1]), 128);
        mbar_init(smem_u32(q_full), 1);
        mbar_init(smem_u32(q_free), 1);
        mbar_init(smem_u32(p_full), 128);
        mbar_init(smem_u32(pv_done), 1);
        mbar_init(smem_u32(drained), 2);
        *abort_flag = 0;
        issued[0] = issued[1] = issued[2] = 0;
        mbar_fence_init();
        tma_prefetch_map(&tmap_q);
        tma_prefetch_map(&tmap_k);
        if (!SHARED || C::kExtra) tma_prefetch_map(&tmap_v);
    }
    if (warp == 5) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    griddep_wait();  // everything read below may come from the previous kernel

    // ---- the line: its length, and where this CTA's first unit lies ----
    // Up to 128 sequences: every warp for itself (no thread waits for another warp); more: the CTA.
    AttnLine ln;
    ln.total = ln.x1 = static_cast<uint32_t>(a.batch) * a.kv_heads;  // uncut: the items
    ln.x0 = cta;
    ln.ctas = a.ctas;
    ln.base = 0;
    ln.b0 = ln.len0 = 0;
    if (a.split) {
        const bool by_warp = a.batch <= 128;
        const int tn = by_warp ? 32 : kAttnThreads, tno = by_warp ? lane : tid;
        const int per = (a.batch + tn - 1) / tn;
        const int bfirst = min(a.batch, tno * per), blast = min(a.batch, bfirst + per);
        uint32_t mine = 0;
        int len = 0;
        for (int b = bfirst; b < blast; ++b) {
            len = attn_len(a, b);
            mine += len > 0 ? attn_tiles(len) + a.weight : 0;
        }
        uint32_t incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        uint32_t before = incl - mine, all = __shfl_sync(0xffffffffu, incl, 31);
        if (!by_warp) {
            if (lane == 31) warp_sum[warp] = static_cast<int>(incl);
            __syncthreads();
            all = 0;
#pragma unroll
            for (int w = 0; w < kAttnThreads / 32; ++w) {
                if (w < warp) before += warp_sum[w];
                all += warp_sum[w];
            }
        }
        ln.total = all * a.kv_heads;
        ln.ctas = min(ln.total, static_cast<uint32_t>(a.ctas));
        ln.x0 = ln.x1 = 0;
        bool here = false;  // this thread's sequences hold the CTA's first unit
        uint32_t first = before * a.kv_heads;
        int b = bfirst;
        if (cta < ln.ctas) {
            ln.x0 = line_start(ln.total, cta, ln.ctas);
            ln.x1 = line_start(ln.total, cta + 1, ln.ctas);
            here = ln.x0 >= first && ln.x0 < first + mine * a.kv_heads;
        }
        if (here) {
            if (per > 1) {  // walk to the sequence
                for (;; ++b) {
                    len = attn_len(a, b);
                    const uint32_t units = len > 0 ? (attn_tiles(len) + a.weight) * a.kv_heads : 0;
                    if (ln.x0 < first + units || b + 1 >= blast) break;
                    first += units;
                }
            }
            // its first page id, on its way before the copy producer asks for it
            const uint32_t units = attn_tiles(len) + a.weight;
            const uint32_t t = (ln.x0 - first) % units;
            const int64_t page = (static_cast<int64_t>(max(0, static_cast<int>(t) - a.weight)) * kAttnTile) >> a.page_shift;
            prefetch_l1(a.table + (a.rows ? a.rows[b] : b) * a.table_stride + page);
        }
        if (by_warp) {
            const uint32_t who = __ballot_sync(0xffffffffu, here);
            const int from = who ? __ffs(who) - 1 : 0;
            ln.b0 = __shfl_sync(0xffffffffu, b, from);
            ln.base = __shfl_sync(0xffffffffu, first, from);
            ln.len0 = __shfl_sync(0xffffffffu, len, from);
        } else {
            if (here) {
                place[0] = b;
                place[1] = static_cast<int>(first);
                place[2] = len;
            }
            __syncthreads();
            ln.b0 = place[0];
            ln.base = static_cast<uint32_t>(place[1]);
            ln.len0 = place[2];
        }
    }
    const uint32_t tmem = *tmem_slot;
    const uint32_t tmem_s = tmem + C::kOT * N;

    if (warp == 4) {
        // ---------------- copy producer: one thread reads the table a tile ahead and issues ----------------
        if (elect_one()) {
            AttnWalk walk(ln);
            int i = 0;
            AttnSegment sg;
            RingPos rp, xp;
            int ng = 0;
            uint32_t seg = 0;
            const int pbox = min(kAttnTile, 1 << a.page_shift);     // tokens per box
            const int boxes = kAttnTile / pbox;                     // pages that meet a tile (1, 2 or 4)
            const uint32_t line_bytes = static_cast<uint32_t>(pbox) * 128;
            bool alive = true;
            while (alive && attn_next_segment(a, ln, walk, sg)) {
                const int row = a.rows ? a.rows[sg.b] : sg.b;
                const int32_t *tbl = a.table + row * a.table_stride;
                const int pages = static_cast<int>((static_cast<int64_t>(sg.len) + (1 << a.page_shift) - 1) >> a.page_shift);
                auto ids_of = [&](int tile, int (&id)[4]) {
                    const int p0 = static_cast<int>((static_cast<int64_t>(tile) * kAttnTile) >> a.page_shift);
#pragma unroll
                    for (int e = 0; e < 4; ++e) id[e] = (e < boxes && p0 + e < pages) ? tbl[p0 + e] : 0;
                };
                // the sequence's queries for this head tile, once the scores of the last sequence are done
                // with theirs (heads past the group are another group's, or zero past the last: columns
                // that nothing reads); behind the first tile, which does not have to wait for that
                auto queries = [&]() {
                    alive = attn_wait(smem_u32(q_free), (seg & 1u) ^ 1u, a.wait_limit_ns, abort_flag);
                    if (!alive) return;
                    mbar_arrive_expect_tx(smem_u32(q_full), C::kQBytes);
                    tma_load_5d(smem_u32(q_smem), &tmap_q, 0, sg.kv * a.group + ht * N, 0, sg.b, 0, smem_u32(q_full));
                    issued[2] = static_cast<int>(++seg);
                };
                int next[4];
                ids_of(sg.t0, next);
                if (seg == 0) queries();
                const uint32_t seg0 = seg;
                for (int k = 0; k < sg.n && alive; ++k, ++i) {
                    int id[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        id[e] = next[e];
                        if (id[e] < 0 || id[e] >= a.num_pages) {
                            atomicCAS(a.err_word, 0, kDeviceErrIndex);
                            id[e] = 0;  // stays inside the pool; the call is reported
                        }
                    }
                    if (k + 1 < sg.n) ids_of(sg.t0 + k + 1, next);
                    const int64_t tok = static_cast<int64_t>(sg.t0 + k) * kAttnTile;
                    const int np = min(boxes, pages - static_cast<int>(tok >> a.page_shift));
                    const int off = static_cast<int>(tok & ((1 << a.page_shift) - 1));
                    // one group: `n` boxes from box `box` of a map; small pages: one copy per page and box
                    auto load = [&](const CUtensorMap *map, int box, int n, uint32_t dst, uint32_t fb) {
                        mbar_arrive_expect_tx(fb, static_cast<uint32_t>(np * n) * line_bytes);
                        if (boxes == 1) {
                            tma_load_5d(dst, map, 0, off, box, sg.kv, id[0], fb);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (e < np)
                                    for (int kb = 0; kb < n; ++kb)
                                        tma_load_5d(dst + kb * C::kBoxBytes + e * line_bytes, map, 0, 0, box + kb, sg.kv, id[e], fb);
                        }
                    };
                    // Two tiles are all that shared memory holds beside 64 latent queries, too few to hide DRAM
                    // behind the products: with several head tiles one of them sends the next tile to L2
                    // (48 ragged sequences, 128 heads: 66.4 -> 62.8 us; two tiles ahead 65.5; one head tile,
                    // 16 to 64 heads: mostly 1 us slower).
                    if (SHARED && N == 64 && gridDim.x > 1 && boxes == 1 && k + 1 < sg.n && (k + 1) % static_cast<int>(gridDim.x) == ht && next[0] >= 0 &&
                        next[0] < a.num_pages) {
                        const int to = static_cast<int>((tok + kAttnTile) & ((1 << a.page_shift) - 1));
#pragma unroll
                        for (int g = 0; g < C::kGroups; ++g)
                            tma_prefetch_5d(SHARED || g < C::kKG ? &tmap_k : &tmap_v, 0, to, SHARED ? g * C::kGB : 0, sg.kv, next[0]);
                        if (C::kExtra) tma_prefetch_5d(&tmap_v, 0, to, VB, sg.kv, next[0]);
                    }
                    const bool skip = i == a.skip_tile;
#pragma unroll 1
                    for (int g = 0; g < C::kGroups; ++g) {
                        // (a fresh barrier's phase before the first counts as complete)
                        alive = attn_wait(smem_u32(&empty[rp.slot]), rp.phase ^ 1u, a.wait_limit_ns, abort_flag);
                        if (!alive) break;
                        ++ng;
                        if (!skip) {
                            load(SHARED || g < C::kKG ? &tmap_k : &tmap_v, SHARED ? g * C::kGB : 0, C::kGB,
                                 ring + rp.slot * C::kGroupBytes, smem_u32(&full[rp.slot]));
                            issued[0] = ng;
                        }
                        rp.next(a.slots);
                    }
                    if (C::kExtra && alive) {
                        alive = attn_wait(smem_u32(&x_empty[xp.slot]), xp.phase ^ 1u, a.wait_limit_ns, abort_flag);
                        if (!alive) break;
                        if (!skip) {
                            load(&tmap_v, VB, 1, extra + xp.slot * C::kBoxBytes, smem_u32(&x_full[xp.slot]));
                            issued[1] = i + 1;
                        }
                        xp.next(2);
                    }
                    if (k == 0 && alive && i > 0 && seg == seg0) queries();
                }
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        // ---------------- issuer of the scores ----------------
        if (elect_one()) {
            constexpr uint32_t kDesc = kIdescBase<N> | (static_cast<uint32_t>(kAttnTile >> 4) << 24);
            AttnWalk walk(ln);
            uint32_t seg = 0;
            AttnSegment sg;
            bool alive = true;
            const uint64_t qd = umma_desc_sw128(smem_u32(q_smem));
            RingPos rp, xp, sp;
            auto ready = [&](uint64_t *bar, uint32_t phase) {
                return attn_wait(smem_u32(bar), phase, a.wait_limit_ns, abort_flag);
            };
            while (alive && attn_next_segment(a, ln, walk, sg)) {
                if (!ready(q_full, seg & 1u)) break;
                ++seg;
                for (int k = 0; k < sg.n; ++k) {
                    // the scores of the tile before last have been read out of this accumulator
                    if (!(alive = ready(&s_free[sp.slot], sp.phase ^ 1u))) break;
                    const uint32_t d = tmem_s + sp.slot * N;
                    constexpr int kGroupsK = SHARED ? C::kVG : C::kKG;
#pragma unroll
                    for (int g = 0; g < kGroupsK; ++g) {
                        if (alive) alive = ready(&full[rp.slot], rp.phase);
                        if (!alive) break;
                        tc_fence_after_sync();
                        const uint64_t kd = umma_desc_sw128(ring + rp.slot * C::kGroupBytes);
#pragma unroll
                        for (int e = 0; e < C::kGB * 4; ++e)  // (descriptors count 16 bytes)
                            umma_f16(d, kd + (e >> 2) * (C::kBoxBytes / 16) + (e & 3) * 2,
                                     qd + (g * C::kGB + (e >> 2)) * (N * 8) + (e & 3) * 2, kDesc, (g | e) != 0 ? 1u : 0u);
                        if (!SHARED) umma_commit(smem_u32(&empty[rp.slot]));
                        rp.next(a.slots);
                    }
                    if (!alive) break;
                    if (!SHARED) rp.next(a.slots);  // the value group
                    if (C::kExtra) {
                        if (!(alive = ready(&x_full[xp.slot], xp.phase))) break;
                        tc_fence_after_sync();
                        const uint64_t kd = umma_desc_sw128(extra + xp.slot * C::kBoxBytes);
#pragma unroll
                        for (int e = 0; e < 4; ++e) umma_f16(d, kd + e * 2, qd + VB * (N * 8) + e * 2, kDesc, 1u);
                        umma_commit(smem_u32(&x_empty[xp.slot]));
                        xp.next(2);
                    }
                    umma_commit(smem_u32(&s_full[sp.slot]));
                    sp.next(2);
                }
                umma_commit(smem_u32(q_free));
            }
            umma_commit(smem_u32(drained));
        }
        __syncwarp();
    } else if (warp == 6) {
        // ---------------- issuer of the products with the values ----------------
        if (elect_one()) {
            constexpr uint32_t kDesc = kIdescBase<N> | (1u << 15) | (1u << 16) | (static_cast<uint32_t>(C::kMV >> 4) << 24);
            AttnWalk walk(ln);
            int i = 0;
            AttnSegment sg;
            bool alive = true;
            const uint64_t pd = umma_desc_mn_sw128(smem_u32(p_smem), C::kBoxBytes);
            RingPos rp;
            while (alive && attn_next_segment(a, ln, walk, sg)) {
                for (int k = 0; k < sg.n; ++k, ++i) {
                    const int valid = min(kAttnTile, sg.len - (sg.t0 + k) * kAttnTile);  // tokens of this tile
                    alive = attn_wait(smem_u32(p_full), static_cast<uint32_t>(i) & 1u, a.wait_limit_ns, abort_flag);
                    if (!alive) break;
                    tc_fence_after_sync();
                    if (!SHARED) {
                        rp.next(a.slots);  // the key group
                        alive = attn_wait(smem_u32(&full[rp.slot]), rp.phase, a.wait_limit_ns, abort_flag);
                        if (!alive) break;
                        tc_fence_after_sync();
                    }
#pragma unroll
                    for (int jt = 0; jt < C::kOT; ++jt) {
                        const uint64_t vd = umma_desc_mn_sw128(ring + rp.slot * C::kGroupBytes, C::kBoxBytes);
#pragma unroll
                        for (int e = 0; e < kAttnTile / 16; ++e)
                            if (e * 16 < valid) umma_f16(tmem + jt * N, vd + e * 128, pd + e * 128, kDesc, (k | e) != 0 ? 1u : 0u);
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
    } else {
        // ---------------- softmax warps ----------------
        AttnWalk walk(ln);
        int i = 0;
        AttnSegment sg;
        const int head0 = ht * N;                              // of the group
        const int nheads = min(N, a.group - head0);            // real heads of this tile
        const int all_heads = a.kv_heads * a.group;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
        const int r0 = warp * 16 + (lane >> 2);                // this thread's token rows: r0 and r0 + 8
        const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
        constexpr float kFloor = -3.0e38f;
        if (a.split && ht == 0 && tid == 96) {
            AttnEntry e;
            e.batch = -1;
            e.kv_head = e.last = e.slot = 0;
            a.entries[cta] = e;
        }
        while (attn_next_segment(a, ln, walk, sg)) {
            const bool begins = sg.t0 == 0, ends = sg.t0 + sg.n == sg.tiles;
            float m[kS * 2];     // reference point
            float2 l[kS], u[kS];  // sums of the rounded and the unrounded weights
#pragma unroll
            for (int e = 0; e < kS * 2; ++e) m[e] = kFloor;
#pragma unroll
            for (int j = 0; j < kS; ++j) l[j] = u[j] = make_float2(0.f, 0.f);
            for (int k = 0; k < sg.n; ++k, ++i) {
                const int64_t tok0 = static_cast<int64_t>(sg.t0 + k) * kAttnTile;
                const int valid = static_cast<int>(min(static_cast<int64_t>(kAttnTile), sg.len - tok0));
                attn_wait(smem_u32(&s_full[i & 1]), static_cast<uint32_t>(i >> 1) & 1u, a.wait_limit_ns, abort_flag);
                tc_fence_after_sync();
                float s[kS * 4];
                tmem_ld_frag<kS>(tmem_s + (i & 1) * N + lane_base, s);
                tmem_wait_ld();
                tc_fence_before_sync();
                mbar_arrive(smem_u32(&s_free[i & 1]));
#pragma unroll
                for (int e = 0; e < kS * 4; ++e) s[e] *= a.scale_log2;
                if (valid < kAttnTile) {
#pragma unroll
                    for (int j = 0; j < kS; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (r0 >= valid) s[4 * j + e] = -INFINITY;
                            if (r0 + 8 >= valid) s[4 * j + 2 + e] = -INFINITY;
                        }
                }
                float most = -INFINITY;
#pragma unroll
                for (int j = 0; j < kS; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) most = fmaxf(most, fmaxf(s[4 * j + e], s[4 * j + 2 + e]) - m[2 * j + e]);
                const bool over = k == 0 || most > 8.f;
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
                            const float2 o = *reinterpret_cast<const float2 *>(red + w * N + c);
                            t.x = fmaxf(t.x, o.x);
                            t.y = fmaxf(t.y, o.y);
                        }
                        const float n0 = fmaxf(m[2 * j], t.x), n1 = fmaxf(m[2 * j + 1], t.y);
                        const float f0 = fast_exp2(m[2 * j] - n0), f1 = fast_exp2(m[2 * j + 1] - n1);
                        m[2 * j] = n0;
                        m[2 * j + 1] = n1;
                        l[j] = make_float2(l[j].x * f0, l[j].y * f1);
                        u[j] = make_float2(u[j].x * f0, u[j].y * f1);
                        if (warp == 0 && lane < 4) *reinterpret_cast<float2 *>(fac + c) = make_float2(f0, f1);
                    }
                    if (k > 0) {
                        attn_wait(smem_u32(pv_done), static_cast<uint32_t>(i - 1) & 1u, a.wait_limit_ns, abort_flag);
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
                if (valid < kAttnTile) {
                    // the last tile: what lies behind the sequence must not reach the product (0 x NaN).  Its last
                    // step of 16 tokens is filled up with zeros; the steps behind that are not taken.
                    const int first = i * C::kGroups + C::kKG;  // its first value group in the ring
                    if (!SHARED)                                // (a latent tile's scores have waited for it)
                        attn_wait(smem_u32(&full[first % a.slots]), static_cast<uint32_t>(first / a.slots) & 1u, a.wait_limit_ns, abort_flag);
                    if (tid < (-valid & 15) * 8) {
                        int at = first % a.slots;
#pragma unroll
                        for (int g = 0; g < C::kVG; ++g) {
#pragma unroll
                            for (int e = 0; e < C::kGB; ++e)
                                *reinterpret_cast<uint4 *>(smem + at * C::kGroupBytes + e * C::kBoxBytes + valid * 128 + tid * 16) =
                                    make_uint4(0, 0, 0, 0);
                            at = at + 1 == a.slots ? 0 : at + 1;
                        }
                    }
                }
                // the probabilities of tile i - 1 have been read before these replace them
                if (i > 0)
                    attn_wait(smem_u32(pv_done), static_cast<uint32_t>(i - 1) & 1u, a.wait_limit_ns, abort_flag);
                uint32_t pb[kS * 2];  // the rounded weights, two columns each
#pragma unroll
                for (int j = 0; j < kS; ++j) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[4 * j + e] = fast_exp2(s[4 * j + e] - m[2 * j + (e & 1)]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(s[4 * j + 2 * e], s[4 * j + 2 * e + 1]);
                        pb[2 * j + e] = *reinterpret_cast<const uint32_t *>(&b);
                        *reinterpret_cast<uint32_t *>(p_smem + (r0 + 8 * e) * 128 + ((j ^ (r0 & 7)) << 4) + (lane & 3) * 4) = pb[2 * j + e];
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                mbar_arrive(smem_u32(p_full));
                // the sums, beside the product (48 sequences with 128 heads: 61.5 us before the arrival, 60.2 behind it)
#pragma unroll
                for (int j = 0; j < kS; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        add2(u[j], make_float2(s[4 * j + 2 * e], s[4 * j + 2 * e + 1]));
                        add2(l[j], make_float2(__uint_as_float(pb[2 * j + e] << 16), __uint_as_float(pb[2 * j + e] & 0xffff0000u)));
                    }
            }
            // ---- the part is done: l (and u) over the tokens, then O^T out of tensor memory ----
            auto over_tokens = [&](float2 (&v)[kS]) {  // a warp's sums to `red`
#pragma unroll
                for (int j = 0; j < kS; ++j)
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        v[j].x += __shfl_xor_sync(0xffffffffu, v[j].x, d);
                        v[j].y += __shfl_xor_sync(0xffffffffu, v[j].y, d);
                    }
                softmax_sync();  // the last tile's maxima and factors (l), the sums l (u) have been read
                if (lane < 4) {
#pragma unroll
                    for (int j = 0; j < kS; ++j) *reinterpret_cast<float2 *>(red + warp * N + 8 * j + 2 * lane) = v[j];
                }
            };
            over_tokens(l);
            if (warp == 0 && lane < 4) {
#pragma unroll
                for (int j = 0; j < kS; ++j) *reinterpret_cast<float2 *>(fac + 8 * j + 2 * lane) = make_float2(m[2 * j], m[2 * j + 1]);
            }
            softmax_sync();
            const bool whole = begins && ends;
            const int slot = sg.x0 == ln.x0 ? 0 : 1;
            float *part = a.parts + (static_cast<int64_t>(ht) * a.ctas + cta) * 2 * attn_part(kDV, N) + slot * attn_part(kDV, N);
            float top = 0.f;
            if (tid < N) {  // a column per thread
                const float t = red[tid] + red[N + tid] + red[2 * N + tid] + red[3 * N + tid];
                top = fac[tid];
                if (whole) {
                    fac[tid] = t == 0.f ? 0.f : 1.f / t;
                } else {
                    part[N * kDV + tid] = top;
                    part[N * kDV + N + tid] = t;
                }
            }
            if (a.lse) {
                over_tokens(u);
                softmax_sync();
                if (tid < N) {
                    const float t = red[tid] + red[N + tid] + red[2 * N + tid] + red[3 * N + tid];
                    if (!whole)
                        part[N * kDV + 2 * N + tid] = t;
                    else if (tid < nheads && *abort_flag == 0)
                        a.lse[static_cast<int64_t>(sg.b) * all_heads + sg.kv * a.group + head0 + tid] =
                            t == 0.f ? -INFINITY : (top + log2f(t)) * 0.6931471805599453f;
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
            attn_wait(smem_u32(pv_done), static_cast<uint32_t>(i - 1) & 1u, a.wait_limit_ns, abort_flag);
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
                        __nv_bfloat16 *to = out + obase + static_cast<int64_t>(h0) * kDV + dv;
                        if (h0 + 16 <= nheads) {  // (16 tests take longer than the stores)
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(fac + h0 + e);
                                to[e * kDV] = __float2bfloat16_rn(o[e] * f.x);
                                to[(e + 1) * kDV] = __float2bfloat16_rn(o[e + 1] * f.y);
                                to[(e + 2) * kDV] = __float2bfloat16_rn(o[e + 2] * f.z);
                                to[(e + 3) * kDV] = __float2bfloat16_rn(o[e + 3] * f.w);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 15; ++e)
                                if (h0 + e < nheads) to[e * kDV] = __float2bfloat16_rn(o[e] * fac[h0 + e]);
                        }
                    } else {
                        float *to = part + h0 * kDV + dv;
                        if (h0 + 16 <= nheads) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) to[e * kDV] = o[e];
                        } else {
#pragma unroll
                            for (int e = 0; e < 15; ++e)
                                if (h0 + e < nheads) to[e * kDV] = o[e];
                        }
                    }
                }
            }
            tc_fence_before_sync();
            softmax_sync();  // red and fac are free again
        }
        // sequences without a token: zeros, and no weight at all
        for (int e = cta; e < a.batch; e += a.ctas) {
            if (attn_len<true>(a, e) != 0) continue;
            for (int kv = 0; kv < a.kv_heads; ++kv) {
                const int64_t h = static_cast<int64_t>(e) * all_heads + kv * a.group + head0;
                uint4 *to = reinterpret_cast<uint4 *>(out + h * kDV);  // (its heads lie one after another)
                for (int c = tid; c < nheads * kDV / 8; c += 128) to[c] = make_uint4(0, 0, 0, 0);
                if (a.lse)
                    for (int c = tid; c < nheads; c += 128) a.lse[h + c] = -INFINITY;
            }
        }
    }
    tc_fence_before_sync();
    // (Triggered at the start, the join's CTAs crowded on the SMs that were free first: 43 -> 47 us
    // for one sequence of 131071 tokens and 64 heads.)
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
        for (int j = max(0, nx - 2); j < nx; ++j)
            if (j != a.skip_tile) land(&x_full[j & 1], j >> 1);
        if (issued[2] > 0) land(q_full, issued[2] - 1);
    }
    if (warp == 5) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    __syncthreads();
}

// ---- join ------------------------------------------------------------------------------
//
// Sequences cut over several CTAs: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i, and with u_i
// for l_i the sum of lse, the parts in a fixed order.  Few parts, or heads enough for all warps: a warp takes a head, part
// after part.  Else (one long sequence): a CTA takes 64 or 128 columns of a head, its half warps
// or warps take the parts in turn and their sums are added in a fixed order.  Which of the two depends on
// the lengths only.

constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32, kJoinPerSm = 4;
constexpr int kJoinWarpParts = 32;  // most parts of a head that one warp joins

template <int W>
struct JoinWidth {
    static constexpr int value = W;
};

template <int DV, int N>
__global__ void __launch_bounds__(kJoinThreads, kJoinPerSm) hsp_attn_join_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int kParts = DV / 64;             // units of 64 columns of a head with many parts
    constexpr int kPart = attn_part(DV, N);     // floats of one partial
    __shared__ float4 acc_s[kJoinWarps][32];
    __shared__ float weight[kAttnMaxCtas], red_s[3 * kJoinWarps];
    __shared__ uint16_t few[kAttnMaxCtas], many[kAttnMaxCtas];  // the CTAs that began them
    __shared__ AttnEntry entries[kAttnMaxCtas];
    __shared__ uint32_t bits[2][kAttnMaxCtas / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_wait();
    // the sequences to join, in CTA order in every CTA of this kernel: its units are shared out by their place
    int parts_of[kAttnMaxCtas / kJoinThreads];
#pragma unroll
    for (int k = 0; k < kAttnMaxCtas / kJoinThreads; ++k) {
        const int c = tid + k * kJoinThreads;
        int begun = -1, last = 0;
        if (c < a.ctas) {
            const AttnEntry e = a.entries[c];
            entries[c] = e;
            begun = e.batch;
            last = e.last;
        }
        parts_of[k] = begun >= 0 ? last - c + 1 : 0;
        const uint32_t mm = __ballot_sync(0xffffffffu, begun >= 0);
        if (lane == 0) bits[1][c >> 5] = mm;
    }
    __syncthreads();
    // A warp joins a head in about half as many steps as it has parts, a CTA 64 columns of one in
    // about five; with R such units for every CTA, up to 5 R parts are a warp's.
    int items = 0;
    for (int w = 0; w * 32 < a.ctas; ++w) items += __popc(bits[1][w]);
    const int units = static_cast<int>(min(static_cast<int64_t>(1) << 20, static_cast<int64_t>(items) * a.group * kParts / gridDim.x));
    const int by_warp = min(kJoinWarpParts, 5 * max(1, units));
#pragma unroll
    for (int k = 0; k < kAttnMaxCtas / kJoinThreads; ++k) {
        const uint32_t mf = __ballot_sync(0xffffffffu, parts_of[k] > 0 && parts_of[k] <= by_warp);
        if (lane == 0) bits[0][(tid + k * kJoinThreads) >> 5] = mf;
    }
    __syncthreads();
    int nfew = 0, nmany = 0;
    for (int w = 0; w * 32 < a.ctas; ++w) {
        const uint32_t f = bits[0][w], m = bits[1][w] & ~f;
        if (warp == w % kJoinWarps) {
            const uint32_t low = (1u << lane) - 1u;
            if ((f >> lane) & 1u) few[nfew + __popc(f & low)] = static_cast<uint16_t>(w * 32 + lane);
            if ((m >> lane) & 1u) many[nmany + __popc(m & low)] = static_cast<uint16_t>(w * 32 + lane);
        }
        nfew += __popc(f);
        nmany += __popc(m);
    }
    __syncthreads();
    auto store = [&](const AttnEntry &e, int h, int col, float4 acc, float inv) {
        const int64_t oh = (static_cast<int64_t>(e.batch) * a.kv_heads + e.kv_head) * a.group + h;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        uint2 o;
        o.x = *reinterpret_cast<const uint32_t *>(&lo);
        o.y = *reinterpret_cast<const uint32_t *>(&hi);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + oh * DV + col) = o;
    };
    auto store_lse = [&](const AttnEntry &e, int h, float M, float U) {
        a.lse[(static_cast<int64_t>(e.batch) * a.kv_heads + e.kv_head) * a.group + h] =
            U == 0.f ? -INFINITY : (M + log2f(U)) * 0.6931471805599453f;
    };
    // part p of head h of CTA c's sequence: its own slot, then slot 0 of the CTAs behind it
    auto part = [&](int c, int slot, int h, int p) {
        const int at = p == 0 ? c * 2 + slot : (c + p) * 2;
        return a.parts + (static_cast<int64_t>(h / N) * a.ctas * 2 + at) * kPart;
    };
    // few parts: a warp takes a head, all of its columns
    constexpr int kVec = DV >= 128 ? DV / 128 : 1;  // float4 per lane and part
    for (int u = blockIdx.x * kJoinWarps + warp; u < nfew * a.group; u += gridDim.x * kJoinWarps) {
        const int c = few[u / a.group], h = u % a.group, col = h % N;
        const AttnEntry e = entries[c];
        const int parts = min(e.last, a.ctas - 1) - c + 1;
        float m = -3.0e38f, l = 0.f, un = 0.f;
        if (lane < parts) {
            const float *pp = part(c, e.slot, h, lane);
            m = pp[N * DV + col];
            l = pp[N * DV + N + col];
            if (a.lse) un = pp[N * DV + 2 * N + col];
        }
        float4 v[2][kVec];
        auto load = [&](int p, float4 (&to)[kVec]) {
            if (p < parts && lane * 4 < DV) {
                const float *pp = part(c, e.slot, h, p) + col * DV + lane * 4;
#pragma unroll
                for (int k = 0; k < kVec; ++k) to[k] = *reinterpret_cast<const float4 *>(pp + k * 128);
            }
        };
        load(0, v[0]);
        load(1, v[1]);
        float M = m;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        const float w = lane < parts ? fast_exp2(m - M) : 0.f;
        float L = w * l, U = w * un;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            L += __shfl_xor_sync(0xffffffffu, L, d);
            U += __shfl_xor_sync(0xffffffffu, U, d);
        }
        float4 acc[kVec];
#pragma unroll
        for (int k = 0; k < kVec; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = 0; p0 < parts; p0 += 2) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float wk = __shfl_sync(0xffffffffu, w, (p0 + q) & 31);
                if (p0 + q < parts) {
#pragma unroll
                    for (int k = 0; k < kVec; ++k) {
                        acc[k].x += wk * v[q][k].x;
                        acc[k].y += wk * v[q][k].y;
                        acc[k].z += wk * v[q][k].z;
                        acc[k].w += wk * v[q][k].w;
                    }
                }
                load(p0 + q + 2, v[q]);
            }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        if (lane * 4 < DV) {
#pragma unroll
            for (int k = 0; k < kVec; ++k) store(e, h, k * 128 + lane * 4, acc[k], inv);
        }
        if (a.lse && lane == 0) store_lse(e, h, M, U);
    }
    // one head, `width` columns from dp * width on
    auto join_cta = [&](int c, int h, int dp, auto width) {
        const AttnEntry e = entries[c];
        const int col = h % N;
        const int parts = min(e.last, a.ctas - 1) - c + 1;
        // the values are on their way while the weights are made
        constexpr int kAhead = 10, kLanes = decltype(width)::value / 4, kRows = kJoinThreads / kLanes;
        const int at = dp * (kLanes * 4) + tid % kLanes * 4, p_first = tid / kLanes;
        float4 v[kAhead];
        auto load = [&](int p0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (p0 + kRows * k < parts) v[k] = *reinterpret_cast<const float4 *>(part(c, e.slot, h, p0 + kRows * k) + col * DV + at);
        };
        load(p_first);
        float m[kAttnMaxCtas / kJoinThreads], lw[kAttnMaxCtas / kJoinThreads], uw[kAttnMaxCtas / kJoinThreads];
        const bool sums_u = a.lse && dp == 0;  // (one CTA of a head stores its lse)
        float M = -3.0e38f;
#pragma unroll
        for (int k = 0; k < kAttnMaxCtas / kJoinThreads; ++k) {
            const int p = tid + k * kJoinThreads;
            m[k] = -3.0e38f;
            lw[k] = uw[k] = 0.f;
            if (p < parts) {
                const float *pp = part(c, e.slot, h, p) + N * DV + col;
                m[k] = pp[0];
                lw[k] = pp[N];
                if (sums_u) uw[k] = pp[2 * N];
            }
            M = fmaxf(M, m[k]);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        if (lane == 0) red_s[warp] = M;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) M = fmaxf(M, red_s[k]);
        float L = 0.f, U = 0.f;
#pragma unroll
        for (int k = 0; k < kAttnMaxCtas / kJoinThreads; ++k) {
            const int p = tid + k * kJoinThreads;
            const float w = fast_exp2(m[k] - M);
            if (p < parts) weight[p] = w;
            L += lw[k] * w;
            U += uw[k] * w;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            L += __shfl_xor_sync(0xffffffffu, L, d);
            U += __shfl_xor_sync(0xffffffffu, U, d);
        }
        if (lane == 0) {
            red_s[kJoinWarps + warp] = L;
            red_s[2 * kJoinWarps + warp] = U;
        }
        __syncthreads();
        L = U = 0.f;
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) {
            L += red_s[kJoinWarps + k];
            U += red_s[2 * kJoinWarps + k];
        }
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = p_first; p0 < parts; p0 += kRows * kAhead) {
            if (p0 != p_first) load(p0);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (p0 + kRows * k < parts) {
                    const float w = weight[p0 + kRows * k];
                    acc.x += w * v[k].x;
                    acc.y += w * v[k].y;
                    acc.z += w * v[k].z;
                    acc.w += w * v[k].w;
                }
        }
        if (kLanes == 16) {
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
            acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
            acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
        }
        if (lane < kLanes) acc_s[warp][lane] = acc;
        __syncthreads();
        if (tid < kLanes) {
#pragma unroll
            for (int k = 1; k < kJoinWarps; ++k) {
                const float4 o = acc_s[k][lane];
                acc.x += o.x;
                acc.y += o.y;
                acc.z += o.z;
                acc.w += o.w;
            }
            store(e, h, at, acc, L == 0.f ? 0.f : 1.f / L);
            if (sums_u && lane == 0) store_lse(e, h, M, U);
        }
        __syncthreads();
    };
    // 64 columns while that leaves CTAs without any work, else 128
    const bool wide = DV >= 128 && static_cast<int64_t>(nmany) * a.group * (DV / 128) >= gridDim.x;
    const int pieces = wide ? DV / 128 : DV / 64, per_item = a.group * pieces;
    for (int u = blockIdx.x; u < nmany * per_item; u += gridDim.x) {
        const int c = many[u / per_item], rem = u % per_item, h = rem / pieces, dp = rem % pieces;
        if (wide) join_cta(c, h, dp, JoinWidth<DV >= 128 ? 128 : 64>{});
        else join_cta(c, h, dp, JoinWidth<64>{});
    }
    cta_release_and_trigger();
}

}  // namespace hsp
