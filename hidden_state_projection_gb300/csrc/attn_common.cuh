// attn_common.cuh -- what the attention kernels over a paged cache share (attn_kernel.cuh: bf16, attn8_kernel.cuh: 8
// bits): tcgen05 pieces, the line of tiles that is cut over the CTAs, the way of O^T out of tensor memory.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "cache_args.h"
#include "packed.cuh"
#include "ptx.cuh"
#include "stream_args.h"

namespace hsp {

// ---- tcgen05 pieces ------------------------------------------------------------------

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

// Barrier 1 of the softmax threads, and the same with an OR over their predicates.
template <int THREADS = 128>
__device__ __forceinline__ void softmax_sync() {
    asm volatile("barrier.cta.sync.aligned 1, %0;" ::"n"(THREADS) : "memory");
}
template <int THREADS = 128>
__device__ __forceinline__ bool softmax_any(bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred.aligned q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(p)), "n"(THREADS)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
template <int TILE>
__device__ __forceinline__ int attn_tiles(int len) {
    return static_cast<int>((static_cast<uint32_t>(len) + TILE - 1) / TILE);
}

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

template <int TILE>
__device__ __forceinline__ bool attn_next_segment(const AttnArgs &a, const AttnLine &ln, AttnWalk &w, AttnSegment &s) {
    while (w.x < ln.x1) {
        if (!a.split) {  // whole sequences, taken in turn
            const int item = static_cast<int>(w.x);
            w.x += a.ctas;
            s.b = item / a.kv_heads;
            s.kv = item - s.b * a.kv_heads;
            s.len = attn_len(a, s.b);
            s.n = s.tiles = attn_tiles<TILE>(s.len);
            s.t0 = 0;
            s.x0 = item;
            s.end = item + 1;
            if (s.n > 0) return true;
            continue;
        }
        uint32_t units;
        for (;;) {
            units = w.len > 0 ? attn_tiles<TILE>(w.len) + a.weight : 0;
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

// The length of the line, and where this CTA's first unit lies (called by all of its threads).
// Up to 128 sequences: every warp for itself (no thread waits for another warp); more: the CTA.
// place: three ints, warp_sum: one for each warp, in shared memory.
template <int TILE, int THREADS>
__device__ __forceinline__ AttnLine attn_find_line(const AttnArgs &a, int cta, int *place, int *warp_sum) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    AttnLine ln;
    ln.total = ln.x1 = static_cast<uint32_t>(a.batch) * a.kv_heads;  // uncut: the items
    ln.x0 = cta;
    ln.ctas = a.ctas;
    ln.base = 0;
    ln.b0 = ln.len0 = 0;
    if (a.split) {
        const bool by_warp = a.batch <= 128;
        const int tn = by_warp ? 32 : THREADS, tno = by_warp ? lane : tid;
        const int per = (a.batch + tn - 1) / tn;
        const int bfirst = min(a.batch, tno * per), blast = min(a.batch, bfirst + per);
        uint32_t mine = 0;
        int len = 0;
        for (int b = bfirst; b < blast; ++b) {
            len = attn_len(a, b);
            mine += len > 0 ? attn_tiles<TILE>(len) + a.weight : 0;
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
            for (int w = 0; w < THREADS / 32; ++w) {
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
                    const uint32_t units = len > 0 ? (attn_tiles<TILE>(len) + a.weight) * a.kv_heads : 0;
                    if (ln.x0 < first + units || b + 1 >= blast) break;
                    first += units;
                }
            }
            // its first page id, on its way before the copy producer asks for it
            const uint32_t units = attn_tiles<TILE>(len) + a.weight;
            const uint32_t t = (ln.x0 - first) % units;
            const int64_t page = (static_cast<int64_t>(max(0, static_cast<int>(t) - a.weight)) * TILE) >> a.page_shift;
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
    return ln;
}

// ---- the end of a part -----------------------------------------------------------------
//
// O^T (OT tiles of MV value columns, N heads each) out of tensor memory by SETS times four warps (warp: of the four, set:
// which steps of 16 columns): a whole sequence's rows times fac[head] to `out`, of a cut one to its partial, as they
// are.  Heads from `nheads` on go nowhere.
template <int N, int DV, int MV, int OT, int SETS = 1>
__device__ __forceinline__ void attn_store_part(uint32_t tmem, int warp, int lane, bool good, bool whole, int nheads, const float *fac,
                                                __nv_bfloat16 *out, float *part, int set = 0) {
    constexpr int rpw = MV / 4;
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
#pragma unroll 1
    for (int c0 = set * 16; c0 < OT * N; c0 += SETS * 16) {
        const int h0 = c0 & (N - 1);
        if (h0 >= nheads) continue;
        float o[16];
        tmem_ld16(tmem + c0 + lane_base, o);
        tmem_wait_ld();
        const int dv = (c0 / N) * MV + warp * rpw + lane;
        if (lane < rpw && good) {
            if (whole) {
                __nv_bfloat16 *to = out + static_cast<int64_t>(h0) * DV + dv;
                if (h0 + 16 <= nheads) {  // (16 tests take longer than the stores)
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(fac + h0 + e);
                        to[e * DV] = __float2bfloat16_rn(o[e] * f.x);
                        to[(e + 1) * DV] = __float2bfloat16_rn(o[e + 1] * f.y);
                        to[(e + 2) * DV] = __float2bfloat16_rn(o[e + 2] * f.z);
                        to[(e + 3) * DV] = __float2bfloat16_rn(o[e + 3] * f.w);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 15; ++e)
                        if (h0 + e < nheads) to[e * DV] = __float2bfloat16_rn(o[e] * fac[h0 + e]);
                }
            } else {
                float *to = part + h0 * DV + dv;
                if (h0 + 16 <= nheads) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) to[e * DV] = o[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 15; ++e)
                        if (h0 + e < nheads) to[e * DV] = o[e];
                }
            }
        }
    }
}

// Sequences without a token: zeros, and no weight at all (128 threads of each CTA).
template <int DV>
__device__ __forceinline__ void attn_store_empty(const AttnArgs &a, int cta, int head0, int nheads) {
    const int tid = threadIdx.x, all_heads = a.kv_heads * a.group;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
    for (int e = cta; e < a.batch; e += a.ctas) {
        if (attn_len<true>(a, e) != 0) continue;
        for (int kv = 0; kv < a.kv_heads; ++kv) {
            const int64_t h = static_cast<int64_t>(e) * all_heads + kv * a.group + head0;
            uint4 *to = reinterpret_cast<uint4 *>(out + h * DV);  // (its heads lie one after another)
            for (int c = tid; c < nheads * DV / 8; c += 128) to[c] = make_uint4(0, 0, 0, 0);
            if (a.lse)
                for (int c = tid; c < nheads; c += 128) a.lse[h + c] = -INFINITY;
        }
    }
}

}  // namespace hsp
