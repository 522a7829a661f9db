// kernels_append.cu -- the new tokens' keys and values into their pages, with the rotary
// turn of keys and queries on the way.
//
//   k row of token i -> page table[rows[i]][pos / page size], line pos mod page size, its last
//   `rot` columns turned by the angles of pos:
//     (a, b) -> (a cos - b sin, b cos + a sin),
//   pairs (2j, 2j + 1) or (j, j + rot / 2); v rows as they are; query rows turned alike.
//
// Every value is read once and written once in 16-byte pieces; products and sums in fp32, one
// rounding to bf16.  A thread takes pieces (pairs of pieces where the pairs lie rot / 2 apart),
// two requested before either is stored.  A CTA looks up the places of its tokens first (row and
// position, then the page and the length: two dependent loads, which bound the small calls, and
// the large ones where their rows come from DRAM: none is requested before).  On a GB300, graph
// replay: 8 latent tokens with 16 query heads 2.3 us; 2047 tokens of 8 + 8 + 32 heads of 128
// (51 MB) held by L2 15.1 us with a CTA per token and a fence per thread, 9.9 with up to eight
// tokens behind one look-up and one fence, 8.5 with multiplications for the divisions by the rows'
// pieces; 8.7 with the rows' lengths read too and the trigger behind the fence, 11.8 from DRAM.
#include <cuda_bf16.h>
#include <stdint.h>

#include "cache_args.h"
#include "ptx.cuh"

namespace hsp {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;  // most tokens per CTA

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Four interleaved pairs of one piece.
__device__ __forceinline__ uint4 turn_pairs(uint4 v, const float4 c, const float4 s) {
    uint4 o;
    o.x = pack_bf16(bf_lo(v.x) * c.x - bf_hi(v.x) * s.x, bf_hi(v.x) * c.x + bf_lo(v.x) * s.x);
    o.y = pack_bf16(bf_lo(v.y) * c.y - bf_hi(v.y) * s.y, bf_hi(v.y) * c.y + bf_lo(v.y) * s.y);
    o.z = pack_bf16(bf_lo(v.z) * c.z - bf_hi(v.z) * s.z, bf_hi(v.z) * c.z + bf_lo(v.z) * s.z);
    o.w = pack_bf16(bf_lo(v.w) * c.w - bf_hi(v.w) * s.w, bf_hi(v.w) * c.w + bf_lo(v.w) * s.w);
    return o;
}
// Two columns of either half: a (first half) and b (second half).
__device__ __forceinline__ void turn_halves(uint32_t &a, uint32_t &b, float c0, float c1, float s0, float s1) {
    const float a0 = bf_lo(a), a1 = bf_hi(a), b0 = bf_lo(b), b1 = bf_hi(b);
    a = pack_bf16(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
    b = pack_bf16(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
}

// n / d for n < 2^31: multiply by floor(2^(32 + s) / d) + 1, s = floor(log2 d), and shift (the
// product is too large by at most n d <= 2^(32 + s), so the quotient is exact); a power of two
// only shifts.
struct FastDiv {
    uint32_t mul, shift;
    explicit FastDiv(int d) {
        shift = 0;
        while (d >> (shift + 1)) ++shift;
        mul = (d & (d - 1)) == 0 ? 0u : static_cast<uint32_t>((1ull << (32 + shift)) / static_cast<uint32_t>(d)) + 1u;
    }
    __device__ __forceinline__ int operator()(int n) const {
        return static_cast<int>(mul ? __umulhi(static_cast<uint32_t>(n), mul) >> shift : static_cast<uint32_t>(n) >> shift);
    }
};
struct AppendShape {  // pieces of a token
    int plain, per_row, per_v, nk, nv, total;
    FastDiv by_total, by_row, by_v;
};

struct AppendPlace {
    int64_t k, v;      // element offsets of the token's line in the cache, -1: nowhere
    const float *cs;   // its angles; null: none (or outside the table)
};

__global__ void __launch_bounds__(kAppendThreads, 4) hsp_append_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ AppendShape g,
                                                                     int per_cta) {
    __shared__ AppendPlace places[kAppendTokens];
    griddep_wait();
    const int first = blockIdx.x * per_cta, here = min(per_cta, a.tokens - first);
    if (threadIdx.x < here) {
        const int i = first + threadIdx.x;
        const int row = a.rows ? a.rows[i] : i;
        const bool row_ok = row >= 0 && row < a.num_rows;
        const int len = row_ok ? a.lens[row] : 0;
        const int pos = a.positions ? a.positions[i] : len - 1;
        int page = -1;
        if (row_ok && pos >= 0 && (pos >> a.page_shift) < a.max_pages)
            page = a.table[row * a.table_stride + (pos >> a.page_shift)];
        if (pos >= len) page = -1;  // behind the row's end, as where its growth found no free page (on the way with the table's entry)
        if (a.refs && page >= 0 && page < a.num_pages && a.refs[page] > 1) page = -1;  // others hold it too
        const bool angle = a.rot > 0 && pos >= 0 && pos < a.max_pos;
        const int64_t line = pos & ((1 << a.page_shift) - 1);
        AppendPlace p;
        p.k = p.v = -1;
        p.cs = angle ? a.cos_sin + static_cast<int64_t>(pos) * a.rot : nullptr;
        if (page >= 0 && page < a.num_pages && (angle || a.rot == 0)) {
            p.k = page * a.k_page + line * a.k_token;
            p.v = page * a.v_page + line * a.v_token;
        } else if (blockIdx.y == 0) {
            atomicCAS(a.err_word, 0, kDeviceErrIndex);
        }
        places[threadIdx.x] = p;
    }
    __syncthreads();
    const int half = a.rot / 2, total = g.total;
    const int step = gridDim.y * kAppendThreads;
    for (int e0 = blockIdx.y * kAppendThreads + threadIdx.x; e0 < total * here; e0 += 2 * step) {
        uint4 v[2], w[2];
        __nv_bfloat16 *to[2];
        const float *cs[2];  // angles of a piece that is turned
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int e = e0 + u * step;
            to[u] = nullptr;
            cs[u] = nullptr;
            if (e >= total * here) continue;
            const int tok = g.by_total(e), x = e - tok * total, i = first + tok;
            const AppendPlace p = places[tok];
            // piece t of head h of k (kind 0), v (1) or q (2)
            const int kind = x < g.nk ? 0 : x < g.nk + g.nv ? 1 : 2;
            const int r = x - (kind == 0 ? 0 : kind == 1 ? g.nk : g.nk + g.nv);
            const int h = kind == 1 ? g.by_v(r) : g.by_row(r), t = r - h * (kind == 1 ? g.per_v : g.per_row);
            const __nv_bfloat16 *from;
            if (kind == 0) {
                from = static_cast<const __nv_bfloat16 *>(a.k_new) + i * a.k_row + h * a.k_dim;
                if (p.k >= 0) to[u] = static_cast<__nv_bfloat16 *>(a.k) + p.k + h * a.k_head + t * 8;
            } else if (kind == 1) {
                from = static_cast<const __nv_bfloat16 *>(a.v_new) + i * a.v_row + h * a.v_dim;
                if (p.v >= 0) to[u] = static_cast<__nv_bfloat16 *>(a.v) + p.v + h * a.v_head + t * 8;
            } else {
                from = static_cast<const __nv_bfloat16 *>(a.q) + i * a.q_row + h * a.q_head;
                if (p.cs) to[u] = static_cast<__nv_bfloat16 *>(a.q_out) + i * a.qo_row + h * a.qo_head + t * 8;
            }
            if (!to[u]) continue;
            v[u] = *reinterpret_cast<const uint4 *>(from + t * 8);
            if (kind != 1 && t >= g.plain) {
                cs[u] = p.cs + (t - g.plain) * (a.interleaved ? 4 : 8);
                if (!a.interleaved) w[u] = *reinterpret_cast<const uint4 *>(from + t * 8 + half);
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (!to[u]) continue;
            if (cs[u]) {
                const float4 c0 = *reinterpret_cast<const float4 *>(cs[u]), s0 = *reinterpret_cast<const float4 *>(cs[u] + half);
                if (a.interleaved) {
                    v[u] = turn_pairs(v[u], c0, s0);
                } else {
                    const float4 c1 = *reinterpret_cast<const float4 *>(cs[u] + 4);
                    const float4 s1 = *reinterpret_cast<const float4 *>(cs[u] + half + 4);
                    turn_halves(v[u].x, w[u].x, c0.x, c0.y, s0.x, s0.y);
                    turn_halves(v[u].y, w[u].y, c0.z, c0.w, s0.z, s0.w);
                    turn_halves(v[u].z, w[u].z, c1.x, c1.y, s1.x, s1.y);
                    turn_halves(v[u].w, w[u].w, c1.z, c1.w, s1.z, s1.w);
                    *reinterpret_cast<uint4 *>(to[u] + half) = w[u];
                }
            }
            *reinterpret_cast<uint4 *>(to[u]) = v[u];
        }
    }
    cta_release_and_trigger();
}

cudaError_t launch_append(const AppendArgs &a, int sms, int pdl, cudaStream_t stream) {
    // pieces of a k or q row: copied ones, then turned ones (a pair of pieces each where the pairs lie apart)
    const int plain = (a.k_dim - a.rot) / 8, per_row = plain + a.rot / (a.interleaved ? 8 : 16);
    const int per_v = a.v_new ? a.v_dim / 8 : 0, nk = a.kv_heads * per_row, nv = a.kv_heads * per_v;
    const int total = nk + nv + (a.q ? a.heads * per_row : 0);
    const AppendShape g{plain, per_row, per_v, nk, nv, total, FastDiv(total), FastDiv(per_row), FastDiv(per_v > 0 ? per_v : 1)};
    // as many CTAs as fit the GPU at once (four per SM): few tokens are spread over several CTAs each,
    // a piece per thread at least; of many, a CTA takes up to kAppendTokens
    const int fit = sms * 4;
    int y = (total + kAppendThreads - 1) / kAppendThreads, per_cta = 1;
    if (static_cast<int64_t>(a.tokens) * y > fit) y = fit / a.tokens > 1 ? fit / a.tokens : 1;
    if (a.tokens > fit) per_cta = (a.tokens + fit - 1) / fit;
    if (per_cta > kAppendTokens) per_cta = kAppendTokens;
    if (y > 65535) y = 65535;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.tokens + per_cta - 1) / per_cta), static_cast<unsigned>(y), 1);
    cfg.blockDim = dim3(kAppendThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[1];
    unsigned n = 0;
    if (pdl) {
        attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attrs;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, hsp_append_kernel, a, g, per_cta);
}

}  // namespace hsp
