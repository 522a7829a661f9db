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
// position, then the page: two dependent loads, which bound the small calls): one token, its
// pieces spread over several CTAs, while that does not fill the GPU, up to eight behind one
// look-up and one release fence otherwise (2047 tokens of 48 heads of 128: 16.7 us with a CTA
// per token, 51 MB).
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

struct AppendPlace {
    int64_t k, v;      // element offsets of the token's line in the cache, -1: nowhere
    const float *cs;   // its angles; null: none (or outside the table)
};

__global__ void __launch_bounds__(kAppendThreads, 4) hsp_append_kernel(const __grid_constant__ AppendArgs a, int per_cta) {
    __shared__ AppendPlace places[kAppendTokens];
    griddep_wait();
    const int first = blockIdx.x * per_cta, here = min(per_cta, a.tokens - first);
    if (threadIdx.x < here) {
        const int i = first + threadIdx.x;
        const int row = a.rows ? a.rows[i] : i;
        const bool row_ok = row >= 0 && row < a.num_rows;
        const int pos = a.positions ? a.positions[i] : row_ok ? a.lens[row] - 1 : -1;
        int page = -1;
        if (row_ok && pos >= 0 && (pos >> a.page_shift) < a.max_pages)
            page = a.table[row * a.table_stride + (pos >> a.page_shift)];
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
    const int plain = (a.k_dim - a.rot) / 8;                               // pieces of a k or q row that are copied
    const int turned = a.rot / (a.interleaved ? 8 : 16);                   // and those that are turned
    const int per_row = plain + turned, per_v = a.v_new ? a.v_dim / 8 : 0;
    const int nk = a.kv_heads * per_row, nv = a.kv_heads * per_v, nq = a.q ? a.heads * per_row : 0;
    const int total = nk + nv + nq, half = a.rot / 2;
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
            const int tok = e / total, x = e - tok * total, i = first + tok;
            const AppendPlace p = places[tok];
            // piece t of head h of k (kind 0), v (1) or q (2)
            const int kind = x < nk ? 0 : x < nk + nv ? 1 : 2;
            const int r = x - (kind == 0 ? 0 : kind == 1 ? nk : nk + nv), per = kind == 1 ? per_v : per_row;
            const int h = r / per, t = r - h * per;
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
            if (kind != 1 && t >= plain) {
                cs[u] = p.cs + (t - plain) * (a.interleaved ? 4 : 8);
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
    __syncthreads();
    if (threadIdx.x == 0) fence_release_gpu();  // (cumulative over the barrier)
    griddep_launch_dependents();
}

cudaError_t launch_append(const AppendArgs &a, int sms, int pdl, cudaStream_t stream) {
    const int per_row = (a.k_dim - a.rot) / 8 + a.rot / (a.interleaved ? 8 : 16);
    const int total = a.kv_heads * (per_row + (a.v_new ? a.v_dim / 8 : 0)) + (a.q ? a.heads * per_row : 0);
    // one token per CTA and a thread per piece while the CTAs fit the GPU at once, else more tokens
    int y = (total + kAppendThreads - 1) / kAppendThreads;
    if (y > 65535) y = 65535;
    int per_cta = 1;
    while (per_cta < kAppendTokens && static_cast<int64_t>(a.tokens) * y > static_cast<int64_t>(sms) * 4 * per_cta) per_cta *= 2;
    if (per_cta > 1) y = 1;
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
    return cudaLaunchKernelEx(&cfg, hsp_append_kernel, a, per_cta);
}

}  // namespace hsp
