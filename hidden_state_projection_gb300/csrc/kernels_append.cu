// kernels_append.cu -- the new tokens' keys and values into their pages, with the rotary
// turn of keys and queries on the way.
//
//   k row of token i -> page table[rows[i]][pos / page size], line pos mod page size, its last
//   `rot` columns turned by the angles of pos:
//     (a, b) -> (a cos - b sin, b cos + a sin),
//   pairs (2j, 2j + 1) or (j, j + rot / 2); v rows as they are; query rows turned alike.
//
// Every value is read once and written once in 16-byte pieces; products and sums in fp32, one
// rounding to bf16.  A thread takes one piece (a pair of pieces where the pairs lie rot / 2
// apart); a token's pieces are spread over enough CTAs that a decode step of a few tokens is
// one round of loads.  The page lookup (row, position, table) is a chain of dependent loads:
// it bounds the small calls, the copied bytes the large ones.
#include <cuda_bf16.h>
#include <stdint.h>

#include "cache_args.h"
#include "ptx.cuh"

namespace hsp {

constexpr int kAppendThreads = 128;
constexpr int kAppendPieces = 2;  // pieces per thread, all loads before the stores

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

__global__ void __launch_bounds__(kAppendThreads) hsp_append_kernel(const __grid_constant__ AppendArgs a) {
    griddep_wait();
    const int i = blockIdx.x;
    const int plain = (a.k_dim - a.rot) / 8;                               // pieces of a k or q row that are copied
    const int turned = a.rot / (a.interleaved ? 8 : 16);                   // and those that are turned
    const int per_row = plain + turned, per_v = a.v_new ? a.v_dim / 8 : 0;
    const int nk = a.kv_heads * per_row, nv = a.kv_heads * per_v, nq = a.q ? a.heads * per_row : 0;
    const int row = a.rows ? a.rows[i] : i;
    const bool row_ok = row >= 0 && row < a.num_rows;
    const int pos = a.positions ? a.positions[i] : (row_ok ? a.lens[row] - 1 : -1);
    const bool pos_ok = pos >= 0 && (pos >> a.page_shift) < a.max_pages;
    int page = -1;
    if (row_ok && pos_ok) page = a.table[row * a.table_stride + (pos >> a.page_shift)];
    const bool write = page >= 0 && page < a.num_pages;
    const bool turn = a.rot > 0;
    const bool angle = !turn || (pos >= 0 && pos < a.max_pos);
    if ((!write || !angle) && threadIdx.x == 0 && blockIdx.y == 0) atomicCAS(a.err_word, 0, kDeviceErrIndex);
    if (!angle) return;
    const int64_t line = pos & ((1 << a.page_shift) - 1);
    const float *cs = turn ? a.cos_sin + static_cast<int64_t>(pos) * a.rot : nullptr;
    const int total = nk + nv + nq;
    const int step = gridDim.y * kAppendThreads;
    for (int e0 = blockIdx.y * kAppendThreads + threadIdx.x; e0 < total; e0 += step * kAppendPieces) {
        uint4 v[kAppendPieces], w[kAppendPieces];
        __nv_bfloat16 *to[kAppendPieces], *to2[kAppendPieces];
#pragma unroll
        for (int u = 0; u < kAppendPieces; ++u) {
            const int e = e0 + u * step;
            to[u] = to2[u] = nullptr;
            if (e >= total) continue;
            const __nv_bfloat16 *from;
            __nv_bfloat16 *dst;
            int t;
            bool is_v = false;
            if (e < nk) {
                const int h = e / per_row;
                t = e - h * per_row;
                from = static_cast<const __nv_bfloat16 *>(a.k_new) + i * a.k_row + static_cast<int64_t>(h) * a.k_dim;
                dst = write ? static_cast<__nv_bfloat16 *>(a.k) + page * a.k_page + line * a.k_token + h * a.k_head : nullptr;
            } else if (e < nk + nv) {
                const int h = (e - nk) / per_v;
                t = e - nk - h * per_v;
                is_v = true;
                from = static_cast<const __nv_bfloat16 *>(a.v_new) + i * a.v_row + static_cast<int64_t>(h) * a.v_dim;
                dst = write ? static_cast<__nv_bfloat16 *>(a.v) + page * a.v_page + line * a.v_token + h * a.v_head : nullptr;
            } else {
                const int h = (e - nk - nv) / per_row;
                t = e - nk - nv - h * per_row;
                from = static_cast<const __nv_bfloat16 *>(a.q) + i * a.q_row + h * a.q_head;
                dst = static_cast<__nv_bfloat16 *>(a.q_out) + i * a.qo_row + h * a.qo_head;
            }
            if (!dst) continue;
            v[u] = *reinterpret_cast<const uint4 *>(from + t * 8);
            to[u] = dst + t * 8;
            if (is_v || t < plain) continue;
            const int j = t - plain;  // piece of the turned columns
            if (a.interleaved) {
                const float4 c = *reinterpret_cast<const float4 *>(cs + 4 * j);
                const float4 s = *reinterpret_cast<const float4 *>(cs + a.rot / 2 + 4 * j);
                v[u] = turn_pairs(v[u], c, s);
            } else {
                const int half = a.rot / 2;
                w[u] = *reinterpret_cast<const uint4 *>(from + t * 8 + half);
                to2[u] = dst + t * 8 + half;
                const float4 c0 = *reinterpret_cast<const float4 *>(cs + 8 * j), c1 = *reinterpret_cast<const float4 *>(cs + 8 * j + 4);
                const float4 s0 = *reinterpret_cast<const float4 *>(cs + half + 8 * j);
                const float4 s1 = *reinterpret_cast<const float4 *>(cs + half + 8 * j + 4);
                turn_halves(v[u].x, w[u].x, c0.x, c0.y, s0.x, s0.y);
                turn_halves(v[u].y, w[u].y, c0.z, c0.w, s0.z, s0.w);
                turn_halves(v[u].z, w[u].z, c1.x, c1.y, s1.x, s1.y);
                turn_halves(v[u].w, w[u].w, c1.z, c1.w, s1.z, s1.w);
            }
        }
#pragma unroll
        for (int u = 0; u < kAppendPieces; ++u) {
            if (to[u]) *reinterpret_cast<uint4 *>(to[u]) = v[u];
            if (to2[u]) *reinterpret_cast<uint4 *>(to2[u]) = w[u];
        }
    }
    fence_release_gpu();
    __syncthreads();
    griddep_launch_dependents();
}

cudaError_t launch_append(const AppendArgs &a, int pdl, cudaStream_t stream) {
    const int per_row = (a.k_dim - a.rot) / 8 + a.rot / (a.interleaved ? 8 : 16);
    const int total = a.kv_heads * (per_row + (a.v_new ? a.v_dim / 8 : 0)) + (a.q ? a.heads * per_row : 0);
    int y = (total + kAppendThreads * kAppendPieces - 1) / (kAppendThreads * kAppendPieces);
    if (y > 65535) y = 65535;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.tokens), static_cast<unsigned>(y), 1);
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
    return cudaLaunchKernelEx(&cfg, hsp_append_kernel, a);
}

}  // namespace hsp
