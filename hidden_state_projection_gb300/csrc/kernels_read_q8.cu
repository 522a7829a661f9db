// kernels_read_q8.cu -- tokens of a cache held in 8 bits, in bf16: out = round(code * scale).
//
// One byte read and two written per element.  A CTA looks up the places of up to 32 tokens (three dependent loads), then its
// threads take pieces of 16 codes, keys first, four requested before the first is stored; where outputs are 32-byte
// aligned a piece goes out in one store.  Memory bounds it: 40009 tokens of 8 heads of 128 columns, keys and values, 246 MB in
// 42.9 us (5.7 TB/s; 36.8 at the copy rate); 16001 latent tokens 5.8 us (4.2); 77 2.4, a launch and three dependent loads.
#include <cuda_bf16.h>
#include <stdint.h>

#include "append_common.cuh"
#include "cache_args.h"
#include "ptx.cuh"
#include "q8.cuh"

namespace hsp {

constexpr int kRead8Threads = 256;
constexpr int kRead8Tokens = 32;
constexpr int kRead8Ahead = 4;

struct Read8Shape {
    int per_cta, krow, vrow, wide;   // tokens per CTA; pieces of 16 codes of a key and a value row; whether 32-byte stores may be used
    FastDiv by_k, by_v, by_krow, by_vrow;
};

struct Read8Place {
    int64_t codes, scales;           // offsets of the token's line and block, codes -1: zeros
};

__device__ __forceinline__ void store32(void *p, const uint32_t (&o)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]),
                 "r"(o[5]), "r"(o[6]), "r"(o[7])
                 : "memory");
}

// Two codes times s, in bf16, where fp32 does not hold the products.  (A function of its own: in line it made the usual case's code longer,
// 2.4 -> 2.5 us for 77 tokens.)
__device__ __noinline__ uint32_t products_odd(uint32_t codes, float s) {
    const float2 x = __half22float2(e4m3x2_to_half2(codes));
    return pack_bf16(product_odd(x.x, s), product_odd(x.y, s));
}

__global__ void __launch_bounds__(kRead8Threads, 4) hsp_read_q8_kernel(const __grid_constant__ ReadQ8Args a, const __grid_constant__ Read8Shape g) {
    __shared__ Read8Place places[2][kRead8Tokens];
    griddep_wait();
    const int first = blockIdx.x * g.per_cta, here = min(g.per_cta, a.tokens - first);
    if (threadIdx.x < here) {
        const int i = first + threadIdx.x;
        const int row = a.rows ? a.rows[i] : i;
        const int given = a.positions ? a.positions[i] : 0;
        const bool row_ok = row >= 0 && row < a.num_rows;
        const int len = row_ok ? a.lens[row] : 0;
        const int pos = a.positions ? given : len - 1;
        int page = -1;
        if (row_ok && pos >= 0 && (pos >> a.page_shift) < a.max_pages) page = a.table[row * a.table_stride + (pos >> a.page_shift)];
        if (pos >= len || page < 0 || page >= a.num_pages) {
            page = -1;
            if (blockIdx.y == 0) atomicCAS(a.err_word, 0, kDeviceErrIndex);
        }
        const int line = pos & ((1 << a.page_shift) - 1), blk = line >> a.block_shift;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Q8Side &s = k == 0 ? a.k : a.v;
            places[k][threadIdx.x].codes = page < 0 ? -1 : page * s.page + line * s.token;
            places[k][threadIdx.x].scales = page * s.s_page + blk * s.s_block;
        }
    }
    __syncthreads();
    const int step = gridDim.y * kRead8Threads, from = blockIdx.y * kRead8Threads + threadIdx.x;
#pragma unroll 1
    for (int side = 0; side < (a.v.codes ? 2 : 1); ++side) {
        const Q8Side s = side == 0 ? a.k : a.v;
        const FastDiv by = side == 0 ? g.by_k : g.by_v, by_row = side == 0 ? g.by_krow : g.by_vrow;
        const int row = side == 0 ? g.krow : g.vrow, per = row * a.kv_heads, all = per * here;
        const int64_t out_row = side == 0 ? a.k_row : a.v_row;
        __nv_bfloat16 *const out = static_cast<__nv_bfloat16 *>(side == 0 ? a.k_out : a.v_out) + first * out_row;
#pragma unroll 1
        for (int e0 = from; e0 < all; e0 += kRead8Ahead * step) {
            uint4 c[kRead8Ahead];
            float scale[kRead8Ahead];
#pragma unroll
            for (int u = 0; u < kRead8Ahead; ++u) {
                const int e = e0 + u * step;
                c[u] = make_uint4(0, 0, 0, 0);
                scale[u] = 0.f;
                if (e >= all) continue;
                const int tok = by(e), x = e - tok * per, h = by_row(x);
                const Read8Place p = places[side][tok];
                if (p.codes < 0) continue;
                c[u] = *reinterpret_cast<const uint4 *>(s.codes + p.codes + h * s.head + (x - h * row) * 16);
                scale[u] = s.scales[p.scales + h * s.s_head];
            }
#pragma unroll
            for (int u = 0; u < kRead8Ahead; ++u) {
                const int e = e0 + u * step;
                if (e >= all) continue;
                const int tok = by(e), x = e - tok * per;
                const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
                uint32_t o[8];
                if (__builtin_expect((__float_as_uint(scale[u]) & 15u) == 0u, true)) {  // (a code has four bits: the product is exact)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float2 x = __half22float2(e4m3x2_to_half2(k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu));
                        o[k] = pack_bf16(x.x * scale[u], x.y * scale[u]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = products_odd(k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu, scale[u]);
                }
                __nv_bfloat16 *to = out + tok * out_row + x * 16;  // (a token's heads lie one after another)
                if (g.wide) {
                    store32(to, o);
                } else {
                    reinterpret_cast<uint4 *>(to)[0] = make_uint4(o[0], o[1], o[2], o[3]);
                    reinterpret_cast<uint4 *>(to)[1] = make_uint4(o[4], o[5], o[6], o[7]);
                }
            }
        }
    }
    cta_release_and_trigger();
}

cudaError_t launch_read_q8(const ReadQ8Args &a, int sms, int pdl, cudaStream_t stream) {
    const int krow = a.k.dim / 16, vrow = a.v.codes ? a.v.dim / 16 : 1;
    const int kper = a.kv_heads * krow, vper = a.v.codes ? a.kv_heads * vrow : 1;
    const int total = kper > vper ? kper : vper;
    const int fit = sms * 4;
    int y = (total + kRead8Threads - 1) / kRead8Threads, per_cta = 1;
    if (static_cast<int64_t>(a.tokens) * y > fit) y = fit / a.tokens > 1 ? fit / a.tokens : 1;
    if (a.tokens > fit) per_cta = static_cast<int>((static_cast<int64_t>(a.tokens) + fit - 1) / fit);
    if (per_cta > kRead8Tokens) per_cta = kRead8Tokens;
    if (y > 65535) y = 65535;
    auto wide = [&](const void *p, int64_t row) { return reinterpret_cast<uintptr_t>(p) % 32 == 0 && row % 16 == 0; };
    const Read8Shape g{per_cta, krow, vrow, wide(a.k_out, a.k_row) && wide(a.v_out, a.v_row) ? 1 : 0, FastDiv(kper), FastDiv(vper), FastDiv(krow), FastDiv(vrow)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(a.tokens) + per_cta - 1) / per_cta), static_cast<unsigned>(y), 1);
    cfg.blockDim = dim3(kRead8Threads, 1, 1);
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
    return cudaLaunchKernelEx(&cfg, hsp_read_q8_kernel, a, g);
}

}  // namespace hsp
