// kernels_read_q8.cu -- tokens of a cache held in 8 bits, in bf16: out = round(code * scale).
//
// One byte read and two written per element.  A CTA looks up the places of up to eight tokens, then its threads take
// pieces of 16 codes, four requested before the first is stored.
#include <cuda_bf16.h>
#include <stdint.h>

#include "append_common.cuh"
#include "cache_args.h"
#include "ptx.cuh"
#include "q8.cuh"

namespace hsp {

constexpr int kRead8Threads = 256;
constexpr int kRead8Tokens = 8;
constexpr int kRead8Ahead = 4;

struct Read8Shape {
    int per_cta, parts, nk, row, vrow, total;  // pieces of 16 codes: of a token's keys, of a key row, a value row, a token
    FastDiv by_total, by_row, by_vrow;
};

struct Read8Place {
    int page, line;  // page -1: zeros
};

__global__ void __launch_bounds__(kRead8Threads) hsp_read_q8_kernel(const __grid_constant__ ReadQ8Args a, const __grid_constant__ Read8Shape g) {
    __shared__ Read8Place places[kRead8Tokens];
    griddep_wait();
    const int first = blockIdx.x * g.per_cta, here = min(g.per_cta, a.tokens - first);
    if (threadIdx.x < here) {
        const int i = first + threadIdx.x;
        const int row = a.rows ? a.rows[i] : i;
        const bool row_ok = row >= 0 && row < a.num_rows;
        const int len = row_ok ? a.lens[row] : 0;
        const int pos = a.positions ? a.positions[i] : len - 1;
        int page = -1;
        if (row_ok && pos >= 0 && (pos >> a.page_shift) < a.max_pages) page = a.table[row * a.table_stride + (pos >> a.page_shift)];
        if (pos >= len || page < 0 || page >= a.num_pages) {
            page = -1;
            if (blockIdx.y == 0) atomicCAS(a.err_word, 0, kDeviceErrIndex);
        }
        places[threadIdx.x].page = page;
        places[threadIdx.x].line = pos & ((1 << a.page_shift) - 1);
    }
    __syncthreads();
    const int step = gridDim.y * kRead8Threads, all = g.total * here;
    for (int e0 = blockIdx.y * kRead8Threads + threadIdx.x; e0 < all; e0 += kRead8Ahead * step) {
        uint4 c[kRead8Ahead];
        float scale[kRead8Ahead];
        __nv_bfloat16 *to[kRead8Ahead];
#pragma unroll
        for (int u = 0; u < kRead8Ahead; ++u) {
            const int e = e0 + u * step;
            to[u] = nullptr;
            if (e >= all) continue;
            const int tok = g.by_total(e), x = e - tok * g.total;
            const bool is_k = x < g.nk;
            const int r = is_k ? x : x - g.nk;
            const int h = is_k ? g.by_row(r) : g.by_vrow(r), t = r - h * (is_k ? g.row : g.vrow);
            const Q8Side &s = is_k ? a.k : a.v;
            to[u] = static_cast<__nv_bfloat16 *>(is_k ? a.k_out : a.v_out) + (first + tok) * (is_k ? a.k_row : a.v_row) + h * s.dim + t * 16;
            const Read8Place p = places[tok];
            c[u] = make_uint4(0, 0, 0, 0);
            scale[u] = 0.f;
            if (p.page < 0) continue;
            c[u] = *reinterpret_cast<const uint4 *>(s.codes + p.page * s.page + p.line * s.token + h * s.head + t * 16);
            scale[u] = s.scales[p.page * s.s_page + (p.line >> a.block_shift) * s.s_block + h * s.s_head];
        }
#pragma unroll
        for (int u = 0; u < kRead8Ahead; ++u) {
            if (!to[u]) continue;
            const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 lo = __half22float2(e4m3x2_to_half2(w[k] & 0xffffu)), hi = __half22float2(e4m3x2_to_half2(w[k] >> 16));
                o[2 * k] = pack_bf16(lo.x * scale[u], lo.y * scale[u]);
                o[2 * k + 1] = pack_bf16(hi.x * scale[u], hi.y * scale[u]);
            }
            reinterpret_cast<uint4 *>(to[u])[0] = make_uint4(o[0], o[1], o[2], o[3]);
            reinterpret_cast<uint4 *>(to[u])[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
    cta_release_and_trigger();
}

cudaError_t launch_read_q8(const ReadQ8Args &a, int sms, int pdl, cudaStream_t stream) {
    const int row = a.k.dim / 16, vrow = a.v.codes ? a.v.dim / 16 : 1;
    const int nk = a.kv_heads * row, total = nk + (a.v.codes ? a.kv_heads * vrow : 0);
    const int fit = sms * 4;
    int y = (total + kRead8Threads - 1) / kRead8Threads, per_cta = 1;
    if (static_cast<int64_t>(a.tokens) * y > fit) y = fit / a.tokens > 1 ? fit / a.tokens : 1;
    if (a.tokens > fit) per_cta = (a.tokens + fit - 1) / fit;
    if (per_cta > kRead8Tokens) per_cta = kRead8Tokens;
    if (y > 65535) y = 65535;
    const Read8Shape g{per_cta, y, nk, row, vrow, total, FastDiv(total), FastDiv(row), FastDiv(vrow)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.tokens + per_cta - 1) / per_cta), static_cast<unsigned>(y), 1);
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
