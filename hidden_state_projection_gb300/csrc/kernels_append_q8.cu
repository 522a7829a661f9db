// kernels_append_q8.cu -- new tokens into the pages of a cache held in 8 bits: the rotary turn of keys and
// queries, a scale for each block of tokens and head, and the codes.
//
// For the new tokens of one block and head, x their key (turned) or value rows:
//   s = the smallest power of two with amax |x| <= 448 s; not below the block's old scale where tokens
//       stand in front of them;  code = round(x / s);
//   where s grew, the codes in front are rounded to it (a shift of their exponents, exact unless the result
//   is below the smallest normal code).
// A turned value is rounded once, from the exact sum of its two products (dot2_odd), so a code does not
// depend on the order of operations.
//
// Two kinds of CTA in one launch.  The first `kv_ctas` write the cache: a CTA looks at `per_cta` tokens of
// the call, finds the runs of neighbouring tokens that share a row and block (a run belongs to the CTA that
// holds its first token), and takes (run, side, head) units: 8 lanes, a warp or the CTA, whichever leaves a lane at most
// eight 16-byte pieces.  The pieces are read twice, for the largest and for the codes.  The others turn queries, four pieces
// (or pairs) per thread requested at once.
#include <cuda_bf16.h>
#include <stdint.h>

#include "append_common.cuh"
#include "cache_args.h"
#include "ptx.cuh"
#include "q8.cuh"

namespace hsp {

constexpr int kAppend8Threads = 256;
constexpr int kAppend8Tokens = 32;   // most tokens that a CTA looks at (a lane each)
constexpr int kAppend8Lines = kAppend8Tokens + 1024;  // and those of the last one's block
constexpr int kAppend8Items = 8;     // pieces of a unit for a lane, where a larger group would leave fewer
constexpr int kAppend8Ahead = 4;     // pieces of queries that a lane has requested

struct Append8Shape {
    int kv_ctas, per_cta, parts;     // CTAs of the cache; tokens and CTAs of a chunk
    int q_per_cta;                   // tokens per CTA of the queries
    int q_parts;                     // CTAs of such a chunk
    int plain, row;                  // pieces of a query row (copied ones; all, turned pairs as one)
    int krow, vrow;                  // pieces of a key and a value row
    FastDiv by_row, by_krow, by_vrow, by_units, by_q, by_kv_heads;
};

struct Append8Run {
    int first, n;                    // its tokens
    int page;                        // -1: nowhere to write
    int block;                       // of the page
};

__device__ __forceinline__ int append8_pos(const AppendQ8Args &a, int i, int len) { return a.positions ? a.positions[i] : len - 1; }

// A group of G lanes (the CTA: G = 256) makes one unit's scale and codes.
template <int G>
struct Append8Unit {
    const AppendQ8Args &a;
    const Append8Shape &g;
    int t;          // this thread's place in the group
    uint32_t mask;  // lanes of the group

    // The eight numbers of piece x of a token's row: turned, where they are keys of a turned column.
    __device__ __forceinline__ void numbers(bool is_k, const __nv_bfloat16 *from, const uint4 &raw, int x, int pos, float2 (&v)[4]) const {
        v[0] = make_float2(bf_lo(raw.x), bf_hi(raw.x)), v[1] = make_float2(bf_lo(raw.y), bf_hi(raw.y));
        v[2] = make_float2(bf_lo(raw.z), bf_hi(raw.z)), v[3] = make_float2(bf_lo(raw.w), bf_hi(raw.w));
        if (!is_k || x < g.plain) return;
        const int half = a.rot / 2, y = (x - g.plain) * 8;
        const float *cs = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
        // partners w, cosines c and sines s (with the sign that they have in the sum) of the eight
        float2 w[4], c[4], s[4];
        if (a.interleaved) {
            const float4 cc = *reinterpret_cast<const float4 *>(cs + y / 2), ss = *reinterpret_cast<const float4 *>(cs + half + y / 2);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = make_float2(v[e].y, v[e].x);
            c[0] = make_float2(cc.x, cc.x), c[1] = make_float2(cc.y, cc.y), c[2] = make_float2(cc.z, cc.z), c[3] = make_float2(cc.w, cc.w);
            s[0] = make_float2(-ss.x, ss.x), s[1] = make_float2(-ss.y, ss.y), s[2] = make_float2(-ss.z, ss.z), s[3] = make_float2(-ss.w, ss.w);
        } else {
            // the piece's columns are all of the first or all of the second half, their partners half a turn away
            const bool second = y >= half;
            const int z = second ? y - half : y;
            const uint4 other = *reinterpret_cast<const uint4 *>(from + x * 8 + (second ? -half : half));
            w[0] = make_float2(bf_lo(other.x), bf_hi(other.x)), w[1] = make_float2(bf_lo(other.y), bf_hi(other.y));
            w[2] = make_float2(bf_lo(other.z), bf_hi(other.z)), w[3] = make_float2(bf_lo(other.w), bf_hi(other.w));
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float4 cc = *reinterpret_cast<const float4 *>(cs + z + 2 * e), ss = *reinterpret_cast<const float4 *>(cs + half + z + 2 * e);
                c[e] = make_float2(cc.x, cc.y), c[e + 1] = make_float2(cc.z, cc.w);
                s[e] = make_float2(second ? ss.x : -ss.x, second ? ss.y : -ss.y), s[e + 1] = make_float2(second ? ss.z : -ss.z, second ? ss.w : -ss.w);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = dot2_odd(v[e], c[e], w[e], s[e]);
    }

    // The largest of amax and the smallest of line over the group.
    __device__ __forceinline__ void reduce(float &amax, int &line, float *red, int *redi) const {
#pragma unroll
        for (int d = (G < 32 ? G : 32) / 2; d > 0; d >>= 1) {
            amax = fmaxf(amax, __shfl_xor_sync(mask, amax, d));
            line = min(line, __shfl_xor_sync(mask, line, d));
        }
        if (G > 32) {
            __syncthreads();  // what the last unit left there has been read
            if ((t & 31) == 0) {
                red[t >> 5] = amax;
                redi[t >> 5] = line;
            }
            __syncthreads();
#pragma unroll
            for (int w = 0; w < G / 32; ++w) {
                amax = fmaxf(amax, red[w]);
                line = min(line, redi[w]);
            }
        }
    }

    // lines: of the run's tokens in their page, -1: written nowhere; pos0: the first position of that page.
    __device__ void operator()(const Append8Run &r, const int16_t *lines, int pos0, bool is_k, int head, float *red, int *redi) const {
        const Q8Side &s = is_k ? a.k : a.v;
        const int per = is_k ? g.krow : g.vrow;
        const FastDiv &by = is_k ? g.by_krow : g.by_vrow;
        const int block = 1 << a.block_shift, items = r.n * per;
        float *const scale = s.scales + r.page * s.s_page + r.block * s.s_block + head * s.s_head;
        uint8_t *const codes = s.codes + r.page * s.page + head * s.head;
        const int64_t stride = is_k ? a.k_row : a.v_row;
        const __nv_bfloat16 *const rows = static_cast<const __nv_bfloat16 *>(is_k ? a.k_new : a.v_new) + r.first * stride + static_cast<int64_t>(head) * s.dim;
        const float old = *scale;
        constexpr float limit = kQ8Top * 1152921504606846976.f;  // 448 * 2^60
        float amax = 0.f;
        int line = block;  // first new line of the block
        auto piece = [&](int e) {
            const int j = by(e);
            return *reinterpret_cast<const uint4 *>(rows + j * stride + (e - j * per) * 8);
        };
        // Pieces one after the other, the next one requested before this one is worked on, as `each(line, x, numbers)`.
        // (Rolled, and twice from memory: with nine pieces in registers, unrolled, the code's way from L2 took longer than
        // the work, 2047 tokens of 8 heads of 128 columns 39 us for 29.)
        auto walk = [&](auto each) {
            uint4 next = t < items ? piece(t) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
            for (int e = t; e < items; e += G) {
                const uint4 raw = next;
                if (e + G < items) next = piece(e + G);
                const int j = by(e), x = e - j * per, at = lines[j];
                if (at < 0) continue;
                float2 v[4];
                numbers(is_k, rows + j * stride, raw, x, pos0 + at, v);
                each(at, x, v);
            }
        };
        walk([&](int at, int, const float2 (&v)[4]) {
            line = min(line, at & (block - 1));
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const float y = fabsf(v[f].x), z = fabsf(v[f].y);
                if (y <= limit) amax = fmaxf(amax, y);
                if (z <= limit) amax = fmaxf(amax, z);
            }
        });
        reduce(amax, line, red, redi);
        if (line == block) return;  // no token of the run is written
        float now = two_to(q8_exponent(amax));
        if (line > 0 && old >= now) now = old;
        const float inv = 1.f / now;  // (exact for the powers of two that this kernel writes)
        if (line > 0 && now > old) {
            // the codes in front, under the new scale
            const float by_new = old * inv;
            const int p16 = s.dim / 16;
            for (int e = t; e < line * p16; e += G) {
                const int l = e / p16, x = e - l * p16;
                uint4 *at = reinterpret_cast<uint4 *>(codes + (static_cast<int64_t>(r.block) * block + l) * s.token + x * 16);
                uint4 c = *at;
                uint32_t *w = reinterpret_cast<uint32_t *>(&c);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 lo = __half22float2(e4m3x2_to_half2(w[k] & 0xffffu)), hi = __half22float2(e4m3x2_to_half2(w[k] >> 16));
                    w[k] = float2_to_e4m3x2(lo.x * by_new, lo.y * by_new) | float2_to_e4m3x2(hi.x * by_new, hi.y * by_new) << 16;
                }
                *at = c;
            }
        }
        walk([&](int at, int x, const float2 (&v)[4]) {
            float2 y[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) y[f] = make_float2(q8_scaled(v[f].x, inv), q8_scaled(v[f].y, inv));
            uint2 c;
            c.x = float2_to_e4m3x2(y[0].x, y[0].y) | float2_to_e4m3x2(y[1].x, y[1].y) << 16;
            c.y = float2_to_e4m3x2(y[2].x, y[2].y) | float2_to_e4m3x2(y[3].x, y[3].y) << 16;
            *reinterpret_cast<uint2 *>(codes + static_cast<int64_t>(at) * s.token + x * 8) = c;
        });
        if (t == 0) *scale = now;
    }
};

template <int G>
__global__ void __launch_bounds__(kAppend8Threads, 3) hsp_append_q8_kernel(const __grid_constant__ AppendQ8Args a, const __grid_constant__ Append8Shape g) {
    __shared__ Append8Run runs[kAppend8Tokens];
    __shared__ int num_runs, first_pos[kAppend8Tokens];
    __shared__ int16_t lines[kAppend8Lines];
    __shared__ const float *angles[kAppend8Tokens];
    __shared__ float red[kAppend8Threads / 32];
    __shared__ int redi[kAppend8Threads / 32];
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    if (static_cast<int>(blockIdx.x) < g.kv_ctas) {
        const int chunk = blockIdx.x / g.parts, part = blockIdx.x - chunk * g.parts;
        const int first = chunk * g.per_cta, here = min(g.per_cta, a.tokens - first);
        if (tid < 32) {
            const int page_mask = (1 << a.page_shift) - 1;
            auto row_of = [&](int i) { return a.rows ? a.rows[i] : i; };
            auto line_of = [&](int pos, int len) {
                return static_cast<int16_t>(pos >= 0 && pos < len && (a.rot == 0 || pos < a.max_pos) ? pos & page_mask : -1);
            };
            const int i = first + min(lane, here - 1);
            const int row = row_of(i), prow = i > 0 ? row_of(i - 1) : -1;
            const int given = a.positions ? a.positions[i] : 0, before = a.positions && i > 0 ? a.positions[i - 1] : 0;
            const bool row_ok = row >= 0 && row < a.num_rows;
            const int len = row_ok ? a.lens[row] : 0;
            const int pos = a.positions ? given : len - 1;
            const int blk = pos >> a.block_shift;
            int page = -1;
            if (row_ok && pos >= 0 && (pos >> a.page_shift) < a.max_pages) page = a.table[row * a.table_stride + (pos >> a.page_shift)];
            const bool same = i > 0 && row_ok && prow == row && ((a.positions ? before : len - 1) >> a.block_shift) == blk;
            const uint32_t live = here == 32 ? 0xffffffffu : (1u << here) - 1u;
            const uint32_t leaders = __ballot_sync(0xffffffffu, !same) & live;
            // the last run goes on behind the chunk
            int behind = 0;
            if (leaders) {
                const int last = 31 - __clz(leaders);
                const int lrow = __shfl_sync(0xffffffffu, row, last), lblk = __shfl_sync(0xffffffffu, blk, last), llen = __shfl_sync(0xffffffffu, len, last);
                const bool lok = __shfl_sync(0xffffffffu, static_cast<int>(row_ok), last) != 0;
                for (int from = first + here; lok; from += 32) {
                    const int k = from + lane;
                    bool on = k < a.tokens && row_of(k) == lrow;
                    if (on) {
                        const int p = append8_pos(a, k, llen);
                        on = (p >> a.block_shift) == lblk;
                        // (more than a block's tokens only where places are named again: those are left out)
                        if (on && k - first >= kAppend8Lines) atomicCAS(a.err_word, 0, kDeviceErrIndex);
                        else if (on) lines[k - first] = line_of(p, llen);
                    }
                    const uint32_t off = ~__ballot_sync(0xffffffffu, on);
                    behind += off ? __ffs(off) - 1 : 32;
                    if (off || behind >= kAppend8Lines - here) break;
                }
                behind = min(behind, kAppend8Lines - here);
            }
            bool bad = page < 0 || page >= a.num_pages || line_of(pos, len) < 0;
            if (page < 0 || page >= a.num_pages) page = -1;
            if (a.refs && page >= 0 && a.refs[page] > 1) page = -1, bad = true;  // others hold it too
            if (part == 0 && lane < here && bad) atomicCAS(a.err_word, 0, kDeviceErrIndex);
            if (lane < here) lines[lane] = line_of(pos, len);
            if (lane < here && ((leaders >> lane) & 1u)) {
                const uint32_t later = lane == 31 ? 0u : leaders >> (lane + 1);
                const int at = __popc(leaders & ((1u << lane) - 1u));
                Append8Run r;
                r.first = i;
                r.n = later ? __ffs(later) : here - lane + behind;
                r.page = page;
                r.block = (pos & page_mask) >> a.block_shift;
                runs[at] = r;
                first_pos[at] = pos & ~page_mask;
            }
            if (lane == 0) num_runs = __popc(leaders);
        }
        __syncthreads();
        const int units_per_run = a.kv_heads * (a.v.codes ? 2 : 1);
        constexpr int kGroups = kAppend8Threads / G;  // of the CTA
        const Append8Unit<G> unit{a, g, tid % G, G >= 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u) << (lane / G * G)};
#pragma unroll 1
        for (int u = part * kGroups + tid / G; u < num_runs * units_per_run; u += g.parts * kGroups) {
            const int r = g.by_units(u), x = u - r * units_per_run;
            const int side = g.by_kv_heads(x);
            const Append8Run run = runs[r];
            if (run.page >= 0) unit(run, lines + (run.first - first), first_pos[r], side == 0, x - side * a.kv_heads, red, redi);
        }
    } else {
        const int cta = blockIdx.x - g.kv_ctas;
        const int chunk = cta / g.q_parts, part = cta - chunk * g.q_parts;
        const int first = chunk * g.q_per_cta, here = min(g.q_per_cta, a.tokens - first);
        if (tid < here) {
            const int i = first + tid;
            const int row = a.rows ? a.rows[i] : i;
            const int len = a.positions || row < 0 || row >= a.num_rows ? 0 : a.lens[row];
            const int pos = append8_pos(a, i, len);
            const bool ok = pos >= 0 && pos < a.max_pos;
            if (!ok && part == 0) atomicCAS(a.err_word, 0, kDeviceErrIndex);
            angles[tid] = ok ? a.cos_sin + static_cast<int64_t>(pos) * a.rot : nullptr;
        }
        __syncthreads();
        const int half = a.rot / 2, per_token = a.heads * g.row;
        const int step = g.q_parts * kAppend8Threads;
#pragma unroll 1
        for (int e0 = part * kAppend8Threads + tid; e0 < per_token * here; e0 += kAppend8Ahead * step) {
            uint4 v[kAppend8Ahead], w[kAppend8Ahead];
            __nv_bfloat16 *to[kAppend8Ahead];
            const float *cs[kAppend8Ahead];
#pragma unroll
            for (int u = 0; u < kAppend8Ahead; ++u) {
                const int e = e0 + u * step;
                to[u] = nullptr;
                cs[u] = nullptr;
                if (e >= per_token * here) continue;
                const int tok = g.by_q(e), x = e - tok * per_token, i = first + tok;
                if (!angles[tok]) continue;
                const int h = g.by_row(x), t = x - h * g.row;
                const __nv_bfloat16 *from = static_cast<const __nv_bfloat16 *>(a.q) + i * a.q_row + h * a.q_head + t * 8;
                to[u] = static_cast<__nv_bfloat16 *>(a.q_out) + i * a.qo_row + h * a.qo_head + t * 8;
                v[u] = *reinterpret_cast<const uint4 *>(from);
                if (t >= g.plain) {
                    cs[u] = angles[tok] + (t - g.plain) * (a.interleaved ? 4 : 8);
                    if (!a.interleaved) w[u] = *reinterpret_cast<const uint4 *>(from + half);
                }
            }
#pragma unroll
            for (int u = 0; u < kAppend8Ahead; ++u) {
                if (!to[u]) continue;
                if (cs[u]) {
                    const float4 c0 = *reinterpret_cast<const float4 *>(cs[u]), s0 = *reinterpret_cast<const float4 *>(cs[u] + half);
                    if (a.interleaved) {
                        v[u] = turn_pairs(v[u], c0, s0);
                    } else {
                        const float4 c1 = *reinterpret_cast<const float4 *>(cs[u] + 4), s1 = *reinterpret_cast<const float4 *>(cs[u] + half + 4);
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
    }
    cta_release_and_trigger();
}

template <int G>
cudaError_t launch_append_q8_group(const AppendQ8Args &a, int sms, int pdl, cudaStream_t stream) {
    const int fit = sms * 4;
    const int units = a.kv_heads * (a.v.codes ? 2 : 1), groups = kAppend8Threads / G;
    const int plain = (a.k.dim - a.rot) / 8, row = plain + a.rot / (a.interleaved ? 8 : 16);
    const int krow = a.k.dim / 8, vrow = a.v.codes ? a.v.dim / 8 : 1;
    const int per_q = a.q ? a.heads * row : 1;
    Append8Shape g{0,    1,    1,    1, 1, plain, row, krow, vrow, FastDiv(row), FastDiv(krow), FastDiv(vrow), FastDiv(units), FastDiv(per_q),
                   FastDiv(a.kv_heads)};
    // few tokens: a CTA for each and for as many of its units as it has groups; many: chunks of 32 tokens, whose runs
    // are at least their share of a block
    const int64_t alone = static_cast<int64_t>(a.tokens) * ((units + groups - 1) / groups);
    if (alone <= fit) {
        g.per_cta = 1;
        g.parts = (units + groups - 1) / groups;
    } else {
        g.per_cta = kAppend8Tokens;
        const int chunks = (a.tokens + g.per_cta - 1) / g.per_cta;
        const int block = 1 << a.block_shift;
        const int64_t work = static_cast<int64_t>(units) * (block >= g.per_cta ? 1 : g.per_cta / block);
        int64_t parts = (work + groups - 1) / groups;
        const int64_t most = fit / chunks > 1 ? fit / chunks : 1;
        if (parts > most) parts = most;
        g.parts = static_cast<int>(parts);
    }
    g.kv_ctas = (a.tokens + g.per_cta - 1) / g.per_cta * g.parts;
    int q_ctas = 0;
    if (a.q) {
        int y = (per_q + kAppend8Threads - 1) / kAppend8Threads;
        if (static_cast<int64_t>(a.tokens) * y > fit) y = fit / a.tokens > 1 ? fit / a.tokens : 1;
        if (a.tokens > fit) g.q_per_cta = (a.tokens + fit - 1) / fit;
        if (g.q_per_cta > 8) g.q_per_cta = 8;
        g.q_parts = y;
        q_ctas = (a.tokens + g.q_per_cta - 1) / g.q_per_cta * y;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(g.kv_ctas + q_ctas), 1, 1);
    cfg.blockDim = dim3(kAppend8Threads, 1, 1);
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
    return cudaLaunchKernelEx(&cfg, hsp_append_q8_kernel<G>, a, g);
}

cudaError_t launch_append_q8(const AppendQ8Args &a, int sms, int pdl, cudaStream_t stream) {
    // pieces of a unit at most
    const int64_t block = 1 << a.block_shift;
    const int64_t dim = a.v.codes && a.v.dim > a.k.dim ? a.v.dim : a.k.dim;
    const int64_t pieces = (block < a.tokens ? block : a.tokens) * dim / 8;
    if (pieces <= 8 * kAppend8Items) return launch_append_q8_group<8>(a, sms, pdl, stream);
    if (pieces <= 32 * kAppend8Items) return launch_append_q8_group<32>(a, sms, pdl, stream);
    return launch_append_q8_group<256>(a, sms, pdl, stream);
}

}  // namespace hsp
