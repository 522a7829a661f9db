// kernels_append_q8.cu -- new tokens into the pages of a cache held in 8 bits: the rotary turn of keys and
// queries, a scale for each block of tokens and head, and the codes.
//
// For the new tokens of one block and head, x their key (turned) or value rows:
//   s = the smallest power of two with amax |x| <= 448 s; not below the block's old scale where tokens
//       stand in front of them;  code = round(x / s);
//   where s grew, the codes in front are rounded to it (a shift of their exponents, exact unless the result
//   is below the smallest normal code).
// Under a scale that is another writer's and no power of two the quotients are made in 64 bits, element by element.
// A turned value is rounded once, from the exact sum of its two products, so a code does not depend on the order of
// operations: the sum is made in fp32, and again exactly (dot2_odd) where its error could carry it over the border between
// two codes or two scales.
//
// A CTA looks at `per_cta` tokens of the call, finds the runs of neighbouring tokens that share a row and block (a run
// belongs to the CTA that holds its first token), and takes (run, side, head) units, each by 8, 32, 128 or 256 lanes, by
// the longest of its runs: a lane has two 16-byte pieces, requested at once, and keeps their numbers from the search for
// the largest to the codes (of larger units it reads them twice; where units are few, a cluster of CTAs shares one).  Further
// CTAs of the launch turn the queries.
//
// Bytes: two read and one written per number of the cache, two and two per query's.  What bounds it is latency (row,
// position, length and page before the first new row, a scale between the two looks at the numbers), so what counts are short
// code and many lanes: with a warp for 256 pieces, eight each, 2047 tokens of 8 heads of 128 columns took 29 us.  One GB300,
// us: 8 latent tokens with 16 query heads 4.1; 2047 tokens of 8 kv and 32 query heads of 128 columns 19.9 (14.3 without
// queries, 7.1 at the copy rate); 1501 latent tokens with 16 query heads 19.0 (11.3; 8.7): most of the queries' CTAs start where the
// cache's, which fill the GPU, end.  With the queries in a second launch beside this one 5.1, 21.4 and 21.7.
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
constexpr int kAppend8Chunk = 16;    // tokens of a CTA where they are many and have few heads
constexpr int kAppend8Items = 2;     // pieces that a lane works on at once

struct Append8Shape {
    int per_cta, parts;              // tokens and CTAs of a chunk
    int plain;                       // copied pieces of a key row
    int krow, vrow;                  // pieces of a key and a value row
    int subs;                        // CTAs that share a unit (a cluster), 1: none
    FastDiv by_krow, by_vrow, by_units, by_kv_heads;
    // CTAs from cache_ctas on turn queries: q_slices of them q_per_cta tokens
    int cache_ctas, q_per_cta, q_slices;
    int q_row, q_total;              // pieces (pairs of pieces where the turn's pairs lie apart) of a head and of a token
    FastDiv by_q_row, by_q_total;
};

struct Append8Run {
    int first, n;                    // its tokens
    int page;                        // -1: nowhere to write
    int block;                       // of the page
};

__device__ __forceinline__ int append8_pos(const AppendQ8Args &a, int i, int len) { return a.positions ? a.positions[i] : len - 1; }

// (a c + b d) / s rounded to odd (NaN where the sum is beyond 448 * 2^60): in 64 bits the products (of 32 bits) are exact, the sum is
// made odd, so that it lies on the exact sum's side of s times any number of few bits, and the quotient by its remainder's sign.
static __device__ __noinline__ float quotient_odd(float a, float c, float b, float d, float s) {
    const double p = static_cast<double>(a) * c, q = static_cast<double>(b) * d, t = s;
    auto odd64 = [](double h, double rest) {  // h, moved towards the rest unless its last bit is set
        long long u = __double_as_longlong(h);
        if (rest != 0. && (u & 1) == 0 && h != 0.) u += (rest > 0.) == (h > 0.) ? 1 : -1;
        return __longlong_as_double(u);
    };
    const double sum = __dadd_rn(p, q), bb = __dsub_rn(sum, p);
    const double h = odd64(sum, __dadd_rn(__dsub_rn(p, __dsub_rn(sum, bb)), __dsub_rn(q, bb)));
    if (!(fabs(h) <= static_cast<double>(kQ8Top * 0x1p60f))) return __uint_as_float(0x7fc00000u);
    const double r = __ddiv_rn(h, t), y = odd64(r, __fma_rn(-r, t, h));
    const float f = __double2float_rz(y);
    return __uint_as_float(__float_as_uint(f) | (static_cast<double>(f) != y ? 1u : 0u));
}

// The codes of pieces e, e + step, ... below `items` of a run under a scale that is no power of two: what another writer left in a
// block whose new tokens ask for no more.  Columns from `turned` on are turned.
static __device__ __noinline__ void append8_divided(const AppendQ8Args &a, const __nv_bfloat16 *rows, int64_t stride, int per, int turned, const int16_t *lines,
                                             int pos0, uint8_t *codes, int64_t token, float scale, int e, int step, int items) {
    const int half = a.rot / 2;
#pragma unroll 1
    for (; e < items; e += step) {
        const int j = e / per, line = lines[j];
        if (line < 0) continue;
        const __nv_bfloat16 *row = rows + j * stride;
#pragma unroll 1
        for (int x = (e - j * per) * 8, end = x + 8; x < end; ++x) {
            float c = 1.f, s = 0.f, w = 0.f;
            if (x >= turned) {
                const int y = x - turned, pair = a.interleaved ? y >> 1 : y < half ? y : y - half;
                const bool second = a.interleaved ? (y & 1) != 0 : y >= half;
                const int away = a.interleaved ? 1 : half;
                const float *cs = a.cos_sin + static_cast<int64_t>(pos0 + line) * a.rot;
                c = cs[pair];
                s = cs[half + pair];
                w = second ? __bfloat162float(row[x - away]) : -__bfloat162float(row[x + away]);
            }
            const float y = quotient_odd(__bfloat162float(row[x]), c, w, s, scale);
            codes[line * token + x] = static_cast<uint8_t>(float2_to_e4m3x2(y, 0.f) & 0xffu);
        }
    }
}

// A group of G lanes (8, 32, 128 or the CTA's 256) makes one unit's scale and codes.
template <int G>
struct Append8Unit {
    const AppendQ8Args &a;
    const Append8Shape &g;
    int t;          // this thread's place in the group
    uint32_t mask;  // lanes of the group

    // The eight numbers of piece x of a token's row, turned where they are keys of a turned column, and the largest of them.
    // Turned fast (one rounding of one product, one of the sum: off by at most 2^-23 of |product| + |sum|, and `size` is not
    // below any of these) or exactly (size 0).
    __device__ __forceinline__ void numbers(bool is_k, const uint4 *row, int x, int pos, bool exact, float2 (&v)[4], float &most, float &size) const {
        const uint4 raw = row[x];
        v[0] = make_float2(bf_lo(raw.x), bf_hi(raw.x)), v[1] = make_float2(bf_lo(raw.y), bf_hi(raw.y));
        v[2] = make_float2(bf_lo(raw.z), bf_hi(raw.z)), v[3] = make_float2(bf_lo(raw.w), bf_hi(raw.w));
        size = 0.f;
        if (is_k && x >= g.plain) {
            const int half = a.rot / 2, y = (x - g.plain) * 8;
            const float *cs = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
            // partners w (with the sign that they have in the sum), cosines c and sines s of the eight
            float2 w[4], c[4], s[4];
            if (a.interleaved) {
                const float4 cc = *reinterpret_cast<const float4 *>(cs + y / 2), ss = *reinterpret_cast<const float4 *>(cs + half + y / 2);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = make_float2(-v[e].y, v[e].x);
                c[0] = make_float2(cc.x, cc.x), c[1] = make_float2(cc.y, cc.y), c[2] = make_float2(cc.z, cc.z), c[3] = make_float2(cc.w, cc.w);
                s[0] = make_float2(ss.x, ss.x), s[1] = make_float2(ss.y, ss.y), s[2] = make_float2(ss.z, ss.z), s[3] = make_float2(ss.w, ss.w);
            } else {
                // the piece's columns are all of the first or all of the second half, their partners half a turn away
                const bool second = y >= half;
                const uint32_t flip = second ? 0u : 0x80000000u;
                const float *from = cs + (second ? y - half : y);
                const uint4 o = row[x + (second ? -half : half) / 8];
                auto lo = [&](uint32_t f) { return __uint_as_float((f << 16) ^ flip); };
                auto hi = [&](uint32_t f) { return __uint_as_float((f & 0xffff0000u) ^ flip); };
                w[0] = make_float2(lo(o.x), hi(o.x)), w[1] = make_float2(lo(o.y), hi(o.y));
                w[2] = make_float2(lo(o.z), hi(o.z)), w[3] = make_float2(lo(o.w), hi(o.w));
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float4 cc = *reinterpret_cast<const float4 *>(from + 2 * e), ss = *reinterpret_cast<const float4 *>(from + half + 2 * e);
                    c[e] = make_float2(cc.x, cc.y), c[e + 1] = make_float2(cc.z, cc.w);
                    s[e] = make_float2(ss.x, ss.y), s[e + 1] = make_float2(ss.z, ss.w);
                }
            }
            if (exact) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = dot2_odd(v[e], c[e], w[e], s[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 p = mul2(w[e], s[e]);
                    v[e] = fma2(v[e], c[e], p);
                    size = fmaxf(size, fmaxf(fabsf(p.x), fabsf(p.y)));
                }
            }
        }
        auto largest = [&]() {
            most = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) most = fmaxf(most, fmaxf(fabsf(v[e].x), fabsf(v[e].y)));
        };
        largest();
        if (most > kQ8Top * 0x1p60f * (1.f - 0x1p-20f)) {  // out of range: NaN, and none that counts (a fast sum may lie on either side)
            if (size > 0.f) size = INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (fabsf(v[e].x) > kQ8Top * 0x1p60f) v[e].x = __uint_as_float(0x7fc00000u);
                if (fabsf(v[e].y) > kQ8Top * 0x1p60f) v[e].y = __uint_as_float(0x7fc00000u);
            }
            largest();
        }
        if (size > 0.f) size += most;
    }

    // The group meets (G > 32: at a barrier of its own).
    __device__ __forceinline__ void meet() const {
        if (G == 256) __syncthreads();
        else if (G == 128) asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + static_cast<int>(threadIdx.x >> 7)) : "memory");
        else __syncwarp(mask);
    }

    // The largest of lo and hi and the smallest of line over the group (and the cluster that shares the unit).
    __device__ __forceinline__ void reduce(float &lo, float &hi, int &line, float (*red)[2], int *redi, float (*shared)[3], int &turn) const {
#pragma unroll
        for (int d = (G < 32 ? G : 32) / 2; d > 0; d >>= 1) {
            lo = fmaxf(lo, __shfl_xor_sync(mask, lo, d));
            hi = fmaxf(hi, __shfl_xor_sync(mask, hi, d));
            line = min(line, __shfl_xor_sync(mask, line, d));
        }
        if (G > 32) {
            meet();  // what the last unit left there has been read
            if ((t & 31) == 0) {
                red[t >> 5][0] = lo;
                red[t >> 5][1] = hi;
                redi[t >> 5] = line;
            }
            meet();
#pragma unroll
            for (int w = 0; w < G / 32; ++w) {
                lo = fmaxf(lo, red[w][0]);
                hi = fmaxf(hi, red[w][1]);
                line = min(line, redi[w]);
            }
        }
        if (G == 256 && g.subs > 1) {  // and over the cluster
            float *mine = shared[turn];
            if (t == 0) {
                mine[0] = lo;
                mine[1] = hi;
                mine[2] = __int_as_float(line);
            }
            cluster_sync_all();
#pragma unroll 1
            for (int c = 0; c < g.subs; ++c) {
                const uint32_t at = cluster_map_shared(smem_u32(mine), static_cast<uint32_t>(c));
                lo = fmaxf(lo, ld_shared_cluster_f32(at));
                hi = fmaxf(hi, ld_shared_cluster_f32(at + 4));
                line = min(line, __float_as_int(ld_shared_cluster_f32(at + 8)));
            }
            turn ^= 1;  // (a CTA that is ahead writes the other one)
        }
    }

    // lines: of the run's tokens in their page, -1: written nowhere; pos0: the first position of that page; sub: which CTA of
    // the cluster that shares the unit this is.
    __device__ __forceinline__ void operator()(const Append8Run &r, const int16_t *lines, int pos0, bool is_k, int head, int sub, float (*red)[2], int *redi,
                                               float (*shared)[3], int &turn) const {
        const Q8Side &s = is_k ? a.k : a.v;
        const int per = is_k ? g.krow : g.vrow;
        const FastDiv &by = is_k ? g.by_krow : g.by_vrow;
        const int block = 1 << a.block_shift, items = r.n * per;
        float *const scale = s.scales + r.page * s.s_page + r.block * s.s_block + head * s.s_head;
        uint8_t *const codes = s.codes + r.page * s.page + head * s.head;
        const int64_t stride = is_k ? a.k_row : a.v_row;
        const __nv_bfloat16 *const rows = static_cast<const __nv_bfloat16 *>(is_k ? a.k_new : a.v_new) + r.first * stride + static_cast<int64_t>(head) * s.dim;
        const float old = *scale;
        constexpr int kBatch = kAppend8Items * G;
        const int all = kBatch * (G == 256 ? g.subs : 1);
        float2 v[kAppend8Items][4];
        float most[kAppend8Items], size[kAppend8Items];
        int where[kAppend8Items], column[kAppend8Items];  // line (-1: none) and first column of the pieces
        // The largest number lies between lo and hi (fast sums); they ask for the same scale unless it lies at the border of
        // two, and then it is sought again, exactly.
        enum { kLargest, kLargestExact, kCodes } phase = kLargest;
        float lo, hi, inv = 0.f;  // inv: 1 / scale (below zero: minus the scale, which is no power of two)
        int line;  // first new line of the block
#pragma unroll 1
        for (;;) {
            if (inv < 0.f) {
                append8_divided(a, rows, stride, per, is_k ? g.plain * 8 : s.dim, lines, pos0, codes, s.token, -inv, t + sub * G,
                                G * (G == 256 ? g.subs : 1), items);
                return;
            }
            lo = hi = 0.f;
            line = block;
#pragma unroll 1
            for (int e0 = t + sub * kBatch; e0 < items; e0 += all) {
                bool exact = phase == kLargestExact;
                bool load = phase != kCodes || items > all;
#pragma unroll 1
                for (;;) {
                    if (load) {
#pragma unroll
                        for (int k = 0; k < kAppend8Items; ++k) {
                            const int e = e0 + k * G;
                            where[k] = -1;
                            if (e >= items) continue;
                            const int j = by(e), x = e - j * per;
                            where[k] = lines[j];
                            column[k] = x * 8;
                            numbers(is_k, reinterpret_cast<const uint4 *>(rows + j * stride), x, pos0 + max(where[k], 0), exact, v[k], most[k], size[k]);
                        }
                    }
                    if (phase != kCodes) break;
                    // where both ends of a fast sum's range have the same code, that is its code; else once more, exactly
                    bool near = false;
#pragma unroll
                    for (int k = 0; k < kAppend8Items; ++k) {
                        if (where[k] < 0) continue;
                        uint2 c;
                        const float2 i2 = make_float2(inv, inv);
                        auto codes4 = [&](float slack, int f) {
                            const float2 d = make_float2(slack, slack);
                            const float2 y = sum2(mul2(v[k][f], i2), d), z = sum2(mul2(v[k][f + 1], i2), d);
                            return __byte_perm(float2_to_e4m3x2(y.x, y.y), float2_to_e4m3x2(z.x, z.y), 0x5410);
                        };
                        const float slack = exact ? 0.f : size[k] * inv * 0x1p-22f;
                        c.x = codes4(slack, 0);
                        c.y = codes4(slack, 2);
                        if (slack > 0.f) near |= slack > kQ8Top || c.x != codes4(-slack, 0) || c.y != codes4(-slack, 2);
                        *reinterpret_cast<uint2 *>(codes + static_cast<int64_t>(where[k]) * s.token + column[k]) = c;
                    }
                    if (!near) break;
                    exact = load = true;
                }
                if (phase == kCodes) continue;
#pragma unroll
                for (int k = 0; k < kAppend8Items; ++k) {
                    if (where[k] < 0) continue;
                    line = min(line, where[k] & (block - 1));
                    lo = fmaxf(lo, most[k] - size[k] * 0x1p-22f);
                    hi = fmaxf(hi, most[k] + size[k] * 0x1p-22f);
                }
            }
            if (phase == kCodes) break;
            reduce(lo, hi, line, red, redi, shared, turn);
            if (line == block) return;  // no token of the run is written
            if (phase == kLargest && q8_exponent(lo) != q8_exponent(hi)) {
                phase = kLargestExact;
                continue;
            }
            phase = kCodes;
            float now = two_to(q8_exponent(hi));
            if (line > 0 && old >= now) now = old;  // (also where another CTA of the cluster has written it already)
            inv = (__float_as_uint(now) & 0x7fffffu) == 0 ? 1.f / now : -now;  // (1 / now is exact)
            if (sub != 0) continue;
            if (line > 0 && now > old) {
                // the codes in front, under the new scale
                const float by_new = old * inv;
                const int p16 = s.dim / 16;
#pragma unroll 1
                for (int e = t; e < line * p16; e += G) {
                    const int l = e / p16, x = e - l * p16;
                    uint4 *at = reinterpret_cast<uint4 *>(codes + (static_cast<int64_t>(r.block) * block + l) * s.token + x * 16);
                    uint4 c = *at;
                    uint32_t *w = reinterpret_cast<uint32_t *>(&c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 p = __half22float2(e4m3x2_to_half2(w[k] & 0xffffu)), q = __half22float2(e4m3x2_to_half2(w[k] >> 16));
                        // (to odd: an old scale of another writer's may have more bits than a product with it holds)
                        w[k] = float2_to_e4m3x2(product_odd(p.x, by_new), product_odd(p.y, by_new)) |
                               float2_to_e4m3x2(product_odd(q.x, by_new), product_odd(q.y, by_new)) << 16;
                    }
                    *at = c;
                }
            }
            if (t == 0) *scale = now;  // (the group's lanes have read the old one: they have met since)
        }
    }
};

// The units of a CTA, by groups of G lanes (a cluster's: all of the chunk's, by all of its CTAs together).
template <int G>
__device__ __forceinline__ void append8_units(const AppendQ8Args &a, const Append8Shape &g, const Append8Run *runs, int num_runs, const int16_t *lines,
                                              const int *first_pos, int first, int part, float (*red)[2], int *redi, float (*shared)[3]) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int units_per_run = a.kv_heads * (a.v.codes ? 2 : 1);
    constexpr int kGroups = kAppend8Threads / G;  // of the CTA
    const bool together = G == 256 && g.subs > 1;
    const Append8Unit<G> unit{a, g, tid % G, G >= 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u) << (lane / G * G)};
    int turn = 0;
#pragma unroll 1
    for (int u = together ? 0 : part * kGroups + tid / G; u < num_runs * units_per_run; u += together ? 1 : g.parts * kGroups) {
        const int r = g.by_units(u), x = u - r * units_per_run;
        const int side = g.by_kv_heads(x);
        const Append8Run run = runs[r];
        if (run.page >= 0)
            unit(run, lines + (run.first - first), first_pos[r], side == 0, x - side * a.kv_heads, together ? part : 0, red + tid / G * (G / 32),
                 redi + tid / G * (G / 32), shared, turn);
    }
}

// Queries: copied columns, turned columns.  Pieces are requested before their token's position is known, several by a
// lane at once.  (A token without angles is reported with its keys; its queries stay as they are.)
template <bool INTERLEAVED>
__device__ __forceinline__ void append8_queries(const AppendQ8Args &a, const Append8Shape &g, int cta) {
    constexpr int kMany = INTERLEAVED ? 8 : 4;
    const int group = cta / g.q_slices, slice = cta - group * g.q_slices;
    const int64_t first = static_cast<int64_t>(group) * g.q_per_cta;
    const int here = static_cast<int>(min(static_cast<int64_t>(g.q_per_cta), a.tokens - first));  // (0 or less: none)
    const int all = here * g.q_total, step = g.q_slices * kAppend8Threads, half = a.rot / 2;
    const __nv_bfloat16 *const q = static_cast<const __nv_bfloat16 *>(a.q) + first * a.q_row;
    __nv_bfloat16 *const out = static_cast<__nv_bfloat16 *>(a.q_out) + first * a.qo_row;
#pragma unroll 1
    for (int e0 = slice * kAppend8Threads + threadIdx.x; e0 < all; e0 += kMany * step) {
        uint4 v[kMany], w[INTERLEAVED ? 1 : kMany];
        int pos[kMany];
#pragma unroll
        for (int u = 0; u < kMany; ++u) {
            const int e = e0 + u * step;
            pos[u] = -1;
            if (e >= all) continue;
            const int tok = g.by_q_total(e), x = e - tok * g.q_total, h = g.by_q_row(x), t = x - h * g.q_row;
            const __nv_bfloat16 *from = q + tok * a.q_row + h * a.q_head + t * 8;
            v[u] = *reinterpret_cast<const uint4 *>(from);
            if (!INTERLEAVED && t >= g.plain) w[INTERLEAVED ? 0 : u] = *reinterpret_cast<const uint4 *>(from + half);
            const int i = static_cast<int>(first) + tok;
            if (a.positions) {
                pos[u] = a.positions[i];
            } else {
                const int row = a.rows ? a.rows[i] : i;
                if (row >= 0 && row < a.num_rows) pos[u] = a.lens[row] - 1;
            }
        }
#pragma unroll
        for (int u = 0; u < kMany; ++u) {
            const int e = e0 + u * step;
            if (e >= all || pos[u] < 0 || pos[u] >= a.max_pos) continue;
            const int tok = g.by_q_total(e), x = e - tok * g.q_total, h = g.by_q_row(x), t = x - h * g.q_row;
            __nv_bfloat16 *to = out + tok * a.qo_row + h * a.qo_head + t * 8;
            if (t >= g.plain) {
                const float *cs = a.cos_sin + static_cast<int64_t>(pos[u]) * a.rot + (t - g.plain) * (INTERLEAVED ? 4 : 8);
                const float4 c0 = *reinterpret_cast<const float4 *>(cs), s0 = *reinterpret_cast<const float4 *>(cs + half);
                if (INTERLEAVED) {
                    v[u] = turn_pairs(v[u], c0, s0);
                } else {
                    const float4 c1 = *reinterpret_cast<const float4 *>(cs + 4), s1 = *reinterpret_cast<const float4 *>(cs + half + 4);
                    turn_halves(v[u].x, w[INTERLEAVED ? 0 : u].x, c0.x, c0.y, s0.x, s0.y);
                    turn_halves(v[u].y, w[INTERLEAVED ? 0 : u].y, c0.z, c0.w, s0.z, s0.w);
                    turn_halves(v[u].z, w[INTERLEAVED ? 0 : u].z, c1.x, c1.y, s1.x, s1.y);
                    turn_halves(v[u].w, w[INTERLEAVED ? 0 : u].w, c1.z, c1.w, s1.z, s1.w);
                    *reinterpret_cast<uint4 *>(to + half) = w[INTERLEAVED ? 0 : u];
                }
            }
            *reinterpret_cast<uint4 *>(to) = v[u];
        }
    }
}

__global__ void __launch_bounds__(kAppend8Threads, 3) hsp_append_q8_kernel(const __grid_constant__ AppendQ8Args a, const __grid_constant__ Append8Shape g) {
    __shared__ Append8Run runs[kAppend8Tokens];
    __shared__ int num_runs, longest, first_pos[kAppend8Tokens];
    __shared__ int16_t lines[kAppend8Lines];
    __shared__ float red[kAppend8Threads / 32][2];
    __shared__ int redi[kAppend8Threads / 32];
    __shared__ float shared[2][3];
    griddep_wait();
    if (static_cast<int>(blockIdx.x) >= g.cache_ctas) {
        if (a.interleaved) append8_queries<true>(a, g, static_cast<int>(blockIdx.x) - g.cache_ctas);
        else append8_queries<false>(a, g, static_cast<int>(blockIdx.x) - g.cache_ctas);
        cta_release_and_trigger();
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31;
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
                bool on = static_cast<uint32_t>(k) < static_cast<uint32_t>(a.tokens) && row_of(k) == lrow;  // (k may have passed 2^31)
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
        if (a.rot > 0 && (pos & ~page_mask) >= a.max_pos) page = -1;  // no token of this page is written: no angle may be read either
        if (a.refs && page >= 0 && a.refs[page] > 1) page = -1, bad = true;  // others hold it too
        if (part == 0 && lane < here && bad) atomicCAS(a.err_word, 0, kDeviceErrIndex);
        if (lane < here) lines[lane] = line_of(pos, len);
        int n = 0;
        if (lane < here && ((leaders >> lane) & 1u)) {
            const uint32_t later = lane == 31 ? 0u : leaders >> (lane + 1);
            const int at = __popc(leaders & ((1u << lane) - 1u));
            Append8Run r;
            r.first = i;
            r.n = n = later ? __ffs(later) : here - lane + behind;
            r.page = page;
            r.block = (pos & page_mask) >> a.block_shift;
            runs[at] = r;
            first_pos[at] = pos & ~page_mask;
        }
        n = __reduce_max_sync(0xffffffffu, n);
        if (lane == 0) {
            num_runs = __popc(leaders);
            longest = n;
        }
    }
    __syncthreads();
    // as many lanes for a unit as have their pieces of its longest run at once
    const int64_t pieces = static_cast<int64_t>(longest) * max(g.krow, g.vrow);
    if (g.subs > 1) append8_units<256>(a, g, runs, num_runs, lines, first_pos, first, part, red, redi, shared);
    else if (pieces <= 8 * kAppend8Items) append8_units<8>(a, g, runs, num_runs, lines, first_pos, first, part, red, redi, shared);
    else if (pieces <= 32 * kAppend8Items) append8_units<32>(a, g, runs, num_runs, lines, first_pos, first, part, red, redi, shared);
    else if (pieces <= 128 * kAppend8Items) append8_units<128>(a, g, runs, num_runs, lines, first_pos, first, part, red, redi, shared);
    else append8_units<256>(a, g, runs, num_runs, lines, first_pos, first, part, red, redi, shared);
    if (g.subs > 1) cluster_sync_all();  // (nobody reads another CTA's memory any more)
    cta_release_and_trigger();
}

cudaError_t launch_append_q8(const AppendQ8Args &a, int sms, int pdl, cudaStream_t stream) {
    const int fit = sms * 3;  // CTAs on the GPU at once
    const int units = a.kv_heads * (a.v.codes ? 2 : 1), block = 1 << a.block_shift;
    const int krow = a.k.dim / 8, vrow = a.v.codes ? a.v.dim / 8 : 1;
    // A few tokens: a CTA for each and, of its units, for four pieces per thread.  Many: chunks of 32 tokens (or 16), and as
    // many CTAs for the chunk's units as fit the GPU; where the units are fewer than those, and larger than a CTA has in hand at
    // once (latent rows in long blocks), a cluster shares a unit.
    const int64_t per_token = static_cast<int64_t>(a.kv_heads) * (krow + (a.v.codes ? vrow : 0));
    int64_t parts = (per_token + 4 * kAppend8Threads - 1) / (4 * kAppend8Threads);
    int per_cta = 1, subs = 1;
    if (parts > units) parts = units;
    if (a.tokens * parts > fit) {
        // (2047 tokens of 8 heads of 128 columns and values, blocks of 16: 25.3 us in chunks of 16, 21.5 of 32; latent rows, one
        // unit to a run: 1501 tokens in blocks of 16 9.9 and 12.6)
        per_cta = units >= 4 || block > kAppend8Chunk ? kAppend8Tokens : kAppend8Chunk;
        const int chunks = static_cast<int>((static_cast<int64_t>(a.tokens) + per_cta - 1) / per_cta);
        parts = fit / chunks > 1 ? fit / chunks : 1;
        const int64_t runs = static_cast<int64_t>(units) * (block < per_cta ? per_cta / block : 1);  // units of a chunk, at least
        const int64_t batches = (static_cast<int64_t>(block) * krow + kAppend8Items * 256 - 1) / (kAppend8Items * 256);
        if (parts > runs) {
            parts = parts / runs < batches ? parts / runs : batches;
            subs = static_cast<int>(parts < 8 ? parts : 8);
            parts = subs > 1 ? subs : runs;
        }
    }
    const int64_t cache_ctas = (static_cast<int64_t>(a.tokens) + per_cta - 1) / per_cta * parts;
    // Queries: a piece per lane where they are few, else twice the CTAs that fit the GPU (2047 tokens with 32 heads of 128 columns: as
    // many as fit 20.9 us, twice 19.9, four times 20.5; 1501 with 16 of 576 21.4, 18.9, 20.0).
    const int plain = (a.k.dim - a.rot) / 8, q_row = plain + a.rot / (a.interleaved ? 8 : 16), q_total = a.q ? a.heads * q_row : 1;
    int64_t q_slices = (q_total + kAppend8Threads - 1) / kAppend8Threads, q_per_cta = 1, q_ctas = 0;
    if (a.q) {
        if (a.tokens * q_slices > 2 * fit) q_slices = 2 * fit / a.tokens > 1 ? 2 * fit / a.tokens : 1;
        if (a.tokens > 2 * fit) q_per_cta = (static_cast<int64_t>(a.tokens) + 2 * fit - 1) / (2 * fit);
        const int64_t most = (int64_t(1) << 30) / q_total;  // (pieces of a CTA are counted in 32 bits)
        if (q_per_cta > most) q_per_cta = most;
        q_ctas = (a.tokens + q_per_cta - 1) / q_per_cta * q_slices;
        q_ctas = (q_ctas + subs - 1) / subs * subs;         // (whole clusters)
    }
    const Append8Shape g{per_cta, static_cast<int>(parts), plain, krow, vrow, subs, FastDiv(krow), FastDiv(vrow), FastDiv(units), FastDiv(a.kv_heads),
                         static_cast<int>(cache_ctas), static_cast<int>(q_per_cta), static_cast<int>(q_slices), q_row, q_total, FastDiv(q_row), FastDiv(q_total)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cache_ctas + q_ctas), 1, 1);
    cfg.blockDim = dim3(kAppend8Threads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    unsigned n = 0;
    if (subs > 1) {
        attrs[n].id = cudaLaunchAttributeClusterDimension;
        attrs[n].val.clusterDim.x = static_cast<unsigned>(subs);
        attrs[n].val.clusterDim.y = 1;
        attrs[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl) {
        attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attrs;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, hsp_append_q8_kernel, a, g);
}

}  // namespace hsp
