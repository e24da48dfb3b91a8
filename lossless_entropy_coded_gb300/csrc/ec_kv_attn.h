/*
 * ec_kv_attn.h -- arguments of the attention kernels, shared by the register form
 * (ec_kv_attn.cu: few rows) and the tensor-memory form (ec_kv_prefill.cu: many rows).
 */
#ifndef EC_KV_ATTN_H_
#define EC_KV_ATTN_H_

#include <float.h>

#include "ec_kv_internal.h"

namespace kv {

struct AttnArgs {
    Pool P;
    Seqs S;
    Rows q, out;
    float* lse;       /* [n_rows, n_q_heads] or NULL */
    float* part;
    int32_t n_q_heads, group;   /* query heads, per key/value head */
    int32_t window, sinks;
    float scale;
    int32_t max_new, max_len;
    int32_t solo;     /* few rows: > 0: one CTA per tile, this many places of work each; 0: even shares */
    int32_t splits, row_tiles;  /* many rows: parts of a row tile's tokens, row tiles per head */
    int* status;
};

/* The least factor of a score, so that no factor is 0 (the smallest denormal: FLT_MIN would raise
 * the scores of queries near 2^-110, whose keys may be as large as 2^100). */
constexpr float kTiny = 1.4e-45f;

/* One query row, and the units of its sequence that are taken in: u0 .. u1 - 1 of sink_u units
 * at the front and those from lo_u on. */
struct RowJob {
    int b, h, head, pos;
    int sink_u, lo_u, u0, u1;
    int64_t row;
};

/* The row by one warp in FP32 on the CUDA cores, for tokens whose scales lie further apart than
 * the FP16 operands of the matrix instructions hold: every product takes its block's own
 * scale, so what a row gives depends on the tokens that it sees alone.  A lane finds in each
 * word what the formats put there: channels 32 b + 8 c + 0..7 of keys g and g + 8, channels
 * 16 i + 8 r + g of values 2c, 2c + 1, 2c + 8, 2c + 9.  Bound by its instructions: 2.2 us per 16
 * tokens and row for each of an SM's 16 warps (one token over 400003, 32 query over 8 key/value
 * heads of 128 channels, 822 us for 83), so only data that needs it comes here.
 *
 * dst: the unnormalised sums of weights 2^(s - m + bias) go there, m and the weights' sum to
 * *dst_m and *dst_l; NULL: the row's output and lse are written. */
template <int NB>
__device__ __forceinline__ void wide_row(const AttnArgs& a, const RowJob& j, float bias, float* dst, float* dst_m, float* dst_l) {
    constexpr int D = 32 * NB;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const float f = a.scale * 1.4426950408889634f;
    float q[NB][8], acc[4 * NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) q[b][i] = load_elem(a.q, j.row * a.q.row + (int64_t)j.head * a.q.head + 32 * b + 8 * c + i);
#pragma unroll
    for (int i = 0; i < 4 * NB; ++i) acc[i] = 0.f;
    float m = -FLT_MAX, l = 0.f;
    auto sees = [&](int t) { return t <= j.pos && (!a.window || j.pos - t < a.window || t < a.sinks); };
#pragma unroll 1
    for (int u = j.u0; u < j.u1; ++u) {
        const int unit = u < j.sink_u ? u : u - j.sink_u + j.lo_u, tok = unit * kUnit;
        int page = a.S.table[(int64_t)j.b * a.S.table_stride + (unit >> (a.P.page_shift - 4))];
        if (page < 0 || page >= a.P.n_pages) page = 0; /* flagged where the unit was first copied */
        const uint8_t* src = page_ptr(a.P, page, j.h, unit & ((1 << (a.P.page_shift - 4)) - 1));
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i4 = 0; i4 < NB / 2; ++i4) {
            const uint4 w = *(const uint4*)(src + i4 * 512 + lane * 16);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) { /* block 2 i4 + k / 2 of key g + 8 (k % 2) */
                const int blk = 2 * i4 + (k >> 1);
                uint32_t h[4];
                e2m1x8_f16(ww[k], h);
                float d = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 x = __half22float2(*(const __half2*)&h[i]);
                    d = fmaf(q[blk][2 * i], x.x, fmaf(q[blk][2 * i + 1], x.y, d));
                }
                s[k & 1] = fmaf(d, scale_value(src[16 * D + (g + 8 * (k & 1)) * NB + blk]), s[k & 1]);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            s[r] += __shfl_xor_sync(kAll, s[r], 1);
            s[r] += __shfl_xor_sync(kAll, s[r], 2);
            s[r] = sees(tok + g + 8 * r) ? __fmul_rn(s[r], f) : -INFINITY;
        }
        float mx = fmaxf(s[0], s[1]);
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, w));
        const float nm = fmaxf(m, mx), al = ex2(m - nm);
        m = nm;
        const float p[2] = {ex2(s[0] - m + bias), ex2(s[1] - m + bias)};
        l = fmaf(l, al, p[0] + p[1]);
        float pt[4]; /* weights of tokens 2c, 2c + 1, 2c + 8, 2c + 9 */
        bool on[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            pt[k] = __shfl_sync(kAll, p[k >> 1], 4 * (2 * c + (k & 1)));
            on[k] = sees(tok + 2 * c + (k & 1) + 8 * (k >> 1));
        }
#pragma unroll
        for (int i4 = 0; i4 < NB / 2; ++i4) {
            const uint4 w = *(const uint4*)(src + 8 * D + i4 * 512 + lane * 16);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = 4 * i4 + k;
                const uint32_t sc = *(const uint32_t*)(src + 16 * D + D / 2 + (c * NB + i / 2) * 4);
                float pv[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) pv[t] = on[t] ? pt[t] * scale_value((sc >> (8 * t)) & 0xFFu) : 0.f;
                uint32_t h[4]; /* byte r + 2 p: channel 16 i + 8 r + g of tokens 2c + 8p, 2c + 8p + 1 */
                e2m1x8_f16(ww[k], h);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 x = __half22float2(*(const __half2*)&h[r]), y = __half22float2(*(const __half2*)&h[r + 2]);
                    float& o = acc[2 * i + r];
                    o = fmaf(o, al, fmaf(x.x, pv[0], fmaf(x.y, pv[1], fmaf(y.x, pv[2], y.y * pv[3]))));
                }
            }
        }
    }
#pragma unroll
    for (int w = 4; w < 32; w <<= 1) l += __shfl_xor_sync(kAll, l, w);
    const float inv = dst ? 1.f : l == 0.f ? 0.f : 1.f / l;
    const int64_t off = j.row * a.out.row + (int64_t)j.head * a.out.head;
#pragma unroll
    for (int i = 0; i < 4 * NB; ++i) {
        acc[i] += __shfl_xor_sync(kAll, acc[i], 1);
        acc[i] += __shfl_xor_sync(kAll, acc[i], 2);
        if ((i & 3) != c) continue;
        const int d = 16 * (i >> 1) + 8 * (i & 1) + g;
        if (dst) dst[d] = acc[i];
        else store_elem(a.out, off + d, acc[i] * inv);
    }
    if (lane) return;
    if (dst) *dst_m = m, *dst_l = l;
    else if (a.lse) a.lse[j.row * a.n_q_heads + j.head] = l == 0.f ? -INFINITY : (m - bias + log2f(l)) * 0.6931471805599453f;
}

struct PrefillPlan {
    int row_tiles, splits;
    int64_t grid;
    size_t work, most; /* bytes of this call's parts, and of any call's of at most these sizes */
};
bool plan_prefill(const ec_kv* C, int sms, int n_seqs, int max_new, int64_t max_units, int group, int dtype, PrefillPlan* p);
int launch_prefill(const AttnArgs& a, const PrefillPlan& p, cudaStream_t stream);

}  // namespace kv

#endif
