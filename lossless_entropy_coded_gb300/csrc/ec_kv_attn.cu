/*
 * ec_kv_attn.cu -- attention of new tokens over the 4-bit cache (ec_kv_attend).
 *
 * For a query row q, head by head: s_t = scale q . k_t over the visible tokens, p = exp
 * (s - m), o = sum p v / sum p.  All rows of a key/value head's query group, times a few
 * new tokens, form the columns of the products S^T = K Q^T and O^T = V^T P^T, 8 to a tile,
 * so each 4-bit key or value is expanded once for 8 rows (and read from HBM once; further
 * tiles of a head find it in L2).  16 columns per tile need 168 registers and leave 12
 * warps per SM for 16: 16 rows over 400000 tokens 154 us for 160, but 63 for 51 with 1 to 5
 * new tokens of 16 sequences and 72 for 54 over 100000 tokens, so there is one width.
 *
 * Bounds.  The floor is HBM: 4.25 bits per element of every visible key and value.  An SM
 * gets 45 bytes/ns of it, a unit (16 tokens, 2176 bytes at 128 channels) every 94 clocks;
 * the four schedulers then have 375 issue slots for it.  A unit takes about 270
 * instructions, 140 of them on the integer pipe, which issues every second clock (the
 * expansion of E2M1 to FP16 alone is 64), so the integer pipe and the dependent chain of
 * a warp bound the kernel, not HBM.  Measured, 128 channels, 32 query over 8 key/value
 * heads: 400003 tokens 82.6 us (5.27 TB/s, 0.79 of the measured copy rate; 113 us with
 * one unit per step and all segment state in registers); 64 sequences of 1 to 8192 tokens
 * 36.2 us for 92 MB (245 us with one CTA per tile and fixed chunks: most tiles are short,
 * and their fixed cost, about that of 10 units, has to be shared out too).
 * mma.sync, whose operands a warp expands in its own registers; the pipe is 28 % busy at the
 * rate above.  tcgen05 with the tokens as its 128 rows and the query rows as columns would
 * expand a tile once for all of a head's rows, in shared memory; it has not been tried.
 */
#include "ec_kv_attn.h"

namespace kv {

constexpr int64_t kMaxLen = 0x7FFFFFF0; /* tokens of a sequence: lens are 32-bit, and a unit past them too */
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

/* Work is counted in units of 16 tokens of one tile (the rows of one key/value head's
 * group, 8 at a time), plus kTileCost for a tile's queries and outputs.  Measured (us, cost 6 /
 * 10 / 14 / 20), 32 query over 8 key/value heads of 128 channels: 64 sequences of 1 to 8192
 * tokens 30.7 / 27.1 / 28.8 / 28.4, with FP32 queries 42.3 / 35.9 / 37.3 / 36.8; 200 of 16 to 2000
 * 43.0 / 39.4 / 41.8 / 44.9; 1000 of 1 to 300 62.9 / 62.5 / 63.1 / 66.9; 64 over 8: 16 of 500 to 30000
 * 37.9 / 35.6 / 35.5 / 34.6; 16 over 16 of 64 channels, 100 of 64 to 4000 37.6 / 35.4 / 36.0 / 38.3. */
constexpr int kTileCost = 10;

/* The keys that a sequence's new rows see, in units: the sinks' units, then lo_u ..
 * ceil(len / 16) - 1. */
struct Span {
    int sink_u, lo_u, units;   /* units >= 1 (one empty step where there is no token) */
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int len, int m) {
    Span s;
    const int all = (len + kUnit - 1) / kUnit;
    const int64_t lo = a.window ? (int64_t)(len - m) - a.window + 1 : 0; /* first token of row 0's window */
    s.lo_u = lo > 0 ? (int)min(lo / kUnit, (int64_t)all) : 0;
    s.sink_u = min((a.sinks + kUnit - 1) / kUnit, s.lo_u);
    s.units = max(1, s.sink_u + all - s.lo_u);
    return s;
}
__device__ __forceinline__ int tile_cost(const AttnArgs& a, int units) { return a.solo ? a.solo : units + kTileCost; }

/* Per sequence, in shared memory: pre[b], the work in front of it (pre[n_seqs]: all work),
 * and {len, new tokens, first row}.  Every thread of the CTA takes part. */
__device__ __forceinline__ void scan_seqs(const AttnArgs& a, int rows_per_tile, int64_t* pre, int3* info, bool flag) {
    __shared__ int64_t warp_work[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    int64_t at = 0;
    for (int base = 0; base < a.S.n_seqs; base += 32 * W) {
        const int b = base + threadIdx.x;
        int64_t n = 0;
        if (b < a.S.n_seqs) {
            Seq q = seq_of(a.S, a.P.page_shift, b);
            if (q.len > a.max_len) {
                q.len = a.max_len;
                q.bad = true;
            }
            if (q.m > a.max_new) {
                q.m = a.max_new;
                q.bad = true;
            }
            if (flag && q.bad) flag_corrupt(a.status);
            const int units = span_of(a, q.len, q.m).units;
            info[b] = make_int3(q.len, q.m, (int)q.row0);
            n = (int64_t)((q.m * a.group + rows_per_tile - 1) / rows_per_tile) * a.P.n_heads * tile_cost(a, units);
        }
        int64_t x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(kAll, x, o);
            if (lane >= o) x += y;
        }
        if (base) __syncthreads(); /* the sums of the sequences before have been read */
        if (lane == 31) warp_work[warp] = x;
        __syncthreads();
        int64_t front = at;
        for (int w = 0; w < W; ++w) {
            const int64_t y = warp_work[w];
            if (w < warp) front += y;
            at += y;
        }
        if (b < a.S.n_seqs) pre[b] = front + x - n;
    }
    if (threadIdx.x == 0) pre[a.S.n_seqs] = at;
    __syncthreads();
}

/* Where a place of work lies: sequence, head, first row of the tile, units u0 .. u1 - 1 up
 * to the place `end`, and the place of the tile's first unit (its name). */
struct Seg {
    int b, h, r0, u0, u1, units;
    int64_t tile, next;
};
__device__ __forceinline__ Seg seg_at(const AttnArgs& a, const int64_t* pre, const int3* info, int rows_per_tile, int64_t x, int64_t end) {
    int lo = 0, hi = a.S.n_seqs - 1; /* the last sequence whose work begins at x or before (those without any come before it) */
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (pre[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    Seg s;
    s.b = lo;
    s.units = span_of(a, info[lo].x, info[lo].y).units;
    const uint32_t per = (uint32_t)tile_cost(a, s.units), local = (uint32_t)(x - pre[lo]), tile = local / per, off = local - tile * per;
    s.tile = x - off;
    s.next = min(s.tile + per, end);
    s.u0 = min((int)off, s.units);
    s.u1 = (int)min((int64_t)s.units, s.next - s.tile);
    s.h = (int)(tile % (uint32_t)a.P.n_heads);
    s.r0 = (int)(tile / (uint32_t)a.P.n_heads) * rows_per_tile;
    return s;
}

/* The tile that begins in a share and ends in a later one. */
struct JoinJob {
    int parts, h, r0, R, row0, pad[3];
};

/* The share of CTA i of n: places i * share .. . */
__device__ __forceinline__ int64_t share_of(const AttnArgs& a, int64_t X, int n, int warps) {
    if (a.solo) return a.solo;
    const int64_t s = (X + n - 1) / n;
    return max((s + warps - 1) / warps, (int64_t)4) * warps;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

/* Bits of the probabilities: p is held as 2^kBias p in FP16, the running reference of a
 * row moves only when weights pass 2^(kBias + 3), and value scales lie up to 2^7 above their
 * block's reference: 2^(5 + 3 + 7) < 65504.  They lie down to 2^-8 below it, where a weight is
 * good to 2^-22 of the row's largest; what a step of two units holds outside moves the
 * reference, up or down. */
constexpr float kBias = 5.f;
constexpr int kRefUp = 7, kRefDown = 8;
/* A step whose scales span more than the two, or a reference that is more than kRefSpan from its
 * segment's first, sends the rest of the warp's work to redo_wide: the accumulators' FP32 range is far from
 * its ends, and tokens that weigh little cannot drown those that count. */
constexpr int kRefSpan = 16;

/* Warps per SM and stages of a warp's ring by the tile's registers; `keep` floats hold a
 * warp's partial result of a tile: [rows][LD], maxima, sums.  All warps of an SM form one
 * CTA: of two CTAs the SM favours one, whose warps are done at 66 us of 81 with 400000
 * tokens, and the other's go on alone.  Where a tile has a CTA of its own (solo) it has half
 * the warps. */
template <int NB>
struct Shape {
    static constexpr int D = 32 * NB, RB = 8, LD = D + 4, UB = 17 * D;
    static constexpr int W = NB <= 4 ? 16 : 8;
    static constexpr int S = NB == 2 ? 4 : 2; /* of two units each; a power of two */
    static constexpr int KEEP = RB * LD + 2 * RB;
    static constexpr int RING = S * 2 * UB, WARP_BYTES = RING + KEEP * 4 + 64; /* + the warp's segment */
    static_assert(KEEP * 4 <= RING, "a second partial result fits the ring");
    static constexpr size_t smem(int n_seqs, int warps) {
        return (size_t)warps * (WARP_BYTES + 8 * S + 2 * 8 + 2 * 4) + 8 * ((size_t)n_seqs + 1) + 12 * (size_t)n_seqs;
    }
    static_assert(W <= 16 && smem(EC_KV_MAX_SEQS, W) + 16 * 8 <= 232448, "shared memory");
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, w));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) v += __shfl_xor_sync(kAll, v, w);
    return v;
}

/* Four channels of a tile's row r from its unnormalised sums v, L relative to M. */
__device__ __forceinline__ void write_row(const AttnArgs& a, int row0, int h, int r, int d, const float4& v, float M, float L) {
    const int64_t row = row0 + r / a.group;
    const int head = h * a.group + r % a.group;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int64_t off = row * a.out.row + (int64_t)head * a.out.head + d;
    store_elem(a.out, off, v.x * inv);
    store_elem(a.out, off + 1, v.y * inv);
    store_elem(a.out, off + 2, v.z * inv);
    store_elem(a.out, off + 3, v.w * inv);
    if (d == 0 && a.lse) a.lse[row * a.n_q_heads + head] = L == 0.f ? -INFINITY : (M - kBias + log2f(L)) * kLn2;
}

/* A warp's work again, row by row in FP32, from the place whose lower half is `from`; `own`: the
 * warp's shared memory. */
template <int NB>
__device__ __forceinline__ void redo_wide(const AttnArgs& a, const int64_t* pre, const int3* info, uint32_t from, float* own) {
    using H = Shape<NB>;
    constexpr int RB = H::RB, LD = H::LD;
    const int warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int64_t X = pre[a.S.n_seqs], share = share_of(a, X, gridDim.x, W), x1 = min(X, (blockIdx.x + 1) * share);
    int64_t x = min(x1, blockIdx.x * share + warp * (share / W));
    const int64_t x_end = min(x1, x + share / W);
    x += from - (uint32_t)x; /* a warp's places are fewer than 2^32 */
    while (x < x_end) {
        const Seg s = seg_at(a, pre, info, RB, x, x_end);
        x = s.next;
        const int3 f = info[s.b];
        if (s.u0 >= s.u1 || f.x == 0) continue;
        const Span sp = span_of(a, f.x, f.y);
        float* mine = own + (s.u0 == 0 ? 0 : H::RING / 4);
        for (int r = 0; r < min(RB, f.y * a.group - s.r0); ++r) {
            const int t = (s.r0 + r) / a.group;
            const RowJob j{s.b, s.h, s.h * a.group + (s.r0 + r) % a.group, f.x - f.y + t, sp.sink_u, sp.lo_u, s.u0, s.u1, (int64_t)f.z + t};
            const bool whole = s.u0 == 0 && s.u1 == s.units;
            wide_row<NB>(a, j, kBias, whole ? nullptr : mine + r * LD, mine + RB * LD + r, mine + RB * LD + RB + r);
        }
    }
}

/* Each CTA takes a share of the work (or one tile), each of its warps an even part of
 * that: a run of units, which may cover the end of a tile, whole tiles and the begin of
 * another.  Per unit: S^T, 32 channels at a time (each block with its own scale, applied
 * to the FP32 products), weights against a lazily moved reference, O^T with the value
 * scales folded into the FP16 weights; work whose value scales FP16 does not hold is done again
 * in FP32 at the end.  A warp writes tiles that it has seen whole; parts
 * meet in shared memory at the end, and what the CTA has not seen whole goes to `part`.
 * Units come by bulk copies through a ring of the warp's own, several ahead and across
 * tiles. */
template <int NB, int QT>
__global__ void __launch_bounds__(Shape<NB>::W * 32, 1) kv_attn_kernel(const __grid_constant__ AttnArgs a) {
    using H = Shape<NB>;
    constexpr int D = H::D, RB = H::RB, S = H::S, UB = H::UB, LD = H::LD;
    extern __shared__ __align__(128) uint8_t at_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5, g = lane >> 2, c = lane & 3;
    const uint32_t ring = smem_u32(at_smem) + warp * H::WARP_BYTES;
    uint8_t* tail = at_smem + W * H::WARP_BYTES;
    const uint32_t bars = smem_u32(tail) + warp * S * 8, own = ring + H::RING + H::KEEP * 4;
    int64_t* slot_tile = (int64_t*)(tail + W * S * 8);   /* [2 W]: a warp's first and last partial tile, -1: none */
    int32_t* slot_flags = (int32_t*)(slot_tile + 2 * W); /* bit 0: the tile's first unit is in, bit 1: its last */
    int64_t* pre = (int64_t*)(slot_flags + 2 * W);
    int3* info = (int3*)(pre + a.S.n_seqs + 1);
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(bars + 8 * s, 1);
        mbar_fence_init();
        sts32(own + 60, 0u); /* not 0: redo_wide takes the warp's work from the place in the word before */
        slot_tile[2 * warp] = slot_tile[2 * warp + 1] = -1;
    }
    grid_dep_launch();
    grid_dep_wait();
    scan_seqs(a, RB, pre, info, blockIdx.x == 0);
    const int64_t X = pre[a.S.n_seqs];
    const int64_t share = share_of(a, X, gridDim.x, W);
    const int64_t x0 = min(X, blockIdx.x * share), x1 = min(X, x0 + share);
    JoinJob* todo = (JoinJob*)(a.part + (int64_t)gridDim.x * 2 * RB * (D + 2)) + blockIdx.x;
    if (!a.solo && threadIdx.x == 0) todo->parts = 0;
    if (x0 >= x1) return;
    int64_t x = min(x1, x0 + warp * (share / W));
    const int64_t x_end = min(x1, x + share / W);
    const int unit_mask = (1 << (a.P.page_shift - 4)) - 1;

    /* the ring's filling side: a cursor of its own over the warp's segments.  The lanes hold the
     * next units' addresses, up to 32 at a time, and issue the copies, two units to a stage. */
    int64_t px = x;
    int pk = 0, pn = 0;
    uint32_t p_count = 0;
    const uint8_t* p_src = nullptr;
    auto fill = [&]() {
        if (pk >= pn) {
            pk = pn = 0;
            while (pn == 0) {
                if (px >= x_end) return;
                const Seg s = seg_at(a, pre, info, RB, px, x_end);
                const int3 f = info[s.b];
                const Span sp = span_of(a, f.x, f.y);
                pn = f.x > 0 ? min(32, max(0, s.u1 - s.u0)) : 0;
                px = pn == 32 ? s.tile + s.u0 + 32 : s.next;
                if (lane < pn) {
                    int u = s.u0 + lane;
                    u = u < sp.sink_u ? u : u - sp.sink_u + sp.lo_u;
                    int page = a.S.table[(int64_t)s.b * a.S.table_stride + (u >> (a.P.page_shift - 4))];
                    if (page < 0 || page >= a.P.n_pages) {
                        page = 0;
                        flag_corrupt(a.status);
                    }
                    p_src = page_ptr(a.P, page, s.h, u & unit_mask);
                }
            }
        }
        /* two units, or a segment's last one (a reload starts a pair) */
        const int n = min(2, pn - pk), k = lane - pk;
        if (k >= 0 && k < n) {
            const uint32_t st = p_count & (S - 1);
            if (k == 0) mbar_arrive_tx(bars + 8 * st, n * UB);
            bulk_g2s(ring + (2 * st + k) * UB, p_src, UB, bars + 8 * st);
        }
        pk += 2;
        ++p_count;
    };
#pragma unroll 1
    for (int k = 0; k < S; ++k) fill();

    uint32_t count = 0; /* stages taken from the ring */
    bool live = true;   /* no wait has run out */
    while (live && x < x_end) {
        /* (the segment lies in shared memory for its masked ends and for what follows the loop,
         * so that the loop need not keep it in registers) */
        auto look_up = [&](Seg& sg, int3& f) {
            const uint4 p = lds128(own), q = lds128(own + 16), r = lds128(own + 32);
            sg.b = (int)p.x, sg.h = (int)p.y, sg.r0 = (int)p.z, sg.u0 = (int)p.w;
            sg.u1 = (int)q.x, sg.units = (int)q.y, sg.tile = (int64_t)((uint64_t)q.w << 32 | q.z);
            f = make_int3((int)r.x, (int)r.y, (int)r.z);
        };
        int u = 0, u1 = 0, all_lo = 0, all_hi = 0;
        uint32_t qf[QT][NB][4];
        float fac[2];
        {
            const Seg sg = seg_at(a, pre, info, RB, x, x_end);
            const int3 f = info[sg.b];
            const uint32_t place = (uint32_t)x;
            x = sg.next;
            if (sg.u0 >= sg.u1) continue;
            __syncwarp();
            if (lane == 0) {
                uint4* o = (uint4*)(at_smem + warp * H::WARP_BYTES + H::RING + H::KEEP * 4);
                o[0] = make_uint4(sg.b, sg.h, sg.r0, sg.u0);
                o[1] = make_uint4(sg.u1, sg.units, (uint32_t)sg.tile, (uint32_t)((uint64_t)sg.tile >> 32));
                o[2] = make_uint4(f.x, f.y, f.z, place);
            }
            __syncwarp();
            const Span sp = span_of(a, f.x, f.y);
            const int h = sg.h, r0 = sg.r0, R = f.y * a.group, first = f.x - f.y;
            u = sg.u0;
            u1 = f.x > 0 ? sg.u1 : 0;
            /* units all_lo .. all_hi - 1 are seen whole by every row (with a window: those of
             * its middle; the sinks' units take the masked way) */
            const int pos_lo = first + min(r0, R - 1) / a.group, pos_hi = first + min(r0 + RB - 1, R - 1) / a.group, skip = sp.lo_u - sp.sink_u;
            all_hi = min(u1, (pos_lo + 1 < 0 ? 0 : (pos_lo + 1) / kUnit) - skip);
            all_lo = a.window ? max(sp.sink_u, (max(0, pos_hi - a.window + 1) + kUnit - 1) / kUnit - skip) : 0;

            /* queries: lane 4 g + c holds row g's channels 32 b + 8 c + 0..7, scaled by a power
             * of two so that the row's largest lies in [2^14, 2^15): BF16 and FP16 rows are
             * exact in one FP16 part but for elements 2^-28 of the row's largest, FP32 rows
             * take two parts (22 bits) */
            const int r = r0 + g;
            const bool on = r < R;
            const int64_t off = on ? (int64_t)(f.z + r / a.group) * a.q.row + (int64_t)(h * a.group + r % a.group) * a.q.head : 0;
            float xq[NB][8];
            if constexpr (QT == 2) {
                const float* p = (const float*)a.q.data + off + 8 * c;
#pragma unroll
                for (int k = 0; k < NB; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) xq[k][i] = 0.f;
                if (on && a.q.wide) {
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        const float4 u = *(const float4*)(p + 32 * k), v = *(const float4*)(p + 32 * k + 4);
                        xq[k][0] = u.x, xq[k][1] = u.y, xq[k][2] = u.z, xq[k][3] = u.w;
                        xq[k][4] = v.x, xq[k][5] = v.y, xq[k][6] = v.z, xq[k][7] = v.w;
                    }
                } else if (on) {
#pragma unroll
                    for (int k = 0; k < NB; ++k)
#pragma unroll
                        for (int i = 0; i < 8; ++i) xq[k][i] = p[32 * k + i];
                }
            } else {
                const uint16_t* p = (const uint16_t*)a.q.data + off + 8 * c;
                uint4 w[NB];
#pragma unroll
                for (int k = 0; k < NB; ++k) w[k] = make_uint4(0, 0, 0, 0);
                if (on && a.q.wide) {
#pragma unroll
                    for (int k = 0; k < NB; ++k) w[k] = *(const uint4*)(p + 32 * k);
                } else if (on) {
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        const uint16_t* e = p + 32 * k;
                        w[k] = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                    }
                }
                const bool half = a.q.dtype == EC_DTYPE_FP16;
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = __half22float2(*(const __half2*)&u[i]);
                        xq[k][2 * i] = half ? f.x : __uint_as_float(u[i] << 16);
                        xq[k][2 * i + 1] = half ? f.y : __uint_as_float(u[i] & 0xFFFF0000u);
                    }
                }
            }
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(xq[k][i]) & 0x7FFFFFFFu);
            top = max(top, __shfl_xor_sync(kAll, top, 1));
            top = max(top, __shfl_xor_sync(kAll, top, 2));
            const int E = (int)(top >> 23);
            const int up = E == 255 ? 127 : min(253, 268 - E);
            const float s = __uint_as_float((uint32_t)up << 23);
            const float inv = fmaxf(__uint_as_float((uint32_t)(254 - up) << 23) * a.scale * kLog2e, kTiny); /* > 0: a masked -inf stays one */
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y0 = xq[k][2 * i] * s, y1 = xq[k][2 * i + 1] * s;
                    qf[0][k][i] = pack_f16(y0, y1);
                    if constexpr (QT == 2) {
                        const float2 hi = __half22float2(*(const __half2*)&qf[0][k][i]);
                        qf[QT - 1][k][i] = pack_f16(y0 - hi.x, y1 - hi.y);
                    }
                }
#pragma unroll
            for (int j = 0; j < 2; ++j) fac[j] = __shfl_sync(kAll, inv, 8 * c + 4 * j);
        }

        float o[2 * NB][4];
        float m[2], l[2];
        uint32_t add[NB]; /* kRefDown - the block's reference in both halves; 300: none yet, any scale passes it */
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        m[0] = m[1] = -FLT_MAX;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int k = 0; k < NB; ++k) add[k] = both_halves(300);

#pragma unroll 1
        for (; u < u1; u += 2) {
            const uint32_t st = count & (S - 1), buf = ring + st * (2 * UB);
            if (!mbar_wait(bars + 8 * st, (count / S) & 1u)) {
                live = false;
                if (lane == 0) flag_corrupt(a.status);
                break;
            }
            ++count;

            /* S^T: rows = tokens g, g + 8 of unit v, columns = query rows 2c, 2c + 1 */
            float s[2][4];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
#pragma unroll
                for (int i4 = 0; i4 < NB / 2; ++i4) {
                    const uint4 w = lds128(buf + v * UB + i4 * 512 + lane * 16);
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int bb = 0; bb < 2; ++bb) {
                        const int blk = 2 * i4 + bb;
                        uint32_t ra[4], rb[4];
                        e2m1x8_f16(ww[2 * bb], ra);
                        e2m1x8_f16(ww[2 * bb + 1], rb);
                        const float sa = __uint_as_float(lds8(buf + v * UB + 16 * D + g * NB + blk) << 23);
                        const float sb = __uint_as_float(lds8(buf + v * UB + 16 * D + (g + 8) * NB + blk) << 23);
                        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int q = 0; q < QT; ++q) {
                            mma16816(d, ra[0], rb[0], ra[1], rb[1], qf[q][blk][0], qf[q][blk][1]);
                            mma16816(d, ra[2], rb[2], ra[3], rb[3], qf[q][blk][2], qf[q][blk][3]);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[v][j] = blk == 0 ? d[j] * (j < 2 ? sa : sb) : fmaf(d[j], j < 2 ? sa : sb, s[v][j]);
                    }
                }
            }
            const bool masked = u < all_lo || u + 1 >= all_hi;
            uint32_t vmask[2] = {0u, 0u}; /* masked: bytes of tokens 2c, 2c + 1, 2c + 8, 2c + 9 that some row sees */
            if (masked) { /* a place that a row does not see: score -inf */
                Seg sg;
                int3 f;
                look_up(sg, f);
                const Span sp = span_of(a, f.x, f.y);
                const int R = f.y * a.group, first = f.x - f.y, skip = sp.lo_u - sp.sink_u;
                const int pos_lo = first + min(sg.r0, R - 1) / a.group, pos_hi = first + min(sg.r0 + RB - 1, R - 1) / a.group;
                int tok[2];
#pragma unroll
                for (int v = 0; v < 2; ++v) tok[v] = u + v < u1 ? (u + v < sp.sink_u ? u + v : u + v + skip) * kUnit : (int)kMaxLen; /* past every token */
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int p = first + min(sg.r0 + 2 * c + j, R - 1) / a.group;
#pragma unroll
                    for (int v = 0; v < 2; ++v)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int at = tok[v] + g + 8 * k;
                            if (at > p || (a.window && at <= p - a.window && at >= a.sinks)) s[v][j + 2 * k] = -INFINITY;
                        }
                }
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = tok[v] + 2 * c + (j & 1) + 8 * (j >> 1);
                        if (at <= pos_hi && (!a.window || at > pos_lo - a.window || at < a.sinks)) vmask[v] |= 0xFFu << (8 * j);
                    }
            }

            /* weights 2^(s - m + kBias); the references move when a lane's eight weights add to
             * more than 2^(kBias + 3), or to NaN: one row's must not hide the other's (fac > 0, so
             * a masked -inf stays one) */
            float p[2][4], sum[2];
            auto weights = [&]() {
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[v][j] = ex2(fmaf(s[v][j], fac[j & 1], kBias - m[j & 1]));
                sum[0] = (p[0][0] + p[0][2]) + (p[1][0] + p[1][2]);
                sum[1] = (p[0][1] + p[0][3]) + (p[1][1] + p[1][3]);
                return !(sum[0] + sum[1] <= 256.f);
            };
            if (__any_sync(kAll, weights())) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float mx = fmaxf(fmaxf(s[0][j], s[0][j + 2]), fmaxf(s[1][j], s[1][j + 2])) * fac[j];
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, w));
                    const float nm = fmaxf(m[j], mx), al = ex2(m[j] - nm);
                    m[j] = nm;
                    l[j] *= al;
#pragma unroll
                    for (int i = 0; i < 2 * NB; ++i) {
                        o[i][j] *= al;
                        o[i][j + 2] *= al;
                    }
                }
                if (__any_sync(kAll, weights())) {
                    /* Scores of 2^22 and more: what rounds off the product of the largest one is more than
                     * weights can bear, so the products are rounded as the reference was.  (A row of NaN
                     * comes by as well.) */
#pragma unroll
                    for (int v = 0; v < 2; ++v)
#pragma unroll
                        for (int j = 0; j < 4; ++j) p[v][j] = ex2(__fadd_rn(__fmul_rn(s[v][j], fac[j & 1]), -m[j & 1]) + kBias);
                    sum[0] = (p[0][0] + p[0][2]) + (p[1][0] + p[1][2]);
                    sum[1] = (p[0][1] + p[0][3]) + (p[1][1] + p[1][3]);
                }
            }
            /* their transposition into the second product's operand */
            uint32_t p0[2], p1[2];
            l[0] += sum[0];
            l[1] += sum[1];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                p0[v] = transpose8x8(pack_f16(p[v][0], p[v][1]));
                p1[v] = transpose8x8(pack_f16(p[v][2], p[v][3]));
            }

            /* value scales 2^(e - ref) as FP16 pairs: z = e - ref + kRefDown, exponent field z + 7;
             * z outside 0..15 means more than 2^7 above the reference or 2^-8 below it (or a block
             * of zeros or NaN) */
            uint32_t vw[2][NB], z0[2][NB], z1[2][NB], over = 0;
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int i = 0; i < NB / 2; ++i) {
                    const uint32_t at = buf + v * UB + 16 * D + D / 2 + (c * NB + 2 * i) * 4;
                    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(vw[v][2 * i]), "=r"(vw[v][2 * i + 1]) : "r"(at) : "memory");
                }
            if (masked) { /* scales of tokens that no row sees: the reference, or none (their weights are 0) */
#pragma unroll
                for (int k2 = 0; k2 < NB; ++k2) {
                    const uint32_t ref = (uint32_t)max(kRefDown - (int)(int16_t)(add[k2] & 0xFFFFu), 0) * 0x01010101u;
#pragma unroll
                    for (int v = 0; v < 2; ++v) vw[v][k2] = (vw[v][k2] & vmask[v]) | (ref & ~vmask[v]);
                }
            }
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int k2 = 0; k2 < NB; ++k2) {
                    z0[v][k2] = __viaddmax_s16x2(__byte_perm(vw[v][k2], 0, 0x4140), add[k2], 0x80008000u);
                    z1[v][k2] = __viaddmax_s16x2(__byte_perm(vw[v][k2], 0, 0x4342), add[k2], 0x80008000u);
                    over |= z0[v][k2] | z1[v][k2];
                }
            bool bad = false;
            if (__any_sync(kAll, (over & 0xFFF0FFF0u) != 0)) {
                uint32_t ends[NB]; /* the largest and smallest scale, but zeros and NaN */
                uint32_t nan = 0;
#pragma unroll
                for (int k2 = 0; k2 < NB; ++k2) {
                    uint32_t hi = 0, lo = 0xFFFFFFFFu;
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t x = __byte_perm(vw[v][k2], 0, k ? 0x4342 : 0x4140), y = x + 0x00010001u;
                            nan |= y;
                            hi = __vmaxu2(hi, y & 0x00FF00FFu);
                            lo = __viaddmin_u16x2(x, 0xFFFFFFFFu, lo);
                        }
                    }
                    ends[k2] = __reduce_max_sync(kAll, max(hi & 0xFFFFu, hi >> 16)) | __reduce_min_sync(kAll, min(lo & 0xFFFFu, lo >> 16)) << 16;
                }
                bad = __any_sync(kAll, (nan & 0x01000100u) != 0);
                bool wide = false;
#pragma unroll
                for (int k2 = 0; k2 < NB; ++k2) {
                    const int ref = kRefDown - (int)(int16_t)(add[k2] & 0xFFFFu); /* < 0: none yet, o is 0 or NaN */
                    const int mx = (int)(ends[k2] & 0xFFFFu) - 1, mn = (int)(ends[k2] >> 16) + 1;
                    const bool move = mx > 0 && (mx > ref + kRefUp || mn < ref - kRefDown), again = move && ref >= 0;
                    const int to = !move ? ref : mx - mn <= kRefDown ? mx : max(mx - kRefUp, 1);
                    const float f = again ? __uint_as_float((uint32_t)(127 + max(-126, min(126, ref - to))) << 23) : 1.f;
                    add[k2] = both_halves(kRefDown - to);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        o[2 * k2][j] *= f;
                        o[2 * k2 + 1][j] *= f;
                    }
                    wide |= move && mx - mn > kRefUp + kRefDown;
                    if (again) wide |= abs(to - (int)lds8(own + 48 + k2)) > kRefSpan;
                    else if (move) sts8(own + 48 + k2, (uint32_t)to);
                    const uint32_t add7 = both_halves((int)(int16_t)(add[k2] & 0xFFFFu) + 7);
#pragma unroll
                    for (int v = 0; v < 2; ++v) { /* (what lies outside is zeros, NaN, unseen, or wide_row's) */
                        z0[v][k2] = __vmins2(__viaddmax_s16x2(__byte_perm(vw[v][k2], 0, 0x4140), add7, 0u), 0x00160016u) - 0x00070007u;
                        z1[v][k2] = __vmins2(__viaddmax_s16x2(__byte_perm(vw[v][k2], 0, 0x4342), add7, 0u), 0x00160016u) - 0x00070007u;
                    }
                }
                if (wide && lds32(own + 60) == 0) {
                    sts32(own + 56, lds32(own + 44));
                    sts32(own + 60, 1u);
                }
            }

            /* O^T: rows = channels, columns = query rows */
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int i4 = 0; i4 < NB / 2; ++i4) {
                    const uint4 w = lds128(buf + v * UB + 8 * D + i4 * 512 + lane * 16);
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int bb = 0; bb < 2; ++bb) {
                        const int blk = 2 * i4 + bb;
                        const uint32_t s0 = z0[v][blk] * 1024u + 0x1C001C00u, s1 = z1[v][blk] * 1024u + 0x1C001C00u;
                        uint32_t b0 = hmul2(p0[v], s0), b1 = hmul2(p1[v], s1);
                        if (bad) { /* a block of NaN makes its channels NaN for every row that sees the token */
                            Seg sg;
                            int3 f;
                            look_up(sg, f);
                            const Span sp = span_of(a, f.x, f.y);
                            const int R = f.y * a.group, tok = (u + v < sp.sink_u ? u + v : u + v + sp.lo_u - sp.sink_u) * kUnit;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (lds8(buf + v * UB + 16 * D + D / 2 + (c * NB + blk) * 4 + j) != 255u) continue;
                                const int at = tok + 2 * c + (j & 1) + 8 * (j >> 1);
                                const int p = f.x - f.y + min(sg.r0 + g, R - 1) / a.group;
                                if (u + v >= u1 || at > p || (a.window && at <= p - a.window && at >= a.sinks)) continue;
                                (j < 2 ? b0 : b1) |= 0x7FFFu << (16 * (j & 1));
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t ra[4];
                            e2m1x8_f16(ww[2 * bb + j], ra);
                            mma16816(o[2 * blk + j], ra[0], ra[1], ra[2], ra[3], b0, b1);
                        }
                    }
                }
            __syncwarp(); /* every lane has read the stage */
            fill();
        }

        /* the lanes' sums; values are held relative to 2^(ref - 127) per block (ref < 0:
         * nothing but blocks of zeros so far, a NaN there stays one) */
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) l[j] += __shfl_xor_sync(kAll, l[j], w);
        Seg sg;
        int3 f;
        look_up(sg, f);
        const int h = sg.h, r0 = sg.r0, R = f.y * a.group;
        float back[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int ref = kRefDown - (int)(int16_t)(add[k] & 0xFFFFu);
            back[k] = ref > 0 ? __uint_as_float((uint32_t)ref << 23) : 0.f;
        }
        if (sg.u0 == 0 && sg.u1 == sg.units) {
            if (lds32(own + 60)) continue; /* nothing is written over queries that are still to be read, should out be q */
            float inv[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                inv[j] = l[j] == 0.f ? 0.f : 1.f / l[j];
                const int r = r0 + 2 * c + j;
                if (a.lse && g == 0 && r < R)
                    a.lse[(int64_t)(f.z + r / a.group) * a.n_q_heads + h * a.group + r % a.group] =
                        l[j] == 0.f ? -INFINITY : (m[j] - kBias + log2f(l[j])) * kLn2;
            }
            /* 8 x 8 transpositions turn channels g of rows 2c, 2c + 1 into channels 2c,
             * 2c + 1 of row g (FP32 rows are stored as they lie) */
            if (a.out.dtype != EC_DTYPE_FP32) {
                const int r = r0 + g;
                const int64_t off = (int64_t)(f.z + r / a.group) * a.out.row + (int64_t)(h * a.group + r % a.group) * a.out.head + 2 * c;
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float v0 = o[i][2 * j] * back[i / 2] * inv[0], v1 = o[i][2 * j + 1] * back[i / 2] * inv[1];
                        uint32_t w;
                        if (a.out.dtype == EC_DTYPE_FP16) w = pack_f16(v0, v1);
                        else {
                            const __nv_bfloat162 y = __floats2bfloat162_rn(v0, v1);
                            w = *(const uint32_t*)&y;
                        }
                        w = transpose8x8(w);
                        if (r < R) {
                            uint16_t* at = (uint16_t*)a.out.data + off + 16 * i + 8 * j;
                            if (a.out.wide) *(uint32_t*)at = w;
                            else {
                                at[0] = (uint16_t)w;
                                at[1] = (uint16_t)(w >> 16);
                            }
                        }
                    }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = r0 + 2 * c + j;
                    if (r >= R) continue;
                    float* at = (float*)a.out.data + (int64_t)(f.z + r / a.group) * a.out.row + (int64_t)(h * a.group + r % a.group) * a.out.head + g;
#pragma unroll
                    for (int i = 0; i < 2 * NB; ++i) {
                        at[16 * i] = o[i][j] * back[i / 2] * inv[j];
                        at[16 * i + 8] = o[i][j + 2] * back[i / 2] * inv[j];
                    }
                }
            }
        } else {
            /* the end of a tile is the warp's first segment, the begin of another its last,
             * when the ring is empty */
            const int slot = sg.u0 == 0 ? 1 : 0;
            float* mine = (float*)(at_smem + warp * H::WARP_BYTES + (slot ? 0 : H::RING));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 2 * c + j;
                if (g == 0) {
                    mine[RB * LD + r] = m[j];
                    mine[RB * LD + RB + r] = l[j];
                }
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) {
                    mine[r * LD + 16 * i + g] = o[i][j] * back[i / 2];
                    mine[r * LD + 16 * i + 8 + g] = o[i][j + 2] * back[i / 2];
                }
            }
            if (lane == 0) {
                slot_tile[2 * warp + slot] = sg.tile;
                slot_flags[2 * warp + slot] = (sg.u0 == 0 ? 1 : 0) | (sg.u1 == sg.units ? 2 : 0);
            }
        }
    }
    if (!live) /* the copies in flight end before the shared memory is given back */
        for (; count != p_count; ++count) mbar_wait(bars + 8 * (count & (S - 1)), (count / S) & 1u);
    __syncwarp();
    if (lds32(own + 60)) redo_wide<NB>(a, pre, info, lds32(own + 56), (float*)(at_smem + warp * H::WARP_BYTES));

    /* join the warps' parts, tile by tile, in order: lane k holds slot k's tile; 8, 4, 2 or one
     * warps take a tile, a row at a time, so that most warps have one */
    __syncthreads();
    const int64_t slot = lane < 2 * W ? slot_tile[lane] : -1;
    const int flags = lane < 2 * W ? slot_flags[lane] : 0;
    const float* kept = (const float*)(at_smem + (lane / 2) * H::WARP_BYTES + (lane & 1 ? 0 : H::RING));
    const uint32_t same = __match_any_sync(kAll, slot);
    uint32_t firsts = __ballot_sync(kAll, slot >= 0 && __ffs(same) - 1 == lane);
    const int nt = __popc(firsts);
    const int G = 8 * nt <= W ? 8 : 4 * nt <= W ? 4 : 2 * nt <= W ? 2 : 1; /* 4 at most with 4 warps */
    for (int n = 0; firsts; ++n, firsts &= firsts - 1) {
        if (n % (W / G) != warp / G) continue;
        const int s0 = __ffs(firsts) - 1;
        const int64_t tile = __shfl_sync(kAll, slot, s0);
        const uint32_t of = __shfl_sync(kAll, same, s0);
        const bool begins = __shfl_sync(kAll, flags, s0) & 1, whole = begins && (__shfl_sync(kAll, flags, 31 - __clz(of)) & 2);
        const Seg sg = seg_at(a, pre, info, RB, tile, X);
        const int3 f = info[sg.b];
        const int R = f.y * a.group;
        if (warp % G == 0 && lane == 0 && !whole && begins) { /* the tile begins here: how many shares it covers */
            todo->parts = (int)((tile + sg.units - 1) / share) - (int)blockIdx.x + 1;
            todo->h = sg.h, todo->r0 = sg.r0, todo->R = R, todo->row0 = f.z;
        }
        float* part = a.part + ((int64_t)blockIdx.x * 2 + begins) * (RB * (D + 2));
        const bool in = (of >> lane) & 1u;
#pragma unroll 1
        for (int r = warp % G; r < min(RB, R - sg.r0); r += G) {
            const float pm = in ? kept[RB * LD + r] : -FLT_MAX;
            const float M = warp_max(pm);
            const float w = in ? ex2(pm - M) : 0.f;
            const float L = warp_sum(in ? w * kept[RB * LD + RB + r] : 0.f);
#pragma unroll
            for (int d0 = 0; d0 < D; d0 += 128) {
                const int d = d0 + 4 * lane;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                for (uint32_t k = of; k;) {
                    float wi[4];
                    float4 y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int i = k ? __ffs(k) - 1 : s0;
                        wi[j] = __shfl_sync(kAll, w, i);
                        y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (k && d < D) y[j] = *(const float4*)((const float*)(at_smem + (i / 2) * H::WARP_BYTES + (i & 1 ? 0 : H::RING)) + r * LD + d);
                        k &= k - 1;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v.x = fmaf(y[j].x, wi[j], v.x), v.y = fmaf(y[j].y, wi[j], v.y), v.z = fmaf(y[j].z, wi[j], v.z), v.w = fmaf(y[j].w, wi[j], v.w);
                }
                if (d >= D) continue;
                if (whole) write_row(a, f.z, sg.h, sg.r0 + r, d, v, M, L);
                else *(float4*)&part[r * D + d] = v;
            }
            if (!whole && lane == 0) {
                part[RB * D + r] = M;
                part[RB * D + RB + r] = L;
            }
        }
    }
}

/* Join the partial results of a tile that several shares cover: CTA i adds, in order, the
 * parts of the tile that begins in share i and does not end there (if there is one).  A
 * warp takes a row, 32 parts at a time: each lane one part's maximum and sum, then four
 * channels of every part, eight parts at a time, whose loads wait for nothing.  Bound by
 * three round trips to memory: 2.3 us (19 parts of 8 tiles; 8.8 us with a loop over 38
 * parts, 1.3 us where tiles have two or three). */
template <int NB>
__global__ void __launch_bounds__(256, 2) kv_join_kernel(const __grid_constant__ AttnArgs a) {
    using H = Shape<NB>;
    constexpr int D = H::D, RB = H::RB, PS = RB * (D + 2), NV = (D + 127) / 128;
    grid_dep_launch();
    grid_dep_wait();
    const JoinJob job = ((const JoinJob*)(a.part + (int64_t)gridDim.x * 2 * PS))[blockIdx.x];
    const int n = job.parts, lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    if (n == 0 || job.r0 + r >= job.R) return;
    const float* p1 = a.part + ((int64_t)blockIdx.x * 2) * PS; /* share i's part; the first share's is its second */
    auto part = [&](int i) { return p1 + (int64_t)(i ? 2 * i : 1) * PS; };
    float M = -FLT_MAX, L = 0.f;
    float4 v[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int cnt = min(32, n - i0);
        float4 y[8][NV];
        auto load = [&](int j0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    y[j][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (j0 + j < cnt && 128 * k + 4 * lane < D) y[j][k] = *(const float4*)(part(i0 + j0 + j) + r * D + 128 * k + 4 * lane);
                }
        };
        const float pm = lane < cnt ? part(i0 + lane)[RB * D + r] : -FLT_MAX, pl = lane < cnt ? part(i0 + lane)[RB * D + RB + r] : 0.f;
        load(0);
        const float top = fmaxf(M, warp_max(pm)), old = ex2(M - top), w = ex2(pm - top);
        M = top;
        L = fmaf(L, old, pl * w);
#pragma unroll
        for (int k = 0; k < NV; ++k) v[k].x *= old, v[k].y *= old, v[k].z *= old, v[k].w *= old;
        for (int j0 = 0; j0 < cnt; j0 += 8) {
            if (j0) load(j0);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float wj = __shfl_sync(kAll, w, j0 + j);
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    v[k].x = fmaf(y[j][k].x, wj, v[k].x), v[k].y = fmaf(y[j][k].y, wj, v[k].y), v[k].z = fmaf(y[j][k].z, wj, v[k].z), v[k].w = fmaf(y[j][k].w, wj, v[k].w);
            }
        }
    }
    L = warp_sum(L);
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if (128 * k + 4 * lane < D) write_row(a, job.row0, job.h, job.r0 + r, 128 * k + 4 * lane, v[k], M, L);
}

/* ------------------------------------------------------------ launch */
struct Plan {
    int grid, solo, warps;
    size_t work;
    bool many;         /* the tensor-memory form */
    PrefillPlan pre;
};

template <int NB>
static void plan_shape(Plan* p, int sms, int64_t tiles, int64_t units) {
    using H = Shape<NB>;
    /* up to 4 units per warp there is nothing to gain from splitting a tile, and one launch
     * does, as long as the tiles run at the same time (us, a CTA per tile / split: 8 tiles of
     * 17 tokens 7.1 / 8.4, 128 of 500 12.1 / 15.2, 512 of 500 25.0 / 21.7, 2048 of 300 87 / 37) */
    const int w = H::W / 2;
    const bool solo = units <= 4 * w && tiles <= 2 * sms;
    p->solo = solo ? (int)((units + w - 1) / w) * w : 0;
    p->warps = solo ? w : H::W;
    p->grid = solo ? (int)tiles : sms;
    p->work = solo ? 0 : (size_t)p->grid * (2 * H::RB * (H::D + 2) * sizeof(float) + sizeof(JoinJob));
}

/* Query rows per sequence and key/value head, on average, up to which the register form
 * runs (with up to twice as many in any one sequence): it expands the tokens once per 8
 * rows, the tensor-memory form once per 128 or 256.
 * Measured (us, register form / tensor-memory form), 16 sequences of 4100 tokens, 128
 * channels: 16 rows 40 / 66, 24 rows 53 / 66, 32 rows 65 / 66, 40 rows 78 / 66, 8 to 40 rows
 * (24 on average) 51 / 68; 64 channels: 40 rows 50 / 61, 64 rows 72 / 61; 256 channels: 16
 * rows 81 / 118, 24 rows 109 / 119, 32 rows 137 / 118; 192 channels: 24 rows 78 / 107, 40
 * rows 118 / 107.  One sequence of 30000 and 128 channels, 40 rows: 41 / 42. */
constexpr int64_t few_rows(int nb) { return nb == 2 ? 40 : nb == 4 ? 32 : 24; }

/* The mask as the kernels take it: a window that hides none of max_len tokens is none, and there
 * are no more sinks than tokens, so that sums with either stay within 31 bits. */
static ec_kv_attn within(ec_kv_attn at, int64_t max_len) {
    if (at.window >= max_len) at.window = at.sinks = 0;
    if (at.sinks > max_len) at.sinks = (int32_t)max_len;
    return at;
}

/* Sizes that both forms are planned by; none shrinks when a bound grows. */
struct Extent {
    int group, nb;
    int64_t rows;            /* per sequence and key/value head */
    int64_t units;           /* that a sequence's rows see */
    int64_t per_seq, tiles;  /* of 8 rows */
    bool past;               /* more work per sequence than the register form counts (31 bits) */
};
static Extent extent_of(const ec_kv* C, int n_seqs, int max_new, int64_t max_len, const ec_kv_attn* at) {
    Extent x;
    x.group = at->n_q_heads / C->p.n_kv_heads;
    x.nb = C->p.head_dim / 32;
    x.rows = (int64_t)x.group * max_new;
    x.units = (max_len + kUnit - 1) / kUnit;
    if (at->window) {
        const int64_t w = ((int64_t)at->window + max_new + kUnit) / kUnit + 1 + (at->sinks + kUnit - 1) / kUnit;
        if (w < x.units) x.units = w;
    }
    if (x.units < 1) x.units = 1;
    x.per_seq = (x.rows + 7) / 8 * C->p.n_kv_heads;
    x.tiles = x.per_seq * n_seqs;
    x.past = x.per_seq > 0x7FFFFFFF / (x.units + kTileCost);
    return x;
}
static void plan_few(Plan* p, int sms, const Extent& x) {
    switch (x.nb) {
        case 2: plan_shape<2>(p, sms, x.tiles, x.units); break;
        case 4: plan_shape<4>(p, sms, x.tiles, x.units); break;
        case 6: plan_shape<6>(p, sms, x.tiles, x.units); break;
        default: plan_shape<8>(p, sms, x.tiles, x.units);
    }
}

/* false: more work than the kernels count */
static bool plan_of(const ec_kv* C, int sms, int n_seqs, int64_t n_rows, int max_new, int64_t max_len, const ec_kv_attn* at, int dtype, Plan* p) {
    const Extent x = extent_of(C, n_seqs, max_new, max_len, at);
    const int64_t few = few_rows(x.nb);
    p->many = x.rows > 2 * few || (x.rows > few && n_rows > few * n_seqs / x.group) || x.past;
    if (!p->many) {
        plan_few(p, sms, x);
        return true;
    }
    p->grid = p->solo = 0;
    if (!plan_prefill(C, sms, n_seqs, max_new, x.units, x.group, dtype, &p->pre)) return false;
    p->work = p->pre.work;
    return true;
}

/* The most work that any call of at most these sizes plans.  Both forms' parts are bounded: the
 * register form's by its grid of one CTA per SM (a call whose tiles have a CTA each has smaller
 * ones that do too), the tensor-memory form's by the same many row tiles and splits; fewer rows
 * of the same bounds may take either. */
static bool most_work(const ec_kv* C, int sms, int n_seqs, int max_new, int64_t max_len, const ec_kv_attn* at, int dtype, size_t* bytes) {
    const Extent x = extent_of(C, n_seqs, max_new, max_len, at);
    Plan p;
    plan_few(&p, sms, x);
    *bytes = p.work;
    if (x.rows <= few_rows(x.nb) && !x.past) return true;
    if (!plan_prefill(C, sms, n_seqs, max_new, x.units, x.group, dtype, &p.pre)) return false;
    if (p.pre.most > *bytes) *bytes = p.pre.most;
    return true;
}

template <int NB, int QT>
static int run_attn(const AttnArgs& a, const Plan& p, cudaStream_t stream) {
    using H = Shape<NB>;
    static SmemOnce once;
    int rc = once.set(kv_attn_kernel<NB, QT>, H::smem(EC_KV_MAX_SEQS, H::W));
    if (rc != EC_OK) return rc;
    rc = launch(kv_attn_kernel<NB, QT>, dim3(p.grid), p.warps * 32, H::smem(a.S.n_seqs, p.warps), stream, a);
    if (rc == EC_OK && !p.solo)
        rc = launch(kv_join_kernel<NB>, dim3(p.grid), 256, 0, stream, a);
    return rc;
}

template <int NB>
static int run_terms(const AttnArgs& a, const Plan& p, cudaStream_t stream) {
    return a.q.dtype == EC_DTYPE_FP32 ? run_attn<NB, 2>(a, p, stream) : run_attn<NB, 1>(a, p, stream);
}

static int check_attn(const ec_kv* C, int n_seqs, int64_t n_rows, int max_new, int64_t max_len, const ec_kv_attn* at) {
    if (!C || !at) return EC_ERR_INVALID_ARG;
    if (n_seqs < 0 || n_rows < 0 || max_new < 0 || max_len < 0) return EC_ERR_SHAPE;
    if (max_len > kMaxLen) return EC_ERR_UNSUPPORTED;
    if (n_seqs > EC_KV_MAX_SEQS || max_new > (1 << 24) || at->n_q_heads > 65536) return EC_ERR_UNSUPPORTED;
    if (at->n_q_heads < 1 || at->n_q_heads % C->p.n_kv_heads) return EC_ERR_SHAPE;
    if (at->window < 0 || at->sinks < 0 || (at->sinks > 0 && at->window == 0)) return EC_ERR_INVALID_ARG;
    if (!(at->scale >= 0.f) || at->scale > FLT_MAX) return EC_ERR_INVALID_ARG;
    return EC_OK;
}

}  // namespace kv

using namespace kv;

extern "C" int ec_kv_attend_work_bytes(const ec_kv* C, int n_seqs, int64_t n_rows, int max_new, int64_t max_len,
                                       const ec_kv_attn* attn, size_t* bytes) {
    if (!bytes) return EC_ERR_INVALID_ARG;
    int rc = check_attn(C, n_seqs, n_rows, max_new, max_len, attn);
    if (rc != EC_OK) return rc;
    int sms = 0, dev = 0;
    if (C->pool) {
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return EC_ERR_CUDA;
    } else sms = 152;
    *bytes = 0;
    if (n_seqs == 0 || max_new == 0) return EC_OK;
    if (max_len == 0) max_len = kMaxLen;
    const ec_kv_attn at = within(*attn, max_len);
    for (int dtype : {EC_DTYPE_BF16, EC_DTYPE_FP32}) {
        size_t most = 0;
        if (!most_work(C, sms, n_seqs, max_new, max_len, &at, dtype, &most)) return EC_ERR_UNSUPPORTED;
        if (most > *bytes) *bytes = most;
    }
    return EC_OK;
}

extern "C" int ec_kv_attend(const ec_kv* C, const ec_kv_attention* t, cudaStream_t stream) {
    if (!C || !t) return EC_ERR_INVALID_ARG;
    int rc = check_seqs(&t->seqs);
    if (rc != EC_OK) return rc;
    int64_t max_len = t->max_len;
    if (max_len == 0) {
        max_len = t->seqs.table_stride * C->p.page_tokens;
        if (max_len > kMaxLen) max_len = kMaxLen;
    }
    if ((rc = check_attn(C, t->seqs.n_seqs, t->n_rows, t->max_new, max_len, &t->attn)) != EC_OK) return rc;
    const ec_kv_attn at = within(t->attn, max_len);
    if (!t->starts && t->n_rows < t->seqs.n_seqs) return EC_ERR_SHAPE;
    AttnArgs a{};
    if (!pool_view(C, t->layer, &a.P)) return EC_ERR_INVALID_ARG;
    if ((rc = check_rows(&t->q, at.n_q_heads, t->n_rows, &a.q)) != EC_OK) return rc;
    if ((rc = check_rows(&t->out, at.n_q_heads, t->n_rows, &a.out)) != EC_OK) return rc;
    if ((uintptr_t)t->lse % 4) return EC_ERR_INVALID_ARG;
    Device d;
    if ((rc = device_of(C, &d)) != EC_OK) return rc;
    if (t->seqs.n_seqs == 0 || t->n_rows == 0 || t->max_new == 0) return EC_OK;
    Plan p;
    if (!plan_of(C, d.sms, t->seqs.n_seqs, t->n_rows, t->max_new, max_len, &at, t->q.dtype, &p)) return EC_ERR_UNSUPPORTED;
    if (p.work && (!t->work || (uintptr_t)t->work % 16 || t->work_bytes < p.work)) return EC_ERR_INVALID_ARG;
    a.S = Seqs{t->seqs.table, t->seqs.lens, t->starts, t->seqs.table_stride, t->n_rows, t->seqs.n_seqs};
    a.lse = t->lse;
    a.part = (float*)t->work;
    a.n_q_heads = at.n_q_heads;
    a.group = at.n_q_heads / C->p.n_kv_heads;
    a.window = at.window;
    a.sinks = at.sinks;
    a.scale = at.scale > 0.f ? at.scale : 1.f / sqrtf((float)C->p.head_dim);
    a.max_new = t->max_new;
    a.max_len = (int32_t)max_len;
    a.solo = p.solo;
    a.status = d.status;
    if (p.many) return launch_prefill(a, p.pre, stream);
    switch (C->p.head_dim / 32) {
        case 2: return run_terms<2>(a, p, stream);
        case 4: return run_terms<4>(a, p, stream);
        case 6: return run_terms<6>(a, p, stream);
        default: return run_terms<8>(a, p, stream);
    }
}
