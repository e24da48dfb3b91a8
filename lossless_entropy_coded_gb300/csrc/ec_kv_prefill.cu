/*
 * ec_kv_prefill.cu -- attention of many new rows over the 4-bit cache on the tensor
 * cores (tcgen05), the form of ec_kv_attend for more rows per key/value head than the
 * register kernel holds at once.
 *
 * One CTA takes 128 NQ rows (row r of a sequence: new token r / group, query head r %
 * group of one key/value head) and walks the tokens they see in tiles.  A tile is
 * expanded from 4 bits once for all rows:
 *   keys    FP16 k 2^(e - kref + 13), kref the tile's largest scale, so S = Q K^T comes
 *           out times a power of two of the tile;
 *   values  FP16 v 2^(e - vref), vref per 32 channels: it moves (and the accumulators with
 *           it) only when a tile's scales lie more than 2^13 above or 2^14 below.
 * Where a tile's value scales span more, or vref would go further than kVSpan from its
 * first, or a key's scale lies 2^-28 below the largest kref, the CTA's rows are done again in
 * FP32 at the end (wide_row); and a warp's rows, where a score passes kMost.
 * S (FP32, in tensor memory) is read one row per thread, the weights 2^(s - m + 6) go
 * back as FP16 in S's place and are the tensor-memory operand of O += P V.  The row's
 * reference m moves, and O with it, only when a score passes it by 2^8.
 *
 * Bounds.  The floor is the tensor pipe: 4 D operations per visible (query, token) pair.
 * Two prompts (2999 and 5003 new rows of 32 query over 8 key/value heads, 128 channels, up
 * to 13000 tokens): 1135 us, 1.16 PFLOP/s, 0.59 of the measured BF16 rate; tensor pipe 47 %
 * active over a whole launch.  What bounds it is the chain of one row tile: softmax of 128
 * tokens (about 1850 clocks), then its product and the next scores (1500), of which the
 * other row tile hides only its own share; shared memory carries the products' operands
 * (192 KB per 128 tokens), the expanded tiles (64 KB) and the 4-bit ones (17 KB) at 128
 * bytes per clock, 2100 clocks of the 3400.  Tiles of 64 tokens with two score tiles per row
 * tile, which break the chain, took 1476 us (twice the barriers, and products of 64 columns
 * read 6 KB for 32 clocks of work).
 *
 * Warps: NQ groups of four for the softmax, four that expand tiles, one that issues the
 * matrix instructions, one that copies units in, one that finds their largest scales.
 * Matrix instructions of the NQ row tiles alternate (P0 V, Q0 K', P1 V, Q1 K', ...), so that
 * one tile's softmax runs under the other's products.
 */
#include "ec_kv_attn.h"

namespace kv {

constexpr float kPBias = 6.f, kPSlack = 8.f;
constexpr int kVUp = 13, kVDown = 14, kVSpan = 16;
/* A reference from which what rounds off a score's product may raise a weight twofold. */
constexpr float kMost = 4194304.f;

template <int NB, int NQ, int QT>
struct PShape {
    static constexpr int D = 32 * NB, UB = 17 * D;
    static constexpr int TN = NB <= 4 ? 128 : 64;        /* tokens per tile */
    static constexpr int UT = TN / kUnit;                /* units per tile */
    static constexpr int QBYTES = 128 * D * 2;           /* one row tile, one part */
    static constexpr int BUF = TN * D * 2;               /* one expanded tile */
    static constexpr int RAW = UT * UB;                  /* one tile in 4 bits */
    static constexpr int META = 16 + 64 + TN;            /* kref, flags, vref[8], factors[8], NaN masks */
    static constexpr int MS = 4;                         /* tiles' metas */
    static constexpr int RS = NB == 8 && QT == 2 ? 1 : 2; /* tiles in 4 bits */
    static constexpr int FIXED = NQ * QT * QBYTES + RS * RAW + MS * META + 256;
    static constexpr int ROOM = (232448 - 1024 - FIXED) / BUF;
    static constexpr int NBUF = ROOM > 4 ? 4 : ROOM;
    static_assert(NBUF >= 2, "a key and a value tile fit");
    static_assert(NQ * QT * QBYTES + NBUF * BUF + RS * RAW + MS * META + 256 + 1024 <= 232448, "shared memory");
    static constexpr int EW = 4;                         /* warps that expand */
    static constexpr int WARPS = 4 * NQ + EW + 4;        /* whole warpgroups; one warp idles */
    static constexpr int SMEM = NQ * QT * QBYTES + NBUF * BUF + RS * RAW + MS * META + 256 + 1024;
    static constexpr int O_COL = NQ * TN;                /* accumulators behind the scores */
    static constexpr uint32_t COLS = NQ * (TN + D) <= 256 ? 256 : 512;
    static_assert(NQ * (TN + D) <= 512, "tensor memory");
};

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
/* 32 lanes x 32 columns of 32 bits; the wait ties the registers, so nothing uses them before. */
__device__ __forceinline__ void tc_ld32(uint32_t at, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(at)
        : "memory");
}
/* The same with the largest of the 32 columns (FP32), found on the way. */
__device__ __forceinline__ void tc_ld32_max(uint32_t at, uint32_t (&v)[32], float& mx) {
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]), "=f"(mx)
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tc_wait_ld(float& a, float& b) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(a), "+f"(b)::"memory");
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                   "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                   "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])::"memory");
}
__device__ __forceinline__ void tc_st32(uint32_t at, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
        ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
          "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
          "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
          "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(at)
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t at, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
          "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(at)
        : "memory");
}
/* Descriptor of a K-major operand in 128-byte-swizzled atoms of 64 FP16 columns, 8-row
 * groups 1024 bytes apart: start address >> 4, stride 1024 B >> 4 at bit 32, version 1 at
 * bit 46, swizzle mode 2 (128 B) at bit 61.  16 columns on: 32 bytes further. */
__device__ __forceinline__ uint64_t sw128_desc(uint32_t at) {
    return (uint64_t)((at >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) |
           ((uint64_t)2u << 61);
}
/* Four matrix instructions, 16 columns of the operands each, by one elected lane of a
 * converged warp: A from shared memory, or from tensor memory. */
__device__ __forceinline__ void tc_mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\tadd.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\tadd.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\tadd.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tc_mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 y;\n\t.reg .b32 x;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\tadd.s32 x, %1, 8;\n\tadd.s64 y, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\tadd.s32 x, %1, 16;\n\tadd.s64 y, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\tadd.s32 x, %1, 24;\n\tadd.s64 y, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

/* (a f + c, b f + c) and acc + (a, b): the two-wide FP32 instructions. */
__device__ __forceinline__ float2 fma2(uint32_t a, uint32_t b, float f, float c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, d;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %5};\n\t"
        "fma.rn.f32x2 d, x, y, z;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(a), "r"(b), "f"(f), "f"(c));
    return r;
}
__device__ __forceinline__ float2 add2(float2 acc, float a, float b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, d;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 d, x, y;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(acc.x), "f"(acc.y), "f"(a), "f"(b));
    return r;
}

/* Largest bytes, as two 16-bit halves to be joined by half_max. */
__device__ __forceinline__ uint32_t bytes_max(uint32_t m, uint32_t w) {
    return __vmaxu2(m, __vmaxu2(w & 0x00FF00FFu, (w >> 8) & 0x00FF00FFu));
}
/* Smallest bytes but zeros, less 1 (65535: none). */
__device__ __forceinline__ uint32_t bytes_min(uint32_t m, uint32_t w) {
    return __viaddmin_u16x2(w & 0x00FF00FFu, 0xFFFFFFFFu, __viaddmin_u16x2((w >> 8) & 0x00FF00FFu, 0xFFFFFFFFu, m));
}
__device__ __forceinline__ int half_min(uint32_t m) { return (int)min(m & 0xFFFFu, m >> 16) + 1; }
__device__ __forceinline__ int half_max(uint32_t m) { return (int)max(m & 0xFFFFu, m >> 16); }
/* A word's bytes with 255 (NaN) as 0. */
__device__ __forceinline__ uint32_t drop_nan(uint32_t w) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (((w >> (8 * i)) & 0xFFu) == 0xFFu) w &= ~(0xFFu << (8 * i));
    return w;
}

/* What a CTA works on. */
struct PJob {
    int b, h, r0, R, len, first, group;
    int sink_u, lo_u, units; /* units that its rows see */
    int u0, u1;              /* this split's */
    int64_t row0;
};

template <int NB, int NQ, int QT>
__global__ void __launch_bounds__(PShape<NB, NQ, QT>::WARPS * 32, 1) kv_prefill_kernel(const __grid_constant__ AttnArgs a) {
    using H = PShape<NB, NQ, QT>;
    constexpr int D = H::D, TN = H::TN, UT = H::UT, UB = H::UB, NBUF = H::NBUF;
    extern __shared__ __align__(1024) uint8_t pf_smem[];
    /* (warp-uniform values are taken from lane 0, so that the compiler knows them for such) */
    const int lane = threadIdx.x & 31, warp = __shfl_sync(kAll, (int)threadIdx.x >> 5, 0), g = lane >> 2, c = lane & 3;
    const uint32_t base = (smem_u32(pf_smem) + 1023u) & ~1023u;
    const uint32_t q_at = base, buf_at = q_at + NQ * QT * H::QBYTES, raw_at = buf_at + NBUF * H::BUF, meta_at = raw_at + H::RS * H::RAW,
                   bars = meta_at + H::MS * H::META;
    static_assert(H::META % 16 == 0 && H::RAW % 16 == 0, "sections stay aligned");
    const uint32_t raw_full = bars, raw_empty = bars + 16, buf_full = bars + 32, buf_empty = buf_full + 8 * NBUF,
                   s_full = buf_empty + 8 * NBUF, p_full = s_full + 8 * NQ, o_done = p_full + 8 * NQ, q_full = o_done + 8 * NQ,
                   meta_full = q_full + 8, tslot = meta_full + 8 * H::MS, drained = bars + 240, wide = bars + 248;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, H::EW);
        }
        for (int i = 0; i < NBUF; ++i) {
            mbar_init(buf_full + 8 * i, H::EW);
            mbar_init(buf_empty + 8 * i, 1);
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 4);
            mbar_init(o_done + 8 * i, 1);
        }
        for (int i = 0; i < H::MS; ++i) mbar_init(meta_full + 8 * i, 1);
        mbar_init(q_full, 4 * NQ);
        mbar_init(drained, 1);
        sts32(wide, 0u); /* bit w: the rows of softmax warp w are done again */
        mbar_fence_init();
    }
    if (warp == 4 * NQ + H::EW) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tslot), "r"(H::COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kAll, lds32(tslot), 0);
    grid_dep_launch();
    grid_dep_wait();

    /* late row tiles see the most tokens and come first */
    PJob J;
    {
        int i = blockIdx.x;
        const int sp = i % a.splits;
        i /= a.splits;
        J.h = i % a.P.n_heads;
        i /= a.P.n_heads;
        J.b = i % a.S.n_seqs;
        const int rt = a.row_tiles - 1 - i / a.S.n_seqs;
        Seq q = seq_of(a.S, a.P.page_shift, J.b);
        if (q.len > a.max_len) q.len = a.max_len, q.bad = true;
        if (q.m > a.max_new) q.m = a.max_new, q.bad = true;
        if (q.bad && J.h == 0 && sp == 0 && rt == 0 && threadIdx.x == 0) flag_corrupt(a.status);
        J.group = a.group;
        J.len = q.len;
        J.row0 = q.row0;
        J.first = q.len - q.m;
        J.R = q.m * a.group;
        J.r0 = rt * (128 * NQ);
        J.u0 = J.u1 = 0;
        if (J.r0 < J.R) {
            const int pos0 = J.first + J.r0 / a.group, pos1 = J.first + min(J.r0 + 128 * NQ - 1, J.R - 1) / a.group;
            const int all = pos1 < 0 ? 0 : pos1 / kUnit + 1;
            const int64_t lo = a.window ? (int64_t)pos0 - a.window + 1 : 0;
            J.lo_u = lo > 0 ? (int)min(lo / kUnit, (int64_t)all) : 0;
            J.sink_u = min((a.sinks + kUnit - 1) / kUnit, J.lo_u);
            J.units = J.sink_u + all - J.lo_u;
            const int tiles = (J.units + UT - 1) / UT, per = (tiles + a.splits - 1) / a.splits;
            J.u0 = min(J.units, sp * per * UT);
            J.u1 = min(J.units, (sp + 1) * per * UT);
        }
    }
    const int T = __shfl_sync(kAll, (J.u1 - J.u0 + UT - 1) / UT, 0);
    const int NA = __shfl_sync(kAll, min(NQ, (J.R - J.r0 + 127) / 128), 0); /* row tiles that hold rows */
    bool live = true; /* no wait of this warp has run out; its role ends when one has */
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (live && !mbar_wait(bar, parity)) {
            live = false;
            flag_corrupt(a.status);
        }
        __syncwarp();
    };
    auto unit_of = [&](int u) { return u < J.sink_u ? u : u - J.sink_u + J.lo_u; };

    if (J.r0 >= J.R) {
        /* a row tile that this sequence does not have */
    } else if (warp < 4 * NQ) {
        /* ---------------------------------------------------------------- softmax */
        const int t = warp >> 2, q4 = warp & 3, r = J.r0 + 128 * t + 32 * q4 + lane;
        const bool on = r < J.R;
        const uint32_t lanes = (uint32_t)(32 * q4) << 16;
        const uint32_t s_at = tmem + lanes + t * TN, o_at = tmem + lanes + H::O_COL + t * D;
        const int rr = min(r, J.R - 1), pos = J.first + rr / J.group, head = J.h * J.group + rr % J.group;
        const int64_t row = J.row0 + rr / J.group;
        float rowfac;
        /* the row's query: a power of two brings its largest element to [2^14, 2^15) */
        {
            const int64_t off = row * a.q.row + (int64_t)head * a.q.head;
            uint32_t top = 0;
            auto get8 = [&](int d, float (&x)[8]) {
                if (a.q.wide && a.q.dtype == EC_DTYPE_FP32) {
                    const float4 u = *(const float4*)((const float*)a.q.data + off + d), v = *(const float4*)((const float*)a.q.data + off + d + 4);
                    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
                } else if (a.q.wide) {
                    const uint4 w = *(const uint4*)((const uint16_t*)a.q.data + off + d);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (a.q.dtype == EC_DTYPE_FP16) {
                            const float2 f = __half22float2(*(const __half2*)&u[i]);
                            x[2 * i] = f.x, x[2 * i + 1] = f.y;
                        } else x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = load_elem(a.q, off + d + i);
                }
                if (!on)
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = 0.f;
            };
            for (int d = 0; d < D; d += 8) {
                float x[8];
                get8(d, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
            }
            const int E = (int)(top >> 23), up = E == 255 ? 127 : min(253, 268 - E);
            const float s = __uint_as_float((uint32_t)up << 23);
            rowfac = __uint_as_float((uint32_t)(254 - up) << 23) * a.scale * 1.4426950408889634f;
            const int lr = 32 * q4 + lane;
            for (int d = 0; d < D; d += 8) {
                float x[8];
                get8(d, x);
                uint32_t w[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y0 = x[2 * i] * s, y1 = x[2 * i + 1] * s;
                    w[i] = pack_f16(y0, y1);
                    const float2 hi = __half22float2(*(const __half2*)&w[i]);
                    lo[i] = pack_f16(y0 - hi.x, y1 - hi.y);
                }
                const uint32_t at = q_at + t * QT * H::QBYTES + (d >> 6) * (128 * 128) + lr * 128 + ((((d >> 3) & 7) ^ (lr & 7)) << 4);
                sts128(at, w[0], w[1], w[2], w[3]);
                if constexpr (QT == 2) sts128(at + H::QBYTES, lo[0], lo[1], lo[2], lo[3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }

        float m = 0.f, l = 0.f;
        bool set = false; /* the row has seen a token: m is its reference */
        uint32_t nan_blocks = 0;
        const int pos_lo = __shfl_sync(kAll, pos, 0), pos_hi = __shfl_sync(kAll, pos, 31);

        for (int j = 0; j < (t < NA ? T : 0); ++j) {
            const uint32_t meta = meta_at + j % H::MS * H::META;
            wait(meta_full + 8 * (j % H::MS), (j / H::MS) & 1);
            wait(s_full + 8 * t, j & 1);
            if (!live) break;
            tc_fence_after();
            const float f = fmaxf(rowfac * __uint_as_float((lds32(meta) - 13u) << 23), kTiny); /* > 0: a masked -inf stays one */
            const uint32_t flags = lds32(meta + 4);
            const int ut = J.u0 + j * UT; /* the tile's first unit */
            const int tok_a = unit_of(ut) * kUnit, tok_z = unit_of(min(ut + UT, J.u1) - 1) * kUnit + kUnit - 1;
            const bool all = ut + UT <= J.u1 && tok_z <= pos_lo &&
                             (!a.window || tok_a > pos_hi - a.window || tok_z < a.sinks);
            /* scores of 32 columns; a place that the row does not see is -inf */
            auto mask_of = [&](int u) { /* tokens of a unit that the row sees */
                if (u >= J.u1) return 0u;
                const int tok = unit_of(u) * kUnit, last = pos - tok;
                uint32_t w = last < 0 ? 0u : last >= 15 ? 0xFFFFu : (2u << last) - 1u;
                if (a.window) {
                    const int gone = last - a.window + 1; /* the first `gone` tokens lie before the window, */
                    uint32_t x = gone <= 0 ? 0xFFFFu : gone >= 16 ? 0u : 0xFFFFu << gone;
                    const int keep = a.sinks - tok;       /* but the first `keep` stay */
                    x |= keep <= 0 ? 0u : keep >= 16 ? 0xFFFFu : (1u << keep) - 1u;
                    w &= x;
                }
                return w;
            };
            auto hide = [&](int k, uint32_t (&v)[32]) {
                const uint32_t w = mask_of(ut + 2 * k) | mask_of(ut + 2 * k + 1) << 16;
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = w >> i & 1u ? v[i] : 0xFF800000u;
            };
            /* (the loops stay rolled: with five roles side by side the instruction cache decides;
             * unrolled they took 2.2 times as long) */
            float mx = -INFINITY;
            if (all) {
#pragma unroll 1
                for (int k = 0; k < TN / 32; k += 2) {
                    uint32_t va[32], vb[32];
                    float ma, mb;
                    tc_ld32_max(s_at + 32 * k, va, ma);
                    tc_ld32_max(s_at + 32 * k + 32, vb, mb);
                    tc_wait_ld(ma, mb);
                    mx = fmaxf(mx, fmaxf(ma, mb));
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < TN / 32; ++k) {
                    uint32_t v[32];
                    tc_ld32(s_at + 32 * k, v);
                    tc_wait_ld(v);
                    hide(k, v);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) mx = fmaxf(mx, fmaxf(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
                }
            }
            mx *= f; /* f > 0 */
            if (__any_sync(kAll, mx > m + kPSlack || (!set && mx > -INFINITY)) || (flags & 4u)) {
                /* references move: the accumulators follow once the products before are done */
                const float nm = set ? fmaxf(m, mx) : mx > -INFINITY ? mx : 0.f, al = set ? ex2(m - nm) : 0.f;
                set |= mx > -INFINITY;
                if (fabsf(nm) > kMost) atomicOr((uint32_t*)__cvta_shared_to_generic(wide), 1u << warp);
                if (j > 0) {
                    wait(o_done + 8 * t, (j - 1) & 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < NB; ++k) {
                        uint32_t v[32];
                        tc_ld32(o_at + 32 * k, v);
                        tc_wait_ld(v);
                        const float fk = al * __uint_as_float(lds32(meta + 48 + 4 * k));
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * fk);
                        tc_st32(o_at + 32 * k, v);
                    }
                    tc_wait_st();
                }
                m = nm;
                l *= al;
            }
            /* weights 2^(s - m + kPBias) take the scores' place, behind the reads */
            const float off = kPBias - m;
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int k = 0; k < TN / 32; ++k) {
                uint32_t v[32], p[16];
                tc_ld32(s_at + 32 * k, v);
                tc_wait_ld(v);
                if (!all) hide(k, v);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 y = fma2(v[i], v[i + 1], f, off);
                    const float p0 = ex2(y.x), p1 = ex2(y.y);
                    acc = add2(acc, p0, p1);
                    p[i / 2] = pack_f16(p0, p1);
                }
                tc_st16(s_at + 16 * k, p);
            }
            l += acc.x + acc.y;
            tc_wait_st();
            tc_fence_before();
            if (flags & 1u) { /* tokens with NaN values: their blocks are NaN for the rows that see them */
                for (int i = 0; i < TN; ++i) {
                    const int u = ut + (i >> 4);
                    if (u >= J.u1) break;
                    const uint32_t w = lds8(meta + 80 + i);
                    const int tok = unit_of(u) * kUnit + (i & 15);
                    if (w && tok <= pos && (!a.window || tok > pos - a.window || tok < a.sinks)) nan_blocks |= w;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 8 * t);
        }

        /* outputs */
        if (t < NA && T > 0) {
            wait(o_done + 8 * t, (T - 1) & 1);
            tc_fence_after();
        }
        __syncwarp();
        const bool redo = lds32(wide) >> warp & 1u; /* nothing is written over queries that are still to be read, should out be q */
        const float inv = a.splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
        float* part = a.part + ((int64_t)blockIdx.x * NQ + t) * (128 * (D + 2));
#pragma unroll 1
        for (int k = 0; k < NB; ++k) {
            uint32_t v[32];
            const int vr = T > 0 ? (int)lds32(meta_at + (T - 1) % H::MS * H::META + 16 + 4 * k) : 0;
            const float back = vr > 0 ? __uint_as_float((uint32_t)vr << 23) : 0.f;
            if (t < NA && T > 0) {
                tc_ld32(o_at + 32 * k, v);
                tc_wait_ld(v);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0;
            }
            const bool nan = nan_blocks >> k & 1u;
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = nan ? __uint_as_float(0x7FC00000u) : __uint_as_float(v[i]) * back * inv;
            if (!on || redo) continue;
            if (a.splits > 1) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *(float4*)&part[(32 * q4 + lane) * D + 32 * k + i] = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            } else {
                const int64_t off = row * a.out.row + (int64_t)head * a.out.head + 32 * k;
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    const float y[8] = {x[i], x[i + 1], x[i + 2], x[i + 3], x[i + 4], x[i + 5], x[i + 6], x[i + 7]};
                    store8(a.out, off + i, y);
                }
            }
        }
        if (on && !redo) {
            if (a.splits > 1) {
                part[128 * D + 32 * q4 + lane] = set || !(l == 0.f) ? m : -FLT_MAX;
                part[128 * D + 128 + 32 * q4 + lane] = l;
            } else if (a.lse) a.lse[row * a.n_q_heads + head] = l == 0.f ? -INFINITY : (m - kPBias + log2f(l)) * 0.6931471805599453f;
        }
    } else if (warp < 4 * NQ + H::EW) {
        /* ---------------------------------------------------------------- expansion */
        /* warp w takes the units w, w + 4 of a tile */
        const int we = warp - 4 * NQ;
        /* which words a lane takes of the keys: rows q and q + 4 share a quarter of the warp, so
         * that its eight 16-byte stores fall into eight different bank groups */
        const int kg = (lane >> 3) + 4 * ((lane >> 2) & 1), kl = kg * 4 + c;
        int n = 0; /* tiles expanded: keys 2 j, values 2 j + 1 */
        for (int j = 0; j < T; ++j) {
            const int rs = j % H::RS, ut = J.u0 + j * UT;
            const uint32_t raw = raw_at + rs * H::RAW, meta = meta_at + j % H::MS * H::META;
            wait(raw_full + 8 * rs, (j / H::RS) & 1);
            wait(meta_full + 8 * (j % H::MS), (j / H::MS) & 1);
            const uint32_t flags = lds32(meta + 4); /* bit 0: NaN values, bit 1: NaN keys */
            {
                const int buf = n % NBUF;
                const uint32_t add = both_halves(28 - (int)lds32(meta));
                wait(buf_empty + 8 * buf, ((n / NBUF) & 1) ^ 1u);
                if (!live) break;
#pragma unroll 1
                for (int u = we; u < UT; u += 4) {
                    const uint32_t src = raw + u * UB;
                    /* a row's 16-byte chunk 4 b + c goes to chunk (4 b + c) ^ (row % 8) of its 128 bytes */
                    const uint32_t dst = buf_at + buf * H::BUF + (u * kUnit + kg) * 128;
                    const uint32_t even = dst + ((c ^ kg) << 4), odd = dst + (((4 + c) ^ kg) << 4);
#pragma unroll 1
                    for (int i = 0; i < NB / 2; ++i) {
                        const uint4 wv = lds128(src + i * 512 + kl * 16);
                        uint32_t e2[2]; /* scales of blocks 2 i, 2 i + 1, tokens kg and kg + 8 */
                        e2[0] = lds16(src + 16 * D + kg * NB + 2 * i);
                        e2[1] = lds16(src + 16 * D + (kg + 8) * NB + 2 * i);
                        const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
                        for (int r = 0; r < 2; ++r)
#pragma unroll
                            for (int bb = 0; bb < 2; ++bb) {
                                /* 2^(e - kref + 13) in both halves, 0 below 2^-27 of the largest */
                                uint32_t sc = __viaddmax_s16x2(__byte_perm(e2[r], 0, bb ? 0x4141 : 0x4040), add, 0u) * 1024u;
                                if ((flags & 2u) && ((e2[r] >> (8 * bb)) & 0xFFu) == 255u) sc = 0x7E007E00u;
                                uint32_t h4[4];
                                e2m1x8_f16(ww[2 * bb + r], h4);
                                sts128((bb ? odd : even) + i * (TN * 128) + r * 1024, hmul2(h4[0], sc), hmul2(h4[1], sc),
                                       hmul2(h4[2], sc), hmul2(h4[3], sc));
                            }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(buf_full + 8 * buf);
                ++n;
            }
            {
                const int buf = n % NBUF;
                wait(buf_empty + 8 * buf, ((n / NBUF) & 1) ^ 1u);
                if (!live) break;
#pragma unroll 1
                for (int u = we; u < UT; u += 4) {
                    const uint32_t src = raw + u * UB;
                    const int nv = ut + u < J.u1 ? min(kUnit, J.len - unit_of(ut + u) * kUnit) : 0; /* tokens of the unit that hold something */
                    /* channel d's row: tokens 16 u + 8 p + 2 c, + 1 are 4 bytes of chunk 2 u + p */
                    const uint32_t dst = buf_at + buf * H::BUF + (u >> 2) * (D * 128) + g * 128 + 4 * c;
                    const uint32_t at0 = dst + (((2 * (u & 3)) ^ g) << 4), at1 = dst + (((2 * (u & 3) + 1) ^ g) << 4);
                    const bool odd = (flags & 1u) || nv < kUnit;
#pragma unroll 1
                    for (int i4 = 0; i4 < NB / 2; ++i4) {
                        const uint4 wv = lds128(src + 8 * D + i4 * 512 + lane * 16);
                        uint32_t x[2], v[2], s0[2], s1[2];
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(src + 16 * D + D / 2 + (c * NB + 2 * i4) * 4) : "memory");
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(meta + 16 + 8 * i4) : "memory");
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (odd) { /* scales of NaN blocks (their codes are zeros) and of tokens that hold nothing */
                                x[k] = drop_nan(x[k]);
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    if (2 * c + (q & 1) + 8 * (q >> 1) >= nv) x[k] &= ~(0xFFu << (8 * q));
                            }
                            /* 2^(e - vref): 0 below 2^-14, at most 2^13 by the choice of vref */
                            const uint32_t add = both_halves(15 - (int)v[k]);
                            s0[k] = __viaddmax_s16x2(__byte_perm(x[k], 0, 0x4140), add, 0u) * 1024u;
                            s1[k] = __viaddmax_s16x2(__byte_perm(x[k], 0, 0x4342), add, 0u) * 1024u;
                            if (odd) { /* with vref < 15 a scale byte of 0 is no zero: the codes of nothing must not count */
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    if (2 * c + q >= nv) s0[k] &= ~(0xFFFFu << (16 * q));
                                    if (2 * c + q + 8 >= nv) s1[k] &= ~(0xFFFFu << (16 * q));
                                }
                            }
                        }
                        const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) { /* channels 16 (4 i4 + i) .. + 15: block 2 i4 + i / 2 */
                            uint32_t h4[4]; /* byte r + 2 p: channel 8 r + g of them */
                            e2m1x8_f16(ww[i], h4);
                            const uint32_t o = (64 * i4 + 16 * i) * 128;
                            sts32(at0 + o, hmul2(h4[0], s0[i / 2]));
                            sts32(at0 + o + 1024, hmul2(h4[1], s0[i / 2]));
                            sts32(at1 + o, hmul2(h4[2], s1[i / 2]));
                            sts32(at1 + o + 1024, hmul2(h4[3], s1[i / 2]));
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(buf_full + 8 * buf);
                    mbar_arrive(raw_empty + 8 * rs);
                }
                ++n;
            }
        }
    } else if (warp == 4 * NQ + H::EW) {
        /* ---------------------------------------------------------------- matrix instructions */
        if (T > 0) {
            /* kind::f16, FP32 accumulators, FP16 operands, both K-major: N / 8 at bit 17, M / 16 at bit 24 */
            const uint32_t id_s = (1u << 4) | ((uint32_t)(TN / 8) << 17) | (8u << 24), id_o = (1u << 4) | ((uint32_t)(D / 8) << 17) | (8u << 24);
            auto scores = [&](int t, int kb) {
                uint64_t qa = sw128_desc(q_at + t * QT * H::QBYTES);
#pragma unroll 1
                for (int x = 0; x < QT; ++x) {
                    uint64_t ka = sw128_desc(buf_at + kb * H::BUF);
#pragma unroll 1
                    for (int k = 0; k < D / 64; ++k) {
                        tc_mma4_ss(tmem + t * TN, qa, ka, id_s, x + k);
                        qa += (128 * 128) >> 4;
                        ka += (TN * 128) >> 4;
                    }
                }
            };
            auto values = [&](int t, int vb, int j) {
                uint64_t va = sw128_desc(buf_at + vb * H::BUF);
#pragma unroll 1
                for (int k = 0; k < TN / 64; ++k) {
                    tc_mma4_ts(tmem + H::O_COL + t * D, tmem + t * TN + 32 * k, va, id_o, j + k);
                    va += (D * 128) >> 4;
                }
            };
            wait(q_full, 0);
            wait(buf_full, 0);
            tc_fence_after();
#pragma unroll 1
            for (int t = 0; t < NA && live; ++t) {
                scores(t, 0);
                tc_commit(s_full + 8 * t);
            }
            tc_commit(buf_empty);
            for (int j = 0; j < T && live; ++j) {
                const int vn = 2 * j + 1, kn = 2 * j + 2, vb = vn % NBUF, kb = kn % NBUF;
                wait(buf_full + 8 * vb, (vn / NBUF) & 1);
#pragma unroll 1
                for (int t = 0; t < NA; ++t) {
                    wait(p_full + 8 * t, j & 1);
                    if (!live) break;
                    tc_fence_after();
                    values(t, vb, j);
                    tc_commit(o_done + 8 * t);
                    if (t == NA - 1) tc_commit(buf_empty + 8 * vb);
                    if (j + 1 < T) {
                        if (t == 0) {
                            wait(buf_full + 8 * kb, (kn / NBUF) & 1);
                            tc_fence_after();
                        }
                        /* the scores take the weights' place: not before their product is done
                         * (products of other shapes and accumulators may overtake it) */
                        wait(o_done + 8 * t, j & 1);
                        if (!live) break;
                        scores(t, kb);
                        tc_commit(s_full + 8 * t);
                        if (t == NA - 1) tc_commit(buf_empty + 8 * kb);
                    }
                }
            }
            /* nothing is in flight when the tensor memory is given back, whatever ran out */
            tc_commit(drained);
            mbar_wait(drained, 0);
        }
        __syncwarp();
    } else if (warp == 4 * NQ + H::EW + 1) {
        /* ---------------------------------------------------------------- copies */
        int j = 0;
        for (; j < T; ++j) {
            const int s = j % H::RS, ut = J.u0 + j * UT, have = min(UT, J.u1 - ut);
            int page = 0, unit = 0;
            if (lane < have) {
                unit = unit_of(ut + lane);
                page = a.S.table[(int64_t)J.b * a.S.table_stride + (unit >> (a.P.page_shift - 4))];
                if (page < 0 || page >= a.P.n_pages) {
                    page = 0;
                    flag_corrupt(a.status);
                }
            }
            const uint8_t* src = page_ptr(a.P, page, J.h, unit & ((1 << (a.P.page_shift - 4)) - 1));
            wait(raw_empty + 8 * s, ((j / H::RS) & 1) ^ 1u);
            if (!live) break;
            if (lane == 0) mbar_arrive_tx(raw_full + 8 * s, have * UB);
            __syncwarp();
            if (lane < have) bulk_g2s(raw_at + s * H::RAW + lane * UB, src, UB, raw_full + 8 * s);
        }
        for (int i = max(0, j - H::RS); i < j; ++i) mbar_wait(raw_full + 8 * (i % H::RS), (i / H::RS) & 1); /* nor any copy */
    } else if (warp == 4 * NQ + H::EW + 2) {
        /* ---------------------------------------------------------------- references */
        constexpr int WU = 4 * NB;             /* words of scales per unit, keys' or values' */
        constexpr int LANES = 32 / NB * NB;    /* lanes that stride whole blocks: word i of the values' is of block i % NB */
        constexpr int PER = (UT * WU + LANES - 1) / LANES;
        int vref = 0, first = 0; /* lane: of block lane % NB, now and when it was set (0: not yet) */
        uint32_t kl = 0xFFFFFFFFu; /* of all keys; kmost the largest kref */
        int kmost = 0;
        bool far = false;
        for (int j = 0; j < T; ++j) {
            const int s = j % H::RS, ut = J.u0 + j * UT, have = min(UT, J.u1 - ut);
            const uint32_t raw = raw_at + s * H::RAW, meta = meta_at + j % H::MS * H::META;
            wait(raw_full + 8 * s, (j / H::RS) & 1);
            if (!live) break;
            const int last = ut + have >= J.units ? min(kUnit, J.len - unit_of(ut + have - 1) * kUnit) : kUnit; /* tokens of the last unit */
            uint32_t kw[PER], vw[PER];
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                const int i = lane + q * LANES, v = i / WU;
                kw[q] = vw[q] = 0;
                if (lane < LANES && v < have) {
                    const uint32_t at = raw + v * UB + 16 * D + 4 * (i % WU);
                    kw[q] = lds32(at);
                    vw[q] = lds32(at + D / 2);
                }
            }
            if (last < kUnit) { /* scales past the sequence's end are none */
#pragma unroll
                for (int q = 0; q < PER; ++q) {
                    const int i = lane + q * LANES, k = i % WU;
                    if (i / WU != have - 1) continue;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        if ((4 * k + x) / NB >= last) kw[q] &= ~(0xFFu << (8 * x));
                        if (2 * (k / NB) + (x & 1) + 8 * (x >> 1) >= last) vw[q] &= ~(0xFFu << (8 * x));
                    }
                }
            }
            uint32_t km = 0, vm = 0, vl = 0xFFFFFFFFu;
#pragma unroll
            for (int q = 0; q < PER; ++q) km = bytes_max(km, kw[q]), vm = bytes_max(vm, vw[q]), vl = bytes_min(vl, vw[q]);
            uint32_t flags = 0;
            if (__any_sync(kAll, half_max(km) == 255 || half_max(vm) == 255)) {
                flags = (__any_sync(kAll, half_max(vm) == 255) ? 1u : 0u) | (__any_sync(kAll, half_max(km) == 255) ? 2u : 0u);
                km = vm = 0;
#pragma unroll
                for (int q = 0; q < PER; ++q) km = bytes_max(km, drop_nan(kw[q])), vm = bytes_max(vm, drop_nan(vw[q]));
            }
            const int kref = max(16, __reduce_max_sync(kAll, half_max(km)));
            int best = half_max(vm), least = half_min(vl);
            if constexpr (32 % NB == 0) {
#pragma unroll
                for (int o = NB; o < 32; o <<= 1) {
                    best = max(best, __shfl_xor_sync(kAll, best, o));
                    least = min(least, __shfl_xor_sync(kAll, least, o));
                }
            } else {
                const int mine = best, low = least;
#pragma unroll
                for (int k = 0; k < LANES / NB; ++k) {
                    best = max(best, __shfl_sync(kAll, mine, lane % NB + k * NB));
                    least = min(least, __shfl_sync(kAll, low, lane % NB + k * NB));
                }
            }
            const int was = vref;
            if (best > 0 && (vref == 0 || best > vref + kVUp || least < vref - kVDown)) {
                vref = best - least <= kVDown ? best : max(best - kVUp, 1);
                if (first == 0) first = vref;
                far |= best - least > kVUp + kVDown || abs(vref - first) > kVSpan;
            }
            if (__any_sync(kAll, was != 0 && was != vref)) flags |= 4u;
            if (lane == 0) {
                sts32(meta, (uint32_t)kref);
                sts32(meta + 4, flags);
            }
            if (lane < NB) {
                sts32(meta + 16 + 4 * lane, (uint32_t)vref);
                sts32(meta + 48 + 4 * lane, __float_as_uint(was ? ex2((float)(was - vref)) : 1.f));
            }
            if (flags & 1u) { /* which blocks of which tokens are NaN */
                for (int i = lane; i < TN; i += 32) {
                    const int v = i >> 4, tk = i & 15;
                    uint32_t mask = 0;
                    if (v < have && (v < have - 1 || tk < last))
                        for (int k = 0; k < NB; ++k)
                            if (lds8(raw + v * UB + 16 * D + D / 2 + ((((tk >> 1) & 3) * NB + k) * 2 + (tk >> 3)) * 2 + (tk & 1)) == 255u)
                                mask |= 1u << k;
                    sts8(meta + 80 + i, mask);
                }
            }
            __syncwarp();
            /* (behind the arrival, where nobody waits for it: ahead of it this cost 29 us of 1146; but
             * the last tile's waiters learn whether the rows are done again) */
            if (lane == 0 && j + 1 < T) mbar_arrive(meta_full + 8 * (j % H::MS));
#pragma unroll
            for (int q = 0; q < PER; ++q) kl = bytes_min(kl, kw[q]);
            kmost = max(kmost, kref);
        }
        if (far || half_min(kl) < kmost - 27) sts32(wide, ~0u);
        __syncwarp();
        if (lane == 0 && T > 0) mbar_arrive(meta_full + 8 * ((T - 1) % H::MS));
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4 * NQ + H::EW) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(H::COLS) : "memory");
    }
    if (lds32(wide)) {
#pragma unroll 1
        for (int i = warp; i < min(128 * NQ, J.R - J.r0); i += H::WARPS) {
            if (!(lds32(wide) >> (i / 32) & 1u)) continue;
            const int t = (J.r0 + i) / J.group;
            const RowJob row{J.b, J.h, J.h * J.group + (J.r0 + i) % J.group, J.first + t, J.sink_u, J.lo_u, J.u0, J.u1, J.row0 + t};
            float* part = a.part + ((int64_t)blockIdx.x * NQ + i / 128) * (128 * (D + 2)) + 128 * D + i % 128;
            wide_row<NB>(a, row, kPBias, a.splits > 1 ? part - 128 * D - i % 128 + i % 128 * D : nullptr, part, part + 128);
        }
    }
}

/* Join the splits of a row tile: one warp per row. */
template <int NB, int NQ>
__global__ void __launch_bounds__(256) kv_prefill_join_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int D = 32 * NB, PS = 128 * (D + 2);
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * 8 + warp; /* row r of tile: (((rt, b), h), row) */
    int64_t i = item / (128 * NQ);
    const int lr = (int)(item % (128 * NQ));
    const int64_t tile = i;
    const int h = (int)(i % a.P.n_heads);
    i /= a.P.n_heads;
    const int b = (int)(i % a.S.n_seqs);
    const int64_t rt = a.row_tiles - 1 - i / a.S.n_seqs;
    if (rt < 0) return;
    const Seq q = seq_of(a.S, a.P.page_shift, b);
    const int64_t r = rt * (128 * NQ) + lr;
    if (r >= (int64_t)min(q.m, a.max_new) * a.group) return;
    const float* p0 = a.part + (tile * a.splits * NQ + lr / 128) * PS;
    float M = -FLT_MAX;
    for (int s = 0; s < a.splits; ++s) M = fmaxf(M, p0[(int64_t)s * NQ * PS + 128 * D + lr % 128]);
    float L = 0.f, v[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) v[k] = 0.f;
    for (int s = 0; s < a.splits; ++s) {
        const float* p = p0 + (int64_t)s * NQ * PS;
        const float w = ex2(p[128 * D + lr % 128] - M);
        L = fmaf(p[128 * D + 128 + lr % 128], w, L);
#pragma unroll
        for (int k = 0; k < NB; ++k) v[k] = fmaf(p[(int64_t)(lr % 128) * D + 32 * k + lane], w, v[k]);
    }
    const int64_t row = q.row0 + r / a.group;
    const int head = h * a.group + (int)(r % a.group);
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int k = 0; k < NB; ++k) store_elem(a.out, row * a.out.row + (int64_t)head * a.out.head + 32 * k + lane, v[k] * inv);
    if (lane == 0 && a.lse) a.lse[row * a.n_q_heads + head] = L == 0.f ? -INFINITY : (M - kPBias + log2f(L)) * 0.6931471805599453f;
}

/* ------------------------------------------------------------ launch */
template <int NB, int NQ, int QT>
static int run_prefill(AttnArgs a, const PrefillPlan& p, cudaStream_t stream) {
    using H = PShape<NB, NQ, QT>;
    static SmemOnce once;
    int rc = once.set(kv_prefill_kernel<NB, NQ, QT>, H::SMEM);
    if (rc != EC_OK) return rc;
    a.splits = p.splits;
    a.row_tiles = p.row_tiles;
    rc = launch(kv_prefill_kernel<NB, NQ, QT>, dim3((unsigned)p.grid), H::WARPS * 32, H::SMEM, stream, a);
    if (rc == EC_OK && p.splits > 1)
        rc = launch(kv_prefill_join_kernel<NB, NQ>, dim3((unsigned)(p.grid / p.splits * 16 * NQ)), 256, 0, stream, a);
    return rc;
}

/* Two row tiles per CTA for FP16 and BF16 queries of up to 128 channels.  (64 channels with FP32
 * queries and 192 with 16-bit ones would fit shared and tensor memory too; not measured.) */
static int row_tiles_per_cta(int nb, int dtype) { return nb <= 4 && dtype != EC_DTYPE_FP32 ? 2 : 1; }

bool plan_prefill(const ec_kv* C, int sms, int n_seqs, int max_new, int64_t max_units, int group, int dtype, PrefillPlan* p) {
    const int nb = C->p.head_dim / 32, nq = row_tiles_per_cta(nb, dtype), ut = nb <= 4 ? 8 : 4;
    const int64_t rows = (int64_t)group * max_new;
    if (rows > 0x7FFFFFFF - 255) return false; /* the kernel's row numbers, rounded up to a tile, are 32-bit */
    const int64_t rt = (rows + 128 * nq - 1) / (128 * nq), tiles = rt * n_seqs * C->p.n_kv_heads;
    const int64_t steps = (max_units + ut - 1) / ut, finest = (steps + 3) / 4;
    int64_t s = 1;
    /* fewer row tiles than SMs: split the tokens, no finer than 4 tiles each */
    if (tiles < sms) s = sms / tiles;
    if (s > finest) s = finest;
    if (s < 1) s = 1;
    if (tiles * s > 0x7FFFFFF || tiles * 16 * nq > 0x7FFFFFFF) return false;
    p->row_tiles = (int)rt;
    p->splits = (int)s;
    p->grid = tiles * s;
    const size_t part = (size_t)nq * 128 * (C->p.head_dim + 2) * sizeof(float);
    const int64_t most = tiles < (sms + finest - 1) / finest ? tiles * finest : sms;
    p->work = s > 1 ? tiles * s * part : 0;
    p->most = finest > 1 ? most * part : 0;
    return true;
}

int launch_prefill(const AttnArgs& a, const PrefillPlan& p, cudaStream_t stream) {
    const bool two = a.q.dtype == EC_DTYPE_FP32;
    switch (a.P.dim / 32) {
        case 2: return two ? run_prefill<2, 1, 2>(a, p, stream) : run_prefill<2, 2, 1>(a, p, stream);
        case 4: return two ? run_prefill<4, 1, 2>(a, p, stream) : run_prefill<4, 2, 1>(a, p, stream);
        case 6: return two ? run_prefill<6, 1, 2>(a, p, stream) : run_prefill<6, 1, 1>(a, p, stream);
        default: return two ? run_prefill<8, 1, 2>(a, p, stream) : run_prefill<8, 1, 1>(a, p, stream);
    }
}

}  // namespace kv
