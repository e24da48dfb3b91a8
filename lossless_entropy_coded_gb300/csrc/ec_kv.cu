/*
 * ec_kv.cu -- the paged 4-bit key/value cache: its descriptor, quantising new tokens
 * into pages (ec_kv_append), reading values back (ec_kv_read), and the page operations
 * (ec_kv_fork, ec_kv_compact).  The format and the contracts are in ec.h.
 */
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "ec_kv_internal.h"

namespace kv {

/* ============================================================ host helpers */
bool use_pdl() {
    static const bool on = [] {
        const char* e = std::getenv("EC_NO_PDL");
        return !(e && e[0] == '1');
    }();
    return on;
}

int device_of(const ec_kv* C, Device* out) {
    if (!C->pool) return EC_ERR_INVALID_ARG;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return EC_ERR_CUDA;
    if (dev != C->device) return EC_ERR_INVALID_ARG;
    static std::mutex mu;
    static std::vector<int> sms;
    {
        std::lock_guard<std::mutex> lk(mu);
        if ((int)sms.size() <= dev) sms.resize(dev + 1, 0);
        if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            sms[dev] = 0;
            return EC_ERR_CUDA;
        }
        out->sms = sms[dev];
    }
    return ec_internal_status_ptr(dev, &out->status);
}

static int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

bool pool_view(const ec_kv* C, int layer, Pool* o) {
    const ec_kv_params& p = C->p;
    if (layer < 0 || layer >= p.n_layers) return false;
    o->base = C->pool;
    o->dim = p.head_dim;
    o->n_heads = p.n_kv_heads;
    o->n_pages = (int32_t)p.n_pages;
    o->page_shift = log2_of(p.page_tokens);
    o->unit_bytes = 17 * p.head_dim;
    o->head_bytes = (int64_t)o->unit_bytes * (p.page_tokens / kUnit);
    o->layer_off = o->head_bytes * p.n_kv_heads * layer;
    o->page_bytes = o->head_bytes * p.n_kv_heads * p.n_layers;
    return true;
}

int check_seqs(const ec_kv_seqs* S) {
    if (S->n_seqs < 0 || S->table_stride < 0) return EC_ERR_SHAPE;
    if (S->n_seqs > EC_KV_MAX_SEQS) return EC_ERR_UNSUPPORTED;
    if (S->table_stride > (int64_t(1) << 26)) return EC_ERR_UNSUPPORTED;
    if (S->n_seqs > 0 && (!S->lens || (S->table_stride > 0 && !S->table))) return EC_ERR_INVALID_ARG;
    return EC_OK;
}

int check_rows(const ec_kv_rows* r, int heads, int64_t n_rows, Rows* o) {
    int size = 0;
    if (r->dtype == EC_DTYPE_FP32) size = 4;
    else if (r->dtype == EC_DTYPE_BF16 || r->dtype == EC_DTYPE_FP16) size = 2;
    else return EC_ERR_INVALID_ARG;
    if (n_rows < 0) return EC_ERR_SHAPE;
    if (r->row_stride < 0 || r->head_stride < 0) return EC_ERR_SHAPE;
    /* the last element's offset in bytes fits 62 bits */
    const int64_t lim = int64_t(1) << 60;
    if (n_rows > 1 && r->row_stride > lim / (n_rows - 1)) return EC_ERR_OVERFLOW;
    if (heads > 1 && r->head_stride > lim / (heads - 1)) return EC_ERR_OVERFLOW;
    if (n_rows > 0 && (!r->data || (uintptr_t)r->data % size)) return EC_ERR_INVALID_ARG;
    o->data = r->data;
    o->row = r->row_stride;
    o->head = r->head_stride;
    o->dtype = r->dtype;
    o->wide = ((uintptr_t)r->data % 16 == 0 && r->row_stride * size % 16 == 0 && r->head_stride * size % 16 == 0) ? 1 : 0;
    return EC_OK;
}

/* The checks that every call on new tokens makes; *go = false when there is nothing to do. */
static int check_call(const ec_kv* C, int layer, const ec_kv_seqs* seqs, const int32_t* starts, int64_t n_rows,
                      int max_new, Pool* P, Seqs* S, bool* go) {
    int rc = check_seqs(seqs);
    if (rc != EC_OK) return rc;
    if (!pool_view(C, layer, P)) return EC_ERR_INVALID_ARG;
    if (n_rows < 0 || max_new < 0) return EC_ERR_SHAPE;
    if (max_new > (1 << 24)) return EC_ERR_UNSUPPORTED;
    if (!starts && n_rows < seqs->n_seqs) return EC_ERR_SHAPE;
    S->table = seqs->table;
    S->lens = seqs->lens;
    S->starts = starts;
    S->table_stride = seqs->table_stride;
    S->n_rows = n_rows;
    S->n_seqs = seqs->n_seqs;
    *go = seqs->n_seqs > 0 && n_rows > 0 && max_new > 0;
    return EC_OK;
}

/* ============================================================ append and read */
/* One warp owns the keys, another the values of a unit of 16 tokens of one head, so nothing
 * else writes its bytes and a token's nibbles can share bytes with its neighbour's.  Lane
 * 4 g + c takes channels 32 b + 8 c + 0..7 of tokens g and g + 8: a quad of lanes holds a
 * block, whose largest magnitude takes two shuffles, and the eight codes are one word.
 *
 * A word of the keys is a word of the unit: it is stored as it is.  A word of the values
 * holds 2 channels of 4 tokens; lanes 4 apart (the tokens of a pair) and 1 apart (channels
 * 8 apart) exchange halves: with own words w0, w1 (tokens g, g + 8)
 *   pair step     lane with g even keeps channels 0..3 of both tokens, g odd 4..7: a byte
 *                 per channel, the even token in the low nibble; x[p] for p = 0, 1
 *   channel step  lane with c even keeps the first two of its four channels, c odd the last
 *                 two, of both lanes: bytes (r, p) of two words, r = c % 2
 * which land at words i = 2 b + c / 2 of lanes 4 (4 (g % 2) + k) + g / 2, k = 2 (c % 2), + 1.
 * Reading runs the same steps backwards.
 *
 * Every byte moves once; all loads of a warp are issued before the first is used.  The floor
 * is HBM, the integer pipe (magnitudes, conversions, exchanges) is next: 65 % busy.  18900
 * rows of 8 heads x 128 channels in BF16: append 21 us, read 17 us back to back, 39.6 us
 * together for 196 MB (4.95 TB/s); 64 single tokens take 8.3 us for both, which is the
 * latency of lens, table and rows, one after the other. */
constexpr int kIoWarps = 4;

struct IoArgs {
    Pool P;
    Seqs S;
    Rows k, v;
    int32_t has_k, has_v;
    int32_t units;       /* units that max_new tokens can touch */
    int32_t max_new;
    int* status;
};

/* Which unit of which head a warp works on. */
struct UnitJob {
    int b, h, which, unit, tok0;  /* sequence, head, keys (0) or values (1), unit of the sequence, token of its first place */
    int u;                        /* unit among those that the call can touch */
    int64_t row0;                 /* dense row of token tok0 (may lie before the first) */
    int lo, hi;                   /* places of the unit that the call covers */
    bool in, any;
    Seq q;
};

__device__ __forceinline__ UnitJob unit_job(const IoArgs& a) {
    UnitJob j;
    const int64_t item = (int64_t)blockIdx.x * kIoWarps + (threadIdx.x >> 5);
    j.which = (int)(item & 1);
    const uint32_t r = (uint32_t)(item >> 1), rh = r / (uint32_t)a.P.n_heads; /* fewer than 2^31 items */
    j.h = (int)(r - rh * (uint32_t)a.P.n_heads);
    j.b = (int)(rh / (uint32_t)a.units);
    j.u = (int)(rh - (uint32_t)j.b * (uint32_t)a.units);
    j.in = j.b < a.S.n_seqs;
    j.any = false;
    if (!j.in) return j;
    j.q = seq_of(a.S, a.P.page_shift, j.b);
    if ((j.q.bad || j.q.m > a.max_new) && j.u == 0 && j.h == 0 && (threadIdx.x & 31) == 0) flag_corrupt(a.status);
    const int first = j.q.len - j.q.m; /* position of the first new token; < 0: rows without a token */
    const int f = first < 0 ? 0 : first;
    j.unit = f / kUnit + j.u;
    const bool past = j.unit >= 1 << 27; /* of 2^31 tokens */
    j.tok0 = past ? 0 : j.unit * kUnit;
    j.lo = f - j.tok0 > 0 ? f - j.tok0 : 0;
    j.hi = j.q.len - j.tok0 < kUnit ? j.q.len - j.tok0 : kUnit;
    j.row0 = j.q.row0 + (j.tok0 - first);
    j.any = !past && j.hi > j.lo && !(j.which == 0 ? !a.has_k : !a.has_v);
    return j;
}

__device__ __forceinline__ int32_t page_at(const IoArgs& a, const UnitJob& j) {
    return a.S.table[(int64_t)j.b * a.S.table_stride + (j.tok0 >> a.P.page_shift)];
}
__device__ __forceinline__ uint8_t* unit_ptr(const IoArgs& a, const UnitJob& j, int32_t page) {
    if (page < 0 || page >= a.P.n_pages) {
        if ((threadIdx.x & 31) == 0) flag_corrupt(a.status);
        return nullptr;
    }
    return (uint8_t*)page_ptr(a.P, page, j.h, (j.tok0 & ((1 << a.P.page_shift) - 1)) / kUnit);
}

/* Eight consecutive elements of type T (EC_DTYPE_*) as they lie in memory. */
template <int T>
struct Raw8 {
    uint32_t w[T == EC_DTYPE_FP32 ? 8 : 4];
};
template <int T, bool kWide>
__device__ __forceinline__ Raw8<T> load_raw(const void* data, int64_t off, bool on) {
    constexpr int N = T == EC_DTYPE_FP32 ? 8 : 4;
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = 0;
    if (!on) return r;
    if constexpr (kWide) {
        const uint4* p = (const uint4*)((const uint8_t*)data + off * (T == EC_DTYPE_FP32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 x = p[i];
            r.w[4 * i] = x.x, r.w[4 * i + 1] = x.y, r.w[4 * i + 2] = x.z, r.w[4 * i + 3] = x.w;
        }
    } else if constexpr (T == EC_DTYPE_FP32) {
        const uint32_t* p = (const uint32_t*)data + off;
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = p[i];
    } else {
        const uint16_t* p = (const uint16_t*)data + off;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
    }
    return r;
}

/* Eight channels of one token -> their word and the block's scale byte (the quad's four
 * lanes take part).  The largest magnitude is found on the bits (NaN and infinity are the
 * largest), for 16-bit types two at a time. */
template <int T>
__device__ __forceinline__ uint32_t quantise8(const Raw8<T>& r, int& e) {
    uint32_t top = 0;
    float x[8];
    if constexpr (T == EC_DTYPE_FP32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = __uint_as_float(r.w[i]);
            top = max(top, r.w[i] & 0x7FFFFFFFu);
        }
    } else {
        const uint32_t m2 = __vmaxu2(__vmaxu2(r.w[0] & 0x7FFF7FFFu, r.w[1] & 0x7FFF7FFFu), __vmaxu2(r.w[2] & 0x7FFF7FFFu, r.w[3] & 0x7FFF7FFFu));
        const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (T == EC_DTYPE_FP16) {
                const float2 f = __half22float2(*(const __half2*)&r.w[i]);
                x[2 * i] = f.x, x[2 * i + 1] = f.y;
            } else x[2 * i] = __uint_as_float(r.w[i] << 16), x[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
        }
        top = T == EC_DTYPE_FP16 ? __float_as_uint(__half2float(__ushort_as_half((unsigned short)m))) : m << 16;
    }
    top = max(top, __shfl_xor_sync(kAll, top, 1));
    top = max(top, __shfl_xor_sync(kAll, top, 2));
    bool none;
    e = scale_byte(top, &none);
    const float s = none ? 0.f : inv_scale(e);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= s;
    const uint32_t w = f32x8_e2m1(x);
    return none ? 0u : w;
}

/* Four nibbles to the low halves of four bytes, and back. */
__device__ __forceinline__ uint32_t spread4(uint32_t x) {
    x = (x | x << 8) & 0x00FF00FFu;
    return (x | x << 4) & 0x0F0F0F0Fu;
}
__device__ __forceinline__ uint32_t gather4(uint32_t x) {
    x = (x | x >> 4) & 0x00FF00FFu;
    return (x | x >> 8) & 0xFFFFu;
}

template <int NB, int T>
__global__ void __launch_bounds__(kIoWarps * 32) kv_append_kernel(const __grid_constant__ IoArgs a) {
    constexpr int D = 32 * NB, SECTION = 8 * D + D / 2; /* a warp's codes and scales */
    __shared__ __align__(16) uint8_t io_smem[kIoWarps][SECTION];
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint8_t* buf = io_smem[threadIdx.x >> 5];
    grid_dep_launch();
    grid_dep_wait();
    const UnitJob j = unit_job(a);
    if (!j.any) return;
    const int32_t page = page_at(a, j);
    const Rows& R = j.which ? a.v : a.k;
    const bool on[2] = {g >= j.lo && g < j.hi, g + 8 >= j.lo && g + 8 < j.hi};
    Raw8<T> raw[NB][2];
    const int64_t off = (j.row0 + g) * R.row + (int64_t)j.h * R.head + 8 * c;
    if (R.wide) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < NB; ++b) raw[b][r] = load_raw<T, true>(R.data, off + 8 * r * R.row + 32 * b, on[r]);
    } else {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < NB; ++b) raw[b][r] = load_raw<T, false>(R.data, off + 8 * r * R.row + 32 * b, on[r]);
    }
    uint8_t* dst = unit_ptr(a, j, page);
    if (!dst) return;
    const bool full = j.lo == 0 && j.hi == kUnit;
    if (j.which == 0) {
        uint32_t word[2 * NB];
        uint8_t es[2][NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                int e;
                word[2 * b + r] = quantise8<T>(raw[b][r], e);
                es[r][b] = (uint8_t)e;
            }
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
            uint32_t* at = (uint32_t*)(dst + i * 512 + lane * 16);
            if (full) *(uint4*)at = make_uint4(word[4 * i], word[4 * i + 1], word[4 * i + 2], word[4 * i + 3]);
            else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (on[k & 1]) at[k] = word[4 * i + k];
            }
        }
        if (c == 0) { /* a token's scales, two at a time */
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int b = 0; b < NB; b += 2)
                    if (on[r]) *(uint16_t*)(dst + 16 * D + (g + 8 * r) * NB + b) = (uint16_t)(es[r][b] | es[r][b + 1] << 8);
        }
    } else {
        uint8_t* codes = dst + 8 * D;
        uint8_t* scales = dst + 16 * D + D / 2;
        if (j.lo > 0) { /* older tokens stay */
            for (int i = lane; i < 8 * D / 16; i += 32) ((uint4*)buf)[i] = ((const uint4*)codes)[i];
            for (int i = lane; i < D / 2 / 16; i += 32) ((uint4*)(buf + 8 * D))[i] = ((const uint4*)scales)[i];
            __syncwarp();
        }
        /* nibbles of the pair's places that are written: tokens 2 m, 2 m + 1, + 8 of pair m = g / 2 */
        const int m = g >> 1;
        uint32_t mask = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int tok = 2 * m + (t & 1) + 8 * (t >> 1);
            if (tok >= j.lo && tok < j.hi) mask |= (t & 1 ? 0xF0F0u : 0x0F0Fu) << (16 * (t >> 1));
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t w[2], x[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                int e;
                w[r] = quantise8<T>(raw[b][r], e);
                if (c == 0 && on[r]) buf[8 * D + ((m * NB + b) * 2 + r) * 2 + (g & 1)] = (uint8_t)e;
                /* pair step */
                const uint32_t other = __shfl_xor_sync(kAll, w[r], 4), sh = g & 1 ? 16 : 0;
                const uint32_t ev = ((g & 1 ? other : w[r]) >> sh) & 0xFFFFu, od = ((g & 1 ? w[r] : other) >> sh) & 0xFFFFu;
                x[r] = spread4(ev) | spread4(od) << 4;
            }
            /* channel step: word k = bytes (r 0, p 0), (r 1, p 0), (r 0, p 1), (r 1, p 1) of channel k */
            const uint32_t y0 = __shfl_xor_sync(kAll, x[0], 1), y1 = __shfl_xor_sync(kAll, x[1], 1);
            const uint32_t a0 = c & 1 ? y0 : x[0], b0 = c & 1 ? x[0] : y0, a1 = c & 1 ? y1 : x[1], b1 = c & 1 ? x[1] : y1;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int ch = 2 * (c & 1) + k;
                const uint32_t sel = (uint32_t)ch | (uint32_t)(4 + ch) << 4;
                const uint32_t lo = __byte_perm(a0, b0, sel), hi = __byte_perm(a1, b1, sel);
                const uint32_t word = __byte_perm(lo, hi, 0x5410);
                const int i = 2 * b + (c >> 1);
                uint32_t* at = (uint32_t*)(buf + (i >> 2) * 512 + ((4 * (g & 1) + ch) * 4 + m) * 16 + (i & 3) * 4);
                *at = full ? word : ((j.lo > 0 ? *at : 0u) & ~mask) | (word & mask);
            }
        }
        __syncwarp();
        for (int i = lane; i < 8 * D / 16; i += 32) ((uint4*)codes)[i] = ((const uint4*)buf)[i];
        if (full || j.lo > 0) {
            for (int i = lane; i < D / 2 / 16; i += 32) ((uint4*)scales)[i] = ((const uint4*)(buf + 8 * D))[i];
        } else { /* a new unit with places left: bytes of its tokens only */
            for (int i = lane; i < D / 2; i += 32) {
                const int tok = 2 * (i / (4 * NB)) + (i & 1) + 8 * ((i >> 1) & 1);
                if (tok < j.hi) scales[i] = buf[8 * D + i];
            }
        }
    }
}

__device__ __forceinline__ void word_values(uint32_t w, float s, float (&x)[8]) {
    uint32_t h[4];
    e2m1x8_f16(w, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*(const __half2*)&h[i]);
        x[2 * i] = f.x * s, x[2 * i + 1] = f.y * s;
    }
}

template <int NB>
__global__ void __launch_bounds__(kIoWarps * 32) kv_read_kernel(const __grid_constant__ IoArgs a) {
    constexpr int D = 32 * NB;
    __shared__ __align__(16) uint8_t io_smem[kIoWarps][8 * D];
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint8_t* buf = io_smem[threadIdx.x >> 5];
    grid_dep_launch();
    grid_dep_wait();
    const UnitJob j = unit_job(a);
    if (!j.in) return;
    const Rows& R = j.which ? a.v : a.k;
    const int none = j.q.m - j.q.len;
    if (none > 0 && (j.which ? a.has_v : a.has_k)) { /* rows of tokens before the sequence's first: zeros, 16 at a time */
        const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int64_t r0 = j.u * kUnit; r0 < none; r0 += a.units * kUnit)
            for (int64_t r = r0; r < min((int64_t)none, r0 + kUnit); ++r)
                for (int d = 8 * lane; d < D; d += 256) store8(R, (j.q.row0 + r) * R.row + (int64_t)j.h * R.head + d, z);
    }
    if (!j.any) return;
    const uint8_t* src = unit_ptr(a, j, page_at(a, j));
    if (!src) return;
    const bool on[2] = {g >= j.lo && g < j.hi, g + 8 >= j.lo && g + 8 < j.hi};
    uint32_t word[2][NB]; /* channels 32 b + 8 c + 0..7 of tokens g, g + 8 */
    uint32_t es[2][NB];
    uint4 w[NB / 2];
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) w[i] = *(const uint4*)(src + (j.which ? 8 * D : 0) + i * 512 + lane * 16);
    if (j.which == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < NB; ++b) es[r][b] = src[16 * D + (g + 8 * r) * NB + b];
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
            word[0][2 * i] = w[i].x, word[1][2 * i] = w[i].y;
            word[0][2 * i + 1] = w[i].z, word[1][2 * i + 1] = w[i].w;
        }
    } else {
        const int m = g >> 1;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < NB; ++b) es[r][b] = src[16 * D + D / 2 + ((m * NB + b) * 2 + r) * 2 + (g & 1)];
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) *(uint4*)(buf + i * 512 + lane * 16) = w[i];
        __syncwarp();
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int i = 2 * b + (c >> 1);
            uint32_t v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                v[k] = *(const uint32_t*)(buf + (i >> 2) * 512 + ((4 * (g & 1) + 2 * (c & 1) + k) * 4 + m) * 16 + (i & 3) * 4);
            /* channel step: bytes (p 0 of channels k, k + 1 | p 1 of them) of r = c % 2, and of the other r for lane c ^ 1 */
            const uint32_t mine = __byte_perm(v[0], v[1], c & 1 ? 0x7351 : 0x6240), theirs = __byte_perm(v[0], v[1], c & 1 ? 0x6240 : 0x7351);
            const uint32_t got = __shfl_xor_sync(kAll, theirs, 1);
            const uint32_t first = c & 1 ? got : mine, second = c & 1 ? mine : got; /* channels 0, 1 and 2, 3 of the four */
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t x = __byte_perm(first, second, r ? 0x7632 : 0x5410);
                /* pair step: low nibbles are the even token's */
                const uint32_t ev = gather4(x & 0x0F0F0F0Fu), od = gather4((x >> 4) & 0x0F0F0F0Fu);
                const uint32_t other = __shfl_xor_sync(kAll, g & 1 ? ev : od, 4);
                word[r][b] = g & 1 ? other | od << 16 : ev | other << 16;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (!on[r]) continue;
        const int64_t off = (j.row0 + g + 8 * r) * R.row + (int64_t)j.h * R.head + 8 * c;
        if (R.wide && R.dtype == EC_DTYPE_BF16) {
            uint16_t* at = (uint16_t*)R.data + off;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float x[8];
                word_values(word[r][b], scale_value((int)es[r][b]), x);
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                    u[i] = *(const uint32_t*)&y;
                }
                *(uint4*)(at + 32 * b) = make_uint4(u[0], u[1], u[2], u[3]);
            }
        } else {
#pragma unroll 1
            for (int b = 0; b < NB; ++b) {
                float x[8];
                uint32_t w2 = 0, e2 = 0;
#pragma unroll
                for (int k = 0; k < NB; ++k)
                    if (k == b) w2 = word[r][k], e2 = es[r][k];
                word_values(w2, scale_value((int)e2), x);
                store8(R, off + 32 * b, x);
            }
        }
    }
}

/* units that n consecutive tokens can touch */
static int units_of(int n) { return (n + 14) / kUnit + 1; }

/* ============================================================ page operations */
/* What a plan leaves in `work` for the copy kernel: the number of copies, then
 * (source page, destination page, units per head) triples.  A fork has at most one copy
 * per sequence, a compaction at most n_pages / 2.
 *
 * A plan is one CTA: the work is a few passes over small integer arrays with a barrier
 * between them, bound by the latency of each pass (about 4 us of the 7.7 us of a step of 8
 * beams over 32 layers); up to kSmallPool pages the counts are kept in shared memory, above
 * that in refs_out itself. */
struct PlanArgs {
    Pool P;
    const int32_t *table, *lens, *refs, *parents, *grow;
    int32_t *table_out, *lens_out, *refs_out, *map;
    int64_t in_stride, out_stride;
    int32_t n_in, n_out;
    int32_t* count;     /* [1] */
    int32_t* copies;    /* [.][3] */
    int* status;
};

constexpr int kPlanThreads = 1024; /* one sequence each: EC_KV_MAX_SEQS */
constexpr int kSmallPool = 24576;  /* 96 KB of counts */
static_assert(EC_KV_MAX_SEQS <= kPlanThreads, "one thread per sequence");

/* Exclusive scan of one value per thread over the CTA; *total gets the sum. */
template <class T>
__device__ __forceinline__ T block_scan(T v, T* total, T* tmp /* [33] */) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(kAll, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        T y = tmp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T z = __shfl_up_sync(kAll, y, o);
            if (lane >= o) y += z;
        }
        tmp[lane] = y;
        if (lane == 31) tmp[32] = y;
    }
    __syncthreads();
    *total = tmp[32];
    return x - v + (warp ? tmp[warp - 1] : 0);
}

__global__ void __launch_bounds__(kPlanThreads) kv_fork_plan_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ __align__(16) int32_t plan_smem[];
    __shared__ int64_t tmp[33];
    __shared__ int n_copies;
    __shared__ int32_t first[EC_KV_MAX_SEQS], len_of[EC_KV_MAX_SEQS], kept_of[EC_KV_MAX_SEQS], need_of[EC_KV_MAX_SEQS],
        parent_of[EC_KV_MAX_SEQS];
    __shared__ int64_t begin_of[EC_KV_MAX_SEQS];
    const int tid = threadIdx.x, lane = tid & 31, shift = a.P.page_shift, T = 1 << shift, N = a.P.n_pages;
    const int64_t in_cap = a.in_stride << shift;
    int32_t* cnt = N <= kSmallPool ? plan_smem : a.refs_out;
    grid_dep_launch();
    grid_dep_wait();
    for (int i = tid; i < N; i += kPlanThreads) cnt[i] = a.refs[i];
    int parent = -1;
    int64_t more = 0;
    if (tid < a.n_in) {
        const int64_t n = a.lens[tid];
        if (n > in_cap) flag_corrupt(a.status);
        len_of[tid] = (int)(n < 0 ? 0 : n > in_cap ? in_cap : n);
        first[tid] = a.n_out;
    }
    if (tid < a.n_out) {
        const int p = a.parents ? a.parents[tid] : tid;
        if (p < -1 || p >= a.n_in) flag_corrupt(a.status);
        else parent = p;
        more = a.grow ? max(a.grow[tid], 0) : 0;
        parent_of[tid] = parent;
    }
    if (tid == 0) n_copies = 0;
    __syncthreads();
    if (parent >= 0) atomicMin(&first[parent], tid);
    __syncthreads();
    auto pages_of = [&](int len) { return (int)(((int64_t)len + T - 1) >> shift); };
    auto page_in = [&](int s, int k) {
        const int p = a.table[(int64_t)s * a.in_stride + k];
        return p < 0 || p >= N ? -1 : p;
    };
    /* pages shared (kept) and wanted */
    int kept = 0, need = 0;
    int64_t want = 0, now = 0;
    if (parent >= 0) {
        const int len = len_of[parent];
        now = len + more;
        kept = (len >> shift) + ((len & (T - 1)) && first[parent] == tid ? 1 : 0);
        const int64_t n = (now + T - 1) >> shift;
        need = n > a.out_stride || now > 0x7FFFFFFF ? -1 : (int)n;
        want = need < 0 ? 0 : need - kept;
    }
    int64_t wanted;
    const int64_t begin = block_scan(want, &wanted, tmp);
    if (tid < a.n_out) kept_of[tid] = kept, need_of[tid] = need, begin_of[tid] = begin;
    __syncthreads();
    /* reference counts: sequences without a child give their pages up; children past the
     * first add theirs (a first child takes its parent's place in every count) */
    for (int s = tid >> 5; s < a.n_in; s += kPlanThreads / 32)
        if (first[s] == a.n_out)
            for (int k = lane; k < pages_of(len_of[s]); k += 32) {
                const int p = page_in(s, k);
                if (p >= 0) atomicSub(&cnt[p], 1);
                else flag_corrupt(a.status);
            }
    for (int i = tid >> 5; i < a.n_out; i += kPlanThreads / 32) {
        const int s = parent_of[i];
        if (s < 0 || first[s] == i) continue;
        for (int k = lane; k < kept_of[i]; k += 32) {
            const int p = page_in(s, k);
            if (p < 0) flag_corrupt(a.status);
            else atomicAdd(&cnt[p], 1);
        }
    }
    __syncthreads();
    /* the free pages in ascending order go to the ranks begin .. ; a thread looks at a run of pages */
    const int run = (N + kPlanThreads - 1) / kPlanThreads, p0 = min(N, tid * run), p1 = min(N, p0 + run);
    int64_t mine = 0, F;
    for (int p = p0; p < p1; ++p) mine += cnt[p] == 0;
    int64_t rank = block_scan(mine, &F, tmp);
    auto fits = [&](int i) { return need_of[i] >= 0 && (need_of[i] == kept_of[i] || begin_of[i] + (need_of[i] - kept_of[i]) <= F); };
    if (mine)
        for (int p = p0; p < p1 && rank < wanted; ++p) {
            if (cnt[p] != 0) continue;
            int lo = 0, hi = a.n_out - 1; /* the last sequence that begins at the rank or before (those that want nothing come before it) */
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (begin_of[mid] <= rank) lo = mid;
                else hi = mid - 1;
            }
            if (fits(lo)) {
                a.table_out[(int64_t)lo * a.out_stride + kept_of[lo] + (int)(rank - begin_of[lo])] = p;
                cnt[p] = 1;
            }
            ++rank;
        }
    __syncthreads();
    /* rows, lengths, copies */
    for (int i = tid >> 5; i < a.n_out; i += kPlanThreads / 32) {
        const int s = parent_of[i], k0 = kept_of[i], k1 = need_of[i];
        const bool ok = fits(i);
        int32_t* row = a.table_out + (int64_t)i * a.out_stride;
        for (int64_t k = lane; k < a.out_stride; k += 32) {
            if (ok && k < k0) {
                const int p = a.table[(int64_t)s * a.in_stride + k];
                if (p < 0 || p >= N) flag_corrupt(a.status);
                row[k] = p;
            } else if (!ok || k >= k1) row[k] = -1;
        }
        if (!ok)
            for (int k = lane; k < k0; k += 32) {
                const int p = page_in(s, k);
                if (p >= 0) atomicSub(&cnt[p], 1);
            }
        if (lane == 0 && ok && s >= 0 && (len_of[s] & (T - 1)) && first[s] != i) {
            const int from = page_in(s, len_of[s] >> shift);
            if (from >= 0) {
                const int n = atomicAdd(&n_copies, 1);
                a.copies[3 * n] = from;
                a.copies[3 * n + 1] = row[k0];
                a.copies[3 * n + 2] = ((len_of[s] & (T - 1)) + kUnit - 1) / kUnit;
            } else flag_corrupt(a.status);
        }
    }
    if (tid < a.n_out) a.lens_out[tid] = !fits(tid) ? -1 : (int)now;
    __syncthreads();
    if (cnt != a.refs_out)
        for (int i = tid; i < N; i += kPlanThreads) a.refs_out[i] = cnt[i];
    if (tid == 0) *a.count = n_copies;
}

__global__ void __launch_bounds__(kPlanThreads) kv_compact_plan_kernel(const __grid_constant__ PlanArgs a) {
    __shared__ int64_t tmp[33];
    const int tid = threadIdx.x, N = a.P.n_pages;
    grid_dep_launch();
    grid_dep_wait();
    int64_t mine = 0, total;
    for (int i = tid; i < N; i += kPlanThreads) mine += a.refs[i] > 0;
    block_scan(mine, &total, tmp);
    const int n = (int)total;
    int holes = 0, movers = 0;
    for (int base = 0; base < N; base += kPlanThreads) {
        const int i = base + tid;
        const int ref = i < N ? a.refs[i] : 0;
        const bool live = ref > 0, hole = i < n && !live, mover = live && i >= n;
        const int64_t x = block_scan<int64_t>((hole ? 1 : 0) | (mover ? int64_t(1) << 32 : 0), &total, tmp);
        if (hole) a.copies[3 * (holes + (int)x) + 1] = i;
        if (mover) a.copies[3 * (movers + (int)(x >> 32))] = i;
        holes += (int)total;
        movers += (int)(total >> 32);
        if (i < N) {
            a.refs_out[i] = live && i < n ? ref : 0;
            a.map[i] = live && i < n ? i : -1;
        }
    }
    __syncthreads();
    for (int k = tid; k < movers; k += kPlanThreads) {
        const int src = a.copies[3 * k], dst = a.copies[3 * k + 1];
        a.copies[3 * k + 2] = 1 << (a.P.page_shift - 4);
        a.map[src] = dst;
        a.refs_out[dst] = a.refs[src];
    }
    __syncthreads();
    if (tid == 0) *a.count = movers;
    for (int s = tid; s < a.n_in; s += kPlanThreads) {
        if (a.lens[s] > a.in_stride << a.P.page_shift) flag_corrupt(a.status);
        a.lens_out[s] = a.lens[s];
    }
    for (int s = tid >> 5; s < a.n_in; s += kPlanThreads / 32)
        for (int64_t col = tid & 31; col < a.out_stride; col += 32) {
            const int p = col < a.in_stride ? a.table[s * a.in_stride + col] : -1;
            a.table_out[s * a.out_stride + col] = p >= 0 && p < N ? a.map[p] : p;
        }
}

struct CopyArgs {
    Pool P;
    const int32_t* count;
    const int32_t* copies;
    int32_t heads;   /* heads of all layers */
};

/* A copy moves the first `units` units of every head of every layer of a page: runs of
 * units * 17 D contiguous bytes, one CTA per (copy, head) run at a time.  Bound by HBM: a
 * compaction that moves 0.2 GB takes 68 to 74 us with its plan (5.4 to 5.9 TB/s, 0.81 to 0.88 of
 * the measured copy rate), 64 samples of 6 prompts over 32 layers 22 to 23.5 us (112 MB, 5 TB/s). */
constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const __grid_constant__ CopyArgs a) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t items = (int64_t)*a.count * a.heads;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t c = it / a.heads, h = it % a.heads;
        const int64_t src = a.copies[3 * c], dst = a.copies[3 * c + 1];
        const int n = a.copies[3 * c + 2] * (a.P.unit_bytes / 16);
        const uint4* s = (const uint4*)(a.P.base + src * a.P.page_bytes + h * a.P.head_bytes);
        uint4* d = (uint4*)(a.P.base + dst * a.P.page_bytes + h * a.P.head_bytes);
        for (int i = threadIdx.x; i < n; i += 4 * kCopyThreads) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k * kCopyThreads < n) v[k] = s[i + k * kCopyThreads];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k * kCopyThreads < n) d[i + k * kCopyThreads] = v[k];
        }
    }
}

static size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }

/* work: count (16 bytes) | copies | map (compact) */
static size_t pages_work(const ec_kv* C, int64_t n_out) {
    const size_t fork = 16 + align16(12 * (size_t)n_out);
    const size_t compact = 16 + align16(12 * ((size_t)C->p.n_pages / 2 + 1)) + align16(4 * (size_t)C->p.n_pages);
    return fork > compact ? fork : compact;
}

static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    return a && b && na && nb && (const uint8_t*)a < (const uint8_t*)b + nb && (const uint8_t*)b < (const uint8_t*)a + na;
}

static int check_pages(const ec_kv* C, const ec_kv_pages* g) {
    if (!C || !g) return EC_ERR_INVALID_ARG;
    const ec_kv_seqs &from = g->from, &to = g->to;
    int rc = check_seqs(&from);
    if (rc == EC_OK) rc = check_seqs(&to);
    if (rc != EC_OK) return rc;
    if (!g->refs || !g->refs_out || !g->work || (uintptr_t)g->work % 16) return EC_ERR_INVALID_ARG;
    if (g->work_bytes < pages_work(C, to.n_seqs)) return EC_ERR_INVALID_ARG;
    const size_t in = sizeof(int32_t) * (size_t)(from.n_seqs * from.table_stride), nr = sizeof(int32_t) * (size_t)C->p.n_pages,
                 out = sizeof(int32_t) * (size_t)(to.n_seqs * to.table_stride);
    if (overlap(from.table, in, to.table, out) || overlap(g->refs, nr, g->refs_out, nr) ||
        overlap(from.lens, sizeof(int32_t) * (size_t)from.n_seqs, to.lens, sizeof(int32_t) * (size_t)to.n_seqs))
        return EC_ERR_INVALID_ARG;
    return EC_OK;
}

static int run_copies(const ec_kv* C, const PlanArgs& a, int64_t most, const Device& d, cudaStream_t stream) {
    CopyArgs c{};
    c.P = a.P;
    c.count = a.count;
    c.copies = a.copies;
    c.heads = C->p.n_layers * C->p.n_kv_heads;
    const int64_t items = most * c.heads;
    const int64_t full = (int64_t)d.sms * 8;
    const int grid = (int)(items < 1 ? 1 : items < full ? items : full);
    return launch(kv_copy_kernel, dim3(grid), kCopyThreads, 0, stream, c);
}

}  // namespace kv

using namespace kv;

/* ============================================================ C ABI */
static int check_params(const ec_kv_params* p, size_t* bytes) {
    if (!p) return EC_ERR_INVALID_ARG;
    if (p->n_layers < 1 || p->n_kv_heads < 1 || p->head_dim < 1 || p->page_tokens < 1 || p->n_pages < 1) return EC_ERR_SHAPE;
    if (p->n_layers > 1024 || p->n_kv_heads > 1024 || p->n_pages > (int64_t(1) << 30)) return EC_ERR_UNSUPPORTED;
    if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 192 && p->head_dim != 256) return EC_ERR_UNSUPPORTED;
    if (p->page_tokens != 16 && p->page_tokens != 32 && p->page_tokens != 64 && p->page_tokens != 128 && p->page_tokens != 256)
        return EC_ERR_UNSUPPORTED;
    /* at most 1024 * 1024 * 16 * 4352 < 2^37 bytes per page, 2^30 pages: checked before the product */
    const int64_t page = (int64_t)p->n_layers * p->n_kv_heads * (p->page_tokens / kUnit) * 17 * p->head_dim;
    if (p->n_pages > (int64_t(1) << 62) / page) return EC_ERR_OVERFLOW;
    *bytes = (size_t)(page * p->n_pages);
    return EC_OK;
}

extern "C" int ec_kv_pool_bytes(const ec_kv_params* params, size_t* bytes) {
    if (!bytes) return EC_ERR_INVALID_ARG;
    return check_params(params, bytes);
}

extern "C" int ec_kv_create(const ec_kv_params* params, void* pool, size_t pool_bytes, int device, ec_kv** out) {
    if (!out) return EC_ERR_INVALID_ARG;
    *out = nullptr;
    size_t need = 0;
    const int rc = check_params(params, &need);
    if (rc != EC_OK) return rc;
    if (device >= 0) {
        if (!pool || (uintptr_t)pool % 16 || pool_bytes < need) return EC_ERR_INVALID_ARG;
        int n = 0;
        if (cudaGetDeviceCount(&n) != cudaSuccess) return EC_ERR_CUDA;
        if (device >= n) return EC_ERR_INVALID_ARG;
    }
    ec_kv* C = new (std::nothrow) ec_kv;
    if (!C) return EC_ERR_OOM;
    C->p = *params;
    C->pool = device >= 0 ? (uint8_t*)pool : nullptr;
    C->device = device;
    *out = C;
    return EC_OK;
}

extern "C" void ec_kv_free(ec_kv* C) { delete C; }

template <class Kernel>
static int run_io(const ec_kv* C, const ec_kv_tokens* t, IoArgs& a, Kernel k2, Kernel k4, Kernel k6, Kernel k8, cudaStream_t stream) {
    a.units = units_of(t->max_new);
    a.max_new = t->max_new;
    const int64_t items = (int64_t)a.S.n_seqs * a.units * a.P.n_heads * 2, grid = (items + kIoWarps - 1) / kIoWarps;
    if (items > 0x7FFFFFFF) return EC_ERR_UNSUPPORTED;
    const int nb = C->p.head_dim / 32;
    return launch(nb == 2 ? k2 : nb == 4 ? k4 : nb == 6 ? k6 : k8, dim3((unsigned)grid), kIoWarps * 32, 0, stream, a);
}

template <int T>
static int run_append(const ec_kv* C, const ec_kv_tokens* t, IoArgs& a, cudaStream_t stream) {
    return run_io(C, t, a, kv_append_kernel<2, T>, kv_append_kernel<4, T>, kv_append_kernel<6, T>, kv_append_kernel<8, T>, stream);
}

extern "C" int ec_kv_append(const ec_kv* C, const ec_kv_tokens* t, cudaStream_t stream) {
    if (!C || !t) return EC_ERR_INVALID_ARG;
    IoArgs a{};
    bool go = false;
    int rc = check_call(C, t->layer, &t->seqs, t->starts, t->n_rows, t->max_new, &a.P, &a.S, &go);
    if (rc == EC_OK) rc = check_rows(&t->k, a.P.n_heads, t->n_rows, &a.k);
    if (rc == EC_OK) rc = check_rows(&t->v, a.P.n_heads, t->n_rows, &a.v);
    if (rc != EC_OK) return rc;
    if (t->k.dtype != t->v.dtype) return EC_ERR_UNSUPPORTED;
    Device d;
    if ((rc = device_of(C, &d)) != EC_OK) return rc;
    if (!go) return EC_OK;
    a.has_k = a.has_v = 1;
    a.status = d.status;
    switch (t->k.dtype) {
        case EC_DTYPE_FP32: return run_append<EC_DTYPE_FP32>(C, t, a, stream);
        case EC_DTYPE_FP16: return run_append<EC_DTYPE_FP16>(C, t, a, stream);
        default: return run_append<EC_DTYPE_BF16>(C, t, a, stream);
    }
}

extern "C" int ec_kv_read(const ec_kv* C, const ec_kv_tokens* t, cudaStream_t stream) {
    if (!C || !t) return EC_ERR_INVALID_ARG;
    IoArgs a{};
    bool go = false;
    int rc = check_call(C, t->layer, &t->seqs, t->starts, t->n_rows, t->max_new, &a.P, &a.S, &go);
    a.has_k = t->k.data != nullptr;
    a.has_v = t->v.data != nullptr;
    if (rc == EC_OK && t->n_rows > 0 && !a.has_k && !a.has_v) rc = EC_ERR_INVALID_ARG;
    if (rc == EC_OK && a.has_k) rc = check_rows(&t->k, a.P.n_heads, t->n_rows, &a.k);
    if (rc == EC_OK && a.has_v) rc = check_rows(&t->v, a.P.n_heads, t->n_rows, &a.v);
    if (rc != EC_OK) return rc;
    Device d;
    if ((rc = device_of(C, &d)) != EC_OK) return rc;
    if (!go) return EC_OK;
    a.status = d.status;
    return run_io(C, t, a, kv_read_kernel<2>, kv_read_kernel<4>, kv_read_kernel<6>, kv_read_kernel<8>, stream);
}

extern "C" int ec_kv_pages_work_bytes(const ec_kv* C, int n_from, int n_to, size_t* bytes) {
    if (!C || !bytes) return EC_ERR_INVALID_ARG;
    if (n_from < 0 || n_to < 0) return EC_ERR_SHAPE;
    if (n_from > EC_KV_MAX_SEQS || n_to > EC_KV_MAX_SEQS) return EC_ERR_UNSUPPORTED;
    *bytes = pages_work(C, n_to);
    return EC_OK;
}

extern "C" int ec_kv_fork(const ec_kv* C, const ec_kv_pages* g, cudaStream_t stream) {
    int rc = check_pages(C, g);
    if (rc != EC_OK) return rc;
    const ec_kv_seqs *from = &g->from, *to = &g->to;
    if (!g->parents && to->n_seqs > 0 && from->n_seqs != to->n_seqs) return EC_ERR_SHAPE;
    PlanArgs a{};
    if (!pool_view(C, 0, &a.P)) return EC_ERR_INVALID_ARG;
    Device d;
    if ((rc = device_of(C, &d)) != EC_OK) return rc;
    a.table = from->table, a.lens = from->lens, a.refs = g->refs, a.parents = g->parents, a.grow = g->grow;
    a.table_out = to->table, a.lens_out = to->lens, a.refs_out = g->refs_out;
    a.in_stride = from->table_stride, a.out_stride = to->table_stride;
    a.n_in = from->n_seqs, a.n_out = to->n_seqs;
    uint8_t* w = (uint8_t*)g->work;
    a.count = (int32_t*)w;
    w += 16;
    a.copies = (int32_t*)w;
    a.status = d.status;
    static SmemOnce once;
    if ((rc = once.set(kv_fork_plan_kernel, sizeof(int32_t) * kSmallPool)) != EC_OK) return rc;
    const size_t counts = a.P.n_pages <= kSmallPool ? sizeof(int32_t) * (size_t)a.P.n_pages : 0;
    if ((rc = launch(kv_fork_plan_kernel, dim3(1), kPlanThreads, counts, stream, a)) != EC_OK) return rc;
    return run_copies(C, a, a.n_out, d, stream);
}

extern "C" int ec_kv_compact(const ec_kv* C, const ec_kv_pages* g, cudaStream_t stream) {
    int rc = check_pages(C, g);
    if (rc != EC_OK) return rc;
    const ec_kv_seqs *from = &g->from, *to = &g->to;
    if (from->n_seqs != to->n_seqs) return EC_ERR_SHAPE;
    if (to->table_stride < from->table_stride) return EC_ERR_SHAPE;
    const size_t nr = sizeof(int32_t) * (size_t)C->p.n_pages;
    if (overlap(g->map, nr, g->refs, nr) || overlap(g->map, nr, g->refs_out, nr)) return EC_ERR_INVALID_ARG;
    PlanArgs a{};
    if (!pool_view(C, 0, &a.P)) return EC_ERR_INVALID_ARG;
    Device d;
    if ((rc = device_of(C, &d)) != EC_OK) return rc;
    a.table = from->table, a.lens = from->lens, a.refs = g->refs;
    a.table_out = to->table, a.lens_out = to->lens, a.refs_out = g->refs_out;
    a.in_stride = from->table_stride, a.out_stride = to->table_stride;
    a.n_in = from->n_seqs, a.n_out = to->n_seqs;
    uint8_t* w = (uint8_t*)g->work;
    a.count = (int32_t*)w;
    w += 16;
    a.copies = (int32_t*)w;
    w += align16(12 * ((size_t)C->p.n_pages / 2 + 1));
    a.map = g->map ? g->map : (int32_t*)w;
    a.status = d.status;
    if ((rc = launch(kv_compact_plan_kernel, dim3(1), kPlanThreads, 0, stream, a)) != EC_OK) return rc;
    return run_copies(C, a, C->p.n_pages / 2 + 1, d, stream);
}
