/*
 * ec_kv_internal.h -- what the cache's translation units share: the descriptor, the
 * device view of it and of the sequences, the 4-bit format, and small PTX helpers.
 */
#ifndef EC_KV_INTERNAL_H_
#define EC_KV_INTERNAL_H_

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "ec_internal.h"

struct ec_kv {
    ec_kv_params p;
    uint8_t* pool; /* the caller's; NULL for a descriptor without a device */
    int32_t device;
};

namespace kv {

constexpr int kUnit = 16;        /* tokens per unit */
constexpr unsigned kAll = 0xFFFFFFFFu;

/* ------------------------------------------------------------ device views */
struct Pool {
    uint8_t* base;
    int64_t page_bytes;   /* all layers of a page */
    int64_t layer_off;    /* the call's layer inside a page */
    int64_t head_bytes;   /* one head of one layer of a page */
    int32_t n_pages, n_heads, dim;
    int32_t page_shift;   /* log2(page_tokens) */
    int32_t unit_bytes;   /* 17 dim */
};

struct Seqs {
    const int32_t* table;
    const int32_t* lens;
    const int32_t* starts;
    int64_t table_stride;
    int64_t n_rows;
    int32_t n_seqs;
};

struct Rows {
    void* data;
    int64_t row, head;  /* strides in elements */
    int32_t dtype;
    int32_t wide;       /* 16-byte loads and stores allowed */
};

/* What a sequence holds and which dense rows are its: len tokens, the last m of them
 * new, rows row0 .. row0 + m - 1 of the dense arguments. */
struct Seq {
    int32_t len, m;
    int64_t row0;
    bool bad;
};

__device__ __forceinline__ Seq seq_of(const Seqs& S, int page_shift, int b) {
    Seq q;
    q.bad = false;
    int64_t len = S.lens[b];
    if (len < 0) len = 0;
    const int64_t cap = S.table_stride << page_shift;
    if (len > cap) {
        len = cap;
        q.bad = true;
    }
    int64_t r0 = b, m = 1;
    if (S.starts) {
        r0 = S.starts[b];
        m = (int64_t)S.starts[b + 1] - r0;
    }
    if (m < 0 || r0 < 0 || r0 + m > S.n_rows) {
        m = 0;
        q.bad = true;
    }
    q.len = (int32_t)len;
    q.m = (int32_t)m;
    q.row0 = r0;
    return q;
}

/* Address of unit u (16 tokens) of head h of sequence b; a page number outside the pool
 * reads page 0 and is flagged. */
__device__ __forceinline__ const uint8_t* page_ptr(const Pool& P, int32_t page, int h, int unit_in_page) {
    return P.base + (int64_t)page * P.page_bytes + P.layer_off + (int64_t)h * P.head_bytes +
           (int64_t)unit_in_page * P.unit_bytes;
}

__device__ __forceinline__ void flag_corrupt(int* status) { atomicOr(status, 1); }

/* ------------------------------------------------------------ E2M1 and E8M0 */
/* The four bytes of a word -> four FP16 pairs. */
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
/* Eight FP32 values -> a word of eight elements (the first in the low nibble), nearest even, 6 the largest. */
__device__ __forceinline__ uint32_t f32x8_e2m1(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}
/* The scale byte of a block whose largest magnitude has these bits: the smallest e >= 1 with
 * top <= 6 * 2^(e - 127), 0 for a block of zeros, 255 for one with an infinity or NaN
 * (*none in both cases).  With top = 1.f * 2^(E - 127) that e is E - 2, or E - 1 when 1.f >
 * 1.5, which is when adding 2^22 - 1 carries into the exponent; at most 253. */
__device__ __forceinline__ int scale_byte(uint32_t top, bool* none) {
    *none = top - 1u >= 0x7F7FFFFFu;
    const int e = max((int)((top + 0x3FFFFFu) >> 23) - 2, 1);
    return *none ? (top ? 255 : 0) : e;
}
/* 2^(e - 127), NaN for 255 (e = 0: blocks of zeros). */
__device__ __forceinline__ float scale_value(int e) {
    return e == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)e << 23);
}
/* 2^(127 - e), e in 1..253. */
__device__ __forceinline__ float inv_scale(int e) { return __uint_as_float((uint32_t)(254 - e) << 23); }

/* ------------------------------------------------------------ pairs of 16 bits */
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t both_halves(int v) { return ((uint32_t)v & 0xFFFFu) * 0x10001u; }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *(const uint32_t*)&h;
}

/* ------------------------------------------------------------ PTX helpers */
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory"); }
__device__ __forceinline__ void sts8(uint32_t a, uint32_t x) { asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(x) : "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_fence_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
/* Bounded wait for phase `parity`; false when the bound ran out. */
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    for (int i = 0; i < (1 << 20); ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return false;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

/* One element of a dense row as FP32, and back. */
__device__ __forceinline__ float load_elem(const Rows& R, int64_t off) {
    if (R.dtype == EC_DTYPE_FP32) return ((const float*)R.data)[off];
    if (R.dtype == EC_DTYPE_FP16) return __half2float(((const __half*)R.data)[off]);
    return __bfloat162float(((const __nv_bfloat16*)R.data)[off]);
}
__device__ __forceinline__ void store_elem(const Rows& R, int64_t off, float v) {
    if (R.dtype == EC_DTYPE_FP32) ((float*)R.data)[off] = v;
    else if (R.dtype == EC_DTYPE_FP16) ((__half*)R.data)[off] = __float2half_rn(v);
    else ((__nv_bfloat16*)R.data)[off] = __float2bfloat16_rn(v);
}

/* Eight consecutive elements. */
__device__ __forceinline__ void store8(const Rows& R, int64_t off, const float (&x)[8]) {
    if (R.wide) {
        if (R.dtype == EC_DTYPE_FP32) {
            *(float4*)((float*)R.data + off) = make_float4(x[0], x[1], x[2], x[3]);
            *(float4*)((float*)R.data + off + 4) = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (R.dtype == EC_DTYPE_FP16) {
                    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                    u[i] = *(const uint32_t*)&h;
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                    u[i] = *(const uint32_t*)&h;
                }
            }
            *(uint4*)((uint16_t*)R.data + off) = make_uint4(u[0], u[1], u[2], u[3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) store_elem(R, off + i, x[i]);
    }
}

/* ------------------------------------------------------------ host side */
struct Device {
    int sms;
    int* status;
};
int device_of(const ec_kv* C, Device* out);              /* EC_ERR_* unless C's pool is on the current device */
bool pool_view(const ec_kv* C, int layer, Pool* out);    /* false: layer out of range */
int check_seqs(const ec_kv_seqs* S);
int check_rows(const ec_kv_rows* r, int heads, int64_t n_rows, Rows* out);
bool use_pdl();

/* A kernel's dynamic shared-memory limit, raised before its first launch on a device. */
struct SmemOnce {
    std::atomic<uint64_t> done{0};
    template <class K>
    int set(K kernel, size_t bytes) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return EC_ERR_CUDA;
        if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1u)) return EC_OK;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
            return EC_ERR_CUDA;
        if (dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
        return EC_OK;
    }
};

template <class... KArgs, class... Args>
int launch(void (*kernel)(KArgs...), dim3 grid, int block, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = use_pdl() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? EC_OK : EC_ERR_CUDA;
}

}  // namespace kv

#endif
