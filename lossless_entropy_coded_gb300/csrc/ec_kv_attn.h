/*
 * ec_kv_attn.h -- arguments of the attention kernels, shared by the register form
 * (ec_kv_attn.cu: few rows) and the tensor-memory form (ec_kv_prefill.cu: many rows).
 */
#ifndef EC_KV_ATTN_H_
#define EC_KV_ATTN_H_

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

struct PrefillPlan {
    int row_tiles, splits;
    int64_t grid;
    size_t work;
};
bool plan_prefill(const ec_kv* C, int sms, int n_seqs, int max_new, int64_t max_units, int group, int dtype, PrefillPlan* p);
int launch_prefill(const AttnArgs& a, const PrefillPlan& p, cudaStream_t stream);

}  // namespace kv

#endif
