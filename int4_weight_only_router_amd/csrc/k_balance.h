// k_balance.h -- arguments of the balance loss kernels.
#pragma once

#include "moe_common.h"

namespace moe {

constexpr int BL_MAX_E = 1024;

struct BalanceArgs {
    const void *logits;       // [T] rows, ld elements apart
    int64_t ld;
    const int32_t *idx;       // [T][k] choices, or null: counts are given
    const uint8_t *mask;      // [T], 0: a token that does not count; or null
    int T, E, k, score;
    float coef, zcoef;
    int32_t *counts;          // [E]
    float *mean_prob;         // [E] or null
    float *losses;            // [2] or null
    const float *d_loss;      // [1] or null (one)
    void *dlogits;            // [T] rows, ldd elements apart, or null
    int64_t ldd;
    int gtype;
    // workspace
    int count_groups;         // workgroups that count, 0: every one for itself
    int *n, *part_counts, *part_n;
    float *part_p;
};

size_t balance_ws(int T, int E);
int launch_balance(BalanceArgs, int dtype, void *ws, hipStream_t);

}  // namespace moe
