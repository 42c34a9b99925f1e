// nosa_decode_work.cuh -- the work lists of the decode kernels: items are (unit, block) pairs, a unit's
// items lie one after the other, and each CTA takes a contiguous range of them.
#pragma once

#include "nosa_attend.cuh"

namespace nosa {

namespace {
// Work items of unit u in the kernel's mode.
__device__ __forceinline__ int32_t unit_work(const DecodeParams &p, int32_t u) {
    const int32_t L = p.seq_len[u];
    if (L <= 0) return 0;
    switch (p.mode) {
    case kModeSel: return max(0, min(p.nsel[u], p.max_sel));
    case kModeResident: return min(max(p.gamma_n[u], 0), p.k_e) + 1;
    case kModeRest: return p.k_q;
    default: return (L + kBlock - 1) / kBlock;
    }
}

// Block id (lb; -1 = nothing to attend) and buffer block index (pb) of item j of unit u.
__device__ __forceinline__ void item_block(const DecodeParams &p, int32_t u, int32_t j, int32_t &lb, int32_t &pb) {
    if (p.mode == kModeSel) {
        lb = p.sel[(int64_t)u * p.max_sel + j];
        pb = p.block_table ? p.block_table[(int64_t)u * p.max_sel + j] : lb;
        return;
    }
    if (p.mode == kModeDense) {
        lb = pb = j;
        return;
    }
    if (p.mode == kModeResident) {
        const int32_t ne = min(max(p.gamma_n[u], 0), p.k_e);
        lb = (j < ne) ? p.gamma_e[(int64_t)u * p.k_e + j] : (p.seq_len[u] - 1) / kBlock;
    } else {  // kModeRest: Gamma_q entries not already attended by the resident pass
        lb = p.gq[(int64_t)u * p.k_q + j];
        if (lb >= 0 && lb < p.nblk &&
            ((p.res_bits[(int64_t)u * p.bits_words + (lb >> 5)] >> (lb & 31)) & 1u))
            lb = -1;
    }
    pb = (p.block_slot && lb >= 0 && lb < p.nblk) ? p.block_slot[(int64_t)u * p.nblk + lb] : lb;
}

// Merge the resident pass's state of unit u (head h, dim d) into (M, acc, lsum) in place.
__device__ __forceinline__ void merge_resident(const DecodeParams &p, int32_t u, int h, int d, float &M, float &acc,
                                               float &lsum) {
    const float *r = p.res_part + (int64_t)u * kPartFloats;
    const float rm = r[h];
    const float Mn = fmaxf(M, rm);
    if (Mn == -__builtin_huge_valf()) return;
    const float fa = (M == -__builtin_huge_valf()) ? 0.f : exp2f(M - Mn);
    const float fr = (rm == -__builtin_huge_valf()) ? 0.f : exp2f(rm - Mn);
    acc = fmaf(fr, r[2 * kMaxG + h * kD + d], fa * acc);
    lsum = fmaf(fr, r[kMaxG + h], fa * lsum);
    M = Mn;
}

// Largest u with P[u] <= x, for 0 <= x < P[U] (skips units without work).
__device__ __forceinline__ int32_t find_unit(const int32_t *P, int32_t U, int64_t x) {
    int32_t lo = 0, hi = U;
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (P[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// CTA whose range [c*W/G, (c+1)*W/G) holds item x (every range non-empty: W >= G).
__device__ __forceinline__ int32_t cta_of(int64_t x, int64_t W, int32_t G) {
    return (int32_t)(((x + 1) * G - 1) / W);
}

}  // namespace

}  // namespace nosa
