// nosa_attend8.cuh -- attention of one staged block of the 8-bit KV store.
//
// NOSA pages: montaan.com summary of arXiv:2510.13602, "Empirical Results and Analysis" item 4
// (decoding is bound by KV loading); the pages keep the cache in 16 bits.
//
// Formula.  A block's keys stand for s_K c_jd and its values for s_V c'_jd, with 8-bit codes c
// (int8, or e4m3) and one fp32 scale each.  With x_j = s_K scale log2(e) (q . c_j) + e_j log2(e):
//   o = s_V sum_j 2^(x_j - m) c'_j,   l = sum_j 2^(x_j - m),   out = o / l.
// The scales come out of both products, so the matrix instructions run on the codes: every int8 and
// every e4m3 value is exact in f16, as is a bf16 query row once it is scaled by a power of two to
// [1, 2) (its smallest values, 2^-24 below the largest and less, are rounded by at most 2^-25 of it,
// below the fp32 sum's own rounding).  2^(x - m) goes to f16, 11 bits where the bf16 store's
// path has 8; m is kept 14 below the running maximum, so that the largest is 2^14 and the smallest
// normal one 2^-28 of it: a token loses bits only below that, and is lost only below 2^-39 of the
// largest (2^20 tokens of that size are 2^-19 of the sum).
//
// Layout.  As attend_block: warp w of a group owns tokens 16w..16w+15, S^T = C Q^T and
// O^T += C'^T P^T in m16n8k16 tiles.  One 16-byte shared load holds 16 dims of a row (half as many
// loads as bf16); the codes become f16 pairs in registers: int8 by placing the byte under the
// exponent of 1024 (one permute) and subtracting 1152, e4m3 by the conversion instruction.
#pragma once

#include "nosa_attend.cuh"

namespace nosa {

// The two low (two high) codes of a word as an f16 pair.  int8 codes come biased: c ^ 0x80.
template <int kFmt>
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
    if constexpr (kFmt == kFmtInt8) {
        const uint32_t x = __byte_perm(w, 0x64646464u, 0x4140);  // 1024 + 128 + c
        const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        uint32_t r;
        asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo; }" : "=r"(r) : "r"(w));
        return r;
    }
}
template <int kFmt>
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
    if constexpr (kFmt == kFmtInt8) {
        const uint32_t x = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        uint32_t r;
        asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi; }" : "=r"(r) : "r"(w));
        return r;
    }
}
template <int kFmt>
__device__ __forceinline__ uint32_t biased(uint32_t w) {
    return kFmt == kFmtInt8 ? w ^ 0x80808080u : w;
}

// A unit's queries as f16 fragments (dims ordered as attend8's key loads) and the powers of two
// they were divided by, for heads 2c and 2c + 1.
struct Query8 {
    uint32_t f[8][2];
    float s0, s1;
};

__device__ __forceinline__ void load_query8(Query8 &Q, const uint16_t *q, int G, int r, int c) {
    uint4 x[4];  // dims 16c..16c+15 and 64+16c..64+16c+15 of head r
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = r < G ? reinterpret_cast<const uint4 *>(q + r * kD)[8 * (i >> 1) + 2 * c + (i & 1)]
                     : make_uint4(0, 0, 0, 0);
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            a = max_nan(a, max_nan(fabsf(bf16_lo(word(x[i], j))), fabsf(bf16_hi(word(x[i], j)))));
    a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
    uint32_t E = (__float_as_uint(a) >> 23) & 255u;  // 255: not finite, nor are the scores
    E = E == 255u ? 127u : min(max(E, 15u), 253u);
    const float inv = __uint_as_float((254u + 14u - E) << 23);  // 2^(127 + 14 - E)
    const float s = __uint_as_float((E - 14u) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            Q.f[2 * i + (j >> 1)][j & 1] =
                pack_f16x2(bf16_lo(word(x[i], j)) * inv, bf16_hi(word(x[i], j)) * inv);
    Q.s0 = __shfl_sync(0xFFFFFFFFu, s, 8 * c);
    Q.s1 = __shfl_sync(0xFFFFFFFFu, s, 8 * c + 4);
}

constexpr float kPBias = 14.f;  // m is the running maximum less this

// One block of codes (t: 64 key rows, then 64 value rows, 128 bytes each, 128-byte swizzle), every
// token of it before the newest block.  sK, sV: its scales.  kWeights: as attend_block.
template <int kFmt, bool kWeights>
__device__ __forceinline__ void attend8(WarpState &st, const Query8 &Q, const uint8_t *t, const float *eb, float sK,
                                        float sV, float qk_log2, int warp, int r, int c, int sig, float *rec) {
    const int rowA = warp * 16 + sig, rowB = rowA + 8;
    // ---- S^T (16 tokens x 8 heads), two independent accumulation chains ----
    float sacc[4] = {0.f, 0.f, 0.f, 0.f};
    float sacc2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int off = (((c + 4 * j) ^ sig) << 4);
        const uint4 ka = lds128(t + rowA * kRow8Bytes + off);
        const uint4 kb = lds128(t + rowB * kRow8Bytes + off);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t x = biased<kFmt>(word(ka, w)), y = biased<kFmt>(word(kb, w));
            const uint32_t a[4] = {codes_lo<kFmt>(x), codes_lo<kFmt>(y), codes_hi<kFmt>(x), codes_hi<kFmt>(y)};
            mma_16816_f16((w & 1) ? sacc2 : sacc, a, Q.f[4 * j + w]);
        }
    }
    const float f0 = qk_log2 * sK * Q.s0, f1 = qk_log2 * sK * Q.s1;
    const float eA = bias_log2(eb[rowA]), eB = bias_log2(eb[rowB]);
    const float x0 = fmaf(sacc[0] + sacc2[0], f0, eA), x1 = fmaf(sacc[1] + sacc2[1], f1, eA);
    const float x2 = fmaf(sacc[2] + sacc2[2], f0, eB), x3 = fmaf(sacc[3] + sacc2[3], f1, eB);
    float bm0 = max_nan(x0, x2), bm1 = max_nan(x1, x3);
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
        bm0 = max_nan(bm0, __shfl_xor_sync(0xFFFFFFFFu, bm0, sh));
        bm1 = max_nan(bm1, __shfl_xor_sync(0xFFFFFFFFu, bm1, sh));
    }
    const float mn0 = max_nan(st.m0, bm0 - kPBias), mn1 = max_nan(st.m1, bm1 - kPBias);
    const float ms0 = mn0 == kNegInf ? 0.f : mn0, ms1 = mn1 == kNegInf ? 0.f : mn1;  // nothing seen yet: all zeros
    const float c0 = exp2f(st.m0 - ms0), c1 = exp2f(st.m1 - ms1);
    const float p0 = exp2f(x0 - ms0), p1 = exp2f(x1 - ms1), p2 = exp2f(x2 - ms0), p3 = exp2f(x3 - ms1);
    st.m0 = mn0;
    st.m1 = mn1;
    if constexpr (kWeights) leave_weights(rec, p0 + p2, p1 + p3, ms0, ms1, warp, r, c);
    // rounded to f16 once; the denominator sums what the numerator sums (kWeights: as attend_block)
    const uint32_t plo = pack_f16x2(p0, p1), phi = pack_f16x2(p2, p3);
    const float2 lo = unpack_f16x2(plo), hi = unpack_f16x2(phi);
    st.l0 = fmaf(st.l0, c0, kWeights ? p0 + p2 : lo.x + hi.x);
    st.l1 = fmaf(st.l1, c1, kWeights ? p1 + p3 : lo.y + hi.y);
    if (__any_sync(0xFFFFFFFFu, c0 != 1.f || c1 != 1.f)) {  // the maximum rises a few times in a long context
#pragma unroll
        for (int tt = 0; tt < 8; ++tt) {
            st.o[tt][0] *= c0; st.o[tt][1] *= c1;
            st.o[tt][2] *= c0; st.o[tt][3] *= c1;
        }
    }
    const uint32_t pb[2] = {movmatrix_trans(plo), movmatrix_trans(phi)};
    // ---- O^T (128 dims x 8 heads) += s_V C'^T P^T ----
    const uint8_t *vb = t + kHalfBlock8Bytes + (warp * 16 + c) * kRow8Bytes;
    const int off0 = ((sig ^ c) << 4), off1 = ((sig ^ (c + 4)) << 4);
    const uint4 v0 = lds128(vb + off0), v1 = lds128(vb + 4 * kRow8Bytes + off1);
    const uint4 v2 = lds128(vb + 8 * kRow8Bytes + off0), v3 = lds128(vb + 12 * kRow8Bytes + off1);
#pragma unroll
    for (int wi = 0; wi < 4; ++wi) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // dims 4 wi + 2 half, + 1 of the chunk: bytes of two tokens side by side
            const uint32_t z = biased<kFmt>(__byte_perm(word(v0, wi), word(v1, wi), half ? 0x7362 : 0x5140));
            const uint32_t y = biased<kFmt>(__byte_perm(word(v2, wi), word(v3, wi), half ? 0x7362 : 0x5140));
            const uint32_t a[4] = {codes_lo<kFmt>(z), codes_hi<kFmt>(z), codes_lo<kFmt>(y), codes_hi<kFmt>(y)};
            float d[4];
            mma_16816_f16_zero(d, a, pb);
            float(&o)[4] = st.o[2 * wi + half];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = fmaf(d[i], sV, o[i]);
        }
    }
}

}  // namespace nosa
