// nosa_attend8.cuh -- attention of one staged block of the 8-bit KV store.
//
// NOSA pages: montaan.com summary of arXiv:2510.13602, "Empirical Results and Analysis" item 4
// (decoding is bound by KV loading); the pages keep the cache in 16 bits.
//
// Formula.  A block's keys stand for s_K c_jd and its values for s_V c'_jd, with 8-bit codes c
// (int8, or e4m3) and one fp32 scale each.  With x_j = s_K scale log2(e) (q . c_j) + e_j log2(e):
//   o = s_V sum_j 2^(x_j - m) c'_j,   l = sum_j 2^(x_j - m),   out = o / l.
// The scales come out of both products, so the matrix instructions run on the codes.
//
// int8: both products are exact in integers.  A query row becomes 23-bit integers against its largest
// value, three signed bytes each (a bf16 value down to 2^-14 of the largest keeps every bit, a smaller
// one is off by at most 2^-22 of it); where some row's largest value is 64 times its mean or more,
// 31-bit integers and a fourth byte (2^-22, 2^-30).  P becomes 16-bit integers against the block's own largest weight
// (off by at most 2^-17 of that), two bytes each.  An int8 instruction covers twice the depth of an f16
// one in the same 8 clocks (measured), and nothing has to be converted: attending a block takes a warp
// 2400 clocks by way of f16 pairs and 2100 this way, two warps on one scheduler 1780 and 1600 each.
// The int32 sums start at the bits of 1.5 * 2^23: read as floats less that number they are
// themselves, since all stay below 2^22.
//
// e4m3: every value is exact in f16, as is a bf16 query row once a power of two brings its largest
// value to [2^14, 2^15): values down to 2^-31 of the largest keep every bit, smaller ones are off by at
// most 2^-39 of it.  2^(x - m) goes to f16, 11 bits where the bf16 store's path has 8; m is kept 14
// below the running maximum, by the newest block (bf16) too, so that the largest is 2^14 and the smallest
// normal one 2^-28 of it: a token loses bits only below that, and is lost only below 2^-39 of the largest
// (2^20 tokens of that size are 2^-19 of the sum).  The codes become f16 pairs by the conversion
// instruction.
//
// Layout.  One warp attends a whole block of 64 tokens, in four slices of 16: S^T = C Q^T and
// O^T += C'^T P^T (attend_block gives a block to four warps).  The maximum, its two reductions over
// lanes, the rescaling and the scale of the values are paid once per block, and the four slices keep
// the matrix instructions' latency covered.  One 16-byte shared load holds 16 dims of a row.
#pragma once

#include <type_traits>

#include "nosa_attend.cuh"

namespace nosa {

// The dims of a lane's accumulators: o[t][0..1] hold dim psi(t, sig) of heads 2c, 2c+1 and
// o[t][2..3] dim psi(t, sig) + 1; at() places a dim in the merge scratch so that a warp's stores of
// one t hit 32 distinct banks.
struct DimsBf16 {  // two 16-byte chunks of a 256-byte row, one in each 128-byte half
    static __device__ __forceinline__ int psi(int t, int sig) { return 64 * (t >> 2) + 8 * sig + 2 * (t & 3); }
    static __device__ __forceinline__ int at(int x) { return swz(x); }
};
struct Dims8 {  // one 16-byte chunk of a 128-byte row
    static __device__ __forceinline__ int psi(int t, int sig) { return 16 * sig + 2 * t; }
    static __device__ __forceinline__ int at(int x) { return x ^ ((x >> 5) & 1) ^ (((x >> 6) & 1) << 3); }
};

// An item's sums of 2^x, for heads 2c and 2c + 1 and this lane's tokens: s0 and s1, relative to m0 and m1.
struct ItemSums {
    float s0, s1, m0, m1;
};

// Leave an item's weights, per head, for the unit's last CTA: rec[h] = v, the log2 of the sum of 2^x over
// its tokens, -inf where nothing is seen.  A weight wants v to an absolute error, and next to a large m a
// float holds none of log2(s): a unit whose logits all lie at -1e9, or at the lowest finite value, would have no
// shares left.  What the heads' x have in common is the logit.  So there v is taken against the item's
// largest logit, which is found again in the store when it is wanted (e, n: the item's logits in
// shared memory), and left as 2^40 v, at least 2^16 in magnitude; a plain v stays below 2^12.  Up to kNear a
// plain v, below 256, is off by no more than an x of that size (half a step: 2^-17).  *far: set if some v is not
// plain; adding the weights up then reads the logits once more (8 sequences of 16K: 38 us instead of 24).
// After the block's attention: within it, the rare branch cost 1.0 us of 26 (8 sequences of up to 16K, int8).
constexpr float kNear = 240.f, kFarScale = 0x1p40f, kFarLeast = 4096.f;
__device__ __forceinline__ float item_value(float s, float m, float top) {
    const float l = log2_fast(s), d = m - top;
    if (s == 0.f) return kNegInf;
    if (fabsf(m) <= kNear) return m + l;
    const float v = l + d;
    return (fabsf(v) < 0x1p-24f ? 0x1p-24f : v) * kFarScale;
}
__device__ __forceinline__ bool is_far(float v) { return fabsf(v) >= kFarLeast && v != kNegInf; }
__device__ __forceinline__ void leave_weights(float *rec, volatile int *far, ItemSums w, const float *e, int n, int r,
                                              int c) {
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
        w.s0 += __shfl_xor_sync(0xFFFFFFFFu, w.s0, sh);
        w.s1 += __shfl_xor_sync(0xFFFFFFFFu, w.s1, sh);
    }
    float2 v = make_float2(w.m0 + log2_fast(w.s0), w.m1 + log2_fast(w.s1));
    if (__any_sync(0xFFFFFFFFu, fmaxf(fabsf(w.m0), fabsf(w.m1)) > kNear)) {
        float top = kNegInf;
        for (int i = r; i < n; i += 8) top = fmaxf(top, bias_log2(e[i]));
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, sh));
        v = make_float2(item_value(w.s0, w.m0, top), item_value(w.s1, w.m1, top));
        if (is_far(v.x) || is_far(v.y)) *far = 1;
    }
    if (r == 0) *reinterpret_cast<float2 *>(rec + 2 * c) = v;
}

// The item has nothing to attend: its weights are zero.
__device__ __forceinline__ void leave_none(float *rec, int r, int c) {
    if (r == 0) *reinterpret_cast<float2 *>(rec + 2 * c) = make_float2(kNegInf, kNegInf);
}

// The two low (two high) e4m3 codes of a word as an f16 pair.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
    uint32_t r;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo; }" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
    uint32_t r;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi; }" : "=r"(r) : "r"(w));
    return r;
}

// A unit's queries as fragments (dims ordered as the key loads), and for heads 2c and 2c + 1 what a unit
// of them stands for: f16 pairs over the e4m3 store, three signed bytes over the int8 store (the top
// one first).
constexpr int kQueryBytes = 3;
template <int kFmt>
struct Query8 {
    uint32_t f[8][2];
    float s0, s1;
};
template <>
struct Query8<kFmtInt8> {
    uint32_t f[kQueryBytes][4][2];
    float s0, s1;
    bool four;  // a fourth byte is wanted (the same in all lanes); fourth_byte makes it when it is used
};

// This lane's dims 16c..16c+15 and 64+16c..64+16c+15 of head r, the head's largest magnitude's
// exponent field (255: not finite), and whether the unit wants a fourth byte.
__device__ __forceinline__ void load_row(uint4 (&x)[4], const uint16_t *q, int G, int r, int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = r < G ? reinterpret_cast<const uint4 *>(q + r * kD)[8 * (i >> 1) + 2 * c + (i & 1)]
                     : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ uint32_t row_exponent(const uint4 (&x)[4], bool &four) {
    float a = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float y = fabsf(bf16_lo(word(x[i], j))), z = fabsf(bf16_hi(word(x[i], j)));
            a = max_nan(a, max_nan(y, z));
            sum += y + z;
        }
#pragma unroll
    for (int sh = 1; sh < 4; sh <<= 1) {
        a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, sh));
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, sh);
    }
    four = __any_sync(0xFFFFFFFFu, a > 0.f && a * (kD / 64) >= sum);  // 64 times the mean
    return (__float_as_uint(a) >> 23) & 255u;  // a in [2^(E - 127), 2^(E - 126))
}

// Dims 8i + 4h .. + 3 of a lane's as integers: times 2^29 (a fourth byte) or 2^21 over 2^(E - 127).
__device__ __forceinline__ void row_ints(int (&v)[4], const uint4 &x, int h, uint32_t E, bool four) {
    const float up = __uint_as_float(((four ? 283u : 275u) - E) << 23);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t w = word(x, 2 * h + (d >> 1));
        v[d] = __float2int_rn((d & 1 ? bf16_hi(w) : bf16_lo(w)) * up);
    }
}
// Their lowest signed bytes as one word, which leave them (v becomes (v - byte) / 256).
__device__ __forceinline__ uint32_t take_bytes(int (&v)[4]) {
    const uint32_t b = __byte_perm(__byte_perm(v[0], v[1], 0x0040), __byte_perm(v[2], v[3], 0x0040), 0x5410);
#pragma unroll
    for (int d = 0; d < 4; ++d) v[d] = (v[d] - (int)(int8_t)v[d]) >> 8;
    return b;
}
__device__ __forceinline__ uint32_t int_exponent(uint32_t E) { return min(max(E, 30u), 254u); }

template <int kFmt>
__device__ __forceinline__ void load_query8(Query8<kFmt> &Q, const uint16_t *q, int G, int r, int c) {
    uint4 x[4];
    bool four;
    load_row(x, q, G, r, c);
    const uint32_t E0 = row_exponent(x, four);
    float s;
    if constexpr (kFmt == kFmtInt8) {
        const uint32_t E = int_exponent(E0);
        Q.four = four;
        s = E0 == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((E - (four ? 29u : 21u)) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int v[4];
                row_ints(v, x[i], h, E, four);
                if (four) take_bytes(v);
#pragma unroll
                for (int k = kQueryBytes - 1; k >= 0; --k) Q.f[k][i][h] = take_bytes(v);
            }
    } else {
        const uint32_t E = E0 == 255u ? 127u : min(max(E0, 15u), 253u);  // not finite, nor are the scores
        const float up = __uint_as_float((254u + 14u - E) << 23);         // 2^(127 + 14 - E)
        s = __uint_as_float((E - 14u) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                Q.f[2 * i + (j >> 1)][j & 1] = pack_f16x2(bf16_lo(word(x[i], j)) * up, bf16_hi(word(x[i], j)) * up);
    }
    Q.s0 = __shfl_sync(0xFFFFFFFFu, s, 8 * c);
    Q.s1 = __shfl_sync(0xFFFFFFFFu, s, 8 * c + 4);
}

constexpr float kPBias = 14.f;  // e4m3: m is the running maximum less this

// The softmax step of one block in a warp: x[i] holds slice i's logits (rows r and r + 8 of the slice,
// heads 2c and 2c + 1) in the log2 domain.  Updates m and l, rescales o, leaves P in p.  NaN is
// carried on (attend_block passes over it).  bias: m is the maximum less this. ws (with kWeights):
// the block's sums.
template <bool kWeights, bool kF16>
__device__ __forceinline__ void softmax_step(WarpState &st, float (&x)[4][4], uint32_t (&pb)[4][2], float bias,
                                             ItemSums &ws) {
    float bm0 = max_nan(x[0][0], x[0][2]), bm1 = max_nan(x[0][1], x[0][3]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        bm0 = max_nan(bm0, max_nan(x[i][0], x[i][2]));
        bm1 = max_nan(bm1, max_nan(x[i][1], x[i][3]));
    }
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
        bm0 = max_nan(bm0, __shfl_xor_sync(0xFFFFFFFFu, bm0, sh));
        bm1 = max_nan(bm1, __shfl_xor_sync(0xFFFFFFFFu, bm1, sh));
    }
    const float mn0 = max_nan(st.m0, bm0 - bias), mn1 = max_nan(st.m1, bm1 - bias);
    const float ms0 = mn0 == kNegInf ? 0.f : mn0, ms1 = mn1 == kNegInf ? 0.f : mn1;  // nothing seen yet: all zeros
    const float c0 = exp2_fast(st.m0 - ms0), c1 = exp2_fast(st.m1 - ms1);
    float s0 = 0.f, s1 = 0.f;    // of P as it goes into the product: the denominator sums what the numerator sums
    float w0 = 0.f, w1 = 0.f;    // of P before its rounding
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float p0 = exp2_fast(x[i][0] - ms0), p1 = exp2_fast(x[i][1] - ms1);
        const float p2 = exp2_fast(x[i][2] - ms0), p3 = exp2_fast(x[i][3] - ms1);
        const uint32_t lo = kF16 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
        const uint32_t hi = kF16 ? pack_f16x2(p2, p3) : pack_bf16x2(p2, p3);
        pb[i][0] = movmatrix_trans(lo);
        pb[i][1] = movmatrix_trans(hi);
        if constexpr (kWeights) {
            w0 += p0 + p2;
            w1 += p1 + p3;
        } else {
            const float2 a = kF16 ? unpack_f16x2(lo) : make_float2(bf16_lo(lo), bf16_hi(lo));
            const float2 b = kF16 ? unpack_f16x2(hi) : make_float2(bf16_lo(hi), bf16_hi(hi));
            s0 += a.x + b.x;
            s1 += a.y + b.y;
        }
    }
    // with weights, both sums without P's rounding (which is unbiased: out moves by less than its own last bit)
    st.l0 = fmaf(st.l0, c0, kWeights ? w0 : s0);
    st.l1 = fmaf(st.l1, c1, kWeights ? w1 : s1);
    st.m0 = mn0;
    st.m1 = mn1;
    if constexpr (kWeights) ws = ItemSums{w0, w1, ms0, ms1};
    if (__any_sync(0xFFFFFFFFu, c0 != 1.f || c1 != 1.f)) {  // the maximum rises a few times in a long context
#pragma unroll
        for (int tt = 0; tt < 8; ++tt) {
            st.o[tt][0] *= c0; st.o[tt][1] *= c1;
            st.o[tt][2] *= c0; st.o[tt][3] *= c1;
        }
    }
}

// One block of codes (t: 64 key rows, then 64 value rows, 128 bytes each, 128-byte swizzle), every
// token of it before the newest block.  sK, sV: its scales.  kWeights: leave its weights in rec.
template <bool kWeights>
__device__ __forceinline__ void attend8(WarpState &st, const Query8<kFmtE4m3> &Q, const uint16_t *, int,
                                        const uint8_t *t, const float *eb, float sK, float sV, float qk_log2, int r,
                                        int c, int sig, ItemSums &ws) {
    float x[4][4];
    // ---- S^T (4 slices of 16 tokens x 8 heads) ----
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint8_t *kp = t + sig * kRow8Bytes + (((c + 4 * j) ^ sig) << 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 ka = lds128(kp + 16 * i * kRow8Bytes), kb = lds128(kp + (16 * i + 8) * kRow8Bytes);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t y = word(ka, w), z = word(kb, w);
                const uint32_t a[4] = {codes_lo(y), codes_lo(z), codes_hi(y), codes_hi(z)};
                mma_16816_f16(x[i], a, Q.f[4 * j + w]);
            }
        }
    }
    const float f0 = qk_log2 * sK * Q.s0, f1 = qk_log2 * sK * Q.s1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float eA = bias_log2(eb[16 * i + sig]), eB = bias_log2(eb[16 * i + sig + 8]);
        x[i][0] = fmaf(x[i][0], f0, eA);
        x[i][1] = fmaf(x[i][1], f1, eA);
        x[i][2] = fmaf(x[i][2], f0, eB);
        x[i][3] = fmaf(x[i][3], f1, eB);
    }
    uint32_t pb[4][2];
    softmax_step<kWeights, true>(st, x, pb, kPBias, ws);
    // ---- O^T (128 dims x 8 heads) += s_V C'^T P^T ----
    float d[8][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t *vb = t + kHalfBlock8Bytes + (16 * i + c) * kRow8Bytes;
        const int off0 = ((sig ^ c) << 4), off1 = ((sig ^ (c + 4)) << 4);
        const uint4 v0 = lds128(vb + off0), v1 = lds128(vb + 4 * kRow8Bytes + off1);
        const uint4 v2 = lds128(vb + 8 * kRow8Bytes + off0), v3 = lds128(vb + 12 * kRow8Bytes + off1);
#pragma unroll
        for (int tt = 0; tt < 8; ++tt) {  // dims 2 tt, 2 tt + 1 of the chunk: bytes of two tokens side by side
            const int sel = (tt & 1) ? 0x7362 : 0x5140;
            const uint32_t z = __byte_perm(word(v0, tt >> 1), word(v1, tt >> 1), sel);
            const uint32_t y = __byte_perm(word(v2, tt >> 1), word(v3, tt >> 1), sel);
            const uint32_t a[4] = {codes_lo(z), codes_hi(z), codes_lo(y), codes_hi(y)};
            if (i == 0) mma_16816_f16_zero(d[tt], a, pb[i]);
            else mma_16816_f16(d[tt], a, pb[i]);
        }
    }
#pragma unroll
    for (int tt = 0; tt < 8; ++tt)
#pragma unroll
        for (int j = 0; j < 4; ++j) st.o[tt][j] = fmaf(d[tt][j], sV, st.o[tt][j]);
}

// The int32 sums' start, and a sum as a float.
constexpr int32_t kSumBits = 0x4B400000;  // 1.5 * 2^23
__device__ __forceinline__ float sum_value(int32_t d) { return __int_as_float(d) - 12582912.f; }

// The queries' fourth byte, for a unit that wants it (made here from the queries in memory: the
// registers of the usual case are worth more).
__device__ __forceinline__ void fourth_byte(float (&x)[4][4], const uint16_t *q, int G, const uint8_t *t, int r, int c,
                                            int sig) {
    uint4 row[4];
    bool four;
    load_row(row, q, G, r, c);
    const uint32_t E = int_exponent(row_exponent(row, four));
    uint32_t f[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int v[4];
            row_ints(v, row[i], h, E, true);
            f[i][h] = take_bytes(v);
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int32_t d[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint8_t *kp = t + (16 * i + sig) * kRow8Bytes + (((c + 4 * j) ^ sig) << 4);
            const uint4 ka = lds128(kp), kb = lds128(kp + 8 * kRow8Bytes);
            const uint32_t a0[4] = {ka.x, kb.x, ka.y, kb.y}, a1[4] = {ka.z, kb.z, ka.w, kb.w};
            if (j == 0) mma_16832_s8<true>(d, a0, f[0], kSumBits);
            else mma_16832_s8<false>(d, a0, f[2], 0);
            mma_16832_s8<false>(d, a1, f[2 * j + 1], 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = fmaf(x[i][j], 256.f, sum_value(d[j]));
    }
}

// The same over int8 codes.  q: the unit's queries in memory, G rows.
template <bool kWeights>
__device__ __forceinline__ void attend8(WarpState &st, const Query8<kFmtInt8> &Q, const uint16_t *q, int G,
                                        const uint8_t *t, const float *eb, float sK, float sV, float qk_log2, int r,
                                        int c, int sig, ItemSums &ws) {
    // ---- S^T (4 slices of 16 tokens x 8 heads), a sum per byte of the queries ----
    float x[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int32_t d[kQueryBytes][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint8_t *kp = t + (16 * i + sig) * kRow8Bytes + (((c + 4 * j) ^ sig) << 4);
            const uint4 ka = lds128(kp), kb = lds128(kp + 8 * kRow8Bytes);
            const uint32_t a0[4] = {ka.x, kb.x, ka.y, kb.y}, a1[4] = {ka.z, kb.z, ka.w, kb.w};
#pragma unroll
            for (int k = 0; k < kQueryBytes; ++k) {
                if (j == 0) mma_16832_s8<true>(d[k], a0, Q.f[k][0], kSumBits);
                else mma_16832_s8<false>(d[k], a0, Q.f[k][2], 0);
            }
#pragma unroll
            for (int k = 0; k < kQueryBytes; ++k) mma_16832_s8<false>(d[k], a1, Q.f[k][2 * j + 1], 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[i][j] = fmaf(fmaf(sum_value(d[0][j]), 256.f, sum_value(d[1][j])), 256.f, sum_value(d[2][j]));
    }
    if (Q.four) fourth_byte(x, q, G, t, r, c, sig);
    const float f0 = qk_log2 * sK * Q.s0, f1 = qk_log2 * sK * Q.s1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float eA = bias_log2(eb[16 * i + sig]), eB = bias_log2(eb[16 * i + sig + 8]);
        x[i][0] = fmaf(x[i][0], f0, eA);
        x[i][1] = fmaf(x[i][1], f1, eA);
        x[i][2] = fmaf(x[i][2], f0, eB);
        x[i][3] = fmaf(x[i][3], f1, eB);
    }
    // ---- the block's largest logits and its weights against them ----
    float bm0 = max_nan(x[0][0], x[0][2]), bm1 = max_nan(x[0][1], x[0][3]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        bm0 = max_nan(bm0, max_nan(x[i][0], x[i][2]));
        bm1 = max_nan(bm1, max_nan(x[i][1], x[i][3]));
    }
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
        bm0 = max_nan(bm0, __shfl_xor_sync(0xFFFFFFFFu, bm0, sh));
        bm1 = max_nan(bm1, __shfl_xor_sync(0xFFFFFFFFu, bm1, sh));
    }
    const float bs0 = bm0 == kNegInf ? 0.f : bm0, bs1 = bm1 == kNegInf ? 0.f : bm1;  // nothing seen: all zeros
    float w0 = 0.f, w1 = 0.f;
    uint32_t ph[4], pl[4];  // this lane's four tokens of slice i (rows c, c + 4, c + 8, c + 12) for head r
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        constexpr float kTop = 65535.f, kBig = 8388608.f;  // 2^23 + n has n in its low bits
        const float p0 = exp2_fast(x[i][0] - bs0), p1 = exp2_fast(x[i][1] - bs1);
        const float p2 = exp2_fast(x[i][2] - bs0), p3 = exp2_fast(x[i][3] - bs1);
        w0 += p0 + p2;
        w1 += p1 + p3;
        const uint32_t n0 = __float_as_uint(fmaf(p0, kTop, kBig)), n1 = __float_as_uint(fmaf(p1, kTop, kBig));
        const uint32_t n2 = __float_as_uint(fmaf(p2, kTop, kBig)), n3 = __float_as_uint(fmaf(p3, kTop, kBig));
        const uint32_t lo = movmatrix_trans(__byte_perm(n0, n1, 0x5410));
        const uint32_t hi = movmatrix_trans(__byte_perm(n2, n3, 0x5410));
        ph[i] = __byte_perm(lo, hi, 0x7531);
        pl[i] = __byte_perm(lo, hi, 0x6420);
    }
    if constexpr (kWeights) ws = ItemSums{w0, w1, bs0, bs1};
    const float mn0 = max_nan(st.m0, bm0), mn1 = max_nan(st.m1, bm1);
    const float ms0 = mn0 == kNegInf ? 0.f : mn0, ms1 = mn1 == kNegInf ? 0.f : mn1;
    const float c0 = exp2_fast(st.m0 - ms0), c1 = exp2_fast(st.m1 - ms1);
    const float b0 = exp2_fast(bm0 - ms0), b1 = exp2_fast(bm1 - ms1);  // the block against the whole
    // the denominator sums the weights before their rounding (to the nearest, without a bias)
    st.l0 = fmaf(st.l0, c0, b0 * w0);
    st.l1 = fmaf(st.l1, c1, b1 * w1);
    st.m0 = mn0;
    st.m1 = mn1;
    if (__any_sync(0xFFFFFFFFu, c0 != 1.f || c1 != 1.f)) {  // the maximum rises a few times in a long context
#pragma unroll
        for (int tt = 0; tt < 8; ++tt) {
            st.o[tt][0] *= c0; st.o[tt][1] *= c1;
            st.o[tt][2] *= c0; st.o[tt][3] *= c1;
        }
    }
    // ---- O^T (128 dims x 8 heads) += s_V C'^T P^T, a sum per byte of P ----
    int32_t dh[8][4], dl[8][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // two slices, 32 tokens
        const uint32_t Bh[2] = {ph[2 * k], ph[2 * k + 1]}, Bl[2] = {pl[2 * k], pl[2 * k + 1]};
        uint4 v[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t *vb = t + kHalfBlock8Bytes + (16 * (2 * k + i) + c) * kRow8Bytes;
            const int off0 = ((sig ^ c) << 4), off1 = ((sig ^ (c + 4)) << 4);
            v[i][0] = lds128(vb + off0);
            v[i][1] = lds128(vb + 4 * kRow8Bytes + off1);
            v[i][2] = lds128(vb + 8 * kRow8Bytes + off0);
            v[i][3] = lds128(vb + 12 * kRow8Bytes + off1);
        }
#pragma unroll
        for (int tt = 0; tt < 8; ++tt) {  // dims 2 tt, 2 tt + 1 of the chunk: a byte of each of four tokens side by side
            const int sel = (tt & 1) ? 0x7362 : 0x5140, w = tt >> 1;
            uint32_t a[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t y = __byte_perm(word(v[i][0], w), word(v[i][1], w), sel);
                const uint32_t z = __byte_perm(word(v[i][2], w), word(v[i][3], w), sel);
                a[2 * i] = __byte_perm(y, z, 0x5410);
                a[2 * i + 1] = __byte_perm(y, z, 0x7632);
            }
            if (k == 0) {
                mma_16832_s8u8<true>(dh[tt], a, Bh, kSumBits);
                mma_16832_s8u8<true>(dl[tt], a, Bl, kSumBits);
            } else {
                mma_16832_s8u8<false>(dh[tt], a, Bh, 0);
                mma_16832_s8u8<false>(dl[tt], a, Bl, 0);
            }
        }
    }
    const float k0 = b0 * (sV * (1.f / 65535.f)), k1 = b1 * (sV * (1.f / 65535.f));
#pragma unroll
    for (int tt = 0; tt < 8; ++tt)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            st.o[tt][j] = fmaf(fmaf(sum_value(dh[tt][j]), 256.f, sum_value(dl[tt][j])), (j & 1) ? k1 : k0, st.o[tt][j]);
}

// One bf16 block by one warp (kt: its key rows, vt: its value rows, two boxes each): the tail of an 8-bit store (Dims8: the value loads then have a two-way
// bank conflict, on one block of a unit), or a block of the bf16 store whose weights are kept.  Tokens
// at or beyond L are not seen.
// kBias: softmax_step's, that of the unit's other blocks.
template <class Dims, bool kWeights, bool kBias>
__device__ __forceinline__ void attend16(WarpState &st, const uint32_t (&qf)[8][2], const uint8_t *kt, const uint8_t *vt,
                                         const float *eb, int32_t lb, int32_t L, float qk_log2, int r, int c, int sig, ItemSums &ws) {
    constexpr bool kWide = std::is_same<Dims, Dims8>::value;  // chunks 2 sig, 2 sig + 1 of the row
    const int32_t n = min(L - lb * kBlock, kBlock);            // tokens seen
    float x[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint8_t *kp = kt + (j >> 1) * kBoxBytes + sig * 128 + (((((j & 1) << 2) + c) ^ sig) << 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 ka = lds128(kp + 16 * i * 128), kb = lds128(kp + (16 * i + 8) * 128);
            const uint32_t a0[4] = {ka.x, kb.x, ka.y, kb.y};
            const uint32_t a1[4] = {ka.z, kb.z, ka.w, kb.w};
            mma_16816(x[i], a0, qf[2 * j]);
            mma_16816(x[i], a1, qf[2 * j + 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int rowA = 16 * i + sig, rowB = rowA + 8;
        const float eA = bias_log2(eb[rowA]), eB = bias_log2(eb[rowB]);
        x[i][0] = rowA < n ? fmaf(x[i][0], qk_log2, eA) : kNegInf;
        x[i][1] = rowA < n ? fmaf(x[i][1], qk_log2, eA) : kNegInf;
        x[i][2] = rowB < n ? fmaf(x[i][2], qk_log2, eB) : kNegInf;
        x[i][3] = rowB < n ? fmaf(x[i][3], qk_log2, eB) : kNegInf;
    }
    uint32_t pb[4][2];
    softmax_step<kWeights, false>(st, x, pb, kBias ? kPBias : 0.f, ws);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (16 * i >= n) break;  // every P left is zero
        const int vt0 = 16 * i + c;
#pragma unroll
        for (int bx = 0; bx < 2; ++bx) {
            const uint8_t *vb = vt + (kWide ? sig >> 2 : bx) * kBoxBytes;
            const int ch = kWide ? 2 * (sig & 3) + bx : sig;
            uint4 v0 = lds128(vb + (vt0 + 0) * 128 + ((ch ^ c) << 4));
            uint4 v1 = lds128(vb + (vt0 + 4) * 128 + ((ch ^ (c + 4)) << 4));
            uint4 v2 = lds128(vb + (vt0 + 8) * 128 + ((ch ^ c) << 4));
            uint4 v3 = lds128(vb + (vt0 + 12) * 128 + ((ch ^ (c + 4)) << 4));
            if (n < kBlock) {  // rows at or beyond L hold stale bits: keep them out of 0 * x
                const uint4 z = make_uint4(0, 0, 0, 0);
                if (vt0 >= n) v0 = z;
                if (vt0 + 4 >= n) v1 = z;
                if (vt0 + 8 >= n) v2 = z;
                if (vt0 + 12 >= n) v3 = z;
            }
#pragma unroll
            for (int wi = 0; wi < 4; ++wi) {
                const uint32_t y0 = word(v0, wi), y1 = word(v1, wi), y2 = word(v2, wi), y3 = word(v3, wi);
                const uint32_t a[4] = {__byte_perm(y0, y1, 0x5410), __byte_perm(y0, y1, 0x7632),
                                       __byte_perm(y2, y3, 0x5410), __byte_perm(y2, y3, 0x7632)};
                mma_16816(st.o[4 * bx + wi], a, pb[i]);
            }
        }
    }
}

}  // namespace nosa
