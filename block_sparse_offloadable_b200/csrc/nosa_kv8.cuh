// nosa_kv8.cuh -- a block's keys and values in 8 bits, with one scale each.
//
// NOSA pages: montaan.com summary of arXiv:2510.13602, "System Optimization (NOSI)" item 2 (the KV
// cache in block-sized units on both sides); the pages keep it in 16 bits.
//
// Formula, per 64 x 128 half (keys or values) of a block, with M = 127 (int8) or 448 (e4m3):
//   a = max |x|;  s = fl32(a fl32(1 / M)), r = fl32(fl32(1 / a) M);  code = rint(x r) (int8: one rounding of the exact
//   product, ties to even) or e4m3(fl32(x r)) (nearest, ties to even, saturating);  value = code s.
//   a < 2^-100: s = 0 and codes 0.  Some x not finite: s = NaN and codes 0, so that attention over
//   the block is NaN rather than silently wrong.
// A block is coded once, from its bf16 rows, when it becomes a candidate: no token is coded twice.
#pragma once

#include "nosa_internal.cuh"

namespace nosa {

constexpr float kInt8Max = 127.f, kE4m3Max = 448.f;
constexpr uint32_t kBf16Inf = 0x7F80u;

// Largest |x| of a bf16 pair's halves, as bf16 bits (integer order is the order of magnitudes, and
// infinity and NaN are the largest, so nothing that is not finite gets lost).
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) { return __vmaxu2(a, b & 0x7FFF7FFFu); }
__device__ __forceinline__ uint32_t absmax4(uint32_t a, const uint4 &v) {
    return absmax2(absmax2(absmax2(absmax2(a, v.x), v.y), v.z), v.w);
}
__device__ __forceinline__ uint32_t absmax_warp(uint32_t a) {
    a = max(a & 0xFFFFu, a >> 16);
    return __reduce_max_sync(0xFFFFFFFFu, a);
}

// (s, r) of a half whose largest magnitude has these bf16 bits; r = 0 where every code is 0.
__device__ __forceinline__ float2 scale_of(uint32_t bits, int fmt) {
    const float a = __uint_as_float(bits << 16), M = fmt == kFmtInt8 ? kInt8Max : kE4m3Max;
    if (bits >= kBf16Inf) return make_float2(__uint_as_float(0x7FC00000u), 0.f);
    if (a < 0x1p-100f) return make_float2(0.f, 0.f);
    return make_float2(__fmul_rn(a, fmt == kFmtInt8 ? 1.f / kInt8Max : 1.f / kE4m3Max), __fmul_rn(__frcp_rn(a), M));
}

// Four bf16 values (two words) to four codes (one word, first value in the low byte).
__device__ __forceinline__ uint32_t code4(uint32_t w0, uint32_t w1, float r, int fmt) {
    const float x0 = bf16_lo(w0), x1 = bf16_hi(w0), x2 = bf16_lo(w1), x3 = bf16_hi(w1);
    if (r == 0.f) return 0u;  // zeros, and rows beside a value that is not finite
    if (fmt == kFmtInt8) {
        // 1.5 * 2^23 + n has n in its low bits: the fused multiply-add rounds x r once
        constexpr float kBig = 12582912.f;
        const uint32_t a = __float_as_uint(__fmaf_rn(x0, r, kBig)), b = __float_as_uint(__fmaf_rn(x1, r, kBig));
        const uint32_t c = __float_as_uint(__fmaf_rn(x2, r, kBig)), d = __float_as_uint(__fmaf_rn(x3, r, kBig));
        return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
    }
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(x0, r), __fmul_rn(x1, r)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(x2, r), __fmul_rn(x3, r)), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ uint2 code8(const uint4 &v, float r, int fmt) {
    return make_uint2(code4(v.x, v.y, r, fmt), code4(v.z, v.w, r, fmt));
}

// Code the block in `tail` (64 key rows, 64 value rows, bf16), whose logits are e, into the record
// dst, by one warp.  Twice over the 32 KiB, which the L2 holds; eight loads in flight.
__device__ __forceinline__ void code_tail(const uint8_t *tail, const float *e, uint8_t *dst, int lane, int fmt) {
    constexpr int kPer = kHalfBlockBytes / 16 / 32;  // 16-byte pieces per lane and half
    float *side = reinterpret_cast<float *>(dst + kBlock8Bytes);
    float2 s[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint4 *src = reinterpret_cast<const uint4 *>(tail + half * kHalfBlockBytes) + lane;
        uint32_t a = 0;
#pragma unroll 8
        for (int i = 0; i < kPer; ++i) a = absmax4(a, src[32 * i]);
        s[half] = scale_of(absmax_warp(a), fmt);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint4 *src = reinterpret_cast<const uint4 *>(tail + half * kHalfBlockBytes) + lane;
        uint2 *to = reinterpret_cast<uint2 *>(dst + half * kHalfBlock8Bytes) + lane;
#pragma unroll 8
        for (int i = 0; i < kPer; ++i) to[32 * i] = code8(src[32 * i], s[half].y, fmt);
    }
    side[lane] = e[lane];
    side[lane + 32] = e[lane + 32];
    if (lane < 2) side[kBlock + lane] = lane ? s[1].x : s[0].x;
}

}  // namespace nosa
