// nosa_topk.cuh -- the k largest of n keys in shared memory, by one CTA of 256 threads.
//
// Radix selection: 8 bits at a time from the top, a histogram of the keys that agree with the digits
// found so far, and the digit in which the k-th largest lies; done early once every key of that bucket
// is among the k (for random keys after two or three digits).  A pass takes about 0.3 us.
#pragma once

#include "nosa_common.cuh"

namespace nosa {

constexpr int kTopThreads = 256;

struct TopShared {
    int32_t hist[256], warp_sum[kTopThreads / 32], digit, left, count;
};

// Exclusive prefix sum over the CTA; the total to *sum.  Two barriers.
__device__ __forceinline__ int32_t cta_scan(int32_t v, TopShared &s, int32_t *sum) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) s.warp_sum[warp] = incl;
    __syncthreads();
    int32_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kTopThreads / 32; ++w) {
        if (w < warp) base += s.warp_sum[w];
        all += s.warp_sum[w];
    }
    *sum = all;
    return base + incl - v;
}

// The k largest keys are those with (key & mask) > value, and the first `ties`, by index, of those with
// (key & mask) == value.
template <class Key>
struct TopK {
    Key value, mask;
    int32_t ties;
};

// keys[0 .. n), 0 < k < n, written before a barrier.
template <class Key>
__device__ __forceinline__ TopK<Key> top_k(const Key *keys, int32_t n, int32_t k, TopShared &s) {
    TopK<Key> t = {0, 0, k};
    const int tid = threadIdx.x;
#pragma unroll 1
    for (int shift = 8 * (int)sizeof(Key) - 8; shift >= 0; shift -= 8) {
        s.hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kTopThreads)
            if ((keys[i] & t.mask) == t.value) atomicAdd(&s.hist[(int)(keys[i] >> shift) & 255], 1);
        __syncthreads();
        int32_t sum;
        const int32_t mine = s.hist[255 - tid];
        const int32_t above = cta_scan(mine, s, &sum);  // keys with a larger digit
        if (above < t.ties && t.ties <= above + mine) {
            s.digit = 255 - tid;
            s.left = t.ties - above;
            s.count = mine;
        }
        __syncthreads();
        t.value |= (Key)s.digit << shift;
        t.mask |= (Key)255 << shift;
        t.ties = s.left;
        if (s.count == t.ties) break;
    }
    return t;
}

// Number the chosen of n keys in index order: keys[i] becomes its number, or all ones.  A thread takes
// consecutive keys.  Returns how many are chosen.  `all`: every key is.
template <class Key>
__device__ __forceinline__ int32_t number_chosen(Key *keys, int32_t n, bool all, int32_t k, TopShared &s) {
    TopK<Key> t = {0, 0, 0};
    const bool some = !all && k > 0;
    if (some) t = top_k(keys, n, k, s);
    const int32_t per = (n + kTopThreads - 1) / kTopThreads;
    const int32_t b0 = min((int)threadIdx.x * per, n), b1 = min(b0 + per, n);
    int32_t eq = 0, sum;
    if (some)
        for (int b = b0; b < b1; ++b) eq += (keys[b] & t.mask) == t.value;
    int32_t eq_at = cta_scan(eq, s, &sum);
    int32_t cnt = 0;
    for (int b = b0; b < b1; ++b) {
        bool stay = all;
        if (some) {
            const Key v = keys[b] & t.mask;
            stay = v > t.value || (v == t.value && eq_at++ < t.ties);
        }
        keys[b] = stay ? (Key)1 : (Key)0;
        cnt += stay;
    }
    int32_t at = cta_scan(cnt, s, &sum);
    for (int b = b0; b < b1; ++b) keys[b] = keys[b] ? (Key)at++ : ~(Key)0;
    __syncthreads();
    return sum;
}

}  // namespace nosa
