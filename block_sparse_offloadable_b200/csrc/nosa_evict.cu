// nosa_evict.cu -- eviction by accumulated attention weight: the blocks of a unit that are kept,
// moved into a state of smaller capacity.
//
// NOSA pages: montaan.com summary of arXiv:2510.13602, "Key Design Components" item 1 (a block the
// query-agnostic selection lets go is never selected by it again); the pages score blocks with a
// trained head, here the score is the attention weight that the block has got.
//
// Rule.  Of a unit's candidates (blocks 0 .. nb-1, the local block nb stays in any case) the first
// `sink` and the last `recent` are kept, and of the others those with the largest weight, `keep` in
// all; equal weights go to the lower block; a weight that is NaN counts as the largest.  The kept
// blocks keep their order and are numbered from 0.
//
// Two kernels.  choose: a CTA per unit finds the keep-th largest of the weights' order-preserving
// integer keys by four 8-bit histogram passes in shared memory, numbers the kept blocks with a scan,
// and writes what a unit has once (lengths, Gamma_e and the pool renumbered, weights).  move: a CTA
// per kept block copies its rows or codes, logits, pooled keys and score; only what the unit's
// tokens have filled is read or written.  Bound by HBM: every kept byte is read and written once.
#include "nosa_internal.cuh"

namespace nosa {

namespace {
constexpr int kChooseThreads = 256;
constexpr int kMoveThreads = 256;

// Larger weight, larger key; -0 and +0 the same; NaN above every number.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xFFFFFFFEu;
    return float_order(w == 0.f ? 0.f : w);
}
constexpr uint32_t kProtected = 0xFFFFFFFFu;

// Exclusive prefix sum over the CTA; total to *sum.  s_w: one word per warp.
__device__ __forceinline__ int32_t cta_scan(int32_t v, int32_t *s_w, int32_t *sum) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) s_w[warp] = incl;
    __syncthreads();
    int32_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kChooseThreads / 32; ++w) {
        if (w < warp) base += s_w[w];
        all += s_w[w];
    }
    *sum = all;
    return base + incl - v;
}

// Renumber a list of blocks (ids in order, those not kept left out) into dst; one warp.
__device__ __forceinline__ int32_t renumber(const int32_t *src, int32_t n, const int32_t *map, int32_t nb, int32_t *dst,
                                            int lane) {
    int32_t m = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const int32_t b = i < n ? src[i] : -1;
        const int32_t to = b >= 0 && b < nb ? map[b] : -1;
        const unsigned got = __ballot_sync(0xFFFFFFFFu, to >= 0);
        if (to >= 0) dst[m + __popc(got & ((1u << lane) - 1u))] = to;
        m += __popc(got);
    }
    return m;
}
}  // namespace

__global__ void __launch_bounds__(kChooseThreads) evict_choose_kernel(const EvictParams p) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ uint32_t keys[];  // [nblk]: the candidates' keys, then their new numbers
    __shared__ int32_t hist[256], s_w[kChooseThreads / 32], s_digit, s_left;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t u = blockIdx.x;
    const int32_t L = max(p.seq_len[u], 0);
    const int32_t nb = L > 0 ? (L - 1) / kBlock : 0;
    const float *w = p.weights + (int64_t)u * p.nblk;
    int32_t *kept = p.kept + (int64_t)u * (p.keep + 1);
    for (int i = tid; i < nb; i += kChooseThreads)
        keys[i] = (i < p.sink || i >= nb - p.recent) ? kProtected : weight_key(w[i]);
    // the keep-th largest key, and how many of the blocks with that key are kept
    uint32_t thr = 0;
    int32_t ties = 0;
    const bool all = nb <= p.keep;
    if (!all && p.keep > 0) {
        uint32_t mask = 0;
        int32_t left = p.keep;
        for (int shift = 24; shift >= 0; shift -= 8) {
            hist[tid] = 0;
            __syncthreads();
            for (int i = tid; i < nb; i += kChooseThreads)
                if ((keys[i] & mask) == thr) atomicAdd(&hist[(keys[i] >> shift) & 255u], 1);
            __syncthreads();
            int32_t sum;
            const int32_t above = cta_scan(hist[255 - tid], s_w, &sum);  // keys in larger digits
            if (above < left && left <= above + hist[255 - tid]) {
                s_digit = 255 - tid;
                s_left = left - above;
            }
            __syncthreads();
            thr |= (uint32_t)s_digit << shift;
            mask |= 255u << shift;
            left = s_left;
        }
        ties = left;
    }
    __syncthreads();
    // new numbers, in block order: a thread takes consecutive blocks
    const int32_t per = (nb + kChooseThreads - 1) / kChooseThreads;
    const int32_t b0 = min(tid * per, nb), b1 = min(b0 + per, nb);
    int32_t eq = 0, n = 0;
    if (!all && p.keep > 0)
        for (int b = b0; b < b1; ++b) eq += keys[b] == thr;
    int32_t sum;
    int32_t eq_at = cta_scan(eq, s_w, &sum);
    for (int b = b0; b < b1; ++b) {
        bool stay = all;
        if (!all && p.keep > 0) stay = keys[b] > thr || (keys[b] == thr && eq_at++ < ties);
        keys[b] = stay ? 1u : 0u;
        n += stay;
    }
    int32_t at = cta_scan(n, s_w, &sum);
    for (int b = b0; b < b1; ++b) {
        if (keys[b]) {
            kept[at] = b;
            keys[b] = (uint32_t)at++;
        } else {
            keys[b] = 0xFFFFFFFFu;  // -1
        }
    }
    const int32_t n_kept = sum;
    for (int i = n_kept + tid; i <= p.keep; i += kChooseThreads) kept[i] = (i == n_kept && L > 0) ? nb : -1;
    __syncthreads();  // kept (device memory, this CTA) and the numbers are written
    const int32_t n_blk = n_kept + (L > 0 ? 1 : 0);
    float *dw = p.dst_weights + (int64_t)u * p.dst_nblk;
    for (int i = tid; i < p.dst_nblk; i += kChooseThreads) dw[i] = i < n_blk ? w[kept[i]] : 0.f;
    const int32_t *map = reinterpret_cast<const int32_t *>(keys);
    if (warp == 0) {
        if (lane == 0) p.dst_seq_len[u] = L > 0 ? n_kept * kBlock + (L - nb * kBlock) : 0;
        if (p.k_e > 0) {
            const int32_t m = renumber(p.gamma_e + (int64_t)u * p.k_e, min(max(p.gamma_n[u], 0), p.k_e), map, nb,
                                       p.dst_gamma_e + (int64_t)u * p.k_e, lane);
            if (lane == 0) p.dst_gamma_n[u] = m;
        } else if (lane == 0) {
            p.dst_gamma_n[u] = 0;
        }
    }
    if (warp == 1 && p.pool) {
        const int32_t m = renumber(p.pool + (int64_t)u * p.nblk, min(max(p.pool_n[u], 0), p.nblk), map, nb,
                                   p.dst_pool + (int64_t)u * p.dst_nblk, lane);
        if (lane == 0) p.dst_pool_n[u] = m;
    }
}

// Copy n 16-byte pieces.
__device__ __forceinline__ void move16(uint8_t *dst, const uint8_t *src, int n) {
    const uint4 *s = reinterpret_cast<const uint4 *>(src);
    uint4 *d = reinterpret_cast<uint4 *>(dst);
    for (int i0 = threadIdx.x; i0 < n; i0 += 4 * kMoveThreads) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + j * kMoveThreads < n) v[j] = __ldcs(s + i0 + j * kMoveThreads);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + j * kMoveThreads < n) d[i0 + j * kMoveThreads] = v[j];
    }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
    pdl_wait();
    const int tid = threadIdx.x;
    const int32_t i = (int32_t)(blockIdx.x % (uint32_t)(p.keep + 1)), u = (int32_t)(blockIdx.x / (uint32_t)(p.keep + 1));
    const int32_t b = p.kept[(int64_t)u * (p.keep + 1) + i];
    if (b < 0) return;
    const int32_t rows = min(p.seq_len[u] - b * kBlock, kBlock);  // of the block's 64, those with a token
    const bool local = b == (p.seq_len[u] - 1) / kBlock;
    const int64_t sb = (int64_t)u * p.nblk + b, db = (int64_t)u * p.dst_nblk + i;
    if (p.fmt == kFmtBf16) {
        const uint8_t *s = p.store + sb * kBlockBytes;
        uint8_t *d = p.dst_store + db * kBlockBytes;
        move16(d, s, rows * (kRowBytes / 16));
        move16(d + kHalfBlockBytes, s + kHalfBlockBytes, rows * (kRowBytes / 16));
    } else if (local) {
        const uint8_t *s = p.tail + (int64_t)u * kBlockBytes;
        uint8_t *d = p.dst_tail + (int64_t)u * kBlockBytes;
        move16(d, s, rows * (kRowBytes / 16));
        move16(d + kHalfBlockBytes, s + kHalfBlockBytes, rows * (kRowBytes / 16));
    } else {
        move16(p.dst_store + db * kRec8Bytes, p.store + sb * kRec8Bytes, kHeld8Bytes / 16);
    }
    const int ck_bytes = kD * (p.ck_bf16 ? 2 : 4);  // one pooled key
    move16(p.dst_ck + db * kSubPerBlock * ck_bytes, p.ck + sb * kSubPerBlock * ck_bytes, rows / kSub * (ck_bytes / 16));
    if (tid < rows) p.dst_e[(int64_t)u * p.dst_max_ctx + i * kBlock + tid] = p.e[(int64_t)u * p.max_ctx + b * kBlock + tid];
    if (tid == 0 && rows == kBlock) p.dst_blk_evict[db] = p.blk_evict[sb];
}

int launch_evict(const EvictParams &p, cudaStream_t stream) {
    const size_t smem = (size_t)p.nblk * sizeof(uint32_t);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(evict_choose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return NOSA_ERR_CUDA;
    if (launch_pdl(evict_choose_kernel, dim3(p.units), dim3(kChooseThreads), smem, stream, p) != cudaSuccess)
        return NOSA_ERR_CUDA;
    return launch_pdl(evict_move_kernel, dim3((unsigned)p.units * (unsigned)(p.keep + 1)), dim3(kMoveThreads), 0, stream,
                      p) == cudaSuccess
               ? NOSA_OK
               : NOSA_ERR_CUDA;
}

}  // namespace nosa
