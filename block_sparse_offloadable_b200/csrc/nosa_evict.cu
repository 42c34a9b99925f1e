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
// Two kernels.  choose: a CTA per unit finds the keep largest of the weights' order-preserving integer
// keys by radix selection in shared memory, numbers the kept blocks with a scan, and writes what a unit
// has once (lengths, Gamma_e and the pool renumbered, weights).  move: a CTA per kept block copies its
// rows or codes, logits, pooled keys and score; only what the unit's tokens have filled is read or
// written.  Bound by HBM: every kept byte is read and written once.  Measured: 16 units of 512 blocks,
// 64 kept, bf16: 21.8 us; 64 units of up to 256 blocks, 128 kept, int8: 56 us, 0.84 of the measured HBM
// rate (both as calls within 2 %).  One kernel in which teams of CTAs choose and then copy, each its share: 26.5 and 99.9 us (a CTA's
// blocks one after the other leave too little in flight).
#include "nosa_internal.cuh"
#include "nosa_topk.cuh"

namespace nosa {

namespace {

// Larger weight, larger key; -0 and +0 the same; NaN above every number.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xFFFFFFFEu;
    return float_order(w == 0.f ? 0.f : w);
}
constexpr uint32_t kProtected = 0xFFFFFFFFu;

// Renumber a list of blocks (ids in order, those not kept left out) into dst; one warp.
__device__ __forceinline__ int32_t renumber(const int32_t *src, int32_t n, const uint32_t *number, int32_t nb,
                                            int32_t *dst, int lane) {
    int32_t m = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const int32_t b = i < n ? src[i] : -1;
        const int32_t to = b >= 0 && b < nb ? (int32_t)number[b] : -1;
        const unsigned got = __ballot_sync(0xFFFFFFFFu, to >= 0);
        if (to >= 0) dst[m + __popc(got & ((1u << lane) - 1u))] = to;
        m += __popc(got);
    }
    return m;
}
}  // namespace

__global__ void __launch_bounds__(kTopThreads) evict_choose_kernel(const EvictParams p) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ uint32_t keys[];  // [nblk]: the candidates' keys, then their new numbers (or -1)
    __shared__ TopShared top;
    __shared__ int32_t ge[kMaxKe];
    static_assert(kMaxKe <= kTopThreads, "a thread per member");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t u = blockIdx.x;
    const float *w = p.weights + (int64_t)u * p.nblk;
    int32_t *kept = p.kept + (int64_t)u * (p.keep + 1);
    float *dw = p.dst_weights + (int64_t)u * p.dst_nblk;
    // everything that is read, at once: a chain of loads from HBM is most of this kernel's time
    const int32_t L = max(p.seq_len[u], 0);
    const int32_t n_ge = p.k_e > 0 ? min(max(p.gamma_n[u], 0), p.k_e) : 0;
    const int32_t n_pool = p.pool ? min(max(p.pool_n[u], 0), p.nblk) : 0;
    if (tid < p.k_e) ge[tid] = p.gamma_e[(int64_t)u * p.k_e + tid];
    for (int i = tid; i < p.nblk; i += kTopThreads) keys[i] = weight_key(w[i]);
    const int32_t nb = L > 0 ? (L - 1) / kBlock : 0;
    for (int i = tid; i < nb; i += kTopThreads)
        if (i < p.sink || i >= nb - p.recent) keys[i] = kProtected;
    __syncthreads();
    const int32_t n_kept = number_chosen(keys, nb, nb <= p.keep, p.keep, top);
    for (int i = tid; i < nb; i += kTopThreads) {
        const int32_t at = (int32_t)keys[i];
        if (at < 0) continue;
        kept[at] = i;
        dw[at] = w[i];
    }
    for (int i = n_kept + tid; i <= p.keep; i += kTopThreads) kept[i] = (i == n_kept && L > 0) ? nb : -1;
    for (int i = n_kept + tid; i < p.dst_nblk; i += kTopThreads) dw[i] = (i == n_kept && L > 0) ? w[nb] : 0.f;
    if (warp == 0) {
        const int32_t m = renumber(ge, n_ge, keys, nb, p.dst_gamma_e + (int64_t)u * p.k_e, lane);
        if (lane == 0) {
            p.dst_seq_len[u] = L > 0 ? n_kept * kBlock + (L - nb * kBlock) : 0;
            p.dst_gamma_n[u] = m;
        }
    }
    if (warp == 1 && p.pool) {
        const int32_t m = renumber(p.pool + (int64_t)u * p.nblk, n_pool, keys, nb,
                                   p.dst_pool + (int64_t)u * p.dst_nblk, lane);
        if (lane == 0) p.dst_pool_n[u] = m;
    }
}

// Copy n 16-byte pieces.
template <int kAtOnce>
__device__ __forceinline__ void move16(uint8_t *dst, const uint8_t *src, int n) {
    const uint4 *s = reinterpret_cast<const uint4 *>(src);
    uint4 *d = reinterpret_cast<uint4 *>(dst);
    for (int i0 = threadIdx.x; i0 < n; i0 += kAtOnce * kTopThreads) {
        uint4 v[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (i0 + j * kTopThreads < n) v[j] = __ldcs(s + i0 + j * kTopThreads);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (i0 + j * kTopThreads < n) d[i0 + j * kTopThreads] = v[j];
    }
}

__global__ void __launch_bounds__(kTopThreads) evict_move_kernel(const EvictParams p) {
    pdl_wait();
    const int tid = threadIdx.x;
    const int32_t i = (int32_t)(blockIdx.x % (uint32_t)(p.keep + 1)), u = (int32_t)(blockIdx.x / (uint32_t)(p.keep + 1));
    const int32_t b = p.kept[(int64_t)u * (p.keep + 1) + i];
    const int32_t L = p.seq_len[u];
    if (b < 0) return;
    const int32_t rows = min(L - b * kBlock, kBlock);  // of the block's 64, those with a token
    const bool local = b == (L - 1) / kBlock;
    const int64_t sb = (int64_t)u * p.nblk + b, db = (int64_t)u * p.dst_nblk + i;
    const int ck_bytes = kD * (p.ck_bf16 ? 2 : 4);  // one pooled key
    float e = 0.f;
    if (tid < rows) e = p.e[(int64_t)u * p.max_ctx + b * kBlock + tid];
    if (p.fmt != kFmtBf16 && !local) {
        move16<5>(p.dst_store + db * kRec8Bytes, p.store + sb * kRec8Bytes, kHeld8Bytes / 16);
    } else {
        const bool tail = p.fmt != kFmtBf16;
        const uint8_t *s = tail ? p.tail + (int64_t)u * kBlockBytes : p.store + sb * kBlockBytes;
        uint8_t *d = tail ? p.dst_tail + (int64_t)u * kBlockBytes : p.dst_store + db * kBlockBytes;
        if (rows == kBlock) {
            move16<8>(d, s, kBlockBytes / 16);
        } else {
            move16<4>(d, s, rows * (kRowBytes / 16));
            move16<4>(d + kHalfBlockBytes, s + kHalfBlockBytes, rows * (kRowBytes / 16));
        }
    }
    move16<1>(p.dst_ck + db * kSubPerBlock * ck_bytes, p.ck + sb * kSubPerBlock * ck_bytes,
              rows / kSub * (ck_bytes / 16));
    if (tid < rows) p.dst_e[(int64_t)u * p.dst_max_ctx + i * kBlock + tid] = e;
    if (tid == 0 && rows == kBlock) p.dst_blk_evict[db] = p.blk_evict[sb];
}

int launch_evict(const EvictParams &p, cudaStream_t stream) {
    const size_t smem = (size_t)p.nblk * sizeof(uint32_t);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(evict_choose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return NOSA_ERR_CUDA;
    if (launch_pdl(evict_choose_kernel, dim3(p.units), dim3(kTopThreads), smem, stream, p) != cudaSuccess)
        return NOSA_ERR_CUDA;
    return launch_pdl(evict_move_kernel, dim3((unsigned)p.units * (unsigned)(p.keep + 1)), dim3(kTopThreads), 0, stream,
                      p) == cudaSuccess
               ? NOSA_OK
               : NOSA_ERR_CUDA;
}

}  // namespace nosa
