// nosa_decode_items.cu -- steps a5 and a6 over the 8-bit KV store, and over any store when the blocks'
// attention weights are kept.
//
// NOSA pages: gist.science summary of arXiv:2510.13602, "ED-DMA" (the eviction score enters the
// softmax as the additive logit e_j); montaan.com "Empirical Results and Analysis" item 4 (decoding
// is bound by KV loading).  Neither the 8-bit store nor eviction by attention weight is on the pages.
//
// The split of nosa_decode.cu's kernel (work items are (unit, block) pairs; equal pieces of a unit
// per CTA where the units are fewer than the SMs, else balanced ranges; partial states merged by a
// unit's last CTA), with a different inside, since an 8-bit block is half the bytes and more
// instructions than a bf16 one:
//  * One consumer warp attends a whole block (nosa_attend8.cuh).  Five of them (three over the bf16
//    store) with two stages each: a stage's next block is in flight while its other one is
//    attended.  Eight warps with ten stages leave two blocks in flight while all attend: 93 us at
//    32 ragged sequences of up to 32K (e4m3, 16 q / 2 kv heads) where five warps took 75 (70.3 now,
//    0.89 of the measured HBM rate; 76 as calls one after the other, 0.83).
//  * Two producer warps, for the even and the odd items: one issue (expected bytes, a tensor copy of
//    the codes, a bulk copy of the logits and scales) takes 0.27 us of one thread's time, and a
//    block must come every 0.38 us to keep the memory busy; the first items are issued by the
//    consumer warps and the producers at once.
//  * The newest block of a unit (bf16 tail of the 8-bit store) takes longest and comes first.
//  * Seven warps leave 255 registers a thread: attend8 wants about 200.
// Times in these files are replays of a captured graph over several states, unless they say calls.
#include "nosa_attend8.cuh"
#include "nosa_decode_work.cuh"

namespace nosa {

namespace {

constexpr int kItemCons = 5;                       // consumer warps
constexpr int kItemProd = 2;                       // producer warps
constexpr int kAlignItems = 6;                     // about what a segment's end costs, in items
constexpr int kItemConsThreads = kItemCons * 32;
constexpr int kItemThreads = (kItemCons + kItemProd) * 32;

// Stages, and consumer warps that take items (two stages each; stage s always belongs to consumer
// s % kTakers and producer s % 2, so that every barrier has one waiter, which meets its phases in
// order: a parity cannot tell phase n from n - 2).  The resident pass of the split decode leaves
// room for a select CTA on the SM.
template <int kFmt, bool kResident>
struct ItemGeo {
    static constexpr bool k8 = kFmt != kFmtBf16;
    static constexpr int kStages = (k8 && !kResident) ? 10 : 6;
    static constexpr int kTakers = kStages / 2;
    static constexpr int kStageBytes = k8 ? kBlock8Bytes : kBlockBytes;
    static constexpr int kTails = !k8 ? 0 : (kResident ? 1 : 2);  // buffers for a tail's values (its keys take a stage)
    static constexpr int kSide = k8 ? kSide8Bytes / 4 : kBlock;   // floats a stage: logits (8-bit store: and scales)
    static_assert(kTakers <= kItemCons && kStages % kItemProd == 0, "one waiter per barrier");

    static size_t smem_bytes(int32_t prefix) {
        return 1024 + (size_t)kStages * kStageBytes + (size_t)kTails * kHalfBlockBytes +
               (size_t)kStages * kSide * sizeof(float) + (2 * kStages + 2) * sizeof(uint64_t) +
               (size_t)kStages * sizeof(int4) + (size_t)kTakers * kScr * sizeof(float) +
               (size_t)prefix * sizeof(int32_t);
    }
};

// Wait until *at == n (shared memory, written by another warp); false if the bound ran out.
__device__ __forceinline__ bool reached_or_abort(const volatile int32_t *at, int32_t n, volatile int *abort_flag,
                                                 uint32_t *err) {
    const long long t0 = clock64();
    while (*at != n) {
        if (*abort_flag) return false;
        if (clock64() - t0 > kWaitCycles) {
            *abort_flag = 1;
            set_error(err, NOSA_EFLAG_TIMEOUT);
            return false;
        }
    }
    return true;
}

// Segment end, first half: this warp's (m, l, o) to its slot of the scratch.
template <class Dims>
__device__ __forceinline__ void leave_state(const WarpState &st, float *mine, int r, int c, int sig) {
    float l0 = st.l0, l1 = st.l1;
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
        l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, sh);
        l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, sh);
    }
    if (r == 0) {
        mine[2 * c] = st.m0; mine[2 * c + 1] = st.m1;
        mine[kMaxG + 2 * c] = l0; mine[kMaxG + 2 * c + 1] = l1;
    }
    float *oo = mine + 2 * kMaxG;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const int psi = Dims::psi(t, sig);
        oo[(2 * c) * kHS + Dims::at(psi)] = st.o[t][0];
        oo[(2 * c + 1) * kHS + Dims::at(psi)] = st.o[t][1];
        oo[(2 * c) * kHS + Dims::at(psi + 1)] = st.o[t][2];
        oo[(2 * c + 1) * kHS + Dims::at(psi + 1)] = st.o[t][3];
    }
}

// Second half, for head h and dims d .. d + 3: the warps' states merged into (M, acc, lsum).
template <class Dims, int kTakers>
__device__ __forceinline__ void join_states(const float *scratch, int h, int d, float &M, float4 &acc, float &lsum) {
    M = kNegInf;
#pragma unroll
    for (int w = 0; w < kTakers; ++w) M = fmaxf(M, scratch[w * kScr + h]);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kTakers; ++w) {
        const float mw = scratch[w * kScr + h];
        const float f = (mw == kNegInf) ? 0.f : exp2f(mw - M);
        const float *o = scratch + w * kScr + 2 * kMaxG + h * kHS;
        acc.x = fmaf(f, o[Dims::at(d)], acc.x);
        acc.y = fmaf(f, o[Dims::at(d + 1)], acc.y);
        acc.z = fmaf(f, o[Dims::at(d + 2)], acc.z);
        acc.w = fmaf(f, o[Dims::at(d + 3)], acc.w);
        lsum = fmaf(f, scratch[w * kScr + kMaxG + h], lsum);
    }
}

// merge_resident for dims d4 .. d4 + 3.  Where neither state has a maximum, both are empty or NaN, and NaN is carried on.
__device__ __forceinline__ void merge_resident4(const DecodeParams &p, int32_t u, int h, int d4, float &M, float4 &acc,
                                                float &lsum) {
    const float *res = p.res_part + (int64_t)u * kPartFloats;
    if (M == kNegInf && res[h] == kNegInf) {
        const float4 o = *reinterpret_cast<const float4 *>(res + 2 * kMaxG + h * kD + d4);
        acc.x += o.x; acc.y += o.y; acc.z += o.z; acc.w += o.w;
        lsum += res[kMaxG + h];
        return;
    }
    float m = M, l = lsum;
    merge_resident(p, u, h, d4, m, acc.x, l);
    m = M, l = lsum;
    merge_resident(p, u, h, d4 + 1, m, acc.y, l);
    m = M, l = lsum;
    merge_resident(p, u, h, d4 + 2, m, acc.z, l);
    merge_resident(p, u, h, d4 + 3, M, acc.w, lsum);
}

// A unit's whole softmax per head: the log2 of its sum, and where that is far from 0 its two parts.
struct WholeSums {
    float lse[kMaxG], M[kMaxG], l[kMaxG];
    __device__ __forceinline__ void set(int h, float m, float sum) {
        lse[h] = m + log2f(sum);
        M[h] = m;
        l[h] = sum;
    }
};

// The last CTA of a unit merges the nc partial records src[], in order.  A thread takes 8 dims of a
// head and has the loads of kBatch records in flight at once, since a round trip to the L2 (0.7 us) is
// what this costs.  Writes bf16 out, or the merged record to res (the split decode's state), and the
// heads' whole sums to *all.
__device__ __forceinline__ void merge_records(const float *const *src, int nc, int G, uint16_t *out, float *res,
                                              WholeSums *all, int ctid) {
    constexpr int kBatch = 4;
#pragma unroll 1
    for (int v = ctid; v < G * (kD / 8); v += kItemConsThreads) {
        const int h = v / (kD / 8), d = (v % (kD / 8)) * 8;
        float M = kNegInf, ls = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 1
        for (int t0 = 0; t0 < nc; t0 += kBatch) {
            float m[kBatch], l[kBatch];
            float4 x[kBatch], y[kBatch];
#pragma unroll
            for (int t = 0; t < kBatch; ++t) {
                m[t] = kNegInf;
                if (t0 + t < nc) {
                    const float *rec = src[t0 + t];
                    const float4 *o = reinterpret_cast<const float4 *>(rec + 2 * kMaxG + h * kD + d);
                    m[t] = __ldcg(rec + h);
                    l[t] = __ldcg(rec + kMaxG + h);
                    x[t] = __ldcg(o);
                    y[t] = __ldcg(o + 1);
                }
            }
            float Mn = M;
#pragma unroll
            for (int t = 0; t < kBatch; ++t) Mn = fmaxf(Mn, m[t]);
            const float f0 = (M == kNegInf) ? 0.f : exp2f(M - Mn);
            a.x *= f0; a.y *= f0; a.z *= f0; a.w *= f0;
            b.x *= f0; b.y *= f0; b.z *= f0; b.w *= f0;
            ls *= f0;
#pragma unroll
            for (int t = 0; t < kBatch; ++t)
                if (t0 + t < nc) {
                    const float f = (m[t] == kNegInf) ? 0.f : exp2f(m[t] - Mn);
                    a.x = fmaf(f, x[t].x, a.x); a.y = fmaf(f, x[t].y, a.y);
                    a.z = fmaf(f, x[t].z, a.z); a.w = fmaf(f, x[t].w, a.w);
                    b.x = fmaf(f, y[t].x, b.x); b.y = fmaf(f, y[t].y, b.y);
                    b.z = fmaf(f, y[t].z, b.z); b.w = fmaf(f, y[t].w, b.w);
                    ls = fmaf(f, l[t], ls);
                }
            M = Mn;
        }
        if (res) {
            *reinterpret_cast<float4 *>(res + 2 * kMaxG + h * kD + d) = a;
            *reinterpret_cast<float4 *>(res + 2 * kMaxG + h * kD + d + 4) = b;
            if (d == 0) {
                res[h] = M;
                res[kMaxG + h] = ls;
            }
        } else {
            const uint2 lo = pack_out4<true>(a, ls), hi = pack_out4<true>(b, ls);
            *reinterpret_cast<uint4 *>(out + h * kD + d) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
        if (all && d == 0) all->set(h, M, ls);
    }
}

// A block's weight: its item's values (left by the warp that attended it) against the whole sums per head.
struct Weight {
    int32_t lb, pb;  // the block's number (-1: none) and its place in the buffer
    float4 a, b;
};

__device__ __forceinline__ Weight load_weight(const DecodeParams &p, int32_t u, int32_t item0, int32_t n, int32_t j) {
    Weight w;
    w.lb = w.pb = -1;
    if (j >= n) return w;
    const float4 *rec = reinterpret_cast<const float4 *>(p.rec + (int64_t)(item0 + j) * kRecFloats);
    w.a = __ldcg(rec);
    w.b = __ldcg(rec + 1);
    const int32_t L = p.seq_len[u];
    item_block(p, u, n - 1 - j, w.lb, w.pb);  // the items' order, see look_up
    if ((int64_t)w.lb * kBlock >= L) w.lb = -1;
    return w;
}

// The largest of a block's logits in the log2 domain (n of its 64 are seen).  A call: it is wanted only where some
// item's value is not plain, see leave_weights.
__device__ __noinline__ float largest_logit(const float *e, int32_t n) {
    float top = kNegInf;
#pragma unroll 4
    for (int i = 0; i < kBlock; i += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(e + i);
        if (i < n) top = fmaxf(top, bias_log2(x.x));
        if (i + 1 < n) top = fmaxf(top, bias_log2(x.y));
        if (i + 2 < n) top = fmaxf(top, bias_log2(x.z));
        if (i + 3 < n) top = fmaxf(top, bias_log2(x.w));
    }
    return top;
}

template <bool k8>
__device__ __forceinline__ void add_weight(const DecodeParams &p, int32_t u, const Weight &w, const WholeSums &all,
                                           bool far) {
    if (w.lb < 0) return;
    const float v[kMaxG] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
    float sum = 0.f;
    if (far) {
        float top = 0.f;
        bool any = false;
#pragma unroll
        for (int h = 0; h < kMaxG; ++h) any |= is_far(v[h]);
        if (any) {  // the logits, from where the attention read them
            const int32_t L = p.seq_len[u];
            const float *e = p.e + (int64_t)u * p.max_ctx + (int64_t)w.lb * kBlock;
            if (k8 && w.lb < (L - 1) / kBlock)
                e = reinterpret_cast<const float *>(
                    p.records + ((int64_t)u * p.blocks_per_unit + w.pb) * kRec8Bytes + kBlock8Bytes);
            top = largest_logit(e, L - w.lb * kBlock);
        }
#pragma unroll 1
        for (int h = 0; h < p.G; ++h)
            if (all.l[h] != 0.f)
                sum += exp2f(is_far(v[h]) ? v[h] * (1.f / kFarScale) + (top - all.M[h]) : v[h] - all.M[h]) / all.l[h];
    } else {
#pragma unroll
        for (int h = 0; h < kMaxG; ++h)  // a head that sees nothing gives no weight
            if (h < p.G && all.lse[h] != kNegInf) sum += exp2f(v[h] - all.lse[h]);
    }
    atomicAdd(p.weights + (int64_t)u * p.nblk + w.lb, sum);  // a caller's list may name a block twice
}

// An item: its unit, the unit's length, the block's number (-1: nothing) and its place in the buffer.
struct Item {
    int32_t u, L, lb, pb;
    __device__ __forceinline__ int32_t local() const { return L > 0 ? (L - 1) / kBlock : -1; }
    __device__ __forceinline__ bool tail() const { return lb >= 0 && lb == local(); }
};

}  // namespace

// Pieces (p.pieces > 0) only with kModeSel.
template <int kFmt, bool kWeights, bool kResident>
__global__ void __launch_bounds__(kItemThreads, 1)
    decode_items_kernel(const __grid_constant__ CUtensorMap tmap, const __grid_constant__ CUtensorMap tail_map,
                        const DecodeParams p) {
    using Geo = ItemGeo<kFmt, kResident>;
    constexpr bool k8 = Geo::k8;
    constexpr int kStages = Geo::kStages, kTakers = Geo::kTakers, kStageBytes = Geo::kStageBytes, kTails = Geo::kTails,
                  kSide = Geo::kSide;
    using Dims = std::conditional_t<k8, Dims8, DimsBf16>;
    pdl_trigger();  // the next append's CTAs are tiny; they wait for this grid
    extern __shared__ uint8_t smem_raw[];
    uint8_t *tiles = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *tails = tiles + kStages * kStageBytes;
    float *ebuf = reinterpret_cast<float *>(tails + kTails * kHalfBlockBytes);
    uint64_t *full = reinterpret_cast<uint64_t *>(ebuf + kStages * kSide);
    uint64_t *empty = full + kStages;
    uint64_t *tempty = empty + kStages;
    int4 *s_item = reinterpret_cast<int4 *>(tempty + 2);  // what a stage holds: (block number, tail buffer or -1, -, -)
    float *scratch = reinterpret_cast<float *>(s_item + kStages);
    int32_t *P = reinterpret_cast<int32_t *>(scratch + kTakers * kScr);
    __shared__ int32_t s_wsum[kItemThreads / 32];
    __shared__ volatile int32_t s_tail_no[2];  // the tail last issued into each buffer
    __shared__ int s_last;
    __shared__ volatile int s_abort;
    __shared__ WholeSums s_all;
    __shared__ volatile int s_far;  // some item's weights of this CTA, or of one whose unit it ends, are not plain

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t U = p.units, grid = (int32_t)gridDim.x, cta = (int32_t)blockIdx.x;
    const bool nominal = p.mode == kModeSel;  // max_sel items per unit, whatever nsel (-1 padded past it)

    if (warp == kItemCons) {
        if (lane < kStages) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], 1);
        }
        if (lane < kTails) {
            mbar_init(&tempty[lane], 1);
            s_tail_no[lane] = lane - kTails;
        }
        fence_mbar_init();
        if (lane == 0) {
            prefetch_tmap(&tmap);
            if (k8) prefetch_tmap(&tail_map);
            s_abort = 0;
            s_far = 0;
        }
    }
    // ---- items of units < u ----
    if (nominal) {
        __syncthreads();
        pdl_wait();  // nothing before it reads global memory
    } else {
        pdl_wait();
        const int per = (U + kItemThreads - 1) / kItemThreads;
        const int u0 = min((int)threadIdx.x * per, U), u1 = min(u0 + per, U);
        int32_t sum = 0;
        for (int u = u0; u < u1; ++u) {
            const int32_t w = unit_work(p, u);
            P[u + 1] = w;
            sum += w;
        }
        int32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) s_wsum[warp] = incl;
        __syncthreads();
        int32_t run = incl - sum;
        for (int w = 0; w < warp; ++w) run += s_wsum[w];
        for (int u = u0; u < u1; ++u) {
            run += P[u + 1];
            P[u + 1] = run;
        }
        if (threadIdx.x == 0) P[0] = 0;
        __syncthreads();
    }
    const auto first_item = [&](int32_t u) { return nominal ? u * p.max_sel : P[u]; };
    const auto unit_of = [&](int32_t x) { return nominal ? x / p.max_sel : find_unit(P, U, x); };
    const int32_t W = first_item(U);  // < 2^25
    // Balanced: ranges over Ge CTAs of no fewer items than consumer warps, where there are as many: a
    // CTA with one item costs a merge of its state and saves nothing (65 blocks a unit, 2 units: 12.0 us
    // with ranges of 5, 14.4 of 8 over 4 warps, 15.6 of 4).
    const int32_t We = (W + kTakers - 1) / kTakers;
    const int32_t Ge = min(max(We, 1), grid);
    // Where a CTA has items of one unit alone, that unit's CTAs: `team` of them from team_first on.
    int32_t lo, hi, team = p.pieces, team_first = 0;
    if (team > 0) {  // equal pieces of every unit
        team_first = cta / team * team;
        lo = cta / team * p.max_sel + (cta - team_first) * p.max_sel / team;
        hi = cta / team * p.max_sel + (cta - team_first + 1) * p.max_sel / team;
    } else {
        lo = (int32_t)((cta < Ge) ? (int64_t)cta * W / Ge : W);
        hi = (int32_t)((cta < Ge) ? (int64_t)(cta + 1) * W / Ge : W);
    }
    if (p.pieces <= 0 && U <= 32 && U <= Ge && W > 0) {
        // Few units, of any lengths: a CTA for each and the others in proportion to the units' items, equal
        // pieces of a unit each, if that gives no CTA more than kAlignItems items more than balanced
        // ranges.  It spares ranges with two units in them, whose first one's end holds up the stream.
        // int8 with weights, units of 129 to 257 blocks, against balanced ranges: 16 units 23.7 us (27.4), 24
        // units 28.8 (31.5), 32 units 35.7 (35.2); 32 units of 33 to 65 blocks 16.7 (21.2).  A warp holds 32
        // units, and there the gain ends where the units are long.  Balanced, 40 units take 39.0 (bytes alone
        // 20.3), 100 units 71.5 (51.9).
        const int32_t n = lane < U ? first_item(lane + 1) - first_item(lane) : 0;
        const int32_t mine = n > 0 ? 1 + (int32_t)((int64_t)n * (Ge - U) / W) : 0;  // Ge in all at most
        const int32_t most = (int32_t)__reduce_max_sync(0xFFFFFFFFu, n > 0 ? (uint32_t)((n + mine - 1) / mine) : 0u);
        int32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += x;
        }
        const int uc = __popc(__ballot_sync(0xFFFFFFFFu, incl <= cta));  // 32: no unit's
        const int32_t t = __shfl_sync(0xFFFFFFFFu, mine, uc & 31), tf = __shfl_sync(0xFFFFFFFFu, incl - mine, uc & 31);
        if (most <= (W + Ge - 1) / Ge + kAlignItems) {
            team = t;
            team_first = tf;
            lo = hi = W;
            if (uc < U) {
                const int32_t at = first_item(uc), nu = first_item(uc + 1) - at;
                lo = at + (cta - team_first) * nu / team;
                hi = at + (cta - team_first + 1) * nu / team;
            }
        }
    }
    const int32_t n_items = hi - lo;

    // The lanes of a warp look up 32 items at a time.  A unit's items run from its last block to its first.
    const auto look_up = [&](int32_t x) {
        Item i = {0, 0, -1, -1};
        if (x < hi) {
            i.u = unit_of(x);
            i.L = p.seq_len[i.u];  // in flight with the block number
            item_block(p, i.u, first_item(i.u + 1) - 1 - x, i.lb, i.pb);
        }
        return i;
    };
    const uint64_t once = evict_first_policy();
    // Item number `it` of the CTA, by one thread; nt: the tails before it.
    const auto issue = [&](const Item &i, int it, int nt) {
        const int s = it % kStages;
        uint8_t *t = tiles + s * kStageBytes;
        float *es = ebuf + s * kSide;
        if (it >= kStages && !wait_or_abort(&empty[s], ((it / kStages) - 1) & 1, &s_abort, p.err)) return;
        const bool held = i.pb >= 0 && i.pb < p.blocks_per_unit;
        if constexpr (!k8) {
            const bool ok = i.lb >= 0 && (int64_t)i.lb * kBlock < p.max_ctx && held;
            if (!ok && i.lb >= 0) set_error(p.err, NOSA_EFLAG_STATE);  // a block with no buffer
            s_item[s].x = ok ? i.lb : -1;
            if (ok) {
                const int32_t y = (int32_t)(((int64_t)i.u * p.blocks_per_unit + i.pb) * 2 * kBlock);
                mbar_arrive_expect_tx(&full[s], kBlockBytes + kBlock * sizeof(float));
                tma_load_2d_hint(t, &tmap, &full[s], 0, y, once);
                tma_load_2d_hint(t + kBoxBytes, &tmap, &full[s], 64, y, once);
                tma_load_2d_hint(t + 2 * kBoxBytes, &tmap, &full[s], 0, y + kBlock, once);
                tma_load_2d_hint(t + 3 * kBoxBytes, &tmap, &full[s], 64, y + kBlock, once);
                bulk_load_hint(es, p.e + (int64_t)i.u * p.max_ctx + (int64_t)i.lb * kBlock, kBlock * sizeof(float), &full[s], once);
            } else {
                mbar_arrive(&full[s]);
            }
        } else if (i.tail()) {
            constexpr int kT = kTails ? kTails : 1;
            const int tb = nt % kT;
            // The buffer's phases in order, whichever producer has the tail: the tail before it in
            // this buffer has been issued, then consumed.
            bool have = true;
            if (nt >= kTails)
                have = reached_or_abort(&s_tail_no[tb], nt - kT, &s_abort, p.err) &&
                       wait_or_abort(&tempty[tb], ((nt / kT) - 1) & 1, &s_abort, p.err);
            s_item[s] = make_int4(have ? i.lb : -1, tb, 0, 0);
            if (have) {
                s_tail_no[tb] = nt;
                const int32_t y = i.u * 2 * kBlock;
                uint8_t *tv = tails + tb * kHalfBlockBytes;
                mbar_arrive_expect_tx(&full[s], kBlockBytes + kBlock * sizeof(float));
                tma_load_2d_hint(t, &tail_map, &full[s], 0, y, once);
                tma_load_2d_hint(t + kBoxBytes, &tail_map, &full[s], 64, y, once);
                tma_load_2d_hint(tv, &tail_map, &full[s], 0, y + kBlock, once);
                tma_load_2d_hint(tv + kBoxBytes, &tail_map, &full[s], 64, y + kBlock, once);
                bulk_load_hint(es, p.e + (int64_t)i.u * p.max_ctx + (int64_t)i.lb * kBlock, kBlock * sizeof(float), &full[s], once);
            } else {
                mbar_arrive(&full[s]);
            }
        } else {
            const bool ok = i.lb >= 0 && i.lb < i.local() && held;
            // a block with no buffer; blocks past the newest hold nothing to attend
            if (!ok && i.lb >= 0 && (i.lb < i.local() || (int64_t)i.lb * kBlock >= p.max_ctx))
                set_error(p.err, NOSA_EFLAG_STATE);
            s_item[s] = make_int4(ok ? i.lb : -1, -1, 0, 0);
            if (ok) {
                const int64_t rb = (int64_t)i.u * p.blocks_per_unit + i.pb;
                mbar_arrive_expect_tx(&full[s], kHeld8Bytes);
                tma_load_3d_hint(t, &tmap, &full[s], 0, 0, (int32_t)rb, once);
                bulk_load_hint(es, p.records + rb * kRec8Bytes + kBlock8Bytes, kSide8Bytes, &full[s], once);
            } else {
                mbar_arrive(&full[s]);
            }
        }
    };
    // Each consumer warp issues its own first item where that waits for nothing (a consumer that waited
    // for a tail's buffer could hold up the one that frees it).
    const auto by_consumer = [&](const Item &i, int it, int nt) {
        return it < kTakers && !(k8 && i.tail() && nt >= kTails);
    };

    if (warp >= kItemCons) {
        // ---------------- producers ----------------
        const int odd = warp - kItemCons;
        int it = 0, nt = 0;
        Item next = look_up(lo + lane);  // the next batch, looked up while one is issued
        for (int32_t xb = lo; xb < hi && !s_abort; xb += 32) {
            const int nb = min(hi - xb, 32);
            const Item mine = next;
            next = look_up(xb + 32 + lane);
            const unsigned tail_lanes = __ballot_sync(0xFFFFFFFFu, mine.tail());
            const int my_nt = nt + __popc(tail_lanes & ((1u << lane) - 1u));
            nt += __popc(tail_lanes);
            for (int k = 0; k < nb; ++k, ++it) {
                if (lane == k && it % kItemProd == odd && !by_consumer(mine, it, my_nt)) issue(mine, it, my_nt);
                __syncwarp();
            }
        }
        // never leave with copies in flight
        if (lane == 0)
            for (int i = max(0, it - kStages); i < it; ++i) mbar_wait(&full[i % kStages], (i / kStages) & 1);
    } else {
        // ---------------- consumers ----------------
        const int r = lane >> 2, c = lane & 3;
        const int sig = (r >> 1) + ((r & 1) << 2);  // row permutation 0,4,1,5,2,6,3,7
        const int ctid = threadIdx.x;                // 0..kItemConsThreads-1
        {
            const Item mine = look_up(lane < kTakers ? lo + lane : hi);
            const unsigned tail_lanes = __ballot_sync(0xFFFFFFFFu, mine.tail());
            const int nt = __popc(tail_lanes & ((1u << lane) - 1u));
            if (lane == warp && warp < n_items && by_consumer(mine, warp, nt)) issue(mine, warp, nt);
            __syncwarp();
        }
        uint32_t qf[8][2];
        [[maybe_unused]] Query8<k8 ? kFmt : kFmtE4m3> q8;
        int32_t L = 0;
        // a unit's queries (B fragments, dims permuted as the key loads) and length
        auto load_q = [&](int32_t uu) {
            const uint4 *qrow = reinterpret_cast<const uint4 *>(p.q + ((int64_t)uu * p.G + r) * kD);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                const uint4 x = (r < p.G) ? qrow[4 * jj + c] : make_uint4(0, 0, 0, 0);
                qf[2 * jj][0] = x.x; qf[2 * jj][1] = x.y;
                qf[2 * jj + 1][0] = x.z; qf[2 * jj + 1][1] = x.w;
            }
        };
        auto load_unit = [&](int32_t uu) {
            if constexpr (k8) load_query8(q8, p.q + (int64_t)uu * p.G * kD, p.G, r, c);
            else load_q(uu);
            L = p.seq_len[uu];
        };
        const int32_t first_unit = n_items > 0 ? unit_of(lo) : 0;
        int32_t u = first_unit, last_first = -1, last_other = -1;
        for (int32_t x = lo; x < hi;) {
            load_unit(u);
            WarpState st;
            st.reset();
            const int32_t u_begin = first_item(u), u_end = first_item(u + 1);
            const int32_t seg_end = min(hi, u_end);
            const bool whole = x == u_begin && seg_end == u_end;
            const int slot = (u == first_unit) ? 0 : 1;
            if (warp < kTakers) {
                for (int32_t xi = x + ((warp - (x - lo)) % kTakers + kTakers) % kTakers; xi < seg_end; xi += kTakers) {
                    const int it = xi - lo;
                    const int s = it % kStages;
                    if (wait_or_abort(&full[s], (it / kStages) & 1, &s_abort, p.err)) {
                        const int32_t lb = s_item[s].x, tb = k8 ? s_item[s].y : -1;
                        float *rec = kWeights ? p.rec + (int64_t)xi * kRecFloats : nullptr;
                        const uint8_t *t = tiles + s * kStageBytes;
                        const float *e = ebuf + s * kSide;
                        [[maybe_unused]] ItemSums ws;
                        if (lb < 0) {
                            if (kWeights) leave_none(rec, r, c);
                        } else if constexpr (k8) {
                            if (tb >= 0) {
                                load_q(u);  // once a unit
                                attend16<Dims, kWeights, kFmt == kFmtE4m3>(st, qf, t, tails + tb * kHalfBlockBytes, e, lb,
                                                                           L, p.qk_log2, r, c, sig, ws);
                            } else {
                                attend8<kWeights>(st, q8, p.q + (int64_t)u * p.G * kD, p.G, t, e, e[kBlock], e[kBlock + 1],
                                                  p.qk_log2, r, c, sig, ws);
                            }
                        } else {
                            attend16<Dims, kWeights, false>(st, qf, t, t + kHalfBlockBytes, e, lb, L, p.qk_log2, r, c,
                                                            sig, ws);
                        }
                        if (kWeights && lb >= 0) leave_weights(rec, &s_far, ws, e, min(L - lb * kBlock, kBlock), r, c);
                        __syncwarp();
                        if (lane == 0 && tb >= 0) mbar_arrive(&tempty[tb]);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[s]);
                }
                leave_state<Dims>(st, scratch + warp * kScr, r, c, sig);
            }
            const int32_t u_next = (seg_end < hi) ? unit_of(seg_end) : u;
            consumer_sync<kItemConsThreads>();
            uint16_t *out = p.out + (int64_t)u * p.G * kD;
            float *part = p.part + ((int64_t)cta * 2 + slot) * kPartFloats;
            for (int v = ctid; v < p.G * (kD / 4); v += kItemConsThreads) {
                const int h = v / (kD / 4), d4 = (v % (kD / 4)) * 4;
                float M, lsum;
                float4 acc;
                join_states<Dims, kTakers>(scratch, h, d4, M, acc, lsum);
                if (whole && !kResident) {
                    if (p.mode == kModeRest) merge_resident4(p, u, h, d4, M, acc, lsum);
                    *reinterpret_cast<uint2 *>(out + h * kD + d4) = pack_out4<true>(acc, lsum);
                    if (kWeights && d4 == 0) s_all.set(h, M, lsum);
                } else {
                    float *rec = whole ? p.res_part + (int64_t)u * kPartFloats : part;
                    *reinterpret_cast<float4 *>(rec + 2 * kMaxG + h * kD + d4) = acc;
                    if (d4 == 0) {
                        rec[h] = M;
                        rec[kMaxG + h] = lsum;
                    }
                }
            }
            consumer_sync<kItemConsThreads>();
            if (!whole) {
                // hand-off: the partial is written (barrier), one thread counts it with release
                // semantics; the unit's last contributor acquired the others' partials with the same
                // atomic, and the barrier after it orders every thread's later loads after them
                const int32_t others = team > 0 ? team - 1 : cta_of((int64_t)u_end - 1, W, Ge) - cta_of(u_begin, W, Ge);
                // (with weights: and in the upper half, that some of the CTA's are not plain)
                if (ctid == 0) {
                    const uint32_t mine = kWeights && s_far ? 0x10001u : 1u;
                    const uint32_t n = atom_add_acq_rel_gpu(p.counter + u, mine) + mine;
                    s_last = (int32_t)(n & 0xFFFFu) == others + 1;
                    if (kWeights && s_last && n >> 16) s_far = 1;
                }
                consumer_sync<kItemConsThreads>();
                if (s_last) (slot == 0 ? last_first : last_other) = u;
            } else if (kWeights) {
                for (int32_t j = ctid; j < u_end - u_begin; j += kItemConsThreads)
                    add_weight<k8>(p, u, load_weight(p, u, u_begin, u_end - u_begin, j), s_all, s_far);
                consumer_sync<kItemConsThreads>();
            }
            x = seg_end;
            u = u_next;
        }
        // The units whose last contributor this CTA is, at most its first and its last: merged here, after
        // the stream, where the registers of the attention are free (a first unit's merge is rarely
        // here: the CTA before it streams the rest of that unit at its end).
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const int32_t um = k ? last_other : last_first;
            if (um < 0) continue;
            const int32_t u_begin = first_item(um), u_end = first_item(um + 1);
            const int32_t cf = team > 0 ? team_first : cta_of(u_begin, W, Ge);
            const int32_t cl = team > 0 ? team_first + team - 1 : cta_of((int64_t)u_end - 1, W, Ge);
            if (ctid == 0) p.counter[um] = 0;
            // the CTA partials in CTA order (and, merging the rest pass, the resident state)
            const int nc = cl - cf + 1 + (p.mode == kModeRest ? 1 : 0);  // <= Ge + 1
            const float **src = reinterpret_cast<const float **>(scratch);
            for (int t = ctid; t < nc; t += kItemConsThreads) {
                const int32_t cc = cf + t;
                if (cc > cl) {
                    src[t] = p.res_part + (int64_t)um * kPartFloats;
                } else {
                    const int sl = (team > 0 || unit_of((int32_t)((int64_t)cc * W / Ge)) == um) ? 0 : 1;
                    src[t] = p.part + (int64_t)(cc * 2 + sl) * kPartFloats;
                }
            }
            consumer_sync<kItemConsThreads>();
            Weight w0;  // the first blocks' weights, in flight while the states are merged
            if (kWeights) w0 = load_weight(p, um, u_begin, u_end - u_begin, ctid);
            merge_records(src, nc, p.G, p.out + (int64_t)um * p.G * kD,
                              kResident ? p.res_part + (int64_t)um * kPartFloats : nullptr, kWeights ? &s_all : nullptr,
                              ctid);
            consumer_sync<kItemConsThreads>();
            if (kWeights) {
                add_weight<k8>(p, um, w0, s_all, s_far);
                for (int32_t j = ctid + kItemConsThreads; j < u_end - u_begin; j += kItemConsThreads)
                    add_weight<k8>(p, um, load_weight(p, um, u_begin, u_end - u_begin, j), s_all, s_far);
                consumer_sync<kItemConsThreads>();
            }
        }
        // units without work, one CTA each: zero output (an empty state in the
        // resident pass; the resident state alone in the rest pass)
        for (int32_t uz = cta; uz < U; uz += grid) {
            if (first_item(uz + 1) != first_item(uz)) continue;
            if (kResident) {
                float *rp = p.res_part + (int64_t)uz * kPartFloats;
                for (int i = ctid; i < kPartFloats; i += kItemConsThreads) rp[i] = (i < kMaxG) ? kNegInf : 0.f;
                continue;
            }
            uint16_t *out = p.out + (int64_t)uz * p.G * kD;
            for (int v = ctid; v < p.G * (kD / 4); v += kItemConsThreads) {
                float M = kNegInf, lsum = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                const int h = v / (kD / 4), d4 = (v % (kD / 4)) * 4;
                if (p.mode == kModeRest) merge_resident4(p, uz, h, d4, M, acc, lsum);
                *reinterpret_cast<uint2 *>(out + h * kD + d4) = pack_out4<true>(acc, lsum);
            }
        }
        // the resident pass also leaves, per unit, the set it covered (for the rest pass)
        if (kResident) {
            for (int32_t uz = cta; uz < U; uz += grid) {
                uint32_t *bits = p.res_bits + (int64_t)uz * p.bits_words;
                for (int i = ctid; i < p.bits_words; i += kItemConsThreads) bits[i] = 0u;
                consumer_sync<kItemConsThreads>();
                const int32_t Lz = p.seq_len[uz];
                const int32_t ne = Lz > 0 ? min(max(p.gamma_n[uz], 0), p.k_e) : -1;
                for (int j = ctid; j <= ne; j += kItemConsThreads) {
                    const int32_t b = (j < ne) ? p.gamma_e[(int64_t)uz * p.k_e + j] : (Lz - 1) / kBlock;
                    if (b >= 0 && b < p.nblk) atomicOr(&bits[b >> 5], 1u << (b & 31));
                }
            }
        }
    }
}

namespace {

template <int kFmt, bool kWeights, bool kResident>
int launch_items(const DecodeParams &p, const CUtensorMap &tmap, const CUtensorMap &tail_map, cudaStream_t stream) {
    const auto kernel = decode_items_kernel<kFmt, kWeights, kResident>;
    const size_t smem = ItemGeo<kFmt, kResident>::smem_bytes(p.mode == kModeSel ? 0 : p.units + 1);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return NOSA_ERR_CUDA;
    const int grid = p.pieces > 0 ? p.units * p.pieces : decode_ctas();
    return launch_pdl(kernel, dim3(grid), dim3(kItemThreads), smem, stream, tmap, tail_map, p) == cudaSuccess
               ? NOSA_OK
               : NOSA_ERR_CUDA;
}

template <int kFmt>
int launch_items8(const DecodeParams &p, const CUtensorMap &tmap, const CUtensorMap &tail_map, cudaStream_t stream) {
    if (p.mode == kModeResident) return launch_items<kFmt, false, true>(p, tmap, tail_map, stream);
    return p.weights ? launch_items<kFmt, true, false>(p, tmap, tail_map, stream)
                     : launch_items<kFmt, false, false>(p, tmap, tail_map, stream);
}

}  // namespace

int launch_decode_items(const DecodeParams &p, const CUtensorMap &tmap, const CUtensorMap &tail_map, cudaStream_t stream) {
    if (p.fmt == kFmtInt8) return launch_items8<kFmtInt8>(p, tmap, tail_map, stream);
    if (p.fmt == kFmtE4m3) return launch_items8<kFmtE4m3>(p, tmap, tail_map, stream);
    return launch_items<kFmtBf16, true, false>(p, tmap, tail_map, stream);
}

}  // namespace nosa
