// attention_packed_backward.cu -- causal softmax attention of a packed batch with
// grouped key/value heads, backward.
//
// With P rebuilt from the saved lse, P = 2^(scale log2(e) q.k - lse):
//
//   delta = rowsum(dO O) ; dP = dO V^T ; dS = P (dP - delta)
//   dQ = scale dS K ; dV = sum over the group's heads of P^T dO ;
//   dK = scale sum over the group's heads of dS^T Q
//
// Two tensor-core kernels, so that every gradient is summed by one CTA in a fixed
// order (fp32, in tensor memory) and written once, without atomics; the price is
// that both rebuild S and dP, seven products where five would do.
//   packed_dq_kernel    items: (128 queries, head); streams the K and V tiles.
//   packed_dkdv_kernel  items: (128 keys, key/value head); streams the Q and dO
//                       tiles of every head of the group.
// P and dS are rounded to bf16 where they become operands of the next product, and dS
// of a sequence's first 128 tokens in two parts, dS = hi + lo, each with a product of its
// own.  Over many keys the roundings average out; a gradient that is one or two terms (a
// sequence of two tokens: dQ_1 = dS_10 K_0 + dS_11 K_1) has the whole of one, 2^-8, which
// made batches of short sequences up to twice as far off as the rounding of the result.
// Elsewhere the gradients are 1.35 to 1.45 times as far from 64 bits as their own rounding
// leaves them, which is what one product for each of P and dS costs.
//
// Tiles are 128 x 128 (128 x 64 for d = 160, whose accumulators leave tensor memory
// no more): with N = 128 an MMA of two shared-memory operands reads them at exactly
// the rate that shared memory delivers, with N = 64 it waits a third of the time.
// Eight softmax warps own half a row of the tile each.  They work in two steps,
// each of which frees one accumulator early: S is read (and P made) while dP is
// computed, dS is made while the next tile's S is computed, so the tensor cores
// always have a product of this or the next tile to work on.
//
// 8 x 1024 tokens, 32 heads on 8 of 128: 228 us (tensor cores 51 and 54 % busy, delta and
// plan 20 us of it); 23 sequences in 6007 tokens, 16 heads on 4 of 160: 110 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_packed.cuh"
#include "kernels.h"

namespace tpmlp {
namespace {

// 8 softmax warps, the producer's, and those that issue the MMAs: one warp for each
// chain of products, because a lone thread spends 55 clocks on an MMA that takes 64
// and some 240 on each barrier, ready or not, while the MMAs load shared memory.
// With one warp for all, the issuer and not the tensor cores set the pace (3400 to
// 4400 clocks a tile against 1536 and 2048 of MMAs).
constexpr int kDqThreads = 384;    // S, dP and dQ
constexpr int kDkvThreads = 352;   // dV with S^T, and dK with dP^T, in each other's place

template <int D>
struct BwdCfg {
    static constexpr int NB = (D + 63) / 64;                // 64-column boxes per row
    static constexpr int BS = D <= 128 ? 128 : 64;          // rows of a streamed tile
    static constexpr int HALF = BS / 2;                     // columns of a tile a softmax warp owns
    static constexpr int OWN = NB * 128 * kRowBytes;        // a resident operand: 128 rows
    static constexpr int STREAM = NB * BS * kRowBytes;      // a streamed operand
    static constexpr int STATS = 2 * 2 * 2 * HALF * 4;      // two tiles' lse and delta, by halves
    static constexpr int BARS = 512;
    // Rings of the streamed operands: FAR holds the one whose last use is a tile behind
    // its first (K for dQ, Q for dK), NEAR the other.  Three and two slots for d = 96
    // and 128 are all that fits, and what keeps a load a tile ahead of its use.
    static constexpr int FIT = (227 * 1024 - 2 * OWN - STATS - BARS) / STREAM;
    static constexpr int NEAR = FIT / 2 > 4 ? 4 : FIT / 2;
    static constexpr int FAR = FIT - NEAR > 4 ? 4 : FIT - NEAR;
    static constexpr int SMEM = 2 * OWN + (FAR + NEAR) * STREAM + STATS + BARS;
    static_assert(NEAR >= 2 && FAR >= 3, "slots");
    // Tensor memory.  Packed P or dS of softmax half w overlays the first columns of
    // that half's fp32 columns, at HALF w.  Accumulators of N >= 128 start on
    // multiples of 128.  dQ kernel: S, two dP, dQ; dK/dV kernel: S^T, dP^T, dV, dK.
    static constexpr uint32_t kS = 0;
    static constexpr uint32_t dp(int b) { return BS * (1u + b); }
    static constexpr uint32_t kDQ = D <= 128 ? 384 : 256;
    static constexpr uint32_t kDQTail = D <= 128 ? kDQ + (D / 64) * 64 : 384;
    static constexpr uint32_t acc(int x) { return D <= 128 ? 256u + 128u * x : 128u + 128u * x; }
    static constexpr uint32_t acc_tail(int x) { return D <= 128 ? acc(x) + (D / 64) * 64 : 384u + 32u * x; }
};

// The kernels' tiles start on 1024-byte boundaries (the swizzle's period), and their
// shared memory leaves no room to look for one.
__device__ __forceinline__ bool tiles_aligned(const uint8_t* smem, int* status) {
    if ((smem_u32(smem) & 1023u) == 0) return true;
    if (threadIdx.x == 0) atomicExch(status, kStatusTimeout);
    return false;
}

struct BwdArgs {
    const int4* entries;
    unsigned* plan;
    int nh, nkv, group;
    int split;           // parts of a group's heads (dK/dV kernel)
    int part_heads;      // a part's heads; the first part_more parts have one more
    int part_more;
    float* parts;        // [split][T][nkv][dV, dK][d] where split > 1
    long long T;
    float scale, scale2;
    const float* lse;    // [nh, T]
    const float* delta;  // [nh, T]
    __nv_bfloat16 *dQ, *dK, *dV;
    long long ldq, ldk, ldv;
    int* status;
};

// A role's place in a ring of N slots.
template <int N>
struct RingSlot {
    int at = 0;
    uint32_t phase = 0, issued = 0, issued_phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) {
            at = 0;
            phase ^= 1u;
        }
    }
    // the producer's: remembers the copy it has started
    __device__ __forceinline__ void issue() {
        issued |= 1u << at;
        issued_phase = (issued_phase & ~(1u << at)) | (phase << at);
        next();
    }
    __device__ __forceinline__ void drain(uint64_t* full, int* status, int site) {
        for (int i = 0; i < N; ++i)
            if (issued & (1u << i)) wait_drain(&full[i], (issued_phase >> i) & 1u, status, site);
    }
};

// HALF consecutive 32-bit columns of this thread's lane.
template <int HALF>
__device__ __forceinline__ void tmem_ld_half(uint32_t addr, uint32_t (&v)[HALF / 32][32]) {
#pragma unroll
    for (int c = 0; c < HALF / 32; ++c) warp_tmem_ld32(addr + 32 * c, v[c]);
#pragma unroll
    for (int c = 0; c < HALF / 32; ++c) tmem_loaded(v[c]);
}

// The same value, or the columns' own (in shared memory, the same for every lane), as
// pairs for columns 4 i .. 4 i + 3.
struct OneValue {
    uint64_t v;
    __device__ __forceinline__ ulonglong2 operator()(int) const { return make_ulonglong2(v, v); }
};
struct ColumnValues {
    const float* p;
    __device__ __forceinline__ ulonglong2 operator()(int i) const {
        return reinterpret_cast<const ulonglong2*>(p)[i];
    }
};

__device__ __forceinline__ uint64_t pair_of(const uint32_t (&v)[32], int i) {
    return f32x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
}

// x = scale2 s + neg_lse, p = 2^x of 32 columns of a row.  With MASK, columns outside
// [lo, hi) give an exact zero whatever s holds.
template <bool MASK, typename Lse>
__device__ __forceinline__ void weights(const uint32_t (&v)[32], uint64_t scale2, Lse neg_lse, int lo, int hi,
                                        float (&p)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const ulonglong2 l = neg_lse(i / 4);
        float x[4];
        f32x2_split(fma_f32x2(pair_of(v, i), scale2, l.x), x[0], x[1]);
        f32x2_split(fma_f32x2(pair_of(v, i + 2), scale2, l.y), x[2], x[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (MASK && (i + e < lo || i + e >= hi)) x[e] = -INFINITY;
            p[i + e] = ex2(x[e]);
        }
    }
}

// dS = p (dP + neg_delta), packed; masked columns are exact zeros here too.
template <bool MASK, typename Delta>
__device__ __forceinline__ void score_grads(const uint32_t (&v)[32], const float (&p)[32], Delta neg_dlt, int lo, int hi,
                                            uint32_t (&dd)[16]) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const ulonglong2 l = neg_dlt(i / 4);
        float x[4];
        f32x2_split(mul_f32x2(f32x2(p[i], p[i + 1]), add_f32x2(pair_of(v, i), l.x)), x[0], x[1]);
        f32x2_split(mul_f32x2(f32x2(p[i + 2], p[i + 3]), add_f32x2(pair_of(v, i + 2), l.y)), x[2], x[3]);
        if (MASK) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < lo || i + e >= hi) x[e] = 0.0f;
        }
        dd[i / 2] = pack_bf16x2(x[0], x[1]);
        dd[i / 2 + 1] = pack_bf16x2(x[2], x[3]);
    }
}

// The same in two parts, each packed: dS rounded, and what that leaves.
template <typename Delta>
__device__ __forceinline__ void score_grads_two(const uint32_t (&v)[32], const float (&p)[32], Delta neg_dlt, int lo,
                                                int hi, uint32_t (&dd)[16], uint32_t (&rest)[16]) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const ulonglong2 l = neg_dlt(i / 4);
        float x[4];
        f32x2_split(mul_f32x2(f32x2(p[i], p[i + 1]), add_f32x2(pair_of(v, i), l.x)), x[0], x[1]);
        f32x2_split(mul_f32x2(f32x2(p[i + 2], p[i + 3]), add_f32x2(pair_of(v, i + 2), l.y)), x[2], x[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < lo || i + e >= hi) x[e] = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const uint32_t w = pack_bf16x2(x[e], x[e + 1]);
            dd[(i + e) / 2] = w;
            rest[(i + e) / 2] = pack_bf16x2(x[e] - __uint_as_float(w << 16), x[e + 1] - __uint_as_float(w & 0xFFFF0000u));
        }
    }
}

// delta = rowsum(dO O) of every token and head; the first CTA makes the plan.  A warp
// takes a head of 8 tokens, all of their loads at once, a row to as many lanes as it has
// 16-byte pieces; the next warp the next head, whose rows lie behind.
constexpr int kPrepareThreads = 256, kPrepareTokens = 8;

template <int D>
__global__ void __launch_bounds__(kPrepareThreads)
    packed_prepare_kernel(const __nv_bfloat16* dO, const __nv_bfloat16* O, long long T, int nh, float* delta,
                          const int* cu, int nb, int4* entries, unsigned* plan, int* ranks, int* status) {
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0) {
        plan_block(cu, nb, static_cast<int>(T), 128, entries, plan, ranks, status);
        return;
    }
    constexpr int PIECES = D / 8, LANES = PIECES <= 8 ? 8 : PIECES <= 16 ? 16 : 32;
    constexpr int ROWS = 32 / LANES, PASSES = kPrepareTokens / ROWS;
    const int lane = threadIdx.x & 31, sub = lane % LANES;
    const long long unit = static_cast<long long>(blockIdx.x - 1) * (kPrepareThreads / 32) + threadIdx.x / 32;
    const long long tok0 = unit / nh * kPrepareTokens + lane / LANES;
    const long long head = unit % nh;
    uint4 g[PASSES], o[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const long long tok = tok0 + i * ROWS;
        g[i] = o[i] = make_uint4(0u, 0u, 0u, 0u);
        if (tok < T && sub < PIECES) {
            const long long at = (tok * nh + head) * PIECES + sub;
            g[i] = __ldg(reinterpret_cast<const uint4*>(dO) + at);
            o[i] = __ldg(reinterpret_cast<const uint4*>(O) + at);
        }
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const uint32_t gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w}, ow[4] = {o[i].x, o[i].y, o[i].z, o[i].w};
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            sum = fmaf(__uint_as_float(gw[k] << 16), __uint_as_float(ow[k] << 16), sum);
            sum = fmaf(__uint_as_float(gw[k] & 0xFFFF0000u), __uint_as_float(ow[k] & 0xFFFF0000u), sum);
        }
#pragma unroll
        for (int x = LANES / 2; x > 0; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
        const long long tok = tok0 + i * ROWS;
        if (sub == 0 && tok < T) delta[head * T + tok] = sum;
    }
}

// ------------------------------------------------------------- dQ

template <int D>
__global__ void __launch_bounds__(kDqThreads, 1)
    packed_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,  // 128 rows
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,   // BS rows
                     const BwdArgs a) {
    using C = BwdCfg<D>;
    constexpr int FAR = C::FAR, NEAR = C::NEAR, BS = C::BS, HALF = C::HALF;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (!tiles_aligned(smem, a.status)) return;
    uint8_t* sQ = smem;
    uint8_t* sdO = sQ + C::OWN;
    uint8_t* sK = sdO + C::OWN;           // [FAR]
    uint8_t* sV = sK + FAR * C::STREAM;   // [NEAR]
    uint64_t* bars = reinterpret_cast<uint64_t*>(sV + NEAR * C::STREAM + C::STATS);
    uint64_t* q_full = bars;              // the item's Q has landed
    uint64_t* q_empty = bars + 1;         // its last S has read it
    uint64_t* do_full = bars + 2;         // the same for dO and dP
    uint64_t* do_empty = bars + 3;
    uint64_t* s_full = bars + 4;          // S is complete
    uint64_t* s_read = bars + 5;          // the softmax warps have read it
    uint64_t* dq_done = bars + 6;         // the item's dQ is complete
    uint64_t* dq_free = bars + 7;         // the softmax warps have read it out
    uint64_t* dp_full = bars + 8;         // [2] dP is complete
    uint64_t* ds_full = bars + 10;        // [2] dS is in its place
    uint64_t* item_full = bars + 12;      // [2]
    uint64_t* item_empty = bars + 14;     // [2]
    uint64_t* drain = bars + 16;
    uint64_t* k_full = bars + 17;         // [FAR]
    uint64_t* k_empty = bars + 21;
    uint64_t* v_full = bars + 25;         // [NEAR]
    uint64_t* v_empty = bars + 29;
    uint64_t* ds_used = bars + 33;        // [2] dQ has read dS
    int* items = reinterpret_cast<int*>(bars + 35);  // [2] x {first row, length, tile, head}
    uint32_t* misc = reinterpret_cast<uint32_t*>(items + 8);
    volatile uint32_t* abort_flag = misc + 1;
    static_assert(35 * 8 + 8 * 4 + 8 <= C::BARS && FAR <= 4 && NEAR <= 4, "barrier space");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    struct Item {
        int row0, len, q0, head, n_kv;
    };
    auto decode = [&](int slot) {
        const volatile int* p = items + 4 * slot;
        Item it;
        it.row0 = p[0];
        it.len = p[1];
        it.q0 = p[2] * 128;
        it.head = p[3];
        it.n_kv = (min(it.q0 + 128, it.len) - 1) / BS + 1;  // tiles with keys up to the last query
        return it;
    };

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(do_full, 1);
        mbar_init(do_empty, 1);
        mbar_init(s_full, 1);
        mbar_init(s_read, 8);
        mbar_init(dq_done, 1);
        mbar_init(dq_free, 8);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&dp_full[b], 1);
            mbar_init(&ds_full[b], 8);
            mbar_init(&item_full[b], 1);
            mbar_init(&ds_used[b], 1);
            mbar_init(&item_empty[b], 11);  // the 3 MMA threads and the 8 softmax warps
        }
        for (int i = 0; i < FAR; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NEAR; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(drain, 3);
        misc[1] = 0u;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&misc[0], 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    pdl_wait();  // the plan and delta are there
    pdl_launch_dependents();  // the dK/dV kernel needs nothing else

    if (warp == 8) {
        // ------------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_do);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            const unsigned total = a.plan[kPlanCount] * static_cast<unsigned>(a.nh);
            RingSlot<FAR> ks;
            RingSlot<NEAR> vs;
            int q_loads = 0, do_loads = 0;
            bool ok = true;
            for (int k = 0;; ++k) {
                const int slot = k & 1;
                if (k >= 2 && !thread_wait(&item_empty[slot], static_cast<uint32_t>((k - 2) >> 1) & 1u, abort_flag,
                                            a.status, 0x511))
                    ok = false;
                unsigned item = total;
                if (ok) item = atomicAdd(&a.plan[kPlanWork0], 1u);
                if (item >= total) {
                    items[4 * slot + 1] = 0;  // no sequence: the end
                    mbar_arrive(&item_full[slot]);
                    break;
                }
                {
                    const int4 e = a.entries[item / a.nh];
                    items[4 * slot] = e.x;
                    items[4 * slot + 1] = e.y;
                    items[4 * slot + 2] = e.z;
                    items[4 * slot + 3] = static_cast<int>(item % a.nh);
                }
                mbar_arrive(&item_full[slot]);
                const Item it = decode(slot);
                const int qcol = it.head * D, kcol = it.head / a.group * D, row = it.row0 + it.q0;
                const uint32_t before = static_cast<uint32_t>(k - 1) & 1u;
                // Q goes first: the next S needs it while dP still needs the last dO
                if (k >= 1 && !thread_wait(q_empty, before, abort_flag, a.status, 0x512)) break;
                mbar_arrive_expect_tx(q_full, C::OWN);
                for (int b = 0; b < C::NB; ++b)
                    tma_load_3d(&tm_q, smem_u32(q_full), smem_u32(sQ) + b * 128 * kRowBytes, qcol + 64 * b, row, 0);
                ++q_loads;
                for (int j = 0; j < it.n_kv; ++j) {
                    if (!thread_wait(&k_empty[ks.at], ks.phase ^ 1u, abort_flag, a.status, 0x501)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&k_full[ks.at], C::STREAM);
                    for (int b = 0; b < C::NB; ++b)
                        tma_load_3d(&tm_k, smem_u32(&k_full[ks.at]),
                                    smem_u32(sK) + ks.at * C::STREAM + b * BS * kRowBytes, kcol + 64 * b,
                                    it.row0 + j * BS, 0);
                    ks.issue();
                    if (j == 0) {
                        if (k >= 1 && !thread_wait(do_empty, before, abort_flag, a.status, 0x513)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(do_full, C::OWN);
                        for (int b = 0; b < C::NB; ++b)
                            tma_load_3d(&tm_do, smem_u32(do_full), smem_u32(sdO) + b * 128 * kRowBytes, qcol + 64 * b,
                                        row, 0);
                        ++do_loads;
                    }
                    if (!thread_wait(&v_empty[vs.at], vs.phase ^ 1u, abort_flag, a.status, 0x517)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&v_full[vs.at], C::STREAM);
                    for (int b = 0; b < C::NB; ++b)
                        tma_load_3d(&tm_v, smem_u32(&v_full[vs.at]),
                                    smem_u32(sV) + vs.at * C::STREAM + b * BS * kRowBytes, kcol + 64 * b,
                                    it.row0 + j * BS, 0);
                    vs.issue();
                }
                if (!ok) break;
            }
            // every copy this thread started lands before the CTA may exit
            if (q_loads > 0) wait_drain(q_full, static_cast<uint32_t>(q_loads - 1) & 1u, a.status, 0x502);
            if (do_loads > 0) wait_drain(do_full, static_cast<uint32_t>(do_loads - 1) & 1u, a.status, 0x503);
            ks.drain(k_full, a.status, 0x504);
            vs.drain(v_full, a.status, 0x518);
        }
        __syncwarp();
    } else if (warp >= 9) {
        // ----------------------- MMA issuers: S (warp 9), dP (warp 10), dQ (warp 11)
        {
            int g = 0;  // tiles so far
            RingSlot<FAR> ks;
            RingSlot<NEAR> vs;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int slot = k & 1;
                if (!warp_wait(&item_full[slot], static_cast<uint32_t>(k >> 1) & 1u, abort_flag, a.status, 0x515))
                    break;
                const Item it = decode(slot);
                __syncwarp();
                warp_arrive(&item_empty[slot]);
                if (it.len == 0) break;
                const uint32_t item_parity = static_cast<uint32_t>(k) & 1u;
                if (warp == 9) {
                    const uint32_t qdesc = desc_low(smem_u32(sQ), 16);
                    ok = warp_wait(q_full, item_parity, abort_flag, a.status, 0x506);
                    for (int j = 0; j < it.n_kv && ok; ++j, ++g, ks.next()) {
                        // (parity 1 of a barrier that has seen no phase counts as complete)
                        if (!(ok = warp_wait_both(&k_full[ks.at], ks.phase, s_read, static_cast<uint32_t>(g + 1) & 1u,
                                                  abort_flag, a.status, 0x507)))
                            break;
                        tc_fence_after();
                        warp_mma_scores<D, BS>(tmem + C::kS, qdesc, desc_low(smem_u32(sK) + ks.at * C::STREAM, 16));
                        warp_commit(s_full);
                    }
                    if (ok) warp_commit(q_empty);
                } else if (warp == 10) {
                    const uint32_t dodesc = desc_low(smem_u32(sdO), 16);
                    ok = warp_wait(do_full, item_parity, abort_flag, a.status, 0x509);
                    for (int j = 0; j < it.n_kv && ok; ++j, ++g, vs.next()) {
                        const int b = g & 1;
                        // over the dS of the tile before the last, which its dQ has read
                        if (!(ok = warp_wait_both(&v_full[vs.at], vs.phase, &ds_used[b],
                                                  static_cast<uint32_t>((g >> 1) + 1) & 1u, abort_flag, a.status, 0x519)))
                            break;
                        tc_fence_after();
                        warp_mma_scores<D, BS>(tmem + C::dp(b), dodesc,
                                      desc_low(smem_u32(sV) + vs.at * C::STREAM, 16));
                        warp_commit(&dp_full[b]);
                        warp_commit(&v_empty[vs.at]);
                    }
                    if (ok) warp_commit(do_empty);
                } else {
                    // the first product of an item overwrites the last item's dQ
                    ok = k == 0 || warp_wait(dq_free, static_cast<uint32_t>(k - 1) & 1u, abort_flag, a.status, 0x514);
                    for (int j = 0; j < it.n_kv && ok; ++j, ++g, ks.next()) {
                        const int b = g & 1;
                        if (!(ok = warp_wait(&ds_full[b], static_cast<uint32_t>(g >> 1) & 1u, abort_flag, a.status,
                                               0x505)))
                            break;
                        tc_fence_after();
                        warp_mma_values<D, BS, HALF>(tmem + C::kDQ, tmem + C::kDQTail, tmem + C::dp(b),
                                      desc_low(smem_u32(sK) + ks.at * C::STREAM, BS * kRowBytes), j > 0);
                        if (it.q0 == 0)  // dS's second part
                            warp_mma_values<D, BS, HALF>(tmem + C::kDQ, tmem + C::kDQTail, tmem + C::dp(b) + HALF / 2,
                                      desc_low(smem_u32(sK) + ks.at * C::STREAM, BS * kRowBytes), true);
                        warp_commit(&ds_used[b]);
                        warp_commit(&k_empty[ks.at]);
                    }
                    if (ok) warp_commit(dq_done);
                }
            }
            warp_commit(drain);
            if (lane == 0) wait_drain(drain, 0, a.status, 0x50A);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------- softmax warps
        const int w = warp >> 2;            // which half of a tile's columns
        const int r = threadIdx.x & 127;    // query row = TMEM lane
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        constexpr int CH = D / 32, MID = (CH + 1) / 2;  // dQ chunks of half 0: [0, MID)
        bool ok = true;
        int g = 0, k_slot = 0;
        struct Pending {
            int k, head, valid;
            long long row;
        };
        Pending pend{-1, 0, 0, 0};
        auto readout = [&]() -> bool {
            if (!warp_wait(dq_done, static_cast<uint32_t>(pend.k) & 1u, abort_flag, a.status, 0x50B))
                return false;
            tc_fence_after();
            const RowsOut out(a.dQ, a.ldq, pend.row, pend.head * D, pend.valid);
            for (int c = w ? MID : 0; c < (w ? CH : MID); ++c)
                read_out(out, c, lane_addr + (c < (D / 64) * 2 ? C::kDQ + 32 * c : C::kDQTail + 32 * (c - (D / 64) * 2)),
                         a.scale);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dq_free);
            pend.k = -1;
            return true;
        };
        for (int k = 0; ok; ++k) {
            const int slot = k & 1;
            if (!warp_wait(&item_full[slot], static_cast<uint32_t>(k >> 1) & 1u, abort_flag, a.status, 0x516))
                break;
            const Item it = decode(slot);
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[slot]);
            if (it.len == 0) break;
            const int first_q = it.q0 + (warp & 3) * 32, q = it.q0 + r;  // the warp's first, this lane's
            const bool q_ok = q < it.len;
            const long long tok = static_cast<long long>(it.row0) + q;
            const float lse = q_ok ? __ldg(a.lse + it.head * a.T + tok) : 0.0f;
            const float dlt = q_ok ? __ldg(a.delta + it.head * a.T + tok) : 0.0f;
            const OneValue neg_lse{f32x2(-lse, -lse)}, neg_dlt{f32x2(-dlt, -dlt)};
            const uint64_t scale2 = f32x2(a.scale2, a.scale2);
            for (int j = 0; j < it.n_kv; ++j, ++g) {
                const int b = g & 1, key0 = j * BS + w * HALF;  // first key of this half
                // chunks of 32 keys: the warp's queries see the first `live`, the last of
                // those up to the diagonal if that is in this half (keys behind the
                // sequence's end come after its last query)
                const int live = ((first_q - key0) >> 5) + 1;
                if (!warp_wait(s_full, static_cast<uint32_t>(g) & 1u, abort_flag, a.status, 0x50C)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t v[HALF / 32][32];
                tmem_ld_half<HALF>(lane_addr + C::kS + w * HALF, v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_read);
                float p[HALF / 32][32];
#pragma unroll
                for (int c = 0; c < HALF / 32; ++c)
                    if (c < live) weights<false>(v[c], scale2, neg_lse, 0, 0, p[c]);
                if (!warp_wait(&dp_full[b], static_cast<uint32_t>(g >> 1) & 1u, abort_flag, a.status, 0x50D)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t dp = lane_addr + C::dp(b) + w * HALF;
                tmem_ld_half<HALF>(dp, v);
#pragma unroll
                for (int c = 0; c < HALF / 32; ++c) {
                    uint32_t dd[16];
                    if (c >= live) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) dd[i] = 0u;
                        if (it.q0 == 0) warp_tmem_st16(dp + HALF / 2 + 16 * c, dd);
                    } else if (it.q0 == 0) {  // the second part goes behind the first of the whole half
                        uint32_t rest[16];
                        score_grads_two(v[c], p[c], neg_dlt, 0, c == live - 1 ? lane + 1 : 32, dd, rest);
                        warp_tmem_st16(dp + HALF / 2 + 16 * c, rest);
                    } else if (c == live - 1) {
                        score_grads<true>(v[c], p[c], neg_dlt, 0, lane + 1, dd);
                    } else {
                        score_grads<false>(v[c], p[c], neg_dlt, 0, 0, dd);
                    }
                    warp_tmem_st16(dp + 16 * c, dd);
                }
                __syncwarp();
                tmem_wait_st();
                tc_fence_before();
                // K rows behind the sequence's end (S, their first use, is done)
                if ((j + 1) * BS > it.len)
                    zero_rows<C::NB>(smem_u32(sK) + k_slot * C::STREAM, BS, it.len - j * BS, threadIdx.x, 256);
                __syncwarp();
                if (lane == 0) mbar_arrive(&ds_full[b]);
                if (++k_slot == FAR) k_slot = 0;
                // the last item's dQ, while the tensor cores have this item's next tile
                if (pend.k >= 0 && !readout()) {
                    ok = false;
                    break;
                }
            }
            if (!ok) break;
            pend = Pending{k, it.head, it.len - first_q, static_cast<long long>(it.row0) + first_q};
        }
        if (ok && pend.k >= 0) readout();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------- dK, dV

template <int D>
__global__ void __launch_bounds__(kDkvThreads, 1)
    packed_dkdv_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,   // 128 rows
                       const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,  // BS rows
                       const BwdArgs a) {
    using C = BwdCfg<D>;
    constexpr int FAR = C::FAR, NEAR = C::NEAR, BS = C::BS, HALF = C::HALF;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (!tiles_aligned(smem, a.status)) return;
    uint8_t* sK = smem;
    uint8_t* sV = sK + C::OWN;
    uint8_t* sQ = sV + C::OWN;            // [FAR]
    uint8_t* sdO = sQ + FAR * C::STREAM;  // [NEAR]
    float* stats = reinterpret_cast<float*>(sdO + NEAR * C::STREAM);  // [tile & 1][half][lse, delta][HALF], negated
    uint64_t* bars = reinterpret_cast<uint64_t*>(sdO + NEAR * C::STREAM + C::STATS);
    uint64_t* k_full = bars;              // the item's K has landed
    uint64_t* k_empty = bars + 1;         // its last S^T has read it
    uint64_t* v_full = bars + 2;          // the same for V and dP^T
    uint64_t* v_empty = bars + 3;
    uint64_t* s_full = bars + 4;          // S^T is complete
    uint64_t* p_full = bars + 5;          // P^T is in its place
    uint64_t* dp_full = bars + 6;         // dP^T is complete
    uint64_t* ds_full = bars + 7;         // dS^T is in its place
    uint64_t* grad_done = bars + 8;       // the item's dV and dK are complete
    uint64_t* grad_free = bars + 9;       // the softmax warps have read them out
    uint64_t* item_full = bars + 10;      // [2]
    uint64_t* item_empty = bars + 12;     // [2]
    uint64_t* drain = bars + 14;
    uint64_t* q_full = bars + 15;         // [FAR]
    uint64_t* q_empty = bars + 19;
    uint64_t* do_full = bars + 23;        // [NEAR]
    uint64_t* do_empty = bars + 27;
    uint64_t* stat_full = bars + 31;      // [2] the half's lse and delta of the tile are there
    int* items = reinterpret_cast<int*>(bars + 33);  // [2] x {first row, length, key tile, head}
    uint32_t* misc = reinterpret_cast<uint32_t*>(items + 8);
    volatile uint32_t* abort_flag = misc + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    struct Item {
        int row0, len, k0, kv_head, part, head, i0, nq, tiles;
    };
    auto decode = [&](int slot) {
        const volatile int* p = items + 4 * slot;
        Item it;
        it.row0 = p[0];
        it.len = p[1];
        it.k0 = p[2] * 128;
        it.kv_head = p[3] / a.split;
        it.part = p[3] - it.kv_head * a.split;
        it.head = it.kv_head * a.group + it.part * a.part_heads + min(it.part, a.part_more);
        it.i0 = it.k0 / BS;                         // first query tile that sees the keys
        it.nq = (it.len + BS - 1) / BS - it.i0;     // query tiles of each head
        it.tiles = it.nq * (a.part_heads + (it.part < a.part_more));
        return it;
    };

    if (threadIdx.x == 0) {
        mbar_init(k_full, 1);
        mbar_init(k_empty, 1);
        mbar_init(v_full, 1);
        mbar_init(v_empty, 1);
        mbar_init(s_full, 1);
        mbar_init(p_full, 8);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, 8);
        mbar_init(grad_done, 2);
        mbar_init(grad_free, 8);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&item_full[b], 1);
            mbar_init(&item_empty[b], 10);  // the 2 MMA threads and the 8 softmax warps
            mbar_init(&stat_full[b], 4);
        }
        for (int i = 0; i < FAR; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < NEAR; ++i) {
            mbar_init(&do_full[i], 1);
            mbar_init(&do_empty[i], 2);  // read for dP^T and dV
        }
        mbar_init(drain, 2);
        misc[1] = 0u;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&misc[0], 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    // No pdl_wait() here: the dQ kernel lets this one begin once the plan and delta are
    // complete, and where its CTAs run out of items this one's take the SMs over.  What
    // was written since (plan, delta) is read past the first-level cache.

    if (warp == 8) {
        // ------------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_do);
            const unsigned units = static_cast<unsigned>(a.nkv * a.split);
            const unsigned total = __ldcg(&a.plan[kPlanCount]) * units;
            RingSlot<FAR> qs;
            RingSlot<NEAR> os;
            int k_loads = 0, v_loads = 0;
            bool ok = true;
            for (int k = 0;; ++k) {
                const int slot = k & 1;
                if (k >= 2 && !thread_wait(&item_empty[slot], static_cast<uint32_t>((k - 2) >> 1) & 1u, abort_flag,
                                            a.status, 0x611))
                    ok = false;
                unsigned item = total;
                if (ok) item = atomicAdd(&a.plan[kPlanWork1], 1u);
                if (item >= total) {
                    items[4 * slot + 1] = 0;  // no sequence: the end
                    mbar_arrive(&item_full[slot]);
                    break;
                }
                {
                    const int4 e = __ldcg(&a.entries[item / units]);
                    items[4 * slot] = e.x;
                    items[4 * slot + 1] = e.y;
                    items[4 * slot + 2] = e.w - 1 - e.z;  // the highest rank is the first key tile
                    items[4 * slot + 3] = static_cast<int>(item % units);
                }
                mbar_arrive(&item_full[slot]);
                const Item it = decode(slot);
                const int kcol = it.kv_head * D, row = it.row0 + it.k0;
                const uint32_t before = static_cast<uint32_t>(k - 1) & 1u;
                if (k >= 1 && !thread_wait(k_empty, before, abort_flag, a.status, 0x612)) break;
                mbar_arrive_expect_tx(k_full, C::OWN);
                for (int b = 0; b < C::NB; ++b)
                    tma_load_3d(&tm_k, smem_u32(k_full), smem_u32(sK) + b * 128 * kRowBytes, kcol + 64 * b, row, 0);
                ++k_loads;
                int head = it.head, i = 0;
                for (int n = 0; n < it.tiles; ++n) {
                    const int qrow = it.row0 + (it.i0 + i) * BS;
                    if (!thread_wait(&q_empty[qs.at], qs.phase ^ 1u, abort_flag, a.status, 0x601)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&q_full[qs.at], C::STREAM);
                    for (int b = 0; b < C::NB; ++b)
                        tma_load_3d(&tm_q, smem_u32(&q_full[qs.at]),
                                    smem_u32(sQ) + qs.at * C::STREAM + b * BS * kRowBytes, head * D + 64 * b, qrow, 0);
                    qs.issue();
                    if (n == 0) {
                        if (k >= 1 && !thread_wait(v_empty, before, abort_flag, a.status, 0x613)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(v_full, C::OWN);
                        for (int b = 0; b < C::NB; ++b)
                            tma_load_3d(&tm_v, smem_u32(v_full), smem_u32(sV) + b * 128 * kRowBytes, kcol + 64 * b, row,
                                        0);
                        ++v_loads;
                    }
                    if (!thread_wait(&do_empty[os.at], os.phase ^ 1u, abort_flag, a.status, 0x617)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&do_full[os.at], C::STREAM);
                    for (int b = 0; b < C::NB; ++b)
                        tma_load_3d(&tm_do, smem_u32(&do_full[os.at]),
                                    smem_u32(sdO) + os.at * C::STREAM + b * BS * kRowBytes, head * D + 64 * b, qrow,
                                    0);
                    os.issue();
                    if (++i == it.nq) {
                        i = 0;
                        ++head;
                    }
                }
                if (!ok) break;
            }
            // every copy this thread started lands before the CTA may exit
            if (k_loads > 0) wait_drain(k_full, static_cast<uint32_t>(k_loads - 1) & 1u, a.status, 0x602);
            if (v_loads > 0) wait_drain(v_full, static_cast<uint32_t>(v_loads - 1) & 1u, a.status, 0x603);
            qs.drain(q_full, a.status, 0x604);
            os.drain(do_full, a.status, 0x618);
        }
        __syncwarp();
    } else if (warp >= 9) {
        // -------- MMA issuers: dV and S^T (warp 9), dK and dP^T (warp 10).  The product
        // of a tile that reads P^T (dS^T) goes before the next tile's S^T (dP^T), which
        // overwrites it: MMAs of one thread run in order.
        {
            const bool first = warp == 9;
            const uint32_t own = desc_low(smem_u32(first ? sK : sV), 16);
            const uint32_t tile = tmem + (first ? C::kS : C::dp(0));
            const uint32_t acc = tmem + (first ? C::acc(0) : C::acc(1));
            const uint32_t tail = tmem + (first ? C::acc_tail(0) : C::acc_tail(1));
            int g = 0;  // tiles so far
            RingSlot<FAR> qs;
            RingSlot<NEAR> os;
            bool ok = true;
            // the tile whose gradient product is still to be issued
            int last_q = 0, last_o = 0, last_k = -1;
            uint32_t last_o_phase = 0;
            bool last_first = false, last_final = false, last_two = false;
            auto issue_grad = [&]() {
                if (last_k < 0 || !ok) return;
                const uint32_t parity = static_cast<uint32_t>(g - 1) & 1u;
                // the first products of an item overwrite the last item's gradients
                if (last_first && last_k >= 1)
                    ok = warp_wait(grad_free, static_cast<uint32_t>(last_k - 1) & 1u, abort_flag, a.status, 0x614);
                ok = ok && (first ? warp_wait_both(&do_full[last_o], last_o_phase, p_full, parity, abort_flag, a.status,
                                                   0x605)
                                  : warp_wait(ds_full, parity, abort_flag, a.status, 0x60E));
                if (!ok) return;
                tc_fence_after();
                // dV += P^T dO, dK += dS^T Q
                const uint32_t rows = first ? smem_u32(sdO) + last_o * C::STREAM : smem_u32(sQ) + last_q * C::STREAM;
                warp_mma_values<D, BS, HALF>(acc, tail, tile, desc_low(rows, BS * kRowBytes), !last_first);
                if (last_two)  // dS's second part
                    warp_mma_values<D, BS, HALF>(acc, tail, tile + HALF / 2, desc_low(rows, BS * kRowBytes), true);
                warp_commit(first ? &do_empty[last_o] : &q_empty[last_q]);
                if (last_final) warp_commit(grad_done);
                last_k = -1;
            };
            for (int k = 0; ok; ++k) {
                const int slot = k & 1;
                if (!warp_wait(&item_full[slot], static_cast<uint32_t>(k >> 1) & 1u, abort_flag, a.status, 0x615))
                    break;
                const Item it = decode(slot);
                __syncwarp();
                warp_arrive(&item_empty[slot]);
                if (it.len == 0) break;
                int i = 0;  // the tile of its head
                for (int n = 0; n < it.tiles; ++n) {
                    uint64_t* full = first ? &q_full[qs.at] : &do_full[os.at];
                    const uint32_t phase = first ? qs.phase : os.phase;
                    if (n == 0) {
                        issue_grad();
                        ok = ok && warp_wait_both(first ? k_full : v_full, static_cast<uint32_t>(k) & 1u, full, phase,
                                                  abort_flag, a.status, 0x607);
                    } else {
                        // landed by now as a rule: the wait is over before the softmax is
                        ok = warp_wait(full, phase, abort_flag, a.status, 0x608);
                        issue_grad();
                    }
                    if (!ok) break;
                    tc_fence_after();
                    // S^T = K Q^T, dP^T = V dO^T
                    const uint32_t rows = first ? smem_u32(sQ) + qs.at * C::STREAM : smem_u32(sdO) + os.at * C::STREAM;
                    warp_mma_scores<D, BS>(tile, own, desc_low(rows, 16));
                    warp_commit(first ? s_full : dp_full);
                    if (!first) warp_commit(&do_empty[os.at]);
                    if (n == it.tiles - 1) warp_commit(first ? k_empty : v_empty);
                    last_q = qs.at;
                    last_o = os.at;
                    last_o_phase = os.phase;
                    last_k = k;
                    last_first = n == 0;
                    last_final = n == it.tiles - 1;
                    last_two = !first && (it.i0 + i) * BS < 128;
                    if (++i == it.nq) i = 0;
                    ++g;
                    qs.next();
                    os.next();
                }
            }
            issue_grad();
            warp_commit(drain);
            if (lane == 0) wait_drain(drain, 0, a.status, 0x60A);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------- softmax warps
        const int w = warp >> 2;            // which half of a tile's columns (queries)
        const int r = threadIdx.x & 127;    // key row = TMEM lane
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint64_t scale2 = f32x2(a.scale2, a.scale2);
        bool ok = true;
        int g = 0;
        RingSlot<FAR> qs;
        RingSlot<NEAR> os;
        for (int k = 0; ok; ++k) {
            const int slot = k & 1;
            if (!warp_wait(&item_full[slot], static_cast<uint32_t>(k >> 1) & 1u, abort_flag, a.status, 0x616))
                break;
            const Item it = decode(slot);
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[slot]);
            if (it.len == 0) break;
            const int first_key = it.k0 + (warp & 3) * 32;  // the warp's
            // a value of the tile's lse or delta per thread, loaded a tile ahead
            float stat_n = 0.0f;
            auto fetch = [&](int head, int i) {
                if (r < 2 * HALF) {
                    const int qq = (it.i0 + i) * BS + w * HALF + r % HALF;
                    stat_n = qq < it.len ? -__ldcg((r < HALF ? a.lse : a.delta) + head * a.T + it.row0 + qq) : 0.0f;
                }
            };
            int head = it.head, i = 0;
            fetch(head, 0);
            for (int n = 0; n < it.tiles; ++n, ++g) {
                const uint32_t parity = static_cast<uint32_t>(g) & 1u;
                const int q0 = (it.i0 + i) * BS + w * HALF;  // first query of this half
                const int valid = it.len - (it.i0 + i) * BS;  // queries of the tile inside the sequence
                const bool tail = valid < BS;
                const bool two = (it.i0 + i) * BS < 128;  // dS in two parts
                // chunks of 32 queries: all of them see the warp's keys (full), none does or
                // none is inside the sequence (dead), or those in [lo, hi)
                auto full = [&](int c) { return q0 + 32 * c > first_key && q0 + 32 * c + 32 <= it.len; };
                auto dead = [&](int c) { return q0 + 32 * c < first_key || q0 + 32 * c >= it.len; };
                auto lo = [&](int c) { return q0 + 32 * c == first_key ? lane : q0 + 32 * c < first_key ? 32 : 0; };
                auto hi = [&](int c) { return it.len - q0 - 32 * c; };
                float* stat = stats + ((g & 1) * 2 + w) * 2 * HALF;
                if (r < 2 * HALF) stat[r] = stat_n;
                __syncwarp();
                if (lane == 0) mbar_arrive(&stat_full[w]);
                if (++i == it.nq) {
                    i = 0;
                    ++head;
                }
                if (n + 1 < it.tiles) fetch(head, i);
                // (a warp that passes has left the tile before the last, whose place this was)
                if (!warp_wait_both(&stat_full[w], parity, s_full, parity, abort_flag, a.status, 0x60B)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float p[HALF / 32][32];
#pragma unroll
                for (int c = 0; c < HALF / 32; ++c) {
                    uint32_t v[32];
                    warp_tmem_ld32(lane_addr + C::kS + w * HALF + 32 * c, v);
                    tmem_loaded(v);
                    const ColumnValues neg_lse{stat + 32 * c};
                    if (full(c)) {
                        weights<false>(v, scale2, neg_lse, 0, 0, p[c]);
                    } else if (dead(c)) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) p[c][e] = 0.0f;
                    } else {
                        weights<true>(v, scale2, neg_lse, lo(c), hi(c), p[c]);
                    }
                    uint32_t pp[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) pp[e] = pack_bf16x2(p[c][2 * e], p[c][2 * e + 1]);
                    warp_tmem_st16(lane_addr + C::kS + w * HALF + 16 * c, pp);
                }
                __syncwarp();
                tmem_wait_st();
                tc_fence_before();
                if (tail) {  // dO rows behind the end
                    if (!warp_wait(&do_full[os.at], os.phase, abort_flag, a.status, 0x61A)) {
                        ok = false;
                        break;
                    }
                    zero_rows<C::NB>(smem_u32(sdO) + os.at * C::STREAM, BS, valid, threadIdx.x, 256);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
                if (!warp_wait(dp_full, parity, abort_flag, a.status, 0x60C)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t dp = lane_addr + C::dp(0) + w * HALF;
                if (two) {
                    uint32_t rest[HALF / 32][16];
#pragma unroll
                    for (int c = 0; c < HALF / 32; ++c) {
                        uint32_t v[32], dd[16];
                        warp_tmem_ld32(dp + 32 * c, v);
                        tmem_loaded(v);
                        score_grads_two(v, p[c], ColumnValues{stat + HALF + 32 * c}, lo(c), hi(c), dd, rest[c]);
                        warp_tmem_st16(dp + 16 * c, dd);
                    }
                    // over the end of the half, which has all been read now
#pragma unroll
                    for (int c = 0; c < HALF / 32; ++c) warp_tmem_st16(dp + HALF / 2 + 16 * c, rest[c]);
                } else {
#pragma unroll
                    for (int c = 0; c < HALF / 32; ++c) {
                        uint32_t v[32], dd[16];
                        warp_tmem_ld32(dp + 32 * c, v);
                        tmem_loaded(v);
                        const ColumnValues neg_dlt{stat + HALF + 32 * c};
                        if (full(c)) {
                            score_grads<false>(v, p[c], neg_dlt, 0, 0, dd);
                        } else if (dead(c)) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) dd[e] = 0u;
                        } else {
                            score_grads<true>(v, p[c], neg_dlt, lo(c), hi(c), dd);
                        }
                        warp_tmem_st16(dp + 16 * c, dd);
                    }
                }
                __syncwarp();
                tmem_wait_st();
                tc_fence_before();
                // Q rows behind the end (S^T, their first use, is done)
                if (tail) zero_rows<C::NB>(smem_u32(sQ) + qs.at * C::STREAM, BS, valid, threadIdx.x, 256);
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full);
                qs.next();
                os.next();
            }
            if (!ok || !warp_wait(grad_done, static_cast<uint32_t>(k) & 1u, abort_flag, a.status, 0x60D)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // half 0 reads dV out, half 1 dK
            auto chunk = [&](int c) {
                return lane_addr + (c < (D / 64) * 2 ? C::acc(w) + 32 * c : C::acc_tail(w) + 32 * (c - (D / 64) * 2));
            };
            const long long first_row = static_cast<long long>(it.row0) + first_key;
            if (a.split == 1) {
                const RowsOut out(w ? a.dK : a.dV, w ? a.ldk : a.ldv, first_row, it.kv_head * D, it.len - first_key);
                for (int c = 0; c < D / 32; ++c) read_out(out, c, chunk(c), w ? a.scale : 1.0f);
            } else {
                // a part of the group's heads: its fp32 sum
                const bool wide = (reinterpret_cast<uintptr_t>(a.parts) & 31u) == 0;
                float* row = a.parts + (((it.part * a.T + first_row + lane) * a.nkv + it.kv_head) * 2 + w) * D;
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    warp_tmem_ld32(chunk(c), v);
                    tmem_loaded(v);
                    if (lane < it.len - first_key)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t u[8];
#pragma unroll
                            for (int f = 0; f < 8; ++f) u[f] = v[8 * e + f];
                            store_32(row + 32 * c + 8 * e, u, wide);
                        }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(grad_free);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    pdl_wait();  // what follows this kernel follows the dQ kernel too
    pdl_launch_dependents();
}

// dK and dV from the parts' sums, added in order: 8 values a thread, of the tokens that
// are in sequences.
__global__ void __launch_bounds__(256)
    packed_parts_kernel(const BwdArgs a, int d, const int* cu, int nb) {
    pdl_launch_dependents();
    pdl_wait();
    const int pieces = d / 8;
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;  // [token][kv head][dV, dK][piece]
    const long long tok = i / (2 * pieces * a.nkv);
    if (a.plan[kPlanCount] == 0u || tok < cu[0] || tok >= cu[nb]) return;
    const int rest = static_cast<int>(i - tok * (2 * pieces * a.nkv));
    const int head = rest / (2 * pieces), x = rest / pieces & 1, c = rest % pieces * 8;
    const long long plane = a.T * a.nkv * 2 * d;
    const float* p = a.parts + i * 8;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < a.split; ++s) {
        const float4 lo = *reinterpret_cast<const float4*>(p + s * plane);
        const float4 hi = *reinterpret_cast<const float4*>(p + s * plane + 4);
        v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
        v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
    }
    const float f = x ? a.scale : 1.0f;
    __nv_bfloat16* out = (x ? a.dK + tok * a.ldk : a.dV + tok * a.ldv) + head * d + c;
    *reinterpret_cast<uint4*>(out) = make_uint4(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f),
                                                pack_bf16x2(v[4] * f, v[5] * f), pack_bf16x2(v[6] * f, v[7] * f));
}

template <int D>
cudaError_t launch_bwd(const CUtensorMap& q128, const CUtensorMap& do128, const CUtensorMap& k128,
                       const CUtensorMap& v128, const CUtensorMap& q_s, const CUtensorMap& do_s,
                       const CUtensorMap& k_s, const CUtensorMap& v_s, const PackedAttn& p, const BwdArgs& a,
                       cudaStream_t st, int* launches) {
    const long long warps = (static_cast<long long>(p.T) + kPrepareTokens - 1) / kPrepareTokens * p.nh;
    const unsigned blocks = static_cast<unsigned>((warps + kPrepareThreads / 32 - 1) / (kPrepareThreads / 32));
    cudaError_t e = launch_dependent(packed_prepare_kernel<D>, dim3(blocks + 1), dim3(kPrepareThreads), 0, st, p.dO,
                                     p.O_in, static_cast<long long>(p.T), p.nh, p.delta, p.cu_seqlens, p.nb, p.entries,
                                     p.plan, p.ranks, p.status);
    if (e != cudaSuccess) return e;
    ++*launches;
    const long long most = packed_attn_entries(p.nb, p.T, 128);
    auto grid = [&](long long heads) {
        return dim3(static_cast<unsigned>(most * heads < p.sms ? most * heads : p.sms));
    };
    constexpr int smem = BwdCfg<D>::SMEM;
    auto kq = packed_dq_kernel<D>;
    auto kk = packed_dkdv_kernel<D>;
    if ((e = allow_shared<packed_dq_kernel<D>>(smem)) != cudaSuccess ||
        (e = allow_shared<packed_dkdv_kernel<D>>(smem)) != cudaSuccess ||
        (e = launch_dependent(kq, grid(p.nh), dim3(kDqThreads), smem, st, q128, do128, k_s, v_s, a)) != cudaSuccess)
        return e;
    ++*launches;
    if ((e = launch_dependent(kk, grid(static_cast<long long>(p.nkv) * a.split), dim3(kDkvThreads), smem, st, k128, v128,
                              q_s, do_s, a)) != cudaSuccess)
        return e;
    ++*launches;
    if (a.split > 1) {
        const long long pieces = static_cast<long long>(p.T) * p.nkv * 2 * (D / 8);
        e = launch_dependent(packed_parts_kernel, dim3(static_cast<unsigned>((pieces + 255) / 256)), dim3(256), 0, st, a,
                             D, p.cu_seqlens, p.nb);
        if (e == cudaSuccess) ++*launches;
    }
    return e;
}

}  // namespace

// Parts that a group's heads are dealt to in the dK/dV kernel: one where key tiles and
// key/value heads make an item and a half for each SM, else the fewest that do.  Whole
// groups of 16 heads of 128 on one key/value head took 250 us (8 x 1024 tokens) and
// 1688 us (one sequence of 8192), in parts 144 and 585; two parts where the items were
// 256 cost 15 % at 8 x 1024 tokens (their sums go through memory) and gained 5 % at 8192.
// Parts of one size where less than twice as many give that, and their sums stay in
// bounds: split T nkv <= kPartRows, 75 MB at d = 160, which the fewest parts always
// keep ((items + kPartItems - 1) / items parts of 128 items rows, items < kPartItems).
constexpr long long kPartItems = 3 * 152 / 2, kPartRows = 2 * kPartItems * 128;

int packed_attn_split(int nb, int T, int nh, int nkv) {
    const int group = nh / nkv;
    const long long items = ((static_cast<long long>(T) + 127) / 128 + nb / 2) * nkv;  // half a tile each lost to ends
    if (items >= kPartItems || items == 0) return 1;
    const int fewest = static_cast<int>((kPartItems + items - 1) / items);
    if (fewest >= group) return group;
    for (int s = fewest; s < 2 * fewest && s <= group; ++s)
        if (group % s == 0 && 1LL * s * T * nkv <= kPartRows) return s;
    return fewest;
}

int packed_attn_parts_tokens(int nh, int nkv) {
    return nh == nkv ? 0 : static_cast<int>((kPartItems - 1) / nkv * 128);
}

long long packed_attn_parts_rows(int T, int nh) {
    return 1LL * T * nh < kPartRows ? 1LL * T * nh : kPartRows;
}

int packed_attn_stream_rows(int d) { return d <= 128 ? 128 : 64; }

cudaError_t launch_packed_backward(const CUtensorMap& q128, const CUtensorMap& do128, const CUtensorMap& k128,
                                   const CUtensorMap& v128, const CUtensorMap& q_s, const CUtensorMap& do_s,
                                   const CUtensorMap& k_s, const CUtensorMap& v_s, int d, const PackedAttn& p,
                                   cudaStream_t st, int* launches) {
    BwdArgs a{};
    a.entries = p.entries;
    a.plan = p.plan;
    a.nh = p.nh;
    a.nkv = p.nkv;
    a.group = p.nh / p.nkv;
    a.T = p.T;
    a.scale = p.scale;
    a.scale2 = 1.4426950408889634f * p.scale;
    a.lse = p.lse_in;
    a.delta = p.delta;
    a.split = packed_attn_split(p.nb, p.T, p.nh, p.nkv);
    a.part_heads = a.group / a.split;
    a.part_more = a.group % a.split;
    a.parts = p.parts;
    a.dQ = p.dQ;
    a.dK = p.dK;
    a.dV = p.dV;
    a.ldq = p.ldq;
    a.ldk = p.ldk;
    a.ldv = p.ldv;
    a.status = p.status;
    switch (d) {
        case 64: return launch_bwd<64>(q128, do128, k128, v128, q_s, do_s, k_s, v_s, p, a, st, launches);
        case 96: return launch_bwd<96>(q128, do128, k128, v128, q_s, do_s, k_s, v_s, p, a, st, launches);
        case 128: return launch_bwd<128>(q128, do128, k128, v128, q_s, do_s, k_s, v_s, p, a, st, launches);
        default: return launch_bwd<160>(q128, do128, k128, v128, q_s, do_s, k_s, v_s, p, a, st, launches);
    }
}

}  // namespace tpmlp
