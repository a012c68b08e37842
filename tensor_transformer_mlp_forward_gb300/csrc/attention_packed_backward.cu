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
// P and dS are rounded to bf16 where they become operands of the next product.
//
// Tiles are 128 x 128 (128 x 64 for d = 160, whose accumulators leave tensor memory
// no more): with N = 128 an MMA of two shared-memory operands reads them at exactly
// the rate that shared memory delivers, with N = 64 it waits a third of the time.
// Eight softmax warps own half a row of the tile each.  They work in two steps,
// each of which frees one accumulator early: S is read (and P made) while dP is
// computed, dS is made while the next tile's S is computed, so the tensor cores
// always have a product of this or the next tile to work on.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_packed.cuh"
#include "kernels.h"

namespace tpmlp {
namespace {

constexpr int kBwdThreads = 320;  // 8 softmax warps, producer, MMA

template <int D>
struct BwdCfg {
    static constexpr int NB = (D + 63) / 64;                // 64-column boxes per row
    static constexpr int BS = D <= 128 ? 128 : 64;          // rows of a streamed tile
    static constexpr int HALF = BS / 2;                     // columns of a tile a softmax warp owns
    static constexpr int OWN = NB * 128 * kRowBytes;        // a resident operand: 128 rows
    static constexpr int STREAM = NB * BS * kRowBytes;      // a streamed operand
    static constexpr int STATS = 8 * 2 * HALF * 4;          // lse and delta of each warp's columns
    static constexpr int BARS = 512;
    static constexpr int FIXED = 2 * OWN + STATS + BARS;
    static constexpr int FIT = (226 * 1024 - FIXED) / (2 * STREAM);
    static constexpr int STAGES = FIT > 4 ? 4 : FIT;
    static constexpr int SMEM = 1024 + FIXED + STAGES * 2 * STREAM;
    static_assert(STAGES >= 2, "two stages at least");
    // Tensor memory.  Tiles: S (or S^T) at 0, dP (or dP^T) at BS.  The packed
    // P or dS of softmax half w overlays the first columns of that half's fp32
    // columns, at HALF w.  Accumulators of N >= 128 start on multiples of 128,
    // with the 32-column tails of d = 160 at 384 and 416 (dK/dV) or 256 and 288 (dQ).
    static constexpr uint32_t kS = 0, kP = BS;
    static constexpr uint32_t acc(int x) { return D <= 128 ? 256u + 128u * x : 128u + 128u * x; }
    static constexpr uint32_t acc_tail(int x) { return D <= 128 ? acc(x) + (D / 64) * 64 : 384u + 32u * x; }
    static constexpr uint32_t dq(int x) { return D <= 128 ? 256u + 128u * x : 128u + 256u * x; }
    static constexpr uint32_t dq_tail(int x) { return D <= 128 ? dq(x) + (D / 64) * 64 : 256u + 32u * x; }
};

struct BwdArgs {
    const int4* entries;
    unsigned* plan;
    int nh, nkv, group;
    long long T;
    float scale, scale2;
    const float* lse;    // [nh, T]
    const float* delta;  // [nh, T]
    __nv_bfloat16 *dQ, *dK, *dV;
    long long ldq, ldk, ldv;
    int* status;
};

// D (+)= A B^T with A the packed bf16 halves of a tile in tensor memory (half w at
// a_tmem + HALF w, 8 columns a k-step) and B MN-major along d in shared memory: N in
// whole 64-wide swizzle atoms, then a 32-wide tail.
template <int D>
__device__ __forceinline__ void mma_halves(uint32_t acc, uint32_t tail, uint32_t a_tmem, uint64_t b_desc,
                                           bool accumulate) {
    using C = BwdCfg<D>;
    constexpr int N1 = (D / 64) * 64, N2 = D - N1, STEPS = C::BS / 16;
    constexpr uint32_t id1 = idesc_bf16_f32(128, N1, false, true);
    constexpr uint32_t id2 = idesc_bf16_f32(128, N2 > 0 ? N2 : 32, false, true);
#pragma unroll
    for (int kk = 0; kk < STEPS; ++kk) {
        const uint32_t on = (accumulate || kk > 0) ? 1u : 0u;
        const uint32_t at = a_tmem + (kk / (STEPS / 2)) * C::HALF + (kk % (STEPS / 2)) * 8;
        const uint64_t bd = desc_add(b_desc, mnmajor_step(kk));
        tc_mma_f16_ts(acc, at, bd, id1, on);
        if constexpr (N2 > 0) tc_mma_f16_ts(tail, at, desc_add(bd, (N1 / 64) * C::BS * kRowBytes), id2, on);
    }
}

// D = A B^T over the head dim, A 128 rows and B BS rows, both K-major.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc) {
    using C = BwdCfg<D>;
    constexpr uint32_t id = idesc_bf16_f32(128, C::BS, false, false);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        tc_mma_f16(d_tmem, desc_add(a_desc, kmajor_step<128>(kk)), desc_add(b_desc, kmajor_step<C::BS>(kk)), id,
                   kk > 0 ? 1u : 0u);
}

// HALF consecutive 32-bit columns of this thread's lane.
template <int HALF>
__device__ __forceinline__ void tmem_ld_half(uint32_t addr, uint32_t (&v)[HALF / 32][32]) {
#pragma unroll
    for (int c = 0; c < HALF / 32; ++c) tmem_ld32(addr + 32 * c, v[c]);
    tmem_wait_ld();
}

// Reads chunks [c0, c1) of 32 accumulator columns of this thread's row, scales and
// rounds them, and stores them at dst (a row of D values) when `store`.
template <int D>
__device__ __forceinline__ void read_out(uint32_t acc, uint32_t tail, int c0, int c1, float f, bool store,
                                         __nv_bfloat16* row) {
    uint4* dst = reinterpret_cast<uint4*>(row);
    for (int c = c0; c < c1; ++c) {
        uint32_t v[32];
        // tcgen05.ld is warp-collective: every lane loads
        tmem_ld32(c < (D / 64) * 2 ? acc + 32 * c : tail + 32 * (c - (D / 64) * 2), v);
        tmem_wait_ld();
        if (store) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dst[c * 4 + i] = make_uint4(pack_scaled(v[8 * i], v[8 * i + 1], f), pack_scaled(v[8 * i + 2], v[8 * i + 3], f),
                                            pack_scaled(v[8 * i + 4], v[8 * i + 5], f),
                                            pack_scaled(v[8 * i + 6], v[8 * i + 7], f));
        }
    }
}

// delta = rowsum(dO O) of every token and head; the last CTA makes the plan.
template <int D>
__global__ void __launch_bounds__(kDeltaThreads)
    packed_prepare_kernel(const __nv_bfloat16* dO, const __nv_bfloat16* O, long long T, int nh, float* delta,
                          const int* cu, int nb, int4* entries, unsigned* plan, int* ranks, int* status) {
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0)
        plan_block(cu, nb, static_cast<int>(T), 128, entries, plan, ranks, status);
    else
        attn_delta_block<D>(dO, O, T, nh, delta, blockIdx.x - 1);
}

// ------------------------------------------------------------- dQ

template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1)
    packed_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,  // 128 rows
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,   // BS rows
                     const BwdArgs a) {
    pdl_launch_dependents();
    using C = BwdCfg<D>;
    constexpr int S = C::STAGES, BS = C::BS, HALF = C::HALF;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t* sQ = smem;
    uint8_t* sdO = sQ + C::OWN;
    uint8_t* ring = sdO + C::OWN;
    uint64_t* bars = reinterpret_cast<uint64_t*>(ring + S * 2 * C::STREAM + C::STATS);
    uint64_t* q_full = bars;              // the item's Q has landed
    uint64_t* q_empty = bars + 1;         // its last S has read it
    uint64_t* do_full = bars + 2;         // the same for dO and dP
    uint64_t* do_empty = bars + 3;
    uint64_t* s_full = bars + 4;          // S is complete
    uint64_t* s_read = bars + 5;          // the softmax warps have read it
    uint64_t* dp_full = bars + 6;         // dP is complete
    uint64_t* ds_full = bars + 7;         // dS is in its place
    uint64_t* dq_done = bars + 8;         // [2] the item's dQ is complete
    uint64_t* dq_free = bars + 10;        // [2] the softmax warps have read it out
    uint64_t* item_full = bars + 12;      // [2]
    uint64_t* item_empty = bars + 14;     // [2]
    uint64_t* drain = bars + 16;
    uint64_t* kv_full = bars + 17;        // [S]
    uint64_t* kv_empty = kv_full + S;     // [S]
    int* items = reinterpret_cast<int*>(bars + 17 + 2 * 4);  // [2] x {first row, length, tile, head}
    uint32_t* misc = reinterpret_cast<uint32_t*>(items + 8);
    volatile uint32_t* abort_flag = misc + 1;
    static_assert((17 + 8) * 8 + 8 * 4 + 8 <= C::BARS, "barrier space");

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
        mbar_init(dp_full, 1);
        mbar_init(ds_full, 8);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&dq_done[b], 1);
            mbar_init(&dq_free[b], 8);
            mbar_init(&item_full[b], 1);
            mbar_init(&item_empty[b], 9);  // the MMA thread and the 8 softmax warps
        }
        for (int i = 0; i < S; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        mbar_init(drain, 1);
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

    if (warp == 8) {
        // ------------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_do);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            const unsigned total = a.plan[kPlanCount] * static_cast<unsigned>(a.nh);
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_phase = 0;
            int q_loads = 0, do_loads = 0;
            bool ok = true;
            for (int k = 0;; ++k) {
                const int slot = k & 1;
                if (k >= 2 && !wait_bounded(&item_empty[slot], static_cast<uint32_t>((k - 2) >> 1) & 1u, abort_flag,
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
                if (k >= 1 && !wait_bounded(q_empty, before, abort_flag, a.status, 0x512)) break;
                mbar_arrive_expect_tx(q_full, C::OWN);
                for (int b = 0; b < C::NB; ++b)
                    tma_load_3d(&tm_q, smem_u32(q_full), smem_u32(sQ) + b * 128 * kRowBytes, qcol + 64 * b, row, 0);
                ++q_loads;
                for (int j = 0; j < it.n_kv; ++j) {
                    if (!wait_bounded(&kv_empty[stage], phase ^ 1u, abort_flag, a.status, 0x501)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&kv_full[stage], 2 * C::STREAM);
                    const uint32_t dst = smem_u32(ring) + stage * 2 * C::STREAM;
                    for (int b = 0; b < C::NB; ++b) {
                        tma_load_3d(&tm_k, smem_u32(&kv_full[stage]), dst + b * BS * kRowBytes, kcol + 64 * b,
                                    it.row0 + j * BS, 0);
                        tma_load_3d(&tm_v, smem_u32(&kv_full[stage]), dst + C::STREAM + b * BS * kRowBytes,
                                    kcol + 64 * b, it.row0 + j * BS, 0);
                    }
                    issued |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (j == 0) {
                        if (k >= 1 && !wait_bounded(do_empty, before, abort_flag, a.status, 0x513)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(do_full, C::OWN);
                        for (int b = 0; b < C::NB; ++b)
                            tma_load_3d(&tm_do, smem_u32(do_full), smem_u32(sdO) + b * 128 * kRowBytes, qcol + 64 * b,
                                        row, 0);
                        ++do_loads;
                    }
                }
                if (!ok) break;
            }
            // every copy this thread started lands before the CTA may exit
            if (q_loads > 0) wait_drain(q_full, static_cast<uint32_t>(q_loads - 1) & 1u, a.status, 0x502);
            if (do_loads > 0) wait_drain(do_full, static_cast<uint32_t>(do_loads - 1) & 1u, a.status, 0x503);
            for (int i = 0; i < S; ++i)
                if (issued & (1u << i)) wait_drain(&kv_full[i], (issued_phase >> i) & 1u, a.status, 0x504);
        }
        __syncwarp();
    } else if (warp == 9) {
        // ------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint64_t qdesc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
            const uint64_t dodesc = smem_desc_sw128(smem_u32(sdO), 16, 1024);
            int stage = 0, g = 0;  // g: tiles so far
            uint32_t phase = 0;
            bool ok = true;
            // the tile whose dQ product is still to be issued
            int last_stage = 0, last_k = -1;
            bool last_first = false, last_final = false;
            auto issue_dq = [&]() {  // dQ += dS K of tile g - 1
                if (last_k < 0 || !ok) return;
                const int x = last_k & 1;
                if (last_first && last_k >= 2 &&
                    !wait_bounded(&dq_free[x], static_cast<uint32_t>((last_k - 2) >> 1) & 1u, abort_flag, a.status,
                                  0x514)) {
                    ok = false;
                    return;
                }
                if (!wait_bounded(ds_full, static_cast<uint32_t>(g - 1) & 1u, abort_flag, a.status, 0x505)) {
                    ok = false;
                    return;
                }
                tc_fence_after();
                const uint64_t kdesc =
                    smem_desc_sw128(smem_u32(ring) + last_stage * 2 * C::STREAM, BS * kRowBytes, 1024);
                mma_halves<D>(tmem + C::dq(x), tmem + C::dq_tail(x), tmem + C::kP, kdesc, !last_first);
                tc_commit(&kv_empty[last_stage]);
                if (last_final) tc_commit(&dq_done[x]);
                last_k = -1;
            };
            for (int k = 0; ok; ++k) {
                const int slot = k & 1;
                if (!wait_bounded(&item_full[slot], static_cast<uint32_t>(k >> 1) & 1u, abort_flag, a.status, 0x515))
                    break;
                const Item it = decode(slot);
                mbar_arrive(&item_empty[slot]);
                if (it.len == 0) break;
                for (int j = 0; j < it.n_kv && ok; ++j) {
                    // where the next item's Q is still on its way, the last dQ goes first
                    if (j == 0 && !mbar_test(q_full, static_cast<uint32_t>(k) & 1u)) issue_dq();
                    if (!ok) break;
                    if ((j == 0 && !wait_bounded(q_full, static_cast<uint32_t>(k) & 1u, abort_flag, a.status, 0x506)) ||
                        !wait_bounded(&kv_full[stage], phase, abort_flag, a.status, 0x507) ||
                        (g > 0 &&
                         !wait_bounded(s_read, static_cast<uint32_t>(g - 1) & 1u, abort_flag, a.status, 0x508))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t kv = smem_u32(ring) + stage * 2 * C::STREAM;
                    mma_scores<D>(tmem + C::kS, qdesc, smem_desc_sw128(kv, 16, 1024));
                    tc_commit(s_full);
                    if (j == it.n_kv - 1) tc_commit(q_empty);
                    issue_dq();  // reads dS, which lies over the last dP
                    if (!ok) break;
                    if (j == 0 &&
                        !wait_bounded(do_full, static_cast<uint32_t>(k) & 1u, abort_flag, a.status, 0x509)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mma_scores<D>(tmem + C::kP, dodesc, smem_desc_sw128(kv + C::STREAM, 16, 1024));
                    tc_commit(dp_full);
                    if (j == it.n_kv - 1) tc_commit(do_empty);
                    last_stage = stage;
                    last_k = k;
                    last_first = j == 0;
                    last_final = j == it.n_kv - 1;
                    ++g;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            issue_dq();
            tc_commit(drain);
            wait_drain(drain, 0, a.status, 0x50A);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------- softmax warps
        const int w = warp >> 2;            // which half of a tile's columns
        const int r = threadIdx.x & 127;    // query row = TMEM lane
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        constexpr int CH = D / 32, MID = (CH + 1) / 2;  // dQ chunks of half 0: [0, MID)
        bool ok = true;
        int g = 0, stage = 0;
        struct Pending {
            int k, head;
            bool q_ok;
            long long tok;
        };
        Pending pend{-1, 0, false, 0};
        auto readout = [&]() -> bool {
            const int x = pend.k & 1;
            if (!warp_wait_bounded(&dq_done[x], static_cast<uint32_t>(pend.k >> 1) & 1u, abort_flag, a.status, 0x50B))
                return false;
            tc_fence_after();
            read_out<D>(lane_addr + C::dq(x), lane_addr + C::dq_tail(x), w ? MID : 0, w ? CH : MID, a.scale, pend.q_ok,
                        a.dQ + pend.tok * a.ldq + pend.head * D);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&dq_free[x]);
            pend.k = -1;
            return true;
        };
        for (int k = 0; ok; ++k) {
            const int slot = k & 1;
            if (!warp_wait_bounded(&item_full[slot], static_cast<uint32_t>(k >> 1) & 1u, abort_flag, a.status, 0x516))
                break;
            const Item it = decode(slot);
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[slot]);
            if (it.len == 0) break;
            const int q = it.q0 + r;
            const bool q_ok = q < it.len;
            const long long tok = static_cast<long long>(it.row0) + q;
            const float lse = q_ok ? __ldg(a.lse + it.head * a.T + tok) : 0.0f;
            const float dlt = q_ok ? __ldg(a.delta + it.head * a.T + tok) : 0.0f;
            for (int j = 0; j < it.n_kv; ++j, ++g) {
                const uint32_t parity = static_cast<uint32_t>(g) & 1u;
                const int key0 = j * BS + w * HALF;  // first key of this half
                const bool masked = key0 + HALF - 1 > it.q0 + (warp & 3) * 32;
                if (!warp_wait_bounded(s_full, parity, abort_flag, a.status, 0x50C)) {
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
                const uint64_t scale2 = f32x2(a.scale2, a.scale2), neg_lse = f32x2(-lse, -lse);
#pragma unroll
                for (int c = 0; c < HALF / 32; ++c)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x0, x1;
                        f32x2_split(fma_f32x2(f32x2(__uint_as_float(v[c][2 * i]), __uint_as_float(v[c][2 * i + 1])),
                                              scale2, neg_lse), x0, x1);
                        p[c][2 * i] = ex2(x0);
                        p[c][2 * i + 1] = ex2(x1);
                    }
                if (!warp_wait_bounded(dp_full, parity, abort_flag, a.status, 0x50D)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                tmem_ld_half<HALF>(lane_addr + C::kP + w * HALF, v);
                const uint64_t neg_dlt = f32x2(-dlt, -dlt);
#pragma unroll
                for (int c = 0; c < HALF / 32; ++c) {
                    uint32_t dd[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float d0, d1;
                        f32x2_split(mul_f32x2(f32x2(p[c][2 * i], p[c][2 * i + 1]),
                                              add_f32x2(f32x2(__uint_as_float(v[c][2 * i]),
                                                              __uint_as_float(v[c][2 * i + 1])), neg_dlt)), d0, d1);
                        // an exact zero whatever the masked scores and values hold
                        if (masked) {
                            if (key0 + 32 * c + 2 * i > q) d0 = 0.0f;
                            if (key0 + 32 * c + 2 * i + 1 > q) d1 = 0.0f;
                        }
                        dd[i] = pack_bf16x2(d0, d1);
                    }
                    tmem_st16(lane_addr + C::kP + w * HALF + 16 * c, dd);
                }
                tmem_wait_st();
                tc_fence_before();
                // K rows behind the sequence's end (S, their first use, is done)
                if ((j + 1) * BS > it.len)
                    zero_rows<C::NB>(smem_u32(ring) + stage * 2 * C::STREAM, BS, it.len - j * BS, threadIdx.x, 256);
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full);
                if (++stage == S) stage = 0;
                // the last item's dQ, once this item's first tiles keep the tensor cores busy
                if (pend.k >= 0 && j == (it.n_kv > 1 ? 1 : 0) && !readout()) {
                    ok = false;
                    break;
                }
            }
            if (!ok) break;
            pend = Pending{k, it.head, q_ok, tok};
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
__global__ void __launch_bounds__(kBwdThreads, 1)
    packed_dkdv_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,   // 128 rows
                       const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,  // BS rows
                       const BwdArgs a) {
    pdl_launch_dependents();
    using C = BwdCfg<D>;
    constexpr int S = C::STAGES, BS = C::BS, HALF = C::HALF;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t* sK = smem;
    uint8_t* sV = sK + C::OWN;
    uint8_t* ring = sV + C::OWN;
    float* stats = reinterpret_cast<float*>(ring + S * 2 * C::STREAM);  // [warp][lse, delta][HALF], negated
    uint64_t* bars = reinterpret_cast<uint64_t*>(ring + S * 2 * C::STREAM + C::STATS);
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
    uint64_t* q_full = bars + 15;         // [S]
    uint64_t* q_empty = q_full + S;       // [S]
    int* items = reinterpret_cast<int*>(bars + 15 + 2 * 4);  // [2] x {first row, length, key tile, head}
    uint32_t* misc = reinterpret_cast<uint32_t*>(items + 8);
    volatile uint32_t* abort_flag = misc + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    struct Item {
        int row0, len, k0, kv_head, i0, nq, tiles;
    };
    auto decode = [&](int slot) {
        const volatile int* p = items + 4 * slot;
        Item it;
        it.row0 = p[0];
        it.len = p[1];
        it.k0 = p[2] * 128;
        it.kv_head = p[3];
        it.i0 = it.k0 / BS;                         // first query tile that sees the keys
        it.nq = (it.len + BS - 1) / BS - it.i0;     // query tiles of each head
        it.tiles = it.nq * a.group;
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
        mbar_init(grad_done, 1);
        mbar_init(grad_free, 8);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&item_full[b], 1);
            mbar_init(&item_empty[b], 9);  // the MMA thread and the 8 softmax warps
        }
        for (int i = 0; i < S; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        mbar_init(drain, 1);
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

    if (warp == 8) {
        // ------------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_do);
            const unsigned total = a.plan[kPlanCount] * static_cast<unsigned>(a.nkv);
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_phase = 0;
            int k_loads = 0, v_loads = 0;
            bool ok = true;
            for (int k = 0;; ++k) {
                const int slot = k & 1;
                if (k >= 2 && !wait_bounded(&item_empty[slot], static_cast<uint32_t>((k - 2) >> 1) & 1u, abort_flag,
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
                    const int4 e = a.entries[item / a.nkv];
                    items[4 * slot] = e.x;
                    items[4 * slot + 1] = e.y;
                    items[4 * slot + 2] = e.w - 1 - e.z;  // the highest rank is the first key tile
                    items[4 * slot + 3] = static_cast<int>(item % a.nkv);
                }
                mbar_arrive(&item_full[slot]);
                const Item it = decode(slot);
                const int kcol = it.kv_head * D, row = it.row0 + it.k0;
                const uint32_t before = static_cast<uint32_t>(k - 1) & 1u;
                if (k >= 1 && !wait_bounded(k_empty, before, abort_flag, a.status, 0x612)) break;
                mbar_arrive_expect_tx(k_full, C::OWN);
                for (int b = 0; b < C::NB; ++b)
                    tma_load_3d(&tm_k, smem_u32(k_full), smem_u32(sK) + b * 128 * kRowBytes, kcol + 64 * b, row, 0);
                ++k_loads;
                int head = it.kv_head * a.group, i = 0;
                for (int n = 0; n < it.tiles; ++n) {
                    if (!wait_bounded(&q_empty[stage], phase ^ 1u, abort_flag, a.status, 0x601)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&q_full[stage], 2 * C::STREAM);
                    const uint32_t dst = smem_u32(ring) + stage * 2 * C::STREAM;
                    const int qrow = it.row0 + (it.i0 + i) * BS;
                    for (int b = 0; b < C::NB; ++b) {
                        tma_load_3d(&tm_q, smem_u32(&q_full[stage]), dst + b * BS * kRowBytes, head * D + 64 * b, qrow,
                                    0);
                        tma_load_3d(&tm_do, smem_u32(&q_full[stage]), dst + C::STREAM + b * BS * kRowBytes,
                                    head * D + 64 * b, qrow, 0);
                    }
                    issued |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++i == it.nq) {
                        i = 0;
                        ++head;
                    }
                    if (n == 0) {
                        if (k >= 1 && !wait_bounded(v_empty, before, abort_flag, a.status, 0x613)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(v_full, C::OWN);
                        for (int b = 0; b < C::NB; ++b)
                            tma_load_3d(&tm_v, smem_u32(v_full), smem_u32(sV) + b * 128 * kRowBytes, kcol + 64 * b, row,
                                        0);
                        ++v_loads;
                    }
                }
                if (!ok) break;
            }
            // every copy this thread started lands before the CTA may exit
            if (k_loads > 0) wait_drain(k_full, static_cast<uint32_t>(k_loads - 1) & 1u, a.status, 0x602);
            if (v_loads > 0) wait_drain(v_full, static_cast<uint32_t>(v_loads - 1) & 1u, a.status, 0x603);
            for (int i = 0; i < S; ++i)
                if (issued & (1u << i)) wait_drain(&q_full[i], (issued_phase >> i) & 1u, a.status, 0x604);
        }
        __syncwarp();
    } else if (warp == 9) {
        // ------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint64_t kdesc = smem_desc_sw128(smem_u32(sK), 16, 1024);
            const uint64_t vdesc = smem_desc_sw128(smem_u32(sV), 16, 1024);
            int stage = 0, g = 0;  // g: tiles so far
            uint32_t phase = 0;
            bool ok = true;
            // the tile whose dV and dK products are still to be issued
            int last_stage = 0, last_k = -1;
            bool last_first = false, last_final = false, dv_issued = false;
            auto issue_dv = [&]() {  // dV += P^T dO of tile g - 1
                if (last_k < 0 || dv_issued || !ok) return;
                // the first products of an item overwrite the last item's gradients
                if ((last_first && last_k >= 1 &&
                     !wait_bounded(grad_free, static_cast<uint32_t>(last_k - 1) & 1u, abort_flag, a.status, 0x614)) ||
                    !wait_bounded(p_full, static_cast<uint32_t>(g - 1) & 1u, abort_flag, a.status, 0x605)) {
                    ok = false;
                    return;
                }
                tc_fence_after();
                mma_halves<D>(tmem + C::acc(0), tmem + C::acc_tail(0), tmem + C::kS,
                              smem_desc_sw128(smem_u32(ring) + last_stage * 2 * C::STREAM + C::STREAM, BS * kRowBytes,
                                              1024), !last_first);
                dv_issued = true;
            };
            auto issue_dk = [&]() {  // dK += dS^T Q of tile g - 1
                if (last_k < 0 || !ok) return;
                if (!wait_bounded(ds_full, static_cast<uint32_t>(g - 1) & 1u, abort_flag, a.status, 0x606)) {
                    ok = false;
                    return;
                }
                tc_fence_after();
                mma_halves<D>(tmem + C::acc(1), tmem + C::acc_tail(1), tmem + C::kP,
                              smem_desc_sw128(smem_u32(ring) + last_stage * 2 * C::STREAM, BS * kRowBytes, 1024),
                              !last_first);
                tc_commit(&q_empty[last_stage]);
                if (last_final) tc_commit(grad_done);
                last_k = -1;
            };
            for (int k = 0; ok; ++k) {
                const int slot = k & 1;
                if (!wait_bounded(&item_full[slot], static_cast<uint32_t>(k >> 1) & 1u, abort_flag, a.status, 0x615))
                    break;
                const Item it = decode(slot);
                mbar_arrive(&item_empty[slot]);
                if (it.len == 0) break;
                for (int n = 0; n < it.tiles && ok; ++n) {
                    issue_dv();  // reads P^T, which lies over the last S^T
                    // where the next item's K is still on its way, the last dK goes first
                    if (n == 0 && ok && !mbar_test(k_full, static_cast<uint32_t>(k) & 1u)) issue_dk();
                    if (!ok) break;
                    if ((n == 0 && !wait_bounded(k_full, static_cast<uint32_t>(k) & 1u, abort_flag, a.status, 0x607)) ||
                        !wait_bounded(&q_full[stage], phase, abort_flag, a.status, 0x608)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t qd = smem_u32(ring) + stage * 2 * C::STREAM;
                    mma_scores<D>(tmem + C::kS, kdesc, smem_desc_sw128(qd, 16, 1024));
                    tc_commit(s_full);
                    if (n == it.tiles - 1) tc_commit(k_empty);
                    issue_dk();  // reads dS^T, which lies over the last dP^T
                    if (!ok) break;
                    if (n == 0 && !wait_bounded(v_full, static_cast<uint32_t>(k) & 1u, abort_flag, a.status, 0x609)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mma_scores<D>(tmem + C::kP, vdesc, smem_desc_sw128(qd + C::STREAM, 16, 1024));
                    tc_commit(dp_full);
                    if (n == it.tiles - 1) tc_commit(v_empty);
                    last_stage = stage;
                    last_k = k;
                    last_first = n == 0;
                    last_final = n == it.tiles - 1;
                    dv_issued = false;
                    ++g;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            issue_dv();
            issue_dk();
            tc_commit(drain);
            wait_drain(drain, 0, a.status, 0x60A);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------- softmax warps
        const int w = warp >> 2;            // which half of a tile's columns (queries)
        const int r = threadIdx.x & 127;    // key row = TMEM lane
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        float* neg_lse = stats + warp * 2 * HALF;
        float* neg_dlt = neg_lse + HALF;
        bool ok = true;
        int g = 0, stage = 0;
        for (int k = 0; ok; ++k) {
            const int slot = k & 1;
            if (!warp_wait_bounded(&item_full[slot], static_cast<uint32_t>(k >> 1) & 1u, abort_flag, a.status, 0x616))
                break;
            const Item it = decode(slot);
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[slot]);
            if (it.len == 0) break;
            const int key = it.k0 + r;
            // lse and delta of the tile's queries, loaded a tile ahead
            float lse_n[HALF / 32], dlt_n[HALF / 32];
            auto fetch = [&](int head, int i) {
                const long long at = head * a.T + it.row0;
#pragma unroll
                for (int c = 0; c < HALF / 32; ++c) {
                    const int qq = (it.i0 + i) * BS + w * HALF + 32 * c + lane;
                    const bool in = qq < it.len;
                    lse_n[c] = in ? -__ldg(a.lse + at + qq) : 0.0f;
                    dlt_n[c] = in ? -__ldg(a.delta + at + qq) : 0.0f;
                }
            };
            int head = it.kv_head * a.group, i = 0;
            fetch(head, 0);
            for (int n = 0; n < it.tiles; ++n, ++g) {
                const uint32_t parity = static_cast<uint32_t>(g) & 1u;
                const int q0 = (it.i0 + i) * BS + w * HALF;  // first query of this half
                const bool masked = q0 < it.k0 + (warp & 3) * 32 + 31 || q0 + HALF > it.len;
                const bool tail = (it.i0 + i + 1) * BS > it.len;
                const int valid = it.len - (it.i0 + i) * BS;  // queries of the tile inside the sequence
                __syncwarp();  // the last tile's values have been read
#pragma unroll
                for (int c = 0; c < HALF / 32; ++c) {
                    neg_lse[32 * c + lane] = lse_n[c];
                    neg_dlt[32 * c + lane] = dlt_n[c];
                }
                __syncwarp();
                if (++i == it.nq) {
                    i = 0;
                    ++head;
                }
                if (n + 1 < it.tiles) fetch(head, i);
                if (!warp_wait_bounded(s_full, parity, abort_flag, a.status, 0x60B)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t v[HALF / 32][32];
                tmem_ld_half<HALF>(lane_addr + C::kS + w * HALF, v);
                float p[HALF / 32][32];
                const uint64_t scale2 = f32x2(a.scale2, a.scale2);
#pragma unroll
                for (int c = 0; c < HALF / 32; ++c) {
                    uint32_t pp[16];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const float4 l4 = *reinterpret_cast<const float4*>(neg_lse + 32 * c + 4 * u);
                        float x[4];
                        f32x2_split(fma_f32x2(f32x2(__uint_as_float(v[c][4 * u]), __uint_as_float(v[c][4 * u + 1])),
                                              scale2, f32x2(l4.x, l4.y)), x[0], x[1]);
                        f32x2_split(fma_f32x2(f32x2(__uint_as_float(v[c][4 * u + 2]), __uint_as_float(v[c][4 * u + 3])),
                                              scale2, f32x2(l4.z, l4.w)), x[2], x[3]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float pe = ex2(x[e]);
                            // keys after the query, and queries behind the sequence's end
                            if (masked) {
                                const int qq = q0 + 32 * c + 4 * u + e;
                                if (qq < key || qq >= it.len) pe = 0.0f;
                            }
                            p[c][4 * u + e] = pe;
                        }
                        pp[2 * u] = pack_bf16x2(p[c][4 * u], p[c][4 * u + 1]);
                        pp[2 * u + 1] = pack_bf16x2(p[c][4 * u + 2], p[c][4 * u + 3]);
                    }
                    tmem_st16(lane_addr + C::kS + w * HALF + 16 * c, pp);
                }
                tmem_wait_st();
                tc_fence_before();
                const uint32_t qd = smem_u32(ring) + stage * 2 * C::STREAM;
                // dO rows behind the end: S^T is there, so Q and dO have landed
                if (tail) zero_rows<C::NB>(qd + C::STREAM, BS, valid, threadIdx.x, 256);
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
                if (!warp_wait_bounded(dp_full, parity, abort_flag, a.status, 0x60C)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                tmem_ld_half<HALF>(lane_addr + C::kP + w * HALF, v);
#pragma unroll
                for (int c = 0; c < HALF / 32; ++c) {
                    uint32_t dd[16];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const float4 d4 = *reinterpret_cast<const float4*>(neg_dlt + 32 * c + 4 * u);
                        float x[4];
                        f32x2_split(mul_f32x2(f32x2(p[c][4 * u], p[c][4 * u + 1]),
                                              add_f32x2(f32x2(__uint_as_float(v[c][4 * u]),
                                                              __uint_as_float(v[c][4 * u + 1])), f32x2(d4.x, d4.y))),
                                    x[0], x[1]);
                        f32x2_split(mul_f32x2(f32x2(p[c][4 * u + 2], p[c][4 * u + 3]),
                                              add_f32x2(f32x2(__uint_as_float(v[c][4 * u + 2]),
                                                              __uint_as_float(v[c][4 * u + 3])), f32x2(d4.z, d4.w))),
                                    x[2], x[3]);
                        if (masked) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int qq = q0 + 32 * c + 4 * u + e;
                                if (qq < key || qq >= it.len) x[e] = 0.0f;
                            }
                        }
                        dd[2 * u] = pack_bf16x2(x[0], x[1]);
                        dd[2 * u + 1] = pack_bf16x2(x[2], x[3]);
                    }
                    tmem_st16(lane_addr + C::kP + w * HALF + 16 * c, dd);
                }
                tmem_wait_st();
                tc_fence_before();
                if (tail) zero_rows<C::NB>(qd, BS, valid, threadIdx.x, 256);  // Q rows
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full);
                if (++stage == S) stage = 0;
            }
            if (!ok || !warp_wait_bounded(grad_done, static_cast<uint32_t>(k) & 1u, abort_flag, a.status, 0x60D)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // half 0 reads dV out, half 1 dK
            const long long tok = static_cast<long long>(it.row0) + key;
            const bool key_ok = key < it.len;
            if (w == 0)
                read_out<D>(lane_addr + C::acc(0), lane_addr + C::acc_tail(0), 0, D / 32, 1.0f, key_ok,
                            a.dV + tok * a.ldv + it.kv_head * D);
            else
                read_out<D>(lane_addr + C::acc(1), lane_addr + C::acc_tail(1), 0, D / 32, a.scale, key_ok,
                            a.dK + tok * a.ldk + it.kv_head * D);
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
}

template <int D>
cudaError_t launch_bwd(const CUtensorMap& q128, const CUtensorMap& do128, const CUtensorMap& k128,
                       const CUtensorMap& v128, const CUtensorMap& q_s, const CUtensorMap& do_s,
                       const CUtensorMap& k_s, const CUtensorMap& v_s, const PackedAttn& p, const BwdArgs& a,
                       cudaStream_t st, int* launches) {
    const long long segs = static_cast<long long>(p.T) * p.nh;
    const unsigned blocks = static_cast<unsigned>((segs + delta_segs<D>() - 1) / delta_segs<D>());
    cudaError_t e = launch_dependent(packed_prepare_kernel<D>, dim3(blocks + 1), dim3(kDeltaThreads), 0, st, p.dO,
                                     p.O_in, static_cast<long long>(p.T), p.nh, p.delta, p.cu_seqlens, p.nb, p.entries,
                                     p.plan, p.ranks, p.status);
    if (e != cudaSuccess) return e;
    ++*launches;
    const long long most = static_cast<long long>(p.T) / 128 + p.nb;  // entries at most
    auto grid = [&](long long heads) {
        return dim3(static_cast<unsigned>(most * heads < p.sms ? most * heads : p.sms));
    };
    constexpr int smem = BwdCfg<D>::SMEM;
    auto kq = packed_dq_kernel<D>;
    auto kk = packed_dkdv_kernel<D>;
    if ((e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(kk, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
        (e = launch_dependent(kq, grid(p.nh), dim3(kBwdThreads), smem, st, q128, do128, k_s, v_s, a)) != cudaSuccess)
        return e;
    ++*launches;
    e = launch_dependent(kk, grid(p.nkv), dim3(kBwdThreads), smem, st, k128, v128, q_s, do_s, a);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace

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
