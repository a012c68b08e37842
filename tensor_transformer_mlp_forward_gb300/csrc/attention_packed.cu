// attention_packed.cu -- causal softmax attention of a packed batch with grouped
// key/value heads, forward.
//
// Query head j of nh reads key/value head j / (nh / nkv).  Per sequence (rows
// cu_seqlens[i] .. cu_seqlens[i + 1] - 1) and head:
//
//   S = scale Q K^T (keys up to the query) ; P = softmax_rows(S) ; O = P V
//
// in one pass over the keys with a running maximum and sum, in the log2 domain
// (u = scale log2(e) q.k, P = 2^(u - m) / l, lse = m + log2(l)).  S, l and O are
// fp32; P is rounded to bf16 where it becomes an operand of P V, as the tensor cores
// take it beside a bf16 V.  That leaves O 1.2 to 1.35 times as far from 64 bits (in the
// 2-norm) as its own rounding to bf16 alone.
//
// The kernel is that of attention.cu (two 128-query tiles A and B in ping-pong,
// S and O in tensor memory, P written back over S as the A operand of P V) with
// other work: items come from a list of the sequences' tiles, tiles of a sequence
// are read by row coordinates, and A and B are, where the heads of a group come
// in pairs, two heads' tiles of the same queries, so that both share every K/V
// tile, need the same number of them, and a sequence of 128 tokens or fewer keeps
// both busy; else two adjacent tiles of one head.
//
// Long sequences are bound by the tensor cores and the softmax between their products
// (16384 tokens, 16 heads on 2 of 128: 641-690 us, 1590-1710 TFLOP/s), short ones by an
// item's chain of load, S, softmax, P V and store (8 x 1024 tokens, 32 heads on 8 of 128:
// 70.7 us; 37 sequences in 8191 tokens, 20 heads of 64: 48 to 50 us).  For the latter neither a
// deeper ring (50.9 against 49.3 us) nor a second place for O (49.7 against 48.6) helped.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_packed.cuh"
#include "kernels.h"

namespace tpmlp {
namespace {

// 8 softmax warps, the producer's, the MMAs', and one that zeroes V's rows behind the
// sequences' ends as soon as they land (left to the softmax warps, that was a wait for V
// and for stores between the scores and P V: 72.4 us for 8 x 1024 tokens against 70.5).
constexpr int kPackedFwdThreads = 352;

// The Q tiles have two places where they fit (d = 64), so that the next item's are there
// when the last product of this one is done.
template <int D>
struct PackedFwdCfg : FwdCfg<D> {
    using F = FwdCfg<D>;
    static constexpr int QPLACES = 2 * F::FIXED + F::STAGES * F::KVTILE <= 224 * 1024 ? 2 : 1;
    static constexpr int BARS = 384;
    static constexpr int SMEM = 1024 + QPLACES * F::FIXED + F::STAGES * F::KVTILE + BARS;
};

struct FwdArgs {
    const int4* entries;  // the plan's tiles
    unsigned* plan;       // its header words
    int nh, group;        // query heads, query heads per key/value head
    int units;            // items per entry (heads, or pairs of heads)
    int pair_heads;
    long long T;
    float scale2;         // scale * log2(e)
    __nv_bfloat16* O;     // [T, nh, D]
    float* lse;           // [nh, T]
    int* status;
};

__global__ void __launch_bounds__(1024) packed_plan_kernel(const int* cu, int nb, int T, int tile, int4* entries,
                                                           unsigned* head, int* ranks, int* status) {
    pdl_launch_dependents();
    pdl_wait();
    plan_block(cu, nb, T, tile, entries, head, ranks, status);
}

__device__ __forceinline__ void row_max(const uint32_t (&v)[32], float (&mx)[8]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) mx[i & 7] = fmaxf(mx[i & 7], __uint_as_float(v[i]));
}

// p = 2^(scale2 s - m) of 32 scores (masked ones are -inf: 2^-inf = 0), packed bf16, and
// their sums in fp32.
__device__ __forceinline__ void row_weights(const uint32_t (&v)[32], uint64_t scale2, uint64_t neg_m, uint32_t (&pk)[16],
                                            uint64_t (&sum)[4]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float x0, x1;
        f32x2_split(fma_f32x2(f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), scale2, neg_m), x0, x1);
        const float p0 = ex2(x0), p1 = ex2(x1);
        sum[i & 3] = add_f32x2(sum[i & 3], f32x2(p0, p1));
        pk[i] = pack_bf16x2(p0, p1);
    }
}

template <int D>
__global__ void __launch_bounds__(kPackedFwdThreads, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,  // 128-row boxes
                      const __grid_constant__ CUtensorMap tm_k,  // BKV-row boxes
                      const __grid_constant__ CUtensorMap tm_v, const FwdArgs a) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    using C = PackedFwdCfg<D>;
    constexpr int S = C::STAGES;
    constexpr int BKV = C::BKV;
    constexpr int SCH = BKV / 32;  // 32-key chunks of S per key tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    constexpr int QP = C::QPLACES;
    uint8_t* sQ = smem;                   // [QP] x {Q_A, Q_B}
    uint8_t* ring = smem + QP * 2 * C::QTILE;  // K_0, V_0, K_1, V_1, ... of every item in turn
    uint64_t* bars = reinterpret_cast<uint64_t*>(ring + S * C::KVTILE);
    uint64_t* q_full = bars;              // [QP] the item's Q tiles have landed
    uint64_t* q_empty = bars + 2;         // [QP] the item's last S MMAs have read them
    uint64_t* kv_full = bars + 4;
    uint64_t* kv_empty = kv_full + S;
    uint64_t* s_full = kv_empty + S;      // [tile]
    uint64_t* p_full = s_full + 2;        // [tile]
    uint64_t* o_full = p_full + 2;       // [tile]
    uint64_t* o_free = o_full + 2;       // [tile] the softmax warps have read O_x out
    uint64_t* item_full = o_free + 2;     // [2]
    uint64_t* item_empty = item_full + 2; // [2]
    uint64_t* v_clean = item_empty + 2;   // [4] V's rows behind the end are zeros (ends in turn)
    uint64_t* v_issued = v_clean + 4;     // [4] the load of such a V has been started
    uint64_t* drain = v_issued + 4;
    static_assert((4 + 2 * S + 12 + 8 + 1) * 8 + 8 * 4 + 8 <= C::BARS, "barrier space");
    int* items = reinterpret_cast<int*>(drain + 1);  // [2] x {first row, length, tile, head}
    uint32_t* misc = reinterpret_cast<uint32_t*>(items + 8);
    volatile uint32_t* abort_flag = misc + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    struct Item {
        int row0, len, n_kv;
        int q0[2], head[2];
        bool has_b, ends;  // ends: the last key tile reaches behind the sequence's end
        int last[2];  // last key tile each query tile sees
    };
    auto decode = [&](int slot) {
        const volatile int* p = items + 4 * slot;
        Item it;
        it.row0 = p[0];
        it.len = p[1];
        it.head[0] = p[3];
        if (a.pair_heads) {
            it.q0[0] = it.q0[1] = p[2] * 128;
            it.head[1] = it.head[0] + 1;
            it.has_b = true;
        } else {
            it.q0[0] = p[2] * 256;
            it.q0[1] = it.q0[0] + 128;
            it.head[1] = it.head[0];
            it.has_b = it.q0[1] < it.len;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) it.last[x] = (min(it.q0[x] + 128, it.len) - 1) / BKV;
        it.n_kv = it.has_b ? it.last[1] + 1 : it.last[0] + 1;
        it.ends = it.n_kv * BKV > it.len;
        return it;
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < QP; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < S; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 4);  // one arrival per warp of the tile's warpgroup
            mbar_init(&o_full[x], 1);
            mbar_init(&o_free[x], 4);
            mbar_init(&item_full[x], 1);
            mbar_init(&item_empty[x], 10);  // the MMA thread, the 8 softmax warps and V's
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&v_clean[i], 1);
            mbar_init(&v_issued[i], 1);
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
    pdl_wait();  // the plan, and whatever wrote the inputs, is done

    if (warp == 8) {
        // ------------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            const unsigned units = static_cast<unsigned>(a.units);
            const unsigned total = a.plan[kPlanCount] * units;
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_phase = 0;
            int q_loads = 0;
            unsigned ends = 0;
            bool ok = true;
            for (int k = 0;; ++k) {
                const int slot = k & 1;
                if (k >= 2 && !thread_wait(&item_empty[slot], static_cast<uint32_t>((k - 2) >> 1) & 1u,
                                            abort_flag, a.status, 0x411))
                    ok = false;
                unsigned item = total;
                if (ok) item = atomicAdd(&a.plan[kPlanWork0], 1u);
                if (item >= total) {
                    items[4 * slot + 1] = 0;  // no sequence: the end
                    mbar_arrive(&item_full[slot]);
                    break;
                }
                {
                    const int4 e = a.entries[item / units];
                    items[4 * slot] = e.x;
                    items[4 * slot + 1] = e.y;
                    items[4 * slot + 2] = e.z;
                    items[4 * slot + 3] = static_cast<int>(item % units) * (a.pair_heads ? 2 : 1);
                }
                mbar_arrive(&item_full[slot]);
                const Item it = decode(slot);
                const int kcol = it.head[0] / a.group * D;
                // the previous item's S MMAs are done with the Q tiles
                const int qp = k % QP;
                if (k >= QP && !thread_wait(&q_empty[qp], static_cast<uint32_t>(k / QP - 1) & 1u, abort_flag, a.status,
                                            0x412))
                    break;
                mbar_arrive_expect_tx(&q_full[qp], (it.has_b ? 2 : 1) * C::QTILE);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    for (int b = 0; b < C::NB && (x == 0 || it.has_b); ++b)
                        tma_load_3d(&tm_q, smem_u32(&q_full[qp]),
                                    smem_u32(sQ) + (2 * qp + x) * C::QTILE + b * 128 * kRowBytes,
                                    it.head[x] * D + 64 * b, it.row0 + it.q0[x], 0);
                ++q_loads;
                for (int idx = 0; idx < 2 * it.n_kv; ++idx) {  // K_j = 2j, V_j = 2j + 1
                    if (!thread_wait(&kv_empty[stage], phase ^ 1u, abort_flag, a.status, 0x401)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&kv_full[stage], C::KVTILE);
                    const uint32_t dst = smem_u32(ring) + stage * C::KVTILE;
                    for (int b = 0; b < C::NB; ++b)
                        tma_load_3d((idx & 1) ? &tm_v : &tm_k, smem_u32(&kv_full[stage]),
                                    dst + b * BKV * kRowBytes, kcol + 64 * b, it.row0 + (idx >> 1) * BKV, 0);
                    issued |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if (it.ends) mbar_arrive(&v_issued[ends++ % 4]);
            }
            for (int k = q_loads > QP ? q_loads - QP : 0; k < q_loads; ++k)
                wait_drain(&q_full[k % QP], static_cast<uint32_t>(k / QP) & 1u, a.status, 0x402);
            for (int i = 0; i < S; ++i)
                if (issued & (1u << i)) wait_drain(&kv_full[i], (issued_phase >> i) & 1u, a.status, 0x403);
        }
        __syncwarp();
    } else if (warp == 9) {
        // ------------------------------------------------------ MMA issuer
        {
            bool ok = true;
            int rstage = 0;  // ring entries are taken in order, across items
            uint32_t rphase = 0;
            int gx[2] = {0, 0};  // S / P V MMAs of each tile over the items so far
            int cx[2] = {0, 0};  // items each tile has taken part in
            auto next = [&]() {
                if (++rstage == S) {
                    rstage = 0;
                    rphase ^= 1u;
                }
            };
            unsigned ends = 0;  // items so far whose V has rows behind the end
            int s_left = 0;  // S MMAs of the item still to issue
            int qp = 0;      // where the item's Q tiles lie
            auto issue_s = [&](int x, int stage) {  // S_x = Q_x K^T
                warp_mma_scores<D, BKV>(tmem + C::s_col(x), desc_low(smem_u32(sQ) + (2 * qp + x) * C::QTILE, 16),
                                        desc_low(smem_u32(ring) + stage * C::KVTILE, 16));
                warp_commit(&s_full[x]);
                // the item's last S: once done, the Q tiles may be replaced
                if (--s_left == 0) warp_commit(&q_empty[qp]);
            };
            // O_x (+)= P_x V: A = P_x from TMEM (packed over S_x's first columns), B = V
            // (MN-major: d along the rows, keys down the box)
            auto issue_pv = [&](int x, int j, int stage, bool final) {
                warp_mma_values<D, BKV, BKV / 4>(tmem + C::o_col(x), tmem + C::o_tail(x), tmem + C::s_col(x),
                                                 desc_low(smem_u32(ring) + stage * C::KVTILE, BKV * kRowBytes), j > 0);
                if (final) warp_commit(&o_full[x]);
            };
            // P_x of key tile j is there, and (j == 0) O_x of the last item is read out
            auto wait_p = [&](int x, int j) {
                if (j == 0 && cx[x] >= 1)
                    ok = ok && warp_wait(&o_free[x], static_cast<uint32_t>(cx[x] - 1) & 1u, abort_flag, a.status,
                                           0x413 + x);
                ok = ok && warp_wait(&p_full[x], static_cast<uint32_t>(gx[x] + j) & 1u, abort_flag, a.status,
                                       0x405 + x);
                tc_fence_after();
            };
            for (int k = 0; ok; ++k) {
                const int slot = k & 1;
                if (!warp_wait(&item_full[slot], static_cast<uint32_t>(k >> 1) & 1u, abort_flag, a.status, 0x415))
                    break;
                const Item it = decode(slot);
                __syncwarp();
                warp_arrive(&item_empty[slot]);
                if (it.len == 0) break;
                qp = k % QP;
                if (!warp_wait_both(&q_full[qp], static_cast<uint32_t>(k / QP) & 1u, &kv_full[rstage], rphase, abort_flag,
                                      a.status, 0x404))
                    break;
                tc_fence_after();
                s_left = it.last[0] + 1 + (it.has_b ? it.last[1] + 1 : 0);
                // S of both tiles for key tile 0
                issue_s(0, rstage);
                if (it.has_b) issue_s(1, rstage);
                warp_commit(&kv_empty[rstage]);
                next();
                for (int j = 0; j < it.n_kv && ok; ++j) {
                    // V of this key tile and K of the next: by now both have landed as a
                    // rule, and one wait for the two is spent while tile A's softmax runs
                    const int vs = rstage;
                    const uint32_t vp = rphase;
                    next();
                    const bool more = j + 1 < it.n_kv;
                    const int kn = rstage;
                    if (more) {
                        ok = warp_wait_both(&kv_full[vs], vp, &kv_full[kn], rphase, abort_flag, a.status, 0x408);
                        next();
                    } else if (it.ends) {
                        // (warp 10 is at most two items ahead: four barriers tell its ends apart)
                        ok = warp_wait_both(&kv_full[vs], vp, &v_clean[ends % 4], ends / 4 & 1u, abort_flag, a.status,
                                            0x409);
                        ++ends;
                    } else {
                        ok = warp_wait(&kv_full[vs], vp, abort_flag, a.status, 0x409);
                    }
                    if (!ok) break;
                    if (j <= it.last[0]) {
                        wait_p(0, j);
                        if (!ok) break;
                        issue_pv(0, j, vs, j == it.last[0]);
                        if (j + 1 <= it.last[0]) issue_s(0, kn);
                    }
                    if (it.has_b) {
                        wait_p(1, j);
                        if (!ok) break;
                        issue_pv(1, j, vs, j == it.last[1]);
                        warp_commit(&kv_empty[vs]);
                        if (more) issue_s(1, kn);
                    } else {
                        warp_commit(&kv_empty[vs]);
                    }
                    if (more) warp_commit(&kv_empty[kn]);
                }
                gx[0] += it.last[0] + 1;
                cx[0] += 1;
                if (it.has_b) {
                    gx[1] += it.last[1] + 1;
                    cx[1] += 1;
                }
            }
            warp_commit(drain);
            if (lane == 0) wait_drain(drain, 0, a.status, 0x40B);
        }
        __syncwarp();
    } else if (warp == 10) {
        // -------------------- zeroes of V's rows behind the sequences' ends
        unsigned ends = 0, ring_at = 0;  // of the items so far
        for (int k = 0;; ++k) {
            const int slot = k & 1;
            if (!warp_wait(&item_full[slot], static_cast<uint32_t>(k >> 1) & 1u, abort_flag, a.status, 0x417)) break;
            const Item it = decode(slot);
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[slot]);
            if (it.len == 0) break;
            ring_at += 2u * static_cast<unsigned>(it.n_kv);
            if (!it.ends) continue;
            const unsigned v_at = ring_at - 1u;  // the last V
            const int vs = static_cast<int>(v_at % S);
            // its load first: from then on the slot is in V's phase, and stays in it until
            // V is used, for which this warp's word is needed
            if (!warp_wait(&v_issued[ends % 4], ends / 4 & 1u, abort_flag, a.status, 0x418) ||
                !warp_wait(&kv_full[vs], (v_at / S) & 1u, abort_flag, a.status, 0x414))
                break;
            zero_rows<C::NB>(smem_u32(ring) + vs * C::KVTILE, BKV, it.len - (it.n_kv - 1) * BKV, lane, 32);
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_clean[ends % 4]);
            ++ends;
        }
        __syncwarp();
    } else {
        // -------------------------------------------------- softmax warps
        const int x = warp >> 2;               // tile: 0 = A, 1 = B
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_addr = lane_addr + C::s_col(x);
        int gxl = 0;  // this tile's S / P V MMAs over the items so far
        int taken = 0;         // items this tile has taken part in
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int slot = k & 1;
            if (!warp_wait(&item_full[slot], static_cast<uint32_t>(k >> 1) & 1u, abort_flag,
                                   a.status, 0x416))
                break;
            const Item it = decode(slot);
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[slot]);
            if (it.len == 0) break;
            if (x == 1 && !it.has_b) continue;  // no B tile in this item
            const int first_q = (x ? it.q0[1] : it.q0[0]) + (warp & 3) * 32;  // the warp's
            const int q = first_q + lane;
            const int head = x ? it.head[1] : it.head[0];
            const int jl = x ? it.last[1] : it.last[0];
            // (finite: scores that are all -inf so far weigh 2^-inf, not 2^(-inf + inf))
            float m = -3.4e38f, l = 0.0f;
            for (int j = 0; j <= jl; ++j) {
                const int k0 = j * BKV;
                if (!warp_wait(&s_full[x], static_cast<uint32_t>(gxl + j) & 1u, abort_flag,
                                       a.status, 0x40C + x)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t v[SCH][32];
#pragma unroll
                for (int c = 0; c < SCH; ++c) warp_tmem_ld32(s_addr + c * 32, v[c]);
#pragma unroll
                for (int c = 0; c < SCH; ++c) tmem_loaded(v[c]);
                // chunks of 32 keys: the warp's queries see the first `live`, the last of
                // those up to the diagonal if that is in this key tile; the rest holds
                // nothing for any of them
                const int live = ((first_q - k0) >> 5) + 1;
                // eight independent max / sum chains: the row is one thread's
                // work, so its reductions must not be one serial chain
                float mx8[8];
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) mx8[kk] = -INFINITY;
                if (live > SCH) {
#pragma unroll
                    for (int c = 0; c < SCH; ++c) row_max(v[c], mx8);
                } else {
#pragma unroll
                    for (int c = 0; c < SCH; ++c) {
                        if (c == live - 1) {
#pragma unroll
                            for (int i = 1; i < 32; ++i)
                                if (i > lane) v[c][i] = __float_as_uint(-INFINITY);
                        }
                        if (c < live) row_max(v[c], mx8);
                    }
                }
                const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                       fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
                // the reference max only moves when the row max outgrows it by
                // more than 2^8, so the O rescale below is rare.  A row whose
                // keys in this tile are all masked keeps its reference.
                const float m_new = fmaxf(m, mx * a.scale2);
                const bool move = j == 0 || m_new > m + kRescaleLog2;
                const float alpha = move ? ex2(m - m_new) : 1.0f;
                if (move) m = m_new;
                uint64_t rs2[4];
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) rs2[kk] = 0ull;  // (0.0f, 0.0f)
                const uint64_t scale2 = f32x2(a.scale2, a.scale2), neg_m = f32x2(-m, -m);
                // P_x, packed bf16, over the first columns of S_x (already read)
                if (live > SCH) {
#pragma unroll
                    for (int c = 0; c < SCH; ++c) {
                        uint32_t pk[16];
                        row_weights(v[c], scale2, neg_m, pk, rs2);
                        warp_tmem_st16(s_addr + 16 * c, pk);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < SCH; ++c) {
                        uint32_t pk[16];
                        if (c < live) {
                            row_weights(v[c], scale2, neg_m, pk, rs2);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) pk[i] = 0u;
                        }
                        warp_tmem_st16(s_addr + 16 * c, pk);
                    }
                }
                float rsv[8];
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) f32x2_split(rs2[kk], rsv[2 * kk], rsv[2 * kk + 1]);
                const float rs = ((rsv[0] + rsv[1]) + (rsv[2] + rsv[3])) + ((rsv[4] + rsv[5]) + (rsv[6] + rsv[7]));
                l = fmaf(l, alpha, rs);
                // S_x(j) was issued after P_x V of the previous key tile, and the
                // commit that signalled S_x covers every earlier MMA: that P V
                // has finished, so O_x is final and P_x's columns are free
                if (j >= 1) {
                    if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            warp_tmem_ld32(lane_addr + C::o_chunk(x, c), o);
                            tmem_loaded(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            warp_tmem_st32(lane_addr + C::o_chunk(x, c), o);
                        }
                        __syncwarp();
                        tmem_wait_st();
                    }
                }
                __syncwarp();
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x]);
            }
            if (!ok) break;
            // while the last P V runs
            const float inv = 1.0f / l;
            if (q < it.len) a.lse[head * a.T + it.row0 + q] = m + lg2(l);
            const RowsOut out(a.O, static_cast<long long>(a.nh) * D, static_cast<long long>(it.row0) + first_q, head * D,
                              it.len - first_q);
            if (!warp_wait(&o_full[x], static_cast<uint32_t>(taken) & 1u, abort_flag, a.status, 0x410 + x)) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) read_out(out, c, lane_addr + C::o_chunk(x, c), inv);
            // O_x is in registers or on its way to memory: the MMA may reuse it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[x]);
            gxl += jl + 1;
            ++taken;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// CTAs of a persistent kernel: one per SM at most.
unsigned persistent_grid(long long items, int sms) {
    return static_cast<unsigned>(items < sms ? items : sms);
}

template <int D>
cudaError_t launch_fwd(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const FwdArgs& a,
                       unsigned grid, cudaStream_t st) {
    const cudaError_t e = allow_shared<packed_fwd_kernel<D>>(PackedFwdCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_dependent(packed_fwd_kernel<D>, dim3(grid), dim3(kPackedFwdThreads), PackedFwdCfg<D>::SMEM, st, q, k, v, a);
}

}  // namespace

int packed_attn_kv_rows(int d) { return d <= 128 ? 128 : 64; }

cudaError_t launch_packed_forward(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, int d,
                                  const PackedAttn& p, cudaStream_t st, int* launches) {
    FwdArgs a{};
    a.nh = p.nh;
    a.group = p.nh / p.nkv;
    a.pair_heads = a.group % 2 == 0;
    a.units = a.pair_heads ? p.nh / 2 : p.nh;
    a.T = p.T;
    a.scale2 = 1.4426950408889634f * p.scale;
    a.O = p.O;
    a.lse = p.lse;
    a.plan = p.plan;
    a.entries = p.entries;
    a.status = p.status;
    const int tile = a.pair_heads ? 128 : 256;
    // the plan's scans cross the CTA's warps: few of them where there is little to plan
    // (a prompt of one token: 12.0 us of device time with 1024 threads, 9.9 with 256)
    const unsigned planners = packed_attn_entries(p.nb, p.T, tile) <= 512 ? 256 : 1024;
    cudaError_t e = launch_dependent(packed_plan_kernel, dim3(1), dim3(planners), 0, st, p.cu_seqlens, p.nb, p.T, tile,
                                     p.entries, p.plan, p.ranks, p.status);
    if (e != cudaSuccess) return e;
    ++*launches;
    const unsigned grid = persistent_grid(packed_attn_entries(p.nb, p.T, tile) * a.units, p.sms);
    switch (d) {
        case 64: e = launch_fwd<64>(q, k, v, a, grid, st); break;
        case 96: e = launch_fwd<96>(q, k, v, a, grid, st); break;
        case 128: e = launch_fwd<128>(q, k, v, a, grid, st); break;
        default: e = launch_fwd<160>(q, k, v, a, grid, st); break;
    }
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace tpmlp
