// Differential attention of prompts on sm_103a (D = 128, two maps of width 64 over one V):
//   O = (softmax(scale q1 k1^T) - lambda_h softmax(scale q2 k2^T)) V, then diff.cuh's normalisation,
// with FP16 Q/K/V/P/O, FP32 accumulation in tensor memory and an FP32 online softmax per map.  Causal
// or not, shared-KV heads, ragged query and key lengths, key ranges split over CTAs when there are
// few query rows.
//
// Mathematics and work.  O1 = P1 V and O2 = P2 V are accumulated apart: each map has its own running
// max and sum, and only O1 / l1 - lambda O2 / l2 at the end joins them.  A visible (query, key) pair
// costs 2 * 64 FLOPs of QK and 2 * 128 of PV per map: 768 in all, against 512 for an ordinary head,
// and two exponentials instead of one.  So the tensor pipe bounds it (1536 cycles per 128 x 128 tile)
// with the softmax close behind.
//
// One CTA owns a 128-row query tile of one head and walks its 128-key tiles; a step is one map of one
// tile, and the steps alternate between the maps, so both maps use each K and V tile while it is in
// shared memory.  Warp roles (352 threads) are the dense kernel's (attn_dense.cu):
//   warp 0      TMA producer: Q once, then K_0, V_0, K_1, V_1, ... through a ring of 32 KB slots.
//   warp 1      allocates tensor memory and issues S_m = Q_m K_m^T (SMEM x SMEM, 4 MMAs).
//   warp 10     issues O_m += P_m V (P from TMEM).
//   warps 2..5, 6..9  softmax of map 0, of map 1: one thread per query row (TMEM lane = row).
// Tensor memory (512 columns): one S, P of each map (FP16 pairs), O of each map.  S is handed back as
// soon as the softmax has it in registers, so the other map's QK runs under this one's exponentials,
// and PV of a tile under the next tile's.
//
// Split keys: with fewer query tiles than SMs the key tiles of each are cut into C chunks of their
// own CTAs, which write unnormalised O_m, max and sum to `workspace`; a merge kernel joins them.
//
// Every wait is bounded in time (see WaitCtl): a wait that runs out records
// GBATTN_DEV_WAIT_TIMEOUT in the device status word, the CTA stops, waits a
// bounded time for its copies and MMAs in flight, frees tensor memory and exits.
#include <cuda_fp16.h>

#include <cmath>
#include <mutex>

#include "diff.cuh"
#include "host.h"
#include "ptx.cuh"

namespace gbattn {
namespace {

constexpr int kD = 128;              // head width: two maps of 64, values of 128
constexpr int kBM = 128;             // query rows per CTA
constexpr int kBN = 128;             // keys per tile (two halves of 64)
constexpr int kNS = 4;               // K/V ring slots (even: K tiles, odd: V tiles)
constexpr int kThreads = 352;
constexpr int kPvWarp = 10;
constexpr int kSoftmaxThreads = 128;   // per map
constexpr int kChunk = 128 * 128;    // 128 rows x 64 FP16 columns
constexpr int kQBytes = kBM * kD * 2;
constexpr int kSlotBytes = kBN * kD * 2;
// Tensor memory columns: S, then P of map 0 and of map 1 (FP16 pairs), then O of map 0 and of map 1.
constexpr uint32_t kTP = 128, kTO = 256;
constexpr uint32_t kIdescQK = idesc_f16(kBM, kBN, false, false);
constexpr uint32_t kIdescPV = idesc_f16(kBM, kD, false, true);
constexpr uint64_t kDrainNs = 200000000ull;   // 0.2 s for draining after an abort
constexpr float kLn2 = 0.69314718055994531f;

struct DiffPrefillArgs {
    int Sq, Skv, Hq, grp, causal;
    int chunks;         // CTAs per query tile along the keys
    const int32_t *q_lens, *kv_lens;   // [B] or null
    float scale_log2;   // scale * log2(e)
    __half* o;
    long long o_sb, o_sh, o_sr;   // element strides of O between batch entries, heads, rows
    float* lse;         // optional natural-log LSE [B][Hq][2][Sq]
    float* part_o;      // chunks > 1: [record][map][128][128], unnormalised
    float2* part_ml;    // [record][map][128]: (max in log2 units, sum)
    uint32_t* status;
    uint64_t wait_limit;
    int fault;          // test hook: 1 = the TMA warp never loads Q; 2 = it stops after 2*NS K/V items
    DiffArgs diff;
};

struct Ctrl {
    uint64_t q_full;
    uint64_t full[kNS];
    uint64_t empty[kNS];
    uint64_t s_full[2];       // S of a map's tile computed
    uint64_t s_free;          // S read into registers (once per step)
    uint64_t p_full[2];       // P of a map written
    uint64_t pv_done[2];      // PV of a map done: its P buffer is free, its O up to date
    uint64_t drain;
    uint64_t drain_pv;        // the PV issuer's own drain after an abort
    uint64_t xchg[4];         // per row quarter: the two threads of a row exchange values
    uint32_t tmem_base;
    int abort;
};

// Values exchanged in the epilogue between the two threads of a query row.
struct Exchange {
    float mx[2][128];   // [map][row] running max
    float l[2][128];    // [map][row] row sum
    float sq[2][128];   // [column half][row] partial sum of squares
};

constexpr int kCtrlBytes = 256 + static_cast<int>(sizeof(Exchange));
static_assert(sizeof(Ctrl) <= 256, "control block");
constexpr int kSmemBytes = 1024 + kQBytes + kNS * kSlotBytes + kCtrlBytes;

// Bounded wait that ignores the abort flag (used only to drain after an abort).
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > kDrainNs) return;
    }
}

// The lengths of batch entry b; one out of range counts as no queries.
struct Lens {
    int q, kv;
};
__device__ __forceinline__ Lens lens_of(const DiffPrefillArgs& a, int b) {
    Lens n{a.q_lens ? a.q_lens[b] : a.Sq, a.kv_lens ? a.kv_lens[b] : a.Skv};
    if (n.q < 0 || n.q > a.Sq || n.kv < 0 || n.kv > a.Skv) {
        atomicOr(a.status, kDevBadLength);
        n.q = n.kv = 0;
    }
    return n;
}

// Keys that query row i sees: the first visible(i).
__device__ __forceinline__ int visible(const Lens& n, int i, int causal) {
    if (i >= n.q) return 0;
    return causal ? max(0, n.kv - n.q + i + 1) : n.kv;
}

__device__ __forceinline__ void store_f32x8(float* p, const float* v) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
                 "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_diff_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const DiffPrefillArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sQ = smem;
    uint8_t* sKV = smem + kQBytes;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(sKV + kNS * kSlotBytes);
    Exchange* ex = reinterpret_cast<Exchange*>(reinterpret_cast<uint8_t*>(ctrl) + 256);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bh = static_cast<int>(blockIdx.x);
    const int b = bh / a.Hq, head = bh - b * a.Hq, hk = head / a.grp;
    // the longest (causal) query tiles first, so that the short ones fill the last wave
    const int q_row0 = static_cast<int>(gridDim.y - 1 - blockIdx.y) * kBM;
    const Lens n = lens_of(a, b);
    const int last = min(q_row0 + kBM, n.q) - 1;   // last query row of the tile
    const int seen = last < q_row0 ? 0 : visible(n, last, a.causal);
    const int all_tiles = (seen + kBN - 1) / kBN;
    const int per = (all_tiles + a.chunks - 1) / a.chunks;
    const int tile0 = min(static_cast<int>(blockIdx.z) * per, all_tiles);
    const int n_tiles = min(per, all_tiles - tile0);

    // ---- prologue
    if (threadIdx.x == 0) {
        mbar_init(&ctrl->q_full, 1);
        for (int i = 0; i < kNS; ++i) {
            mbar_init(&ctrl->full[i], 1);
            mbar_init(&ctrl->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctrl->s_full[i], 1);
            mbar_init(&ctrl->p_full[i], kSoftmaxThreads);
            mbar_init(&ctrl->pv_done[i], 1);
        }
        mbar_init(&ctrl->s_free, kSoftmaxThreads);
        for (int i = 0; i < 4; ++i) mbar_init(&ctrl->xchg[i], 64);
        mbar_init(&ctrl->drain, 1);
        mbar_init(&ctrl->drain_pv, 1);
        ctrl->abort = 0;
        mbar_init_fence();
    }
    const bool load_q = a.fault != 1;
    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        __syncwarp();   // the barriers thread 0 initialised are visible to the warp
    }
    if (warp == 1) {
        tmem_alloc(&ctrl->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctrl->tmem_base;
    const WaitCtl w{a.wait_limit, a.status, &ctrl->abort};

    if (warp == 0) {
        // ================= TMA producer (whole warp; one elected lane issues)
        if (n_tiles > 0) {
            int last_it[kNS] = {-1, -1, -1, -1};
            if (load_q) {
                if (elect_one()) {
                    mbar_arrive_expect_tx(&ctrl->q_full, kQBytes);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tma_load_4d(sQ + c * kChunk, &tmQ, &ctrl->q_full, c * 64, q_row0, head, b);
                }
                __syncwarp();
            }
            bool ok = true;
            for (int it = 0; it < 2 * n_tiles; ++it) {
                if (a.fault == 2 && it >= 2 * kNS) {   // test hook: stop mid-stream, drain, leave
                    ok = false;
                    break;
                }
                const int slot = it % kNS;
                if (!wait_warp(&ctrl->empty[slot], ((it / kNS) & 1) ^ 1u, w)) { ok = false; break; }
                const int k0 = (tile0 + (it >> 1)) * kBN;
                const CUtensorMap* m = (it & 1) ? &tmV : &tmK;
                uint8_t* dst = sKV + slot * kSlotBytes;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&ctrl->full[slot], kSlotBytes);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tma_load_4d(dst + c * kChunk, m, &ctrl->full[slot], c * 64, k0, hk, b);
                }
                __syncwarp();
                last_it[slot] = it;
            }
            if (!ok && lane == 0) {   // let copies in flight land before the CTA exits
                if (load_q) drain_wait(&ctrl->q_full, 0);
                for (int s = 0; s < kNS; ++s)
                    if (last_it[s] >= 0) drain_wait(&ctrl->full[s], (last_it[s] / kNS) & 1);
            }
        }
    } else if (warp == 1) {
        // ================= QK issuer.  A step's QK overwrites the S that the step before
        // it left, as soon as the softmax has that in registers.  K_t sits at ring
        // position 2 t; the previous item of its slot, K_{t - 2}, was waited for by
        // this warp.
        if (n_tiles > 0) {
            bool ok = wait_warp(&ctrl->q_full, 0, w);
            const uint32_t qa = smem_addr(sQ);
            for (int t = 0; ok && t < n_tiles; ++t) {
                const int slot = (2 * t) % kNS;
                const uint32_t ka = smem_addr(sKV + slot * kSlotBytes);
                for (int m = 0; m < 2; ++m) {
                    const int s = 2 * t + m;
                    if (s > 0) ok = wait_warp(&ctrl->s_free, (s - 1) & 1, w);
                    if (m == 0) ok = ok && wait_warp(&ctrl->full[slot], (2 * t / kNS) & 1, w);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k16 = 0; k16 < 4; ++k16) {
                            const uint32_t off = m * kChunk + k16 * 32;
                            mma_ss(tmem, sdesc_sw128(qa + off, 16, 1024),
                                   sdesc_sw128(ka + off, 16, 1024), kIdescQK, k16 > 0 ? 1u : 0u);
                        }
                        mma_commit(&ctrl->s_full[m]);
                        if (m == 1) mma_commit(&ctrl->empty[slot]);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {   // wait for issued MMAs before tensor memory is freed
                if (elect_one()) mma_commit(&ctrl->drain);
                __syncwarp();
                if (lane == 0) drain_wait(&ctrl->drain, 0);
            }
        }
    } else if (warp == kPvWarp) {
        // ================= PV issuer: waits for P of the step and, once a tile, for V_t
        // (ring position 2 t + 1; the slot's previous item is V_{t - 2}).
        if (n_tiles > 0) {
            bool ok = true;
            for (int t = 0; ok && t < n_tiles; ++t) {
                const int slot = (2 * t + 1) % kNS;
                const uint32_t va = smem_addr(sKV + slot * kSlotBytes);
                for (int m = 0; m < 2; ++m) {
                    if (m == 0) {
                        ok = wait_warp(&ctrl->full[slot], ((2 * t + 1) / kNS) & 1, w);
                        const int live = n.kv - (tile0 + t) * kBN;   // keys of the tile that exist
                        if (ok && live < kBN && n.kv < a.Skv) {
                            // Rows past this entry's keys may hold anything, and P = 0 times
                            // a NaN is a NaN: clear them.
                            uint4* v16 = reinterpret_cast<uint4*>(sKV + slot * kSlotBytes);
                            for (int x = live * 8 + lane; x < kBN * 8; x += 32)
                                v16[x] = v16[kChunk / 16 + x] = make_uint4(0, 0, 0, 0);
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                        }
                    }
                    ok = ok && wait_warp(&ctrl->p_full[m], t & 1, w);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k16 = 0; k16 < kBN / 16; ++k16)
                            mma_ts(tmem + kTO + m * 128, tmem + kTP + m * 64 + k16 * 8,
                                   sdesc_sw128(va + k16 * 2048, kChunk, 1024), kIdescPV,
                                   (t > 0 || k16 > 0) ? 1u : 0u);
                        if (m == 1) mma_commit(&ctrl->empty[slot]);
                        mma_commit(&ctrl->pv_done[m]);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {   // wait for issued MMAs before tensor memory is freed
                if (elect_one()) mma_commit(&ctrl->drain_pv);
                __syncwarp();
                if (lane == 0) drain_wait(&ctrl->drain_pv, 0);
            }
        }
    } else {
        // ================= softmax / correction / epilogue (warps 2..5 map 0, 6..9 map 1)
        // A thread owns one query row of one map (TMEM lane quarter = warp % 4), so nothing is
        // exchanged until the epilogue and the two maps' warps run out of step: while one map's
        // are in their exponentials, the other's load scores or wait for the tensor core.
        const int quarter = warp & 3;
        const int m = (warp - 2) >> 2;
        const int row = quarter * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t pbuf = tl + kTP + m * 64, obuf = tl + kTO + m * 128;
        const int row_g = q_row0 + row;
        uint64_t* xbar = &ctrl->xchg[quarter];
        const int lim = visible(n, row_g, a.causal);   // keys >= lim are invisible
        const float sl2 = a.scale_log2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        float m_run = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int t = 0; t < n_tiles; ++t) {
            ok = wait_warp(&ctrl->s_full[m], t & 1, w);
            if (!ok) break;
            tc_fence_after();
            uint32_t x[kBN];
#pragma unroll
            for (int c = 0; c < kBN; c += 32) tmem_ld32(tl + c, x + c);
            tmem_ld_wait();
            tc_fence_before();
            mbar_arrive(&ctrl->s_free);

            const int k0 = (tile0 + t) * kBN;
            if (k0 + kBN > lim) {   // keys the row does not see
#pragma unroll
                for (int c = 0; c < kBN; ++c)
                    if (k0 + c >= lim) x[c] = __float_as_uint(-INFINITY);
            }
            // row max with four independent chains (short latency)
            float m4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = __uint_as_float(x[k]);
#pragma unroll
            for (int c = 4; c < 124; c += 8) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    m4[k] = max3f(m4[k], __uint_as_float(x[c + k]), __uint_as_float(x[c + 4 + k]));
            }
            m4[0] = max3f(m4[0], __uint_as_float(x[124]), __uint_as_float(x[125]));
            m4[1] = max3f(m4[1], __uint_as_float(x[126]), __uint_as_float(x[127]));
            const float mx = fmaxf(max3f(m4[0], m4[1], m4[2]), m4[3]);
            const float m_new = fmaxf(m_run, mx * sl2);
            const bool need = m_new > m_run + 8.0f;
            float alpha = 1.0f;
            if (need) {
                alpha = fast_exp2(m_run - m_new);
                m_run = m_new;
            }
            const bool warp_need = __any_sync(0xffffffffu, need);
            const float m_use = m_run == -INFINITY ? 0.0f : m_run;
            const uint64_t negm = f2_pack(-m_use, -m_use);
            if (t > 0) {   // the P buffer is free and O complete up to the last tile
                ok = wait_warp(&ctrl->pv_done[m], (t - 1) & 1, w);
                if (!ok) break;
                tc_fence_after();
            }
            uint64_t rs[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) rs[k] = f2_pack(0.0f, 0.0f);
#pragma unroll
            for (int c = 0; c < kBN; c += 32) {
                uint32_t p2[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x0, x1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c + 2 * i]),
                                             __uint_as_float(x[c + 2 * i + 1])),
                                     sl2x2, negm),
                              x0, x1);
                    const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                    rs[i & 3] = f2_add(rs[i & 3], f2_pack(p0, p1));   // four independent sums
                    p2[i] = pack_half2(p0, p1);
                }
                tmem_st16(pbuf + c / 2, p2);
            }
            float r0, r1, r2, r3, r4, r5, r6, r7;
            f2_unpack(rs[0], r0, r1);
            f2_unpack(rs[1], r2, r3);
            f2_unpack(rs[2], r4, r5);
            f2_unpack(rs[3], r6, r7);
            l = l * alpha + (((r0 + r1) + (r2 + r3)) + ((r4 + r5) + (r6 + r7)));
            tmem_st_wait();
            if (warp_need && t > 0) {   // rescale the row of O
                const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
                for (int cc = 0; cc < 4; ++cc) {
                    uint32_t o[32];
                    tmem_ld32(obuf + cc * 32, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float y0, y1;
                        f2_unpack(f2_mul(f2_pack(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), a2),
                                  y0, y1);
                        o[2 * e] = __float_as_uint(y0);
                        o[2 * e + 1] = __float_as_uint(y1);
                    }
                    tmem_st32(obuf + cc * 32, o);
                }
                tmem_st_wait();
            }
            tc_fence_before();
            mbar_arrive(&ctrl->p_full[m]);
        }
        if (ok && n_tiles > 0) {
            ok = wait_warp(&ctrl->pv_done[0], (n_tiles - 1) & 1, w) &&
                 wait_warp(&ctrl->pv_done[1], (n_tiles - 1) & 1, w);
            tc_fence_after();
        }
        // From here a thread works on half of the columns of both maps.
        const int half = m;
        uint32_t xphase = 0;
        float l2[2] = {0.0f, 0.0f}, mr[2] = {-INFINITY, -INFINITY};
        if (ok) {
            ex->mx[m][row] = m_run;
            ex->l[m][row] = l;
            mbar_arrive(xbar);
            ok = wait_warp(xbar, xphase, w);
            xphase ^= 1u;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                l2[k] = ex->l[k][row];
                mr[k] = ex->mx[k][row];
            }
        }
        const bool row_ok = row_g < a.Sq;
        if (ok && a.chunks > 1) {   // a partial record per map
            const long long rec =
                (static_cast<long long>(bh) * gridDim.y + q_row0 / kBM) * a.chunks + blockIdx.z;
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
                const int m = x >> 1, c0 = half * 64 + (x & 1) * 32;
                uint32_t o[32];
                if (n_tiles > 0) {
                    tmem_ld32(tl + kTO + m * 128 + c0, o);
                    tmem_ld_wait();
                }
                if (!row_ok || n_tiles == 0) continue;
                float* dst = a.part_o + ((rec * 2 + m) * kBM + row) * kD + c0;
#pragma unroll
                for (int e = 0; e < 32; e += 8) store_f32x8(dst + e, reinterpret_cast<float*>(o) + e);
            }
            if (half == 0) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    a.part_ml[(rec * 2 + m) * kBM + row] = make_float2(mr[m], l2[m]);
            }
        } else if (ok) {
            const float lambda = diff_lambda(a.diff, head, kD / 2, lane);
            const float f0 = l2[0] == 0.0f ? 0.0f : 1.0f / l2[0];
            const float f1 = l2[1] == 0.0f ? 0.0f : -lambda / l2[1];
            float y[64];   // this thread's columns
            float sq = 0.0f;
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                const int c0 = half * 64 + cc * 32;
                uint32_t o0[32], o1[32];
                if (n_tiles > 0) {
                    tmem_ld32(tl + kTO + c0, o0);
                    tmem_ld32(tl + kTO + 128 + c0, o1);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o0[e] = o1[e] = 0u;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float v = __uint_as_float(o0[e]) * f0 + __uint_as_float(o1[e]) * f1;
                    y[cc * 32 + e] = v;
                    sq += v * v;
                }
            }
            if (a.diff.norm) {
                ex->sq[half][row] = sq;
                mbar_arrive(xbar);
                ok = wait_warp(xbar, xphase, w);
                sq += ex->sq[half ^ 1][row];
                const float rn = rsqrtf(sq * (1.0f / kD) + a.diff.eps) * (1.0f - a.diff.init);
#pragma unroll
                for (int e = 0; e < 64; ++e) y[e] *= rn * a.diff.norm[half * 64 + e];
            }
            if (ok && row_ok) {
                uint4* dst = reinterpret_cast<uint4*>(a.o + b * a.o_sb + head * a.o_sh +
                                                      row_g * a.o_sr + half * 64);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    uint32_t hw[4];
#pragma unroll
                    for (int f = 0; f < 4; ++f) hw[f] = pack_half2(y[8 * e + 2 * f], y[8 * e + 2 * f + 1]);
                    dst[e] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
                }
                if (half == 0 && a.lse) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        a.lse[(static_cast<long long>(bh) * 2 + m) * a.Sq + row_g] =
                            l2[m] == 0.0f ? -INFINITY : (mr[m] + log2f(l2[m])) * kLn2;
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the chunks of one query row per warp (four columns a lane): per map M = max_c m_c,
// l = sum_c 2^(m_c - M) l_c, O_m = sum_c 2^(m_c - M) O_c / l, then the difference and the norm.
// Every chunk reads its records once; a chunk that saw nothing has sum 0 and no O.
__global__ void __launch_bounds__(256) attn_diff_merge_kernel(const DiffPrefillArgs a, int q_tiles) {
    const int lane = threadIdx.x & 31;
    const int bh = static_cast<int>(blockIdx.x);
    const int row_g = static_cast<int>(blockIdx.y) * 8 + static_cast<int>(threadIdx.x >> 5);
    const int b = bh / a.Hq, head = bh - b * a.Hq;
    const float lambda = diff_lambda(a.diff, head, kD / 2, lane);
    // a programmatic dependent of the attention grid
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row_g >= a.Sq) return;
    const long long rec0 = (static_cast<long long>(bh) * q_tiles + row_g / kBM) * a.chunks;
    const int row = row_g % kBM;
    float out[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        float M = -INFINITY, L = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int c = 0; c < a.chunks; ++c)
            M = fmaxf(M, a.part_ml[((rec0 + c) * 2 + m) * kBM + row].x);
        for (int c = 0; c < a.chunks; ++c) {
            const long long at = ((rec0 + c) * 2 + m) * kBM + row;
            const float2 ml = a.part_ml[at];
            if (ml.y == 0.0f) continue;
            const float wt = exp2f(ml.x - M);
            const float4 v = *reinterpret_cast<const float4*>(a.part_o + at * kD + lane * 4);
            acc[0] += wt * v.x;
            acc[1] += wt * v.y;
            acc[2] += wt * v.z;
            acc[3] += wt * v.w;
            L += wt * ml.y;
        }
        const float f = L == 0.0f ? 0.0f : (m == 0 ? 1.0f : -lambda) / L;
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] += acc[e] * f;
        if (a.lse && lane == 0)
            a.lse[(static_cast<long long>(bh) * 2 + m) * a.Sq + row_g] =
                L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
    if (a.diff.norm) {
        float sq = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) sq += out[e] * out[e];
        const float rn = rsqrtf(warp_sum(sq) * (1.0f / kD) + a.diff.eps) * (1.0f - a.diff.init);
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] *= rn * a.diff.norm[lane * 4 + e];
    }
    *reinterpret_cast<uint2*>(a.o + b * a.o_sb + head * a.o_sh + row_g * a.o_sr + lane * 4) =
        make_uint2(pack_half2(out[0], out[1]), pack_half2(out[2], out[3]));
}

size_t record_bytes() { return 2ull * kBM * (kD * 4 + 8); }

// Chunks along the keys for `units` query tiles of all heads with `tiles` key tiles each: the number
// that minimises waves * (tiles per chunk + 3 for a CTA's start and end) plus, for more than one,
// the records' trip through memory (about 20 records written and read per tile time and wave).
int pick_chunks(long long units, int tiles, int sms) {
    int best = 1;
    double best_cost = 1e30;
    for (int c = 1; c <= 16 && (c == 1 || tiles / c >= 4); ++c) {
        const double waves = static_cast<double>((units * c + sms - 1) / sms);
        const double cost = waves * ((tiles + c - 1) / c + 3) + (c > 1 ? units * c / 20.0 : 0.0);
        if (cost < best_cost) {
            best_cost = cost;
            best = c;
        }
    }
    return best;
}

int sm_count_or_default() {
    DeviceState d;
    return current_device(&d) == GBATTN_OK ? d.num_sms : 152;
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" size_t attn_diff_prefill_workspace_size(int B, int Hq, int Sq, int Skv, int D) {
    if (B <= 0 || Hq <= 0 || Sq <= 0 || Skv <= 0 || D != kD) return 0;
    const long long units = static_cast<long long>(B) * Hq * ((static_cast<long long>(Sq) + kBM - 1) / kBM);
    const int c = pick_chunks(units, static_cast<int>((static_cast<long long>(Skv) + kBN - 1) / kBN),
                              sm_count_or_default());
    return c > 1 ? static_cast<size_t>(units) * c * record_bytes() : 0;
}

extern "C" int attn_diff_prefill_fwd(const void* q, const void* k, const void* v,
                                     const float* lambda_vecs, int lambda_heads, float lambda_init,
                                     const float* norm_weight, float eps, const int32_t* q_lens,
                                     const int32_t* kv_lens, void* o, float* lse, int B, int Hq,
                                     int Hkv, int Sq, int Skv, int D, const int64_t* q_strides,
                                     const int64_t* kv_strides, const int64_t* o_strides,
                                     float scale, int causal, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    CallRange nvtx_range("attn_diff_prefill_fwd");
    if (!q || !k || !v || !lambda_vecs || !o) return GBATTN_ERR_NULL;
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Skv <= 0 || Hq % Hkv != 0) return GBATTN_ERR_SHAPE;
    if (static_cast<long long>(B) * Hq > 65535 || Sq > (1 << 22) || Skv > (1 << 30))
        return GBATTN_ERR_SHAPE;
    if (lambda_heads != 1 && lambda_heads != Hq) return GBATTN_ERR_SHAPE;
    if (causal != 0 && causal != 1) return GBATTN_ERR_SHAPE;
    if (D != kD) return GBATTN_ERR_UNSUPPORTED;
    Strides qs, kvs, os;
    if (!make_strides(q_strides, B, Hq, Sq, D, false, &qs) ||
        !make_strides(kv_strides, B, Hkv, Skv, D, false, &kvs) ||
        !make_strides(o_strides, B, Hq, Sq, D, true, &os))
        return GBATTN_ERR_SHAPE;
    if (!finite_positive(scale) || !(std::fabs(lambda_init) <= 3.402823466e38f) ||
        (norm_weight && !finite_positive(eps)))
        return GBATTN_ERR_SCALE;
    auto misaligned4 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (reinterpret_cast<uintptr_t>(workspace) & 31u) || misaligned4(lambda_vecs) ||
        misaligned4(norm_weight) || misaligned4(q_lens) || misaligned4(kv_lens) || misaligned4(lse))
        return GBATTN_ERR_ALIGN;
    DeviceState dev;
    const int q_tiles = (Sq + kBM - 1) / kBM;
    const long long units = static_cast<long long>(B) * Hq * q_tiles;
    const int tiles = static_cast<int>((static_cast<long long>(Skv) + kBN - 1) / kBN);
    int chunks = pick_chunks(units, tiles, sm_count_or_default());
    if (Sq > 8 * 65535) chunks = 1;   // the merge's grid
    while (chunks > 1 &&
           (!workspace || static_cast<size_t>(units) * chunks * record_bytes() > workspace_bytes))
        --chunks;
    struct Range { const void* p; size_t n; };
    const size_t kb = strided_bytes(kvs, B, Hkv, Skv, D);
    const Range in[] = {{q, strided_bytes(qs, B, Hq, Sq, D)},
                        {k, kb},
                        {v, kb},
                        {lambda_vecs, static_cast<size_t>(lambda_heads) * 4 * (kD / 2) * 4},
                        {norm_weight, static_cast<size_t>(kD) * 4},
                        {q_lens, static_cast<size_t>(B) * 4},
                        {kv_lens, static_cast<size_t>(B) * 4}};
    const Range out[] = {{o, strided_bytes(os, B, Hq, Sq, D)},
                         {lse, static_cast<size_t>(B) * Hq * 2 * Sq * 4},
                         {workspace, chunks > 1 ? static_cast<size_t>(units) * chunks * record_bytes() : 0}};
    for (int i = 0; i < 3; ++i) {
        for (const Range& y : in)
            if (overlaps(out[i].p, out[i].n, y.p, y.n)) return GBATTN_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return GBATTN_ERR_ALIAS;
    }
    int rc = current_device(&dev);
    if (rc != GBATTN_OK) return rc;
    if (dev.device < 0 || dev.device >= 64) return GBATTN_ERR_CUDA;
    DiffPrefillArgs a{};
    a.Sq = Sq;
    a.Skv = Skv;
    a.Hq = Hq;
    a.grp = Hq / Hkv;
    a.causal = causal;
    a.chunks = chunks;
    a.q_lens = q_lens;
    a.kv_lens = kv_lens;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.o = static_cast<__half*>(o);
    a.o_sb = os.b;
    a.o_sh = os.h;
    a.o_sr = os.r;
    a.lse = lse;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(units) * chunks * 2 * kBM * kD);
    a.status = dev.status;
    a.wait_limit = wait_limit_ns();
    a.fault = fault_mode();
    a.diff = DiffArgs{lambda_vecs, norm_weight, lambda_heads, lambda_init, eps};
    CUtensorMap tq, tk, tv;
    if (encode_tmap_f16_4d(&tq, q, D, Sq, Hq, B, qs.r, qs.h, qs.b, 64, kBM) != GBATTN_OK ||
        encode_tmap_f16_4d(&tk, k, D, Skv, Hkv, B, kvs.r, kvs.h, kvs.b, 64, kBN) != GBATTN_OK ||
        encode_tmap_f16_4d(&tv, v, D, Skv, Hkv, B, kvs.r, kvs.h, kvs.b, 64, kBN) != GBATTN_OK)
        return GBATTN_ERR_CUDA;
    static std::once_flag once[64];
    static int attr_rc[64];
    std::call_once(once[dev.device], [&] {
        attr_rc[dev.device] = cudaFuncSetAttribute(attn_diff_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kSmemBytes) == cudaSuccess
                                  ? GBATTN_OK
                                  : GBATTN_ERR_CUDA;
    });
    if (attr_rc[dev.device] != GBATTN_OK) return attr_rc[dev.device];
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    attn_diff_kernel<<<dim3(B * Hq, q_tiles, chunks), kThreads, kSmemBytes, s>>>(tq, tk, tv, a);
    count_launches(1);
    rc = launch_status();
    if (rc != GBATTN_OK || chunks == 1) return rc;
    // The merge's CTAs may be placed as attention CTAs retire; they wait for the whole grid.
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(B * Hq, (Sq + 7) / 8);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_diff_merge_kernel, a, q_tiles);
    count_launches(1);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GBATTN_ERR_CUDA;
    }
    return launch_status();
}
