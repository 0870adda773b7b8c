// Differential attention of prompts on sm_103a (D = 128, two maps of width 64 over one V):
//   O = (softmax(scale q1 k1^T) - lambda_h softmax(scale q2 k2^T)) V, then diff.cuh's normalisation,
// with FP16 Q/K/V/O, P as FP16 hi + lo, FP32 accumulation in tensor memory and an FP32 online softmax
// per map.  Causal or not, shared-KV heads, ragged query and key lengths, key ranges split over CTAs
// when there are few query rows.
//
// Mathematics and work.  O1 = P1 V and O2 = P2 V are accumulated apart: each map has its own running
// max and sum, and only O1 / l1 - lambda O2 / l2 at the end joins them.  A visible (query, key) pair
// costs 2 * 64 FLOPs of QK and 2 * 128 of PV per map: 768 in all, against 512 for an ordinary head,
// and two exponentials instead of one.
//
// P is rounded to two FP16 halves, hi = RNE(p) and lo = RNE(p - hi), 2^-22 of p, with the largest p
// near the top of FP16's range so that small ones keep their bits (kShift in tiles.cuh).  What the maps have
// in common cancels in the difference and the norm brings the rest back to unit size, so P's rounding
// grows as the output shrinks: with one FP16 value the error against float64 was 2.6 to 3.2e-4 of
// unrelated maps' output and 9.9e-4 of maps correlated by 0.999 (lambda 0.78), of which the output's
// own rounding is 2.1e-4.  The second half costs another PV: 1280 tensor cycles per 64 keys and both
// maps instead of 768, and a third of the softmax's instructions.
//
// Persistent CTAs, one per SM, work through items: a 128-row query tile of one head (a unit) and its
// 64-key tiles, or a part of them.  A step is one map of one key tile; the steps alternate between
// the maps, so both maps use each K and V tile while it is in shared memory.  Warp roles (352 threads):
//   warp 0      TMA producer: Q of each item into one of two buffers, then K_0, V_0, K_1, V_1, ...
//               through a ring of 16 KB slots, on into the next item.
//   warp 1      allocates tensor memory and issues S_m = Q_m K_m^T (SMEM x SMEM, 4 MMAs).
//   warp 10     issues O_m += hi_m V + lo_m V (P from TMEM).
//   warps 2..5, 6..9  softmax of map 0, of map 1: one thread per query row (TMEM lane = row); at an
//               item's end each takes half of the columns of both O, and the next item's QK runs
//               under this epilogue.
// Tensor memory (512 columns): S of each map (64), P of each map (FP16 pairs: 32 hi, 32 lo), O of each
// map (128).  With 128 keys a tile, hi and lo would leave no columns for S beside them.  S is handed
// back as soon as the softmax has it in registers, so the next tile's QK runs under this one's
// exponentials, and PV of a tile under the next tile's.
//
// Which CTA does what: with many units, whole units, the longest (causal) first, in rounds that run
// over the CTAs forth and back, so that every CTA gets the same work to about one key tile a round.
// With few, the key tiles of all units are laid end to end and every CTA takes an equal contiguous
// range of them (as the decode kernels do); the parts of a unit that ranges cut leave unnormalised
// O_m, max and sum in `workspace`, and a merge kernel joins them.
//
// Measured (graph replays): 16 heads x 8192 causal 464 us (447 with kShift 7, 479 with 13), 500
// queries on 32,500 keys 243 us.  The softmax's chain bounds it: copies of a version that took 420 us
// took 358 us without any softmax, 430 without MMAs (one k-step each) and 342 without the lo halves in
// softmax and PV.  Of a softmax warp's 1,750 cycles per tile 800 are the exponentials with both
// roundings, 256 and 211 the waits for S and for the P buffer, 180 the maximum, 240 loads and stores.
// Slower: P written in two or four chunks between the exponentials (457 to 492), PV's lo half without
// a gap behind its hi half (434).
//
// Every wait is bounded in time (see WaitCtl): a wait that runs out records
// GBATTN_DEV_WAIT_TIMEOUT in the device status word, the CTA stops, waits a
// bounded time for its copies and MMAs in flight, frees tensor memory and exits.
#include <cuda_fp16.h>

#include <cmath>
#include <cstddef>
#include <mutex>

#include "diff.cuh"
#include "host.h"
#include "ptx.cuh"
#include "tiles.cuh"

namespace gbattn {
namespace {

constexpr int kD = 128;              // head width: two maps of 64, values of 128
constexpr int kBM = 128;             // query rows per CTA
constexpr int kBN = 64;              // keys per tile
constexpr int kNS = 8;               // K/V ring slots (even: K tiles, odd: V tiles)
constexpr int kThreads = 352;
constexpr int kPvWarp = 10;
constexpr int kSoftmaxThreads = 128;   // per map
constexpr int kQChunk = kBM * 128;   // 64 FP16 columns of a Q tile's rows
constexpr int kKvChunk = kBN * 128;  // and of a K or V tile's
constexpr int kQBytes = kBM * kD * 2;
constexpr int kSlotBytes = kBN * kD * 2;
// Tensor memory columns: S of each map, P of each map (FP16 pairs: 32 columns of hi, 32 of lo), O of
// each map.
constexpr uint32_t kTS = 64, kTP = 128, kTPMap = 64, kTPLo = 32, kTO = 256;
constexpr uint32_t kIdescQK = idesc_f16(kBM, kBN, false, false);
constexpr uint32_t kIdescPV = idesc_f16(kBM, kD, false, true);
constexpr uint64_t kDrainNs = 200000000ull;   // 0.2 s for draining after an abort
constexpr float kLn2 = 0.69314718055994531f;

struct DiffPrefillArgs {
    int Sq, Skv, Hq, grp, causal;
    int units, q_tiles;   // query tiles of all heads, of one head
    int split;            // 1: equal ranges of all units' key tiles
    const int32_t *q_lens, *kv_lens;   // [B] or null
    float scale_log2;   // scale * log2(e)
    __half* o;
    long long o_sb, o_sh, o_sr;   // element strides of O between batch entries, heads, rows
    float* lse;         // optional natural-log LSE [B][Hq][2][Sq]
    // split: records 2 c (the unit that CTA c's range begins in) and 2 c + 1 (the one that begins in
    // the range and goes on behind it)
    float* part_o;        // [record][map][128][128], unnormalised
    float2* part_ml;      // [record][map][128]: (reference in log2 units, sum)
    uint32_t* prefix;     // [units + 1]: key tiles of the units before u
    uint32_t* status;
    uint64_t wait_limit;
    int fault;          // test hook: 1 = the TMA warp never loads Q; 2 = it stops after 2*NS K/V items
    DiffArgs diff;
};

struct Ctrl {
    uint64_t q_full[2];
    uint64_t q_empty[2];      // the last QK of the buffer's item is done
    uint64_t full[kNS];
    uint64_t empty[kNS];
    uint64_t s_full[2];       // S of a map's tile computed
    uint64_t s_free[2];       // S of a map read into registers
    uint64_t p_full[2];       // P of a map written
    uint64_t pv_done[2];      // PV of a map done: its P buffer is free, its O up to date
    uint64_t o_free;          // an item's O read into registers
    uint64_t drain;
    uint64_t drain_pv;        // the PV issuer's own drain after an abort
    uint64_t xchg[4];         // per row quarter: the two threads of a row exchange values
    uint32_t tmem_base;
    int abort;
};

// Values exchanged in the epilogue between the two threads of a query row.
struct Exchange {
    float mx[2][128];      // [map][row] reference of the exponentials
    float l[2][128];       // [map][row] row sum
    float sq[2][128];      // [column half][row] partial sum of squares
    float norm[128];       // the norm weight * (1 - lambda_init)
};

constexpr int kBarBytes = 320;
constexpr int kCtrlBytes = kBarBytes + static_cast<int>(sizeof(Exchange));
constexpr int kItemBytes = 64;       // a warp's place in its items
static_assert(sizeof(Ctrl) <= kBarBytes, "control block");
constexpr int kMaxUnits = 512;       // units of a split launch (prefix table in shared memory)
constexpr int kSmemBytes = 1024 + 2 * kQBytes + kNS * kSlotBytes + kCtrlBytes +
                           kItemBytes * (kThreads / 32) + 4 * (kMaxUnits + 4);

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

__device__ __forceinline__ void store_f32x8(float* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Key tiles that query tile qt of a batch entry walks.
__device__ __forceinline__ int unit_tiles(const Lens& n, int qt, int causal) {
    const int last = min((qt + 1) * kBM, n.q) - 1;   // last query row of the tile
    return last < qt * kBM ? 0 : (visible(n, last, causal) + kBN - 1) / kBN;
}

// One item of a CTA's work: n_tiles key tiles from tile0 of a unit; rec >= 0: a part of the unit,
// left in that record.
struct Item {
    int bh, qt, tile0, n_tiles, rec;
    Lens n;
};

// The items of one CTA in order.  Every warp walks them by itself, lane 0 for the others, in a
// place of its own in shared memory: the softmax has no registers to spare for it.
struct Items {
    int k;                       // items drawn (whole units)
    uint32_t pos, end, first;    // the CTA's range of key tiles (split)
    Item it;
    float lambda;
};

__device__ __forceinline__ void items_begin(Items& s, const DiffPrefillArgs& a, const uint32_t* prefix) {
    if ((threadIdx.x & 31) == 0) {
        s.k = 0;
        s.pos = s.end = s.first = 0;
        if (a.split) {
            const uint32_t U = prefix[a.units], W = min(gridDim.x, U);
            if (blockIdx.x < W) {
                s.first = s.pos = warp_start(blockIdx.x, W, U);
                s.end = warp_start(blockIdx.x + 1, W, U);
            }
        }
    }
}

// The next item, or false behind the last.
__device__ __forceinline__ bool items_next(Items& s, const DiffPrefillArgs& a, const uint32_t* prefix) {
    bool more = false;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        Item& it = s.it;
        if (!a.split) {   // rounds over the CTAs, forth and back; the last query tiles first
            const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
            const long long i = static_cast<long long>(s.k) * g + ((s.k & 1) ? g - 1 - c : c);
            ++s.k;
            more = i < a.units;
            if (more) {
                const int heads = a.units / a.q_tiles;
                it.qt = a.q_tiles - 1 - static_cast<int>(i / heads);
                it.bh = static_cast<int>(i % heads);
                it.n = lens_of(a, it.bh / a.Hq);
                it.tile0 = 0;
                it.n_tiles = unit_tiles(it.n, it.qt, a.causal);
                it.rec = -1;
            }
        } else if (s.pos < s.end) {
            more = true;
            int lo = 0, hi = a.units - 1;   // largest unit whose first tile is <= pos
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (prefix[mid] <= s.pos) lo = mid; else hi = mid - 1;
            }
            const uint32_t u0 = prefix[lo], u1 = prefix[lo + 1], stop = min(s.end, u1);
            it.bh = lo / a.q_tiles;
            it.qt = lo - it.bh * a.q_tiles;
            it.n = lens_of(a, it.bh / a.Hq);
            it.tile0 = static_cast<int>(s.pos - u0);
            it.n_tiles = static_cast<int>(stop - s.pos);
            it.rec = (s.pos == u0 && stop == u1)
                         ? -1
                         : 2 * static_cast<int>(blockIdx.x) + (s.pos == s.first ? 0 : 1);
            s.pos = stop;
        }
    }
    return __shfl_sync(0xffffffffu, more, 0);   // orders lane 0's writes before the others' reads
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_diff_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const DiffPrefillArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sQ = smem;
    uint8_t* sKV = smem + 2 * kQBytes;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(sKV + kNS * kSlotBytes);
    Exchange* ex = reinterpret_cast<Exchange*>(reinterpret_cast<uint8_t*>(ctrl) + kBarBytes);
    uint8_t* item_mem = reinterpret_cast<uint8_t*>(ctrl) + kCtrlBytes;
    uint32_t* prefix = reinterpret_cast<uint32_t*>(item_mem + kItemBytes * (kThreads / 32));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // ---- prologue
    if (threadIdx.x == 0) {
        for (int i = 0; i < kNS; ++i) {
            mbar_init(&ctrl->full[i], 1);
            mbar_init(&ctrl->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctrl->q_full[i], 1);
            mbar_init(&ctrl->q_empty[i], 1);
            mbar_init(&ctrl->s_full[i], 1);
            mbar_init(&ctrl->s_free[i], kSoftmaxThreads);
            mbar_init(&ctrl->p_full[i], kSoftmaxThreads);
            mbar_init(&ctrl->pv_done[i], 1);
        }
        mbar_init(&ctrl->o_free, 2 * kSoftmaxThreads);
        for (int i = 0; i < 4; ++i) mbar_init(&ctrl->xchg[i], 64);
        mbar_init(&ctrl->drain, 1);
        mbar_init(&ctrl->drain_pv, 1);
        ctrl->abort = 0;
        mbar_init_fence();
    }
    if (a.diff.norm && threadIdx.x < kD)
        ex->norm[threadIdx.x] = a.diff.norm[threadIdx.x] * (1.0f - a.diff.init);
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
    if (a.split) {   // key tiles before each unit
        for (int u = threadIdx.x; u < a.units; u += kThreads) {
            const int bh = u / a.q_tiles;
            prefix[u + 1] = unit_tiles(lens_of(a, bh / a.Hq), u - bh * a.q_tiles, a.causal);
        }
        if (threadIdx.x == 0) prefix[0] = 0;
        __syncthreads();
        if (warp == 2) {   // inclusive scan, 32 units at a time
            uint32_t run = 0;
            for (int u0 = 1; u0 <= a.units; u0 += 32) {
                uint32_t x = u0 + lane <= a.units ? prefix[u0 + lane] : 0u;
#pragma unroll
                for (int sh = 1; sh < 32; sh <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, x, sh);
                    if (lane >= sh) x += y;
                }
                x += run;
                if (u0 + lane <= a.units) prefix[u0 + lane] = x;
                run = __shfl_sync(0xffffffffu, x, 31);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (a.split && blockIdx.x == 0)
        for (int u = threadIdx.x; u <= a.units; u += kThreads) a.prefix[u] = prefix[u];
    const uint32_t tmem = ctrl->tmem_base;
    static_assert(sizeof(Items) <= kItemBytes, "a warp's place in its items");
    const WaitCtl w{a.wait_limit, a.status, &ctrl->abort};
    // Counts that run on over the items: key tiles (tc), items with any (ic).  Items without key
    // tiles concern the softmax warps alone.
    uint32_t tc = 0, ic = 0, pos = 0;   // pos: ring positions loaded (TMA warp)
    Items& items = *reinterpret_cast<Items*>(item_mem + kItemBytes * warp);
    const Item& it = items.it;
    items_begin(items, a, prefix);

    if (warp == 0) {
        // ================= TMA producer (whole warp; one elected lane issues)
        bool ok = true;
        while (ok && items_next(items, a, prefix)) {
            const int n_tiles = it.n_tiles, tile0 = it.tile0;
            if (n_tiles == 0) continue;
            const int b = it.bh / a.Hq, head = it.bh - b * a.Hq, hk = head / a.grp;
            const int qb = ic & 1;
            if (ic >= 2) ok = wait_warp(&ctrl->q_empty[qb], ((ic >> 1) - 1) & 1, w);
            if (!ok) break;
            if (a.fault != 1 && elect_one()) {
                mbar_arrive_expect_tx(&ctrl->q_full[qb], kQBytes);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    tma_load_4d(sQ + qb * kQBytes + c * kQChunk, &tmQ, &ctrl->q_full[qb], c * 64,
                                it.qt * kBM, head, b);
            }
            __syncwarp();
            ++ic;
            for (int x = 0; x < 2 * n_tiles; ++x, ++pos) {
                if (a.fault == 2 && pos >= 2 * kNS) {   // test hook: stop mid-stream, drain, leave
                    ok = false;
                    break;
                }
                const int slot = pos % kNS;
                ok = wait_warp(&ctrl->empty[slot], ((pos / kNS) & 1) ^ 1u, w);
                if (!ok) break;
                const int k0 = (tile0 + (x >> 1)) * kBN;
                const CUtensorMap* m = (x & 1) ? &tmV : &tmK;
                uint8_t* dst = sKV + slot * kSlotBytes;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&ctrl->full[slot], kSlotBytes);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tma_load_4d(dst + c * kKvChunk, m, &ctrl->full[slot], c * 64, k0, hk, b);
                }
                __syncwarp();
            }
        }
    } else if (warp == 1) {
        // ================= QK issuer.  A step's QK overwrites its map's S of the last tile as
        // soon as the softmax has that in registers.  K of tile tc sits at ring position 2 tc;
        // the previous item of its slot, K of tile tc - kNS / 2, was waited for by this warp.
        bool ok = true;
        while (ok && items_next(items, a, prefix)) {
            const int n_tiles = it.n_tiles;
            if (n_tiles == 0) continue;
            const int qb = ic & 1;
            ok = wait_warp(&ctrl->q_full[qb], (ic >> 1) & 1, w);
            ++ic;
            const uint32_t qa = smem_addr(sQ + qb * kQBytes);
            for (int t = 0; ok && t < n_tiles; ++t, ++tc) {
                const int slot = (2 * tc) % kNS;
                const uint32_t ka = smem_addr(sKV + slot * kSlotBytes);
                for (int m = 0; m < 2; ++m) {
                    if (m == 0) ok = wait_warp(&ctrl->full[slot], (2 * tc / kNS) & 1, w);
                    if (tc > 0) ok = ok && wait_warp(&ctrl->s_free[m], (tc - 1) & 1, w);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k16 = 0; k16 < 4; ++k16) {
                            mma_ss(tmem + m * kTS, sdesc_sw128(qa + m * kQChunk + k16 * 32, 16, 1024),
                                   sdesc_sw128(ka + m * kKvChunk + k16 * 32, 16, 1024), kIdescQK,
                                   k16 > 0 ? 1u : 0u);
                        }
                        mma_commit(&ctrl->s_full[m]);
                        if (m == 1) mma_commit(&ctrl->empty[slot]);
                        if (m == 1 && t + 1 == n_tiles) mma_commit(&ctrl->q_empty[qb]);
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp == kPvWarp) {
        // ================= PV issuer: waits for P of the step and, once a tile, for V
        // (ring position 2 tc + 1; the slot's previous item is V of tile tc - kNS / 2).  The first
        // PV of an item overwrites O, so it waits until the softmax has read the last item's.
        bool ok = true;
        while (ok && items_next(items, a, prefix)) {
            const int n_tiles = it.n_tiles;
            const int keys = it.n.kv < a.Skv ? it.n.kv - it.tile0 * kBN : 0x7FFFFFFF;
            if (n_tiles == 0) continue;
            if (ic > 0) ok = wait_warp(&ctrl->o_free, (ic - 1) & 1, w);
            ++ic;
            for (int t = 0; ok && t < n_tiles; ++t, ++tc) {
                const int slot = (2 * tc + 1) % kNS;
                const uint32_t va = smem_addr(sKV + slot * kSlotBytes);
                for (int m = 0; m < 2; ++m) {
                    if (m == 0) {
                        ok = wait_warp(&ctrl->full[slot], ((2 * tc + 1) / kNS) & 1, w);
                        const int live = keys - t * kBN;   // keys of the tile that exist
                        if (ok && live < kBN) {
                            // Rows past this entry's keys may hold anything, and P = 0 times
                            // a NaN is a NaN: clear them.
                            uint4* v16 = reinterpret_cast<uint4*>(sKV + slot * kSlotBytes);
                            for (int x = live * 8 + lane; x < kBN * 8; x += 32)
                                v16[x] = v16[kKvChunk / 16 + x] = make_uint4(0, 0, 0, 0);
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                        }
                    }
                    ok = ok && wait_warp(&ctrl->p_full[m], tc & 1, w);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        // hi, then lo, each 256 tensor-core cycles, the second's issue 128 cycles
                        // behind the first's: the tensor core works in order, and a QK that gets
                        // ready meanwhile goes in between (8192 x 16 heads 434 -> 420 us).
                        const long long begun = clock64();
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if (half == 1)
                                while (clock64() - begun < 128) {}
#pragma unroll
                            for (int k16 = 0; k16 < kBN / 16; ++k16)
                                mma_ts(tmem + kTO + m * 128,
                                       tmem + kTP + m * kTPMap + half * kTPLo + k16 * 8,
                                       sdesc_sw128(va + k16 * 2048, kKvChunk, 1024), kIdescPV,
                                       (t > 0 || half > 0 || k16 > 0) ? 1u : 0u);
                        }
                        if (m == 1) mma_commit(&ctrl->empty[slot]);
                        mma_commit(&ctrl->pv_done[m]);
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        // ================= softmax / correction / epilogue (warps 2..5 map 0, 6..9 map 1)
        // A thread owns one query row of one map (TMEM lane quarter = warp % 4), so nothing is
        // exchanged until the epilogue and the two maps' warps run out of step: while one map's
        // are in their exponentials, the other's load scores or wait for the tensor core.
        // The scores and both halves of P leave few registers: barriers are named by address, the
        // loop keeps only what it needs, and the epilogue works its own values out anew.
        const uint32_t bars = smem_addr(&ctrl->s_full[0]) + 8 * ((warp - 2) >> 2);   // of this map
        constexpr uint32_t kPFull = offsetof(Ctrl, p_full) - offsetof(Ctrl, s_full);
        constexpr uint32_t kPvDone = offsetof(Ctrl, pv_done) - offsetof(Ctrl, s_full);
        constexpr uint32_t kSFree = offsetof(Ctrl, s_free) - offsetof(Ctrl, s_full);
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const float sl2 = a.scale_log2;
        bool ok = true;
        while (ok && items_next(items, a, prefix)) {
        // keys >= lim, counted from the tile's first, are invisible
        int lim = visible(it.n, it.qt * kBM + (warp & 3) * 32 + lane, a.causal) - it.tile0 * kBN;
        int left = it.n_tiles;
        {
            const float lambda = diff_lambda<kD / 2>(a.diff, it.bh % a.Hq, lane);
            if (lane == 0) items.lambda = lambda;
        }
        float m_run = -INFINITY, l = 0.0f;   // the exponentials' reference (tiles.cuh) and their sum
        bool first = true;
        for (; left > 0; --left, ++tc, lim -= kBN, first = false) {
            ok = wait_warp(bars, tc & 1, w);
            if (!ok) break;
            tc_fence_after();
            uint32_t x[kBN];
#pragma unroll
            for (int c = 0; c < kBN; c += 32) tmem_ld32(tl + ((warp - 2) >> 2) * kTS + c, x + c);
            tmem_ld_wait();
            tc_fence_before();
            mbar_arrive(bars + kSFree);

            if (lim < kBN) {   // keys the row does not see
#pragma unroll
                for (int c = 0; c < kBN; ++c)
                    if (c >= lim) x[c] = __float_as_uint(-INFINITY);
            }
            // row max with four independent chains (short latency)
            float m4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = __uint_as_float(x[k]);
#pragma unroll
            for (int c = 4; c < kBN - 4; c += 8) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    m4[k] = max3f(m4[k], __uint_as_float(x[c + k]), __uint_as_float(x[c + 4 + k]));
            }
            m4[0] = max3f(m4[0], __uint_as_float(x[kBN - 4]), __uint_as_float(x[kBN - 3]));
            m4[1] = max3f(m4[1], __uint_as_float(x[kBN - 2]), __uint_as_float(x[kBN - 1]));
            const float mx = fmaxf(max3f(m4[0], m4[1], m4[2]), m4[3]);
            const float top = mx * sl2;
            const bool need = top > m_run + kTop;
            float alpha = 1.0f;
            if (need) {
                alpha = fast_exp2(m_run - (top - kShift));
                m_run = top - kShift;
            }
            const bool warp_need = __any_sync(0xffffffffu, need);
            const float m_use = m_run == -INFINITY ? 0.0f : m_run;
            const uint64_t sl2x2 = f2_pack(sl2, sl2), negm = f2_pack(-m_use, -m_use);
            // P as two FP16 halves, hi = RNE(p) and lo = RNE(p - hi), packed over the keys
            uint64_t rs[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) rs[k] = f2_pack(0.0f, 0.0f);
            uint32_t hi[kBN / 2], lo[kBN / 2];
#pragma unroll
            for (int i = 0; i < kBN / 2; ++i) {
                float x0, x1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])),
                                 sl2x2, negm),
                          x0, x1);
                const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                rs[i & 3] = f2_add(rs[i & 3], f2_pack(p0, p1));   // four independent sums
                const __half2 h = __floats2half2_rn(p0, p1);
                const float2 f = __half22float2(h);
                hi[i] = *reinterpret_cast<const uint32_t*>(&h);
                lo[i] = pack_half2(p0 - f.x, p1 - f.y);
            }
            if (!first) {   // the P buffer is free and O complete up to the last tile
                ok = wait_warp(bars + kPvDone, (tc - 1) & 1, w);
                if (!ok) break;
                tc_fence_after();
            }
            const uint32_t pbuf = tl + kTP + ((warp - 2) >> 2) * kTPMap;
            tmem_st32(pbuf, hi);
            tmem_st32(pbuf + kTPLo, lo);
            float r0, r1, r2, r3, r4, r5, r6, r7;
            f2_unpack(rs[0], r0, r1);
            f2_unpack(rs[1], r2, r3);
            f2_unpack(rs[2], r4, r5);
            f2_unpack(rs[3], r6, r7);
            l = l * alpha + (((r0 + r1) + (r2 + r3)) + ((r4 + r5) + (r6 + r7)));
            tmem_st_wait();
            if (warp_need && !first) {   // rescale the row of O
                const uint32_t obuf = tl + kTO + ((warp - 2) >> 2) * 128;
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
            mbar_arrive(bars + kPFull);
        }
        if (!ok) break;
        const bool any = it.n_tiles > 0;
        if (any) {
            ok = wait_warp(&ctrl->pv_done[0], (tc - 1) & 1, w) &&
                 wait_warp(&ctrl->pv_done[1], (tc - 1) & 1, w);
            if (!ok) break;
            tc_fence_after();
        }
        // From here a thread works on half of the columns of both maps.  Two exchanges with the
        // row's other thread, always both, so that each orders the other's reads before the next
        // writes.
        int tid;
        asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
        const int quarter = (tid >> 5) & 3, half = (tid - 64) >> 7;   // half: also the thread's map
        const int row = quarter * 32 + (tid & 31);
        uint64_t* xbar = &ctrl->xchg[quarter];
        float l2[2], mr[2];
        ex->mx[half][row] = m_run;
        ex->l[half][row] = l;
        mbar_arrive(xbar);
        ok = wait_warp(xbar, 0, w);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            l2[k] = ex->l[k][row];
            mr[k] = ex->mx[k][row];
        }
        const int rec = it.rec, row_g = it.qt * kBM + row;
        const bool row_ok = row_g < a.Sq;
        const float f0 = l2[0] == 0.0f ? 0.0f : 1.0f / l2[0];
        const float f1 = l2[1] == 0.0f ? 0.0f : -items.lambda / l2[1];
        const uint32_t o_tm = tl + kTO + half * 64;
        // O is read twice, 32 columns at a time in loops that stay rolled: the code runs once an
        // item, and unrolled over 64 columns it spent its time fetching itself.
        float sq = 0.0f;
        if (rec < 0 && a.diff.norm && any) {
#pragma unroll 1
            for (uint32_t c = 0; c < 64; c += 32) {
                uint32_t o0[32], o1[32];
                tmem_ld32(o_tm + c, o0);
                tmem_ld32(o_tm + 128 + c, o1);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float v = __uint_as_float(o0[e]) * f0 + __uint_as_float(o1[e]) * f1;
                    sq += v * v;
                }
            }
        }
        ex->sq[half][row] = sq;
        mbar_arrive(xbar);
        ok = wait_warp(xbar, 1, w);
        if (!ok) break;
        const float rn = rsqrtf((ex->sq[0][row] + ex->sq[1][row]) * (1.0f / kD) + a.diff.eps);
        const int b = it.bh / a.Hq;
        __half* op = a.o + b * a.o_sb + (it.bh - b * a.Hq) * a.o_sh + row_g * a.o_sr + half * 64;
        float* part = a.part_o + (2LL * rec * kBM + row) * kD + half * 64;
#pragma unroll 1
        for (uint32_t c = 0; c < 64; c += 32) {
            uint32_t o0[32], o1[32];
            if (any) {
                tmem_ld32(o_tm + c, o0);
                tmem_ld32(o_tm + 128 + c, o1);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o0[e] = o1[e] = 0u;
            }
            if (any && c == 32) {
                tc_fence_before();
                mbar_arrive(&ctrl->o_free);   // the next item's PV may overwrite O
            }
            if (!row_ok) continue;
            if (rec >= 0) {   // a partial record per map
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    store_f32x8(part + c + e, o0 + e);
                    store_f32x8(part + kBM * kD + c + e, o1 + e);
                }
                continue;
            }
            const float4* nw = reinterpret_cast<const float4*>(ex->norm + half * 64 + c);
            uint32_t hw[16];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                float v[4];
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    v[f] = __uint_as_float(o0[e + f]) * f0 + __uint_as_float(o1[e + f]) * f1;
                if (a.diff.norm) {
                    const float4 g = nw[e / 4];
                    v[0] *= rn * g.x;
                    v[1] *= rn * g.y;
                    v[2] *= rn * g.z;
                    v[3] *= rn * g.w;
                }
                hw[e / 2] = pack_half2(v[0], v[1]);
                hw[e / 2 + 1] = pack_half2(v[2], v[3]);
            }
            if (l2[0] + l2[1] == 0.0f) {   // sees no key; O may hold 0 times an infinite value
#pragma unroll
                for (int e = 0; e < 16; ++e) hw[e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                reinterpret_cast<uint4*>(op + c)[e] =
                    make_uint4(hw[4 * e], hw[4 * e + 1], hw[4 * e + 2], hw[4 * e + 3]);
        }
        // max and sum of map `half`
        const float mh = half ? mr[1] : mr[0], lh = half ? l2[1] : l2[0];
        if (rec >= 0)
            a.part_ml[(2LL * rec + half) * kBM + row] = make_float2(mh, lh);
        else if (row_ok && a.lse)
            a.lse[(2LL * it.bh + half) * a.Sq + row_g] =
                lh == 0.0f ? -INFINITY : (mh + log2f(lh)) * kLn2;
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*static_cast<volatile int*>(&ctrl->abort)) {
        // After an abort: copies in flight land and issued MMAs end (each waited for by its
        // own issuer) before shared and tensor memory go away.
        if (warp == 0 && lane == 0) {
            if (a.fault != 1)
                for (uint32_t i = ic > 2 ? ic - 2 : 0; i < ic; ++i)
                    drain_wait(&ctrl->q_full[i & 1], (i >> 1) & 1);
            for (uint32_t i = pos > kNS ? pos - kNS : 0; i < pos; ++i)
                drain_wait(&ctrl->full[i % kNS], (i / kNS) & 1);
        }
        if (warp == 1 || warp == kPvWarp) {
            uint64_t* bar = warp == 1 ? &ctrl->drain : &ctrl->drain_pv;
            if (elect_one()) mma_commit(bar);
            __syncwarp();
            if (lane == 0) drain_wait(bar, 0);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of a unit that the CTAs' ranges cut: one query row per warp (four columns a
// lane).  Per map M = max_c m_c, l = sum_c 2^(m_c - M) l_c, O_m = sum_c 2^(m_c - M) O_c / l, then the
// difference and the norm.  A unit inside one range was finished there; one without key tiles is
// nobody's, and its rows are written here (O = 0, lse = -inf).
__global__ void __launch_bounds__(256) attn_diff_merge_kernel(const DiffPrefillArgs a, uint32_t grid) {
    const int lane = threadIdx.x & 31;
    const int u = static_cast<int>(blockIdx.x);
    const int row = static_cast<int>(blockIdx.y) * 8 + static_cast<int>(threadIdx.x >> 5);
    const int bh = u / a.q_tiles, row_g = (u - bh * a.q_tiles) * kBM + row;
    const int b = bh / a.Hq, head = bh - b * a.Hq;
    const float lambda = diff_lambda<kD / 2>(a.diff, head, lane);
    // a programmatic dependent of the attention grid
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row_g >= a.Sq) return;
    const uint32_t U = a.prefix[a.units], u0 = a.prefix[u], u1 = a.prefix[u + 1];
    const uint32_t W = min(grid, U);
    uint32_t c0 = 0, parts = 0;   // the CTAs whose ranges meet the unit: c0 .. c0 + parts - 1
    long long rec0 = 0;           // the first one's record; CTA c's is 2 c for the others
    if (u1 > u0) {
        c0 = warp_of(u0, W, U);
        parts = warp_of(u1 - 1, W, U) - c0 + 1;
        if (parts == 1) return;
        rec0 = 2LL * c0 + (warp_start(c0, W, U) < u0 ? 1 : 0);
    }
    auto at_of = [&](uint32_t i, int m) -> long long {   // row of part i, map m
        const long long rec = i == 0 ? rec0 : 2LL * (c0 + i);
        return (rec * 2 + m) * kBM + row;
    };
    float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.0f, 0.0f};
    float acc[2][4] = {};
    // 32 parts at a time, their (max, sum) one a lane
    for (uint32_t i0 = 0; i0 < parts; i0 += 32) {
        const uint32_t n = min(32u, parts - i0);
        float wt[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float2 ml = make_float2(-INFINITY, 0.0f);
            if (lane < n) ml = a.part_ml[at_of(i0 + lane, m)];
            float mx = fmaxf(M[m], ml.x);
#pragma unroll
            for (int sh = 16; sh > 0; sh >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
            const float keep = M[m] == -INFINITY ? 0.0f : exp2f(M[m] - mx);
            M[m] = mx;
            wt[m] = ml.y == 0.0f ? 0.0f : (ml.x == -INFINITY ? 1.0f : exp2f(ml.x - mx));
            L[m] = L[m] * keep + warp_sum(wt[m] * ml.y);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][e] *= keep;
        }
#pragma unroll 4
        for (uint32_t i = 0; i < n; ++i) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float w = __shfl_sync(0xffffffffu, wt[m], i);
                if (w == 0.0f) continue;   // a part in which the row saw nothing holds no O
                const float4 v = *reinterpret_cast<const float4*>(a.part_o + at_of(i0 + i, m) * kD + lane * 4);
                acc[m][0] += w * v.x;
                acc[m][1] += w * v.y;
                acc[m][2] += w * v.z;
                acc[m][3] += w * v.w;
            }
        }
    }
    float out[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const float f = L[m] == 0.0f ? 0.0f : (m == 0 ? 1.0f : -lambda) / L[m];
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] += acc[m][e] * f;
        if (a.lse && lane == 0)
            a.lse[(static_cast<long long>(bh) * 2 + m) * a.Sq + row_g] =
                L[m] == 0.0f ? -INFINITY : (M[m] + log2f(L[m])) * kLn2;
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

// Whether to split the keys, by the time of both ways in key tiles per CTA (0.95 to 1.0 us each): whole
// units cost their rounds (at least the longest unit) and about 6 tiles for the start and the ends; a
// split costs an even share and about 30 tiles for its start, the records and the merge.  Measured,
// whole against split: 16 heads, 500 queries on 32,500 keys 522 and 240 us; 8 heads, 128 on 4,000 59
// and 23 us; 16 heads, 1,024 on 9,000 124 and 124 us; 32 heads, 512 on 8,192 113 and 117 us; 8 heads
// x 4,096 causal 61 and 99 us.
bool split_pays(long long units, int Sq, int Skv, int sms) {
    const int longest = (Skv + kBN - 1) / kBN;
    if (units > kMaxUnits || units * longest > 0x7FFFFFFFLL) return false;
    // a causal launch's mean; without the mask whole units cost at least as much more
    const double mean = longest - (Sq < Skv ? Sq : Skv) / (2.0 * kBN);
    const double rounds = static_cast<double>((units + sms - 1) / sms);
    const double whole = rounds * mean > longest ? rounds * mean : longest;
    return units * mean / sms + 30 < whole + 6;
}

// Workspace of a split launch: two records per CTA and the units' tile prefix.
size_t split_workspace(long long ctas) {
    return static_cast<size_t>(2 * ctas) * record_bytes() + 4 * (kMaxUnits + 1);
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
    const int sms = sm_count_or_default();
    return split_pays(units, Sq, Skv, sms) ? split_workspace(sms) : 0;
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
    const int sms = sm_count_or_default();
    const bool split = workspace && workspace_bytes >= split_workspace(sms) &&
                       split_pays(units, Sq, Skv, sms);
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
                         {workspace, split ? split_workspace(sms) : 0}};
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
    a.units = static_cast<int>(units);
    a.q_tiles = q_tiles;
    a.split = split ? 1 : 0;
    a.q_lens = q_lens;
    a.kv_lens = kv_lens;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.o = static_cast<__half*>(o);
    a.o_sb = os.b;
    a.o_sh = os.h;
    a.o_sr = os.r;
    a.lse = lse;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(2 * sms) * 2 * kBM * kD);
    a.prefix = reinterpret_cast<uint32_t*>(a.part_ml + static_cast<size_t>(2 * sms) * 2 * kBM);
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
    const unsigned grid = static_cast<unsigned>(split || units > sms ? sms : units);
    attn_diff_kernel<<<grid, kThreads, kSmemBytes, s>>>(tq, tk, tv, a);
    count_launches(1);
    rc = launch_status();
    if (rc != GBATTN_OK || !split) return rc;
    // The merge's CTAs may be placed as attention CTAs retire; they wait for the whole grid.
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(units), kBM / 8);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_diff_merge_kernel, a, grid);
    count_launches(1);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GBATTN_ERR_CUDA;
    }
    return launch_status();
}
