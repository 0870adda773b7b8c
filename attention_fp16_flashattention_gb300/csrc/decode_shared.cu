// Decode attention over a paged FP16 KV cache for a batch whose requests share prefixes: the sequences of a
// group have their first tokens' pages in common, and those are read once for all of them.  Over its
// own tokens every sequence is decoded as in decode_f16.cu ("Integrate FP32 v37 prefill and exact E4M3 bridge",
// Validation: decode of long caches with shared-KV heads; prefixes in common have no counterpart there).
//
// Mathematics.  Query row r of a sequence sees the prefix's tokens t < p and its own behind them; softmax over
// both is the join of two partial (max, sum, O) with one exponential each.  Over the prefix all rows of all
// sequences of the group meet the same keys, so for a KV head they are one matrix Q [rows][D], and
// S = Q K^T and O = P V are matrix products with 4 D FLOPs per row and 4 D bytes per token: above some 190 rows
// (with P in two halves) the tensor cores bound it, below them the bytes.
//
// One grid, one CTA per SM, and two kinds of work, so that the one's memory time runs beside the other's
// arithmetic.  Every CTA works out the same tile counts from the lengths (a few loads, two scans): `prefix_split`
// of them share the prefixes' tiles evenly, the others the own tokens' (decode_f16_body), each a contiguous
// range of tiles laid end to end.  A merge kernel joins the records of both.
//
// The prefix CTAs.  A unit is 256 query rows of one KV head and group (128 at D = 256); its prefix goes by in
// tiles of 64 tokens, and a step is 128 rows against a tile.  Warp roles:
//   warp 0     TMA producer: K_0, V_0, K_1, V_1, ... through a ring, the pages looked up 32 boxes at a time.
//   warp 1     allocates tensor memory and issues S = Q K^T (tcgen05, 128 x 64 x D); a buffer is handed back as soon as
//              the softmax has it in registers.
//   last warp  issues O += hi V + lo V (P from tensor memory).
//   the others softmax: one thread per query row (TMEM lane).  D <= 128: two sets of four warps take the steps in
//              turn, each with its own running max, sum and O, so that a step's exponentials run beside the
//              next one's.  With more than 128 rows the sets are the unit's two halves and share every
//              tile; with fewer they take its tiles in turn and are joined at its end.  D = 256: O fills half of the
//              tensor memory and there is one set; a tile's bytes take as long as its softmax.
// P = hi + lo in FP16 as everywhere in the decode (decode_f16.cu).  Tensor memory: S and P (hi, lo) of 64 columns
// a buffer, one for each set, O of D columns a set, and at D = 256 Q in its 128, so that the 64 KB that it would
// take of the shared memory hold another tile under way.
//
// Measured (graph replays): 64 sequences behind 16,384 tokens with 100 to 2,001 of their own, 32 on 8 heads of 128
// (351 MB; 67 of them the prefix) 71 to 76 us, where the ordinary decode, to which that is 4.6 GB, takes 345; at D = 64 48;
// 8 behind 131,072 (32 rows a KV head) 91 to 99 us, 0.80 to 0.87 of the measured copy; 64 behind as many (256 rows) 147 to 156 us,
// 880 to 935 TFLOP/s without the lo halves, a step of 128 rows and 64 tokens in 1,030 cycles of which the tensor pipe has 900
// to do.  8 behind 1,024 with up to 300 of their own in the form for short caches 10.7 us (the ordinary decode 10.5).
//
// Against the ordinary decode (one group with up to 300 own tokens each; this call's time first): the form for short
// caches costs 0.2 to 0.7 us for the groups.  Beyond it, 32 on 8 heads of 128: 16 sequences behind 1,024 tokens 16.9 and
// 17.2 us, 4 behind 4,096 16.2 and 16.8, 2 15.1 and 12.7; 6 on 1 of 256: 32 behind 1,024 15.8 and 16.4, 4 behind 4,096
// 13.5 and 14.3, 2 13.2 and 12.4.  Prefixes of a tile or two are better read with the sequences' own tokens: 32 sequences
// behind 64 on 8 heads of 128 36 and 15 us, since few CTAs then take several units each, one after the other.
//
// Every wait is bounded in time (WaitCtl): one that runs out records GBATTN_DEV_WAIT_TIMEOUT, the CTA stops,
// waits a bounded time for its copies and MMAs in flight, frees tensor memory and exits.
#include <cstddef>

#include "decode_f16.cuh"

namespace gbattn {
namespace {

constexpr uint64_t kDrainNs = 200000000ull;   // 0.2 s for draining after an abort
// Tensor memory columns: S (64 a buffer), P (32 of hi, 32 of lo a buffer), Q where it is kept there, O.
constexpr uint32_t kTBuf = 64, kTPLo = 32, kTO = 256;

template <int D>
struct Pre {
    static constexpr int kSets = D == 256 ? 1 : 2;
    static constexpr int kBufs = kSets;                            // S and P buffers
    static constexpr bool kQTmem = D == 256;                       // Q in tensor memory
    static constexpr uint32_t kTP = kBufs * kTBuf;                 // tensor memory columns of P and, behind it, Q
    static constexpr int kThreads = 32 * (3 + 4 * kSets);
    static constexpr int kPvWarp = 2 + 4 * kSets;
    static constexpr int kChunks = D / 64;                         // 64-column chunks of a row
    static constexpr int kQTile = kStepRows * D * 2;
    static constexpr int kQBytes = kQTmem ? 0 : kSets * kQTile;
    static constexpr int kSlot = kPreTile * D * 2;                 // a K or V tile
    static constexpr int kNS = D == 256 ? 6 : D == 128 ? 8 : 20;   // ring slots (even: K, odd: V)
    static constexpr int kQChunk = kStepRows * 128, kKvChunk = kPreTile * 128;
    static constexpr uint32_t kIdescQK = idesc_f16(kStepRows, kPreTile, false, false);
    static constexpr uint32_t kIdescPV = idesc_f16(kStepRows, D, false, true);
};

constexpr int kMaxSlots = 20;
struct Ctrl {
    uint64_t q_full;
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t s_full[2];    // S buffer computed
    uint64_t s_free[2];    // and read into registers
    uint64_t p_full[2];    // P buffer written
    uint64_t pv_done[2];   // its PV done: the buffer is free, its O up to date
    uint64_t o_free;       // a unit's O read into registers
    uint64_t xchg[4];      // per row quarter: the two threads of a row exchange max and sum
    uint64_t drain, drain_pv;
    uint32_t tmem_base;
    int abort;
};
struct Exchange {   // the two sets' (reference, sum) of a row
    float m[2][kStepRows], l[2][kStepRows];
};

// Shared memory: the role's own part, then two tables: the tile prefix over groups or, in a CTA of the own
// tokens, over sequences; and every sequence's prefix length, which a prefix CTA has no use for and puts the
// sets' exchange there.
constexpr int kTable = 4 * (kMaxSeqs + 4);
constexpr int kCtrlBytes = (static_cast<int>(sizeof(Ctrl)) + 15) / 16 * 16;
template <int D>
struct Smem {
    static constexpr int kOwn = Cfg<D>::kRing + Cfg<D>::kBarBytes;
    static constexpr int kPre = Pre<D>::kQBytes + Pre<D>::kNS * Pre<D>::kSlot + kCtrlBytes;
    static_assert(Pre<D>::kNS <= kMaxSlots && Pre<D>::kNS % 2 == 0 && sizeof(Exchange) <= kTable, "prefix role");
    static constexpr int kRole = ((kOwn > kPre ? kOwn : kPre) + 15) / 16 * 16;
    static constexpr int kBytes = kRole + 2 * kTable + 1024;
    static_assert(kBytes <= 232448 - 1200, "shared memory of a CTA, beside its static variables");
};

struct SharedArgs {
    DecodeF16Args dec;
    const int32_t *starts, *prefix_lens;   // [groups + 1], [groups]
    float* pre_o;                          // PrefixRecords
    float2* pre_ml;
    uint32_t* work_out;
    int2* seq_out;
    uint32_t* total_out;
    int groups, max_prefix, max_own, box_rows, box_bits;
    int cap;                               // slots of a page-table row
};

// Exclusive sums over the block; `all` gets the total.  One barrier before and one inside.
template <int kThreads>
__device__ __forceinline__ uint32_t block_sum(uint32_t x, uint32_t& all) {
    __shared__ uint32_t s_sum[kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t incl = x;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, sh);
        if (lane >= sh) incl += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    uint32_t run = incl - x;
    all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) run += s_sum[w];
        all += s_sum[w];
    }
    return run;
}

// A shared-memory descriptor `bytes` further on: only the address field changes, and within 32 bits.  (Made anew
// for every MMA, the descriptors took as long as the MMAs: behind 131,072 tokens 256 rows on each of 8 KV heads took 170 us
// and so 155, 512 on each of 4 167 and 150.)
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, int bytes) {
    return (desc & 0xFFFFFFFF00000000ull) | (static_cast<uint32_t>(desc) + static_cast<uint32_t>(bytes >> 4));
}

// Bounded wait that ignores the abort flag (used only to drain after an abort).
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > kDrainNs) return;
    }
}

__device__ __forceinline__ void store_f32x8(float* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// 32 columns of each of the warp's 32 rows (a lane a row, at `out`, where live): by way of `stage` in shared memory,
// so that a store writes whole lines of four rows and not a sector of 32.  Without a stage (Q in tensor memory) a
// lane stores its own.
constexpr int kStageBytes = 32 * 32 * 4;
template <int D>
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint32_t (&o)[32], float* out, bool live, int lane) {
    if constexpr (Pre<D>::kQTmem) {
        if (live) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) store_f32x8(out + e, o + e);
        }
        __syncwarp();
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)   // 16-byte pieces, exchanged within the row so that eight lanes meet all banks
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        __syncwarp();
        const long long to = live ? reinterpret_cast<long long>(out) : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3), e = lane & 7;
            const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((e ^ (r & 7)) << 4));
            float* row = reinterpret_cast<float*>(__shfl_sync(0xffffffffu, to, r));
            if (row) *reinterpret_cast<uint4*>(row + 4 * e) = v;
        }
        __syncwarp();
    }
}

// A part of a unit: steps [s0, s1) of it, for rows row0 .. of KV head hk of group g.
struct Part {
    int hk, row0, rows;   // rows: of the group and KV head, in all
    int first, prefix;    // the group's first sequence, its prefix's tokens
    int pair;             // 1: two steps a tile
    int s0, s1;
    __device__ __forceinline__ int tile_of(int step) const { return step >> pair; }
    __device__ __forceinline__ int tile0() const { return s0 >> pair; }
    __device__ __forceinline__ int tiles() const { return ((s1 - 1) >> pair) - (s0 >> pair) + 1; }
};
// The part that begins with step `pos` of a range that ends before `end`; pos moves behind it.
template <int D>
__device__ __forceinline__ Part next_part(const SharedArgs& a, const uint32_t* work, uint32_t& pos, uint32_t end) {
    int lo = 0, hi = a.groups - 1;   // the last group whose steps begin at or before pos
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (work[mid] <= pos) lo = mid; else hi = mid - 1;
    }
    constexpr uint32_t kPer = Unit<D>::kRows / kStepRows;   // steps a tile of a full unit
    Part p;
    p.first = a.starts[lo];
    p.prefix = a.prefix_lens[lo];
    p.rows = (a.starts[lo + 1] - p.first) * a.dec.G;
    const uint32_t T = (p.prefix + kPreTile - 1) / kPreTile, per_tile = steps_of_rows(p.rows);
    const uint32_t off = pos - work[lo];
    p.hk = static_cast<int>(off / (per_tile * T));
    const uint32_t in_head = off - p.hk * (per_tile * T), unit = in_head / (kPer * T);
    const uint32_t per = min(per_tile - unit * kPer, kPer);
    p.pair = per == 2;
    p.row0 = static_cast<int>(unit * Unit<D>::kRows);
    p.s0 = static_cast<int>(in_head - unit * kPer * T);
    p.s1 = static_cast<int>(min(per * T, p.s0 + (end - pos)));
    pos += p.s1 - p.s0;
    return p;
}

template <int D>
__device__ __forceinline__ void prefix_body(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& a,
                                            uint8_t* smem, const uint32_t* work, Exchange* ex,
                                            uint32_t cta, const PreSplit& split) {
    using C = Pre<D>;
    uint8_t* sQ = smem;
    uint8_t* sKV = smem + C::kQBytes;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(sKV + C::kNS * C::kSlot);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const DecodeF16Args& d = a.dec;
    if (threadIdx.x == 0) {
        mbar_init(&ctrl->q_full, 128 * C::kSets);
        for (int i = 0; i < C::kNS; ++i) {
            mbar_init(&ctrl->full[i], 1);
            mbar_init(&ctrl->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctrl->s_full[i], 1);
            mbar_init(&ctrl->s_free[i], 128);
            mbar_init(&ctrl->p_full[i], 128);
            mbar_init(&ctrl->pv_done[i], 1);
        }
        mbar_init(&ctrl->o_free, 128 * C::kSets);
        for (int i = 0; i < 4; ++i) mbar_init(&ctrl->xchg[i], 64);
        mbar_init(&ctrl->drain, 1);
        mbar_init(&ctrl->drain_pv, 1);
        ctrl->abort = 0;
        mbar_init_fence();
    }
    if (warp == 1) {
        tmem_alloc(&ctrl->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctrl->tmem_base;
    const WaitCtl w{d.wait_limit, d.status, &ctrl->abort};
    const uint32_t end = min(warp_start(cta + 1, split.ctas, split.total), work[a.groups]);
    uint32_t pos = warp_start(cta, split.ctas, split.total);
    // Counts over all parts: steps (sc; its parity is the S and P buffer and, with two, the set), tiles (tc), parts
    // (ic), ring places.
    uint32_t sc = 0, tc = 0, ic = 0, ring = 0;

    if (warp == 0) {
        // ================= TMA producer
        const int bpt = kPreTile >> a.box_bits;   // boxes of a tile, at most 4
        bool ok = d.fault != 1;                   // test hook
        while (ok && pos < end) {
            const Part p = next_part<D>(a, work, pos, end);
            const int tile0 = p.tile0(), n_tiles = p.tiles();
            const int32_t* row = d.table + static_cast<long long>(p.first) * d.max_pages;
            const int boxes = (p.prefix + a.box_rows - 1) >> a.box_bits;
            // the cache row of box 32 c + lane
            auto look_up = [&](int c) -> int {
                const int box = 32 * c + lane;
                if (box >= boxes || box >= (tile0 + n_tiles) * bpt || 32 * c + 31 < tile0 * bpt) return 0;
                const int tok = box << a.box_bits;
                int page = row[tok / d.ps];
                if (page < 0 || page >= d.num_phys) {
                    atomicOr(d.status, kDevBadPage);
                    page = 0;
                }
                return page * d.ps + tok % d.ps;
            };
            int c = tile0 * bpt >> 5, cur = look_up(c), next = look_up(c + 1);
            for (int x = 0; x < 2 * n_tiles; ++x, ++ring) {
                if (d.fault == 2 && ring >= 2 * C::kNS) {   // test hook: stop mid-stream, drain, leave
                    ok = false;
                    break;
                }
                const int slot = ring % C::kNS;
                ok = wait_warp(&ctrl->empty[slot], ((ring / C::kNS) & 1) ^ 1u, w);
                if (!ok) break;
                const int box0 = (tile0 + (x >> 1)) * bpt;
                if (box0 >> 5 != c) {
                    ++c;
                    cur = next;
                    next = look_up(c + 1);
                }
                const int n = min(bpt, boxes - box0);
                int src[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) src[j] = __shfl_sync(0xffffffffu, cur, (box0 + j) & 31);
                const CUtensorMap* m = (x & 1) ? &tv : &tk;
                uint8_t* dst = sKV + slot * C::kSlot;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&ctrl->full[slot], n * a.box_rows * (D * 2));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= n) break;
#pragma unroll
                        for (int ch = 0; ch < C::kChunks; ++ch)
                            tma_load_3d(dst + ch * C::kKvChunk + j * a.box_rows * 128, m, &ctrl->full[slot],
                                        64 * ch, p.hk, src[j]);
                    }
                }
                __syncwarp();
            }
        }
    } else if (warp == 1) {
        // ================= QK issuer: K of tile tc sits at ring place 2 tc
        bool ok = true;
        for (; ok && pos < end; ++ic) {
            const Part p = next_part<D>(a, work, pos, end);
            ok = wait_warp(&ctrl->q_full, ic & 1, w);
            if constexpr (C::kQTmem) tc_fence_after();
            for (int s = p.s0; ok && s < p.s1; ++s, ++sc) {
                const int slot = (2 * tc) % C::kNS, buf = sc % C::kBufs;
                if (s == p.s0 || !p.pair || !(s & 1)) ok = wait_warp(&ctrl->full[slot], (2 * tc / C::kNS) & 1, w);
                if (sc >= C::kBufs) ok = ok && wait_warp(&ctrl->s_free[buf], (sc / C::kBufs - 1) & 1, w);
                if (!ok) break;
                const bool last = s + 1 == p.s1 || !p.pair || (s & 1);   // of the tile, here
                const uint64_t qd = sdesc_sw128(smem_addr(sQ + (p.pair ? buf : 0) * C::kQTile), 16, 1024);
                const uint64_t kd = sdesc_sw128(smem_addr(sKV + slot * C::kSlot), 16, 1024);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k16 = 0; k16 < D / 16; ++k16) {
                        const uint64_t k = desc_at(kd, (k16 >> 2) * C::kKvChunk + (k16 & 3) * 32);
                        if constexpr (C::kQTmem)
                            mma_ts(tmem + buf * kTBuf, tmem + 2 * C::kTP + k16 * 8, k, C::kIdescQK, k16 > 0 ? 1u : 0u);
                        else
                            mma_ss(tmem + buf * kTBuf, desc_at(qd, (k16 >> 2) * C::kQChunk + (k16 & 3) * 32), k,
                                   C::kIdescQK, k16 > 0 ? 1u : 0u);
                    }
                    mma_commit(&ctrl->s_full[buf]);
                    if (last) mma_commit(&ctrl->empty[slot]);
                }
                __syncwarp();
                tc += last;
            }
        }
    } else if (warp == C::kPvWarp) {
        // ================= PV issuer: V of tile tc sits at ring place 2 tc + 1.  A part's first PV into an O
        // overwrites it, so the softmax must have read the last part's.
        bool ok = true;
        for (; ok && pos < end; ++ic) {
            const Part p = next_part<D>(a, work, pos, end);
            if (ic > 0) ok = wait_warp(&ctrl->o_free, (ic - 1) & 1, w);
            for (int s = p.s0; ok && s < p.s1; ++s, ++sc) {
                const int slot = (2 * tc + 1) % C::kNS, buf = sc % C::kBufs;
                const uint64_t vd = sdesc_sw128(smem_addr(sKV + slot * C::kSlot), C::kKvChunk, 1024);
                if (s == p.s0 || !p.pair || !(s & 1)) {
                    ok = wait_warp(&ctrl->full[slot], ((2 * tc + 1) / C::kNS) & 1, w);
                    if (!ok) break;
                    const int live = p.prefix - p.tile_of(s) * kPreTile;
                    if (live < kPreTile) {
                        // Rows past the prefix were not loaded and may hold anything; P = 0 times a NaN is one.
                        uint4* v16 = reinterpret_cast<uint4*>(sKV + slot * C::kSlot);
                        for (int x = live * 8 + lane; x < kPreTile * 8; x += 32) {
#pragma unroll
                            for (int ch = 0; ch < C::kChunks; ++ch)
                                v16[ch * (C::kKvChunk / 16) + x] = make_uint4(0, 0, 0, 0);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                }
                ok = wait_warp(&ctrl->p_full[buf], (sc / C::kBufs) & 1, w);
                if (!ok) break;
                tc_fence_after();
                const bool last = s + 1 == p.s1 || !p.pair || (s & 1);
                const uint32_t o = tmem + kTO + (C::kSets == 2 ? buf * D : 0);
                const bool begun = s - p.s0 >= C::kSets;   // this O holds a step of the part
                if (elect_one()) {
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int k16 = 0; k16 < kPreTile / 16; ++k16)
                            mma_ts(o, tmem + C::kTP + buf * kTBuf + half * kTPLo + k16 * 8,
                                   desc_at(vd, k16 * 2048), C::kIdescPV,
                                   (begun || half > 0 || k16 > 0) ? 1u : 0u);
                    if (last) mma_commit(&ctrl->empty[slot]);
                    mma_commit(&ctrl->pv_done[buf]);
                }
                __syncwarp();
                tc += last;
            }
        }
    } else {
        // ================= softmax: set (warp - 2) / 4, TMEM lane quarter warp % 4, a thread per query row
        const int set = C::kSets == 2 ? (warp - 2) >> 2 : 0;
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        uint32_t xc = 0;   // exchanges between the sets
        bool ok = true;
        for (; ok && pos < end; ++ic) {
            const Part p = next_part<D>(a, work, pos, end);
            // The unit's half that the set's steps are of: the buffers' order runs on over the parts.
            const int half = p.pair ? set ^ static_cast<int>((sc ^ p.s0) & 1) : 0;
            const int gr = p.row0 + half * kStepRows + row;          // the row among its KV head's of the group
            const bool live = gr < p.rows;
            const bool warp_live = p.row0 + half * kStepRows + quarter * 32 < p.rows;
            // Q of the part.  The last part's products with the old one are done (its epilogue waited for them); that
            // its rows no longer pass through the Q tiles has to be waited for.
            if (!C::kQTmem && ic > 0) ok = wait_warp(&ctrl->o_free, (ic - 1) & 1, w);
            if (!ok) break;
            int lim = 0;   // the row sees prefix tokens t < lim
            {
                const int member = gr / d.G, rem = gr - member * d.G, b = p.first + member;
                const int len = live ? d.kv_lens[b] : 0;   // under way beside Q
                const __half* q = d.q + ((static_cast<long long>(b) * d.Hkv + p.hk) * d.G + rem) * D;
                if constexpr (C::kQTmem) {
#pragma unroll 2
                    for (int ch = 0; ch < C::kChunks; ++ch) {
                        uint32_t v[32];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint4 x = live ? reinterpret_cast<const uint4*>(q + ch * 64)[e] : make_uint4(0, 0, 0, 0);
                            v[4 * e] = x.x;
                            v[4 * e + 1] = x.y;
                            v[4 * e + 2] = x.z;
                            v[4 * e + 3] = x.w;
                        }
                        tmem_st32(tl + 2 * C::kTP + ch * 32, v);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                } else if (p.pair) {
                    // The warp's 32 rows, kRowLanes lanes a row, so that a load takes whole lines (a thread a row takes
                    // 32 lines a load).
                    constexpr int kRowLanes = D / 8, kAt = 32 / kRowLanes;
                    uint8_t* dst = sQ + set * C::kQTile;
                    const int c16 = lane % kRowLanes;
                    const long long at = live ? q - d.q : -1;
#pragma unroll 1
                    for (int i = 0; i < 32; i += 8 * kAt) {
                        uint4 v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const long long from = __shfl_sync(0xffffffffu, at, i + e * kAt + lane / kRowLanes);
                            v[e] = make_uint4(0, 0, 0, 0);
                            if (from >= 0) v[e] = reinterpret_cast<const uint4*>(d.q + from)[c16];
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int qrow = quarter * 32 + i + e * kAt + lane / kRowLanes;
                            *reinterpret_cast<uint4*>(dst + (c16 >> 3) * C::kQChunk + qrow * 128 +
                                                      (((c16 & 7) ^ (qrow & 7)) << 4)) = v[e];
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                } else {
                    // Two sets on the same rows, often few of them: a thread a row, half of the row's pieces.
                    constexpr int kPieces = D / 16;
                    uint4 v[kPieces];
#pragma unroll
                    for (int e = 0; e < kPieces; ++e)
                        v[e] = live ? reinterpret_cast<const uint4*>(q)[set * kPieces + e] : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < kPieces; ++e) {
                        const int c16 = set * kPieces + e;
                        *reinterpret_cast<uint4*>(sQ + (c16 >> 3) * C::kQChunk + row * 128 +
                                                  (((c16 & 7) ^ (row & 7)) << 4)) = v[e];
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                if (live) {
                    const int own = len - p.prefix;   // (outside [0, max_own]: the merge drops the row)
                    if (own >= 0 && own <= a.max_own) lim = min(p.prefix, p.prefix + own - d.nq + rem % d.nq + 1);
                }
            }
            mbar_arrive(&ctrl->q_full);
            float m_run = -INFINITY, l = 0.0f;   // the exponentials' reference (tiles.cuh) and their sum
            bool first = true;
            for (int s = p.s0; s < p.s1; ++s, ++sc) {
                const int buf = sc % C::kBufs;
                if (C::kSets == 2 && buf != set) continue;
                ok = wait_warp(&ctrl->s_full[buf], (sc / C::kBufs) & 1, w);
                if (!ok) break;
                tc_fence_after();
                float alpha = 1.0f;
                bool warp_need = false;
                uint32_t hi[kPreTile / 2], lo[kPreTile / 2];
                if (warp_live) {
                    uint32_t x[kPreTile];
#pragma unroll
                    for (int c = 0; c < kPreTile; c += 32) tmem_ld32(tl + buf * kTBuf + c, x + c);
                    tmem_ld_wait();
                    tc_fence_before();
                    mbar_arrive(&ctrl->s_free[buf]);
                    const int seen = lim - p.tile_of(s) * kPreTile;
                    if (seen < kPreTile) {
#pragma unroll
                        for (int c = 0; c < kPreTile; ++c)
                            if (c >= seen) x[c] = __float_as_uint(-INFINITY);
                    }
                    float m4[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) m4[k] = __uint_as_float(x[k]);
#pragma unroll
                    for (int c = 4; c < kPreTile - 4; c += 8) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            m4[k] = max3f(m4[k], __uint_as_float(x[c + k]), __uint_as_float(x[c + 4 + k]));
                    }
                    m4[0] = max3f(m4[0], __uint_as_float(x[kPreTile - 4]), __uint_as_float(x[kPreTile - 3]));
                    m4[1] = max3f(m4[1], __uint_as_float(x[kPreTile - 2]), __uint_as_float(x[kPreTile - 1]));
                    const float top = fmaxf(max3f(m4[0], m4[1], m4[2]), m4[3]) * d.sl2;
                    const bool need = top > m_run + kTop;
                    if (need) {
                        alpha = fast_exp2(m_run - (top - kShift));
                        m_run = top - kShift;
                    }
                    warp_need = __any_sync(0xffffffffu, need);
                    const float m_use = m_run == -INFINITY ? 0.0f : m_run;
                    const uint64_t sl2x2 = f2_pack(d.sl2, d.sl2), negm = f2_pack(-m_use, -m_use);
                    uint64_t rs[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) rs[k] = f2_pack(0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < kPreTile / 2; ++i) {
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), sl2x2,
                                         negm),
                                  x0, x1);
                        const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                        rs[i & 3] = f2_add(rs[i & 3], f2_pack(p0, p1));
                        const __half2 h = __floats2half2_rn(p0, p1);
                        const float2 f = __half22float2(h);
                        hi[i] = *reinterpret_cast<const uint32_t*>(&h);
                        lo[i] = pack_half2(p0 - f.x, p1 - f.y);
                    }
                    float r0, r1, r2, r3, r4, r5, r6, r7;
                    f2_unpack(rs[0], r0, r1);
                    f2_unpack(rs[1], r2, r3);
                    f2_unpack(rs[2], r4, r5);
                    f2_unpack(rs[3], r6, r7);
                    l = l * alpha + (((r0 + r1) + (r2 + r3)) + ((r4 + r5) + (r6 + r7)));
                } else {
                    tc_fence_before();
                    mbar_arrive(&ctrl->s_free[buf]);
                }
                // the P buffer is free and its O up to date
                if (sc >= C::kBufs) ok = wait_warp(&ctrl->pv_done[buf], (sc / C::kBufs - 1) & 1, w);
                if (!ok) break;
                tc_fence_after();
                if (warp_live) {
                    const uint32_t pbuf = tl + C::kTP + buf * kTBuf;
                    tmem_st32(pbuf, hi);
                    tmem_st32(pbuf + kTPLo, lo);
                    tmem_st_wait();
                    if (warp_need && !first) {   // rescale the row of O
                        const uint32_t obuf = tl + kTO + set * D;
                        const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
                        for (int cc = 0; cc < D / 32; ++cc) {
                            uint32_t o[32];
                            tmem_ld32(obuf + cc * 32, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float y0, y1;
                                f2_unpack(f2_mul(f2_pack(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])),
                                                 a2),
                                          y0, y1);
                                o[2 * e] = __float_as_uint(y0);
                                o[2 * e + 1] = __float_as_uint(y1);
                            }
                            tmem_st32(obuf + cc * 32, o);
                        }
                        tmem_st_wait();
                    }
                }
                first = false;
                tc_fence_before();
                mbar_arrive(&ctrl->p_full[buf]);
            }
            if (!ok) break;
            // ---- the part's record: unnormalised O, reference and sum
            // (first the last step but one: the other set's barrier has then left the phase before its
            // last step's, which a wait for that would otherwise take for it)
            if (C::kBufs == 2 && sc >= 2) ok = wait_warp(&ctrl->pv_done[sc & 1], ((sc - 2) >> 1) & 1, w);
            ok = ok && wait_warp(&ctrl->pv_done[(sc - 1) % C::kBufs], ((sc - 1) / C::kBufs) & 1, w);
            if (!ok) break;
            tc_fence_after();
            const long long rec = static_cast<long long>(cta) * Unit<D>::kRows +
                                  static_cast<long long>(p.first) * d.Hq * d.nq +
                                  static_cast<long long>(p.hk) * p.rows + gr;
            if (C::kSets == 2 && !p.pair) {
                ex->m[set][row] = m_run;
                ex->l[set][row] = l;
                mbar_arrive(&ctrl->xchg[quarter]);
                ok = wait_warp(&ctrl->xchg[quarter], xc & 1, w);
                ++xc;
                if (!ok) break;
                const float2 ml0 = make_float2(ex->m[0][row], ex->l[0][row]);
                const float2 ml1 = make_float2(ex->m[1][row], ex->l[1][row]);
                const float M = fmaxf(ml0.x, ml1.x);
                const bool any0 = ml0.y != 0.0f, any1 = ml1.y != 0.0f;   // (a set without a step has no O)
                const float f0 = record_weight(ml0, M), f1 = record_weight(ml1, M);
                constexpr int kCols = D / 2;   // a thread joins half of the columns
                const uint32_t o_tm = tl + kTO + set * kCols;
#pragma unroll 1
                for (int c = 0; c < kCols; c += 32) {
                    uint32_t o0[32], o1[32];
                    tmem_ld32(o_tm + c, o0);
                    tmem_ld32(o_tm + D + c, o1);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o0[e] = __float_as_uint((any0 ? f0 * __uint_as_float(o0[e]) : 0.0f) +
                                                (any1 ? f1 * __uint_as_float(o1[e]) : 0.0f));
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            store_f32x8(a.pre_o + rec * D + set * kCols + c + e, o0 + e);
                    }
                    __syncwarp();
                }
                if (live && set == 0) a.pre_ml[rec] = make_float2(M, f0 * ml0.y + f1 * ml1.y);
            } else {
                // (through the warp's part of the Q tiles, which no product reads any more)
                uint8_t* stage = sQ + (warp - 2) * kStageBytes;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o0[32];
                    tmem_ld32(tl + kTO + set * D + c, o0);
                    tmem_ld_wait();
                    store_rows<D>(stage, o0, a.pre_o + rec * D + c, live, lane);
                }
                if (live) a.pre_ml[rec] = make_float2(m_run, l);   // (a sum of 0: the record holds no O)
            }
            tc_fence_before();
            mbar_arrive(&ctrl->o_free);
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*static_cast<volatile int*>(&ctrl->abort)) {
        // After an abort: copies in flight land and issued MMAs end (each waited for by its
        // own issuer) before shared and tensor memory go away.
        if (warp == 0 && lane == 0)
            for (uint32_t i = ring > C::kNS ? ring - C::kNS : 0; i < ring; ++i)
                drain_wait(&ctrl->full[i % C::kNS], (i / C::kNS) & 1);
        if (warp == 1 || warp == C::kPvWarp) {
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

// (tk, tv) have boxes of kTile rows, (pk, pv) of box_rows, both over the same pages.
template <int D, int NB>
__global__ void __launch_bounds__(Pre<D>::kThreads, 1)
    decode_shared_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                         const __grid_constant__ CUtensorMap pk, const __grid_constant__ CUtensorMap pv,
                         const SharedArgs a) {
    constexpr int kThreads = Pre<D>::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint32_t* tiles = reinterpret_cast<uint32_t*>(smem + Smem<D>::kRole);   // and the decode's abort flag behind it
    int* pre = reinterpret_cast<int*>(smem + Smem<D>::kRole + kTable);
    const DecodeF16Args& d = a.dec;
    const int tid = threadIdx.x;
    const bool lead = blockIdx.x == 0;
    if (tid == 0) {
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
        tma_prefetch_desc(&pk);
        tma_prefetch_desc(&pv);
    }
    const int my_len = d.B <= kThreads && tid < d.B ? d.kv_lens[tid] : 0;   // under way beside the groups
    // ---- steps over every group's prefix
    const int per_g = (a.groups + kThreads - 1) / kThreads;
    const int g0 = min(tid * per_g, a.groups), g1 = min(g0 + per_g, a.groups);
    __shared__ uint32_t s_shortest, s_longest;   // units
    if (tid == 0) s_shortest = 0xFFFFFFFFu, s_longest = 0;
    bool order = true;
    uint32_t sum = 0, shortest = 0xFFFFFFFFu, longest = 0;
    for (int g = g0; g < g1; ++g) {
        const int s = a.starts[g], e = a.starts[g + 1], p = a.prefix_lens[g];
        const bool in_order = s >= 0 && s <= e && e <= d.B && (g > 0 || s == 0) && (g + 1 < a.groups || e == d.B);
        const bool good = p >= 0 && p <= a.max_prefix && p % d.ps == 0;
        order = order && in_order;
        if (!good && lead) atomicOr(d.status, kDevBadLength);
        uint32_t n = 0;
        if (in_order && good)
            n = static_cast<uint32_t>(d.Hkv) * steps_of_rows((e - s) * d.G) * ((p + kPreTile - 1) / kPreTile);
        if (n > 0) {
            const uint32_t u = unit_steps<D>((e - s) * d.G, (p + kPreTile - 1) / kPreTile);
            shortest = min(shortest, u);
            longest = max(longest, u);
        }
        tiles[g] = n;
        sum += n;
    }
    order = __syncthreads_and(order);
    if (order && shortest <= longest) {   // (a group of unlike units has 0 for its length: neither may be left out)
        atomicMin(&s_shortest, shortest);
        atomicMax(&s_longest, longest);
    }
    uint32_t Up = 0;
    uint32_t run = block_sum<kThreads>(order ? sum : 0, Up);
    for (int g = g0; g < g1; ++g) {
        const uint32_t n = order ? tiles[g] : 0;
        tiles[g] = run;
        if (lead) a.work_out[g] = run;
        run += n;
    }
    if (tid == 0) {
        tiles[a.groups] = Up;
        if (lead) {
            a.work_out[a.groups] = Up;
            if (!order) atomicOr(d.status, kDevBadIndex);
        }
    }
    // ---- every sequence's prefix, and the tiles of its own tokens
    const int per_seq = d.Hkv * d.sets;
    const int per = (d.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, d.B), b1 = min(b0 + per, d.B);
    sum = 0;
    for (int b = b0; b < b1; ++b) {
        int p = -1, g = 0;
        if (order) {
            int hi = a.groups - 1;   // the last group that begins at or before b
            while (g < hi) {
                const int mid = (g + hi + 1) >> 1;
                if (a.starts[mid] <= b) g = mid; else hi = mid - 1;
            }
            p = a.prefix_lens[g];
            if (p < 0 || p > a.max_prefix || p % d.ps != 0) {
                p = -1;
            } else {
                const int n = d.B <= kThreads ? my_len : d.kv_lens[b];
                if (n < p || n - p > a.max_own || n > a.cap) {
                    p = -1;
                    if (lead) atomicOr(d.status, kDevBadLength);
                } else {
                    sum += seq_tiles(n - p, a.max_own) * static_cast<uint32_t>(per_seq);
                }
            }
        }
        pre[b] = p;
        if (lead) a.seq_out[b] = make_int2(p, g);
    }
    uint32_t own = 0;
    run = block_sum<kThreads>(sum, own);   // (its barriers also make `tiles` and `pre` whole)
    // The merge grid may start launching now; it waits for this grid to finish.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const PreSplit split = prefix_split<D>(gridDim.x, Up, own, s_shortest == s_longest ? s_longest : 0u, 8 * NB);
    const uint32_t P = split.ctas;
    if (lead && tid == 0) {
        a.total_out[0] = own;
        a.total_out[1] = split.ctas;
        a.total_out[2] = split.total;
    }
    if (blockIdx.x < P) {
        prefix_body<D>(pk, pv, a, smem, tiles, reinterpret_cast<Exchange*>(pre), blockIdx.x, split);
        return;
    }
    if (own == 0) return;
    __syncthreads();   // nobody reads the groups' tiles any more
    for (int b = b0; b < b1; ++b) {
        tiles[b] = run;
        if (blockIdx.x == P) d.prefix_out[b] = run;
        run += seq_tiles(seq_len<kOwn>(d, pre, FlatSeq{}, b), a.max_own) * static_cast<uint32_t>(per_seq);
    }
    if (tid == 0) {
        tiles[d.B] = own;
        if (blockIdx.x == P) d.prefix_out[d.B] = own;
    }
    __syncthreads();
    if (tid >= Cfg<D>::kThreads) return;
    decode_f16_body<D, NB, false, kOwn>(tk, tv, d, smem, tiles, pre, FlatSeq{}, blockIdx.x - P, gridDim.x - P);
}

// Short caches: clusters as in the FP16 decode's short form, one for each stream, which read the prefix for each
// sequence; the rule is that form's (cluster_of), for the longest prefix and own part together.  8 sequences behind
// 1,024 tokens: 10.7 us, where two kinds of CTAs and a merge take 14.5.
template <int D, int NB>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    decode_shared_flat_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                              const SharedArgs a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const DecodeF16Args& d = a.dec;
    const bool lead = blockIdx.x == 0;
    const int b = static_cast<int>(blockIdx.x / cg::this_cluster().num_blocks()) / (d.Hkv * d.sets);
    const int n = d.kv_lens[b];
    bool order = true;
    for (int g = threadIdx.x; g < a.groups; g += C::kThreads) {
        const int s = a.starts[g], e = a.starts[g + 1];
        order = order && s >= 0 && s <= e && e <= d.B && (g > 0 || s == 0) && (g + 1 < a.groups || e == d.B);
        if (lead) {
            const int p = a.prefix_lens[g];
            if (p < 0 || p > a.max_prefix || p % d.ps != 0) atomicOr(d.status, kDevBadLength);
        }
    }
    order = __syncthreads_and(order);
    FlatSeq flat{0, 0, b};
    if (order) {
        int g = 0, hi = a.groups - 1;   // the last group that begins at or before b
        while (g < hi) {
            const int mid = (g + hi + 1) >> 1;
            if (a.starts[mid] <= b) g = mid; else hi = mid - 1;
        }
        const int p = a.prefix_lens[g];
        if (p >= 0 && p <= a.max_prefix && p % d.ps == 0) {
            if (n >= p && n - p <= a.max_own && n <= a.cap) flat = FlatSeq{n, p, a.starts[g]};
            else if (threadIdx.x == 0) atomicOr(d.status, kDevBadLength);
        }
    } else if (lead && threadIdx.x == 0) {
        atomicOr(d.status, kDevBadIndex);
    }
    decode_f16_body<D, NB, true, kFlat>(tk, tv, d, smem,
                                        reinterpret_cast<uint32_t*>(smem + C::kRing + C::kBarBytes), nullptr,
                                        flat, blockIdx.x, gridDim.x);
}

// Workspace: the own tokens' records and tile prefix (decode_layout), then the prefixes' records, a unit's rows a
// CTA and one for every row of the call, the groups' steps, the sequences' prefixes and the total.
struct SharedLayout {
    Layout dec;
    size_t o, ml, work, seq, total_at, total;
};
SharedLayout shared_layout(long long ctas, int B, int Hkv, int G, int groups, int max_own, int D) {
    SharedLayout l{};
    l.dec = decode_layout(ctas, B, Hkv, G, max_own, D, false);
    const size_t rows = static_cast<size_t>(ctas) * (D == 256 ? Unit<256>::kRows : Unit<128>::kRows) +
                        static_cast<size_t>(B) * Hkv * G;
    size_t at = round16(l.dec.total);
    at = (at + 31) & ~static_cast<size_t>(31);
    l.o = at;
    at += rows * D * 4;
    l.ml = at;
    at += round16(rows * 8);
    l.work = at;
    at += round16((static_cast<size_t>(groups) + 1) * 4);
    l.seq = at;
    at += round16(static_cast<size_t>(B) * 8);
    l.total_at = at;
    l.total = at + 16;
    return l;
}

template <int D, int NB>
int launch_shared(const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& pk, const CUtensorMap& pv,
                  int ctas, int device, const SharedArgs& a, cudaStream_t s) {
    static std::once_flag once[64];
    static int rc[64];
    if (device < 0 || device >= 64) return GBATTN_ERR_CUDA;
    auto* kernel = decode_shared_kernel<D, NB>;
    std::call_once(once[device], [&] {
        rc[device] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          Smem<D>::kBytes) == cudaSuccess
                         ? GBATTN_OK
                         : GBATTN_ERR_CUDA;
        if (rc[device] != GBATTN_OK) cudaGetLastError();
    });
    if (rc[device] != GBATTN_OK) return rc[device];
    kernel<<<ctas, Pre<D>::kThreads, Smem<D>::kBytes, s>>>(tk, tv, pk, pv, a);
    count_launches(1);
    return launch_status();
}

// The short form, where its rule takes it: `launched` says whether.
template <int D, int NB>
int launch_flat(const CUtensorMap& tk, const CUtensorMap& tv, long long streams, int device, const SharedArgs& a,
                cudaStream_t s, bool& launched) {
    launched = false;
    const long long most = static_cast<long long>(a.max_prefix) + a.max_own;
    if (most > (1 << 30)) return GBATTN_OK;
    const int* resident = resident_clusters<D, NB, decode_shared_flat_kernel<D, NB>>(device);
    if (!resident) return GBATTN_ERR_CUDA;
    const int cl = cluster_of(streams, static_cast<int>(most), D, false, resident);
    if (cl == 0) return GBATTN_OK;
    launched = true;
    SharedArgs f = a;
    f.dec.max_kv = static_cast<int>(most);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(streams * cl));
    cfg.blockDim = dim3(Cfg<D>::kThreads);
    cfg.dynamicSmemBytes = Cfg<D>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cl);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_shared_flat_kernel<D, NB>, tk, tv, f);
    count_launches(1);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GBATTN_ERR_CUDA;
    }
    return launch_status();
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" size_t attn_paged_decode_shared_f16_workspace_size(int B, int Hq, int Hkv, int nq, int groups,
                                                              int max_prefix_len, int max_own_len, int D) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || nq <= 0 || groups <= 0 || max_prefix_len < 0 || max_own_len < 0 ||
        D <= 0 || Hq % Hkv != 0)
        return 0;
    const long long G = static_cast<long long>(Hq / Hkv) * nq;
    if (G > 0x7FFFFFFFLL) return 0;
    return shared_layout(sm_count_or_default(), B, Hkv, static_cast<int>(G), groups, max_own_len, D).total;
}

extern "C" int attn_paged_decode_shared_f16_fwd(const void* q, const void* k_pages, const void* v_pages,
                                                const int32_t* page_table, const int32_t* kv_lens,
                                                const int32_t* group_starts, const int32_t* prefix_lens,
                                                void* o, float* lse, int B, int Hq, int Hkv, int nq, int D,
                                                int groups, int num_phys_pages, int page_size,
                                                int max_pages, int max_prefix_len, int max_own_len,
                                                float scale, void* workspace, size_t workspace_bytes,
                                                void* stream) {
    CallRange nvtx_range("attn_paged_decode_shared_f16_fwd");
    if (!q || !k_pages || !v_pages || !page_table || !kv_lens || !group_starts || !prefix_lens || !o)
        return GBATTN_ERR_NULL;
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || nq <= 0 || groups <= 0 || num_phys_pages <= 0 || page_size <= 0 ||
        max_pages <= 0 || max_prefix_len < 0 || max_own_len < 0)
        return GBATTN_ERR_SHAPE;
    if (D != 64 && D != 128 && D != 256) return GBATTN_ERR_UNSUPPORTED;
    if (!pool_supported(num_phys_pages, page_size) || B > kMaxSeqs || groups > kMaxSeqs)
        return GBATTN_ERR_UNSUPPORTED;
    const long long slots_row = static_cast<long long>(max_pages) * page_size;
    if (Hq % Hkv != 0 || max_prefix_len > slots_row || max_own_len > slots_row ||
        max_prefix_len > (1 << 30) || max_own_len > (1 << 30))
        return GBATTN_ERR_SHAPE;
    const long long rows = static_cast<long long>(B) * Hq * nq;
    const long long G64 = static_cast<long long>(Hq / Hkv) * nq;
    if (rows > (1 << 30) || G64 > (1 << 30)) return GBATTN_ERR_SHAPE;
    const int G = static_cast<int>(G64);
    const RowPlan plan = row_plan(G, D, B, Hkv, max_own_len);
    const int R = plan.R;
    const long long streams = static_cast<long long>(B) * Hkv * plan.sets * plan.side;
    const long long own_tiles = (max_own_len + kTile - 1LL) / kTile;
    // steps a tile of all groups, each at most one short of a whole number of them per KV head
    const long long units = (static_cast<long long>(B) * G / kStepRows + groups) * Hkv;
    const long long pre_tiles = (max_prefix_len + kPreTile - 1LL) / kPreTile;
    if (streams > 0x7FFFFFFFLL || streams * own_tiles > 0x7FFFFFFFLL || units > 0x7FFFFFFFLL ||
        units * pre_tiles > 0x7FFFFFFFLL)
        return GBATTN_ERR_SHAPE;
    if (!finite_positive(scale)) return GBATTN_ERR_SCALE;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) ||
        (reinterpret_cast<uintptr_t>(workspace) & 31u) || misaligned4(page_table) || misaligned4(kv_lens) ||
        misaligned4(group_starts) || misaligned4(prefix_lens) || misaligned4(lse))
        return GBATTN_ERR_ALIGN;
    const size_t slots = static_cast<size_t>(num_phys_pages) * page_size * Hkv;
    const Range in[] = {{q, static_cast<size_t>(rows) * D * 2},
                        {k_pages, slots * D * 2},
                        {v_pages, slots * D * 2},
                        {page_table, static_cast<size_t>(B) * max_pages * 4},
                        {kv_lens, static_cast<size_t>(B) * 4},
                        {group_starts, (static_cast<size_t>(groups) + 1) * 4},
                        {prefix_lens, static_cast<size_t>(groups) * 4}};
    const Range out[] = {{o, static_cast<size_t>(rows) * D * 2},
                         {lse, static_cast<size_t>(rows) * 4}};
    if (any_overlap(in, out)) return GBATTN_ERR_ALIAS;
    if (!workspace) return GBATTN_ERR_WORKSPACE;
    DeviceState dev;
    int rc = current_device(&dev);
    if (rc != GBATTN_OK) return rc;
    auto layout = [&](long long ctas) { return shared_layout(ctas, B, Hkv, G, groups, max_own_len, D); };
    // One CTA per SM; fewer, down to two, when the workspace holds fewer records.
    long long ctas = dev.num_sms;
    while (ctas > 2 && layout(ctas).total > workspace_bytes) --ctas;
    const SharedLayout lay = layout(ctas);
    if (lay.total > workspace_bytes) return GBATTN_ERR_WORKSPACE;
    const Range ws[] = {{workspace, lay.total}};
    if (any_overlap(in, ws) || any_overlap(out, ws)) return GBATTN_ERR_ALIAS;

    SharedArgs a{};
    a.box_rows = page_size < kPreTile ? page_size : kPreTile;
    while ((1 << a.box_bits) < a.box_rows) ++a.box_bits;
    CUtensorMap tk, tv, pk, pv;
    const uint64_t total_rows = static_cast<uint64_t>(num_phys_pages) * page_size;
    if (encode_tmap_f16_pages(&tk, k_pages, D, Hkv, total_rows, kTile) != GBATTN_OK ||
        encode_tmap_f16_pages(&tv, v_pages, D, Hkv, total_rows, kTile) != GBATTN_OK)
        return GBATTN_ERR_CUDA;
    uint8_t* wsp = static_cast<uint8_t*>(workspace);
    DecodeF16Args& d = a.dec;
    d.q = static_cast<const __half*>(q);
    d.table = page_table;
    d.kv_lens = kv_lens;
    d.part_o = reinterpret_cast<float*>(wsp + lay.dec.o);
    d.part_ml = reinterpret_cast<float2*>(wsp + lay.dec.ml);
    d.tail0 = static_cast<long long>(lay.dec.tail0);
    d.prefix_out = reinterpret_cast<uint32_t*>(wsp + lay.dec.prefix);
    d.status = dev.status;
    d.wait_limit = wait_limit_ns();
    d.fault = fault_mode();
    d.B = B;
    d.Hq = Hq;
    d.Hkv = Hkv;
    d.nq = nq;
    d.G = G;
    d.side_bits = plan.side_bits;
    d.sets = plan.sets;
    d.pairs = row_pairs(plan.groups, R, G);
    d.num_phys = num_phys_pages;
    d.ps = page_size;
    d.max_pages = max_pages;
    d.max_kv = max_own_len;
    d.maps = 1;
    d.sl2 = scale * 1.4426950408889634f;
    d.out = RowOut{static_cast<__half*>(o), lse, Hq, nq, DiffArgs{}};
    a.starts = group_starts;
    a.prefix_lens = prefix_lens;
    a.pre_o = reinterpret_cast<float*>(wsp + lay.o);
    a.pre_ml = reinterpret_cast<float2*>(wsp + lay.ml);
    a.work_out = reinterpret_cast<uint32_t*>(wsp + lay.work);
    a.seq_out = reinterpret_cast<int2*>(wsp + lay.seq);
    a.total_out = reinterpret_cast<uint32_t*>(wsp + lay.total_at);
    a.groups = groups;
    a.max_prefix = max_prefix_len;
    a.max_own = max_own_len;
    a.cap = slots_row < 0x7FFFFFFFLL ? static_cast<int>(slots_row) : 0x7FFFFFFF;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (plan.side == 1) {   // short caches (row groups as streams of their own read the cache again, as there)
        bool launched = false;
        auto flat = [&](auto launch) { return launch(tk, tv, streams, dev.device, a, s, launched); };
        if (R == 8)
            rc = D == 64 ? flat(launch_flat<64, 1>) : D == 128 ? flat(launch_flat<128, 1>) : flat(launch_flat<256, 1>);
        else
            rc = D == 64 ? flat(launch_flat<64, 2>) : D == 128 ? flat(launch_flat<128, 2>) : flat(launch_flat<256, 2>);
        if (rc != GBATTN_OK || launched) return rc;
    }
    if (encode_tmap_f16_pages(&pk, k_pages, D, Hkv, total_rows, a.box_rows) != GBATTN_OK ||
        encode_tmap_f16_pages(&pv, v_pages, D, Hkv, total_rows, a.box_rows) != GBATTN_OK)
        return GBATTN_ERR_CUDA;
    const int n = static_cast<int>(ctas);
    auto go = [&](auto launch) { return launch(tk, tv, pk, pv, n, dev.device, a, s); };
    if (R == 8)
        rc = D == 64 ? go(launch_shared<64, 1>) : D == 128 ? go(launch_shared<128, 1>) : go(launch_shared<256, 1>);
    else
        rc = D == 64 ? go(launch_shared<64, 2>) : D == 128 ? go(launch_shared<128, 2>) : go(launch_shared<256, 2>);
    if (rc != GBATTN_OK) return rc;

    MergeArgs m{};
    m.part_o = d.part_o;
    m.part_ml = d.part_ml;
    m.prefix = d.prefix_out;
    m.kv_lens = kv_lens;
    m.max_kv = max_own_len;
    m.B = B;
    m.Hq = Hq;
    m.Hkv = Hkv;
    m.nq = nq;
    m.side_bits = plan.side_bits;
    m.sets = plan.sets;
    m.R = R;
    m.tail0 = d.tail0;
    m.grid = static_cast<uint32_t>(ctas);
    m.parts = static_cast<uint32_t>(warps_of(D) / plan.side);
    m.out = d.out;
    m.pre = PrefixRecords{a.pre_o, a.pre_ml, a.work_out, a.seq_out, a.total_out, group_starts, prefix_lens,
                          groups, max_prefix_len, page_size, a.cap};
    // Warps per row by the records of an average row, of either kind, as long as all of them fit the GPU at once:
    // every warp places its row's records by itself (1024 rows 29.4 us with two warps, 33.0 with four; 512 rows 38.8
    // and 35.8; 2048 rows 73.5 with one, 77.9 with two).  Eight records a warp are one trip to L2: 16 warps instead of
    // eight for 152 records took 5 sequences behind 196,608 tokens of one KV head from 49.6 to 47.4 us, 16 behind 65,536 at
    // D = 64 from 24.9 to 22.3; eight instead of four for 31 records, six groups behind 16,384, from 21.6 to 20.7.
    const long long recs = ctas * plan.side / streams + ctas / (units < 1 ? 1 : units) + 2;
    int mw = recs > 64 ? 16 : recs > 16 ? 8 : recs > 8 ? 4 : 1;
    while (mw > 1 && rows * mw > 2048) mw /= 2;
    const dim3 mgrid(static_cast<unsigned>(rows));
    const size_t msmem = static_cast<size_t>(mw) * (D * sizeof(float) + sizeof(float2));
    return D == 64    ? launch_dependent(decode_f16_merge_kernel<64, false, true>, mgrid, 32 * mw, msmem, s, m)
           : D == 128 ? launch_dependent(decode_f16_merge_kernel<128, false, true>, mgrid, 32 * mw, msmem, s, m)
                      : launch_dependent(decode_f16_merge_kernel<256, false, true>, mgrid, 32 * mw, msmem, s, m);
}
