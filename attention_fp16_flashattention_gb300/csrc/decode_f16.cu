// Decode attention over a paged FP16 KV cache, with the attention weight every
// cached token receives added up for eviction, and its differential form.  The
// FP16 counterpart of the E4M3 decode in decode.cu ("Integrate FP32 v37 prefill
// and exact E4M3 bridge", Validation: decode of long caches with shared-KV heads).
//
// Mathematics.  Row r of a (sequence, KV head) is one query of one head of the
// group; x[r][t] = scale q_r . k_t over the tokens it sees, p = softmax(x),
// o_r = sum_t p[r][t] v_t.  In the differential form a query head has two rows,
// q's halves q1 and q2 against k's halves: the rows are [q1 | 0] and [0 | q2], so
// both maps are ordinary rows of the same kernel over the same cached bytes, and
// the merge takes o1 - lambda o2 (diff.cuh).
//
// What bounds it: the cache's bytes, 4 D per token and KV head read once, against
// 4 D FLOPs per row.  So the split is the E4M3 decode's (tiles.cuh): every warp of
// a persistent grid takes an equal contiguous range of 16-token tiles whatever the
// lengths and runs its own TMA ring (about 192 KB in flight per SM).  The partial
// (max, sum, O) of a stream that ends inside a warp's range goes to memory; those
// that the ranges' ends cut are first joined over the CTA's warps in shared memory
// (consecutive warps mostly work on one stream), so a stream leaves one record per
// CTA it meets and not one per warp.  A merge kernel joins the records.
//   * S^T = K Q^T and O^T += V^T P^T on mma.sync m16n8k16: tokens (QK) and head
//     width (PV) fill M, the query rows N (8, or 16 where a group has more).  K and
//     V fragments come from the swizzled stage by ldmatrix (V transposed).
//   * Probabilities enter the PV product as two FP16 halves, hi = RNE(p) and
//     lo = RNE(p - hi), 22 bits: one FP16 value alone would add an error as
//     large as the output's own rounding, and the extra MMAs are hidden behind the
//     loads.  p is 2^(x - reference), where the reference lies kShift below a maximum, so
//     that the largest p fill FP16's range and the smallest keep their bits (tiles.cuh).
//   * With `weights` the warps also store their scores (FP32, 1/16 of the cache's
//     bytes at D = 128 and four rows); when the merge has the rows' final max and
//     sum, a third kernel adds sum_r 2^(x - max) / sum to every token's weight.
//     Every (token, KV head) is added to once per call, so the result does not
//     depend on any order unless two sequences share a page.
//   * Short caches: a cluster of up to eight CTAs takes each stream, joins the partials
//     through its shared memory and adds the weights; one kernel (rule at cluster_of).
// Measured (graph replays): 4 sequences of 65,571 to 131,072 tokens, 6 query heads on
// one KV head of 256 (450 MB) 75 us, 6.0 TB/s, 0.89 of the measured copy; 32 of 257
// to 8,191, 32 on 8 of 128, with weights (581 MB) 109 us, 15 of them for the weights (a
// kernel of its own, and 17 MB of scores written beside the cache's stream); one sequence of 511
// 7.4 us in clusters (9.1 with a merge kernel), latency of the loads behind each other.
// What the decode kernel loses against the copy rate is its start (lengths, then page
// table, then the first tiles: three trips to memory) and the joins at its end, 6 us
// together.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <mutex>

#include "diff.cuh"
#include "host.h"
#include "ptx.cuh"
#include "tiles.cuh"

namespace cg = cooperative_groups;

namespace gbattn {
namespace {

constexpr int kTile = 16;        // tokens per tile (one MMA M block)
constexpr int kMaxSeqs = 4096;   // sequences per launch (prefix table in shared memory)
constexpr int kMaxCluster = 8;      // CTAs of a stream's cluster
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
struct Cfg {
    static constexpr int kWarps = D == 256 ? 4 : 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kStages = D == 64 ? 6 : 3;            // 192 KB per CTA at every width
    static constexpr int kBoxes = D / 64;                      // 64-column boxes of a row
    static constexpr int kBox = kTile * 128;                   // bytes of one TMA box
    static constexpr int kStageBytes = 2 * kBoxes * kBox;      // K boxes, then V boxes
    static constexpr int kSteps = D / 16;                      // QK k-steps, PV d-blocks
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kBarBytes = kWarps * kStages * 8;
    static constexpr int kSmem = kRing + kBarBytes + 4 * (kMaxSeqs + 1) + 16 + 1024;
};

// Where a finished row goes, and what the differential form does to it.
struct RowOut {
    __half* o;
    float* lse;       // [B][Hq][maps][nq] or null
    int Hq, nq;
    DiffArgs diff;
};

struct DecodeF16Args {
    const __half* q;
    const int32_t* table;
    const int32_t* kv_lens;
    // Records of R = 8 NB rows: O [R][D] unnormalised and (reference in log2 units, sum) [R], for
    // every row group i of a stream's `side`.  Record (CTA + stream) side + i holds what the
    // ends of the CTA's warp ranges cut of the stream; record (tail0 + stream) side + i what
    // a warp finished inside its range.
    float* part_o;
    float2* part_ml;
    long long tail0;
    uint32_t* prefix_out; // [B + 1]: tiles of all streams of the sequences before b
    float* scores;        // log2-unit scores [tile][pairs][8][2][2]: of rows 2 p and 2 p + 1, tokens
                          // g and g + 8, as one lane has them; or null
    uint4* tiles;         // with scores: what the weights kernel needs to know of each tile
    uint32_t* status;
    uint64_t wait_limit;
    int fault;   // test hook: 1 = no stage is loaded, 2 = loads stop after two ring rounds
    int B, Hq, Hkv, nq, G, pairs, num_phys, ps, max_pages, max_kv;
    int side_bits, sets;  // row groups: `side` = 2^side_bits side by side in a CTA, `sets` such sets
    int maps;             // 1, or 2: row r is map r % 2 of query r / 2
    float sl2;            // softmax scale * log2(e)
    RowOut out;           // a cluster a stream: where its rows go
    float* weights;       // and their weights, with `scores`
};

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Tiles of one stream of a sequence (0 for a rejected length).
__device__ __forceinline__ uint32_t seq_tiles(int len, int max_kv) {
    return (len >= 0 && len <= max_kv) ? static_cast<uint32_t>((len + kTile - 1) / kTile) : 0u;
}

// A CTA's warps are `parts` equal shares of its tile range, each of `side` warps on as many
// row groups.  How many CTAs of a grid work on U tiles, and how many parts of each: all of
// them when every part gets a tile, else as many as every CTA can feed.
struct Split {
    uint32_t ctas, parts;
};
__device__ __forceinline__ Split split_of(uint32_t U, uint32_t grid, uint32_t parts) {
    return Split{min(grid, U), min(parts, max(U / grid, 1u))};
}

// The row sums of a lane's two query columns over the eight lanes that share them.
__device__ __forceinline__ void quad_sum(const float (&l)[2], float (&out)[2]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        out[e] = l[e];
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) out[e] += __shfl_xor_sync(0xffffffffu, out[e], sh);
    }
}

// The factor of a partial (max, sum) under the joint max M.  A row that saw nothing
// has max -inf, sum 0 and factor 0 (and its O does not count); one whose scores are all
// NaN keeps its NaN.
__device__ __forceinline__ float record_weight(float2 ml, float M) {
    return ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : exp2f(ml.x - M);
}

// The end of a row, a warp on D columns (V a lane): map mp's joint (M, sum Ls) and O scaled by
// 2^(x - M) give O / Ls and lse = (M + log2 Ls) ln 2; a row that sees nothing gets 0 and -inf.
template <int V>
__device__ __forceinline__ void add_map(float (&out)[V], const float (&so)[V], float M, float Ls, int mp,
                                        float lambda, const RowOut& t, int b, int head, int i, int maps,
                                        int lane) {
    const float inv = Ls == 0.0f ? 0.0f : 1.0f / Ls;
    const float f = mp == 0 ? inv : -lambda * inv;
#pragma unroll
    for (int e = 0; e < V; ++e) out[e] += so[e] * f;
    if (lane == 0 && t.lse)
        t.lse[((static_cast<long long>(b) * t.Hq + head) * maps + mp) * t.nq + i] =
            Ls == 0.0f ? -INFINITY : (M + log2f(Ls)) * kLn2;
}
// The lane's norm weights, loaded where there is time for it.
template <int V>
__device__ __forceinline__ void load_norm(float (&gain)[V], bool diff, const RowOut& t, int lane) {
#pragma unroll
    for (int e = 0; e < V; ++e) gain[e] = diff && t.diff.norm ? t.diff.norm[lane * V + e] : 1.0f;
}
template <int D>
__device__ __forceinline__ void store_row(float (&out)[D / 32], const float (&gain)[D / 32], bool diff,
                                          const RowOut& t, int b, int head, int i, int lane) {
    constexpr int V = D / 32;
    if (diff && t.diff.norm) {
        float sq = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) sq += out[e] * out[e];
        const float rn = rsqrtf(warp_sum(sq) * (1.0f / D) + t.diff.eps) * (1.0f - t.diff.init);
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] *= rn * gain[e];
    }
    __half* op = t.o + ((static_cast<long long>(b) * t.Hq + head) * t.nq + i) * D + lane * V;
    if constexpr (V == 2) {
        *reinterpret_cast<uint32_t*>(op) = pack_half2(out[0], out[1]);
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 4)
            *reinterpret_cast<uint2*>(op + e) =
                make_uint2(pack_half2(out[e], out[e + 1]), pack_half2(out[e + 2], out[e + 3]));
    }
}

// kOne: a cluster takes one stream, its CTAs' warps equal shares of the stream's tiles, and joins the
// partials in its shared memory: short caches, where the merge kernel would cost more than an uneven
// split (rule and times at cluster_of).
template <int D, int NB, bool kOne>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    decode_f16_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                      DecodeF16Args a) {
    using C = Cfg<D>;
    constexpr int R = 8 * NB;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t warp_sums[C::kWarps];
    __shared__ float2 s_ml[C::kWarps][R];      // each warp's last segment: row max and sum
    __shared__ long long s_stream[C::kWarps];  // its stream, -1 for an idle warp
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kRing);
    uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + C::kRing + C::kBarBytes);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(prefix + kMaxSeqs + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp >> a.side_bits, beside = warp & ((1 << a.side_bits) - 1);
    const int per_seq = a.Hkv * a.sets;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    cg::cluster_group cluster = cg::this_cluster();
    const int C_one = kOne ? static_cast<int>(cluster.num_blocks()) : 1;
    TileLoc one{};   // kOne: the stream and its tiles
    if constexpr (kOne) {
        const int stream = static_cast<int>(blockIdx.x) / C_one;
        one.b = stream / per_seq;
        one.sis = stream - one.b * per_seq;
        const int len = a.kv_lens[one.b];
        if ((len < 0 || len > a.max_kv) && threadIdx.x == 0) atomicOr(a.status, kDevBadLength);
        one.s_end = seq_tiles(len, a.max_kv);
        if (threadIdx.x == 0) {
            for (int s = 0; s < C::kWarps * C::kStages; ++s) mbar_init(&bars[s], 1);
            *abort_flag = 0;
            mbar_init_fence();
        }
        __syncthreads();
    } else {   // ---- tile prefix over sequences (block-wide scan of per-sequence tile counts)
        const int per = (a.B + C::kThreads) / C::kThreads;   // entries 0..B over the threads
        const int b0 = threadIdx.x * per;
        uint32_t sum = 0;
        for (int b = b0; b < min(b0 + per, a.B); ++b) {
            const int len = a.kv_lens[b];
            if ((len < 0 || len > a.max_kv) && blockIdx.x == 0) atomicOr(a.status, kDevBadLength);
            const uint32_t n = seq_tiles(len, a.max_kv) * static_cast<uint32_t>(per_seq);
            prefix[b] = n;   // this thread's own entries; turned into the prefix below
            sum += n;
        }
        uint32_t incl = sum;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, sh);
            if (lane >= sh) incl += y;
        }
        if (lane == 31) warp_sums[warp] = incl;
        if (threadIdx.x == 0) {
            for (int s = 0; s < C::kWarps * C::kStages; ++s) mbar_init(&bars[s], 1);
            *abort_flag = 0;
            mbar_init_fence();
        }
        __syncthreads();
        uint32_t run = incl - sum;
        for (int w = 0; w < warp; ++w) run += warp_sums[w];
        for (int b = b0; b < min(b0 + per, a.B + 1); ++b) {
            const uint32_t n = b < a.B ? prefix[b] : 0u;
            prefix[b] = run;   // prefix[B] = total
            run += n;
        }
        __syncthreads();
        if (blockIdx.x == 0)
            for (int b = threadIdx.x; b <= a.B; b += C::kThreads) a.prefix_out[b] = prefix[b];
    }
    // The merge grid may start launching now; it waits for this grid to finish.
    if constexpr (!kOne) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t U = kOne ? one.s_end : prefix[a.B];
    const Split sp = kOne ? Split{static_cast<uint32_t>(C_one), static_cast<uint32_t>(C::kWarps)}
                          : split_of(U, gridDim.x, C::kWarps >> a.side_bits);
    if (!kOne && blockIdx.x >= sp.ctas) return;
    // every part below sp.parts has at least one tile; the others wait at the end
    const uint32_t cta = kOne ? cluster.block_rank() : blockIdx.x;
    const uint32_t W = sp.ctas * sp.parts;
    const uint32_t w = cta * sp.parts + min(static_cast<uint32_t>(part), sp.parts - 1);
    const bool idle = static_cast<uint32_t>(part) >= sp.parts;
    const uint32_t u_beg = warp_start(w, W, U), u_end = idle ? u_beg : warp_start(w + 1, W, U);
    auto place = [&](uint32_t u) -> TileLoc {
        if constexpr (kOne) return TileLoc{one.b, one.sis, static_cast<int>(u), one.s_end};
        return locate(u, prefix, a.B, per_seq);
    };

    const WaitCtl wc{a.wait_limit, a.status, abort_flag};
    const uint64_t policy = l2_evict_first();   // the cache is read once; records and scores stay
    // scores are read back soon: kept in L2 (without this ncu saw 9 to 15 of their 17 MB written out
    // to memory while the cache streams through, and the call took 1.4 us more; 65 MB of them cost a
    // later kernel 2.3 us, once, until its own lines have taken their place)
    const uint64_t keep = l2_evict_last();
    uint8_t* ring = smem + warp * C::kStages * C::kStageBytes;
    uint64_t* full = bars + warp * C::kStages;

    // First cache row ([page * ps + slot] space) of tile u and its KV head, packed
    // as (head, row) in 64 bits.
    auto tile_src = [&](uint32_t u, bool dead = false) -> long long {
        if (u >= u_end) return 0;
        const TileLoc L = place(u);
        const int tok = L.t * kTile;
        int page = a.table[static_cast<long long>(L.b) * a.max_pages + tok / a.ps];
        const bool bad = page < 0 || page >= a.num_phys;
        if (bad) {
            atomicOr(a.status, kDevBadPage);
            page = 0;
        }
        const int hk = L.sis / a.sets;
        if (!kOne && a.scores) {
            // One description for all row groups: group 0's tile leaves (first slot, sequence and
            // KV head, its own number, live tokens + 32 * tiles of the stream); none live on a
            // bad page, or where the warp gave up (dead).  Row group r's tile is side * (number + (r / side) tiles) + r % side.
            if (beside == 0 && L.sis == hk * a.sets) {
                const uint32_t first = prefix[L.b], T = (prefix[L.b + 1] - first) / per_seq;
                const uint32_t live = bad || dead ? 0 : min(kTile, a.kv_lens[L.b] - tok);
                a.tiles[first / a.sets + hk * T + L.t] =
                    make_uint4(page * a.ps + tok % a.ps, L.b * a.Hkv + hk, u, live + 32 * T);
            }
        }
        return (static_cast<long long>(hk) << 32) | static_cast<uint32_t>(page * a.ps + tok % a.ps);
    };
    auto issue = [&](uint32_t k, long long src) {   // stage k of this warp's range
        if (elect_one()) {
            const int slot = k % C::kStages;
            uint8_t* dst = ring + slot * C::kStageBytes;
            const int row = static_cast<int>(src & 0xFFFFFFFFLL), hk = static_cast<int>(src >> 32);
            mbar_arrive_expect_tx(&full[slot], C::kStageBytes);
#pragma unroll
            for (int h = 0; h < C::kBoxes; ++h) {
                tma_load_3d_hint(dst + h * C::kBox, &tk, &full[slot], 64 * h, hk, row, policy);
                tma_load_3d_hint(dst + (C::kBoxes + h) * C::kBox, &tv, &full[slot], 64 * h, hk, row,
                                 policy);
            }
        }
        __syncwarp();
    };

    const uint32_t n_tiles = u_end - u_beg;
    // test hook: the waits for stages never loaded run out (bounded) mid-range
    const uint32_t n_load = a.fault == 1 ? 0u
                            : a.fault == 2 ? min(n_tiles, static_cast<uint32_t>(2 * C::kStages))
                                           : n_tiles;
    long long src_cur = tile_src(u_beg + lane);          // tiles 0..31 of the range, one per lane
    long long src_next = tile_src(u_beg + 32 + lane);    // tiles 32..63
    uint32_t issued = 0;
    for (; issued < static_cast<uint32_t>(C::kStages - 1) && issued < n_load; ++issued)
        issue(issued, __shfl_sync(0xffffffffu, src_cur, issued));

    const int g = lane >> 2, c = lane & 3;
    const int grp = a.Hq / a.Hkv;
    float o[NB][C::kSteps][4];
    float m_ref[NB][2], l_sum[NB][2];
    uint32_t qf[NB][C::kSteps][2];
    TileLoc L = place(u_beg);
    int kv_len = 0, lim[NB][2], first_masked = 0;
    // Start of a stream segment: state reset and the Q operand of the stream's rows.
    auto begin_stream = [&]() {
        kv_len = a.kv_lens[L.b];
        const int hk = L.sis / a.sets, rg = ((L.sis - hk * a.sets) << a.side_bits) + beside;
        first_masked = kv_len - a.nq + 1;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = rg * R + 8 * n + 2 * c + e;
                lim[n][e] = r < a.G ? kv_len - a.nq + (r / a.maps) % a.nq : kv_len - 1;
                m_ref[n][e] = -INFINITY;
                l_sum[n][e] = 0.0f;
            }
            const int r = rg * R + 8 * n + g;
            const int rq = r / a.maps, sub = r - rq * a.maps;   // query of the group, map
            const __half* qp = nullptr;
            if (r < a.G)
                qp = a.q + ((static_cast<long long>(L.b) * a.Hq + hk * grp + rq / a.nq) * a.nq +
                            rq % a.nq) * D;
#pragma unroll
            for (int st = 0; st < C::kSteps; ++st) {
                uint32_t x0 = 0, x1 = 0;
                // map 0 holds q's first half and zeros, map 1 zeros and its second half
                if (qp && (a.maps == 1 || (st >= C::kSteps / 2) == (sub == 1))) {
                    x0 = *reinterpret_cast<const uint32_t*>(qp + 16 * st + 2 * c);
                    x1 = *reinterpret_cast<const uint32_t*>(qp + 16 * st + 8 + 2 * c);
                }
                qf[n][st][0] = x0;
                qf[n][st][1] = x1;
            }
#pragma unroll
            for (int j = 0; j < C::kSteps; ++j)
                o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.0f;
        }
    };
    begin_stream();

    // ldmatrix lane addresses within a box: K rows (tokens) lane % 16, column chunk
    // lane / 16; V rows (lane % 8) + 8 (lane / 16), chunk (lane / 8) % 2.
    const int k_row = lane & 15, k_ch = lane >> 4;
    const int v_row = (lane & 7) + ((lane >> 4) << 3), v_ch = (lane >> 3) & 1;

    // kOne: the warp's first query at the end; what its lambda and norm need is on its way from here
    const int hk_one = one.sis / a.sets, rg_one = one.sis - hk_one * a.sets;
    const int queries = min(R, a.G - rg_one * R) / a.maps;   // R and G are multiples of maps
    const int j_first = static_cast<int>(cta) * C::kWarps + warp;
    const long long one_tile0 = (static_cast<long long>(one.b) * per_seq + one.sis) *
                                ((a.max_kv + kTile - 1) / kTile);   // the stream's tiles in `scores`
    // (kOne: D == 128 in the differential form)
    LambdaTerms<64> terms{};
    float gain[D / 32] = {};
    if constexpr (kOne) {
        const bool diff = D == 128 && a.maps == 2 && j_first < queries;
        if (diff)
            terms.load(a.out.diff, hk_one * (a.Hq / a.Hkv) + (rg_one * (R / 2) + j_first) / a.nq, lane);
        load_norm<D / 32>(gain, diff, a.out, lane);
    }

    bool aborted = false;
    for (uint32_t k = 0; k < n_tiles; ++k) {
        // keep the ring kStages - 1 tiles ahead
        if (issued < n_load) {
            if ((issued & 31u) == 0) {
                src_cur = src_next;
                src_next = tile_src(u_beg + issued + 32 + lane);
            }
            issue(issued, __shfl_sync(0xffffffffu, src_cur, issued & 31u));
            ++issued;
        }
        const int slot = k % C::kStages;
        if (!wait_warp(&full[slot], (k / C::kStages) & 1, wc)) {
            aborted = true;
            break;
        }
        const uint32_t kst = smem_addr(ring + slot * C::kStageBytes);
        const uint32_t vst = kst + C::kBoxes * C::kBox;
        const int tb = L.t * kTile;   // first token of the tile

        // ---- S^T = K Q^T: 16 tokens (rows) x R query rows
        float acc[NB][2][4];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) acc[n][x][0] = acc[n][x][1] = acc[n][x][2] = acc[n][x][3] = 0.0f;
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) {
            uint32_t f[4];
            const int ch = 2 * (st & 3) + k_ch;
            ldmatrix_x4(f, kst + (st >> 2) * C::kBox + k_row * 128 + ((ch ^ (k_row & 7)) << 4));
#pragma unroll
            for (int n = 0; n < NB; ++n)
                mma_16816(acc[n][st & 1], f[0], f[1], f[2], f[3], qf[n][st][0], qf[n][st][1]);
        }
        uint32_t ph[NB][2], pl[NB][2];   // P^T operands: hi and lo halves
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            // x[0]: token g, query 2c; x[1]: token g, query 2c+1; x[2], x[3]: token g+8.
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (acc[n][0][e] + acc[n][1][e]) * a.sl2;
            if (tb + kTile > first_masked) {
                const int t0 = tb + g, t1 = tb + g + 8;
                if (t0 > lim[n][0]) x[0] = -INFINITY;
                if (t0 > lim[n][1]) x[1] = -INFINITY;
                if (t1 > lim[n][0]) x[2] = -INFINITY;
                if (t1 > lim[n][1]) x[3] = -INFINITY;
            }
            if (a.scores) {
                const int r0 = 8 * n + 2 * c;
                const int real = a.G - (((L.sis % a.sets) << a.side_bits) + beside) * R;
                const long long tile = kOne ? one_tile0 + u_beg + k
                                            : (static_cast<long long>(u_beg + k) << a.side_bits) + beside;
                if (r0 < real)
                    store_f32x4_hint(a.scores + (tile * a.pairs + r0 / 2) * (2 * kTile) + 4 * g, x, keep);
            }
            // ---- online softmax for this lane's query columns 2c, 2c+1
            float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
            }
            const bool up0 = mx0 > m_ref[n][0] + kTop, up1 = mx1 > m_ref[n][1] + kTop;
            if (__any_sync(0xffffffffu, up0 || up1)) {
                const float n0 = up0 ? mx0 - kShift : m_ref[n][0], n1 = up1 ? mx1 - kShift : m_ref[n][1];
                const float al0 = up0 ? fast_exp2(m_ref[n][0] - n0) : 1.0f;
                const float al1 = up1 ? fast_exp2(m_ref[n][1] - n1) : 1.0f;
                m_ref[n][0] = n0;
                m_ref[n][1] = n1;
                l_sum[n][0] *= al0;
                l_sum[n][1] *= al1;
#pragma unroll
                for (int j = 0; j < C::kSteps; ++j) {
                    o[n][j][0] *= al0;
                    o[n][j][2] *= al0;
                    o[n][j][1] *= al1;
                    o[n][j][3] *= al1;
                }
            }
            const float mu0 = m_ref[n][0] == -INFINITY ? 0.0f : m_ref[n][0];
            const float mu1 = m_ref[n][1] == -INFINITY ? 0.0f : m_ref[n][1];
            const float p0 = fast_exp2(x[0] - mu0), p1 = fast_exp2(x[1] - mu1);
            const float p2 = fast_exp2(x[2] - mu0), p3 = fast_exp2(x[3] - mu1);
            l_sum[n][0] += p0 + p2;
            l_sum[n][1] += p1 + p3;
            const __half2 h01 = __floats2half2_rn(p0, p1), h23 = __floats2half2_rn(p2, p3);
            const float2 f01 = __half22float2(h01), f23 = __half22float2(h23);
            const __half2 l01 = __floats2half2_rn(p0 - f01.x, p1 - f01.y);
            const __half2 l23 = __floats2half2_rn(p2 - f23.x, p3 - f23.y);
            ph[n][0] = movmatrix_trans(h2_bits(h01));
            ph[n][1] = movmatrix_trans(h2_bits(h23));
            pl[n][0] = movmatrix_trans(h2_bits(l01));
            pl[n][1] = movmatrix_trans(h2_bits(l23));
        }
        // ---- O^T += V^T P^T: d-block j, rows d = 16 j + g (+ 8)
        auto pv = [&](uint32_t m01, uint32_t m89) {
#pragma unroll
            for (int j = 0; j < C::kSteps; ++j) {
                uint32_t f[4];
                const int ch = 2 * (j & 3) + v_ch;
                ldmatrix_x4_trans(f, vst + (j >> 2) * C::kBox + v_row * 128 +
                                         ((ch ^ (v_row & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    mma_16816(o[n][j], f[0] & m01, f[1] & m01, f[2] & m89, f[3] & m89, ph[n][0],
                              ph[n][1]);
                    mma_16816(o[n][j], f[0] & m01, f[1] & m01, f[2] & m89, f[3] & m89, pl[n][0],
                              pl[n][1]);
                }
            }
        };
        if (tb + kTile > kv_len) {   // slots past the cache end may hold anything, NaN too
            const int t0 = tb + 2 * c;
            const uint32_t m01 = (t0 < kv_len ? 0xFFFFu : 0u) | (t0 + 1 < kv_len ? 0xFFFF0000u : 0u);
            const uint32_t m89 = (t0 + 8 < kv_len ? 0xFFFFu : 0u) | (t0 + 9 < kv_len ? 0xFFFF0000u : 0u);
            pv(m01, m89);
        } else {
            pv(0xFFFFFFFFu, 0xFFFFFFFFu);
        }

        // ---- the stream ends inside the range: write its record, move on
        const uint32_t u = u_beg + k;
        if (!kOne && u + 1 == L.s_end && k + 1 < n_tiles) {
            // query rows of padding are skipped
            const int rbase = (((L.sis % a.sets) << a.side_bits) + beside) * R;
            const long long rec =
                ((a.tail0 + static_cast<long long>(L.b) * per_seq + L.sis) << a.side_bits) + beside;
            float* po = a.part_o + rec * R * D;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                float ls[2];
                quad_sum(l_sum[n], ls);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * n + 2 * c + e;
                    if (rbase + r >= a.G) continue;
#pragma unroll
                    for (int j = 0; j < C::kSteps; ++j) {
                        po[r * D + 16 * j + g] = o[n][j][e];
                        po[r * D + 16 * j + g + 8] = o[n][j][e + 2];
                    }
                    if (g == 0) a.part_ml[rec * R + r] = make_float2(m_ref[n][e], ls[e]);
                }
            }
            L = locate(u + 1, prefix, a.B, per_seq);
            begin_stream();
        } else {
            ++L.t;
        }
    }
    if (aborted) {
        // The weights kernel follows every description: none may be left unwritten.
        if (!kOne && a.scores)
            for (uint32_t k = lane; k < n_tiles; k += 32) tile_src(u_beg + k, true);
        // Stages already issued must land before the CTA's shared memory goes away.
        if (lane == 0) {
            for (uint32_t k = issued > C::kStages ? issued - C::kStages : 0; k < issued; ++k) {
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(&full[k % C::kStages], (k / C::kStages) & 1))
                    if (global_timer_ns() - t0 > a.wait_limit) break;
            }
        }
        __syncwarp();
    }

    // ---- the ranges' last segments: joined over the warps that hold the same stream.
    // A warp's ring is its own and empty by now; rows are padded by four floats, which
    // spreads the fragments' rows over the banks.
    constexpr int kPitch = D + 4;
    static_assert(R * kPitch * 4 <= C::kStages * C::kStageBytes, "segment fits the warp's ring");
    if (lane == 0)
        s_stream[warp] = idle ? -1 : static_cast<long long>(L.b) * per_seq + L.sis;
    if (!idle) {
        float* so = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            float ls[2];
            quad_sum(l_sum[n], ls);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * n + 2 * c + e;
#pragma unroll
                for (int j = 0; j < C::kSteps; ++j) {
                    so[r * kPitch + 16 * j + g] = o[n][j][e];
                    so[r * kPitch + 16 * j + g + 8] = o[n][j][e + 2];
                }
                if (g == 0) s_ml[warp][r] = make_float2(m_ref[n][e], ls[e]);
            }
        }
    }
    __syncthreads();
    constexpr int kRingFloats = C::kStages * C::kStageBytes / 4;
    const float* all = reinterpret_cast<const float*>(smem);
    if constexpr (kOne) {
        // The CTA's record in the place of the prefix table, then every row's over the cluster: a warp a
        // query, both maps of it.
        static_assert(R * D * 4 <= 4 * (kMaxSeqs + 1), "record fits the prefix table");
        __shared__ float2 s_rec[R];
        float* rec_o = reinterpret_cast<float*>(prefix);
        for (int x = threadIdx.x; x < R * (D / 4); x += C::kThreads) {
            const int r = x / (D / 4), d = 4 * (x % (D / 4));
            float M = -INFINITY, l = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int p = 0; p < C::kWarps; ++p) M = fmaxf(M, s_ml[p][r].x);
#pragma unroll
            for (int p = 0; p < C::kWarps; ++p) {
                const float2 ml = s_ml[p][r];
                if (ml.y == 0.0f) continue;   // no tile, or saw nothing
                const float wt = record_weight(ml, M);
                const float4 v = *reinterpret_cast<const float4*>(all + p * kRingFloats + r * kPitch + d);
                acc = make_float4(acc.x + wt * v.x, acc.y + wt * v.y, acc.z + wt * v.z, acc.w + wt * v.w);
                l += wt * ml.y;
            }
            *reinterpret_cast<float4*>(rec_o + r * D + d) = acc;
            if (d == 0) s_rec[r] = make_float2(M, l);
        }
        cluster.sync();
        if (a.scores) {
            // The weights, by the lanes that hold the scores: every row's joint max and sum, then
            // sum_r 2^(x - max) / sum over the lane's rows and the four lanes of a token.
            __shared__ float2 s_row[R];
            if (threadIdx.x < R) {
                float M = -INFINITY, l = 0.0f;
                for (int c8 = 0; c8 < C_one; ++c8)
                    M = fmaxf(M, cluster.map_shared_rank(s_rec, c8)[threadIdx.x].x);
                for (int c8 = 0; c8 < C_one; ++c8) {
                    const float2 ml = cluster.map_shared_rank(s_rec, c8)[threadIdx.x];
                    l += ml.y == 0.0f ? 0.0f : record_weight(ml, M) * ml.y;
                }
                s_row[threadIdx.x] = make_float2(M, l == 0.0f ? 0.0f : 1.0f / l);
            }
            __syncthreads();
            for (uint32_t k = 0; k < (aborted ? 0u : n_tiles); ++k) {
                const int tok = static_cast<int>(u_beg + k) * kTile;
                const int page = a.table[static_cast<long long>(one.b) * a.max_pages + tok / a.ps];
                float w0 = 0.0f, w1 = 0.0f;   // tokens g and g + 8
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const int r0 = 8 * n + 2 * c;
                    if (r0 >= a.G) continue;
                    const float4 x = *reinterpret_cast<const float4*>(
                        a.scores + ((one_tile0 + u_beg + k) * a.pairs + r0 / 2) * (2 * kTile) + 4 * g);
                    const float2 m0 = s_row[r0], m1 = s_row[r0 + 1];
                    if (x.x != -INFINITY) w0 += fast_exp2(x.x - m0.x) * m0.y;
                    if (x.z != -INFINITY) w1 += fast_exp2(x.z - m0.x) * m0.y;
                    if (r0 + 1 < a.G) {   // an odd last row has no partner
                        if (x.y != -INFINITY) w0 += fast_exp2(x.y - m1.x) * m1.y;
                        if (x.w != -INFINITY) w1 += fast_exp2(x.w - m1.x) * m1.y;
                    }
                }
#pragma unroll
                for (int sh = 1; sh < 4; sh <<= 1) {
                    w0 += __shfl_xor_sync(0xffffffffu, w0, sh);
                    w1 += __shfl_xor_sync(0xffffffffu, w1, sh);
                }
                const int t = tok + g + 8 * c;   // lane c = 0 adds token g's, c = 1 token g + 8's
                if (c < 2 && t < kv_len && page >= 0 && page < a.num_phys)
                    atomicAdd(a.weights + (static_cast<long long>(page) * a.Hkv + hk_one) * a.ps + t % a.ps,
                              c == 0 ? w0 : w1);
            }
        }
        constexpr int V = D / 32;
        for (int j = j_first; j < queries; j += C_one * C::kWarps) {
            const int rq = rg_one * (R / a.maps) + j;
            const int head = hk_one * (a.Hq / a.Hkv) + rq / a.nq, i = rq % a.nq;
            float lambda = 0.0f;
            if (D == 128 && a.maps == 2) {
                if (j != j_first) terms.load(a.out.diff, head, lane);
                lambda = terms.value(a.out.diff);
            }
            // lane c holds CTA c's (max, sum) of the query's row in each map
            float M[2], Ls[2], wt_c[2], so[2][V];
#pragma unroll
            for (int mp = 0; mp < 2; ++mp) {
                float2 ml = make_float2(-INFINITY, 0.0f);
                if (mp < a.maps && lane < C_one)
                    ml = cluster.map_shared_rank(s_rec, lane)[j * a.maps + mp];
                M[mp] = ml.x;
#pragma unroll
                for (int sh = 1; sh < kMaxCluster; sh <<= 1)
                    M[mp] = fmaxf(M[mp], __shfl_xor_sync(0xffffffffu, M[mp], sh));
                M[mp] = __shfl_sync(0xffffffffu, M[mp], 0);
                wt_c[mp] = ml.y == 0.0f ? 0.0f : record_weight(ml, M[mp]);
                Ls[mp] = warp_sum(wt_c[mp] * ml.y);
#pragma unroll
                for (int e = 0; e < V; ++e) so[mp][e] = 0.0f;
            }
#pragma unroll
            for (int c8 = 0; c8 < kMaxCluster; ++c8) {
                if (c8 >= C_one) break;
                const float* p = cluster.map_shared_rank(rec_o, c8) + j * a.maps * D + lane * V;
#pragma unroll
                for (int mp = 0; mp < 2; ++mp) {
                    if (mp >= a.maps) break;
                    const float wt = __shfl_sync(0xffffffffu, wt_c[mp], c8);
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        const float2 v = *reinterpret_cast<const float2*>(p + mp * D + e);
                        so[mp][e] += wt * v.x;
                        so[mp][e + 1] += wt * v.y;
                    }
                }
            }
            float out[V];
#pragma unroll
            for (int e = 0; e < V; ++e) out[e] = 0.0f;
            add_map<V>(out, so[0], M[0], Ls[0], 0, lambda, a.out, one.b, head, i, a.maps, lane);
            if (a.maps == 2)
                add_map<V>(out, so[1], M[1], Ls[1], 1, lambda, a.out, one.b, head, i, a.maps, lane);
            store_row<D>(out, gain, a.maps == 2, a.out, one.b, head, i, lane);
        }
        cluster.sync();   // nobody leaves while another CTA reads its record
        return;
    }
    for (uint32_t p0 = 0, p1; p0 < sp.parts; p0 = p1) {
        const long long stream = s_stream[p0 << a.side_bits];
        for (p1 = p0 + 1; p1 < sp.parts && s_stream[p1 << a.side_bits] == stream; ++p1) {}
        for (int i = 0; i < 1 << a.side_bits; ++i) {
            const long long rec = ((static_cast<long long>(blockIdx.x) + stream) << a.side_bits) + i;
            const int rg = (static_cast<int>(stream % a.sets) << a.side_bits) + i;
            const int real = min(R, a.G - rg * R);
            for (int x = threadIdx.x; x < real * (D / 4); x += C::kThreads) {
                const int r = x / (D / 4), d = 4 * (x % (D / 4));
                float M = -INFINITY, l = 0.0f;
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (uint32_t p = p0; p < p1; ++p) M = fmaxf(M, s_ml[(p << a.side_bits) + i][r].x);
                for (uint32_t p = p0; p < p1; ++p) {
                    const uint32_t wi = (p << a.side_bits) + i;
                    const float2 ml = s_ml[wi][r];
                    if (ml.y == 0.0f) continue;   // saw nothing: O may hold 0 times a cached infinity
                    const float wt = record_weight(ml, M);
                    const float4 v =
                        *reinterpret_cast<const float4*>(all + wi * kRingFloats + r * kPitch + d);
                    acc = make_float4(acc.x + wt * v.x, acc.y + wt * v.y, acc.z + wt * v.z,
                                      acc.w + wt * v.w);
                    l += wt * ml.y;
                }
                *reinterpret_cast<float4*>(a.part_o + (rec * R + r) * D + d) = acc;
                if (d == 0) a.part_ml[rec * R + r] = make_float2(M, l);
            }
        }
    }
}

// Joins the partial records of every query row: with m_r, l_r the reference (log2
// units) and sum of record r, M = max_r m_r, L = sum_r 2^(m_r - M) l_r,
// O = sum_r 2^(m_r - M) O_r / L and lse = (M + log2 L) ln 2.  One CTA takes one
// query of one head, its warps every blockDim/32-th record (kBatch in flight each,
// a lane on D/32 columns); the differential form gives each map half the warps
// and ends with diff.cuh's combination.  A row that sees nothing gets O = 0,
// lse = -inf.
struct MergeArgs {
    const float* part_o;
    const float2* part_ml;
    const uint32_t* prefix;
    const int32_t* kv_lens;
    long long tail0;
    int B, Hq, Hkv, nq, R, side_bits, sets, max_kv;
    uint32_t grid, parts;   // of the decode kernel
    float2* row_ml;   // [B][Hkv][G, made even]: (M, 1 / L) for the weights kernel, or null
    RowOut out;
};

constexpr int kMergeMaxWarps = 16;
constexpr int kEarlySeqs = 64;   // two lengths a lane

template <int D, bool kDiff>
__global__ void __launch_bounds__(32 * kMergeMaxWarps)
    decode_f16_merge_kernel(const MergeArgs a) {
    constexpr int V = D / 32;
    constexpr int kMaps = kDiff ? 2 : 1;
    constexpr int kBatch = 8;
    // Sized by the launch, so that as many CTAs as can be wait beside the decode's: with this and the early
    // sums below a call of 16 sequences to 16,001 went from 54.2 to 52.5 us, 4 to 131,072 from 76.5 to 75.5.
    extern __shared__ float s_merge[];   // [warps][D] O, then [warps] (max, sum)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    float2* s_ml = reinterpret_cast<float2*>(s_merge + warps * D);
    const long long row = blockIdx.x;
    const int per_b = a.Hq * a.nq;
    const int b = static_cast<int>(row / per_b);
    const int within = static_cast<int>(row - static_cast<long long>(b) * per_b);
    const int head = within / a.nq, i = within - head * a.nq;
    const int grp = a.Hq / a.Hkv;
    const int hk = head / grp;
    const int map = kDiff ? warp & 1 : 0;
    const int r = ((head - hk * grp) * a.nq + i) * kMaps + map;
    const int rg = r / a.R, n = r - rg * a.R;
    const int set = rg >> a.side_bits, per_seq = a.Hkv * a.sets, sis = hk * a.sets + set;
    float lambda = 0.0f;
    float gain[V];
    load_norm<V>(gain, kDiff && warp == 0, a.out, lane);
    if constexpr (kDiff) {
        if (warp == 0) lambda = diff_lambda<D / 2>(a.out.diff, head, lane);
    }
    // Launched as a programmatic dependent of the decode grid.  With few sequences the tiles before
    // this one's are summed up from the lengths while that runs; else the grid's prefix table is read.
    uint32_t T = 0, before = 0, U = 0;
    const bool early = a.B <= kEarlySeqs;
    if (early) {
        uint32_t mine = 0, total = 0;
#pragma unroll
        for (int e = 0; e < kEarlySeqs; e += 32) {
            const uint32_t n = e + lane < a.B ? seq_tiles(a.kv_lens[e + lane], a.max_kv) : 0u;
            total += n;
            mine += e + lane < b ? n : 0u;
            if (e + lane == b) T = n;
        }
        T = __reduce_add_sync(0xffffffffu, T);
        before = __reduce_add_sync(0xffffffffu, mine) * per_seq;
        U = __reduce_add_sync(0xffffffffu, total) * per_seq;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!early) {
        before = a.prefix[b];
        T = (a.prefix[b + 1] - before) / per_seq;
        U = a.prefix[a.B];
    }
    // The stream's records: `cut` of CTAs c0 .. c0 + cut - 1, and the tail when the
    // stream ends inside a warp's range.
    uint32_t c0 = 0, cut = 0, tail = 0;
    const long long stream = static_cast<long long>(b) * per_seq + sis;
    if (T > 0) {
        const Split sp = split_of(U, a.grid, a.parts);
        const uint32_t W = sp.ctas * sp.parts;
        const uint32_t u0 = before + sis * T;
        const uint32_t wf = warp_of(u0, W, U), wl = warp_of(u0 + T - 1, W, U);
        tail = warp_start(wl + 1, W, U) != u0 + T ? 1 : 0;
        c0 = wf / sp.parts;
        if (wl + 1 - tail > wf) cut = (wl - tail) / sp.parts - c0 + 1;
    }
    const uint32_t n_rec = cut + tail;
    const int lanes = warps / kMaps, wl = kDiff ? warp >> 1 : warp;
    float mx = -INFINITY, lw = 0.0f, acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.0f;
    for (uint32_t xb = wl; xb < n_rec; xb += lanes * kBatch) {
        float2 ml[kBatch];
        float v[kBatch][V];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const uint32_t x = xb + lanes * j;
            ml[j] = make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int e = 0; e < V; ++e) v[j][e] = 0.0f;
            if (x < n_rec) {
                const long long at = ((x < cut ? c0 + x : a.tail0) + stream) << a.side_bits;
                const long long rec = (at + rg - (set << a.side_bits)) * a.R + n;
                ml[j] = a.part_ml[rec];
                const float* p = a.part_o + rec * D + lane * V;
                if constexpr (V == 2) {
                    const float2 t = *reinterpret_cast<const float2*>(p);
                    v[j][0] = t.x;
                    v[j][1] = t.y;
                } else {
#pragma unroll
                    for (int e = 0; e < V; e += 4) {
                        const float4 t = *reinterpret_cast<const float4*>(p + e);
                        v[j][e] = t.x;
                        v[j][e + 1] = t.y;
                        v[j][e + 2] = t.z;
                        v[j][e + 3] = t.w;
                    }
                }
            }
        }
        float M = mx;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) M = fmaxf(M, ml[j].x);
        const float sc = mx == -INFINITY ? 1.0f : exp2f(mx - M);   // what the warp holds so far
        lw *= sc;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] *= sc;
        mx = M;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (ml[j].y == 0.0f) continue;   // saw nothing (or past the last record)
            const float wt = record_weight(ml[j], M);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += wt * v[j][e];
            lw += wt * ml[j].y;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) s_merge[warp * D + lane * V + e] = acc[e];
    if (lane == 0) s_ml[warp] = make_float2(mx, lw);
    __syncthreads();
    if (warp != 0) return;
    float out[V];
#pragma unroll
    for (int e = 0; e < V; ++e) out[e] = 0.0f;
#pragma unroll
    for (int mp = 0; mp < kMaps; ++mp) {
        float M = -INFINITY, Ls = 0.0f, so[V];
#pragma unroll
        for (int e = 0; e < V; ++e) so[e] = 0.0f;
        for (int k = mp; k < warps; k += kMaps) M = fmaxf(M, s_ml[k].x);
        for (int k = mp; k < warps; k += kMaps) {
            const float2 ml = s_ml[k];
            const float wt = record_weight(ml, M);
            Ls += wt * ml.y;
#pragma unroll
            for (int e = 0; e < V; ++e) so[e] += wt * s_merge[k * D + lane * V + e];
        }
        add_map<V>(out, so, M, Ls, mp, lambda, a.out, b, head, i, kMaps, lane);
        if (!kDiff && lane == 0 && a.row_ml)
            a.row_ml[(static_cast<long long>(b) * a.Hkv + hk) * ((grp * a.nq + 1) & ~1) + r] =
                make_float2(M, Ls == 0.0f ? 0.0f : 1.0f / Ls);
    }
    store_row<D>(out, gain, kDiff, a.out, b, head, i, lane);
}

// weights[slot] += sum over the group's rows of 2^(x - M) / L for every cached
// token.  A half-warp takes a tile (one token a lane) with every row group's scores of
// it, kTiles tiles at once so that their loads overlap; what it has to know of a tile
// the decode kernel left beside the scores.  The sum runs in row order in one thread and
// reaches memory by one atomic add per (token, KV head).
struct WeightArgs {
    const float* scores;
    const uint4* tiles;
    const float2* row_ml;
    const uint32_t* prefix;
    float* weights;   // [num_phys][Hkv][ps]
    int B, Hkv, G, row_groups, R, pairs, page_bits, side_bits, sets;
};

// Bound by the latency of its loads (under ncu 20% of the DRAM rate, 30% of the issue slots).  What the
// weights add to a call of 32 sequences (67,000 tiles of four rows), by tiles in flight and CTAs per SM:
// 4 and 3 19.0 us, 2 and 3 17.0, 2 and 4 15.8, 2 and 5 15.0, 1 and 6 15.9, 1 and 4 17.7.
constexpr int kWeightCtas = 5;
__global__ void __launch_bounds__(256, kWeightCtas) decode_f16_weights_kernel(const WeightArgs a) {
    constexpr int kTiles = 2;
    // A programmatic dependent of the merge, which itself waited for the decode.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t N = a.prefix[a.B] / a.sets;   // (sequence, KV head, tile) triples
    const uint32_t step = gridDim.x * 16;
    const int tok = threadIdx.x & 15, g_even = (a.G + 1) & ~1;
    for (uint32_t x0 = blockIdx.x * 16 + (threadIdx.x >> 4); x0 < N; x0 += kTiles * step) {
        uint4 info[kTiles];
        float sum[kTiles];
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
            const uint32_t x = x0 + j * step;
            info[j] = x < N ? a.tiles[x] : make_uint4(0, 0, 0, 0);
            sum[j] = 0.0f;
        }
        for (int rg = 0; rg < a.row_groups; ++rg) {
            const int set = rg >> a.side_bits, beside = rg - (set << a.side_bits);
            const int real = min(a.R, a.G - rg * a.R);
#pragma unroll 2
            for (int r = 0; r < real; r += 2) {
                float2 s[kTiles];
                float4 m[kTiles];
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    // with one row group a triple's tile has its number: no wait for info
                    const uint32_t x = x0 + j * step;
                    const long long u = a.row_groups == 1
                                            ? x
                                            : ((info[j].z + static_cast<long long>(set) * (info[j].w >> 5))
                                               << a.side_bits) + beside;
                    s[j] = make_float2(-INFINITY, -INFINITY);
                    if (x < N)
                        s[j] = *reinterpret_cast<const float2*>(
                            a.scores + (u * a.pairs + r / 2) * (2 * kTile) + 4 * (tok & 7) + 2 * (tok >> 3));
                }
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
                    m[j] = *reinterpret_cast<const float4*>(
                        a.row_ml + static_cast<long long>(info[j].y) * g_even + rg * a.R + r);
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    if (s[j].x != -INFINITY) sum[j] += fast_exp2(s[j].x - m[j].x) * m[j].y;
                    // an odd last row has no partner
                    if (s[j].y != -INFINITY && r + 1 < real) sum[j] += fast_exp2(s[j].y - m[j].z) * m[j].w;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
            if (tok >= static_cast<int>(info[j].w & 31u)) continue;
            const long long page = info[j].x >> a.page_bits;
            const int off = info[j].x & ((1u << a.page_bits) - 1u), hk = info[j].y % a.Hkv;
            atomicAdd(a.weights + ((page * a.Hkv + hk) << a.page_bits) + off + tok, sum[j]);
        }
    }
}

int rows_per_group(int G) { return G <= 8 ? 8 : 16; }

int warps_of(int D) { return D == 256 ? 4 : 8; }

// Row groups of G rows, `side` of them side by side.  Groups are streams of their own, each reading
// the cache: from memory once and from L2 for the others while the caches fit there about twice over;
// above that, groups that fill a CTA's warps evenly (2, 4, 8) take the same tiles at the same time.
// Measured, streams against side by side: 8 sequences of 10,000 to 30,000, 4 KV heads of 128, 32 rows
// (328 MB) 109 and 84 us; 16 of 3,000 to 9,000, 2 KV heads of 128, 20 rows (100 MB) 32.7 and 34.6 us.
struct RowPlan {
    int R, groups, side_bits, side, sets;
};
RowPlan row_plan(int G, int D, int B, int Hkv, int max_kv) {
    RowPlan p{};
    p.R = rows_per_group(G);
    p.groups = (G + p.R - 1) / p.R;
    const bool large = static_cast<double>(B) * Hkv * max_kv * D * 4 > 256e6;
    p.side = large && p.groups <= warps_of(D) && warps_of(D) % p.groups == 0 ? p.groups : 1;
    while ((1 << p.side_bits) < p.side) ++p.side_bits;
    p.sets = p.groups / p.side;
    return p;
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

// Workspace: partial records, one per CTA and two per stream (of each row group), the (B + 1)-entry
// tile prefix and, for the weights, every row's (max, 1 / sum) and the description
// and scores of every tile that max_kv_len allows.
struct Layout {
    size_t tail0, o, ml, prefix, row_ml, tiles, scores, total;
};

// Pairs of rows whose scores a tile of a row group has.
int row_pairs(int groups, int R, int G) { return groups > 1 ? R / 2 : (G + 1) / 2; }

Layout decode_layout(long long ctas, int B, int Hkv, int G, int max_kv, int D, bool weights) {
    const RowPlan rows = row_plan(G, D, B, Hkv, max_kv);
    const int R = rows.R;
    const size_t streams = static_cast<size_t>(B) * Hkv * rows.sets;
    const size_t recs = (static_cast<size_t>(ctas) + 2 * streams) * rows.side;
    Layout l{};
    l.tail0 = static_cast<size_t>(ctas) + streams;
    size_t at = 0;
    l.o = at;
    at += recs * R * D * 4;
    l.ml = at;
    at += recs * R * 8;
    l.prefix = at;
    at += round16((static_cast<size_t>(B) + 1) * 4);
    l.row_ml = at;
    if (weights) at += static_cast<size_t>(B) * Hkv * ((G + 1) & ~1) * 8;
    const size_t triples = static_cast<size_t>(B) * Hkv * ((static_cast<size_t>(max_kv) + kTile - 1) / kTile);
    const size_t tiles = triples * rows.groups;
    l.tiles = at;
    if (weights) at += triples * 16;
    l.scores = at;
    if (weights) at += tiles * row_pairs(rows.groups, R, G) * (2 * kTile * 4);
    l.total = at + 16;
    return l;
}

int sm_count_or_default() {
    DeviceState d;
    return current_device(&d) == GBATTN_OK ? d.num_sms : 152;
}

size_t decode_workspace_size(int B, int Hq, int Hkv, int nq, int max_kv, int D, int maps,
                             bool weights) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || nq <= 0 || max_kv <= 0 || D <= 0 || Hq % Hkv != 0) return 0;
    const long long G = static_cast<long long>(Hq / Hkv) * nq * maps;
    if (G > 0x7FFFFFFFLL) return 0;
    return decode_layout(sm_count_or_default(), B, Hkv, static_cast<int>(G), max_kv, D, weights).total;
}

// How many clusters of 1, 2, 4 and 8 CTAs of the one-kernel form run at once on a device: a CTA takes an SM,
// and a cluster's SMs lie in one GPC (152 SMs hold 152, 76, 36 and 15).  null: the device refused.
template <int D, int NB>
const int* resident_clusters(int device) {
    static std::once_flag once[64];
    static int n[64][4];
    static bool ok[64];
    if (device < 0 || device >= 64) return nullptr;
    std::call_once(once[device], [&] {
        auto* kernel = decode_f16_kernel<D, NB, true>;
        ok[device] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          Cfg<D>::kSmem) == cudaSuccess;
        for (int i = 0; i < 4 && ok[device]; ++i) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(1u << i);
            cfg.blockDim = dim3(Cfg<D>::kThreads);
            cfg.dynamicSmemBytes = Cfg<D>::kSmem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << i;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            ok[device] = cudaOccupancyMaxActiveClusters(&n[device][i], kernel, &cfg) == cudaSuccess;
        }
        if (!ok[device]) cudaGetLastError();
    });
    return ok[device] ? n[device] : nullptr;
}
const int* resident_clusters(int D, int R, int device) {
    if (D == 64) return R == 8 ? resident_clusters<64, 1>(device) : resident_clusters<64, 2>(device);
    if (D == 128) return R == 8 ? resident_clusters<128, 1>(device) : resident_clusters<128, 2>(device);
    return R == 8 ? resident_clusters<256, 1>(device) : resident_clusters<256, 2>(device);
}

// CTAs of a cluster when every stream gets one (kOne), 0 when the streams' tiles are laid end to end.  A
// cluster saves the merge kernel, the tile prefix and the records' way through memory, but its SMs read
// one stream only, whatever the others' lengths, and its warps add the weights of their own tiles one
// after the other.  So where all clusters run at once, the largest that do, and max_kv_len gives a warp
// at most `per_warp` tiles.  Measured, clusters against laid end to end, in us (streams: sequences with
// one KV head of four rows, one length unless said):
//   D = 128   1 stream 4,096 tokens 9.7 and 11.1, 8,192 11.9 and 11.2; 15 streams 6,144 13.0 and 16.1; 32
//             of half to all of 2,048 9.7 and 13.7; 152 of half to all of 768 11.8 and 17.0
//   D = 64    1 stream 8,192 9.9 and 10.8, 12,288 12.1 and 11.1; 8 streams 12,288 12.1 and 13.1; 152 of
//             half to all of 1,536 13.2 and 18.5
//   D = 256   1 stream 512 8.8 and 8.2; 8 streams 8.9 and 9.5; 15 streams 9.4 and 10.3
//   weights   D = 128: 8 streams 2,048 11.1 and 12.1, 4,096 13.8 and 12.8; 15 of 6,144 6% less, 8 tiles a
//             warp no gain; 152 of half to all of 768 16.4 and 19.3, of 1,536 27.3 and 25.8.  D = 64 alike.
//             D = 256: 1 stream 512 10.6 and 10.7, 8 streams 11.0 and 11.9
// With clusters of eight for up to 19 streams (152 SMs, of which 15 such clusters fit) 16 streams of half to
// all of 512 took 13.2 us, in two waves; end to end takes 10.1, clusters of four 7.2.
int cluster_of(long long streams, int max_kv, int D, bool weights, const int* resident) {
    static_assert(kMaxCluster == 8, "resident_clusters asks for up to eight CTAs");
    int bits = 3;
    while (bits > 0 && streams > resident[bits]) --bits;
    if (streams > resident[bits]) return 0;
    const int per_warp = weights    ? D == 256 ? 1 : streams < 12 ? 2 : 6
                         : D == 64  ? streams < 8 ? 8 : 12
                         : D == 128 ? 6
                                    : streams < 8 ? 0 : 1;
    const int tiles = (max_kv + kTile - 1) / kTile;
    return tiles <= per_warp * (warps_of(D) << bits) ? 1 << bits : 0;
}

template <int D, int NB, bool kOne>
int launch_decode(const CUtensorMap& tk, const CUtensorMap& tv, int ctas, int cluster,
                  const DecodeF16Args& a, cudaStream_t s) {
    static std::once_flag once[64];
    static int rc[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GBATTN_ERR_CUDA;
    auto* kernel = decode_f16_kernel<D, NB, kOne>;
    std::call_once(once[dev], [&] {
        rc[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D>::kSmem) == cudaSuccess
                      ? GBATTN_OK
                      : GBATTN_ERR_CUDA;
    });
    if (rc[dev] != GBATTN_OK) return rc[dev];
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(Cfg<D>::kThreads);
    cfg.dynamicSmemBytes = Cfg<D>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kOne ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tk, tv, a);
    count_launches(1);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GBATTN_ERR_CUDA;
    }
    return launch_status();
}

// cluster: CTAs of a stream's cluster, or 0.
template <int D>
int launch_decode_rows(int R, const CUtensorMap& tk, const CUtensorMap& tv, int ctas, int cluster,
                       const DecodeF16Args& a, cudaStream_t s) {
    if (cluster)
        return R == 8 ? launch_decode<D, 1, true>(tk, tv, ctas, cluster, a, s)
                      : launch_decode<D, 2, true>(tk, tv, ctas, cluster, a, s);
    return R == 8 ? launch_decode<D, 1, false>(tk, tv, ctas, 1, a, s)
                  : launch_decode<D, 2, false>(tk, tv, ctas, 1, a, s);
}

// A launch whose CTAs may be placed while the grid before it on the stream still
// runs; the kernel waits for that grid itself (griddepcontrol.wait).
template <typename Args>
int launch_dependent(void (*kernel)(Args), dim3 grid, int threads, size_t smem, cudaStream_t s,
                     const Args& args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
    count_launches(1);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GBATTN_ERR_CUDA;
    }
    return launch_status();
}

struct DecodeCall {
    const void *q, *k_pages, *v_pages;
    const int32_t *page_table, *kv_lens;
    void* o;
    float *lse, *weights;
    int B, Hq, Hkv, nq, D, num_phys, ps, max_pages, max_kv;
    float scale;
    void* workspace;
    size_t workspace_bytes;
    void* stream;
    const DiffArgs* diff;   // null: ordinary attention
};

int run_decode(const DecodeCall& c) {
    if (!c.q || !c.k_pages || !c.v_pages || !c.page_table || !c.kv_lens || !c.o)
        return GBATTN_ERR_NULL;
    if (c.diff && !c.diff->vecs) return GBATTN_ERR_NULL;
    if (c.B <= 0 || c.Hq <= 0 || c.Hkv <= 0 || c.nq <= 0 || c.num_phys <= 0 || c.ps <= 0 ||
        c.max_pages <= 0 || c.max_kv <= 0)
        return GBATTN_ERR_SHAPE;
    if (c.Hq % c.Hkv != 0 || c.max_kv > (1 << 30) ||
        static_cast<long long>(c.max_kv) > static_cast<long long>(c.max_pages) * c.ps)
        return GBATTN_ERR_SHAPE;
    if (c.diff && c.diff->heads != 1 && c.diff->heads != c.Hq) return GBATTN_ERR_SHAPE;
    if (c.diff ? c.D != 128 : (c.D != 64 && c.D != 128 && c.D != 256)) return GBATTN_ERR_UNSUPPORTED;
    if (c.ps < kTile || (c.ps & (c.ps - 1)) != 0 ||
        static_cast<long long>(c.num_phys) * c.ps > 0x7FFFFFFFLL)
        return GBATTN_ERR_UNSUPPORTED;
    if (c.B > kMaxSeqs) return GBATTN_ERR_UNSUPPORTED;
    const int maps = c.diff ? 2 : 1;
    const long long rows = static_cast<long long>(c.B) * c.Hq * c.nq;
    const long long G64 = static_cast<long long>(c.Hq / c.Hkv) * c.nq * maps;
    if (rows * maps > 0x7FFFFFFFLL || G64 > 0x7FFFFFFFLL) return GBATTN_ERR_SHAPE;
    const int G = static_cast<int>(G64);
    const RowPlan plan = row_plan(G, c.D, c.B, c.Hkv, c.max_kv);
    const int R = plan.R;
    const long long streams = static_cast<long long>(c.B) * c.Hkv * plan.sets * plan.side;
    if (streams > 0x7FFFFFFFLL ||
        streams * ((static_cast<long long>(c.max_kv) + kTile - 1) / kTile) > 0x7FFFFFFFLL)
        return GBATTN_ERR_SHAPE;
    if (!finite_positive(c.scale)) return GBATTN_ERR_SCALE;
    if (c.diff && (!(fabsf(c.diff->init) <= 3.402823466e38f) ||
                   (c.diff->norm && !finite_positive(c.diff->eps))))
        return GBATTN_ERR_SCALE;
    auto misaligned4 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
    if (!aligned16(c.q) || !aligned16(c.k_pages) || !aligned16(c.v_pages) || !aligned16(c.o) ||
        !aligned16(c.workspace) || misaligned4(c.page_table) || misaligned4(c.kv_lens) ||
        misaligned4(c.lse) || misaligned4(c.weights) ||
        (c.diff && (misaligned4(c.diff->vecs) || misaligned4(c.diff->norm))))
        return GBATTN_ERR_ALIGN;
    struct Range { const void* p; size_t n; };
    const size_t slots = static_cast<size_t>(c.num_phys) * c.ps * c.Hkv;
    const Range in[] = {{c.q, static_cast<size_t>(rows) * c.D * 2},
                        {c.k_pages, slots * c.D * 2},
                        {c.v_pages, slots * c.D * 2},
                        {c.page_table, static_cast<size_t>(c.B) * c.max_pages * 4},
                        {c.kv_lens, static_cast<size_t>(c.B) * 4},
                        {c.diff ? c.diff->vecs : nullptr,
                         c.diff ? static_cast<size_t>(c.diff->heads) * 4 * (c.D / 2) * 4 : 0},
                        {c.diff ? c.diff->norm : nullptr, static_cast<size_t>(c.D) * 4}};
    const Range out[] = {{c.o, static_cast<size_t>(rows) * c.D * 2},
                         {c.lse, static_cast<size_t>(rows) * maps * 4},
                         {c.weights, slots * 4}};
    auto clash = [&](const Range& x) {
        for (const Range& y : in)
            if (overlaps(x.p, x.n, y.p, y.n)) return true;
        return false;
    };
    for (int i = 0; i < 3; ++i) {
        if (clash(out[i])) return GBATTN_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return GBATTN_ERR_ALIAS;
    }
    if (!c.workspace) return GBATTN_ERR_WORKSPACE;
    DeviceState dev;
    int rc = current_device(&dev);
    if (rc != GBATTN_OK) return rc;

    // One CTA per SM; fewer when the workspace holds fewer records.
    auto layout = [&](long long ctas) {
        return decode_layout(ctas, c.B, c.Hkv, G, c.max_kv, c.D, c.weights != nullptr);
    };
    long long ctas = dev.num_sms;
    while (ctas > 1 && layout(ctas).total > c.workspace_bytes) --ctas;
    const Layout lay = layout(ctas);
    if (lay.total > c.workspace_bytes) return GBATTN_ERR_WORKSPACE;
    const Range ws{c.workspace, lay.total};
    if (clash(ws)) return GBATTN_ERR_ALIAS;
    for (const Range& x : out)
        if (overlaps(ws.p, ws.n, x.p, x.n)) return GBATTN_ERR_ALIAS;

    CUtensorMap tk, tv;
    const uint64_t total_rows = static_cast<uint64_t>(c.num_phys) * c.ps;
    if (encode_tmap_f16_pages(&tk, c.k_pages, c.D, c.Hkv, total_rows, kTile) != GBATTN_OK ||
        encode_tmap_f16_pages(&tv, c.v_pages, c.D, c.Hkv, total_rows, kTile) != GBATTN_OK)
        return GBATTN_ERR_CUDA;

    uint8_t* wsp = static_cast<uint8_t*>(c.workspace);
    DecodeF16Args a{};
    a.q = static_cast<const __half*>(c.q);
    a.table = c.page_table;
    a.kv_lens = c.kv_lens;
    a.part_o = reinterpret_cast<float*>(wsp + lay.o);
    a.part_ml = reinterpret_cast<float2*>(wsp + lay.ml);
    a.tail0 = static_cast<long long>(lay.tail0);
    a.prefix_out = reinterpret_cast<uint32_t*>(wsp + lay.prefix);
    a.scores = c.weights ? reinterpret_cast<float*>(wsp + lay.scores) : nullptr;
    a.tiles = reinterpret_cast<uint4*>(wsp + lay.tiles);
    a.status = dev.status;
    a.wait_limit = wait_limit_ns();
    a.fault = fault_mode();
    a.B = c.B;
    a.Hq = c.Hq;
    a.Hkv = c.Hkv;
    a.nq = c.nq;
    a.G = G;
    a.side_bits = plan.side_bits;
    a.sets = plan.sets;
    a.pairs = row_pairs(plan.groups, R, G);
    a.num_phys = c.num_phys;
    a.ps = c.ps;
    a.max_pages = c.max_pages;
    a.max_kv = c.max_kv;
    a.maps = maps;
    a.sl2 = c.scale * 1.4426950408889634f;
    a.weights = c.weights;
    a.out = RowOut{static_cast<__half*>(c.o), c.lse, c.Hq, c.nq, c.diff ? *c.diff : DiffArgs{}};
    cudaStream_t s = static_cast<cudaStream_t>(c.stream);
    // (row groups of their own would add to the weights in any order)
    int cl = 0;
    if (plan.side == 1 && !(c.weights && plan.groups > 1)) {
        const int* resident = resident_clusters(c.D, R, dev.device);
        if (!resident) return GBATTN_ERR_CUDA;
        cl = cluster_of(streams, c.max_kv, c.D, c.weights != nullptr, resident);
    }
    const int n = static_cast<int>(cl ? streams * cl : ctas);
    rc = c.D == 64    ? launch_decode_rows<64>(R, tk, tv, n, cl, a, s)
         : c.D == 128 ? launch_decode_rows<128>(R, tk, tv, n, cl, a, s)
                      : launch_decode_rows<256>(R, tk, tv, n, cl, a, s);
    if (rc != GBATTN_OK || cl) return rc;

    MergeArgs m{};
    m.part_o = a.part_o;
    m.part_ml = a.part_ml;
    m.prefix = a.prefix_out;
    m.kv_lens = c.kv_lens;
    m.max_kv = c.max_kv;
    m.B = c.B;
    m.Hq = c.Hq;
    m.Hkv = c.Hkv;
    m.nq = c.nq;
    m.side_bits = plan.side_bits;
    m.sets = plan.sets;
    m.R = R;
    m.tail0 = a.tail0;
    m.grid = static_cast<uint32_t>(ctas);
    m.parts = static_cast<uint32_t>(warps_of(c.D) / plan.side);
    m.out = a.out;
    m.row_ml = c.weights ? reinterpret_cast<float2*>(wsp + lay.row_ml) : nullptr;
    // Warps per row by the records of an average row (a map of a row): one up to a batch of 8.
    const long long recs = ctas * plan.side / streams + 1;
    const int mw = (recs > 32 ? 8 : recs > 8 ? 4 : 1) * maps;
    const dim3 mgrid(static_cast<unsigned>(rows));
    const size_t msmem = static_cast<size_t>(mw) * (c.D * sizeof(float) + sizeof(float2));
    rc = c.diff       ? launch_dependent(decode_f16_merge_kernel<128, true>, mgrid, 32 * mw, msmem, s, m)
         : c.D == 64  ? launch_dependent(decode_f16_merge_kernel<64, false>, mgrid, 32 * mw, msmem, s, m)
         : c.D == 128 ? launch_dependent(decode_f16_merge_kernel<128, false>, mgrid, 32 * mw, msmem, s, m)
                      : launch_dependent(decode_f16_merge_kernel<256, false>, mgrid, 32 * mw, msmem, s, m);
    if (rc != GBATTN_OK || !c.weights) return rc;

    WeightArgs x{};
    x.scores = a.scores;
    x.tiles = a.tiles;
    x.row_ml = m.row_ml;
    x.prefix = a.prefix_out;
    x.weights = c.weights;
    x.B = c.B;
    x.Hkv = c.Hkv;
    x.G = G;
    x.row_groups = plan.groups;
    x.side_bits = plan.side_bits;
    x.sets = plan.sets;
    x.R = R;
    x.pairs = a.pairs;
    x.page_bits = 0;
    while ((1 << x.page_bits) < c.ps) ++x.page_bits;
    const long long tiles = static_cast<long long>(c.B) * c.Hkv * ((c.max_kv + kTile - 1) / kTile);
    const long long want = (tiles + 15) / 16;
    const unsigned grid = static_cast<unsigned>(want < 1LL * kWeightCtas * dev.num_sms ? want : 1LL * kWeightCtas * dev.num_sms);
    return launch_dependent(decode_f16_weights_kernel, dim3(grid), 256, 0, s, x);
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" size_t attn_paged_decode_f16_workspace_size(int B, int Hq, int Hkv, int nq,
                                                       int max_kv_len, int D, int weights) {
    return decode_workspace_size(B, Hq, Hkv, nq, max_kv_len, D, 1, weights != 0);
}

extern "C" int attn_paged_decode_f16_fwd(const void* q, const void* k_pages, const void* v_pages,
                                         const int32_t* page_table, const int32_t* kv_lens, void* o,
                                         float* lse, float* weights, int B, int Hq, int Hkv, int nq,
                                         int D, int num_phys_pages, int page_size, int max_pages,
                                         int max_kv_len, float scale, void* workspace,
                                         size_t workspace_bytes, void* stream) {
    CallRange nvtx_range("attn_paged_decode_f16_fwd");
    return run_decode({q, k_pages, v_pages, page_table, kv_lens, o, lse, weights, B, Hq, Hkv, nq, D,
                       num_phys_pages, page_size, max_pages, max_kv_len, scale, workspace,
                       workspace_bytes, stream, nullptr});
}

extern "C" size_t attn_diff_paged_decode_f16_workspace_size(int B, int Hq, int Hkv, int nq,
                                                            int max_kv_len, int D) {
    return decode_workspace_size(B, Hq, Hkv, nq, max_kv_len, D, 2, false);
}

extern "C" int attn_diff_paged_decode_f16_fwd(const void* q, const void* k_pages,
                                              const void* v_pages, const int32_t* page_table,
                                              const int32_t* kv_lens, const float* lambda_vecs,
                                              int lambda_heads, float lambda_init,
                                              const float* norm_weight, float eps, void* o,
                                              float* lse, int B, int Hq, int Hkv, int nq, int D,
                                              int num_phys_pages, int page_size, int max_pages,
                                              int max_kv_len, float scale, void* workspace,
                                              size_t workspace_bytes, void* stream) {
    CallRange nvtx_range("attn_diff_paged_decode_f16_fwd");
    const DiffArgs diff{lambda_vecs, norm_weight, lambda_heads, lambda_init, eps};
    return run_decode({q, k_pages, v_pages, page_table, kv_lens, o, lse, nullptr, B, Hq, Hkv, nq, D,
                       num_phys_pages, page_size, max_pages, max_kv_len, scale, workspace,
                       workspace_bytes, stream, &diff});
}
