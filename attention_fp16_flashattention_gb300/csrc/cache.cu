// The paged KV cache around the decode kernels: new tokens are appended to the
// pages, and tokens that received little attention are evicted.  The pages name
// the cache and its page table ("Integrate FP32 v37 prefill and exact E4M3
// bridge", Implementation: paged cache, live length); how it is filled and kept
// within a budget is this library's own.
//
// Both are copies: nothing but bytes moves, so HBM bounds them.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <mutex>

#include "host.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace gbattn {
namespace {

// ---------------------------------------------------------------- append

struct AppendArgs {
    const uint4 *k, *v;          // new rows, 16-byte chunks
    uint4 *k_pages, *v_pages;
    const int32_t *table, *kv_lens, *new_lens;
    float* weights;              // [num_phys][Hkv][ps] or null
    uint32_t* status;
    long long k_sb, k_sh, k_sr;  // source strides in chunks (k and v share them)
    int n, Hkv, chunk_bits, num_phys, ps, max_pages;
};

constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;   // chunks of K and of V in flight per thread

// One thread moves 16-byte chunk c of head h of new token i (chunks of one token are
// contiguous in the page: h and c are the fast indexes), kAppendUnroll of them
// blockDim apart.  Four prompts of 4,096 to 8,192 tokens (8 KV heads of 128, 226 MB) take
// 35 us, 0.95 of the measured copy rate; one token for each of 64 sequences 1.8 us.
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a) {
    const int b = blockIdx.y;
    const int len = a.kv_lens[b];
    const int count = a.new_lens ? a.new_lens[b] : a.n;
    if (count < 0 || count > a.n || len < count ||
        len > static_cast<long long>(a.max_pages) * a.ps) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, kDevBadLength);
        return;
    }
    const int row_chunks = a.Hkv << a.chunk_bits;
    const long long total = static_cast<long long>(count) * row_chunks;
    long long x = static_cast<long long>(blockIdx.x) * (kAppendThreads * kAppendUnroll) + threadIdx.x;
    uint4 kv[kAppendUnroll], vv[kAppendUnroll];
    long long dst[kAppendUnroll];
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u, x += kAppendThreads) {
        dst[u] = -1;
        if (x >= total) continue;
        const int i = static_cast<int>(x / row_chunks);
        const int hc = static_cast<int>(x - static_cast<long long>(i) * row_chunks);
        const int h = hc >> a.chunk_bits, c = hc & ((1 << a.chunk_bits) - 1);
        const int token = len - count + i;
        const int page = a.table[static_cast<long long>(b) * a.max_pages + token / a.ps];
        if (page < 0 || page >= a.num_phys) {
            atomicOr(a.status, kDevBadPage);
            continue;
        }
        const long long slot = token % a.ps;
        const long long src = b * a.k_sb + h * a.k_sh + i * a.k_sr + c;
        kv[u] = a.k[src];
        vv[u] = a.v[src];
        dst[u] = (static_cast<long long>(page) * a.ps + slot) * row_chunks + hc;
        if (a.weights && c == 0)
            a.weights[(static_cast<long long>(page) * a.Hkv + h) * a.ps + slot] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u) {
        if (dst[u] < 0) continue;
        a.k_pages[dst[u]] = kv[u];
        a.v_pages[dst[u]] = vv[u];
    }
}

// ---------------------------------------------------------------- eviction
//
// Selection.  One cluster of 1..8 CTAs takes one (sequence, KV head).  Of its L > budget
// slots the first `sink` and the last `recent` stay, and of the middle the M = budget -
// sink - recent heaviest.  The M-th largest weight is found by radix selection on
// order-preserving 32-bit keys, by digits of 11, 11 and 10 bits.  For the first, each CTA
// counts its part of the slots (keys held in shared memory) into 2048 bins and adds the
// counts to every CTA of the cluster.  Eleven bits hold the sign, the exponent and two bits
// of the mantissa, so the bin that holds the M-th has a few percent of the keys as a rule:
// the CTAs exchange those, and each counts the other digits by itself.  Where most weights
// are alike they pass the lists, and the counts are exchanged for every digit.  Keys above
// the M-th are kept, and of those equal to it the first slots up to M.  Prefix counts over
// warps and CTAs give every kept slot its place, in slot order.
//
// Moving.  Into other pages a second kernel copies the rows, shared evenly over the GPU's
// warps whatever the number of heads.  In place a row's new slot j is never above its old
// one, so rows may move in steps of consecutive j: a step's reads end (cluster barrier)
// before its writes begin, and a write of this step lands below every later step's reads,
// which may therefore run ahead; the cluster that selected moves its own rows.
//
// Bound by HBM: the kept rows read and written.  16 sequences of about 1,100 tokens kept to
// 1,024 (8 KV heads of 128, 136 MB): 7.5 us of selection, half of it the wait for lengths, pages
// and weights, one behind the other, and 20 us of copies (6.7 TB/s), 31 us in all.  4 of
// 20,011 to 32,768 kept to 8,192 (274 MB): 15 us in clusters of eight and 40 us, 63 us in all
// (67 with the counts of every digit exchanged; 66 and 77 in clusters of four and two); in
// place 76 us (and the former 38).

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictStages = 6;          // row steps in flight per thread
constexpr int kEvictMaxCluster = 8;
// Shared memory: the ring (K and V chunks, a weight per row) or the keys, 99 KB: two CTAs per SM.
constexpr int kEvictRing = kEvictStages * kEvictThreads * (2 * 16 + 1);   // >= 4 chunks a row
constexpr int kDigits = 3, kBins = 2048;   // 11, 11 and 10 bits of the key
constexpr int kEvictMaxKeys = kEvictRing / 4 - (kDigits + 1) * kBins;
static_assert(kBins == 4 * kEvictThreads, "four bins a thread");

struct EvictArgs {
    uint4 *k_pages, *v_pages;
    float* weights;             // [num_phys][Hkv][ps]
    const int32_t *table, *dst_table, *kv_lens;
    int32_t *new_lens, *kept;   // [B], [B][Hkv][budget]
    uint32_t* status;
    int Hkv, chunk_bits, page_bits, num_phys, ps, max_pages, dst_pages, max_kv, budget, sink, recent;
    int keys;                   // capacity of the CTA's key array
};

// Larger key = larger weight; NaN is below everything, -0 equals 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w == 0.0f ? 0.0f : w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Writes new_lens and kept[] of the cluster's (sequence, KV head).  False: nothing is to be
// moved (the same answer in every CTA of the cluster).
template <bool kInPlace>
__device__ __forceinline__ bool evict_select(const EvictArgs& a, uint32_t* s_dyn,
                                             cg::cluster_group& cluster) {
    uint32_t* s_total = s_dyn;                          // [kDigits][kBins] of the whole cluster
    uint32_t* s_hist = s_total + kDigits * kBins;       // [kBins] of this CTA
    uint32_t* s_keys = s_hist + kBins;                  // [a.keys]; behind the first min(per, keys) the
                                                        // cluster's keys of the chosen first digit
    __shared__ uint32_t s_pick[2];                      // digit, keys still wanted at it
    __shared__ uint2 s_warp[kEvictWarps], s_cta;        // (above, equal) counts
    __shared__ uint32_t s_bad, s_own;                   // s_own: keys this CTA has listed
    const int C = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long stream = blockIdx.x / C;
    const int b = static_cast<int>(stream / a.Hkv), h = static_cast<int>(stream - static_cast<long long>(b) * a.Hkv);
    const int32_t* table = a.table + static_cast<long long>(b) * a.max_pages;
    const int32_t* dst_table = a.dst_table + static_cast<long long>(b) * a.dst_pages;
    int32_t* kept = a.kept + stream * a.budget;
    const int L = a.kv_lens[b];
    const int first = rank * kEvictThreads + tid, step = C * kEvictThreads;

    const bool bad_len = L < 0 || L > a.max_kv;
    if (bad_len && first == 0) atomicOr(a.status, kDevBadLength);
    const int n = bad_len ? 0 : min(L, a.budget);
    const int want = !bad_len && L > a.budget ? n - a.sink - a.recent : 0;   // M
    // this CTA's part [lo, hi) of the middle slots
    const int mid = want > 0 ? L - a.sink - a.recent : 0;
    const int per = (mid + C - 1) / C;
    const int lo = min(rank * per, mid), hi = min(lo + per, mid);
    const bool together = C > 1 && want > 0;   // the cluster's CTAs exchange anything at all
    for (int x = tid; x < (kDigits + 1) * kBins; x += kEvictThreads) s_total[x] = 0;   // s_hist too
    if (tid == 0) s_bad = s_own = 0;
    if (together) cluster.barrier_arrive();    // waited for before the first remote access
    uint32_t* s_list = s_keys + min(per, a.keys);
    auto weight_at = [&](int t) -> float* {
        return a.weights + ((static_cast<long long>(table[t >> a.page_bits]) * a.Hkv + h) << a.page_bits) +
               (t & (a.ps - 1));
    };
    auto key_at = [&](int i) -> uint32_t {   // i relative to lo
        return i < a.keys ? s_keys[i] : weight_key(*weight_at(a.sink + lo + i));
    };

    // ---- the keys of this CTA's part, and whether any page is out of range
    bool bad = false;
    if (!bad_len) {
        const int held = min(hi - lo, a.keys);
        // The pages of every slot whose weight is not loaded here, one after the other: with a middle
        // those of the sinks, of the recent and of what the key array does not hold, else all; then the
        // destination's.  The first of them are on their way before the weights.
        auto pages_to = [&](int t) -> int { return (t + a.ps - 1) >> a.page_bits; };
        const int p0 = mid == 0 ? pages_to(L) : pages_to(a.sink);
        const int at1 = (L - a.recent) >> a.page_bits, p1 = mid == 0 ? 0 : pages_to(L) - at1;
        const int at2 = (a.sink + lo + held) >> a.page_bits;
        const int p2 = mid == 0 || held == hi - lo ? 0 : pages_to(a.sink + hi) - at2;
        const int p3 = kInPlace ? 0 : pages_to(n);
        // A destination that is the sequence's own page of the same place, as in a copy of the page table,
        // would be written while it is read: refused like a page out of range, wherever the call reads
        // that page (all of a cache within the budget or with weights to compare, else sinks and recent).
        const bool read_all = L <= a.budget || want > 0;
        const int sinks_end = pages_to(a.sink), recent_at = (L - a.recent) >> a.page_bits;
        auto destination = [&](int x) -> int {
            const int page = dst_table[x];
            return page == table[x] && (read_all || x < sinks_end || x >= recent_at) ? -1 : page;
        };
        auto page_at = [&](int x) -> int {
            if (x < p0) return table[x];
            if ((x -= p0) < p1) return table[at1 + x];
            if ((x -= p1) < p2) return table[at2 + x];
            return (x -= p2) < p3 ? destination(x) : 0;
        };
        const int early = page_at(tid);
        // eight weights a thread at a time, so that the loads (each behind a page-table
        // entry) wait together
        for (int i0 = tid; i0 < held; i0 += 8 * kEvictThreads) {
            int page[8];
            float wt[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e * kEvictThreads;
                page[e] = i < held ? table[(a.sink + lo + i) >> a.page_bits] : 0;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e * kEvictThreads;
                const bool out = page[e] < 0 || page[e] >= a.num_phys;
                bad |= out;
                wt[e] = 0.0f;
                if (i < held && !out)
                    wt[e] = a.weights[((static_cast<long long>(page[e]) * a.Hkv + h) << a.page_bits) +
                                      ((a.sink + lo + i) & (a.ps - 1))];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e * kEvictThreads;
                if (i < held) s_keys[i] = weight_key(wt[e]);
            }
        }
        bad |= early < 0 || early >= a.num_phys;
        for (int x = tid + kEvictThreads; x < p0 + p1 + p2 + p3; x += kEvictThreads) {
            const int page = page_at(x);
            bad |= page < 0 || page >= a.num_phys;
        }
    }
    bad = __syncthreads_or(bad) != 0;

    // ---- the first digit, over the whole cluster.  Its CTAs checked different pages: what one
    // found goes to all of them on the way.
    auto count_keys = [&](uint32_t* hist, int pass, uint32_t chosen) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        const int above_shift = pass == 1 ? 21 : 10;   // of the digits chosen so far
        for (int i = tid; i < hi - lo; i += kEvictThreads) {
            const uint32_t key = key_at(i);
            if (pass == 0 || (key >> above_shift) == chosen) atomicAdd(&hist[(key >> shift) & mask], 1u);
        }
    };
    auto share_counts = [&](uint32_t* total) {   // few bins are in use: theirs go to every CTA
        for (int x = tid; x < kBins; x += kEvictThreads) {
            const uint32_t count = s_hist[x];
            if (count)
                for (int r = 0; r < C; ++r) atomicAdd(cluster.map_shared_rank(total, r) + x, count);
        }
    };
    if (want > 0 && (together || !bad)) {
        if (!bad) count_keys(together ? s_hist : s_total, 0, 0);   // (it may look pages up again)
        __syncthreads();
        if (together) {
            cluster.barrier_wait();
            if (bad && tid < C) *cluster.map_shared_rank(&s_bad, tid) = 1;
            share_counts(s_total);
            cluster.sync();
            bad = s_bad != 0;
        }
    }
    if (bad && first == 0) atomicOr(a.status, kDevBadPage);
    bad |= bad_len;

    // ---- a sequence whose length or pages are out of range stays as it is
    if (h == 0 && first == 0) a.new_lens[b] = bad ? L : n;
    for (int j = (bad ? 0 : n) + first; j < a.budget; j += step) kept[j] = -1;
    if (bad) return false;
    if (L <= a.budget) {
        for (int j = first; j < n; j += step) kept[j] = j;
        if (kInPlace) return false;
    } else {
        for (int j = first; j < a.sink; j += step) kept[j] = j;
        for (int j = first; j < a.recent; j += step) kept[n - a.recent + j] = L - a.recent + j;
        if (want > 0) {
            uint32_t chosen = 0, left = static_cast<uint32_t>(want);
            uint32_t gathered = 0;   // keys of the chosen first digit, in s_list behind the CTA's own
#pragma unroll 1
            for (int pass = 0; pass < kDigits; ++pass) {
                uint32_t* total = s_total + pass * kBins;
                if (pass > 0 && gathered > 0) {   // every CTA counts the cluster's few by itself
                    const int shift = pass == 1 ? 10 : 0, above_shift = pass == 1 ? 21 : 10;
                    const uint32_t mask = pass == 1 ? 2047u : 1023u;
                    for (uint32_t i = tid; i < gathered; i += kEvictThreads) {
                        const uint32_t key = s_list[gathered + i];
                        if ((key >> above_shift) == chosen) atomicAdd(&total[(key >> shift) & mask], 1u);
                    }
                    __syncthreads();
                } else if (pass > 0 && C > 1) {
                    for (int x = tid; x < kBins; x += kEvictThreads) s_hist[x] = 0;
                    __syncthreads();
                    count_keys(s_hist, pass, chosen);
                    __syncthreads();
                    share_counts(total);
                    cluster.sync();
                } else if (pass > 0) {
                    count_keys(total, pass, chosen);
                    __syncthreads();
                }
                // the bin that holds the left-th largest key: four bins a thread, from the top
                const int top = kBins - 4 - 4 * tid;
                const uint4 bins = *reinterpret_cast<const uint4*>(total + top);
                const uint32_t own = bins.x + bins.y + bins.z + bins.w;
                uint32_t incl = own;
#pragma unroll
                for (int sh = 1; sh < 32; sh <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, sh);
                    if (lane >= sh) incl += y;
                }
                if (lane == 31) s_warp[warp].x = incl;
                __syncthreads();
                for (int k = 0; k < warp; ++k) incl += s_warp[k].x;
                uint32_t above = incl - own;
                if (above < left && left <= incl) {
                    const uint32_t count[4] = {bins.w, bins.z, bins.y, bins.x};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (above < left && left <= above + count[e]) {
                            s_pick[0] = top + 3 - e;
                            s_pick[1] = left - above;
                        }
                        above += count[e];
                    }
                }
                __syncthreads();
                const uint32_t digit = s_pick[0];
                chosen = (chosen << (pass == 2 ? 10 : 11)) | digit;
                left = s_pick[1];
                // The keys of the chosen first digit are few unless most weights are alike.  Every CTA
                // lists its own, then reads all lists, and the other digits need no more of the cluster.
                if (C > 1 && pass == 0 &&
                    2 * total[digit] <= static_cast<uint32_t>(a.keys - min(per, a.keys))) {
                    gathered = total[digit];
                    for (int i = tid; i < hi - lo; i += kEvictThreads) {
                        const uint32_t key = key_at(i);
                        if ((key >> 21) == digit) s_list[atomicAdd(&s_own, 1u)] = key;
                    }
                    cluster.sync();
                    const int warps = kEvictWarps / C, r = warp / warps;   // a list's warps, and the list
                    const uint32_t own = lane < C ? *cluster.map_shared_rank(&s_own, lane) : 0u;
                    const uint32_t before = __reduce_add_sync(0xffffffffu, lane < r ? own : 0u);
                    const uint32_t here = __shfl_sync(0xffffffffu, own, r);
                    const uint32_t* list = cluster.map_shared_rank(s_list, r);
#pragma unroll 4
                    for (uint32_t i = (warp - r * warps) * 32 + lane; i < here; i += warps * 32)
                        s_list[gathered + before + i] = list[i];
                    __syncthreads();
                }
            }
            // ---- places: a warp takes consecutive slots; (above, equal) counts before it
            const int wper = ((hi - lo + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
            const int w0 = min(warp * wper, hi - lo), w1 = min(w0 + wper, hi - lo);
            uint32_t above = 0, equal = 0;
            for (int i0 = w0; i0 < w1; i0 += 32) {
                const int i = i0 + lane;
                const uint32_t key = i < w1 ? key_at(i) : 0u;
                above += __popc(__ballot_sync(0xffffffffu, i < w1 && key > chosen));
                equal += __popc(__ballot_sync(0xffffffffu, i < w1 && key == chosen));
            }
            if (lane == 0) s_warp[warp] = make_uint2(above, equal);
            __syncthreads();
            above = equal = 0;
            for (int k = 0; k < kEvictWarps; ++k) {
                if (k == warp) break;
                above += s_warp[k].x;
                equal += s_warp[k].y;
            }
            if (tid == kEvictThreads - 1)
                s_cta = make_uint2(above + s_warp[warp].x, equal + s_warp[warp].y);
            if (C > 1) cluster.sync();
            if (rank > 0) {
                uint2 t = make_uint2(0u, 0u);
                if (lane < rank) t = *cluster.map_shared_rank(&s_cta, lane);
                above += __reduce_add_sync(0xffffffffu, t.x);
                equal += __reduce_add_sync(0xffffffffu, t.y);
            }
            const uint32_t below = (1u << lane) - 1u;
            for (int i0 = w0; i0 < w1; i0 += 32) {
                const int i = i0 + lane;
                const uint32_t key = i < w1 ? key_at(i) : 0u;
                const uint32_t ma = __ballot_sync(0xffffffffu, i < w1 && key > chosen);
                const uint32_t me = __ballot_sync(0xffffffffu, i < w1 && key == chosen);
                const uint32_t eq = equal + __popc(me & below);
                if (i < w1 && (key > chosen || (key == chosen && eq < left)))
                    kept[a.sink + above + __popc(ma & below) + min(eq, left)] = a.sink + lo + i;
                above += __popc(ma);
                equal += __popc(me);
            }
        }
    }
    return true;
}

// The shared-memory ring of row copies in flight: stage, K or V, thread; then a weight per row.
struct EvictRing {
    uint4* data;
    float* w;
    int tid, rows, row, c;   // rows of a stage; this thread's row and chunk of it
    long long row_chunks;
    __device__ __forceinline__ EvictRing(uint32_t* smem, const EvictArgs& a, int t)
        : data(reinterpret_cast<uint4*>(smem)),
          w(reinterpret_cast<float*>(data + kEvictStages * 2 * kEvictThreads)),
          tid(t),
          rows(kEvictThreads >> a.chunk_bits),
          row(t >> a.chunk_bits),
          c(t & ((1 << a.chunk_bits) - 1)),
          row_chunks(static_cast<long long>(a.Hkv) << a.chunk_bits) {}
    // Starts the copy of slot t (on physical page `page`) of head h into the stage of `step`.
    __device__ __forceinline__ void fetch(const EvictArgs& a, int step, int page, int t, int h) {
        const int st = step % kEvictStages, off = t & (a.ps - 1);
        const long long at =
            ((static_cast<long long>(page) << a.page_bits) + off) * row_chunks + (h << a.chunk_bits) + c;
        cp_async16(data + (2 * st) * kEvictThreads + tid, a.k_pages + at);
        cp_async16(data + (2 * st + 1) * kEvictThreads + tid, a.v_pages + at);
        if (c == 0)
            cp_async4(w + st * rows + row,
                      a.weights + ((static_cast<long long>(page) * a.Hkv + h) << a.page_bits) + off);
    }
    // Writes the stage of `step` to slot j (on physical page `page`).
    __device__ __forceinline__ void store(const EvictArgs& a, int step, int page, int j, int h) {
        const int st = step % kEvictStages, off = j & (a.ps - 1);
        const long long at =
            ((static_cast<long long>(page) << a.page_bits) + off) * row_chunks + (h << a.chunk_bits) + c;
        a.k_pages[at] = data[(2 * st) * kEvictThreads + tid];
        a.v_pages[at] = data[(2 * st + 1) * kEvictThreads + tid];
        if (c == 0)
            a.weights[((static_cast<long long>(page) * a.Hkv + h) << a.page_bits) + off] =
                w[st * rows + row];
    }
};

// In place: selection, then the cluster moves its rows.  A step moves rows_step rows per CTA, a
// thread one 16-byte chunk of K and of V of its row (and the row's weight); the copies to shared
// memory run ahead of the stores.  A thread reads back only what it copied itself, so the ring
// needs no barrier of its own; the selection's shared memory is free by then.
__global__ void __launch_bounds__(kEvictThreads, 2) kv_evict_in_place_kernel(const EvictArgs a) {
    extern __shared__ __align__(16) uint32_t s_dyn[];   // selection: counts and keys; then the ring
    cg::cluster_group cluster = cg::this_cluster();
    const bool move = evict_select<true>(a, s_dyn, cluster);
    cluster.sync();   // kept[] is complete; nobody uses another CTA's shared memory any more
    if (!move) return;
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x;
    const long long stream = blockIdx.x / C;
    const int b = static_cast<int>(stream / a.Hkv), h = static_cast<int>(stream - static_cast<long long>(b) * a.Hkv);
    const int32_t* table = a.table + static_cast<long long>(b) * a.max_pages;
    const int32_t* kept = a.kept + stream * a.budget;
    const int n = a.budget;   // the selection returned true: the cache was longer

    EvictRing ring(s_dyn, a, tid);
    const int stride = C * ring.rows, r0 = rank * ring.rows + ring.row;
    const int steps = (n + stride - 1) / stride;   // the same in every CTA of the cluster
    // The index chain of a row, old slot then page, is fetched two steps before its copy: each
    // link has a step's time to arrive.
    auto old_slot = [&](int step) -> int {   // -1: no row, or one that stays where it is
        const int j = step * stride + r0;
        if (j >= n) return -1;
        const int t = __ldcg(kept + j);
        return t == j ? -1 : t;
    };
    auto page_of = [&](int t) -> int { return t < 0 ? 0 : table[t >> a.page_bits]; };
    uint32_t moved = 0;   // bit step % 32: this thread's row of the step has to be stored
    int t0 = old_slot(0), t1 = old_slot(1);
    int page0 = page_of(t0);
    auto advance = [&](int step) {   // copy `step`, move the chain on
        const int t2 = old_slot(step + 2), page1 = page_of(t1);
        const uint32_t bit = 1u << (step & 31);
        moved = t0 < 0 ? moved & ~bit : moved | bit;
        if (t0 >= 0) ring.fetch(a, step, page0, t0, h);
        cp_async_commit();
        t0 = t1;
        t1 = t2;
        page0 = page1;
    };
    // A cluster barrier stands between the reads of three steps and their writes.
    constexpr int kGroup = 3, kAhead = kEvictStages - kGroup;
    for (int step = 0; step < kAhead; ++step) advance(step);   // past the last: nothing
    for (int base = 0; base < steps; base += kGroup) {
        bool mine[kGroup];
        int dst_page[kGroup];
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            mine[u] = (moved >> ((base + u) & 31)) & 1u;   // false past the last step
            dst_page[u] = mine[u] ? table[((base + u) * stride + r0) >> a.page_bits] : 0;
        }
#pragma unroll
        for (int u = 0; u < kGroup; ++u) advance(base + kAhead + u);
        cp_async_wait<kAhead>();   // these steps' copies have landed
        cluster.sync();            // and those of every other row of them
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
            if (mine[u]) ring.store(a, base + u, dst_page[u], (base + u) * stride + r0, h);
    }
    cp_async_wait<0>();
}

// Into other pages: the selection alone, and a copy kernel whose CTAs share all heads' rows evenly.
__global__ void __launch_bounds__(kEvictThreads, 2) kv_evict_select_kernel(const EvictArgs a) {
    extern __shared__ __align__(16) uint32_t s_dyn[];
    cg::cluster_group cluster = cg::this_cluster();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    evict_select<false>(a, s_dyn, cluster);
    cluster.sync();   // nobody leaves while another CTA adds to or reads its shared memory
}

// A warp takes 32 consecutive kept rows of a head at a time.  Lane l finds where row l comes from
// and goes to (one batch ahead: kept slot, then pages) and moves its weight; then the warp copies the
// rows, as many a step as its lanes' 16-byte chunks cover, through a ring of its own in shared
// memory, kEvictStages - 1 steps ahead of the stores, each lane reading back only what it copied.
// The index work is once a row and not once a chunk: with each thread following its own row the
// kernel issued 66% of the cycles and moved 268 MB in 43 us.  Batch u goes to CTA u % grid.
__global__ void __launch_bounds__(kEvictThreads, 2) kv_evict_copy_kernel(const EvictArgs a, int most,
                                                                         int head_batches,
                                                                         int batches) {
    extern __shared__ __align__(16) uint32_t s_dyn[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint4* ring = reinterpret_cast<uint4*>(s_dyn) + warp * (kEvictStages * 64);
    const int c = lane & ((1 << a.chunk_bits) - 1), sub = lane >> a.chunk_bits;
    const int rows = 32 >> a.chunk_bits, steps = 1 << a.chunk_bits;   // rows a step, steps a batch
    const long long row_chunks = static_cast<long long>(a.Hkv) << a.chunk_bits;
    const int stride = static_cast<int>(gridDim.x) * kEvictWarps;
    struct Row {
        int b, h, j, t;   // sequence, head, new slot, old slot (-1: no row)
    };
    auto find = [&](int u) -> Row {
        Row x{0, 0, 0, -1};
        if (u >= batches) return x;
        const int stream = u / head_batches;
        x.b = stream / a.Hkv;
        x.h = stream - x.b * a.Hkv;
        x.j = (u - stream * head_batches) * 32 + lane;
        if (x.j < most) x.t = a.kept[static_cast<long long>(stream) * a.budget + x.j];
        return x;
    };
    struct Move {
        long long src, dst;   // in chunks; src -1: no row
    };
    auto place = [&](const Row& x) -> Move {
        Move m{-1, 0};
        if (x.t < 0) return m;
        const long long from = a.table[static_cast<long long>(x.b) * a.max_pages + (x.t >> a.page_bits)];
        const long long to = a.dst_table[static_cast<long long>(x.b) * a.dst_pages + (x.j >> a.page_bits)];
        const int t_off = x.t & (a.ps - 1), j_off = x.j & (a.ps - 1);
        m.src = ((from << a.page_bits) + t_off) * row_chunks + (x.h << a.chunk_bits);
        m.dst = ((to << a.page_bits) + j_off) * row_chunks + (x.h << a.chunk_bits);
        a.weights[((to * a.Hkv + x.h) << a.page_bits) + j_off] =
            a.weights[((from * a.Hkv + x.h) << a.page_bits) + t_off];
        return m;
    };
    int u = warp * static_cast<int>(gridDim.x) + blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Row row = find(u);
    Move now = place(row);
    row = find(u + stride);
    int filled = 0, drained = 0;   // ring positions
    // The copies run on into the next batch while this one's last stores are due: `now` is the
    // batch being fetched, `old` the one being stored.
    Move old = now;
    auto fetch = [&](int s) {
        const int r = s * rows + sub;
        const long long src = __shfl_sync(0xffffffffu, now.src, r);
        if (src >= 0) {
            uint4* slot = ring + (filled % kEvictStages) * 64 + lane;
            cp_async16(slot, a.k_pages + src + c);
            cp_async16(slot + 32, a.v_pages + src + c);
        }
        cp_async_commit();
        ++filled;
    };
    auto store = [&](int s) {
        const int r = s * rows + sub;
        const long long src = __shfl_sync(0xffffffffu, old.src, r);
        const long long dst = __shfl_sync(0xffffffffu, old.dst, r) + c;
        if (src >= 0) {
            const uint4* slot = ring + (drained % kEvictStages) * 64 + lane;
            a.k_pages[dst] = slot[0];
            a.v_pages[dst] = slot[32];
        }
        ++drained;
    };
    constexpr int kAhead = kEvictStages - 1;
    const int lead = min(kAhead, steps);   // steps of the next batch that a batch's stores overlap
    if (u >= batches) return;
    for (int s = 0; s < lead; ++s) fetch(s);
    for (; u < batches; u += stride) {
        old = now;
        const bool more = u + stride < batches;
        for (int s = 0; s < steps; ++s) {
            if (s + lead < steps) {
                fetch(s + lead);
            } else {
                if (s + lead == steps) {   // on to the next batch
                    now = place(row);
                    row = find(u + 2 * stride);
                }
                if (more) fetch(s + lead - steps);
                else cp_async_commit();   // an empty group keeps the count of those in flight
            }
            // `lead` groups are younger than this step's
            if (lead == kAhead) cp_async_wait<kAhead>();
            else cp_async_wait<4>();   // rows of four chunks: four steps a batch
            store(s);
        }
    }
    cp_async_wait<0>();
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// log2 of the 16-byte chunks of one row of D elements, or -1.
int row_chunk_bits(int D, int elem) {
    if ((D != 64 && D != 128 && D != 256) || (elem != 1 && elem != 2)) return -1;
    int bits = 0;
    while ((16 << bits) < D * elem) ++bits;
    return bits;
}

bool pool_supported(int num_phys, int ps) {
    return ps >= 16 && (ps & (ps - 1)) == 0 && static_cast<long long>(num_phys) * ps <= 0x7FFFFFFFLL;
}

struct Range {
    const void* p;
    size_t n;
};

// Whether any of the outputs overlaps an input or another output.
template <int NI, int NO>
bool any_overlap(const Range (&in)[NI], const Range (&out)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
    }
    return false;
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" int kv_paged_append_f16(const void* k_new, const void* v_new, void* k_pages, void* v_pages,
                                   const int32_t* page_table, const int32_t* kv_lens,
                                   const int32_t* new_lens, float* weights, int B, int Hkv, int n,
                                   int D, const int64_t* new_strides, int num_phys_pages,
                                   int page_size, int max_pages, void* stream) {
    CallRange nvtx_range("kv_paged_append_f16");
    if (!k_new || !v_new || !k_pages || !v_pages || !page_table || !kv_lens) return GBATTN_ERR_NULL;
    if (B <= 0 || Hkv <= 0 || n <= 0 || num_phys_pages <= 0 || page_size <= 0 || max_pages <= 0)
        return GBATTN_ERR_SHAPE;
    const int bits = row_chunk_bits(D, 2);
    if (bits < 0 || !pool_supported(num_phys_pages, page_size)) return GBATTN_ERR_UNSUPPORTED;
    if (B > 65535 || static_cast<long long>(Hkv) * n > (1LL << 40) / D ||
        static_cast<long long>(Hkv) > (1 << 24))
        return GBATTN_ERR_SHAPE;
    Strides st;
    if (!make_strides(new_strides, B, Hkv, n, D, false, &st)) return GBATTN_ERR_SHAPE;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages) ||
        misaligned4(page_table) || misaligned4(kv_lens) || misaligned4(new_lens) ||
        misaligned4(weights))
        return GBATTN_ERR_ALIGN;
    const size_t nb = strided_bytes(st, B, Hkv, n, D);
    const size_t slots = static_cast<size_t>(num_phys_pages) * page_size * Hkv;
    const Range in[] = {{k_new, nb},
                        {v_new, nb},
                        {page_table, static_cast<size_t>(B) * max_pages * 4},
                        {kv_lens, static_cast<size_t>(B) * 4},
                        {new_lens, static_cast<size_t>(B) * 4}};
    const Range out[] = {{k_pages, slots * D * 2}, {v_pages, slots * D * 2}, {weights, slots * 4}};
    if (any_overlap(in, out)) return GBATTN_ERR_ALIAS;
    DeviceState dev;
    const int rc = current_device(&dev);
    if (rc != GBATTN_OK) return rc;
    AppendArgs a{};
    a.k = static_cast<const uint4*>(k_new);
    a.v = static_cast<const uint4*>(v_new);
    a.k_pages = static_cast<uint4*>(k_pages);
    a.v_pages = static_cast<uint4*>(v_pages);
    a.table = page_table;
    a.kv_lens = kv_lens;
    a.new_lens = new_lens;
    a.weights = weights;
    a.status = dev.status;
    a.k_sb = st.b / 8;
    a.k_sh = st.h / 8;
    a.k_sr = st.r / 8;
    a.n = n;
    a.Hkv = Hkv;
    a.chunk_bits = bits;
    a.num_phys = num_phys_pages;
    a.ps = page_size;
    a.max_pages = max_pages;
    const long long per_block = kAppendThreads * kAppendUnroll;
    const long long blocks = ((static_cast<long long>(n) * Hkv << bits) + per_block - 1) / per_block;
    if (blocks > 0x7FFFFFFFLL) return GBATTN_ERR_SHAPE;
    kv_append_kernel<<<dim3(static_cast<unsigned>(blocks), B), kAppendThreads, 0,
                       static_cast<cudaStream_t>(stream)>>>(a);
    count_launches(1);
    return launch_status();
}

extern "C" int kv_paged_evict(void* k_pages, void* v_pages, float* weights,
                              const int32_t* page_table, const int32_t* dst_table,
                              const int32_t* kv_lens, int32_t* new_lens, int32_t* kept, int B,
                              int Hkv, int D, int elem_size, int num_phys_pages, int page_size,
                              int max_pages, int dst_pages, int max_kv_len, int budget, int sink,
                              int recent, void* stream) {
    CallRange nvtx_range("kv_paged_evict");
    if (!k_pages || !v_pages || !weights || !page_table || !dst_table || !kv_lens || !new_lens ||
        !kept)
        return GBATTN_ERR_NULL;
    if (B <= 0 || Hkv <= 0 || num_phys_pages <= 0 || page_size <= 0 || max_pages <= 0 ||
        dst_pages <= 0 || max_kv_len <= 0 || budget <= 0 || sink < 0 || recent < 0 ||
        static_cast<long long>(sink) + recent > budget || max_kv_len > (1 << 30) ||
        static_cast<long long>(max_kv_len) > static_cast<long long>(max_pages) * page_size)
        return GBATTN_ERR_SHAPE;
    const bool in_place = dst_table == page_table;
    if (in_place && dst_pages != max_pages) return GBATTN_ERR_SHAPE;
    const int most = budget < max_kv_len ? budget : max_kv_len;
    if (static_cast<long long>(most) > static_cast<long long>(dst_pages) * page_size)
        return GBATTN_ERR_SHAPE;
    const int bits = row_chunk_bits(D, elem_size);
    if (bits < 0 || !pool_supported(num_phys_pages, page_size)) return GBATTN_ERR_UNSUPPORTED;
    const long long streams = static_cast<long long>(B) * Hkv;
    if (streams > 0x7FFFFFFFLL / kEvictMaxCluster || Hkv > (1 << 24) ||
        streams * ((most + 31LL) / 32) > (1 << 30))
        return GBATTN_ERR_SHAPE;
    if (!aligned16(k_pages) || !aligned16(v_pages) || misaligned4(weights) ||
        misaligned4(page_table) || misaligned4(dst_table) || misaligned4(kv_lens) ||
        misaligned4(new_lens) || misaligned4(kept))
        return GBATTN_ERR_ALIGN;
    const size_t slots = static_cast<size_t>(num_phys_pages) * page_size * Hkv;
    const size_t rows = slots * D * elem_size;
    const Range in[] = {{page_table, static_cast<size_t>(B) * max_pages * 4},
                        {dst_table, static_cast<size_t>(B) * dst_pages * 4},
                        {kv_lens, static_cast<size_t>(B) * 4}};
    const Range out[] = {{k_pages, rows},
                         {v_pages, rows},
                         {weights, slots * 4},
                         {new_lens, static_cast<size_t>(B) * 4},
                         {kept, static_cast<size_t>(streams) * budget * 4}};
    if (any_overlap(in, out)) return GBATTN_ERR_ALIAS;
    DeviceState dev;
    const int rc = current_device(&dev);
    if (rc != GBATTN_OK) return rc;

    // Selection: a CTA for 2048 to 4096 slots, as long as all CTAs are resident at once (two per SM).
    // In place the cluster also moves its rows, so it is as large as that allows.
    int C = kEvictMaxCluster;
    while (C > 1 && (streams * C > 2LL * dev.num_sms || (!in_place && max_kv_len <= 2048LL * C))) C /= 2;
    EvictArgs a{};
    a.k_pages = static_cast<uint4*>(k_pages);
    a.v_pages = static_cast<uint4*>(v_pages);
    a.weights = weights;
    a.table = page_table;
    a.dst_table = dst_table;
    a.kv_lens = kv_lens;
    a.new_lens = new_lens;
    a.kept = kept;
    a.status = dev.status;
    a.Hkv = Hkv;
    a.chunk_bits = bits;
    a.num_phys = num_phys_pages;
    a.ps = page_size;
    a.max_pages = max_pages;
    a.dst_pages = dst_pages;
    a.max_kv = max_kv_len;
    a.budget = budget;
    a.sink = sink;
    a.recent = recent;
    while ((1 << a.page_bits) < page_size) ++a.page_bits;
    a.keys = kEvictMaxKeys;
    static std::once_flag once[64];
    static int attr_rc[64];
    if (dev.device < 0 || dev.device >= 64) return GBATTN_ERR_CUDA;
    std::call_once(once[dev.device], [&] {
        bool ok = cudaFuncSetAttribute(kv_evict_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kEvictRing) == cudaSuccess;
        for (auto* k : {kv_evict_in_place_kernel, kv_evict_select_kernel})
            ok = ok && cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            kEvictRing) == cudaSuccess;
        attr_rc[dev.device] = ok ? GBATTN_OK : GBATTN_ERR_CUDA;
    });
    if (attr_rc[dev.device] != GBATTN_OK) return attr_rc[dev.device];
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(streams * C));
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = kEvictRing;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, in_place ? kv_evict_in_place_kernel : kv_evict_select_kernel, a);
    count_launches(1);
    if (e == cudaSuccess && !in_place) {
        // Its CTAs may be placed as the selection's leave; they wait for all of it.
        const int head_batches = (most + 31) / 32;
        const long long batches = streams * head_batches;
        const int grid = static_cast<int>(batches < 2LL * dev.num_sms ? batches : 2LL * dev.num_sms);
        cudaLaunchConfig_t copy{};
        copy.gridDim = dim3(static_cast<unsigned>(grid));
        copy.blockDim = dim3(kEvictThreads);
        copy.dynamicSmemBytes = kEvictRing;
        copy.stream = cfg.stream;
        cudaLaunchAttribute dep[1];
        dep[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        dep[0].val.programmaticStreamSerializationAllowed = 1;
        copy.attrs = dep;
        copy.numAttrs = 1;
        e = cudaLaunchKernelEx(&copy, kv_evict_copy_kernel, a, most, head_batches,
                               static_cast<int>(batches));
        count_launches(1);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GBATTN_ERR_CUDA;
    }
    return launch_status();
}
