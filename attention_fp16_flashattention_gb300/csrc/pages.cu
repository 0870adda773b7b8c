// Page tables on the GPU: pages and slots for the new tokens of a batch of requests
// from a stack of free pages, and pages given back.  The pages name the paged cache
// and its table ("Integrate FP32 v37 prefill and exact E4M3 bridge", Implementation:
// paged cache, page table, live length); where the tables come from is this library's own.
//
// Mathematics.  Sequence b with n_b cached and m_b new tokens needs
// need_b = ceil((n_b + m_b) / ps) - ceil(n_b / ps) pages, and first_b = sum_{a < b} need_a of the
// stack's top go to the sequences before it, so page j of its new ones is
// free_pages[count - 1 - first_b - j].  Every CTA scans all sequences by itself (at most 4096, a few
// a thread) into shared memory, and then every page and every token is found by a binary
// search in the two prefixes: any number of CTAs work without waiting for each other.
// Only where the new lengths or the new count overwrite the old ones do all CTAs have to
// have read them first: then one cluster does the work, and its barrier comes in between.
//
// Bound by latency: the lengths, the stack's or the table's entries and the stores, one
// behind the other; 8 bytes a token and 8 a page are nothing beside that.  Measured (graph replays): one
// token for 64 sequences 4.0 us, 32 prompts of 131,000 tokens 4.7, drafted tokens of 64 sequences back 4.0,
// 100,000 pages back 7.3, 262,000 27 (a cluster of 16 CTAs looks at each of them; of eight 13.8 and 56, with 1024 threads
// a CTA 9.5 and 34, but then 4.9 for the few).
#include <cooperative_groups.h>

#include <mutex>

#include "host.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace gbattn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSeqs = 4096;
constexpr int kMaxCluster = 16;
constexpr int kUnroll = 4;   // tokens (or pages) a thread has under way at once

__device__ __forceinline__ int sat_add(int a, int b) {   // of counts >= 0
    const uint32_t s = static_cast<uint32_t>(a) + static_cast<uint32_t>(b);
    return s > 0x7FFFFFFFu ? 0x7FFFFFFF : static_cast<int>(s);
}
__device__ __forceinline__ int pages_of(int tokens, int page_bits) {   // tokens <= 2^30
    return (tokens + (1 << page_bits) - 1) >> page_bits;
}

// Sums of the threads before this one, and of all, of two counts (x saturates at 2^31 - 1).
struct Sums {
    int x, y, all_x, all_y;
};
__device__ __forceinline__ Sums block_scan(int x, int y) {
    __shared__ int s_x[kWarps], s_y[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int ix = x, iy = y;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, ix, sh), b = __shfl_up_sync(0xffffffffu, iy, sh);
        if (lane >= sh) {
            ix = sat_add(ix, a);
            iy += b;
        }
    }
    __syncthreads();   // s_x and s_y may still be read from the scan before
    if (lane == 31) {
        s_x[warp] = ix;
        s_y[warp] = iy;
    }
    // a saturated inclusive sum cannot be taken back by one's own part
    int ex = __shfl_up_sync(0xffffffffu, ix, 1), ey = __shfl_up_sync(0xffffffffu, iy, 1);
    if (lane == 0) ex = ey = 0;
    __syncthreads();
    Sums r{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) {
            r.x = r.all_x;
            r.y = r.all_y;
        }
        r.all_x = sat_add(r.all_x, s_x[w]);
        r.all_y += s_y[w];
    }
    r.x = sat_add(r.x, ex);
    r.y += ey;
    return r;
}

// The largest b with at[b] <= i (at[0] = 0 <= i).
__device__ __forceinline__ int find(const int* at, int B, int i) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (at[mid] <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
}

struct TableArgs {
    int32_t* table;              // [B][max_pages]
    const int32_t *kv_lens, *other;   // other: new_lens, or keep_lens or null (nothing is kept)
    int32_t* free_pages;         // [capacity]
    const int32_t* free_count;
    int32_t *lens_out, *count_out, *starts, *positions, *slots;
    uint32_t* status;
    int B, max_pages, page_bits, num_phys, capacity, row_tokens, max_tokens;
    int in_place;                // lens_out is kv_lens or count_out is free_count
};

__device__ __forceinline__ int valid_count(const TableArgs& a, bool report) {
    const int n = *a.free_count;
    if (n >= 0 && n <= a.capacity) return n;
    if (report) atomicOr(a.status, kDevBadLength);
    return 0;
}

constexpr int kRefused = 0x7FFFFFFF, kRejected = -1;

// What kv_extend_kernel does where there are more places than entries, out of its way (inlined, the code that calls
// hardly ever take cost 0.1 us of 4).
//
// Beside a sequence by whose length nobody can have packed, places that are together beyond the entries are nobody's
// either: then only the sound sequences have theirs.  The thread's own of those, or -1 where all stay.
__device__ __noinline__ int drop_rejected(const int32_t* new_lens, int* start, const int* old, int b0, int b1, int most) {
    bool wild = false;
    int tokens = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        if (old[b] == kRejected) wild = wild || new_lens[b] < 0 || new_lens[b] > most;
        else tokens = sat_add(tokens, start[b]);
    }
    if (!__syncthreads_or(wild)) return -1;
#pragma unroll 1
    for (int b = b0; b < b1; ++b)
        if (old[b] == kRejected) start[b] = 0;
    return tokens;
}
// A token without an entry is not a cached one, and its page stays on the stack (though the row has it, behind what
// the sequence holds, where nobody reads).
__device__ __noinline__ void cut_tokens(const int* start, const int* first, const int* old, int* after, int b0, int b1,
                                        int entries, int page_bits, int* gone) {
    int most = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const int n = old[b];
        if (n == kRejected || first[b] == kRefused) continue;
        const int have = max(min(after[b] - n, entries - start[b]), 0);
        after[b] = n + have;
        const int pages = pages_of(n + have, page_bits) - pages_of(n, page_bits);
        if (pages) most = first[b] + pages;   // (of one that needs none, first counts what others did not get)
    }
    if (most) atomicMax(gone, most);
}

__global__ void __launch_bounds__(kThreads) kv_extend_kernel(const TableArgs a) {
    extern __shared__ int s_dyn[];
    int* start = s_dyn;             // [B] places of the tokens of the sequences before b
    int* first = s_dyn + a.B;       // [B] pages that they take; kRefused: the stack has none for b
    int* old = s_dyn + 2 * a.B;     // [B] cached tokens; kRejected: the sequence's lengths were
    int* after = s_dyn + 3 * a.B;   // [B] and after the call
    __shared__ int s_taken, s_gone;
    const int tid = threadIdx.x;
    const bool lead = blockIdx.x == 0;
    const int cap = a.max_pages << a.page_bits;   // at most 2^30
    const int stack = valid_count(a, lead && tid == 0);
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    if (tid == 0) s_taken = s_gone = 0;
    // Tokens end to end lie where whoever packed them by new_lens put them, so the tokens of a rejected sequence keep
    // their places between the others' -- unless nobody can have packed by its length: a negative one, or one that neither
    // the entries nor a row could hold.  (In rows of their own nobody's places depend on the others.)
    const int entries = a.slots && !a.row_tokens ? a.max_tokens : 0x7FFFFFFF;
    const int most = max(entries, cap);
    int tokens = 0, pages = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = a.kv_lens[b], m = a.other[b];
        int places = m, need = 0, known = n;
        if (n < 0 || n > cap || m < 0 || m > cap - n || (a.row_tokens && m > a.row_tokens)) {
            if (lead) atomicOr(a.status, kDevBadLength);
            if (a.row_tokens || m < 0 || m > most) places = 0;
            known = kRejected;
        } else {
            need = pages_of(n + m, a.page_bits) - pages_of(n, a.page_bits);
            pages += need;
        }
        start[b] = places;   // this thread's own entries; turned into the prefixes below
        first[b] = need;
        old[b] = known;
        tokens = sat_add(tokens, places);
    }
    Sums at;
#pragma unroll 1
    for (bool again = false;; again = true) {
        at = block_scan(tokens, pages);
        if (at.all_x <= entries || again) break;
        tokens = drop_rejected(a.other, start, old, b0, b1, most);
        if (tokens < 0) break;
    }
    int taken = 0;
    for (int b = b0; b < b1; ++b) {
        const int places = start[b], need = first[b], n = old[b];
        const bool served = need == 0 || at.y + need <= stack;
        if (!served && lead) atomicOr(a.status, kDevNoPages);
        after[b] = n == kRejected ? a.kv_lens[b] : served ? n + places : n;
        start[b] = at.x;
        first[b] = served ? at.y : kRefused;
        at.x = sat_add(at.x, places);
        at.y += need;
        if (served && need) taken = at.y;
    }
    const bool cut = at.all_x > entries;
    if (cut) cut_tokens(start, first, old, after, b0, b1, entries, a.page_bits, &s_gone);
    taken = __reduce_max_sync(0xffffffffu, taken);
    if ((tid & 31) == 0 && taken) atomicMax(&s_taken, taken);   // (set to 0 two barriers ago)
    if (a.in_place) cg::this_cluster().sync();   // every CTA has read the old lengths and count
    else __syncthreads();
    taken = s_taken;
    if (lead) {
        for (int b = tid; b < a.B; b += kThreads) {
            a.lens_out[b] = after[b];
            if (a.starts) a.starts[b] = start[b];
        }
        if (tid == 0) {
            *a.count_out = stack - (cut ? s_gone : taken);
            if (a.starts) a.starts[a.B] = at.all_x;
            if (cut) atomicOr(a.status, kDevBadLength);
        }
    }
    const int step = kThreads * gridDim.x, self = blockIdx.x * kThreads + tid;
    for (int x = self; x < taken; x += step) {
        const int b = find(first, a.B, x);   // the refused ones lie behind all that are served
        const int page = a.free_pages[stack - 1 - x];
        if (page < 0 || page >= a.num_phys) atomicOr(a.status, kDevBadPage);
        a.table[static_cast<long long>(b) * a.max_pages + pages_of(old[b], a.page_bits) + x - first[b]] = page;
    }
    if (!a.slots) return;
    const int total = a.row_tokens ? a.max_tokens : min(at.all_x, a.max_tokens);
    for (long long i0 = self; i0 < a.max_tokens; i0 += static_cast<long long>(kUnroll) * step) {
        int pos[kUnroll], page[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long i = i0 + static_cast<long long>(u) * step;
            pos[u] = page[u] = -1;
            if (i >= total) continue;
            int b, off;
            if (a.row_tokens) {
                b = static_cast<int>(i) / a.row_tokens;
                off = static_cast<int>(i) - b * a.row_tokens;
                if (off >= after[b] - old[b]) continue;
            } else {
                b = find(start, a.B, static_cast<int>(i));
                off = static_cast<int>(i) - start[b];
            }
            const int n = old[b], t = n + off;
            if (n == kRejected || first[b] == kRefused) continue;
            const int fresh = (t >> a.page_bits) - pages_of(n, a.page_bits);
            // a token of the page that the old ones end in, or of a new one
            const int32_t* at_page = fresh < 0 ? a.table + static_cast<long long>(b) * a.max_pages + (t >> a.page_bits)
                                               : a.free_pages + (stack - 1 - first[b] - fresh);
            page[u] = *at_page;
            pos[u] = t;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long i = i0 + static_cast<long long>(u) * step;
            if (i >= a.max_tokens) continue;
            int slot = -1;
            if (pos[u] >= 0) {
                if (page[u] >= 0 && page[u] < a.num_phys)
                    slot = (page[u] << a.page_bits) + (pos[u] & ((1 << a.page_bits) - 1));
                else
                    atomicOr(a.status, kDevBadPage);
            }
            a.positions[i] = pos[u];
            a.slots[i] = slot;
        }
    }
}

// One cluster: it has to know that a sequence's entries are pages before any of them goes onto the
// stack, and each CTA looks at its share of them.  Entries stay in registers between the check and
// the store as far as kKeep goes.
__global__ void __launch_bounds__(kThreads) kv_release_kernel(const TableArgs a) {
    extern __shared__ int s_dyn[];
    int* first = s_dyn;                // [B] pages that the sequences before b give back
    int* from = s_dyn + a.B;           // [B] the row's first page that goes
    int* count = s_dyn + 2 * a.B;      // [B] how many go
    __shared__ int s_bad, s_given;
    constexpr int kKeep = 16;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x;
    const bool lead = blockIdx.x == 0;
    const int cap = a.max_pages << a.page_bits;
    const int stack = valid_count(a, lead && tid == 0);
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    if (tid == 0) s_bad = s_given = 0;
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = a.kv_lens[b], keep = a.other ? a.other[b] : 0;
        int p0 = 0, c = 0;
        if (n < 0 || n > cap || keep < 0 || keep > n) {
            if (lead) atomicOr(a.status, kDevBadLength);
        } else {
            p0 = pages_of(keep, a.page_bits);
            c = pages_of(n, a.page_bits) - p0;
        }
        from[b] = p0;
        count[b] = c;
        sum += c;
    }
    auto place = [&](int mine) -> int {   // prefix of the counts; returns their sum
        const Sums at = block_scan(0, mine);
        int run = at.y;
        for (int b = b0; b < b1; ++b) {
            first[b] = run;
            run += count[b];
        }
        __syncthreads();
        return at.all_y;
    };
    int total = place(sum);
    const int step = kThreads * gridDim.x, self = blockIdx.x * kThreads + tid;
    // Entries x0, x0 + step, ... below `end`, all under way at once.
    auto load = [&](int (&page)[kKeep], int x0, int end) {
#pragma unroll
        for (int u = 0; u < kKeep; ++u) {
            const int x = x0 + u * step;
            page[u] = 0;
            if (x >= end) continue;
            const int b = find(first, a.B, x);
            page[u] = a.table[static_cast<long long>(b) * a.max_pages + from[b] + x - first[b]];
        }
    };
    auto check = [&](const int (&page)[kKeep], int x0) {
        bool bad = false;
#pragma unroll
        for (int u = 0; u < kKeep; ++u) bad |= page[u] < 0 || page[u] >= a.num_phys;
        if (!bad) return;
        atomicOr(a.status, kDevBadPage);
#pragma unroll 1
        for (int u = 0; u < kKeep; ++u) {
            const int x = x0 + u * step;
            if (x >= total) break;
            const int b = find(first, a.B, x);
            const int page_x = a.table[static_cast<long long>(b) * a.max_pages + from[b] + x - first[b]];
            if (page_x >= 0 && page_x < a.num_phys) continue;
            for (unsigned r = 0; r < gridDim.x; ++r) {   // the sequence keeps all of its pages
                cluster.map_shared_rank(count, r)[b] = 0;
                *cluster.map_shared_rank(&s_bad, r) = 1;
            }
        }
    };
    int kept[kKeep];
    load(kept, self, total);
    cluster.sync();   // every CTA's tables are laid out before another marks a sequence in them
    check(kept, self);
    for (int x0 = self + kKeep * step; x0 < total; x0 += kKeep * step) {
        int page[kKeep];
        load(page, x0, total);
        check(page, x0);
    }
    cluster.sync();   // (and every CTA has read the old count)
    const bool again = s_bad != 0;
    if (again) {
        sum = 0;
        for (int b = b0; b < b1; ++b) sum += count[b];
        total = place(sum);
    }
    // In order, and all of a sequence's pages or none: those that the stack has room for.
    int given = 0;
    for (int b = b0; b < b1; ++b) {
        if (count[b] == 0) continue;
        if (first[b] + count[b] <= a.capacity - stack) given = first[b] + count[b];
        else if (lead) atomicOr(a.status, kDevNoPages);
    }
    given = __reduce_max_sync(0xffffffffu, given);
    if ((tid & 31) == 0 && given) atomicMax(&s_given, given);
    __syncthreads();
    given = s_given;
    if (lead && tid == 0) *a.count_out = stack + given;
    for (int x0 = self; x0 < given; x0 += kKeep * step) {
        if (again || x0 != self) load(kept, x0, given);
#pragma unroll
        for (int u = 0; u < kKeep; ++u) {
            const int x = x0 + u * step;
            if (x < given) a.free_pages[stack + x] = kept[u];
        }
    }
}

// What a device allows a kernel, asked for once: shared memory above the default, and clusters of 16 CTAs, which need
// a GPC with as many SMs, or of eight, which every one has.
struct Allowed {
    std::once_flag once;
    int rc, cluster;
};
int allow(void (*kernel)(TableArgs), int device, Allowed* all, int& cluster) {
    if (device < 0 || device >= 64) return GBATTN_ERR_CUDA;
    Allowed& d = all[device];
    std::call_once(d.once, [&] {
        constexpr int kSmem = 4 * kMaxSeqs * static_cast<int>(sizeof(int));
        d.cluster = 8;
        d.rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess
                   ? GBATTN_OK
                   : GBATTN_ERR_CUDA;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(kMaxCluster);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kMaxCluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0)
            d.cluster = kMaxCluster;
        cudaGetLastError();
    });
    cluster = d.cluster;
    return d.rc;
}

int launch(void (*kernel)(TableArgs), int ctas, int cluster, size_t smem, cudaStream_t s,
           const TableArgs& a) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    count_launches(1);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GBATTN_ERR_CUDA;
    }
    return launch_status();
}

int page_bits_of(int ps) {
    int bits = 0;
    while ((1 << bits) < ps) ++bits;
    return bits;
}

// Sizes that both calls take.
int check_sizes(int B, int max_pages, int page_size, int num_phys, int capacity) {
    if (B <= 0 || max_pages <= 0 || page_size <= 0 || num_phys <= 0 || capacity <= 0)
        return GBATTN_ERR_SHAPE;
    if (!pool_supported(num_phys, page_size) || B > kMaxSeqs) return GBATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(max_pages) * page_size > (1 << 30) ||
        static_cast<long long>(B) * max_pages > (1 << 30))
        return GBATTN_ERR_SHAPE;
    return GBATTN_OK;
}

// CTAs for n tokens or pages, `each` of them a CTA, up to `most` (a power of two for a cluster).
int ctas_for(long long n, int each, int most) {
    int c = 1;
    while (c < most && static_cast<long long>(c) * each < n) c *= 2;
    return c < most ? c : most;
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" int kv_paged_extend(int32_t* page_table, const int32_t* kv_lens, const int32_t* new_lens,
                               const int32_t* free_pages, const int32_t* free_count,
                               int32_t* kv_lens_out, int32_t* free_count_out, int32_t* token_starts,
                               int32_t* positions, int32_t* slots, int B, int max_pages,
                               int page_size, int num_phys_pages, int capacity, int row_tokens,
                               int max_tokens, void* stream) {
    CallRange nvtx_range("kv_paged_extend");
    if (!page_table || !kv_lens || !new_lens || !free_pages || !free_count || !kv_lens_out ||
        !free_count_out || !positions != !slots)
        return GBATTN_ERR_NULL;
    int rc = check_sizes(B, max_pages, page_size, num_phys_pages, capacity);
    if (rc != GBATTN_OK) return rc;
    if (row_tokens < 0 || max_tokens < 0 || (slots && max_tokens == 0) ||
        (row_tokens && static_cast<long long>(B) * row_tokens != max_tokens))
        return GBATTN_ERR_SHAPE;
    for (const void* p : {static_cast<const void*>(page_table), static_cast<const void*>(kv_lens),
                          static_cast<const void*>(new_lens), static_cast<const void*>(free_pages),
                          static_cast<const void*>(free_count), static_cast<const void*>(kv_lens_out),
                          static_cast<const void*>(free_count_out), static_cast<const void*>(token_starts),
                          static_cast<const void*>(positions), static_cast<const void*>(slots)})
        if (misaligned4(p)) return GBATTN_ERR_ALIGN;
    const size_t b4 = static_cast<size_t>(B) * 4, t4 = static_cast<size_t>(max_tokens) * 4;
    const bool same_lens = kv_lens_out == kv_lens, same_count = free_count_out == free_count;
    const Range in[] = {{same_lens ? nullptr : kv_lens, b4},
                        {new_lens, b4},
                        {free_pages, static_cast<size_t>(capacity) * 4},
                        {same_count ? nullptr : free_count, 4}};
    const Range out[] = {{page_table, static_cast<size_t>(B) * max_pages * 4},
                         {kv_lens_out, b4},
                         {free_count_out, 4},
                         {token_starts, b4 + 4},
                         {positions, t4},
                         {slots, t4}};
    if (any_overlap(in, out)) return GBATTN_ERR_ALIAS;
    DeviceState dev;
    rc = current_device(&dev);
    if (rc != GBATTN_OK) return rc;
    TableArgs a{};
    a.table = page_table;
    a.kv_lens = kv_lens;
    a.other = new_lens;
    a.free_pages = const_cast<int32_t*>(free_pages);   // only read
    a.free_count = free_count;
    a.lens_out = kv_lens_out;
    a.count_out = free_count_out;
    a.starts = token_starts;
    a.positions = positions;
    a.slots = slots;
    a.status = dev.status;
    a.B = B;
    a.max_pages = max_pages;
    a.page_bits = page_bits_of(page_size);
    a.num_phys = num_phys_pages;
    a.capacity = capacity;
    a.row_tokens = row_tokens;
    a.max_tokens = slots ? max_tokens : 0;
    a.in_place = same_lens || same_count;
    static Allowed allowed[64];
    int cluster = 0;
    rc = allow(kv_extend_kernel, dev.device, allowed, cluster);
    if (rc != GBATTN_OK) return rc;
    const int ctas = ctas_for(max_tokens > B ? max_tokens : B, kThreads * kUnroll,
                              a.in_place ? cluster : 128);
    return launch(kv_extend_kernel, ctas, a.in_place ? ctas : 1, 4 * b4,
                  static_cast<cudaStream_t>(stream), a);
}

extern "C" int kv_paged_release(const int32_t* page_table, const int32_t* kv_lens,
                                const int32_t* keep_lens, int32_t* free_pages,
                                const int32_t* free_count, int32_t* free_count_out, int B,
                                int max_pages, int page_size, int num_phys_pages, int capacity,
                                void* stream) {
    CallRange nvtx_range("kv_paged_release");
    if (!page_table || !kv_lens || !free_pages || !free_count || !free_count_out) return GBATTN_ERR_NULL;
    int rc = check_sizes(B, max_pages, page_size, num_phys_pages, capacity);
    if (rc != GBATTN_OK) return rc;
    for (const void* p : {static_cast<const void*>(page_table), static_cast<const void*>(kv_lens),
                          static_cast<const void*>(keep_lens), static_cast<const void*>(free_pages),
                          static_cast<const void*>(free_count), static_cast<const void*>(free_count_out)})
        if (misaligned4(p)) return GBATTN_ERR_ALIGN;
    const size_t b4 = static_cast<size_t>(B) * 4;
    const Range in[] = {{page_table, static_cast<size_t>(B) * max_pages * 4},
                        {kv_lens, b4},
                        {keep_lens, b4},
                        {free_count == free_count_out ? nullptr : free_count, 4}};
    const Range out[] = {{free_pages, static_cast<size_t>(capacity) * 4}, {free_count_out, 4}};
    if (any_overlap(in, out)) return GBATTN_ERR_ALIAS;
    DeviceState dev;
    rc = current_device(&dev);
    if (rc != GBATTN_OK) return rc;
    TableArgs a{};
    a.table = const_cast<int32_t*>(page_table);   // only read
    a.kv_lens = kv_lens;
    a.other = keep_lens;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.count_out = free_count_out;
    a.status = dev.status;
    a.B = B;
    a.max_pages = max_pages;
    a.page_bits = page_bits_of(page_size);
    a.num_phys = num_phys_pages;
    a.capacity = capacity;
    static Allowed allowed[64];
    int cluster = 0;
    rc = allow(kv_release_kernel, dev.device, allowed, cluster);
    if (rc != GBATTN_OK) return rc;
    // how many pages go is known on the device only; the table's size bounds it
    const int ctas = ctas_for(static_cast<long long>(B) * max_pages, kThreads * kUnroll, cluster);
    return launch(kv_release_kernel, ctas, ctas, 3 * b4, static_cast<cudaStream_t>(stream), a);
}
