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
#include "decode_f16.cuh"

namespace gbattn {
namespace {

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

size_t decode_workspace_size(int B, int Hq, int Hkv, int nq, int max_kv, int D, int maps,
                             bool weights) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || nq <= 0 || max_kv <= 0 || D <= 0 || Hq % Hkv != 0) return 0;
    const long long G = static_cast<long long>(Hq / Hkv) * nq * maps;
    if (G > 0x7FFFFFFFLL) return 0;
    return decode_layout(sm_count_or_default(), B, Hkv, static_cast<int>(G), max_kv, D, weights).total;
}

template <int D, int NB>
const int* resident_clusters(int device) {
    return resident_clusters<D, NB, decode_f16_kernel<D, NB, true>>(device);
}
const int* resident_clusters(int D, int R, int device) {
    if (D == 64) return R == 8 ? resident_clusters<64, 1>(device) : resident_clusters<64, 2>(device);
    if (D == 128) return R == 8 ? resident_clusters<128, 1>(device) : resident_clusters<128, 2>(device);
    return R == 8 ? resident_clusters<256, 1>(device) : resident_clusters<256, 2>(device);
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
    rc = c.diff       ? launch_dependent(decode_f16_merge_kernel<128, true, false>, mgrid, 32 * mw, msmem, s, m)
         : c.D == 64  ? launch_dependent(decode_f16_merge_kernel<64, false, false>, mgrid, 32 * mw, msmem, s, m)
         : c.D == 128 ? launch_dependent(decode_f16_merge_kernel<128, false, false>, mgrid, 32 * mw, msmem, s, m)
                      : launch_dependent(decode_f16_merge_kernel<256, false, false>, mgrid, 32 * mw, msmem, s, m);
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
