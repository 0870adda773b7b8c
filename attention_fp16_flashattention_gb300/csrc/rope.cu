// Norms of queries and keys for each head and the rotation by their positions in one pass,
// for prompts and on the way into a paged cache ("Integrate FP32 v37 prefill and exact E4M3 bridge",
// Implementation: paged E4M3 cache; the FP16 cache is the same with FP16 elements).
//
// Mathematics.  A head's row x of D elements becomes y = x / sqrt(mean(x^2) + eps) * w (or stays as
// it is without w), and pair p of its first `rot` elements, (y_p, y_{p + rot/2}) or (y_2p, y_2p+1), is
// turned by the angle pos * freq_p and scaled:  (c y_a - s y_b, s y_a + c y_b).  All in FP32, rounded
// once to FP16, or to E4M3 after a division by the cache's scale.
//
// The angle of a far position has to be known to a small part of a turn, and an FP32 product
// of 10^6 has lost three digits of it.  So a frequency becomes the part of a turn per position
// as a 64-bit fraction of 2^64 (once per CTA, in FP64, 2^-53 of itself); its integer product with the
// position wraps at whole turns by itself, and its upper 32 bits are the angle, exact to 2^-32 turns and
// pos 2^-53 of the frequency.  A token's angles are worked out once for all of its heads.
//
// Bound by HBM: 2 bytes in and 2 (1) out per element.  D / 8 lanes take a row, each eight elements of it:
// four pairs, so that the two elements of a pair are in one lane and only the norm crosses lanes.
#include <cuda_fp16.h>

#include <cstring>

#include "host.h"
#include "ptx.cuh"

namespace gbattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxAxes = 3;

struct View {   // [B][H][S][D] rows
    __half* p;
    long long b, h, s;
};

struct RopeArgs {
    View q, k, v, q_out, k_out;      // v, or k_out, with p null: not there
    void *k_pages, *v_pages;
    float* weights;                  // [num_phys][Hkv][ps] or null
    const int32_t *positions;        // [axes][B][S]
    const int32_t* slots;            // [B][S]
    const float *freqs, *q_weight, *k_weight;
    uint32_t* status;
    long long tokens;                // B * S
    int B, S, Hq, Hk, rot8;          // rot8: rot / 8, lanes with pairs
    int axis_end[kMaxAxes];          // pairs before the end of each axis
    int axes, slots_total, page_bits;
    int rows, rows_per, parts;       // rows of a token, of a warp, warps a token
    float eps, scale, k_scale, v_scale;
};

enum Store { kDense, kF16Pages, kE4m3Pages };

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    uint16_t lo, hi;   // saturating; the second operand goes to the low byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Four elements of a cached row at p (element offset `at`).
template <Store kStore>
__device__ __forceinline__ void store_cached(void* p, long long at, const float (&x)[4], float scale) {
    if constexpr (kStore == kE4m3Pages)
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p) + at) =
            pack_e4m3(x[0] / scale, x[1] / scale, x[2] / scale, x[3] / scale);
    else
        *reinterpret_cast<uint2*>(static_cast<__half*>(p) + at) =
            make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
}

__device__ __forceinline__ void load4(const __half* p, float (&x)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}

// A warp takes rows_per rows (of q, then k, then v) of one token, 32 / (D / 8) of them at a time.
template <int D, bool kInterleaved, Store kStore>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int kLanes = D / 8;          // lanes of a row
    constexpr int kSide = 32 / kLanes;     // rows of a warp at a time
    __shared__ unsigned long long s_turn[D / 2];   // parts of a turn per position, in 2^-64
    for (int p = threadIdx.x; p < 4 * a.rot8; p += kThreads) {
        double t = static_cast<double>(a.freqs[p]) * 0.15915494309189535;   // 1 / (2 pi)
        t -= floor(t);
        s_turn[p] = static_cast<unsigned long long>(t * 18446744073709551616.0);
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lr = lane & (kLanes - 1), side = lane / kLanes;
    // The lane's eight elements: two groups of four, at c0 and c1.
    const bool turns = lr < a.rot8;
    const int c0 = kInterleaved ? 8 * lr : turns ? 4 * lr : 8 * lr;
    const int c1 = kInterleaved || !turns ? c0 + 4 : c0 + 4 * a.rot8;
    float wq[8], wk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = e < 4 ? c0 + e : c1 + e - 4;
        wq[e] = a.q_weight ? a.q_weight[c] : 1.0f;
        wk[e] = a.k_weight ? a.k_weight[c] : 1.0f;
    }
    int axis[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int p = 4 * lr + e;
        axis[e] = (p >= a.axis_end[0]) + (p >= a.axis_end[1]);
    }
    const long long units = a.tokens * a.parts;
    for (long long u = static_cast<long long>(blockIdx.x) * kWarps + warp; u < units;
         u += static_cast<long long>(gridDim.x) * kWarps) {
        const long long token = u / a.parts;
        const int part = static_cast<int>(u - token * a.parts);
        const int b = static_cast<int>(token / a.S), s = static_cast<int>(token - static_cast<long long>(b) * a.S);
        long long slot = 0;
        bool cached = true;
        if constexpr (kStore != kDense) {
            slot = a.slots[token];
            if (slot < 0) continue;   // padding
            if (slot >= a.slots_total) {
                cached = false;
                if (lane == 0 && part == 0) atomicOr(a.status, kDevBadPage);
            }
        }
        float cs[4], sn[4];
        if (a.positions) {
            const bool skip = lane < a.axes && a.positions[lane * a.tokens + token] < 0;
            if (__any_sync(0xffffffffu, skip)) continue;   // padding
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int pos = a.positions[(turns ? axis[e] : 0) * a.tokens + token];
                const unsigned long long angle =
                    turns ? s_turn[turns ? 4 * lr + e : 0] * static_cast<unsigned long long>(static_cast<uint32_t>(pos)) : 0;
                // half turns in [-1, 1)
                const float x = static_cast<float>(static_cast<int>(angle >> 32)) * 4.656612873077393e-10f;
                sincospif(x, &sn[e], &cs[e]);
                sn[e] *= a.scale;
                cs[e] *= a.scale;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) sn[e] = 0.0f, cs[e] = 1.0f;
        }
        const int r_end = min((part + 1) * a.rows_per, a.rows);
#pragma unroll 2
        for (int r0 = part * a.rows_per; r0 < r_end; r0 += kSide) {
            const int r = r0 + side;
            const bool live = r < r_end;
            const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hk;
            const int h = is_q ? r : is_v ? r - a.Hq - a.Hk : r - a.Hq;
            const View& in = is_q ? a.q : is_v ? a.v : a.k;
            float x[8];
            float lo[4] = {0.0f, 0.0f, 0.0f, 0.0f}, hi[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (live) {
                const __half* row = in.p + b * in.b + h * in.h + s * in.s;
                load4(row + c0, lo);
                load4(row + c1, hi);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = lo[e], x[4 + e] = hi[e];
            float sq = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sq += x[e] * x[e];
#pragma unroll
            for (int sh = 1; sh < kLanes; sh <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, sh);
            if (!live) continue;
            if (!is_v) {
                const bool norm = is_q ? a.q_weight != nullptr : a.k_weight != nullptr;
                const float rn = norm ? rsqrtf(sq * (1.0f / D) + a.eps) : 1.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= rn * (is_q ? wq[e] : wk[e]);
                if (turns) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float& m = kInterleaved ? x[2 * e] : x[e];
                        float& n = kInterleaved ? x[2 * e + 1] : x[4 + e];
                        const float y = cs[e] * m - sn[e] * n;
                        n = sn[e] * m + cs[e] * n;
                        m = y;
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) lo[e] = x[e], hi[e] = x[4 + e];
            if (is_q || kStore == kDense) {
                const View& out = is_q ? a.q_out : a.k_out;
                __half* row = out.p + b * out.b + h * out.h + s * out.s;
                *reinterpret_cast<uint2*>(row + c0) = make_uint2(pack_half2(lo[0], lo[1]), pack_half2(lo[2], lo[3]));
                *reinterpret_cast<uint2*>(row + c1) = make_uint2(pack_half2(hi[0], hi[1]), pack_half2(hi[2], hi[3]));
            } else if (cached) {
                const long long at = (slot * a.Hk + h) * D;
                void* pages = is_v ? a.v_pages : a.k_pages;
                store_cached<kStore>(pages, at + c0, lo, is_v ? a.v_scale : a.k_scale);
                store_cached<kStore>(pages, at + c1, hi, is_v ? a.v_scale : a.k_scale);
                if (!is_v && lr == 0 && a.weights)
                    a.weights[((slot >> a.page_bits) * a.Hk + h) * (1LL << a.page_bits) +
                              (slot & ((1LL << a.page_bits) - 1))] = 0.0f;
            }
        }
    }
}

template <Store kStore>
int launch_rope(const RopeArgs& a, int D, bool interleaved, int grid, cudaStream_t s) {
    auto go = [&](auto* kernel) {
        kernel<<<grid, kThreads, 0, s>>>(a);
        count_launches(1);
        return launch_status();
    };
    if (interleaved)
        return D == 64    ? go(qk_norm_rope_kernel<64, true, kStore>)
               : D == 128 ? go(qk_norm_rope_kernel<128, true, kStore>)
                          : go(qk_norm_rope_kernel<256, true, kStore>);
    return D == 64    ? go(qk_norm_rope_kernel<64, false, kStore>)
           : D == 128 ? go(qk_norm_rope_kernel<128, false, kStore>)
                      : go(qk_norm_rope_kernel<256, false, kStore>);
}

// Two views that share no element although their spans may meet: slices of one packed tensor, whose
// heads lie in different parts of every row.
bool packed_apart(const void* pa, const Strides& a, int Ha, const void* pb, const Strides& b, int Hb,
                  int B, int S, int D) {
    const long long sa = (Ha - 1) * a.h + D, sb = (Hb - 1) * b.h + D;   // what a row's heads span
    long long ra = a.r, rb = b.r;
    if (S == 1) ra = a.b, rb = b.b;   // one row per batch entry
    if (ra != rb || sa > ra || sb > ra) return false;
    if (B > 1 && (a.b != b.b || a.b % ra != 0 || a.b < static_cast<long long>(S) * ra)) return false;
    const long long bytes = static_cast<long long>(reinterpret_cast<uintptr_t>(pb)) -
                            static_cast<long long>(reinterpret_cast<uintptr_t>(pa));
    if (bytes % 2 != 0) return false;
    long long d = bytes / 2 % ra;
    if (d < 0) d += ra;
    // b's heads begin d behind a's in a row: between a's end and the next row's
    return d >= sa && d + sb <= ra;
}

struct RopeCall {
    const void *q, *k, *v;
    const int32_t *positions, *slots;
    const float *freqs, *q_weight, *k_weight;
    const int32_t* sections;
    void *q_out, *k_out, *k_pages, *v_pages;
    float* weights;
    int B, Hq, Hk, S, D, rot, axes, interleaved, elem, num_phys, ps;
    const int64_t *q_strides, *kv_strides, *qo_strides, *ko_strides;
    float eps, rope_scale, k_scale, v_scale;
    void* stream;
    bool append;
};

int run_rope(const RopeCall& c) {
    if (!c.q || !c.q_out) return GBATTN_ERR_NULL;
    if (c.append) {
        if (!c.k || !c.v || !c.slots || !c.k_pages || !c.v_pages) return GBATTN_ERR_NULL;
    } else if (!c.k != !c.k_out || (!c.k && c.Hk != 0)) {
        return GBATTN_ERR_NULL;
    }
    if (c.rot > 0 && (!c.positions || !c.freqs)) return GBATTN_ERR_NULL;
    if (c.B <= 0 || c.Hq <= 0 || c.S <= 0 || c.Hk < (c.k ? 1 : 0) || c.rot < 0 || c.axes < 1 ||
        c.axes > kMaxAxes || (c.interleaved != 0 && c.interleaved != 1))
        return GBATTN_ERR_SHAPE;
    if (c.append && (c.num_phys <= 0 || c.ps <= 0)) return GBATTN_ERR_SHAPE;
    if (c.D != 64 && c.D != 128 && c.D != 256) return GBATTN_ERR_UNSUPPORTED;
    if (c.rot % 8 != 0) return GBATTN_ERR_UNSUPPORTED;
    if (c.append && ((c.elem != 1 && c.elem != 2) || !pool_supported(c.num_phys, c.ps)))
        return GBATTN_ERR_UNSUPPORTED;
    if (c.rot > c.D || c.Hq > (1 << 24) || c.Hk > (1 << 24) ||
        static_cast<long long>(c.B) * c.S > 0x7FFFFFFFLL)
        return GBATTN_ERR_SHAPE;
    if (c.axes > 1 && !c.sections) return GBATTN_ERR_NULL;
    long long pairs = 0;
    if (c.sections && c.rot > 0) {
        for (int i = 0; i < c.axes; ++i) {
            if (c.sections[i] < 0) return GBATTN_ERR_SHAPE;
            pairs += c.sections[i];
        }
        if (2 * pairs != c.rot) return GBATTN_ERR_SHAPE;
    }
    if (((c.q_weight || c.k_weight) && !finite_positive(c.eps)) ||
        (c.rot > 0 && !finite_positive(c.rope_scale)) ||
        (c.append && c.elem == 1 && (!finite_positive(c.k_scale) || !finite_positive(c.v_scale))))
        return GBATTN_ERR_SCALE;
    const int Hk1 = c.Hk > 0 ? c.Hk : 1;
    Strides qs, ks, qo, ko;
    if (!make_strides(c.q_strides, c.B, c.Hq, c.S, c.D, false, &qs) ||
        !make_strides(c.kv_strides, c.B, Hk1, c.S, c.D, false, &ks) ||
        !make_strides(c.qo_strides, c.B, c.Hq, c.S, c.D, true, &qo) ||
        !make_strides(c.ko_strides, c.B, Hk1, c.S, c.D, true, &ko))
        return GBATTN_ERR_SHAPE;
    if (!aligned16(c.q) || !aligned16(c.k) || !aligned16(c.v) || !aligned16(c.q_out) ||
        !aligned16(c.k_out) || !aligned16(c.k_pages) || !aligned16(c.v_pages) ||
        misaligned4(c.positions) || misaligned4(c.slots) || misaligned4(c.freqs) ||
        misaligned4(c.q_weight) || misaligned4(c.k_weight) || misaligned4(c.weights))
        return GBATTN_ERR_ALIGN;

    const long long tokens = static_cast<long long>(c.B) * c.S;
    const size_t t4 = static_cast<size_t>(tokens) * 4;
    const size_t kb = strided_bytes(ks, c.B, Hk1, c.S, c.D), d4 = static_cast<size_t>(c.D) * 4;
    const size_t slots = c.append ? static_cast<size_t>(c.num_phys) * c.ps * c.Hk : 0;
    const Range qi{c.q, strided_bytes(qs, c.B, c.Hq, c.S, c.D)}, ki{c.k, kb}, vi{c.v, kb};
    const Range qr{c.q_out, strided_bytes(qo, c.B, c.Hq, c.S, c.D)};
    const Range kr{c.k_out, strided_bytes(ko, c.B, Hk1, c.S, c.D)};
    const Range kp{c.k_pages, slots * c.D * c.elem}, vp{c.v_pages, slots * c.D * c.elem};
    const Range w{c.weights, slots * 4};
    // Rows in place: the very elements of the input, each read by the warp that writes it.
    auto same = [](const void* a, const Strides& x, const void* b, const Strides& y) {
        return a == b && x.b == y.b && x.h == y.h && x.r == y.r;
    };
    auto hits = [](const Range& a, const Range& b) { return overlaps(a.p, a.n, b.p, b.n); };
    auto meet = [&](const Range& ra, const Strides& a, int Ha, const Range& rb, const Strides& b, int Hb) {
        return hits(ra, rb) && !packed_apart(ra.p, a, Ha, rb.p, b, Hb, c.B, c.S, c.D);
    };
    if (!same(c.q_out, qo, c.q, qs) && hits(qr, qi)) return GBATTN_ERR_ALIAS;
    if (!same(c.k_out, ko, c.k, ks) && hits(kr, ki)) return GBATTN_ERR_ALIAS;
    if (meet(qr, qo, c.Hq, ki, ks, Hk1) || meet(qr, qo, c.Hq, vi, ks, Hk1) ||
        meet(kr, ko, Hk1, qi, qs, c.Hq) || meet(qr, qo, c.Hq, kr, ko, Hk1))
        return GBATTN_ERR_ALIAS;
    const Range in[] = {{c.positions, t4 * c.axes}, {c.slots, t4}, {c.freqs, static_cast<size_t>(c.rot) * 2},
                        {c.q_weight, d4}, {c.k_weight, d4}};
    const Range rows[] = {qi, ki, vi, qr, kr};
    const Range pool[] = {kp, vp, w};
    if (any_overlap(in, pool) || any_overlap(rows, pool)) return GBATTN_ERR_ALIAS;
    for (const Range& x : in)
        if (hits(x, qr) || hits(x, kr)) return GBATTN_ERR_ALIAS;

    DeviceState dev;
    const int rc = current_device(&dev);
    if (rc != GBATTN_OK) return rc;
    auto view = [](const void* p, const Strides& s) {
        return View{static_cast<__half*>(const_cast<void*>(p)), s.b, s.h, s.r};
    };
    RopeArgs a{};
    a.q = view(c.q, qs);
    a.k = view(c.k, ks);
    a.v = view(c.v, ks);
    a.q_out = view(c.q_out, qo);
    a.k_out = view(c.k_out, ko);
    a.k_pages = c.k_pages;
    a.v_pages = c.v_pages;
    a.weights = c.weights;
    a.positions = c.positions;
    a.slots = c.slots;
    a.freqs = c.freqs;
    a.q_weight = c.q_weight;
    a.k_weight = c.k_weight;
    a.status = dev.status;
    a.tokens = tokens;
    a.B = c.B;
    a.S = c.S;
    a.Hq = c.Hq;
    a.Hk = c.Hk;
    a.rot8 = c.rot / 8;
    int end = 0;
    for (int i = 0; i < kMaxAxes; ++i) {
        if (c.sections && i < c.axes) end += c.sections[i];
        a.axis_end[i] = c.axes > 1 && i + 1 < c.axes ? end : 0x7FFFFFFF;
    }
    a.axes = c.axes;
    if (c.append) {
        a.slots_total = c.num_phys * c.ps;
        while ((1 << a.page_bits) < c.ps) ++a.page_bits;
    }
    a.eps = c.eps;
    a.scale = c.rope_scale;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    // A warp takes all rows of a token, or with few tokens a part of them, so that the GPU is filled.
    const int side = 256 / c.D;
    a.rows = c.Hq + (c.append ? 2 : 1) * c.Hk;
    const long long warps = 32LL * dev.num_sms;
    long long parts = (warps + tokens - 1) / tokens;
    const long long most = (a.rows + side - 1) / side;
    if (parts > most) parts = most;
    a.rows_per = static_cast<int>((most + parts - 1) / parts) * side;
    a.parts = (a.rows + a.rows_per - 1) / a.rows_per;
    const long long blocks = (tokens * a.parts + kWarps - 1) / kWarps;
    const long long resident = 8LL * dev.num_sms;
    const int grid = static_cast<int>(blocks < resident ? blocks : resident);
    cudaStream_t s = static_cast<cudaStream_t>(c.stream);
    const bool il = c.interleaved != 0;
    if (!c.append) return launch_rope<kDense>(a, c.D, il, grid, s);
    return c.elem == 2 ? launch_rope<kF16Pages>(a, c.D, il, grid, s)
                       : launch_rope<kE4m3Pages>(a, c.D, il, grid, s);
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" int qk_norm_rope_f16(const void* q, const void* k, const int32_t* positions,
                                const float* freqs, const float* q_weight, const float* k_weight,
                                void* q_out, void* k_out, int B, int Hq, int Hk, int S, int D, int rot,
                                int interleaved, int axes, const int32_t* sections,
                                const int64_t* q_strides, const int64_t* k_strides,
                                const int64_t* q_out_strides, const int64_t* k_out_strides, float eps,
                                float rope_scale, void* stream) {
    CallRange nvtx_range("qk_norm_rope_f16");
    RopeCall c{};
    c.q = q;
    c.k = k;
    c.positions = positions;
    c.freqs = freqs;
    c.q_weight = q_weight;
    c.k_weight = k_weight;
    c.sections = sections;
    c.q_out = q_out;
    c.k_out = k_out;
    c.B = B;
    c.Hq = Hq;
    c.Hk = Hk;
    c.S = S;
    c.D = D;
    c.rot = rot;
    c.axes = axes;
    c.interleaved = interleaved;
    c.q_strides = q_strides;
    c.kv_strides = k_strides;
    c.qo_strides = q_out_strides;
    c.ko_strides = k_out_strides;
    c.eps = eps;
    c.rope_scale = rope_scale;
    c.stream = stream;
    return run_rope(c);
}

extern "C" int kv_paged_rope_append(const void* q, const void* k_new, const void* v_new,
                                    const int32_t* slots, const int32_t* positions, const float* freqs,
                                    const float* q_weight, const float* k_weight, void* q_out,
                                    void* k_pages, void* v_pages, float* weights, int B, int Hq,
                                    int Hkv, int S, int D, int rot, int interleaved, int axes,
                                    const int32_t* sections, const int64_t* q_strides,
                                    const int64_t* kv_strides, const int64_t* q_out_strides,
                                    int elem_size, int num_phys_pages, int page_size, float eps,
                                    float rope_scale, float k_scale, float v_scale, void* stream) {
    CallRange nvtx_range("kv_paged_rope_append");
    RopeCall c{};
    c.append = true;
    c.q = q;
    c.k = k_new;
    c.v = v_new;
    c.slots = slots;
    c.positions = positions;
    c.freqs = freqs;
    c.q_weight = q_weight;
    c.k_weight = k_weight;
    c.sections = sections;
    c.q_out = q_out;
    c.k_pages = k_pages;
    c.v_pages = v_pages;
    c.weights = weights;
    c.B = B;
    c.Hq = Hq;
    c.Hk = Hkv;
    c.S = S;
    c.D = D;
    c.rot = rot;
    c.axes = axes;
    c.interleaved = interleaved;
    c.q_strides = q_strides;
    c.kv_strides = kv_strides;
    c.qo_strides = q_out_strides;
    c.elem = elem_size;
    c.num_phys = num_phys_pages;
    c.ps = page_size;
    c.eps = eps;
    c.rope_scale = rope_scale;
    c.k_scale = k_scale;
    c.v_scale = v_scale;
    c.stream = stream;
    return run_rope(c);
}
