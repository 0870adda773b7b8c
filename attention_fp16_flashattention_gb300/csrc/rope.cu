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
// four pairs, so that the two elements of a pair are in one lane and only the norm crosses lanes.  A row step
// (32 lanes) is about 85 instructions, two pairs in each (f32x2); with 190, as selects by row had it, the
// issue slots bound it and not the memory.  Measured (graph replays): 32,768 video tokens x 48 heads of 128 with
// norms (806 MB) 133 us, 6.05 TB/s, 0.89 of the measured copy; 20,000 prompt tokens into FP16 pages (487 MB) 86 us, 0.83;
// 8,192 into E4M3 pages (63 MB) 16 us; one token of 64 sequences 4.0 us.
#include <cuda_fp16.h>

#include <cstring>

#include "host.h"
#include "ptx.cuh"

namespace gbattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxAxes = 3;
// Blocks per SM (80 registers) and row steps under way in a warp: 3 and 4.  Video tokens, prompts, E4M3: 133, 86, 16.1
// us; 3 and 2 144, 94, 15.1; 4 and 2 139, 95, 17.9; 2 and 4 147, 94, 15.3.  One pair for all stores, though E4M3 would be a
// little quicker with two steps.  80 registers are not quite enough: 8 to 36 bytes are spilled for dense rows, 40 to 52 for
// FP16 pages, 52 to 68 for E4M3.
constexpr int kBlocks = 3, kAhead = 4;

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
    uint32_t tokens, S;              // B * S tokens
    int Hq, Hk, rot8;                // rot8: rot / 8, lanes with pairs
    int axis_end[kMaxAxes - 1];      // pairs before the end of each axis
    int axes, slots_total, page_bits;
    int q_steps, k_steps, steps;     // row steps of q, of k (and of v), of a token
    uint32_t steps_per, parts;       // of a warp; warps a token
    float eps, scale, k_scale, v_scale;
};

enum Store { kDense, kF16Pages, kE4m3Pages };

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    uint16_t lo, hi;   // saturating; the second operand goes to the low byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The eight elements of a lane as they lie in memory: two groups of four.
struct Raw {
    uint2 lo, hi;
};
__device__ __forceinline__ float2 unpack_half2(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// First and second elements of the lane's pairs, two pairs in each (f32x2).
struct Pairs {
    uint64_t a[2], b[2];
};
template <bool kInterleaved>
__device__ __forceinline__ Pairs to_pairs(const Raw& r) {
    const float2 x = unpack_half2(r.lo.x), y = unpack_half2(r.lo.y);
    const float2 z = unpack_half2(r.hi.x), w = unpack_half2(r.hi.y);
    if constexpr (kInterleaved)
        return Pairs{{f2_pack(x.x, y.x), f2_pack(z.x, w.x)}, {f2_pack(x.y, y.y), f2_pack(z.y, w.y)}};
    else
        return Pairs{{f2_pack(x.x, x.y), f2_pack(y.x, y.y)}, {f2_pack(z.x, z.y), f2_pack(w.x, w.y)}};
}
template <bool kInterleaved>
__device__ __forceinline__ void from_pairs(const Pairs& p, float (&lo)[4], float (&hi)[4]) {
    float a[4], b[4];
    f2_unpack(p.a[0], a[0], a[1]);
    f2_unpack(p.a[1], a[2], a[3]);
    f2_unpack(p.b[0], b[0], b[1]);
    f2_unpack(p.b[1], b[2], b[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (kInterleaved) {
            lo[e] = e % 2 == 0 ? a[e / 2] : b[e / 2];
            hi[e] = e % 2 == 0 ? a[2 + e / 2] : b[2 + e / 2];
        } else {
            lo[e] = a[e];
            hi[e] = b[e];
        }
    }
}

// A warp takes a range of a token's row steps -- q's, then k's, then v's; a step is 32 / (D / 8) rows -- and loads
// kAhead of them at a time.
template <int D, bool kInterleaved, Store kStore>
__global__ void __launch_bounds__(kThreads, kBlocks) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int kLanes = D / 8;          // lanes of a row
    constexpr int kSide = 32 / kLanes;     // rows of a step
    constexpr int kOwn = 4 / kSide;        // of a lane's four angles, those that it works out itself
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
    const uint32_t units = a.tokens * a.parts, stride = gridDim.x * kWarps;
    // What a unit's token needs to know first is loaded for 32 units of the warp at once, a lane each.
    int my_slot = 0, my_pos[kMaxAxes] = {0, 0, 0};
    uint32_t turn = 0;
    for (uint32_t u = blockIdx.x * kWarps + warp; u < units; u += stride, ++turn) {
        const uint32_t token = u / a.parts, part = u - token * a.parts;
        if ((turn & 31) == 0) {
            const unsigned long long ahead = u + static_cast<unsigned long long>(stride) * lane;
            if (ahead < units) {
                const uint32_t t = static_cast<uint32_t>(ahead) / a.parts;
                if (kStore != kDense) my_slot = a.slots[t];
#pragma unroll
                for (int i = 0; i < kMaxAxes; ++i)
                    if (a.positions && i < a.axes)
                        my_pos[i] = a.positions[static_cast<long long>(i) * a.tokens + t];
            }
        }
        const long long slot = __shfl_sync(0xffffffffu, my_slot, turn & 31);
        int pos[kMaxAxes];
#pragma unroll
        for (int i = 0; i < kMaxAxes; ++i) pos[i] = __shfl_sync(0xffffffffu, my_pos[i], turn & 31);
        if (slot < 0 || pos[0] < 0 || pos[1] < 0 || pos[2] < 0) continue;   // padding
        const bool cached = kStore == kDense || slot < a.slots_total;
        if (!cached && lane == 0 && part == 0) atomicOr(a.status, kDevBadPage);
        const uint32_t b = token / a.S, s = token - b * a.S;
        const int t_beg = static_cast<int>(part * a.steps_per);
        const int t_end = min(t_beg + static_cast<int>(a.steps_per), a.steps);
        // One tensor's rows from step t on, two pointers a lane.
        Raw raw[kAhead];
        const __half *p0 = nullptr, *p1 = nullptr;
        long long apart = 0;   // of a step's rows
        int h = 0;             // the row that is loaded next
        auto load = [&](Raw& r, bool in_range, int H) {
            if (in_range && h < H) {
                r.lo = *reinterpret_cast<const uint2*>(p0);
                r.hi = *reinterpret_cast<const uint2*>(p1);
            }
            p0 += apart;
            p1 += apart;
            h += kSide;
        };
        auto begin = [&](const View& v, int t0, int t1, int H) {
            h = t0 * kSide + side;
            const __half* row = v.p + b * v.b + s * v.s + h * v.h;
            p0 = row + c0;
            p1 = row + c1;
            apart = kSide * v.h;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                raw[i] = Raw{};
                load(raw[i], t0 + i < t1, H);
            }
        };
        const bool has_q = t_beg < a.q_steps;
        const int q_end = min(t_end, a.q_steps);
        if (has_q) begin(a.q, t_beg, q_end, a.Hq);
        float cs[4], sn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) sn[e] = 0.0f, cs[e] = 1.0f;
        if (a.rot8) {
            // The rows side by side in the warp share their angles: each side works out its part.
            float own_c[kOwn], own_s[kOwn];
#pragma unroll
            for (int e = 0; e < kOwn; ++e) {
                const int p = 4 * lr + side * kOwn + e;
                const int at = p < a.axis_end[0] ? pos[0] : p < a.axis_end[1] ? pos[1] : pos[2];
                const unsigned long long angle =
                    s_turn[turns ? p : 0] * static_cast<unsigned long long>(static_cast<uint32_t>(at));
                // half turns in [-1, 1)
                const float x = static_cast<float>(static_cast<int>(angle >> 32)) * 4.656612873077393e-10f;
                sincospif(x, &own_s[e], &own_c[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int from = lr + kLanes * (e / kOwn);
                const float c = __shfl_sync(0xffffffffu, own_c[e % kOwn], from);
                const float n = __shfl_sync(0xffffffffu, own_s[e % kOwn], from);
                if (turns) cs[e] = c * a.scale, sn[e] = n * a.scale;
            }
        }
        // Steps t0 .. t1 - 1 of the tensor that `begin` began, through `put(row, live, Pairs)`.
        auto rows = [&](int t0, int t1, int H, const float* weight, auto put) {
            // Coefficients of the two elements of each pair, the norm's weights in them:
            // (aa x_a - ab x_b, ba x_a + bb x_b)
            uint64_t aa[2], ab[2], ba[2], bb[2];
            float wa[4], wb[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                wa[e] = weight ? weight[kInterleaved ? c0 + 2 * e : c0 + e] : 1.0f;
                wb[e] = weight ? weight[kInterleaved ? c0 + 2 * e + 1 : c1 + e] : 1.0f;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                aa[i] = f2_pack(cs[2 * i] * wa[2 * i], cs[2 * i + 1] * wa[2 * i + 1]);
                ab[i] = f2_pack(-sn[2 * i] * wb[2 * i], -sn[2 * i + 1] * wb[2 * i + 1]);
                ba[i] = f2_pack(sn[2 * i] * wa[2 * i], sn[2 * i + 1] * wa[2 * i + 1]);
                bb[i] = f2_pack(cs[2 * i] * wb[2 * i], cs[2 * i + 1] * wb[2 * i + 1]);
            }
            for (int t = t0; t < t1; t += kAhead) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (t + i >= t1) break;
                    const Pairs x = to_pairs<kInterleaved>(raw[i]);
                    load(raw[i], t + i + kAhead < t1, H);
                    const int row = h - (kAhead + 1) * kSide;   // h is kAhead steps on and one more
                    Pairs y;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        y.a[j] = f2_mul(aa[j], x.a[j]);
                        y.b[j] = f2_mul(bb[j], x.b[j]);
                        if (turns) {
                            y.a[j] = f2_fma(ab[j], x.b[j], y.a[j]);
                            y.b[j] = f2_fma(ba[j], x.a[j], y.b[j]);
                        }
                    }
                    if (weight) {
                        uint64_t s2 = f2_mul(x.a[0], x.a[0]);
                        s2 = f2_fma(x.a[1], x.a[1], s2);
                        s2 = f2_fma(x.b[0], x.b[0], s2);
                        s2 = f2_fma(x.b[1], x.b[1], s2);
                        float s0, s1;
                        f2_unpack(s2, s0, s1);
                        float sq = s0 + s1;
#pragma unroll
                        for (int sh = 1; sh < kLanes; sh <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, sh);
                        const float rn = rsqrtf(sq * (1.0f / D) + a.eps);
                        const uint64_t rn2 = f2_pack(rn, rn);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            y.a[j] = f2_mul(y.a[j], rn2);
                            y.b[j] = f2_mul(y.b[j], rn2);
                        }
                    }
                    put(row, row < H, y);
                }
            }
        };
        // FP16 rows from `out` on, out_h apart
        auto to_half = [&](__half* out, long long out_h) {
            return [=](int h, bool live, const Pairs& y) {
                float lo[4], hi[4];
                from_pairs<kInterleaved>(y, lo, hi);
                if (!live) return;
                __half* row = out + h * out_h;
                *reinterpret_cast<uint2*>(row + c0) = make_uint2(pack_half2(lo[0], lo[1]), pack_half2(lo[2], lo[3]));
                *reinterpret_cast<uint2*>(row + c1) = make_uint2(pack_half2(hi[0], hi[1]), pack_half2(hi[2], hi[3]));
            };
        };
        // E4M3 codes of the values over `scale`
        auto to_codes = [&](void* pages, float scale) {
            uint8_t* out = static_cast<uint8_t*>(pages) + slot * a.Hk * D;
            return [=](int h, bool live, const Pairs& y) {
                float lo[4], hi[4];
                from_pairs<kInterleaved>(y, lo, hi);
                if (!live) return;
                uint8_t* row = out + h * D;
                *reinterpret_cast<uint32_t*>(row + c0) =
                    pack_e4m3(lo[0] / scale, lo[1] / scale, lo[2] / scale, lo[3] / scale);
                *reinterpret_cast<uint32_t*>(row + c1) =
                    pack_e4m3(hi[0] / scale, hi[1] / scale, hi[2] / scale, hi[3] / scale);
            };
        };
        if (has_q)
            rows(t_beg, q_end, a.Hq, a.q_weight,
                 to_half(a.q_out.p + b * a.q_out.b + s * a.q_out.s, a.q_out.h));
        if (!cached) continue;
        const int k_beg = max(t_beg - a.q_steps, 0), k_end = min(t_end - a.q_steps, a.k_steps);
        if (k_beg < k_end) {
            begin(a.k, k_beg, k_end, a.Hk);
            if constexpr (kStore == kDense)
                rows(k_beg, k_end, a.Hk, a.k_weight,
                     to_half(a.k_out.p + b * a.k_out.b + s * a.k_out.s, a.k_out.h));
            else if constexpr (kStore == kF16Pages)
                rows(k_beg, k_end, a.Hk, a.k_weight,
                     to_half(static_cast<__half*>(a.k_pages) + slot * a.Hk * D, D));
            else
                rows(k_beg, k_end, a.Hk, a.k_weight, to_codes(a.k_pages, a.k_scale));
            if (kStore != kDense && a.weights) {
                float* w = a.weights + (slot >> a.page_bits) * a.Hk * (1LL << a.page_bits) +
                           (slot & ((1LL << a.page_bits) - 1));
                for (int x = k_beg * kSide + lane; x < min(k_end * kSide, a.Hk); x += 32)
                    w[static_cast<long long>(x) << a.page_bits] = 0.0f;
            }
        }
        if constexpr (kStore != kDense) {   // v: as it is
            const int v_beg = max(t_beg - a.q_steps - a.k_steps, 0), v_end = t_end - a.q_steps - a.k_steps;
            if (v_beg < v_end) begin(a.v, v_beg, v_end, a.Hk);
            for (int t = v_beg; t < v_end; t += kAhead) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (t + i >= v_end) break;
                    const Raw r = raw[i];
                    load(raw[i], t + i + kAhead < v_end, a.Hk);
                    const int row_h = (t + i) * kSide + side;
                    if (row_h >= a.Hk) continue;
                    if constexpr (kStore == kF16Pages) {
                        __half* row = static_cast<__half*>(a.v_pages) + (slot * a.Hk + row_h) * D;
                        *reinterpret_cast<uint2*>(row + c0) = r.lo;
                        *reinterpret_cast<uint2*>(row + c1) = r.hi;
                    } else {
                        to_codes(a.v_pages, a.v_scale)(row_h, true, to_pairs<kInterleaved>(r));
                    }
                }
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
    if (c.rot > 0 && c.axes > 1 && !c.sections) return GBATTN_ERR_NULL;
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
    a.tokens = static_cast<uint32_t>(tokens);
    a.S = static_cast<uint32_t>(c.S);
    a.Hq = c.Hq;
    a.Hk = c.Hk;
    a.rot8 = c.rot / 8;
    int end = 0;
    for (int i = 0; i + 1 < kMaxAxes; ++i) {
        if (c.sections && i < c.axes) end += c.sections[i];
        a.axis_end[i] = i + 1 < c.axes ? end : 0x7FFFFFFF;
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
    const int side = 256 / c.D;
    a.q_steps = (c.Hq + side - 1) / side;
    a.k_steps = (c.Hk + side - 1) / side;
    a.steps = a.q_steps + (c.append ? 2 : 1) * a.k_steps;
    // A warp takes all rows of a token, or with few tokens a part of them, so that the GPU is filled.
    const long long warps = static_cast<long long>(kBlocks) * kWarps * dev.num_sms;
    long long parts = (warps + tokens - 1) / tokens;
    if (parts > a.steps) parts = a.steps;
    a.steps_per = static_cast<uint32_t>((a.steps + parts - 1) / parts);
    a.parts = (a.steps + a.steps_per - 1) / a.steps_per;
    const long long blocks = (tokens * a.parts + kWarps - 1) / kWarps;
    const long long resident = static_cast<long long>(kBlocks) * dev.num_sms;
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
