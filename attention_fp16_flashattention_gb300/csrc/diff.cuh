// What differential attention does to the two maps' outputs of one row:
//   o = o1 - lambda_h o2,  lambda_h = exp(lq1 . lk1) - exp(lq2 . lk2) + lambda_init,
// and, with a norm weight w, o = o / sqrt(mean(o^2) + eps) * w * (1 - lambda_init) over the head
// width.  The four vectors of a head are learned; they lie in one FP32 array [4][heads][d] in the
// order lq1, lk1, lq2, lk2 (heads = 1: shared by every head).
#pragma once

#include <cuda_fp16.h>

#include "ptx.cuh"

namespace gbattn {

struct DiffArgs {
    const float* vecs;   // [4][heads][d]
    const float* norm;   // [2 d] or null
    int heads;           // 1 or the query head count
    float init, eps;
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) x += __shfl_xor_sync(0xffffffffu, x, sh);
    return x;
}

// lambda of query head `head`, computed by a whole warp (kHalf = head width of one map), in two parts, so
// that the loads can be under way long before the sums are due.
template <int kHalf>
struct LambdaTerms {
    float q1[kHalf / 32], k1[kHalf / 32], q2[kHalf / 32], k2[kHalf / 32];
    __device__ __forceinline__ void load(const DiffArgs& f, int head, int lane) {
        const int h = f.heads == 1 ? 0 : head;
        const size_t plane = static_cast<size_t>(f.heads) * kHalf;
        const float* p = f.vecs + static_cast<size_t>(h) * kHalf;
#pragma unroll
        for (int i = 0; i < kHalf / 32; ++i) {
            q1[i] = p[lane + 32 * i];
            k1[i] = p[plane + lane + 32 * i];
            q2[i] = p[2 * plane + lane + 32 * i];
            k2[i] = p[3 * plane + lane + 32 * i];
        }
    }
    __device__ __forceinline__ float value(const DiffArgs& f) const {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < kHalf / 32; ++i) {
            a = fmaf(q1[i], k1[i], a);
            b = fmaf(q2[i], k2[i], b);
        }
        return expf(warp_sum(a)) - expf(warp_sum(b)) + f.init;
    }
};
template <int kHalf>
__device__ __forceinline__ float diff_lambda(const DiffArgs& f, int head, int lane) {
    LambdaTerms<kHalf> t;
    t.load(f, head, lane);
    return t.value(f);
}

}  // namespace gbattn
