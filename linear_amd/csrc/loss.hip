// loss.hip -- the row passes of the linear head's cross entropy: the tiles' statistics joined
// into lse and loss, and the factor that dz is rounded under.
#include "loss.h"

namespace lin {

namespace {

// f(v of this thread, v of another) over a workgroup of NW waves, on every thread; lds: a float each.
template <int NW, typename F>
__device__ inline float group_fold(float v, float* lds, F f) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o, 64));
    __syncthreads();                                 // the last use of lds is over
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) v = f(v, lds[w]);
    return v;
}

// A workgroup per row.  The sum of the row's exp(z - top) is the tiles' sums, each brought
// to the common reference; the order is fixed.
__global__ void __launch_bounds__(256) loss_join(LossJoinArgs j) {
    __shared__ float lds[4];
    const int64_t m = blockIdx.x;
    const RowPart* p = j.parts + m * j.ldparts;
    float top = -3.402823466e38f;                    // no reference is lower
    for (int64_t i = threadIdx.x; i < j.count; i += 256) top = fmaxf(top, p[i].ref);
    top = group_fold<4>(top, lds, [](float a, float b) { return fmaxf(a, b); });
    float sum = 0.f;
    for (int64_t i = threadIdx.x; i < j.count; i += 256) sum += p[i].sum * __expf(p[i].ref - top);
    sum = group_fold<4>(sum, lds, [](float a, float b) { return a + b; });
    if (threadIdx.x != 0) return;
    const float lse = top + logf(sum);
    if (j.lse) j.lse[m] = lse;
    if (j.loss) {
        const int64_t t = j.target[m];
        j.loss[m] = t >= 0 && t < j.cols ? lse - j.at_target[m] : 0.f;
    }
}

__global__ void __launch_bounds__(1024) loss_scale(const int64_t* target, int64_t cols, const float* dloss,
                                                   const float* dlse, int64_t M, float* head) {
    __shared__ float lds[16];
    float base = 0.f, most = 0.f;
    for (int64_t m = threadIdx.x; m < M; m += 1024) {
        const int64_t t = target[m];
        const float d = t >= 0 && t < cols ? dloss[m] : 0.f;
        const float v = __builtin_fabsf(dlse ? d + dlse[m] : d) + __builtin_fabsf(d);
        if (!(v < __builtin_inff())) continue;
        base = fmaxf(base, __builtin_fabsf(d));
        most = fmaxf(most, v);
    }
    const auto largest = [](float a, float b) { return fmaxf(a, b); };
    base = group_fold<16>(base, lds, largest);
    most = group_fold<16>(most, lds, largest);
    if (threadIdx.x != 0) return;
    // (rows below 2^-80 are left smaller: the factor stays finite)
    base = fmaxf(base > 0.f ? base : most, 0x1p-80f);
    int x = 1;
    if (most > 0.f) __builtin_frexpf(most / base, &x);   // most / base < 2^x
    head[0] = __builtin_ldexpf(base, x - 15);
    head[1] = __builtin_ldexpf(1.f, 15 - x) / base;
}

}  // namespace

hipError_t launch_loss_join(const LossJoinArgs& j, int64_t M, hipStream_t stream) {
    LossJoinArgs args = j;
    void* params[] = {&args};
    return launch_kernel((const void*)loss_join, dim3((unsigned)M), dim3(256), params, 0, stream);
}

hipError_t launch_loss_scale(const int64_t* target, int64_t cols, const float* dloss, const float* dlse, int64_t M,
                             float* head, hipStream_t stream) {
    void* params[] = {&target, &cols, &dloss, &dlse, &M, &head};
    return launch_kernel((const void*)loss_scale, dim3(1), dim3(1024), params, 0, stream);
}

}  // namespace lin
