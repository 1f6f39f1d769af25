// gradnorm.hip -- the global norm of many gradient tensors, and clipping by it.
//
//     norm = sqrt(sum over tensors and elements of g^2)
//     out  = round(g * s),  s = min(1, max_norm / (norm + 1e-6))   (NaN norm: NaN)
//
// Both passes are bound by memory: the norm reads every gradient once, clipping
// reads and writes each once.  Up to kGradTensors tensors go into one launch, their
// table in the kernel's arguments (so a captured launch keeps it, and nothing is
// copied).  A tensor is cut into chunks of at most kGradChunk elements of one row
// (a contiguous tensor is one row); workgroup w takes chunks w, w + grid, ...
// Squares are taken and added in FP64: no finite binary32 gradient overflows or
// vanishes, and the order of additions is fixed, so reruns give the same bits.
#include "train.h"

namespace lin {

namespace {

// The tensor that holds chunk c (the table's last entry whose first chunk is <= c).
__device__ inline int find_tensor(const GradTable& t, int64_t c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

struct Chunk {
    int64_t row, col;
    int n;               // elements
};
__device__ inline Chunk locate(const GradTable& t, int i, int64_t c) {
    const int64_t per_row = (t.cols[i] + kGradChunk - 1) / kGradChunk;
    const int64_t j = c - t.first[i];
    Chunk k;
    k.row = j / per_row;
    k.col = (j - k.row * per_row) * kGradChunk;
    const int64_t left = t.cols[i] - k.col;
    k.n = (int)(left < kGradChunk ? left : kGradChunk);
    return k;
}

__device__ inline double square(float v) { return (double)v * (double)v; }

template <int E>
__device__ inline double squares16(const uint16_t* p, int n, bool vec) {
    double s = 0.0;
    int done = 0;
    if (vec) {
        done = n & ~7;
        for (int i = threadIdx.x * 8; i < done; i += 256 * 8) {
            const u32x4 v = *(const u32x4*)(p + i);
#pragma unroll
            for (int q = 0; q < 4; ++q) s += square(widen<E>((uint16_t)v[q])) + square(widen<E>((uint16_t)(v[q] >> 16)));
        }
    }
    for (int i = done + threadIdx.x; i < n; i += 256) s += square(widen<E>(p[i]));
    return s;
}

__device__ inline double squares32(const float* p, int n, bool vec) {
    double s = 0.0;
    int done = 0;
    if (vec) {
        done = n & ~3;
        for (int i = threadIdx.x * 4; i < done; i += 256 * 4) {
            const f32x4 v = *(const f32x4*)(p + i);
#pragma unroll
            for (int q = 0; q < 4; ++q) s += square(v[q]);
        }
    }
    for (int i = done + threadIdx.x; i < n; i += 256) s += square(p[i]);
    return s;
}

// The sum of v over the workgroup's NW waves, in one fixed order; thread 0 has it.
template <int NW>
__device__ inline double group_sum(double v, double* lds) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = lds[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += lds[w];
    return s;
}

__global__ void __launch_bounds__(256) grad_partials(GradTable t, double* partial) {
    __shared__ double lds[4];
    double s = 0.0;
    const int64_t chunks = t.first[t.count];
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = find_tensor(t, c);
        const Chunk k = locate(t, i, c);
        const int64_t at = k.row * t.ld[i] + k.col;
        if (t.type[i] == kGradF32) s += squares32((const float*)t.src[i] + at, k.n, t.vec[i]);
        else if (t.type[i] == kGradBF16) s += squares16<kBF16>((const uint16_t*)t.src[i] + at, k.n, t.vec[i]);
        else s += squares16<kF16>((const uint16_t*)t.src[i] + at, k.n, t.vec[i]);
    }
    s = group_sum<4>(s, lds);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ void __launch_bounds__(1024) grad_norm(const double* partial, int count, float* norm) {
    __shared__ double lds[16];
    double s = 0.0;
    for (int i = threadIdx.x; i < count; i += 1024) s += partial[i];
    s = group_sum<16>(s, lds);
    if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

template <int E>
__device__ inline void scale16(const uint16_t* p, uint16_t* q, int n, bool vec, float s) {
    int done = 0;
    if (vec) {
        done = n & ~7;
        for (int i = threadIdx.x * 8; i < done; i += 256 * 8) {
            const u32x4 v = *(const u32x4*)(p + i);
            u32x4 o;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[j] = (uint32_t)narrow<E>(widen<E>((uint16_t)v[j]) * s) |
                       ((uint32_t)narrow<E>(widen<E>((uint16_t)(v[j] >> 16)) * s) << 16);
            *(u32x4*)(q + i) = o;
        }
    }
    for (int i = done + threadIdx.x; i < n; i += 256) q[i] = narrow<E>(widen<E>(p[i]) * s);
}

__device__ inline void scale32(const float* p, float* q, int n, bool vec, float s) {
    int done = 0;
    if (vec) {
        done = n & ~3;
        for (int i = threadIdx.x * 4; i < done; i += 256 * 4) *(f32x4*)(q + i) = *(const f32x4*)(p + i) * s;
    }
    for (int i = done + threadIdx.x; i < n; i += 256) q[i] = p[i] * s;
}

__global__ void __launch_bounds__(256) grad_clip(GradTable t, const float* norm, float max_norm) {
    float s = max_norm / (*norm + 1e-6f);
    if (s >= 1.f) s = 1.f;                           // a NaN scale stays
    const int64_t chunks = t.first[t.count];
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = find_tensor(t, c);
        const Chunk k = locate(t, i, c);
        const int64_t from = k.row * t.ld[i] + k.col, to = k.row * t.ldd[i] + k.col;
        if (t.type[i] == kGradF32) scale32((const float*)t.src[i] + from, (float*)t.dst[i] + to, k.n, t.vec[i], s);
        else if (t.type[i] == kGradBF16)
            scale16<kBF16>((const uint16_t*)t.src[i] + from, (uint16_t*)t.dst[i] + to, k.n, t.vec[i], s);
        else scale16<kF16>((const uint16_t*)t.src[i] + from, (uint16_t*)t.dst[i] + to, k.n, t.vec[i], s);
    }
}

}  // namespace

hipError_t launch_grad_partials(const GradTable& t, double* partial, int grid, hipStream_t stream) {
    GradTable table = t;
    void* params[] = {&table, &partial};
    return launch_kernel((const void*)grad_partials, dim3((unsigned)grid), dim3(256), params, 0, stream);
}

hipError_t launch_grad_norm(const double* partial, int count, float* norm, hipStream_t stream) {
    void* params[] = {&partial, &count, &norm};
    return launch_kernel((const void*)grad_norm, dim3(1), dim3(1024), params, 0, stream);
}

hipError_t launch_grad_clip(const GradTable& t, const float* norm, float max_norm, int grid, hipStream_t stream) {
    GradTable table = t;
    void* params[] = {&table, &norm, &max_norm};
    return launch_kernel((const void*)grad_clip, dim3((unsigned)grid), dim3(256), params, 0, stream);
}

}  // namespace lin
