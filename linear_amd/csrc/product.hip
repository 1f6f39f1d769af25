// product.hip -- the gated block's and the gradients' products for any layout,
// the elementwise half of the gated backward, and column sums.
//
// product_any computes one 64 x 64 output tile per workgroup of 4 waves with
// v_mfma_f32_32x32x16 (a 32 x 32 block each; columns as the A operand, rows as B,
// so a lane holds four consecutive columns of one row).  Both operands are read
// element by element at their own strides with 64-bit addresses (masked past the
// edges), along whichever of row and k is contiguous, and staged in LDS as
// [row][k]: it takes every alignment, stride and transposition.  It is the path
// for layouts that the streaming kernels refuse (odd row strides or bases).
#include "activation.h"
#include "columns.h"
#include "train.h"

namespace lin {

namespace {

constexpr int PB = kProdTile;        // output tile
constexpr int PK = 32;               // k per stage
constexpr int PITCH = PK + 8;        // LDS row, in words: 16-byte aligned rows

// A [PB, PK] operand tile at rows r0.., k0.. into registers: thread t of 256
// takes 8 elements.  Consecutive threads walk the contiguous direction.
__device__ inline void any_load(const uint16_t* p, int64_t sr, int64_t sk, int r0, int R, int k0, int L, int tid,
                                uint16_t (&v)[8]) {
    const bool along_k = sk == 1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = e * 256 + tid;
        const int r = r0 + (along_k ? i / PK : i % PB), k = k0 + (along_k ? i % PK : i / PB);
        v[e] = (r < R && k < L) ? p[(int64_t)r * sr + (int64_t)k * sk] : (uint16_t)0;
    }
}
__device__ inline void any_stage(uint16_t* lds, int64_t sk, int tid, const uint16_t (&v)[8]) {
    const bool along_k = sk == 1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = e * 256 + tid;
        lds[(along_k ? i / PK : i % PB) * PITCH + (along_k ? i % PK : i / PB)] = v[e];
    }
}

template <int E, int MODE>
__global__ void __launch_bounds__(256) product_any(ProductArgs p) {
    constexpr int NB = MODE == kProdGated ? 2 : 1;
    __shared__ __attribute__((aligned(16))) uint16_t sa[PB * PITCH];
    __shared__ __attribute__((aligned(16))) uint16_t sb[NB][PB * PITCH];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int tr = blockIdx.x / p.tiles_c, tc = blockIdx.x % p.tiles_c;
    const int r0 = tr * PB, c0 = tc * PB;
    const int wr = (wave >> 1) * 32, wc = (wave & 1) * 32;
    const int lr = lane & 31, lh = lane >> 5;
    f32x16 acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = (f32x16){};
    const int passes = MODE == kProdGated ? 1 : p.segs;
    for (int s = 0; s < passes; ++s) {
        for (int k0 = 0; k0 < p.L; k0 += PK) {
            uint16_t va[8], vb[NB][8];
            any_load(p.a[s], p.sar, p.sak, r0, p.R, k0, p.L, tid, va);
#pragma unroll
            for (int b = 0; b < NB; ++b) any_load(p.b[s + b], p.sbr[s + b], p.sbk[s + b], c0, p.C, k0, p.L, tid, vb[b]);
            __syncthreads();                       // the last stage has been read
            any_stage(sa, p.sak, tid, va);
#pragma unroll
            for (int b = 0; b < NB; ++b) any_stage(sb[b], p.sbk[s + b], tid, vb[b]);
            __syncthreads();
#pragma unroll
            for (int ks = 0; ks < PK / 16; ++ks) {
                const u32x4 fr = *(const u32x4*)(sa + (wr + lr) * PITCH + ks * 16 + lh * 8);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const u32x4 fc = *(const u32x4*)(sb[b] + (wc + lr) * PITCH + ks * 16 + lh * 8);
                    acc[b] = mfma32x32x16<E>(fc, fr, acc[b]);
                }
            }
        }
    }
    const int r = r0 + wr + lr;
    if (r >= p.R) return;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int c = c0 + wc + 8 * (v / 4) + 4 * lh + (v % 4);
        if (c >= p.C) continue;
        if constexpr (MODE == kProdF32) {
            float* y = (float*)p.y + (int64_t)r * p.ldy + c;
            *y = p.accumulate ? *y + acc[0][v] : acc[0][v];
        } else if constexpr (MODE == kProdRound) {
            ((uint16_t*)p.y)[(int64_t)r * p.ldy + c] = narrow<E>(acc[0][v]);
        } else {
            ((uint16_t*)p.y)[(int64_t)r * p.ldy + c] = narrow<E>(gated_act(p.act, acc[0][v]) * acc[NB - 1][v]);
            if (p.gate) p.gate[(int64_t)r * p.ldgate + c] = narrow<E>(acc[0][v]);
            if (p.up) p.up[(int64_t)r * p.ldup + c] = narrow<E>(acc[NB - 1][v]);
        }
    }
}

// One thread per four columns of a row; the splits are added in their order.
template <int E, bool F32>
__global__ void __launch_bounds__(256) split_sum(StreamProduct a) {
    const int chunks = (a.C + 3) / 4;
    const int64_t total = (int64_t)a.groups * a.R * chunks, plane = (int64_t)a.groups * a.R * a.ldp;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t gr = i / chunks;                   // group * R + row
        const int c = (int)(i - gr * chunks) * 4;
        const float* p = a.partial + gr * a.ldp + c;
        f32x4 v = *(const f32x4*)p;
        int s = 1;
        for (; s + 3 < a.splits; s += 4) {              // four loads in flight
            f32x4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = *(const f32x4*)(p + (s + j) * plane);
#pragma unroll
            for (int j = 0; j < 4; ++j) v += w[j];
        }
        f32x4 w[3];
#pragma unroll
        for (int j = 0; j < 3; ++j) w[j] = s + j < a.splits ? *(const f32x4*)(p + (s + j) * plane) : (f32x4){};
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (s + j < a.splits) v += w[j];
        const int g = gr >= a.R ? 1 : 0;
        const int64_t at = (gr - (int64_t)g * a.R) * a.ldy[g] + c;
        const bool vec = ((a.vec >> g) & 1) && c + 3 < a.C;
        if constexpr (F32) {
            float* y = (float*)a.y[g] + at;
            if (vec) {
                *(f32x4*)y = a.accumulate ? *(const f32x4*)y + v : v;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < a.C) y[e] = a.accumulate ? y[e] + v[e] : v[e];
            }
        } else {
            uint16_t* y = (uint16_t*)a.y[g] + at;
            uint2 u;
            u.x = (uint32_t)narrow<E>(v[0]) | ((uint32_t)narrow<E>(v[1]) << 16);
            u.y = (uint32_t)narrow<E>(v[2]) | ((uint32_t)narrow<E>(v[3]) << 16);
            if (vec) {
                *(uint2*)y = u;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < a.C) y[e] = narrow<E>(v[e]);
            }
        }
    }
}

template <int E>
__global__ void __launch_bounds__(256) gated_grad(GatedGradArgs g) {
    const int chunks = g.Np / 8;                     // 8-column pieces of a row of one half
    const int64_t total = (int64_t)g.M * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / chunks;
        const int c = (int)(i - m * chunks) * 8;
        const u32x4 h = load8(g.dh + m * g.lddh + c, true, c, g.N, g.vec);
        const u32x4 a = load8(g.gate + m * g.ldgate + c, true, c, g.N, g.vec);
        const u32x4 u = load8(g.up + m * g.ldup + c, true, c, g.N, g.vec);
        u32x4 dg = (u32x4){0u, 0u, 0u, 0u}, du = (u32x4){0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (c + e >= g.N) continue;
            const int q = e >> 1, sh = 16 * (e & 1);
            const float hv = widen<E>((uint16_t)(h[q] >> sh)), uv = widen<E>((uint16_t)(u[q] >> sh));
            float av, dv;
            gated_act_grad(g.act, widen<E>((uint16_t)(a[q] >> sh)), av, dv);
            dg[q] |= (uint32_t)narrow<E>(hv * uv * dv) << sh;
            du[q] |= (uint32_t)narrow<E>(hv * av) << sh;
        }
        uint16_t* row = g.d + m * 2 * g.Np + c;
        *(u32x4*)row = dg;
        *(u32x4*)(row + g.Np) = du;
    }
}

template <int E>
__global__ void __launch_bounds__(1024) column_partials(ColumnSumArgs c) {
    __shared__ float lds[column_lds(1024)];
    column_block<E, 1024>(c, blockIdx.x, blockIdx.y, lds);
}

// The splits' sums, in their order.
template <int E>
__global__ void __launch_bounds__(64) column_finish(ColumnSumArgs c) {
    const int n = blockIdx.x * 64 + threadIdx.x;
    if (n >= c.N) return;
    float sum = c.partial[n];
#pragma unroll 8
    for (int s = 1; s < c.splits; ++s) sum += c.partial[(int64_t)s * c.N + n];
    store_sum<E>(c, n, sum);
}

template <int E>
const void* any_fn(int mode) {
    if (mode == kProdF32) return (const void*)product_any<E, kProdF32>;
    if (mode == kProdGated) return (const void*)product_any<E, kProdGated>;
    return (const void*)product_any<E, kProdRound>;
}

}  // namespace

hipError_t launch_product_any(int elem, int mode, const ProductArgs& p, hipStream_t stream) {
    ProductArgs args = p;
    void* params[] = {&args};
    return hipLaunchKernel(elem == kBF16 ? any_fn<kBF16>(mode) : any_fn<kF16>(mode),
                           dim3((unsigned)(p.tiles_r * p.tiles_c)), dim3(256), params, 0, stream);
}

hipError_t launch_split_sum(int elem, bool f32, const StreamProduct& a, hipStream_t stream) {
    StreamProduct args = a;
    void* params[] = {&args};
    const int64_t blocks = ((int64_t)a.groups * a.R * ((a.C + 3) / 4) + 255) / 256;
    const void* fn = f32 ? (const void*)split_sum<kF16, true>
                         : elem == kBF16 ? (const void*)split_sum<kBF16, false> : (const void*)split_sum<kF16, false>;
    return hipLaunchKernel(fn, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), params, 0, stream);
}

hipError_t launch_gated_grad(int elem, const GatedGradArgs& g, hipStream_t stream) {
    GatedGradArgs args = g;
    void* params[] = {&args};
    const int64_t blocks = ((int64_t)g.M * (g.Np / 8) + 255) / 256;
    return hipLaunchKernel(elem == kBF16 ? (const void*)gated_grad<kBF16> : (const void*)gated_grad<kF16>,
                           dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), params, 0, stream);
}

hipError_t launch_column_sum(int elem, const ColumnSumArgs& c, hipStream_t stream) {
    ColumnSumArgs args = c;
    void* params[] = {&args};
    const unsigned gx = (unsigned)((c.N + 63) / 64);
    hipError_t e = hipLaunchKernel(elem == kBF16 ? (const void*)column_partials<kBF16> : (const void*)column_partials<kF16>,
                                   dim3(gx, (unsigned)c.splits), dim3(1024), params, 0, stream);
    if (e != hipSuccess || c.splits == 1) return e;
    return hipLaunchKernel(elem == kBF16 ? (const void*)column_finish<kBF16> : (const void*)column_finish<kF16>,
                           dim3(gx), dim3(64), params, 0, stream);
}

}  // namespace lin
