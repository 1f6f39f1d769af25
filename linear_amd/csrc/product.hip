// product.hip -- the gated block's and the gradients' products for any layout,
// the elementwise half of the gated backward, and column sums.
//
// product_any computes one T x T output tile per workgroup of 4 waves with
// v_mfma_f32_32x32x16 (a quarter of the tile each; columns as the A operand, rows as
// B, so a lane holds four consecutive columns of one row).  It is the path for layouts
// that the streaming kernels refuse (odd row strides or bases): it takes every
// alignment and stride, with 64-bit addresses.  A thread reads 8 words along an
// operand's contiguous direction as one 16-byte load of 2-byte alignment (word by word
// at the edges), the next stage's while this one is multiplied.  A k-contiguous
// operand is staged as [row][k], a k-major one as [k][row] and read with the
// transposing read, as in the streaming kernels.
#include <algorithm>

#include "abi.h"
#include "columns.h"
#include "grad_impl.h"
#include "train.h"

namespace lin {

namespace {

constexpr int PK = 32;               // k per stage
constexpr int PITCH = PK + 8;        // words of a [row][k] LDS row: 16-byte aligned rows

// The 8-word pieces of a stage of T rows by PK that thread tid of 256 takes.
template <int T>
struct Pieces {
    u32x4 v[T * PK / 2048];
};

// ALONG_K: k contiguous (row stride ld), 4 pieces a row; else k-major (ld between
// k's), T / 8 pieces of 8 rows per k.
template <int T, bool ALONG_K>
__device__ inline Pieces<T> any_load(const uint16_t* p, int64_t ld, int r0, int R, int64_t k0, int L, int tid) {
    Pieces<T> out;
#pragma unroll
    for (int i = 0; i < T * PK / 2048; ++i) {
        const int c = i * 256 + tid;
        const int r = r0 + (ALONG_K ? c / (PK / 8) : c % (T / 8) * 8);
        const int64_t k = k0 + (ALONG_K ? c % (PK / 8) * 8 : c / (T / 8));
        const bool row = ALONG_K ? r < R : k < L;              // the line that holds the piece
        const int64_t at = ALONG_K ? k : r, end = ALONG_K ? L : R;
        const uint16_t* q = p + (ALONG_K ? (int64_t)r : k) * ld + at;
        if (row && at + 8 <= end) {
            __builtin_memcpy(&out.v[i], q, 16);
        } else {
            out.v[i] = (u32x4){0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (row && at + e < end) out.v[i][e >> 1] |= (uint32_t)q[e] << (16 * (e & 1));
        }
    }
    return out;
}

// LDS bytes of a stage.
template <int T, bool ALONG_K>
constexpr int any_bytes = ALONG_K ? T * PITCH * 2 : PK * T * 2;

template <int T, bool ALONG_K>
__device__ inline void any_stage(unsigned char* lds, int tid, const Pieces<T>& in) {
#pragma unroll
    for (int i = 0; i < T * PK / 2048; ++i) {
        const int c = i * 256 + tid;
        if constexpr (ALONG_K) {
            *(u32x4*)(lds + c / (PK / 8) * PITCH * 2 + c % (PK / 8) * 16) = in.v[i];
        } else {
            const int k = c / (T / 8), c8 = c % (T / 8);
            *(u32x4*)(lds + k * T * 2 + ((c8 ^ (2 * panel_swz<T>(k))) << 4)) = in.v[i];
        }
    }
}

// The 32-row fragment of rows base .. base + 31 at K step ks: 8 k's from 16 ks + 8 (lane / 32).
template <int T, bool ALONG_K>
__device__ inline u32x4 any_frag(const unsigned char* lds, int base, int ks, int lane) {
    if constexpr (ALONG_K) {
        return *(const u32x4*)(lds + (base + (lane & 31)) * PITCH * 2 + ks * 32 + (lane >> 5) * 16);
    } else {
        // 16 lanes q address rows 16 ks + 8 (q / 2) + s / 4 (+ 4) and the piece at 16 (q % 2) + 4 (s % 4)
        const int q = lane >> 4, s = lane & 15, k = 16 * ks + 8 * (q >> 1) + (s >> 2);
        const int r = base + 16 * (q & 1);
        lds_byte* p = lds_at(lds_address(lds) + k * T * 2 + (((r >> 4) ^ panel_swz<T>(k)) << 5) + 8 * (s & 3));
        const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * T * 2);
        return (u32x4){lo.x, lo.y, hi.x, hi.y};
    }
}

template <int T, int E, int MODE, bool AK, bool BK>
__global__ void __launch_bounds__(256) product_any(ProductArgs p) {
    constexpr int NB = MODE == kProdGated ? 2 : 1;
    constexpr int F = T / 64;                         // 32 x 32 blocks per wave and direction
    __shared__ __attribute__((aligned(16))) unsigned char sa[any_bytes<T, AK>];
    __shared__ __attribute__((aligned(16))) unsigned char sb[NB][any_bytes<T, BK>];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int tr = blockIdx.x / p.tiles_c, tc = blockIdx.x % p.tiles_c;
    const int r0 = tr * T, c0 = tc * T;
    const int wr = (wave >> 1) * (T / 2), wc = (wave & 1) * (T / 2);
    f32x16 acc[NB][F][F];                             // [operand][column block][row block]
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j) acc[b][i][j] = (f32x16){};
    const int passes = MODE == kProdGated ? 1 : p.segs;
    for (int s = 0; s < passes; ++s) {
        Pieces<T> va, vb[NB];
        auto load = [&](int64_t k0) {
            va = any_load<T, AK>(p.a[s], p.lda, r0, p.R, k0, p.L, tid);
#pragma unroll
            for (int b = 0; b < NB; ++b) vb[b] = any_load<T, BK>(p.b[s + b], p.ldb[s + b], c0, p.C, k0, p.L, tid);
            if constexpr (MODE == kProdRound) {
                if (p.finite_from && s >= p.finite_from) {
#pragma unroll
                    for (int i = 0; i < T * PK / 2048; ++i) vb[0].v[i] = finite_words<E>(vb[0].v[i]);
                }
            }
        };
        if (p.L > 0) load(0);
        for (int64_t k0 = 0; k0 < p.L; k0 += PK) {
            __syncthreads();                       // the last stage has been read
            any_stage<T, AK>(sa, tid, va);
#pragma unroll
            for (int b = 0; b < NB; ++b) any_stage<T, BK>(sb[b], tid, vb[b]);
            __syncthreads();
            if (k0 + PK < p.L) load(k0 + PK);
#pragma unroll
            for (int ks = 0; ks < PK / 16; ++ks) {
                u32x4 fr[F];
#pragma unroll
                for (int j = 0; j < F; ++j) fr[j] = any_frag<T, AK>(sa, wr + 32 * j, ks, lane);
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < F; ++i) {
                        const u32x4 fc = any_frag<T, BK>(sb[b], wc + 32 * i, ks, lane);
#pragma unroll
                        for (int j = 0; j < F; ++j) acc[b][i][j] = mfma32x32x16<E>(fc, fr[j], acc[b][i][j]);
                    }
            }
        }
    }
    const int lr = lane & 31, lh = lane >> 5;
    const float back = MODE == kProdRound && p.unscale ? *p.unscale : 1.f;
#pragma unroll
    for (int j = 0; j < F; ++j) {
        const int r = r0 + wr + 32 * j + lr;
        if (r >= p.R) continue;
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int c = c0 + wc + 32 * i + 8 * (v / 4) + 4 * lh + (v % 4);
                if (c >= p.C) continue;
                const float sum = acc[0][i][j][v];
                if constexpr (MODE == kProdF32) {
                    float* y = (float*)p.y + (int64_t)r * p.ldy + c;
                    *y = p.accumulate ? *y + sum : sum;
                } else if constexpr (MODE == kProdRound) {
                    ((uint16_t*)p.y)[(int64_t)r * p.ldy + c] = narrow<E>(sum * back);
                } else {
                    const float up = acc[NB - 1][i][j][v];
                    ((uint16_t*)p.y)[(int64_t)r * p.ldy + c] = narrow<E>(gated_act(p.act, sum) * up);
                    if (p.gate) p.gate[(int64_t)r * p.ldgate + c] = narrow<E>(sum);
                    if (p.up) p.up[(int64_t)r * p.ldup + c] = narrow<E>(up);
                }
            }
    }
}

// The gated block's few-row form for any layout: a wave takes one row of both weights
// and up to 4 rows of x (grid y: row groups), 8 words per lane and step; 4 steps'
// loads in flight.  (1 x 4001 x 4095 bf16; a 64 x 64 tile per workgroup leaves most
// CUs without work there.)
constexpr int ROWS = kAnyRows;

__device__ inline u32x4 any_piece(const uint16_t* p, int k, int K) {
    u32x4 v = (u32x4){0u, 0u, 0u, 0u};
    if (k + 8 <= K) __builtin_memcpy(&v, p + k, 16);
    else
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < K) v[e >> 1] |= (uint32_t)p[k + e] << (16 * (e & 1));
    return v;
}

template <int E>
__global__ void __launch_bounds__(256) gated_rows_any(ProductArgs p) {
    constexpr int U = 4;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = (int64_t)blockIdx.x * 4 + wave, m0 = (int64_t)blockIdx.y * ROWS;
    if (n >= p.C) return;
    const uint16_t *g = p.b[0] + n * p.ldb[0], *u = p.b[1] + n * p.ldb[1];
    const int rows = (int)min((int64_t)ROWS, p.R - m0);
    float gs[ROWS] = {}, us[ROWS] = {};
    for (int64_t k0 = 0; k0 < p.L; k0 += U * 512) {
        u32x4 gv[U], uv[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t k = min(k0 + j * 512 + lane * 8, (int64_t)p.L);
            gv[j] = any_piece(g, (int)k, p.L);
            uv[j] = any_piece(u, (int)k, p.L);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t k = min(k0 + j * 512 + lane * 8, (int64_t)p.L);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                if (r >= rows) break;
                const u32x4 xv = any_piece(p.a[0] + (m0 + r) * p.lda, (int)k, p.L);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = widen<E>((uint16_t)(xv[e >> 1] >> (16 * (e & 1))));
                    gs[r] = __builtin_fmaf(widen<E>((uint16_t)(gv[j][e >> 1] >> (16 * (e & 1)))), x, gs[r]);
                    us[r] = __builtin_fmaf(widen<E>((uint16_t)(uv[j][e >> 1] >> (16 * (e & 1)))), x, us[r]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float gt = wave_sum(gs[r]), ut = wave_sum(us[r]);
        if (lane != 0 || r >= rows) continue;
        const int64_t m = m0 + r;
        ((uint16_t*)p.y)[m * p.ldy + n] = narrow<E>(gated_act(p.act, gt) * ut);
        if (p.gate) p.gate[m * p.ldgate + n] = narrow<E>(gt);
        if (p.up) p.up[m * p.ldup + n] = narrow<E>(ut);
    }
}

// A matrix [rows, cols] of any stride and base into rows of ldo words (a multiple of
// 8, 16-byte aligned), the columns past cols zeroed: operands of odd widths become
// ones that the streaming kernels read.  A thread copies 8 words.
__global__ void __launch_bounds__(256) repack(const uint16_t* in, int64_t ld, int64_t rows, int cols, uint16_t* out,
                                              int64_t ldo) {
    const int64_t chunks = ldo / 8, total = rows * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / chunks;
        const int c = (int)(i - r * chunks) * 8;
        *(u32x4*)(out + r * ldo + c) = any_piece(in + r * ld, c, cols);
    }
}

// One thread per four columns of a row; the splits are added in their order.
template <int E, bool F32>
__global__ void __launch_bounds__(256) split_sum(StreamProduct a) {
    const int chunks = (a.C + 3) / 4;
    const int64_t total = (a.rows ? (int64_t)*a.rows : (int64_t)a.groups * a.R) * chunks, plane = (int64_t)a.groups * a.R * a.ldp;
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
        if (a.sum_unscale) v *= *a.sum_unscale;
        const int g = gr >= a.R ? 1 : 0;
        const int64_t row = a.list ? a.list[gr] : gr - (int64_t)g * a.R;
        const int64_t at = row * a.ldy[g] + c;
        const bool whole = c + 3 < a.C;                  // stored at any alignment
        if constexpr (F32) {
            float* y = (float*)a.y[g] + at;
            if (whole) {
                f32x4 old = (f32x4){};
                if (a.accumulate) {
                    __builtin_memcpy(&old, y, 16);
                    v = old + v;
                }
                __builtin_memcpy(y, &v, 16);
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
            if (whole) {
                __builtin_memcpy(y, &u, 8);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < a.C) y[e] = narrow<E>(v[e]);
            }
        }
    }
}

// What the rounding of v to `word` leaves, rounded: 0 where the word is an infinity or NaN.
template <int E>
__device__ inline uint16_t low_word(float v, uint16_t word) {
    const float rest = v - widen<E>(word);
    return narrow<E>(__builtin_fabsf(rest) < __builtin_inff() ? rest : 0.f);
}

// dg and du of the 8 columns from c of row m; 0 past N.
template <int E>
__device__ inline void gated_piece(const GatedGradArgs& g, int64_t m, int c, float (&dg)[8], float (&du)[8]) {
    const u32x4 h = load8(g.dh + m * g.lddh + c, true, c, g.N);
    const u32x4 a = load8(g.gate + m * g.ldgate + c, true, c, g.N);
    const u32x4 u = load8(g.up + m * g.ldup + c, true, c, g.N);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        dg[e] = du[e] = 0.f;
        if (c + e >= g.N) continue;
        const int q = e >> 1, sh = 16 * (e & 1);
        const float hv = widen<E>((uint16_t)(h[q] >> sh)), uv = widen<E>((uint16_t)(u[q] >> sh));
        float av, dv;
        gated_act_grad(g.act, widen<E>((uint16_t)(a[q] >> sh)), av, dv);
        dg[e] = hv * uv * dv;
        du[e] = hv * av;
    }
}

// The largest of v >= 0 over the workgroup, on every thread; lds: a float per wave.
__device__ inline float group_max(float v, float* lds) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
    for (int w = 1; w < (int)blockDim.x / 64; ++w) v = fmaxf(v, lds[w]);
    return v;
}

// The largest finite |dg| and |du| that each workgroup meets, into head[4 + workgroup].
// Bound by the reads of dh, gate and up, which gated_grad makes again (4096 x 14336: 93 us, a
// bound without exp or division 80; 517 x 2720: 6.1; on top of gated_grad's 95 and 8.1).
template <int E>
__global__ void __launch_bounds__(1024) gated_max(GatedGradArgs g) {
    __shared__ float lds[16];
    const int chunks = g.Np / 8;
    const int64_t total = (int64_t)g.M * chunks;
    float most = 0.f;
    for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 1024) {
        const int64_t m = i / chunks;
        float dg[8], du[8];
        gated_piece<E>(g, m, (int)(i - m * chunks) * 8, dg, du);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = __builtin_fabsf(dg[e]), y = __builtin_fabsf(du[e]);
            if (x < __builtin_inff()) most = fmaxf(most, x);
            if (y < __builtin_inff()) most = fmaxf(most, y);
        }
    }
    most = group_max(most, lds);
    if (threadIdx.x == 0) g.head[4 + blockIdx.x] = most;
}

template <int E, bool LOW, bool SCALED>
__global__ void __launch_bounds__(256) gated_grad(GatedGradArgs g) {
    const int chunks = g.Np / 8;                     // 8-column pieces of a row of one half
    const int64_t total = (int64_t)g.M * chunks;
    float scale = 1.f;
    if constexpr (SCALED) {
        __shared__ float lds[4];
        float most = 0.f;
        for (int i = threadIdx.x; i < g.parts; i += 256) most = fmaxf(most, g.head[4 + i]);
        most = group_max(most, lds);
        // most = f 2^x with f in [1/2, 1): most 2^(15 - x) in [2^14, 2^15).  (Past 2^100, for
        // gradients below 2^-86, the outputs are zero anyway.)
        int x = 15;
        if (most > 0.f) __builtin_frexpf(most, &x);
        const int s = min(15 - x, 100);
        scale = __builtin_ldexpf(1.f, s);
        if (blockIdx.x == 0 && threadIdx.x == 0) g.head[0] = __builtin_ldexpf(1.f, -s);
    }
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / chunks;
        const int c = (int)(i - m * chunks) * 8;
        float gf[8], uf[8];
        gated_piece<E>(g, m, c, gf, uf);
        u32x4 dg = (u32x4){0u, 0u, 0u, 0u}, du = dg, dgl = dg, dul = dg;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int q = e >> 1, sh = 16 * (e & 1);
            if constexpr (SCALED) {
                gf[e] *= scale;
                uf[e] *= scale;
            }
            const uint16_t gw = narrow<E>(gf[e]), uw = narrow<E>(uf[e]);
            dg[q] |= (uint32_t)gw << sh;
            du[q] |= (uint32_t)uw << sh;
            if constexpr (LOW) {
                dgl[q] |= (uint32_t)low_word<E>(gf[e], gw) << sh;
                dul[q] |= (uint32_t)low_word<E>(uf[e], uw) << sh;
            }
        }
        uint16_t* row = g.d + m * 2 * g.Np + c;
        *(u32x4*)row = dg;
        *(u32x4*)(row + g.Np) = du;
        if constexpr (LOW) {
            row += (int64_t)kLowRow * 2 * g.Np;
            *(u32x4*)row = dgl;
            *(u32x4*)(row + g.Np) = dul;
        }
    }
}

template <int E, bool COUNTED>
__global__ void __launch_bounds__(1024) column_partials(ColumnSumArgs c) {
    __shared__ float lds[column_lds(1024)];
    column_block<E, 1024, COUNTED>(c, blockIdx.x, blockIdx.y, lds);
}

// The splits' sums, in their order.
template <int E, bool COUNTED>
__global__ void __launch_bounds__(64) column_finish(ColumnSumArgs c) {
    const int n = blockIdx.x * 64 + threadIdx.x;
    if (n >= c.N) return;
    float sum = c.partial[n];
#pragma unroll 8
    for (int s = 1; s < c.splits; ++s) sum += c.partial[(int64_t)s * c.N + n];
    store_sum<E, COUNTED>(c, n, sum);
}

template <int T, int E>
const void* any_fn(int mode, bool rowt) {
    if (mode == kProdGated) return (const void*)product_any<T, E, kProdGated, true, true>;
    if (mode == kProdF32) return (const void*)product_any<T, E, kProdF32, false, false>;
    return rowt ? (const void*)product_any<T, E, kProdRound, false, false>
                : (const void*)product_any<T, E, kProdRound, true, false>;
}

}  // namespace

hipError_t launch_product_any(int elem, int mode, bool rowt, const ProductArgs& p, hipStream_t stream) {
    if ((mode == kProdF32) > rowt || (mode == kProdGated && rowt)) return hipErrorInvalidValue;
    ProductArgs args = p;
    void* params[] = {&args};
    if (mode == kProdGated && p.R <= 8 * ROWS)
        return launch_kernel(elem == kBF16 ? (const void*)gated_rows_any<kBF16> : (const void*)gated_rows_any<kF16>,
                               dim3((unsigned)((p.C + 3) / 4), (unsigned)((p.R + ROWS - 1) / ROWS)), dim3(256), params, 0,
                               stream);
    const auto tiles = [&](int t) { return ((int64_t)p.R + t - 1) / t * (((int64_t)p.C + t - 1) / t); };
    const bool large = tiles(128) >= 256;             // enough tiles of 128 for every CU
    const int t = large ? 128 : kProdTile;
    args.tiles_c = (p.C + t - 1) / t;
    const void* fn = elem == kBF16 ? (large ? any_fn<128, kBF16>(mode, rowt) : any_fn<kProdTile, kBF16>(mode, rowt))
                                   : (large ? any_fn<128, kF16>(mode, rowt) : any_fn<kProdTile, kF16>(mode, rowt));
    return launch_kernel(fn, dim3((unsigned)tiles(t)), dim3(256), params, 0, stream);
}

hipError_t launch_repack(const uint16_t* in, int64_t ld, int64_t rows, int cols, uint16_t* out, int64_t ldo,
                         hipStream_t stream) {
    void* params[] = {&in, &ld, &rows, &cols, &out, &ldo};
    const int64_t blocks = (rows * (ldo / 8) + 255) / 256;
    return launch_kernel((const void*)repack, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), params, 0,
                           stream);
}

hipError_t launch_split_sum(int elem, bool f32, const StreamProduct& a, hipStream_t stream) {
    StreamProduct args = a;
    void* params[] = {&args};
    const int64_t blocks = ((int64_t)a.groups * a.R * ((a.C + 3) / 4) + 255) / 256;
    const void* fn = f32 ? (const void*)split_sum<kF16, true>
                         : elem == kBF16 ? (const void*)split_sum<kBF16, false> : (const void*)split_sum<kF16, false>;
    return launch_kernel(fn, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), params, 0, stream);
}

hipError_t launch_gated_grad(int elem, const GatedGradArgs& g, hipStream_t stream) {
    if ((elem == kF16) != (g.head != nullptr)) return hipErrorInvalidValue;
    GatedGradArgs args = g;
    void* params[] = {&args};
    const int64_t pieces = (int64_t)g.M * (g.Np / 8), blocks = (pieces + 255) / 256;
    if (g.head) {
        const int64_t parts = (pieces + 1023) / 1024;
        args.parts = (int)(parts < kGradMaxGrid ? parts : kGradMaxGrid);
        const hipError_t e = launch_kernel((const void*)gated_max<kF16>, dim3((unsigned)args.parts), dim3(1024), params, 0,
                                             stream);
        if (e != hipSuccess) return e;
    }
    const void* fn = elem == kBF16
                         ? (g.low ? (const void*)gated_grad<kBF16, true, false> : (const void*)gated_grad<kBF16, false, false>)
                         : (g.low ? (const void*)gated_grad<kF16, true, true> : (const void*)gated_grad<kF16, false, true>);
    return launch_kernel(fn, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), params, 0, stream);
}

hipError_t launch_column_sum(int elem, const ColumnSumArgs& c, hipStream_t stream) {
    ColumnSumArgs args = c;
    void* params[] = {&args};
    if (c.N > kColumnPart) {                          // (one split: so many columns fill the chip)
        for (int64_t n = 0; n < c.N; n += kColumnPart) {
            args.dy = c.dy + n;
            args.db = (char*)c.db + n * (c.f32 ? 4 : 2);
            args.N = (int)std::min((int64_t)c.N - n, kColumnPart);
            const hipError_t e = launch_column_sum(elem, args, stream);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    const unsigned gx = (unsigned)((c.N + 63) / 64);
    const void *sums, *finish;
    if (c.rows) {
        sums = elem == kBF16 ? (const void*)column_partials<kBF16, true> : (const void*)column_partials<kF16, true>;
        finish = elem == kBF16 ? (const void*)column_finish<kBF16, true> : (const void*)column_finish<kF16, true>;
    } else {
        sums = elem == kBF16 ? (const void*)column_partials<kBF16, false> : (const void*)column_partials<kF16, false>;
        finish = elem == kBF16 ? (const void*)column_finish<kBF16, false> : (const void*)column_finish<kF16, false>;
    }
    hipError_t e = launch_kernel(sums, dim3(gx, (unsigned)c.splits), dim3(1024), params, 0, stream);
    if (e != hipSuccess || c.splits == 1) return e;
    return launch_kernel(finish, dim3(gx), dim3(64), params, 0, stream);
}

}  // namespace lin
