// adamw.hip -- an AdamW step over many tensors.
//
//     g = grad * s,  s = 1 or min(1, max_norm / (norm + 1e-6))
//     m = beta1 m + (1 - beta1) g        v = beta2 v + (1 - beta2) g^2
//     p = p (1 - lr weight_decay) - lr / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)
//
// One pass: weights, gradients and moments are read once, weights and moments written.  Up to
// 72 tensors (40 with copies or gaps between rows) go into one launch, their table in its arguments; a tensor's
// values, in row-major order, are cut into chunks, one for each workgroup (shares of
// many chunks a workgroup read and wrote as many distant streams at once: 10% slower).  A thread
// takes 8 consecutive values.
//
// 8-bit moments: n codes, then a byte k + 127 for each block of 32 values, whose codes count in
// units of 2^k.  The first moment's codes are a sign, 4 bits of exponent and 3 of mantissa (the
// hardware's e4m3: 448 at most, 127 is NaN); the second's have no sign and 5 bits of exponent
// (the upper bits of a binary16 word: 61440 at most, 248 infinity, past it NaN).  m / sqrt(v)
// needs about the same range of m and of sqrt(v): 2^17 and 2^16 under a block's largest.  k is
// the smallest, from -100 on, for which the largest finite value stays under the border where it
// would round past the last code, 464 or 63488 times 2^k.  A power of two makes the division by
// it exact, so a stored moment is one rounding (half a step: 2^-4) from its value.  The moments
// are formed in FP64: sums of such few-bit numbers often lie on, or within FP32's error of, the
// border between two codes.  A second moment over zero is never stored as zero, which the next
// step would divide by.
#include "adamw.h"
#include "train.h"

namespace lin {

namespace {

constexpr int RUN = kAdamRun;

// 8 consecutive values of type T (kGradF16, kGradBF16 or kGradF32) as loaded.
template <int T>
struct Run {
    u32x4 w[T == kGradF32 ? 2 : 1];
};

template <int T>
__device__ inline Run<T> load_run(const void* p, int64_t i) {
    Run<T> r;
    __builtin_memcpy(&r, (const char*)p + i * (T == kGradF32 ? 4 : 2), sizeof r);   // at any alignment
    return r;
}

template <int T>
__device__ inline void widen_run(const Run<T>& r, float (&out)[RUN]) {
#pragma unroll
    for (int e = 0; e < RUN; ++e) {
        const uint32_t word = r.w[T == kGradF32 ? e >> 2 : 0][e & 3];   // (a bit cast of a vector's element takes its first)
        if constexpr (T == kGradF32) out[e] = __builtin_bit_cast(float, word);
        else out[e] = widen<T == kGradBF16 ? kBF16 : kF16>((uint16_t)(r.w[0][e >> 1] >> (16 * (e & 1))));
    }
}

template <int T>
__device__ inline void store_run(void* p, const float (&v)[RUN], int64_t i) {
    Run<T> r;
#pragma unroll
    for (int e = 0; e < RUN; e += 2) {
        if constexpr (T == kGradF32) {
            r.w[e >> 2][e & 3] = __builtin_bit_cast(uint32_t, v[e]);
            r.w[e >> 2][(e & 3) + 1] = __builtin_bit_cast(uint32_t, v[e + 1]);
        } else {
            constexpr int E = T == kGradBF16 ? kBF16 : kF16;
            r.w[0][e >> 1] = (uint32_t)narrow<E>(v[e]) | ((uint32_t)narrow<E>(v[e + 1]) << 16);
        }
    }
    __builtin_memcpy((char*)p + i * (T == kGradF32 ? 4 : 2), &r, sizeof r);
}

// Value by value: a tensor's last run, and tensors with gaps between their rows.
__device__ inline float value_at(const void* p, int type, int64_t at) {
    if (type == kGradF32) return ((const float*)p)[at];
    const uint16_t u = ((const uint16_t*)p)[at];
    return type == kGradBF16 ? widen<kBF16>(u) : widen<kF16>(u);
}
__device__ inline void put_at(void* p, int type, int64_t at, float v) {
    if (type == kGradF32) ((float*)p)[at] = v;
    else ((uint16_t*)p)[at] = type == kGradBF16 ? narrow<kBF16>(v) : narrow<kF16>(v);
}

// f(e, offset) for the first `count` values from value i on of a tensor with rows of cols values
// (0: no gaps) and a row stride of ld.
template <typename F>
__device__ inline void each_value(int64_t i, int count, int64_t cols, int64_t ld, F f) {
    int64_t row = cols ? i / cols : 0, col = i - row * cols;
    const int64_t end = cols ? cols : INT64_MAX;
#pragma unroll
    for (int e = 0; e < RUN; ++e) {
        if (e < count) f(e, row * ld + col);
        if (++col == end) {
            col = 0;
            ++row;
        }
    }
}

__device__ inline uint2 load_codes(const uint8_t* p) {
    uint2 r;
    __builtin_memcpy(&r, p, 8);
    return r;
}
__device__ inline void store_codes(uint8_t* p, uint2 c) { __builtin_memcpy(p, &c, 8); }

// The first `count` of 8 codes (zeros past them).
__device__ inline uint2 load_codes(const uint8_t* p, int count) {
    uint2 r{0u, 0u};
#pragma unroll
    for (int e = 0; e < RUN; ++e)
        if (e < count) (e < 4 ? r.x : r.y) |= (uint32_t)p[e] << (8 * (e & 3));
    return r;
}
__device__ inline void store_codes(uint8_t* p, uint2 c, int count) {
#pragma unroll
    for (int e = 0; e < RUN; ++e)
        if (e < count) p[e] = (uint8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
}

// 2^k of a block's byte k + 127 (0 for a byte of 0: a state of zero bytes is a state of zeros).
__device__ inline float block_unit(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// The numbers of 4 codes, in units of their block.
template <bool SECOND>
__device__ inline void decode4(uint32_t codes, float* out) {
    if constexpr (SECOND) {
        // a code is bits 7 .. 14 of a binary16 word
        const uint32_t a = __builtin_amdgcn_perm(0u, codes, 0x0c010c00u) << 7, b = __builtin_amdgcn_perm(0u, codes, 0x0c030c02u) << 7;
        out[0] = widen<kF16>((uint16_t)a);
        out[1] = widen<kF16>((uint16_t)(a >> 16));
        out[2] = widen<kF16>((uint16_t)b);
        out[3] = widen<kF16>((uint16_t)(b >> 16));
    } else {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(codes, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(codes, true);
        out[0] = a[0];
        out[1] = a[1];
        out[2] = b[0];
        out[3] = b[1];
    }
}

template <bool SECOND>
__device__ inline void decode8(uint2 codes, float (&out)[RUN]) {
    decode4<SECOND>(codes.x, out);
    decode4<SECOND>(codes.y, out + 4);
}

__device__ inline uint32_t high_word(double v) { return (uint32_t)(__builtin_bit_cast(uint64_t, v) >> 32); }
__device__ inline double from_high(uint32_t hi) { return __builtin_bit_cast(double, (uint64_t)hi << 32); }

// max(a, |b|, |c|) and min(a, b, c), a NaN left out (fmaxf makes three instructions of each maximum:
// it quiets its operands first).
__device__ inline float max3_abs(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, abs(%2), abs(%3)" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ inline float min3(float a, float b, float c) {
    float r;
    asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

template <int CTRL>
__device__ inline float dpp_max(float v) {
    const float o = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
    return max3_abs(v, o, o);
}

// The largest over the four lanes of a quad, which hold a block.
__device__ inline float block_max(float v) { return dpp_max<0x4E>(dpp_max<0xB1>(v)); }   // quad_perm [1, 0, 3, 2], [2, 3, 0, 1]

// From here on a magnitude counts as infinite: rounded to a code, it could leave binary32's range.
constexpr float kEndless = 0x1.fp127f;

// The codes of 8 values (0 past a tensor's end), given in FP32 too, and their block's byte.  What is
// rare (infinities, second moments that would round to zero) is looked for once a run and put right
// behind a branch.
template <bool SECOND>
__device__ inline uint2 encode8(const double (&v)[RUN], const float (&f)[RUN], uint32_t& byte) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < RUN; e += 2) top = max3_abs(top, f[e], f[e + 1]);
    top = block_max(top);
    const bool endless = top >= kEndless;
    if (endless) {
        top = 0.f;
#pragma unroll
        for (int e = 0; e < RUN; ++e) top = __builtin_fabsf(f[e]) < kEndless ? fmaxf(top, __builtin_fabsf(f[e])) : top;
        top = block_max(top);                         // (a quad takes this branch as one)
    }
    // 464 = 1.8125 * 2^8, 63488 = 1.9375 * 2^15: from there on the next power of two
    const int x = (int)((__builtin_bit_cast(uint32_t, top) + (SECOND ? 0x80000u : 0x180000u)) >> 23) - 127;
    const int k = max(x - (SECOND ? 15 : 8), -100);
    byte = (uint32_t)(k + 127);
    const float inverse = __builtin_bit_cast(float, (uint32_t)(127 - k) << 23);
    const uint32_t low = (uint32_t)(1023 + k - (SECOND ? 14 : 6)) << 20;   // the smallest normal code, as an upper word
    float r[RUN];
#pragma unroll
    for (int e = 0; e < RUN; ++e) {
        // Rounded to 4 significant bits (the subnormals to their spacing) by adding, and taking away,
        // 2^49 times the number's upper word: the sum's last place is then the code's, and the large
        // number an even count of those.
        const uint32_t h = SECOND ? high_word(v[e]) : high_word(v[e]) & 0x7fffffffu;
        const double big = from_high(max(h, low) + (49u << 20));
        r[e] = (float)((__builtin_fabs(v[e]) + big) - big) * inverse;
    }
    if constexpr (SECOND) {
        float least = __builtin_inff();
#pragma unroll
        for (int e = 0; e < RUN; e += 2) least = min3(least, r[e], r[e + 1]);
        if (least == 0.f) {
#pragma unroll
            for (int e = 0; e < RUN; ++e) r[e] = r[e] == 0.f && v[e] > 0.0 ? 0x1p-17f : r[e];
        }
    }
    if (endless) {
#pragma unroll
        for (int e = 0; e < RUN; ++e)
            r[e] = __builtin_fabsf(f[e]) >= kEndless ? (SECOND ? __builtin_inff() : __builtin_nanf("")) : r[e];
    }
    uint2 c;
    if constexpr (SECOND) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)                   // exact: the values are binary16's
            w[q] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(r[2 * q], r[2 * q + 1])) >> 7;
        c.x = __builtin_amdgcn_perm(w[1], w[0], 0x06040200u);
        c.y = __builtin_amdgcn_perm(w[3], w[2], 0x06040200u);
    } else {
#pragma unroll
        for (int e = 0; e < RUN; ++e) r[e] = __builtin_copysignf(r[e], f[e]);
        int a = __builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], 0, false), b = __builtin_amdgcn_cvt_pk_fp8_f32(r[4], r[5], 0, false);
        a = __builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], a, true);
        b = __builtin_amdgcn_cvt_pk_fp8_f32(r[6], r[7], b, true);
        c.x = (uint32_t)a;
        c.y = (uint32_t)b;
    }
    return c;
}

// A step's factors, the same on every thread.  What the host knows it has computed; a step or rate in
// device memory costs every thread two powers in FP64 (486 M bf16 values, device lr and step: 32-bit moments
// 1967 -> 1977 us, 8-bit ones, whose step is bound by its instructions, 922 -> 1171).
struct Factors {
    double scale;                    // of the gradients
    float keep, rate, root;          // 1 - lr weight_decay, lr / bias1, 1 / sqrt(bias2)
};

__device__ inline Factors factors(const AdamArgs& a) {
    Factors f{1.0, a.keep, a.rate, a.root};
    if (a.device_lr || a.device_step) {
        const double lr = a.device_lr ? (double)*a.device_lr : a.lr;
        double bias1 = a.bias1, bias2 = a.bias2;
        if (a.device_step) {
            const double step = (double)*a.device_step;
            bias1 = 1.0 - pow(a.beta1, step);
            bias2 = 1.0 - pow(a.beta2, step);
        }
        f.keep = (float)(1.0 - lr * a.weight_decay);
        f.rate = (float)(lr / bias1);
        f.root = (float)(1.0 / sqrt(bias2));
    }
    if (a.norm) {
        const double s = (double)a.max_norm / ((double)*a.norm + 1e-6);
        f.scale = s >= 1.0 ? 1.0 : s;                 // a NaN scale stays
    }
    return f;
}

// sqrt(v) within 2 FP32 steps, for subnormal v too (which the instruction takes for zero).
__device__ inline float root_of(float v) {
    const bool low = v < 0x1p-60f;
    const float s = __builtin_amdgcn_sqrtf(low ? v * 0x1p80f : v);
    return low ? s * 0x1p-40f : s;
}

__device__ inline float updated(float p, float m, float root, const Factors& f, float eps) {
    return p * f.keep - (f.rate * m) * __builtin_amdgcn_rcpf(root * f.root + eps);
}

// The moments of 8 values after the step, and the values.
__device__ inline void step32(const AdamArgs& a, const Factors& f, float (&p)[RUN], const float (&g)[RUN], float (&m)[RUN],
                              float (&v)[RUN]) {
    const float b1 = (float)a.beta1, r1 = (float)(1.0 - a.beta1), b2 = (float)a.beta2, r2 = (float)(1.0 - a.beta2);
    const float s = (float)f.scale;
#pragma unroll
    for (int e = 0; e < RUN; ++e) {
        const float gs = g[e] * s;
        m[e] = m[e] * b1 + gs * r1;
        v[e] = v[e] * b2 + gs * gs * r2;
        p[e] = updated(p[e], m[e], root_of(v[e]), f, a.eps);
    }
}

__device__ inline void step8(const AdamArgs& a, const Factors& f, float (&p)[RUN], const float (&g)[RUN], uint2& mc, uint2& vc,
                             uint32_t& mb, uint32_t& vb) {
    float mf[RUN], vf[RUN];
    decode8<false>(mc, mf);
    // (a block's unit is a power of two: in the factor it changes no rounding)
    const double m1 = (double)block_unit(mb) * a.beta1, m2 = (double)block_unit(vb) * a.beta2;
    const double r1 = 1.0 - a.beta1, r2 = 1.0 - a.beta2;
    // one moment after the other, held apart: together they take registers that waves could have
    double gd[RUN], w[RUN];
#pragma unroll
    for (int e = 0; e < RUN; ++e) {
        gd[e] = (double)g[e] * f.scale;
        w[e] = (double)mf[e] * m1 + gd[e] * r1;
        mf[e] = (float)w[e];
    }
    mc = encode8<false>(w, mf, mb);
    __builtin_amdgcn_sched_barrier(0);
    decode8<true>(vc, vf);
#pragma unroll
    for (int e = 0; e < RUN; ++e) {
        w[e] = (double)vf[e] * m2 + gd[e] * gd[e] * r2;
        vf[e] = (float)w[e];
    }
    vc = encode8<true>(w, vf, vb);
    __builtin_amdgcn_sched_barrier(0);
    // the root of a subnormal v is under 2^-63: nothing beside an eps of 2^-36 or more
    if (a.eps < 0x1p-36f) {                           // uniform
#pragma unroll
        for (int e = 0; e < RUN; ++e) p[e] = updated(p[e], mf[e], root_of(vf[e]), f, a.eps);
    } else {
#pragma unroll
        for (int e = 0; e < RUN; ++e) p[e] = updated(p[e], mf[e], __builtin_amdgcn_sqrtf(vf[e]), f, a.eps);
    }
}

// A chunk of a tensor without gaps that lies inside it, of types P and G: every load is issued
// before the first is used.
template <bool EIGHT, int P, int G, typename Table>
__device__ __forceinline__ void chunk_fast(const Table& t, const AdamArgs& a, const Factors& f, int i, int64_t begin) {
    constexpr int U = adam_runs(EIGHT);
    const int64_t at = begin + threadIdx.x * RUN;
    Run<P> pr[U];
    Run<G> gr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        pr[u] = load_run<P>(t.param[i], at + u * kAdamRuns);
        gr[u] = load_run<G>(t.grad[i], at + u * kAdamRuns);
    }
    float p[RUN], g[RUN];
    const auto leave = [&](int u) {
        store_run<P>(t.param[i], p, at + u * kAdamRuns);
        if constexpr (!Table::kPlain) {
            if (t.ctype[i] == kGradBF16) store_run<kGradBF16>(t.copy[i], p, at + u * kAdamRuns);
            else if (t.ctype[i] == kGradF16) store_run<kGradF16>(t.copy[i], p, at + u * kAdamRuns);
        }
    };
    if constexpr (EIGHT) {
        uint8_t *ms = (uint8_t*)t.m[i] + at, *vs = (uint8_t*)t.v[i] + at;
        uint8_t *mk = (uint8_t*)t.m[i] + t.n[i] + at / kAdamBlock, *vk = (uint8_t*)t.v[i] + t.n[i] + at / kAdamBlock;
        uint2 mc[U], vc[U];
        uint32_t mb[U], vb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mc[u] = load_codes(ms + u * kAdamRuns);
            vc[u] = load_codes(vs + u * kAdamRuns);
            mb[u] = mk[u * kAdamRuns / kAdamBlock];
            vb[u] = vk[u * kAdamRuns / kAdamBlock];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            widen_run<P>(pr[u], p);
            widen_run<G>(gr[u], g);
            step8(a, f, p, g, mc[u], vc[u], mb[u], vb[u]);
            store_codes(ms + u * kAdamRuns, mc[u]);
            store_codes(vs + u * kAdamRuns, vc[u]);
            if ((threadIdx.x & 3) == 0) {
                mk[u * kAdamRuns / kAdamBlock] = (uint8_t)mb[u];
                vk[u * kAdamRuns / kAdamBlock] = (uint8_t)vb[u];
            }
            leave(u);
        }
    } else {
        static_assert(U == 1, "one run");
        const Run<kGradF32> mr = load_run<kGradF32>(t.m[i], at), vr = load_run<kGradF32>(t.v[i], at);
        float m[RUN], v[RUN];
        widen_run<P>(pr[0], p);
        widen_run<G>(gr[0], g);
        widen_run<kGradF32>(mr, m);
        widen_run<kGradF32>(vr, v);
        step32(a, f, p, g, m, v);
        store_run<kGradF32>(t.m[i], m, at);
        store_run<kGradF32>(t.v[i], v, at);
        leave(0);
    }
}

// Any run.  Lanes past the end take part in their block's maximum with zeros.
template <bool EIGHT, typename Table>
__device__ __forceinline__ void run_any(const Table& t, const AdamArgs& a, const Factors& f, int i, int64_t at) {
    const int64_t n = t.n[i], left = n - at;
    int64_t cols = 0, ldp = 0, ldg = 0;
    if constexpr (!Table::kPlain) {
        cols = t.cols[i];
        ldp = t.ldp[i];
        ldg = t.ldg[i];
    }
    const int ptype = t.types[i] / 3, gtype = t.types[i] % 3;
    const int count = left >= RUN ? RUN : left > 0 ? (int)left : 0;
    float p[RUN] = {}, g[RUN] = {};
    const bool whole = cols == 0 && count == RUN;     // (of a tensor's last chunk, all runs but one)
    const auto get = [&](const void* from, int type, int64_t ld, float (&out)[RUN]) {
        if (!whole) each_value(at, count, cols, ld, [&](int e, int64_t o) { out[e] = value_at(from, type, o); });
        else if (type == kGradF32) widen_run<kGradF32>(load_run<kGradF32>(from, at), out);
        else if (type == kGradBF16) widen_run<kGradBF16>(load_run<kGradBF16>(from, at), out);
        else widen_run<kGradF16>(load_run<kGradF16>(from, at), out);
    };
    const auto put = [&](void* to, int type, int64_t ld, const float (&v)[RUN]) {
        if (!whole) each_value(at, count, cols, ld, [&](int e, int64_t o) { put_at(to, type, o, v[e]); });
        else if (type == kGradF32) store_run<kGradF32>(to, v, at);
        else if (type == kGradBF16) store_run<kGradBF16>(to, v, at);
        else store_run<kGradF16>(to, v, at);
    };
    get(t.param[i], ptype, ldp, p);
    get(t.grad[i], gtype, ldg, g);
    if constexpr (EIGHT) {
        uint8_t *ms = (uint8_t*)t.m[i], *vs = (uint8_t*)t.v[i];
        const int64_t block = n + at / kAdamBlock;
        const bool full = count == RUN;
        uint2 mc = full ? load_codes(ms + at) : load_codes(ms + at, count);
        uint2 vc = full ? load_codes(vs + at) : load_codes(vs + at, count);
        uint32_t mb = count ? ms[block] : 0u, vb = count ? vs[block] : 0u;
        step8(a, f, p, g, mc, vc, mb, vb);
        if (full) {
            store_codes(ms + at, mc);
            store_codes(vs + at, vc);
        } else {
            store_codes(ms + at, mc, count);
            store_codes(vs + at, vc, count);
        }
        if (count && (threadIdx.x & 3) == 0) {
            ms[block] = (uint8_t)mb;
            vs[block] = (uint8_t)vb;
        }
    } else {
        float *mp = (float*)t.m[i] + at, *vp = (float*)t.v[i] + at;
        float m[RUN] = {}, v[RUN] = {};
        if (count == RUN) {
            widen_run<kGradF32>(load_run<kGradF32>(mp, 0), m);
            widen_run<kGradF32>(load_run<kGradF32>(vp, 0), v);
            step32(a, f, p, g, m, v);
            store_run<kGradF32>(mp, m, 0);
            store_run<kGradF32>(vp, v, 0);
        } else {
#pragma unroll
            for (int e = 0; e < RUN; ++e)
                if (e < count) {
                    m[e] = mp[e];
                    v[e] = vp[e];
                }
            step32(a, f, p, g, m, v);
#pragma unroll
            for (int e = 0; e < RUN; ++e)
                if (e < count) {
                    mp[e] = m[e];
                    vp[e] = v[e];
                }
        }
    }
    put(t.param[i], ptype, ldp, p);
    if constexpr (!Table::kPlain)
        if (t.ctype[i] != kNoCopy) put(t.copy[i], t.ctype[i], t.ldc[i], p);
}

// The tensor that holds chunk c: the last whose first chunk is <= c.
template <typename Table>
__device__ inline int tensor_of(const Table& t, int64_t c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// One chunk per workgroup, in their order (past the grid's limit the next ones after it).
template <bool EIGHT, typename Table>
__global__ void __launch_bounds__(256, 4) adamw(Table t, AdamArgs a) {
    const Factors f = factors(a);
    for (int64_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const int64_t begin = (c - t.first[i]) * adam_chunk(EIGHT);
        bool gaps = false;
        if constexpr (!Table::kPlain) gaps = t.cols[i] != 0;
        if (gaps || begin + adam_chunk(EIGHT) > t.n[i]) {
            for (int u = 0; u < adam_runs(EIGHT) && begin + u * kAdamRuns < t.n[i]; ++u)
                run_any<EIGHT>(t, a, f, i, begin + u * kAdamRuns + threadIdx.x * RUN);
            continue;
        }
        switch (t.types[i]) {                         // uniform
            case 0: chunk_fast<EIGHT, 0, 0>(t, a, f, i, begin); break;
            case 1: chunk_fast<EIGHT, 0, 1>(t, a, f, i, begin); break;
            case 2: chunk_fast<EIGHT, 0, 2>(t, a, f, i, begin); break;
            case 3: chunk_fast<EIGHT, 1, 0>(t, a, f, i, begin); break;
            case 4: chunk_fast<EIGHT, 1, 1>(t, a, f, i, begin); break;
            case 5: chunk_fast<EIGHT, 1, 2>(t, a, f, i, begin); break;
            case 6: chunk_fast<EIGHT, 2, 0>(t, a, f, i, begin); break;
            case 7: chunk_fast<EIGHT, 2, 1>(t, a, f, i, begin); break;
            default: chunk_fast<EIGHT, 2, 2>(t, a, f, i, begin); break;
        }
    }
}

template <bool SECOND>
__global__ void __launch_bounds__(256) adamw_values(ValueTable t) {
    for (int64_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const int64_t n = t.n[i], begin = (c - t.first[i]) * kValueChunk, at = begin + threadIdx.x * RUN;
        const uint8_t *s = t.state[i] + at, *k = t.state[i] + n + at / kAdamBlock;
        float v[RUN];
        if (t.cols[i] == 0 && begin + kValueChunk <= n) {
            uint2 codes[kValueRuns];
            uint32_t byte[kValueRuns];
#pragma unroll
            for (int u = 0; u < kValueRuns; ++u) {
                codes[u] = load_codes(s + u * kAdamRuns);
                byte[u] = k[u * kAdamRuns / kAdamBlock];
            }
#pragma unroll
            for (int u = 0; u < kValueRuns; ++u) {
                decode8<SECOND>(codes[u], v);
#pragma unroll
                for (int e = 0; e < RUN; ++e) v[e] *= block_unit(byte[u]);
                if (t.f32[i]) store_run<kGradF32>(t.out[i], v, at + u * kAdamRuns);
                else store_run<kGradBF16>(t.out[i], v, at + u * kAdamRuns);
            }
            continue;
        }
        for (int u = 0; u < kValueRuns; ++u) {
            const int64_t left = n - at - u * kAdamRuns;
            if (left <= 0) break;
            const int count = left >= RUN ? RUN : (int)left;
            decode8<SECOND>(load_codes(s + u * kAdamRuns, count), v);
#pragma unroll
            for (int e = 0; e < RUN; ++e) v[e] *= block_unit(k[u * kAdamRuns / kAdamBlock]);
            each_value(at + u * kAdamRuns, count, t.cols[i], t.ld[i],
                       [&](int e, int64_t o) { put_at(t.out[i], t.f32[i] ? kGradF32 : kGradBF16, o, v[e]); });
        }
    }
}

}  // namespace

template <typename Table>
static hipError_t launch_table(bool eight, const Table& t, const AdamArgs& a, int grid, hipStream_t stream) {
    Table table = t;
    AdamArgs args = a;
    void* params[] = {&table, &args};
    return launch_kernel(eight ? (const void*)adamw<true, Table> : (const void*)adamw<false, Table>, dim3((unsigned)grid),
                         dim3(256), params, 0, stream);
}

hipError_t launch_adamw(bool eight, const AdamTable& t, const AdamArgs& a, int grid, hipStream_t stream) {
    return launch_table(eight, t, a, grid, stream);
}
hipError_t launch_adamw(bool eight, const AdamPlainTable& t, const AdamArgs& a, int grid, hipStream_t stream) {
    return launch_table(eight, t, a, grid, stream);
}

hipError_t launch_adamw_values(bool second, const ValueTable& t, int grid, hipStream_t stream) {
    ValueTable table = t;
    void* params[] = {&table};
    return launch_kernel(second ? (const void*)adamw_values<true> : (const void*)adamw_values<false>, dim3((unsigned)grid),
                         dim3(256), params, 0, stream);
}

}  // namespace lin
