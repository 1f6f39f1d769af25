// grad_impl.h -- the streaming MFMA kernels of the gradients' products (templates).
//
//     dx [M, K] = dy [M, N] . weight [N, K]        contraction over n
//     dw [N, K] = dy [M, N]^T . x [M, K]           contraction over m
//
// In both the operand that supplies the output columns (weight, x) is contraction-
// major: one contraction index is a row of memory.  So is dy in dw.  A matrix-core
// operand holds 8 consecutive contraction indices per lane, so these panels are
// read out of LDS with the transposing read ds_read_b64_tr_b16: within each group
// of 16 lanes, lane i receives the elements that lanes 4j + i/4 (j = 0..3) address
// at their offset i % 4; when the lanes address 4 contraction rows x 16 columns in
// 8-byte pieces, lane i receives 4 consecutive contraction indices of column i.
// Nothing is transposed in memory.
//
// The tile is the layer's own: columns are the MFMA A operand and rows the B
// operand, so a lane ends with four consecutive columns of a row; slices of 64
// contraction indices stream through an LDS ring by direct-to-LDS loads; the
// fragments of the next K step are read while the MFMAs of the current one run;
// ends in finish_tile.  v_mfma_f32_16x16x32 throughout.
//
// Layout in LDS of a panel slice: 64 rows of B columns (2B bytes), 32-byte column
// pair u of row k at pair u ^ swz(k), swz(k) = 2 (k mod 4) + (k / 8) mod 2.  The LDS
// serves a 64-lane 8-byte read 32 lanes at a time: those fetch the pieces of rows
// 4i .. 4i + 3 and 4i + 8 .. 4i + 11 in one pair, which swz sends to eight
// different 32-byte bank groups.  A 64-column panel has four pairs a row and two rows
// in 256 bytes: there swz(k) = (k / 2) mod 2 + 2 ((k / 8) mod 2).  A contraction-contiguous row operand (dy in dx)
// is laid out as in the layer's kernel.
//
// The resources are made anew for each slice, from its own first row and with its
// own length: offsets within a slice stay small whatever the operand's size, rows
// past the contraction's end read as zero, and a lane's offsets never change.
#pragma once

#include "columns.h"
#include "gemm_impl.h"
#include "train.h"

namespace lin {

template <int B>
__host__ __device__ constexpr int panel_swz(int k) {
    return B == 64 ? ((k >> 1) & 1) | (((k >> 3) & 1) << 1) : 2 * (k & 3) | ((k >> 3) & 1);
}

// Direct-to-LDS load as lds_dma16, in inline assembly: the compiler does not see an
// LDS write, so it puts no wait for every load in flight (vmcnt 0) before the
// transposing reads, which name no LDS bytes it could tell apart.  The ring's own
// waits (an explicit vmcnt and a barrier per slice) order the two.  There is no
// register output.  The s_nop covers the wait states after the write of m0, and
// those between a vector write of a resource word and its use.  m0 cannot be named as
// clobbered (the compiler reserves it): the build checks that no other instruction of
// these kernels uses it.  (Handing back its old value after each load would need no
// check, and takes 2 to 4% more of dx: 8192 x 4096 x 4096 bf16 214.5 -> 223.4 us.)
__device__ __forceinline__ void lds_dma16_raw(__amdgpu_buffer_rsrc_t r, uint32_t lds, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(r));
}

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) unsigned char lds_byte;

// LDS bytes at an address (constant offsets from it go into the read instruction).
__device__ __forceinline__ lds_byte* lds_at(uint32_t addr) { return (lds_byte*)(uintptr_t)addr; }

// The transposing read of 8 bytes per lane.
__device__ __forceinline__ uint2 lds_tr(lds_byte* p) {
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p));
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// A resource over `bytes` bytes from p (none when negative).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t slice_rsrc(const uint16_t* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, max(bytes, 0), kRsrcWord3);
}

// Workgroup: one BM x BN tile of one group's output.  ROWT: the row operand is
// contraction-major too (dw); else contraction-contiguous (dx).
//
// KG sets of WM x WN waves share the tile's slices, each set with a ring of its own,
// and add their sums in LDS at the end: a small tile's slice is bound by the latency of
// its reads, so several in flight cost one's time (no traffic, unlike a split over
// workgroups).  The sets run the same number of slices, empty ones at the end.
template <int BM, int BN, int KG, int STAGES>
constexpr int grad_lds = KG * STAGES * 64 * (BM + BN) * 2;   // bytes of the rings

template <int BM, int BN, int WM, int WN, int KG, int STAGES, bool ROWT, int E, int MODE>
__device__ __forceinline__ void grad_tile(const StreamProduct& a, int block, unsigned char* smem) {
    constexpr int BK = 64, R = 16, KS = 2;            // slice, MFMA block, K steps of 32 per slice
    constexpr int NW = WM * WN;
    constexpr int TM = BM / WM, TN = BN / WN;
    constexpr int FM = TM / R, FN = TN / R;
    constexpr int CROW = 2 * BN, RROW = ROWT ? 2 * BM : 2 * BK;   // LDS bytes per row of each panel
    constexpr int CBYTES = BK * CROW, RBYTES = BM * BK * 2;
    constexpr int SLICE = CBYTES + RBYTES;
    constexpr int GC = CBYTES / 1024 / NW, GR = RBYTES / 1024 / NW;   // loads per wave and slice
    constexpr int GPW = GC + GR;
    static_assert(CBYTES % (1024 * NW) == 0 && RBYTES % (1024 * NW) == 0, "loads must divide evenly over the waves");
    static_assert(BN >= 64 && BM >= 64, "panel rows of 4 or more pairs");
    static_assert(TM % R == 0 && TN % R == 0, "whole fragments");
    constexpr int RING = STAGES * SLICE;
    static_assert(STAGES >= 2 && KG * RING <= 160 * 1024, "LDS rings too large");
    static_assert(KG == 1 || (KG - 1) * BM * BN * 4 <= KG * RING, "the sets' sums must fit in the rings");
    static_assert(grad_lds<BM, BN, KG, STAGES> == KG * RING, "the rings' bytes");

    // the bias gradient's share of the launch (small tiles, which leave CUs to spare)
    if constexpr (ROWT && BM == 64) {
        const int tiles = a.splits * a.groups * a.tiles_r * a.tiles_c;
        if (block >= tiles) {
            static_assert(column_lds(KG * NW * 64) * 4 <= KG * RING, "the column sums fit in the rings");
            column_block<E, KG * NW * 64>(a.sums, block - tiles, 0, (float*)smem);
            return;
        }
    }

    int tr, tc;
    // row tiles of every group of every split, stacked into one grid
    tile_coords(block, a.splits * a.groups * a.tiles_r, a.tiles_c, a.xcd_shift, tr, tc);
    const int stack = tr / a.tiles_r;                 // split * groups + group
    const int split = stack / a.groups, group = stack - split * a.groups;
    const int r0 = (tr - stack * a.tiles_r) * BM, c0 = tc * BN;
    const uint16_t* rbase = a.r + group * a.rgroup;
    float back = 1.f;                                 // (read here: its latency passes under the loop)
    if constexpr (E == kF16 && MODE != kOutF32Add) {
        if (a.unscale) back = *a.unscale;
    }

    const int lane = threadIdx.x & 63;
    const int set = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane((int)threadIdx.x / (NW * 64));
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) - set * NW;
    const uint32_t base = lds_address(smem) + set * RING;

    // This wave's loads: GC of the column panel, then GR of the row operand; lane l
    // lands at byte 16 l of its KB and fetches what the layout places there.
    uint32_t goff[GPW];
    const int lines = ROWT && a.fold ? kLowRow - 1 : BK - 1, whole = ROWT && a.fold ? a.fold : BK;
    // contiguous row operand: the first contraction index fetched, which repeats every
    // second load (8 rows each, a swizzle of period 16)
    static_assert(GR % 2 == 0, "a wave's first load must start the swizzle's period");
    int gk[2];
#pragma unroll
    for (int j = 0; j < GPW; ++j) {
        const bool col = j < GC;
        const int byte = (col ? wave * GC + j : wave * GR + j - GC) * 1024 + 16 * lane;
        if (col || ROWT) {
            const int row = col ? CROW : RROW;
            const int k = byte / row, c = (byte % row / 16) ^ (2 * (col ? panel_swz<BN>(k) : panel_swz<BM>(k)));
            const int at = (col ? c0 : r0) + 8 * c;
            const int line = col ? k & lines : k;
            goff[j] = (int)(at < (col ? a.C : a.R)) & (int)(k % kLowRow < whole)
                          ? (uint32_t)((line * (int)(col ? a.ldc : a.ldr) + at) * 2) : kOOB;
        } else {
            const int r = byte / RROW, c = (byte % RROW / 16) ^ ((r >> 1) & 7);
            gk[(j - GC) % 2] = 8 * c;
            goff[j] = r0 + r < a.R ? (uint32_t)((r * (int)a.ldr + 8 * c) * 2) : kOOB;
        }
    }

    // slices: each segment's contraction in slices of BK, the segments one after the other
    // (split s takes a contiguous share of all of them, and a set of it)
    const int per = (a.L + BK - 1) / BK;
    const int s0 = (int)((int64_t)per * a.segs * split / a.splits);
    const int s1 = (int)((int64_t)per * a.segs * (split + 1) / a.splits);
    const int nk = (s1 - s0 + KG - 1) / KG;           // slices a set runs
    const int t0 = s0 + set * nk, mine = max(min(nk, s1 - t0), 0);

    // the next slice to request: its LDS slot and resources, from running scalar state.
    // A row's last 16-byte chunk is read whole (a partly valid one would be dropped): it
    // is aligned, so it lies in the page of its valid words, and what it holds past
    // them goes to outputs that are not stored.  With nothing left the lengths are not
    // positive (ld >= its columns), so the column panel and a contraction-major row
    // operand read zeros; a contiguous one is masked by its lanes' own indices.
    int seg = t0 >= per && a.segs > 1 ? 1 : 0;
    const int first = (t0 - seg * per) * BK;
    const uint16_t* cp = a.c[seg] + (int64_t)first * a.ldc;
    const uint16_t* rp = ROWT ? rbase + (int64_t)first * a.ldr : rbase + r0 * a.ldr + (int64_t)t0 * BK;
    int left = mine > 0 ? a.L - first : 0;            // contraction indices left in the segment
    int todo = mine;                                  // slices left to request
    uint32_t fill = base;
    const int ldc = (int)a.ldc, ldr = (int)a.ldr;
    const int cend = (a.C + 7) & ~7, rend = (a.R + 7) & ~7;
    const int rbytes = ((min(BM, a.R - r0) - 1) * ldr + BK) * 2;
    auto request = [&]<int J0, int J1>() {
        const int n = min(left, BK);
        const __amdgpu_buffer_rsrc_t rc = slice_rsrc(cp, ((n - 1) * ldc + cend) * 2);
        const __amdgpu_buffer_rsrc_t rr = slice_rsrc(rp, ROWT ? ((n - 1) * ldr + rend) * 2 : rbytes);
        static_for<J0, J1>([&]<int j>() {
            if constexpr (j < GC) lds_dma16_raw(rc, fill + (wave * GC + j) * 1024, goff[j]);
            else if constexpr (ROWT) lds_dma16_raw(rr, fill + CBYTES + (wave * GR + j - GC) * 1024, goff[j]);
            else
                lds_dma16_raw(rr, fill + CBYTES + (wave * GR + j - GC) * 1024, gk[(j - GC) % 2] < left ? goff[j] : kOOB);
        });
    };
    auto next = [&]() {
        fill = fill == base + (STAGES - 1) * SLICE ? base : fill + SLICE;
        left -= BK;
        cp += BK * ldc;
        rp += ROWT ? BK * ldr : BK;
        if (left <= 0 && seg + 1 < a.segs) {
            ++seg;
            left = a.L;
            cp = a.c[1];
        }
        if (--todo <= 0) left = 0;
    };

    const int wn = wave % WN, wm = wave / WN;
    // transposing reads: lane (q = lane / 16, s = lane % 16) addresses row 32 ks + 8 q +
    // s / 4 (+ 4 for the second read) and the 8-byte piece at column 4 (s % 4) of its
    // fragment's 16; the row's swizzle is the same for both reads and every ks
    const int q = lane >> 4, s = lane & 15;
    const int kq = 8 * q + (s >> 2);
    uint32_t coff[FN], roff[ROWT ? FM : KS];
#pragma unroll
    for (int i = 0; i < FN; ++i)
        coff[i] = kq * CROW + ((((wn * TN) / 16 + i) ^ panel_swz<BN>(kq)) << 5) + 8 * (s & 3);
    if constexpr (ROWT) {
#pragma unroll
        for (int j = 0; j < FM; ++j)
            roff[j] = CBYTES + kq * RROW + ((((wm * TM) / 16 + j) ^ panel_swz<BM>(kq)) << 5) + 8 * (s & 3);
    } else {
        // row lr of fragment j, chunk 4 ks + q: the swizzle (r / 2) % 8 is the same for every j
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) roff[ks] = CBYTES + (wm * TM + s) * RROW + (((4 * ks + q) ^ ((s >> 1) & 7)) << 4);
    }
    auto read_col = [&]<int ks, int i>(uint32_t slot) {
        lds_byte* p = lds_at(slot + coff[i]);
        const uint2 lo = lds_tr(p + 32 * ks * CROW), hi = lds_tr(p + (32 * ks + 4) * CROW);
        return (u32x4){lo.x, lo.y, hi.x, hi.y};
    };
    auto read_row = [&]<int ks, int j>(uint32_t slot) {
        if constexpr (ROWT) {
            lds_byte* p = lds_at(slot + roff[j]);
            const uint2 lo = lds_tr(p + 32 * ks * RROW), hi = lds_tr(p + (32 * ks + 4) * RROW);
            return (u32x4){lo.x, lo.y, hi.x, hi.y};
        } else {
            return *(lds_u32x4*)(lds_at(slot + roff[ks]) + j * R * RROW);
        }
    };

    f32x4 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = (f32x4){};

    if (nk > 0) {
        // requests past the last slice carry empty resources, so every wait is static
#pragma unroll
        for (int t = 0; t < STAGES; ++t) {
            request.template operator()<0, GPW>();
            next();
        }
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((STAGES - 1) * GPW) : "memory");
        lds_barrier();
        if constexpr (ROWT) {
            if (a.fold) {                             // uniform: one slice
                // rows kLowRow .. of the column panel, which the second words meet: an infinity of x
                // is the first words' alone, a zero or a word of the other sign would make it NaN (16 x
                // 14336 x 4096 bf16: 2.5 us of 147)
                for (int o = (int)threadIdx.x % (NW * 64) * 16; o < a.fold * CROW; o += NW * 1024) {
                    u32x4* v = (u32x4*)(smem + set * RING + kLowRow * CROW + o);
                    *v = finite_words<E>(*v);
                }
                lds_barrier();
            }
        }
        // the column fragments are double buffered; a row fragment's next value is read
        // right after the MFMAs that use it
        u32x4 ca[2][FN], rb[FM];
        static_for<0, FN>([&]<int i>() { ca[0][i] = read_col.template operator()<0, i>(base); });
        static_for<0, FM>([&]<int j>() { rb[j] = read_row.template operator()<0, j>(base); });
        // the MFMAs of the step in buffer CUR while step NKS of the slice at `slot` is read
        auto step = [&]<int CUR, int NKS, bool LOADS>(uint32_t slot) {
            static_for<0, FN>([&]<int i>() { ca[CUR ^ 1][i] = read_col.template operator()<NKS, i>(slot); });
            __builtin_amdgcn_sched_barrier(0);
            static_for<0, FM>([&]<int j>() {
#pragma unroll
                for (int i = 0; i < FN; ++i) acc[i][j] = mfma16x16x32<E>(ca[CUR][i], rb[j], acc[i][j]);
                rb[j] = read_row.template operator()<NKS, j>(slot);
                if constexpr (LOADS) {
                    constexpr int J0 = GPW * j / FM, J1 = GPW * (j + 1) / FM;
                    if constexpr (J1 > J0) request.template operator()<J0, J1>();
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        uint32_t slot = base;
        for (int t = 0; t + 1 < nk; ++t) {
            step.template operator()<0, 1, false>(slot);
            slot = (t + 1) % STAGES == 0 ? base : slot + SLICE;
            // slice t + 1 has landed, and every wave has read slot t's last step
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((STAGES - 2) * GPW) : "memory");
            lds_barrier();
            step.template operator()<1, 0, true>(slot);
            next();
        }
        step.template operator()<0, 1, false>(slot);
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
            for (int i = 0; i < FN; ++i) acc[i][j] = mfma16x16x32<E>(ca[1][i], rb[j], acc[i][j]);
        // the empty requests past the end must land before the LDS is used again
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

    if constexpr (KG > 1) {
        // set s > 0 leaves its sums in LDS (thread-contiguous, one accumulator after the
        // other) and ends; set 0 adds them in order
        f32x4* sums = (f32x4*)smem;
        const int t = threadIdx.x % (NW * 64);
        __syncthreads();
        if (set > 0) {
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) sums[((set - 1) * FN * FM + i * FM + j) * NW * 64 + t] = acc[i][j];
        }
        __syncthreads();
        if (set > 0) return;
#pragma unroll
        for (int g = 0; g < KG - 1; ++g)
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[i][j] += sums[(g * FN * FM + i * FM + j) * NW * 64 + t];
    }

    // the second words' rows, 32 further down, are the same fragments of the tile's other waves
    if constexpr (!ROWT && BM == 64) {
        static_assert(WM == 2 && TM == kLowRow, "rows r and kLowRow + r in the waves wm = 0 and 1");
        if (a.fold) {                                 // uniform
            f32x4* low = (f32x4*)smem;
            __syncthreads();
            if (wm == 1) {
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int j = 0; j < FM; ++j) low[((i * FM + j) * WN + wn) * 64 + lane] = acc[i][j];
            }
            __syncthreads();
            if (wm == 0) {
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int j = 0; j < FM; ++j) {
                        // (the second words' sum is left out where the first's is infinite or NaN:
                        // with an infinite weight it may be of the other sign, or NaN)
                        const f32x4 lo = low[((i * FM + j) * WN + wn) * 64 + lane];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[i][j][e] += __builtin_fabsf(acc[i][j][e]) < __builtin_inff() ? lo[e] : 0.f;
                    }
            }
        }
    }

    if constexpr (E == kF16 && MODE != kOutF32Add) {
        if (a.unscale) {                              // uniform
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[i][j] *= back;
        }
    }

    LinearArgs o;
    o.M = !ROWT && a.fold ? a.fold : a.R;
    o.N = a.C;
    if (a.splits > 1) {                               // FP32 partial sums (kOutF32)
        o.y = a.partial + (int64_t)stack * o.M * a.ldp;
        o.ldy = a.ldp;
    } else {
        o.y = group ? a.y[1] : a.y[0];
        o.ldy = group ? a.ldy[1] : a.ldy[0];
    }
    if constexpr (MODE == kOutF32 || MODE == kOutF32Add) {
        // FP32 sums leave straight from the registers: the four lanes of a row write 64
        // bytes of it, the wave's next fragment the 64 beside them, and the workgroup
        // ends without waiting for its stores (0.5 to 2.5% faster than staged in LDS:
        // 8192 x 4096 x 4096 214 -> 211 us, adding to the output 224 -> 218)
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int r = r0 + wm * TM + j * R + s;
            if (r >= o.M) continue;
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                const int c = c0 + wn * TN + i * R + 4 * q;
                float* y = (float*)o.y + (int64_t)r * o.ldy + c;
                if (c + 3 < o.N) {                     // at any alignment
                    f32x4 v = acc[i][j];
                    if constexpr (MODE == kOutF32Add) {
                        f32x4 old;
                        __builtin_memcpy(&old, y, 16);
                        v = old + v;
                    }
                    __builtin_memcpy(y, &v, 16);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < o.N) y[e] = MODE == kOutF32Add ? y[e] + acc[i][j][e] : acc[i][j][e];
                }
            }
        }
    } else {
        finish_tile<BM, BN, WM, WN, KG * RING, E, MODE, R>(o, smem, acc, r0, c0, wave, lane);
    }
}

template <int BM, int BN, int WM, int WN, int KG, int STAGES, bool ROWT, int E, int MODE>
__global__ void __launch_bounds__(KG * WM * WN * 64)
grad_stream(StreamProduct a) {
    __shared__ __attribute__((aligned(1024))) unsigned char smem[grad_lds<BM, BN, KG, STAGES>];
    grad_tile<BM, BN, WM, WN, KG, STAGES, ROWT, E, MODE>(a, blockIdx.x, smem);
}

// Two products that do not depend on each other in one launch, the gated block's dx (on
// 64 x 64 tiles of two sets, or 128 x 128) and dWg, dWu (128 x 128): where each alone
// leaves CUs idle in its last round, the other's tiles fill them.  dx's tiles, the
// longer ones, come first.
template <bool SMALL, int E>
__global__ void __launch_bounds__(512) grad_pair(StreamProduct a, StreamProduct b) {
    __shared__ __attribute__((aligned(1024))) unsigned char smem[grad_lds<128, 128, 1, 4>];
    static_assert(grad_lds<64, 64, 2, 4> <= grad_lds<128, 128, 1, 4>, "one LDS block for both");
    const int tiles = a.tiles_r * a.tiles_c;
    if ((int)blockIdx.x < tiles) {
        if constexpr (SMALL) grad_tile<64, 64, 2, 2, 2, 4, false, E, kOutRound>(a, blockIdx.x, smem);
        else grad_tile<128, 128, 2, 4, 1, 4, false, E, kOutRound>(a, blockIdx.x, smem);
    } else {
        grad_tile<128, 128, 2, 4, 1, 4, true, E, kOutRound>(b, blockIdx.x - tiles, smem);
    }
}

static hipError_t launch_product(const void* fn, const StreamProduct& a, int threads, hipStream_t stream) {
    StreamProduct args = a;
    void* params[] = {&args};
    return launch_kernel(fn, dim3((unsigned)(a.splits * a.groups * a.tiles_r * a.tiles_c + a.sum_blocks)), dim3(threads),
                           params, 0, stream);
}

template <int BM, int BN, int WM, int WN, int KG, int STAGES, int E>
static const void* grad_fn(bool rowt, int mode) {
    if (!rowt) {
        if constexpr (BM < 256 && STAGES > 2)         // partial sums (the tiles that split contractions take)
            if (mode == kOutF32) return (const void*)grad_stream<BM, BN, WM, WN, KG, STAGES, false, E, kOutF32>;
        return (const void*)grad_stream<BM, BN, WM, WN, KG, STAGES, false, E, kOutRound>;
    }
    if (mode == kOutF32) return (const void*)grad_stream<BM, BN, WM, WN, KG, STAGES, true, E, kOutF32>;
    if (mode == kOutF32Add) return (const void*)grad_stream<BM, BN, WM, WN, KG, STAGES, true, E, kOutF32Add>;
    return (const void*)grad_stream<BM, BN, WM, WN, KG, STAGES, true, E, kOutRound>;
}

template <int E>
hipError_t launch_grad_stream_t(int cfg, bool rowt, int mode, const StreamProduct& a, hipStream_t stream) {
    switch (cfg) {
        case 0: return launch_product(grad_fn<256, 256, 2, 4, 1, 2, E>(rowt, mode), a, 512, stream);
        case 1: return launch_product(grad_fn<256, 128, 4, 2, 1, 3, E>(rowt, mode), a, 512, stream);
        case 2: return launch_product(grad_fn<128, 128, 2, 4, 1, 4, E>(rowt, mode), a, 512, stream);
        case 3: return launch_product(grad_fn<64, 64, 2, 2, 1, 5, E>(rowt, mode), a, 256, stream);
        case 4: return launch_product(grad_fn<64, 64, 2, 2, 2, 4, E>(rowt, mode), a, 512, stream);
        case 5: return launch_product(grad_fn<128, 128, 2, 4, 1, 2, E>(rowt, mode), a, 512, stream);
        default: return hipErrorInvalidValue;
    }
}

template <int E>
hipError_t launch_grad_pair_t(bool small, const StreamProduct& a, const StreamProduct& b, hipStream_t stream) {
    StreamProduct aa = a, bb = b;
    void* params[] = {&aa, &bb};
    return launch_kernel(small ? (const void*)grad_pair<true, E> : (const void*)grad_pair<false, E>,
                           dim3((unsigned)(a.tiles_r * a.tiles_c + b.groups * b.tiles_r * b.tiles_c)), dim3(512), params, 0,
                           stream);
}

}  // namespace lin
