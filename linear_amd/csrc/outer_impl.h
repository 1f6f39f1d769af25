// outer_impl.h -- a weight's gradient from few rows (templates).
//
//     y[r, c] = sum_{k < L} row[k, r] * col[k, c]          L <= 256, both contraction-major
//
// With one to four slices of contraction indices the product is bound by writing y, and a tile that
// ends after them overlaps its stores with nothing (262 MB of dW from 20 rows: 74 us on the 256 x 256 tile,
// 3.5 TB/s).  Here a workgroup of 4 waves keeps its 256 columns of the column panel in registers, as
// matrix-core operands, and walks down the rows in blocks of 64: a block's slice of the row operand
// comes through an LDS ring by direct-to-LDS loads, three blocks ahead, and its sums leave from the
// registers while later blocks are multiplied.
//
// Columns are dealt to a fragment's 16 rows so that a lane ends with 8 consecutive columns of a row
// in two fragments: 32 p + 8 h + 4 b + e for fragment 2 p + b, lane group h, element e.  Four lanes
// then store 64 bytes of a row (16-bit words), the next two fragments the 64 beside them.
//
// Loads and stores share a counter and finish in the order of their issue.  Stores go through a
// buffer resource, masked by their offset and not by a branch, so that every block issues the same
// number of them and the wait for a block's slice counts past the stores of three blocks.
#pragma once

#include "grad_impl.h"

namespace lin {

// Words are stored past the caches: y is larger than those or is read by nobody soon, and the weight
// that the next call reads stays in them (backward without dx, 64 x 128259 x 4096 bf16: 520 us with
// plain stores, 508 with the bit nt alone, 417 with nt and sc1; 20 x 32000 x 4096: 133, 122, 96).  Stores that do
// not fill parts of lines at once keep to the caches, which put them together: rows that end inside a
// cache line (loss and gradients of 20 x 32000 x 4104 373 -> 253 us, of 2 x 11771 x 2248 90 -> 65), and
// floats, 16 of whose bytes a lane stores at a time, 32 apart (backward without dx, FP32 dW: 20 x 32000 x 4096 491
// us past the caches, 197; 128 x 32000 x 4096 497, 226; on the 64-row tiles 212 and 247).
constexpr int kOuterCols = 256, kOuterRows = 64, kOuterStages = 4;

// KS: K steps of 32 contraction indices, 2, 4 or 8; POLICY: the stores' cache policy.
template <int KS, int E, int MODE, int POLICY>
__global__ void __launch_bounds__(256) outer_stream(StreamProduct a) {
    constexpr int BK = 32 * KS, CROW = 2 * kOuterCols, RROW = 2 * kOuterRows, SLOT = BK * RROW;
    constexpr int LOADS = SLOT / 4096, CLOADS = BK * CROW / 4096;   // of a slice and of the panel, per wave
    constexpr int STORES = MODE == kOutRound ? 8 : 16;
    static_assert(kOuterStages * SLOT == BK * CROW, "the ring takes the column panel's place");
    __shared__ __attribute__((aligned(1024))) unsigned char smem[BK * CROW];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int q = lane >> 4, s = lane & 15, kq = 8 * q + (s >> 2);
    const int L = a.rows ? *a.rows : a.L;
    const float back = a.unscale ? *a.unscale : 1.f;
    const int step = (int)(gridDim.x / a.tiles_c), dies = 1 << a.xcd_shift;
    int tile = (int)blockIdx.x;
    // a share's column tiles on one XCD, whose L2 then reads a slice once for all of them (256 x 32000 x
    // 4096 bf16 loss and gradients 331 -> 324 us; the shorter panels, whose slices are small, lose 1 to 2%)
    if (KS == 8 && step % dies == 0) tile = (tile / dies / a.tiles_c * dies + tile % dies) * a.tiles_c + tile / dies % a.tiles_c;
    const int c0 = tile % a.tiles_c * kOuterCols, share = tile / a.tiles_c;
    const int ldc = (int)a.ldc, ldr = (int)a.ldr;
    const uint32_t base = lds_address(smem);

    // the column panel: rows of 512 bytes in loads of 1 KB; rows past L read zero
    {
        const __amdgpu_buffer_rsrc_t rc = slice_rsrc(a.c[0] + c0, L > 0 ? ((L - 1) * ldc + ((a.C + 7) & ~7) - c0) * 2 : 0);
        static_for<0, CLOADS>([&]<int j>() {
            const int byte = (wave * CLOADS + j) * 1024 + 16 * lane, k = byte / CROW;
            const int c = (byte % CROW / 16) ^ (2 * panel_swz<kOuterCols>(k));
            lds_dma16_raw(rc, base + (wave * CLOADS + j) * 1024, c0 + 8 * c < a.C ? (uint32_t)((k * ldc + 8 * c) * 2) : kOOB);
        });
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
    u32x4 col[KS][4];                                 // [K step][fragment]
    static_for<0, KS>([&]<int ks>() {
        static_for<0, 4>([&]<int i>() {
            const int unit = wave * 4 + 2 * (i >> 1) + ((s & 3) >> 1);
            lds_byte* p = lds_at(base + (kq + 32 * ks) * CROW + ((unit ^ panel_swz<kOuterCols>(kq)) << 5) + 16 * (s & 1) + 8 * (i & 1));
            const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * CROW);
            col[ks][i] = (u32x4){lo.x, lo.y, hi.x, hi.y};
        });
    });
    lds_barrier();                                    // the panel's place is the ring's from here on

    uint32_t goff[LOADS];
    static_for<0, LOADS>([&]<int j>() {
        const int byte = (wave * LOADS + j) * 1024 + 16 * lane, k = byte / RROW;
        goff[j] = (uint32_t)((k * ldr + 8 * ((byte % RROW / 16) ^ (2 * panel_swz<kOuterRows>(k)))) * 2);
    });
    const int blocks = (a.R + kOuterRows - 1) / kOuterRows;
    const int rend = (a.R + 7) & ~7;
    int asked = share, fill = 0;                      // the next block to request, its slot
    auto request = [&]() {
        // (a resource of no bytes past the last block: nothing is read, and the count stays)
        const bool some = asked < blocks && L > 0;
        const int r0 = some ? asked * kOuterRows : 0;
        const __amdgpu_buffer_rsrc_t rr = slice_rsrc(a.r + r0, some ? ((L - 1) * ldr + rend - r0) * 2 : 0);
        static_for<0, LOADS>([&]<int j>() { lds_dma16_raw(rr, base + fill * SLOT + (wave * LOADS + j) * 1024, goff[j]); });
        asked += step;
        fill = (fill + 1) % kOuterStages;
    };
#pragma unroll
    for (int t = 0; t < kOuterStages - 1; ++t) request();

    constexpr int WORD = MODE == kOutRound ? 2 : 4;
    const int cl = c0 + wave * 64 + 8 * q;            // this lane's first column; its others are 32 further on
    int slot = 0, turn = 0;
    for (int block = share; block < blocks; block += step) {
        // the slice asked for kOuterStages - 1 blocks ago (or ahead of the loop) has landed once only
        // what was issued after it is outstanding
        static_for<0, kOuterStages>([&]<int k>() {
            constexpr int after = k * STORES + (kOuterStages - 2) * LOADS;   // (the counter's wait ends at 63)
            if (turn == k) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(after < 63 ? after : 63) : "memory");
        });
        turn = turn < kOuterStages - 1 ? turn + 1 : turn;
        lds_barrier();
        request();
        const uint32_t from = base + slot * SLOT + kq * RROW + 8 * (s & 3);
        slot = (slot + 1) % kOuterStages;
        const int r0 = block * kOuterRows, left = min(a.R - r0, kOuterRows);
        char* y = (char*)a.y[0] + (int64_t)r0 * a.ldy[0] * WORD;
        const __amdgpu_buffer_rsrc_t ry = __builtin_amdgcn_make_buffer_rsrc((void*)y, (short)0, 0x7fffffff, kRsrcWord3);
        static_for<0, 4>([&]<int j>() {
            f32x4 acc[4] = {};
            static_for<0, KS>([&]<int ks>() {
                lds_byte* p = lds_at(from + 32 * ks * RROW + ((j ^ panel_swz<kOuterRows>(kq)) << 5));
                const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * RROW);
                const u32x4 row = (u32x4){lo.x, lo.y, hi.x, hi.y};
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = mfma16x16x32<E>(col[ks][i], row, acc[i]);
            });
            const int r = 16 * j + s;
            static_for<0, 2>([&]<int p>() {
                const int c = cl + 32 * p;
                const uint32_t off = r < left && c < a.C ? (uint32_t)((r * (int)a.ldy[0] + c) * WORD) : kOOB;
                if constexpr (MODE == kOutRound) {
                    u32x4 w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x4 v = acc[2 * p + e / 2] * back;
                        w[e] = (uint32_t)narrow<E>(v[2 * (e & 1)]) | ((uint32_t)narrow<E>(v[2 * (e & 1) + 1]) << 16);
                    }
                    __builtin_amdgcn_raw_buffer_store_b128(w, ry, off, 0, POLICY);
                } else {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const f32x4 v = acc[2 * p + b] * back;
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), ry, off == kOOB ? kOOB : off + 16 * b, 0, POLICY);
                    }
                }
            });
        });
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the empty requests land before the LDS is released
}

template <int KS, int E>
static const void* outer_fn(bool words, bool past) {
    if (!words) return (const void*)outer_stream<KS, E, kOutF32, 0>;
    return past ? (const void*)outer_stream<KS, E, kOutRound, kPastCaches> : (const void*)outer_stream<KS, E, kOutRound, 0>;
}

// mode kOutRound or kOutF32.
template <int E>
hipError_t launch_outer_t(int mode, const StreamProduct& a, hipStream_t stream) {
    StreamProduct args = a;
    args.tiles_c = (a.C + kOuterCols - 1) / kOuterCols;
    const int64_t blocks = ((int64_t)a.R + kOuterRows - 1) / kOuterRows;
    // eight workgroups for each of 256 CUs, each taking every shares-th block (four: 2 to 4% slower);
    // of the longest panels, which fill a CU's LDS, one
    const int64_t shares = a.L <= 128 ? (2048 + args.tiles_c - 1) / args.tiles_c : args.tiles_c < 256 ? 256 / args.tiles_c : 1;
    int64_t used = blocks < shares ? blocks : shares;
    if (a.L > 128 && used >> a.xcd_shift) used = used >> a.xcd_shift << a.xcd_shift;
    void* params[] = {&args};
    const bool words = mode == kOutRound, past = words && whole_lines(a.y[0], a.ldy[0]);
    const void* fn = a.L <= 64    ? outer_fn<2, E>(words, past)
                     : a.L <= 128 ? outer_fn<4, E>(words, past)
                                  : outer_fn<8, E>(words, past);
    return launch_kernel(fn, dim3((unsigned)(used * args.tiles_c)), dim3(256), params, 0, stream);
}

}  // namespace lin
