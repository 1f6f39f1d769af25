// train_host.h -- what the C ABI's files of the training operators share on the host:
// operand checks, copies of operands that the streaming kernels cannot read, and the plans
// and launches of the gradients' streaming products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "../../include/linear_amd.h"
#include "abi.h"
#include "train.h"

namespace lin {

inline int32_t launched(hipError_t e) {
    if (e == hipSuccess) return LINEAR_OK;
    set_last_hip_error((int32_t)e);
    return LINEAR_E_LAUNCH;
}

// Elements that one operand may span: byte addresses stay far inside 64 bits.
constexpr int64_t kMaxElems = int64_t(1) << 58;

// Sizes leave room below 2^31 for the last tile's rows and columns.
constexpr int64_t kMaxSize = kMaxDim - 65535;

inline bool dims_ok(int64_t M, int64_t N, int64_t K) {
    return M >= 0 && N >= 0 && K >= 0 && M <= kMaxSize && N <= kMaxSize && K <= kMaxSize;
}

// A [rows, cols] operand of a call: its checks in the order NULL, stride.
struct Operand {
    const void* p;
    int64_t rows, ld, cols;
    int64_t bytes = 2;
    bool empty() const { return rows == 0 || cols == 0; }
    Extent range() const { return extent(p, rows, ld, cols, bytes); }
};

inline int32_t check_operand(const Operand& o) {
    if (o.empty()) return LINEAR_OK;
    if (!o.p) return LINEAR_E_NULL;
    if (o.ld < o.cols || (o.rows > 1 && o.ld > kMaxLdOut)) return LINEAR_E_STRIDE;
    if ((o.rows - 1) * o.ld > kMaxElems - o.cols) return LINEAR_E_STRIDE;
    return LINEAR_OK;
}

// Whether two operands share no byte: apart in memory, or columns of their own in rows of
// one length (the projections side by side in one [M, 2N] tensor).
inline bool apart(const Operand& a, const Operand& b) {
    if (!overlaps(a.range(), b.range())) return true;
    if (a.rows == 1 || b.rows == 1 || a.ld * a.bytes != b.ld * b.bytes) return false;
    const bool swap = (uintptr_t)b.p < (uintptr_t)a.p;
    const Operand &lo = swap ? b : a, &hi = swap ? a : b;
    const int64_t row = a.ld * a.bytes, at = (int64_t)(((uintptr_t)hi.p - (uintptr_t)lo.p) % (uintptr_t)row);
    return at >= lo.cols * lo.bytes && at + hi.cols * hi.bytes <= row;
}

// The operands' own checks, then: no output may overlap an input or another output.
template <int NI, int NO>
inline int32_t check_operands(const Operand (&in)[NI], const Operand (&out)[NO]) {
    int32_t st = LINEAR_OK;
    auto first = [&](int32_t want) {
        for (const Operand& o : in)
            if (check_operand(o) == want) return true;
        for (const Operand& o : out)
            if (o.p && check_operand(o) == want) return true;
        return false;
    };
    for (int32_t code : {LINEAR_E_NULL, LINEAR_E_STRIDE})
        if (st == LINEAR_OK && first(code)) st = code;
    if (st != LINEAR_OK) return st;
    for (int i = 0; i < NO; ++i) {
        if (!out[i].p || out[i].empty()) continue;
        for (const Operand& o : in)
            if (!o.empty() && !apart(out[i], o)) return LINEAR_E_ALIAS;
        for (int j = 0; j < i; ++j)
            if (out[j].p && !out[j].empty() && !apart(out[i], out[j])) return LINEAR_E_ALIAS;
    }
    return LINEAR_OK;
}

inline int64_t tiles_of(int64_t n, int64_t t) { return (n + t - 1) / t; }

inline bool al16(const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0; }

// The time of a streaming launch in microseconds, from measurements on a whole MI355X:
// rounds of tiles over the CUs (the small tiles run several per
// CU), each a start and end plus a time per slice of 64.
struct TileTime {
    double fixed, slice;
    int per_cu;
};

inline double rounds_time(const TileTime& t, int64_t tiles, int64_t slices, int cus) {
    return (double)tiles_of(tiles, (int64_t)cus * t.per_cu) * (t.fixed + t.slice * (double)slices);
}

// What the streaming kernels read: 16-byte chunks of rows, offsets of a tile's rows in 32 bits.
inline bool streamable(const void* p, int64_t ld) { return al16(p, ld) && ld <= kMaxLdIn; }

inline int32_t check_workspace(const void* ws, int64_t have, int64_t need) {
    if (need == 0) return LINEAR_OK;
    if (!ws) return LINEAR_E_NULL;
    if (have < need || (uintptr_t)ws % 16 != 0) return LINEAR_E_WORKSPACE;
    return LINEAR_OK;
}

// Operands whose width is not a multiple of 8 are copied into padded rows in the
// workspace, behind the partial sums (4099 x 4099 x 4099 bf16 dx: 167 us; 4096 x 4096 x
// 4096 off 16-byte alignment, which is read in place: 292).
inline int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }
inline int64_t round256(int64_t bytes) { return (bytes + 255) / 256 * 256; }
inline bool pack_ok(int64_t rows, int64_t cols) { return rows == 0 || round8(cols) <= kMaxElems / 16 / rows; }
inline int64_t packed_bytes(int64_t rows, int64_t cols) { return cols % 8 ? round256(rows * round8(cols) * 2) : 0; }

// The operand p [rows, cols] as the streaming kernels can read it: as it is, or copied
// to `space`, which then moves on.  contracted: its columns are contraction indices, so
// the last piece of a row has to hold zeros past them.  (Rows too long for the
// streaming kernels stay as they are: so does their stride, which those then refuse.)
inline int32_t pack_operand(const uint16_t*& p, int64_t& ld, int64_t rows, int64_t cols, bool contracted, unsigned char*& space,
                     void* stream) {
    if (cols % 8 == 0 || (streamable(p, ld) && !contracted) || rows == 0 || round8(cols) > kMaxLdIn) return LINEAR_OK;
    uint16_t* out = (uint16_t*)space;
    const int32_t st = launched(launch_repack(p, ld, rows, (int)cols, out, round8(cols), (hipStream_t)stream));
    p = out;
    ld = round8(cols);
    space += packed_bytes(rows, cols);
    return st;
}

// A streaming product's plan: the tile, the splits of the contraction, and, where the
// last round of tiles would leave much of the chip idle, the first output column of a
// second launch with a tile of its own (0: one launch).
struct StreamPlan {
    int cfg, splits;
    int64_t c1;
    int cfg1;
    double time;
};

// kGradConfigs' times, from 4096 x 4096 outputs at 1 to 64 slices (and 1024 x 1024 for
// the small tiles).  128 x 128 comes with a deep ring for a single round and, with two
// slots, two to a CU, whose ends overlap: 11960 x 2632 outputs of one slice take 21.4 us
// on the latter, 28 to 33 on the other large tiles.  The splits' partial sums cost a
// launch and their traffic (0.65 us per MB written and read back).
constexpr TileTime kGradTimes[kNumGradConfigs] = {{10.2, 1.50, 1}, {7.0, 0.83, 1}, {4.1, 0.50, 1},
                                                       {2.8, 0.365, 2}, {3.4, 0.20, 1}, {5.7, 0.92, 2}};
constexpr int kPlanCus = 256;      // plans (and so workspaces) do not depend on the device
constexpr double kLaunchGap = 4.0;

inline double tile_time(int cfg, int64_t groups, int64_t R, int64_t C, int64_t slices, int64_t splits) {
    const GradConfig& g = kGradConfigs[cfg];
    const double main = rounds_time(kGradTimes[cfg], splits * groups * tiles_of(R, g.bm) * tiles_of(C, g.bn),
                                    tiles_of(slices, splits), kPlanCus);
    return splits == 1 ? main : main + 3.5 + 0.65e-6 * 4.0 * (double)splits * (double)groups * (double)R * (double)C;
}

// only64: one launch of a 64-row tile.  split_large: the 256-row tiles may share a contraction too,
// for those of a vocabulary's length (cross entropy, loss and gradients: 1000 x 128259 x 4096 3792 ->
// 3489 us, 1999 x 32001 x 2048 982 -> 953).
inline StreamPlan plan_stream(int64_t groups, int64_t R, int64_t C, int64_t slices, bool only64 = false, bool split_large = false) {
    StreamPlan p{only64 ? kPairSmall : 0, 1, 0, 0, 0.0};
    double best = tile_time(p.cfg, groups, R, C, slices, 1);
    for (int c = 0; c < kNumGradConfigs; ++c) {
        if (only64 && kGradConfigs[c].bm != 64) continue;
        for (int64_t s = 1; s <= 16 && (s == 1 || 2 * s <= slices); ++s) {
            // the large tiles fill the chip where splitting pays, and past twice the chip's
            // tiles a split only adds traffic
            if (s > 1 && !split_large && (kGradConfigs[c].bm == 256 || kGradConfigs[c].stages == 2)) break;
            if (s > 1 && s * groups * tiles_of(R, kGradConfigs[c].bm) * tiles_of(C, kGradConfigs[c].bn) >
                             2 * kPlanCus * kGradTimes[c].per_cu)
                break;
            const double t = tile_time(c, groups, R, C, slices, s);
            if (t < best) {
                best = t;
                p.cfg = c;
                p.splits = (int)s;
            }
        }
    }
    const GradConfig& g = kGradConfigs[0];
    const int64_t rows = groups * tiles_of(R, g.bm), cols = tiles_of(C, g.bn);
    const int64_t whole = rows > 0 ? rows * cols / kPlanCus * kPlanCus / rows : 0;   // column tiles in whole rounds
    if (!only64 && whole > 0 && whole < cols) {
        const double head = tile_time(0, groups, R, whole * g.bn, slices, 1) + kLaunchGap;
        for (int c = 0; c < kNumGradConfigs; ++c) {
            const double t = head + tile_time(c, groups, R, C - whole * g.bn, slices, 1);
            if (t < best) {
                best = t;
                p = StreamPlan{0, 1, whole * g.bn, c, 0.0};
            }
        }
    }
    p.time = best;
    return p;
}

// Whether the bias gradient's workgroups fit on the chip beside the product's tiles:
// then they cost neither a launch nor time (1024 x 1024 x 768: 4.5 us saved).
inline bool sums_fit(const StreamPlan& p, int64_t groups, int64_t R, int64_t C, int cus) {
    const GradConfig& g = kGradConfigs[p.cfg];
    if (g.bm != 64 || p.splits != 1 || p.c1 != 0) return false;
    return groups * tiles_of(R, g.bm) * tiles_of(C, g.bn) + tiles_of(R, 64) <= (int64_t)cus * kGradTimes[p.cfg].per_cu;
}

// dx [R, C] over sx slices and dw (groups of [Rw, C]) over sw slices in one launch, where their
// tiles together, spread over the CUs, take less than `time`: whether, and the tiles of both.
// (Both then keep these plans, unsplit, launched together or alone.)  only64: dx on 64-row tiles.
inline bool plan_pair(StreamPlan& dx, StreamPlan& dw, double time, int64_t R, int64_t C, int64_t sx, int64_t groups, int64_t Rw,
                      int64_t sw, bool only64) {
    bool pair = false;
    const GradConfig& gw = kGradConfigs[kPairTile];
    const TileTime& tw = kGradTimes[kPairTile];
    const double wt = tw.fixed + tw.slice * (double)sw;
    const double wsum = wt * (double)(groups * tiles_of(Rw, gw.bm) * tiles_of(C, gw.bn));
    for (int c : {kPairSmall, kPairTile}) {
        const GradConfig& g = kGradConfigs[c];
        if (only64 && g.bm != 64) continue;
        const TileTime& t = kGradTimes[c];
        const double xt = t.fixed + t.slice * (double)sx;
        const double xsum = xt * (double)(tiles_of(R, g.bm) * tiles_of(C, g.bn));
        const double all = std::max(std::max(xt, wt), (xsum + wsum) / kPlanCus + 0.5 * wt);
        if (all < time) {
            time = all;
            pair = true;
            dx = StreamPlan{c, 1, 0, 0, xt};
            dw = StreamPlan{kPairTile, 1, 0, 0, wt};
        }
    }
    return pair;
}

// Bytes of partial sums of a product's plan.
inline int64_t partial_bytes(const StreamPlan& p, int64_t groups, int64_t R, int64_t C) {
    return p.splits > 1 ? p.splits * groups * R * ((C + 7) / 8 * 8) * 4 : 0;
}
inline int64_t partial_bytes(int64_t groups, int64_t R, int64_t C, int64_t slices) {
    return partial_bytes(plan_stream(groups, R, C, slices), groups, R, C);
}

inline int64_t slices_of(int64_t L) { return (L + 63) / 64; }

// A product's tiles under a plan.
inline void set_tiles(StreamProduct& a, const StreamPlan& p, const DevInfo& di) {
    const GradConfig& g = kGradConfigs[p.cfg];
    a.tiles_r = (int)tiles_of(a.R, g.bm);
    a.tiles_c = (int)tiles_of(a.C, g.bn);
    a.xcd_shift = di.xcd_shift;
    a.splits = p.splits;
}

// A streaming product's launches under its plan; the operands are set by the caller.
// partial: device memory of the plan's partial sums.
inline int32_t launch_stream(int elem, bool rowt, int mode, StreamProduct& a, const StreamPlan& p, const DevInfo& di,
                      void* partial, hipStream_t stream) {
    const GradConfig& g = kGradConfigs[p.cfg];
    const bool f32 = mode == kOutF32 || mode == kOutF32Add;
    const int64_t eb = f32 ? 4 : 2;
    set_tiles(a, p, di);
    if (p.c1 > 0) {
        StreamProduct head = a;
        head.C = (int)p.c1;
        head.tiles_c = (int)(p.c1 / g.bn);
        const int32_t st = launched(launch_grad_stream(elem, p.cfg, rowt, mode, head, stream));
        if (st != LINEAR_OK) return st;
        const GradConfig& g1 = kGradConfigs[p.cfg1];
        a.C -= (int)p.c1;
        a.tiles_r = (int)tiles_of(a.R, g1.bm);
        a.tiles_c = (int)tiles_of(a.C, g1.bn);
        for (int i = 0; i < 2; ++i) {
            if (a.c[i]) a.c[i] += p.c1;
            if (a.y[i]) a.y[i] = (char*)a.y[i] + p.c1 * eb;
        }
        return launched(launch_grad_stream(elem, p.cfg1, rowt, mode, a, stream));
    }
    if (p.splits == 1) return launched(launch_grad_stream(elem, p.cfg, rowt, mode, a, stream));
    a.partial = (float*)partial;
    a.ldp = ((int64_t)a.C + 7) / 8 * 8;
    a.accumulate = mode == kOutF32Add;
    const int32_t st = launched(launch_grad_stream(elem, p.cfg, rowt, kOutF32, a, stream));
    if (st != LINEAR_OK) return st;
    if (a.fold) a.R = a.fold;
    if (rowt) a.rows = nullptr;                       // it counted the contraction, not the output's rows
    return launched(launch_split_sum(elem, f32, a, stream));
}

// The weight call's partial sums: db's and dw's, one after the other in the same space.
inline int64_t weight_scratch(int64_t M, int64_t N, int64_t K) {
    const int64_t sums = column_sum_splits(M, N);
    return std::max(sums > 1 ? sums * N * 4 : 0, partial_bytes(1, N, K, slices_of(M)));
}

inline int64_t type_bytes(int64_t type) { return type == LINEAR_TYPE_F32 ? 4 : 2; }

inline int32_t check_tensor(const linear_tensor& t) {
    if (t.type != LINEAR_TYPE_F16 && t.type != LINEAR_TYPE_BF16 && t.type != LINEAR_TYPE_F32) return LINEAR_E_VALUE;
    if (t.rows < 0 || t.cols < 0 || t.rows > kMaxDim || t.cols > (int64_t(1) << 46)) return LINEAR_E_SHAPE;
    if (t.rows == 0 || t.cols == 0) return LINEAR_OK;
    if (!t.data) return LINEAR_E_NULL;
    if (t.rows > 1 && (t.ld < t.cols || t.ld > kMaxLdOut || (t.rows - 1) * t.ld > kMaxElems - t.cols))
        return LINEAR_E_STRIDE;
    return LINEAR_OK;
}

struct Range {
    Extent e;
    bool out;
};

}  // namespace lin
