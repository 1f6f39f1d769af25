// train_abi.hip -- the C ABI of the gated feed-forward block, the layer's
// gradients and the gradient norm: argument checks, kernel choice, launches.
// The conventions are linear_abi.hip's: every check runs on the host before
// anything is enqueued, and only kernels are enqueued.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <memory>
#include <new>

#include "../../include/linear_amd.h"
#include "abi.h"
#include "train.h"

namespace {

using lin::DevInfo;
using lin::Extent;
using lin::extent;
using lin::kMaxDim;
using lin::kMaxGridX;
using lin::kMaxLdOut;
using lin::overlaps;

static_assert(lin::kGradF16 == LINEAR_TYPE_F16 && lin::kGradBF16 == LINEAR_TYPE_BF16 && lin::kGradF32 == LINEAR_TYPE_F32,
              "tensor types");

int32_t launched(hipError_t e) {
    if (e == hipSuccess) return LINEAR_OK;
    lin::set_last_hip_error((int32_t)e);
    return LINEAR_E_LAUNCH;
}

// Elements that one operand may span: byte addresses stay far inside 64 bits.
constexpr int64_t kMaxElems = int64_t(1) << 58;

// Sizes leave room below 2^31 for the last tile's rows and columns.
constexpr int64_t kMaxSize = kMaxDim - 65535;

bool dims_ok(int64_t M, int64_t N, int64_t K) {
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

int32_t check_operand(const Operand& o) {
    if (o.empty()) return LINEAR_OK;
    if (!o.p) return LINEAR_E_NULL;
    if (o.ld < o.cols || (o.rows > 1 && o.ld > kMaxLdOut)) return LINEAR_E_STRIDE;
    if ((o.rows - 1) * o.ld > kMaxElems - o.cols) return LINEAR_E_STRIDE;
    return LINEAR_OK;
}

// Whether two operands share no byte: apart in memory, or columns of their own in rows of
// one length (the projections side by side in one [M, 2N] tensor).
bool apart(const Operand& a, const Operand& b) {
    if (!overlaps(a.range(), b.range())) return true;
    if (a.rows == 1 || b.rows == 1 || a.ld * a.bytes != b.ld * b.bytes) return false;
    const bool swap = (uintptr_t)b.p < (uintptr_t)a.p;
    const Operand &lo = swap ? b : a, &hi = swap ? a : b;
    const int64_t row = a.ld * a.bytes, at = (int64_t)(((uintptr_t)hi.p - (uintptr_t)lo.p) % (uintptr_t)row);
    return at >= lo.cols * lo.bytes && at + hi.cols * hi.bytes <= row;
}

// The operands' own checks, then: no output may overlap an input or another output.
template <int NI, int NO>
int32_t check_operands(const Operand (&in)[NI], const Operand (&out)[NO]) {
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

int64_t tiles_of(int64_t n, int64_t t) { return (n + t - 1) / t; }

bool any_grid_ok(int64_t R, int64_t C) { return tiles_of(R, lin::kProdTile) * tiles_of(C, lin::kProdTile) <= kMaxGridX; }

// A one-segment product with its output shape.
lin::ProductArgs product(const uint16_t* a, int64_t lda, const uint16_t* b, int64_t ldb, void* y, int64_t ldy, int64_t R,
                         int64_t C, int64_t L) {
    lin::ProductArgs p;
    memset(&p, 0, sizeof p);
    p.a[0] = a;
    p.b[0] = b;
    p.lda = lda;
    p.ldb[0] = ldb;
    p.segs = 1;
    p.R = (int)R;
    p.C = (int)C;
    p.L = (int)L;
    p.y = y;
    p.ldy = ldy;
    return p;
}

bool al16(const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0; }

// The time of a streaming launch in microseconds, from measurements on a whole MI355X:
// rounds of tiles over the CUs (the small tiles run several per
// CU), each a start and end plus a time per slice of 64.
struct TileTime {
    double fixed, slice;
    int per_cu;
};

double rounds_time(const TileTime& t, int64_t tiles, int64_t slices, int cus) {
    return (double)tiles_of(tiles, (int64_t)cus * t.per_cu) * (t.fixed + t.slice * (double)slices);
}

// kGatedConfigs' times, at 12 to 64 slices.  The 32-row tile with 16 columns of each weight serves few
// rows (its many small workgroups keep the weights' read at the memory's rate: 16 x
// 4000 x 4096 in 14 us, 21 with the 64-row tile).
constexpr TileTime kGatedTimes[lin::kNumGatedConfigs] = {{6.5, 1.60, 1}, {5.3, 0.80, 1}, {4.9, 0.50, 1}, {2.0, 0.42, 2},
                                                         {2.0, 0.30, 3}};

int choose_gated(int64_t M, int64_t N, int64_t K, int cus) {
    int best = 0;
    double best_time = -1.0;
    for (int c = 0; c < lin::kNumGatedConfigs; ++c) {
        const lin::GemmConfig& g = lin::kGatedConfigs[c];
        const double t = rounds_time(kGatedTimes[c], tiles_of(M, g.bm) * tiles_of(2 * N, g.bn), tiles_of(K, 64), cus);
        if (best_time < 0 || t < best_time) {
            best_time = t;
            best = c;
        }
    }
    return best;
}

// What the streaming kernels read: 16-byte chunks of rows, offsets of a tile's rows in 32 bits.
bool streamable(const void* p, int64_t ld) { return al16(p, ld) && ld <= lin::kMaxLdIn; }

int32_t check_workspace(const void* ws, int64_t have, int64_t need) {
    if (need == 0) return LINEAR_OK;
    if (!ws) return LINEAR_E_NULL;
    if (have < need || (uintptr_t)ws % 16 != 0) return LINEAR_E_WORKSPACE;
    return LINEAR_OK;
}

// Operands whose width is not a multiple of 8 are copied into padded rows in the
// workspace, behind the partial sums (4099 x 4099 x 4099 bf16 dx: 167 us; 4096 x 4096 x
// 4096 off 16-byte alignment, which is read in place: 292).
int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }
int64_t round256(int64_t bytes) { return (bytes + 255) / 256 * 256; }
bool pack_ok(int64_t rows, int64_t cols) { return rows == 0 || round8(cols) <= kMaxElems / 16 / rows; }
int64_t packed_bytes(int64_t rows, int64_t cols) { return cols % 8 ? round256(rows * round8(cols) * 2) : 0; }

// The operand p [rows, cols] as the streaming kernels can read it: as it is, or copied
// to `space`, which then moves on.  contracted: its columns are contraction indices, so
// the last piece of a row has to hold zeros past them.  (Rows too long for the
// streaming kernels stay as they are: so does their stride, which those then refuse.)
int32_t pack_operand(const uint16_t*& p, int64_t& ld, int64_t rows, int64_t cols, bool contracted, unsigned char*& space,
                     void* stream) {
    if (cols % 8 == 0 || (streamable(p, ld) && !contracted) || rows == 0 || round8(cols) > lin::kMaxLdIn) return LINEAR_OK;
    uint16_t* out = (uint16_t*)space;
    const int32_t st = launched(lin::launch_repack(p, ld, rows, (int)cols, out, round8(cols), (hipStream_t)stream));
    p = out;
    ld = round8(cols);
    space += packed_bytes(rows, cols);
    return st;
}

int32_t run_gated(int elem, const uint16_t* x, int64_t ldx, const uint16_t* wg, int64_t ldwg, const uint16_t* wu,
                  int64_t ldwu, int32_t act, uint16_t* h, int64_t ldh, uint16_t* gate, int64_t ldgate, uint16_t* up,
                  int64_t ldup, int64_t M, int64_t N, int64_t K, void* ws, int64_t ws_bytes, void* stream) {
    if (!dims_ok(M, N, K)) return LINEAR_E_SHAPE;
    if (!lin::is_activation(act)) return LINEAR_E_VALUE;
    if (M == 0 || N == 0) return LINEAR_OK;
    if (!h) return LINEAR_E_NULL;
    const int64_t need = linear_gated_forward_workspace_bytes(M, N, K);
    if (need < 0) return LINEAR_E_SHAPE;
    const Operand in[] = {{x, M, ldx, K}, {wg, N, ldwg, K}, {wu, N, ldwu, K}};
    const Operand out[] = {{h, M, ldh, N}, {gate, M, ldgate, N}, {up, M, ldup, N}, {ws, 1, need, need, 1}};
    int32_t st = check_operands(in, out);
    if (st != LINEAR_OK) return st;
    st = check_workspace(ws, ws_bytes, need);
    if (st != LINEAR_OK) return st;
    if (N > lin::kColumnPart) {                       // columns in parts; the workspace serves one after the other
        for (int64_t n = 0; n < N && st == LINEAR_OK; n += lin::kColumnPart)
            st = run_gated(elem, x, ldx, wg + n * ldwg, ldwg, wu + n * ldwu, ldwu, act, h + n, ldh, gate ? gate + n : gate,
                           ldgate, up ? up + n : up, ldup, M, std::min(N - n, lin::kColumnPart), K, ws, ws_bytes, stream);
        return st;
    }
    if (!any_grid_ok(M, N)) return LINEAR_E_SHAPE;
    int dev = 0;
    DevInfo di;
    st = lin::check_device(&dev, &di);
    if (st != LINEAR_OK) return st;
    if (need > 0) {
        unsigned char* space = (unsigned char*)ws;
        if ((st = pack_operand(x, ldx, M, K, true, space, stream)) != LINEAR_OK) return st;
        if ((st = pack_operand(wg, ldwg, N, K, true, space, stream)) != LINEAR_OK) return st;
        if ((st = pack_operand(wu, ldwu, N, K, true, space, stream)) != LINEAR_OK) return st;
    }
    // whole pieces of K only: the copies have them, with zeros past K
    if (streamable(x, ldx) && streamable(wg, ldwg) && streamable(wu, ldwu) && (K % 8 == 0 || need > 0)) {
        lin::LinearArgs a;
        memset(&a, 0, sizeof a);
        a.x = x;
        a.w = wg;
        a.w2 = wu;
        a.y = h;
        a.gate = gate;
        a.up = up;
        a.ldx = ldx;
        a.ldw = ldwg;
        a.ldw2 = ldwu;
        a.ldy = ldh;
        a.ldgate = ldgate;
        a.ldup = ldup;
        a.M = (int)M;
        a.N = (int)N;
        a.K = (int)round8(K);
        a.act = act;
        a.groups = 1;
        a.xcd_shift = di.xcd_shift;
        if (M == 1 && K <= lin::kGemvMaxK) return launched(lin::launch_gated_gemv(elem, a, (hipStream_t)stream));
        const int c = choose_gated(M, N, a.K, di.cus);
        const lin::GemmConfig& g = lin::kGatedConfigs[c];
        a.tiles_m = (int)tiles_of(M, g.bm);
        a.tiles_n = (int)tiles_of(2 * N, g.bn);
        return launched(lin::launch_gated_stream(elem, c, a, (hipStream_t)stream));
    }
    lin::ProductArgs p = product(x, ldx, wg, ldwg, h, ldh, M, N, K);
    p.segs = 2;
    p.b[1] = wu;
    p.ldb[1] = ldwu;
    p.gate = gate;
    p.ldgate = ldgate;
    p.up = up;
    p.ldup = ldup;
    p.act = act;
    return launched(lin::launch_product_any(elem, lin::kProdGated, false, p, (hipStream_t)stream));
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
constexpr TileTime kGradTimes[lin::kNumGradConfigs] = {{10.2, 1.50, 1}, {7.0, 0.83, 1}, {4.1, 0.50, 1},
                                                       {2.8, 0.365, 2}, {3.4, 0.20, 1}, {5.7, 0.92, 2}};
constexpr int kPlanCus = 256;      // plans (and so workspaces) do not depend on the device
constexpr double kLaunchGap = 4.0;

double tile_time(int cfg, int64_t groups, int64_t R, int64_t C, int64_t slices, int64_t splits) {
    const lin::GradConfig& g = lin::kGradConfigs[cfg];
    const double main = rounds_time(kGradTimes[cfg], splits * groups * tiles_of(R, g.bm) * tiles_of(C, g.bn),
                                    tiles_of(slices, splits), kPlanCus);
    return splits == 1 ? main : main + 3.5 + 0.65e-6 * 4.0 * (double)splits * (double)groups * (double)R * (double)C;
}

// only64: one launch of a 64-row tile.
StreamPlan plan_stream(int64_t groups, int64_t R, int64_t C, int64_t slices, bool only64 = false) {
    StreamPlan p{only64 ? lin::kPairSmall : 0, 1, 0, 0, 0.0};
    double best = tile_time(p.cfg, groups, R, C, slices, 1);
    for (int c = 0; c < lin::kNumGradConfigs; ++c) {
        if (only64 && lin::kGradConfigs[c].bm != 64) continue;
        for (int64_t s = 1; s <= 16 && (s == 1 || 2 * s <= slices); ++s) {
            // the large tiles fill the chip where splitting pays, and past twice the chip's
            // tiles a split only adds traffic
            if (s > 1 && (lin::kGradConfigs[c].bm == 256 || lin::kGradConfigs[c].stages == 2)) break;
            if (s > 1 && s * groups * tiles_of(R, lin::kGradConfigs[c].bm) * tiles_of(C, lin::kGradConfigs[c].bn) >
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
    const lin::GradConfig& g = lin::kGradConfigs[0];
    const int64_t rows = groups * tiles_of(R, g.bm), cols = tiles_of(C, g.bn);
    const int64_t whole = rows > 0 ? rows * cols / kPlanCus * kPlanCus / rows : 0;   // column tiles in whole rounds
    if (!only64 && whole > 0 && whole < cols) {
        const double head = tile_time(0, groups, R, whole * g.bn, slices, 1) + kLaunchGap;
        for (int c = 0; c < lin::kNumGradConfigs; ++c) {
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
bool sums_fit(int64_t groups, int64_t R, int64_t C, int64_t slices, int cus) {
    const StreamPlan p = plan_stream(groups, R, C, slices);
    const lin::GradConfig& g = lin::kGradConfigs[p.cfg];
    if (g.bm != 64 || p.splits != 1 || p.c1 != 0) return false;
    return groups * tiles_of(R, g.bm) * tiles_of(C, g.bn) + tiles_of(R, 64) <= (int64_t)cus * kGradTimes[p.cfg].per_cu;
}

// Bytes of partial sums of a product's plan.
int64_t partial_bytes(const StreamPlan& p, int64_t groups, int64_t R, int64_t C) {
    return p.splits > 1 ? p.splits * groups * R * ((C + 7) / 8 * 8) * 4 : 0;
}
int64_t partial_bytes(int64_t groups, int64_t R, int64_t C, int64_t slices) {
    return partial_bytes(plan_stream(groups, R, C, slices), groups, R, C);
}

int64_t slices_of(int64_t L) { return (L + 63) / 64; }

// A product's tiles under a plan.
void set_tiles(lin::StreamProduct& a, const StreamPlan& p, const DevInfo& di) {
    const lin::GradConfig& g = lin::kGradConfigs[p.cfg];
    a.tiles_r = (int)tiles_of(a.R, g.bm);
    a.tiles_c = (int)tiles_of(a.C, g.bn);
    a.xcd_shift = di.xcd_shift;
    a.splits = p.splits;
}

// A streaming product's launches under its plan; the operands are set by the caller.
// partial: device memory of the plan's partial sums.
int32_t launch_stream(int elem, bool rowt, int mode, lin::StreamProduct& a, const StreamPlan& p, const DevInfo& di,
                      void* partial, hipStream_t stream) {
    const lin::GradConfig& g = lin::kGradConfigs[p.cfg];
    const int64_t eb = mode == lin::kOutRound ? 2 : 4;
    set_tiles(a, p, di);
    if (p.c1 > 0) {
        lin::StreamProduct head = a;
        head.C = (int)p.c1;
        head.tiles_c = (int)(p.c1 / g.bn);
        const int32_t st = launched(lin::launch_grad_stream(elem, p.cfg, rowt, mode, head, stream));
        if (st != LINEAR_OK) return st;
        const lin::GradConfig& g1 = lin::kGradConfigs[p.cfg1];
        a.C -= (int)p.c1;
        a.tiles_r = (int)tiles_of(a.R, g1.bm);
        a.tiles_c = (int)tiles_of(a.C, g1.bn);
        for (int i = 0; i < 2; ++i) {
            if (a.c[i]) a.c[i] += p.c1;
            if (a.y[i]) a.y[i] = (char*)a.y[i] + p.c1 * eb;
        }
        return launched(lin::launch_grad_stream(elem, p.cfg1, rowt, mode, a, stream));
    }
    if (p.splits == 1) return launched(lin::launch_grad_stream(elem, p.cfg, rowt, mode, a, stream));
    a.partial = (float*)partial;
    a.ldp = ((int64_t)a.C + 7) / 8 * 8;
    a.accumulate = mode == lin::kOutF32Add;
    const int32_t st = launched(lin::launch_grad_stream(elem, p.cfg, rowt, lin::kOutF32, a, stream));
    if (st != LINEAR_OK) return st;
    if (a.fold) a.R = a.fold;
    return launched(lin::launch_split_sum(elem, mode != lin::kOutRound, a, stream));
}


// dx [M, K] = dy [M, N] . weight [N, K].
int32_t run_backward_input(int elem, const uint16_t* dy, int64_t lddy, const uint16_t* w, int64_t ldw, uint16_t* dx,
                           int64_t lddx, int64_t M, int64_t N, int64_t K, void* ws, int64_t ws_bytes, void* stream) {
    if (!dims_ok(M, N, K)) return LINEAR_E_SHAPE;
    if (M == 0 || K == 0) return LINEAR_OK;
    if (!dx) return LINEAR_E_NULL;
    const int64_t need = linear_backward_workspace_bytes(M, N, K);
    if (need < 0) return LINEAR_E_SHAPE;
    const Operand in[] = {{dy, M, lddy, N}, {w, N, ldw, K}};
    const Operand out[] = {{dx, M, lddx, K}, {ws, 1, need, need, 1}};
    int32_t st = check_operands(in, out);
    if (st != LINEAR_OK) return st;
    st = check_workspace(ws, ws_bytes, need);
    if (st != LINEAR_OK) return st;
    if (!any_grid_ok(M, K)) return LINEAR_E_SHAPE;
    int dev = 0;
    DevInfo di;
    st = lin::check_device(&dev, &di);
    if (st != LINEAR_OK) return st;
    unsigned char* space = (unsigned char*)ws + round256(partial_bytes(1, M, K, slices_of(N)));
    if ((st = pack_operand(dy, lddy, M, N, true, space, stream)) != LINEAR_OK) return st;
    if ((st = pack_operand(w, ldw, N, K, false, space, stream)) != LINEAR_OK) return st;
    if (streamable(dy, lddy) && streamable(w, ldw)) {
        lin::StreamProduct a;
        memset(&a, 0, sizeof a);
        a.r = dy;
        a.ldr = lddy;
        a.c[0] = w;
        a.ldc = ldw;
        a.y[0] = dx;
        a.ldy[0] = lddx;
        a.R = (int)M;
        a.C = (int)K;
        a.L = (int)N;
        a.segs = a.groups = 1;
        return launch_stream(elem, false, lin::kOutRound, a, plan_stream(1, M, K, slices_of(N)), di, ws, (hipStream_t)stream);
    }
    const lin::ProductArgs p = product(dy, lddy, w, ldw, dx, lddx, M, K, N);
    return launched(lin::launch_product_any(elem, lin::kProdRound, false, p, (hipStream_t)stream));
}

// The weight call's partial sums: db's and dw's, one after the other in the same space.
int64_t weight_scratch(int64_t M, int64_t N, int64_t K) {
    const int64_t sums = lin::column_sum_splits(M, N);
    return std::max(sums > 1 ? sums * N * 4 : 0, partial_bytes(1, N, K, slices_of(M)));
}

// dw [N, K] = dy [M, N]^T . x [M, K], db [N] = column sums of dy.
int32_t run_backward_weight(int elem, bool f32, const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx, void* dw,
                            int64_t lddw, void* db, int32_t accumulate, int64_t M, int64_t N, int64_t K, void* ws,
                            int64_t ws_bytes, void* stream) {
    if (!dims_ok(M, N, K)) return LINEAR_E_SHAPE;
    if (N == 0 || (K == 0 && !db)) return LINEAR_OK;
    if (K > 0 && !dw) return LINEAR_E_NULL;
    const int64_t eb = f32 ? 4 : 2;
    const int64_t need = linear_backward_workspace_bytes(M, N, K);
    if (need < 0) return LINEAR_E_SHAPE;
    const Operand in[] = {{dy, M, lddy, N}, {x, M, ldx, K}};
    const Operand out[] = {{dw, N, lddw, K, eb}, {db, 1, N, N, eb}, {ws, 1, need, need, 1}};
    int32_t st = check_operands(in, out);
    if (st != LINEAR_OK) return st;
    st = check_workspace(ws, ws_bytes, need);
    if (st != LINEAR_OK) return st;
    if (!any_grid_ok(N, K)) return LINEAR_E_SHAPE;
    if (M == 0 && f32 && accumulate) return LINEAR_OK;   // adds nothing (and leaves a -0)
    int dev = 0;
    DevInfo di;
    st = lin::check_device(&dev, &di);
    if (st != LINEAR_OK) return st;
    lin::ColumnSumArgs c;
    memset(&c, 0, sizeof c);
    c.partial = (float*)ws;
    c.db = db;
    c.M = (int)M;
    c.N = (int)N;
    c.splits = (int)lin::column_sum_splits(M, N);
    c.f32 = f32;
    c.accumulate = accumulate != 0;
    unsigned char* space = (unsigned char*)ws + round256(weight_scratch(M, N, K));
    if (K > 0) {
        if ((st = pack_operand(dy, lddy, M, N, false, space, stream)) != LINEAR_OK) return st;
        if ((st = pack_operand(x, ldx, M, K, false, space, stream)) != LINEAR_OK) return st;
    }
    const bool streams = K > 0 && streamable(dy, lddy) && streamable(x, ldx);
    c.dy = dy;
    c.lddy = lddy;
    const bool with_sums = db && streams && c.splits == 1 && sums_fit(1, N, K, slices_of(M), di.cus);
    if (db && !with_sums) {
        st = launched(lin::launch_column_sum(elem, c, (hipStream_t)stream));
        if (st != LINEAR_OK) return st;
    }
    if (K == 0) return LINEAR_OK;
    if (streams) {
        lin::StreamProduct a;
        memset(&a, 0, sizeof a);
        a.r = dy;
        a.ldr = lddy;
        a.c[0] = x;
        a.ldc = ldx;
        a.y[0] = dw;
        a.ldy[0] = lddw;
        a.R = (int)N;
        a.C = (int)K;
        a.L = (int)M;
        a.segs = a.groups = 1;
        if (with_sums) {
            a.sum_blocks = (int)tiles_of(N, 64);
            a.sums = c;
        }
        const int mode = !f32 ? lin::kOutRound : accumulate ? lin::kOutF32Add : lin::kOutF32;
        return launch_stream(elem, true, mode, a, plan_stream(1, N, K, slices_of(M)), di, ws, (hipStream_t)stream);
    }
    lin::ProductArgs p = product(dy, lddy, x, ldx, dw, lddw, N, K, M);
    p.accumulate = f32 && accumulate != 0;
    return launched(lin::launch_product_any(elem, f32 ? lin::kProdF32 : lin::kProdRound, true, p, (hipStream_t)stream));
}


// The gated block's dg | du matrix: columns of one half, a whole number of 64-wide slices.
int64_t gated_half(int64_t N) { return (N + 63) / 64 * 64; }

// Up to 32 rows leave half of a 64-row tile, and half of a slice of 64 rows, empty: there
// dg and du are two words each, the second in the empty half, and their rounding costs the
// outputs nothing (whole backward of 16 x 14336 x 4096 bf16 146 us, 141 with one word).  With
// more rows it would double the products; the outputs' errors are then 1.4 times one rounding's.
bool low_words(int64_t M) { return M > 0 && M <= lin::kLowRow; }
int64_t gated_rows(int64_t M) { return low_words(M) ? 2 * lin::kLowRow : M; }

// The plans of the gated block's dx and of dWg, dWu.  pair: both run in one launch, where
// their tiles together, spread over the CUs, take less than two launches.  Whole backward,
// with and without, bf16: 517 x 2720 x 1024 34.1 us, 41.1; 1000 x 1928 x 1296 42.0, 56.9; 2000
// x 4096 x 1024 89, 106 (f16 40.5, 47.3; 49.0, 63.5; 108, 124); 1000 x 11008 x 4096 is large
// enough for two.  The plans depend on
// the sizes alone, so either gradient has the same words with and without the other.
struct GatedPlan {
    StreamPlan dx, dw;
    bool pair;
};

GatedPlan plan_gated(int64_t M, int64_t N, int64_t K) {
    const bool low = low_words(M);
    const int64_t sx = 2 * slices_of(N), sw = slices_of(M);
    GatedPlan p{plan_stream(1, M, K, sx, low), plan_stream(2, N, K, sw), false};
    if (M == 0 || N == 0) return p;
    double best = p.dx.time + p.dw.time + kLaunchGap;
    const lin::GradConfig& gw = lin::kGradConfigs[lin::kPairTile];
    const TileTime& tw = kGradTimes[lin::kPairTile];
    const double wt = tw.fixed + tw.slice * (double)sw;
    const double wsum = wt * 2.0 * (double)(tiles_of(N, gw.bm) * tiles_of(K, gw.bn));
    for (int c : {lin::kPairSmall, lin::kPairTile}) {
        const lin::GradConfig& g = lin::kGradConfigs[c];
        if (low && g.bm != 64) continue;
        const TileTime& t = kGradTimes[c];
        const double xt = t.fixed + t.slice * (double)sx;
        const double xsum = xt * (double)(tiles_of(M, g.bm) * tiles_of(K, g.bn));
        const double all = std::max(std::max(xt, wt), (xsum + wsum) / kPlanCus + 0.5 * wt);
        if (all < best) {
            best = all;
            p.pair = true;
            p.dx = StreamPlan{c, 1, 0, 0, xt};
            p.dw = StreamPlan{lin::kPairTile, 1, 0, 0, wt};
        }
    }
    return p;
}

int64_t gated_partials(int64_t M, int64_t N, int64_t K) {
    const GatedPlan p = plan_gated(M, N, K);
    return std::max(partial_bytes(p.dx, 1, M, K), partial_bytes(p.dw, 2, N, K));
}

int32_t run_gated_backward(int elem, const uint16_t* dh, int64_t lddh, const uint16_t* x, int64_t ldx, const uint16_t* wg,
                           int64_t ldwg, const uint16_t* wu, int64_t ldwu, const uint16_t* gate, int64_t ldgate,
                           const uint16_t* up, int64_t ldup, int32_t act, uint16_t* dx, int64_t lddx, uint16_t* dwg,
                           int64_t lddwg, uint16_t* dwu, int64_t lddwu, int64_t M, int64_t N, int64_t K, void* ws,
                           int64_t ws_bytes, void* stream) {
    if (!dims_ok(M, N, K)) return LINEAR_E_SHAPE;
    if (!lin::is_activation(act)) return LINEAR_E_VALUE;
    if (K == 0 || (M == 0 && N == 0)) return LINEAR_OK;
    if ((dwg == nullptr) != (dwu == nullptr)) return LINEAR_E_NULL;
    const bool want_dx = dx && M > 0, want_dw = dwg && N > 0;
    // (an empty output has no address, like one that is not wanted)
    if (!want_dx && !want_dw) return M == 0 || N == 0 || dx || dwg ? LINEAR_OK : LINEAR_E_NULL;
    const int64_t need = linear_gated_workspace_bytes(M, N, K);
    if (need < 0) return LINEAR_E_SHAPE;
    const Operand in[] = {{dh, M, lddh, N}, {x, M, ldx, want_dw ? K : 0}, {wg, N, ldwg, want_dx ? K : 0},
                          {wu, N, ldwu, want_dx ? K : 0}, {gate, M, ldgate, N}, {up, M, ldup, N}};
    const Operand out[] = {{dx, M, lddx, K}, {dwg, N, lddwg, K}, {dwu, N, lddwu, K}, {ws, 1, need, need, 1}};
    int32_t st = check_operands(in, out);
    if (st != LINEAR_OK) return st;
    st = check_workspace(ws, ws_bytes, need);
    if (st != LINEAR_OK) return st;
    const int64_t Np = gated_half(N);
    if ((want_dx && !any_grid_ok(M, K)) || (want_dw && !any_grid_ok(N, K))) return LINEAR_E_SHAPE;
    int dev = 0;
    DevInfo di;
    st = lin::check_device(&dev, &di);
    if (st != LINEAR_OK) return st;
    uint16_t* d = (uint16_t*)((char*)ws + lin::kGradHead);
    // binary16 words are scaled; the products' sums are then multiplied by the factor's inverse
    float* const head = elem == lin::kF16 && M > 0 && N > 0 ? (float*)ws : nullptr;
    if (M > 0 && N > 0) {
        lin::GatedGradArgs g;
        memset(&g, 0, sizeof g);
        g.head = head;
        g.dh = dh;
        g.gate = gate;
        g.up = up;
        g.lddh = lddh;
        g.ldgate = ldgate;
        g.ldup = ldup;
        g.d = d;
        g.M = (int)M;
        g.N = (int)N;
        g.Np = (int)Np;
        g.act = act;
        g.low = low_words(M);
        st = launched(lin::launch_gated_grad(elem, g, (hipStream_t)stream));
        if (st != LINEAR_OK) return st;
    }
    const bool low = low_words(M);
    uint16_t* partials = d + gated_rows(M) * 2 * Np;
    const uint16_t* dl = d + (int64_t)lin::kLowRow * 2 * Np;
    unsigned char* space = (unsigned char*)partials + round256(gated_partials(M, N, K));
    if (want_dx) {
        if ((st = pack_operand(wg, ldwg, N, K, false, space, stream)) != LINEAR_OK) return st;
        if ((st = pack_operand(wu, ldwu, N, K, false, space, stream)) != LINEAR_OK) return st;
    }
    if (want_dw && (st = pack_operand(x, ldx, M, K, false, space, stream)) != LINEAR_OK) return st;
    // weights of two row strides run the any-layout kernel, as unaligned ones do
    const bool dx_streams = streamable(wg, ldwg) && ldwu == ldwg && al16(wu, ldwu) && 2 * Np <= lin::kMaxLdIn;
    const bool dw_streams = streamable(x, ldx) && 2 * Np <= lin::kMaxLdIn;
    const GatedPlan plan = plan_gated(M, N, K);
    lin::StreamProduct px, pw;
    memset(&px, 0, sizeof px);
    memset(&pw, 0, sizeof pw);
    px.r = d;
    px.ldr = 2 * Np;
    px.c[0] = wg;
    px.c[1] = wu;
    px.ldc = ldwg;
    px.y[0] = dx;
    px.ldy[0] = lddx;
    px.R = (int)(low ? 2 * lin::kLowRow : M);
    px.fold = low ? (int)M : 0;
    px.C = (int)K;
    px.L = (int)N;
    px.segs = 2;
    px.groups = 1;
    px.unscale = pw.unscale = head;
    pw.r = d;
    pw.ldr = 2 * Np;
    pw.rgroup = Np;
    pw.c[0] = x;
    pw.ldc = ldx;
    pw.y[0] = dwg;
    pw.y[1] = dwu;
    pw.ldy[0] = lddwg;
    pw.ldy[1] = lddwu;
    pw.R = (int)N;
    pw.C = (int)K;
    pw.L = (int)(low ? 2 * lin::kLowRow : M);
    pw.fold = px.fold;
    pw.segs = 1;
    pw.groups = 2;
    if (want_dx && want_dw && dx_streams && dw_streams && plan.pair) {
        set_tiles(px, plan.dx, di);
        set_tiles(pw, plan.dw, di);
        return launched(lin::launch_grad_pair(elem, plan.dx.cfg == lin::kPairSmall, px, pw, (hipStream_t)stream));
    }
    if (want_dx && dx_streams) {
        st = launch_stream(elem, false, lin::kOutRound, px, plan.dx, di, partials, (hipStream_t)stream);
        if (st != LINEAR_OK) return st;
    } else if (want_dx) {
        lin::ProductArgs p = product(d, 2 * Np, wg, ldwg, dx, lddx, M, K, N);
        p.segs = low ? 4 : 2;
        p.finite_from = low ? 2 : 0;                  // the second words'
        p.unscale = head;
        for (int s = 0; s < p.segs; ++s) {
            p.a[s] = (s < 2 ? d : dl) + s % 2 * Np;
            p.b[s] = s % 2 ? wu : wg;
            p.ldb[s] = s % 2 ? ldwu : ldwg;
        }
        st = launched(lin::launch_product_any(elem, lin::kProdRound, false, p, (hipStream_t)stream));
        if (st != LINEAR_OK) return st;
    }
    if (want_dw && dw_streams) {
        return launch_stream(elem, true, lin::kOutRound, pw, plan.dw, di, partials, (hipStream_t)stream);
    } else if (want_dw) {
        for (int s = 0; s < 2; ++s) {
            lin::ProductArgs p = product(d + s * Np, 2 * Np, x, ldx, s ? dwu : dwg, s ? lddwu : lddwg, N, K, M);
            p.unscale = head;
            if (low) {
                p.segs = 2;
                p.finite_from = 1;
                p.a[1] = dl + s * Np;
                p.b[1] = x;
                p.ldb[1] = ldx;
            }
            st = launched(lin::launch_product_any(elem, lin::kProdRound, true, p, (hipStream_t)stream));
            if (st != LINEAR_OK) return st;
        }
    }
    return LINEAR_OK;
}

// ---------------------------------------------------------------------------
// Gradient norm and clipping

int64_t type_bytes(int64_t type) { return type == LINEAR_TYPE_F32 ? 4 : 2; }

int32_t check_tensor(const linear_tensor& t) {
    if (t.type != LINEAR_TYPE_F16 && t.type != LINEAR_TYPE_BF16 && t.type != LINEAR_TYPE_F32) return LINEAR_E_VALUE;
    if (t.rows < 0 || t.cols < 0 || t.rows > kMaxDim || t.cols > (int64_t(1) << 46)) return LINEAR_E_SHAPE;
    if (t.rows == 0 || t.cols == 0) return LINEAR_OK;
    if (!t.data) return LINEAR_E_NULL;
    if (t.rows > 1 && (t.ld < t.cols || t.ld > kMaxLdOut || (t.rows - 1) * t.ld > kMaxElems - t.cols))
        return LINEAR_E_STRIDE;
    return LINEAR_OK;
}

// Tables of up to kGradTensors tensors, empty ones left out; rows without gaps
// between them count as one row.  f(table, chunks) launches each.
template <typename F>
int32_t each_table(const linear_tensor* src, const linear_tensor* dst, int64_t count, F f) {
    lin::GradTable t;
    memset(&t, 0, sizeof t);
    for (int64_t i = 0; i < count; ++i) {
        const linear_tensor& s = src[i];
        if (s.rows > 0 && s.cols > 0) {
            const linear_tensor& d = dst ? dst[i] : s;
            const int k = t.count;
            const bool one = s.rows == 1 || (s.ld == s.cols && d.ld == s.cols);
            const int64_t rows = one ? 1 : s.rows;
            t.src[k] = s.data;
            t.dst[k] = d.data;
            t.cols[k] = one ? s.rows * s.cols : s.cols;
            t.ld[k] = one ? 0 : s.ld;
            t.ldd[k] = one ? 0 : d.ld;
            t.type[k] = (uint8_t)s.type;
            const int64_t eb = type_bytes(s.type);
            t.vec[k] = (uintptr_t)s.data % 16 == 0 && (uintptr_t)d.data % 16 == 0 && t.ld[k] * eb % 16 == 0 &&
                       t.ldd[k] * eb % 16 == 0;
            t.first[k + 1] = t.first[k] + rows * ((t.cols[k] + lin::kGradChunk - 1) / lin::kGradChunk);
            t.count = k + 1;
        }
        if (t.count == lin::kGradTensors || (i + 1 == count && t.count > 0)) {
            const int32_t st = f(t, (int)std::min<int64_t>(t.first[t.count], lin::kGradGrid));
            if (st != LINEAR_OK) return st;
            t.count = 0;
        }
    }
    return LINEAR_OK;
}

struct Range {
    Extent e;
    bool out;
};

}  // namespace

extern "C" {

int64_t linear_gated_forward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!dims_ok(M, N, K) || !pack_ok(M, K) || !pack_ok(N, K)) return -1;
    // a few rows read their weights once, in place
    return M <= lin::kAnyRows ? 0 : packed_bytes(M, K) + 2 * packed_bytes(N, K);
}

int64_t linear_gated_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!dims_ok(M, N, K) || 2 * gated_half(N) > kMaxLdOut) return -1;   // dg | du in one row
    if (!pack_ok(M, gated_half(N)) || !pack_ok(M, K) || !pack_ok(N, K)) return -1;
    const int64_t partials = gated_partials(M, N, K), packed = 2 * packed_bytes(N, K) + packed_bytes(M, K);
    return lin::kGradHead + gated_rows(M) * gated_half(N) * 2 * 2 + (packed ? round256(partials) + packed : partials);
}

int32_t linear_gated_backward_plan(int64_t M, int64_t N, int64_t K, linear_gated_plan* plan) {
    if (linear_gated_workspace_bytes(M, N, K) < 0) return LINEAR_E_SHAPE;
    if (!plan) return LINEAR_E_NULL;
    memset(plan, 0, sizeof *plan);
    const GatedPlan p = plan_gated(M, N, K);
    auto fill = [](linear_product_plan& out, const StreamPlan& s) {
        const lin::GradConfig &g = lin::kGradConfigs[s.cfg], &g1 = lin::kGradConfigs[s.cfg1];
        out.tile_m = g.bm;
        out.tile_n = g.bn;
        out.stages = g.stages;
        out.sets = g.sets;
        out.splits = s.splits;
        out.split_c = s.c1;
        if (s.c1 > 0) {
            out.tile_m2 = g1.bm;
            out.tile_n2 = g1.bn;
        }
    };
    fill(plan->dx, p.dx);
    fill(plan->dw, p.dw);
    plan->joint = p.pair;
    plan->two_words = low_words(M);
    return LINEAR_OK;
}

int64_t linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!dims_ok(M, N, K) || !pack_ok(M, N) || !pack_ok(M, K) || !pack_ok(N, K)) return -1;
    const int64_t in = partial_bytes(1, M, K, slices_of(N)), in_packed = packed_bytes(M, N) + packed_bytes(N, K);
    const int64_t wt = weight_scratch(M, N, K), wt_packed = packed_bytes(M, N) + packed_bytes(M, K);
    return std::max(in_packed ? round256(in) + in_packed : in, wt_packed ? round256(wt) + wt_packed : wt);
}

int32_t linear_f16_gated(const uint16_t* x, int64_t ldx, const uint16_t* wg, int64_t ldwg, const uint16_t* wu,
                         int64_t ldwu, int32_t act, uint16_t* h, int64_t ldh, uint16_t* gate, int64_t ldgate, uint16_t* up,
                         int64_t ldup, int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                         void* stream) {
    return run_gated(lin::kF16, x, ldx, wg, ldwg, wu, ldwu, act, h, ldh, gate, ldgate, up, ldup, M, N, K, workspace,
                     workspace_bytes, stream);
}

int32_t linear_bf16_gated(const uint16_t* x, int64_t ldx, const uint16_t* wg, int64_t ldwg, const uint16_t* wu,
                          int64_t ldwu, int32_t act, uint16_t* h, int64_t ldh, uint16_t* gate, int64_t ldgate, uint16_t* up,
                          int64_t ldup, int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                          void* stream) {
    return run_gated(lin::kBF16, x, ldx, wg, ldwg, wu, ldwu, act, h, ldh, gate, ldgate, up, ldup, M, N, K, workspace,
                     workspace_bytes, stream);
}

int32_t linear_f16_gated_backward(const uint16_t* dh, int64_t lddh, const uint16_t* x, int64_t ldx, const uint16_t* wg,
                                  int64_t ldwg, const uint16_t* wu, int64_t ldwu, const uint16_t* gate, int64_t ldgate,
                                  const uint16_t* up, int64_t ldup, int32_t act, uint16_t* dx, int64_t lddx, uint16_t* dwg,
                                  int64_t lddwg, uint16_t* dwu, int64_t lddwu, int64_t M, int64_t N, int64_t K,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
    return run_gated_backward(lin::kF16, dh, lddh, x, ldx, wg, ldwg, wu, ldwu, gate, ldgate, up, ldup, act, dx, lddx, dwg,
                              lddwg, dwu, lddwu, M, N, K, workspace, workspace_bytes, stream);
}

int32_t linear_bf16_gated_backward(const uint16_t* dh, int64_t lddh, const uint16_t* x, int64_t ldx, const uint16_t* wg,
                                   int64_t ldwg, const uint16_t* wu, int64_t ldwu, const uint16_t* gate, int64_t ldgate,
                                   const uint16_t* up, int64_t ldup, int32_t act, uint16_t* dx, int64_t lddx, uint16_t* dwg,
                                   int64_t lddwg, uint16_t* dwu, int64_t lddwu, int64_t M, int64_t N, int64_t K,
                                   void* workspace, int64_t workspace_bytes, void* stream) {
    return run_gated_backward(lin::kBF16, dh, lddh, x, ldx, wg, ldwg, wu, ldwu, gate, ldgate, up, ldup, act, dx, lddx, dwg,
                              lddwg, dwu, lddwu, M, N, K, workspace, workspace_bytes, stream);
}

int32_t linear_f16_backward_input(const uint16_t* dy, int64_t lddy, const uint16_t* weight, int64_t ldw, uint16_t* dx,
                                  int64_t lddx, int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                                  void* stream) {
    return run_backward_input(lin::kF16, dy, lddy, weight, ldw, dx, lddx, M, N, K, workspace, workspace_bytes, stream);
}

int32_t linear_bf16_backward_input(const uint16_t* dy, int64_t lddy, const uint16_t* weight, int64_t ldw, uint16_t* dx,
                                   int64_t lddx, int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                                   void* stream) {
    return run_backward_input(lin::kBF16, dy, lddy, weight, ldw, dx, lddx, M, N, K, workspace, workspace_bytes, stream);
}

int32_t linear_f16_backward_weight(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx, uint16_t* dw,
                                   int64_t lddw, uint16_t* db, int64_t M, int64_t N, int64_t K, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
    return run_backward_weight(lin::kF16, false, dy, lddy, x, ldx, dw, lddw, db, 0, M, N, K, workspace, workspace_bytes,
                               stream);
}

int32_t linear_bf16_backward_weight(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx, uint16_t* dw,
                                    int64_t lddw, uint16_t* db, int64_t M, int64_t N, int64_t K, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
    return run_backward_weight(lin::kBF16, false, dy, lddy, x, ldx, dw, lddw, db, 0, M, N, K, workspace, workspace_bytes,
                               stream);
}

int32_t linear_f16_backward_weight_f32out(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx, float* dw,
                                          int64_t lddw, float* db, int32_t accumulate, int64_t M, int64_t N, int64_t K,
                                          void* workspace, int64_t workspace_bytes, void* stream) {
    return run_backward_weight(lin::kF16, true, dy, lddy, x, ldx, dw, lddw, db, accumulate, M, N, K, workspace,
                               workspace_bytes, stream);
}

int32_t linear_bf16_backward_weight_f32out(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx, float* dw,
                                           int64_t lddw, float* db, int32_t accumulate, int64_t M, int64_t N, int64_t K,
                                           void* workspace, int64_t workspace_bytes, void* stream) {
    return run_backward_weight(lin::kBF16, true, dy, lddy, x, ldx, dw, lddw, db, accumulate, M, N, K, workspace,
                               workspace_bytes, stream);
}

int64_t linear_grad_workspace_bytes(int64_t count) {
    if (count < 0 || count > LINEAR_GRAD_MAX_TENSORS) return -1;
    return (count + lin::kGradTensors - 1) / lin::kGradTensors * lin::kGradGrid * 8;
}

int32_t linear_grad_norm(const linear_tensor* grads, int64_t count, float* norm, void* workspace, int64_t workspace_bytes,
                         void* stream) {
    const int64_t need = linear_grad_workspace_bytes(count);
    if (need < 0) return LINEAR_E_SHAPE;
    if (!norm || (count > 0 && !grads)) return LINEAR_E_NULL;
    int32_t st;
    const Extent en = extent(norm, 1, 1, 1, 4), ew = extent(workspace, 1, need, need, 1);
    for (int64_t i = 0; i < count; ++i)
        if ((st = check_tensor(grads[i])) != LINEAR_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != LINEAR_OK) return st;
    if (overlaps(en, ew)) return LINEAR_E_ALIAS;
    for (int64_t i = 0; i < count; ++i) {
        const linear_tensor& t = grads[i];
        const Extent e = extent(t.data, t.rows, t.ld, t.cols, type_bytes(t.type));
        if (overlaps(e, en) || overlaps(e, ew)) return LINEAR_E_ALIAS;
    }
    int dev = 0;
    if ((st = lin::check_device(&dev)) != LINEAR_OK) return st;
    double* partial = (double*)workspace;
    int used = 0;
    st = each_table(grads, nullptr, count, [&](const lin::GradTable& t, int grid) {
        const int32_t r = launched(lin::launch_grad_partials(t, partial + used, grid, (hipStream_t)stream));
        used += grid;
        return r;
    });
    if (st != LINEAR_OK) return st;
    return launched(lin::launch_grad_norm(partial, used, norm, (hipStream_t)stream));
}

int32_t linear_grad_clip(const linear_tensor* grads, const linear_tensor* out, int64_t count, const float* norm,
                         float max_norm, void* stream) {
    if (count < 0 || count > LINEAR_GRAD_MAX_TENSORS) return LINEAR_E_SHAPE;
    if (isnan(max_norm) || max_norm < 0.f) return LINEAR_E_VALUE;
    if (count == 0) return LINEAR_OK;
    if (!grads || !norm) return LINEAR_E_NULL;
    int32_t st;
    for (int64_t i = 0; i < count; ++i) {
        if ((st = check_tensor(grads[i])) != LINEAR_OK) return st;
        if (!out) continue;
        if ((st = check_tensor(out[i])) != LINEAR_OK) return st;
        if (out[i].type != grads[i].type) return LINEAR_E_VALUE;
        if (out[i].rows != grads[i].rows || out[i].cols != grads[i].cols) return LINEAR_E_SHAPE;
    }
    // every output must be apart from every other tensor and from the norm, but a
    // tensor may be its own output: sorted by address, an output may not begin
    // before an earlier range ends, nor an input before an earlier output ends
    std::unique_ptr<Range[]> ranges(new (std::nothrow) Range[2 * count + 1]);
    if (!ranges) return LINEAR_E_MEMORY;
    int64_t n = 0;
    ranges[n++] = {extent(norm, 1, 1, 1, 4), false};
    for (int64_t i = 0; i < count; ++i) {
        const linear_tensor &s = grads[i], &d = out ? out[i] : grads[i];
        if (s.rows == 0 || s.cols == 0) continue;
        const int64_t eb = type_bytes(s.type);
        ranges[n++] = {extent(d.data, d.rows, d.ld, d.cols, eb), true};
        const bool in_place = d.data == s.data && (d.rows == 1 || d.ld == s.ld);
        if (!in_place) ranges[n++] = {extent(s.data, s.rows, s.ld, s.cols, eb), false};
    }
    std::sort(ranges.get(), ranges.get() + n, [](const Range& a, const Range& b) { return a.e.lo < b.e.lo; });
    uintptr_t all = 0, outs = 0;
    for (int64_t i = 0; i < n; ++i) {
        const Range& r = ranges[i];
        if (r.e.lo < (r.out ? all : outs)) return LINEAR_E_ALIAS;
        all = std::max(all, r.e.hi);
        if (r.out) outs = std::max(outs, r.e.hi);
    }
    int dev = 0;
    if ((st = lin::check_device(&dev)) != LINEAR_OK) return st;
    return each_table(grads, out, count, [&](const lin::GradTable& t, int grid) {
        return launched(lin::launch_grad_clip(t, norm, max_norm, grid, (hipStream_t)stream));
    });
}

}  // extern "C"
