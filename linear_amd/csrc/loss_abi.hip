// loss_abi.hip -- the C ABI of the linear head's cross entropy: argument checks, the plan of
// the vocabulary's pieces, launches.  The conventions are linear_abi.hip's: every check runs
// on the host before anything is enqueued, and only kernels are enqueued.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "../../include/linear_amd.h"
#include "abi.h"
#include "loss.h"
#include "train.h"
#include "train_host.h"

namespace {

using namespace lin;

constexpr int64_t kMaxLossRows = int64_t(1) << 24;
constexpr int64_t kMaxLossK = kMaxLdIn / 8 * 8;       // rows that the streaming kernels read
static_assert(kMaxLossK == LINEAR_CROSS_ENTROPY_MAX_K && kMaxLossRows == LINEAR_CROSS_ENTROPY_MAX_M, "limits");

bool loss_dims_ok(int64_t M, int64_t N, int64_t K) {
    return M >= 0 && N >= 0 && K >= 0 && M <= kMaxLossRows && N <= kMaxSize && K <= kMaxLossK;
}

// kLossConfigs' times, near those measured and set so that the choice is the fastest of the five tiles, or
// close to it, at M from 1 to 2000, N from 8000 to 128259, K of 768 and 4096.  Measured beside those, with every
// tile (bf16 loss; M of 1, 16, 48, 100, 200, 400, 700, 1500, N of 16000 and 50000, K of 384, 1536, 2048, 2560, 6144):
// 76 of the 80 within 4% of the fastest, the others 6 to 14% (700 x 16000 x 6144 172 us, 151 on 256 x 256).
constexpr TileTime kLossTimes[kNumLossConfigs] = {{6.5, 1.60, 1}, {5.3, 0.80, 1}, {4.9, 0.50, 1}, {2.0, 0.42, 2}, {2.0, 0.30, 3}};

// The tile of a product of M rows and N columns (by sizes alone: workspaces depend on it).
int choose_loss(int64_t M, int64_t N, int64_t K) {
    int best = 0;
    double best_time = -1.0;
    for (int c = 0; c < kNumLossConfigs; ++c) {
        const GemmConfig& g = kLossConfigs[c];
        const double t = rounds_time(kLossTimes[c], tiles_of(M, g.bm) * tiles_of(N, g.bn), tiles_of(K, 64), kPlanCus);
        if (best_time < 0 || t < best_time) {
            best_time = t;
            best = c;
        }
    }
    return best;
}

// Rows of the weight that are copied at a time where the streaming kernels cannot read them
// in place: 256 MiB of copies, whole tiles (bf16 loss and gradients of 170 x 30000 x 4001 741 us with
// 64 MiB, 536 with 256; of 312 x 106631 x 3204 2163, 2146, and 2041 with 1 GiB).
int64_t pack_rows(int64_t N, int64_t K) {
    const int64_t rows = std::max<int64_t>((int64_t(128) << 20) / std::max<int64_t>(round8(K), 1) / 256 * 256, 256);
    return std::min(rows, N);
}

// What both calls keep at the end of their workspace: copies of x and, behind it, of a piece of the
// weight, for layouts that the streaming kernels cannot read.  (Calls that read the weight in place need,
// and may be given, the workspace without them.)
int64_t copies_bytes(int64_t M, int64_t N, int64_t K) {
    return round256(M * round8(K) * 2) + round256(pack_rows(N, K) * round8(K) * 2);
}

struct Copies {
    uint16_t *x, *w;
};
Copies copies_at(unsigned char* space, int64_t M, int64_t K) {
    return {(uint16_t*)space, (uint16_t*)(space + round256(M * round8(K) * 2))};
}

bool in_place(const uint16_t* p, int64_t ld, int64_t rows, int64_t K) {
    return K == 0 || (K % 8 == 0 && (rows <= 1 ? (uintptr_t)p % 16 == 0 : streamable(p, ld)));
}

// A row stride that is never used may be anything: the kernels get a readable one.
int64_t row_stride(int64_t ld, int64_t rows, int64_t K) { return rows <= 1 ? round8(K) : ld; }

// Columns of one launch: its threads are counted in 32 bits.
int64_t launch_columns(int64_t M, const GemmConfig& g) {
    const int64_t tiles = ((int64_t(1) << 32) - 1) / (g.wm * g.wn * 64) / tiles_of(std::max<int64_t>(M, 1), g.bm);
    return std::min(tiles * g.bn, kColumnPart);
}

LossArgs loss_args(const uint16_t* x, int64_t ldx, const int64_t* target, int64_t M, int64_t N, int64_t K, const DevInfo& di) {
    LossArgs a;
    memset(&a, 0, sizeof a);
    a.x = x;
    a.ldx = ldx;
    a.target = target;
    a.cols = N;
    a.M = (int)M;
    a.K = (int)round8(K);
    a.groups = 1;
    a.xcd_shift = di.xcd_shift;
    return a;
}

int32_t launch_piece(int elem, int cfg, int mode, LossArgs a, const uint16_t* w, int64_t ldw, const uint16_t* b, int64_t col,
                     int64_t n, hipStream_t stream) {
    const GemmConfig& g = kLossConfigs[cfg];
    a.w = w;
    a.ldw = ldw;
    a.b = b ? b + col : nullptr;
    a.col0 = col;
    a.N = (int)n;
    a.tiles_m = (int)tiles_of(a.M, g.bm);
    a.tiles_n = (int)tiles_of(n, g.bn);
    return launched(launch_loss_stream(elem, cfg, mode, a, stream));
}

// Bytes of the forward call's row statistics and logits at the targets.
int64_t parts_bytes(int64_t M, int64_t N, int64_t K) {
    return round256(M * tiles_of(N, kLossConfigs[choose_loss(M, N, K)].bn) * (int64_t)sizeof(RowPart));
}

int32_t run_loss(int elem, const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw, const uint16_t* b,
                 const int64_t* target, float* loss, float* lse, int64_t M, int64_t N, int64_t K, void* ws, int64_t ws_bytes,
                 hipStream_t stream) {
    if (!loss_dims_ok(M, N, K)) return LINEAR_E_SHAPE;
    if (M == 0) return LINEAR_OK;
    if (!target || (!loss && !lse)) return LINEAR_E_NULL;
    const bool packed = !in_place(w, ldw, N, K), aligned = !packed && in_place(x, ldx, M, K);
    const int64_t need = aligned ? linear_cross_entropy_workspace_bytes_aligned(M, N, K) : linear_cross_entropy_workspace_bytes(M, N, K);
    const Operand in[] = {{x, M, ldx, K}, {w, N, ldw, K}, {b, b ? 1 : 0, N, N}, {target, 1, M, M, 8}};
    const Operand out[] = {{loss, 1, M, M, 4}, {lse, 1, M, M, 4}, {ws, 1, need, need, 1}};
    int32_t st = check_operands(in, out);
    if (st != LINEAR_OK) return st;
    if ((st = check_workspace(ws, ws_bytes, need)) != LINEAR_OK) return st;
    int dev = 0;
    DevInfo di;
    if ((st = check_device(&dev, &di)) != LINEAR_OK) return st;
    const int cfg = choose_loss(M, N, K);
    const GemmConfig& g = kLossConfigs[cfg];
    RowPart* parts = (RowPart*)ws;
    float* at_target = (float*)((unsigned char*)ws + parts_bytes(M, N, K));
    const Copies copies = copies_at((unsigned char*)at_target + round256(M * 4), M, K);
    if (!in_place(x, ldx, M, K)) {
        if ((st = launched(launch_repack(x, ldx, M, (int)K, copies.x, round8(K), stream))) != LINEAR_OK) return st;
        x = copies.x;
        ldx = round8(K);
    }
    LossArgs a = loss_args(x, row_stride(ldx, M, K), target, M, N, K, di);
    a.ldparts = tiles_of(N, g.bn);
    a.at_target = at_target;
    int64_t step = launch_columns(M, g);
    if (packed) step = std::min(step, pack_rows(N, K));
    for (int64_t n = 0; n < N; n += step) {          // (whole tiles, but for the last)
        const int64_t cols = std::min(N - n, step);
        if (packed && (st = launched(launch_repack(w + n * ldw, ldw, cols, (int)K, copies.w, round8(K), stream))) != LINEAR_OK)
            return st;
        a.parts = parts + n / g.bn;
        st = launch_piece(elem, cfg, kOutLse, a, packed ? copies.w : w + n * ldw, packed ? round8(K) : row_stride(ldw, N, K), b, n,
                          cols, stream);
        if (st != LINEAR_OK) return st;
    }
    const LossJoinArgs j{parts, a.ldparts, a.ldparts, at_target, target, N, M, lse, loss};
    return launched(launch_loss_join(j, stream));
}

// The gradient call's plan.  The vocabulary is taken in pieces of `cols` columns (whole
// tiles): dz of one piece is formed, multiplied into dx (FP32 sums over the pieces) and into
// its rows of dw.  One piece where dz is at most 256 MiB; else pieces of 128 MiB (they stay in
// the memory-side cache until both products have read them), of 8192 columns at least.
// Both products in one launch where that is faster (plan_pair), with db's column sums.
struct LossPlan {
    int64_t pieces, cols, ldz;
    StreamPlan dx, dw;
    bool pair;
    bool outer;                                       // dw by launch_outer, where its layout allows
};
// From how many values of dw on launch_outer is the faster, for up to 128 rows and up to 256 (bf16
// loss and gradients of 256 x 32000 x 4096 361 -> 324 us, 256 x 16000 x 2048 117 -> 107, 160 x 60000 x 520
// 131 -> 125; under the limit 256 x 5000 x 1000 55 -> 59).
constexpr int64_t kOuterValues = int64_t(1) << 20, kOuterLong = int64_t(1) << 24;
LossPlan plan_loss(int64_t M, int64_t N, int64_t K, bool packed) {
    LossPlan p;
    int64_t most = std::max<int64_t>(N, 1);
    const int64_t rows = std::max<int64_t>(M, 1);
    if (rows * most > int64_t(1) << 27) most = std::max<int64_t>((int64_t(1) << 26) / rows, 8192);
    if (packed) most = std::min(most, std::max<int64_t>(pack_rows(N, K), 1));
    most = std::min(most, kMaxLdIn / 256 * 256);      // a stride that the products' kernels read
    p.pieces = std::max<int64_t>(tiles_of(N, most), 1);
    p.cols = p.pieces == 1 ? N : std::min(tiles_of(tiles_of(N, p.pieces), 256) * 256, N);
    p.pieces = std::max<int64_t>(p.cols ? tiles_of(N, p.cols) : 1, 1);
    p.ldz = (p.cols + 63) / 64 * 64;
    p.dx = plan_stream(1, M, K, slices_of(p.cols), false, true);
    p.dw = plan_stream(1, p.cols, K, slices_of(M));
    p.outer = M <= 128 ? N * K >= kOuterValues : M <= kOuterL && N * K >= kOuterLong;
    p.pair = !p.outer && p.pieces == 1 && M > 0 && N > 0 && K > 0 &&
             plan_pair(p.dx, p.dw, p.dx.time + p.dw.time + kLaunchGap, M, K, slices_of(N), 1, N, slices_of(M), false);
    return p;
}

constexpr int64_t kLossHead = 256;                    // the factor and its inverse, the number of rows
int64_t sums_bytes(int64_t M, int64_t cols) { return M > 2048 ? round256(64 * cols * 4) : 0; }

// Bytes ahead of the copies: the head, the rows' places, list and terms, dz, dx's FP32 sums, the
// products' partial sums.
struct LossSpace {
    int64_t place, list, terms, dz, dx, partials, end;
};
LossSpace space_of(const LossPlan& p, int64_t M, int64_t K) {
    LossSpace s;
    s.place = kLossHead;
    s.list = s.place + round256(M * 4);
    s.terms = s.list + round256(M * 4);
    s.dz = s.terms + round256(M * (int64_t)sizeof(RowTerms));
    s.dx = s.dz + round256(M * p.ldz * 2);
    s.partials = s.dx + (p.pieces > 1 ? round256(M * round8(K) * 4) : 0);
    s.end = s.partials + round256(std::max({partial_bytes(p.dx, 1, M, K), partial_bytes(p.dw, 1, p.cols, K), sums_bytes(M, p.cols)}));
    return s;
}

int32_t run_loss_backward(int elem, bool f32, const float* dloss, const float* dlse, const uint16_t* x, int64_t ldx,
                          const uint16_t* w, int64_t ldw, const uint16_t* b, const int64_t* target, const float* lse,
                          uint16_t* dx, int64_t lddx, void* dw, int64_t lddw, void* db, int32_t accumulate, int64_t M, int64_t N,
                          int64_t K, void* ws, int64_t ws_bytes, hipStream_t stream) {
    if (!loss_dims_ok(M, N, K)) return LINEAR_E_SHAPE;
    if (M == 0 && N == 0) return LINEAR_OK;
    const bool want_dx = dx && M > 0 && K > 0, want_dw = dw && N > 0 && K > 0, want_db = db && N > 0;
    // (an empty output has no address, like one that is not wanted)
    if (!want_dx && !want_dw && !want_db) return M == 0 || N == 0 || K == 0 || dx || dw ? LINEAR_OK : LINEAR_E_NULL;
    const bool packed = !in_place(w, ldw, N, K);
    const int64_t need = packed ? linear_cross_entropy_backward_workspace_bytes(M, N, K)
                                : linear_cross_entropy_backward_workspace_bytes_aligned(M, N, K);
    const int64_t eb = f32 ? 4 : 2;
    const Operand in[] = {{x, M, ldx, N > 0 ? K : 0}, {w, M > 0 ? N : 0, ldw, K}, {b, b ? 1 : 0, N, N}, {target, 1, M, M, 8},
                          {lse, 1, M, M, 4}, {dloss, 1, M, M, 4}, {dlse, dlse ? 1 : 0, M, M, 4}};
    const Operand out[] = {{dx, M, lddx, K}, {dw, N, lddw, K, eb}, {db, 1, N, N, eb}, {ws, 1, need, need, 1}};
    int32_t st = check_operands(in, out);
    if (st != LINEAR_OK) return st;
    if ((st = check_workspace(ws, ws_bytes, need)) != LINEAR_OK) return st;
    if (M == 0 && f32 && accumulate) return LINEAR_OK;   // adds nothing (and leaves a -0)
    int dev = 0;
    DevInfo di;
    if ((st = check_device(&dev, &di)) != LINEAR_OK) return st;
    const LossPlan p = plan_loss(M, N, K, packed);
    const LossSpace at = space_of(p, M, K);
    unsigned char* space = (unsigned char*)ws;
    const bool any = M > 0 && N > 0;
    // dz is scaled; the products' sums are then multiplied by the factor's inverse
    float* const head = any ? (float*)ws : nullptr;
    int32_t* const rows = any ? (int32_t*)ws + 2 : nullptr;
    int32_t *place = (int32_t*)(space + at.place), *list = any ? (int32_t*)(space + at.list) : nullptr;
    uint16_t* dz = (uint16_t*)(space + at.dz);
    float* sums = (float*)(space + at.dx);
    void* partials = space + at.partials;
    const Copies copies = copies_at(space + at.end, M, K);
    LossArgs a = loss_args(copies.x, round8(K), target, M, N, K, di);
    if (any) {
        a.terms = (RowTerms*)(space + at.terms);
        a.rows = rows;
        const LossRowsArgs r{target, dloss, dlse, lse, N, M, head, rows, place, list, (RowTerms*)(space + at.terms)};
        const LossGatherArgs g{x, ldx, (int)K, copies.x, round8(K), want_dx ? dx : nullptr, lddx};
        if ((st = launched(launch_loss_rows(r, g, stream))) != LINEAR_OK) return st;
    }
    a.y = dz;
    a.ldy = p.ldz;
    for (int64_t piece = 0; piece < p.pieces; ++piece) {
        const int64_t n = piece * p.cols, cols = std::min(N - n, p.cols);
        const uint16_t* wp = w + n * ldw;
        int64_t ldp = row_stride(ldw, N, K);
        if (packed && M > 0 && cols > 0) {
            if ((st = launched(launch_repack(wp, ldw, cols, (int)K, copies.w, round8(K), stream))) != LINEAR_OK) return st;
            wp = copies.w;
            ldp = round8(K);
        }
        if (M > 0 && cols > 0) {
            const int cfg = choose_loss(M, cols, K);
            const int64_t step = launch_columns(M, kLossConfigs[cfg]);
            for (int64_t c = 0; c < cols; c += step) {
                a.y = dz + c;
                st = launch_piece(elem, cfg, kOutDz, a, wp + c * ldp, ldp, b, n + c, std::min(cols - c, step), stream);
                if (st != LINEAR_OK) return st;
            }
        }
        StreamProduct sx, sw;
        memset(&sx, 0, sizeof sx);
        memset(&sw, 0, sizeof sw);
        sx.r = sw.r = dz;
        sx.ldr = sw.ldr = p.ldz;
        sx.segs = sx.groups = sw.segs = sw.groups = 1;
        sx.rows = sw.rows = rows;
        sx.c[0] = wp;
        sx.ldc = ldp;
        sx.y[0] = p.pieces > 1 ? (void*)sums : (void*)dx;
        sx.ldy[0] = p.pieces > 1 ? round8(K) : lddx;
        sx.R = (int)M;
        sx.C = (int)K;
        sx.L = (int)cols;
        sx.unscale = p.pieces > 1 ? nullptr : head;
        sx.list = p.pieces > 1 ? nullptr : list;
        sw.c[0] = copies.x;
        sw.ldc = round8(K);
        sw.y[0] = (char*)dw + n * lddw * eb;
        sw.ldy[0] = lddw;
        sw.R = (int)cols;
        sw.C = (int)K;
        sw.L = (int)M;
        sw.unscale = head;
        ColumnSumArgs c;
        memset(&c, 0, sizeof c);
        c.dy = dz;
        c.lddy = p.ldz;
        c.partial = (float*)partials;
        c.db = want_db ? (char*)db + n * eb : nullptr;
        c.M = (int)M;
        c.N = (int)cols;
        c.splits = (int)column_sum_splits(M, cols);
        c.f32 = f32;
        c.accumulate = accumulate != 0;
        c.unscale = head;
        c.rows = rows;
        const bool together = p.pair && want_dx && want_dw && !f32 && any;
        const bool outer = want_dw && p.outer && K % 8 == 0 && streamable(dw, lddw) && !(f32 && accumulate);
        const bool with_sums = want_db && want_dw && !outer && c.splits == 1 && (together || sums_fit(p.dw, 1, cols, K, di.cus));
        if (with_sums) {
            sw.sum_blocks = (int)tiles_of(cols, 64);
            sw.sums = c;
        } else if (want_db && (st = launched(launch_column_sum(elem, c, stream))) != LINEAR_OK) {
            return st;
        }
        if (together) {
            set_tiles(sx, p.dx, di);
            set_tiles(sw, p.dw, di);
            return launched(launch_grad_pair(elem, p.dx.cfg == kPairSmall, sx, sw, stream));
        }
        if (want_dx) {
            const int mode = p.pieces > 1 ? (piece == 0 ? kOutF32 : kOutF32Add) : list ? kOutList : kOutRound;
            if ((st = launch_stream(elem, false, mode, sx, p.dx, di, partials, stream)) != LINEAR_OK) return st;
        }
        // dw's words go past the caches, which hold the weight and dz (256 x 32000 x 4096 bf16 loss and
        // gradients: 376 us, 361; 4096 x 128259 x 4096 12.52 ms, 12.41)
        if (outer) {
            sw.xcd_shift = di.xcd_shift;
            if ((st = launched(launch_outer(elem, f32 ? kOutF32 : kOutRound, sw, stream))) != LINEAR_OK) return st;
        } else if (want_dw) {
            const int mode = !f32 ? (any && streamable(dw, lddw) && whole_lines(dw, lddw) ? kOutStream : kOutRound)
                                  : accumulate ? kOutF32Add : kOutF32;
            if ((st = launch_stream(elem, true, mode, sw, p.dw, di, partials, stream)) != LINEAR_OK) return st;
        }
    }
    if (!want_dx || p.pieces == 1) return LINEAR_OK;
    StreamProduct s;                                  // the sums over the pieces, rounded
    memset(&s, 0, sizeof s);
    s.partial = sums;
    s.ldp = round8(K);
    s.y[0] = dx;
    s.ldy[0] = lddx;
    s.R = (int)M;
    s.C = (int)K;
    s.splits = s.groups = 1;
    s.sum_unscale = head;
    s.rows = rows;
    s.list = list;
    return launched(launch_split_sum(elem, false, s, stream));
}

}  // namespace

extern "C" {

int64_t linear_cross_entropy_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!loss_dims_ok(M, N, K)) return -1;
    return parts_bytes(M, N, K) + round256(M * 4) + copies_bytes(M, N, K);
}

int64_t linear_cross_entropy_workspace_bytes_aligned(int64_t M, int64_t N, int64_t K) {
    if (K % 8 != 0 || !loss_dims_ok(M, N, K)) return linear_cross_entropy_workspace_bytes(M, N, K);
    return parts_bytes(M, N, K) + round256(M * 4);
}

int64_t linear_cross_entropy_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!loss_dims_ok(M, N, K)) return -1;
    const int64_t in_place = space_of(plan_loss(M, N, K, false), M, K).end, packed = space_of(plan_loss(M, N, K, true), M, K).end;
    return std::max(in_place, packed) + copies_bytes(M, N, K);
}

int64_t linear_cross_entropy_backward_workspace_bytes_aligned(int64_t M, int64_t N, int64_t K) {
    if (K % 8 != 0 || !loss_dims_ok(M, N, K)) return linear_cross_entropy_backward_workspace_bytes(M, N, K);
    return space_of(plan_loss(M, N, K, false), M, K).end + round256(M * K * 2);   // (x is gathered there in any layout)
}

int32_t linear_f16_cross_entropy(const uint16_t* x, int64_t ldx, const uint16_t* weight, int64_t ldw, const uint16_t* b,
                                 const int64_t* target, float* loss, float* lse, int64_t M, int64_t N, int64_t K,
                                 void* workspace, int64_t workspace_bytes, void* stream) {
    return run_loss(kF16, x, ldx, weight, ldw, b, target, loss, lse, M, N, K, workspace, workspace_bytes, (hipStream_t)stream);
}

int32_t linear_bf16_cross_entropy(const uint16_t* x, int64_t ldx, const uint16_t* weight, int64_t ldw, const uint16_t* b,
                                  const int64_t* target, float* loss, float* lse, int64_t M, int64_t N, int64_t K,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
    return run_loss(kBF16, x, ldx, weight, ldw, b, target, loss, lse, M, N, K, workspace, workspace_bytes, (hipStream_t)stream);
}

int32_t linear_f16_cross_entropy_backward(const float* dloss, const float* dlse, const uint16_t* x, int64_t ldx,
                                          const uint16_t* weight, int64_t ldw, const uint16_t* b, const int64_t* target,
                                          const float* lse, uint16_t* dx, int64_t lddx, uint16_t* dw, int64_t lddw,
                                          uint16_t* db, int64_t M, int64_t N, int64_t K, void* workspace,
                                          int64_t workspace_bytes, void* stream) {
    return run_loss_backward(kF16, false, dloss, dlse, x, ldx, weight, ldw, b, target, lse, dx, lddx, dw, lddw, db, 0, M, N, K,
                             workspace, workspace_bytes, (hipStream_t)stream);
}

int32_t linear_bf16_cross_entropy_backward(const float* dloss, const float* dlse, const uint16_t* x, int64_t ldx,
                                           const uint16_t* weight, int64_t ldw, const uint16_t* b, const int64_t* target,
                                           const float* lse, uint16_t* dx, int64_t lddx, uint16_t* dw, int64_t lddw,
                                           uint16_t* db, int64_t M, int64_t N, int64_t K, void* workspace,
                                           int64_t workspace_bytes, void* stream) {
    return run_loss_backward(kBF16, false, dloss, dlse, x, ldx, weight, ldw, b, target, lse, dx, lddx, dw, lddw, db, 0, M, N, K,
                             workspace, workspace_bytes, (hipStream_t)stream);
}

int32_t linear_f16_cross_entropy_backward_f32out(const float* dloss, const float* dlse, const uint16_t* x, int64_t ldx,
                                                 const uint16_t* weight, int64_t ldw, const uint16_t* b, const int64_t* target,
                                                 const float* lse, uint16_t* dx, int64_t lddx, float* dw, int64_t lddw,
                                                 float* db, int32_t accumulate, int64_t M, int64_t N, int64_t K,
                                                 void* workspace, int64_t workspace_bytes, void* stream) {
    return run_loss_backward(kF16, true, dloss, dlse, x, ldx, weight, ldw, b, target, lse, dx, lddx, dw, lddw, db, accumulate, M,
                             N, K, workspace, workspace_bytes, (hipStream_t)stream);
}

int32_t linear_bf16_cross_entropy_backward_f32out(const float* dloss, const float* dlse, const uint16_t* x, int64_t ldx,
                                                  const uint16_t* weight, int64_t ldw, const uint16_t* b, const int64_t* target,
                                                  const float* lse, uint16_t* dx, int64_t lddx, float* dw, int64_t lddw,
                                                  float* db, int32_t accumulate, int64_t M, int64_t N, int64_t K,
                                                  void* workspace, int64_t workspace_bytes, void* stream) {
    return run_loss_backward(kBF16, true, dloss, dlse, x, ldx, weight, ldw, b, target, lse, dx, lddx, dw, lddw, db, accumulate, M,
                             N, K, workspace, workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"
