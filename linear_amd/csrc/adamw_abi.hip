// adamw_abi.hip -- the C ABI of the AdamW step: argument checks, tables of tensors, launches.
// The conventions are linear_abi.hip's: every check runs on the host before anything is
// enqueued, and only kernels are enqueued.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <memory>
#include <new>

#include "../../include/linear_amd.h"
#include "abi.h"
#include "adamw.h"
#include "train.h"
#include "train_host.h"

namespace {

using namespace lin;

static_assert(kAdamBlock == LINEAR_ADAMW_BLOCK, "values of a block");

int64_t state_bytes(int64_t n, int32_t bits) { return bits == 8 ? n + tiles_of(n, kAdamBlock) : 4 * n; }

bool empty(const linear_tensor& t) { return t.rows == 0 || t.cols == 0; }

int32_t check_like(const linear_tensor& t, const linear_tensor& like) {
    const int32_t st = check_tensor(t);
    if (st != LINEAR_OK) return st;
    return t.rows == like.rows && t.cols == like.cols ? LINEAR_OK : LINEAR_E_SHAPE;
}

// Whether a tensor's rows follow each other without gaps.
bool whole(const linear_tensor& t) { return t.rows == 1 || t.ld == t.cols; }

Extent extent_of(const linear_tensor& t) { return extent(t.data, t.rows, t.ld, t.cols, type_bytes(t.type)); }

// An output must be apart from every other range, an input from every output.
int32_t check_ranges(Range* ranges, int64_t n) {
    std::sort(ranges, ranges + n, [](const Range& a, const Range& b) { return a.e.lo < b.e.lo; });
    uintptr_t all = 0, outs = 0;
    for (int64_t i = 0; i < n; ++i) {
        const Range& r = ranges[i];
        if (r.e.lo < (r.out ? all : outs)) return LINEAR_E_ALIAS;
        all = std::max(all, r.e.hi);
        if (r.out) outs = std::max(outs, r.e.hi);
    }
    return LINEAR_OK;
}

bool share(double v) { return v >= 0.0 && v < 1.0; }
bool amount(double v) { return v >= 0.0 && v <= 1.7e308; }

int32_t check_options(const linear_adamw_options& o) {
    if (o.state_bits != 8 && o.state_bits != 32) return LINEAR_E_VALUE;
    if (!amount(o.lr) || !share(o.beta1) || !share(o.beta2) || !amount(o.eps) || !amount(o.weight_decay)) return LINEAR_E_VALUE;
    if (!o.device_step && o.step < 1) return LINEAR_E_VALUE;
    if (o.norm && !(o.max_norm >= 0.f)) return LINEAR_E_VALUE;
    return LINEAR_OK;
}

int grid_of(int64_t chunks) { return (int)std::min<int64_t>(chunks, kAdamGrid); }

// The launches over the tensors that are not empty.
template <typename Table>
int32_t launch_tables(const linear_tensor* params, const linear_tensor* grads, void* const* m, void* const* v,
                      const linear_tensor* copies, int64_t count, bool eight, const AdamArgs& a, hipStream_t stream) {
    Table t;
    memset(&t, 0, sizeof t);
    for (int64_t i = 0; i < count; ++i) {
        const linear_tensor &p = params[i], &g = grads[i];
        if (!empty(p)) {
            const int k = t.count;
            t.param[k] = p.data;
            t.grad[k] = g.data;
            t.m[k] = m[i];
            t.v[k] = v[i];
            t.n[k] = p.rows * p.cols;
            t.types[k] = (uint8_t)(3 * p.type + g.type);
            if constexpr (!Table::kPlain) {
                t.copy[k] = copies ? copies[i].data : nullptr;
                t.cols[k] = whole(p) && whole(g) && (!copies || whole(copies[i])) ? 0 : p.cols;
                t.ldp[k] = (int32_t)(p.rows == 1 ? 0 : p.ld);
                t.ldg[k] = (int32_t)(g.rows == 1 ? 0 : g.ld);
                t.ldc[k] = (int32_t)(!copies || p.rows == 1 ? 0 : copies[i].ld);
                t.ctype[k] = (uint8_t)(copies ? copies[i].type : (int64_t)kNoCopy);
            }
            t.first[k + 1] = t.first[k] + tiles_of(t.n[k], adam_chunk(eight));
            t.count = k + 1;
        }
        if (t.count == Table::kMost || (i + 1 == count && t.count > 0)) {
            const int32_t st = launched(launch_adamw(eight, t, a, grid_of(t.first[t.count]), stream));
            if (st != LINEAR_OK) return st;
            t.count = 0;
        }
    }
    return LINEAR_OK;
}

}  // namespace

extern "C" {

int64_t linear_adamw_state_bytes(int64_t n, int32_t bits) {
    if (n < 0 || n > kMaxElems || (bits != 8 && bits != 32)) return -1;
    return state_bytes(n, bits);
}

int32_t linear_adamw(const linear_tensor* params, const linear_tensor* grads, void* const* m, void* const* v,
                     const linear_tensor* copies, int64_t count, const linear_adamw_options* options, void* stream) {
    if (count < 0 || count > LINEAR_GRAD_MAX_TENSORS) return LINEAR_E_SHAPE;
    if (!options) return LINEAR_E_NULL;
    int32_t st = check_options(*options);
    if (st != LINEAR_OK) return st;
    if (count == 0) return LINEAR_OK;
    if (!params || !grads || !m || !v) return LINEAR_E_NULL;
    const linear_adamw_options& o = *options;
    std::unique_ptr<Range[]> ranges(new (std::nothrow) Range[5 * count + 3]);
    if (!ranges) return LINEAR_E_MEMORY;
    int64_t n = 0;
    const auto add = [&](Extent e, bool out) {
        if (e.hi > e.lo) ranges[n++] = {e, out};
    };
    add(extent(o.norm, 1, 1, 1, 4), false);
    add(extent(o.device_lr, 1, 1, 1, 4), false);
    add(extent(o.device_step, 1, 1, 1, 8), false);
    for (int64_t i = 0; i < count; ++i) {
        const linear_tensor& p = params[i];
        if ((st = check_tensor(p)) != LINEAR_OK || (st = check_like(grads[i], p)) != LINEAR_OK) return st;
        if (copies) {
            if ((st = check_like(copies[i], p)) != LINEAR_OK) return st;
            if (copies[i].type == LINEAR_TYPE_F32) return LINEAR_E_VALUE;
            add(extent_of(copies[i]), true);
        }
        if (empty(p)) continue;
        if (p.cols > kMaxElems / p.rows) return LINEAR_E_SHAPE;
        if (!m[i] || !v[i]) return LINEAR_E_NULL;
        const int64_t bytes = state_bytes(p.rows * p.cols, o.state_bits);
        add(extent_of(p), true);
        add(extent_of(grads[i]), false);
        add(extent(m[i], 1, bytes, bytes, 1), true);
        add(extent(v[i], 1, bytes, bytes, 1), true);
    }
    if ((st = check_ranges(ranges.get(), n)) != LINEAR_OK) return st;
    int dev = 0;
    if ((st = check_device(&dev)) != LINEAR_OK) return st;
    AdamArgs a;
    memset(&a, 0, sizeof a);
    a.lr = o.lr;
    a.beta1 = o.beta1;
    a.beta2 = o.beta2;
    a.weight_decay = o.weight_decay;
    a.bias1 = 1.0 - pow(o.beta1, (double)o.step);
    a.bias2 = 1.0 - pow(o.beta2, (double)o.step);
    a.keep = (float)(1.0 - o.lr * o.weight_decay);
    a.rate = (float)(o.lr / a.bias1);
    a.root = (float)(1.0 / sqrt(a.bias2));
    // the kernels' reciprocal takes a subnormal denominator for zero: 0 / eps would be NaN.  (Beside a root, of
    // 2^-75 at least, an eps under 2^-126 is nothing.)
    a.eps = o.eps > 0.0 ? std::max((float)o.eps, 0x1p-126f) : 0.f;
    a.max_norm = o.max_norm;
    a.norm = o.norm;
    a.device_lr = o.device_lr;
    a.device_step = o.device_step;
    bool plain = !copies;
    for (int64_t i = 0; i < count && plain; ++i) plain = empty(params[i]) || (whole(params[i]) && whole(grads[i]));
    if (plain) return launch_tables<AdamPlainTable>(params, grads, m, v, nullptr, count, o.state_bits == 8, a, (hipStream_t)stream);
    return launch_tables<AdamTable>(params, grads, m, v, copies, count, o.state_bits == 8, a, (hipStream_t)stream);
}

int32_t linear_adamw_values(const linear_tensor* out, const void* const* states, int32_t second, int64_t count, void* stream) {
    if (count < 0 || count > LINEAR_GRAD_MAX_TENSORS) return LINEAR_E_SHAPE;
    if (count == 0) return LINEAR_OK;
    if (!out || !states) return LINEAR_E_NULL;
    std::unique_ptr<Range[]> ranges(new (std::nothrow) Range[2 * count]);
    if (!ranges) return LINEAR_E_MEMORY;
    int64_t n = 0;
    int32_t st;
    for (int64_t i = 0; i < count; ++i) {
        if ((st = check_tensor(out[i])) != LINEAR_OK) return st;
        if (out[i].type == LINEAR_TYPE_F16) return LINEAR_E_VALUE;   // a state's range is binary32's
        if (empty(out[i])) continue;
        if (out[i].cols > kMaxElems / out[i].rows) return LINEAR_E_SHAPE;
        if (!states[i]) return LINEAR_E_NULL;
        const int64_t bytes = state_bytes(out[i].rows * out[i].cols, 8);
        ranges[n++] = {extent_of(out[i]), true};
        ranges[n++] = {extent(states[i], 1, bytes, bytes, 1), false};
    }
    if ((st = check_ranges(ranges.get(), n)) != LINEAR_OK) return st;
    int dev = 0;
    if ((st = check_device(&dev)) != LINEAR_OK) return st;
    ValueTable t;
    memset(&t, 0, sizeof t);
    for (int64_t i = 0; i < count; ++i) {
        const linear_tensor& y = out[i];
        if (!empty(y)) {
            const int k = t.count;
            t.state[k] = (const uint8_t*)states[i];
            t.out[k] = y.data;
            t.n[k] = y.rows * y.cols;
            t.cols[k] = whole(y) ? 0 : y.cols;
            t.ld[k] = (int32_t)(y.rows == 1 ? 0 : y.ld);
            t.f32[k] = y.type == LINEAR_TYPE_F32;
            t.first[k + 1] = t.first[k] + tiles_of(t.n[k], kValueChunk);
            t.count = k + 1;
        }
        if (t.count == kValueTensors || (i + 1 == count && t.count > 0)) {
            st = launched(launch_adamw_values(second != 0, t, grid_of(t.first[t.count]), (hipStream_t)stream));
            if (st != LINEAR_OK) return st;
            t.count = 0;
        }
    }
    return LINEAR_OK;
}

}  // extern "C"
