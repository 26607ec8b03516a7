// fsdp_ops_capi.cpp -- argument checks and the extern "C" entry points of the
// training-step operators (fsdp_ops.h). Host code only.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
#include <limits>
#include <mutex>
#include <unordered_map>

#include <cuda_runtime.h>

#include "fsdp_ops_internal.h"

namespace fsdp {

cudaError_t norm_wait_timeouts(unsigned long long *n);
cudaError_t loss_wait_timeouts(unsigned long long *n);
cudaError_t muon_wait_timeouts(unsigned long long *n);
cudaError_t team_wait_timeouts(unsigned long long *n);

Record *&current_record()
{
    static thread_local Record *r = nullptr;
    return r;
}

fsdp_status Record::add(const char *fmt, ...)
{
    char line[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(line, sizeof line, fmt, ap);
    va_end(ap);
    text += line;
    text += '\n';
    return FSDP_OK;
}

int device_sms(int dev)
{
    if (const Record *r = current_record())
        return r->sms;
    static std::mutex mu;
    static std::unordered_map<int, int> known;
    std::lock_guard<std::mutex> lk(mu);
    int &n = known[dev];
    if (n == 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        n = 0;
    return n > 0 ? n : 1;
}

namespace {

// Sizes whose coordinates the tensor maps and kernels hold in 32 bits, with
// room for what a loop's last step reaches past them (the loss's pass over the
// rows: four steps of 2048 columns, and segments rounded up by 8 columns each).
constexpr int64_t kMaxDim = (int64_t(1) << 31) - (1 << 16);
constexpr int64_t kMaxElems = int64_t(1) << 40;
// Elements from the first to the last of a matrix, gaps included: with the
// batch's (65,535 strides of at most kMaxElems) their bytes stay in int64.
constexpr int64_t kMaxRange = int64_t(1) << 56;

int64_t esize(fsdp_dtype d) { return d == FSDP_BF16 ? 2 : 4; }
bool known(fsdp_dtype d) { return d == FSDP_F32 || d == FSDP_BF16; }

// Whether fp32, in which the kernels take the numbers, holds v: finite, and 0
// only for 0.
bool in_f32(double v) { return std::isfinite((float)v) && ((float)v != 0.0f || v == 0.0); }

// One call's buffers: each is checked as it is named, the rest in done().
class Buffers {
  public:
    explicit Buffers(const char *fn) : fn_(fn) {}

    // [rows, cols] with row stride ld, of `size`-byte elements, `batch` of
    // them `stride` elements apart.
    void matrix(const char *what, const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t size,
                bool out, int64_t batch = 1, int64_t stride = 0, int index = -1)
    {
        if (st_ != FSDP_OK || rows == 0 || cols == 0 || batch == 0)
            return;
        if (p == nullptr)
            fail(FSDP_EINVAL, what, index, "is NULL");
        else if (reinterpret_cast<uintptr_t>(p) % (uintptr_t)size)
            fail(FSDP_EALIGN, what, index, "is not aligned to its element");
        else if (ld < cols || ld > kMaxElems)
            fail(FSDP_EINVAL, what, index, "has a row stride below its columns");
        else if (rows - 1 > kMaxRange / ld)
            fail(FSDP_ERANGE, what, index, "has a range that is too large");
        else if (batch > 1 && (stride < (rows - 1) * ld + cols || stride > kMaxElems))
            fail(FSDP_EINVAL, what, index, "has a batch stride below its matrices");
        else {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
            const int64_t n = (batch - 1) * stride + (rows - 1) * ld + cols;
            spans_.push_back({lo, lo + (uintptr_t)(n * size), out, what, index});
        }
    }
    void vector(const char *what, const void *p, int64_t n, int64_t size, bool out)
    {
        matrix(what, p, n ? 1 : 0, n, n, size, out);
    }
    void workspace(const void *p, int64_t have, int64_t need)
    {
        if (st_ != FSDP_OK || need == 0)
            return;
        if (have < need)
            st_ = set_error(FSDP_EINVAL, "%s: workspace of %lld bytes, needs %lld", fn_, (long long)have,
                            (long long)need);
        else if (p == nullptr)
            fail(FSDP_EINVAL, "workspace", -1, "is NULL");
        else if (reinterpret_cast<uintptr_t>(p) & 255u)
            fail(FSDP_EALIGN, "workspace", -1, "is not 256-byte aligned");
        else {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
            spans_.push_back({lo, lo + (uintptr_t)need, true, "workspace", -1});
        }
    }

    // Overlaps and devices; on success makes the buffers' device current for
    // the life of this object.
    fsdp_status done()
    {
        if (st_ != FSDP_OK)
            return st_;
        std::sort(spans_.begin(), spans_.end(), [](const Span &a, const Span &b) { return a.lo < b.lo; });
        const Span *any = nullptr, *out = nullptr;  // those that reach furthest
        for (const Span &s : spans_) {
            const Span *hit = s.out && any && s.lo < any->hi ? any : out && s.lo < out->hi ? out : nullptr;
            if (hit)
                return set_error(FSDP_EINVAL, "%s: %s overlaps %s", fn_, s.what, hit->what);
            if (!any || s.hi > any->hi)
                any = &s;
            if (s.out && (!out || s.hi > out->hi))
                out = &s;
        }
        for (const Span &s : spans_) {
            cudaPointerAttributes a;
            const cudaError_t err = cudaPointerGetAttributes(&a, reinterpret_cast<const void *>(s.lo));
            if (err != cudaSuccess) {
                cudaGetLastError();
                return set_error(FSDP_ECUDA, "%s: cudaPointerGetAttributes(%s): %s", fn_, s.what,
                                 cudaGetErrorString(err));
            }
            if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)
                return set_error(FSDP_EINVAL, "%s: %s is not device memory", fn_, s.what);
            if (dev_ >= 0 && a.device != dev_)
                return set_error(FSDP_EINVAL, "%s: %s is on device %d, other buffers on device %d", fn_, s.what,
                                 a.device, dev_);
            dev_ = a.device;
        }
        if (dev_ < 0)
            return FSDP_OK;
        cudaError_t err = cudaGetDevice(&prev_);
        if (err == cudaSuccess && prev_ != dev_) {
            err = cudaSetDevice(dev_);
            changed_ = err == cudaSuccess;
        }
        return err == cudaSuccess ? FSDP_OK
                                  : set_error(FSDP_ECUDA, "%s: device %d: %s", fn_, dev_, cudaGetErrorString(err));
    }
    int device() const { return dev_; }
    ~Buffers()
    {
        if (changed_)
            cudaSetDevice(prev_);
    }
    Buffers(const Buffers &) = delete;
    Buffers &operator=(const Buffers &) = delete;

  private:
    struct Span {
        uintptr_t lo, hi;
        bool out;
        const char *what;
        int index;
    };
    void fail(fsdp_status st, const char *what, int index, const char *why)
    {
        st_ = index < 0 ? set_error(st, "%s: %s %s", fn_, what, why)
                        : set_error(st, "%s: %s[%d] %s", fn_, what, index, why);
    }
    const char *fn_;
    fsdp_status st_ = FSDP_OK;
    std::vector<Span> spans_;
    int dev_ = -1, prev_ = -1;
    bool changed_ = false;
};

// Runs a call's body; no exception passes the C interface.
template <class F>
fsdp_status guarded(const char *fn, F f)
{
    try {
        return f();
    } catch (const std::exception &e) {
        try {
            return set_error(FSDP_EINVAL, "%s: %s", fn, e.what());
        } catch (...) {
            return FSDP_EINVAL;
        }
    } catch (...) {
        return FSDP_EINVAL;
    }
}

fsdp_status check_size(const char *fn, const char *what, int64_t v, int64_t least)
{
    if (v < least)
        return set_error(FSDP_EINVAL, "%s: %s = %lld, must be at least %lld", fn, what, (long long)v, (long long)least);
    if (v > kMaxDim)
        return set_error(FSDP_ERANGE, "%s: %s = %lld is too large", fn, what, (long long)v);
    return FSDP_OK;
}

fsdp_status check_norm(const char *fn, int64_t rows, int64_t cols, fsdp_dtype dtype, fsdp_dtype param_dtype)
{
    fsdp_status st;
    if ((st = check_size(fn, "rows", rows, 0)) != FSDP_OK || (st = check_size(fn, "cols", cols, 1)) != FSDP_OK)
        return st;
    if (!known(dtype) || !known(param_dtype))
        return set_error(FSDP_EUNSUPPORTED, "%s: unsupported dtype", fn);
    if (rows > kMaxElems / cols)
        return set_error(FSDP_ERANGE, "%s: %lld x %lld is too large", fn, (long long)rows, (long long)cols);
    return FSDP_OK;
}

fsdp_status check_loss(const char *fn, int64_t rows, int64_t cols, int64_t vocab, int64_t piece_rows)
{
    fsdp_status st;
    if ((st = check_size(fn, "rows", rows, 0)) != FSDP_OK || (st = check_size(fn, "cols", cols, 1)) != FSDP_OK ||
        (st = check_size(fn, "vocab", vocab, 1)) != FSDP_OK ||
        (st = check_size(fn, "piece_rows", piece_rows, 0)) != FSDP_OK)
        return st;
    if (rows > kMaxElems / cols || vocab > kMaxElems / cols || rows > kMaxElems / vocab)
        return set_error(FSDP_ERANGE, "%s: %lld x %lld x %lld is too large", fn, (long long)rows, (long long)cols,
                         (long long)vocab);
    return FSDP_OK;
}

fsdp_status check_schulz(const char *fn, int64_t batch, int64_t m, int64_t n)
{
    fsdp_status st;
    if ((st = check_size(fn, "m", m, 1)) != FSDP_OK || (st = check_size(fn, "n", n, 1)) != FSDP_OK)
        return st;
    if (batch < 0 || batch > 65535)
        return set_error(FSDP_EINVAL, "%s: batch = %lld outside [0, 65535]", fn, (long long)batch);
    if (m > kMaxElems / n || (batch > 0 && m * n > kMaxElems / batch))
        return set_error(FSDP_ERANGE, "%s: %lld x %lld x %lld is too large", fn, (long long)batch, (long long)m,
                         (long long)n);
    return FSDP_OK;
}

fsdp_status check_iteration(const char *fn, int steps, double eps, double a, double b, double c)
{
    if (steps < 0 || steps > 64)
        return set_error(FSDP_EINVAL, "%s: steps = %d outside [0, 64]", fn, steps);
    if (!(in_f32(eps) && eps >= 0) || !std::isfinite((float)a) || !std::isfinite((float)b) || !std::isfinite((float)c))
        return set_error(FSDP_EINVAL, "%s: bad eps or coefficients", fn);
    return FSDP_OK;
}

// Runs f with a record set and hands the text out.
template <class F>
fsdp_status recorded(const char *fn, int sms, char *text, int64_t bytes, F f)
{
    if (sms < 1 || text == nullptr || bytes < 1)
        return set_error(FSDP_EINVAL, "%s: bad sms or text", fn);
    struct Set {
        explicit Set(Record *r) { current_record() = r; }
        ~Set() { current_record() = nullptr; }
    };
    Record r{sms, {}};
    fsdp_status st;
    {
        const Set set(&r);
        st = f();
    }
    if (st == FSDP_OK && (int64_t)r.text.size() >= bytes)
        return set_error(FSDP_EINVAL, "%s: the text has %lld bytes", fn, (long long)r.text.size() + 1);
    if (st == FSDP_OK)
        memcpy(text, r.text.c_str(), r.text.size() + 1);
    return st;
}

}  // namespace
}  // namespace fsdp

using namespace fsdp;

extern "C" {

fsdp_status fsdp_layer_norm(int64_t rows, int64_t cols, const void *x, int64_t ldx, fsdp_dtype dtype,
                            const void *gamma, const void *beta, fsdp_dtype param_dtype, double eps, void *y,
                            int64_t ldy, float *mean, float *rstd, void *stream)
{
    const char *fn = "fsdp_layer_norm";
    return guarded(fn, [&]() -> fsdp_status {
        fsdp_status st = check_norm(fn, rows, cols, dtype, param_dtype);
        if (st != FSDP_OK)
            return st;
        if (!(in_f32(eps) && eps > 0))
            return set_error(FSDP_EINVAL, "%s: eps = %g, must be above 0 and an fp32 number", fn, eps);
        if ((mean == nullptr) != (rstd == nullptr))
            return set_error(FSDP_EINVAL, "%s: mean and rstd are given together", fn);
        if (rows == 0)
            return FSDP_OK;
        Buffers b(fn);
        b.matrix("x", x, rows, cols, ldx, esize(dtype), false);
        b.vector("gamma", gamma, cols, esize(param_dtype), false);
        if (beta)
            b.vector("beta", beta, cols, esize(param_dtype), false);
        b.matrix("y", y, rows, cols, ldy, esize(dtype), true);
        if (mean) {
            b.vector("mean", mean, rows, 4, true);
            b.vector("rstd", rstd, rows, 4, true);
        }
        if ((st = b.done()) != FSDP_OK)
            return st;
        NormArgs a{};
        a.rows = rows, a.cols = cols, a.x = x, a.ldx = ldx, a.gamma = gamma, a.beta = beta;
        a.dtype = dtype, a.param_dtype = param_dtype, a.eps = (float)eps;
        a.y = y, a.ldy = ldy, a.mean = mean, a.rstd = rstd;
        return launch_layer_norm(a, b.device(), stream);
    });
}

fsdp_status fsdp_layer_norm_backward_workspace(int64_t rows, int64_t cols, int64_t *bytes)
{
    const char *fn = "fsdp_layer_norm_backward_workspace";
    return guarded(fn, [&]() -> fsdp_status {
        if (bytes == nullptr)
            return set_error(FSDP_EINVAL, "%s: bytes is NULL", fn);
        fsdp_status st = check_norm(fn, rows, cols, FSDP_F32, FSDP_F32);
        if (st != FSDP_OK)
            return st;
        *bytes = norm_backward_workspace(rows, cols);
        return FSDP_OK;
    });
}

fsdp_status fsdp_layer_norm_backward(int64_t rows, int64_t cols, const void *dy, int64_t lddy, const void *x,
                                     int64_t ldx, fsdp_dtype dtype, const void *gamma, fsdp_dtype param_dtype,
                                     const float *mean, const float *rstd, void *dx, int64_t lddx, void *dgamma,
                                     void *dbeta, void *workspace, int64_t workspace_bytes, void *stream)
{
    const char *fn = "fsdp_layer_norm_backward";
    return guarded(fn, [&]() -> fsdp_status {
        fsdp_status st = check_norm(fn, rows, cols, dtype, param_dtype);
        if (st != FSDP_OK)
            return st;
        Buffers b(fn);
        b.matrix("dy", dy, rows, cols, lddy, esize(dtype), false);
        b.matrix("x", x, rows, cols, ldx, esize(dtype), false);
        b.vector("gamma", gamma, cols, esize(param_dtype), false);
        b.vector("mean", mean, rows, 4, false);
        b.vector("rstd", rstd, rows, 4, false);
        b.matrix("dx", dx, rows, cols, lddx, esize(dtype), true);
        b.vector("dgamma", dgamma, cols, esize(param_dtype), true);
        if (dbeta)
            b.vector("dbeta", dbeta, cols, esize(param_dtype), true);
        b.workspace(workspace, workspace_bytes, norm_backward_workspace(rows, cols));
        if ((st = b.done()) != FSDP_OK)
            return st;
        NormArgs a{};
        a.rows = rows, a.cols = cols, a.x = x, a.ldx = ldx, a.gamma = gamma;
        a.dtype = dtype, a.param_dtype = param_dtype;
        a.dy = dy, a.lddy = lddy, a.mean_in = mean, a.rstd_in = rstd, a.dx = dx, a.lddx = lddx;
        a.dgamma = dgamma, a.dbeta = dbeta, a.partial = static_cast<float *>(workspace);
        return launch_layer_norm_backward(a, b.device(), stream);
    });
}

fsdp_status fsdp_linear_cross_entropy_workspace(int64_t rows, int64_t cols, int64_t vocab, int with_gradients,
                                                int aligned_weight, int64_t piece_rows, int64_t *bytes)
{
    const char *fn = "fsdp_linear_cross_entropy_workspace";
    return guarded(fn, [&]() -> fsdp_status {
        if (bytes == nullptr)
            return set_error(FSDP_EINVAL, "%s: bytes is NULL", fn);
        fsdp_status st = check_loss(fn, rows, cols, vocab, piece_rows);
        if (st != FSDP_OK)
            return st;
        LossArgs a{};
        a.rows = rows, a.cols = cols, a.vocab = vocab, a.piece_rows = piece_rows;
        *bytes = loss_workspace(a, with_gradients != 0, aligned_weight != 0);
        return FSDP_OK;
    });
}

fsdp_status fsdp_linear_cross_entropy(int64_t rows, int64_t cols, int64_t vocab, const void *hidden, int64_t ldh,
                                      const void *weight, int64_t ldw, const int64_t *targets, int64_t ignore_index,
                                      fsdp_reduction reduction, double grad_scale, float *loss, float *row_loss,
                                      void *dhidden, int64_t lddh, void *dweight, int64_t lddw, int64_t piece_rows,
                                      void *workspace, int64_t workspace_bytes, void *stream)
{
    const char *fn = "fsdp_linear_cross_entropy";
    return guarded(fn, [&]() -> fsdp_status {
        fsdp_status st = check_loss(fn, rows, cols, vocab, piece_rows);
        if (st != FSDP_OK)
            return st;
        if (reduction != FSDP_MEAN && reduction != FSDP_SUM)
            return set_error(FSDP_EINVAL, "%s: unknown reduction %d", fn, (int)reduction);
        if (!std::isfinite(grad_scale) || !std::isfinite((float)grad_scale))
            return set_error(FSDP_EINVAL, "%s: grad_scale = %g", fn, grad_scale);
        if ((dhidden == nullptr) != (dweight == nullptr) && rows > 0)
            return set_error(FSDP_EINVAL, "%s: dhidden and dweight are given together", fn);
        LossArgs a{};
        a.rows = rows, a.cols = cols, a.vocab = vocab, a.piece_rows = piece_rows;
        a.hidden = hidden, a.ldh = ldh, a.weight = weight, a.ldw = ldw, a.targets = targets;
        a.ignore_index = ignore_index, a.mean = reduction == FSDP_MEAN, a.grad_scale = (float)grad_scale;
        a.loss = loss, a.row_loss = row_loss, a.dhidden = dhidden, a.lddh = lddh, a.dweight = dweight, a.lddw = lddw;
        const bool grad = dweight != nullptr;
        Buffers b(fn);
        b.matrix("hidden", hidden, rows, cols, ldh, 2, false);
        b.matrix("weight", weight, vocab, cols, ldw, 2, false);
        b.vector("targets", targets, rows, 8, false);
        b.vector("loss", loss, 1, 4, true);
        b.vector("row_loss", row_loss, rows, 4, true);
        if (grad) {
            b.matrix("dhidden", dhidden, rows, cols, lddh, 2, true);
            b.matrix("dweight", dweight, vocab, cols, lddw, 2, true);
        }
        b.workspace(workspace, workspace_bytes, loss_workspace(a, grad, loss_weight_aligned(weight, ldw)));
        if ((st = b.done()) != FSDP_OK)
            return st;
        return launch_linear_cross_entropy(a, workspace, b.device(), stream);
    });
}

fsdp_status fsdp_newton_schulz_workspace(int64_t batch, int64_t m, int64_t n, int64_t *bytes)
{
    const char *fn = "fsdp_newton_schulz_workspace";
    return guarded(fn, [&]() -> fsdp_status {
        if (bytes == nullptr)
            return set_error(FSDP_EINVAL, "%s: bytes is NULL", fn);
        fsdp_status st = check_schulz(fn, batch, m, n);
        if (st != FSDP_OK)
            return st;
        *bytes = schulz_workspace(batch, m, n, false);
        return FSDP_OK;
    });
}

fsdp_status fsdp_newton_schulz(int64_t batch, int64_t m, int64_t n, const void *g, int64_t ldg, int64_t batch_stride,
                               fsdp_dtype dtype, void *out, int64_t ldo, int64_t out_batch_stride, int steps,
                               double eps, double a, double b, double c, void *workspace, int64_t workspace_bytes,
                               void *stream)
{
    const char *fn = "fsdp_newton_schulz";
    return guarded(fn, [&]() -> fsdp_status {
        fsdp_status st = check_schulz(fn, batch, m, n);
        if (st != FSDP_OK || (st = check_iteration(fn, steps, eps, a, b, c)) != FSDP_OK)
            return st;
        if (!known(dtype))
            return set_error(FSDP_EUNSUPPORTED, "%s: unsupported dtype", fn);
        if (batch == 0)
            return FSDP_OK;
        Buffers buf(fn);
        buf.matrix("g", g, m, n, ldg, esize(dtype), false, batch, batch_stride);
        buf.matrix("out", out, m, n, ldo, 2, true, batch, out_batch_stride);
        buf.workspace(workspace, workspace_bytes, schulz_workspace(batch, m, n, false));
        if ((st = buf.done()) != FSDP_OK)
            return st;
        SchulzArgs s{};
        s.batch = batch, s.m = m, s.n = n, s.steps = steps;
        s.eps = (float)eps, s.a = (float)a, s.b = (float)b, s.c = (float)c;
        s.g = g, s.ldg = ldg, s.g_stride = batch > 1 ? batch_stride : 0, s.dtype = dtype;
        s.out = out, s.ldo = ldo, s.out_stride = batch > 1 ? out_batch_stride : 0;
        return launch_newton_schulz(s, workspace, buf.device(), stream);
    });
}

fsdp_status fsdp_muon_workspace(int n_mats, int64_t m, int64_t n, int64_t *bytes)
{
    const char *fn = "fsdp_muon_workspace";
    return guarded(fn, [&]() -> fsdp_status {
        if (bytes == nullptr)
            return set_error(FSDP_EINVAL, "%s: bytes is NULL", fn);
        fsdp_status st = check_schulz(fn, n_mats, m, n);
        if (st != FSDP_OK)
            return st;
        *bytes = schulz_workspace(n_mats, m, n, true);
        return FSDP_OK;
    });
}

fsdp_status fsdp_muon(int n_mats, int64_t m, int64_t n, int R, const void *const *grads, fsdp_dtype grad_dtype,
                      float *const *momentum, float *const *master, void *const *param_out, const fsdp_muon_hp *hp,
                      void *workspace, int64_t workspace_bytes, void *stream)
{
    const char *fn = "fsdp_muon";
    return guarded(fn, [&]() -> fsdp_status {
        if (n_mats < 1 || n_mats > FSDP_MUON_MAX_MATRICES)
            return set_error(FSDP_EINVAL, "%s: n_mats = %d outside [1, %d]", fn, n_mats, FSDP_MUON_MAX_MATRICES);
        if (R < 1 || R > FSDP_MAX_RANKS)
            return set_error(FSDP_EINVAL, "%s: R = %d outside [1, %d]", fn, R, FSDP_MAX_RANKS);
        if (n_mats * R > kMuonMaxGrads)
            return set_error(FSDP_EINVAL, "%s: n_mats * R = %d is above %d", fn, n_mats * R, kMuonMaxGrads);
        fsdp_status st = check_schulz(fn, n_mats, m, n);
        if (st != FSDP_OK)
            return st;
        if (hp == nullptr)
            return set_error(FSDP_EINVAL, "%s: hp is NULL", fn);
        if ((st = check_iteration(fn, hp->steps, hp->eps, hp->a, hp->b, hp->c)) != FSDP_OK)
            return st;
        if (!(std::isfinite(hp->lr) && hp->lr >= 0) || !(hp->momentum >= 0 && (float)hp->momentum < 1) ||
            !std::isfinite(hp->weight_decay) || !(std::isfinite(hp->update_scale) && hp->update_scale > 0) ||
            !std::isfinite((float)(hp->lr * hp->update_scale)) ||
            !std::isfinite((float)(1.0 - hp->lr * hp->weight_decay)))
            return set_error(FSDP_EINVAL, "%s: bad hyper-parameters", fn);
        if (!known(grad_dtype))
            return set_error(FSDP_EUNSUPPORTED, "%s: unsupported dtype", fn);
        if (grads == nullptr || momentum == nullptr || master == nullptr)
            return set_error(FSDP_EINVAL, "%s: a pointer array is NULL", fn);
        Buffers b(fn);
        for (int i = 0; i < n_mats * R; i++)
            b.matrix("grads", grads[i], m, n, n, esize(grad_dtype), false, 1, 0, i);
        for (int i = 0; i < n_mats; i++) {
            b.matrix("momentum", momentum[i], m, n, n, 4, true, 1, 0, i);
            b.matrix("master", master[i], m, n, n, 4, true, 1, 0, i);
            if (param_out)
                b.matrix("param_out", param_out[i], m, n, n, 2, true, 1, 0, i);
        }
        b.workspace(workspace, workspace_bytes, schulz_workspace(n_mats, m, n, true));
        if ((st = b.done()) != FSDP_OK)
            return st;
        SchulzArgs s{};
        s.batch = n_mats, s.m = m, s.n = n, s.steps = hp->steps;
        s.eps = (float)hp->eps, s.a = (float)hp->a, s.b = (float)hp->b, s.c = (float)hp->c;
        s.dtype = grad_dtype, s.grads = grads, s.R = R;
        s.momentum = momentum, s.master = master, s.param_out = param_out;
        s.mu = (float)hp->momentum, s.decay = (float)(1.0 - hp->lr * hp->weight_decay);
        s.lr = (float)(hp->lr * hp->update_scale), s.nesterov = hp->nesterov != 0;
        return launch_newton_schulz(s, workspace, b.device(), stream);
    });
}

fsdp_status fsdp_ops_wait_timeouts(int device, uint64_t *count)
{
    const char *fn = "fsdp_ops_wait_timeouts";
    return guarded(fn, [&]() -> fsdp_status {
        if (count == nullptr || device < 0)
            return set_error(FSDP_EINVAL, "%s: count is NULL or device < 0", fn);
        int prev = -1;
        cudaError_t err = cudaGetDevice(&prev);
        if (err != cudaSuccess)
            return set_error(FSDP_ECUDA, "%s: cudaGetDevice: %s", fn, cudaGetErrorString(err));
        if (prev != device && (err = cudaSetDevice(device)) != cudaSuccess)
            return set_error(FSDP_ECUDA, "%s: cudaSetDevice(%d): %s", fn, device, cudaGetErrorString(err));
        unsigned long long n[4] = {0, 0, 0, 0};
        err = cudaDeviceSynchronize();
        if (err == cudaSuccess)
            err = norm_wait_timeouts(&n[0]);
        if (err == cudaSuccess)
            err = loss_wait_timeouts(&n[1]);
        if (err == cudaSuccess)
            err = muon_wait_timeouts(&n[2]);
        if (err == cudaSuccess)
            err = team_wait_timeouts(&n[3]);
        if (prev != device)
            cudaSetDevice(prev);
        if (err != cudaSuccess)
            return set_error(FSDP_ECUDA, "%s: %s", fn, cudaGetErrorString(err));
        *count = n[0] + n[1] + n[2] + n[3];
        return FSDP_OK;
    });
}

// Pointers are looked at for their alignment alone.
fsdp_status fsdp_ops_plan_newton_schulz(int64_t batch, int64_t m, int64_t n, int ranks, int steps, int sms, char *text,
                                        int64_t bytes)
{
    const char *fn = "fsdp_ops_plan_newton_schulz";
    return guarded(fn, [&]() -> fsdp_status {
        fsdp_status st = check_schulz(fn, batch, m, n);
        if (st != FSDP_OK || (st = check_iteration(fn, steps, 1e-7, 0, 0, 0)) != FSDP_OK)
            return st;
        if (batch < 1 || ranks < 0 || (ranks > 0 && (batch > kMuonMaxMats || batch * ranks > kMuonMaxGrads)))
            return set_error(FSDP_EINVAL, "%s: bad batch or ranks", fn);
        SchulzArgs s{};
        s.batch = batch, s.m = m, s.n = n, s.steps = steps;
        s.a = 3.4445f, s.b = -4.7750f, s.c = 2.0315f;
        s.ldg = s.ldo = n, s.g_stride = s.out_stride = m * n;
        const std::vector<const void *> grads((size_t)(ranks > 0 ? batch * ranks : 1));
        const std::vector<float *> state((size_t)batch);
        if (ranks > 0)
            s.grads = grads.data(), s.momentum = s.master = state.data(), s.R = ranks;
        return recorded(fn, sms, text, bytes, [&] { return launch_newton_schulz(s, nullptr, 0, nullptr); });
    });
}

fsdp_status fsdp_ops_plan_linear_cross_entropy(int64_t rows, int64_t cols, int64_t vocab, int with_gradients, int aligned,
                                               int64_t piece_rows, int sms, char *text, int64_t bytes)
{
    const char *fn = "fsdp_ops_plan_linear_cross_entropy";
    return guarded(fn, [&]() -> fsdp_status {
        fsdp_status st = check_loss(fn, rows, cols, vocab, piece_rows);
        if (st != FSDP_OK)
            return st;
        if (rows < 1)
            return set_error(FSDP_EINVAL, "%s: no rows", fn);
        LossArgs a{};
        a.rows = rows, a.cols = cols, a.vocab = vocab, a.piece_rows = piece_rows;
        a.ldh = a.ldw = a.lddh = a.lddw = aligned ? ceil_to(cols, 8) : cols | 1;
        if (with_gradients)
            a.dhidden = a.dweight = reinterpret_cast<void *>(uintptr_t(256));
        return recorded(fn, sms, text, bytes, [&] { return launch_linear_cross_entropy(a, nullptr, 0, nullptr); });
    });
}

}  // extern "C"
