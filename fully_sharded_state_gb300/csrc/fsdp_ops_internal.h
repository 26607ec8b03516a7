// fsdp_ops_internal.h -- types shared by the operators' host code
// (fsdp_ops_capi.cpp) and their kernels (fsdp_norm.cu, fsdp_loss.cu,
// fsdp_muon.cu). Not part of the public ABI.
#pragma once

#include <cstdint>
#include <string>

#include "fsdp_internal.h"
#include "fsdp_ops.h"

namespace fsdp {

// What a call would launch, one line per launch, written instead of launched
// where a thread has one set: the tests ask so which kernels a call takes, on
// the host and for any number of multiprocessors.
struct Record {
    int sms;
    std::string text;
    fsdp_status add(const char *fmt, ...) __attribute__((format(printf, 2, 3)));
};
Record *&current_record();  // this thread's, or NULL

// Multiprocessors of `dev`, read once per device.
int device_sms(int dev);

inline int64_t ceil_to(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

// Splits one workspace into 256-byte aligned parts. With a null base it only
// counts, which is how the workspace queries get their sizes.
class Carver {
  public:
    explicit Carver(void *base) : base_(static_cast<char *>(base)) {}
    template <typename T>
    T *take(int64_t count)
    {
        T *p = base_ ? reinterpret_cast<T *>(base_ + used_) : nullptr;
        used_ += ceil_to(count * (int64_t)sizeof(T), 256);
        return p;
    }
    int64_t used() const { return used_; }

  private:
    char *base_;
    int64_t used_ = 0;
};

struct NormArgs {
    int64_t rows, cols;
    const void *x;
    int64_t ldx;
    const void *gamma, *beta;
    fsdp_dtype dtype, param_dtype;
    float eps;
    // forward
    void *y;
    int64_t ldy;
    float *mean, *rstd;
    // backward
    const void *dy;
    int64_t lddy;
    const float *mean_in, *rstd_in;
    void *dx;
    int64_t lddx;
    void *dgamma, *dbeta;
    float *partial;  // one line of dgamma and one of dbeta per block
};
int64_t norm_backward_workspace(int64_t rows, int64_t cols);  // bytes
fsdp_status launch_layer_norm(const NormArgs &a, int dev, void *stream);
fsdp_status launch_layer_norm_backward(const NormArgs &a, int dev, void *stream);

struct LossArgs {
    int64_t rows, cols, vocab;
    const void *hidden;
    int64_t ldh;
    const void *weight;
    int64_t ldw;
    const int64_t *targets;
    int64_t ignore_index;
    int mean;
    float grad_scale;
    float *loss, *row_loss;
    void *dhidden;  // NULL: loss alone
    int64_t lddh;
    void *dweight;
    int64_t lddw;
    int64_t piece_rows;
};
// Whether the weight's rows can be copied as they lie; else a copy of it that
// can be is part of the workspace.
inline bool loss_weight_aligned(const void *weight, int64_t ldw)
{
    return (reinterpret_cast<uintptr_t>(weight) & 15u) == 0 && ldw % 8 == 0;
}
int64_t loss_workspace(const LossArgs &a, bool grad, bool aligned_weight);  // bytes
fsdp_status launch_linear_cross_entropy(const LossArgs &a, void *workspace, int dev, void *stream);

constexpr int kMuonMaxMats = FSDP_MUON_MAX_MATRICES;
constexpr int kMuonMaxGrads = 1024;  // n_mats * R pointers of one launch

struct SchulzArgs {
    int64_t batch, m, n;
    int steps;
    float eps, a, b, c;
    // fsdp_newton_schulz
    const void *g;
    int64_t ldg, g_stride;
    fsdp_dtype dtype;
    void *out;
    int64_t ldo, out_stride;
    // fsdp_muon (grads != NULL)
    const void *const *grads;
    int R;
    float *const *momentum;
    float *const *master;
    void *const *param_out;
    float mu, decay, lr;  // lr includes update_scale
    int nesterov;
};
int64_t schulz_workspace(int64_t batch, int64_t m, int64_t n, bool muon);  // bytes
fsdp_status launch_newton_schulz(const SchulzArgs &a, void *workspace, int dev, void *stream);

// The launches of a call of these sizes on `sms` multiprocessors, as text (at
// most `bytes` of it, its end included). ranks > 0: a Muon step. aligned: the
// caller's matrices start on 16 bytes and so do their rows.
extern "C" {
fsdp_status fsdp_ops_plan_newton_schulz(int64_t batch, int64_t m, int64_t n, int ranks, int steps, int sms, char *text,
                                        int64_t bytes);
fsdp_status fsdp_ops_plan_linear_cross_entropy(int64_t rows, int64_t cols, int64_t vocab, int with_gradients, int aligned,
                                               int64_t piece_rows, int sms, char *text, int64_t bytes);
}

}  // namespace fsdp
