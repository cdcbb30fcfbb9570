// api_ops.cu -- the C ABI of the operators around the memory (convolution, q/k norm, selective
// scan), declared in include/falcon.h: host-side argument checks and status codes.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "launch.h"
#include "ops.h"

namespace falcon {
namespace {

constexpr int kMaxTokens = 1 << 30;
constexpr long long kMaxSpan = 1LL << 50;   // elements: addresses stay far inside 64 bits

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t elem_size(int io) { return io == FALCON_BF16 ? 2 : 4; }

// Sizes common to all: nonnegative, and products that 64 (heads: 31) bits hold.
falcon_status_t check_sizes(int io, int B, long long heads, int T, int d) {
    if (io != FALCON_F32 && io != FALCON_BF16) return FALCON_ERR_INVALID_ARG;
    if (B < 0 || heads < 0 || T < 0 || d <= 0) return FALCON_ERR_INVALID_ARG;
    if (T > kMaxTokens || heads > 0x7fffffffLL || (long long)B * heads > 0x7fffffffLL) return FALCON_ERR_UNSUPPORTED;
    if (heads * d > 0x7fffffffLL) return FALCON_ERR_UNSUPPORTED;
    if ((long long)B * heads > 0 && (long long)B * heads * d > kMaxSpan / (T > 0 ? T : 1)) return FALCON_ERR_UNSUPPORTED;
    return FALCON_OK;
}

// A view of B x H x T rows of d elements of es bytes; `out`: its rows must not overlap.
falcon_status_t check_view(const falcon_view_t &v, int B, int H, int T, int d, size_t es, bool out) {
    if ((long long)B * H * T == 0) return FALCON_OK;   // nothing is read or written
    if (!v.p || !aligned(v.p, es)) return FALCON_ERR_INVALID_ARG;
    if (v.sb < 0 || v.sh < 0 || v.st < 0) return FALCON_ERR_INVALID_ARG;
    const long long size[3] = {B, H, T}, stride[3] = {v.sb, v.sh, v.st};
    long long span = d;
    for (int i = 0; i < 3; ++i) {
        if (size[i] > 1 && stride[i] > kMaxSpan / (size[i] - 1)) return FALCON_ERR_UNSUPPORTED;
        span += (size[i] - 1) * (size[i] > 1 ? stride[i] : 0);
    }
    if (span > kMaxSpan) return FALCON_ERR_UNSUPPORTED;
    if (!out) return FALCON_OK;
    // ascending by stride, each axis has to step over everything below it
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (stride[order[j]] > stride[order[j + 1]]) {
                const int x = order[j];
                order[j] = order[j + 1];
                order[j + 1] = x;
            }
    long long extent = d;
    for (int i = 0; i < 3; ++i) {
        const int x = order[i];
        if (size[x] <= 1) continue;
        if (stride[x] < extent) return FALCON_ERR_INVALID_ARG;
        extent += (size[x] - 1) * stride[x];
    }
    return FALCON_OK;
}

// Where `rows` rows of a view start, NULL where there is none.
const void *start(const falcon_view_t &v, long long rows) { return rows > 0 ? v.p : nullptr; }

// No output starts where another one or an input does (what overlaps in another way is not seen here).
bool apart(std::initializer_list<const void *> outs, std::initializer_list<const void *> ins) {
    for (const void *const *o = outs.begin(); o != outs.end(); ++o) {
        if (!*o) continue;
        for (const void *const *p = outs.begin(); p != o; ++p)
            if (*p == *o) return false;
        for (const void *i : ins)
            if (i == *o) return false;
    }
    return true;
}

// Parameters, lengths and states: device arrays of 4-byte elements (or io elements of es bytes).
bool ok_array(const void *p, bool required, size_t es = 4) { return p ? aligned(p, es) : !required; }

#define FALCON_TRY(x)                                   \
    do {                                                \
        const falcon_status_t st_ = (x);                \
        if (st_ != FALCON_OK) return st_;               \
    } while (0)
#define FALCON_NEED(x)                                  \
    do {                                                \
        if (!(x)) return FALCON_ERR_INVALID_ARG;        \
    } while (0)

falcon_status_t status_of(cudaError_t e) {
    if (e == cudaSuccess) return FALCON_OK;
    return e == cudaErrorInvalidConfiguration ? FALCON_ERR_UNSUPPORTED : FALCON_ERR_CUDA;
}

falcon_status_t check_workspace(void *ws, size_t bytes, size_t need) {
    if (need == 0) return FALCON_OK;
    if (!ws || bytes < need) return FALCON_ERR_WORKSPACE;
    return aligned(ws, 16) ? FALCON_OK : FALCON_ERR_INVALID_ARG;
}

// Fails where there is no device to launch on.
falcon_status_t device(int *sms) {
    int *err = nullptr;
    return device_info(&err, sms) ? FALCON_OK : FALCON_ERR_CUDA;
}

// ---- convolution

falcon_status_t check_conv(const falcon_conv_args_t *a) {
    FALCON_NEED(a);
    FALCON_TRY(check_sizes(a->io_dtype, a->B, a->H, a->T, a->d));
    FALCON_NEED(a->K >= 1 && (a->act == FALCON_ACT_NONE || a->act == FALCON_ACT_SILU));
    if (a->K > 8) return FALCON_ERR_UNSUPPORTED;
    const size_t es = elem_size(a->io_dtype);
    FALCON_TRY(check_view(a->x, a->B, a->H, a->T, a->d, es, false));
    FALCON_NEED(ok_array(a->w, (long long)a->B * a->H > 0) && ok_array(a->bias, false) && ok_array(a->lengths, false));
    FALCON_NEED(ok_array(a->state, false, es));
    return FALCON_OK;
}

falcon_status_t check_conv_out(const falcon_conv_args_t *a) {
    const size_t es = elem_size(a->io_dtype);
    FALCON_TRY(check_view(a->y, a->B, a->H, a->T, a->d, es, true));
    FALCON_NEED(ok_array(a->state_out, false, es));
    FALCON_NEED(!a->y.p || a->y.p != a->x.p);   // a row is read again after its successors are written
    const long long rows = (long long)a->B * a->H * a->T, tail = (long long)a->B * a->H * (a->K - 1);
    const void *const state_out = tail > 0 ? a->state_out : nullptr;
    FALCON_NEED(apart({start(a->y, rows), state_out}, {start(a->x, rows)}));
    FALCON_NEED(apart({start(a->y, rows)}, {tail > 0 ? a->state : nullptr}));   // state_out may be state
    return FALCON_OK;
}

// ---- scan

constexpr int kMaxChannels = 0x7fffffff - 511;   // channel numbers of a block that dv does not fill stay in 31 bits

// The scan's kernels take token strides of up to 2^28 elements (32 bits of bytes).
bool far_tokens(const falcon_view_t &v, int T) { return v.p && T > 1 && v.st > (1LL << 28); }

falcon_status_t check_scan(const falcon_scan_args_t *a) {
    FALCON_NEED(a);
    FALCON_NEED(a->dk > 0);
    FALCON_TRY(check_sizes(a->io_dtype, a->B, a->H, a->T, a->dv));
    if (a->dk > 128 || a->dv > kMaxChannels) return FALCON_ERR_UNSUPPORTED;
    FALCON_TRY(check_sizes(a->io_dtype, a->B, a->H, a->T, a->dk));
    if ((long long)a->B * a->H * a->dv > kMaxSpan / a->dk) return FALCON_ERR_UNSUPPORTED;
    FALCON_NEED((a->flags & ~FALCON_SCAN_SOFTPLUS) == 0);
    const size_t es = elem_size(a->io_dtype);
    FALCON_TRY(check_view(a->q, a->B, a->H, a->T, a->dk, es, false));
    FALCON_TRY(check_view(a->k, a->B, a->H, a->T, a->dk, es, false));
    FALCON_TRY(check_view(a->v, a->B, a->H, a->T, a->dv, es, false));
    FALCON_TRY(check_view(a->delta, a->B, a->H, a->T, a->dv, es, false));
    if (a->z.p) FALCON_TRY(check_view(a->z, a->B, a->H, a->T, a->dv, es, false));
    if (far_tokens(a->v, a->T) || far_tokens(a->delta, a->T) || far_tokens(a->z, a->T)) return FALCON_ERR_UNSUPPORTED;
    FALCON_NEED(ok_array(a->A, (long long)a->B * a->H > 0) && ok_array(a->D, false) && ok_array(a->delta_bias, false));
    FALCON_NEED(ok_array(a->lengths, false) && ok_array(a->S0, false));
    return FALCON_OK;
}

falcon_status_t check_scan_out(const falcon_scan_args_t *a) {
    FALCON_TRY(check_view(a->o, a->B, a->H, a->T, a->dv, elem_size(a->io_dtype), true));
    if (far_tokens(a->o, a->T)) return FALCON_ERR_UNSUPPORTED;
    FALCON_NEED(ok_array(a->S_out, false));
    const long long rows = (long long)a->B * a->H * a->T;   // other blocks still read q and k of a token that is written
    FALCON_NEED(apart({start(a->o, rows), a->S_out}, {start(a->q, rows), start(a->k, rows), start(a->v, rows),
                                                      start(a->delta, rows), start(a->z, rows)}));
    FALCON_NEED(apart({start(a->o, rows)}, {a->S0}));       // S_out may be S0
    return FALCON_OK;
}

// ---- q/k norm

falcon_status_t check_qknorm(const falcon_qknorm_args_t *a) {
    FALCON_NEED(a);
    FALCON_NEED(a->Hq >= 0 && a->Hk >= 0);
    FALCON_TRY(check_sizes(a->io_dtype, a->B, (long long)a->Hq + a->Hk, a->T, a->d));
    FALCON_NEED(a->norm >= FALCON_NORM_NONE && a->norm <= FALCON_NORM_L2);
    FALCON_NEED(a->rot_layout == FALCON_ROT_HALF || a->rot_layout == FALCON_ROT_PAIRS);
    FALCON_NEED(a->rot >= 0 && a->rot % 2 == 0 && a->rot <= a->d);
    FALCON_NEED(a->eps >= 0.f && isfinite(a->eps));
    if (a->Hq > 65536 || a->Hk > 65536) return FALCON_ERR_UNSUPPORTED;   // rows of a group of tokens: 32 bits
    if (a->d > 256) return FALCON_ERR_UNSUPPORTED;
    const size_t es = elem_size(a->io_dtype);
    FALCON_TRY(check_view(a->q, a->B, a->Hq, a->T, a->d, es, false));
    FALCON_TRY(check_view(a->k, a->B, a->Hk, a->T, a->d, es, false));
    FALCON_NEED(ok_array(a->wq, false) && ok_array(a->wk, false) && ok_array(a->lengths, false));
    const bool any = (long long)a->B * a->T * (a->Hq + a->Hk) > 0;
    FALCON_NEED(ok_array(a->freq, a->rot > 0 && any) && ok_array(a->positions, false));
    return FALCON_OK;
}

// In place: the same memory in the same order (the stride of an axis of one does not count), or nothing at all.
bool same_place(const falcon_view_t &x, const falcon_view_t &y, int B, int H, int T) {
    if ((long long)B * H * T == 0) return true;
    return x.p != y.p || ((B == 1 || x.sb == y.sb) && (H == 1 || x.sh == y.sh) && (T == 1 || x.st == y.st));
}

falcon_status_t check_qknorm_out(const falcon_qknorm_args_t *a) {
    const size_t es = elem_size(a->io_dtype);
    FALCON_TRY(check_view(a->q_out, a->B, a->Hq, a->T, a->d, es, true));
    FALCON_TRY(check_view(a->k_out, a->B, a->Hk, a->T, a->d, es, true));
    FALCON_NEED(same_place(a->q, a->q_out, a->B, a->Hq, a->T) && same_place(a->k, a->k_out, a->B, a->Hk, a->T));
    const long long tokens = (long long)a->B * a->T;
    const void *const q = start(a->q, tokens * a->Hq), *const k = start(a->k, tokens * a->Hk);
    const void *const q_out = start(a->q_out, tokens * a->Hq), *const k_out = start(a->k_out, tokens * a->Hk);
    FALCON_NEED(apart({q_out, k_out}, {}) && apart({q_out}, {k}) && apart({k_out}, {q}));
    return FALCON_OK;
}

}  // namespace
}  // namespace falcon

using namespace falcon;

extern "C" {

falcon_status_t falcon_conv_fwd(const falcon_conv_args_t *a, falcon_stream_t stream) {
    FALCON_TRY(check_conv(a));
    FALCON_TRY(check_conv_out(a));
    if ((long long)a->B * a->H == 0) return FALCON_OK;
    int sms = 0;
    FALCON_TRY(device(&sms));
    return status_of(launch_conv_fwd(*a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

falcon_status_t falcon_conv_step(const falcon_conv_args_t *a, falcon_stream_t stream) {
    FALCON_TRY(check_conv(a));
    FALCON_TRY(check_conv_out(a));
    FALCON_NEED(a->T == 1 && !a->lengths);
    if ((long long)a->B * a->H == 0) return FALCON_OK;
    FALCON_NEED(a->K == 1 || (a->state && a->state_out));
    int sms = 0;
    FALCON_TRY(device(&sms));
    return status_of(launch_conv_step(*a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t falcon_conv_bwd_workspace_size(const falcon_conv_args_t *a) {
    return check_conv(a) == FALCON_OK ? conv_bwd_workspace(*a) : 0;
}

falcon_status_t falcon_conv_bwd(const falcon_conv_args_t *a, const falcon_conv_grads_t *g, void *workspace,
                                size_t workspace_bytes, falcon_stream_t stream) {
    FALCON_TRY(check_conv(a));
    FALCON_NEED(g);
    FALCON_TRY(check_view(g->dy, a->B, a->H, a->T, a->d, 4, false));
    FALCON_TRY(check_view(g->dx, a->B, a->H, a->T, a->d, 4, true));
    FALCON_NEED(!g->dx.p || g->dx.p != g->dy.p);
    FALCON_NEED(ok_array(g->dw, a->H > 0) && ok_array(g->dbias, false) && ok_array(g->dstate_out, false) &&
                ok_array(g->dstate, false));
    const long long rows = (long long)a->B * a->H * a->T;
    const bool tail = (long long)a->B * a->H * (a->K - 1) > 0;
    FALCON_NEED(apart({start(g->dx, rows), g->dw, g->dbias, tail ? g->dstate : nullptr},
                      {start(a->x, rows), start(g->dy, rows), tail ? a->state : nullptr, tail ? g->dstate_out : nullptr}));
    if (a->H == 0) return FALCON_OK;
    FALCON_TRY(check_workspace(workspace, workspace_bytes, conv_bwd_workspace(*a)));
    int sms = 0;
    FALCON_TRY(device(&sms));
    return status_of(launch_conv_bwd(*a, *g, static_cast<float *>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

size_t falcon_scan_workspace_size(const falcon_scan_args_t *a) {
    int sms = 0;
    if (check_scan(a) != FALCON_OK || device(&sms) != FALCON_OK) return 0;
    return scan_plan(*a, sms).bytes;
}

falcon_status_t falcon_scan_fwd(const falcon_scan_args_t *a, void *workspace, size_t workspace_bytes,
                                falcon_stream_t stream) {
    FALCON_TRY(check_scan(a));
    FALCON_TRY(check_scan_out(a));
    if ((long long)a->B * a->H == 0) return FALCON_OK;
    int sms = 0;
    FALCON_TRY(device(&sms));
    ScanPlan plan = scan_plan(*a, sms);
    if (plan.bytes && workspace && workspace_bytes >= plan.bytes) {
        FALCON_NEED(aligned(workspace, 16));
    } else {
        plan = ScanPlan{};
        plan.seg = a->T;
    }
    return status_of(launch_scan_fwd(*a, plan, static_cast<float *>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

falcon_status_t falcon_scan_step(const falcon_scan_args_t *a, falcon_stream_t stream) {
    FALCON_TRY(check_scan(a));
    FALCON_TRY(check_scan_out(a));
    FALCON_NEED(a->T == 1 && !a->lengths);
    if ((long long)a->B * a->H == 0) return FALCON_OK;
    FALCON_NEED(a->S0 && a->S_out);
    int sms = 0;
    FALCON_TRY(device(&sms));
    return status_of(launch_scan_step(*a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t falcon_scan_bwd_workspace_size(const falcon_scan_args_t *a) {
    return check_scan(a) == FALCON_OK ? scan_bwd_workspace(*a) : 0;
}

falcon_status_t falcon_scan_bwd(const falcon_scan_args_t *a, const falcon_scan_grads_t *g, void *workspace,
                                size_t workspace_bytes, falcon_stream_t stream) {
    FALCON_TRY(check_scan(a));
    FALCON_NEED(g);
    FALCON_TRY(check_view(g->dO, a->B, a->H, a->T, a->dv, 4, false));
    FALCON_TRY(check_view(g->dq, a->B, a->H, a->T, a->dk, 4, true));
    FALCON_TRY(check_view(g->dk, a->B, a->H, a->T, a->dk, 4, true));
    FALCON_TRY(check_view(g->dv, a->B, a->H, a->T, a->dv, 4, true));
    FALCON_TRY(check_view(g->ddelta, a->B, a->H, a->T, a->dv, 4, true));
    if (far_tokens(g->dO, a->T)) return FALCON_ERR_UNSUPPORTED;
    if (g->dz.p) {
        FALCON_NEED(a->z.p);
        FALCON_TRY(check_view(g->dz, a->B, a->H, a->T, a->dv, 4, true));
    }
    FALCON_NEED(ok_array(g->dS_T, false) && ok_array(g->dA, a->H > 0) && ok_array(g->dD, false) &&
                ok_array(g->ddelta_bias, false) && ok_array(g->dS0, false));
    const long long rows = (long long)a->B * a->H * a->T;
    const void *const dS0 = a->B > 0 ? g->dS0 : nullptr;
    FALCON_NEED(apart({start(g->dq, rows), start(g->dk, rows), start(g->dv, rows), start(g->ddelta, rows), start(g->dz, rows),
                       g->dA, g->dD, g->ddelta_bias, dS0},
                      {start(g->dO, rows), start(a->q, rows), start(a->k, rows), start(a->v, rows), start(a->delta, rows),
                       start(a->z, rows), a->S0}));
    if (a->H == 0) return FALCON_OK;
    if (!scan_bwd_fits(*a)) return FALCON_ERR_UNSUPPORTED;
    FALCON_TRY(check_workspace(workspace, workspace_bytes, scan_bwd_workspace(*a)));
    int sms = 0;
    FALCON_TRY(device(&sms));
    return status_of(launch_scan_bwd(*a, *g, static_cast<float *>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

falcon_status_t falcon_qknorm_fwd(const falcon_qknorm_args_t *a, falcon_stream_t stream) {
    FALCON_TRY(check_qknorm(a));
    FALCON_TRY(check_qknorm_out(a));
    if ((long long)a->B * a->T * (a->Hq + a->Hk) == 0) return FALCON_OK;
    int sms = 0;
    FALCON_TRY(device(&sms));
    return status_of(launch_qknorm_fwd(*a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t falcon_qknorm_bwd_workspace_size(const falcon_qknorm_args_t *a) {
    return check_qknorm(a) == FALCON_OK ? qknorm_bwd_workspace(*a) : 0;
}

falcon_status_t falcon_qknorm_bwd(const falcon_qknorm_args_t *a, const falcon_qknorm_grads_t *g, void *workspace,
                                  size_t workspace_bytes, falcon_stream_t stream) {
    FALCON_TRY(check_qknorm(a));
    FALCON_NEED(g);
    FALCON_TRY(check_view(g->dq_out, a->B, a->Hq, a->T, a->d, 4, false));
    FALCON_TRY(check_view(g->dk_out, a->B, a->Hk, a->T, a->d, 4, false));
    FALCON_TRY(check_view(g->dq, a->B, a->Hq, a->T, a->d, 4, true));
    FALCON_TRY(check_view(g->dk, a->B, a->Hk, a->T, a->d, 4, true));
    FALCON_NEED(same_place(g->dq, g->dq_out, a->B, a->Hq, a->T) && same_place(g->dk, g->dk_out, a->B, a->Hk, a->T));
    const long long tokens = (long long)a->B * a->T;
    const void *const q = start(a->q, tokens * a->Hq), *const k = start(a->k, tokens * a->Hk);
    const void *const q_up = start(g->dq_out, tokens * a->Hq), *const k_up = start(g->dk_out, tokens * a->Hk);
    const void *const dq = start(g->dq, tokens * a->Hq), *const dk = start(g->dk, tokens * a->Hk);
    FALCON_NEED(apart({dq, dk, g->dwq, g->dwk}, {q, k}) && apart({dq}, {k_up}) && apart({dk}, {q_up}));
    FALCON_NEED(ok_array(g->dwq, false) && ok_array(g->dwk, false));
    if (g->dwq || g->dwk) FALCON_TRY(check_workspace(workspace, workspace_bytes, qknorm_bwd_workspace(*a)));
    int sms = 0;
    FALCON_TRY(device(&sms));
    return status_of(launch_qknorm_bwd(*a, *g, static_cast<float *>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
