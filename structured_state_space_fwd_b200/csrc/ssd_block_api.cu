// C ABI of the operators around the layer: the short causal convolution and the
// selective scan with a diagonal A. Host-side argument checks only; every call is
// one kernel launch on the caller's stream, and nothing here allocates or waits.
#include <cuda_runtime.h>

#include <cstdio>
#include <initializer_list>

#include "ssd.h"
#include "ssd_internal.h"

namespace {

using ssd::aligned;
using ssd::overlaps;
using ssd::Range;

constexpr int64_t kMaxDocs = 1 << 24;
constexpr int64_t kMaxTokens = 0x7fff0000;   // tokens and rows of the scan's kernels are 32-bit
constexpr int64_t kMaxRow = 0x7fffffff;      // numbers, so that an offset is one 32 x 32 product
constexpr double kMaxElems = 4.0e15;      // keeps every element index well inside int64

size_t elem_size(int dtype) { return dtype == SSD_BF16 ? 2 : 4; }
bool dtype_ok(int dtype) { return dtype == SSD_F32 || dtype == SSD_BF16; }

ssd_status_t cuda_status(const char* what, cudaError_t e) {
    if (e == cudaSuccess) return SSD_OK;
    if (e == cudaErrorInvalidConfiguration) return SSD_ERR_UNSUPPORTED;   // more blocks than a grid has
    char msg[256];
    snprintf(msg, sizeof(msg), "%s: %s (%d)", what, cudaGetErrorString(e), (int)e);
    ssd::set_error_detail(msg);
    return SSD_ERR_CUDA;
}

bool stride_ok(const ssd_strides_t& s, int64_t b, int64_t T) {
    if (s.batch < 0 || s.row < 0) return false;
    return (double)s.batch * (double)b + (double)s.row * (double)T <= kMaxElems;
}
// Bytes from the first to behind the last element of an input of b x T rows of n elements.
size_t span(const ssd_strides_t& s, int64_t b, int64_t T, int64_t n, size_t es) {
    if (b == 0 || T == 0) return 0;
    return (size_t)((b - 1) * s.batch + (T - 1) * s.row + n) * es;
}

// Outputs overlap no input and no other output.
bool disjoint(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range* o = outs.begin(); o != outs.end(); ++o) {
        for (const Range& i : ins)
            if (overlaps(*o, i)) return false;
        for (const Range* p = outs.begin(); p != o; ++p)
            if (overlaps(*o, *p)) return false;
    }
    return true;
}

ssd_status_t check_docs(int64_t batch, int64_t T, int64_t n_docs, const int32_t* cu) {
    if (batch != 1 || n_docs < 0 || (n_docs == 0 && T != 0)) return SSD_ERR_INVALID_ARG;
    if (n_docs > kMaxDocs || T > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
    if (n_docs > 0 && (!cu || !aligned(cu, 4))) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

ssd_status_t check_conv_shape(const ssd_conv_shape_t* s) {
    if (!s) return SSD_ERR_INVALID_ARG;
    if (s->batch < 0 || s->seqlen < 0 || s->channels < 1 || s->width < 1) return SSD_ERR_INVALID_ARG;
    if (!dtype_ok(s->dtype) || (s->silu != 0 && s->silu != 1)) return SSD_ERR_INVALID_ARG;
    if ((double)s->batch * (double)s->seqlen * (double)s->channels > kMaxElems ||
        (double)s->batch * (double)s->channels * 4.0 > kMaxElems || s->channels > (1LL << 40))
        return SSD_ERR_UNSUPPORTED;
    int64_t sum = 0;
    for (int64_t c : s->out_channels) {
        if (c < 0 || c > s->channels) return SSD_ERR_INVALID_ARG;
        sum += c;
    }
    if (sum != s->channels) return SSD_ERR_INVALID_ARG;
    if (s->width < 2 || s->width > 4) return SSD_ERR_UNSUPPORTED;
    if (!stride_ok(s->u, s->batch, s->seqlen)) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

// Shared by the three convolution entries; `init` and `fin` are [nseq, W-1, C] (the step's state is `fin`).
ssd_status_t check_conv(const ssd_conv_shape_t* s, int64_t nseq, const void* u, const float* weight,
                        const float* bias, const int32_t* cu, const void* init, void* const* y, void* fin,
                        ssd::ConvArgs* a) {
    const size_t es = elem_size(s->dtype);
    const size_t zu = span(s->u, s->batch, s->seqlen, s->channels, es);
    const size_t zst = (size_t)(nseq * (s->width - 1) * s->channels) * es;
    size_t zy[3];
    for (int i = 0; i < 3; ++i) {
        zy[i] = (size_t)(s->batch * s->seqlen * s->out_channels[i]) * es;
        if (zy[i] && !y[i]) return SSD_ERR_INVALID_ARG;
        if (!aligned(y[i], es)) return SSD_ERR_INVALID_ARG;
    }
    if ((zu && !u) || !weight) return SSD_ERR_INVALID_ARG;
    if (!aligned(u, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(init, es) || !aligned(fin, es))
        return SSD_ERR_INVALID_ARG;
    if (!disjoint({{y[0], zy[0]}, {y[1], zy[1]}, {y[2], zy[2]}, {fin, zst}},
                  {{u, zu}, {weight, (size_t)(s->channels * s->width) * 4}, {bias, (size_t)s->channels * 4},
                   {init, zst}, {cu, cu ? (size_t)(nseq + 1) * 4 : 0}}))
        return SSD_ERR_INVALID_ARG;
    *a = ssd::ConvArgs{};
    a->b = s->batch; a->T = s->seqlen; a->C = s->channels; a->nseq = nseq;
    for (int i = 0; i < 3; ++i) {
        a->oc[i] = s->out_channels[i];
        a->y[i] = y[i];
    }
    a->ub = s->u.batch; a->ur = s->u.row;
    a->W = (int)s->width; a->dtype = s->dtype; a->silu = s->silu;
    a->u = u; a->weight = weight; a->bias = bias; a->cu = cu;
    a->init = init; a->final_states = fin;
    return SSD_OK;
}

ssd_status_t check_selective_shape(const ssd_selective_shape_t* s) {
    if (!s) return SSD_ERR_INVALID_ARG;
    if (s->reserved != 0 || s->batch < 0 || s->seqlen < 0 || s->channels < 1 || s->ngroups < 1 || s->dstate < 1)
        return SSD_ERR_INVALID_ARG;
    if (s->channels % s->ngroups != 0) return SSD_ERR_INVALID_ARG;
    if (!dtype_ok(s->dtype) || !dtype_ok(s->dt_dtype) || (s->dt_dtype != SSD_F32 && s->dt_dtype != s->dtype) ||
        (s->dt_softplus != 0 && s->dt_softplus != 1))
        return SSD_ERR_INVALID_ARG;
    if (s->dstate > ssd::kMaxSelectiveStates || s->seqlen > kMaxTokens) return SSD_ERR_UNSUPPORTED;
    if ((double)s->batch * (double)s->seqlen * (double)s->channels > kMaxElems ||
        (double)s->batch * (double)s->seqlen * (double)s->ngroups * (double)s->dstate > kMaxElems ||
        (double)s->batch * (double)s->channels * (double)s->dstate > kMaxElems)
        return SSD_ERR_UNSUPPORTED;
    if (s->channels > kMaxRow) return SSD_ERR_UNSUPPORTED;
    for (const ssd_strides_t* p : {&s->u, &s->dt, &s->B, &s->C}) {
        if (!stride_ok(*p, s->batch, s->seqlen)) return SSD_ERR_INVALID_ARG;
        if (s->seqlen > 1 && p->row > kMaxRow) return SSD_ERR_UNSUPPORTED;
    }
    return SSD_OK;
}

// Shared by the three scan entries. in_place: init and fin are the one state.
ssd_status_t check_selective(const ssd_selective_shape_t* s, int64_t nseq, const void* u, const void* dt,
                             const float* A, const void* B, const void* C, const float* D, const void* z,
                             const float* dt_bias, const int32_t* cu, const float* init, void* y, float* fin,
                             bool in_place, ssd::SelectiveArgs* a) {
    if (z && !stride_ok(s->z, s->batch, s->seqlen)) return SSD_ERR_INVALID_ARG;
    if (z && s->seqlen > 1 && s->z.row > kMaxRow) return SSD_ERR_UNSUPPORTED;
    const size_t es = elem_size(s->dtype), des = elem_size(s->dt_dtype);
    const int64_t b = s->batch, T = s->seqlen, Dc = s->channels, GN = s->ngroups * s->dstate;
    const size_t zu = span(s->u, b, T, Dc, es), zdt = span(s->dt, b, T, Dc, des);
    const size_t zz = z ? span(s->z, b, T, Dc, es) : 0;
    const size_t zB = span(s->B, b, T, GN, es), zC = span(s->C, b, T, GN, es);
    const size_t zy = (size_t)(b * T * Dc) * es, zst = (size_t)(nseq * Dc * s->dstate) * 4;
    if ((zu && (!u || !dt || !B || !C || !y)) || !A) return SSD_ERR_INVALID_ARG;
    if (!aligned(u, es) || !aligned(dt, des) || !aligned(z, es) || !aligned(B, es) || !aligned(C, es) ||
        !aligned(y, es) || !aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(init, 4) ||
        !aligned(fin, 4))
        return SSD_ERR_INVALID_ARG;
    if (!disjoint({{y, zy}, {fin, zst}},
                  {{u, zu}, {dt, zdt}, {z, zz}, {B, zB}, {C, zC}, {A, (size_t)(Dc * s->dstate) * 4},
                   {D, (size_t)Dc * 4}, {dt_bias, (size_t)Dc * 4}, {init, in_place ? 0 : zst},
                   {cu, cu ? (size_t)(nseq + 1) * 4 : 0}}))
        return SSD_ERR_INVALID_ARG;
    *a = ssd::SelectiveArgs{};
    a->b = b; a->T = T; a->D = Dc; a->G = s->ngroups; a->N = s->dstate; a->nseq = nseq;
    a->us = s->u; a->dts = s->dt; a->zs = s->z; a->Bs = s->B; a->Cs = s->C;
    a->dtype = s->dtype; a->dt_dtype = s->dt_dtype; a->softplus = s->dt_softplus;
    a->u = u; a->dt = dt; a->A = A; a->B = B; a->C = C; a->Dskip = D; a->z = z; a->dt_bias = dt_bias;
    a->cu = cu; a->init = init; a->y = y; a->fin = fin;
    return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status_t ssd_causal_conv1d(const ssd_conv_shape_t* shape, const void* u, const float* weight,
                               const float* bias, const void* initial_states, void* y0, void* y1, void* y2,
                               void* final_states, void* stream) {
    ssd_status_t st = check_conv_shape(shape);
    if (st != SSD_OK) return st;
    ssd::ConvArgs a;
    void* y[3] = {y0, y1, y2};
    if ((st = check_conv(shape, shape->batch, u, weight, bias, nullptr, initial_states, y, final_states, &a)) !=
        SSD_OK)
        return st;
    return cuda_status("causal convolution", ssd::launch_conv(a, (cudaStream_t)stream));
}

ssd_status_t ssd_causal_conv1d_varlen(const ssd_conv_shape_t* shape, const void* u, const float* weight,
                                      const float* bias, const int32_t* cu_seqlens, int64_t n_docs,
                                      const void* initial_states, void* y0, void* y1, void* y2,
                                      void* final_states, void* stream) {
    ssd_status_t st = check_conv_shape(shape);
    if (st != SSD_OK) return st;
    if ((st = check_docs(shape->batch, shape->seqlen, n_docs, cu_seqlens)) != SSD_OK) return st;
    if ((double)n_docs * (double)shape->channels * 4.0 > kMaxElems) return SSD_ERR_UNSUPPORTED;
    if (n_docs == 0) return SSD_OK;
    ssd::ConvArgs a;
    void* y[3] = {y0, y1, y2};
    if ((st = check_conv(shape, n_docs, u, weight, bias, cu_seqlens, initial_states, y, final_states, &a)) !=
        SSD_OK)
        return st;
    return cuda_status("causal convolution (packed documents)", ssd::launch_conv(a, (cudaStream_t)stream));
}

ssd_status_t ssd_causal_conv1d_step(const ssd_conv_shape_t* shape, const void* u, const float* weight,
                                    const float* bias, void* state, void* y0, void* y1, void* y2, void* stream) {
    ssd_status_t st = check_conv_shape(shape);
    if (st != SSD_OK) return st;
    if (!state && shape->batch > 0) return SSD_ERR_INVALID_ARG;
    ssd::ConvArgs a;
    void* y[3] = {y0, y1, y2};
    if ((st = check_conv(shape, shape->batch, u, weight, bias, nullptr, nullptr, y, state, &a)) != SSD_OK) return st;
    return cuda_status("causal convolution step", ssd::launch_conv_step(a, state, (cudaStream_t)stream));
}

ssd_status_t ssd_selective_scan(const ssd_selective_shape_t* shape, const void* u, const void* dt, const float* A,
                                const void* B, const void* C, const float* D, const void* z, const float* dt_bias,
                                const float* initial_states, void* y, float* final_states, void* stream) {
    ssd_status_t st = check_selective_shape(shape);
    if (st != SSD_OK) return st;
    ssd::SelectiveArgs a;
    if ((st = check_selective(shape, shape->batch, u, dt, A, B, C, D, z, dt_bias, nullptr, initial_states, y,
                              final_states, false, &a)) != SSD_OK)
        return st;
    return cuda_status("selective scan", ssd::launch_selective_scan(a, (cudaStream_t)stream));
}

ssd_status_t ssd_selective_scan_varlen(const ssd_selective_shape_t* shape, const void* u, const void* dt,
                                       const float* A, const void* B, const void* C, const float* D, const void* z,
                                       const float* dt_bias, const int32_t* cu_seqlens, int64_t n_docs,
                                       const float* initial_states, void* y, float* final_states, void* stream) {
    ssd_status_t st = check_selective_shape(shape);
    if (st != SSD_OK) return st;
    if ((st = check_docs(shape->batch, shape->seqlen, n_docs, cu_seqlens)) != SSD_OK) return st;
    if ((double)n_docs * (double)shape->channels * (double)shape->dstate > kMaxElems) return SSD_ERR_UNSUPPORTED;
    if (n_docs == 0) return SSD_OK;
    ssd::SelectiveArgs a;
    if ((st = check_selective(shape, n_docs, u, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_states, y,
                              final_states, false, &a)) != SSD_OK)
        return st;
    return cuda_status("selective scan (packed documents)", ssd::launch_selective_scan(a, (cudaStream_t)stream));
}

ssd_status_t ssd_selective_step(const ssd_selective_shape_t* shape, const void* u, const void* dt, const float* A,
                                const void* B, const void* C, const float* D, const void* z, const float* dt_bias,
                                float* state, void* y, void* stream) {
    ssd_status_t st = check_selective_shape(shape);
    if (st != SSD_OK) return st;
    if (!state && shape->batch > 0) return SSD_ERR_INVALID_ARG;
    ssd::SelectiveArgs a;
    if ((st = check_selective(shape, shape->batch, u, dt, A, B, C, D, z, dt_bias, nullptr, state, y, state, true,
                              &a)) != SSD_OK)
        return st;
    return cuda_status("selective step", ssd::launch_selective_step(a, (cudaStream_t)stream));
}

}  // extern "C"
