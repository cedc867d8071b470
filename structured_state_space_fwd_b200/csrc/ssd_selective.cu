// Selective scan with a diagonal A: the recurrence of Knowl 3's general form with a
// diagonal transition ("Transformers are SSMs: Generalized Models and Efficient
// Algorithms Through Structured State Space Duality"). Per sequence, channel d
// (group g) and state n:
//
//     h_t[n] = exp(dt_t A[n]) h_{t-1}[n] + dt_t u_t B_t[n],   y_t = sum_n C_t[n] h_t[n] + D u_t
//
// and y_t *= SiLU(z_t) with a gate. One warp per channel, the states over its lanes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_block.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kWarps = 4;
constexpr int kPieces = 8;       // states of a lane: up to 256 over 32 lanes

template <typename E, typename Td>
__global__ void __launch_bounds__(kWarps * 32) selective_kernel(const SelectiveArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t idx = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t seq = idx / a.D, d = idx % a.D;
    if (seq >= a.nseq) return;
    int64_t t0 = 0, t1 = a.T, b = seq;
    if (a.cu) {
        b = 0;
        t0 = min((int64_t)max(a.cu[seq], 0), a.T);
        t1 = min((int64_t)max(a.cu[seq + 1], 0), a.T);
    }
    const int64_t g = d / (a.D / a.G);
    const int N = (int)a.N;
    float h[kPieces], A[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const int n = lane + 32 * k;
        A[k] = n < N ? a.A[d * N + n] * kLog2e : 0.f;
        h[k] = n < N && a.init ? a.init[(seq * a.D + d) * N + n] : 0.f;
    }
    const float D = a.Dskip ? a.Dskip[d] : 0.f, bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    for (int64_t t = t0; t < t1; ++t) {
        const float u = to_float(static_cast<const E*>(a.u)[b * a.us.batch + t * a.us.row + d]);
        float dt = to_float(static_cast<const Td*>(a.dt)[b * a.dts.batch + t * a.dts.row + d]) + bias;
        if (a.softplus) dt = softplus(dt);
        const E* B = static_cast<const E*>(a.B) + b * a.Bs.batch + t * a.Bs.row + g * N;
        const E* C = static_cast<const E*>(a.C) + b * a.Cs.batch + t * a.Cs.row + g * N;
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int n = lane + 32 * k;
            if (n < N) {
                h[k] = fmaf(ex2(dt * A[k]), h[k], dt * u * to_float(B[n]));
                y = fmaf(to_float(C[n]), h[k], y);
            }
        }
        for (int off = 16; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        if (lane == 0) {
            y = fmaf(D, u, y);
            if (a.z) y *= silu(to_float(static_cast<const E*>(a.z)[b * a.zs.batch + t * a.zs.row + d]));
            store_elem(static_cast<E*>(a.y) + (b * a.T + t) * a.D + d, y);
        }
    }
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const int n = lane + 32 * k;
        if (n < N && a.fin) a.fin[(seq * a.D + d) * N + n] = h[k];
    }
}

}  // namespace

cudaError_t launch_selective_scan(const SelectiveArgs& a, cudaStream_t st) {
    const int64_t blocks = (a.nseq * a.D + kWarps - 1) / kWarps;
    if (blocks == 0 || (a.T == 0 && !a.fin)) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned g = (unsigned)blocks;
    if (a.dtype == SSD_F32)
        selective_kernel<float, float><<<g, kWarps * 32, 0, st>>>(a);
    else if (a.dt_dtype == SSD_F32)
        selective_kernel<__nv_bfloat16, float><<<g, kWarps * 32, 0, st>>>(a);
    else
        selective_kernel<__nv_bfloat16, __nv_bfloat16><<<g, kWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_selective_step(const SelectiveArgs& a, cudaStream_t st) {
    return a.T == 0 ? cudaSuccess : launch_selective_scan(a, st);
}

}  // namespace ssd
