// Selective scan with a diagonal A: the recurrence of Knowl 3's general form with a
// diagonal transition ("Transformers are SSMs: Generalized Models and Efficient
// Algorithms Through Structured State Space Duality"). Per sequence, channel d
// (group g) and state n:
//
//     h_t[n] = a_t[n] h_{t-1}[n] + dt_t u_t B_t[n],  a_t[n] = exp(dt_t A[n]),
//     y_t = sum_n C_t[n] h_t[n] + D u_t,             y_t *= SiLU(z_t) with a gate.
//
// What bounds it: one exponential for each (token, channel, state) on the special-function
// unit, 16 a clock and SM (with 16 states: 16 + 4 for softplus and SiLU against 8 bytes of HBM
// traffic in bf16, 3.6 times the time of the bytes), and beside it about as many issue slots.
// So every exponential is computed once, also where the sequence is cut.
//
// Layout: a warp takes 32 / SL channels, SL lanes a channel, 4 states a lane (more than 4 SL
// states in blocks), and kTok tokens at a time: its tokens' inputs arrive by asynchronous copies
// a tile ahead, softplus and dt u are computed once per (token, channel), and each lane then runs
// its 4 states through the tokens with packed fp32x2 arithmetic. The lanes' parts of y are summed
// by exchanges that leave every lane kTok / SL tokens.
//
// The cut (kSplit): where there are few channels, the warps of a CTA take consecutive runs of
// kTok tokens of the same channels. Each runs from a state of zero and keeps, per token and
// state, C_t times the product of its decays so far: the state entering the run, the fold of the
// runs before it, h <- P h + h_local, then adds sum_n (C_t prod a)[n] h_in[n] to each y_t, at two
// packed operations per pair and no second exponential.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "ssd_block.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kTok = 16;         // tokens of a warp's tile
constexpr int kMaxWarps = 8;

struct ScanParams {
    SelectiveArgs a;
    int64_t per;                 // channels of a group
    int64_t cblocks;             // channel blocks of a group
    int nblocks;                 // state blocks
    bool rows16, bc16;           // u, dt, z (B, C) take 16-byte copies
};

__device__ __forceinline__ void copy16(void* dst, const void* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(ok ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// kTok rows of W elements from src (row stride `row`) to dst [kTok][W], zeros where the token is not
// below `tokens` or the column not below `cols`. wide: 16-byte pieces (a piece is then inside or
// outside as a whole).
template <int W, typename E>
__device__ __forceinline__ void stage(E* dst, const E* src, int64_t row, int tokens, int cols, bool wide, int lane) {
    constexpr int V = 16 / sizeof(E);
    if (W >= V && wide) {
        constexpr int P = W >= V ? W / V : 1;
#pragma unroll
        for (int i = 0; i < (kTok * P + 31) / 32; ++i) {
            const int idx = lane + 32 * i, k = idx / P, c = (idx % P) * V;
            const bool ok = k < tokens && c < cols;
            if (kTok * P % 32 == 0 || idx < kTok * P) copy16(dst + k * W + c, ok ? src + k * row + c : src, ok);
        }
    } else {
#pragma unroll 4
        for (int idx = lane; idx < kTok * W; idx += 32) {
            const int k = idx / W, c = idx % W;
            const bool ok = k < tokens && c < cols;
            if constexpr (sizeof(E) == 4) {
                copy4(dst + idx, ok ? src + k * row + c : src, ok);
            } else {
                dst[idx] = ok ? src[k * row + c] : E(0.f);
            }
        }
    }
}

// A warp's shared memory: two stages of raw inputs, the tile's (dt, dt u), and B, C in fp32.
template <typename E, typename Td, int SL>
struct WarpMem {
    static constexpr int CH = 32 / SL, NS = 4 * SL;
    alignas(16) E u[2][kTok][CH];
    alignas(16) E z[2][kTok][CH];
    alignas(16) Td dt[2][kTok][CH];
    alignas(16) E B[2][kTok][NS];
    alignas(16) E C[2][kTok][NS];
    alignas(16) float2 s[kTok][CH];
    alignas(16) float Bf[sizeof(E) == 2 ? kTok : 1][NS];
    alignas(16) float Cf[sizeof(E) == 2 ? kTok : 1][NS];
};

template <int NS>
__device__ __forceinline__ void widen(float (*dst)[NS], const __nv_bfloat16 (*src)[NS], int lane) {
    // kTok * NS values, 8 a lane and round
#pragma unroll
    for (int i = 0; i < (kTok * NS + 255) / 256; ++i) {
        const int at = (lane + 32 * i) * 8;
        if (kTok * NS % 256 == 0 || at < kTok * NS) {
            float v[8];
            unpack(*reinterpret_cast<const uint4*>(&src[0][0] + at), v);
            float4* d = reinterpret_cast<float4*>(&dst[0][0] + at);
            d[0] = make_float4(v[0], v[1], v[2], v[3]);
            d[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
}

template <typename E, typename Td, int SL, bool kSplit>
__global__ void __launch_bounds__(kMaxWarps * 32, 2) scan_kernel(const ScanParams p) {
    constexpr int CH = 32 / SL, NS = 4 * SL;
    using Mem = WarpMem<E, Td, SL>;
    extern __shared__ __align__(16) unsigned char smem[];
    const SelectiveArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int ch = lane % CH, j = lane / CH;
    const int NB = p.nblocks;
    Mem& m = reinterpret_cast<Mem*>(smem)[warp];
    // split: per run and parity, local states and decays; then the carried states, by parity and state block.
    // Not split: each warp's own carried states.
    float4* const exchange = reinterpret_cast<float4*>(smem + warps * sizeof(Mem));
    float4* const carry = exchange + (kSplit ? 4 * warps * 32 : warp * NB * 32);

    // the warp's sequence, group and channels
    int64_t unit = blockIdx.x;
    if constexpr (!kSplit) unit = unit * warps + warp;
    const int64_t per_seq = p.cblocks * a.G;
    const int64_t seq = unit / per_seq, g = unit % per_seq / p.cblocks, c0 = unit % p.cblocks * CH;
    if (!kSplit && seq >= a.nseq) return;
    const int64_t b = a.cu ? 0 : seq;
    int64_t t0 = 0, t1 = a.T;
    if (a.cu) {
        t0 = min((int64_t)max(a.cu[seq], 0), a.T);
        t1 = min((int64_t)max(a.cu[seq + 1], 0), a.T);
    }
    const int cols = (int)min(p.per - c0, (int64_t)CH);
    const int64_t d0 = g * p.per + c0;
    const int64_t d = d0 + (ch < cols ? ch : 0);
    const int N = (int)a.N;
    const E* const u = static_cast<const E*>(a.u) + b * a.us.batch + d0;
    const Td* const dt = static_cast<const Td*>(a.dt) + b * a.dts.batch + d0;
    const E* const z = a.z ? static_cast<const E*>(a.z) + b * a.zs.batch + d0 : nullptr;
    const E* const B = static_cast<const E*>(a.B) + b * a.Bs.batch + g * N;
    const E* const C = static_cast<const E*>(a.C) + b * a.Cs.batch + g * N;
    E* const y = static_cast<E*>(a.y) + b * a.T * a.D + d0;
    const float skip = a.Dskip ? a.Dskip[d] : 0.f, bias = a.dt_bias ? a.dt_bias[d] : 0.f;

    const int64_t state0 = (seq * a.D + d) * N;
    if (!kSplit || warp == 0) {
        for (int nb = 0; nb < NB; ++nb) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = nb * NS + j * 4 + i;
                v[i] = a.init && n < N ? a.init[state0 + n] : 0.f;
            }
            carry[nb * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
        }
    }

    const int64_t tile = kSplit ? (int64_t)warps * kTok : kTok;
    const int64_t ntiles = t1 > t0 ? (t1 - t0 + tile - 1) / tile : 0;
    const int64_t iters = ntiles * NB;
    auto tokens_at = [&](int64_t it, int64_t* t) {     // the warp's first token of iteration it, and how many
        *t = t0 + it * tile + (kSplit ? warp * kTok : 0);
        const int64_t left = t1 - *t;
        return (int)(left < 0 ? 0 : (left > kTok ? kTok : left));
    };
    auto issue = [&](int64_t it, int nb) {
        int64_t t;
        const int n = tokens_at(it, &t);
        if (n > 0) {
            if (nb == 0) {
                const int s = (int)(it & 1);
                stage<CH>(&m.u[s][0][0], u + t * a.us.row, a.us.row, n, cols, p.rows16, lane);
                stage<CH>(&m.dt[s][0][0], dt + t * a.dts.row, a.dts.row, n, cols, p.rows16, lane);
                if (z) stage<CH>(&m.z[s][0][0], z + t * a.zs.row, a.zs.row, n, cols, p.rows16, lane);
            }
            const int s = (int)((it * NB + nb) & 1);
            stage<NS>(&m.B[s][0][0], B + t * a.Bs.row + nb * NS, a.Bs.row, n, N - nb * NS, p.bc16, lane);
            stage<NS>(&m.C[s][0][0], C + t * a.Cs.row + nb * NS, a.Cs.row, n, N - nb * NS, p.bc16, lane);
        }
        copy_commit();
    };

    float yv[kTok];
    float2 A0, A1;
    auto rates = [&](int nb) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = nb * NS + j * 4 + i;
            v[i] = n < N ? a.A[d * N + n] * kLog2e : 0.f;
        }
        A0 = make_float2(v[0], v[1]);
        A1 = make_float2(v[2], v[3]);
    };
    if (NB == 1) rates(0);
    if (iters > 0) issue(0, 0);
    int64_t it = 0;
    int nb = 0;
    for (int64_t i = 0; i < iters; ++i) {
        __syncwarp();                                   // the stage that is filled next has been read
        const int nb1 = nb + 1 == NB ? 0 : nb + 1;
        const int64_t it1 = nb1 == 0 ? it + 1 : it;
        if (i + 1 < iters) issue(it1, nb1);
        else copy_commit();
        copy_wait<1>();
        __syncwarp();
        int64_t t;
        const int n = tokens_at(it, &t);
        const int sr = (int)(it & 1), sb = (int)(i & 1);
        if (nb == 0) {
#pragma unroll
            for (int k = 0; k < kTok; ++k) yv[k] = 0.f;
        }
        if (NB > 1) rates(nb);
        float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
        float4 decay = make_float4(1.f, 1.f, 1.f, 1.f);
        float2 gc[kSplit ? kTok : 1][2];
        if (!kSplit) h = carry[nb * 32 + lane];
        if (n > 0) {
            if (nb == 0) {
                // once per (token, channel): the step and dt u; past the end both are 0, which
                // leaves the state as it is
#pragma unroll
                for (int q = 0; q < kTok / SL; ++q) {
                    const int k = q * SL + j;
                    float v = to_float(m.dt[sr][k][ch]) + bias;
                    if (a.softplus) v = softplus(v);
                    v = k < n ? v : 0.f;
                    m.s[k][ch] = make_float2(v, v * to_float(m.u[sr][k][ch]));
                }
            }
            if constexpr (sizeof(E) == 2) {
                widen<NS>(m.Bf, m.B[sb], lane);
                widen<NS>(m.Cf, m.C[sb], lane);
            }
            __syncwarp();
            const float* Bt;
            const float* Ct;
            if constexpr (sizeof(E) == 2) {
                Bt = &m.Bf[0][0];
                Ct = &m.Cf[0][0];
            } else {
                Bt = &m.B[sb][0][0];
                Ct = &m.C[sb][0][0];
            }
            float2 h0 = make_float2(h.x, h.y), h1 = make_float2(h.z, h.w);
            float2 p0 = make_float2(1.f, 1.f), p1 = p0;
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                const float2 s = m.s[k][ch];
                const float4 Bk = *reinterpret_cast<const float4*>(Bt + k * NS + j * 4);
                const float4 Ck = *reinterpret_cast<const float4*>(Ct + k * NS + j * 4);
                const float2 st = make_float2(s.x, s.x), su = make_float2(s.y, s.y);
                float2 a0 = __fmul2_rn(st, A0), a1 = __fmul2_rn(st, A1);
                a0 = make_float2(ex2(a0.x), ex2(a0.y));
                a1 = make_float2(ex2(a1.x), ex2(a1.y));
                h0 = __ffma2_rn(a0, h0, __fmul2_rn(su, make_float2(Bk.x, Bk.y)));
                h1 = __ffma2_rn(a1, h1, __fmul2_rn(su, make_float2(Bk.z, Bk.w)));
                const float2 C0 = make_float2(Ck.x, Ck.y), C1 = make_float2(Ck.z, Ck.w);
                const float2 r = __ffma2_rn(C1, h1, __fmul2_rn(C0, h0));
                yv[k] += r.x + r.y;
                if constexpr (kSplit) {
                    p0 = __fmul2_rn(p0, a0);
                    p1 = __fmul2_rn(p1, a1);
                    gc[k][0] = __fmul2_rn(C0, p0);
                    gc[k][1] = __fmul2_rn(C1, p1);
                }
            }
            h = make_float4(h0.x, h0.y, h1.x, h1.y);
            decay = make_float4(p0.x, p0.y, p1.x, p1.y);
        }
        if constexpr (kSplit) {
            // One barrier per iteration: run w's part is written before it and read behind it, and the
            // parity keeps a warp that is ahead by one iteration off what others still read.
            float4* const ex = exchange + (i & 1) * (2 * warps * 32);
            ex[(2 * warp) * 32 + lane] = h;
            ex[(2 * warp + 1) * 32 + lane] = decay;
            __syncthreads();
            float4 in = carry[((it & 1) * NB + nb) * 32 + lane];
            for (int w = 0; w < warp; ++w) {
                const float4 hl = ex[(2 * w) * 32 + lane], pl = ex[(2 * w + 1) * 32 + lane];
                in.x = fmaf(pl.x, in.x, hl.x);
                in.y = fmaf(pl.y, in.y, hl.y);
                in.z = fmaf(pl.z, in.z, hl.z);
                in.w = fmaf(pl.w, in.w, hl.w);
            }
            if (warp == warps - 1)
                carry[(((it + 1) & 1) * NB + nb) * 32 + lane] =
                    make_float4(fmaf(decay.x, in.x, h.x), fmaf(decay.y, in.y, h.y), fmaf(decay.z, in.z, h.z),
                                fmaf(decay.w, in.w, h.w));
            if (n > 0) {
                const float2 i0 = make_float2(in.x, in.y), i1 = make_float2(in.z, in.w);
#pragma unroll
                for (int k = 0; k < kTok; ++k) {
                    const float2 r = __ffma2_rn(gc[k][1], i1, __fmul2_rn(gc[k][0], i0));
                    yv[k] += r.x + r.y;
                }
            }
        } else {
            carry[nb * 32 + lane] = h;
        }
        if (nb == NB - 1 && n > 0) {
            // sums over a channel's SL lanes: after the exchanges lane j holds tokens k with k % SL == j
            float r[kTok / SL];
            if constexpr (SL == 4) {
                float half[kTok / 2];
                const bool up = j & 2, odd = j & 1;
#pragma unroll
                for (int q = 0; q < kTok / 2; ++q) {
                    const int k = (q / 2) * 4 + q % 2;         // tokens with bit 1 clear; k + 2 has it set
                    const float send = up ? yv[k] : yv[k + 2];
                    half[q] = (up ? yv[k + 2] : yv[k]) + __shfl_xor_sync(0xffffffffu, send, 2 * CH);
                }
#pragma unroll
                for (int q = 0; q < kTok / 4; ++q) {
                    const float send = odd ? half[2 * q] : half[2 * q + 1];
                    r[q] = (odd ? half[2 * q + 1] : half[2 * q]) + __shfl_xor_sync(0xffffffffu, send, CH);
                }
            } else if constexpr (SL == 2) {
                const bool odd = j & 1;
#pragma unroll
                for (int q = 0; q < kTok / 2; ++q) {
                    const float send = odd ? yv[2 * q] : yv[2 * q + 1];
                    r[q] = (odd ? yv[2 * q + 1] : yv[2 * q]) + __shfl_xor_sync(0xffffffffu, send, CH);
                }
            } else {
#pragma unroll
                for (int q = 0; q < kTok; ++q) r[q] = yv[q];
            }
#pragma unroll
            for (int q = 0; q < kTok / SL; ++q) {
                const int k = q * SL + j;
                float v = fmaf(skip, to_float(m.u[sr][k][ch]), r[q]);
                if (z) v *= silu(to_float(m.z[sr][k][ch]));
                if (k < n && ch < cols) store_elem(y + (t + k) * a.D + ch, v);
            }
        }
        nb = nb1;
        it = it1;
    }
    copy_wait<0>();
    if (!a.fin) return;
    if constexpr (kSplit) __syncthreads();              // the last warp's carried states
    if (kSplit && warp != 0) return;
    if (ch >= cols) return;
    for (int nb2 = 0; nb2 < NB; ++nb2) {
        const float4 h = carry[((kSplit ? (ntiles & 1) * NB : 0) + nb2) * 32 + lane];
        const float v[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = nb2 * NS + j * 4 + i;
            if (n < N) a.fin[state0 + n] = v[i];
        }
    }
}

template <typename E, typename Td, int SL>
cudaError_t launch_scan(ScanParams p, cudaStream_t st) {
    constexpr int CH = 32 / SL, NS = 4 * SL;
    const SelectiveArgs& a = p.a;
    p.cblocks = (p.per + CH - 1) / CH;
    p.nblocks = (int)((a.N + NS - 1) / NS);
    const int64_t units = a.nseq * a.G * p.cblocks;      // warps without a cut
    const int64_t len = (a.T + (a.cu ? a.nseq : 1) - 1) / (a.cu ? a.nseq : 1);
    // Cut the tokens where the channels alone leave the SMs with few warps.
    int warps = 1;
    while (warps < kMaxWarps && units * warps < 148 * 12 && len > warps * kTok) warps *= 2;
    const bool split = warps > 1;
    if (!split) warps = 4;
    const int64_t blocks = split ? units : (units + warps - 1) / warps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const size_t shared = warps * sizeof(WarpMem<E, Td, SL>) +
                          (split ? (size_t)(4 * warps * 32 + 2 * p.nblocks * 32) : (size_t)warps * p.nblocks * 32) * 16;
    auto kernel = split ? scan_kernel<E, Td, SL, true> : scan_kernel<E, Td, SL, false>;
    if (shared > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
        if (e != cudaSuccess) return e;
    }
    kernel<<<(unsigned)blocks, warps * 32, shared, st>>>(p);
    return cudaGetLastError();
}

template <typename E, typename Td>
cudaError_t scan_any(const SelectiveArgs& a, cudaStream_t st) {
    if (a.nseq == 0 || (a.T == 0 && !a.fin)) return cudaSuccess;
    ScanParams p = {};
    p.a = a;
    p.per = a.D / a.G;
    const int64_t v = 16 / sizeof(E), vd = 16 / sizeof(Td);
    auto ok = [](const void* q, const ssd_strides_t& s, int64_t n) {
        return aligned(q, 16) && s.batch % n == 0 && s.row % n == 0;
    };
    p.rows16 = p.per % v == 0 && ok(a.u, a.us, v) && ok(a.dt, a.dts, vd) && (!a.z || ok(a.z, a.zs, v));
    p.bc16 = a.N % v == 0 && ok(a.B, a.Bs, v) && ok(a.C, a.Cs, v);
    if (a.N <= 4) return launch_scan<E, Td, 1>(p, st);
    if (a.N <= 8) return launch_scan<E, Td, 2>(p, st);
    return launch_scan<E, Td, 4>(p, st);
}

// ---- decoding --------------------------------------------------------------
constexpr int kWarps = 4;
constexpr int kPieces = 8;       // states of a lane: up to 256 over 32 lanes

// One warp per channel, the states over its lanes.
template <typename E, typename Td>
__global__ void __launch_bounds__(kWarps * 32) step_kernel(const SelectiveArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t idx = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t b = idx / a.D, d = idx % a.D;
    if (b >= a.b) return;
    const int64_t g = d / (a.D / a.G);
    const int N = (int)a.N;
    float h[kPieces], A[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const int n = lane + 32 * k;
        A[k] = n < N ? a.A[d * N + n] * kLog2e : 0.f;
        h[k] = n < N ? a.init[(b * a.D + d) * N + n] : 0.f;
    }
    const float D = a.Dskip ? a.Dskip[d] : 0.f, bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    for (int64_t t = 0; t < a.T; ++t) {
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
        if (n < N) a.fin[(b * a.D + d) * N + n] = h[k];
    }
}

template <typename E, typename Td>
cudaError_t step_any(const SelectiveArgs& a, cudaStream_t st) {
    const int64_t blocks = (a.nseq * a.D + kWarps - 1) / kWarps;
    if (blocks == 0 || a.T == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    step_kernel<E, Td><<<(unsigned)blocks, kWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_selective_scan(const SelectiveArgs& a, cudaStream_t st) {
    if (a.dtype == SSD_F32) return scan_any<float, float>(a, st);
    return a.dt_dtype == SSD_F32 ? scan_any<__nv_bfloat16, float>(a, st)
                                 : scan_any<__nv_bfloat16, __nv_bfloat16>(a, st);
}

cudaError_t launch_selective_step(const SelectiveArgs& a, cudaStream_t st) {
    if (a.dtype == SSD_F32) return step_any<float, float>(a, st);
    return a.dt_dtype == SSD_F32 ? step_any<__nv_bfloat16, float>(a, st)
                                 : step_any<__nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace ssd
