// Short causal depthwise convolution with SiLU, before the layer ("Transformers are
// SSMs: Generalized Models and Efficient Algorithms Through Structured State Space
// Duality", Knowl 6, step 2 of the Mamba-2 block). Per sequence and channel:
//
//     v[t] = bias + sum_{k<W} w[k] u[t - (W-1) + k],     y[t] = v / (1 + exp(-v)) or v
//
// HBM-bound: u read once, y written once (4 bytes per element in bf16) against
// 2 W + about 6 operations, two of them on the special-function unit. A thread owns
// VW neighbouring channels (4, or 1 where the tensors do not take accesses of 4) and
// walks a run of tokens with the last W - 1 of them in registers, so a token is
// loaded once per run; the W - 1 rows before the run are read again (from L2). 8
// channels a thread (weights and window alone 64 registers) left too few warps to keep
// the memory busy: 139 us at 16384 tokens of 5376 channels in bf16 against 81, 68 now
// (5.2 TB/s, 0.79 of the copy rate).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "ssd_block.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kRunWarps = 4;     // token runs per CTA: one per warp, on the same 32 channel vectors
constexpr int kBatch = 8;        // tokens whose loads a thread issues together

struct ConvParams {
    const void* u;
    const float* weight;
    const float* bias;
    const int* cu;
    const void* init;
    void* y[3];
    void* fin;
    int64_t T, C, ub, ur;
    int64_t oc[3], off[3];       // channels of the outputs and where they start
    int64_t nvec, nvg;           // channel vectors, and groups of 32 of them
    int64_t run_blocks;          // CTAs along the tokens of a batch row
    int64_t main_blocks;         // CTAs of the convolution; the rest write final states
    int64_t nseq;
    int run;                     // tokens per warp
    int silu;
    bool weight16;               // weight starts on 16 bytes
};

// A thread's VW channels as packed pairs (VW = 1: one value).
template <int VW>
struct Lanes {
    using T = float2;
    static constexpr int M = VW / 2;
};
template <>
struct Lanes<1> {
    using T = float;
    static constexpr int M = 1;
};
template <int VW>
struct Vec {
    using T = typename Lanes<VW>::T;
    static constexpr int M = Lanes<VW>::M;
    T v[M];
};
__device__ __forceinline__ Vec<4> widen(uint2 q) {        // 4 bf16
    return {{make_float2(bf16_lo(q.x), bf16_hi(q.x)), make_float2(bf16_lo(q.y), bf16_hi(q.y))}};
}
__device__ __forceinline__ Vec<4> widen(float4 q) { return {{make_float2(q.x, q.y), make_float2(q.z, q.w)}}; }
__device__ __forceinline__ Vec<1> widen(float q) { return {{q}}; }
__device__ __forceinline__ Vec<1> widen(__nv_bfloat16 q) { return {{__bfloat162float(q)}}; }
__device__ __forceinline__ void narrow(const Vec<4>& v, uint2& q) {
    q = make_uint2(pack_bf16(v.v[0].x, v.v[0].y), pack_bf16(v.v[1].x, v.v[1].y));
}
__device__ __forceinline__ void narrow(const Vec<4>& v, float4& q) {
    q = make_float4(v.v[0].x, v.v[0].y, v.v[1].x, v.v[1].y);
}
__device__ __forceinline__ void narrow(const Vec<1>& v, float& q) { q = v.v[0]; }
__device__ __forceinline__ void narrow(const Vec<1>& v, __nv_bfloat16& q) { q = __float2bfloat16_rn(v.v[0]); }
// VW elements as they lie in memory
template <typename E, int VW>
struct Pack {
    using T = E;
};
template <>
struct Pack<float, 4> {
    using T = float4;
};
template <>
struct Pack<__nv_bfloat16, 4> {
    using T = uint2;
};
template <typename P>
__device__ __forceinline__ P zero_pack() {
    if constexpr (sizeof(P) == 16) return make_float4(0.f, 0.f, 0.f, 0.f);
    else if constexpr (sizeof(P) == 8) return make_uint2(0, 0);
    else return P(0.f);
}

template <int VW, int W>
struct Taps {
    Vec<VW> w[W], bias;
    __device__ __forceinline__ void load(const ConvParams& p, int64_t c) {
        float f[VW][W], b[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            if (W == 4 && p.weight16) {
                const float4 q = __ldg(reinterpret_cast<const float4*>(p.weight + (c + i) * W));
                f[i][0] = q.x; f[i][1] = q.y; f[i][2 % W] = q.z; f[i][3 % W] = q.w;
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k) f[i][k] = __ldg(p.weight + (c + i) * W + k);
            }
            b[i] = p.bias ? __ldg(p.bias + c + i) : 0.f;
        }
#pragma unroll
        for (int m = 0; m < Vec<VW>::M; ++m) {
            if constexpr (VW == 1) {
#pragma unroll
                for (int k = 0; k < W; ++k) w[k].v[0] = f[0][k];
                bias.v[0] = b[0];
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k) w[k].v[m] = make_float2(f[2 * m][k], f[2 * m + 1][k]);
                bias.v[m] = make_float2(b[2 * m], b[2 * m + 1]);
            }
        }
    }
    // window: the W - 1 tokens before x, oldest first
    template <bool kSilu>
    __device__ __forceinline__ Vec<VW> apply(const Vec<VW> (&window)[W - 1], const Vec<VW>& x) const {
        Vec<VW> y;
#pragma unroll
        for (int m = 0; m < Vec<VW>::M; ++m) {
            typename Vec<VW>::T v = bias.v[m];
#pragma unroll
            for (int k = 0; k < W - 1; ++k) v = fma_(w[k].v[m], window[k].v[m], v);
            v = fma_(w[W - 1].v[m], x.v[m], v);
            y.v[m] = kSilu ? silu(v) : v;
        }
        return y;
    }
};
template <int W, int VW>
__device__ __forceinline__ void push(Vec<VW> (&window)[W - 1], const Vec<VW>& x) {
#pragma unroll
    for (int k = 0; k + 1 < W - 1; ++k) window[k] = window[k + 1];
    window[W - 2] = x;
}

// Where channel c of batch row b goes: its output's first token, and the stride of its tokens.
template <typename E>
struct Out {
    E* y;
    int64_t stride;
    __device__ __forceinline__ Out(const ConvParams& p, int64_t b, int64_t c) {
        const int o = c >= p.off[2] ? 2 : (c >= p.off[1] ? 1 : 0);
        stride = p.oc[o];
        y = static_cast<E*>(p.y[o]) + (c - p.off[o]) + b * p.T * stride;
    }
};

__device__ __forceinline__ int64_t clamp_offset(int v, int64_t T) { return v < 0 ? 0 : (v > T ? T : v); }

// The document of token t: the last k with cu[k] <= t (offsets non-decreasing).
__device__ __forceinline__ int64_t find_doc(const int* cu, int64_t n, int64_t t) {
    int64_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <typename E, int VW, int W, bool kPacked, bool kSilu>
__global__ void __launch_bounds__(kRunWarps * 32, sizeof(E) == 2 ? 5 : 4) conv_kernel(const ConvParams p) {
    using Raw = typename Pack<E, VW>::T;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t blk = blockIdx.x;
    const E* init = static_cast<const E*>(p.init);

    if (blk >= p.main_blocks) {
        // final states: one warp per (sequence, group of channel vectors)
        const int64_t idx = (blk - p.main_blocks) * kRunWarps + warp;
        const int64_t seq = idx / p.nvg, vec = (idx % p.nvg) * 32 + lane;
        if (seq >= p.nseq || vec >= p.nvec) return;
        const int64_t start = kPacked ? clamp_offset(p.cu[seq], p.T) : 0;
        const int64_t end = kPacked ? clamp_offset(p.cu[seq + 1], p.T) : p.T;
        const E* u = static_cast<const E*>(p.u) + (kPacked ? 0 : seq * p.ub);
        E* fin = static_cast<E*>(p.fin);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int64_t t = end - (W - 1) + j;             // token, or t - start < 0: of the initial state
            const int64_t old = t - start + (W - 1);         // its row there
            Raw r = zero_pack<Raw>();
            if (t >= start)
                r = *reinterpret_cast<const Raw*>(u + t * p.ur + vec * VW);
            else if (init && old >= 0)
                r = *reinterpret_cast<const Raw*>(init + (seq * (W - 1) + old) * p.C + vec * VW);
            *reinterpret_cast<Raw*>(fin + (seq * (W - 1) + j) * p.C + vec * VW) = r;
        }
        return;
    }

    const int64_t vg = blk % p.nvg, rest = blk / p.nvg;
    const int64_t b = rest / p.run_blocks;
    const int64_t t0 = ((rest % p.run_blocks) * kRunWarps + warp) * p.run;
    const int64_t vec = vg * 32 + lane;
    int64_t limit = p.T;                                     // first token that is no document's
    if constexpr (kPacked) limit = clamp_offset(p.cu[p.nseq], p.T);
    const int64_t t1 = t0 + p.run < limit ? t0 + p.run : limit;
    if (t0 >= t1 || vec >= p.nvec) return;
    const int64_t c = vec * VW;
    const E* u = static_cast<const E*>(p.u) + b * p.ub + c;
    const Out<E> out(p, b, c);
    Taps<VW, W> taps;
    taps.load(p, c);

    int64_t seq = b, start = 0, next = limit;                // the sequence and where it starts and ends
    if constexpr (kPacked) {
        seq = find_doc(p.cu, p.nseq, t0);
        start = p.cu[seq];
        start = start < 0 ? 0 : (start > t0 ? t0 : start);
        next = p.cu[seq + 1];
    }
    Vec<VW> window[W - 1];
    auto open = [&](int64_t t) {                             // the W - 1 tokens before t
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int64_t s = t - (W - 1) + k;
            Raw r = zero_pack<Raw>();
            if (s >= start)
                r = *reinterpret_cast<const Raw*>(u + s * p.ur);
            else if (init && s - start + (W - 1) >= 0)
                r = *reinterpret_cast<const Raw*>(init + (seq * (W - 1) + s - start + (W - 1)) * p.C + c);
            window[k] = widen(r);
        }
    };
    // Addresses are walked: a product of 64-bit strides for every row costs more than its arithmetic.
    const E* ut = u + t0 * p.ur;
    E* yt = out.y + t0 * out.stride;
    const int64_t ys = out.stride;
    auto one = [&](const Vec<VW>& x) {
        Raw o;
        narrow(taps.template apply<kSilu>(window, x), o);
        push<W>(window, x);
        __stcs(reinterpret_cast<Raw*>(yt), o);
        yt += ys;
    };
    Raw raw[kBatch];
    auto fetch = [&](int n) {                                // the next n <= kBatch tokens
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (i < n) {
                raw[i] = __ldcs(reinterpret_cast<const Raw*>(ut));
                ut += p.ur;
            }
    };
    for (int64_t t = t0; t < t1;) {                          // the run's part of each document
        if constexpr (kPacked) {
            if (t >= next && seq + 1 < p.nseq) {             // one starts here: the last that does
                do {
                    ++seq;
                    next = p.cu[seq + 1];
                } while (t >= next && seq + 1 < p.nseq);
                start = t;
            }
        }
        const int64_t stop = kPacked && next > t && next < t1 ? next : t1;
        int left = (int)(stop - t);
        t = stop;
        // whole batches, the next one's loads in flight while this one is computed
        fetch(left);
        open(t - left);
        for (; left >= kBatch; left -= kBatch) {
            Vec<VW> x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) x[i] = widen(raw[i]);
            if (left >= 2 * kBatch) fetch(kBatch);
            else fetch(left - kBatch);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) one(x[i]);
        }
#pragma unroll
        for (int i = 0; i < kBatch - 1; ++i)
            if (i < left) one(widen(raw[i]));
    }
}

// One thread per (sequence, channel vector): the state's rows and the call's tokens.
template <typename E, int VW, int W>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvParams p, E* state) {
    using Raw = typename Pack<E, VW>::T;
    const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t b = idx / p.nvec, c = (idx % p.nvec) * VW;
    if (b >= p.nseq) return;
    E* st = state + b * (W - 1) * p.C + c;
    const E* u = static_cast<const E*>(p.u) + b * p.ub + c;
    const Out<E> out(p, b, c);
    Vec<VW> window[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) window[k] = widen(*reinterpret_cast<const Raw*>(st + k * p.C));
    Taps<VW, W> taps;
    taps.load(p, c);
    for (int64_t t = 0; t < p.T; ++t) {
        const Vec<VW> x = widen(*reinterpret_cast<const Raw*>(u + t * p.ur));
        Raw o;
        narrow(p.silu ? taps.template apply<true>(window, x) : taps.template apply<false>(window, x), o);
        push<W>(window, x);
        *reinterpret_cast<Raw*>(out.y + t * out.stride) = o;
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        Raw o;
        narrow(window[k], o);
        *reinterpret_cast<Raw*>(st + k * p.C) = o;
    }
}

// Whether the tensors take accesses of 4 channels (8 bytes of bf16, 16 of fp32).
bool wide(const ConvArgs& a, const void* state) {
    const int es = a.dtype == SSD_BF16 ? 2 : 4, vw = 4;
    if (a.C % vw || a.ub % vw || a.ur % vw || a.oc[0] % vw || a.oc[1] % vw || a.oc[2] % vw) return false;
    for (const void* q : {a.u, (const void*)a.y[0], (const void*)a.y[1], (const void*)a.y[2], a.init,
                          (const void*)a.final_states, state})
        if (!aligned(q, 4 * es)) return false;
    return true;
}

ConvParams params_of(const ConvArgs& a, int vw) {
    ConvParams p = {};
    p.u = a.u; p.weight = a.weight; p.bias = a.bias; p.cu = a.cu; p.init = a.init; p.fin = a.final_states;
    p.T = a.T; p.C = a.C; p.ub = a.ub; p.ur = a.ur; p.nseq = a.nseq; p.silu = a.silu;
    p.weight16 = aligned(a.weight, 16);
    int64_t off = 0;
    for (int i = 0; i < 3; ++i) {
        p.y[i] = a.y[i];
        p.oc[i] = a.oc[i];
        p.off[i] = off;
        off += a.oc[i];
    }
    // an absent output starts behind the last channel, so that no channel is taken for its
    for (int i = 2; i > 0; --i)
        if (p.oc[i] == 0) p.off[i] = a.C;
    p.nvec = a.C / vw;
    p.nvg = (p.nvec + 31) / 32;
    return p;
}

template <typename E, int VW, int W>
cudaError_t conv_w(const ConvArgs& a, cudaStream_t st) {
    ConvParams p = params_of(a, VW);
    // Runs of 64 tokens read 5 % more rows than they write (L2 holds the halo); shorter ones where
    // there would be too few warps to keep the memory busy.
    int run = 64;
    while (run > kBatch && p.nvg * a.b * ((a.T + run - 1) / run) < 148 * 24) run /= 2;
    p.run = run;
    p.run_blocks = (a.T + (int64_t)run * kRunWarps - 1) / ((int64_t)run * kRunWarps);
    p.main_blocks = p.run_blocks * p.nvg * a.b;
    const int64_t fin_blocks = p.fin ? (p.nseq * p.nvg + kRunWarps - 1) / kRunWarps : 0;
    const int64_t blocks = p.main_blocks + fin_blocks;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto kernel = a.cu ? (a.silu ? conv_kernel<E, VW, W, true, true> : conv_kernel<E, VW, W, true, false>)
                       : (a.silu ? conv_kernel<E, VW, W, false, true> : conv_kernel<E, VW, W, false, false>);
    kernel<<<(unsigned)blocks, kRunWarps * 32, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename E, int VW, int W>
cudaError_t step_w(const ConvArgs& a, void* state, cudaStream_t st) {
    const ConvParams p = params_of(a, VW);
    const int64_t blocks = (p.nseq * p.nvec + 127) / 128;
    if (blocks == 0 || a.T == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    conv_step_kernel<E, VW, W><<<(unsigned)blocks, 128, 0, st>>>(p, static_cast<E*>(state));
    return cudaGetLastError();
}

template <typename E, int VW>
cudaError_t conv_v(const ConvArgs& a, void* state, bool step, cudaStream_t st) {
    switch (a.W) {
        case 2: return step ? step_w<E, VW, 2>(a, state, st) : conv_w<E, VW, 2>(a, st);
        case 3: return step ? step_w<E, VW, 3>(a, state, st) : conv_w<E, VW, 3>(a, st);
        default: return step ? step_w<E, VW, 4>(a, state, st) : conv_w<E, VW, 4>(a, st);
    }
}

cudaError_t conv_any(const ConvArgs& a, void* state, bool step, cudaStream_t st) {
    const bool v = wide(a, state);
    if (a.dtype == SSD_BF16)
        return v ? conv_v<__nv_bfloat16, 4>(a, state, step, st) : conv_v<__nv_bfloat16, 1>(a, state, step, st);
    return v ? conv_v<float, 4>(a, state, step, st) : conv_v<float, 1>(a, state, step, st);
}

}  // namespace

cudaError_t launch_conv(const ConvArgs& a, cudaStream_t st) { return conv_any(a, nullptr, false, st); }
cudaError_t launch_conv_step(const ConvArgs& a, void* state, cudaStream_t st) { return conv_any(a, state, true, st); }

}  // namespace ssd
