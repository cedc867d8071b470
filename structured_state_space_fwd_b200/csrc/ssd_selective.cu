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
// traffic in bf16, 3.6 times the time of the bytes), and beside it nearly as many issue slots:
// four fp32 operations for each exponential, whose packed forms (fp32x2) take two slots each, and
// what a (token, channel) needs once. So every exponential is computed once, also where a sequence
// is cut, and what is left is moved off the inner loop.
//
// Two forms, both with their inputs copied asynchronously a tile ahead:
//   many channels (wide_scan_kernel): one or two lanes hold the states of a channel, and two warps
//     take the tiles of a block of channels in turn;
//   few channels (cut_scan_kernel): lanes share pairs of channels, and the warps of a CTA take
//     consecutive runs of tokens of the same channels; for very few, the CTAs of a cluster take
//     consecutive segments.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "ssd_block.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

struct ScanParams {
    SelectiveArgs a;
    int64_t per;                 // channels of a group
    int64_t cblocks;             // channel blocks of a group
    int nblocks;                 // state blocks
    int row_bytes, bc_bytes;     // pieces in which u, dt, z (B, C) are copied: 16, 4 or one element
    bool y_pairs;                // y takes stores of two channels
    bool ranked;                 // documents in the order of their lengths
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
// Named barriers of two warps: the one that hands over goes on (or waits too), the other waits. The
// ids are immediates, so that a CTA reserves no more barriers than it uses.
template <int kIds>
__device__ __forceinline__ void pair_arrive(int id) {
#define SSD_ARRIVE(i) \
    if constexpr (i < kIds) { if (id == i) asm volatile("bar.arrive " #i ", 64;" ::: "memory"); }
    SSD_ARRIVE(0) SSD_ARRIVE(1) SSD_ARRIVE(2) SSD_ARRIVE(3) SSD_ARRIVE(4) SSD_ARRIVE(5) SSD_ARRIVE(6) SSD_ARRIVE(7)
#undef SSD_ARRIVE
    static_assert(kIds <= 8, "");
}
template <int kIds>
__device__ __forceinline__ void pair_wait(int id) {
#define SSD_WAIT(i) \
    if constexpr (i < kIds) { if (id == i) asm volatile("bar.sync " #i ", 64;" ::: "memory"); }
    SSD_WAIT(0) SSD_WAIT(1) SSD_WAIT(2) SSD_WAIT(3) SSD_WAIT(4) SSD_WAIT(5) SSD_WAIT(6) SSD_WAIT(7)
#undef SSD_WAIT
    static_assert(kIds <= 8, "");
}

// The CTAs of a cluster: rank, a barrier in two halves, and loads from another CTA's shared memory.
__device__ __forceinline__ int cluster_rank() {
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cluster_size() {
    int r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t in_cta(const void* own, int rank) {     // the same place in CTA `rank`
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(own)), "r"(rank));
    return at;
}
__device__ __forceinline__ float4 remote4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 remote2(uint32_t at) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

// Copies K rows of W elements, row stride `row`, to shared memory [K][W], zeros where the row is not
// below `rows` or the column not below `cols`, in pieces of `bytes`: 16 or 4 asynchronously (a piece is
// then inside or outside as a whole), else element by element.
template <int K, int W, typename E>
__device__ __forceinline__ void stage(E* dst, const E* src, int row, int rows, int cols, int lane, int bytes) {
    constexpr int V = 16 / sizeof(E), P = W >= V ? W / V : 1, kPieces = (K * P + 31) / 32;
    if (W >= V && bytes == 16) {
        const int k0 = lane / P, c = (lane % P) * V;
        const E* from = src + ((int64_t)k0 * row + c);
        if (rows == K && cols >= W) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                if (K * P % 32 == 0 || k0 < K)
                    copy16(dst + (k0 + i * (32 / P)) * W + c, from + (int64_t)(i * (32 / P)) * row, true);
        } else {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int k = k0 + i * (32 / P);
                const bool ok = k < rows && c < cols;
                if (K * P % 32 == 0 || k < K)
                    copy16(dst + k * W + c, ok ? from + (int64_t)(i * (32 / P)) * row : src, ok);
            }
        }
    } else if (bytes >= 4) {
        constexpr int V4 = 4 / sizeof(E), P4 = W / V4;
#pragma unroll
        for (int i = 0; i < (K * P4 + 31) / 32; ++i) {
            const int k = (lane + 32 * i) / P4, c = (lane + 32 * i) % P4 * V4;
            const bool ok = k < rows && c < cols;
            if (K * P4 % 32 == 0 || k < K) copy4(dst + k * W + c, ok ? src + ((int64_t)k * row + c) : src, ok);
        }
    } else {
        constexpr int kN = (K * W + 31) / 32, kAtOnce = kN < 4 ? kN : 4;
#pragma unroll 1
        for (int i0 = 0; i0 < kN; i0 += kAtOnce) {
            E v[kAtOnce];                                 // loads before the first store
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int k = (lane + 32 * (i0 + i)) / W, c = (lane + 32 * (i0 + i)) % W;
                v[i] = k < rows && c < cols ? src[(int64_t)k * row + c] : E(0.f);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (K * W % (32 * kAtOnce) == 0 || lane + 32 * (i0 + i) < K * W) dst[lane + 32 * (i0 + i)] = v[i];
        }
    }
}

// Which document of a pack the units of place r take: the longest come first, so that the units that are
// taken last are short (ties by index). A warp ranks the lengths of up to kRanked documents by
// exchanges; all its lanes call it.
constexpr int kRanked = 64;
__device__ __forceinline__ int64_t document_at(const int* cu, int64_t n, int64_t r, int T, int lane) {
    auto length = [&](int k) { return k < n ? min(max(cu[k + 1], 0), T) - min(max(cu[k], 0), T) : INT_MIN; };
    const int mine[2] = {length(lane), length(lane + 32)};
    int before[2] = {0, 0};
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
        const int other[2] = {__shfl_sync(0xffffffffu, mine[0], k), __shfl_sync(0xffffffffu, mine[1], k)};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int o = 0; o < 2; ++o)
                before[i] += other[o] > mine[i] || (other[o] == mine[i] && k + 32 * o < lane + 32 * i);
    }
    const unsigned at0 = __ballot_sync(0xffffffffu, lane < n && before[0] == r);
    const unsigned at1 = __ballot_sync(0xffffffffu, lane + 32 < n && before[1] == r);
    return at0 ? __ffs(at0) - 1 : 31 + __ffs(at1);
}

// Two neighbouring elements.
__device__ __forceinline__ float2 pair_of(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16* p) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(bf16_lo(v), bf16_hi(v));
}
__device__ __forceinline__ void store_pair(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float2 v) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(v.x, v.y);
}
// Four neighbouring elements as two pairs.
__device__ __forceinline__ void quad_of(const float* p, float2* v) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = make_float2(q.x, q.y);
    v[1] = make_float2(q.z, q.w);
}
__device__ __forceinline__ void quad_of(const __nv_bfloat16* p, float2* v) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = make_float2(bf16_lo(q.x), bf16_hi(q.x));
    v[1] = make_float2(bf16_lo(q.y), bf16_hi(q.y));
}

// ---- padded states beside infinities -----------------------------------------
//
// The kernels run states from N on, up to their lanes' number, with rates, B and C of 0. They stay 0 as
// long as the steps and their products with u are finite; 0 times an infinity is NaN, stays NaN to the
// end of the sequence, and reaches y, which may be infinite instead. So where the last padded state is not
// 0 at the end, each warp goes over the y that it stored: where that is NaN, the sum over the N states
// alone takes its place. The kernels' loops have no part in this (checks of every tile's dt u, or of its
// states, cost 3 to 20 %; this up to 10, 2 on average. Going over a channel again costs 0.8 us a token and
// channel of the warp.) Where there is no D, 0 times an infinite u may not be added either. kCare, of the
// kernels: 2 with padded states, 1 without them or D, 0 else, with nothing to look after.
//
// Warp w has stored the tiles of kTok tokens w, w + kWarps, .. from token `from` on to `end`; the sequence
// starts at t0. which: bits of the channels; owner(k, c): the lane that stored token k of a tile. A lane has
// the states lane + 32 i, one token after another.
template <int kTok, int kWarps, typename E, typename Td, typename Owner>
__device__ __noinline__ void sum_again(const ScanParams& p, int64_t seq, int64_t g, int64_t d0, int t0, int from,
                                       int end, unsigned which, Owner owner) {
    const SelectiveArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, N = (int)a.N;
    const int64_t b = a.cu ? 0 : seq;
#pragma unroll 1
    for (; which; which &= which - 1) {
        const int c = __ffs(which) - 1;
        const int64_t d = d0 + c;
        const float skip = a.Dskip ? a.Dskip[d] : 0.f, bias = a.dt_bias ? a.dt_bias[d] : 0.f;
        float h[kMaxSelectiveStates / 32];
#pragma unroll 1
        for (int i = 0; i * 32 + lane < N; ++i) h[i] = a.init ? a.init[(seq * a.D + d) * N + i * 32 + lane] : 0.f;
#pragma unroll 1
        for (int t = t0; t < end; ++t) {
            float dt = to_float(static_cast<const Td*>(a.dt)[b * a.dts.batch + (int64_t)t * a.dts.row + d]) + bias;
            if (a.softplus) dt = softplus(dt);
            const float u = to_float(static_cast<const E*>(a.u)[b * a.us.batch + (int64_t)t * a.us.row + d]);
            const E* const B = static_cast<const E*>(a.B) + b * a.Bs.batch + (int64_t)t * a.Bs.row + g * N;
            const E* const C = static_cast<const E*>(a.C) + b * a.Cs.batch + (int64_t)t * a.Cs.row + g * N;
            float sum = 0.f;
            bool lost = false;
#pragma unroll 1
            for (int i = 0; i * 32 + lane < N; ++i) {
                const int n = i * 32 + lane;
                h[i] = fmaf(decay_of(dt, rate_of(a.A[d * N + n])), h[i], dt * u * to_float(B[n]));
                sum = fmaf(to_float(C[n]), h[i], sum);
                lost |= h[i] != h[i];
            }
            __syncwarp();
            if (__any_sync(0xffffffffu, lost)) break;        // a state that is NaN stays it, and y with it
#pragma unroll
            for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            const int k = t - from;
            if (k < 0 || k / kTok % kWarps != warp || owner(k % kTok, c) != lane) continue;
            E* const y = static_cast<E*>(a.y) + (b * a.T + t) * a.D + d;
            if (to_float(*y) == to_float(*y)) continue;
            if (a.Dskip) sum = fmaf(skip, u, sum);
            if (a.z) sum *= silu(to_float(static_cast<const E*>(a.z)[b * a.zs.batch + (int64_t)t * a.zs.row + d]));
            store_elem(y, sum);
        }
    }
}

inline int care_of(const SelectiveArgs& a, int states) { return a.N % states != 0 ? 2 : a.Dskip ? 0 : 1; }

// ---- many channels -----------------------------------------------------------
//
// S = 2 lanes (1 with up to 4 states) hold a channel's states, 8 each of 16 at a time, and every
// second pair of its tokens' steps, gates and outputs; B and C are read at one address by each half of
// the warp, in less time than distinct ones. The two warps of a CTA take the tiles of 32 / S channels in
// turn and hand the states over through shared memory: while one runs the states through its tile,
// the other computes the steps of its next and finishes its last. 168 registers, which keep the next
// token's decays, B and C in flight, are worth more than twice the warps (4 x 2048 tokens of 5120
// channels, 16 states, bf16: 321 us with 6 CTAs an SM, 328 with 8, 327 with 9, 330 with 11; one lane a
// channel 353; four lanes for a pair of channels 349; but see launch_wide).
constexpr int kWideTok = 16, kWideWarps = 2;

template <typename E, typename Td, int NS, int S>
struct WideMem {
    static constexpr int CH = 32 / S;
    alignas(16) E u[2][kWideTok][CH];
    alignas(16) E z[2][kWideTok][CH];
    alignas(16) Td dt[2][kWideTok][CH];
    alignas(16) E B[2][kWideTok][NS];
    alignas(16) E C[2][kWideTok][NS];
    alignas(16) float Bf[sizeof(E) == 2 ? kWideTok : 1][NS];
    alignas(16) float Cf[sizeof(E) == 2 ? kWideTok : 1][NS];
};
template <int K, int NS>
__device__ __forceinline__ void widen(float (*dst)[NS], const __nv_bfloat16 (*src)[NS], int lane) {
#pragma unroll
    for (int i = 0; i < (K * NS + 127) / 128; ++i) {
        const int at = (lane + 32 * i) * 4;
        if (K * NS % 128 == 0 || at < K * NS) {
            float2 v[2];
            quad_of(&src[0][0] + at, v);
            *reinterpret_cast<float4*>(&dst[0][0] + at) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        }
    }
}
template <typename E, int CH>
__device__ __forceinline__ float2 tokens_of(const E (*rows)[CH], int k, int ch) {      // of tokens k and k + 1
    return make_float2(to_float(rows[k][ch]), to_float(rows[k + 1][ch]));
}

// S: lanes of a channel, each with NS / S of the states and every S-th pair of tokens to prepare and
// finish. kBlocks: more states than NS, which the inner loops then take a block at a time. kCtas: CTAs an
// SM that the registers are capped for.
template <typename E, typename Td, int NS, int S, bool kBlocks, int kCare, int kCtas>
__global__ void __launch_bounds__(kWideWarps * 32, kCtas) wide_scan_kernel(const __grid_constant__ ScanParams p) {
    constexpr int K = kWideTok, P = NS / S / 2, W = kWideWarps, CH = 32 / S, Q = K / 2 / S;
    using Mem = WideMem<E, Td, NS, S>;
    extern __shared__ __align__(16) unsigned char smem[];
    const SelectiveArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int ch = lane % CH, j = lane / CH;             // channel, states j NS / S ..
    const int NB = kBlocks ? p.nblocks : 1;
    Mem& m = reinterpret_cast<Mem*>(smem)[warp];
    // by state block: the states entering the next tile, and (with several blocks) the rates
    float2* const carry = reinterpret_cast<float2*>(smem + W * sizeof(Mem)) + lane;     // [NB][P][32]
    float2* const rates = carry + NB * P * 32;
    const int64_t unit = blockIdx.x, per_seq = p.cblocks * a.G;
    const int64_t seq = p.ranked ? document_at(a.cu, a.nseq, unit / per_seq, (int)a.T, lane) : unit / per_seq;
    const int64_t g = unit % per_seq / p.cblocks, c0 = unit % p.cblocks * CH;
    const int64_t b = a.cu ? 0 : seq;
    int t0 = 0, t1 = (int)a.T;
    if (a.cu) {
        t0 = min(max(a.cu[seq], 0), t1);
        t1 = min(max(a.cu[seq + 1], 0), t1);
    }
    const int cols = (int)min(p.per - c0, (int64_t)CH);
    const int64_t d0 = g * p.per + c0;
    const int N = (int)a.N;
    const bool in = ch < cols;
    const int64_t d = d0 + (in ? ch : 0);
    const float2 skip = both(a.Dskip ? a.Dskip[d] : 0.f), bias = both(a.dt_bias ? a.dt_bias[d] : 0.f);
    float2 A[P];
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float v[2], r[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int n = nb * NS + j * (2 * P) + 2 * i + x;
                v[x] = a.init && n < N ? a.init[(seq * a.D + d) * N + n] : 0.f;
                r[x] = n < N ? rate_of(a.A[d * N + n]) : 0.f;
            }
            A[i] = make_float2(r[0], r[1]);
            if (warp == 0) {
                carry[(nb * P + i) * 32] = make_float2(v[0], v[1]);
                if (NB > 1) rates[(nb * P + i) * 32] = A[i];
            }
        }
    }
    if (NB > 1) __syncthreads();
    const E* const ub = static_cast<const E*>(a.u) + b * a.us.batch + d0;
    const Td* const dtb = static_cast<const Td*>(a.dt) + b * a.dts.batch + d0;
    const E* const zb = a.z ? static_cast<const E*>(a.z) + b * a.zs.batch + d0 : nullptr;
    const E* const Bb = static_cast<const E*>(a.B) + b * a.Bs.batch + g * N;
    const E* const Cb = static_cast<const E*>(a.C) + b * a.Cs.batch + g * N;
    const int ur = (int)a.us.row, dtr = (int)a.dts.row, zr = (int)a.zs.row, Br = (int)a.Bs.row, Cr = (int)a.Cs.row;
    // the copies of the tile at token t, state block nb; u, dt, z (stage sr) with the first block
    auto issue = [&](int t, int nb, int sr, int sb) {
        const int n = min(t1 - t, K);
        if (n > 0) {
            if (nb == 0) {
                stage<K, CH>(&m.u[sr][0][0], ub + (int64_t)t * ur, ur, n, cols, lane, p.row_bytes);
                stage<K, CH>(&m.dt[sr][0][0], dtb + (int64_t)t * dtr, dtr, n, cols, lane, p.row_bytes);
                if (zb) stage<K, CH>(&m.z[sr][0][0], zb + (int64_t)t * zr, zr, n, cols, lane, p.row_bytes);
            }
            stage<K, NS>(&m.B[sb][0][0], Bb + (int64_t)t * Br + nb * NS, Br, n, N - nb * NS, lane, p.bc_bytes);
            stage<K, NS>(&m.C[sb][0][0], Cb + (int64_t)t * Cr + nb * NS, Cr, n, N - nb * NS, lane, p.bc_bytes);
        }
        copy_commit();
    };
    const int tiles = t1 > t0 ? (t1 - t0 + K - 1) / K : 0;
    E* const yb = static_cast<E*>(a.y) + b * a.T * a.D + d0 + ch;
    int t = t0 + warp * K, sr = 0, sb = 0;
    issue(t, 0, 0, 0);
    for (int it = warp; it < tiles; it += W, t += W * K, sr ^= 1) {
        const int n = min(t1 - t, K);
        float2 dt[Q], du[Q], yv[Q];                          // pair q S + j of the tile's tokens
        for (int nb = 0; nb < NB; ++nb, sb ^= 1) {
            __syncwarp();                                    // the stage that is filled next has been read
            if (nb + 1 < NB) issue(t, nb + 1, sr ^ 1, sb ^ 1);
            else issue(t + W * K, 0, sr ^ 1, sb ^ 1);
            copy_wait<1>();
            __syncwarp();
            if (nb == 0) {
                // past the end the step and dt u are 0, which leaves the state as it is
#pragma unroll
                for (int q = 0; q < Q; ++q) dt[q] = add_(tokens_of(m.dt[sr], 2 * (q * S + j), ch), bias);
                if (a.softplus) {
#pragma unroll
                    for (int q = 0; q < Q; ++q) dt[q] = softplus(dt[q]);
                }
                if (n < K) {
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const int k = 2 * (q * S + j);
                        dt[q] = make_float2(k < n ? dt[q].x : 0.f, k + 1 < n ? dt[q].y : 0.f);
                    }
                }
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    du[q] = mul_(dt[q], tokens_of(m.u[sr], 2 * (q * S + j), ch));
                    yv[q] = both(0.f);
                }
            }
            const float* Bt;
            const float* Ct;
            if constexpr (sizeof(E) == 2) {
                widen<K, NS>(m.Bf, m.B[sb], lane);
                widen<K, NS>(m.Cf, m.C[sb], lane);
                __syncwarp();
                Bt = &m.Bf[0][0] + j * (2 * P);
                Ct = &m.Cf[0][0] + j * (2 * P);
            } else {
                Bt = &m.B[sb][0][0] + j * (2 * P);
                Ct = &m.C[sb][0][0] + j * (2 * P);
            }
            // barrier w: the other warp has run its tile, whose states are in carry
            if (nb == 0 && it > 0) pair_wait<W>(warp);
            float2 h[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                h[i] = carry[(nb * P + i) * 32];
                if (NB > 1) A[i] = rates[(nb * P + i) * 32];
            }
            // a token's decays, B and C while the states of the one before are computed
            float2 e[2][P], Bv[2][P], Cv[2][P];
            // a value of token k out of the pairs, from the lane that has it
            auto of = [&](const float2 (&v)[Q], int k) {
                const float x = k % 2 ? v[k / 2 / S].y : v[k / 2 / S].x;
                return S == 1 ? x : __shfl_sync(0xffffffffu, x, k / 2 % S * CH + ch);
            };
            auto prepare = [&](int k) {
                const float st = of(dt, k);
#pragma unroll
                for (int i = 0; i < P; i += 2) {
                    quad_of(Bt + k * NS + 2 * i, Bv[k & 1] + i);
                    quad_of(Ct + k * NS + 2 * i, Cv[k & 1] + i);
                }
#pragma unroll
                for (int i = 0; i < P; ++i) e[k & 1][i] = decay_of(both(st), A[i]);
            };
            float part[2 * S];                               // of y, for S pairs of tokens
            prepare(0);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float su = of(du, k);
                if (k + 1 < K) prepare(k + 1);
                float2 r[2] = {both(0.f), both(0.f)};
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    h[i] = fma_(e[k & 1][i], h[i], mul_(both(su), Bv[k & 1][i]));
                    r[i & 1] = fma_(Cv[k & 1][i], h[i], r[i & 1]);
                }
                r[0] = add_(r[0], r[1]);
                part[k % (2 * S)] = r[0].x + r[0].y;
                if (k % (2 * S) == 2 * S - 1) {              // each lane keeps its pair's sum
                    float2 v = make_float2(part[0], part[1]);
                    if constexpr (S == 2) {
                        const float2 o = make_float2(part[2], part[3]);
                        const float2 send = j ? v : o;
                        v = add_(j ? o : v, make_float2(__shfl_xor_sync(0xffffffffu, send.x, CH),
                                                        __shfl_xor_sync(0xffffffffu, send.y, CH)));
                    }
                    yv[k / (2 * S)] = kBlocks ? add_(yv[k / (2 * S)], v) : v;
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) carry[(nb * P + i) * 32] = h[i];
        }
        if (it + 1 < tiles) pair_arrive<W>(warp ^ 1);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const float2 with = fma_(skip, tokens_of(m.u[sr], 2 * (q * S + j), ch), yv[q]);
            yv[q] = kCare == 0 || (kCare == 2 && a.Dskip) ? with : yv[q];
        }
        if (zb) {
#pragma unroll
            for (int q = 0; q < Q; ++q) yv[q] = mul_(yv[q], silu(tokens_of(m.z[sr], 2 * (q * S + j), ch)));
        }
        E* to = yb + (int64_t)(t + 2 * j) * (int)a.D;
        if (n == K && cols == CH) {
#pragma unroll
            for (int q = 0; q < Q; ++q, to += 2 * S * a.D) {
                store_elem(to, yv[q].x);
                store_elem(to + a.D, yv[q].y);
            }
        } else if (in) {
#pragma unroll
            for (int q = 0; q < Q; ++q, to += 2 * S * a.D) {
                const int k = 2 * (q * S + j);
                if (k < n) store_elem(to, yv[q].x);
                if (k + 1 < n) store_elem(to + a.D, yv[q].y);
            }
        }
    }
    copy_wait<0>();
    if constexpr (kCare == 2) {
        __syncwarp();                                        // lanes part at the stores; the barrier takes whole warps
        asm volatile("bar.sync 2, 64;" ::: "memory");        // (0 and 1 are the warps' own)
        const bool odd = in && j == S - 1 && carry[(NB * P - 1) * 32].y != 0.f;
        const unsigned which = __ballot_sync(0xffffffffu, odd) >> ((S - 1) * CH);
        if (which)
            sum_again<K, W, E, Td>(p, seq, g, d0, t0, t0, t1, which, [](int k, int c) { return k / 2 % S * CH + c; });
    }
    // the warp that wrote the carried states last
    if (!a.fin || !in || warp != (tiles == 0 ? 0 : (tiles - 1) % W)) return;
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 h = carry[(nb * P + i) * 32];
            const int n = nb * NS + j * (2 * P) + 2 * i;
            if (n < N) a.fin[(seq * a.D + d) * N + n] = h.x;
            if (n + 1 < N) a.fin[(seq * a.D + d) * N + n + 1] = h.y;
        }
    }
}

template <typename E, typename Td, int NS, int S, bool kBlocks>
cudaError_t launch_wide(ScanParams p, cudaStream_t st) {
    const SelectiveArgs& a = p.a;
    p.cblocks = (p.per + 32 / S - 1) / (32 / S);
    p.nblocks = (int)((a.N + NS - 1) / NS);
    const int64_t units = a.nseq * a.G * p.cblocks;
    if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto bytes = [](size_t nblocks) {
        return kWideWarps * sizeof(WideMem<E, Td, NS, S>) + nblocks * (NS / S) * 32 * 4 * (kBlocks ? 2 : 1);
    };
    const size_t shared = bytes(p.nblocks);
    // 6 CTAs an SM (168 registers), or 8 (128) where that makes fewer waves. 1024 tokens, 16 states, bf16, us
    // with 6 and with 8: 800 units 101, 105; 960 140, 132; 1280 165, 169; 1920 229, 224; 2560 286, 285 (as
    // many waves: 6); 3840 410, 403; 5120 557, 548; 10240 1070, 1049.
    // Blocks of states: in bf16 9 (96 registers; 128 states of 4 x 512 x 4096 575 us, 642 with 6; 64 states
    // of 16 x 512 x 5120 1175 and 1186), but in fp32 6, whose shared memory leaves room for fewer (32 states
    // of 16 x 256 x 4096 260 us, 302 with 9; 256 states of 8 x 128 x 5120 783 and 1176). With padded states 6
    // in bf16 too (20 states of 8 x 1024 x 5120 623 us, 695 with 9; 200 of 4 x 256 x 5120 586 and 759), unless B
    // and C are copied element by element, which gains from warps (17 states of 8 x 512 x 5120 416 and 394).
    constexpr int kCtas = kBlocks && sizeof(E) == 2 ? 9 : 6;
    const int care = care_of(a, NS);
    auto kernel = care == 2   ? wide_scan_kernel<E, Td, NS, S, kBlocks, 2, kCtas>
                  : care == 1 ? wide_scan_kernel<E, Td, NS, S, kBlocks, 1, kCtas>
                              : wide_scan_kernel<E, Td, NS, S, kBlocks, 0, kCtas>;
    if constexpr (kCtas == 9)
        if (care == 2 && p.bc_bytes >= 4) kernel = wide_scan_kernel<E, Td, NS, S, kBlocks, 2, 6>;
    if constexpr (!kBlocks)
        if ((units + 8 * 148 - 1) / (8 * 148) < (units + 6 * 148 - 1) / (6 * 148))
            kernel = care == 2   ? wide_scan_kernel<E, Td, NS, S, kBlocks, 2, 8>
                     : care == 1 ? wide_scan_kernel<E, Td, NS, S, kBlocks, 1, 8>
                                 : wide_scan_kernel<E, Td, NS, S, kBlocks, 0, 8>;
    const cudaError_t e = allow_shared(kernel, bytes(kBlocks ? kMaxSelectiveStates / NS : 1));
    if (e != cudaSuccess) return e;
    // From one wave of 8 CTAs an SM to four the order decides the tail; with more, short documents are better
    // spread between long ones. 8192 tokens, 16 states, bf16, us ranked and in the pack's order: 16 documents
    // of 2048 channels (2048 units) 139, 176; 16 of 4096 (4096) 236, 270; 40 of 2048 (5120) 142, 152; 48 of
    // 2048 (6144) 145, 146; 64 of 2048 (8192) 157, 149. Within a wave: 4 of 4096 (1024) 438, 341.
    p.ranked = a.cu && a.nseq <= kRanked && units > 8 * 148 && units <= 32 * 148;
    kernel<<<(unsigned)units, kWideWarps * 32, shared, st>>>(p);
    return cudaGetLastError();
}

// ---- few channels ------------------------------------------------------------
//
// A warp takes 64 / SL channels, SL lanes for a pair of channels, 4 states a lane (more than 4 SL
// states in blocks), and kCutTok tokens at a time: softplus and dt u are computed once per (token,
// channel) and shared through shared memory, each lane runs its 2 x 4 states through the tokens (two
// channels a lane halve the reads of B and C), and the lanes' parts of y are summed by exchanges that
// leave every lane kCutTok / SL tokens.
//
// The W = kCutWarps warps of a CTA take consecutive runs of kCutTok tokens of the same channels. Each
// runs from a state of zero and keeps, per token and state, C_t times the product of its decays so far
// (128 registers: one CTA an SM, which is faster than twice the warps with half the tokens each: 2048
// tokens of 2048 channels, 16 states, bf16 54 us for 63, 64 states in 8 groups 161 for 177; 16384 tokens
// in fp32 384 for 378). The entering states go from warp to warp as a chain, h <- (prod a) h + h_local,
// over shared memory and a named barrier of the two warps, so that the warps stay at different phases;
// with its entering state a warp adds sum_n (C_t prod a)[n] h[n] to each y_t, at two packed operations
// per pair of states and no second exponential.
//
// kSegments: with so few channels that most SMs would stay empty, a cluster of CTAs shares a unit's
// tokens, a segment each. Every CTA first runs its segment from a state of zero, without outputs, to
// what it leaves and the sum of its steps, whose exponential with A is its decay; after one barrier of
// the cluster each folds the segments before its own, over distributed shared memory, into its
// entering states, and runs its segment again with outputs. The exponentials are computed twice, on
// SMs that had none.
constexpr int kCutTok = 16, kCutWarps = 8;

template <typename E, typename Td, int SL>
struct CutMem {
    static constexpr int CH = 64 / SL, NS = 4 * SL;
    alignas(16) E u[2][kCutTok][CH];
    alignas(16) E z[2][kCutTok][CH];
    alignas(16) Td dt[2][kCutTok][CH];
    alignas(16) E B[2][kCutTok][NS];
    alignas(16) E C[2][kCutTok][NS];
    alignas(16) float4 s[kCutTok][CH / 2];    // dt, dt u of two channels
};

// 2 x 4 states of a lane (or their decays): [channel of the pair][pair of states]
struct States {
    float2 v[2][2];
    __device__ __forceinline__ void fill(float x) {
        v[0][0] = v[0][1] = v[1][0] = v[1][1] = both(x);
    }
    __device__ __forceinline__ void load(const float4* p) {
        const float4 a = p[0], b = p[32];
        v[0][0] = make_float2(a.x, a.y); v[0][1] = make_float2(a.z, a.w);
        v[1][0] = make_float2(b.x, b.y); v[1][1] = make_float2(b.z, b.w);
    }
    __device__ __forceinline__ void store(float4* p) const {
        p[0] = make_float4(v[0][0].x, v[0][0].y, v[0][1].x, v[0][1].y);
        p[32] = make_float4(v[1][0].x, v[1][0].y, v[1][1].x, v[1][1].y);
    }
};

template <typename E, typename Td, int SL, bool kSegments, int kCare>
__global__ void __launch_bounds__(kCutWarps * 32, 1) cut_scan_kernel(const __grid_constant__ ScanParams p) {
    constexpr int K = kCutTok, W = kCutWarps;
    constexpr int CL = 32 / SL, CH = 2 * CL, NS = 4 * SL;
    using Mem = CutMem<E, Td, SL>;
    extern __shared__ __align__(16) unsigned char smem[];
    const SelectiveArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int cp = lane % CL, j = lane / CL;             // pair of channels, states 4 j ..
    const int NB = p.nblocks;
    Mem& m = reinterpret_cast<Mem*>(smem)[warp];
    // by state block: the states entering the next round of W tiles; two slots a warp for what its
    // predecessor hands over. Segments: also what the segment leaves from a state of zero, and the sums
    // of its steps on their way from warp to warp.
    float4* const carry = reinterpret_cast<float4*>(smem + W * sizeof(Mem));
    float4* const slots = carry + NB * 64;
    float4* const leaves = slots + 2 * W * 64;
    float2* const sums = reinterpret_cast<float2*>(leaves + NB * 64);                   // [2 W + 1][32]

    const int rank = kSegments ? cluster_rank() : 0, ranks = kSegments ? cluster_size() : 1;
    const int64_t unit = blockIdx.x / ranks, per_seq = p.cblocks * a.G;
    const int64_t seq = p.ranked ? document_at(a.cu, a.nseq, unit / per_seq, (int)a.T, lane) : unit / per_seq;
    const int64_t g = unit % per_seq / p.cblocks, c0 = unit % p.cblocks * CH;
    const int64_t b = a.cu ? 0 : seq;
    int t0 = 0, t1 = (int)a.T;
    if (a.cu) {
        t0 = min(max(a.cu[seq], 0), t1);
        t1 = min(max(a.cu[seq + 1], 0), t1);
    }
    // the CTA's segment: whole rounds, as many for each rank but the last ones
    bool last = true;                                    // whether the sequence ends here
    const int first = t0;                                // of the sequence
    if constexpr (kSegments) {
        const int end = t1, part = (max(t1 - t0, 0) + ranks * W * K - 1) / (ranks * W * K) * (W * K);
        const int64_t from = t0 + (int64_t)rank * part;
        last = end > t0 ? from < end && from + part >= end : rank == 0;
        t1 = (int)min((int64_t)end, from + part);
        t0 = (int)min((int64_t)max(end, t0), from);
    }
    const int cols = (int)min(p.per - c0, (int64_t)CH);
    const int64_t d0 = g * p.per + c0;
    const int N = (int)a.N;
    const bool in0 = 2 * cp < cols, in1 = 2 * cp + 1 < cols;
    const int64_t da = d0 + (in0 ? 2 * cp : 0), db = d0 + (in1 ? 2 * cp + 1 : 0);   // the lane's channels
    const float2 skip = a.Dskip ? make_float2(a.Dskip[da], a.Dskip[db]) : both(0.f);
    const float2 bias = a.dt_bias ? make_float2(a.dt_bias[da], a.dt_bias[db]) : both(0.f);

    auto row_of = [&](const float* base, int64_t d, int nb, bool rates, float2& lo, float2& hi) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = nb * NS + j * 4 + i;
            v[i] = base && n < N ? base[d * N + n] : 0.f;
            if (rates) v[i] = rate_of(v[i]);
        }
        lo = make_float2(v[0], v[1]);
        hi = make_float2(v[2], v[3]);
    };
    const float* const init = a.init ? a.init + seq * a.D * N : nullptr;
    if (warp == 0) {
        for (int nb = 0; nb < NB; ++nb) {
            States h;
            row_of(init, da, nb, false, h.v[0][0], h.v[0][1]);
            row_of(init, db, nb, false, h.v[1][0], h.v[1][1]);
            h.store(carry + nb * 64 + lane);
            if (kSegments) {
                h.fill(0.f);
                h.store(leaves + nb * 64 + lane);
            }
        }
        if (kSegments) sums[2 * W * 32 + lane] = both(0.f);
    }

    const E* const ub = static_cast<const E*>(a.u) + b * a.us.batch + d0;
    const Td* const dtb = static_cast<const Td*>(a.dt) + b * a.dts.batch + d0;
    const E* const zb = a.z ? static_cast<const E*>(a.z) + b * a.zs.batch + d0 : nullptr;
    const E* const Bb = static_cast<const E*>(a.B) + b * a.Bs.batch + g * N;
    const E* const Cb = static_cast<const E*>(a.C) + b * a.Cs.batch + g * N;
    const int ur = (int)a.us.row, dtr = (int)a.dts.row, zr = (int)a.zs.row, Br = (int)a.Bs.row, Cr = (int)a.Cs.row;
    // the copies of the tile at token t, state block nb; u, dt, z (stage sr) with the first block
    auto issue = [&](int t, int nb, int sr, int sb, bool out) {
        const int n = min(t1 - t, K);
        if (n > 0) {
            if (nb == 0) {
                stage<K, CH>(&m.u[sr][0][0], ub + (int64_t)t * ur, ur, n, cols, lane, p.row_bytes);
                stage<K, CH>(&m.dt[sr][0][0], dtb + (int64_t)t * dtr, dtr, n, cols, lane, p.row_bytes);
                if (zb && out) stage<K, CH>(&m.z[sr][0][0], zb + (int64_t)t * zr, zr, n, cols, lane, p.row_bytes);
            }
            stage<K, NS>(&m.B[sb][0][0], Bb + (int64_t)t * Br + nb * NS, Br, n, N - nb * NS, lane, p.bc_bytes);
            if (out) stage<K, NS>(&m.C[sb][0][0], Cb + (int64_t)t * Cr + nb * NS, Cr, n, N - nb * NS, lane, p.bc_bytes);
        }
        copy_commit();
    };

    E* const yb = static_cast<E*>(a.y) + b * a.T * a.D + d0 + 2 * cp;
    const int64_t Dr = a.D;
    // all warps take part in every round of W tiles, those past the end too, which pass the states on
    const int rounds = t1 > t0 ? (t1 - t0 + W * K - 1) / (W * K) : 0;
    // y of a pair of channels: the lane's parts, and, summed over the SL lanes that share the pair by
    // exchanges of SL tokens each, the tokens q SL + j that the lane finishes
    float2 yv[K], ysum[K / SL] = {};
    auto give = [&](float2 v, int mask) {
        return make_float2(__shfl_xor_sync(0xffffffffu, v.x, mask), __shfl_xor_sync(0xffffffffu, v.y, mask));
    };
    auto gather = [&](int q) {
        const float2* const v = yv + q * SL;
        float2 r;
        if constexpr (SL == 4) {
            const bool up = j & 2, odd = j & 1;
            const float2 lo = add_(up ? v[2] : v[0], give(up ? v[0] : v[2], 2 * CL));
            const float2 hi = add_(up ? v[3] : v[1], give(up ? v[1] : v[3], 2 * CL));
            r = add_(odd ? hi : lo, give(odd ? lo : hi, CL));
        } else {
            static_assert(SL == 2 || SL == 4, "");
            const bool odd = j & 1;
            r = add_(odd ? v[1] : v[0], give(odd ? v[0] : v[1], CL));
        }
        ysum[q] = add_(ysum[q], r);
    };
    States A;
    auto rates = [&](int nb) {
        row_of(a.A, da, nb, true, A.v[0][0], A.v[0][1]);
        row_of(a.A, db, nb, true, A.v[1][0], A.v[1][1]);
    };
    if (NB == 1) rates(0);
    // The segment's rounds; kOut: with outputs, from the states in `carry`, else only what it leaves
    // from zero, in `leaves`, and the sum of its steps.
    auto run = [&](auto out, float4* const carry) {
        constexpr bool kOut = decltype(out)::value;
        int t = t0 + warp * K, sr = 0, sb = 0;
        if (rounds > 0) issue(t, 0, 0, 0, kOut);
        for (int it = 0; it < rounds; ++it, t += W * K, sr ^= 1) {
            const int n = min(t1 - t, K);
            for (int nb = 0; nb < NB; ++nb, sb ^= 1) {
                __syncwarp();                                // the stage that is filled next has been read
                if (nb + 1 < NB)
                    issue(t, nb + 1, sr ^ 1, sb ^ 1, kOut);
                else if (it + 1 < rounds)
                    issue(t + W * K, 0, sr ^ 1, sb ^ 1, kOut);
                else
                    copy_commit();
                copy_wait<1>();
                __syncwarp();
                if (NB > 1) rates(nb);
                if (n > 0) {
                    if (nb == 0) {
                        // once per (token, channel): the step and dt u; past the end both are 0, which
                        // leaves the state as it is
                        float2 v[K / SL];
#pragma unroll
                        for (int q = 0; q < K / SL; ++q) v[q] = add_(pair_of(&m.dt[sr][q * SL + j][2 * cp]), bias);
                        if (a.softplus) {
#pragma unroll
                            for (int q = 0; q < K / SL; ++q) v[q] = softplus(v[q]);
                        }
                        if (n < K) {
#pragma unroll
                            for (int q = 0; q < K / SL; ++q) v[q] = q * SL + j < n ? v[q] : both(0.f);
                        }
#pragma unroll
                        for (int q = 0; q < K / SL; ++q) {
                            const float2 du = mul_(v[q], pair_of(&m.u[sr][q * SL + j][2 * cp]));
                            m.s[q * SL + j][cp] = make_float4(v[q].x, du.x, v[q].y, du.y);
                        }
                    }
                    __syncwarp();
                }
                if (nb == 0) {
#pragma unroll
                    for (int q = 0; q < K / SL; ++q) ysum[q] = both(0.f);
                }
                States h, decay;
                float2 steps = both(0.f);                    // sum of the tile's
                float2 gc[K][2][2];                          // C_t times the decays up to t
                decay.fill(1.f);
                h.fill(0.f);
                if (n > 0) {
                    const E* const Bt = &m.B[sb][0][0] + j * 4;
                    const E* const Ct = &m.C[sb][0][0] + j * 4;
                    // exps of the next token ahead of the states of this one
                    float2 e[2][2][2];
                    float4 sk = m.s[0][cp];
                    auto exps = [&](float2 (&to)[2][2], const float4& s) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int i = 0; i < 2; ++i) to[c][i] = decay_of(both(c ? s.z : s.x), A.v[c][i]);
                    };
                    exps(e[0], sk);
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        const float4 s = sk;
                        float2 Bv[2], Cv[2];
                        quad_of(Bt + k * NS, Bv);
                        if (kOut) quad_of(Ct + k * NS, Cv);
                        if (k + 1 < K) {
                            sk = m.s[k + 1][cp];
                            exps(e[(k + 1) & 1], sk);
                        }
                        float part[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float2 du = both(c ? s.w : s.y);
                            float2 r = both(0.f);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float2 ek = e[k & 1][c][i];
                                h.v[c][i] = fma_(ek, h.v[c][i], mul_(du, Bv[i]));
                                decay.v[c][i] = k ? mul_(decay.v[c][i], ek) : ek;
                                if constexpr (kOut) {
                                    r = i ? fma_(Cv[i], h.v[c][i], r) : mul_(Cv[i], h.v[c][i]);
                                    gc[k][c][i] = mul_(Cv[i], decay.v[c][i]);
                                }
                            }
                            part[c] = r.x + r.y;
                        }
                        if constexpr (kOut) yv[k] = make_float2(part[0], part[1]);
                        else steps = add_(steps, make_float2(s.x, s.z));
                    }
                }
                // The entering state: the first warp's is what the last one left of the round before,
                // any other's comes from its predecessor (barrier w, and slot w by parity). The first
                // warp is told once a round. With one state block a predecessor cannot come to its
                // next hand-over before this one has gone round the chain, and need not wait; with
                // several, both wait, and the second slot keeps the next hand-over off this one.
                float4* const slot = slots + (((it * NB + nb) & 1) * W + warp) * 64 + lane;
                if (warp == 0) {
                    if (it > 0 && nb == 0) pair_wait<W>(0);
                } else {
                    pair_wait<W>(warp);
                }
                States in;
                in.load(warp == 0 ? carry + nb * 64 + lane : slot);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 2; ++i) h.v[c][i] = fma_(decay.v[c][i], in.v[c][i], h.v[c][i]);
                if constexpr (!kOut) {
                    if (nb == 0) {
                        float2* const sum = sums + (it & 1) * W * 32 + lane;
                        steps = add_(steps, warp == 0 ? sums[2 * W * 32 + lane] : sum[warp * 32]);
                        (warp + 1 < W ? sum[(warp + 1) * 32] : sums[2 * W * 32 + lane]) = steps;
                    }
                }
                if (warp + 1 < W) {
                    h.store(slot + 64);
                    if (NB == 1) pair_arrive<W>(warp + 1);
                    else pair_wait<W>(warp + 1);
                } else {
                    h.store(carry + nb * 64 + lane);
                    if (nb == NB - 1 && it + 1 < rounds) pair_arrive<W>(0);
                }
                if (kOut && n > 0) {
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        float part[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float2 r =
                                fma_(gc[k][c][1], in.v[c][1], mul_(gc[k][c][0], in.v[c][0]));
                            part[c] = r.x + r.y;
                        }
                        yv[k] = add_(yv[k], make_float2(part[0], part[1]));
                        if (k % SL == SL - 1) gather(k / SL);
                    }
                }
            }
            if (!kOut || n <= 0) continue;
            E* to = yb + (int64_t)(t + j) * (int)Dr;
            const int64_t step = SL * Dr;
#pragma unroll
            for (int q = 0; q < K / SL; ++q) {
                const float2 with = fma_(skip, pair_of(&m.u[sr][q * SL + j][2 * cp]), ysum[q]);
                ysum[q] = kCare == 0 || (kCare == 2 && a.Dskip) ? with : ysum[q];
            }
            if (zb) {
#pragma unroll
                for (int q = 0; q < K / SL; ++q) ysum[q] = mul_(ysum[q], silu(pair_of(&m.z[sr][q * SL + j][2 * cp])));
            }
            if (n == K && cols == CH && p.y_pairs) {
#pragma unroll
                for (int q = 0; q < K / SL; ++q, to += step) store_pair(to, ysum[q]);
            } else {
#pragma unroll
                for (int q = 0; q < K / SL; ++q, to += step)
                    if (q * SL + j < n) {
                        if (in0) store_elem(to, ysum[q].x);
                        if (in1) store_elem(to + 1, ysum[q].y);
                    }
            }
        }
        copy_wait<0>();
    };
    if constexpr (kSegments) {
        // What each segment leaves, then the fold of those before this one: the entering state
        run(std::false_type{}, leaves);
        cluster_arrive();
        cluster_wait();
        if (warp == 0) {
            for (int nb = 0; nb < NB; ++nb) {
                States h;
                h.load(carry + nb * 64 + lane);
                rates(nb);
                for (int q = 0; q < rank; ++q) {
                    const float2 sum = remote2(in_cta(sums + 2 * W * 32 + lane, q));
                    const uint32_t at = in_cta(leaves + nb * 64 + lane, q);
                    const float4 l0 = remote4(at), l1 = remote4(at + 32 * 16);
                    const float2 l[2][2] = {{make_float2(l0.x, l0.y), make_float2(l0.z, l0.w)},
                                            {make_float2(l1.x, l1.y), make_float2(l1.z, l1.w)}};
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            // not 0, however long the segment: an infinite state stays infinite
                            const float2 e = ex2(mul_(both(c ? sum.y : sum.x), A.v[c][i]));
                            h.v[c][i] = fma_(make_float2(fmaxf(e.x, FLT_MIN), fmaxf(e.y, FLT_MIN)), h.v[c][i], l[c][i]);
                        }
                }
                h.store(carry + nb * 64 + lane);
            }
        }
        cluster_arrive();
    }
    run(std::true_type{}, carry);
    if constexpr (kCare == 2) {
        __syncthreads();
        States h;
        h.load(carry + (NB - 1) * 64 + lane);
        const unsigned odd0 = __ballot_sync(0xffffffffu, h.v[0][1].y != 0.f) >> ((SL - 1) * CL);
        const unsigned odd1 = __ballot_sync(0xffffffffu, h.v[1][1].y != 0.f) >> ((SL - 1) * CL);
        unsigned which = 0;                              // bits of the pairs' channels, side by side
#pragma unroll
        for (int c = 0; c < CL; ++c) which |= (odd0 >> c & 1) << (2 * c) | (odd1 >> c & 1) << (2 * c + 1);
        which &= ~0u >> (32 - cols);
        if (which)
            sum_again<K, W, E, Td>(p, seq, g, d0, first, t0, t1, which,
                                   [](int k, int c) { return k % SL * CL + c / 2; });
    }
    // the warp that wrote the carried states last
    if (a.fin && last && warp == (rounds == 0 ? 0 : W - 1)) {
        for (int nb = 0; nb < NB; ++nb) {
            States h;
            h.load(carry + nb * 64 + lane);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float v[4] = {h.v[c][0].x, h.v[c][0].y, h.v[c][1].x, h.v[c][1].y};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = nb * NS + j * 4 + i;
                    if (n < N && (c ? in1 : in0)) a.fin[(seq * a.D + (c ? db : da)) * N + n] = v[i];
                }
            }
        }
    }
    if constexpr (kSegments) {
        __syncwarp();                                    // lanes part at the stores above; the barrier is for whole warps
        cluster_wait();                                  // others read this CTA's shared memory until here
    }
}

template <typename E, typename Td, int SL, bool kSegments>
cudaError_t launch_cut(ScanParams p, int64_t units, int ranks, cudaStream_t st) {
    constexpr int W = kCutWarps;
    constexpr auto bytes = [](size_t nblocks) {
        return W * sizeof(CutMem<E, Td, SL>) + (nblocks + 2 * W) * 64 * 16 +
               (kSegments ? nblocks * 64 * 16 + (2 * W + 1) * 32 * 8 : 0);
    };
    const size_t shared = bytes(p.nblocks);
    constexpr size_t most = bytes(SL == 4 ? kMaxSelectiveStates / 16 : 1);     // two lanes: up to 8 states
    static_assert(most <= 227 * 1024, "");
    const int care = care_of(p.a, 4 * SL);
    auto kernel = care == 2   ? cut_scan_kernel<E, Td, SL, kSegments, 2>
                  : care == 1 ? cut_scan_kernel<E, Td, SL, kSegments, 1>
                              : cut_scan_kernel<E, Td, SL, kSegments, 0>;
    const cudaError_t e = allow_shared(kernel, most);
    if (e != cudaSuccess) return e;
    // as in launch_wide, over one to five waves of a CTA an SM (8192 tokens, bf16: 16 documents of 512
    // channels, 48 states 149 us ranked, 169 not; 10 of 640, 32 states 151, 172); more make the uncut form
    p.ranked = p.a.cu && p.a.nseq <= kRanked && units > 148 && units <= 5 * 148;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = (unsigned)ranks;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3((unsigned)(units * ranks));
    config.blockDim = dim3(W * 32);
    config.dynamicSmemBytes = shared;
    config.stream = st;
    config.attrs = &cluster;
    config.numAttrs = kSegments ? 1 : 0;
    return cudaLaunchKernelEx(&config, kernel, p);
}

// SL: lanes for a pair of channels in the cut form; NS: states of a channel's lanes in the uncut one
template <typename E, typename Td, int SL, int NS>
cudaError_t launch_scan(ScanParams p, cudaStream_t st) {
    constexpr int CH = 64 / SL;
    const SelectiveArgs& a = p.a;
    const int64_t cblocks = (p.per + CH - 1) / CH, units = a.nseq * a.G * cblocks;
    const int64_t len = (a.T + (a.cu ? a.nseq : 1) - 1) / (a.cu ? a.nseq : 1);
    const int64_t tiles = (len + kWideTok - 1) / kWideTok;
    const int64_t rounds = (len + kCutWarps * kCutTok - 1) / (kCutWarps * kCutTok);
    constexpr int S = NS >= 8 ? 2 : 1;
    if (a.N <= NS) {
        // A CTA of the cut form fills an SM, so it is for units that one wave takes (2048 tokens, 16
        // states, bf16: 2048 channels 54 us cut, 100 uncut; 3200 channels 107 cut, 102 uncut), and for
        // sequences of a few tiles (64 tokens of 5120 channels 14 cut, 8 uncut).
        if (units > 148 || len <= 64) return launch_wide<E, Td, NS, S, false>(p, st);
    } else if constexpr (SL == 4) {
        // More states than a lane holds make up for few channels, and the uncut form reads their B and C
        // a block at a time. A round of a wave of the cut form takes about 1.5 times a tile of the uncut
        // one, whose tiles slow down above 6 units an SM (64 states: 1024 tokens of 10240 channels 418 us
        // cut, 499 uncut; 512 tokens of 81920 channels 1528 cut, 1186 uncut; 16 tokens of 8192 channels
        // 43 cut, 17 uncut).
        const int64_t waves = (units + 147) / 148, full = 6 * 148;
        if (2 * tiles * std::max(units, full) < 3 * waves * rounds * full)
            return launch_wide<E, Td, NS, S, true>(p, st);
    }
    p.cblocks = cblocks;
    p.nblocks = (int)((a.N + 4 * SL - 1) / (4 * SL));
    // Clusters of 8 and 4 such CTAs as long as the GPU has them at once (the SMs of a cluster lie
    // together) and the segments have a round each (15 states, bf16, 6720 tokens of 2 x 16 channels:
    // 258 us without, 61 with 8; 16 states, 8192 tokens of 512 channels: 200 without, 88 with 4). Two
    // segments would gain nothing, at 1.6 times the work.
    if (units <= 12 && rounds >= 8) return launch_cut<E, Td, SL, true>(p, units, 8, st);
    if (units <= 32 && rounds >= 4) return launch_cut<E, Td, SL, true>(p, units, 4, st);
    return launch_cut<E, Td, SL, false>(p, units, 1, st);
}

template <typename E, typename Td>
cudaError_t scan_any(const SelectiveArgs& a, cudaStream_t st) {
    if (a.nseq == 0 || (a.T == 0 && !a.fin)) return cudaSuccess;
    ScanParams p = {};
    p.a = a;
    p.per = a.D / a.G;
    auto pieces = [](const void* q, const ssd_strides_t& s, int64_t inner, int64_t es) {   // 16, 4 or less
        const int64_t all = (int64_t)(uintptr_t)q | s.batch * es | s.row * es | inner * es;
        return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : (int)es;
    };
    p.row_bytes = std::min(pieces(a.u, a.us, p.per, sizeof(E)), pieces(a.dt, a.dts, p.per, sizeof(Td)));
    if (a.z) p.row_bytes = std::min(p.row_bytes, pieces(a.z, a.zs, p.per, sizeof(E)));
    p.bc_bytes = std::min(pieces(a.B, a.Bs, a.N, sizeof(E)), pieces(a.C, a.Cs, a.N, sizeof(E)));
    p.y_pairs = p.per % 2 == 0 && aligned(a.y, 2 * sizeof(E));
    if (a.N <= 4) return launch_scan<E, Td, 2, 4>(p, st);
    if (a.N <= 8) return launch_scan<E, Td, 2, 8>(p, st);
    return launch_scan<E, Td, 4, 16>(p, st);
}

// ---- decoding --------------------------------------------------------------
//
// One or a few tokens per sequence from a state in HBM: the state's 8 b D N bytes bound it. L lanes
// share a channel, V states a lane and piece; a thread keeps the pieces of R batch rows of its
// channel in registers for all of the call's tokens, so that A (as large as one row's state) is read
// once for them and their loads are in flight together. What a (row, channel) needs once - the step,
// dt u, the gate - is computed by one of the L lanes and handed to the others; the rows' sums are
// exchanged so that each row ends in the lane that holds its u and gate. 128 sequences of 5120 channels,
// 16 states: 20 us for 90 MB (0.68 of the copy rate); all lanes computing the scalars 39 us.
constexpr int kStepThreads = 128;

struct StepParams {
    SelectiveArgs a;
    int64_t cblocks;             // CTAs along the channels
    int L;                       // lanes of a channel, a power of two up to 32
    bool a_wide, bc_wide;        // A (B and C) take loads of V elements
};

// V elements as they lie in memory
template <typename E, int V>
struct alignas(V * sizeof(E)) Piece {
    E v[V];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = E(0.f);
    }
    __device__ __forceinline__ void load(const E* p, bool wide) {
        if (V == 4 && wide) {
            if constexpr (sizeof(E) == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p);
            else *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = p[i];
        }
    }
    __device__ __forceinline__ void widen(float2 (&f)[2]) const { f[0] = pair_of(v); f[1] = pair_of(v + 2 % V); }
    __device__ __forceinline__ void widen(float (&f)[1]) const { f[0] = to_float(v[0]); }
};
__device__ __forceinline__ void load_piece(const float* p, float2 (&v)[2]) {
    const float4 q = __ldcs(reinterpret_cast<const float4*>(p));
    v[0] = make_float2(q.x, q.y);
    v[1] = make_float2(q.z, q.w);
}
__device__ __forceinline__ void load_piece(const float* p, float (&v)[1]) { v[0] = __ldcs(p); }
__device__ __forceinline__ void store_piece(float* p, const float2 (&v)[2]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
}
__device__ __forceinline__ void store_piece(float* p, const float (&v)[1]) { __stcs(p, v[0]); }

// R rows a thread, Q = R / (lanes that prepare them): a lane prepares rows q (R / Q) + j, q < Q.
// Addresses are walked: a row or token further costs an addition, where a product of 64-bit
// strides costs several instructions and made up half of the kernel's.
template <typename E, typename Td, int V, int KP, int R, int Q, bool kCare>
__global__ void __launch_bounds__(kStepThreads, V * KP * R <= 16 ? 6 : 1)
    step_kernel(const __grid_constant__ StepParams p) {
    constexpr int PL = R / Q;                            // lanes that prepare rows, at most L
    constexpr int M = V == 4 ? 2 : 1;                    // packed values of a piece
    using F = typename std::conditional<V == 4, float2, float>::type;
    const SelectiveArgs& a = p.a;
    const int L = p.L, j = threadIdx.x & (L - 1), N = (int)a.N;
    const int64_t d = blockIdx.x % p.cblocks * (kStepThreads / L) + threadIdx.x / L;
    const int64_t b0 = blockIdx.x / p.cblocks * R;
    const bool live = d < a.D;                           // whole groups of L lanes
    const int64_t dc = live ? d : 0;
    const int rows = live ? (int)min(a.b - b0, (int64_t)R) : 0;
    bool in[KP];
#pragma unroll
    for (int k = 0; k < KP; ++k) in[k] = (j + k * L) * V < N;

    F h[R][KP][M], A[KP][M];
    const int64_t next_row = a.D * N;
    float* const state = a.fin + (b0 * a.D + dc) * N + j * V;
    {
        const float* s = state;
#pragma unroll
        for (int r = 0; r < R; ++r, s += next_row)
#pragma unroll
            for (int k = 0; k < KP; ++k) {
                h[r][k][0] = h[r][k][M - 1] = all<F>(0.f);
                if (r < rows && in[k]) load_piece(s + k * L * V, h[r][k]);
            }
    }
    // the rows this lane prepares (with more lanes than rows the others repeat them); an absent row
    // reads the first's inputs
    const int own = j % PL;
    const Td* dtp[Q];
    const E* up[Q];
    const E* zp[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int64_t b = b0 + (q * PL + own < rows ? q * PL + own : 0);
        dtp[q] = static_cast<const Td*>(a.dt) + b * a.dts.batch + dc;
        up[q] = static_cast<const E*>(a.u) + b * a.us.batch + dc;
        zp[q] = a.z ? static_cast<const E*>(a.z) + b * a.zs.batch + dc : nullptr;
    }
    const int64_t g = a.G > 1 ? dc / (a.D / a.G) : 0;
    const E* Bt = static_cast<const E*>(a.B) + b0 * a.Bs.batch + g * N + j * V;
    const E* Ct = static_cast<const E*>(a.C) + b0 * a.Cs.batch + g * N + j * V;
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        Piece<float, V> q;
        q.zero();
        if (in[k]) q.load(a.A + dc * N + (j + k * L) * V, p.a_wide);
        q.widen(A[k]);
#pragma unroll
        for (int m = 0; m < M; ++m) A[k][m] = rate_of(A[k][m]);
    }
    const float skip = a.Dskip ? a.Dskip[dc] : 0.f, bias = a.dt_bias ? a.dt_bias[dc] : 0.f;
    E* y = static_cast<E*>(a.y) + (b0 + own) * a.T * a.D + dc;
    for (int64_t t = 0; t < a.T; ++t, y += a.D) {
        float dt[Q], u[Q], gate[Q], acc[R];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            dt[q] = to_float(*dtp[q]);
            u[q] = to_float(*up[q]);
            gate[q] = a.z ? to_float(*zp[q]) : 0.f;
            dtp[q] += a.dts.row;
            up[q] += a.us.row;
            zp[q] += a.zs.row;
        }
        Piece<E, V> Bv[R][KP], Cv[R][KP];                // all of B and C before the first use
        {
            const E* B = Bt;
            const E* C = Ct;
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    Bv[r][k].zero();
                    Cv[r][k].zero();
                    if (r < rows && in[k]) {
                        Bv[r][k].load(B + k * L * V, p.bc_wide);
                        Cv[r][k].load(C + k * L * V, p.bc_wide);
                    }
                }
                B += a.Bs.batch;
                C += a.Cs.batch;
            }
            Bt += a.Bs.row;
            Ct += a.Cs.row;
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            dt[q] += bias;
            if (a.softplus) dt[q] = softplus(dt[q]);
            gate[q] = a.z ? silu(gate[q]) : 1.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float dtr = __shfl_sync(0xffffffffu, dt[r / PL], r % PL, L);
            const float du = dtr * __shfl_sync(0xffffffffu, u[r / PL], r % PL, L);
            F sum = all<F>(0.f);
#pragma unroll
            for (int k = 0; k < KP; ++k) {
                F Bf[M], Cf[M];
                Bv[r][k].widen(Bf);
                Cv[r][k].widen(Cf);
                // pieces past N, which only the second half can be, stay 0 beside infinite steps
                const bool some = !kCare || k < KP / 2 || in[k];
                const float dtk = some ? dtr : 0.f, duk = some ? du : 0.f;
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    h[r][k][m] = fma_(decay_of(A[k][m], all<F>(dtk)), h[r][k][m], mul_(Bf[m], all<F>(duk)));
                    sum = fma_(Cf[m], h[r][k][m], sum);
                }
            }
            if constexpr (V == 4) acc[r] = sum.x + sum.y;
            else acc[r] = sum;
        }
        // lane j ends with the sums of the rows q PL + j % PL
        float sum[Q];
        if constexpr (PL == 4) {
            const bool up2 = j & 2, odd = j & 1;
            const float lo = (up2 ? acc[2] : acc[0]) + __shfl_xor_sync(0xffffffffu, up2 ? acc[0] : acc[2], 2);
            const float hi = (up2 ? acc[3] : acc[1]) + __shfl_xor_sync(0xffffffffu, up2 ? acc[1] : acc[3], 2);
            sum[0] = (odd ? hi : lo) + __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
        } else if constexpr (PL == 2) {
            const bool odd = j & 1;
#pragma unroll
            for (int q = 0; q < Q; ++q)
                sum[q] = (odd ? acc[2 * q + 1] : acc[2 * q]) +
                         __shfl_xor_sync(0xffffffffu, odd ? acc[2 * q] : acc[2 * q + 1], 1);
        } else {
#pragma unroll
            for (int q = 0; q < Q; ++q) sum[q] = acc[q];
        }
        for (int off = PL; off < L; off <<= 1)
#pragma unroll
            for (int q = 0; q < Q; ++q) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], off);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (j < PL && q * PL + own < rows) {
                const float with = fmaf(skip, u[q], sum[q]);
                store_elem(y + q * PL * a.T * a.D, (!kCare || a.Dskip ? with : sum[q]) * gate[q]);
            }
    }
    float* s = state;
#pragma unroll
    for (int r = 0; r < R; ++r, s += next_row)
#pragma unroll
        for (int k = 0; k < KP; ++k)
            if (r < rows && in[k]) store_piece(s + k * L * V, h[r][k]);
}

template <typename E, typename Td, int V, int KP, int R>
cudaError_t launch_rows(const StepParams& p, int64_t blocks, cudaStream_t st) {
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    // as many lanes prepare rows as there are, of the L lanes (32 with more than one piece)
    constexpr int kMost = R < 4 ? R : 4;
    const bool care = (int64_t)KP * p.L * V != p.a.N || !p.a.Dskip;
    auto kernel = care ? step_kernel<E, Td, V, KP, R, R / kMost, true> : step_kernel<E, Td, V, KP, R, R / kMost, false>;
    if constexpr (KP == 1 && R > 1) {
        if (p.L == 1) kernel = care ? step_kernel<E, Td, V, KP, R, R, true> : step_kernel<E, Td, V, KP, R, R, false>;
        if (p.L == 2)
            kernel = care ? step_kernel<E, Td, V, KP, R, R / 2, true> : step_kernel<E, Td, V, KP, R, R / 2, false>;
    }
    kernel<<<(unsigned)blocks, kStepThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename E, typename Td, int V, int KP>
cudaError_t launch_step(StepParams p, cudaStream_t st) {
    const SelectiveArgs& a = p.a;
    const int per_cta = kStepThreads / p.L;
    p.cblocks = (a.D + per_cta - 1) / per_cta;
    // Several batch rows a thread once that leaves every SM some CTAs; fewer rows finish sooner one each.
    constexpr int R = V * KP <= 4 ? 4 : 2;
    const int64_t grouped = p.cblocks * ((a.b + R - 1) / R);
    return grouped >= 4 * 148 ? launch_rows<E, Td, V, KP, R>(p, grouped, st)
                              : launch_rows<E, Td, V, KP, 1>(p, p.cblocks * a.b, st);
}

template <typename E, typename Td>
cudaError_t step_any(const SelectiveArgs& a, cudaStream_t st) {
    if (a.b == 0 || a.T == 0) return cudaSuccess;
    StepParams p = {};
    p.a = a;
    const bool wide = a.N % 4 == 0 && aligned(a.fin, 16);
    const int64_t pieces = wide ? a.N / 4 : a.N;
    p.L = 1;
    while (p.L < 32 && p.L < pieces) p.L *= 2;
    auto ok = [](const void* q, const ssd_strides_t& s) {
        return aligned(q, 4 * sizeof(E)) && s.batch % 4 == 0 && s.row % 4 == 0;
    };
    p.a_wide = aligned(a.A, 16);
    p.bc_wide = ok(a.B, a.Bs) && ok(a.C, a.Cs);
    const int64_t kp = (pieces + p.L - 1) / p.L;
    if (wide) return kp == 1 ? launch_step<E, Td, 4, 1>(p, st) : launch_step<E, Td, 4, 2>(p, st);
    if (kp == 1) return launch_step<E, Td, 1, 1>(p, st);
    if (kp == 2) return launch_step<E, Td, 1, 2>(p, st);
    if (kp <= 4) return launch_step<E, Td, 1, 4>(p, st);
    return launch_step<E, Td, 1, 8>(p, st);
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
