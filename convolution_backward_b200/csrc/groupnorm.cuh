// groupnorm.cuh -- what the two ways of group norm (groupnorm.cu: streaming over the whole
// GPU; groupnorm_cluster.cu: a group's values kept on the SMs of a cluster) have in common.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "gate_act.cuh"
#include "host_util.h"
#include "launchers.h"
#include "rowvec.cuh"

namespace dgrad {

// VEC elements as pairs of fp32 (of one element: the second of the pair is 0).
template <int VEC>
constexpr int gn_pairs() { return (VEC + 1) / 2; }

template <int EK, int VEC>
__device__ __forceinline__ void gn_unpack(const RowVec<EK, VEC>& v, float2 (&f)[gn_pairs<VEC>()])
{
    float a[VEC];
    v.unpack(a);
    if constexpr (VEC == 1) {
        f[0] = make_float2(a[0], 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) f[i] = make_float2(a[2 * i], a[2 * i + 1]);
    }
}

template <int EK, int VEC>
__device__ __forceinline__ void gn_pack(RowVec<EK, VEC>& v, const float2 (&f)[gn_pairs<VEC>()])
{
    float a[VEC];
    a[0] = f[0].x;
#pragma unroll
    for (int i = 1; i < VEC; ++i) a[i] = i % 2 ? f[i / 2].y : f[i / 2].x;
    v.pack(a);
}

template <int VEC>
__device__ __forceinline__ void gn_set(float2 (&f)[gn_pairs<VEC>()], float v)
{
#pragma unroll
    for (int i = 0; i < gn_pairs<VEC>(); ++i) f[i] = splat(v);
}

// gamma or beta at columns col .. col + VEC - 1.
template <int EK, int VEC>
__device__ __forceinline__ void gn_param(const void* src, int col, float constant, float2 (&f)[gn_pairs<VEC>()])
{
    if (src) {
        RowVec<EK, VEC> v;
        v.load(src, col);
        gn_unpack<EK, VEC>(v, f);
    } else {
        gn_set<VEC>(f, constant);
    }
}

// A thread's first column among groups of D: the group (counted from some first one) and how many
// of its columns are still to come.
struct GnGroup {
    int g, left;
    __device__ __forceinline__ GnGroup(int col, int D) : g(col / D), left(0) { left = D - (col - g * D); }
};

// f[i] = at(group of column i of the thread's).
template <int VEC, typename At>
__device__ __forceinline__ void gn_by_group(GnGroup k, int D, float2 (&f)[gn_pairs<VEC>()], At at)
{
    float a[2 * gn_pairs<VEC>()];
    a[2 * gn_pairs<VEC>() - 1] = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if (k.left == 0) {
            ++k.g;
            k.left = D;
        }
        a[i] = at(k.g);
        --k.left;
    }
#pragma unroll
    for (int i = 0; i < gn_pairs<VEC>(); ++i) f[i] = make_float2(a[2 * i], a[2 * i + 1]);
}

// put(group, value) for each of a thread's columns that is its group's first in the tile; start: the thread's first column
// is the tile's.
template <int VEC, typename Put>
__device__ __forceinline__ void gn_each_first(GnGroup k, int D, bool start, const float2 (&f)[gn_pairs<VEC>()], Put put)
{
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if (k.left == 0) {
            ++k.g;
            k.left = D;
        }
        if (k.left == D || (start && i == 0)) put(k.g, i % 2 ? f[i / 2].y : f[i / 2].x);
        --k.left;
    }
}

__device__ __forceinline__ float2 gn_minus(float2 v) { return make_float2(-v.x, -v.y); }

// A pair's products, each rounded: never one half of a multiply-add with what follows.
__device__ __forceinline__ float2 gn_mul_rounded(float2 a, float2 b) { return make_float2(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y)); }

// n and dz of a pair of elements.  relu's border is where z, formed as in the definition
// with every operation rounded, is zero; elsewhere one rounding less does not matter.
template <int ACT>
__device__ __forceinline__ void gn_dz(float2 x, float2 dy, float2 mean, float2 rstd, float2 gamma, float2 beta, float2& n,
                                      float2& dz)
{
    n = __fmul2_rn(__fadd2_rn(x, gn_minus(mean)), rstd);
    if constexpr (ACT == kNoAct) {
        dz = dy;
    } else {
        const float2 z = ACT == kRelu ? __fadd2_rn(gn_mul_rounded(n, gamma), beta) : ffma2(n, gamma, beta);
        float2 a, d;
        gate_act_grad<ACT>(z, a, d);
        dz = __fmul2_rn(dy, d);
    }
}

// dx from n and dz.  q = dz gamma is rounded before a is taken from it: a group of one value has
// q = a and n = 0, and dx = 0.
__device__ __forceinline__ float2 gn_dx(float2 n, float2 dz, float2 rstd, float2 gamma, float2 a, float2 b)
{
    return __fmul2_rn(rstd, ffma2(gn_minus(n), b, __fadd2_rn(gn_mul_rounded(dz, gamma), gn_minus(a))));
}

// Totals over the R rows of threads of each of tw columns: thread (r, c) brings columns c VEC and
// on.  buf: R tw floats, part: T floats, out: tw.  Whole block; out is complete on return.
// `parts` threads share a column's rows.
template <int T, int VEC>
__device__ __forceinline__ void column_totals(const float2 (&v)[gn_pairs<VEC>()], bool on, int r, int c, int R, int tw, int parts,
                                              float* buf, float* part, float* out)
{
    const int tid = threadIdx.x;
    __syncthreads();
    if (on) {
        float* to = buf + r * tw + c * VEC;
        if constexpr (VEC == 1) {
            *to = v[0].x;
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i)
                reinterpret_cast<float4*>(to)[i] = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
        }
    }
    __syncthreads();
    if (tw <= T) {
        const int p = tid / tw, ch = tid - p * tw;
        if (p < parts) {
            float s = 0.f;
#pragma unroll 4
            for (int q = p; q < R; q += parts) s += buf[q * tw + ch];
            (parts == 1 ? out : part)[tid] = s;
        }
        if (parts > 1) {
            __syncthreads();
            if (tid < tw) {
                float s = 0.f;
#pragma unroll 4
                for (int q = 0; q < parts; ++q) s += part[q * tw + tid];
                out[tid] = s;
            }
        }
    } else {
        for (int ch = tid; ch < tw; ch += T) {
            float s = 0.f;
#pragma unroll 4
            for (int q = 0; q < R; ++q) s += buf[q * tw + ch];
            out[ch] = s;
        }
    }
    __syncthreads();
}

// Threads that share a column in column_totals: as many steps before as after the parts meet.
inline int gn_column_parts(int T, int tw, int R)
{
    if (tw > T) return 1;
    int p = 1;
    while (p * p < R) ++p;
    return p < T / tw ? p : T / tw;
}

// Sums over the columns [c0, c1) that fall into each group: out[q][k - c0 / D] for group k, from
// in[q][row * in_row + column - c0], rows 0 .. rows - 1.  Whole block, T threads, in complete on entry; out is
// complete on return.
template <int T, int NQ>
__device__ __forceinline__ void group_totals(const float* in, int in_stride, int rows, int in_row, int c0, int c1, int D, float* out,
                                             int out_stride)
{
    const int first = c0 / D, n = (c1 - 1) / D - first + 1;
    int L = 32;
    while (L > 1 && L * n > T) L >>= 1;
    const int l = threadIdx.x & (L - 1);
    for (int base = 0; base < n; base += T / L) {
        const int j = base + static_cast<int>(threadIdx.x) / L;
        float s[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) s[q] = 0.f;
        if (j < n) {
            const int lo = max(c0, (first + j) * D) - c0, hi = min(c1, (first + j + 1) * D) - c0;
            for (int r = 0; r < rows; ++r)
#pragma unroll 4
                for (int c = lo + l; c < hi; c += L) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q) s[q] += in[q * in_stride + r * in_row + c];
                }
        }
        for (int o = L >> 1; o > 0; o >>= 1) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) s[q] += __shfl_xor_sync(0xFFFFFFFFu, s[q], o);
        }
        if (l == 0 && j < n) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) out[q * out_stride + j] = s[q];
        }
    }
    __syncthreads();
}

// (mean, rstd) of a group of m values, NaN where one of them, or a sum of them, is no finite number: with one infinity
// the mean alone would be infinite.
__device__ __forceinline__ float2 gn_statistics(float mean, float M2, float m, float eps)
{
    if (!isfinite(mean)) return splat(__int_as_float(0x7FC00000));
    return make_float2(mean, 1.0f / sqrtf(M2 / m + eps));
}

// Whether the mean of `count` values lies so far above their spread (M2: the squares about it) that its own roundings,
// some 2^-22 of it, show in the results: from 8 standard deviations on in fp32, from 128 in 16 bits, whose results are
// rounded to 2^-9 and 2^-12.
template <int EK>
__device__ __forceinline__ bool gn_far(float mean, float M2, float count)
{
    constexpr float far = EK == kF32 ? 8.f : 128.f;
    return mean * mean * count > far * far * M2 || (M2 == 0.f && mean != 0.f);   // squares of small values are 0
}

// A thread's own copies of 16 bytes from global to shared memory: nobody else reads them, so
// waiting for one's own is enough.  Loads through registers stalled on memory eight cycles of
// fourteen (gelu backward, 401408 x 96 bf16): there is no room for enough of them beside the
// parameters and sums.
__device__ __forceinline__ void gn_copy16(void* to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void gn_copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void gn_copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// f(element kind, channels a thread takes at a time) for run-time values.
template <typename F>
cudaError_t gn_with_kind(int ek, int vec, F f)
{
    if (ek == kF32) return vec == 1 ? f(std::integral_constant<int, kF32>{}, std::integral_constant<int, 1>{})
                                    : f(std::integral_constant<int, kF32>{}, std::integral_constant<int, 4>{});
    if (ek == kBF16) return vec == 1 ? f(std::integral_constant<int, kBF16>{}, std::integral_constant<int, 1>{})
                                     : f(std::integral_constant<int, kBF16>{}, std::integral_constant<int, 8>{});
    return vec == 1 ? f(std::integral_constant<int, kF16>{}, std::integral_constant<int, 1>{})
                    : f(std::integral_constant<int, kF16>{}, std::integral_constant<int, 8>{});
}

template <typename F>
cudaError_t gn_with_act(int act, F f)
{
    switch (act) {
    case kSilu: return f(std::integral_constant<int, kSilu>{});
    case kGelu: return f(std::integral_constant<int, kGelu>{});
    case kGeluTanh: return f(std::integral_constant<int, kGeluTanh>{});
    case kRelu: return f(std::integral_constant<int, kRelu>{});
    case kSigmoid: return f(std::integral_constant<int, kSigmoid>{});
    default: return f(std::integral_constant<int, kNoAct>{});
    }
}

constexpr size_t gn_up(size_t n) { return (n + 15) / 16 * 16; }

// The cluster way (groupnorm_cluster.cu): a slice of whole groups of a sample, tw channels at all
// positions, is taken by a cluster of K blocks, which keep it in shared memory.
struct GnSlices {
    int N, S;
    int C, G, D;
    int vec, cols, tw, slices;   // slices of tw channels (the last may be narrower); cols vectors each
    int R, parts;                // positions at a time, column_totals' parts
    int K;                       // blocks of a cluster
    int rpc;                     // positions of a block
    int cap;                     // steps of R positions, at most
    int ng;                      // groups of a slice, at most
    int smem;
};

// How the cluster way would cut a problem; false where the streaming way is to be taken.
bool gn_slices(int64_t N, int64_t S, int64_t C, int64_t G, int ek, bool backward, GnSlices* p);

cudaError_t launch_gn_cluster_forward(const GnSlices& p, const GnFwdArgs& a, cudaStream_t stream);
// cols: [N K][2][C], a block's sums of dz and of dz n over its positions.
cudaError_t launch_gn_cluster_backward(const GnSlices& p, const GnBwdArgs& a, float* cols, cudaStream_t stream);

}  // namespace dgrad
