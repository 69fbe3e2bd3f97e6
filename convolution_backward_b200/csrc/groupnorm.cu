// groupnorm.cu -- group norm over NHWC samples with an activation, forward and backward.
//
// Sample n of X holds S positions of C channels; a group is D = C/G adjacent channels at all
// positions, m = S*D values:
//     mean = sum(x) / m,  rstd = 1 / sqrt(sum((x - mean)^2) / m + eps)
//     z = (x - mean) * rstd * gamma + beta,  y = act(z)
// and with n = (x - mean) * rstd, dz = dy * act'(z) and q = dz * gamma
//     dx = rstd * (q - sum(q)/m - n * sum(q*n)/m)
//     dgamma = sum over samples and positions of dz * n,  dbeta = the same of dz.
// sum(q) over a group is the sum over its channels of gamma_c * (sum of dz over positions),
// and sum(q*n) alike, so the backward pass needs two sums per sample and channel only.
//
// A block takes some positions of one sample and a tile of channels.  A thread keeps its
// columns (one 16-byte vector of channels), with their parameters and sums in registers, and
// goes down the positions.  Squares are summed about the mean of the block's first positions,
// K: those are among the values, so the sum of squares about K is at most 1 + (positions a
// thread takes) times the one about the mean, and that bounds what cancellation costs
// wherever the mean lies.
// All sums and statistics are fp32 in a fixed order (no atomics): results repeat bit for bit.
#include "common.cuh"
#include "gate_act.cuh"
#include "host_util.h"
#include "launchers.h"
#include "rowvec.cuh"

namespace dgrad {
namespace {

constexpr int kGnBlock = 256;
constexpr int kGnTarget = 148 * 4;   // blocks that fill a B200
constexpr int kGnLeast = 4;          // positions a thread takes at least, where there are enough

// How a problem is cut.  Channel tiles need not end where groups do: a part is what a tile
// and a group share, numbered group + tile.
struct GnPlan {
    long long N, S;
    int C, G, D;
    int vec;        // channels per thread: 16 bytes of them, or one
    int cols;       // threads side by side along a tile's channels
    int tw;         // channels per tile
    int tiles;
    int R;          // positions a block takes at a time
    int P;          // blocks along the positions
    long long rpb;  // positions per block
    int parts;      // G + tiles - 1
};

GnPlan gn_plan(int64_t N, int64_t S, int64_t C, int64_t G, int ek)
{
    GnPlan p{};
    p.N = N;
    p.S = S;
    p.C = static_cast<int>(C);
    p.G = static_cast<int>(G);
    p.D = static_cast<int>(C / G);
    const int full = ek == kF32 ? 4 : 8;
    p.vec = C % full == 0 ? full : 1;
    const int nv = p.C / p.vec;
    p.tiles = (nv + kGnBlock - 1) / kGnBlock;
    p.cols = (nv + p.tiles - 1) / p.tiles;
    p.tiles = (nv + p.cols - 1) / p.cols;
    p.tw = p.cols * p.vec;
    p.R = kGnBlock / p.cols;
    const long long most = (S + static_cast<long long>(p.R) * kGnLeast - 1) / (static_cast<long long>(p.R) * kGnLeast);
    long long P = kGnTarget / (N * p.tiles > kGnTarget ? kGnTarget : N * p.tiles);
    if (P > most) P = most;
    if (P < 1) P = 1;
    p.rpb = (S + P - 1) / P;
    p.P = static_cast<int>((S + p.rpb - 1) / p.rpb);
    p.parts = p.G + p.tiles - 1;
    return p;
}

// The channels [lo, hi) that tile t shares with the j-th group that reaches into it.
struct GnTile {
    int c0, c1, g0, n;   // channels, first group, groups
    __device__ __forceinline__ GnTile(const GnPlan& p, int t)
    {
        c0 = t * p.tw;
        c1 = min(p.C, c0 + p.tw);
        g0 = c0 / p.D;
        n = (c1 - 1) / p.D - g0 + 1;
    }
};

// Sums of NQ quantities over rows [0, R) and over each part [max(c0, k D), min(c1, (k+1) D)) of
// the columns, from buf[q][r * tw + c - c0] to out[q][k - c0 / D].  Whole block, T threads; buf
// is complete on entry and out on return.
template <int NQ>
__device__ void part_sums(const float* buf, int q_stride, int R, int tw, int c0, int c1, int D, float* out, int out_stride,
                          float* warps)
{
    const int first = c0 / D, n = (c1 - 1) / D - first + 1;
    int L = kGnBlock;
    while (L > 1 && L * n > kGnBlock) L >>= 1;
    const int tid = threadIdx.x, l = tid & (L - 1);
    __syncthreads();
    for (int base = 0; base < n; base += kGnBlock / L) {
        const int j = base + tid / L;
        float s[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) s[q] = 0.f;
        if (j < n) {
            const int lo = max(c0, (first + j) * D) - c0, hi = min(c1, (first + j + 1) * D) - c0, w = hi - lo;
            int r = l / w, c = l - r * w;
            const int dr = L / w, dc = L - dr * w;
            while (r < R) {
#pragma unroll
                for (int q = 0; q < NQ; ++q) s[q] += buf[q * q_stride + r * tw + lo + c];
                r += dr;
                c += dc;
                if (c >= w) {
                    c -= w;
                    ++r;
                }
            }
        }
        for (int o = min(L, 32) >> 1; o > 0; o >>= 1) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) s[q] += __shfl_xor_sync(0xFFFFFFFFu, s[q], o);
        }
        if (L > 32) {
            if ((tid & 31) == 0) {
#pragma unroll
                for (int q = 0; q < NQ; ++q) warps[q * (kGnBlock / 32) + (tid >> 5)] = s[q];
            }
            __syncthreads();
            if (l == 0) {
                for (int w = 1; w < L / 32; ++w) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q) s[q] += warps[q * (kGnBlock / 32) + (tid >> 5) + w];
                }
            }
        }
        if (l == 0 && j < n) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) out[q * out_stride + j] = s[q];
        }
        __syncthreads();
    }
}

// One thread's columns and rows.
template <int EK, int VEC>
struct GnThread {
    using V = RowVec<EK, VEC>;
    int col, r;        // first channel, first position of the block's
    bool on;
    long long row0, row1;
    long long n;
    __device__ __forceinline__ GnThread(const GnPlan& p, const GnTile& t)
    {
        const int c = threadIdx.x % p.cols;
        r = threadIdx.x / p.cols;
        col = t.c0 + c * VEC;
        on = r < p.R && col < t.c1;
        n = blockIdx.x / p.P;
        row0 = (blockIdx.x - n * p.P) * p.rpb;
        row1 = min(p.S, row0 + p.rpb);
    }
    __device__ __forceinline__ long long at(const GnPlan& p, long long row) const { return (n * p.S + row) * p.C + col; }
};

template <int EK, int VEC>
__device__ __forceinline__ void load_params(const void* src, int col, float constant, float (&f)[VEC])
{
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = constant;
    if (src) {
        RowVec<EK, VEC> v;
        v.load(src, col);
        v.unpack(f);
    }
}

// Reads of this many rows are under way at a time.
template <int VEC>
constexpr int gn_unroll() { return VEC == 1 ? 8 : 4; }

struct GnFwd {
    GnPlan p;
    float eps;
    const void* x;
    const void* gamma;
    const void* beta;
    void* y;
    float* part;    // [N][P][parts] pairs (mean, sum of squares about it)
    float* mean;    // [N][G]
    float* rstd;
    int* status;
};

template <int EK, int VEC>
__global__ void __launch_bounds__(kGnBlock) gn_stats_kernel(const GnFwd a)
{
    __shared__ float buf[2 * kGnBlock * VEC];
    __shared__ float sums[2 * kGnBlock * VEC];
    __shared__ float shift[kGnBlock * VEC];
    __shared__ float warps[2 * kGnBlock / 32];
    const GnPlan& p = a.p;
    const GnTile tile(p, blockIdx.y);
    const GnThread<EK, VEC> th(p, tile);
    constexpr int Q = kGnBlock * VEC;
    pdl_wait();
    pdl_trigger();
    const int place = th.r * p.tw + th.col - tile.c0;
    const long long first = min(th.row1 - th.row0, static_cast<long long>(p.R));
    if (th.on) {
        float f[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = 0.f;
        if (th.r < first) {
            RowVec<EK, VEC> v;
            v.load(a.x, th.at(p, th.row0 + th.r));
            v.unpack(f);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (th.col + i < tile.c1) buf[place + i] = f[i];
    }
    part_sums<1>(buf, Q, p.R, p.tw, tile.c0, tile.c1, p.D, shift, Q, warps);
    float K[VEC], s1[VEC], s2[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int g = min(th.col + i, tile.c1 - 1) / p.D;
        const int w = min(tile.c1, (g + 1) * p.D) - max(tile.c0, g * p.D);
        K[i] = shift[g - tile.g0] / (static_cast<float>(w) * static_cast<float>(first));
        s1[i] = 0.f;
        s2[i] = 0.f;
    }
    if (th.on) {
        constexpr int U = gn_unroll<VEC>();
        long long row = th.row0 + th.r;
        for (; row + (U - 1) * p.R < th.row1; row += U * p.R) {
            RowVec<EK, VEC> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u].load(a.x, th.at(p, row + u * p.R));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[VEC];
                v[u].unpack(f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = f[i] - K[i];
                    s1[i] += d;
                    s2[i] = fmaf(d, d, s2[i]);
                }
            }
        }
        for (; row < th.row1; row += p.R) {
            RowVec<EK, VEC> v;
            float f[VEC];
            v.load(a.x, th.at(p, row));
            v.unpack(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = f[i] - K[i];
                s1[i] += d;
                s2[i] = fmaf(d, d, s2[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            buf[place + i] = s1[i];
            buf[Q + place + i] = s2[i];
        }
    }
    part_sums<2>(buf, Q, p.R, p.tw, tile.c0, tile.c1, p.D, sums, Q, warps);
    float2* out = reinterpret_cast<float2*>(a.part) + static_cast<long long>(blockIdx.x) * p.parts;
    for (int j = threadIdx.x; j < tile.n; j += kGnBlock) {
        const int g = tile.g0 + j;
        const int w = min(tile.c1, (g + 1) * p.D) - max(tile.c0, g * p.D);
        const float count = static_cast<float>(w) * static_cast<float>(th.row1 - th.row0);
        const float k = shift[j] / (static_cast<float>(w) * static_cast<float>(first));
        const float d = sums[j] / count;
        const float sq = fmaf(-sums[j], d, sums[Q + j]);
        out[g + blockIdx.y] = make_float2(k + d, sq < 0.f ? 0.f : sq);
    }
}

// Joins the parts of every group: a warp each.
__global__ void __launch_bounds__(kGnBlock) gn_join_kernel(const GnFwd a)
{
    const GnPlan& p = a.p;
    const long long ng = static_cast<long long>(blockIdx.x) * (kGnBlock / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    if (ng >= p.N * p.G) return;
    const long long n = ng / p.G;
    const int g = static_cast<int>(ng - n * p.G);
    const int t0 = g * p.D / p.tw, t1 = (g * p.D + p.D - 1) / p.tw, nt = t1 - t0 + 1;
    const float2* part = reinterpret_cast<const float2*>(a.part) + n * p.P * p.parts;
    const int e1 = nt * p.P;
    const float m0 = part[g + t0].x;
    const float m = static_cast<float>(p.D) * static_cast<float>(p.S);
    float mean = m0, sq = 0.f;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {   // the mean; the squares about it
        float s = 0.f;
        for (int e = lane; e < e1; e += 32) {
            const int b = e / nt, t = t0 + e - b * nt;
            const int w = min(min(p.C, (t + 1) * p.tw), (g + 1) * p.D) - max(t * p.tw, g * p.D);
            const long long rows = min(p.S, (b + 1) * p.rpb) - b * p.rpb;
            const float count = static_cast<float>(w) * static_cast<float>(rows);
            const float2 v = part[static_cast<long long>(b) * p.parts + g + t];
            const float d = v.x - mean;
            s += pass ? fmaf(d * count, d, v.y) : d * count;
        }
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (pass)
            sq = s;
        else
            mean = m0 + s / m;
    }
    if (lane == 0 && store_ok(a.mean, p.N * p.G * 4, a.mean + ng, 4, a.status)) {
        a.mean[ng] = mean;
        a.rstd[ng] = 1.0f / sqrtf(sq / m + a.eps);
    }
}

// z of a thread's columns, and what they need.
template <int EK, int VEC>
struct GnColumns {
    float mean[VEC], rstd[VEC], gamma[VEC], beta[VEC];
    __device__ __forceinline__ void load(const GnPlan& p, long long n, int col, const float* m, const float* r,
                                         const void* g, const void* b)
    {
        load_params<EK, VEC>(g, col, 1.f, gamma);
        load_params<EK, VEC>(b, col, 0.f, beta);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const long long k = n * p.G + (col + i) / p.D;
            mean[i] = m[k];
            rstd[i] = r[k];
        }
    }
};

template <int EK, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock) gn_apply_kernel(const GnFwd a)
{
    const GnPlan& p = a.p;
    const GnTile tile(p, blockIdx.y);
    const GnThread<EK, VEC> th(p, tile);
    constexpr int es = elem_bytes<EK>();
    pdl_wait();
    pdl_trigger();
    if (!th.on) return;
    GnColumns<EK, VEC> c;
    c.load(p, th.n, th.col, a.mean, a.rstd, a.gamma, a.beta);
#pragma unroll
    for (int i = 0; i < VEC; ++i) c.rstd[i] *= c.gamma[i];
    const long long bytes = p.N * p.S * p.C * es;
    constexpr int U = gn_unroll<VEC>();
    for (long long row = th.row0 + th.r; row < th.row1; row += U * p.R) {
        RowVec<EK, VEC> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (row + u * p.R < th.row1) v[u].load(a.x, th.at(p, row + u * p.R));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row + u * p.R >= th.row1) break;
            float f[VEC];
            v[u].unpack(f);
            if constexpr (VEC == 1) {
                f[0] = gate_act<ACT>(splat(fmaf(f[0] - c.mean[0], c.rstd[0], c.beta[0]))).x;
            } else {
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    const float2 d = __fadd2_rn(make_float2(f[i], f[i + 1]), make_float2(-c.mean[i], -c.mean[i + 1]));
                    const float2 z = ffma2(d, make_float2(c.rstd[i], c.rstd[i + 1]), make_float2(c.beta[i], c.beta[i + 1]));
                    const float2 y = gate_act<ACT>(z);
                    f[i] = y.x;
                    f[i + 1] = y.y;
                }
            }
            v[u].pack(f);
            const long long at = th.at(p, row + u * p.R);
            if (store_ok(a.y, bytes, static_cast<char*>(a.y) + at * es, VEC == 1 ? es : 16, a.status)) v[u].store(a.y, at);
        }
    }
}

// ----------------------------------------------------------------- backward

struct GnBwd {
    GnPlan p;
    const void* dy;
    const void* x;
    const void* gamma;
    const void* beta;
    const float* mean;
    const float* rstd;
    void* dx;
    void* dgamma;
    void* dbeta;
    float* cols;    // [N][P][2][C]: sums of dz and of dz * n over a block's positions
    float* part;    // [N][P][parts] pairs: the sums of gamma times those over a part's channels
    float* ab;      // [N][G] pairs: sum(q)/m, sum(q*n)/m
    int* status;
};

// n and dz of a pair of elements.  relu's border is where z, formed as in the definition
// with every operation rounded, is zero; elsewhere one rounding less does not matter.
template <int ACT>
__device__ __forceinline__ void gn_dz(float2 x, float2 dy, float2 mean, float2 rstd, float2 gamma, float2 beta, float2& n,
                                      float2& dz)
{
    n = __fmul2_rn(__fadd2_rn(x, make_float2(-mean.x, -mean.y)), rstd);
    if constexpr (ACT == kNoAct) {
        dz = dy;
    } else {
        const float2 z = ACT == kRelu ? __fadd2_rn(__fmul2_rn(n, gamma), beta) : ffma2(n, gamma, beta);
        float2 a, d;
        gate_act_grad<ACT>(z, a, d);
        dz = __fmul2_rn(dy, d);
    }
}

template <int EK, int VEC, int ACT>
__device__ __forceinline__ void gn_dz_row(const RowVec<EK, VEC>& xv, const RowVec<EK, VEC>& dv, const GnColumns<EK, VEC>& c,
                                          float (&n)[VEC], float (&dz)[VEC])
{
    float x[VEC], dy[VEC];
    xv.unpack(x);
    dv.unpack(dy);
    if constexpr (VEC == 1) {
        float2 nn, dd;
        gn_dz<ACT>(splat(x[0]), splat(dy[0]), splat(c.mean[0]), splat(c.rstd[0]), splat(c.gamma[0]), splat(c.beta[0]), nn, dd);
        n[0] = nn.x;
        dz[0] = dd.x;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            float2 nn, dd;
            gn_dz<ACT>(make_float2(x[i], x[i + 1]), make_float2(dy[i], dy[i + 1]), make_float2(c.mean[i], c.mean[i + 1]),
                       make_float2(c.rstd[i], c.rstd[i + 1]), make_float2(c.gamma[i], c.gamma[i + 1]),
                       make_float2(c.beta[i], c.beta[i + 1]), nn, dd);
            n[i] = nn.x;
            n[i + 1] = nn.y;
            dz[i] = dd.x;
            dz[i + 1] = dd.y;
        }
    }
}

template <int EK, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock) gn_sums_kernel(const GnBwd a)
{
    __shared__ float buf[2 * kGnBlock * VEC];
    __shared__ float sums[2 * kGnBlock * VEC];
    __shared__ float warps[2 * kGnBlock / 32];
    const GnPlan& p = a.p;
    const GnTile tile(p, blockIdx.y);
    const GnThread<EK, VEC> th(p, tile);
    constexpr int Q = kGnBlock * VEC;
    pdl_wait();
    pdl_trigger();
    if (th.on) {
        GnColumns<EK, VEC> c;
        c.load(p, th.n, th.col, a.mean, a.rstd, a.gamma, a.beta);
        float A[VEC], B[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) A[i] = B[i] = 0.f;
        constexpr int U = gn_unroll<VEC>() / 2;
        for (long long row = th.row0 + th.r; row < th.row1; row += U * p.R) {
            RowVec<EK, VEC> xv[U], dv[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (row + u * p.R < th.row1) {
                    xv[u].load(a.x, th.at(p, row + u * p.R));
                    dv[u].load(a.dy, th.at(p, row + u * p.R));
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (row + u * p.R >= th.row1) break;
                float n[VEC], dz[VEC];
                gn_dz_row<EK, VEC, ACT>(xv[u], dv[u], c, n, dz);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    A[i] += dz[i];
                    B[i] = fmaf(dz[i], n[i], B[i]);
                }
            }
        }
        const int place = th.r * p.tw + th.col - tile.c0;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            buf[place + i] = A[i];
            buf[Q + place + i] = B[i];
        }
    }
    part_sums<2>(buf, Q, p.R, p.tw, tile.c0, tile.c1, 1, sums, Q, warps);
    float* cols = a.cols + static_cast<long long>(blockIdx.x) * 2 * p.C;
    for (int c = threadIdx.x; c < tile.c1 - tile.c0; c += kGnBlock) {
        float g[1];
        load_params<EK, 1>(a.gamma, tile.c0 + c, 1.f, g);
        cols[tile.c0 + c] = sums[c];
        cols[p.C + tile.c0 + c] = sums[Q + c];
        buf[c] = sums[c] * g[0];
        buf[Q + c] = sums[Q + c] * g[0];
    }
    part_sums<2>(buf, Q, 1, p.tw, tile.c0, tile.c1, p.D, sums, Q, warps);
    float2* out = reinterpret_cast<float2*>(a.part) + static_cast<long long>(blockIdx.x) * p.parts;
    for (int j = threadIdx.x; j < tile.n; j += kGnBlock) out[tile.g0 + j + blockIdx.y] = make_float2(sums[j], sums[Q + j]);
}

// A warp per group adds its parts; the blocks behind them add the columns of dgamma and
// dbeta over samples and blocks, eight adjacent channels each.
template <int EK>
__global__ void __launch_bounds__(kGnBlock) gn_join_grads_kernel(const GnBwd a, int group_blocks)
{
    __shared__ float2 buf[kGnBlock];
    const GnPlan& p = a.p;
    pdl_wait();
    pdl_trigger();
    if (static_cast<int>(blockIdx.x) < group_blocks) {
        const long long ng = static_cast<long long>(blockIdx.x) * (kGnBlock / 32) + (threadIdx.x >> 5);
        const int lane = threadIdx.x & 31;
        if (ng >= p.N * p.G) return;
        const long long n = ng / p.G;
        const int g = static_cast<int>(ng - n * p.G);
        const int t0 = g * p.D / p.tw, t1 = (g * p.D + p.D - 1) / p.tw, nt = t1 - t0 + 1;
        const float2* part = reinterpret_cast<const float2*>(a.part) + n * p.P * p.parts;
        float sa = 0.f, sb = 0.f;
        for (int e = lane; e < nt * p.P; e += 32) {
            const int b = e / nt, t = t0 + e - b * nt;
            const float2 v = part[static_cast<long long>(b) * p.parts + g + t];
            sa += v.x;
            sb += v.y;
        }
        for (int o = 16; o > 0; o >>= 1) {
            sa += __shfl_xor_sync(0xFFFFFFFFu, sa, o);
            sb += __shfl_xor_sync(0xFFFFFFFFu, sb, o);
        }
        const float m = static_cast<float>(p.D) * static_cast<float>(p.S);
        if (lane == 0) reinterpret_cast<float2*>(a.ab)[ng] = make_float2(sa / m, sb / m);
        return;
    }
    constexpr int kAcross = 8, kDown = kGnBlock / kAcross;
    const int c = (static_cast<int>(blockIdx.x) - group_blocks) * kAcross + threadIdx.x % kAcross;
    float2 s = make_float2(0.f, 0.f);
    if (c < p.C)
        for (long long b = threadIdx.x / kAcross; b < p.N * p.P; b += kDown) {
            s.x += a.cols[b * 2 * p.C + c];
            s.y += a.cols[b * 2 * p.C + p.C + c];
        }
    buf[threadIdx.x] = s;
    for (int o = kGnBlock / 2; o >= kAcross; o >>= 1) {
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < o) {
            buf[threadIdx.x].x += buf[threadIdx.x + o].x;
            buf[threadIdx.x].y += buf[threadIdx.x + o].y;
        }
    }
    if (threadIdx.x < kAcross && c < p.C) {
        constexpr int es = elem_bytes<EK>();
        RowVec<EK, 1> v;
        float f[1] = {buf[threadIdx.x].y};
        v.pack(f);
        if (a.dgamma && store_ok(a.dgamma, p.C * es, static_cast<char*>(a.dgamma) + c * es, es, a.status)) v.store(a.dgamma, c);
        f[0] = buf[threadIdx.x].x;
        v.pack(f);
        if (a.dbeta && store_ok(a.dbeta, p.C * es, static_cast<char*>(a.dbeta) + c * es, es, a.status)) v.store(a.dbeta, c);
    }
}

template <int EK, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock) gn_dx_kernel(const GnBwd a)
{
    const GnPlan& p = a.p;
    const GnTile tile(p, blockIdx.y);
    const GnThread<EK, VEC> th(p, tile);
    constexpr int es = elem_bytes<EK>();
    pdl_wait();
    pdl_trigger();
    if (!th.on) return;
    GnColumns<EK, VEC> c;
    c.load(p, th.n, th.col, a.mean, a.rstd, a.gamma, a.beta);
    float qa[VEC], qb[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float2 v = reinterpret_cast<const float2*>(a.ab)[th.n * p.G + (th.col + i) / p.D];
        qa[i] = v.x;
        qb[i] = v.y;
    }
    const long long bytes = p.N * p.S * p.C * es;
    constexpr int U = gn_unroll<VEC>() / 2;
    for (long long row = th.row0 + th.r; row < th.row1; row += U * p.R) {
        RowVec<EK, VEC> xv[U], dv[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (row + u * p.R < th.row1) {
                xv[u].load(a.x, th.at(p, row + u * p.R));
                dv[u].load(a.dy, th.at(p, row + u * p.R));
            }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row + u * p.R >= th.row1) break;
            float n[VEC], dz[VEC];
            gn_dz_row<EK, VEC, ACT>(xv[u], dv[u], c, n, dz);
            // q is rounded before a is taken from it: a group of one value has q = a, and dx = 0
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                dz[i] = c.rstd[i] * fmaf(-n[i], qb[i], __fmul_rn(dz[i], c.gamma[i]) - qa[i]);
            xv[u].pack(dz);
            const long long at = th.at(p, row + u * p.R);
            if (store_ok(a.dx, bytes, static_cast<char*>(a.dx) + at * es, VEC == 1 ? es : 16, a.status)) xv[u].store(a.dx, at);
        }
    }
}

// ----------------------------------------------------------------- launches

constexpr size_t kAlign = 16;
size_t up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

// Kernel K<EK, VEC, ACT> for run-time values, through F: f(integral constants).
template <typename F>
cudaError_t with_kind(int ek, int vec, F f)
{
    if (ek == kF32) return vec == 1 ? f(std::integral_constant<int, kF32>{}, std::integral_constant<int, 1>{})
                                    : f(std::integral_constant<int, kF32>{}, std::integral_constant<int, 4>{});
    if (ek == kBF16) return vec == 1 ? f(std::integral_constant<int, kBF16>{}, std::integral_constant<int, 1>{})
                                     : f(std::integral_constant<int, kBF16>{}, std::integral_constant<int, 8>{});
    return vec == 1 ? f(std::integral_constant<int, kF16>{}, std::integral_constant<int, 1>{})
                    : f(std::integral_constant<int, kF16>{}, std::integral_constant<int, 8>{});
}

template <typename F>
cudaError_t with_act_host(int act, F f)
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

}  // namespace

size_t groupnorm_forward_workspace_bytes(int64_t N, int64_t S, int64_t C, int64_t G, int ek)
{
    const GnPlan p = gn_plan(N, S, C, G, ek);
    return up(static_cast<size_t>(N) * p.P * p.parts * 8) + up(static_cast<size_t>(N) * G * 8);
}

cudaError_t launch_groupnorm_forward(const GnFwdArgs& a, cudaStream_t stream)
{
    GnFwd f{gn_plan(a.N, a.S, a.C, a.G, a.ek), a.eps, a.X, a.gamma, a.beta, a.Y, nullptr, a.mean, a.rstd, a.status};
    const GnPlan& p = f.p;
    f.part = a.ws;
    float* stats = a.ws + up(static_cast<size_t>(p.N) * p.P * p.parts * 8) / 4;
    if (!f.mean) f.mean = stats;
    if (!f.rstd) f.rstd = stats + p.N * p.G;
    const dim3 grid(static_cast<unsigned>(p.N * p.P), static_cast<unsigned>(p.tiles));
    cudaError_t e = with_kind(a.ek, p.vec, [&](auto ek, auto vec) {
        return launch_kernel(gn_stats_kernel<ek.value, vec.value>, grid, dim3(kGnBlock), 0, stream, 1, f);
    });
    if (e != cudaSuccess) return e;
    const unsigned joins = static_cast<unsigned>((p.N * p.G + kGnBlock / 32 - 1) / (kGnBlock / 32));
    e = launch_kernel(gn_join_kernel, dim3(joins), dim3(kGnBlock), 0, stream, 1, f);
    if (e != cudaSuccess) return e;
    return with_kind(a.ek, p.vec, [&](auto ek, auto vec) {
        return with_act_host(a.act, [&](auto act) {
            return launch_kernel(gn_apply_kernel<ek.value, vec.value, act.value>, grid, dim3(kGnBlock), 0, stream, 1, f);
        });
    });
}

size_t groupnorm_backward_workspace_bytes(int64_t N, int64_t S, int64_t C, int64_t G, int ek)
{
    const GnPlan p = gn_plan(N, S, C, G, ek);
    return up(static_cast<size_t>(N) * p.P * 2 * C * 4) + up(static_cast<size_t>(N) * p.P * p.parts * 8) +
           up(static_cast<size_t>(N) * G * 8);
}

cudaError_t launch_groupnorm_backward(const GnBwdArgs& a, cudaStream_t stream)
{
    GnBwd f{gn_plan(a.N, a.S, a.C, a.G, a.ek), a.dY, a.X, a.gamma, a.beta, a.mean, a.rstd, a.dX, a.dgamma, a.dbeta,
            nullptr, nullptr, nullptr, a.status};
    const GnPlan& p = f.p;
    f.cols = a.ws;
    f.part = f.cols + up(static_cast<size_t>(p.N) * p.P * 2 * p.C * 4) / 4;
    f.ab = f.part + up(static_cast<size_t>(p.N) * p.P * p.parts * 8) / 4;
    const dim3 grid(static_cast<unsigned>(p.N * p.P), static_cast<unsigned>(p.tiles));
    cudaError_t e = with_kind(a.ek, p.vec, [&](auto ek, auto vec) {
        return with_act_host(a.act, [&](auto act) {
            return launch_kernel(gn_sums_kernel<ek.value, vec.value, act.value>, grid, dim3(kGnBlock), 0, stream, 1, f);
        });
    });
    if (e != cudaSuccess) return e;
    const int groups = static_cast<int>((p.N * p.G + kGnBlock / 32 - 1) / (kGnBlock / 32));
    const int params = a.dgamma || a.dbeta ? (p.C + 7) / 8 : 0;
    auto join = a.ek == kF32 ? gn_join_grads_kernel<kF32> : a.ek == kBF16 ? gn_join_grads_kernel<kBF16> : gn_join_grads_kernel<kF16>;
    e = launch_kernel(join, dim3(static_cast<unsigned>(groups + params)), dim3(kGnBlock), 0, stream, 1, f, groups);
    if (e != cudaSuccess) return e;
    return with_kind(a.ek, p.vec, [&](auto ek, auto vec) {
        return with_act_host(a.act, [&](auto act) {
            return launch_kernel(gn_dx_kernel<ek.value, vec.value, act.value>, grid, dim3(kGnBlock), 0, stream, 1, f);
        });
    });
}

}  // namespace dgrad
