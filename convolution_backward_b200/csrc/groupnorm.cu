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
// Two ways.  Where a slice of channels of a sample fits the shared memory of a cluster of blocks
// and there are enough of them, groupnorm_cluster.cu reads every input once, in one launch.  Here is
// the streaming way, for every other size: two passes over the inputs with a join between them.
// A block takes some positions of one sample and a tile of channels.  A thread keeps its
// columns (one 16-byte vector of channels), with their parameters and sums in registers, and
// goes down the positions.  Squares are summed about the thread's own first value: the sum of k
// squares about one of the k values is at most 1 + k times the one about their mean, and that
// bounds what cancellation costs wherever the mean lies.  From there means and squares about them
// are joined, over the block's threads and over the blocks:
//     mean = sum count_i mean_i / sum count_i,  M2 = sum (M2_i + count_i (mean_i - mean)^2).
// Means are joined as differences to one of them, so that a mean far above the spread is rounded to its own
// last place and no more, and that of equal values is the value.
// All sums and statistics are fp32 in a fixed order (no atomics): results repeat bit for bit.
#include "groupnorm.cuh"

namespace dgrad {
namespace {

constexpr int kGnBlock = 256;
// Blocks that fill a B200, forward (16 x 4096 x 384 silu, bf16: 34.2 us, with 444 blocks 38.3, 888 37.6; fp32 60.1, 54.3, 58.9;
// 32 x 12544 x 96 bf16 49.8, 55.5, 51.4, fp32 87.8, 92.4, 83.7) and backward (32 x 12544 x 96 gelu: 93 us, with 444 97.6, 592 98.4).
constexpr int kGnTarget = 148 * 4, kGnTargetBwd = 148 * 2;
constexpr int kGnLeast = 4;          // positions a thread takes at least, where there are enough

// How a problem is cut.  Channel tiles need not end where groups do: a part is what a tile
// and a group share, numbered group + tile.
struct GnPlan {
    int N, S;
    int C, G, D;
    int vec;        // channels per thread: 16 bytes of them, or one
    int cols;       // threads side by side along a tile's channels
    int tw;         // channels per tile
    int tiles;
    int R;          // positions a block takes at a time
    int down;       // column_totals' parts
    int P;          // blocks along the positions
    int rpb;        // positions per block
    int parts;      // G + tiles - 1
};

GnPlan gn_plan(int64_t N, int64_t S, int64_t C, int64_t G, int ek, bool backward)
{
    GnPlan p{};
    p.N = static_cast<int>(N);
    p.S = static_cast<int>(S);
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
    p.down = gn_column_parts(kGnBlock, p.tw, p.R);
    const long long most = (S + static_cast<long long>(p.R) * kGnLeast - 1) / (static_cast<long long>(p.R) * kGnLeast);
    const long long target = backward ? kGnTargetBwd : kGnTarget;
    long long P = target / (N * p.tiles > target ? target : N * p.tiles);
    if (P > most) P = most;
    if (P < 1) P = 1;
    p.rpb = static_cast<int>((S + P - 1) / P);
    p.P = static_cast<int>((S + p.rpb - 1) / p.rpb);
    p.parts = p.G + p.tiles - 1;
    return p;
}

// A thread's place: columns col .. of the tile's [c0, c1), `steps` positions from the first on.
template <int EK, int VEC>
struct GnThread {
    int c0, c1, g0, groups;
    int col, c, r, steps;
    bool on;
    int n, row0, rows;
    long long first, stride;    // elements
    GnGroup group;              // of col, counted from g0
    __device__ __forceinline__ GnThread(const GnPlan& p, int t) : group(0, 1)
    {
        c0 = t * p.tw;
        c1 = min(p.C, c0 + p.tw);
        g0 = c0 / p.D;
        groups = (c1 - 1) / p.D - g0 + 1;
        r = threadIdx.x / p.cols;
        c = threadIdx.x - r * p.cols;
        col = c0 + c * VEC;
        on = r < p.R && col < c1;
        n = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.P));
        row0 = (static_cast<int>(blockIdx.x) - n * p.P) * p.rpb;
        rows = min(p.S - row0, p.rpb);
        steps = on && r < rows ? (rows - r + p.R - 1) / p.R : 0;
        first = (static_cast<long long>(n) * p.S + row0 + r) * p.C + col;
        stride = static_cast<long long>(p.R) * p.C;
        group = GnGroup(col - g0 * p.D, p.D);
    }
    // Channels of group k inside the tile.
    __device__ __forceinline__ int width(const GnPlan& p, int k) const { return min(c1, (k + 1) * p.D) - max(c0, k * p.D); }
};

constexpr int kAhead = 8;        // 16-byte copies a thread has under way

// All of a thread's steps down NT tensors.  16-byte vectors come through the thread's places in
// `ring` (kAhead of them), single elements directly, eight of each tensor at a time (backward 6 x 4000 x
// 1001 bf16, no activation: 89 us, with four 129).  The constructor has the first ones sent for; run calls
// f(element, vectors) for every step.
template <int EK, int VEC, int NT>
struct GnDown {
    static constexpr int es = elem_bytes<EK>(), W = kAhead / NT;
    const void* src[NT];
    const char* from[NT];
    char* mine;
    long long step;
    int coming;       // steps not yet under way

    __device__ __forceinline__ char* place(int slot, int i) const { return mine + (slot * NT + i) * kGnBlock * 16; }
    __device__ __forceinline__ void bring(int slot)
    {
        if (coming > 0) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                gn_copy16(place(slot, i), from[i]);
                from[i] += step;
            }
        }
        --coming;
        gn_copy_commit();
    }
    __device__ __forceinline__ GnDown(const void* const (&s)[NT], const GnThread<EK, VEC>& t, char* ring)
        : mine(ring + threadIdx.x * 16), step(t.stride * es), coming(t.steps)
    {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            src[i] = s[i];
            from[i] = static_cast<const char*>(s[i]) + t.first * es;
        }
        if constexpr (VEC > 1) {
#pragma unroll
            for (int w = 0; w < W; ++w) bring(w);
        }
    }
    template <typename F>
    __device__ __forceinline__ void run(const GnThread<EK, VEC>& t, F f)
    {
        long long at = t.first;
        int left = t.steps;
        if constexpr (VEC == 1) {
            constexpr int U = 8;
            for (; left >= U; left -= U) {
                RowVec<EK, 1> v[U][NT];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < NT; ++i) v[u][i].load(src[i], at + u * t.stride);
#pragma unroll
                for (int u = 0; u < U; ++u) f(at + u * t.stride, v[u]);
                at += U * t.stride;
            }
            for (; left > 0; --left) {
                RowVec<EK, 1> v[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i) v[i].load(src[i], at);
                f(at, v);
                at += t.stride;
            }
        } else {
            // two steps at a time: the chains of one fill the gaps in the other's
            int w = 0;
            for (; left >= 2; left -= 2) {
                gn_copy_wait<W - 2>();
                RowVec<EK, VEC> v[2][NT];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < NT; ++i) v[u][i].load(place(w + u, i), 0);
                f(at, v[0]);
                f(at + t.stride, v[1]);
                at += 2 * t.stride;
                bring(w);
                bring(w + 1);
                w = w + 2 == W ? 0 : w + 2;
            }
            if (left > 0) {
                gn_copy_wait<0>();
                RowVec<EK, VEC> v[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i) v[i].load(place(w, i), 0);
                f(at, v);
            }
            gn_copy_wait<0>();
        }
    }
};

// Shared memory of a kernel that sums: the ring, and when that is done with, four times Q floats (Q:
// a block's columns) and one a thread.
constexpr int gn_ring(int vec) { return vec == 1 ? 0 : kAhead * kGnBlock * 16; }
constexpr int gn_shared(int vec)
{
    const int sums = (4 * kGnBlock * vec + kGnBlock) * 4;
    return sums > gn_ring(vec) ? sums : gn_ring(vec);
}

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

// The squares about the mean, of squares about another value: not below zero, infinite where those are
// (and the mean's part is too), NaN where they are.
__device__ __forceinline__ float left_of(float squares, float about)
{
    return squares == __int_as_float(0x7F800000) ? squares : about < 0.f ? 0.f : about;
}

// Four blocks an SM: with the registers that the compiler takes by itself the loads of single elements wait for each other
// (3 x 1961 x 1001 fp32 27.0 us, 21.6 so; vectors take the same time either way).
template <int EK, int VEC>
__global__ void __launch_bounds__(kGnBlock, 4) gn_stats_kernel(const GnFwd a)
{
    constexpr int Q = kGnBlock * VEC, NP = gn_pairs<VEC>();
    __shared__ __align__(16) char mem[gn_shared(VEC)];
    float* const buf = reinterpret_cast<float*>(mem);
    float* const out = buf + Q;
    float* const mean = out + Q;
    float* const part = mean + Q;
    __shared__ float one[Q];
    const GnPlan& p = a.p;
    const GnThread<EK, VEC> t(p, blockIdx.y);
    pdl_wait();
    pdl_trigger();
    const void* const src[1] = {a.x};
    GnDown<EK, VEC, 1> down(src, t, mem);
    float2 K[NP], s1[NP], s2[NP];
    gn_set<VEC>(K, 0.f);
    gn_set<VEC>(s1, 0.f);
    gn_set<VEC>(s2, 0.f);
    if (t.steps > 0) {
        RowVec<EK, VEC> v;
        v.load(a.x, t.first);
        gn_unpack<EK, VEC>(v, K);
#pragma unroll
        for (int i = 0; i < NP; ++i) K[i] = gn_minus(K[i]);
    }
    down.run(t, [&](long long, const RowVec<EK, VEC>(&v)[1]) {
        float2 f[NP];
        gn_unpack<EK, VEC>(v[0], f);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float2 d = __fadd2_rn(f[i], K[i]);
            s1[i] = __fadd2_rn(s1[i], d);
            s2[i] = ffma2(d, d, s2[i]);
        }
    });
    // a column's mean and squares about it; the block's mean of every group; the squares about that
    const float k = static_cast<float>(t.steps), rk = t.steps > 0 ? 1.f / k : 0.f;
    float2 w[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const float2 d = __fmul2_rn(s1[i], splat(rk));
        const float2 about = ffma2(gn_minus(s1[i]), d, s2[i]);
        s2[i] = make_float2(left_of(s2[i].x, about.x), left_of(s2[i].y, about.y));
        w[i] = __fadd2_rn(d, gn_minus(K[i]));
    }
    // the means less one of them, each group's own (of the middle row of threads: some steps' mean, not a single value
    // that may lie far from all others)
    if (t.on && t.r == (min(p.R, t.rows) >> 1)) gn_each_first<VEC>(t.group, p.D, t.c == 0, w, [&](int g, float v) { one[g] = v; });
    __syncthreads();
    if (t.on) {
        gn_by_group<VEC>(t.group, p.D, w, [&](int g) { return one[g]; });
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float2 above = gn_minus(__fadd2_rn(K[i], w[i]));
            K[i] = ffma2(s1[i], splat(rk), above);
            s1[i] = ffma2(above, splat(k), s1[i]);
        }
    }
    column_totals<kGnBlock, VEC>(s1, t.on, t.r, t.c, p.R, p.tw, p.down, buf, part, out);
    group_totals<kGnBlock, 1>(out, Q, 1, p.tw, t.c0, t.c1, p.D, mean, Q);
    for (int j = threadIdx.x; j < t.groups; j += kGnBlock)
        mean[j] /= static_cast<float>(t.width(p, t.g0 + j)) * static_cast<float>(t.rows);
    __syncthreads();
    if (t.on) {
        gn_by_group<VEC>(t.group, p.D, s1, [&](int g) { return mean[g]; });
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float2 d = __fadd2_rn(K[i], gn_minus(s1[i]));
            s2[i] = ffma2(__fmul2_rn(d, splat(k)), d, s2[i]);
        }
    }
    column_totals<kGnBlock, VEC>(s2, t.on, t.r, t.c, p.R, p.tw, p.down, buf, part, out);
    group_totals<kGnBlock, 1>(out, Q, 1, p.tw, t.c0, t.c1, p.D, buf, Q);
    float2* to = reinterpret_cast<float2*>(a.part) + static_cast<long long>(blockIdx.x) * p.parts;
    for (int j = threadIdx.x; j < t.groups; j += kGnBlock) to[t.g0 + j + blockIdx.y] = make_float2(one[j] + mean[j], buf[j]);
}

// Joins the parts of every group: a warp each.
__global__ void __launch_bounds__(kGnBlock) gn_join_kernel(const GnFwd a)
{
    const GnPlan& p = a.p;
    const int ng = static_cast<int>(blockIdx.x * (kGnBlock / 32) + (threadIdx.x >> 5));
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    if (ng < 0 || ng >= p.N * p.G) return;
    const int n = ng / p.G, g = ng - n * p.G;
    const int t0 = g * p.D / p.tw, t1 = (g * p.D + p.D - 1) / p.tw, nt = t1 - t0 + 1;
    const float2* part = reinterpret_cast<const float2*>(a.part) + static_cast<long long>(n) * p.P * p.parts;
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
            const int rows = min(p.S - b * p.rpb, p.rpb);
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
    if (lane == 0 && store_ok(a.mean, static_cast<long long>(p.N) * p.G * 4, a.mean + ng, 4, a.status)) {
        const float2 stats = gn_statistics(mean, sq, m, a.eps);
        a.mean[ng] = stats.x;
        a.rstd[ng] = stats.y;
    }
}

template <int EK, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock) gn_apply_kernel(const GnFwd a)
{
    constexpr int es = elem_bytes<EK>(), NP = gn_pairs<VEC>();
    __shared__ __align__(16) char ring[gn_ring(VEC) + 16];
    const GnPlan& p = a.p;
    const GnThread<EK, VEC> t(p, blockIdx.y);
    // the kernels before this one only read X: its first vectors are sent for while they end
    const void* const src[1] = {a.x};
    GnDown<EK, VEC, 1> down(src, t, ring);
    pdl_wait();
    pdl_trigger();
    if (!t.on) return;
    float2 mean[NP], scale[NP], beta[NP];
    const long long at = static_cast<long long>(t.n) * p.G + t.g0;
    gn_by_group<VEC>(t.group, p.D, mean, [&](int g) { return a.mean[at + g]; });
    gn_by_group<VEC>(t.group, p.D, scale, [&](int g) { return a.rstd[at + g]; });
    gn_param<EK, VEC>(a.gamma, t.col, 1.f, beta);
#pragma unroll
    for (int i = 0; i < NP; ++i) scale[i] = __fmul2_rn(scale[i], beta[i]);
    gn_param<EK, VEC>(a.beta, t.col, 0.f, beta);
    const long long bytes = static_cast<long long>(p.N) * p.S * p.C * es;
    down.run(t, [&](long long e, RowVec<EK, VEC>(&v)[1]) {
        float2 f[NP];
        gn_unpack<EK, VEC>(v[0], f);
#pragma unroll
        for (int i = 0; i < NP; ++i) f[i] = gate_act<ACT>(ffma2(__fadd2_rn(f[i], gn_minus(mean[i])), scale[i], beta[i]));
        gn_pack<EK, VEC>(v[0], f);
        if (store_ok(a.y, bytes, static_cast<char*>(a.y) + e * es, VEC * es, a.status)) v[0].store(a.y, e);
    });
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
    float* cols;    // [N][P][2][C]: sums of dz and of dz * n over a block's positions
    float* part;    // [N][P][parts] pairs: the sums of gamma times those over a part's channels
    float* ab;      // [N][G] pairs: sum(q)/m, sum(q*n)/m
    int* status;
};

// What dz needs of a thread's columns.
template <int EK, int VEC>
struct GnColumns {
    static constexpr int NP = gn_pairs<VEC>();
    float2 mean[NP], rstd[NP], gamma[NP], beta[NP];
    __device__ __forceinline__ GnColumns(const GnBwd& a, const GnThread<EK, VEC>& t)
    {
        const long long at = static_cast<long long>(t.n) * a.p.G + t.g0;
        gn_by_group<VEC>(t.group, a.p.D, mean, [&](int g) { return a.mean[at + g]; });
        gn_by_group<VEC>(t.group, a.p.D, rstd, [&](int g) { return a.rstd[at + g]; });
        gn_param<EK, VEC>(a.gamma, t.col, 1.f, gamma);
        gn_param<EK, VEC>(a.beta, t.col, 0.f, beta);
    }
    template <int ACT>
    __device__ __forceinline__ void slope(const RowVec<EK, VEC>& xv, const RowVec<EK, VEC>& dv, float2 (&n)[NP], float2 (&dz)[NP]) const
    {
        float2 x[NP];
        gn_unpack<EK, VEC>(xv, x);
        gn_unpack<EK, VEC>(dv, dz);
#pragma unroll
        for (int i = 0; i < NP; ++i) gn_dz<ACT>(x[i], dz[i], mean[i], rstd[i], gamma[i], beta[i], n[i], dz[i]);
    }
};

template <int EK, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock, 2) gn_sums_kernel(const GnBwd a)
{
    constexpr int Q = kGnBlock * VEC, NP = gn_pairs<VEC>();
    __shared__ __align__(16) char mem[gn_shared(VEC)];
    float* const buf = reinterpret_cast<float*>(mem);
    float* const out = buf + 2 * Q;
    float* const part = out + 2 * Q;
    float* const sums = buf;
    const GnPlan& p = a.p;
    const GnThread<EK, VEC> t(p, blockIdx.y);
    pdl_wait();
    pdl_trigger();
    const void* const src[2] = {a.x, a.dy};
    GnDown<EK, VEC, 2> down(src, t, mem);
    float2 A[NP], B[NP];
    gn_set<VEC>(A, 0.f);
    gn_set<VEC>(B, 0.f);
    if (t.on) {
        const GnColumns<EK, VEC> c(a, t);
        down.run(t, [&](long long, const RowVec<EK, VEC>(&v)[2]) {
            float2 n[NP], dz[NP];
            c.template slope<ACT>(v[0], v[1], n, dz);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                A[i] = __fadd2_rn(A[i], dz[i]);
                B[i] = ffma2(dz[i], n[i], B[i]);
            }
        });
    }
    column_totals<kGnBlock, VEC>(A, t.on, t.r, t.c, p.R, p.tw, p.down, buf, part, out);
    column_totals<kGnBlock, VEC>(B, t.on, t.r, t.c, p.R, p.tw, p.down, buf, part, out + Q);
    float* cols = a.cols + static_cast<long long>(blockIdx.x) * 2 * p.C + t.c0;
    for (int c = threadIdx.x; c < t.c1 - t.c0; c += kGnBlock) {
        float2 g[1];
        gn_param<EK, 1>(a.gamma, t.c0 + c, 1.f, g);
        cols[c] = out[c];
        cols[p.C + c] = out[Q + c];
        out[c] *= g[0].x;
        out[Q + c] *= g[0].x;
    }
    __syncthreads();
    group_totals<kGnBlock, 2>(out, Q, 1, p.tw, t.c0, t.c1, p.D, sums, Q);
    float2* to = reinterpret_cast<float2*>(a.part) + static_cast<long long>(blockIdx.x) * p.parts;
    for (int j = threadIdx.x; j < t.groups; j += kGnBlock) to[t.g0 + j + blockIdx.y] = make_float2(sums[j], sums[Q + j]);
}

// A warp per group adds its parts.
__global__ void __launch_bounds__(kGnBlock) gn_join_sums_kernel(const GnBwd a)
{
    const GnPlan& p = a.p;
    const int ng = static_cast<int>(blockIdx.x * (kGnBlock / 32) + (threadIdx.x >> 5));
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    if (ng < 0 || ng >= p.N * p.G) return;
    const int n = ng / p.G, g = ng - n * p.G;
    const int t0 = g * p.D / p.tw, t1 = (g * p.D + p.D - 1) / p.tw, nt = t1 - t0 + 1;
    const float2* part = reinterpret_cast<const float2*>(a.part) + static_cast<long long>(n) * p.P * p.parts;
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
}

// dgamma and dbeta of eight adjacent channels: columns of [rows][2][C] fp32 sums.
struct GnParams {
    const float* cols;
    long long rows;
    int C;
    void* dgamma;
    void* dbeta;
    int* status;
};
constexpr int kAcross = 8;
template <int EK>
__device__ __forceinline__ void gn_params(const GnParams& a, int block, float2* buf)
{
    constexpr int kDown = kGnBlock / kAcross, es = elem_bytes<EK>();
    const int c = block * kAcross + threadIdx.x % kAcross;
    float2 s = make_float2(0.f, 0.f);
    if (c < a.C) {
        const float* at = a.cols + c;
#pragma unroll 4
        for (long long b = threadIdx.x / kAcross; b < a.rows; b += kDown) {
            s.x += at[b * 2 * a.C];
            s.y += at[b * 2 * a.C + a.C];
        }
    }
    buf[threadIdx.x] = s;
    for (int o = kGnBlock / 2; o >= kAcross; o >>= 1) {
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < o) {
            buf[threadIdx.x].x += buf[threadIdx.x + o].x;
            buf[threadIdx.x].y += buf[threadIdx.x + o].y;
        }
    }
    if (threadIdx.x < kAcross && c < a.C) {
        RowVec<EK, 1> v;
        float f[1] = {buf[threadIdx.x].y};
        v.pack(f);
        if (a.dgamma && store_ok(a.dgamma, a.C * es, static_cast<char*>(a.dgamma) + c * es, es, a.status)) v.store(a.dgamma, c);
        f[0] = buf[threadIdx.x].x;
        v.pack(f);
        if (a.dbeta && store_ok(a.dbeta, a.C * es, static_cast<char*>(a.dbeta) + c * es, es, a.status)) v.store(a.dbeta, c);
    }
}

// Behind the cluster way.
template <int EK>
__global__ void __launch_bounds__(kGnBlock) gn_params_kernel(const GnParams a)
{
    __shared__ float2 buf[kGnBlock];
    pdl_wait();
    pdl_trigger();
    gn_params<EK>(a, static_cast<int>(blockIdx.x), buf);
}

template <int EK, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock, 2) gn_dx_kernel(const GnBwd a, const GnParams params, int blocks)
{
    constexpr int es = elem_bytes<EK>(), NP = gn_pairs<VEC>(), kBuf = kGnBlock * 8;
    __shared__ __align__(16) char ring[gn_ring(VEC) > kBuf ? gn_ring(VEC) : kBuf];
    const GnPlan& p = a.p;
    if (static_cast<int>(blockIdx.x) >= blocks) {    // the blocks behind those of dX
        pdl_wait();
        pdl_trigger();
        if (blockIdx.y == 0) gn_params<EK>(params, static_cast<int>(blockIdx.x) - blocks, reinterpret_cast<float2*>(ring));
        return;
    }
    const GnThread<EK, VEC> t(p, blockIdx.y);
    const void* const src[2] = {a.x, a.dy};
    GnDown<EK, VEC, 2> down(src, t, ring);     // as above: read by the kernels before this one
    pdl_wait();
    pdl_trigger();
    if (!t.on) return;
    const GnColumns<EK, VEC> c(a, t);
    float2 qa[NP], qb[NP];
    const float2* ab = reinterpret_cast<const float2*>(a.ab) + static_cast<long long>(t.n) * p.G + t.g0;
    gn_by_group<VEC>(t.group, p.D, qa, [&](int g) { return ab[g].x; });
    gn_by_group<VEC>(t.group, p.D, qb, [&](int g) { return ab[g].y; });
    const long long bytes = static_cast<long long>(p.N) * p.S * p.C * es;
    down.run(t, [&](long long at, RowVec<EK, VEC>(&v)[2]) {
        float2 n[NP], dz[NP];
        c.template slope<ACT>(v[0], v[1], n, dz);
#pragma unroll
        for (int i = 0; i < NP; ++i) dz[i] = gn_dx(n[i], dz[i], c.rstd[i], c.gamma[i], qa[i], qb[i]);
        gn_pack<EK, VEC>(v[0], dz);
        if (store_ok(a.dx, bytes, static_cast<char*>(a.dx) + at * es, VEC * es, a.status)) v[0].store(a.dx, at);
    });
}

}  // namespace

size_t groupnorm_forward_workspace_bytes(int64_t N, int64_t S, int64_t C, int64_t G, int ek)
{
    GnSlices s;
    if (gn_slices(N, S, C, G, ek, false, &s)) return 0;
    const GnPlan p = gn_plan(N, S, C, G, ek, false);
    return gn_up(static_cast<size_t>(N) * p.P * p.parts * 8) + gn_up(static_cast<size_t>(N) * G * 8);
}

cudaError_t launch_groupnorm_forward(const GnFwdArgs& a, cudaStream_t stream)
{
    GnSlices s;
    if (gn_slices(a.N, a.S, a.C, a.G, a.ek, false, &s)) return launch_gn_cluster_forward(s, a, stream);
    GnFwd f{gn_plan(a.N, a.S, a.C, a.G, a.ek, false), a.eps, a.X, a.gamma, a.beta, a.Y, nullptr, a.mean, a.rstd, a.status};
    const GnPlan& p = f.p;
    f.part = a.ws;
    float* stats = a.ws + gn_up(static_cast<size_t>(p.N) * p.P * p.parts * 8) / 4;
    if (!f.mean) f.mean = stats;
    if (!f.rstd) f.rstd = stats + static_cast<int64_t>(p.N) * p.G;
    const dim3 grid(static_cast<unsigned>(p.N * p.P), static_cast<unsigned>(p.tiles));
    cudaError_t e = gn_with_kind(a.ek, p.vec, [&](auto ek, auto vec) {
        return launch_kernel(gn_stats_kernel<ek.value, vec.value>, grid, dim3(kGnBlock), 0, stream, 1, f);
    });
    if (e != cudaSuccess) return e;
    const unsigned joins = static_cast<unsigned>((p.N * p.G + kGnBlock / 32 - 1) / (kGnBlock / 32));
    e = launch_kernel(gn_join_kernel, dim3(joins), dim3(kGnBlock), 0, stream, 1, f);
    if (e != cudaSuccess) return e;
    return gn_with_kind(a.ek, p.vec, [&](auto ek, auto vec) {
        return gn_with_act(a.act, [&](auto act) {
            return launch_kernel(gn_apply_kernel<ek.value, vec.value, act.value>, grid, dim3(kGnBlock), 0, stream, 1, f);
        });
    });
}

size_t groupnorm_backward_workspace_bytes(int64_t N, int64_t S, int64_t C, int64_t G, int ek)
{
    GnSlices s;
    if (gn_slices(N, S, C, G, ek, true, &s)) return gn_up(static_cast<size_t>(N) * s.K * 2 * C * 4);
    const GnPlan p = gn_plan(N, S, C, G, ek, true);
    return gn_up(static_cast<size_t>(N) * p.P * 2 * C * 4) + gn_up(static_cast<size_t>(N) * p.P * p.parts * 8) +
           gn_up(static_cast<size_t>(N) * G * 8);
}

cudaError_t launch_groupnorm_backward(const GnBwdArgs& a, cudaStream_t stream)
{
    const bool params = a.dgamma || a.dbeta;
    const unsigned across = static_cast<unsigned>((a.C + kAcross - 1) / kAcross);
    GnParams g{a.ws, 0, static_cast<int>(a.C), a.dgamma, a.dbeta, a.status};
    GnSlices s;
    if (gn_slices(a.N, a.S, a.C, a.G, a.ek, true, &s)) {
        const cudaError_t e = launch_gn_cluster_backward(s, a, params ? a.ws : nullptr, stream);
        if (e != cudaSuccess || !params) return e;
        g.rows = static_cast<long long>(s.N) * s.K;
        auto kernel = a.ek == kF32 ? gn_params_kernel<kF32> : a.ek == kBF16 ? gn_params_kernel<kBF16> : gn_params_kernel<kF16>;
        return launch_kernel(kernel, dim3(across), dim3(kGnBlock), 0, stream, 1, g);
    }
    GnBwd f{gn_plan(a.N, a.S, a.C, a.G, a.ek, true), a.dY, a.X, a.gamma, a.beta, a.mean, a.rstd, a.dX, nullptr, nullptr, nullptr,
            a.status};
    const GnPlan& p = f.p;
    f.cols = a.ws;
    f.part = f.cols + gn_up(static_cast<size_t>(p.N) * p.P * 2 * p.C * 4) / 4;
    f.ab = f.part + gn_up(static_cast<size_t>(p.N) * p.P * p.parts * 8) / 4;
    const dim3 grid(static_cast<unsigned>(p.N * p.P), static_cast<unsigned>(p.tiles));
    cudaError_t e = gn_with_kind(a.ek, p.vec, [&](auto ek, auto vec) {
        return gn_with_act(a.act, [&](auto act) {
            return launch_kernel(gn_sums_kernel<ek.value, vec.value, act.value>, grid, dim3(kGnBlock), 0, stream, 1, f);
        });
    });
    if (e != cudaSuccess) return e;
    const unsigned groups = static_cast<unsigned>((p.N * p.G + kGnBlock / 32 - 1) / (kGnBlock / 32));
    e = launch_kernel(gn_join_sums_kernel, dim3(groups), dim3(kGnBlock), 0, stream, 1, f);
    if (e != cudaSuccess) return e;
    // dgamma and dbeta ride behind dX: a launch of their own took 3 us more
    const int blocks = p.N * p.P;
    g.rows = blocks;
    const dim3 both(static_cast<unsigned>(blocks) + (params ? across : 0), grid.y);
    return gn_with_kind(a.ek, p.vec, [&](auto ek, auto vec) {
        return gn_with_act(a.act, [&](auto act) {
            return launch_kernel(gn_dx_kernel<ek.value, vec.value, act.value>, both, dim3(kGnBlock), 0, stream, 1, f, g, blocks);
        });
    });
}

}  // namespace dgrad
