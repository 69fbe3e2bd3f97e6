// groupnorm_cluster.cu -- group norm in one launch: a cluster of blocks holds a slice of
// channels of a sample (whole groups, all positions) in shared memory.
//
// The formulas are groupnorm.cu's.  X is read once from global memory; what the second pass
// needs stays on the SM: forward X, backward X and dz in fp32, so that the activation's
// derivative (two or three of the slow exponential and reciprocal instructions) is formed once.
// A thread's steps lie at its own places in shared memory, 16 bytes next to those of its
// neighbours, and nobody else reads them.  The way is taken where all of them fit.
// The forward pass takes the block's mean, then the squares about it, and the blocks of the
// cluster join both over distributed shared memory:
//     mean = sum count_k mean_k / m,  M2 = sum (M2_k + count_k (mean_k - mean)^2).
// A mean formed as a sum is a few roundings of itself off; one that lies far above the spread, or is that of equal
// values, is formed again from the differences to it (finish_far_slice).  The backward pass adds its blocks' sums.
// A block ends only when the others have read what it left for them.
#include "groupnorm.cuh"

namespace dgrad {
namespace {

constexpr int kT = 384;        // threads of a block; two blocks an SM: 85 registers a thread

// Copies a thread has under way, steps of one vector (forward) and two (backward).
constexpr int kAheadFwd = 8, kAheadBwd = 4;

struct GnCluster {
    GnSlices p;
    float eps;
    const void* x;
    const void* dy;
    const void* gamma;
    const void* beta;
    void* y;           // forward: Y, backward: dX
    float* mean;       // forward: null or [N][G]
    float* rstd;
    const float* mean_in;
    const float* rstd_in;
    float* cols;       // backward: null or [N K][2][C]
    int* status;
};

// Shared memory: kept vectors (x, and behind them dz), then these.
struct GnShared {
    float *buf, *part, *out, *ex, *stat, *all;   // T VEC, T, 2 tw, 2 ng, 2 ng, K 2 ng
    template <int VEC>
    __device__ __forceinline__ GnShared(char* at, const GnSlices& p, std::integral_constant<int, VEC>)
    {
        buf = reinterpret_cast<float*>(at);
        part = buf + kT * VEC;
        out = part + kT;
        ex = out + 2 * p.tw;
        stat = ex + 2 * p.ng;
        all = stat + 2 * p.ng;
    }
};
int gn_shared_bytes(int vec, int tw, int ng, int K) { return (kT * vec + kT + 2 * tw + (4 + 2 * K) * ng) * 4; }

__device__ __forceinline__ float peer_float(const float* p, uint32_t rank)
{
    uint32_t at;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The 2 ng values of every block of the cluster, in this block's shared memory: all remote loads under
// way at once.  Complete on return.
__device__ __forceinline__ const float* gather(const GnShared& sh, const GnSlices& p)
{
    for (int i = threadIdx.x; i < p.K * 2 * p.ng; i += kT) {
        const int q = i / (2 * p.ng);
        sh.all[i] = peer_float(sh.ex + i - q * 2 * p.ng, q);
    }
    __syncthreads();
    return sh.all;
}

// Values of a group that block q of its cluster has.
__device__ __forceinline__ float count_of(const GnSlices& p, int q)
{
    return static_cast<float>(max(0, min(p.S - q * p.rpc, p.rpc))) * static_cast<float>(p.D);
}

// What a thread takes: columns col .. of the slice, positions r, r + R, .. of its block's
// of a sample, `most` steps.
struct GnLane {
    int rank, r, c, col, rows, row, most;
    GnGroup group;          // of col, counted from the slice's first
    template <int VEC>
    __device__ __forceinline__ GnLane(const GnSlices& p, std::integral_constant<int, VEC>) : group(0, 1)
    {
        rank = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.K));
        r = static_cast<int>(threadIdx.x / static_cast<unsigned>(p.cols));
        c = static_cast<int>(threadIdx.x) - r * p.cols;
        col = c * VEC;
        const int row0 = rank * p.rpc;
        rows = max(0, min(p.S - row0, p.rpc));
        row = row0 + r;
        most = r < p.R && r < rows ? (rows - r + p.R - 1) / p.R : 0;
        group = GnGroup(col, p.D);
    }
};

// A cluster's slice of a sample.
struct GnItem {
    int n, c0, width, steps;
    bool on;
    long long first;        // element of the first step
    __device__ __forceinline__ GnItem(const GnSlices& p, const GnLane& t, int item)
    {
        n = item / p.slices;
        c0 = (item - n * p.slices) * p.tw;
        width = min(p.C - c0, p.tw);
        on = t.r < p.R && t.col < width;
        steps = on ? t.most : 0;
        first = (static_cast<long long>(n) * p.S + t.row) * p.C + c0 + t.col;
    }
};

// The statistics of a slice's groups, from what its blocks have in ex: stat on return, and a.mean and a.rstd.  Whole
// block.  MARK: true where a mean is far above the spread, and that group's rstd in stat is negative.  The
// cluster's blocks find the same.
template <int EK, bool MARK>
__device__ __forceinline__ bool slice_statistics(const GnCluster& a, const GnShared& sh, int rank, int ng, long long stat_at)
{
    const GnSlices& p = a.p;
    if (p.K > 1) cluster_sync();
    const float m = static_cast<float>(p.S) * static_cast<float>(p.D);
    const float* all = sh.ex;
    if (p.K > 1) all = gather(sh, p);
    bool far = false;
    for (int j = threadIdx.x; j < ng; j += kT) {
        float mu = sh.ex[j], sq = sh.ex[p.ng + j];
        if (p.K > 1) {
            const float mu0 = all[j];
            float d = 0.f;
            for (int q = 1; q < p.K; ++q) d += (all[q * 2 * p.ng + j] - mu0) * count_of(p, q);
            mu = mu0 + d / m;
            sq = 0.f;
            for (int q = 0; q < p.K; ++q) {
                const float e = all[q * 2 * p.ng + j] - mu;
                sq += fmaf(e * count_of(p, q), e, all[(q * 2 + 1) * p.ng + j]);
            }
        }
        const float2 stats = gn_statistics(mu, sq, m, a.eps);
        sh.stat[j] = stats.x;
        const bool again = MARK && gn_far<EK>(stats.x, sq, m);
        sh.stat[p.ng + j] = again ? -stats.y : stats.y;
        far = far || again;
        if (rank == 0) {
            const long long at = stat_at + j, all_of = static_cast<long long>(p.N) * p.G * 4;
            if (a.mean && store_ok(a.mean, all_of, a.mean + at, 4, a.status)) a.mean[at] = stats.x;
            if (a.rstd && store_ok(a.rstd, all_of, a.rstd + at, 4, a.status)) a.rstd[at] = stats.y;
        }
    }
    if (p.K > 1) cluster_arrive();   // this block has read the others' values
    return __syncthreads_or(far);    // in the place of the barrier behind stat: one more took 0.1 us of 5.1
}

// Y of the values that a thread keeps.
template <int EK, int VEC, int ACT>
__device__ __forceinline__ void slice_results(const GnCluster& a, const GnShared& sh, const char* mine, const GnLane& t, const GnItem& it)
{
    constexpr int es = elem_bytes<EK>(), NP = gn_pairs<VEC>();
    const GnSlices& p = a.p;
    if (!it.on) return;
    float2 mean[NP], scale[NP], beta[NP];
    gn_by_group<VEC>(t.group, p.D, mean, [&](int g) { return sh.stat[g]; });
    gn_by_group<VEC>(t.group, p.D, scale, [&](int g) { return sh.stat[p.ng + g]; });
    gn_param<EK, VEC>(a.gamma, it.c0 + t.col, 1.f, beta);
#pragma unroll
    for (int i = 0; i < NP; ++i) scale[i] = __fmul2_rn(scale[i], beta[i]);
    gn_param<EK, VEC>(a.beta, it.c0 + t.col, 0.f, beta);
    const long long bytes = static_cast<long long>(p.N) * p.S * p.C * es, stride = static_cast<long long>(p.R) * p.C;
    for (int k = 0; k < it.steps; ++k) {
        RowVec<EK, VEC> v;
        float2 f[NP];
        v.load(mine, static_cast<long long>(k) * kT * VEC);
        gn_unpack<EK, VEC>(v, f);
#pragma unroll
        for (int i = 0; i < NP; ++i) f[i] = gate_act<ACT>(ffma2(__fadd2_rn(f[i], gn_minus(mean[i])), scale[i], beta[i]));
        gn_pack<EK, VEC>(v, f);
        const long long at = it.first + k * stride;
        if (store_ok(a.y, bytes, static_cast<char*>(a.y) + at * es, VEC * es, a.status)) v.store(a.y, at);
    }
}

// What is left of a slice where a mean is far above the spread: the statistics once more, with the blocks' means of
// such groups formed from the differences to the first mean, and the results.  A function of its own that the kernel ends
// with: what every other slice goes through keeps its registers (16 x 1024 x 512 bf16 13.0 us; a call that returned 13.4, the
// same code in place 13.4).  A slice that takes it takes 5 us more (2 x 64 x 512 fp32 10.0 us, 4.9 without).
template <int EK, int VEC, int ACT>
__device__ __noinline__ void finish_far_slice(const GnCluster& a)
{
    extern __shared__ __align__(16) char smem[];
    constexpr int es = elem_bytes<EK>(), NP = gn_pairs<VEC>();
    const GnSlices& p = a.p;
    const GnShared sh(smem + gn_up(static_cast<size_t>(p.cap) * kT * VEC * es), p, std::integral_constant<int, VEC>{});
    const char* const mine = smem + threadIdx.x * VEC * es;
    const GnLane t(p, std::integral_constant<int, VEC>{});
    const GnItem it(p, t, static_cast<int>(blockIdx.x / static_cast<unsigned>(p.K)));
    const int ng = it.width / p.D;
    const float count = count_of(p, t.rank);
    if (p.K > 1) cluster_wait();
    float2 s[NP], mean[NP];
    gn_set<VEC>(mean, 0.f);
#pragma unroll 1
    for (int squares = 0; squares < 2; ++squares) {
        if (it.on) gn_by_group<VEC>(t.group, p.D, mean, [&](int g) { return squares ? sh.ex[g] : sh.stat[g]; });
        gn_set<VEC>(s, 0.f);
        for (int k = 0; k < it.steps; ++k) {
            RowVec<EK, VEC> v;
            float2 d[NP];
            v.load(mine, static_cast<long long>(k) * kT * VEC);
            gn_unpack<EK, VEC>(v, d);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                d[i] = __fadd2_rn(d[i], gn_minus(mean[i]));
                s[i] = squares ? ffma2(d[i], d[i], s[i]) : __fadd2_rn(s[i], d[i]);
            }
        }
        column_totals<kT, VEC>(s, it.on, t.r, t.c, p.R, p.tw, p.parts, sh.buf, sh.part, sh.out);
        group_totals<kT, 1>(sh.out, p.tw, 1, p.tw, 0, it.width, p.D, squares ? sh.ex + p.ng : sh.all, p.ng);
        if (!squares) {
            for (int j = threadIdx.x; j < ng; j += kT)
                if (t.rows && sh.stat[p.ng + j] < 0.f) sh.ex[j] = sh.stat[j] + sh.all[j] / count;
            __syncthreads();
        }
    }
    slice_statistics<EK, false>(a, sh, t.rank, ng, static_cast<long long>(it.n) * p.G + it.c0 / p.D);
    slice_results<EK, VEC, ACT>(a, sh, mine, t, it);
    if (p.K > 1) cluster_wait();
}

template <int EK, int VEC, int ACT>
__global__ void __launch_bounds__(kT, 2) gn_cluster_fwd_kernel(const __grid_constant__ GnCluster a)
{
    extern __shared__ __align__(16) char smem[];
    using V = RowVec<EK, VEC>;
    constexpr int es = elem_bytes<EK>(), NP = gn_pairs<VEC>();
    const GnSlices& p = a.p;
    const GnShared sh(smem + gn_up(static_cast<size_t>(p.cap) * kT * VEC * es), p, std::integral_constant<int, VEC>{});
    char* const mine = smem + threadIdx.x * VEC * es;
    const GnLane t(p, std::integral_constant<int, VEC>{});
    const long long stride = static_cast<long long>(p.R) * p.C;     // elements from step to step
    pdl_wait();
    pdl_trigger();
    const GnItem it(p, t, static_cast<int>(blockIdx.x / static_cast<unsigned>(p.K)));
    const int kept = it.steps, ng = it.width / p.D;
    // step q: x to its place
    auto bring = [&](int q) {
        if (VEC > 1) {
            if (q < kept) gn_copy16(mine + q * kT * 16, static_cast<const char*>(a.x) + (it.first + q * stride) * es);
            gn_copy_commit();
        }
    };
#pragma unroll
    for (int q = 0; q < kAheadFwd; ++q) bring(q);
    const long long stat_at = static_cast<long long>(it.n) * p.G + it.c0 / p.D;

    // the block's mean
    float2 s[NP];
    gn_set<VEC>(s, 0.f);
    int k = 0;
    auto add = [&](const V& v) {
        float2 f[NP];
        gn_unpack<EK, VEC>(v, f);
#pragma unroll
        for (int i = 0; i < NP; ++i) s[i] = __fadd2_rn(s[i], f[i]);
    };
    if constexpr (VEC == 1) {
        constexpr int U = 8;
        for (; k + U <= kept; k += U) {
            V v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u].load(a.x, it.first + (k + u) * stride);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v[u].store(mine, static_cast<long long>(k + u) * kT * VEC);
                add(v[u]);
            }
        }
        for (; k < kept; ++k) {
            V v;
            v.load(a.x, it.first + k * stride);
            v.store(mine, static_cast<long long>(k) * kT * VEC);
            add(v);
        }
    } else {
        for (; k < kept; ++k) {
            gn_copy_wait<kAheadFwd - 1>();
            V v;
            v.load(mine, static_cast<long long>(k) * kT * VEC);
            add(v);
            bring(k + kAheadFwd);
        }
    }
    column_totals<kT, VEC>(s, it.on, t.r, t.c, p.R, p.tw, p.parts, sh.buf, sh.part, sh.out);
    group_totals<kT, 1>(sh.out, p.tw, 1, p.tw, 0, it.width, p.D, sh.ex, p.ng);
    const float count = static_cast<float>(t.rows) * static_cast<float>(p.D);
    for (int j = threadIdx.x; j < ng; j += kT) sh.ex[j] = t.rows ? sh.ex[j] / count : 0.f;
    __syncthreads();

    // the squares about it
    float2 mean[NP];
    if (it.on) gn_by_group<VEC>(t.group, p.D, mean, [&](int g) { return sh.ex[g]; });
    gn_set<VEC>(s, 0.f);
    auto square = [&](const V& v) {
        float2 f[NP];
        gn_unpack<EK, VEC>(v, f);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float2 d = __fadd2_rn(f[i], gn_minus(mean[i]));
            s[i] = ffma2(d, d, s[i]);
        }
    };
#pragma unroll 4
    for (k = 0; k < kept; ++k) {
        V v;
        v.load(mine, static_cast<long long>(k) * kT * VEC);
        square(v);
    }
    if constexpr (VEC == 1) s[0].y = 0.f;
    column_totals<kT, VEC>(s, it.on, t.r, t.c, p.R, p.tw, p.parts, sh.buf, sh.part, sh.out);
    group_totals<kT, 1>(sh.out, p.tw, 1, p.tw, 0, it.width, p.D, sh.ex + p.ng, p.ng);

    if (slice_statistics<EK, true>(a, sh, t.rank, ng, stat_at)) {
        finish_far_slice<EK, VEC, ACT>(a);
        return;
    }
    slice_results<EK, VEC, ACT>(a, sh, mine, t, it);
    if (p.K > 1) cluster_wait();
}

template <int EK, int VEC, int ACT>
__global__ void __launch_bounds__(kT, 2) gn_cluster_bwd_kernel(const GnCluster a)
{
    extern __shared__ __align__(16) char smem[];
    using V = RowVec<EK, VEC>;
    constexpr int es = elem_bytes<EK>(), NP = gn_pairs<VEC>(), NQ = VEC == 1 ? 1 : VEC / 4;
    const GnSlices& p = a.p;
    const size_t xs = gn_up(static_cast<size_t>(p.cap) * kT * VEC * es);
    const GnShared sh(smem + xs + gn_up(static_cast<size_t>(p.cap) * kT * VEC * 4), p, std::integral_constant<int, VEC>{});
    char* const mine = smem + threadIdx.x * VEC * es;
    float* const mine_dz = reinterpret_cast<float*>(smem + xs) + threadIdx.x * (VEC == 1 ? 1 : 4);
    const GnLane t(p, std::integral_constant<int, VEC>{});
    const long long stride = static_cast<long long>(p.R) * p.C;     // elements from step to step
    pdl_wait();
    pdl_trigger();
    const GnItem it(p, t, static_cast<int>(blockIdx.x / static_cast<unsigned>(p.K)));
    const int kept = it.steps, ng = it.width / p.D;
    // step q: x to its place, dy to where its dz will be
    auto bring = [&](int q) {
        if (VEC > 1) {
            if (q < kept) {
                gn_copy16(mine + q * kT * 16, static_cast<const char*>(a.x) + (it.first + q * stride) * es);
                gn_copy16(mine_dz + q * NQ * kT * 4, static_cast<const char*>(a.dy) + (it.first + q * stride) * es);
            }
            gn_copy_commit();
        }
    };
#pragma unroll
    for (int q = 0; q < kAheadBwd; ++q) bring(q);
    const long long stat_at = static_cast<long long>(it.n) * p.G + it.c0 / p.D;

    float2 mean[NP], rstd[NP], gamma[NP], beta[NP];
    if (it.on) {
        gn_by_group<VEC>(t.group, p.D, mean, [&](int g) { return a.mean_in[stat_at + g]; });
        gn_by_group<VEC>(t.group, p.D, rstd, [&](int g) { return a.rstd_in[stat_at + g]; });
        gn_param<EK, VEC>(a.gamma, it.c0 + t.col, 1.f, gamma);
        gn_param<EK, VEC>(a.beta, it.c0 + t.col, 0.f, beta);
    }
    float2 A[NP], B[NP];
    gn_set<VEC>(A, 0.f);
    gn_set<VEC>(B, 0.f);
    auto slope = [&](const V& xv, const V& dv, float2 (&n)[NP], float2 (&dz)[NP]) {
        float2 x[NP];
        gn_unpack<EK, VEC>(xv, x);
        gn_unpack<EK, VEC>(dv, dz);
#pragma unroll
        for (int i = 0; i < NP; ++i) gn_dz<ACT>(x[i], dz[i], mean[i], rstd[i], gamma[i], beta[i], n[i], dz[i]);
    };
    auto take = [&](const V& xv, const V& dv, int step) {
        float2 n[NP], dz[NP];
        slope(xv, dv, n, dz);
        if constexpr (VEC == 1) {
            xv.store(mine, static_cast<long long>(step) * kT * VEC);
            mine_dz[step * kT] = dz[0].x;
        } else {
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                *reinterpret_cast<float4*>(mine_dz + (step * NQ + q) * kT * 4) =
                    make_float4(dz[2 * q].x, dz[2 * q].y, dz[2 * q + 1].x, dz[2 * q + 1].y);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            A[i] = __fadd2_rn(A[i], dz[i]);
            B[i] = ffma2(dz[i], n[i], B[i]);
        }
    };
    int k = 0;
    if constexpr (VEC == 1) {
        constexpr int U = 4;
        for (; k + U <= kept; k += U) {
            V xv[U], dv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                xv[u].load(a.x, it.first + (k + u) * stride);
                dv[u].load(a.dy, it.first + (k + u) * stride);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) take(xv[u], dv[u], k + u);
        }
        for (; k < kept; ++k) {
            V xv, dv;
            xv.load(a.x, it.first + k * stride);
            dv.load(a.dy, it.first + k * stride);
            take(xv, dv, k);
        }
    } else {
        for (; k < kept; ++k) {
            gn_copy_wait<kAheadBwd - 1>();
            V xv, dv;
            xv.load(mine, static_cast<long long>(k) * kT * VEC);
            dv.load(mine_dz + k * NQ * kT * 4, 0);
            take(xv, dv, k);
            bring(k + kAheadBwd);
        }
    }
    float* const outA = sh.out;
    float* const outB = sh.out + p.tw;
    column_totals<kT, VEC>(A, it.on, t.r, t.c, p.R, p.tw, p.parts, sh.buf, sh.part, outA);
    column_totals<kT, VEC>(B, it.on, t.r, t.c, p.R, p.tw, p.parts, sh.buf, sh.part, outB);
    for (int c = threadIdx.x; c < it.width; c += kT) {
        if (a.cols) {
            float* cols = a.cols + (static_cast<long long>(it.n) * p.K + t.rank) * 2 * p.C + it.c0 + c;
            cols[0] = outA[c];
            cols[p.C] = outB[c];
        }
        float2 g[1];
        gn_param<EK, 1>(a.gamma, it.c0 + c, 1.f, g);
        outA[c] *= g[0].x;
        outB[c] *= g[0].x;
    }
    __syncthreads();
    group_totals<kT, 2>(sh.out, p.tw, 1, p.tw, 0, it.width, p.D, sh.ex, p.ng);
    if (p.K > 1) cluster_sync();
    const float m = static_cast<float>(p.S) * static_cast<float>(p.D);
    const float* all = sh.ex;
    if (p.K > 1) all = gather(sh, p);
    for (int j = threadIdx.x; j < 2 * ng; j += kT) {
        const int at = j < ng ? j : p.ng + j - ng;
        float v = sh.ex[at];
        if (p.K > 1) {
            v = 0.f;
#pragma unroll 4
            for (int q = 0; q < p.K; ++q) v += all[q * 2 * p.ng + at];
        }
        sh.stat[at] = v / m;
    }
    if (p.K > 1) cluster_arrive();
    __syncthreads();

    k = 0;
    if (it.on) {
        float2 qa[NP], qb[NP];
        gn_by_group<VEC>(t.group, p.D, qa, [&](int g) { return sh.stat[g]; });
        gn_by_group<VEC>(t.group, p.D, qb, [&](int g) { return sh.stat[p.ng + g]; });
        const long long bytes = static_cast<long long>(p.N) * p.S * p.C * es;
        auto finish = [&](V& xv, const float2 (&n)[NP], float2 (&dz)[NP], int step) {
#pragma unroll
            for (int i = 0; i < NP; ++i) dz[i] = gn_dx(n[i], dz[i], rstd[i], gamma[i], qa[i], qb[i]);
            gn_pack<EK, VEC>(xv, dz);
            const long long at = it.first + step * stride;
            if (store_ok(a.y, bytes, static_cast<char*>(a.y) + at * es, VEC * es, a.status)) xv.store(a.y, at);
        };
        for (; k < kept; ++k) {
            V xv;
            float2 n[NP], dz[NP];
            xv.load(mine, static_cast<long long>(k) * kT * VEC);
            if constexpr (VEC == 1) {
                dz[0] = make_float2(mine_dz[k * kT], 0.f);
            } else {
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    const float4 w = *reinterpret_cast<const float4*>(mine_dz + (k * NQ + q) * kT * 4);
                    dz[2 * q] = make_float2(w.x, w.y);
                    dz[2 * q + 1] = make_float2(w.z, w.w);
                }
            }
            gn_unpack<EK, VEC>(xv, n);
#pragma unroll
            for (int i = 0; i < NP; ++i) n[i] = __fmul2_rn(__fadd2_rn(n[i], gn_minus(mean[i])), rstd[i]);
            finish(xv, n, dz, k);
        }
    }
    if (p.K > 1) cluster_wait();
}

template <typename Kernel>
cudaError_t launch(Kernel kernel, const GnCluster& c, cudaStream_t stream)
{
    const GnSlices& p = c.p;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), p.smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(p.N * p.slices * p.K)), dim3(kT), p.smem, stream, p.K, c);
}

int64_t gcd(int64_t a, int64_t b) { return b == 0 ? a : gcd(b, a % b); }

// Both ways were timed over 16 shapes of 0.1 to 230 MB, every cluster size and slice width (bf16, silu;
// device time).  The cluster way is 5.2 us (backward 5.6) and 0.38 us (0.75) for each step of its
// busiest SM, and 1.3 to 2.2 us more for clusters of 2 to 8, as long as everything stays in shared memory
// and rows fill their 32-byte sectors; the streaming way 8.5 us and 0.25 us per MB of tensors (10 and
// 0.33, fp32 0.22), and 0.008 for each block that shares a sample.  So the cluster way takes what one
// wave of blocks holds: 16 x 256 x 1024 channels, 32 groups: 8.8 us forward against 15.2, 1 x 64 x 512: 5.1
// against 7.3, backward 6.0 against 6.8; 16 x 4096 x 384 would be 40 us against 34.
bool choose(int64_t N, int64_t S, int64_t C, int64_t G, int ek, bool backward, GnSlices* out)
{
    const char* way = tuning_env("DGRAD_GN_WAY");      // 's': always the streaming way; 'c': the cluster way wherever it fits
    if (way && way[0] == 's') return false;
    const bool forced = way && way[0] == 'c';
    const int es = ek == kF32 ? 4 : 2, full = 16 / es;
    const int vec = C % full == 0 ? full : 1;
    const int64_t D = C / G, unit = D / gcd(D, vec) * vec;   // channels: whole groups and whole vectors
    if (unit > C || unit / vec > kT) return false;
    const double mb = static_cast<double>(N) * S * C * es * (backward ? 3e-6 : 2e-6);
    const double blocks = (backward ? 296.0 : 592.0) / static_cast<double>(N);
    const double streaming = (backward ? 10.0 + (es == 4 ? 0.22 : 0.33) * mb : 8.5 + 0.25 * mb) + 0.008 * (blocks < S / 16.0 ? blocks : S / 16.0) +
                             (vec == 1 ? 3.0 : 0.0);
    if (!forced && mb > 64.0) return false;
    const int64_t units = C / unit;
    const int64_t step_bytes = static_cast<int64_t>(kT) * vec * (backward ? es + 4 : es);
    // a step's microseconds: some of it per thread, most of it per element
    const double step_us = backward ? 0.15 + 0.075 * vec : 0.10 + 0.035 * vec;
    const char* fk = tuning_env("DGRAD_GN_CLUSTER");
    const char* fs = tuning_env("DGRAD_GN_SLICES");
    double best = 1e300;
    for (int K = 1; K <= 8 && K <= S; K *= 2) {
        if (fk && atoi(fk) != K) continue;
        for (int64_t s = fs ? atoi(fs) : 1, next = 0; s != 0; s = next) {
            next = s >= units || fs ? 0 : s + (s < 4 ? 1 : s / 2) < units ? s + (s < 4 ? 1 : s / 2) : units;
            const int64_t per = (units + s - 1) / s, tw = per * unit, cols = tw / vec, slices = (units + per - 1) / per;
            const int64_t ctas = N * slices * K, R = cols > 0 && cols <= kT ? kT / cols : 0;
            if (R == 0 || ctas > 296 * 8) continue;
            const int64_t rpc = (S + K - 1) / K, steps = (rpc + R - 1) / R;
            const int ng = static_cast<int>(tw / D), rest = gn_shared_bytes(vec, static_cast<int>(tw), ng, K) + 64;
            // clusters lie within one of eight groups of some 18 SMs
            const int64_t room = K == 1 ? 148 : 8 * (18 / K) * K;
            const int64_t on_sm = ctas <= room ? 1 : 2, waves = (ctas + 2 * room - 1) / (2 * room);
            const int64_t limit = on_sm == 1 ? 232448 : 115712;
            if (rest + steps * step_bytes > limit || (!forced && waves > 1)) continue;
            // half-used sectors.  fp32 rows of two vectors: fitted to 1 x 16384 x 128, whose backward pass takes 20.7 us (streaming
            // 13.5); 1 x 8192 x 256 would take 11.7 with such rows and is given wider ones, 17.9
            const double sectors = tw * es < 32 ? 3.5 : tw * es >= 64 ? 1.0 : es == 4 ? 2.2 : 1.2;
            const double cost = (backward ? 5.6 : 5.2) + (K == 1 ? 0.0 : 1.0 + 0.15 * K) +
                                step_us * sectors * static_cast<double>(waves * on_sm * steps);
            if (cost >= best) continue;
            best = cost;
            GnSlices& p = *out;
            p.N = static_cast<int>(N);
            p.S = static_cast<int>(S);
            p.C = static_cast<int>(C);
            p.G = static_cast<int>(G);
            p.D = static_cast<int>(D);
            p.vec = vec;
            p.cols = static_cast<int>(cols);
            p.tw = static_cast<int>(tw);
            p.slices = static_cast<int>(slices);
            p.R = static_cast<int>(R);
            p.K = K;
            p.rpc = static_cast<int>(rpc);
            p.cap = static_cast<int>(steps);
            p.ng = ng;
            p.smem = static_cast<int>(gn_up(static_cast<size_t>(steps) * kT * vec * es) +
                                      (backward ? gn_up(static_cast<size_t>(steps) * kT * vec * 4) : 0)) + rest;
        }
    }
    if (best >= 1e300) return false;
    out->parts = gn_column_parts(kT, out->tw, out->R);
    return forced || best <= streaming;
}

}  // namespace

// The choice takes some microseconds of host time and is asked for up to three times a call: a thread keeps
// its last eight, by their sizes.
bool gn_slices(int64_t N, int64_t S, int64_t C, int64_t G, int ek, bool backward, GnSlices* out)
{
    struct Known {
        int64_t N, S, C, G;
        int kind, ok;     // kind 0: none yet
        GnSlices p;
    };
    if (tuning_env("DGRAD_GN_WAY") || tuning_env("DGRAD_GN_CLUSTER") || tuning_env("DGRAD_GN_SLICES"))
        return choose(N, S, C, G, ek, backward, out);
    static thread_local Known known[8] = {};
    static thread_local unsigned next = 0;
    const int kind = 1 + ek * 2 + (backward ? 1 : 0);
    for (const Known& k : known)
        if (k.kind == kind && k.N == N && k.S == S && k.C == C && k.G == G) {
            if (k.ok) *out = k.p;
            return k.ok != 0;
        }
    Known& k = known[next++ % 8];
    k = Known{N, S, C, G, kind, 0, {}};
    k.ok = choose(N, S, C, G, ek, backward, &k.p);
    if (k.ok) *out = k.p;
    return k.ok != 0;
}

cudaError_t launch_gn_cluster_forward(const GnSlices& p, const GnFwdArgs& a, cudaStream_t stream)
{
    GnCluster c{};
    c.p = p;
    c.eps = a.eps;
    c.x = a.X;
    c.gamma = a.gamma;
    c.beta = a.beta;
    c.y = a.Y;
    c.mean = a.mean;
    c.rstd = a.rstd;
    c.status = a.status;
    return gn_with_kind(a.ek, p.vec, [&](auto ek, auto vec) {
        return gn_with_act(a.act, [&](auto act) { return launch(gn_cluster_fwd_kernel<ek.value, vec.value, act.value>, c, stream); });
    });
}

cudaError_t launch_gn_cluster_backward(const GnSlices& p, const GnBwdArgs& a, float* cols, cudaStream_t stream)
{
    GnCluster c{};
    c.p = p;
    c.x = a.X;
    c.dy = a.dY;
    c.gamma = a.gamma;
    c.beta = a.beta;
    c.y = a.dX;
    c.mean_in = a.mean;
    c.rstd_in = a.rstd;
    c.cols = cols;
    c.status = a.status;
    return gn_with_kind(a.ek, p.vec, [&](auto ek, auto vec) {
        return gn_with_act(a.act, [&](auto act) { return launch(gn_cluster_bwd_kernel<ek.value, vec.value, act.value>, c, stream); });
    });
}

}  // namespace dgrad
