// layernorm.cu -- layer norm over the channels of NHWC rows, forward and backward.
//
// Row m of X holds C channels:
//     mean = sum(x) / C,  rstd = 1 / sqrt(sum((x - mean)^2) / C + eps)
//     y = (x - mean) * rstd * gamma + beta
// and with n = (x - mean) * rstd and q = dy * gamma
//     dx = rstd * (q - sum(q)/C - n * sum(q*n)/C)
//     dgamma = sum over rows of dy * n,  dbeta = sum over rows of dy.
// Both directions do a handful of operations per element, so memory bounds
// them: X once and Y once (forward), dY and X once and dX once (backward).
//
// A row is held in the registers of T threads while it is reduced, so it is read
// once and the variance is the two-pass one (sum of squared differences from the
// row's own mean): no cancellation however far the mean lies from zero.  T is a
// power of two up to 32 (several rows per warp) or whole warps, one row per
// block.  All sums and statistics are fp32; results are rounded once.
//
// The parameter gradients are sums down the columns.  Each block keeps its rows'
// column sums in registers, writes them once as fp32 partials [block][2][C], and
// a second kernel adds the partials of a column in a fixed order: no atomics, so
// results repeat bit for bit.
#include "common.cuh"
#include "host_util.h"
#include "launchers.h"
#include "rowvec.cuh"

namespace dgrad {
namespace {

constexpr int kLnBlock = 256;        // threads of a block whose rows take at most a warp
constexpr int kLnMaxMulti = 384;     // threads of a block that shares one row
constexpr int kLnLoopThreads = 512;  // rows too long for registers

// Sum of (a, b) over the T threads of a row.  MULTI: the whole block (red is
// shared memory for one value pair per warp); else T <= 32 adjacent lanes.
template <bool MULTI>
__device__ __forceinline__ float2 row_sum2(float a, float b, int T, float2* red)
{
    const int top = MULTI ? 16 : T >> 1;
    for (int o = top; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if constexpr (MULTI) {
        const int warps = blockDim.x >> 5;
        __syncthreads();   // the previous use of red has been read
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        a = 0.f;
        b = 0.f;
        for (int w = 0; w < warps; ++w) {
            a += red[w].x;
            b += red[w].y;
        }
    }
    return make_float2(a, b);
}

struct LnFwd {
    const void* x;
    const void* gamma;   // null: ones
    const void* beta;    // null: zeros
    void* y;
    float* mean;         // null: not wanted
    float* rstd;
    long long M;
    int C, T;
    float eps;
    int* status;
};

template <int EK, int VEC, int NV, bool MULTI>
__global__ void __launch_bounds__(MULTI ? kLnMaxMulti : kLnBlock) ln_fwd_kernel(const LnFwd p)
{
    pdl_wait();      // the previous kernel on the stream has finished
    pdl_trigger();   // the next one may start its set-up
    __shared__ float2 red[MULTI ? 32 : 1];
    using V = RowVec<EK, VEC>;
    constexpr int es = elem_bytes<EK>();
    const int lane = MULTI ? threadIdx.x : threadIdx.x & (p.T - 1);
    const int rows = MULTI ? 1 : kLnBlock / p.T;       // rows per block and step
    const int group = MULTI ? 0 : threadIdx.x / p.T;
    const long long step = static_cast<long long>(gridDim.x) * rows;
    const float fc = static_cast<float>(p.C);

    V g[NV], b[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (lane + v * p.T) * VEC;
        g[v].zero();
        b[v].zero();
        if (c < p.C) {
            if (p.gamma) {
                g[v].load(p.gamma, c);
            } else {
                float one[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) one[i] = 1.0f;
                g[v].pack(one);
            }
            if (p.beta) b[v].load(p.beta, c);
        }
    }
    // the condition is the same for the whole block, so every thread takes part in each reduction
    for (long long base = static_cast<long long>(blockIdx.x) * rows; base < p.M; base += step) {
        const long long m = base + group;
        const bool live = m < p.M;
        const long long row = m * p.C;
        V x[NV];
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (lane + v * p.T) * VEC;
            x[v].zero();
            if (live && c < p.C) x[v].load(p.x, row + c);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float f[VEC];
            x[v].unpack(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s += f[i];
        }
        const float mean = row_sum2<MULTI>(s, 0.f, p.T, red).x / fc;
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float f[VEC];
            x[v].unpack(f);
            if ((lane + v * p.T) * VEC < p.C) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) ss = fmaf(f[i] - mean, f[i] - mean, ss);
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum2<MULTI>(ss, 0.f, p.T, red).x / fc + p.eps);
        if (!live) continue;
        if (lane == 0) {
            if (p.mean && store_ok(p.mean, p.M * 4, p.mean + m, 4, p.status)) p.mean[m] = mean;
            if (p.rstd && store_ok(p.rstd, p.M * 4, p.rstd + m, 4, p.status)) p.rstd[m] = rstd;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (lane + v * p.T) * VEC;
            if (c < p.C) {
                float f[VEC], gf[VEC], bf[VEC];
                x[v].unpack(f);
                g[v].unpack(gf);
                b[v].unpack(bf);
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[i] = fmaf((f[i] - mean) * rstd, gf[i], bf[i]);
                V o;
                o.pack(f);
                if (store_ok(p.y, p.M * p.C * es, static_cast<char*>(p.y) + (row + c) * es, VEC * es, p.status))
                    o.store(p.y, row + c);
            }
        }
    }
}

// Rows too long for registers: one block per row, the row read three times (the
// second and third time from L2 or L1).
template <int EK, int VEC>
__global__ void __launch_bounds__(kLnLoopThreads) ln_fwd_loop_kernel(const LnFwd p)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float2 red[32];
    using V = RowVec<EK, VEC>;
    constexpr int es = elem_bytes<EK>();
    const float fc = static_cast<float>(p.C);
    for (long long m = blockIdx.x; m < p.M; m += gridDim.x) {
        const long long row = m * p.C;
        float s = 0.f;
        for (int c = threadIdx.x * VEC; c < p.C; c += kLnLoopThreads * VEC) {
            V x;
            float f[VEC];
            x.load(p.x, row + c);
            x.unpack(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s += f[i];
        }
        const float mean = row_sum2<true>(s, 0.f, 0, red).x / fc;
        float ss = 0.f;
        for (int c = threadIdx.x * VEC; c < p.C; c += kLnLoopThreads * VEC) {
            V x;
            float f[VEC];
            x.load(p.x, row + c);
            x.unpack(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) ss = fmaf(f[i] - mean, f[i] - mean, ss);
        }
        const float rstd = 1.0f / sqrtf(row_sum2<true>(ss, 0.f, 0, red).x / fc + p.eps);
        if (threadIdx.x == 0) {
            if (p.mean && store_ok(p.mean, p.M * 4, p.mean + m, 4, p.status)) p.mean[m] = mean;
            if (p.rstd && store_ok(p.rstd, p.M * 4, p.rstd + m, 4, p.status)) p.rstd[m] = rstd;
        }
        for (int c = threadIdx.x * VEC; c < p.C; c += kLnLoopThreads * VEC) {
            V x, g, b;
            float f[VEC], gf[VEC], bf[VEC];
            x.load(p.x, row + c);
            x.unpack(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                gf[i] = 1.0f;
                bf[i] = 0.f;
            }
            if (p.gamma) {
                g.load(p.gamma, c);
                g.unpack(gf);
            }
            if (p.beta) {
                b.load(p.beta, c);
                b.unpack(bf);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = fmaf((f[i] - mean) * rstd, gf[i], bf[i]);
            x.pack(f);
            if (store_ok(p.y, p.M * p.C * es, static_cast<char*>(p.y) + (row + c) * es, VEC * es, p.status))
                x.store(p.y, row + c);
        }
    }
}

struct LnBwd {
    const void* dy;
    const void* x;
    const void* gamma;   // null: ones
    const float* mean;
    const float* rstd;
    void* dx;
    float* part;         // [blocks][2][C]; null: no parameter gradients
    long long M;
    int C, T, blocks;
    int* status;
};

template <int EK, int VEC, int NV, bool MULTI>
__global__ void __launch_bounds__(MULTI ? kLnMaxMulti : kLnBlock) ln_bwd_kernel(const LnBwd p)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float2 red[MULTI ? 32 : 1];
    extern __shared__ float cols[];   // [2][C] column sums (rows of at most a warp)
    using V = RowVec<EK, VEC>;
    constexpr int es = elem_bytes<EK>();
    const int lane = MULTI ? threadIdx.x : threadIdx.x & (p.T - 1);
    const int rows = MULTI ? 1 : kLnBlock / p.T;
    const int group = MULTI ? 0 : threadIdx.x / p.T;
    const long long step = static_cast<long long>(gridDim.x) * rows;
    const float fc = static_cast<float>(p.C);

    V g[NV];
    float dg[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (lane + v * p.T) * VEC;
        g[v].zero();
        if (c < p.C) {
            if (p.gamma) {
                g[v].load(p.gamma, c);
            } else {
                float one[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) one[i] = 1.0f;
                g[v].pack(one);
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) dg[v][i] = db[v][i] = 0.f;
    }
    for (long long base = static_cast<long long>(blockIdx.x) * rows; base < p.M; base += step) {
        const long long m = base + group;
        const bool live = m < p.M;
        const long long row = m * p.C;
        V x[NV], dy[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (lane + v * p.T) * VEC;
            x[v].zero();
            dy[v].zero();
            if (live && c < p.C) {
                x[v].load(p.x, row + c);
                dy[v].load(p.dy, row + c);
            }
        }
        const float mean = live ? p.mean[m] : 0.f;
        const float rstd = live ? p.rstd[m] : 0.f;
        float sq = 0.f, sqn = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float xf[VEC], df[VEC], gf[VEC];
            x[v].unpack(xf);
            dy[v].unpack(df);
            g[v].unpack(gf);
            // a dead row or column must add exactly nothing, whatever mean and rstd hold
            if (live && (lane + v * p.T) * VEC < p.C) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float n = (xf[i] - mean) * rstd;
                    const float q = df[i] * gf[i];
                    sq += q;
                    sqn = fmaf(q, n, sqn);
                    dg[v][i] = fmaf(df[i], n, dg[v][i]);
                    db[v][i] += df[i];
                }
            }
        }
        const float2 t = row_sum2<MULTI>(sq, sqn, p.T, red);
        const float mq = t.x / fc, mqn = t.y / fc;
        if (!live) continue;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (lane + v * p.T) * VEC;
            if (c < p.C) {
                float xf[VEC], df[VEC], gf[VEC];
                x[v].unpack(xf);
                dy[v].unpack(df);
                g[v].unpack(gf);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float n = (xf[i] - mean) * rstd;
                    xf[i] = (fmaf(df[i], gf[i], -mq) - n * mqn) * rstd;
                }
                V o;
                o.pack(xf);
                if (store_ok(p.dx, p.M * p.C * es, static_cast<char*>(p.dx) + (row + c) * es, VEC * es, p.status))
                    o.store(p.dx, row + c);
            }
        }
    }
    if (!p.part) return;
    float* out = p.part + static_cast<long long>(blockIdx.x) * 2 * p.C;
    const long long part_bytes = static_cast<long long>(p.blocks) * 2 * p.C * 4;
    if constexpr (MULTI) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (lane + v * p.T) * VEC;
            if (c < p.C) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    if (store_ok(p.part, part_bytes, out + c + i, 4, p.status)) out[c + i] = dg[v][i];
                    if (store_ok(p.part, part_bytes, out + p.C + c + i, 4, p.status)) out[p.C + c + i] = db[v][i];
                }
            }
        }
    } else {
        // the rows of a warp, then the warps one after the other: a fixed order
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                for (int o = p.T; o < 32; o <<= 1) {
                    dg[v][i] += __shfl_xor_sync(0xFFFFFFFFu, dg[v][i], o);
                    db[v][i] += __shfl_xor_sync(0xFFFFFFFFu, db[v][i], o);
                }
        const int warp = threadIdx.x >> 5;
        for (int w = 0; w < kLnBlock / 32; ++w) {
            if (warp == w && (threadIdx.x & 31) < p.T) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int c = (lane + v * p.T) * VEC;
                    if (c < p.C) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            cols[c + i] = w == 0 ? dg[v][i] : cols[c + i] + dg[v][i];
                            cols[p.C + c + i] = w == 0 ? db[v][i] : cols[p.C + c + i] + db[v][i];
                        }
                    }
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * p.C; c += kLnBlock)
            if (store_ok(p.part, part_bytes, out + c, 4, p.status)) out[c] = cols[c];
    }
}

// Long rows: the column sums first (dX may be dY or X), then dX row by row.
template <int EK, int VEC>
__global__ void __launch_bounds__(256) ln_cols_kernel(const LnBwd p)
{
    pdl_wait();
    pdl_trigger();
    using V = RowVec<EK, VEC>;
    const int c = (blockIdx.x * 256 + threadIdx.x) * VEC;
    if (c >= p.C) return;
    float dg[VEC], db[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) dg[i] = db[i] = 0.f;
    for (long long m = blockIdx.y; m < p.M; m += gridDim.y) {
        V x, dy;
        float xf[VEC], df[VEC];
        x.load(p.x, m * p.C + c);
        dy.load(p.dy, m * p.C + c);
        x.unpack(xf);
        dy.unpack(df);
        const float mean = p.mean[m], rstd = p.rstd[m];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            dg[i] = fmaf(df[i], (xf[i] - mean) * rstd, dg[i]);
            db[i] += df[i];
        }
    }
    float* out = p.part + static_cast<long long>(blockIdx.y) * 2 * p.C;
    const long long part_bytes = static_cast<long long>(p.blocks) * 2 * p.C * 4;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if (store_ok(p.part, part_bytes, out + c + i, 4, p.status)) out[c + i] = dg[i];
        if (store_ok(p.part, part_bytes, out + p.C + c + i, 4, p.status)) out[p.C + c + i] = db[i];
    }
}

template <int EK, int VEC>
__global__ void __launch_bounds__(kLnLoopThreads) ln_bwd_loop_kernel(const LnBwd p)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float2 red[32];
    using V = RowVec<EK, VEC>;
    constexpr int es = elem_bytes<EK>();
    const float fc = static_cast<float>(p.C);
    for (long long m = blockIdx.x; m < p.M; m += gridDim.x) {
        const long long row = m * p.C;
        const float mean = p.mean[m], rstd = p.rstd[m];
        auto read = [&](int c, float (&n)[VEC], float (&q)[VEC]) {
            V x, dy, g;
            float gf[VEC];
            x.load(p.x, row + c);
            dy.load(p.dy, row + c);
            x.unpack(n);
            dy.unpack(q);
#pragma unroll
            for (int i = 0; i < VEC; ++i) gf[i] = 1.0f;
            if (p.gamma) {
                g.load(p.gamma, c);
                g.unpack(gf);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                n[i] = (n[i] - mean) * rstd;
                q[i] *= gf[i];
            }
        };
        float sq = 0.f, sqn = 0.f;
        for (int c = threadIdx.x * VEC; c < p.C; c += kLnLoopThreads * VEC) {
            float n[VEC], q[VEC];
            read(c, n, q);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                sq += q[i];
                sqn = fmaf(q[i], n[i], sqn);
            }
        }
        const float2 t = row_sum2<true>(sq, sqn, 0, red);
        const float mq = t.x / fc, mqn = t.y / fc;
        for (int c = threadIdx.x * VEC; c < p.C; c += kLnLoopThreads * VEC) {
            float n[VEC], q[VEC];
            read(c, n, q);
#pragma unroll
            for (int i = 0; i < VEC; ++i) q[i] = (q[i] - mq - n[i] * mqn) * rstd;
            V o;
            o.pack(q);
            if (store_ok(p.dx, p.M * p.C * es, static_cast<char*>(p.dx) + (row + c) * es, VEC * es, p.status))
                o.store(p.dx, row + c);
        }
    }
}

// Column j of the partials [blocks][2C], summed over the blocks in a fixed order:
// 32 threads take every 32nd block, then one adds the 32 sums.
template <int EK>
__global__ void __launch_bounds__(1024) ln_params_kernel(const float* __restrict__ part, int blocks, int C,
                                                         void* dgamma, void* dbeta, int* status)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float s[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + x;
    float a = 0.f;
    if (j < 2 * C)
        for (int b = y; b < blocks; b += 32) a += part[static_cast<long long>(b) * 2 * C + j];
    s[y][x] = a;
    __syncthreads();
    // warp y now sums column y
    a = s[x][y];
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    const int k = blockIdx.x * 32 + y;
    if (x == 0 && k < 2 * C) {
        void* out = k < C ? dgamma : dbeta;
        const int c = k < C ? k : k - C;
        constexpr int es = elem_bytes<EK>();
        if (out && store_ok(out, static_cast<long long>(C) * es, static_cast<char*>(out) + c * es, es, status)) {
            RowVec<EK, 1> o;
            const float f[1] = {a};
            o.pack(f);
            o.store(out, c);
        }
    }
}

// How a row of C elements is spread: vec elements per load, T threads, nv vectors
// per thread; nv = 0 means the row does not fit and the looped kernels run.
struct LnPlan {
    int vec, T, nv;
    bool multi;
};

LnPlan ln_plan(int C, int ek, int max_elems)
{
    const int wide = ek == kF32 ? 4 : 8;
    LnPlan p{};
    p.vec = C % wide == 0 ? wide : 1;
    const int n = C / p.vec;
    // vectors per thread the kernels are compiled for
    static const int nv16[] = {1, 2, 3, 4}, nv32[] = {1, 2, 4, 8}, nv1[] = {4, 8, 16, 32};
    const int* nvs = p.vec == 1 ? nv1 : ek == kF32 ? nv32 : nv16;
    const int most = max_elems / p.vec;
    auto round_nv = [&](int need) {
        for (int i = 0; i < 4; ++i)
            if (nvs[i] >= need && nvs[i] <= most) return nvs[i];
        return 0;
    };
    for (int T = 1; T <= 32; T *= 2) {
        const int nv = round_nv((n + T - 1) / T);
        if (nv) {
            p.T = T;
            p.nv = nv;
            return p;
        }
    }
    p.multi = true;
    for (int T = 64; T <= kLnMaxMulti; T += 32) {
        const int nv = round_nv((n + T - 1) / T);
        if (nv) {
            p.T = T;
            p.nv = nv;
            return p;
        }
    }
    return p;
}

constexpr int kSms = 148;                 // a B200; the partial count must not depend on the device asked
constexpr int kLnFwdElems = 32, kLnBwdElems = 32;

int ln_bwd_blocks(int64_t M, const LnPlan& p)
{
    const int64_t rows = p.nv == 0 || p.multi ? 1 : kLnBlock / p.T;
    const int64_t need = (M + rows - 1) / rows;
    const int64_t most = p.nv == 0 ? 64 : p.multi ? 4 * kSms : 2 * kSms;
    return static_cast<int>(need < most ? need : most);
}

template <int EK, int VEC, int NV>
cudaError_t run_fwd(const LnFwd& a, const LnPlan& p, cudaStream_t st)
{
    const int rows = p.multi ? 1 : kLnBlock / p.T;
    const int threads = p.multi ? p.T : kLnBlock;
    auto kern = p.multi ? ln_fwd_kernel<EK, VEC, NV, true> : ln_fwd_kernel<EK, VEC, NV, false>;
    const int64_t need = (a.M + rows - 1) / rows;
    const int64_t most = static_cast<int64_t>(kSms) * (2048 / threads);
    return launch_kernel(kern, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(threads), 0, st, 1, a);
}

template <int EK, int VEC, int NV>
cudaError_t run_bwd(const LnBwd& a, const LnPlan& p, cudaStream_t st)
{
    const int threads = p.multi ? p.T : kLnBlock;
    auto kern = p.multi ? ln_bwd_kernel<EK, VEC, NV, true> : ln_bwd_kernel<EK, VEC, NV, false>;
    const size_t smem = p.multi || !a.part ? 0 : static_cast<size_t>(a.C) * 8;
    return launch_kernel(kern, dim3(static_cast<unsigned>(a.blocks)), dim3(threads), smem, st, 1, a);
}

template <int EK>
cudaError_t dispatch_fwd(const LnFwd& a, const LnPlan& p, cudaStream_t st)
{
    constexpr int W = EK == kF32 ? 4 : 8;
    if (p.nv == 0) {
        auto kern = p.vec == 1 ? ln_fwd_loop_kernel<EK, 1> : ln_fwd_loop_kernel<EK, W>;
        const int64_t most = 4 * kSms;
        return launch_kernel(kern, dim3(static_cast<unsigned>(a.M < most ? a.M : most)), dim3(kLnLoopThreads), 0, st,
                             1, a);
    }
    if (p.vec == 1) {
        switch (p.nv) {
        case 4: return run_fwd<EK, 1, 4>(a, p, st);
        case 8: return run_fwd<EK, 1, 8>(a, p, st);
        case 16: return run_fwd<EK, 1, 16>(a, p, st);
        default: return run_fwd<EK, 1, 32>(a, p, st);
        }
    }
    switch (p.nv) {
    case 1: return run_fwd<EK, W, 1>(a, p, st);
    case 2: return run_fwd<EK, W, 2>(a, p, st);
    case 4: return run_fwd<EK, W, 4>(a, p, st);
    default: return run_fwd<EK, W, EK == kF32 ? 8 : 3>(a, p, st);
    }
}

template <int EK>
cudaError_t dispatch_bwd(const LnBwd& a, const LnPlan& p, cudaStream_t st)
{
    constexpr int W = EK == kF32 ? 4 : 8;
    if (p.nv == 0) {
        cudaError_t e = cudaSuccess;
        if (a.part) {
            auto cols = p.vec == 1 ? ln_cols_kernel<EK, 1> : ln_cols_kernel<EK, W>;
            const int n = a.C / p.vec;
            e = launch_kernel(cols, dim3((n + 255) / 256, a.blocks), dim3(256), 0, st, 1, a);
            if (e != cudaSuccess) return e;
        }
        auto kern = p.vec == 1 ? ln_bwd_loop_kernel<EK, 1> : ln_bwd_loop_kernel<EK, W>;
        const int64_t most = 4 * kSms;
        return launch_kernel(kern, dim3(static_cast<unsigned>(a.M < most ? a.M : most)), dim3(kLnLoopThreads), 0, st,
                             1, a);
    }
    if (p.vec == 1) {
        switch (p.nv) {
        case 4: return run_bwd<EK, 1, 4>(a, p, st);
        case 8: return run_bwd<EK, 1, 8>(a, p, st);
        case 16: return run_bwd<EK, 1, 16>(a, p, st);
        default: return run_bwd<EK, 1, 32>(a, p, st);
        }
    }
    switch (p.nv) {
    case 1: return run_bwd<EK, W, 1>(a, p, st);
    case 2: return run_bwd<EK, W, 2>(a, p, st);
    case 4: return run_bwd<EK, W, 4>(a, p, st);
    default: return run_bwd<EK, W, EK == kF32 ? 8 : 3>(a, p, st);
    }
}

}  // namespace

cudaError_t launch_layernorm_forward(const LnFwdArgs& a, cudaStream_t stream)
{
    const LnFwd k{a.X, a.gamma, a.beta, a.Y, a.mean, a.rstd, a.M, static_cast<int>(a.C), 0, a.eps, a.status};
    const LnPlan p = ln_plan(static_cast<int>(a.C), a.ek, kLnFwdElems);
    LnFwd kk = k;
    kk.T = p.T;
    return a.ek == kF32 ? dispatch_fwd<kF32>(kk, p, stream)
                        : a.ek == kBF16 ? dispatch_fwd<kBF16>(kk, p, stream) : dispatch_fwd<kF16>(kk, p, stream);
}

size_t layernorm_backward_workspace_bytes(int64_t M, int64_t C, int ek)
{
    const LnPlan p = ln_plan(static_cast<int>(C), ek, kLnBwdElems);
    return static_cast<size_t>(ln_bwd_blocks(M, p)) * 2 * static_cast<size_t>(C) * sizeof(float);
}

cudaError_t launch_layernorm_backward(const LnBwdArgs& a, cudaStream_t stream)
{
    const bool params = a.dgamma || a.dbeta;
    const LnPlan p = ln_plan(static_cast<int>(a.C), a.ek, kLnBwdElems);
    LnBwd k{a.dY, a.X, a.gamma, a.mean, a.rstd, a.dX, params ? a.ws : nullptr, a.M, static_cast<int>(a.C), p.T,
            ln_bwd_blocks(a.M, p), a.status};
    cudaError_t e = a.ek == kF32 ? dispatch_bwd<kF32>(k, p, stream)
                                 : a.ek == kBF16 ? dispatch_bwd<kBF16>(k, p, stream) : dispatch_bwd<kF16>(k, p, stream);
    if (e != cudaSuccess || !params) return e;
    auto kern = a.ek == kF32 ? ln_params_kernel<kF32> : a.ek == kBF16 ? ln_params_kernel<kBF16> : ln_params_kernel<kF16>;
    return launch_kernel(kern, dim3(static_cast<unsigned>((2 * a.C + 31) / 32)), dim3(1024), 0, stream, 1, a.ws,
                         k.blocks, k.C, a.dgamma, a.dbeta, a.status);
}

}  // namespace dgrad
