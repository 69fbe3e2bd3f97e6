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
// power of two up to 32 (several rows per warp) or whole warps that meet at a named
// barrier; a block holds G rows at a time.
//
// What bounds these kernels is the bytes in flight per SM (about 45 KB at 6.5 TB/s and
// a microsecond of loaded latency), more than the registers of the threads that an SM
// can hold beside their sums.  So where a block has more than one step of rows, its
// first warp brings whole chunks of rows, which are contiguous, into a ring in shared
// memory with bulk copies, wherever their first byte lies (a copy starts at the 16-byte
// boundary before it), and refills a stage one chunk after it was read.  Blocks with
// one step load from global memory directly.
// All sums and statistics are fp32; results are rounded once.
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

constexpr int kLnBlock = 256;        // most threads of a block of several rows
constexpr int kLnMaxMulti = 384;     // threads of a block that shares one row
constexpr int kLnLoopThreads = 512;  // rows too long for registers

// Sum over the T threads of a row of (a, b), or of a alone: T <= 32 adjacent lanes, or
// (MULTI) the warps of one group, through `red`, 2 x 16 pairs of the group.  `turn`
// alternates between its halves, so one barrier per sum is enough: whoever writes a half
// again has passed the barrier of the sum in between, after everyone read it.
template <bool MULTI, bool TWO>
__device__ __forceinline__ float2 row_sum(float a, float b, int T, int group, float2* red, int& turn)
{
    const int top = MULTI ? 16 : T >> 1;
    for (int o = top; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        if constexpr (TWO) b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if constexpr (MULTI) {
        const int warps = T >> 5;
        float2* r = red + (group * 2 + turn) * 16;
        turn ^= 1;
        const int first = group * warps;
        if ((threadIdx.x & 31) == 0) r[(threadIdx.x >> 5) - first] = make_float2(a, b);
        named_barrier_sync(1 + group, T);
        a = 0.f;
        b = 0.f;
        for (int w = 0; w < warps; ++w) {
            a += r[w].x;
            if constexpr (TWO) b += r[w].y;
        }
    }
    return make_float2(a, b);
}

// gamma or beta as fp32 in shared memory, for rows of at most a warp: vector v's quarters
// (four elements each) lie n vectors apart, so that adjacent lanes' 16-byte reads are
// adjacent.  A null pointer gives the constant.
template <int EK, int VEC>
__device__ __forceinline__ void spread_param(float* dst, const void* src, float constant, int C)
{
    const int n = C / VEC;
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
        float f[1] = {constant};
        if (src) {
            RowVec<EK, 1> v;
            v.load(src, c);
            v.unpack(f);
        }
        const int at = VEC == 1 ? c : ((c % VEC / 4) * n + c / VEC) * 4 + c % 4;
        dst[at] = f[0];
    }
}

// The pairs of unit u (RowPart) of a parameter: from shared memory (rows of at most a warp),
// or from the thread's registers.
template <int EK, int VEC, int NV, bool MULTI>
struct LnParam {
    using P = RowPart<EK, VEC, NV>;
    P reg;
    const float* sm;

    __device__ __forceinline__ void init(float* smem, const void* src, float constant, int C, int T, int lane)
    {
        if constexpr (MULTI) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (lane + v * T) * VEC;
                if (constant != 0.f)
                    reg.v[v].ones();
                else
                    reg.v[v].zero();
                if (src && c < C) reg.v[v].load(src, c);
            }
        } else {
            spread_param<EK, VEC>(smem, src, constant, C);
            sm = smem;
        }
    }

    __device__ __forceinline__ void unit(int u, int C, int T, int lane, float2 (&f)[P::kPer]) const
    {
        if constexpr (MULTI) {
            reg.unit(u, f);
        } else if constexpr (VEC == 1) {
            const int c = lane + 2 * u * T;
            f[0] = make_float2(c < C ? sm[c] : 0.f, c + T < C ? sm[c + T] : 0.f);
        } else {
            const int n = C / VEC;
            const float4* q = reinterpret_cast<const float4*>(sm) + lane + u * T;
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const float4 w = q[i * n];
                f[2 * i] = make_float2(w.x, w.y);
                f[2 * i + 1] = make_float2(w.z, w.w);
            }
        }
    }
};

// Vectors (or elements) of a row that this lane holds: the first `mine` of its NV.
template <int VEC>
__device__ __forceinline__ int lane_vectors(int C, int T, int lane)
{
    const int n = C / VEC;
    return lane < n ? (n - lane + T - 1) / T : 0;
}

// Zero the elements of unit u that lie behind the row's end (whole vectors, or either element).
template <int VEC, int PER>
__device__ __forceinline__ void mask_unit(int u, int mine, float2 (&f)[PER])
{
    if constexpr (VEC == 1) {
        if (2 * u >= mine) f[0].x = 0.f;
        if (2 * u + 1 >= mine) f[0].y = 0.f;
    } else {
        if (u >= mine) {
#pragma unroll
            for (int i = 0; i < PER; ++i) f[i] = make_float2(0.f, 0.f);
        }
    }
}

// How a row's threads meet: 0, within a warp; 1, whole warps of a block of several rows
// (or of 256 threads); 2, a block of more than 256 threads.
constexpr int ln_mode(int T) { return T <= 32 ? 0 : T <= kLnBlock ? 1 : 2; }

// Threads of a block.  Where a warp needs no other (mode 0), the backward pass has many
// instructions per chunk and few warps: with blocks of four warps a chunk waits for fewer
// others (401408 x 96 bf16: 43.9 us, against 47.3 with eight; forward 21.4 against 21.0).
constexpr int ln_block(int mode, bool backward) { return mode == 2 ? kLnMaxMulti : mode == 0 && backward ? 128 : kLnBlock; }

// Blocks an SM holds, by the registers their elements take.
constexpr int ln_per_sm(int mode, int elems, bool backward)
{
    return mode == 2 ? 1 : mode == 0 && backward ? 4 : mode == 0 && elems <= 16 ? 3 : 2;
}

// Shared memory for `count` parameters (rows of at most a warp).
__host__ __device__ constexpr int ln_param_bytes(int mode, int C, int count)
{
    return mode == 0 ? (count * C * 4 + 15) / 16 * 16 : 0;
}

// Elements per thread that fit its registers without spills.  Forward: 48 where the
// parameters are in shared memory, 24 or (one block per SM) 32 beside them.  Backward: the
// column sums take two registers per element.  fp32 and element-wise loads take a register
// for every element where 16-bit pairs take half.
constexpr int ln_most(int mode, bool single, bool f32, bool backward)
{
    if (single || (f32 && backward)) return 16;
    if (backward) return 24;
    return f32 ? (mode == 1 ? 16 : 24) : mode == 0 ? 48 : mode == 1 ? 24 : 32;
}

// --------------------------------------------------------------- ring of chunks
//
// Chunk k of a block covers rows [first, first + R) with first = (blockIdx.x + k *
// gridDim.x) * R; a stage holds NT tensors' bytes of it, `pitch` apart, and for the
// backward pass the rows' mean and rstd.
struct LnRing {
    int R;         // rows per chunk, a multiple of G
    int stages;
    int pitch;     // bytes of one tensor's slot: R rows + 32, a multiple of 16
    int stage;     // bytes of a stage, a multiple of 16
};

constexpr int kMaxStages = 8;

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Arrive on `bar` when this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Where chunk bytes [begin, end) of a tensor of `total` bytes lie in its slot: the copy
// starts at the 16-byte boundary at or before begin.
__device__ __forceinline__ int slot_shift(long long begin) { return static_cast<int>(begin & 15); }

// The first warp's part: brings chunk `first` of this block into `stage`.  src: NT tensors
// of M rows of row_bytes; mean and rstd (null: none) go behind the slots, R floats each.
template <int NT>
__device__ __forceinline__ void ln_fill(const LnRing& rg, const char* const (&src)[NT], const float* mean,
                                        const float* rstd, long long M, long long row_bytes, long long first,
                                        uint8_t* st, uint64_t* full)
{
    const int lane = threadIdx.x & 31;
    const int rows = static_cast<int>(M - first < rg.R ? M - first : rg.R);
    if (mean) {
        float* sm = reinterpret_cast<float*>(st + NT * rg.pitch);
        for (int r = lane; r < rows; r += 32) {
            cp_async_4(smem_u32(sm + r), mean + first + r);
            cp_async_4(smem_u32(sm + rg.R + r), rstd + first + r);
        }
        cp_async_arrive(full);
    }
    if (lane == 0) {
        const long long whole = M * row_bytes & ~15LL;   // bulk copies end here at the latest
        const long long begin = first * row_bytes, end = begin + rows * row_bytes;
        const long long a0 = begin & ~15LL;
        const long long up = (end + 15) & ~15LL;
        const long long a1 = up < whole ? up : whole;
        const uint32_t n = a1 > a0 ? static_cast<uint32_t>(a1 - a0) : 0u;
        // the last bytes of the tensor that do not fill 16
        for (int t = 0; t < NT; ++t)
            for (long long i = a1 > begin ? a1 : begin; i < end; i += 2)
                *reinterpret_cast<uint16_t*>(st + t * rg.pitch + (i - a0)) =
                    *reinterpret_cast<const uint16_t*>(src[t] + i);
        mbar_arrive_expect_tx(full, NT * n);
        if (n)
            for (int t = 0; t < NT; ++t) bulk_load(st + t * rg.pitch, src[t] + a0, n, full);
    }
}

// Before the previous kernel on the stream has finished: this block's first chunks into L2,
// the point of coherence, so that the copies that follow see what that kernel writes.
template <int NT>
__device__ __forceinline__ void ln_prefetch(const LnRing& rg, const char* const (&src)[NT], long long M,
                                            long long row_bytes)
{
    if (threadIdx.x != 0) return;
    long long first = static_cast<long long>(blockIdx.x) * rg.R;
    for (int i = 0; i < rg.stages - 1 && first < M; ++i, first += static_cast<long long>(gridDim.x) * rg.R) {
        const long long rows = M - first < rg.R ? M - first : rg.R;
        const long long a0 = (first * row_bytes + 15) & ~15LL, a1 = (first + rows) * row_bytes & ~15LL;
        if (a1 > a0)
            for (int t = 0; t < NT; ++t)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                 reinterpret_cast<uint64_t>(src[t] + a0)),
                             "r"(static_cast<uint32_t>(a1 - a0))
                             : "memory");
    }
}

// Prepares the ring's barriers and starts the first chunks.
template <int NT>
__device__ __forceinline__ void ln_start(const LnRing& rg, const char* const (&src)[NT], const float* mean,
                                         const float* rstd, long long M, long long row_bytes, uint8_t* ring,
                                         uint64_t* full, uint64_t* empty, int* abort_flag)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < rg.stages; ++i) {
            mbar_init(&full[i], mean ? 33 : 1);
            mbar_init(&empty[i], blockDim.x >> 5);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        long long ahead = static_cast<long long>(blockIdx.x) * rg.R;
        for (int i = 0; i < rg.stages - 1 && ahead < M; ++i, ahead += static_cast<long long>(gridDim.x) * rg.R)
            ln_fill<NT>(rg, src, mean, rstd, M, row_bytes, ahead, ring + i * rg.stage, &full[i]);
    }
}

// Runs `chunk(first row, stage's bytes)` over this block's chunks.  Every thread of the
// block takes part; each warp frees a stage when it has read it.  A wait that runs out
// raises the abort flag: nothing more is brought, and the block runs to its end without
// waiting, but for thread 0, which waits for the copies in flight.
template <int NT, typename F>
__device__ __forceinline__ void ln_chunks(const LnRing& rg, const char* const (&src)[NT], const float* mean,
                                          const float* rstd, long long M, long long row_bytes, uint8_t* ring,
                                          uint64_t* full, uint64_t* empty, int* abort_flag, int* status, F chunk)
{
    volatile int* abort = abort_flag;
    bool bringing = threadIdx.x < 32;
    const long long step = static_cast<long long>(gridDim.x) * rg.R;
    long long ahead = (static_cast<long long>(blockIdx.x) + static_cast<long long>(rg.stages - 1) * gridDim.x) * rg.R;
    if (!bringing) ahead = M;   // the next chunk to bring, behind ln_start's
    int stage = 0, fill = rg.stages - 1;
    uint32_t phase = 0, fill_phase = 1;
    for (long long first = static_cast<long long>(blockIdx.x) * rg.R; first < M; first += step) {
        if (bringing && ahead < M) {   // into the stage that the previous chunk was read from
            bool ok = mbar_wait(&empty[fill], fill_phase, abort);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok) {
                ln_fill<NT>(rg, src, mean, rstd, M, row_bytes, ahead, ring + fill * rg.stage, &full[fill]);
            } else {
                report_timeout(status);
                *abort = 1;
            }
            if (ok) ahead += step;
            bringing = ok;
            if (++fill == rg.stages) {
                fill = 0;
                fill_phase ^= 1u;
            }
        }
        // thread 0 waits for every copy it started, whatever has been aborted
        if (!mbar_wait(&full[stage], phase, threadIdx.x == 0 && first < ahead ? nullptr : abort)) {
            report_timeout(status);
            *abort = 1;
        }
        chunk(first, ring + stage * rg.stage);
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[stage]);
        if (++stage == rg.stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
}

struct LnFwd {
    const void* x;
    const void* gamma;   // null: ones
    const void* beta;    // null: zeros
    void* y;
    float* mean;         // null: not wanted
    float* rstd;
    long long M;
    int C, T, G;
    float eps;
    LnRing ring;
    int* status;
};

template <int EK, int VEC, int NV, int MODE, bool RING>
__global__ void __launch_bounds__(ln_block(MODE, false), ln_per_sm(MODE, VEC * NV, false))
    ln_fwd_kernel(const LnFwd p)
{
    constexpr int es = elem_bytes<EK>();
    const char* const src[1] = {static_cast<const char*>(p.x)};
    const long long row_bytes = static_cast<long long>(p.C) * es;
    if constexpr (RING) ln_prefetch<1>(p.ring, src, p.M, row_bytes);
    pdl_wait();      // the previous kernel on the stream has finished
    pdl_trigger();   // the next one may start its set-up
    constexpr bool MULTI = MODE > 0;
    __shared__ float2 red[MULTI ? 128 : 1];
    __shared__ uint64_t bars[RING ? 2 * kMaxStages : 1];
    __shared__ int abort_flag;
    extern __shared__ __align__(16) uint8_t dyn[];
    float* params = reinterpret_cast<float*>(dyn);
    uint8_t* ring = dyn + ln_param_bytes(MODE, p.C, 2);
    uint64_t* full = bars;
    uint64_t* empty = bars + kMaxStages;
    if constexpr (RING)
        ln_start<1>(p.ring, src, nullptr, nullptr, p.M, row_bytes, ring, full, empty, &abort_flag);
    const int group = threadIdx.x / p.T;
    const int lane = threadIdx.x - group * p.T;
    int turn = 0;
    const float fc = static_cast<float>(p.C);
    const int mine = lane_vectors<VEC>(p.C, p.T, lane);

    // gamma and beta: in registers where whole warps share a row; where a row takes at most a
    // warp, every lane meets few of them often, and reads them widened from shared memory
    using P = RowPart<EK, VEC, NV>;
    constexpr int kPer = P::kPer;
    LnParam<EK, VEC, NV, MULTI> gamma, beta;
    gamma.init(params, p.gamma, 1.0f, p.C, p.T, lane);
    beta.init(params + p.C, p.beta, 0.f, p.C, p.T, lane);
    if constexpr (!MULTI) __syncthreads();
    // row m, read from `from`; every thread of the block takes part in each reduction
    auto one_row = [&](long long m, bool live, const void* from) {
        P x;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            x.v[v].zero();
            if (live && v < mine) x.v[v].load(from, (lane + v * p.T) * VEC);
        }
        float2 f[P::kUnits][kPer];   // widened once: x, then x - mean
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < P::kUnits; ++u) {
            x.unit(u, f[u]);
#pragma unroll
            for (int i = 0; i < kPer; ++i) s = __fadd2_rn(s, f[u][i]);
        }
        const float mean = row_sum<MULTI, false>(s.x + s.y, 0.f, p.T, group, red, turn).x / fc;
        const float2 minus = make_float2(-mean, -mean);
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < P::kUnits; ++u) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) f[u][i] = __fadd2_rn(f[u][i], minus);
            mask_unit<VEC>(u, mine, f[u]);
#pragma unroll
            for (int i = 0; i < kPer; ++i) ss = ffma2(f[u][i], f[u][i], ss);
        }
        const float rstd = rsqrtf(row_sum<MULTI, false>(ss.x + ss.y, 0.f, p.T, group, red, turn).x / fc + p.eps);
        if (!live) return;
        if (lane == 0) {
            if (p.mean && store_ok(p.mean, p.M * 4, p.mean + m, 4, p.status)) p.mean[m] = mean;
            if (p.rstd && store_ok(p.rstd, p.M * 4, p.rstd + m, 4, p.status)) p.rstd[m] = rstd;
        }
        const float2 r2 = make_float2(rstd, rstd);
#pragma unroll
        for (int u = 0; u < P::kUnits; ++u) {
            float2 g[kPer], b[kPer];
            if (VEC > 1 && u >= mine) continue;
            gamma.unit(u, p.C, p.T, lane, g);
            beta.unit(u, p.C, p.T, lane, b);
#pragma unroll
            for (int i = 0; i < kPer; ++i) f[u][i] = ffma2(__fmul2_rn(f[u][i], r2), g[i], b[i]);
            x.set_unit(u, f[u]);
        }
        char* out = static_cast<char*>(p.y) + m * p.C * es;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (lane + v * p.T) * VEC;
            if (v < mine && store_ok(p.y, p.M * p.C * es, out + c * es, VEC * es, p.status)) x.v[v].store(out, c);
        }
    };
    if constexpr (!RING) {
        const long long m = static_cast<long long>(blockIdx.x) * p.G + group;
        one_row(m, m < p.M, static_cast<const char*>(p.x) + m * p.C * es);
    } else {
        ln_chunks<1>(p.ring, src, nullptr, nullptr, p.M, row_bytes, ring, full, empty, &abort_flag, p.status, [&](long long first, const uint8_t* st) {
                         st += slot_shift(first * p.C * es);
                         for (int r = group; r < p.ring.R; r += p.G)
                             one_row(first + r, first + r < p.M, st + r * p.C * es);
                     });
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
    int turn = 0;
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
        const float mean = row_sum<true, false>(s, 0.f, kLnLoopThreads, 0, red, turn).x / fc;
        float ss = 0.f;
        for (int c = threadIdx.x * VEC; c < p.C; c += kLnLoopThreads * VEC) {
            V x;
            float f[VEC];
            x.load(p.x, row + c);
            x.unpack(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) ss = fmaf(f[i] - mean, f[i] - mean, ss);
        }
        const float rstd = 1.0f / sqrtf(row_sum<true, false>(ss, 0.f, kLnLoopThreads, 0, red, turn).x / fc + p.eps);
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
    int C, T, G, blocks;
    LnRing ring;
    int* status;
};

template <int EK, int VEC, int NV, int MODE, bool RING>
__global__ void __launch_bounds__(ln_block(MODE, true), ln_per_sm(MODE, VEC * NV, true))
    ln_bwd_kernel(const LnBwd p)
{
    constexpr int es = elem_bytes<EK>();
    const char* const src[2] = {static_cast<const char*>(p.x), static_cast<const char*>(p.dy)};
    const long long row_bytes = static_cast<long long>(p.C) * es;
    if constexpr (RING) ln_prefetch<2>(p.ring, src, p.M, row_bytes);
    pdl_wait();
    pdl_trigger();
    constexpr bool MULTI = MODE > 0;
    __shared__ float2 red[MULTI ? 128 : 1];
    __shared__ uint64_t bars[RING ? 2 * kMaxStages : 1];
    __shared__ int abort_flag;
    extern __shared__ __align__(16) uint8_t dyn[];
    float* params = reinterpret_cast<float*>(dyn);
    uint8_t* ring = dyn + ln_param_bytes(MODE, p.C, 1);   // at the end column sums [warps or groups][2][C]
    uint64_t* full = bars;
    uint64_t* empty = bars + kMaxStages;
    if constexpr (RING) ln_start<2>(p.ring, src, p.mean, p.rstd, p.M, row_bytes, ring, full, empty, &abort_flag);
    const int group = threadIdx.x / p.T;
    const int lane = threadIdx.x - group * p.T;
    int turn = 0;
    const float inv_c = 1.0f / static_cast<float>(p.C);
    const int mine = lane_vectors<VEC>(p.C, p.T, lane);

    using P = RowPart<EK, VEC, NV>;
    constexpr int kPer = P::kPer;
    LnParam<EK, VEC, NV, MULTI> gamma;   // as in the forward kernel
    gamma.init(params, p.gamma, 1.0f, p.C, p.T, lane);
    if constexpr (!MULTI) __syncthreads();
    float2 dg[P::kUnits][kPer], db[P::kUnits][kPer];   // sums down the rows
#pragma unroll
    for (int u = 0; u < P::kUnits; ++u)
#pragma unroll
        for (int i = 0; i < kPer; ++i) dg[u][i] = db[u][i] = make_float2(0.f, 0.f);
    auto one_row = [&](long long m, bool live, const void* fx, const void* fd, float mean, float rstd) {
        P x, dy;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (lane + v * p.T) * VEC;
            x.v[v].zero();
            dy.v[v].zero();
            if (live && v < mine) {
                x.v[v].load(fx, c);
                dy.v[v].load(fd, c);
            }
        }
        const float2 minus = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
        float2 sq = make_float2(0.f, 0.f), sqn = sq;
#pragma unroll
        for (int u = 0; u < P::kUnits; ++u) {
            // a dead row or column must add exactly nothing, whatever mean and rstd hold
            if (!live || (VEC > 1 && u >= mine)) continue;
            float2 n[kPer], d[kPer], g[kPer];
            x.unit(u, n);
            dy.unit(u, d);
            gamma.unit(u, p.C, p.T, lane, g);
#pragma unroll
            for (int i = 0; i < kPer; ++i) n[i] = __fmul2_rn(__fadd2_rn(n[i], minus), r2);
            mask_unit<VEC>(u, mine, n);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float2 q = __fmul2_rn(d[i], g[i]);
                sq = __fadd2_rn(sq, q);
                sqn = ffma2(q, n[i], sqn);
                dg[u][i] = ffma2(d[i], n[i], dg[u][i]);
                db[u][i] = __fadd2_rn(db[u][i], d[i]);
            }
        }
        const float2 t = row_sum<MULTI, true>(sq.x + sq.y, sqn.x + sqn.y, p.T, group, red, turn);
        if (!live) return;
        // rstd (q - mq - n mqn) = q rstd + ((x - mean) (-rstd^2 mqn) - rstd mq)
        const float a = -rstd * rstd * (t.y * inv_c), b = -rstd * (t.x * inv_c);
        const float2 a2 = make_float2(a, a), b2 = make_float2(b, b);
#pragma unroll
        for (int u = 0; u < P::kUnits; ++u) {
            if (VEC > 1 && u >= mine) continue;
            float2 f[kPer], d[kPer], g[kPer];
            x.unit(u, f);
            dy.unit(u, d);
            gamma.unit(u, p.C, p.T, lane, g);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                f[i] = ffma2(__fmul2_rn(d[i], g[i]), r2, ffma2(__fadd2_rn(f[i], minus), a2, b2));
            x.set_unit(u, f);
        }
        char* out = static_cast<char*>(p.dx) + m * p.C * es;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (lane + v * p.T) * VEC;
            if (v < mine && store_ok(p.dx, p.M * p.C * es, out + c * es, VEC * es, p.status)) x.v[v].store(out, c);
        }
    };
    if constexpr (!RING) {
        const long long m = static_cast<long long>(blockIdx.x) * p.G + group;
        const bool live = m < p.M;
        one_row(m, live, static_cast<const char*>(p.x) + m * p.C * es, static_cast<const char*>(p.dy) + m * p.C * es,
                live ? p.mean[m] : 0.f, live ? p.rstd[m] : 0.f);
    } else {
        ln_chunks<2>(p.ring, src, p.mean, p.rstd, p.M, row_bytes, ring, full, empty, &abort_flag, p.status, [&](long long first, const uint8_t* st) {
                         const float* sm = reinterpret_cast<const float*>(st + 2 * p.ring.pitch);
                         const int shift = slot_shift(first * p.C * es);
                         for (int r = group; r < p.ring.R; r += p.G) {
                             const bool live = first + r < p.M;
                             const uint8_t* at = st + shift + r * p.C * es;
                             one_row(first + r, live, at, at + p.ring.pitch, live ? sm[r] : 0.f,
                                     live ? sm[p.ring.R + r] : 0.f);
                         }
                     });
    }
    if (!p.part) return;
    float* out = p.part + static_cast<long long>(blockIdx.x) * 2 * p.C;
    const long long part_bytes = static_cast<long long>(p.blocks) * 2 * p.C * 4;
    // `put` gets every column this thread holds, with its two sums
    auto each = [&](auto put) {
#pragma unroll
        for (int u = 0; u < P::kUnits; ++u)
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = VEC == 1 ? lane + 2 * u * p.T : (lane + u * p.T) * VEC + 2 * i;
                const int c1 = VEC == 1 ? c + p.T : c + 1;
                if (c < p.C) put(c, dg[u][i].x, db[u][i].x);
                if (c1 < p.C) put(c1, dg[u][i].y, db[u][i].y);
            }
    };
    if (p.G == 1) {
        each([&](int c, float a, float b) {
            if (store_ok(p.part, part_bytes, out + c, 4, p.status)) out[c] = a;
            if (store_ok(p.part, part_bytes, out + p.C + c, 4, p.status)) out[p.C + c] = b;
        });
        return;
    }
    // the rows of a warp, then the warps (or groups of warps) one after the other: a fixed order
    if constexpr (!MULTI) {
#pragma unroll
        for (int u = 0; u < P::kUnits; ++u)
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                for (int o = p.T; o < 32; o <<= 1) {
                    dg[u][i].x += __shfl_xor_sync(0xFFFFFFFFu, dg[u][i].x, o);
                    dg[u][i].y += __shfl_xor_sync(0xFFFFFFFFu, dg[u][i].y, o);
                    db[u][i].x += __shfl_xor_sync(0xFFFFFFFFu, db[u][i].x, o);
                    db[u][i].y += __shfl_xor_sync(0xFFFFFFFFu, db[u][i].y, o);
                }
    }
    // every warp's (or group's) sums side by side, then a thread per column in a fixed order
    float* cols = reinterpret_cast<float*>(ring);
    const int parts = MULTI ? p.G : ln_block(0, true) / 32;
    float* own = cols + (MULTI ? group : threadIdx.x >> 5) * 2 * p.C;
    __syncthreads();   // the ring has been read
    if (MULTI || (threadIdx.x & 31) < p.T)
        each([&](int c, float a, float b) {
            own[c] = a;
            own[p.C + c] = b;
        });
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.C; c += blockDim.x) {
        float a = cols[c];
        for (int w = 1; w < parts; ++w) a += cols[w * 2 * p.C + c];
        if (store_ok(p.part, part_bytes, out + c, 4, p.status)) out[c] = a;
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
    int turn = 0;
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
        const float2 t = row_sum<true, true>(sq, sqn, kLnLoopThreads, 0, red, turn);
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
#pragma unroll 8
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

// How a row of C elements is spread: vec elements per load, T threads, nv vectors per
// thread, G rows per block; nv = 0 means the row does not fit and the looped kernels run.
// blocks: the grid; ring.stages 0: one step per block, loaded directly.
struct LnPlan {
    int vec, T, nv, G, blocks;
    LnRing ring;
};

constexpr int kSms = 148;   // a B200; the partial count must not depend on the device asked

// T is the least that holds the row at no more than ln_most elements per thread.  Where the
// rows are too few to give every SM 768 threads, T grows until a thread has one vector (or
// eight elements): the rows' latency is then all there is.
// per_sm blocks share an SM and its shared memory; tensors: how many a stage holds.
LnPlan ln_plan(int64_t M, int C, int ek, int tensors)
{
    const int es = ek == kF32 ? 4 : 2;
    const int wide = 16 / es;
    LnPlan p{};
    p.vec = C % wide == 0 ? wide : 1;
    const int n = C / p.vec;
    // vectors per thread the kernels are compiled for
    static const int wide_nv[] = {1, 2, 3, 4, 6}, one_nv[] = {4, 8, 16, 16, 16};
    const int* nvs = p.vec == 1 ? one_nv : wide_nv;
    auto fit = [&](int T) {   // the least compiled count that holds the row on T threads
        const int need = (n + T - 1) / T;
        for (int i = 0; i < 5; ++i)
            if (nvs[i] >= need)
                return nvs[i] * p.vec <= ln_most(ln_mode(T), p.vec == 1, ek == kF32, tensors > 1) ? nvs[i] : 0;
        return 0;
    };
    const int least = p.vec == 1 ? 8 : 1;
    for (int T = 1; T <= kLnMaxMulti; T = T < 32 ? T * 2 : T + 32) {
        const int nv = fit(T);
        if (!nv) continue;
        p.T = T;
        p.nv = nv;
        if (nv <= least || T >= 256 || M * T >= static_cast<int64_t>(kSms) * 768) break;
    }
    if (!p.nv) {
        const int64_t cap = tensors == 1 ? 4 * kSms : 64;
        p.blocks = static_cast<int>(M < cap ? M : cap);
        return p;
    }
    p.G = p.T <= kLnBlock ? ln_block(ln_mode(p.T), tensors > 1) / p.T : 1;
    const int64_t steps = (M + p.G - 1) / p.G;
    const int64_t row = static_cast<int64_t>(C) * es;
    // chunks of about 12 KB a tensor, stages for a third of an SM's shared memory (half where
    // threads hold column sums), two at least
    const int per_sm = ln_per_sm(ln_mode(p.T), p.nv * p.vec, tensors > 1);
    int k = static_cast<int>((tensors == 1 ? 16384 : 12288) / (row * p.G));
    if (k < 1) k = 1;
    p.ring.R = p.G * k;
    p.ring.pitch = static_cast<int>((p.ring.R * row + 32 + 15) / 16 * 16);
    p.ring.stage = tensors * p.ring.pitch + (tensors > 1 ? (8 * p.ring.R + 15) / 16 * 16 : 0);
    int blocks_per_sm = per_sm;
    int stages = 0;
    for (; blocks_per_sm >= 1; --blocks_per_sm) {
        stages = (220 * 1024 / blocks_per_sm - 4096 - ln_param_bytes(ln_mode(p.T), C, 3 - tensors)) / p.ring.stage;
        if (stages >= 2) break;
    }
    if (blocks_per_sm < 1) {   // not two stages: the looped kernels
        p = LnPlan{};
        p.vec = C % wide == 0 ? wide : 1;
        const int64_t cap = tensors == 1 ? 4 * kSms : 64;
        p.blocks = static_cast<int>(M < cap ? M : cap);
        return p;
    }
    const int64_t grid = static_cast<int64_t>(kSms) * blocks_per_sm;
    if (steps <= (tensors == 1 ? 2 * grid : grid)) {
        p.blocks = static_cast<int>(steps);
        p.ring.stages = 0;
        return p;
    }
    const int64_t chunks = (M + p.ring.R - 1) / p.ring.R;
    p.blocks = static_cast<int>(chunks < grid ? chunks : grid);
    p.ring.stages = stages < kMaxStages ? stages : kMaxStages;
    return p;
}

LnPlan ln_fwd_plan(int64_t M, int C, int ek) { return ln_plan(M, C, ek, 1); }
LnPlan ln_bwd_plan(int64_t M, int C, int ek) { return ln_plan(M, C, ek, 2); }

template <typename A>
cudaError_t run_ln(void (*kern)(A), const A& a, const LnPlan& p, size_t param_bytes, size_t least_smem, cudaStream_t st)
{
    const bool ring = p.ring.stages > 0;
    size_t smem = ring ? static_cast<size_t>(p.ring.stages) * p.ring.stage : 0;
    if (smem < least_smem) smem = least_smem;
    smem += param_bytes;
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(static_cast<unsigned>(p.blocks)),
                         dim3(static_cast<unsigned>(p.G * p.T)), smem, st, 1, a);
}

template <int EK, int VEC, int NV, int MODE>
cudaError_t run_modes_fwd(const LnFwd& a, const LnPlan& p, cudaStream_t st)
{
    if constexpr (MODE > 2) {
        return cudaErrorInvalidValue;
    } else if constexpr (VEC * NV > ln_most(MODE, VEC == 1, EK == kF32, false)) {
        return run_modes_fwd<EK, VEC, NV, MODE + 1>(a, p, st);   // ln_plan does not choose it
    } else {
        if (ln_mode(p.T) != MODE) return run_modes_fwd<EK, VEC, NV, MODE + 1>(a, p, st);
        const size_t params = ln_param_bytes(MODE, a.C, 2);
        return p.ring.stages ? run_ln(ln_fwd_kernel<EK, VEC, NV, MODE, true>, a, p, params, 0, st)
                             : run_ln(ln_fwd_kernel<EK, VEC, NV, MODE, false>, a, p, params, 0, st);
    }
}

template <int EK, int VEC, int NV>
cudaError_t run_fwd(const LnFwd& a, const LnPlan& p, cudaStream_t st)
{
    return run_modes_fwd<EK, VEC, NV, 0>(a, p, st);
}

template <int EK, int VEC, int NV, int MODE>
cudaError_t run_modes_bwd(const LnBwd& a, const LnPlan& p, size_t cols, cudaStream_t st)
{
    if constexpr (MODE > 2) {
        return cudaErrorInvalidValue;
    } else if constexpr (VEC * NV > ln_most(MODE, VEC == 1, EK == kF32, true)) {
        return run_modes_bwd<EK, VEC, NV, MODE + 1>(a, p, cols, st);   // ln_plan does not choose it
    } else {
        if (ln_mode(p.T) != MODE) return run_modes_bwd<EK, VEC, NV, MODE + 1>(a, p, cols, st);
        const size_t params = ln_param_bytes(MODE, a.C, 1);
        return p.ring.stages ? run_ln(ln_bwd_kernel<EK, VEC, NV, MODE, true>, a, p, params, cols, st)
                             : run_ln(ln_bwd_kernel<EK, VEC, NV, MODE, false>, a, p, params, cols, st);
    }
}

template <int EK, int VEC, int NV>
cudaError_t run_bwd(const LnBwd& a, const LnPlan& p, cudaStream_t st)
{
    const size_t cols = p.G == 1 || !a.part ? 0 : static_cast<size_t>(a.C) * 8 * (p.T > 32 ? p.G : ln_block(0, true) / 32);
    return run_modes_bwd<EK, VEC, NV, 0>(a, p, cols, st);
}

template <int EK>
cudaError_t dispatch_fwd(const LnFwd& a, const LnPlan& p, cudaStream_t st)
{
    constexpr int W = EK == kF32 ? 4 : 8;
    if (p.nv == 0) {
        auto kern = p.vec == 1 ? ln_fwd_loop_kernel<EK, 1> : ln_fwd_loop_kernel<EK, W>;
        return launch_kernel(kern, dim3(static_cast<unsigned>(p.blocks)), dim3(kLnLoopThreads), 0, st, 1, a);
    }
    if (p.vec == 1) {
        switch (p.nv) {
        case 4: return run_fwd<EK, 1, 4>(a, p, st);
        case 8: return run_fwd<EK, 1, 8>(a, p, st);
        default: return run_fwd<EK, 1, 16>(a, p, st);
        }
    }
    switch (p.nv) {
    case 1: return run_fwd<EK, W, 1>(a, p, st);
    case 2: return run_fwd<EK, W, 2>(a, p, st);
    case 3: return run_fwd<EK, W, 3>(a, p, st);
    case 4: return run_fwd<EK, W, 4>(a, p, st);
    default: return run_fwd<EK, W, 6>(a, p, st);
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
        default: return run_bwd<EK, 1, 16>(a, p, st);
        }
    }
    switch (p.nv) {
    case 1: return run_bwd<EK, W, 1>(a, p, st);
    case 2: return run_bwd<EK, W, 2>(a, p, st);
    case 3: return run_bwd<EK, W, 3>(a, p, st);
    default: return run_bwd<EK, W, 4>(a, p, st);
    }
}

}  // namespace

cudaError_t launch_layernorm_forward(const LnFwdArgs& a, cudaStream_t stream)
{
    const LnPlan p = ln_fwd_plan(a.M, static_cast<int>(a.C), a.ek);
    const LnFwd k{a.X, a.gamma, a.beta, a.Y, a.mean, a.rstd, a.M, static_cast<int>(a.C), p.T, p.G, a.eps, p.ring,
                  a.status};
    return a.ek == kF32 ? dispatch_fwd<kF32>(k, p, stream)
                        : a.ek == kBF16 ? dispatch_fwd<kBF16>(k, p, stream) : dispatch_fwd<kF16>(k, p, stream);
}

size_t layernorm_backward_workspace_bytes(int64_t M, int64_t C, int ek)
{
    const LnPlan p = ln_bwd_plan(M, static_cast<int>(C), ek);
    return static_cast<size_t>(p.blocks) * 2 * static_cast<size_t>(C) * sizeof(float);
}

cudaError_t launch_layernorm_backward(const LnBwdArgs& a, cudaStream_t stream)
{
    const bool params = a.dgamma || a.dbeta;
    const LnPlan p = ln_bwd_plan(a.M, static_cast<int>(a.C), a.ek);
    const LnBwd k{a.dY, a.X, a.gamma, a.mean, a.rstd, a.dX, params ? a.ws : nullptr, a.M, static_cast<int>(a.C), p.T,
                  p.G, p.blocks, p.ring, a.status};
    cudaError_t e = a.ek == kF32 ? dispatch_bwd<kF32>(k, p, stream)
                                 : a.ek == kBF16 ? dispatch_bwd<kBF16>(k, p, stream) : dispatch_bwd<kF16>(k, p, stream);
    if (e != cudaSuccess || !params) return e;
    auto kern = a.ek == kF32 ? ln_params_kernel<kF32> : a.ek == kBF16 ? ln_params_kernel<kBF16> : ln_params_kernel<kF16>;
    return launch_kernel(kern, dim3(static_cast<unsigned>((2 * a.C + 31) / 32)), dim3(1024), 0, stream, 1, a.ws,
                         k.blocks, k.C, a.dgamma, a.dbeta, a.status);
}

}  // namespace dgrad
