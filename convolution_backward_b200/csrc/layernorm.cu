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
//
// Rows whose length is no multiple of 16 bytes start anywhere.  They too are read and
// written in the 16-byte vectors that lie wholly inside them; the elements before the
// first and behind the last (at most 14, fp32 6) go to one lane each.  A row's offset on
// the 16-byte grid repeats every eight (fp32: four) rows, and the rows of a thread are a
// multiple of that apart, so a thread keeps its columns, and with them its parameters and
// its column sums, in registers from row to row.
// All sums and statistics are fp32; results are rounded once.
//
// The parameter gradients are sums down the columns.  Each block keeps its rows'
// column sums in registers, writes them once as fp32 partials [block][2][C], and
// a second kernel adds the partials of a column in a fixed order: no atomics, so
// results repeat bit for bit.
#include <type_traits>

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

// One thread's part of a row of C elements.  The row's whole 16-byte vectors start at
// column `head`; the thread holds those numbered lane, lane + T, .., `mine` of them.  SH (the
// row starts off its 16-byte grid, so head may not be 0): also one of the columns outside
// the vectors, `single`, or none (-1).
template <int EK, bool SH>
struct LnLane {
    static constexpr int es = elem_bytes<EK>();
    static constexpr int VEC = 16 / es;
    using V = RowVec<EK, VEC>;
    using S = RowVec<EK, 1>;
    int lane, T, C, head, mine, single;

    __device__ __forceinline__ LnLane(int lane_, int T_, int C_, long long row)
        : lane(lane_), T(T_), C(C_), head(0), single(-1)
    {
        if constexpr (SH) {
            head = static_cast<int>((VEC - row * C % VEC) % VEC);
            if (head > C) head = C;
        }
        const int n = (C - head) / VEC;
        mine = lane < n ? (n - lane + T - 1) / T : 0;
        if constexpr (SH) {
            if (lane < head)
                single = lane;
            else if (lane < C - n * VEC)
                single = n * VEC + lane;
        }
    }
    // Column of vector v's first element.
    __device__ __forceinline__ int col(int v) const { return (SH ? head : 0) + (lane + v * T) * VEC; }

    // Vector v (one of the first `have`), and the single column, of the row at p; zeros where
    // there is none.
    __device__ __forceinline__ void load(V& x, const void* p, int v, int have) const
    {
        x.zero();
        if (v < have) x.load(p, col(v));
    }
    __device__ __forceinline__ float load_single(const void* p) const
    {
        float f[1] = {0.f};
        if (single >= 0) {
            S x;
            x.load(p, single);
            x.unpack(f);
        }
        return f[0];
    }
    __device__ __forceinline__ void store(const V& x, void* p, int v, const void* base, long long bytes, int* status) const
    {
        if (v < mine && store_ok(base, bytes, static_cast<char*>(p) + col(v) * es, 16, status)) x.store(p, col(v));
    }
    __device__ __forceinline__ void store_single(float f, void* p, const void* base, long long bytes, int* status) const
    {
        if (single < 0 || !store_ok(base, bytes, static_cast<char*>(p) + single * es, es, status)) return;
        S x;
        const float a[1] = {f};
        x.pack(a);
        x.store(p, single);
    }
    // Zero what vector v holds when it is none of the thread's.
    __device__ __forceinline__ void mask(int v, float2 (&f)[VEC / 2]) const
    {
        if (v >= mine) {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) f[i] = make_float2(0.f, 0.f);
        }
    }
};

// gamma or beta.  REG: in the thread's registers, at its columns.  Else as fp32 in shared
// memory (rows on the 16-byte grid, at most a warp each): vector v's quarters (four
// elements each) lie n vectors apart, so that adjacent lanes' 16-byte reads are adjacent.
// A null pointer gives the constant.
template <int EK, int NV, bool REG, bool SH>
struct LnParam {
    using L = LnLane<EK, SH>;
    static constexpr int VEC = L::VEC;
    typename L::V reg[NV];
    float single;
    const float* sm;

    __device__ __forceinline__ void init(const L& l, float* smem, const void* src, float constant)
    {
        if constexpr (REG) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (constant != 0.f)
                    reg[v].ones();
                else
                    reg[v].zero();
                // a thread's columns lie anywhere on the parameter's own 16-byte grid
                if (src && v < l.mine) {
                    if constexpr (SH) {
                        float f[VEC];
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            RowVec<EK, 1> x;
                            float e[1];
                            x.load(src, l.col(v) + i);
                            x.unpack(e);
                            f[i] = e[0];
                        }
                        reg[v].pack(f);
                    } else {
                        l.load(reg[v], src, v, l.mine);
                    }
                }
            }
            single = src ? l.load_single(src) : constant;
        } else {
            const int n = l.C / VEC;
            for (int c = threadIdx.x; c < l.C; c += blockDim.x) {
                float f[1] = {constant};
                if (src) {
                    RowVec<EK, 1> x;
                    x.load(src, c);
                    x.unpack(f);
                }
                smem[((c % VEC / 4) * n + c / VEC) * 4 + c % 4] = f[0];
            }
            sm = smem;
        }
    }

    __device__ __forceinline__ void get(const L& l, int v, float2 (&f)[VEC / 2]) const
    {
        if constexpr (REG) {
            unpack_pairs(reg[v], f);
        } else {
            const int n = l.C / VEC;
            const float4* q = reinterpret_cast<const float4*>(sm) + l.lane + v * l.T;
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const float4 w = q[i * n];
                f[2 * i] = make_float2(w.x, w.y);
                f[2 * i + 1] = make_float2(w.z, w.w);
            }
        }
    }
};

// How a row's threads meet: 0, within a warp; 1, whole warps of a block of several rows
// (or of 256 threads); 2, a block of more than 256 threads.
constexpr int ln_mode(int T) { return T <= 32 ? 0 : T <= kLnBlock ? 1 : 2; }

// Threads of a block.  Where a warp needs no other (mode 0), the backward pass has many
// instructions per chunk and few warps: with blocks of four warps a chunk waits for fewer
// others (401408 x 96 bf16: 43.9 us, against 47.3 with eight; forward 21.4 against 21.0).
// Rows off the 16-byte grid need eight rows at a time, and keep eight warps.
constexpr int ln_block(int mode, bool backward, bool sh)
{
    return mode == 2 ? kLnMaxMulti : mode == 0 && backward && !sh ? 128 : kLnBlock;
}

// Threads an SM holds (of ln_block a block), by the registers their elements take.  768 where
// up to 16 elements, with 16-bit parameters beside them or none, leave 80 registers (4882 x
// 4096 bf16 forward: 22.3 us, with 512 threads 24.0); else 512, or one block of up to 384.
constexpr int ln_threads(int mode, int elems, bool backward, bool sh, bool f32)
{
    if (mode == 2) return kLnMaxMulti;
    return !backward && elems <= 16 && !sh && (mode == 0 || !f32) ? 768 : 512;
}
constexpr int ln_per_sm(int mode, int elems, bool backward, bool sh, bool f32)
{
    return ln_threads(mode, elems, backward, sh, f32) / ln_block(mode, backward, sh);
}

// Rows on the 16-byte grid of at most a warp keep their parameters in shared memory.
constexpr bool ln_param_regs(int mode, bool sh) { return mode > 0 || sh; }

// Shared memory for `count` parameters.
__host__ __device__ constexpr int ln_param_bytes(int mode, bool sh, int C, int count)
{
    return ln_param_regs(mode, sh) ? 0 : (count * C * 4 + 15) / 16 * 16;
}

// Elements per thread that fit its registers without spills (but for a few words).  Forward: 64
// where the parameters are in shared memory, 24 or (one block per SM) 32 beside them.  Backward: the
// column sums take two registers per element.  fp32 takes a register for every element
// where 16-bit pairs take half.
constexpr int ln_most(int mode, bool sh, bool f32, bool backward)
{
    if (backward) return mode == 2 ? (f32 ? 24 : 32) : f32 ? 16 : 24;
    if (!ln_param_regs(mode, sh)) return f32 ? 32 : 64;
    return f32 ? (mode == 1 ? 16 : 24) : mode == 2 ? 32 : 24;
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

template <int EK, int NV, int MODE, bool RING, bool SH>
__global__ void __launch_bounds__(ln_block(MODE, false, SH), ln_per_sm(MODE, 16 / elem_bytes<EK>() * NV, false, SH, EK == kF32))
    ln_fwd_kernel(const LnFwd p)
{
    constexpr int es = elem_bytes<EK>();
    const char* const src[1] = {static_cast<const char*>(p.x)};
    const long long row_bytes = static_cast<long long>(p.C) * es;
    if constexpr (RING) ln_prefetch<1>(p.ring, src, p.M, row_bytes);
    pdl_wait();      // the previous kernel on the stream has finished
    pdl_trigger();   // the next one may start its set-up
    constexpr bool MULTI = MODE > 0;
    constexpr bool REG = ln_param_regs(MODE, SH);
    __shared__ float2 red[MULTI ? 128 : 1];
    __shared__ uint64_t bars[RING ? 2 * kMaxStages : 1];
    __shared__ int abort_flag;
    extern __shared__ __align__(16) uint8_t dyn[];
    float* params = reinterpret_cast<float*>(dyn);
    uint8_t* ring = dyn + ln_param_bytes(MODE, SH, p.C, 2);
    uint64_t* full = bars;
    uint64_t* empty = bars + kMaxStages;
    if constexpr (RING)
        ln_start<1>(p.ring, src, nullptr, nullptr, p.M, row_bytes, ring, full, empty, &abort_flag);
    const int group = threadIdx.x / p.T;
    int turn = 0;
    const float fc = static_cast<float>(p.C);
    using L = LnLane<EK, SH>;
    constexpr int H = L::VEC / 2;   // pairs of a vector
    // every row of this thread starts where this one does on its 16-byte grid (ln_plan)
    const L l(threadIdx.x - group * p.T, p.T, p.C, static_cast<long long>(blockIdx.x) * (RING ? p.ring.R : p.G) + group);
    LnParam<EK, NV, REG, SH> gamma, beta;
    gamma.init(l, params, p.gamma, 1.0f);
    beta.init(l, params + p.C, p.beta, 0.f);
    if constexpr (!REG) __syncthreads();
    // row m, read from `from`; every thread of the block takes part in each reduction
    auto one_row = [&](long long m, bool live, const void* from) {
        const int have = live ? l.mine : 0;
        float2 f[NV][H];   // widened once: x, then x - mean
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            typename L::V x;
            l.load(x, from, v, have);
            unpack_pairs(x, f[v]);
#pragma unroll
            for (int i = 0; i < H; ++i) s = __fadd2_rn(s, f[v][i]);
        }
        float one = 0.f;   // the single column
        if constexpr (SH) {
            if (live) one = l.load_single(from);
            s.x += one;
        }
        const float mean = row_sum<MULTI, false>(s.x + s.y, 0.f, p.T, group, red, turn).x / fc;
        const float2 minus = make_float2(-mean, -mean);
        float2 ss = make_float2(0.f, 0.f);
        if constexpr (SH) {
            one = l.single < 0 ? 0.f : one - mean;
            ss.x = one * one;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < H; ++i) f[v][i] = __fadd2_rn(f[v][i], minus);
            l.mask(v, f[v]);
#pragma unroll
            for (int i = 0; i < H; ++i) ss = ffma2(f[v][i], f[v][i], ss);
        }
        const float rstd = rsqrtf(row_sum<MULTI, false>(ss.x + ss.y, 0.f, p.T, group, red, turn).x / fc + p.eps);
        if (!live) return;
        if (l.lane == 0) {
            if (p.mean && store_ok(p.mean, p.M * 4, p.mean + m, 4, p.status)) p.mean[m] = mean;
            if (p.rstd && store_ok(p.rstd, p.M * 4, p.rstd + m, 4, p.status)) p.rstd[m] = rstd;
        }
        const float2 r2 = make_float2(rstd, rstd);
        char* out = static_cast<char*>(p.y) + m * p.C * es;
        if constexpr (SH) l.store_single(fmaf(one * rstd, gamma.single, beta.single), out, p.y, p.M * p.C * es, p.status);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (v >= l.mine) continue;
            float2 g[H], b[H];
            gamma.get(l, v, g);
            beta.get(l, v, b);
#pragma unroll
            for (int i = 0; i < H; ++i) f[v][i] = ffma2(__fmul2_rn(f[v][i], r2), g[i], b[i]);
            typename L::V y;
            pack_pairs(y, f[v]);
            l.store(y, out, v, p.y, p.M * p.C * es, p.status);
        }
    };
    if constexpr (!RING) {
        const long long m = static_cast<long long>(blockIdx.x) * p.G + group;
        one_row(m, m < p.M, static_cast<const char*>(p.x) + m * p.C * es);
    } else {
        ln_chunks<1>(p.ring, src, nullptr, nullptr, p.M, row_bytes, ring, full, empty, &abort_flag, p.status,
                     [&](long long first, const uint8_t* st) {
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

template <int EK, int NV, int MODE, bool RING, bool SH>
__global__ void __launch_bounds__(ln_block(MODE, true, SH), ln_per_sm(MODE, 16 / elem_bytes<EK>() * NV, true, SH, EK == kF32))
    ln_bwd_kernel(const LnBwd p)
{
    constexpr int es = elem_bytes<EK>();
    const char* const src[2] = {static_cast<const char*>(p.x), static_cast<const char*>(p.dy)};
    const long long row_bytes = static_cast<long long>(p.C) * es;
    if constexpr (RING) ln_prefetch<2>(p.ring, src, p.M, row_bytes);
    pdl_wait();
    pdl_trigger();
    constexpr bool MULTI = MODE > 0;
    constexpr bool REG = ln_param_regs(MODE, SH);
    __shared__ float2 red[MULTI ? 128 : 1];
    __shared__ uint64_t bars[RING ? 2 * kMaxStages : 1];
    __shared__ int abort_flag;
    extern __shared__ __align__(16) uint8_t dyn[];
    float* params = reinterpret_cast<float*>(dyn);
    uint8_t* ring = dyn + ln_param_bytes(MODE, SH, p.C, 1);   // at the end column sums [warps or groups][2][C]
    uint64_t* full = bars;
    uint64_t* empty = bars + kMaxStages;
    if constexpr (RING) ln_start<2>(p.ring, src, p.mean, p.rstd, p.M, row_bytes, ring, full, empty, &abort_flag);
    const int group = threadIdx.x / p.T;
    int turn = 0;
    const float inv_c = 1.0f / static_cast<float>(p.C);
    using L = LnLane<EK, SH>;
    constexpr int H = L::VEC / 2;
    const L l(threadIdx.x - group * p.T, p.T, p.C, static_cast<long long>(blockIdx.x) * (RING ? p.ring.R : p.G) + group);
    LnParam<EK, NV, REG, SH> gamma;   // as in the forward kernel
    gamma.init(l, params, p.gamma, 1.0f);
    if constexpr (!REG) __syncthreads();
    float2 dg[NV][H], db[NV][H];   // sums down the rows
    float dg1 = 0.f, db1 = 0.f;    // the single column's
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < H; ++i) dg[v][i] = db[v][i] = make_float2(0.f, 0.f);
    auto one_row = [&](long long m, bool live, const void* fx, const void* fd, float mean, float rstd) {
        const int have = live ? l.mine : 0;
        typename L::V x[NV], dy[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            l.load(x[v], fx, v, have);
            l.load(dy[v], fd, v, have);
        }
        const float2 minus = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
        float2 sq = make_float2(0.f, 0.f), sqn = sq;
        float x1 = 0.f, q1 = 0.f;   // the single column
        if constexpr (SH) {
            if (live && l.single >= 0) {
                const float d = l.load_single(fd);
                x1 = l.load_single(fx) - mean;
                q1 = d * gamma.single;
                sq.x = q1;
                sqn.x = q1 * (x1 * rstd);
                dg1 = fmaf(d, x1 * rstd, dg1);
                db1 += d;
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            // a dead row or column must add exactly nothing, whatever mean and rstd hold
            if (v >= have) continue;
            float2 n[H], d[H], g[H];
            unpack_pairs(x[v], n);
            unpack_pairs(dy[v], d);
            gamma.get(l, v, g);
#pragma unroll
            for (int i = 0; i < H; ++i) n[i] = __fmul2_rn(__fadd2_rn(n[i], minus), r2);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float2 q = __fmul2_rn(d[i], g[i]);
                sq = __fadd2_rn(sq, q);
                sqn = ffma2(q, n[i], sqn);
                dg[v][i] = ffma2(d[i], n[i], dg[v][i]);
                db[v][i] = __fadd2_rn(db[v][i], d[i]);
            }
        }
        const float2 t = row_sum<MULTI, true>(sq.x + sq.y, sqn.x + sqn.y, p.T, group, red, turn);
        if (!live) return;
        // rstd (q - mq - n mqn) = q rstd + (n (-rstd mqn) - rstd mq), with n formed again: rstd^2
        // lies outside fp32's range for rows whose spread is below 2^-64
        const float a = -rstd * (t.y * inv_c), b = -rstd * (t.x * inv_c);
        const float2 a2 = make_float2(a, a), b2 = make_float2(b, b);
        char* out = static_cast<char*>(p.dx) + m * p.C * es;
        if constexpr (SH) l.store_single(fmaf(q1, rstd, fmaf(x1 * rstd, a, b)), out, p.dx, p.M * p.C * es, p.status);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (v >= l.mine) continue;
            float2 f[H], d[H], g[H];
            unpack_pairs(x[v], f);
            unpack_pairs(dy[v], d);
            gamma.get(l, v, g);
#pragma unroll
            for (int i = 0; i < H; ++i)
                f[i] = ffma2(__fmul2_rn(d[i], g[i]), r2, ffma2(__fmul2_rn(__fadd2_rn(f[i], minus), r2), a2, b2));
            pack_pairs(x[v], f);
            l.store(x[v], out, v, p.dx, p.M * p.C * es, p.status);
        }
    };
    if constexpr (!RING) {
        const long long m = static_cast<long long>(blockIdx.x) * p.G + group;
        const bool live = m < p.M;
        one_row(m, live, static_cast<const char*>(p.x) + m * p.C * es, static_cast<const char*>(p.dy) + m * p.C * es,
                live ? p.mean[m] : 0.f, live ? p.rstd[m] : 0.f);
    } else {
        ln_chunks<2>(p.ring, src, p.mean, p.rstd, p.M, row_bytes, ring, full, empty, &abort_flag, p.status,
                     [&](long long first, const uint8_t* st) {
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
    // This thread's columns to dst [2][C]; ADD: added to what is there.  checked: the partials.
    auto put = [&](float* dst, auto add, bool checked) {
        constexpr bool ADD = decltype(add)::value;
        auto one = [&](int c, float v) {
            if (!checked || store_ok(p.part, part_bytes, dst + c, 4, p.status)) dst[c] = ADD ? dst[c] + v : v;
        };
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (v >= l.mine) continue;
            const int c = l.col(v);
            if constexpr (!SH && !ADD) {   // whole quarters, 16 bytes each
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    float* at = dst + c + 2 * i;
                    if (checked && !(store_ok(p.part, part_bytes, at, 16, p.status) &&
                                     store_ok(p.part, part_bytes, at + p.C, 16, p.status)))
                        continue;
                    *reinterpret_cast<float4*>(at) = make_float4(dg[v][i].x, dg[v][i].y, dg[v][i + 1].x, dg[v][i + 1].y);
                    *reinterpret_cast<float4*>(at + p.C) =
                        make_float4(db[v][i].x, db[v][i].y, db[v][i + 1].x, db[v][i + 1].y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    one(c + 2 * i, dg[v][i].x);
                    one(c + 2 * i + 1, dg[v][i].y);
                    one(p.C + c + 2 * i, db[v][i].x);
                    one(p.C + c + 2 * i + 1, db[v][i].y);
                }
            }
        }
        if constexpr (SH) {
            if (l.single >= 0) {
                one(l.single, dg1);
                one(p.C + l.single, db1);
            }
        }
    };
    if (!SH && p.G == 1) {   // (off the grid the columns go through shared memory, to leave in whole lines)
        put(out, std::false_type{}, true);
        return;
    }
    // every warp's (or group's) sums side by side, then a thread per column in a fixed order
    float* cols = reinterpret_cast<float*>(ring);
    const int parts = MULTI ? p.G : static_cast<int>(blockDim.x >> 5);
    float* own = cols + (MULTI ? group : threadIdx.x >> 5) * 2 * p.C;
    __syncthreads();   // the ring has been read
    if constexpr (MULTI) {
        put(own, std::false_type{}, false);
    } else if constexpr (!SH) {
        // the rows of a warp hold the same columns in the same lanes
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < H; ++i)
                for (int o = p.T; o < 32; o <<= 1) {
                    dg[v][i].x += __shfl_xor_sync(0xFFFFFFFFu, dg[v][i].x, o);
                    dg[v][i].y += __shfl_xor_sync(0xFFFFFFFFu, dg[v][i].y, o);
                    db[v][i].x += __shfl_xor_sync(0xFFFFFFFFu, db[v][i].x, o);
                    db[v][i].y += __shfl_xor_sync(0xFFFFFFFFu, db[v][i].y, o);
                }
        if ((threadIdx.x & 31) < p.T) put(own, std::false_type{}, false);
    } else {
        // they do not where rows start at different offsets: one row's threads after the other
        const int turns = 32 / p.T, mine = (threadIdx.x & 31) / p.T;
        for (int k = 0; k < turns; ++k) {
            if (mine == k) {
                if (k == 0)
                    put(own, std::false_type{}, false);
                else
                    put(own, std::true_type{}, false);
            }
            __syncwarp();
        }
    }
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

// How a row of C elements is spread: T threads, nv 16-byte vectors per thread, G rows per
// block; sh: rows off the 16-byte grid; nv = 0 means the row does not fit and the looped
// kernels run.  blocks: the grid; ring.stages 0: one step per block, loaded directly.
struct LnPlan {
    bool sh;
    int T, nv, G, blocks;
    LnRing ring;
};

constexpr int kSms = 148;   // a B200; the partial count must not depend on the device asked

LnPlan ln_plan(int64_t M, int C, int ek, bool backward)
{
    const int es = ek == kF32 ? 4 : 2;
    const int vec = 16 / es;
    const int tensors = backward ? 2 : 1;
    LnPlan p{};
    p.sh = C % vec != 0;
    const int n = C >= vec ? C / vec : 1;   // whole vectors of a row (at most, off the grid)
    static const int nvs[] = {1, 2, 3, 4, 6, 8};   // vectors per thread the kernels are compiled for
    auto fit = [&](int T, int most) {   // the least compiled count that holds the row on T threads
        const int need = (n + T - 1) / T;
        for (int nv : nvs)
            if (nv >= need) return nv * vec <= most ? nv : 0;
        return 0;
    };
    // T is the least that holds the row at no more than ln_most elements per thread (a larger one
    // of at most 128 where that leaves an eighth fewer vectors empty), or at 16 where whole
    // warps share it and that takes no more than 256 threads (9765 x 2048 bf16 backward: 36 us
    // with 16, 46 with 24).  Rows off the grid have up to 2 (vec - 1)
    // columns outside their vectors, a lane each.
    const int least = p.sh ? 2 * vec : 1;
    const auto next = [](int T) { return T < 32 ? T * 2 : T + 32; };
    const auto held = [&](int T, bool wide) {
        const int mode = ln_mode(T);
        const int most = ln_most(mode, p.sh, ek == kF32, backward);
        return fit(T, mode == 1 && !wide && most > 16 ? 16 : most);
    };
    for (int pass = 0; pass < 2 && !p.nv; ++pass)
        for (int T = least; T <= (pass ? kLnMaxMulti : kLnBlock); T = next(T)) {
            const int nv = held(T, pass > 0);
            if (nv && (!p.nv || (T <= 128 && 8 * T * nv <= 7 * p.T * p.nv))) {
                p.T = T;
                p.nv = nv;
            }
        }
    // Rows too few to give every SM 512 threads take more threads each, down to one vector: their
    // latency is then all there is (256 x 768 bf16: 2.6 us forward, 6.2 backward; without 3.9
    // and 7.7).
    for (int T = next(p.T); p.nv > 1 && T <= kLnBlock && M * p.T < static_cast<int64_t>(kSms) * 512; T = next(T)) {
        const int nv = held(T, true);
        if (nv && nv < p.nv) {
            p.T = T;
            p.nv = nv;
        }
    }
    auto looped = [&] {
        const int64_t cap = backward ? 64 : 4 * kSms;
        LnPlan q{};
        q.sh = p.sh;
        q.blocks = static_cast<int>(M < cap ? M : cap);
        return q;
    };
    if (!p.nv) return looped();
    const int mode = ln_mode(p.T);
    p.G = p.T <= kLnBlock ? ln_block(mode, backward, p.sh) / p.T : 1;
    const int64_t steps = (M + p.G - 1) / p.G;
    const int64_t row = static_cast<int64_t>(C) * es;
    // Chunks of up to 12 KB a tensor (16 KB forward), as many stages as the SM's blocks have
    // shared memory for, two at least.  A block's steps are dealt out evenly over its chunks: 12
    // and 16 KB of short rows would else leave most blocks without one (bf16, 9473 x 9: 4.9 us
    // forward and 8.5 backward, else 37 and 24; 160009 x 9: 28 and 29, else 40 and 35).
    int per_sm = mode == 2 ? 1 : ln_threads(mode, p.nv * vec, backward, p.sh, ek == kF32) / (p.G * p.T);
    int k = static_cast<int>((backward ? 12288 : 16384) / (row * p.G));
    if (k < 1 || (p.sh && p.G % vec)) k = 1;
    const int64_t per = (steps + kSms * per_sm - 1) / (kSms * per_sm);
    const int64_t even = (per + k - 1) / k;
    k = static_cast<int>((per + even - 1) / even);
    p.ring.R = p.G * k;
    p.ring.pitch = static_cast<int>((p.ring.R * row + 32 + 15) / 16 * 16);
    p.ring.stage = tensors * p.ring.pitch + (backward ? (8 * p.ring.R + 15) / 16 * 16 : 0);
    int stages = 0;
    for (; per_sm >= 1; --per_sm) {
        stages = (220 * 1024 / per_sm - 4096 - ln_param_bytes(mode, p.sh, C, backward ? 1 : 2)) / p.ring.stage;
        if (stages >= 2) break;
    }
    if (per_sm < 1) return looped();
    // One step per block (forward: two blocks' worth): direct loads (256 x 768 bf16: 2.6 us forward,
    // 6.2 backward; through the ring 6.0 and 6.9).
    int64_t grid = static_cast<int64_t>(kSms) * per_sm;
    if (steps <= (backward ? grid : 2 * grid)) {
        p.blocks = static_cast<int>(steps);
        p.ring.stages = 0;
        return p;
    }
    // rows off the grid: the rows of a thread lie a multiple of vec apart, which G rows at a
    // time give when G is one, and else a grid whose rows are one
    if (p.sh && p.G % vec)
        while (grid * p.G % vec) --grid;
    const int64_t chunks = (M + p.ring.R - 1) / p.ring.R;
    p.blocks = static_cast<int>(chunks < grid ? chunks : grid);
    p.ring.stages = stages < kMaxStages ? stages : kMaxStages;
    return p;
}

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

// Finds the compiled kernel of a plan: mode, vectors per thread, grid or not.
template <int EK, int NV, int MODE, bool SH>
cudaError_t run_fwd(const LnFwd& a, const LnPlan& p, cudaStream_t st)
{
    if constexpr (MODE > 2) {
        return cudaErrorInvalidValue;
    } else {
        if constexpr (16 / elem_bytes<EK>() * NV <= ln_most(MODE, SH, EK == kF32, false)) {
            if (ln_mode(p.T) == MODE) {
                const size_t params = ln_param_bytes(MODE, SH, a.C, 2);
                return p.ring.stages ? run_ln(ln_fwd_kernel<EK, NV, MODE, true, SH>, a, p, params, 0, st)
                                     : run_ln(ln_fwd_kernel<EK, NV, MODE, false, SH>, a, p, params, 0, st);
            }
        }
        return run_fwd<EK, NV, MODE + 1, SH>(a, p, st);
    }
}

template <int EK, bool SH>
cudaError_t pick_fwd(const LnFwd& a, const LnPlan& p, cudaStream_t st)
{
    switch (p.nv) {
    case 1: return run_fwd<EK, 1, 0, SH>(a, p, st);
    case 2: return run_fwd<EK, 2, 0, SH>(a, p, st);
    case 3: return run_fwd<EK, 3, 0, SH>(a, p, st);
    case 4: return run_fwd<EK, 4, 0, SH>(a, p, st);
    case 6: return run_fwd<EK, 6, 0, SH>(a, p, st);
    default: return run_fwd<EK, 8, 0, SH>(a, p, st);
    }
}

// Finds the compiled kernel of a plan: mode, vectors per thread, grid or not.
template <int EK, int NV, int MODE, bool SH>
cudaError_t run_bwd(const LnBwd& a, const LnPlan& p, size_t cols, cudaStream_t st)
{
    if constexpr (MODE > 2) {
        return cudaErrorInvalidValue;
    } else {
        if constexpr (16 / elem_bytes<EK>() * NV <= ln_most(MODE, SH, EK == kF32, true)) {
            if (ln_mode(p.T) == MODE) {
                const size_t params = ln_param_bytes(MODE, SH, a.C, 1);
                return p.ring.stages ? run_ln(ln_bwd_kernel<EK, NV, MODE, true, SH>, a, p, params, cols, st)
                                     : run_ln(ln_bwd_kernel<EK, NV, MODE, false, SH>, a, p, params, cols, st);
            }
        }
        return run_bwd<EK, NV, MODE + 1, SH>(a, p, cols, st);
    }
}

template <int EK, bool SH>
cudaError_t pick_bwd(const LnBwd& a, const LnPlan& p, size_t cols, cudaStream_t st)
{
    switch (p.nv) {
    case 1: return run_bwd<EK, 1, 0, SH>(a, p, cols, st);
    case 2: return run_bwd<EK, 2, 0, SH>(a, p, cols, st);
    case 3: return run_bwd<EK, 3, 0, SH>(a, p, cols, st);
    case 4: return run_bwd<EK, 4, 0, SH>(a, p, cols, st);
    default: return run_bwd<EK, 6, 0, SH>(a, p, cols, st);
    }
}

template <int EK>
cudaError_t dispatch_fwd(const LnFwd& a, const LnPlan& p, cudaStream_t st)
{
    if (p.nv == 0) {
        auto kern = p.sh ? ln_fwd_loop_kernel<EK, 1> : ln_fwd_loop_kernel<EK, 16 / elem_bytes<EK>()>;
        return launch_kernel(kern, dim3(static_cast<unsigned>(p.blocks)), dim3(kLnLoopThreads), 0, st, 1, a);
    }
    return p.sh ? pick_fwd<EK, true>(a, p, st) : pick_fwd<EK, false>(a, p, st);
}

template <int EK>
cudaError_t dispatch_bwd(const LnBwd& a, const LnPlan& p, cudaStream_t st)
{
    constexpr int W = 16 / elem_bytes<EK>();
    if (p.nv == 0) {
        if (a.part) {
            auto cols = p.sh ? ln_cols_kernel<EK, 1> : ln_cols_kernel<EK, W>;
            const int n = p.sh ? a.C : a.C / W;
            const cudaError_t e = launch_kernel(cols, dim3((n + 255) / 256, a.blocks), dim3(256), 0, st, 1, a);
            if (e != cudaSuccess) return e;
        }
        auto kern = p.sh ? ln_bwd_loop_kernel<EK, 1> : ln_bwd_loop_kernel<EK, W>;
        const int64_t most = 4 * kSms;
        return launch_kernel(kern, dim3(static_cast<unsigned>(a.M < most ? a.M : most)), dim3(kLnLoopThreads), 0, st,
                             1, a);
    }
    // the block's column sums, one after the chunks
    const size_t parts = p.T > 32 ? p.G : ln_block(0, true, p.sh) / 32;
    const size_t cols = (p.G == 1 && !p.sh) || !a.part ? 0 : static_cast<size_t>(a.C) * 8 * parts;
    return p.sh ? pick_bwd<EK, true>(a, p, cols, st) : pick_bwd<EK, false>(a, p, cols, st);
}

}  // namespace

cudaError_t launch_layernorm_forward(const LnFwdArgs& a, cudaStream_t stream)
{
    const LnPlan p = ln_plan(a.M, static_cast<int>(a.C), a.ek, false);
    const LnFwd k{a.X, a.gamma, a.beta, a.Y, a.mean, a.rstd, a.M, static_cast<int>(a.C), p.T, p.G, a.eps, p.ring,
                  a.status};
    return a.ek == kF32 ? dispatch_fwd<kF32>(k, p, stream)
                        : a.ek == kBF16 ? dispatch_fwd<kBF16>(k, p, stream) : dispatch_fwd<kF16>(k, p, stream);
}

size_t layernorm_backward_workspace_bytes(int64_t M, int64_t C, int ek)
{
    const LnPlan p = ln_plan(M, static_cast<int>(C), ek, true);
    return static_cast<size_t>(p.blocks) * 2 * static_cast<size_t>(C) * sizeof(float);
}

cudaError_t launch_layernorm_backward(const LnBwdArgs& a, cudaStream_t stream)
{
    const bool params = a.dgamma || a.dbeta;
    const LnPlan p = ln_plan(a.M, static_cast<int>(a.C), a.ek, true);
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
