// gated_bwd.cu -- gradients of the gated pointwise block H = act(G) * U, [G | U] = X W^T.
//
//     dZ = [dH U act'(G) | dH act(G)]          M x 2F, element by element
//     dX = dZ W                                 M x C, sums over 2F
//     dW = dZ^T X                               2F x C, sums over the M rows
//
// 8 M F C operations in two GEMMs of equal size; dZ is formed once, in fp32 from the
// kept pre-activations, and rounded to the operands' 16 bits (the tensor cores take no
// wider type at this rate) into the workspace, from where both GEMMs read it.  That is a
// second rounding: terms and their errors both grow with the root of their number, so the
// gradients' error is about sqrt(2) times that of rounding the results alone, in norm, however
// long the sums (against 64 bits: bf16 2.3e-3 and 1.7e-3, f16 2.9e-4 and 2.1e-4).  dX is the
// pointwise dgrad GEMM with K = 2F.
//
// wgrad_pair_kernel: dW's tiles of 256 x BN on pairs of SMs.  The sums run over rows, so
// both operands lie MN-major in memory (their columns contiguous) and go to the MMA as
// they are: TMA boxes of 64 rows x 64 columns, 128-byte swizzle, descriptors with 8 KB
// between the 64-column atoms.  A weight has few tiles and M is long, so the rows are
// split over pairs until they fill the GPU; each split stores its fp32 tile into the
// workspace and a second kernel adds the splits in order and rounds once (no atomics:
// results repeat).  With one split the tile is rounded and stored directly.
//
// Few values of dZ (few_kernels: M F <= 4096) leave the tensor cores little to do: dZ then
// stays fp32, with no second rounding, and fp32 multiply-adds form dX and dW.  At 4096 values
// the two ways take about the same time, with fewer this one is faster.  The backward pass in bf16,
// us, this way and through the GEMMs:
//     rows, C to F          values                    rows, C to F          values
//     1, 64 to 8                8    3.9   8.1        64, 768 to 64         4096  10.4  11.0
//     8, 64 to 64             512    8.0   8.7        64, 2048 to 64        4096  13.1  11.4
//     1, 768 to 2048         2048   10.9  15.8        128, 768 to 32        4096  10.2  11.1
//     8, 768 to 512          4096    9.5  13.2        256, 768 to 16        4096  13.7  11.8
//     32, 768 to 128         4096   15.3  12.0        512, 768 to 8         4096   9.0  14.1
//     64, 64 to 64           4096    9.8   8.9        4, 768 to 2048        8192  20.0  16.7
//     512, 64 to 8           4096    8.7  10.8        1, 2048 to 8192       8192  76    44
#include "common.cuh"
#include "gate_act.cuh"
#include "host_util.h"
#include "launchers.h"

namespace dgrad {
namespace {

constexpr int kBK = 64;
constexpr int kThreads = 192;
constexpr int kStages = 6;
constexpr int kSms = 148;   // a B200; splits and workspaces must not depend on the device asked

// ------------------------------------------------------------------- dZ

// f16 holds less range than the fp32 values of dZ: products of gradients of some hundreds pass 65504, and
// small ones fall among its subnormals.  So the pass that forms dZ also finds its largest finite
// value, block by block, and where that lies beyond 65504 or below 2^-10 (there the subnormals'
// half step, 2^-25, is more than 2^-15 of it) a second pass writes dZ again, times the power of two that
// takes it to 2^14 .. 2^15.  The products' fp32 sums are multiplied by the inverse before they are
// rounded.  What is then below 2^-29 of the largest value keeps an error of 2^-39 of that.  Where dZ
// needs no scaling the second kernel only reads the blocks' values: f16, 300 rows, 136 to 264
// channels 17.1 us (15.7 without), 25088 rows, 256 to 512 65 (60), 16384 rows, 1024 to 4096
// 508 (505).  With two blocks per SM it reads them a microsecond faster, but scales at half the
// rate.  bf16 has fp32's range.
constexpr int kDzBlocks = 64 * kSms;
constexpr size_t kDzScaleBytes = 256 + (kDzBlocks * sizeof(float) + 255) / 256 * 256;   // the inverse, then the blocks' values

// dZ's vectors of eight columns, times `by`: 16 bytes of dH, G and U in, 16 bytes of dG and dU out.
// Returns (F16) the largest finite value this thread formed.
template <bool F16>
__device__ __forceinline__ float dz_vectors(const uint16_t* dH, const uint16_t* Z, uint16_t* dZ, long long nvec, int nv,
                                            int act, float by, long long bytes, int* status)
{
    constexpr int EK = F16 ? kF16 : kBF16;
    const long long stride = static_cast<long long>(gridDim.x) * 256;
    float top = 0.f;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < nvec; i += stride) {
        const long long m = i / nv;
        const long long g_at = m * 2 * nv + (i - m * nv);
        const uint4 h = reinterpret_cast<const uint4*>(dH)[i];
        const uint4 g = reinterpret_cast<const uint4*>(Z)[g_at];
        const uint4 u = reinterpret_cast<const uint4*>(Z)[g_at + nv];
        const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
        uint32_t a[4], b[4];
        with_act(act, [&](auto which) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                constexpr int A = decltype(which)::value;
                const float2 hf = h16x2_to_float2<EK>(hw[j]), gf = h16x2_to_float2<EK>(gw[j]);
                const float2 uf = h16x2_to_float2<EK>(uw[j]);
                float2 av, dv;
                gate_act_grad<A>(gf, av, dv);
                float2 dg = __fmul2_rn(__fmul2_rn(hf, uf), dv), du = __fmul2_rn(hf, av);
                if constexpr (F16) {
                    const float v[4] = {fabsf(dg.x), fabsf(dg.y), fabsf(du.x), fabsf(du.y)};
#pragma unroll
                    for (int q = 0; q < 4; ++q) top = fmaxf(top, v[q] < 1e30f ? v[q] : 0.f);   // not infinities, NaN
                    dg = __fmul2_rn(dg, splat(by));
                    du = __fmul2_rn(du, splat(by));
                }
                a[j] = float2_to_h16x2<EK>(dg.x, dg.y);
                b[j] = float2_to_h16x2<EK>(du.x, du.y);
            }
        });
        uint4* out = reinterpret_cast<uint4*>(dZ) + g_at;
        if (store_ok(dZ, bytes, out, 16, status)) out[0] = make_uint4(a[0], a[1], a[2], a[3]);
        if (store_ok(dZ, bytes, out + nv, 16, status)) out[nv] = make_uint4(b[0], b[1], b[2], b[3]);
    }
    return top;
}

// The largest of a block's 256 values, in every thread (once per kernel: nothing is read again).
__device__ __forceinline__ float block_max(float v)
{
    __shared__ float s[8];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) v = fmaxf(v, s[w]);
    return v;
}

// top: the blocks' largest values, kDzBlocks of them (F16).
template <bool F16>
__global__ void __launch_bounds__(256) gated_dz_kernel(const uint16_t* dH, const uint16_t* Z, uint16_t* dZ,
                                                       long long nvec, int nv, int act, float* top, long long bytes,
                                                       int* status)
{
    pdl_wait();      // the previous kernel on the stream has finished
    pdl_trigger();   // the next one may start its set-up
    float most = dz_vectors<F16>(dH, Z, dZ, nvec, nv, act, 1.0f, bytes, status);
    if constexpr (F16) {
        most = block_max(most);
        if (threadIdx.x == 0 && store_ok(top, kDzBlocks * 4LL, top + blockIdx.x, 4, status)) top[blockIdx.x] = most;
    }
}

// Writes the inverse of dZ's scale, and dZ again where that is not 1.
__global__ void __launch_bounds__(256) gated_dz_scale_kernel(const uint16_t* dH, const uint16_t* Z, uint16_t* dZ,
                                                             long long nvec, int nv, int act, const float* top, int blocks,
                                                             float* inverse, long long bytes, int* status)
{
    pdl_wait();
    pdl_trigger();
    float most = 0.f;
#pragma unroll 8
    for (int i = threadIdx.x; i < blocks; i += 256) most = fmaxf(most, top[i]);
    most = block_max(most);
    int k = 0;   // the scale is 2^k
    if (most > 65504.f || (most > 0.f && most < 0x1p-10f)) {
        k = 14 + 127 - static_cast<int>(__float_as_uint(most) >> 23);
        k = k < 100 ? k : 100;   // what 2^100 does not lift to f16's range gives zero in any product of f16 values
    }
    if (blockIdx.x == 0 && threadIdx.x == 0 && store_ok(inverse, 4, inverse, 4, status))
        *inverse = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
    if (k != 0) dz_vectors<true>(dH, Z, dZ, nvec, nv, act, __uint_as_float(static_cast<uint32_t>(127 + k) << 23), bytes, status);
}

// ------------------------------------------------------- few values of dZ

constexpr int64_t kFew = 4096;
bool few_kernels(int64_t M, int64_t F) { return M * F <= kFew; }

// dZ in fp32, eight columns per thread.
template <bool F16>
__global__ void __launch_bounds__(128) gated_dz_f32_kernel(const uint16_t* dH, const uint16_t* Z, float* dZ, int nvec,
                                                           int nv, int act, long long bytes, int* status)
{
    pdl_wait();
    pdl_trigger();
    constexpr int EK = F16 ? kF16 : kBF16;
    const int i = blockIdx.x * 128 + threadIdx.x;
    if (i >= nvec) return;
    const int m = i / nv;
    const long long g_at = static_cast<long long>(m) * 2 * nv + (i - m * nv);
    const uint4 h = reinterpret_cast<const uint4*>(dH)[i];
    const uint4 g = reinterpret_cast<const uint4*>(Z)[g_at];
    const uint4 u = reinterpret_cast<const uint4*>(Z)[g_at + nv];
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
    float2* out = reinterpret_cast<float2*>(dZ + g_at * 8);
    with_act(act, [&](auto which) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 hf = h16x2_to_float2<EK>(hw[j]), uf = h16x2_to_float2<EK>(uw[j]);
            float2 av, dv;
            gate_act_grad<decltype(which)::value>(h16x2_to_float2<EK>(gw[j]), av, dv);
            if (store_ok(dZ, bytes, out + j, 8, status)) out[j] = __fmul2_rn(__fmul2_rn(hf, uf), dv);
            if (store_ok(dZ, bytes, out + nv * 4 + j, 8, status)) out[nv * 4 + j] = __fmul2_rn(hf, av);
        }
    });
}

// Eight fp32 values rounded to 16 bytes.
template <int EK>
__device__ __forceinline__ uint4 round8(const float2 (&a)[4])
{
    return make_uint4(float2_to_h16x2<EK>(a[0].x, a[0].y), float2_to_h16x2<EK>(a[1].x, a[1].y),
                      float2_to_h16x2<EK>(a[2].x, a[2].y), float2_to_h16x2<EK>(a[3].x, a[3].y));
}

// out[r][c] = sum over k of A[r ra + k ka] B[k][c], fp32 A, 16-bit B and out: R rows and 8 CV
// columns per block, whose 256 / CV slices of CV lanes take the terms in turn; the slices' sums
// are added in a fixed order.  dX: A = dZ, B = W; dW: A = dZ^T, B = X.
template <int R, int CV, bool F16>
__global__ void __launch_bounds__(256) few_product_kernel(const float* A, long long ra, long long ka, const void* B,
                                                          void* out, int rows, int K, int C, int* status)
{
    pdl_wait();
    pdl_trigger();
    constexpr int EK = F16 ? kF16 : kBF16;
    __shared__ float2 part[8][R][CV][4];   // [warp][row][column vector]
    const int cv = threadIdx.x % CV, slice = threadIdx.x / CV;
    const int c = (blockIdx.x * CV + cv) * 8, r0 = blockIdx.y * R;
    float2 acc[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] = make_float2(0.f, 0.f);
    if (c < C) {
#pragma unroll 4
        for (int k = slice; k < K; k += 256 / CV) {
            const uint4 b = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(B) + static_cast<long long>(k) * C + c);
            const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 a = splat(r0 + r < rows ? A[(r0 + r) * ra + k * ka] : 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][i] = ffma2(a, h16x2_to_float2<EK>(bw[i]), acc[r][i]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = CV; o < 32; o <<= 1) {
                acc[r][i].x += __shfl_xor_sync(0xFFFFFFFFu, acc[r][i].x, o);
                acc[r][i].y += __shfl_xor_sync(0xFFFFFFFFu, acc[r][i].y, o);
            }
            if ((threadIdx.x & 31) < CV) part[threadIdx.x >> 5][r][cv][i] = acc[r][i];
        }
    __syncthreads();
    const int r = threadIdx.x / CV;   // now a thread per row and column vector
    if (r >= R || r0 + r >= rows || c >= C) return;
    float2 sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum[i] = part[0][r][cv][i];
#pragma unroll
        for (int w = 1; w < 8; ++w) sum[i] = __fadd2_rn(sum[i], part[w][r][cv][i]);
    }
    uint16_t* at = static_cast<uint16_t*>(out) + static_cast<long long>(r0 + r) * C + c;
    if (store_ok(out, 2LL * rows * C, at, 16, status)) *reinterpret_cast<uint4*>(at) = round8<EK>(sum);
}

// The same for a short K: eight columns of one row per thread, all of K.
template <bool F16>
__global__ void __launch_bounds__(256) few_outer_kernel(const float* A, long long ra, long long ka, const void* B,
                                                        void* out, int rows, int K, int C, int* status)
{
    pdl_wait();
    pdl_trigger();
    constexpr int EK = F16 ? kF16 : kBF16;
    const int nv = C >> 3;
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= static_cast<long long>(rows) * nv) return;
    const int r = static_cast<int>(i / nv), v = static_cast<int>(i - static_cast<long long>(r) * nv);
    float2 acc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        const uint4 b = static_cast<const uint4*>(B)[static_cast<long long>(k) * nv + v];
        const float2 a = splat(A[r * ra + k * ka]);
        const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = ffma2(a, h16x2_to_float2<EK>(bw[q]), acc[q]);
    }
    uint4* at = static_cast<uint4*>(out) + i;
    if (store_ok(out, 2LL * rows * C, at, 16, status)) *at = round8<EK>(acc);
}

template <int CV, bool F16>
cudaError_t few_slices(const float* A, long long ra, long long ka, const void* B, void* out, int rows, int K, int C,
                       int* status, cudaStream_t stream)
{
    const int R = rows == 1 ? 1 : rows == 2 ? 2 : rows <= 4 ? 4 : 8;
    auto kern = R == 1   ? few_product_kernel<1, CV, F16>
                : R == 2 ? few_product_kernel<2, CV, F16>
                : R == 4 ? few_product_kernel<4, CV, F16>
                         : few_product_kernel<8, CV, F16>;
    return launch_kernel(kern, dim3((C + 8 * CV - 1) / (8 * CV), (rows + R - 1) / R), dim3(256), 0, stream, 1, A, ra, ka, B,
                         out, rows, K, C, status);
}

// Up to 16 terms a thread takes them all; up to 256 in 16 slices, more in 128.  Many slices of a
// short sum idle, and their exchange costs more than the terms; one thread's long sum is all
// latency (64 rows, 2048 to 64 channels, backward: 13 us; 50 with 128 slices, 37 with one).
template <bool F16>
cudaError_t few_product(const float* A, long long ra, long long ka, const void* B, void* out, int rows, int K, int C,
                        int* status, cudaStream_t stream)
{
    if (K > 256) return few_slices<2, F16>(A, ra, ka, B, out, rows, K, C, status, stream);
    if (K > 16) return few_slices<16, F16>(A, ra, ka, B, out, rows, K, C, status, stream);
    const long long n = static_cast<long long>(rows) * (C / 8);
    return launch_kernel(few_outer_kernel<F16>, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream, 1, A, ra,
                         ka, B, out, rows, K, C, status);
}

template <bool F16>
cudaError_t run_few(const GatedBwdArgs& a, cudaStream_t stream)
{
    const int M = static_cast<int>(a.M), N2 = static_cast<int>(2 * a.F), C = static_cast<int>(a.C);
    float* dZ = static_cast<float*>(a.ws);
    const int nv = static_cast<int>(a.F / 8), nvec = M * nv;
    cudaError_t e = launch_kernel(gated_dz_f32_kernel<F16>, dim3((nvec + 127) / 128), dim3(128), 0, stream, 1,
                                  static_cast<const uint16_t*>(a.dH), static_cast<const uint16_t*>(a.Z), dZ, nvec, nv,
                                  a.act, 4LL * M * N2, a.status);
    if (e != cudaSuccess) return e;
    if (a.dX) {
        e = few_product<F16>(dZ, N2, 1, a.W, a.dX, M, N2, C, a.status, stream);
        if (e != cudaSuccess) return e;
    }
    return a.dW ? few_product<F16>(dZ, 1, N2, a.X, a.dW, N2, M, C, a.status, stream) : cudaSuccess;
}

// ------------------------------------------------------------------- dW

template <int BN>
struct WgLayout {
    static constexpr int kBHalf = (BN / 2) * kBK * 2;   // this CTA's X columns, one k-block
    static constexpr int kStage = 16384 + kBHalf;
    static constexpr int kEpi = kStages * kStage;       // 2 x 16 KB staging
    static constexpr int kBars = kEpi + 2 * 16384;
    static constexpr int kNumBars = 2 * kStages + 5;
    static constexpr int kBytes = kBars + kNumBars * 8 + 16;
    static constexpr int kAlloc = kBytes + 1024;
};

struct WgPlan {
    int bn, splits, kb_per;   // k-blocks of 64 rows per split
};

// One launch's units: (tile of 256 x BN, split).  map_a: dZ, map_b: X (both 2-D, box 64 x
// 64); map_d: dW (2-D, box 64 x 128) or, PART, the fp32 partials (3-D [split][2F][C],
// box 32 x 128 x 1), all swizzled.
template <int BN, bool PART, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    wgrad_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ CUtensorMap map_d, int M, int N2, int C, int splits, int kb_per,
                      const float* scale, int* status)
{
    pdl_wait();      // the previous kernel on the stream has finished
    pdl_trigger();   // the next one may start its set-up
    using L = WgLayout<BN>;
    constexpr int EK = F16 ? kF16 : kBF16;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* full = bars;                  // used in the rank-0 CTA
    uint64_t* empty = bars + kStages;       // each CTA's own
    uint64_t* tfull = bars + 2 * kStages;   // each CTA's own
    uint64_t* tempty = tfull + 2;           // used in the rank-0 CTA
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int rank = static_cast<int>(cluster_ctarank());
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int num_n = (C + BN - 1) / BN;
    const int num_kb = (M + kBK - 1) / kBK;
    const int units = ((N2 + 255) / 256) * num_n * splits;
    const int pair = blockIdx.x >> 1;
    const int num_pairs = gridDim.x >> 1;
    // unit -> row block of dW, column block, split; its k-blocks
    auto unit = [&](int t, int& r0, int& c0, int& sp, int& kb0, int& kb1) {
        sp = t % splits;
        const int tile = t / splits;
        r0 = (tile / num_n) * 256 + rank * 128;
        c0 = (tile % num_n) * BN;
        kb0 = sp * kb_per;
        kb1 = min(num_kb, kb0 + kb_per);
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 256);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
        tma_prefetch_desc(&map_d);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 2 * BN);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();                          // barriers of both CTAs exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0 = leader_addr(&full[0]);
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (int t = pair; t < units && ok; t += num_pairs) {
                int r0, c0, sp, kb0, kb1;
                unit(t, r0, c0, sp, kb0, kb1);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * L::kStage);
                    uint8_t* a_tile = smem + stage * L::kStage;
                    uint8_t* b_tile = a_tile + 16384;
                    const uint32_t fb = full0 + static_cast<uint32_t>(stage * 8);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        tma_load_2d_pair(a_tile + j * 8192, &map_a, fb, r0 + j * 64, kb * kBK);
#pragma unroll
                    for (int j = 0; j < BN / 128; ++j)
                        tma_load_2d_pair(b_tile + j * 8192, &map_b, fb, c0 + rank * (BN / 2) + j * 64, kb * kBK);
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                report_timeout(status);
                *abort_flag = 1;
            }
            // the last loads of this CTA land before it may exit: wait until the MMAs
            // that read them have released the stages (multicast commit)
            for (long long i = (issued > kStages ? issued - kStages : 0); i < issued; ++i)
                if (!mbar_wait(&empty[i % kStages], static_cast<uint32_t>((i / kStages) & 1))) {
                    report_timeout(status);
                    *abort_flag = 1;
                }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc =
                (F16 ? idesc_f16_f32(256, BN, /*b_mn_major=*/true) : idesc_bf16_f32(256, BN, true)) | kIdescAMnMajor;
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int t = pair; t < units && ok; t += num_pairs) {
                int r0, c0, sp, kb0, kb1;
                unit(t, r0, c0, sp, kb0, kb1);
                if (!mbar_wait_cluster(&tempty[acc], acc_phase ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&full[stage], phase, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(smem + stage * L::kStage);
                    const uint32_t b_addr = a_addr + 16384;
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)   // 16 rows: two groups of 8 rows of 128 bytes
                        umma_f16_pair(d_tmem, sw128_desc(a_addr + kk * 2048, 8192, 1024),
                                      sw128_desc(b_addr + kk * 2048, 8192, 1024), idesc,
                                      (kb > kb0 || kk > 0) ? 1u : 0u);
                    umma_commit_pair(&empty[stage]);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                umma_commit_pair(&tfull[acc]);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (!ok) {
                report_timeout(status);
                *abort_flag = 1;
            }
            umma_commit_pair(drain);
            if (!mbar_wait(drain, 0)) {
                report_timeout(status);
                *abort_flag = 1;
            }
        }
    } else {
        constexpr int kCols = PART ? 32 : 64;     // columns of one 16 KB staging box
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        const bool issuer = warp == 2 && lane == 0;
        const uint32_t tempty0 = leader_addr(&tempty[0]);
        const float by = F16 && !PART ? *scale : 1.0f;   // (partials are multiplied when they are added)
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int t = pair; t < units; t += num_pairs) {
            int r0, c0, sp, kb0, kb1;
            unit(t, r0, c0, sp, kb0, kb1);
            ok = named_barrier_and(1, 128, mbar_wait_cluster(&tfull[acc], acc_phase, abort_flag));
            if (!ok) break;                       // the epilogue warps leave together
            tc_fence_after();
#pragma unroll 1
            for (int chunk = 0; chunk < BN / kCols; ++chunk) {
                const int c = c0 + chunk * kCols;
                uint8_t* buf = smem + L::kEpi + (chunk & 1) * 16384;
                uint8_t* rowp = buf + row * 128;
                if (issuer) bulk_wait_group_read<1>();
                named_barrier_sync(1, 128);
                uint32_t v[kCols];
#pragma unroll
                for (int q = 0; q < kCols / 32; ++q)
                    tmem_ld_32x32b_x32(tmem_base + lane_addr + static_cast<uint32_t>(acc * BN + chunk * kCols + q * 32),
                                       *reinterpret_cast<uint32_t(*)[32]>(&v[q * 32]));
                tmem_wait_ld();
                if constexpr (F16 && !PART) {
#pragma unroll
                    for (int j = 0; j < kCols; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * by);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint4 o;
                    if constexpr (PART) {
                        o = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    } else {
                        o.x = float2_to_h16x2<EK>(__uint_as_float(v[8 * j + 0]), __uint_as_float(v[8 * j + 1]));
                        o.y = float2_to_h16x2<EK>(__uint_as_float(v[8 * j + 2]), __uint_as_float(v[8 * j + 3]));
                        o.z = float2_to_h16x2<EK>(__uint_as_float(v[8 * j + 4]), __uint_as_float(v[8 * j + 5]));
                        o.w = float2_to_h16x2<EK>(__uint_as_float(v[8 * j + 6]), __uint_as_float(v[8 * j + 7]));
                    }
                    *reinterpret_cast<uint4*>(rowp + ((j ^ (row & 7)) << 4)) = o;
                }
                fence_proxy_async_smem();
                named_barrier_sync(1, 128);
                if (issuer) {
                    if (c < C && r0 < N2) {       // the map clips the tails
                        if constexpr (PART)
                            tma_store_3d(&map_d, buf, c, r0, sp);
                        else
                            tma_store_2d(&map_d, buf, c, r0);
                    }
                    bulk_commit_group();
                }
            }
            tc_fence_before();
            mbar_arrive_cluster(tempty0 + static_cast<uint32_t>(acc * 8));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (!ok) {
            report_timeout(status);
            *abort_flag = 1;
        }
        if (issuer) bulk_wait_group<0>();
    }

    tc_fence_before();
    cluster_sync();                              // no CTA leaves while its pair still needs it
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem_base, 2 * BN);
    }
}

// Tile width (half of a 256-column tile would be empty up to 128 channels) and row splits of
// dW: as many as fill the pairs (25088 rows, 256 to 512 channels: the backward pass takes 60 us
// with 18 splits, 150 with one).
WgPlan wgrad_plan(int64_t M, int64_t N2, int64_t C)
{
    WgPlan p;
    p.bn = C > 128 ? 256 : 128;
    const int64_t tiles = ((N2 + 255) / 256) * ((C + p.bn - 1) / p.bn);
    const int64_t num_kb = (M + kBK - 1) / kBK;
    int64_t s = (kSms / 2) / tiles;
    if (s > num_kb / 4) s = num_kb / 4;   // a split too short is all start-up and epilogue
    if (s < 1) s = 1;
    p.kb_per = static_cast<int>((num_kb + s - 1) / s);
    p.splits = static_cast<int>((num_kb + p.kb_per - 1) / p.kb_per);   // no empty split
    return p;
}

// Splits of dX's sums over K = 2F (1: the SM-pair kernel with tiles of 256 rows).  Few rows
// leave most pairs idle through a long K; the split-K kernel's 128 x 128 tiles then fill the
// SMs.  The count is that of least estimated time, in tensor cycles: a k-block costs a tile
// 512 (256 x 256 on a pair), 256 (256 x 128) or, 128 x 128 on one SM, 520 (its 32 KB come at
// about 64 bytes a cycle); splits add their fp32 partials' traffic (24 bytes a cycle and SM)
// and a launch (4000).  The whole
// backward pass of 1024 rows, 768 to 2048 channels, took 37 us with the pair kernel and 30
// with 3 splits; of 2048 to 5600 channels 101 with the pair kernel and 107 with 2 or 8.
int dx_splits(int64_t M, int64_t K, int64_t C)
{
    const int64_t num_kb = (K + kBK - 1) / kBK;
    const int64_t bn = C > 128 ? 256 : 128;
    const int64_t pair_tiles = ((M + 255) / 256) * ((C + bn - 1) / bn);
    const int64_t pairs = kSms / 2;
    int64_t best = (pair_tiles + pairs - 1) / pairs * num_kb * (2 * bn);
    int count = 1;
    const int64_t tiles = ((M + 127) / 128) * ((C + 127) / 128);
    for (int64_t s = 2; s <= 32 && s <= num_kb / 2; ++s) {
        const int64_t t = (tiles * s + kSms - 1) / kSms * ((num_kb + s - 1) / s) * 520 +
                          s * M * C * 8 / (24 * kSms) + 4000;
        if (t < best) {
            best = t;
            count = static_cast<int>(s);
        }
    }
    return count;
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

template <int BN, bool PART, bool F16>
cudaError_t run_wgrad(const GatedBwdArgs& a, const void* dZ, void* dst, const WgPlan& p, const float* scale,
                      cudaStream_t stream)
{
    using L = WgLayout<BN>;
    static_assert(L::kAlloc <= 232448, "shared memory budget");
    const CUtensorMapDataType t = F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t M = static_cast<uint64_t>(a.M), C = static_cast<uint64_t>(a.C), N2 = 2 * static_cast<uint64_t>(a.F);
    const uint64_t da[2] = {N2, M}, sa[1] = {2 * N2}, db[2] = {C, M}, sb[1] = {2 * C};
    const uint32_t box[2] = {64, 64}, bd[2] = {64, 128}, bp[3] = {32, 128, 1};
    const uint64_t dd[2] = {C, N2}, sd[1] = {2 * C};
    const uint64_t dp[3] = {C, N2, static_cast<uint64_t>(p.splits)}, sp[2] = {4 * C, 4 * C * N2};
    CUtensorMap ma, mb, md;
    if (!encode_map(&ma, t, 2, dZ, da, sa, box, true) || !encode_map(&mb, t, 2, a.X, db, sb, box, true))
        return cudaErrorInvalidValue;
    if (!(PART ? encode_map(&md, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, dst, dp, sp, bp, true)
               : encode_map(&md, t, 2, dst, dd, sd, bd, true)))
        return cudaErrorInvalidValue;
    auto kern = wgrad_pair_kernel<BN, PART, F16>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), L::kAlloc);
    if (e != cudaSuccess) return e;
    const int64_t units = static_cast<int64_t>((N2 + 255) / 256 * ((C + BN - 1) / BN)) * p.splits;
    const int64_t most = device_sm_count() / 2;
    const unsigned pairs = static_cast<unsigned>(units < most ? units : most);
    return launch_kernel(kern, dim3(2 * pairs), dim3(kThreads), L::kAlloc, stream, 2, ma, mb, md,
                         static_cast<int>(a.M), static_cast<int>(N2), static_cast<int>(a.C), p.splits, p.kb_per, scale,
                         a.status);
}

template <bool F16>
cudaError_t run(const GatedBwdArgs& a, cudaStream_t stream)
{
    const int64_t N2 = 2 * a.F;
    uint16_t* dZ = static_cast<uint16_t*>(a.ws);
    const size_t dz_bytes = static_cast<size_t>(a.M) * N2 * 2;
    char* rest = static_cast<char*>(a.ws) + align256(dz_bytes);
    float* inverse = F16 ? reinterpret_cast<float*>(rest) : nullptr;
    float* top = reinterpret_cast<float*>(rest + 256);
    // dX's and dW's partials share the rest: dX's are read before dW's kernel begins to write
    float* part = reinterpret_cast<float*>(rest + kDzScaleBytes);
    const long long nvec = a.M * (a.F / 8);
    const long long need = (nvec + 255) / 256;
    const int blocks = static_cast<int>(need < kDzBlocks ? need : kDzBlocks), nv = static_cast<int>(a.F / 8);
    const uint16_t* dH = static_cast<const uint16_t*>(a.dH);
    const uint16_t* Z = static_cast<const uint16_t*>(a.Z);
    cudaError_t e = launch_kernel(gated_dz_kernel<F16>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, 1, dH, Z,
                                  dZ, nvec, nv, a.act, top, static_cast<long long>(dz_bytes), a.status);
    if (e != cudaSuccess) return e;
    if (F16) {
        const int few = blocks < 5 * kSms ? blocks : 5 * kSms;   // as many as are resident
        e = launch_kernel(gated_dz_scale_kernel, dim3(static_cast<unsigned>(few)), dim3(256), 0, stream, 1, dH, Z, dZ, nvec, nv,
                          a.act, top, blocks, inverse, static_cast<long long>(dz_bytes), a.status);
        if (e != cudaSuccess) return e;
    }
    if (a.dX) {
        const CUtensorMapDataType t = F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        const PwArgs g{a.M, N2, a.C, dZ, a.W, a.dX, a.status, F16, inverse};
        const uint64_t M = static_cast<uint64_t>(a.M), C = static_cast<uint64_t>(a.C), K = static_cast<uint64_t>(N2);
        const uint64_t da[2] = {K, M}, sa[1] = {2 * K}, db[2] = {C, K}, sb[1] = {2 * C}, dd[2] = {C, M};
        const uint32_t tall[2] = {64, 128}, sq[2] = {64, 64};
        CUtensorMap ma, mb, md;
        if (!encode_map(&ma, t, 2, dZ, da, sa, tall, true) || !encode_map(&mb, t, 2, a.W, db, sb, sq, true) ||
            !encode_map(&md, t, 2, a.dX, dd, sb, tall, true))
            return cudaErrorInvalidValue;
        const int splits = dx_splits(a.M, N2, a.C);
        e = splits > 1 ? launch_pointwise_tc_splitk(g, ma, mb, splits, part, device_sm_count(), stream)
                       : launch_pointwise_tc_pair(g, ma, mb, md, a.C > 128 ? 256 : 128, device_sm_count(), stream);
        if (e != cudaSuccess) return e;
    }
    if (!a.dW) return cudaSuccess;
    const WgPlan p = wgrad_plan(a.M, N2, a.C);
    if (p.splits == 1)
        return p.bn == 256 ? run_wgrad<256, false, F16>(a, dZ, a.dW, p, inverse, stream)
                           : run_wgrad<128, false, F16>(a, dZ, a.dW, p, inverse, stream);
    e = p.bn == 256 ? run_wgrad<256, true, F16>(a, dZ, part, p, inverse, stream)
                    : run_wgrad<128, true, F16>(a, dZ, part, p, inverse, stream);
    if (e != cudaSuccess) return e;
    return launch_splitk_reduce(part, a.dW, N2 * a.C, p.splits, F16, inverse, a.status, stream);
}

}  // namespace

size_t gated_backward_workspace_bytes(int64_t M, int64_t C, int64_t F)
{
    const int64_t N2 = 2 * F;
    if (few_kernels(M, F)) return static_cast<size_t>(M) * N2 * 4;
    const WgPlan p = wgrad_plan(M, N2, C);
    const int s = dx_splits(M, N2, C);
    const size_t dw = p.splits > 1 ? static_cast<size_t>(p.splits) * N2 * C * 4 : 0;
    const size_t dx = s > 1 ? static_cast<size_t>(s) * M * C * 4 : 0;
    return align256(static_cast<size_t>(M) * N2 * 2) + kDzScaleBytes + (dw > dx ? dw : dx);
}

cudaError_t launch_gated_backward(const GatedBwdArgs& a, cudaStream_t stream)
{
    if (few_kernels(a.M, a.F)) return a.f16 ? run_few<true>(a, stream) : run_few<false>(a, stream);
    return a.f16 ? run<true>(a, stream) : run<false>(a, stream);
}

}  // namespace dgrad
