// dropout.cu -- dropout from a counter-based generator, with no stored mask.
//
// Elements come in blocks of eight.  Block b takes the 128 bits of Philox-4x32-10
// (J. Salmon, M. Moraes, R. Dror and D. Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", 2011) at counter (b, offset) and key seed: element i draws 16 bits, word
// (i % 8) / 2, the low half for even i.  It is kept where the draw is >= t and then
// scaled by 65536 / (65536 - t), with t = round(65536 p); the backward pass draws the
// same bits again.  A dropped element is not multiplied: an infinity or NaN in its
// place leaves no trace.
//
// One read and one write (and a read of the residual) bound it: HBM.  Sixteen bits
// per element rather than 32 because the generator would bound it otherwise: 128 Mi
// bf16 elements ran at 5.95 TB/s with 16-bit draws, 4.16 TB/s with 32-bit draws and
// 6.24 TB/s with no generator at all.  p is then held to 2^-17; the scale goes by
// the rounded value, so the mean is kept exactly.
#include "common.cuh"
#include "host_util.h"
#include "launchers.h"
#include "rowvec.cuh"

namespace dgrad {
namespace {

constexpr int kDropBlock = 256;

struct Drop {
    const void* x;
    const void* r;       // null: no residual
    void* y;
    long long n;
    uint32_t seed_lo, seed_hi, off_lo, off_hi;
    uint32_t thr;
    float scale;
    int* status;
};

// The eight 16-bit draws of block b, two per word.
__device__ __forceinline__ uint4 philox_block(const Drop& p, long long b)
{
    uint32_t c0 = static_cast<uint32_t>(b), c1 = static_cast<uint32_t>(b >> 32), c2 = p.off_lo, c3 = p.off_hi;
    uint32_t k0 = p.seed_lo, k1 = p.seed_hi;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
        const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
        c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(p1);
        c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Without a residual a kept zero keeps its sign, so that p = 0 changes nothing.
template <bool RES>
__device__ __forceinline__ float drop_one(float x, float r, uint32_t draw, const Drop& p)
{
    return draw >= p.thr ? (RES ? fmaf(x, p.scale, r) : x * p.scale) : r;
}

template <int EK, bool RES>
__global__ void __launch_bounds__(kDropBlock) dropout_kernel(const Drop p)
{
    pdl_wait();      // the previous kernel on the stream has finished
    pdl_trigger();   // the next one may start its set-up
    constexpr int VEC = 16 / elem_bytes<EK>();   // elements per 16-byte vector
    constexpr int NV = 8 / VEC;                  // vectors per block of eight
    using V = RowVec<EK, VEC>;
    constexpr int es = elem_bytes<EK>();
    const long long full = p.n >> 3;
    const long long stride = static_cast<long long>(gridDim.x) * kDropBlock;
    const long long first = static_cast<long long>(blockIdx.x) * kDropBlock + threadIdx.x;
    for (long long b = first; b < full; b += stride) {
        V x[NV], r[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            x[v].load(p.x, b * 8 + v * VEC);
            if constexpr (RES) r[v].load(p.r, b * 8 + v * VEC);
        }
        const uint4 d = philox_block(p, b);
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float f[VEC], rf[VEC];
            x[v].unpack(f);
            if constexpr (RES) r[v].unpack(rf);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int e = v * VEC + i;
                const uint32_t draw = (e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu;
                f[i] = drop_one<RES>(f[i], RES ? rf[i] : 0.f, draw, p);
            }
            V o;
            o.pack(f);
            if (store_ok(p.y, p.n * es, static_cast<char*>(p.y) + (b * 8 + v * VEC) * es, 16, p.status))
                o.store(p.y, b * 8 + v * VEC);
        }
    }
    // the elements behind the last whole block, by one thread
    if (first == 0 && (p.n & 7)) {
        const uint4 d = philox_block(p, full);
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
        for (int e = 0; e < static_cast<int>(p.n & 7); ++e) {
            const long long i = full * 8 + e;
            RowVec<EK, 1> x;
            float f[1], rf[1] = {0.f};
            x.load(p.x, i);
            x.unpack(f);
            if constexpr (RES) {
                RowVec<EK, 1> r;
                r.load(p.r, i);
                r.unpack(rf);
            }
            const uint32_t draw = (e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu;
            f[0] = drop_one<RES>(f[0], rf[0], draw, p);
            x.pack(f);
            if (store_ok(p.y, p.n * es, static_cast<char*>(p.y) + i * es, es, p.status)) x.store(p.y, i);
        }
    }
}

}  // namespace

cudaError_t launch_dropout(const DropArgs& a, cudaStream_t stream)
{
    Drop p{a.X, a.residual, a.Y, a.n, static_cast<uint32_t>(a.seed), static_cast<uint32_t>(a.seed >> 32),
           static_cast<uint32_t>(a.offset), static_cast<uint32_t>(a.offset >> 32), a.threshold,
           a.threshold < 65536 ? static_cast<float>(65536.0 / (65536 - a.threshold)) : 0.f, a.status};
    const long long blocks = ((a.n >> 3) + kDropBlock - 1) / kDropBlock;
    const long long most = 64LL * device_sm_count();
    const unsigned grid = static_cast<unsigned>(blocks < 1 ? 1 : blocks < most ? blocks : most);
    auto kern = a.ek == kF32 ? (a.residual ? dropout_kernel<kF32, true> : dropout_kernel<kF32, false>)
                : a.ek == kBF16 ? (a.residual ? dropout_kernel<kBF16, true> : dropout_kernel<kBF16, false>)
                                : (a.residual ? dropout_kernel<kF16, true> : dropout_kernel<kF16, false>);
    return launch_kernel(kern, dim3(grid), dim3(kDropBlock), 0, stream, 1, p);
}

}  // namespace dgrad
