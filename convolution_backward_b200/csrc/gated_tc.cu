// gated_tc.cu -- the gated pointwise block, H = act(X Wg^T) * (X Wu^T), in one kernel.
//
// X [M][C], W [2F][C] (the gate's rows, then the other projection's): each output
// element needs two dot products of C terms, 4 M F C operations against
// 2 (M C + 2 F C + M F) bytes, so the tensor cores bound it from a few hundred rows
// on and W's bytes below that.
//
// gated_pair_kernel (persistent, pairs of SMs, tcgen05 cta_group::2).  A tile is 256
// rows of X and HN columns of H; the MMA's N = 2 HN columns are HN gate columns and
// the same HN columns of the other projection.  For the pair each CTA stages half of
// the MMA's B operand, so the rank-0 CTA loads the gate's rows of W and the rank-1 CTA
// the others: one accumulator row then holds g in columns [0, HN) and u in [HN, 2 HN),
// and the epilogue's thread has both of its elements in its own TMEM lane.
//   warp 0      TMA producer (X 128 rows x 64, W HN rows x 64 per k-block, both K-major)
//   warp 1      TMEM allocation; the rank-0 CTA's lane 0 issues the pair MMAs
//   warps 2..   eight epilogue warps for every 64 columns of H: TMEM loads 16 columns
//               ahead, the activation in fp32, one rounding, a swizzled staging tile, one
//               TMA store (H, and Z's two halves when the pre-activations are kept).
// Two accumulators let a tile's epilogue run under the next tile's MMAs.
//
// gated_row_kernel (one row) and gated_rows_kernel (up to 32) serve single tokens: W's
// bytes bound them, so W is read once, by plain 16-byte loads straight to registers.
#include "common.cuh"
#include "gate_act.cuh"
#include "host_util.h"
#include "launchers.h"

namespace dgrad {
namespace {

constexpr int kBK = 64;

// Sixteen epilogue warps (HN = 128) rather than eight: at 256 channels, where the epilogue
// bounds the tile, 32768 rows to 2048 took 80 us against 85.  ZK: Z is kept.
template <int HN, bool ZK>
struct GatedLayout {
    static constexpr int kBoxes = HN / 64;   // staging boxes of 64 columns, two warp groups each
    static constexpr int kThreads = 64 + 256 * kBoxes;
    static constexpr int kBBytes = HN * kBK * 2;
    static constexpr int kStage = 16384 + kBBytes;
    static constexpr int kStgPerBox = (ZK ? 3 : 2) * 16384;
    static constexpr int kStages = HN == 128 ? (ZK ? 4 : 5) : (ZK ? 7 : 8);
    static constexpr int kEpi = kStages * kStage;
    static constexpr int kBars = kEpi + kBoxes * kStgPerBox;
    static constexpr int kNumBars = 2 * kStages + 5;
    static constexpr int kBytes = kBars + kNumBars * 8 + 16;
    static constexpr int kAlloc = kBytes + 1024;   // slack to align the tiles to 1024 bytes
    static constexpr uint32_t kCols = 2 * 2 * HN;  // two accumulators
};

template <int HN, bool ZK, bool F16>
__global__ void __launch_bounds__(GatedLayout<HN, ZK>::kThreads, 1)
    gated_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ CUtensorMap map_h, const __grid_constant__ CUtensorMap map_z, int M,
                      int C, int F, int act, int* status)
{
    pdl_wait();      // the previous kernel on the stream has finished
    pdl_trigger();   // the next one may start its set-up
    using L = GatedLayout<HN, ZK>;
    constexpr int EK = F16 ? kF16 : kBF16;
    constexpr int S = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* full = bars;              // used in the rank-0 CTA
    uint64_t* empty = bars + S;         // each CTA's own
    uint64_t* tfull = bars + 2 * S;     // each CTA's own
    uint64_t* tempty = tfull + 2;       // used in the rank-0 CTA
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int rank = static_cast<int>(cluster_ctarank());
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int num_n = (F + HN - 1) / HN;
    const int num_tiles = ((M + 255) / 256) * num_n;
    const int num_kb = (C + kBK - 1) / kBK;
    const int pair = blockIdx.x >> 1;
    const int num_pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 2 * 256 * L::kBoxes);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_h);
        if (ZK) tma_prefetch_desc(&map_z);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, L::kCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();                      // barriers of both CTAs exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0 = leader_addr(&full[0]);
            const uint64_t keep = policy_evict_last();   // both operands are read again by other tiles
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (int t = pair; t < num_tiles && ok; t += num_pairs) {
                const int m0 = (t / num_n) * 256 + rank * 128;
                const int w0 = (t % num_n) * HN + rank * F;   // the gate's rows, or the other projection's
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * L::kStage);
                    uint8_t* a_tile = smem + stage * L::kStage;
                    const uint32_t fb = full0 + static_cast<uint32_t>(stage * 8);
                    tma_load_2d_pair_hint(a_tile, &map_x, fb, kb * kBK, m0, keep);
                    tma_load_2d_pair_hint(a_tile + 16384, &map_w, fb, kb * kBK, w0, keep);
                    ++issued;
                    if (++stage == S) {
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
            for (long long i = (issued > S ? issued - S : 0); i < issued; ++i)
                if (!mbar_wait(&empty[i % S], static_cast<uint32_t>((i / S) & 1))) {
                    report_timeout(status);
                    *abort_flag = 1;
                }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc =
                F16 ? idesc_f16_f32(256, 2 * HN, /*b_mn_major=*/false) : idesc_bf16_f32(256, 2 * HN, false);
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int t = pair; t < num_tiles && ok; t += num_pairs) {
                if (!mbar_wait_cluster(&tempty[acc], acc_phase ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 2 * HN);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(&full[stage], phase, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(smem + stage * L::kStage);
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)   // 16 k: 32 bytes inside the swizzled rows
                        umma_f16_pair(d_tmem, sw128_desc(a_addr + kk * 32, 16, 1024),
                                      sw128_desc(a_addr + 16384 + kk * 32, 16, 1024), idesc, (kb | kk) != 0 ? 1u : 0u);
                    umma_commit_pair(&empty[stage]);
                    if (++stage == S) {
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
        const int box = (warp - 2) >> 3;
        const int half = ((warp - 2) >> 2) & 1;   // columns [32 half, 32 half + 32) of the box
        const int quarter = warp & 3;             // TMEM lanes this warp may read
        const int row = quarter * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        const bool issuer = ((warp - 2) & 7) == 0 && lane == 0;
        const uint32_t tempty0 = leader_addr(&tempty[0]);
        const uint64_t once = policy_evict_first();                // Z is next read in the backward pass
        uint8_t* const base = smem + L::kEpi + box * L::kStgPerBox;
        uint8_t* stg = base;   // H, and with ZK Z's gate and other half behind it
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int t = pair; t < num_tiles; t += num_pairs) {
            const int m0 = (t / num_n) * 256 + rank * 128;
            const int n0 = (t % num_n) * HN + box * 64;
            ok = mbar_wait_cluster(&tfull[acc], acc_phase, abort_flag);
            // the stores that read this staging have read it: the previous tile's, or without Z (two
            // boxes in turn) the one before
            if (issuer) bulk_wait_group_read<ZK ? 0 : 1>();
            ok = named_barrier_and(1 + box, 256, ok);   // the box's warps leave together or not at all
            if (!ok) break;
            tc_fence_after();
            // 16 columns at a time, the next ones on their way from tensor memory meanwhile
            const uint32_t col = tmem_base + lane_addr + static_cast<uint32_t>(acc * 2 * HN + box * 64 + half * 32);
            uint32_t g[2][16], u[2][16];
            tmem_ld_32x32b_x16(col, g[0]);
            tmem_ld_32x32b_x16(col + HN, u[0]);
            with_act(act, [&](auto which) {
                constexpr int A = decltype(which)::value;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    tmem_wait_ld();
                    if (q == 0) {
                        tmem_ld_32x32b_x16(col + 16, g[1]);
                        tmem_ld_32x32b_x16(col + 16 + HN, u[1]);
                    } else {                 // the accumulator is in registers: free it
                        tc_fence_before();
                        mbar_arrive_cluster(tempty0 + static_cast<uint32_t>(acc * 8));
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int at = row * 128 + (((half * 4 + q * 2 + j) ^ (row & 7)) << 4);
                        uint32_t h[4], gz[4], uz[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = 8 * j + 2 * i;
                            const float2 gf = make_float2(__uint_as_float(g[q][e]), __uint_as_float(g[q][e + 1]));
                            const float2 uf = make_float2(__uint_as_float(u[q][e]), __uint_as_float(u[q][e + 1]));
                            const float2 hf = __fmul2_rn(gate_act<A>(gf), uf);
                            h[i] = float2_to_h16x2<EK>(hf.x, hf.y);
                            gz[i] = float2_to_h16x2<EK>(gf.x, gf.y);
                            uz[i] = float2_to_h16x2<EK>(uf.x, uf.y);
                        }
                        *reinterpret_cast<uint4*>(stg + at) = make_uint4(h[0], h[1], h[2], h[3]);
                        if constexpr (ZK) {
                            *reinterpret_cast<uint4*>(stg + 16384 + at) = make_uint4(gz[0], gz[1], gz[2], gz[3]);
                            *reinterpret_cast<uint4*>(stg + 32768 + at) = make_uint4(uz[0], uz[1], uz[2], uz[3]);
                        }
                    }
                }
            });
            fence_proxy_async_smem();
            named_barrier_sync(1 + box, 256);
            if (issuer && n0 < F && m0 < M) {        // the maps clip the tails
                tma_store_2d(&map_h, stg, n0, m0);
                if constexpr (ZK) {
                    tma_store_3d_hint(&map_z, stg + 16384, n0, 0, m0, once);
                    tma_store_3d_hint(&map_z, stg + 32768, n0, 1, m0, once);
                }
            }
            if (issuer) bulk_commit_group();
            if constexpr (!ZK) stg = base + (acc ^ 1) * 16384;
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
    cluster_sync();                      // no CTA leaves while its pair still needs it
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem_base, L::kCols);
    }
}

// H and (when Z is not null) Z of one element from its two sums.
template <bool F16>
__device__ __forceinline__ void gated_out(float g, float u, long long m, int f, uint16_t* H, uint16_t* Z, int M, int F,
                                          int act, int* status)
{
    constexpr int EK = F16 ? kF16 : kBF16;
    with_act(act, [&](auto which) {
        const float h = gate_act<decltype(which)::value>(splat(g)).x * u;
        uint16_t* at = H + m * F + f;
        if (store_ok(H, 2LL * M * F, at, 2, status)) *at = static_cast<uint16_t>(float2_to_h16x2<EK>(h, 0.f));
    });
    if (Z) {
        uint16_t* z = Z + 2 * m * F + f;
        if (store_ok(Z, 4LL * M * F, z, 2, status)) z[0] = static_cast<uint16_t>(float2_to_h16x2<EK>(g, 0.f));
        if (store_ok(Z, 4LL * M * F, z + F, 2, status)) z[F] = static_cast<uint16_t>(float2_to_h16x2<EK>(u, 0.f));
    }
}

// One row: a warp owns column f of H and reads rows f and F + f of W.
template <bool F16>
__global__ void __launch_bounds__(256) gated_row_kernel(const void* X, const void* W, uint16_t* H, uint16_t* Z, int C,
                                                        int F, int act, int* status)
{
    constexpr int EK = F16 ? kF16 : kBF16;
    const int lane = threadIdx.x & 31;
    const int f = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int nv = C >> 3;
    const uint4* wg = static_cast<const uint4*>(W) + static_cast<long long>(f) * nv;
    const uint4* wu = wg + static_cast<long long>(F) * nv;
    pdl_wait();      // the previous kernel on the stream has finished
    pdl_trigger();   // the next one may start its set-up
    if (f >= F) return;
    float2 g = make_float2(0.f, 0.f), u = g;
#pragma unroll 4
    for (int v = lane; v < nv; v += 32) {
        const uint4 a = wg[v], b = wu[v], x = static_cast<const uint4*>(X)[v];
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w}, xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 xf = h16x2_to_float2<EK>(xw[i]);
            g = ffma2(xf, h16x2_to_float2<EK>(aw[i]), g);
            u = ffma2(xf, h16x2_to_float2<EK>(bw[i]), u);
        }
    }
    float gs = g.x + g.y, us = u.x + u.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        gs += __shfl_xor_sync(0xFFFFFFFFu, gs, o);
        us += __shfl_xor_sync(0xFFFFFFFFu, us, o);
    }
    if (lane == 0) gated_out<F16>(gs, us, 0, f, H, Z, 1, F, act, status);
}

template <bool F16>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1)
{
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Up to 8 NT rows: a block owns 16 columns of H, its eight warps split C.  W's 16 gate rows
// and 16 other rows are the left operand of small tensor-core products whose right operand
// is X: the products' order along C is free, so lane (g, t) takes eight consecutive elements
// of W's rows g and g + 8 and of X's row g, 16 bytes each, and feeds four of them at a time
// to two MMAs.  The warps' sums meet in shared memory in a fixed order.  Multiply-adds on
// CUDA cores took 10.5 us at 8 rows, 768 to 2048 channels; this takes 3.3.
template <int NT, bool F16>
__global__ void __launch_bounds__(256) gated_rows_kernel(const void* X, const void* W, uint16_t* H, uint16_t* Z, int M,
                                                         int C, int F, int act, int* status)
{
    __shared__ float part[8][2][NT * 8][17];   // [warp][gate, other][row of X][column]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int f0 = blockIdx.x * 16;
    const int nv = C >> 3;                     // 16-byte vectors of a row
    const uint4* Wv = static_cast<const uint4*>(W);
    const uint4* Xv = static_cast<const uint4*>(X);
    pdl_wait();
    pdl_trigger();
    float d[2][NT][4] = {};
    const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll 2
    for (int v0 = warp * 4; v0 < nv; v0 += 32) {
        const int v = v0 + t;
        const bool in = v < nv;
        uint4 a[2][2], x[NT];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int f = f0 + g + 8 * r;
                a[p][r] = in && f < F ? Wv[static_cast<long long>(p * F + f) * nv + v] : none;
            }
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n] = in && n * 8 + g < M ? Xv[static_cast<long long>(n * 8 + g) * nv + v] : none;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_16x8x16<F16>(d[p][n], a[p][0].x, a[p][1].x, a[p][0].y, a[p][1].y, x[n].x, x[n].y);
                mma_16x8x16<F16>(d[p][n], a[p][0].z, a[p][1].z, a[p][0].w, a[p][1].w, x[n].z, x[n].w);
            }
    }
    // the product's element (column g or g + 8 of H, row 2t or 2t + 1 of X)
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[warp][p][n * 8 + 2 * t + (e & 1)][g + 8 * (e >> 1)] = d[p][n][e];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 8 * 16; i += 256) {
        const int r = i >> 4, c = i & 15;
        if (r >= M || f0 + c >= F) continue;
        float gs = 0.f, us = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            gs += part[w][0][r][c];
            us += part[w][1][r][c];
        }
        gated_out<F16>(gs, us, r, f0 + c, H, Z, M, F, act, status);
    }
}

template <int HN, bool ZK, bool F16>
cudaError_t run_pair(const GatedArgs& a, cudaStream_t stream)
{
    using L = GatedLayout<HN, ZK>;
    static_assert(L::kAlloc <= 232448, "shared memory budget");
    const CUtensorMapDataType t = F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t M = static_cast<uint64_t>(a.M), C = static_cast<uint64_t>(a.C), F = static_cast<uint64_t>(a.F);
    CUtensorMap mx, mw, mh, mz;
    const uint64_t dz[3] = {F, 2, M}, sz[2] = {2 * F, 4 * F};
    const uint64_t dx[2] = {C, M}, sx[1] = {2 * C}, dw[2] = {C, 2 * F}, dh[2] = {F, M}, sh[1] = {2 * F};
    const uint32_t bx[2] = {64, 128}, bw[2] = {64, HN}, bz[3] = {64, 1, 128};
    if (!encode_map(&mx, t, 2, a.X, dx, sx, bx, true) || !encode_map(&mw, t, 2, a.W, dw, sx, bw, true) ||
        !encode_map(&mh, t, 2, a.H, dh, sh, bx, true))
        return cudaErrorInvalidValue;
    if (!ZK)
        mz = mh;   // not used
    else if (!encode_map(&mz, t, 3, a.Z, dz, sz, bz, true))
        return cudaErrorInvalidValue;
    auto kern = gated_pair_kernel<HN, ZK, F16>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), L::kAlloc);
    if (e != cudaSuccess) return e;
    const int64_t tiles = ((a.M + 255) / 256) * ((a.F + HN - 1) / HN);
    const int64_t most = device_sm_count() / 2;
    const unsigned pairs = static_cast<unsigned>(tiles < most ? tiles : most);
    return launch_kernel(kern, dim3(2 * pairs), dim3(L::kThreads), L::kAlloc, stream, 2, mx, mw, mh, mz,
                         static_cast<int>(a.M), static_cast<int>(a.C), static_cast<int>(a.F), a.act, a.status);
}

template <int NT, bool F16>
cudaError_t run_rows(const GatedArgs& a, cudaStream_t stream)
{
    return launch_kernel(gated_rows_kernel<NT, F16>, dim3(static_cast<unsigned>((a.F + 15) / 16)), dim3(256), 0, stream,
                         1, a.X, a.W, static_cast<uint16_t*>(a.H), static_cast<uint16_t*>(a.Z), static_cast<int>(a.M),
                         static_cast<int>(a.C), static_cast<int>(a.F), a.act, a.status);
}

// Measured at 768 to 2048 channels, bf16 (us): one row 2.2 (the 8-row kernel 3.1); 8, 16 and 32
// rows 3.3, 4.0 and 4.6 (the pair kernel 8.3 for each).  Tiles of 64 columns where those of 128
// would leave half the pairs idle: 64 rows 8.0 against 14.5; 600 rows, 48 wide tiles, 10.5 wide
// against 13.3.
template <bool F16>
cudaError_t dispatch(const GatedArgs& a, cudaStream_t stream)
{
    if (a.M <= 1)
        return launch_kernel(gated_row_kernel<F16>, dim3(static_cast<unsigned>((a.F + 7) / 8)), dim3(256), 0, stream, 1,
                             a.X, a.W, static_cast<uint16_t*>(a.H), static_cast<uint16_t*>(a.Z), static_cast<int>(a.C),
                             static_cast<int>(a.F), a.act, a.status);
    if (a.M <= 8) return run_rows<1, F16>(a, stream);
    if (a.M <= 16) return run_rows<2, F16>(a, stream);
    if (a.M <= 32) return run_rows<4, F16>(a, stream);
    const int64_t wide = ((a.M + 255) / 256) * ((a.F + 127) / 128);
    if (2 * wide <= device_sm_count() / 2)
        return a.Z ? run_pair<64, true, F16>(a, stream) : run_pair<64, false, F16>(a, stream);
    return a.Z ? run_pair<128, true, F16>(a, stream) : run_pair<128, false, F16>(a, stream);
}

}  // namespace

cudaError_t launch_gated_forward(const GatedArgs& a, cudaStream_t stream)
{
    return a.f16 ? dispatch<true>(a, stream) : dispatch<false>(a, stream);
}

}  // namespace dgrad
