// adamw.cu -- the AdamW step over many tensors at once (states in 32 or in 8 bits) and the
// norm of many gradients.
//
// For each element, all in fp32, with g = scale * grad:
//     m' = b1 m + (1 - b1) g,   v' = b2 v + (1 - b2) g g
//     p' = p (1 - lr wd) - lr (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps)
// A handful of operations for 22 to 28 bytes (8-bit states 10 to 18): HBM bounds it.  The 8-bit step has 78 to 109
// instructions an element and is bound by nothing alone (slots 59 to 70% busy): a warp loads a block, computes and stores one after
// the other, with three blocks of warps an SM.  A launch takes a table of
// tensors among its parameters (no copy to the device, nothing kept between calls, so a
// captured step carries its own), and its blocks take equal runs of 2048-element chunks.
//
// 8-bit states.  Blocks of 256 elements of a tensor share the largest |m| and the largest v
// (fp32, M and V).  Codes are linear in the square root of a gradient's magnitude:
//     m = c|c| / 127^2 * M, c in -127 .. 127,    v = (c / 255)^4 * V, c in 0 .. 255
// so that both reach down to 6e-5 (m) and 1.5e-5 (v's root) of a block's largest gradient with
// steps of 2/c and 4/c of the value: 1.6% next to the largest, where a linear code's 0.4% of
// the largest would be 100% of what lies 250 times below.  A v' above zero keeps a code above
// zero: m / sqrt(0) would be a step of any size.
// A code stands for the nearer of two values (the lower at a tie), or with a seed for the upper with
// probability (w - low)/(high - low): what nearest rounding keeps losing, a v that moves by less
// than half a step at a time, adds up on average.  The stored bits are defined by fp32
// operations each rounded on its own (no fused multiply-add), given in include/dgrad.h, so that
// a step's states can be reproduced exactly.  A warp holds a block: one reduction for M, one for V.
//
// Random bits: Philox-4x32-10 (J. Salmon, M. Moraes, R. Dror and D. Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011) at counter (b, offset) and key seed; elements are counted
// with every tensor rounded up to whole blocks of 256, element i takes word i % 4 of b = i / 4, its low
// half for m, its high half for v.
#include <type_traits>

#include "common.cuh"
#include "host_util.h"
#include "launchers.h"
#include "rowvec.cuh"

namespace dgrad {
namespace {

constexpr int kOptBlock = 256;                  // threads
constexpr int kQuant = 256;                     // elements that share M and V: a warp's
constexpr int kOptChunk = kQuant * (kOptBlock / 32);   // elements a block takes at a time
constexpr int kSteps = kQuant / (32 * 4);       // vectors of four a thread takes of it

// Tensors of a launch's table (its parameters hold 32764 bytes).  The small one takes the host 2.2 us less
// a call (10 tensors: a step 6.5 us, 8.7 with the large one); the device does not tell them apart.
constexpr int kFewTensors = 24, kManyTensors = 380;

struct OptHyper {
    float lr, b1, c1, b2, c2, eps, decay, wd, ibc1, ibc2, ln_b1, ln_b2, zero;   // zero: -0
    const float* lr_dev;         // null: lr and decay above
    const long long* step_dev;   // null: ibc1 and ibc2 above
    const float* scale;          // null: 1
    uint32_t seed_lo, seed_hi, off_lo, off_hi;
    int* status;
};

struct AdamTensor {
    void* p;
    const void* g;
    void* m;
    void* v;
    float* w;
    float* m_max;
    float* v_max;
    long long n;
    long long block0;   // quantisation blocks before it
    int vec;            // every pointer is aligned for four elements
};

template <int CAP>
struct OptTable {
    OptHyper h;
    int count;
    unsigned chunks;              // of all tensors
    unsigned first[CAP + 1];      // a tensor's first chunk
    AdamTensor t[CAP];
};

// Four elements of kind EK at element i of p: FULL, at once (16 bytes of fp32, 8 of 16 bits); else the
// `have` that there are, one by one.
template <int EK, bool FULL>
__device__ __forceinline__ float4 load4(const void* p, long long i, int have)
{
    if constexpr (FULL && EK == kF32) {
        return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    } else if constexpr (FULL) {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
        const float2 a = h16x2_to_float2<EK>(u.x), b = h16x2_to_float2<EK>(u.y);
        return make_float4(a.x, a.y, b.x, b.y);
    }
    float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < have) {
            RowVec<EK, 1> v;
            float e[1];
            v.load(p, i + k);
            v.unpack(e);
            f[k] = e[0];
        }
    return make_float4(f[0], f[1], f[2], f[3]);
}

template <int EK, bool FULL>
__device__ __forceinline__ void store4(void* p, long long i, int have, float4 x, long long n, int* status)
{
    constexpr int es = elem_bytes<EK>();
    char* at = static_cast<char*>(p) + i * es;
    if constexpr (FULL) {
        if (!store_ok(p, n * es, at, 4 * es, status)) return;
        if constexpr (EK == kF32)
            *reinterpret_cast<float4*>(at) = x;
        else
            *reinterpret_cast<uint2*>(at) = make_uint2(float2_to_h16x2<EK>(x.x, x.y), float2_to_h16x2<EK>(x.z, x.w));
        return;
    }
    const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < have && store_ok(p, n * es, at + k * es, es, status)) {
            RowVec<EK, 1> v;
            const float e[1] = {f[k]};
            v.pack(e);
            v.store(p, i + k);
        }
}

template <bool FULL>
__device__ __forceinline__ uint32_t load_codes(const void* p, long long i, int have)
{
    const uint8_t* c = static_cast<const uint8_t*>(p) + i;
    if constexpr (FULL) return *reinterpret_cast<const uint32_t*>(c);
    uint32_t w = 0;
    for (int k = 0; k < have; ++k) w |= static_cast<uint32_t>(c[k]) << (8 * k);
    return w;
}

template <bool FULL>
__device__ __forceinline__ void store_codes(void* p, long long i, int have, uint32_t w, long long n, int* status)
{
    uint8_t* c = static_cast<uint8_t*>(p) + i;
    if constexpr (FULL) {
        if (store_ok(p, n, c, 4, status)) *reinterpret_cast<uint32_t*>(c) = w;
        return;
    }
    for (int k = 0; k < have; ++k)
        if (store_ok(p, n, c + k, 1, status)) c[k] = static_cast<uint8_t>(w >> (8 * k));
}

__device__ __forceinline__ uint4 opt_philox(const OptHyper& h, unsigned long long b)
{
    uint32_t c0 = static_cast<uint32_t>(b), c1 = static_cast<uint32_t>(b >> 32), c2 = h.off_lo, c3 = h.off_hi;
    uint32_t k0 = h.seed_lo, k1 = h.seed_hi;
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

// Pairs of fp32 operations, each rounded on its own.  A packed product and the sum that follows it
// become one multiply-add in the assembler, rounded once, whatever rounding they name, and so does a
// multiply-add with a -0 that it can see.  One with a -0 that comes with the call does not.
struct Packed {
    float2 zero;     // -0, -0
    __device__ __forceinline__ float2 mul(float2 a, float2 b) const { return __ffma2_rn(a, b, zero); }
};
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }

// 2^23 plus byte k of w, or its half h: numbers without the slow conversions.
__device__ __forceinline__ float byte_float(uint32_t w, int k) { return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | k)); }
__device__ __forceinline__ float half_float(uint32_t w, int h) { return __uint_as_float(__byte_perm(w, 0x4B000000u, h ? 0x7432u : 0x7410u)); }
constexpr float kTwo23 = 8388608.0f;

// Values that codes stand for, as multiples of 1/127^2 and 1/255^4 of the block's largest.
template <bool FOURTH>
__device__ __forceinline__ float code_value(float c)
{
    const float q = __fmul_rn(c, c);
    return FOURTH ? __fmul_rn(q, q) : q;
}
constexpr float kMostM = 16129.0f, kMostV = 4228250625.0f;                 // value(127), value(255)
constexpr float kUnitM = static_cast<float>(1.0 / 16129.0), kUnitV = static_cast<float>(1.0 / 4228250625.0);

// The values of codes k and k + 1 of a word of four.
__device__ __forceinline__ float2 decode_m2(const Packed& P, uint32_t word, int k, float2 top)
{
    const uint32_t w = word ^ 0x80808080u;    // c + 128
    const float2 f = add2(make_float2(byte_float(w, k), byte_float(w, k + 1)), pair(-(kTwo23 + 128.0f)));
    return P.mul(P.mul(make_float2(__fmul_rn(f.x, fabsf(f.x)), __fmul_rn(f.y, fabsf(f.y))), pair(kUnitM)), top);
}
__device__ __forceinline__ float2 decode_v2(const Packed& P, uint32_t word, int k, float2 top)
{
    const float2 f = add2(make_float2(byte_float(word, k), byte_float(word, k + 1)), pair(-kTwo23));
    const float2 q = P.mul(f, f);
    return P.mul(P.mul(P.mul(q, q), pair(kUnitV)), top);
}

// What a block's largest value scales the others by: w = (x k) inv, with k a power of two that
// keeps inv = (1/(top k)) value(most) an ordinary number.  With a NaN for the largest value its whole
// block stands for NaN, whatever the codes.
struct CodeScale {
    float k, inv;
};
template <bool FOURTH>
__device__ __forceinline__ CodeScale code_scale(float top)
{
    CodeScale s;
    s.k = top < 0x1p-60f ? 0x1p64f : top > 0x1p60f ? 0x1p-64f : 1.0f;
    s.inv = top > 0.f ? __fmul_rn(__frcp_rn(__fmul_rn(top, s.k)), FOURTH ? kMostV : kMostM) : 0.f;
    return s;
}

// The code of x >= 0: low is the largest c with value(c) <= w; the upper neighbour is taken where
// (w - value(low)) 65536 > (value(low + 1) - value(low)) draw; nearest: draw = 32768.  The
// approximate root r (2^-21) finds low or, lowered by 2^-11, the code below it; that is seen from
// w - value(low) >= value(low + 1) - value(low).  Then w lies above value(low + 1) by less than 2^-10 of the
// next step, and low + 1 is taken all the same, but for draws below 64, which set `below`: the codes
// are formed again by code_of.
__device__ __forceinline__ float2 low_of(float2 r)
{
    const float2 t = add2(add2(add2(r, pair(-(0.5f + 0x1p-11f))), pair(1.5f * kTwo23)), pair(-1.5f * kTwo23));
    return make_float2(fmaxf(t.x, 0.f), fmaxf(t.y, 0.f));
}
template <bool FOURTH>
__device__ __noinline__ float code_of(float w, float low, float draw)
{
    while (code_value<FOURTH>(low + 1.f) <= w && low < 256.f) low += 1.f;
    const float at = code_value<FOURTH>(low);
    const float d = __fsub_rn(w, at), step = __fsub_rn(code_value<FOURTH>(low + 1.f), at);
    return fminf(__fmul_rn(d, 65536.f) > __fmul_rn(step, draw) ? low + 1.f : low, FOURTH ? 255.0f : 127.0f);
}
template <bool FOURTH, bool NEAREST>
__device__ __forceinline__ float2 code2(const Packed& P, float2 w, float2 r, float2 draw, bool& below)
{
    float2 low = low_of(r), d, step;    // the largest of a block has low = 126 (254) and goes up: no code passes 127 (255)
    if constexpr (FOURTH) {
        const float2 q = P.mul(low, low), next = add2(low, pair(1.f)), q1 = P.mul(next, next);
        const float2 minus = P.mul(P.mul(q, pair(-1.f)), q);
        step = add2(P.mul(q1, q1), minus);
        d = add2(w, minus);
    } else {     // whole numbers below 2^24: exact
        step = ffma2(low, pair(2.f), pair(1.f));
        d = ffma2(P.mul(low, pair(-1.f)), low, w);
    }
    if constexpr (NEAREST) {
        d = add2(d, d);
    } else {
        below = below || (d.x >= step.x && draw.x < 64.f) || (d.y >= step.y && draw.y < 64.f);
        d = P.mul(d, pair(65536.f));
        step = P.mul(step, draw);
    }
    low.x = d.x > step.x ? low.x + 1.f : low.x;
    low.y = d.y > step.y ? low.y + 1.f : low.y;
    return low;
}

__device__ __forceinline__ float root_of(float v)
{
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The largest of a warp's values >= 0 (the order of the bits is that of the values); NaN where
// one is no finite number.
__device__ __forceinline__ float warp_largest(float x)
{
    const uint32_t big = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x) & 0x7FFFFFFFu);
    return __uint_as_float(big >= 0x7F800000u ? 0x7FC00000u : big);
}

// The step's scalars, once per block.
struct OptStep {
    float scale, nlr, decay, ibc1, ibc2;
    bool skip;
};
__device__ __forceinline__ OptStep opt_step(const OptHyper& h)
{
    OptStep s{1.f, -h.lr, h.decay, h.ibc1, h.ibc2, false};
    if (h.scale) {
        s.scale = *h.scale;
        s.skip = !isfinite(s.scale);
    }
    if (h.lr_dev) {
        const float lr = *h.lr_dev;
        s.skip = s.skip || !isfinite(lr);
        s.nlr = -lr;
        s.decay = fmaf(-lr, h.wd, 1.f);
    }
    if (h.step_dev) {
        const float t = static_cast<float>(*h.step_dev);
        s.skip = s.skip || t < 1.f;
        s.ibc1 = -1.f / expm1f(t * h.ln_b1);
        s.ibc2 = -1.f / expm1f(t * h.ln_b2);
    }
    return s;
}

// m', v' and the new weights of a pair; root: that of v'/(1 - b2^t).
__device__ __forceinline__ void step2(const Packed& P, float2 g, float2& m, float2& v, float2& w, float2& root, const OptHyper& h, const OptStep& s)
{
    g = P.mul(g, pair(s.scale));
    m = add2(P.mul(m, pair(h.b1)), P.mul(g, pair(h.c1)));
    v = add2(P.mul(v, pair(h.b2)), P.mul(P.mul(g, pair(h.c2)), g));
    const float2 u = P.mul(v, pair(s.ibc2));
    float2 inv, top = P.mul(m, pair(s.ibc1));
    // below 2^-126 the root may be 0 beside an eps from 1e-12 on
    root = make_float2(root_of(u.x), root_of(u.y));
    float2 den = add2(root, pair(h.eps));
    if (h.eps < 1e-12f) {
        asm("sqrt.approx.f32 %0, %1;" : "=f"(root.x) : "f"(u.x));
        asm("sqrt.approx.f32 %0, %1;" : "=f"(root.y) : "f"(u.y));
        den = add2(root, pair(h.eps));
        // a subnormal den has no reciprocal: both ends of the fraction are raised by 2^64
        const float2 up = make_float2(den.x < 0x1p-64f ? 0x1p64f : 1.f, den.y < 0x1p-64f ? 0x1p64f : 1.f);
        den = P.mul(den, up);
        top = P.mul(top, up);
    }
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv.x) : "f"(den.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv.y) : "f"(den.y));
    w = ffma2(pair(s.nlr), P.mul(top, inv), P.mul(w, pair(s.decay)));
}

// The larger magnitude; NaN where one is NaN.
__device__ __forceinline__ float larger(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

// Block q of 256 elements of tensor t, by a warp.  PK, GK: the parameters' and gradients' types; MASTER: an
// fp32 copy of the parameters is what is stepped.  MODE 0: fp32 states; 1: 8 bits, nearest; 2: 8 bits,
// stochastic.  FULL: all of them are there, and every pointer is aligned for four.
template <int PK, int GK, bool MASTER, int MODE, bool FULL>
__device__ __forceinline__ void adamw_block(const AdamTensor& t, long long q, const OptHyper& h, const OptStep& st, const Packed& P)
{
    const int lane = threadIdx.x & 31;
    const long long i0 = q * kQuant + lane * 4;
    float4 g[kSteps], w[kSteps], m[kSteps], v[kSteps];
    uint32_t cm[kSteps], cv[kSteps];
    float mtop = 0.f, vtop = 0.f;
    if constexpr (MODE != 0) {
        mtop = t.m_max[q];
        vtop = t.v_max[q];
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        const long long i = i0 + j * 128;
        const int have = FULL ? 4 : static_cast<int>(max(0LL, min(4LL, t.n - i)));
        g[j] = load4<GK, FULL>(t.g, i, have);
        w[j] = MASTER ? load4<kF32, FULL>(t.w, i, have) : load4<PK, FULL>(t.p, i, have);
        if constexpr (MODE == 0) {
            m[j] = load4<kF32, FULL>(t.m, i, have);
            v[j] = load4<kF32, FULL>(t.v, i, have);
        } else {
            cm[j] = load_codes<FULL>(t.m, i, have);
            cv[j] = load_codes<FULL>(t.v, i, have);
        }
    }
    float big_m = 0.f, big_v = 0.f;
    float2 root[kSteps][2];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        float2 gg[2] = {make_float2(g[j].x, g[j].y), make_float2(g[j].z, g[j].w)};
        float2 ww[2] = {make_float2(w[j].x, w[j].y), make_float2(w[j].z, w[j].w)};
        float2 mm[2], vv[2];
        if constexpr (MODE == 0) {
            mm[0] = make_float2(m[j].x, m[j].y);
            mm[1] = make_float2(m[j].z, m[j].w);
            vv[0] = make_float2(v[j].x, v[j].y);
            vv[1] = make_float2(v[j].z, v[j].w);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if constexpr (MODE != 0) {
                mm[k] = decode_m2(P, cm[j], 2 * k, pair(mtop));
                vv[k] = decode_v2(P, cv[j], 2 * k, pair(vtop));
            }
            step2(P, gg[k], mm[k], vv[k], ww[k], root[j][k], h, st);
            if constexpr (MODE != 0) {
                big_m = larger(larger(big_m, mm[k].x), mm[k].y);
                big_v = larger(larger(big_v, vv[k].x), vv[k].y);
            }
        }
        m[j] = make_float4(mm[0].x, mm[0].y, mm[1].x, mm[1].y);
        v[j] = make_float4(vv[0].x, vv[0].y, vv[1].x, vv[1].y);
        w[j] = make_float4(ww[0].x, ww[0].y, ww[1].x, ww[1].y);
    }
    CodeScale sm, sv;
    float roots = 0.f;      // root_of(v' inv) = root_of(root roots), where ordinary numbers allow it
    if constexpr (MODE != 0) {
        big_m = warp_largest(big_m);
        big_v = warp_largest(big_v);
        sm = code_scale<false>(big_m);
        sv = code_scale<true>(big_v);
        if (sv.k == 1.0f && st.ibc2 < 0x1p30f) roots = root_of(sv.inv / st.ibc2);
        const long long nq = (t.n + kQuant - 1) / kQuant;
        if (lane == 0 && store_ok(t.m_max, nq * 4, t.m_max + q, 4, h.status)) t.m_max[q] = big_m;
        if (lane == 0 && store_ok(t.v_max, nq * 4, t.v_max + q, 4, h.status)) t.v_max[q] = big_v;
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        const long long i = i0 + j * 128;
        const int have = FULL ? 4 : static_cast<int>(max(0LL, min(4LL, t.n - i)));
        if (MASTER) store4<kF32, FULL>(t.w, i, have, w[j], t.n, h.status);
        store4<PK, FULL>(t.p, i, have, w[j], t.n, h.status);
        if constexpr (MODE == 0) {
            store4<kF32, FULL>(t.m, i, have, m[j], t.n, h.status);
            store4<kF32, FULL>(t.v, i, have, v[j], t.n, h.status);
        } else {
            uint4 bits = make_uint4(0, 0, 0, 0);
            if constexpr (MODE == 2)
                bits = opt_philox(h, static_cast<unsigned long long>(t.block0 + q) * (kQuant / 4) + lane + j * 32);
            const uint32_t word[4] = {bits.x, bits.y, bits.z, bits.w};
            uint32_t om[2], ov[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 x = k ? make_float2(m[j].z, m[j].w) : make_float2(m[j].x, m[j].y);
                const float2 y = k ? make_float2(v[j].z, v[j].w) : make_float2(v[j].x, v[j].y);
                float2 dm = pair(0.f), dv = pair(0.f);
                if constexpr (MODE == 2) {
                    dm = add2(make_float2(half_float(word[2 * k], 0), half_float(word[2 * k + 1], 0)), pair(-kTwo23));
                    dv = add2(make_float2(half_float(word[2 * k], 1), half_float(word[2 * k + 1], 1)), pair(-kTwo23));
                }
                float2 wm = make_float2(fabsf(x.x), fabsf(x.y)), wv = y;
                if (sm.k != 1.0f) wm = P.mul(wm, pair(sm.k));
                if (sv.k != 1.0f) wv = P.mul(wv, pair(sv.k));
                wm = P.mul(wm, pair(sm.inv));
                wv = P.mul(wv, pair(sv.inv));
                const float2 rm = make_float2(root_of(wm.x), root_of(wm.y));
                float2 rv = P.mul(root[j][k], pair(roots));
                if (roots == 0.f) rv = make_float2(root_of(wv.x), root_of(wv.y));
                rv = make_float2(root_of(rv.x), root_of(rv.y));
                bool below = false;
                float2 a = code2<false, MODE == 1>(P, wm, rm, dm, below), b = code2<true, MODE == 1>(P, wv, rv, dv, below);
                if (MODE == 2 && below) {
                    const float2 la = low_of(rm), lb = low_of(rv);
                    a = make_float2(code_of<false>(wm.x, la.x, dm.x), code_of<false>(wm.y, la.y, dm.y));
                    b = make_float2(code_of<true>(wv.x, lb.x, dv.x), code_of<true>(wv.y, lb.y, dv.y));
                }
                // the low byte of 2^23 + code; m's codes are 128 higher there
                const float2 as = add2(make_float2(copysignf(a.x, x.x), copysignf(a.y, x.y)), pair(kTwo23 + 128.0f));
                // v' inf is inf, or NaN for 0: 1 or 0
                const float inf = __int_as_float(0x7F800000);
                const float2 bs = add2(make_float2(fmaxf(b.x, __saturatef(y.x * inf)), fmaxf(b.y, __saturatef(y.y * inf))), pair(kTwo23));
                om[k] = __byte_perm(__float_as_uint(as.x), __float_as_uint(as.y), 0x0040);
                ov[k] = __byte_perm(__float_as_uint(bs.x), __float_as_uint(bs.y), 0x0040);
            }
            store_codes<FULL>(t.m, i, have, __byte_perm(om[0], om[1], 0x5410) ^ 0x80808080u, t.n, h.status);
            store_codes<FULL>(t.v, i, have, __byte_perm(ov[0], ov[1], 0x5410), t.n, h.status);
        }
    }
}

// A register more than 64 (80) a thread would leave an SM fewer blocks: 60 M parameters, fp32 states, 274 us with
// four blocks and 301 with three.
template <int PK, int GK, bool MASTER, int MODE, int CAP>
__global__ void __launch_bounds__(kOptBlock, MODE == 0 ? 4 : 3) adamw_kernel(const __grid_constant__ OptTable<CAP> tab)
{
    const int warp = threadIdx.x >> 5;
    // equal runs of chunks
    const unsigned each = tab.chunks / gridDim.x, more = tab.chunks % gridDim.x;
    unsigned c = blockIdx.x * each + min(blockIdx.x, more);
    const unsigned end = c + each + (blockIdx.x < more ? 1 : 0);
    int lo = 0, hi = tab.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    pdl_wait();
    pdl_trigger();
    const OptHyper& h = tab.h;
    const OptStep st = opt_step(h);
    const Packed P{make_float2(h.zero, h.zero)};
    if (st.skip) return;
    for (; c < end; ++c) {
        while (tab.first[lo + 1] <= c) ++lo;
        const AdamTensor& t = tab.t[lo];
        const long long q = static_cast<long long>(c - tab.first[lo]) * (kOptBlock / 32) + warp;   // block of 256
        if (q * kQuant >= t.n) continue;
        if (t.vec != 0 && (q + 1) * kQuant <= t.n)
            adamw_block<PK, GK, MASTER, MODE, true>(t, q, h, st, P);
        else
            adamw_block<PK, GK, MASTER, MODE, false>(t, q, h, st, P);
    }
}

// ------------------------------------------- what 8-bit states stand for, as fp32

struct MomentTensor {
    const void* m;
    const void* v;
    const float* m_max;
    const float* v_max;
    float* m_out;
    float* v_out;
    long long n;
    int vec;
};

template <int CAP>
struct MomentTable {
    float zero;                   // -0
    int count;
    unsigned chunks;
    int* status;
    unsigned first[CAP + 1];
    MomentTensor t[CAP];
};

template <int CAP>
__global__ void __launch_bounds__(kOptBlock) moments_kernel(const __grid_constant__ MomentTable<CAP> tab)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned each = tab.chunks / gridDim.x, more = tab.chunks % gridDim.x;
    unsigned c = blockIdx.x * each + min(blockIdx.x, more);
    const unsigned end = c + each + (blockIdx.x < more ? 1 : 0);
    int lo = 0, hi = tab.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    pdl_wait();
    pdl_trigger();
    for (; c < end; ++c) {
        while (tab.first[lo + 1] <= c) ++lo;
        const MomentTensor& t = tab.t[lo];
        const long long q = static_cast<long long>(c - tab.first[lo]) * (kOptBlock / 32) + warp;
        if (q * kQuant >= t.n) continue;
        const float mtop = t.m_max[q], vtop = t.v_max[q];
        const Packed P{make_float2(tab.zero, tab.zero)};
        const auto block = [&](auto full) {
            constexpr bool FULL = full.value;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                const long long i = q * kQuant + lane * 4 + j * 128;
                const int have = FULL ? 4 : static_cast<int>(max(0LL, min(4LL, t.n - i)));
                const uint32_t cm = load_codes<FULL>(t.m, i, have), cv = load_codes<FULL>(t.v, i, have);
                const float2 m0 = decode_m2(P, cm, 0, pair(mtop)), m1 = decode_m2(P, cm, 2, pair(mtop));
                const float2 v0 = decode_v2(P, cv, 0, pair(vtop)), v1 = decode_v2(P, cv, 2, pair(vtop));
                store4<kF32, FULL>(t.m_out, i, have, make_float4(m0.x, m0.y, m1.x, m1.y), t.n, tab.status);
                store4<kF32, FULL>(t.v_out, i, have, make_float4(v0.x, v0.y, v1.x, v1.y), t.n, tab.status);
            }
        };
        if (t.vec != 0 && (q + 1) * kQuant <= t.n)
            block(std::true_type{});
        else
            block(std::false_type{});
    }
}

// ----------------------------------------------------------- the gradients' norm

constexpr int kFewNorms = 64, kManyNorms = 1600;   // as above: 13.2 us of host time a call, 15.7
constexpr int kNormChunk = 4096;     // elements a block takes at a time: 16 a thread

struct NormTensor {
    const void* g;
    long long n : 63;
    unsigned long long vec : 1;   // on 16 bytes
};

template <int CAP>
struct NormTable {
    int count;
    unsigned chunks;
    double* part;                 // one sum per block of this launch
    int* status;
    unsigned first[CAP + 1];
    NormTensor t[CAP];
};

// Squares of fp32 values are exact in 64 bits, and their sums need not fear overflow, order or length.  A
// thread adds them one after the other, a chain of 64-bit operations that its block's other warps hide.
template <int EK, int CAP>
__global__ void __launch_bounds__(kOptBlock) norm_kernel(const __grid_constant__ NormTable<CAP> tab)
{
    __shared__ double warps[kOptBlock / 32];
    const unsigned each = tab.chunks / gridDim.x, more = tab.chunks % gridDim.x;
    unsigned c = blockIdx.x * each + min(blockIdx.x, more);
    const unsigned end = c + each + (blockIdx.x < more ? 1 : 0);
    int lo = 0, hi = tab.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    pdl_wait();
    pdl_trigger();
    double sum = 0.0;
    constexpr int VEC = 16 / elem_bytes<EK>();
    constexpr int NV = kNormChunk / (kOptBlock * VEC);
    for (; c < end; ++c) {
        while (tab.first[lo + 1] <= c) ++lo;
        const NormTensor& t = tab.t[lo];
        const long long i0 = static_cast<long long>(c - tab.first[lo]) * kNormChunk;
        if (t.vec && i0 + kNormChunk <= t.n) {
            RowVec<EK, VEC> v[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j].load(t.g, i0 + (j * kOptBlock + threadIdx.x) * VEC);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float f[VEC];
                v[j].unpack(f);
#pragma unroll
                for (int k = 0; k < VEC; ++k) sum = fma(static_cast<double>(f[k]), static_cast<double>(f[k]), sum);
            }
        } else {
            const long long i1 = min(t.n, i0 + kNormChunk);
            for (long long i = i0 + threadIdx.x; i < i1; i += kOptBlock) {
                RowVec<EK, 1> v;
                float f[1];
                v.load(t.g, i);
                v.unpack(f);
                sum = fma(static_cast<double>(f[0]), static_cast<double>(f[0]), sum);
            }
        }
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kOptBlock / 32; ++w) sum += warps[w];
        tab.part[blockIdx.x] = sum;
    }
}

// out[0] = the root of the sum of n parts, out[1] = min(1, max_norm/(out[0] + 1e-6)), NaN where
// the norm is no finite number.
__global__ void __launch_bounds__(kOptBlock) norm_join_kernel(const double* part, int n, float max_norm, float* out, int* status)
{
    __shared__ double warps[kOptBlock / 32];
    pdl_wait();
    pdl_trigger();
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += kOptBlock) sum += part[i];
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0 && store_ok(out, 8, out, 8, status)) {
        for (int w = 1; w < kOptBlock / 32; ++w) sum += warps[w];
        const float norm = static_cast<float>(sqrt(sum));
        out[0] = norm;
        out[1] = isfinite(norm) ? fminf(max_norm / (norm + 1e-6f), 1.f) : __int_as_float(0x7FC00000);
    }
}

template <int EK>
bool on4(const void* p)   // aligned for four elements of kind EK
{
    return (reinterpret_cast<uintptr_t>(p) & (4 * elem_bytes<EK>() - 1)) == 0;
}

// Runs of at most CAP tensors; f(begin, end).
template <typename F>
cudaError_t in_runs(int64_t count, int cap, F f)
{
    for (int64_t i = 0; i < count; i += cap) {
        const cudaError_t e = f(i, count - i < cap ? count : i + cap);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

unsigned opt_grid(unsigned chunks, int per_sm)
{
    const unsigned most = static_cast<unsigned>(device_sm_count() * per_sm);
    return chunks < most ? chunks : most;
}

template <int PK, int GK, bool MASTER, int MODE, int CAP>
cudaError_t adamw_run(const AdamWArgs& a, const OptHyper& h, int64_t begin, int64_t end, int64_t& block0, cudaStream_t stream)
{
    OptTable<CAP> tab;
    tab.h = h;
    tab.count = 0;
    unsigned chunks = 0;
    for (int64_t i = begin; i < end; ++i) {
        const dgrad_adamw_tensor_t& s = a.t[i];
        const int64_t at = block0;
        block0 += (s.n + kQuant - 1) / kQuant;
        if (!s.grad || s.n == 0) continue;
        bool vec = on4<PK>(s.param) && on4<GK>(s.grad) && (!MASTER || on4<kF32>(s.master));
        if (MODE == 0)
            vec = vec && on4<kF32>(s.m) && on4<kF32>(s.v);
        else
            vec = vec && ((reinterpret_cast<uintptr_t>(s.m) | reinterpret_cast<uintptr_t>(s.v)) & 3) == 0;
        tab.first[tab.count] = chunks;
        tab.t[tab.count++] = {s.param, s.grad, s.m, s.v, s.master, s.m_max, s.v_max, s.n, at, vec};
        chunks += static_cast<unsigned>((s.n + kOptChunk - 1) / kOptChunk);
    }
    tab.first[tab.count] = chunks;
    tab.chunks = chunks;
    if (chunks == 0) return cudaSuccess;
    return launch_kernel(adamw_kernel<PK, GK, MASTER, MODE, CAP>, dim3(opt_grid(chunks, 8)), dim3(kOptBlock), 0, stream, 1, tab);
}

template <int PK, int GK, bool MASTER, int MODE>
cudaError_t adamw_all(const AdamWArgs& a, const OptHyper& h, cudaStream_t stream)
{
    const int cap = a.count <= kFewTensors ? kFewTensors : kManyTensors;
    int64_t block0 = 0;
    return in_runs(a.count, cap, [&](int64_t b, int64_t e) {
        return cap == kFewTensors ? adamw_run<PK, GK, MASTER, MODE, kFewTensors>(a, h, b, e, block0, stream)
                                  : adamw_run<PK, GK, MASTER, MODE, kManyTensors>(a, h, b, e, block0, stream);
    });
}

template <int PK, int GK, bool MASTER>
cudaError_t adamw_mode(const AdamWArgs& a, const OptHyper& h, cudaStream_t stream)
{
    return a.bits == 32 ? adamw_all<PK, GK, MASTER, 0>(a, h, stream)
           : a.stochastic ? adamw_all<PK, GK, MASTER, 2>(a, h, stream)
                          : adamw_all<PK, GK, MASTER, 1>(a, h, stream);
}

template <int PK>
cudaError_t adamw_types(const AdamWArgs& a, const OptHyper& h, cudaStream_t stream)
{
    if constexpr (PK == kF32) {
        return adamw_mode<kF32, kF32, false>(a, h, stream);
    } else {
        if (a.gk == kF32) return a.master ? adamw_mode<PK, kF32, true>(a, h, stream) : adamw_mode<PK, kF32, false>(a, h, stream);
        return a.master ? adamw_mode<PK, PK, true>(a, h, stream) : adamw_mode<PK, PK, false>(a, h, stream);
    }
}

}  // namespace

cudaError_t launch_adamw(const AdamWArgs& a, cudaStream_t stream)
{
    OptHyper h{};
    h.lr = static_cast<float>(a.lr);
    h.b1 = static_cast<float>(a.beta1);
    h.c1 = static_cast<float>(1.0 - a.beta1);
    h.b2 = static_cast<float>(a.beta2);
    h.c2 = static_cast<float>(1.0 - a.beta2);
    h.eps = static_cast<float>(a.eps);
    h.wd = static_cast<float>(a.weight_decay);
    h.decay = static_cast<float>(1.0 - a.lr * a.weight_decay);
    h.ibc1 = static_cast<float>(a.bias1);
    h.ibc2 = static_cast<float>(a.bias2);
    h.ln_b1 = static_cast<float>(a.ln_beta1);
    h.ln_b2 = static_cast<float>(a.ln_beta2);
    h.lr_dev = a.lr_dev;
    h.step_dev = reinterpret_cast<const long long*>(a.step_dev);
    h.scale = a.scale;
    h.seed_lo = static_cast<uint32_t>(a.seed);
    h.seed_hi = static_cast<uint32_t>(a.seed >> 32);
    h.off_lo = static_cast<uint32_t>(a.offset);
    h.off_hi = static_cast<uint32_t>(a.offset >> 32);
    h.status = a.status;
    h.zero = -0.0f;
    return a.pk == kF32 ? adamw_types<kF32>(a, h, stream) : a.pk == kBF16 ? adamw_types<kBF16>(a, h, stream) : adamw_types<kF16>(a, h, stream);
}

namespace {

template <int CAP>
cudaError_t moments_runs(const dgrad_adamw_tensor_t* t, float* const* m_out, float* const* v_out, int64_t count, int* status,
                         cudaStream_t stream)
{
    return in_runs(count, CAP, [&](int64_t begin, int64_t end) {
        MomentTable<CAP> tab;
        tab.zero = -0.0f;
        tab.count = 0;
        tab.status = status;
        unsigned chunks = 0;
        for (int64_t i = begin; i < end; ++i) {
            if (t[i].n == 0) continue;
            const bool vec = ((reinterpret_cast<uintptr_t>(t[i].m) | reinterpret_cast<uintptr_t>(t[i].v)) & 3) == 0 &&
                             on4<kF32>(m_out[i]) && on4<kF32>(v_out[i]);
            tab.first[tab.count] = chunks;
            tab.t[tab.count++] = {t[i].m, t[i].v, t[i].m_max, t[i].v_max, m_out[i], v_out[i], t[i].n, vec};
            chunks += static_cast<unsigned>((t[i].n + kOptChunk - 1) / kOptChunk);
        }
        tab.first[tab.count] = chunks;
        tab.chunks = chunks;
        if (chunks == 0) return cudaSuccess;
        return launch_kernel(moments_kernel<CAP>, dim3(opt_grid(chunks, 8)), dim3(kOptBlock), 0, stream, 1, tab);
    });
}

}  // namespace

cudaError_t launch_adamw_moments(const dgrad_adamw_tensor_t* t, float* const* m_out, float* const* v_out, int64_t count,
                                 int* status, cudaStream_t stream)
{
    return count <= kFewTensors ? moments_runs<kFewTensors>(t, m_out, v_out, count, status, stream)
                                : moments_runs<kManyTensors>(t, m_out, v_out, count, status, stream);
}

namespace {

constexpr int kNormBlocks = 148 * 8;   // sums a launch leaves at most

template <int EK, int CAP>
cudaError_t norm_runs(const NormArgs& a, int& parts, cudaStream_t stream)
{
    return in_runs(a.count, CAP, [&](int64_t begin, int64_t end) {
        NormTable<CAP> tab;
        tab.count = 0;
        tab.status = a.status;
        unsigned chunks = 0;
        for (int64_t i = begin; i < end; ++i) {
            if (a.n[i] == 0) continue;
            tab.first[tab.count] = chunks;
            tab.t[tab.count].g = a.g[i];
            tab.t[tab.count].n = a.n[i];
            tab.t[tab.count++].vec = (reinterpret_cast<uintptr_t>(a.g[i]) & 15) == 0;
            chunks += static_cast<unsigned>((a.n[i] + kNormChunk - 1) / kNormChunk);
        }
        tab.first[tab.count] = chunks;
        tab.chunks = chunks;
        if (chunks == 0) return cudaSuccess;
        tab.part = a.ws + parts;
        const unsigned grid = chunks < kNormBlocks ? chunks : kNormBlocks;
        parts += static_cast<int>(grid);
        return launch_kernel(norm_kernel<EK, CAP>, dim3(grid), dim3(kOptBlock), 0, stream, 1, tab);
    });
}

template <int EK>
cudaError_t norm_types(const NormArgs& a, int& parts, cudaStream_t stream)
{
    return a.count <= kFewNorms ? norm_runs<EK, kFewNorms>(a, parts, stream) : norm_runs<EK, kManyNorms>(a, parts, stream);
}

}  // namespace

size_t grad_norm_workspace_bytes(int64_t count)
{
    return static_cast<size_t>((count + kManyNorms - 1) / kManyNorms) * kNormBlocks * 8;
}

cudaError_t launch_grad_norm(const NormArgs& a, cudaStream_t stream)
{
    int parts = 0;
    const cudaError_t e = a.ek == kF32 ? norm_types<kF32>(a, parts, stream)
                          : a.ek == kBF16 ? norm_types<kBF16>(a, parts, stream) : norm_types<kF16>(a, parts, stream);
    if (e != cudaSuccess) return e;
    return launch_kernel(norm_join_kernel, dim3(1), dim3(kOptBlock), 0, stream, 1, static_cast<const double*>(a.ws), parts,
                         a.max_norm, a.out, a.status);
}

}  // namespace dgrad
