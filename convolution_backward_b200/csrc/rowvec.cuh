// rowvec.cuh -- vectors of elements along a row, shared by the layer-norm and
// dropout kernels: 16-byte loads and stores where every row starts on 16 bytes,
// single elements where it does not, always widened to fp32 in registers.
#pragma once

#include "common.cuh"

namespace dgrad {

template <int EK>
constexpr int elem_bytes() { return EK == kF32 ? 4 : 2; }

// VEC elements of kind EK as raw words: four words when they are 16 bytes, else
// (VEC == 1) one element in the low bits of one word.
template <int EK, int VEC>
struct RowVec {
    static constexpr int kWords = VEC == 1 ? 1 : 4;
    static_assert(VEC == 1 || VEC * elem_bytes<EK>() == 16, "one element or 16 bytes");
    uint32_t w[kWords];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }

    __device__ __forceinline__ void ones()
    {
        constexpr uint32_t one = EK == kF32 ? 0x3F800000u : EK == kBF16 ? 0x3F80u : 0x3C00u;
        constexpr uint32_t word = EK != kF32 && VEC > 1 ? one | one << 16 : one;
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = word;
    }

    // Element index i of the array at p (a multiple of VEC when VEC > 1).
    __device__ __forceinline__ void load(const void* p, long long i)
    {
        if constexpr (VEC > 1) {
            const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * elem_bytes<EK>());
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else if constexpr (EK == kF32) {
            w[0] = static_cast<const uint32_t*>(p)[i];
        } else {
            w[0] = static_cast<const uint16_t*>(p)[i];
        }
    }

    __device__ __forceinline__ void store(void* p, long long i) const
    {
        if constexpr (VEC > 1)
            *reinterpret_cast<uint4*>(static_cast<char*>(p) + i * elem_bytes<EK>()) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (EK == kF32)
            static_cast<uint32_t*>(p)[i] = w[0];
        else
            static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(w[0]);
    }

    __device__ __forceinline__ void unpack(float (&f)[VEC]) const
    {
        if constexpr (EK == kF32) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(w[i]);
        } else if constexpr (VEC == 1) {
            f[0] = h16x2_to_float2<EK>(w[0]).x;
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const float2 v = h16x2_to_float2<EK>(w[i]);
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    }

    // Round to nearest even.
    __device__ __forceinline__ void pack(const float (&f)[VEC])
    {
        if constexpr (EK == kF32) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(f[i]);
        } else if constexpr (VEC == 1) {
            w[0] = float2_to_h16x2<EK>(f[0], 0.f) & 0xFFFFu;
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) w[i] = float2_to_h16x2<EK>(f[2 * i], f[2 * i + 1]);
        }
    }
};

// A 16-byte vector's elements as pairs of fp32 (packed FP32 instructions take two at a time).
template <int EK, int VEC>
__device__ __forceinline__ void unpack_pairs(const RowVec<EK, VEC>& v, float2 (&f)[VEC / 2])
{
    float a[VEC];
    v.unpack(a);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) f[i] = make_float2(a[2 * i], a[2 * i + 1]);
}

template <int EK, int VEC>
__device__ __forceinline__ void pack_pairs(RowVec<EK, VEC>& v, const float2 (&f)[VEC / 2])
{
    float a[VEC];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        a[2 * i] = f[i].x;
        a[2 * i + 1] = f[i].y;
    }
    v.pack(a);
}

}  // namespace dgrad
