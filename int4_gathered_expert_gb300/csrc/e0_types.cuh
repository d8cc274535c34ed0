// Element types of the calls that take one (E0_F32, E0_F16, E0_BF16, E0_E4M3):
// loads and stores in fp32, and the 8-bit format's conversions.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "e0_common.cuh"

namespace e0 {

// Let kernel f have `bytes` of dynamic shared memory on the current device: asked
// for once a device (`bytes` is the most that any launch of f wants).
inline bool allow_smem(const void* f, size_t bytes, std::atomic<uint64_t>& asked) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (asked.load(std::memory_order_relaxed) & bit)) return true;
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) return false;
    if (dev < 64) asked.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

inline int type_size(int t) { return t == E0_F32 ? 4 : t == E0_E4M3 ? 1 : 2; }

template <int TY>
struct Elem;
template <>
struct Elem<E0_F32> {
    typedef float T;
    static E0_DEV float get(float v) { return v; }
    static E0_DEV float put(float v) { return v; }
};
template <>
struct Elem<E0_F16> {
    typedef __half T;
    static E0_DEV float get(__half v) { return __half2float(v); }
    static E0_DEV __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<E0_BF16> {
    typedef __nv_bfloat16 T;
    static E0_DEV float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static E0_DEV __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

// Two 16-bit values of a 32-bit word as fp32.
template <int TY>
E0_DEV float2 unpack16(uint32_t w) {
    if (TY == E0_F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <int TY>
E0_DEV uint32_t pack16(float a, float b) {
    if (TY == E0_F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// N consecutive elements (N a multiple of 4; the address aligned to their size
// or to 16 bytes, whichever is less).
template <int TY, int N>
E0_DEV void load_vec(const void* p, float (&v)[N]) {
    if constexpr (TY == E0_F32) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
            v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack16<TY>(w[j]);
                v[8 * i + 2 * j] = f.x, v[8 * i + 2 * j + 1] = f.y;
            }
        }
        if constexpr (N % 8 == 4) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(p) + N / 4 - 1);
            const float2 a = unpack16<TY>(u.x), b = unpack16<TY>(u.y);
            v[N - 4] = a.x, v[N - 3] = a.y, v[N - 2] = b.x, v[N - 1] = b.y;
        }
    }
}
template <int TY, int N>
E0_DEV void store_vec(void* p, const float (&v)[N]) {
    if constexpr (TY == E0_F32) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        static_assert(N % 8 == 0, "whole 16-byte stores");
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
            reinterpret_cast<uint4*>(p)[i] =
                make_uint4(pack16<TY>(v[8 * i], v[8 * i + 1]), pack16<TY>(v[8 * i + 2], v[8 * i + 3]),
                           pack16<TY>(v[8 * i + 4], v[8 * i + 5]), pack16<TY>(v[8 * i + 6], v[8 * i + 7]));
    }
}

// fp32 pair -> two e4m3 codes (nearest, ties to even, beyond 448 -> 448), a in
// the low byte.
E0_DEV uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// Two codes (low byte first) -> fp16 pair, exact.
E0_DEV uint32_t e4m3x2_to_half2(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

}  // namespace e0
