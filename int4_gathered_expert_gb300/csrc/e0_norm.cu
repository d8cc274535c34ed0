// Residual addition, RMS norm and e4m3 output with a scale per 64 values
// (e0_rmsnorm_q8).
#include <cuda_runtime.h>

#include "e0_internal.h"
#include "e0_types.cuh"

namespace e0 {
namespace {

// One block per row.  A thread keeps its elements in registers between the
// two uses of a row (the sum of squares, then the outputs), so a row is read
// once: bytes moved are the algorithmic ones and the kernel is bound by them.
// Thread i owns the 8 consecutive elements 8(i + j * blockDim): 8 neighbouring
// threads hold one group of 64, whose maximum is three shuffles.
// VEC: H is a multiple of 8 and every row starts on a 16-byte boundary, so the
// 8 elements are whole vector accesses; otherwise they are checked one by one.
struct NormArgs {
    const void* r;
    const void* d;
    const float* w;
    void* r_out;
    void* h;
    uint8_t* q;
    float* qs;
    uint32_t* st;
    int64_t r_ld, d_ld;
    int H;
    float eps;
};

template <int TY, bool VEC, int CH>
__global__ void __launch_bounds__(512) k_rmsnorm_q8(NormArgs A) {
    typedef typename Elem<TY>::T T;
    __shared__ float red[16];
    const int H = A.H, tid = threadIdx.x, nt = blockDim.x;
    const size_t row = blockIdx.x;
    const T* r = reinterpret_cast<const T*>(A.r) + row * A.r_ld;
    const T* d = A.d ? reinterpret_cast<const T*>(A.d) + row * A.d_ld : nullptr;
    T* r_out = A.r_out ? reinterpret_cast<T*>(A.r_out) + row * H : nullptr;
    float v[CH][8];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int e = 8 * (tid + j * nt);
        float dv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.f, dv[i] = 0.f;
        if (VEC) {
            if (e < H) {
                // plain loads, not the read-only path: r_out may be r or d
                if constexpr (TY == E0_F32) {
                    const float4 a = *reinterpret_cast<const float4*>(r + e), b = *reinterpret_cast<const float4*>(r + e + 4);
                    v[j][0] = a.x, v[j][1] = a.y, v[j][2] = a.z, v[j][3] = a.w;
                    v[j][4] = b.x, v[j][5] = b.y, v[j][6] = b.z, v[j][7] = b.w;
                    if (d) {
                        const float4 f = *reinterpret_cast<const float4*>(d + e), g = *reinterpret_cast<const float4*>(d + e + 4);
                        dv[0] = f.x, dv[1] = f.y, dv[2] = f.z, dv[3] = f.w;
                        dv[4] = g.x, dv[5] = g.y, dv[6] = g.z, dv[7] = g.w;
                    }
                } else {
                    const uint4 a = *reinterpret_cast<const uint4*>(r + e);
                    uint4 b = make_uint4(0, 0, 0, 0);
                    if (d) b = *reinterpret_cast<const uint4*>(d + e);
                    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = unpack16<TY>(wa[i]), g = unpack16<TY>(wb[i]);
                        v[j][2 * i] = f.x, v[j][2 * i + 1] = f.y, dv[2 * i] = g.x, dv[2 * i + 1] = g.y;
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e + i < H) {
                    v[j][i] = Elem<TY>::get(r[e + i]);
                    if (d) dv[i] = Elem<TY>::get(d[e + i]);
                }
        }
        if (d) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = Elem<TY>::get(Elem<TY>::put(v[j][i] + dv[i]));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
        if (r_out) {
            if (VEC) {
                if (e < H) store_vec<TY>(r_out + e, v[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (e + i < H) r_out[e + i] = Elem<TY>::put(v[j][i]);
            }
        }
    }
    ss = warp_sum(ss);
    if ((tid & 31) == 0) red[tid >> 5] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < nt / 32; ++i) ss += red[i];
    const float rstd = 1.f / sqrtf(ss / (float)H + A.eps);

    T* h = A.h ? reinterpret_cast<T*>(A.h) + row * H : nullptr;
    uint8_t* q = A.q ? A.q + row * H : nullptr;
    const int ng = (H + GROUP - 1) / GROUP;
    bool bad_any = false;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int e = 8 * (tid + j * nt);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x = v[j][i] * rstd;
            if (A.w && e + i < H) x *= __ldg(A.w + e + i);
            v[j][i] = x;
            if (e + i < H) m = max(m, __float_as_uint(x) & 0x7FFFFFFFu);  // ordered as |x|, NaN above infinity
        }
        if (h) {
            if (VEC) {
                if (e < H) store_vec<TY>(h + e, v[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (e + i < H) h[e + i] = Elem<TY>::put(v[j][i]);
            }
        }
        if (!q) continue;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool bad = m >= 0x7F800000u;
        bad_any |= bad;
        const float mx = __uint_as_float(m);
        const bool zero = bad || mx < 7.7037198e-34f;  // 2^-110: 448 / mx and mx / 448 stay normal numbers
        const float inv = zero ? 0.f : 448.f / mx;
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = zero ? 0u : e4m3x2(v[j][2 * i] * inv, v[j][2 * i + 1] * inv);
        if (VEC) {
            if (e < H) *reinterpret_cast<uint2*>(q + e) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e + i < H) q[e + i] = (uint8_t)(c[i / 2] >> (8 * (i & 1)));
        }
        if ((tid & 7) == 0 && e < H) A.qs[row * ng + e / GROUP] = zero ? 0.f : mx / 448.f;
    }
    if (bad_any && (tid & 7) == 0) set_status(A.st, E0_ST_NONFINITE);
}

template <int TY, bool VEC>
int launch(const NormArgs& a, int T, cudaStream_t s) {
    const int chunks = (a.H + 7) / 8;
    int nt = (chunks + 31) / 32 * 32;
    if (nt > 512) nt = 512;
    if (chunks <= 512)
        k_rmsnorm_q8<TY, VEC, 1><<<T, nt, 0, s>>>(a);
    else if (chunks <= 1024)
        k_rmsnorm_q8<TY, VEC, 2><<<T, nt, 0, s>>>(a);
    else
        k_rmsnorm_q8<TY, VEC, 4><<<T, nt, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

}  // namespace

int rmsnorm_q8(const void* r, const void* d, const float* w, int T, int H, int dtype, float eps, int64_t r_ld,
               int64_t d_ld, void* r_out, void* h, uint8_t* q, float* qs, uint32_t* st, cudaStream_t s) {
    NormArgs a = {r, d, w, r_out, h, q, qs, st, r_ld, d_ld, H, eps};
    const int sz = type_size(dtype);
    uintptr_t bits = (uintptr_t)r | (uintptr_t)d | (uintptr_t)r_out | (uintptr_t)h | (uintptr_t)(r_ld * sz);
    if (d) bits |= (uintptr_t)(d_ld * sz);
    const bool vec = H % 8 == 0 && !(bits & 15) && !((uintptr_t)q & 7);
    switch (dtype) {
        case E0_F32: return vec ? launch<E0_F32, true>(a, T, s) : launch<E0_F32, false>(a, T, s);
        case E0_F16: return vec ? launch<E0_F16, true>(a, T, s) : launch<E0_F16, false>(a, T, s);
        default: return vec ? launch<E0_BF16, true>(a, T, s) : launch<E0_BF16, false>(a, T, s);
    }
}

}  // namespace e0
