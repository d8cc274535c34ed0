// Residual addition, RMS norm and e4m3 output with a scale per 64 values
// (e0_rmsnorm_q8).
#include <cuda_runtime.h>

#include "e0_internal.h"
#include "e0_types.cuh"

namespace e0 {
namespace {

// A row's elements stay in registers between their two uses (the sum of squares,
// then the outputs), so a row is read once: bytes moved are the algorithmic ones
// and the kernel is bound by them.  Chunk c of a row is the 8 consecutive elements
// 8c...; neighbouring lanes hold neighbouring chunks, so a group of 64 is 8 lanes
// and its maximum three shuffles.  Two shapes: a block per row, and for many short
// rows a warp per row, without the block's barrier.
// VEC: H is a multiple of 8 and every row starts on a 16-byte boundary, so a chunk
// is whole vector accesses; otherwise elements are checked one by one.
//
// Measured (device time, GB300): 16384 x 2048 fp32, 436 MB: 64.1 us, 6.8 TB/s, the
// measured copy rate; 16384 x 1536 bf16, 178 MB: 28.9 us, 6.1 TB/s, 91 % of it; 8 x 2048
// fp32: 1.8 us, a launch.  What got the second there from 43.1 us: all loads before the
// first use, approximate reciprocals in place of divisions, one-instruction maxima.
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
    int T, H;
    float eps, inv_h;
};

// A chunk as it is in memory: the 8 elements from e on (VEC: a place beyond the row
// reads the row's first chunk instead, so that no branch stands between the loads of
// several chunks; what it read counts as zeros).  Plain loads, not the read-only path:
// r_out may be r or d.
template <int TY, bool VEC>
struct Chunk {
    typedef typename Elem<TY>::T T;
    static constexpr int WORDS = VEC ? (TY == E0_F32 ? 8 : 4) : 8;
    uint32_t w[WORDS];
    E0_DEV void load(const T* p, int e, int H) {
        if constexpr (VEC) {
            const uint4* q = reinterpret_cast<const uint4*>(p + (e < H ? e : 0));
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 u = q[i];
                w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = e + i < H ? __float_as_uint(Elem<TY>::get(p[e + i])) : 0u;
        }
    }
    E0_DEV void get(int e, int H, float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (!VEC || TY == E0_F32) {
                v[i] = __uint_as_float(w[i]);
            } else {
                const float2 f = unpack16<TY>(w[i / 2]);
                v[i] = i % 2 ? f.y : f.x;
            }
            if (VEC && e >= H) v[i] = 0.f;
        }
    }
};
// s = r + d, rounded to the type.
template <int TY>
E0_DEV void add_rounded(float (&v)[8], const float (&w)[8]) {
    if constexpr (TY == E0_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack16<TY>(pack16<TY>(v[2 * i] + w[2 * i], v[2 * i + 1] + w[2 * i + 1]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
}
// All chunks of a thread: loads first, then the sums and their squares.
template <int TY, bool VEC, int CH>
E0_DEV float load_row(const NormArgs& A, size_t row, int c0, int step, float (&v)[CH][8]) {
    typedef typename Elem<TY>::T T;
    const T* r = reinterpret_cast<const T*>(A.r) + row * A.r_ld;
    const T* d = A.d ? reinterpret_cast<const T*>(A.d) + row * A.d_ld : nullptr;
    Chunk<TY, VEC> a[CH], b[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) a[j].load(r, 8 * (c0 + j * step), A.H);
    if (d) {
#pragma unroll
        for (int j = 0; j < CH; ++j) b[j].load(d, 8 * (c0 + j * step), A.H);
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int e = 8 * (c0 + j * step);
        a[j].get(e, A.H, v[j]);
        if (d) {
            float w[8];
            b[j].get(e, A.H, w);
            add_rounded<TY>(v[j], w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
    }
    return ss;
}

template <int TY, bool VEC>
E0_DEV void store_chunk(typename Elem<TY>::T* p, int e, int H, const float (&v)[8]) {
    if constexpr (VEC) {
        if (e < H) store_vec<TY>(p + e, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i < H) p[e + i] = Elem<TY>::put(v[i]);
    }
}

// The larger magnitude (its sign says nothing); NaN where either is.
E0_DEV float max_abs(float a, float b) {
    float r;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Whether the squares' sum has passed fp32's range: a root of infinity, whose inverse is 0
// (that of the largest finite number is 2^-64).
E0_DEV bool sum_overflowed(const NormArgs& A, float rstd) { return rstd == 0.f && (A.h || A.q); }

// A chunk's outputs; all lanes of a warp call it.  Returns whether its group holds a
// value that is not finite.
// h / c = 448 t / max|t| whatever the root is, so the codes come from t = s * w (times
// the root's power of two, exact, which keeps t in h's range): their argument has two
// or three roundings, and a code next to a rounding border hardly ever depends on the
// order of the sum of squares.
template <int TY, bool VEC>
E0_DEV bool finish_chunk(const NormArgs& A, size_t row, int e, float rstd, float (&v)[8]) {
    typedef typename Elem<TY>::T T;
    const int H = A.H;
    const uint32_t bits = __float_as_uint(rstd);
    const float pow2 = rstd != rstd ? rstd : __uint_as_float(bits & 0x7F800000u);
    const float rest = __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u);  // rstd = pow2 * rest
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= pow2;
    if (A.w) {
        if constexpr (VEC) {
            if (e < H) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(A.w + e)), g = __ldg(reinterpret_cast<const float4*>(A.w + e) + 1);
                const float u[8] = {f.x, f.y, f.z, f.w, g.x, g.y, g.z, g.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= u[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e + i < H) v[i] *= __ldg(A.w + e + i);
        }
    }
    if (A.h) {
        float h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = v[i] * rest;
        store_chunk<TY, VEC>(reinterpret_cast<T*>(A.h) + row * H, e, H, h);
    }
    if (!A.q) return false;
    float mx = 0.f;  // NaN where a value is
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (VEC || e + i < H) mx = max_abs(mx, v[i]);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) mx = max_abs(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mx = fabsf(mx);
    const float most = mx * rest;  // max|h|
    const bool bad = !(most < INFINITY) && e < H;
    const bool zero = bad || most < 7.7037198e-34f;  // 2^-110: 448 / mx and most / 448 stay normal numbers
    // 448 / mx as 112 / (mx / 4), whose inverse is a normal number up to the largest mx: an
    // approximate inverse, a first quotient, and Newton's step on the quotient's remainder,
    // which a fused multiply-add gives exactly (Markstein, IBM J. Res. Dev. 34, 1990)
    const float quarter = 0.25f * mx;
    float inv, scale;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(quarter));
    scale = 112.f * inv;
    scale = fmaf(fmaf(-quarter, scale, 112.f), inv, scale);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(v[2 * i] * scale, v[2 * i + 1] * scale);
    if (zero) c[0] = c[1] = c[2] = c[3] = 0;
    uint8_t* q = A.q + row * H;
    if constexpr (VEC) {
        if (e < H) *reinterpret_cast<uint2*>(q + e) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i < H) q[e + i] = (uint8_t)(c[i / 2] >> (8 * (i & 1)));
    }
    if ((threadIdx.x & 7) == 0 && e < H)
        A.qs[row * ((H + GROUP - 1) / GROUP) + e / GROUP] = zero ? 0.f : most * (1.f / 448.f);
    return bad;
}

template <int TY, bool VEC, int CH>
__global__ void __launch_bounds__(512) k_rmsnorm_q8(NormArgs A) {
    typedef typename Elem<TY>::T T;
    __shared__ float red[16];
    const int H = A.H, tid = threadIdx.x, nt = blockDim.x;
    const size_t row = blockIdx.x;
    float v[CH][8];
    float ss = warp_sum(load_row<TY, VEC, CH>(A, row, tid, nt, v));
    if (A.r_out) {
#pragma unroll
        for (int j = 0; j < CH; ++j) store_chunk<TY, VEC>(reinterpret_cast<T*>(A.r_out) + row * H, 8 * (tid + j * nt), H, v[j]);
    }
    if ((tid & 31) == 0) red[tid >> 5] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < nt / 32; ++i) ss += red[i];
    const float rstd = rsqrtf(fmaf(ss, A.inv_h, A.eps));
    bool bad = false;
#pragma unroll
    for (int j = 0; j < CH; ++j) bad |= finish_chunk<TY, VEC>(A, row, 8 * (tid + j * nt), rstd, v[j]);
    if ((bad && (tid & 7) == 0) || (tid == 0 && sum_overflowed(A, rstd))) set_status(A.st, E0_ST_NONFINITE);
}

constexpr int NORM_WARPS = 8;

template <int TY, int CH>
__global__ void __launch_bounds__(NORM_WARPS * 32) k_rmsnorm_q8_rows(NormArgs A) {
    typedef typename Elem<TY>::T T;
    const int H = A.H, lane = threadIdx.x & 31;
    const size_t row = (size_t)blockIdx.x * NORM_WARPS + (threadIdx.x >> 5);
    if (row >= (size_t)A.T) return;
    float v[CH][8];
    const float ss = load_row<TY, true, CH>(A, row, lane, 32, v);
    if (A.r_out) {
#pragma unroll
        for (int j = 0; j < CH; ++j) store_chunk<TY, true>(reinterpret_cast<T*>(A.r_out) + row * H, 8 * (lane + j * 32), H, v[j]);
    }
    const float rstd = rsqrtf(fmaf(warp_sum(ss), A.inv_h, A.eps));
    bool bad = false;
#pragma unroll
    for (int j = 0; j < CH; ++j) bad |= finish_chunk<TY, true>(A, row, 8 * (lane + j * 32), rstd, v[j]);
    if ((bad && (lane & 7) == 0) || (lane == 0 && sum_overflowed(A, rstd))) set_status(A.st, E0_ST_NONFINITE);
}

template <int TY, bool VEC>
int launch(const NormArgs& a, cudaStream_t s) {
    const int T = a.T;
    // Short rows, many of them: a warp a row (4800 rows of 512 bf16: 3.7 us against 4.5
    // with a block a row; 600 rows 2.4 against 2.3; rows of 1024 fp32: 14.8 against 12.5).
    if (VEC && a.H <= 512 && T >= NORM_WARPS * num_sms()) {
        k_rmsnorm_q8_rows<TY, 2><<<(T + NORM_WARPS - 1) / NORM_WARPS, NORM_WARPS * 32, 0, s>>>(a);
        return cudaGetLastError() == cudaSuccess ? E0_OK : E0_ERR_CUDA;
    }
    const int chunks = (a.H + 7) / 8;
    // A chunk a thread; two where there is work for the whole machine and a chunk is 16
    // bytes (16384 rows of 1536 bf16: 28.9 us against 32.4, 2400 rows 4.8 against 5.6,
    // 600 rows 3.0 against 2.7; fp32 gains nothing from it).
    const int two = TY != E0_F32 && (long long)T * a.H >= 1 << 21 ? 2 : 1;
    int nt = ((chunks + two - 1) / two + 31) / 32 * 32;
    if (nt > 512) nt = 512;
    if (chunks <= nt)
        k_rmsnorm_q8<TY, VEC, 1><<<T, nt, 0, s>>>(a);
    else if (chunks <= 2 * nt)
        k_rmsnorm_q8<TY, VEC, 2><<<T, nt, 0, s>>>(a);
    else
        k_rmsnorm_q8<TY, VEC, 4><<<T, nt, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

}  // namespace

int rmsnorm_q8(const void* r, const void* d, const float* w, int T, int H, int dtype, float eps, int64_t r_ld,
               int64_t d_ld, void* r_out, void* h, uint8_t* q, float* qs, uint32_t* st, cudaStream_t s) {
    NormArgs a = {r, d, w, r_out, h, q, qs, st, r_ld, d_ld, T, H, eps, (float)(1.0 / H)};
    const int sz = type_size(dtype);
    uintptr_t bits = (uintptr_t)r | (uintptr_t)d | (uintptr_t)r_out | (uintptr_t)h | (uintptr_t)w | (uintptr_t)(r_ld * sz);
    if (d) bits |= (uintptr_t)(d_ld * sz);
    const bool vec = H % 8 == 0 && !(bits & 15) && !((uintptr_t)q & 7);
    switch (dtype) {
        case E0_F32: return vec ? launch<E0_F32, true>(a, s) : launch<E0_F32, false>(a, s);
        case E0_F16: return vec ? launch<E0_F16, true>(a, s) : launch<E0_F16, false>(a, s);
        default: return vec ? launch<E0_BF16, true>(a, s) : launch<E0_BF16, false>(a, s);
    }
}

}  // namespace e0
