// Dense int4 group-64 linear layer for decode batches (e0_linear_forward) and
// its weight layout (e0_pack_linear).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "e0_internal.h"
#include "e0_types.cuh"

namespace cg = cooperative_groups;

namespace e0 {
namespace {

// y = W x with w = s q + b per group of 64 inputs, so for a row and a group
//     sum_k w_k x_k = s * sum_k q_k x_k + b * sum_k x_k.
// Both sums run on the tensor cores (16 rows x 8 tokens x 16 inputs a step,
// fp32 accumulation): the codes are the A operand, unpacked in registers, the
// activations the B operand straight from their rows, and sum x is the product
// with a row of ones, which leaves it in the accumulator layout of the first.
// Decode is bound by reading the weights: 4.5 bits each, once.  The layout gives a
// lane its 16 x 64 tile's fragment with one 16-byte load.
//
// Codes as operands.  fp16: the bits 0..15 of a code are the subnormal number
// code * 2^-24, exact, so a code pair costs a mask (and a shift for three of
// four); the scale takes the 2^24.  bf16: 0x4300 | code is 128 + code, less 128.
// Activations: fp16 and bf16 as they are; e4m3 widened to fp16 (exact), its
// scale applied to the group's sums; fp32 as three bf16 parts (8 significant bits
// each, cut off, the sum exact), three products a step.
// Rounding: products are exact in fp32, sums and the scaling are fp32.

constexpr int REC = 576;          // bytes of one 16-row, 64-input record
constexpr int LIN_WARPS = 8;

struct LinArgs {
    const uint8_t* w;
    const void* x;
    const float* xs;
    const void* add;
    void* y;
    int64_t x_ld, add_ld, y_ld;
    int N, K, T, y_type;
    bool vec;
};

E0_DEV void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool bf) {
    if (bf)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One word of a lane's codes -> its A fragment of one step.
template <bool BF>
E0_DEV void unpack_codes(uint32_t w, uint32_t (&a)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t q = (w >> (4 * i)) & 0x000F000Fu;
        if (BF) {
            q |= 0x43004300u;
            const __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&q), __float2bfloat162_rn(128.f));
            q = *reinterpret_cast<const uint32_t*>(&v);
        }
        a[i] = q;
    }
}

// A lane's 16 consecutive inputs of one token and group as B fragments:
// b[p][2i], b[p][2i+1] for step i and part p (fp32 has three, the others one).
template <int XT>
E0_DEV void load_x(const LinArgs& A, int tok, int g, int t4, uint32_t (&b)[XT == E0_F32 ? 3 : 1][8]) {
    constexpr int P = XT == E0_F32 ? 3 : 1;
    if (tok >= A.T) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < 8; ++i) b[p][i] = 0;
        return;
    }
    const size_t at = (size_t)tok * A.x_ld + g * GROUP + 16 * t4;
    if constexpr (XT == E0_E4M3) {
        const uint8_t* x = reinterpret_cast<const uint8_t*>(A.x) + at;
        uint32_t w[4];
        if (A.vec) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(x));
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = x[4 * i] | (x[4 * i + 1] << 8) | (x[4 * i + 2] << 16) | ((uint32_t)x[4 * i + 3] << 24);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[0][2 * i] = e4m3x2_to_half2((uint16_t)w[i]);
            b[0][2 * i + 1] = e4m3x2_to_half2((uint16_t)(w[i] >> 16));
        }
    } else if constexpr (XT == E0_F32) {
        const float* x = reinterpret_cast<const float*>(A.x) + at;
        float v[16];
        if (A.vec) {
            load_vec<E0_F32, 16>(x, v);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = x[i];
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t lo = __float_as_uint(v[2 * i]), hi = __float_as_uint(v[2 * i + 1]);
                b[p][i] = __byte_perm(lo, hi, 0x7632);
                v[2 * i] -= __uint_as_float(lo & 0xFFFF0000u);
                v[2 * i + 1] -= __uint_as_float(hi & 0xFFFF0000u);
            }
    } else {
        const uint16_t* x = reinterpret_cast<const uint16_t*>(A.x) + at;
        if (A.vec) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(x)), v = __ldg(reinterpret_cast<const uint4*>(x) + 1);
            b[0][0] = u.x, b[0][1] = u.y, b[0][2] = u.z, b[0][3] = u.w;
            b[0][4] = v.x, b[0][5] = v.y, b[0][6] = v.z, b[0][7] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) b[0][i] = x[2 * i] | ((uint32_t)x[2 * i + 1] << 16);
        }
    }
}

E0_DEV float get_any(const void* p, int type, size_t i) {
    return type == E0_F32   ? reinterpret_cast<const float*>(p)[i]
           : type == E0_F16 ? __half2float(reinterpret_cast<const __half*>(p)[i])
                            : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}
E0_DEV void put_any(void* p, int type, size_t i, float v) {
    if (type == E0_F32)
        reinterpret_cast<float*>(p)[i] = v;
    else if (type == E0_F16)
        reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
    else
        reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// One block: 16*RM rows, 8*NT tokens, the groups of its share of K (the blocks
// of a cluster share a row tile and split K); its warps take the groups in
// turn.  The warps' sums meet in shared memory and the cluster's in distributed
// shared memory, always in the same order.
template <int XT, int RM, int NT>
__global__ void __launch_bounds__(LIN_WARPS * 32, RM* NT >= 8 ? 1 : 2) k_linear(LinArgs A) {
    constexpr bool BF = XT == E0_F32 || XT == E0_BF16;
    constexpr int P = XT == E0_F32 ? 3 : 1;
    constexpr int COLS = NT * 8, ROWS = RM * 16;
    __shared__ float part[LIN_WARPS][ROWS][COLS + 1];
    __shared__ float sums[ROWS][COLS + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, t4 = lane & 3;
    const int G = A.K / GROUP, S = gridDim.y;
    const int g0 = (int)((long long)blockIdx.y * G / S), g1 = (int)((long long)(blockIdx.y + 1) * G / S);
    const int nb = (A.N + 15) / 16, rb0 = blockIdx.x * RM, tok0 = blockIdx.z * COLS;
    const uint32_t one = BF ? 0x3F803F80u : 0x3C003C00u;
    const uint32_t ones[4] = {one, one, one, one};
    const float up = BF ? 1.f : 16777216.f;  // fp16 codes stand for code * 2^-24

    float tot[RM][NT][4];
#pragma unroll
    for (int r = 0; r < RM; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[r][n][i] = 0.f;

    for (int g = g0 + warp; g < g1; g += LIN_WARPS) {
        uint4 c[RM];
        uint2 sb[RM];
#pragma unroll
        for (int r = 0; r < RM; ++r) {
            const int rb = min(rb0 + r, nb - 1);  // rows beyond the last block are not stored
            const uint8_t* p = A.w + ((size_t)rb * G + g) * REC;
            c[r] = ldg_stream(p + lane * 16);
            sb[r] = __ldg(reinterpret_cast<const uint2*>(p + 512) + gid);
        }
        uint32_t b[NT][P][8];
        float xs[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            load_x<XT>(A, tok0 + n * 8 + gid, g, t4, b[n]);
            if constexpr (XT == E0_E4M3) {
                const int ta = tok0 + n * 8 + 2 * t4;
                xs[n][0] = ta < A.T ? __ldg(A.xs + (size_t)ta * G + g) : 0.f;
                xs[n][1] = ta + 1 < A.T ? __ldg(A.xs + (size_t)(ta + 1) * G + g) : 0.f;
            }
        }
        float sx[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int p = 0; p < P; ++p) mma16(d, ones, b[n][p][2 * i], b[n][p][2 * i + 1], BF);
            sx[n][0] = d[0], sx[n][1] = d[1];
        }
#pragma unroll
        for (int r = 0; r < RM; ++r) {
            float d[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
            const uint32_t cw[4] = {c[r].x, c[r].y, c[r].z, c[r].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a[4];
                unpack_codes<BF>(cw[i], a);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int p = 0; p < P; ++p) mma16(d[n], a, b[n][p][2 * i], b[n][p][2 * i + 1], BF);
            }
            const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&sb[r].x));
            const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&sb[r].y));
            const float s0 = lo.x * up, s1 = hi.x * up;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if constexpr (XT == E0_E4M3) {
                    tot[r][n][0] = fmaf(xs[n][0], fmaf(s0, d[n][0], lo.y * sx[n][0]), tot[r][n][0]);
                    tot[r][n][1] = fmaf(xs[n][1], fmaf(s0, d[n][1], lo.y * sx[n][1]), tot[r][n][1]);
                    tot[r][n][2] = fmaf(xs[n][0], fmaf(s1, d[n][2], hi.y * sx[n][0]), tot[r][n][2]);
                    tot[r][n][3] = fmaf(xs[n][1], fmaf(s1, d[n][3], hi.y * sx[n][1]), tot[r][n][3]);
                } else {
                    tot[r][n][0] += fmaf(s0, d[n][0], lo.y * sx[n][0]);
                    tot[r][n][1] += fmaf(s0, d[n][1], lo.y * sx[n][1]);
                    tot[r][n][2] += fmaf(s1, d[n][2], hi.y * sx[n][0]);
                    tot[r][n][3] += fmaf(s1, d[n][3], hi.y * sx[n][1]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RM; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            part[warp][16 * r + gid][8 * n + 2 * t4] = tot[r][n][0];
            part[warp][16 * r + gid][8 * n + 2 * t4 + 1] = tot[r][n][1];
            part[warp][16 * r + gid + 8][8 * n + 2 * t4] = tot[r][n][2];
            part[warp][16 * r + gid + 8][8 * n + 2 * t4 + 1] = tot[r][n][3];
        }
    __syncthreads();
    const int rank = blockIdx.y;
    for (int e = threadIdx.x; e < ROWS * COLS; e += LIN_WARPS * 32) {
        const int row = e % ROWS, col = e / ROWS;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < LIN_WARPS; ++w) v += part[w][row][col];
        sums[row][col] = v;
    }
    if (S > 1) cg::this_cluster().sync(); else __syncthreads();
    // the blocks of the cluster finish a share of the tile each; rows run
    // along neighbouring threads, so stores to one token's row are coalesced
    for (int e = threadIdx.x + rank * LIN_WARPS * 32; e < ROWS * COLS; e += S * LIN_WARPS * 32) {
        const int row = e % ROWS, col = e / ROWS;
        const int n = rb0 * 16 + row, t = tok0 + col;
        if (n >= A.N || t >= A.T) continue;
        float v = 0.f;
        if (S > 1) {
            for (int k = 0; k < S; ++k) v += cg::this_cluster().map_shared_rank(&sums[0][0], k)[row * (COLS + 1) + col];
        } else {
            v = sums[row][col];
        }
        if (A.add) v += get_any(A.add, A.y_type, (size_t)t * A.add_ld + n);
        put_any(A.y, A.y_type, (size_t)t * A.y_ld + n, v);
    }
    if (S > 1) cg::this_cluster().sync();  // a block's sums are read until here
}

template <int XT, int RM, int NT>
int launch(const LinArgs& a, int S, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.N + 16 * RM - 1) / (16 * RM), S, (a.T + 8 * NT - 1) / (8 * NT));
    cfg.blockDim = dim3(LIN_WARPS * 32);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1, at[0].val.clusterDim.y = S, at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = S > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_linear<XT, RM, NT>, a) == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

template <int XT>
int linear_type(const LinArgs& a, cudaStream_t s) {
    const int sms = num_sms(), G = a.K / GROUP;
    const long long tiles16 = (a.N + 15) / 16;
    const bool wide = tiles16 >= 8LL * sms;
    const int rows = a.T > 8 ? 32 : wide ? 64 : 16;
    const long long tiles = (a.N + rows - 1) / rows;
    int S = 1;
    while (S < 8 && tiles * S < 2LL * sms && G / (2 * S) >= LIN_WARPS / 2) S *= 2;
    if (a.T > 8) return launch<XT, 2, 4>(a, S, s);
    return wide ? launch<XT, 4, 1>(a, S, s) : launch<XT, 1, 1>(a, S, s);
}

// A thread writes one lane's 16 bytes of codes of one record; lanes 0..7 also
// a pair of rows' (scale, bias).
__global__ void k_pack_linear(e0_qtensor src, int N, int K, uint8_t* dst) {
    const int G = K / GROUP, lane = threadIdx.x & 31, gid = lane >> 2, t4 = lane & 3;
    const long long rec = (long long)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
    const long long recs = (long long)((N + 15) / 16) * G;
    if (rec >= recs) return;
    const int rb = (int)(rec / G), g = (int)(rec % G);
    uint8_t* out = dst + rec * REC;
    uint32_t w[4] = {0, 0, 0, 0};
    for (int h = 0; h < 2; ++h) {
        const int n = rb * 16 + gid + 8 * h;
        if (n >= N) continue;
        const uint8_t* c = src.codes + (size_t)n * (K / 2) + g * 32 + 8 * t4;
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = c[2 * i], hi = c[2 * i + 1];  // inputs 4i, 4i+1 and 4i+2, 4i+3
            const uint32_t v = (lo & 15) | ((lo >> 4) << 16) | ((hi & 15) << 8) | ((hi >> 4) << 24);
            w[i] |= v << (4 * h);
        }
    }
    *reinterpret_cast<uint4*>(out + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    if (lane < 8) {
        uint32_t p[2];
        for (int h = 0; h < 2; ++h) {
            const int n = rb * 16 + lane + 8 * h;
            p[h] = n < N ? src.scale[(size_t)n * G + g] | ((uint32_t)src.bias[(size_t)n * G + g] << 16) : 0u;
        }
        reinterpret_cast<uint2*>(out + 512)[lane] = make_uint2(p[0], p[1]);
    }
}

}  // namespace

size_t linear_bytes(int N, int K) { return (size_t)((N + 15) / 16) * (K / GROUP) * REC; }

int pack_linear(const e0_qtensor* src, int N, int K, uint8_t* dst, cudaStream_t s) {
    const long long recs = (long long)((N + 15) / 16) * (K / GROUP);
    k_pack_linear<<<(int)((recs + 7) / 8), 256, 0, s>>>(*src, N, K, dst);
    return cudaGetLastError() == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

int linear_forward(const uint8_t* w, int N, int K, const void* x, int x_type, int64_t x_ld, const float* xs, int T,
                   const void* add, int64_t add_ld, void* y, int y_type, int64_t y_ld, cudaStream_t s) {
    const int sz = type_size(x_type);
    LinArgs a = {w, x, xs, add, y, x_ld, add_ld, y_ld, N, K, T, y_type, false};
    a.vec = !(((uintptr_t)x | (uintptr_t)(x_ld * sz)) & 15);
    switch (x_type) {
        case E0_F32: return linear_type<E0_F32>(a, s);
        case E0_F16: return linear_type<E0_F16>(a, s);
        case E0_BF16: return linear_type<E0_BF16>(a, s);
        default: return linear_type<E0_E4M3>(a, s);
    }
}

}  // namespace e0
