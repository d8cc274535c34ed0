// Dense int4 group-64 linear layer for decode batches (e0_linear_forward) and
// its weight layout (e0_pack_linear).
#include <climits>
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "e0_first.h"
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
// Codes as operands cost a mask and a shift for some.  fp16: a code in the bits
// 0..3 of a half is the subnormal number code * 2^-24, exact, in the bits 4..7 code *
// 2^-20; the layout gives all codes of the lower row the first place and of the
// upper row the second, and the rows' scales take the factors.  bf16: in the bits
// 3..6, with the exponent of 2^-7 set, it is (16 + code) * 2^-11; the product is then
// too large by 16 sum x, which goes into the bias, and all sums stay times 2^-11 until
// they are stored (sum x is formed with 2^-11 in place of ones), so that a group's
// sums, up to 64 * 31 times a value of x, do not pass fp32's range where y does not.
// (In the bits 0..3 it would be 128 + code and the sums' rounding 5 times as large;
// subtracting the 128 again took a third of the instructions.)
// Activations: fp16 and bf16 as they are; e4m3 widened to fp16 (exact), its
// scale applied to the group's sums; fp32 as three bf16 parts (8 significant bits
// each, cut off, the sum exact), three products a step.
// Rounding: products are exact in fp32, sums and the scaling are fp32.
//
// Measured (device time, GB300): 131071 x 2048, 2 rows of bf16, 152 MB: 29.0 us, 5.2
// TB/s, 77 % of the measured copy rate, bound by instructions (70 for a record of 16
// x 64, 52 of them unpacking, products and scaling; the ALU pipe is busy 55 %).
// 8192 x 8192, one row: 11.1 us; 2048 x 2048, one row of e4m3: 3.5 us (a launch
// and two dependent loads).  One row of fp32, three products a step: 46.2 us on the first,
// 16.5 on the second.  32 rows of fp16 on 8192 x 8192: 22.3 us, of which 12 are 32
// records a warp (these products run at 0.5 a clock and SM and take 8 by themselves, and
// 256 blocks, two a SM, leave 24 SMs idle), 6.5 the start, 1 the sums of x and 2.7 the
// cluster's sum.

constexpr int REC = 576;          // bytes of one 16-row, 64-input record
constexpr int SUPER = 8;          // row blocks whose records of a group stand together
constexpr int SREC = SUPER * REC;
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

// The first product of a sum.
E0_DEV void mma16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool bf) {
    if (bf)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// One word of a lane's codes -> its A fragment of one step.
template <bool BF>
E0_DEV void unpack_codes(uint32_t w, uint32_t (&a)[4]) {
    if (BF) {
        const uint32_t v[4] = {w << 3, w >> 1, w >> 5, w >> 9};
#pragma unroll
        for (int i = 0; i < 4; ++i)  // (v & mask) | exponents in one instruction
            asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(a[i]) : "r"(v[i]), "r"(0x00780078u), "r"(0x3C003C00u));
    } else {
        a[0] = w & 0x000F000Fu;
        a[1] = w & 0x00F000F0u;
        a[2] = (w >> 8) & 0x000F000Fu;
        a[3] = (w >> 8) & 0x00F000F0u;
    }
}
// A pair of the values that sum x is the product with, and what sums are turned back with.
template <bool BF>
constexpr uint32_t ONE = BF ? 0x3A003A00u : 0x3C003C00u;  // 2^-11 in bf16, 1 in fp16
template <bool BF>
constexpr float UNIT = BF ? 2048.f : 1.f;
// What the sums are turned with, from the (scale, bias) word of a lower (i) or
// upper (i + 8) row.
template <bool BF, bool UPPER>
E0_DEV float2 scale_bias(uint32_t w) {
    float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    if (BF)
        f.y = fmaf(-16.f, f.x, f.y);
    else
        f.x *= UPPER ? 1048576.f : 16777216.f;
    return f;
}

// A lane's 16 consecutive inputs of one token and group, as they are in memory ...
template <int XT>
struct RawX {
    static constexpr int WORDS = XT == E0_F32 ? 16 : XT == E0_E4M3 ? 4 : 8;
    static constexpr int PARTS = XT == E0_F32 ? 3 : 1;
    uint32_t w[WORDS];
};
template <int XT>
E0_DEV void load_x(const LinArgs& A, int tok, int g, int t4, RawX<XT>& r) {
    constexpr int SZ = XT == E0_F32 ? 4 : XT == E0_E4M3 ? 1 : 2, W = RawX<XT>::WORDS;
    if (tok >= A.T) {
#pragma unroll
        for (int i = 0; i < W; ++i) r.w[i] = 0;
        return;
    }
    const uint8_t* x = reinterpret_cast<const uint8_t*>(A.x) + ((size_t)tok * A.x_ld + g * GROUP + 16 * t4) * SZ;
    if (A.vec) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(x) + i);
            r.w[4 * i] = u.x, r.w[4 * i + 1] = u.y, r.w[4 * i + 2] = u.z, r.w[4 * i + 3] = u.w;
        }
    } else if constexpr (SZ == 4) {
#pragma unroll
        for (int i = 0; i < W; ++i) r.w[i] = reinterpret_cast<const uint32_t*>(x)[i];
    } else if constexpr (SZ == 2) {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(x);
#pragma unroll
        for (int i = 0; i < W; ++i) r.w[i] = h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            r.w[i] = x[4 * i] | (x[4 * i + 1] << 8) | (x[4 * i + 2] << 16) | ((uint32_t)x[4 * i + 3] << 24);
    }
}
// ... and as B fragments: b[p][2i], b[p][2i+1] for step i and part p.
template <int XT>
E0_DEV void fragments(RawX<XT> r, uint32_t (&b)[RawX<XT>::PARTS][8]) {
    if constexpr (XT == E0_E4M3) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[0][2 * i] = e4m3x2_to_half2((uint16_t)r.w[i]);
            b[0][2 * i + 1] = e4m3x2_to_half2((uint16_t)(r.w[i] >> 16));
        }
    } else if constexpr (XT == E0_F32) {
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t lo = r.w[2 * i], hi = r.w[2 * i + 1];
                b[p][i] = __byte_perm(lo, hi, 0x7632);
                r.w[2 * i] = __float_as_uint(__uint_as_float(lo) - __uint_as_float(lo & 0xFFFF0000u));
                r.w[2 * i + 1] = __float_as_uint(__uint_as_float(hi) - __uint_as_float(hi & 0xFFFF0000u));
            }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[0][i] = r.w[i];
    }
}

E0_DEV void copy16(uint8_t* dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
E0_DEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
E0_DEV void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// y[t][n] = v (+ add[t][n]) from the sum in its unit, where there is such a row and token.
template <bool BF>
E0_DEV void store_y(const LinArgs& A, int n, int t, float v) {
    if (n >= A.N || t >= A.T) return;
    v *= UNIT<BF>;
    if (A.add) v += get_any(A.add, A.y_type, (size_t)t * A.add_ld + n);
    put_any(A.y, A.y_type, (size_t)t * A.y_ld + n, v);
}

// A group's share of rows i and i + 8, tokens 2t and 2t + 1: s * sum q x + b * sum x.
template <bool SCALED>
E0_DEV void add_group(float (&tot)[4], const float (&d)[4], float s0, float b0, float s1, float b1, const float* sx,
                      const float* xs) {
    if (SCALED) {
        tot[0] = fmaf(xs[0], fmaf(s0, d[0], b0 * sx[0]), tot[0]);
        tot[1] = fmaf(xs[1], fmaf(s0, d[1], b0 * sx[1]), tot[1]);
        tot[2] = fmaf(xs[0], fmaf(s1, d[2], b1 * sx[0]), tot[2]);
        tot[3] = fmaf(xs[1], fmaf(s1, d[3], b1 * sx[1]), tot[3]);
    } else {
        tot[0] = fmaf(s0, d[0], fmaf(b0, sx[0], tot[0]));
        tot[1] = fmaf(s0, d[1], fmaf(b0, sx[1], tot[1]));
        tot[2] = fmaf(s1, d[2], fmaf(b1, sx[0], tot[2]));
        tot[3] = fmaf(s1, d[3], fmaf(b1, sx[1], tot[3]));
    }
}

// Up to 8 rows of x.  A tile is 16*RM rows of W; the blocks of a cluster share a
// tile and split K, the warps of a block take the groups of its share in turn,
// and a block goes through tiles blockIdx.x, + gridDim.x, ...  A warp's records
// come through its own ring in shared memory, copied STAGES - 1 groups ahead and
// on into the next tile, so the memory is kept busy while a tile's sums meet.
// The warps' sums meet in shared memory and the cluster's in distributed shared
// memory, always in the same order.
template <int RM>
struct VecRing {
    static constexpr int STAGES = RM == 8 ? 2 : RM == 4 ? 3 : 8;
    static constexpr int BYTES = RM * REC;
    static constexpr int SMEM = LIN_WARPS * STAGES * BYTES;
    // the warps' sums, [warp][row][T | 1], and the cluster's
    static int smem(int T, int S) {
        return SMEM + LIN_WARPS * RM * 16 * (T | 1) * 4 + (S > 1 ? RM * 16 * 8 * 4 : 0);
    }
};

template <int XT, int RM>
__global__ void __launch_bounds__(LIN_WARPS * 32, 2) k_linear_vec(LinArgs A) {
    constexpr bool BF = XT == E0_F32 || XT == E0_BF16;
    constexpr int P = RawX<XT>::PARTS, ROWS = RM * 16, STAGES = VecRing<RM>::STAGES;
    extern __shared__ __align__(128) uint8_t lin_sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, t4 = lane & 3;
    uint8_t* ring = lin_sm + warp * STAGES * VecRing<RM>::BYTES;
    float* part = reinterpret_cast<float*>(lin_sm + VecRing<RM>::SMEM);
    const int LD = A.T | 1;
    const int G = A.K / GROUP, S = gridDim.y, rank = blockIdx.y;
    const int g0 = (int)((long long)rank * G / S), g1 = (int)((long long)(rank + 1) * G / S);
    const int nb = (A.N + 15) / 16, tiles = (nb + RM - 1) / RM;
    const uint32_t ones[4] = {ONE<BF>, ONE<BF>, ONE<BF>, ONE<BF>};

    // where the next copy comes from and goes to
    constexpr int PIECES = (RM * 36 + 31) / 32;  // 16-byte pieces of a step that a lane copies
    int in_tile = blockIdx.x, in_g = g0 + warp, in_stage = 0;
    const auto src_of = [&](int tile) {
        const int rb = tile * RM;
        return A.w + ((size_t)(rb / SUPER) * G + g0 + warp) * SREC + (rb % SUPER) * REC + lane * 16;
    };
    const uint8_t* src = src_of(in_tile);
    const auto issue = [&]() {
        if (in_tile < tiles && in_g < g1) {
            uint8_t* dst = ring + in_stage * VecRing<RM>::BYTES + lane * 16;
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                if (i * 32 + 31 < RM * 36 || i * 32 + lane < RM * 36) copy16(dst + i * 512, src + i * 512);
            if (++in_stage == STAGES) in_stage = 0;
            in_g += LIN_WARPS;
            src += LIN_WARPS * SREC;
            if (in_g >= g1) {
                in_g = g0 + warp, in_tile += gridDim.x;
                src = src_of(in_tile);
            }
        }
        copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < STAGES - 1; ++i) issue();

    int stage = 0;
    RawX<XT> raw;  // of the next group
    float nxt[2] = {0.f, 0.f};
    const auto fetch_x = [&](int g) {
        load_x<XT>(A, gid, g, t4, raw);
        if constexpr (XT == E0_E4M3) {
            nxt[0] = 2 * t4 < A.T ? __ldg(A.xs + (size_t)(2 * t4) * G + g) : 0.f;
            nxt[1] = 2 * t4 + 1 < A.T ? __ldg(A.xs + (size_t)(2 * t4 + 1) * G + g) : 0.f;
        }
    };
    if (g0 + warp < g1) fetch_x(g0 + warp);
#pragma unroll 1
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        float tot[RM][4];
#pragma unroll
        for (int r = 0; r < RM; ++r) tot[r][0] = tot[r][1] = tot[r][2] = tot[r][3] = 0.f;
#pragma unroll 1
        for (int g = g0 + warp; g < g1; g += LIN_WARPS) {
            uint32_t b[P][8];
            fragments<XT>(raw, b);
            const float xs[2] = {nxt[0], nxt[1]};
            fetch_x(g + LIN_WARPS < g1 ? g + LIN_WARPS : g0 + warp);
            copy_wait<STAGES - 2>();
            __syncwarp();  // the group has arrived for all lanes, and all have read the one before it
            const uint8_t* rec = ring + stage * VecRing<RM>::BYTES;
            if (++stage == STAGES) stage = 0;
            issue();
            float sx[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    if (i + p == 0)
                        mma16_first(sx, ones, b[0][0], b[0][1], BF);
                    else
                        mma16(sx, ones, b[p][2 * i], b[p][2 * i + 1], BF);
#pragma unroll
            for (int r = 0; r < RM; ++r) {
                const uint4 c = *reinterpret_cast<const uint4*>(rec + r * REC + lane * 16);
                const uint2 sb = *reinterpret_cast<const uint2*>(rec + r * REC + 512 + gid * 8);
                const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
                float d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t a[4];
                    unpack_codes<BF>(cw[i], a);
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        if (i + p == 0)
                            mma16_first(d, a, b[0][0], b[0][1], BF);
                        else
                            mma16(d, a, b[p][2 * i], b[p][2 * i + 1], BF);
                }
                const float2 lo = scale_bias<BF, false>(sb.x), hi = scale_bias<BF, true>(sb.y);
                add_group<XT == E0_E4M3>(tot[r], d, lo.x, lo.y, hi.x, hi.y, sx, xs);
            }
        }
        if (tile != blockIdx.x) __syncthreads();  // the former tile's sums have been read
#pragma unroll
        for (int r = 0; r < RM; ++r) {
            float* o = part + (warp * ROWS + 16 * r + gid) * LD + 2 * t4;
            if (2 * t4 < A.T) o[0] = tot[r][0], o[8 * LD] = tot[r][2];
            if (2 * t4 + 1 < A.T) o[1] = tot[r][1], o[8 * LD + 1] = tot[r][3];
        }
        __syncthreads();
        const auto sum = [&](int row, int col) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < LIN_WARPS; ++w) v += part[(w * ROWS + row) * LD + col];
            return v;
        };
        // rows run along neighbouring threads, so stores to one token's row are coalesced
        if (S == 1) {
            for (int e = threadIdx.x; e < ROWS * A.T; e += LIN_WARPS * 32)
                store_y<BF>(A, tile * ROWS + e % ROWS, e / ROWS, sum(e % ROWS, e / ROWS));
        } else {  // one tile a cluster
            float* sums = part + LIN_WARPS * ROWS * LD;  // [T][ROWS]
            for (int e = threadIdx.x; e < ROWS * A.T; e += LIN_WARPS * 32) sums[e] = sum(e % ROWS, e / ROWS);
            cg::this_cluster().sync();
            // every block finishes a share
            for (int e = threadIdx.x + rank * LIN_WARPS * 32; e < ROWS * A.T; e += S * LIN_WARPS * 32) {
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < S) v += cg::this_cluster().map_shared_rank(sums, k)[e];
                store_y<BF>(A, tile * ROWS + e % ROWS, e / ROWS, v);
            }
            cg::this_cluster().sync();  // a block's sums are read until here
        }
    }
}

// More than 8 rows of x: 16 or 32 of them (TOK) and 128*RM rows of W a block; a warp has
// 16*RM rows and goes through all groups of the block's share of K, its records
// coming through its ring as above.  x comes through shared memory once for the
// block, CHUNK groups at a time, and its sums over groups are formed there; inside
// a chunk warps do not wait for one another.  The blocks of a cluster split K.
template <int XT, int RM, int TOK>
struct BatchSmem {
    static constexpr int STAGES = 4, ROWS = LIN_WARPS * 16 * RM;
    static constexpr int XROW = GROUP * (XT == E0_F32 ? 4 : XT == E0_E4M3 ? 1 : 2);  // bytes
    static constexpr int CHUNK = XT == E0_F32 ? 8 : 16;
    union {
        struct {
            uint8_t rec[LIN_WARPS][STAGES][RM * REC];
            uint8_t x[CHUNK][TOK * XROW];
            float sx[CHUNK][TOK], xs[CHUNK][TOK];
        };
        float sums[TOK][ROWS + 4];  // at the end: the block's own; 4 more so that what the lanes write has 32 banks
    };
};

// 16-byte chunk c of token t's group: chunks of odd tokens change places in pairs,
// so that the eight lanes of a load's phase (two tokens, every second chunk)
// find eight different ones.
template <int XT>
E0_DEV int x_chunk(int t, int c) {
    constexpr int PER = BatchSmem<XT, 1, 16>::XROW / 16;
    return XT == E0_E4M3 ? t * PER + c : t * PER + (c ^ (t & 1));
}

template <int XT, int RM, int TOK>
__global__ void __launch_bounds__(LIN_WARPS * 32, 2) k_linear_batch(LinArgs A) {
    constexpr bool BF = XT == E0_F32 || XT == E0_BF16;
    constexpr int P = RawX<XT>::PARTS, NT = TOK / 8;
    typedef BatchSmem<XT, RM, TOK> SM;
    constexpr int STAGES = SM::STAGES, PER = SM::XROW / 16, SZ = SM::XROW / GROUP, CHUNK = SM::CHUNK;
    extern __shared__ __align__(128) uint8_t lin_sm[];
    SM& M = *reinterpret_cast<SM*>(lin_sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gid = lane >> 2, t4 = lane & 3;
    const int G = A.K / GROUP, S = gridDim.y, rank = blockIdx.y;
    const int g0 = (int)((long long)rank * G / S), g1 = (int)((long long)(rank + 1) * G / S);
    const int nb = (A.N + 15) / 16, rb0 = (blockIdx.x * LIN_WARPS + warp) * RM, tok0 = blockIdx.z * TOK;

    // the thread's 16-byte pieces of a group of x
    constexpr int XPIECES = (TOK * PER + LIN_WARPS * 32 - 1) / (LIN_WARPS * 32);
    const auto stage_x = [&](int g, int n) {
#pragma unroll
        for (int i = 0; i < XPIECES; ++i) {
            const int e = i * LIN_WARPS * 32 + tid, t = e / PER, c = e % PER;
            if (t >= TOK) continue;
            const uint8_t* src = reinterpret_cast<const uint8_t*>(A.x) + ((size_t)(tok0 + t) * A.x_ld + g * GROUP) * SZ + c * 16;
            uint8_t* to = M.x[0] + 16 * x_chunk<XT>(t, c);
            for (int k = 0; k < n; ++k, src += GROUP * SZ, to += TOK * SM::XROW) {
                if (tok0 + t >= A.T) {
                    *reinterpret_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
                } else if (A.vec) {
                    copy16(to, src);
                } else {
                    for (int b = 0; b < 16; b += SZ) {
                        if (SZ == 4) *reinterpret_cast<uint32_t*>(to + b) = *reinterpret_cast<const uint32_t*>(src + b);
                        if (SZ == 2) *reinterpret_cast<uint16_t*>(to + b) = *reinterpret_cast<const uint16_t*>(src + b);
                        if (SZ == 1) to[b] = src[b];
                    }
                }
            }
        }
        copy_commit();
    };
    // the lane's 16-byte pieces of a group of its warp's records
    constexpr int PIECES = (RM * 36 + 31) / 32;
    static_assert(SUPER % RM == 0, "a warp's records of a group stand together");
    const uint8_t* src = A.w + ((size_t)(rb0 / SUPER) * G + g0) * SREC + (rb0 % SUPER) * REC + lane * 16;
    const bool mine = rb0 < nb;
    int in_stage = 0;
    const auto issue = [&](int g) {
        if (mine && g < g1) {
            uint8_t* dst = M.rec[warp][in_stage] + lane * 16;
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                if (i * 32 + 31 < RM * 36 || i * 32 + lane < RM * 36) copy16(dst + i * 512, src + i * 512);
            src += SREC;
        }
        if (++in_stage == STAGES) in_stage = 0;
        copy_commit();
    };
    const auto fragments_of = [&](const uint8_t* x, int n, uint32_t (&b)[P][8]) {
        RawX<XT> r;
#pragma unroll
        for (int i = 0; i < RawX<XT>::WORDS / 4; ++i) {
            const uint4 u = *reinterpret_cast<const uint4*>(x + 16 * x_chunk<XT>(8 * n + gid, RawX<XT>::WORDS / 4 * t4 + i));
            r.w[4 * i] = u.x, r.w[4 * i + 1] = u.y, r.w[4 * i + 2] = u.z, r.w[4 * i + 3] = u.w;
        }
        fragments<XT>(r, b);
    };
    // sums over a group of 8 tokens' inputs
    const auto sum_x = [&](int g, int k, int n) {
        const uint32_t ones[4] = {ONE<BF>, ONE<BF>, ONE<BF>, ONE<BF>};
        uint32_t b[P][8];
        fragments_of(M.x[k], n, b);
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int p = 0; p < P; ++p) mma16(d, ones, b[p][2 * i], b[p][2 * i + 1], BF);
        if (gid == 0) {
            const int t = 8 * n + 2 * t4;
            *reinterpret_cast<float2*>(&M.sx[k][t]) = make_float2(d[0], d[1]);
            if constexpr (XT == E0_E4M3) {
                M.xs[k][t] = tok0 + t < A.T ? __ldg(A.xs + (size_t)(tok0 + t) * G + g) : 0.f;
                M.xs[k][t + 1] = tok0 + t + 1 < A.T ? __ldg(A.xs + (size_t)(tok0 + t + 1) * G + g) : 0.f;
            }
        }
    };

    float tot[RM][NT][4];
#pragma unroll
    for (int r = 0; r < RM; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) tot[r][n][0] = tot[r][n][1] = tot[r][n][2] = tot[r][n][3] = 0.f;
    int stage = 0;
#pragma unroll 1
    for (int c0 = g0; c0 < g1; c0 += CHUNK) {
        const int n_g = min(CHUNK, g1 - c0);
        if (c0 > g0) __syncthreads();  // the last chunk has been read
        stage_x(c0, n_g);
        if (c0 == g0) {
#pragma unroll 1
            for (int i = 0; i < STAGES - 1; ++i) issue(g0 + i);
            copy_wait<STAGES - 1>();
        } else {
            copy_wait<0>();
        }
        __syncthreads();
#pragma unroll 1
        for (int i = warp; i < n_g * NT; i += LIN_WARPS) sum_x(c0 + i / NT, i / NT, i % NT);
        __syncthreads();
#pragma unroll 1
        for (int k = 0; k < n_g; ++k) {
            copy_wait<STAGES - 2>();
            __syncwarp();  // the group has arrived for all lanes, and all have read the one before it
            const uint8_t* recs = M.rec[warp][stage];
            if (++stage == STAGES) stage = 0;
            issue(c0 + k + STAGES - 1);
            const uint8_t* x = M.x[k];
            uint32_t b[P == 1 ? NT : 1][P][8];  // one part: all tiles' operands stay for the rows to come
            if constexpr (P == 1) {
#pragma unroll
                for (int n = 0; n < NT; ++n) fragments_of(x, n, b[n]);
            }
#pragma unroll
            for (int r = 0; r < RM; ++r) {
                const uint8_t* rec = recs + r * REC;
                const uint4 c = *reinterpret_cast<const uint4*>(rec + lane * 16);
                const uint2 sb = *reinterpret_cast<const uint2*>(rec + 512 + gid * 8);
                const float2 lo = scale_bias<BF, false>(sb.x), hi = scale_bias<BF, true>(sb.y);
                const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
                float d[NT][4];
                if constexpr (P == 1) {  // NT chains of products at once
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t a[4];
                        unpack_codes<BF>(cw[i], a);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            if (i == 0)
                                mma16_first(d[n], a, b[n][0][0], b[n][0][1], BF);
                            else
                                mma16(d[n], a, b[n][0][2 * i], b[n][0][2 * i + 1], BF);
                    }
                } else {
                    uint32_t a[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) unpack_codes<BF>(cw[i], a[i]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        fragments_of(x, n, b[0]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int p = 0; p < P; ++p)
                                if (i + p == 0)
                                    mma16_first(d[n], a[0], b[0][0][0], b[0][0][1], BF);
                                else
                                    mma16(d[n], a[i], b[0][p][2 * i], b[0][p][2 * i + 1], BF);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float2 sx2 = *reinterpret_cast<const float2*>(&M.sx[k][8 * n + 2 * t4]);
                    const float sx[2] = {sx2.x, sx2.y};
                    float xs[2] = {1.f, 1.f};
                    if constexpr (XT == E0_E4M3) {
                        const float2 x2 = *reinterpret_cast<const float2*>(&M.xs[k][8 * n + 2 * t4]);
                        xs[0] = x2.x, xs[1] = x2.y;
                    }
                    add_group<XT == E0_E4M3>(tot[r][n], d[n], lo.x, lo.y, hi.x, hi.y, sx, xs);
                }
            }
        }
    }
    copy_wait<0>();
    __syncthreads();  // all warps are through: the sums stand where x and the records were
#pragma unroll
    for (int r = 0; r < RM; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float* o = &M.sums[8 * n + 2 * t4][(warp * RM + r) * 16 + gid];
            o[0] = tot[r][n][0], o[SM::ROWS + 4] = tot[r][n][1], o[8] = tot[r][n][2], o[SM::ROWS + 12] = tot[r][n][3];
        }
    if (S > 1) cg::this_cluster().sync(); else __syncthreads();
    // every block finishes some of the tokens; four rows a thread
    const int t_end = (rank + 1) * TOK / S;
    for (int i = tid;; i += LIN_WARPS * 32) {
        const int t = rank * TOK / S + i / (SM::ROWS / 4), row = i % (SM::ROWS / 4) * 4;
        if (t >= t_end) break;
        if (tok0 + t >= A.T) break;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < S) {
                const float* from = S > 1 ? cg::this_cluster().map_shared_rank(&M.sums[0][0], k) : &M.sums[0][0];
                const float4 x = *reinterpret_cast<const float4*>(from + t * (SM::ROWS + 4) + row);
                v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
        const int n = blockIdx.x * SM::ROWS + row;
        store_y<BF>(A, n, tok0 + t, v.x);
        store_y<BF>(A, n + 1, tok0 + t, v.y);
        store_y<BF>(A, n + 2, tok0 + t, v.z);
        store_y<BF>(A, n + 3, tok0 + t, v.w);
    }
    if (S > 1) cg::this_cluster().sync();  // a block's sums are read until here
}

void cluster_launch(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* at, dim3 grid, size_t smem, cudaStream_t s) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(LIN_WARPS * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1, at[0].val.clusterDim.y = grid.y, at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = grid.y > 1 ? 1 : 0;
}

// Clusters of S blocks that the current device, dev, holds at once.  The order of y's
// sums depends on it, so the first answer stays.
template <void (*kernel)(LinArgs)>
int room(int dev, int S, size_t smem) {
    static FirstAnswer<9> known;
    return known.get(dev, S, 2 * num_sms() / S, [&]() {
        const cudaError_t before = cudaPeekAtLastError();
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute at[1];
        cluster_launch(cfg, at, dim3(1, S), smem, 0);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) return n;
        if (before == cudaSuccess) cudaGetLastError();  // an error of this question, not of the call
        return 0;
    });
}

// most: the most dynamic shared memory that any launch of the kernel wants.
template <void (*kernel)(LinArgs)>
bool prepare(size_t most) {
    static std::atomic<uint64_t> asked{0};
    return allow_smem((const void*)kernel, most, asked);
}

template <void (*kernel)(LinArgs)>
int launch(const LinArgs& a, dim3 grid, size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cluster_launch(cfg, at, grid, smem, s);
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

// Blocks of a cluster, which split K, for as many tiles: as few groups one after another
// as can be, with a block's start and end counted as START groups (a few microseconds;
// without, 16 rows on 80000 x 2048, 313 tiles, take 72 us instead of 36), and at least
// four groups a block. Clusters that do not find room at once wait for others to end (16
// rows on 10240 x 2560, 40 tiles: 12.3 us with 3 blocks each, 14.7 with 8, 16.1 with 7; 40
// on 7168 x 2048: 13.2 with 5, 17.9 with 8; both in tiles of 32 rows).
template <void (*kernel)(LinArgs)>
int split_of(long long tiles, int G, size_t smem) {
    constexpr int START = 12;
    int best = 1, dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
    long long least = LLONG_MAX;
    for (int S = 1; S <= 8 && (S == 1 || G / S >= 4); ++S) {
        const long long n = room<kernel>(dev, S, smem), groups = (tiles + n - 1) / n * ((G + S - 1) / S + START);
        if (groups < least) least = groups, best = S;
    }
    return best;
}

template <int XT, int RM>
int launch_vec(const LinArgs& a, dim3 grid, cudaStream_t s) {
    if (!prepare<k_linear_vec<XT, RM>>(VecRing<RM>::smem(8, 2))) return E0_ERR_CUDA;
    return launch<k_linear_vec<XT, RM>>(a, grid, VecRing<RM>::smem(a.T, grid.y), s);
}

template <int XT, int TOK>
int linear_batch(const LinArgs& a, int nb, int G, int sms, cudaStream_t s) {
    // two row blocks a warp share the operands of x (8192 x 8192: 22.3 us, 29.8 with
    // one); one where two would leave SMs with no block or most of them with one (32
    // rows on 4096 x 4096: 10.5 us with one, 14.3 with two; 5120 x 5120: 14.3 and 16.7)
    const int zs = (a.T + TOK - 1) / TOK;
    const auto tiles = [&](int rm) { return (nb + LIN_WARPS * rm - 1) / (LIN_WARPS * rm); };
    constexpr size_t sm1 = sizeof(BatchSmem<XT, 1, TOK>), sm2 = sizeof(BatchSmem<XT, 2, TOK>);
    if (!prepare<k_linear_batch<XT, 1, TOK>>(sm1) || !prepare<k_linear_batch<XT, 2, TOK>>(sm2)) return E0_ERR_CUDA;
    const int s2 = split_of<k_linear_batch<XT, 2, TOK>>((long long)tiles(2) * zs, G, sm2);
    if ((long long)tiles(2) * zs * s2 * 4 >= 5LL * sms)
        return launch<k_linear_batch<XT, 2, TOK>>(a, dim3(tiles(2), s2, zs), sm2, s);
    const int s1 = split_of<k_linear_batch<XT, 1, TOK>>((long long)tiles(1) * zs, G, sm1);
    return launch<k_linear_batch<XT, 1, TOK>>(a, dim3(tiles(1), s1, zs), sm1, s);
}

template <int XT>
int linear_type(const LinArgs& a, cudaStream_t s) {
    const int sms = num_sms(), G = a.K / GROUP, nb = (a.N + 15) / 16;
    // A tile of 16 rows takes two thirds of one of 32 (16 rows of fp16 on 8192 x 8192: 14.9 us
    // and 20.6), so one of 16 is better than one of 32, and three than two (48 rows of
    // bf16: 34.4 us and 40.3).
    if (a.T > 8) {
        const bool small = a.T <= 16 || (a.T > 32 && a.T <= 48);
        return small ? linear_batch<XT, 16>(a, nb, G, sms, s) : linear_batch<XT, 32>(a, nb, G, sms, s);
    }
    // The more row blocks a warp has, the less the operands of x cost (131071 x 2048:
    // 37 us with 4, 29 with 8; 8192 x 8192: 19.5 with 1, 11.1 with 8); but there
    // have to be blocks for the whole machine, with K split over up to 8 of them.
    // That costs a cluster's sum: single row blocks are split where a warp keeps four
    // groups of K (2048 x 2048, one row: 3.5 us whole, 4.2 in halves; 512 x 8192: 5.3
    // in halves, 4.3 in quarters), more of them from one and a half on (10240 x 2560: 6.5 us
    // in threes of 8, 8.0 as single ones).
    const auto split = [&](int rm) {
        const int tiles = (nb + rm - 1) / rm, most = rm == 1 ? G / (4 * LIN_WARPS) : G * 2 / (3 * LIN_WARPS);
        return max(1, min(min(8, most), 2 * sms / tiles));
    };
    const auto fills = [&](int rm) { return (long long)((nb + rm - 1) / rm) * split(rm) * 4 >= 5LL * sms; };
    const auto grid = [&](int rm) {
        const int tiles = (nb + rm - 1) / rm, S = split(rm);
        return dim3(S == 1 && tiles > 2 * sms ? 2 * sms : tiles, S);
    };
    if (fills(8)) return launch_vec<XT, 8>(a, grid(8), s);
    if (fills(4)) return launch_vec<XT, 4>(a, grid(4), s);
    return launch_vec<XT, 1>(a, grid(1), s);
}

// A thread writes one lane's 16 bytes of codes of one record; lanes 0..7 also
// a pair of rows' (scale, bias).
__global__ void k_pack_linear(e0_qtensor src, int N, int K, uint8_t* dst) {
    const int G = K / GROUP, lane = threadIdx.x & 31, gid = lane >> 2, t4 = lane & 3;
    const long long rec = (long long)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
    const long long recs = (long long)((N + 16 * SUPER - 1) / (16 * SUPER)) * SUPER * G;
    if (rec >= recs) return;
    const int g = (int)(rec / SUPER % G), rb = (int)(rec / SUPER / G) * SUPER + (int)(rec % SUPER);
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

size_t linear_bytes(int N, int K) { return (size_t)((N + 16 * SUPER - 1) / (16 * SUPER)) * (K / GROUP) * SREC; }

int pack_linear(const e0_qtensor* src, int N, int K, uint8_t* dst, cudaStream_t s) {
    const long long recs = (long long)(linear_bytes(N, K) / REC);
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
