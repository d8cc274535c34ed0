// Norms of queries and keys for each head and their rotation by position, in one pass
// (e0_qk_rope).
#include <cuda_runtime.h>

#include "e0_internal.h"
#include "e0_types.cuh"

namespace e0 {
namespace {

// Pair i of a head turns by the angle a = position * freq[i]:
//     (x0, x1) -> (x0 cos a - x1 sin a, x1 cos a + x0 sin a),
// after h = x / sqrt(mean(x^2) + eps) * w where there is a norm.  A row is read and
// written once, and that bounds the kernel: a head's 16 values a lane (8 pairs) stay in
// registers between the sum of squares and the rotation, the two halves of a lane's pairs
// are a 16-byte vector each whichever way pairs stand, and the angles are found once a
// token, not once a head.
// An angle is needed modulo a turn only, and fp32 has lost it where position * freq is
// large.  So freq / 2 pi is held as a 64-bit fraction of a turn, the product with the
// position is an integer's modulo 2^64, which drops whole turns by itself, and its first
// 32 bits go to the sine: off by less than 2^-22 of a radian at any position.
// The fractions take 64-bit floating point, which this GPU has little of: once a thread
// block, which handles many heads.
constexpr int ROPE_WARPS = 8;
constexpr int MOST_PAIRS = E0_MAX_ROPE_D / 2;
// From here on eps hides what the squares of 256 values lose below fp32's normal numbers (2^-142).  With a smaller one
// the kernel that takes elements one by one looks after them (it has the registers, and nobody's models have such an eps).
constexpr float LEAST_EPS = 0x1p-100f;

struct RopeArgs {
    const void* x;
    void* y;
    const float* freq;
    const uint8_t* axis;
    const float* wq;
    const float* wk;
    const int32_t* pos;
    uint32_t* st;
    int64_t x_ld, y_ld, pos_ld;
    int T, Hq, heads, D, half, axes, per_token, lanes;  // half: pairs that turn; per_token: warps; lanes: of a head
    bool adjacent, norm;
    float eps, inv_d;
};

// Where the pairs 8 item .. 8 item + 7 stand: elements e0.. and e1.. of a head, 8 each.  Adjacent
// pairs are (e0, e0 + 1), ..., then those from e1 on; others (e0, e1), (e0 + 1, e1 + 1), ...
struct Place {
    int e0, e1;
    bool turns;
};
E0_DEV Place place_of(const RopeArgs& A, int item) {
    const int p = 8 * item;
    if (p >= A.half) return {2 * p, 2 * p + 8, false};
    return A.adjacent ? Place{2 * p, 2 * p + 8, true} : Place{p, p + A.half, true};
}

// One pair's elements where vectors do not fit: pair p of D / 2.
E0_DEV void pair_of(const RopeArgs& A, int p, int& a, int& b) {
    const bool apart = p < A.half && !A.adjacent;
    a = apart ? p : 2 * p;
    b = apart ? p + A.half : 2 * p + 1;
}

// t modulo 1, times 2^64.
E0_DEV unsigned long long fraction(double t) {
    return (unsigned long long)(long long)((t - floor(t)) * 9223372036854775808.0) << 1;
}

template <int TY>
struct Raw {
    static constexpr int N = TY == E0_F32 ? 2 : 1;
    uint4 v[N];  // 8 elements
};

// (a0, a1) * (b0, b1) + (c0, c1) and (a0, a1) * (b0, b1), a pair an instruction.
E0_DEV void fma_pair(float& r0, float& r1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
        : "=f"(r0), "=f"(r1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
E0_DEV void mul_pair(float& r0, float& r1, float a0, float a1, float b0, float b1) {
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
        : "=f"(r0), "=f"(r1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

template <int TY>
E0_DEV void to_fp32(const Raw<TY>& r, float (&v)[8]) {
    if constexpr (TY == E0_F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = __uint_as_float(r.v[i].x), v[4 * i + 1] = __uint_as_float(r.v[i].y);
            v[4 * i + 2] = __uint_as_float(r.v[i].z), v[4 * i + 3] = __uint_as_float(r.v[i].w);
        }
    } else {
        const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack16<TY>(w[i]);
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
}

// A head's result is P x + Q x', x' the other element of the pair, with P = w cos and Q = -+ w' sin
// (w' the other's weight): found once for the queries' heads and once for the keys', so that
// a head is a sum of squares and three products a pair of elements.
// VEC: D and twice the pairs that turn are multiples of 16, every row starts on a 16-byte
// boundary, and a norm has an eps of LEAST_EPS or more; otherwise elements come one by one.
// ADJACENT: pairs are neighbours.
//
// Measured (device time, GB300): 16384 rows of 36 heads of 128 bf16, three axes, norms (302 MB):
// 59.1 us, 5.1 TB/s, 75 % of the measured copy rate; what is missing are loads in flight, 24 warps an SM with one head
// ahead each (2.7 of a scheduler's 5.6 warps wait for memory, no pipe is half busy); 64.7 with a block for
// every eight rows, each making the table of turns and the last wave half empty, 87.7 with every lane
// finding its sines, weights and rotation in turn and one value an instruction.  8 rows of 18
// heads of 256: 3.9 us, a launch and two loads behind one another.
template <int TY, bool VEC, bool ADJACENT>
__global__ void __launch_bounds__(ROPE_WARPS * 32, VEC && TY != E0_F32 ? 3 : 2) k_qk_rope(RopeArgs A) {
    typedef typename Elem<TY>::T T;
    __shared__ unsigned long long turn[MOST_PAIRS];
    __shared__ uint8_t axis[MOST_PAIRS];
    __shared__ float2 turned[ROPE_WARPS][MOST_PAIRS];  // a warp's token: cosines and sines
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < A.half; i += ROPE_WARPS * 32) {
        // 1 / 2 pi in two parts, the first of 29 bits: its product with 24 is exact
        const double f = A.freq[i], t = f * 0.15915494272485375, rest = f * 3.6704158172530464e-10;
        turn[i] = fraction(t) + fraction(rest);
        axis[i] = A.axis ? (uint8_t)min((int)A.axis[i], A.axes - 1) : (uint8_t)0;
    }
    __syncthreads();
    const int slots = 32 / A.lanes, item = lane & (A.lanes - 1), items = (A.D + 15) / 16, step = A.per_token * slots;
    const bool live = item < items;
    const Place at = place_of(A, item);
    bool bad = false;
    // (per_token is more than 1 only where T is small: 2^30 at most)
    const int all = A.T * A.per_token;
    for (int w = blockIdx.x * ROPE_WARPS + warp; w < all; w += gridDim.x * ROPE_WARPS) {
        const int t = w / A.per_token;
        if (A.pos[t] < 0) continue;  // no token: the row stays as it is
        const int first = w % A.per_token * slots + lane / A.lanes;
        const T* x = reinterpret_cast<const T*>(A.x) + (size_t)t * A.x_ld;
        T* y = reinterpret_cast<T*>(A.y) + (size_t)t * A.y_ld;
        const auto load = [&](int h, Raw<TY> (&r)[2]) {
            if constexpr (VEC) {
                if (h < A.heads && live) {
                    const uint4* a = reinterpret_cast<const uint4*>(x + (size_t)h * A.D + at.e0);
                    const uint4* b = reinterpret_cast<const uint4*>(x + (size_t)h * A.D + at.e1);
#pragma unroll
                    for (int i = 0; i < Raw<TY>::N; ++i) r[0].v[i] = a[i], r[1].v[i] = b[i];
                }
            }
        };
        Raw<TY> now[2], next[2];
        load(first, now);
        // every angle once a warp
        __syncwarp();
        for (int p = lane; p < A.half; p += 32) {
            const long long pos = A.pos[(size_t)axis[p] * A.pos_ld + t];
            const unsigned long long a = (unsigned long long)pos * turn[p];
            // the nearest turn taken off: -1/2 .. 1/2 of a turn, as half turns
            float sn, cs;
            sincospif((float)(int)(a >> 32) * 4.6566128730773926e-10f, &sn, &cs);
            turned[warp][p] = make_float2(cs, sn);
        }
        __syncwarp();
        float P[2][8], Q[2][8];
        const auto factors = [&](const float* wp) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // the places of a lane's i-th elements, and of their pairs
                float wa = 1.f, wb = 1.f;
                int ea, eb;
                pair_of(A, 8 * item + i, ea, eb);
                const bool in = 8 * item + i < A.D / 2;
                if (wp && in) wa = __ldg(wp + ea), wb = __ldg(wp + eb);
                const float2 f = 8 * item + i < A.half ? turned[warp][8 * item + i] : make_float2(1.f, 0.f);
                const float pa = wa * f.x, qa = -wb * f.y, pb = wb * f.x, qb = wa * f.y;
                if (VEC && (ADJACENT || !at.turns)) {  // neighbours: pair i of 8 is elements 2i, 2i + 1 of 16
                    P[i / 4][2 * (i & 3)] = pa, Q[i / 4][2 * (i & 3)] = qa;
                    P[i / 4][2 * (i & 3) + 1] = pb, Q[i / 4][2 * (i & 3) + 1] = qb;
                } else {
                    P[0][i] = pa, Q[0][i] = qa, P[1][i] = pb, Q[1][i] = qb;
                }
            }
        };
        int have = -1;  // whose factors these are: 0 the queries', 1 the keys'
        for (int h0 = 0; h0 < A.heads; h0 += step) {  // all lanes of a warp take every turn
            const int h = h0 + first;
            const bool mine = h < A.heads && live;
            load(h + step, next);
            const int kind = h < A.Hq ? 0 : 1;
            if (mine && have != kind) {
                factors(!A.norm ? nullptr : kind ? A.wk : A.wq);
                have = kind;
            }
            float a[8], b[8];
            if constexpr (VEC) {
                to_fp32<TY>(now[0], a), to_fp32<TY>(now[1], b);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    int ea, eb;
                    pair_of(A, 8 * item + i, ea, eb);
                    const bool in = mine && 8 * item + i < A.D / 2;
                    a[i] = in ? Elem<TY>::get(x[(size_t)h * A.D + ea]) : 0.f;
                    b[i] = in ? Elem<TY>::get(x[(size_t)h * A.D + eb]) : 0.f;
                }
            }
            if (A.norm) {
                const auto squares = [&]() {
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        fma_pair(s0, s1, a[i], a[i + 1], a[i], a[i + 1], s0, s1);
                        fma_pair(s0, s1, b[i], b[i + 1], b[i], b[i + 1], s0, s1);
                    }
                    float ss = mine ? s0 + s1 : 0.f;
                    for (int o = 1; o < A.lanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    return ss;
                };
                float ss = squares(), eps = A.eps;
                if (!VEC && eps < LEAST_EPS) {  // the squares alone count, and they may be below fp32's normal numbers
                    const float up = ss < 0x1p-100f ? 0x1p100f : 1.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] *= up, b[i] *= up;
                    ss = squares(), eps *= up, eps *= up;
                }
                const float rstd = rsqrtf(fmaf(ss, A.inv_d, eps));
                bad |= mine && !(ss < INFINITY);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    mul_pair(a[i], a[i + 1], a[i], a[i + 1], rstd, rstd);
                    mul_pair(b[i], b[i + 1], b[i], b[i + 1], rstd, rstd);
                }
            }
            float u[8], v[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                // a pair that does not turn has Q = 0, which must not meet an infinity of its partner
                const bool turns = !VEC || at.turns;
                float c0, c1, d0, d1;  // the partners
                if (VEC && ADJACENT) {
                    c0 = a[i + 1], c1 = a[i], d0 = b[i + 1], d1 = b[i];
                } else {
                    c0 = b[i], c1 = b[i + 1], d0 = a[i], d1 = a[i + 1];
                }
                if (turns) {
                    mul_pair(c0, c1, c0, c1, Q[0][i], Q[0][i + 1]);
                    mul_pair(d0, d1, d0, d1, Q[1][i], Q[1][i + 1]);
                } else {
                    c0 = c1 = d0 = d1 = 0.f;
                }
                fma_pair(u[i], u[i + 1], a[i], a[i + 1], P[0][i], P[0][i + 1], c0, c1);
                fma_pair(v[i], v[i + 1], b[i], b[i + 1], P[1][i], P[1][i + 1], d0, d1);
            }
            if (mine) {
                T* to = y + (size_t)h * A.D;
                if constexpr (VEC) {
                    store_vec<TY>(to + at.e0, u);
                    store_vec<TY>(to + at.e1, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        int ea, eb;
                        const int p = 8 * item + i;
                        pair_of(A, p, ea, eb);
                        if (p < A.half) to[ea] = Elem<TY>::put(u[i]), to[eb] = Elem<TY>::put(v[i]);
                        else if (p < A.D / 2) to[ea] = Elem<TY>::put(a[i] * P[0][i]), to[eb] = Elem<TY>::put(b[i] * P[1][i]);
                    }
                }
            }
            now[0] = next[0], now[1] = next[1];
        }
    }
    if (bad && item == 0) set_status(A.st, E0_ST_NONFINITE);
}

template <int TY>
int launch(const RopeArgs& a, bool vec, cudaStream_t s) {
    const long long blocks = ((long long)a.T * a.per_token + ROPE_WARPS - 1) / ROPE_WARPS;
    const long long most = (long long)num_sms() * (vec && TY != E0_F32 ? 3 : 2);
    const auto go = [&](auto kernel) { kernel<<<(unsigned)(blocks < most ? blocks : most), ROPE_WARPS * 32, 0, s>>>(a); };
    if (vec)
        a.adjacent ? go(k_qk_rope<TY, true, true>) : go(k_qk_rope<TY, true, false>);
    else
        a.adjacent ? go(k_qk_rope<TY, false, true>) : go(k_qk_rope<TY, false, false>);
    return cudaGetLastError() == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

}  // namespace

int qk_rope(const void* x, int dtype, int64_t x_ld, int T, int Hq, int Hk, const e0_rope* r, const int32_t* pos,
            int64_t pos_ld, void* y, int64_t y_ld, uint32_t* st, cudaStream_t s) {
    RopeArgs a = {};
    a.x = x, a.y = y, a.freq = r->freq, a.axis = r->axis, a.wq = r->q_norm, a.wk = r->k_norm, a.pos = pos, a.st = st;
    a.x_ld = x_ld, a.y_ld = y_ld, a.pos_ld = pos_ld;
    a.T = T, a.Hq = Hq, a.heads = Hq + Hk, a.D = r->D, a.half = r->rot / 2, a.axes = r->n_axes;
    a.adjacent = r->flags & E0_ROPE_ADJACENT, a.norm = r->flags & E0_QK_NORM;
    a.eps = r->eps, a.inv_d = (float)(1.0 / r->D);
    a.lanes = 1;
    while (16 * a.lanes < r->D) a.lanes *= 2;
    // a warp a token; more of them, down to a head for each of a warp's places, where tokens are few
    const int slots = 32 / a.lanes, most = (a.heads + slots - 1) / slots, want = 16 * num_sms();
    a.per_token = T >= want ? 1 : (want + T - 1) / T;
    if (a.per_token > most) a.per_token = most;
    const int sz = type_size(dtype);
    const uintptr_t bits = (uintptr_t)x | (uintptr_t)y | (uintptr_t)(x_ld * sz) | (uintptr_t)(y_ld * sz);
    const bool vec = r->D % 16 == 0 && r->rot % 16 == 0 && !(bits & 15) && !(a.norm && a.eps < LEAST_EPS);
    switch (dtype) {
        case E0_F32: return launch<E0_F32>(a, vec, s);
        case E0_F16: return launch<E0_F16>(a, vec, s);
        default: return launch<E0_BF16>(a, vec, s);
    }
}

}  // namespace e0
