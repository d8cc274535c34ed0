// Attention of decode queries over the paged 8-bit KV cache (e0_attn_decode).
#include <cuda_runtime.h>

#include "e0_internal.h"
#include "e0_types.cuh"

namespace e0 {
namespace {

// out = softmax(scale q K^T) V in one pass over the context with the running
// maximum and sum.  A job is one (sequence, KV head, 8 query rows): the rows are
// the query heads of the group and the sequence's new tokens, token major.  A
// job's context is cut into units, and the units of all jobs, one after another,
// are dealt out evenly to the thread blocks: every block reads the same number
// of bytes whatever the lengths are.  A job that ends up on several blocks
// leaves one partial result (maximum, sum, unscaled output) on each, at most two
// a block, and k_attn_join adds them in order.
//
// A unit is one step of each of a block's warps.  Products run on the tensor
// cores (16 x 8 x 16, fp16 operands, fp32 accumulation); e4m3 codes widen to fp16
// exactly.  The 16 operand rows hold the 8 query rows twice: rows 0..7 the fp16
// part, rows 8..15 the rest of the value, so neither q nor the probabilities
// lose bits that matter (22 significant bits), at no cost: a decode step has few
// rows and the kernel is bound by reading the cache.
// A warp's codes come through its own ring in shared memory, copied some steps
// ahead, so warps never wait for one another inside a job.  Operand layouts are
// chosen so that every lane reads 16 bytes at a time: the order of D inside the
// first product and of the output columns in the second are permuted (the same
// permutation on both operands).
// The scale of a block of keys multiplies the scores; that of the values goes into
// the exponent: with t_j = score_j + log2(scale_j) and m the running maximum of
// t, the weights of the codes are 2^(t_j - m + 15), which fills fp16's range
// whatever the scales are (the rest of a weight goes in times 2^12, so weights down
// to 2^-51 of the largest count), and the softmax's sum is that of the weights
// over their scales.

constexpr int ROWS = 8;
constexpr int AT_WARPS = 4;

// SUBS: 16-position pieces (the smallest block) of a warp's step.  A step costs a
// chain of dependent instructions (products, maximum, exponentials, products)
// whatever its length, so it is as long as registers and the ring allow.
// STAGES: steps a warp's ring holds; all but one are under way.
template <int D>
struct Tile {
    static constexpr int SUBS = D == 256 ? 1 : 2;
    static constexpr int STEP = 16 * SUBS;
    static constexpr int UNIT = AT_WARPS * STEP;
    static constexpr int STAGES = D == 64 ? 5 : 3;
    static constexpr int BYTES = 2 * STEP * D;  // keys, then values
};

// What a block that starts a job which goes on in the next ones leaves for the join.
struct Cut {
    int parts;  // 0: nothing
    int row0, tile, head, rows;
};

struct AttnArgs {
    const uint8_t* k;
    const uint8_t* v;
    const float* ks;
    const float* vs;
    const int32_t* table;
    const int32_t* ctx;
    const int32_t* cu;
    const void* q;
    void* out;
    float* lse;
    float* part_o;    // [2 * blocks][ROWS][D]
    float2* part_ml;  // [2 * blocks][ROWS]
    Cut* cuts;        // [blocks]
    uint32_t* st;
    int64_t q_ld, out_ld;
    int B, max_blocks, n_blocks, shift, Hq, Hkv, max_q, window, blocks, unit;
    float scale;
};

// One sequence as the schedule sees it.
struct Seq {
    int row0, n, ctx, first;  // first query row, queries, cached tokens, first unit that anyone sees
    int units, tiles;         // units of context, tiles of 8 rows per KV head
    int low;                  // the first position that the first query sees
};

E0_DEV Seq seq_of(const AttnArgs& A, int b, bool tell) {
    Seq s;
    s.row0 = A.cu ? A.cu[b] : b;
    s.n = A.cu ? A.cu[b + 1] - s.row0 : 1;
    s.ctx = A.ctx[b];
    bool bad = false;
    if (s.row0 < 0 || s.n < 0 || s.n > A.max_q) bad = true, s.n = 0;
    if (s.ctx < 0 || (long long)s.ctx > ((long long)A.max_blocks << A.shift)) bad = true, s.ctx = 0;
    if (bad && tell) set_status(A.st, E0_ST_BAD_LENGTH);
    s.low = A.window > 0 ? max(s.ctx - s.n + 1 - A.window, 0) : 0;
    s.first = s.low / A.unit;
    s.units = (int)(((long long)s.ctx + A.unit - 1) / A.unit) - s.first;
    if (s.units < 1) s.units = 1;  // a job without context still writes its rows
    const int G = A.Hq / A.Hkv;
    s.tiles = (int)(((long long)s.n * G + ROWS - 1) / ROWS);
    return s;
}

// First unit of every sequence's jobs, in shared memory; the total.
E0_DEV long long schedule(const AttnArgs& A, long long* first, long long* red, bool tell) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int per = (A.B + blockDim.x - 1) / blockDim.x, b0 = threadIdx.x * per;
    long long sum = 0;
    for (int i = 0; i < per && b0 + i < A.B; ++i) {
        const Seq s = seq_of(A, b0 + i, tell);
        first[b0 + i] = sum;  // from the thread's own first sequence on, for now
        sum += (long long)s.units * s.tiles * A.Hkv;
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) red[warp] = inc;
    __syncthreads();
    long long base = 0, total = 0;
    for (int i = 0; i < nw; ++i) {
        if (i < warp) base += red[i];
        total += red[i];
    }
    for (int i = 0; i < per && b0 + i < A.B; ++i) first[b0 + i] += base + inc - sum;
    if (threadIdx.x == 0) first[A.B] = total;
    __syncthreads();
    return total;
}

// Units of a block: the same for all, at least 2 (a join costs more than a unit).
E0_DEV long long units_per_block(const AttnArgs& A, long long total) {
    const long long per = (total + A.blocks - 1) / A.blocks;
    return per < 2 ? 2 : per;
}

struct Job {
    Seq s;
    int head, tile;
    long long first;  // its first unit among all
    int seq;
};

E0_DEV Job job_at(const AttnArgs& A, const long long* first, long long unit) {
    int lo = 0, hi = A.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= unit) lo = mid; else hi = mid;
    }
    Job j;
    j.seq = lo;
    j.s = seq_of(A, lo, false);
    const int k = (int)((unit - first[lo]) / j.s.units);
    j.head = k / j.s.tiles;
    j.tile = k % j.s.tiles;
    j.first = first[lo] + (long long)k * j.s.units;
    return j;
}

// a's and b's codes at byte (sel & 3) as an fp16 pair: interleave, widen.
E0_DEV uint32_t widen_pair(uint32_t a, uint32_t b, int byte) {
    uint32_t p;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(p) : "r"(a), "r"(b), "r"(0x40u + 0x11u * byte));
    return e4m3x2_to_half2((uint16_t)p);
}
// NaN codes (0x7F, 0xFF) of a word -> 0.
E0_DEV uint32_t without_nan(uint32_t w) {
    const uint32_t m = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // bit 7 where the code is NaN
    return w & ~(m | (m - (m >> 7)));
}
E0_DEV float exp2_of(float x) {  // 2 ulp; results below 2^-126 are 0
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

E0_DEV void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

E0_DEV uint32_t half2_of(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// The fp16 part of a pair and what it leaves, times `up`.
E0_DEV void split_half(float a, float b, uint32_t& hi, uint32_t& lo, float up = 1.f) {
    const __half2 h = __floats2half2_rn(a, b);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const float2 f = __half22float2(h);
    lo = half2_of((a - f.x) * up, (b - f.y) * up);
}

E0_DEV float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
E0_DEV float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float LEAST_SCALE = 7.8886090522101181e-31f;  // 2^-100, the least that e0_kv_append writes
constexpr float LIFT = 15.f;                            // the largest weight is 2^LIFT
constexpr float REST = 4096.f;                          // what the rests of the weights go in times

template <int D>
struct AttnSmem {
    uint8_t ring[AT_WARPS][Tile<D>::STAGES][Tile<D>::BYTES];  // a warp's output at the end of a job
    uint32_t q[D / 16][32][4];
    float4 scales[AT_WARPS][Tile<D>::STAGES][2];  // of a piece: keys' scale (< 0: not seen), values' log2 and inverse
    float m[AT_WARPS][ROWS], l[AT_WARPS][ROWS];
    float f[ROWS];
    long long red[AT_WARPS];
};

template <int D>
E0_DEV float* warp_out(AttnSmem<D>& S, int w) {  // [ROWS][D + 4]
    static_assert(sizeof(S.ring[0]) >= ROWS * (D + 4) * sizeof(float), "the ring holds a warp's output");
    return reinterpret_cast<float*>(S.ring[w]);
}

// Where the 16-byte chunk c of row r of a step's keys or values stands: chunks
// are permuted inside 128 bytes so that the eight lanes of a load's phase, which
// read four chunks of two key rows, or two chunks of four value rows, find
// eight different ones.
template <int D>
E0_DEV int key_chunk(int r, int c) {
    return D == 64 ? r * 4 + c : r * (D / 16) + (c ^ (((r & 1) << 2) | ((r >> 1) & 3)));
}
template <int D>
E0_DEV int value_chunk(int r, int c) {
    return D == 64 ? ((r * 4 + c) ^ (r & 6)) : r * (D / 16) + (c ^ (r & 6));
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

template <int TY>
E0_DEV void store_out(const AttnArgs& A, size_t row, int i, float v) {
    typedef typename Elem<TY>::T T;
    reinterpret_cast<T*>(A.out)[row * A.out_ld + i] = Elem<TY>::put(v);
}

template <int D, int TY>
__global__ void __launch_bounds__(AT_WARPS * 32) k_attn(AttnArgs A) {
    typedef typename Elem<TY>::T T;
    extern __shared__ __align__(16) char attn_sm[];
    AttnSmem<D>& S = *reinterpret_cast<AttnSmem<D>*>(attn_sm);
    long long* first = reinterpret_cast<long long*>(attn_sm + sizeof(AttnSmem<D>));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, t4 = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long total = schedule(A, first, S.red, blockIdx.x == 0);
    const long long per = units_per_block(A, total);
    long long u = blockIdx.x * per;
    const long long u1 = u + per < total ? u + per : total;
    const int G = A.Hq / A.Hkv, bs = 1 << A.shift;
    constexpr int KC = D / 64;          // 16-byte chunks of a key row a lane reads
    constexpr int NT = D / 8;           // output tiles
    constexpr int VC = D >= 128 ? D / 128 : 1;  // 16-byte chunks of a value row
    constexpr int SUBS = Tile<D>::SUBS, STEP = Tile<D>::STEP, UNIT = Tile<D>::UNIT, STAGES = Tile<D>::STAGES;
    constexpr int AHEAD = 32 / SUBS;    // steps whose block ids the lanes hold
    Cut cut = {0, 0, 0, 0, 0};

    while (u < u1) {
        const Job j = job_at(A, first, u);
        const int c0 = (int)(u - j.first);
        const int c1 = (int)(min(j.first + j.s.units, u1) - j.first);
        const int rr = j.tile * ROWS + gid;  // this lane's query row
        const bool row_ok = rr < j.s.n * G;
        const int qi = rr / G;
        const int hq = j.head * G + rr % G;
        const int last = j.s.ctx - j.s.n + qi;  // the last position that the row sees
        const int low = A.window > 0 ? last - A.window + 1 : 0;
        // what every row of the tile sees
        const int last_all = j.s.ctx - j.s.n + j.tile * ROWS / G;
        const int low_all = A.window > 0 ? j.s.ctx - A.window : 0;
        __syncthreads();  // the former job's shared memory has been read

        // block ids and scales of the next pieces, one a lane
        int my_id = -1;
        float4 my_sc = make_float4(-1.f, 0.f, 0.f, 0.f);
        const auto look_up = [&](int c) {
            const int cc = c + lane / SUBS, pos = (j.s.first + cc) * UNIT + STEP * warp + 16 * (lane % SUBS);
            my_id = -1;
            my_sc = make_float4(-1.f, 0.f, 0.f, 0.f);
            if (cc < c1 && pos < j.s.ctx && pos + 16 > j.s.low) {
                my_id = A.table[(size_t)j.seq * A.max_blocks + (pos >> A.shift)];
                if (my_id >= 0 && my_id < A.n_blocks) {
                    const size_t i = (size_t)my_id * A.Hkv + j.head;
                    const float v = fmaxf(A.vs[i], LEAST_SCALE);
                    my_sc = make_float4(A.ks[i], log2f(v), 1.f / v, 0.f);
                } else {
                    my_id = -1;
                    set_status(A.st, E0_ST_BAD_BLOCK);
                }
            }
        };
        int in_stage = 0, in_at = 0;  // where the next copy goes; its place among the lanes' ids
        const auto issue = [&](int c) {
            if (c < c1) {
                if (in_at == 0) look_up(c);
#pragma unroll
                for (int h = 0; h < SUBS; ++h) {
                    const int from = in_at * SUBS + h;
                    const int id = __shfl_sync(0xffffffffu, my_id, from);
                    if (lane == from) S.scales[warp][in_stage][h] = my_sc;
                    if (id >= 0) {
                        const int pos = (j.s.first + c) * UNIT + STEP * warp + 16 * h;
                        const size_t at = ((((size_t)id * A.Hkv + j.head) << A.shift) + (pos & (bs - 1))) * D + 16 * lane;
                        uint8_t* dst = S.ring[warp][in_stage] + h * 16 * D;
#pragma unroll
                        for (int i = 0; i < D / 32; ++i) {
                            const int r = (i * 32 + lane) / (D / 16), ch = (i * 32 + lane) % (D / 16);
                            copy16(dst + 16 * key_chunk<D>(r, ch), A.k + at + 512 * i);
                            copy16(dst + STEP * D + 16 * value_chunk<D>(r, ch), A.v + at + 512 * i);
                        }
                    }
                }
                if (++in_at == AHEAD) in_at = 0;
                if (++in_stage == STAGES) in_stage = 0;
            }
            copy_commit();
        };
        for (int i = 0; i < STAGES - 1; ++i) issue(c0 + i);

        // ---- the job's queries as operand fragments: warps share them through shared memory
        if (warp == 0) {
            float x[KC][16];
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                if (row_ok) {
                    load_vec<TY, 16>(reinterpret_cast<const T*>(A.q) + (size_t)(j.s.row0 + qi) * A.q_ld + (size_t)hq * D +
                                         64 * c + 16 * t4, x[c]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[c][i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[c][i]) & 0x7FFFFFFFu);
            }
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            // rows go in times a power of two that brings the largest near 1
            int e = (int)(m >> 23);
            e = e < 27 ? 27 : e > 253 ? 253 : e;
            const float down = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t a[4];
                    split_half(x[c][4 * i] * down, x[c][4 * i + 1] * down, a[0], a[1]);
                    split_half(x[c][4 * i + 2] * down, x[c][4 * i + 3] * down, a[2], a[3]);
                    *reinterpret_cast<uint4*>(S.q[4 * c + i][lane]) = make_uint4(a[0], a[1], a[2], a[3]);
                }
            // what the product lacks: the power of two, the scale, log2 e
            if (t4 == 0)
                S.f[gid] = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                            : __uint_as_float((uint32_t)e << 23) * A.scale * LOG2E;
        }
        __syncthreads();
        const float f = S.f[gid];
        uint32_t qf[D <= 128 ? D / 16 : 1][4];  // registers hold them where there are enough
        if constexpr (D <= 128) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const uint4 a = *reinterpret_cast<const uint4*>(S.q[i][lane]);
                qf[i][0] = a.x, qf[i][1] = a.y, qf[i][2] = a.z, qf[i][3] = a.w;
            }
        }
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        float mx = -INFINITY, sum = 0.f;

        int stage = 0;
        for (int c = c0; c < c1; ++c) {
            copy_wait<STAGES - 2>();
            __syncwarp();  // the step has arrived for all lanes, and all have read the one before it
            float4 sc[SUBS];
#pragma unroll
            for (int h = 0; h < SUBS; ++h) sc[h] = S.scales[warp][stage][h];
            const uint8_t* kp = S.ring[warp][stage];
            if (++stage == STAGES) stage = 0;
            issue(c + STAGES - 1);
            if (sc[0].x < 0.f && sc[SUBS - 1].x < 0.f) continue;
            const int pos = (j.s.first + c) * UNIT + STEP * warp;
            // whether some row does not see all of the step: masks, and codes that may be anything
            const bool edge = pos + STEP - 1 > last_all || pos < low_all || sc[0].x < 0.f || sc[SUBS - 1].x < 0.f;
            const uint8_t* vp = kp + STEP * D;
            float s[2 * SUBS][4];
#pragma unroll
            for (int h = 0; h < 2 * SUBS; ++h) s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.f;
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                uint4 kw[2 * SUBS];
#pragma unroll
                for (int h = 0; h < 2 * SUBS; ++h)
                    kw[h] = *reinterpret_cast<const uint4*>(kp + 16 * key_chunk<D>(8 * h + gid, 4 * i + t4));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t a[4];
                    if constexpr (D <= 128) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) a[x] = qf[4 * i + k][x];
                    } else {
                        const uint4 x = *reinterpret_cast<const uint4*>(S.q[4 * i + k][lane]);
                        a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w;
                    }
#pragma unroll
                    for (int h = 0; h < 2 * SUBS; ++h) {
                        const uint32_t w = k == 0 ? kw[h].x : k == 1 ? kw[h].y : k == 2 ? kw[h].z : kw[h].w;
                        mma(s[h], a[0], a[1], a[2], a[3], e4m3x2_to_half2((uint16_t)w), e4m3x2_to_half2((uint16_t)(w >> 16)));
                    }
                }
            }
            // t (in units of log2); this lane: row gid, positions 8h + 2t, + 1
            float p[2 * SUBS][2], top = mx;
#pragma unroll
            for (int h = 0; h < 2 * SUBS; ++h) {
                const float fk = f * sc[h / 2].x;
                p[h][0] = fmaf(s[h][0] + s[h][2], fk, sc[h / 2].y);
                p[h][1] = fmaf(s[h][1] + s[h][3], fk, sc[h / 2].y);
            }
            if (edge) {
#pragma unroll
                for (int h = 0; h < 2 * SUBS; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int at = pos + 8 * h + 2 * t4 + i;
                        const bool seen = row_ok && at <= last && at >= low && !(sc[h / 2].x < 0.f);
                        if (!seen) p[h][i] = -INFINITY;
                    }
            }
#pragma unroll
            for (int h = 0; h < 2 * SUBS; ++h) top = fmaxf(top, fmaxf(p[h][0], p[h][1]));
            top = quad_max(top);
            const float base = top == -INFINITY ? 0.f : top;
            const float keep = exp2_of(mx - base);
            mx = top;
            sum *= keep;
            uint32_t ph[2 * SUBS], pl[2 * SUBS];
#pragma unroll
            for (int h = 0; h < 2 * SUBS; ++h) {
                p[h][0] = exp2_of(p[h][0] - (base - LIFT));
                p[h][1] = exp2_of(p[h][1] - (base - LIFT));
                sum = fmaf(p[h][0] + p[h][1], sc[h / 2].z, sum);
                split_half(p[h][0], p[h][1], ph[h], pl[h], REST);
            }
            if (__any_sync(0xffffffffu, keep != 1.f)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][0] *= keep, acc[n][1] *= keep, acc[n][2] *= keep, acc[n][3] *= keep;
            }
#pragma unroll
            for (int b = 0; b < SUBS; ++b)
#pragma unroll
                for (int h = 0; h < VC; ++h) {
                    uint32_t w[4][4];  // tokens 2t, 2t+1, 8+2t, 9+2t
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 16 * b + 2 * t4 + (i & 1) + 8 * (i >> 1);
                        if constexpr (D == 64) {
                            const uint2 x =
                                *reinterpret_cast<const uint2*>(vp + 16 * value_chunk<D>(r, gid >> 1) + 8 * (gid & 1));
                            w[i][0] = x.x, w[i][1] = x.y;
                        } else {
                            const uint4 x = *reinterpret_cast<const uint4*>(vp + 16 * value_chunk<D>(r, 8 * h + gid));
                            w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
                        }
                    }
                    if (edge) {  // a probability of 0 must not meet a NaN
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int k = 0; k < (D == 64 ? 2 : 4); ++k) w[i][k] = without_nan(w[i][k]);
                    }
#pragma unroll
                    for (int n = 0; n < (D == 64 ? 8 : 16); ++n)
                        mma(acc[16 * h + n], ph[2 * b], pl[2 * b], ph[2 * b + 1], pl[2 * b + 1],
                            widen_pair(w[0][n / 4], w[1][n / 4], n & 3), widen_pair(w[2][n / 4], w[3][n / 4], n & 3));
                }
        }
        copy_wait<0>();
        __syncwarp();
        // ---- the warps' results together
        sum = quad_sum(sum);
        if (t4 == 0) S.m[warp][gid] = mx, S.l[warp][gid] = sum;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            // tile n, columns 2t and 2t+1: elements 16 * column + n % 16 of its 128 (8 * column + n of 64)
            const int d0 = D == 64 ? 16 * t4 + n : 128 * (n / 16) + 32 * t4 + n % 16;
            warp_out<D>(S, warp)[gid * (D + 4) + d0] = fmaf(acc[n][2], 1.f / REST, acc[n][0]);
            warp_out<D>(S, warp)[gid * (D + 4) + d0 + (D == 64 ? 8 : 16)] = fmaf(acc[n][3], 1.f / REST, acc[n][1]);
        }
        __syncthreads();
        const bool whole = c0 == 0 && c1 == j.s.units;
        const int slot = 2 * blockIdx.x + (c0 == 0 ? 1 : 0);  // a job that began before this block: its first slot
        for (int e = threadIdx.x; e < ROWS * D; e += AT_WARPS * 32) {
            const int r = e / D, d = e % D, row = j.tile * ROWS + r;
            if (row >= j.s.n * G) break;
            float m = S.m[0][r];
#pragma unroll
            for (int w = 1; w < AT_WARPS; ++w) m = fmaxf(m, S.m[w][r]);
            const float base = m == -INFINITY ? 0.f : m;
            float o = 0.f, l = 0.f;
#pragma unroll
            for (int w = 0; w < AT_WARPS; ++w) {
                const float k = exp2f(S.m[w][r] - base);
                l += k * S.l[w][r];
                o += k * warp_out<D>(S, w)[r * (D + 4) + d];
            }
            if (whole) {
                const size_t tok = (size_t)j.s.row0 + row / G;
                const int head = j.head * G + row % G;
                store_out<TY>(A, tok, head * D + d, l > 0.f || l != l ? o / l : 0.f);
                if (A.lse && d == 0) A.lse[tok * A.Hq + head] = l > 0.f || l != l ? (m - LIFT + log2f(l)) * LN2 : -INFINITY;
            } else {
                A.part_o[((size_t)slot * ROWS + r) * D + d] = o;
                if (d == 0) A.part_ml[(size_t)slot * ROWS + r] = make_float2(m, l);
            }
        }
        if (!whole && c0 == 0)
            cut = {(int)((j.first + j.s.units - 1) / per) - (int)blockIdx.x + 1, j.s.row0, j.tile, j.head,
                   min(ROWS, j.s.n * G - j.tile * ROWS)};
        u = j.first + c1;
    }
    if (threadIdx.x == 0) A.cuts[blockIdx.x] = cut;
}

// Join the partial results of the job that block x started and did not end.
// Few parts: one thread block takes all rows, a thread four columns of a row.
// Many: one row a thread block (y), a thread adds four columns of every
// GROUPS-th part, then the groups' sums are added.
constexpr int JOIN_THREADS = 256;
constexpr int JOIN_PARTS = 512;  // parts a job can have: the thread blocks
constexpr int JOIN_FEW = 8;

template <int D, int TY>
__global__ void __launch_bounds__(JOIN_THREADS) k_attn_join(AttnArgs A) {
    constexpr int GROUPS = JOIN_THREADS / (D / 4);
    __shared__ float weight[JOIN_PARTS];
    __shared__ float part[GROUPS][D + 4];
    __shared__ float wm[JOIN_THREADS / 32], wl[JOIN_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = tid / (D / 4), d4 = tid % (D / 4) * 4, G = A.Hq / A.Hkv, b0 = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial results are there
    const Cut cut = A.cuts[b0];
    const int n = cut.parts;
    const auto write = [&](int r, int d, float o, float m, float l) {
        const int row = cut.tile * ROWS + r, head = cut.head * G + row % G;
        const size_t tok = (size_t)cut.row0 + row / G;
        store_out<TY>(A, tok, head * D + d, l > 0.f || l != l ? o / l : 0.f);
        if (A.lse && d == 0) A.lse[tok * A.Hq + head] = l > 0.f || l != l ? (m - LIFT + log2f(l)) * LN2 : -INFINITY;
    };
    if (n <= JOIN_FEW) {
        if (blockIdx.y != 0) return;
        for (int r = g; r < cut.rows && n > 0; r += GROUPS) {
            const auto slot = [&](int i) { return ((size_t)2 * (b0 + i) + (i == 0)) * ROWS + r; };
            float2 ml[JOIN_FEW];
            float4 x[JOIN_FEW];
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int i = 0; i < JOIN_FEW; ++i)
                if (i < n) {
                    ml[i] = A.part_ml[slot(i)];
                    x[i] = *reinterpret_cast<const float4*>(A.part_o + slot(i) * D + d4);
                    m = fmaxf(m, ml[i].x);
                }
            const float base = m == -INFINITY ? 0.f : m;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < JOIN_FEW; ++i)
                if (i < n) {
                    const float k = exp2f(ml[i].x - base);
                    l += k * ml[i].y;
                    o.x += k * x[i].x, o.y += k * x[i].y, o.z += k * x[i].z, o.w += k * x[i].w;
                }
            write(r, d4, o.x, m, l);
            write(r, d4 + 1, o.y, m, l);
            write(r, d4 + 2, o.z, m, l);
            write(r, d4 + 3, o.w, m, l);
        }
        return;
    }
    const int r = blockIdx.y;
    if (r >= cut.rows) return;
    // the first block left its part in its second slot, the others in their first
    const auto slot = [&](int i) { return ((size_t)2 * (b0 + i) + (i == 0)) * ROWS + r; };
    float m = -INFINITY;
    for (int i = tid; i < n; i += JOIN_THREADS) m = fmaxf(m, A.part_ml[slot(i)].x);
    m = warp_max(m);
    if (lane == 0) wm[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < JOIN_THREADS / 32; ++w) m = fmaxf(m, wm[w]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int i = tid; i < n; i += JOIN_THREADS) {
        const float2 ml = A.part_ml[slot(i)];
        weight[i] = exp2f(ml.x - base);
        l += weight[i] * ml.y;
    }
    l = warp_sum(l);
    if (lane == 0) wl[warp] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < JOIN_THREADS / 32; ++w) l += wl[w];
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = g; i < n; i += GROUPS) {
        const float4 x = *reinterpret_cast<const float4*>(A.part_o + slot(i) * D + d4);
        const float k = weight[i];
        o.x += k * x.x, o.y += k * x.y, o.z += k * x.z, o.w += k * x.w;
    }
    *reinterpret_cast<float4*>(&part[g][d4]) = o;
    __syncthreads();
    if (tid < D) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) v += part[k][tid];
        write(r, tid, v, m, l);
    }
}

constexpr int BLOCKS_PER_SM = 2;

int attn_blocks() {
    const int n = num_sms() * BLOCKS_PER_SM;
    return n < JOIN_PARTS ? n : JOIN_PARTS;
}

template <int D, int TY>
int launch(AttnArgs a, cudaStream_t s) {
    a.unit = Tile<D>::UNIT;
    const size_t sched = (size_t)(a.B + 1) * sizeof(long long);
    const size_t sm = sizeof(AttnSmem<D>) + sched;
    if (cudaFuncSetAttribute(k_attn<D, TY>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm) != cudaSuccess)
        return E0_ERR_CUDA;
    k_attn<D, TY><<<a.blocks, AT_WARPS * 32, sm, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return E0_ERR_CUDA;
    // the join's blocks start while those above still run and wait for all of them
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.blocks, ROWS);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attn_join<D, TY>, a) == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

template <int TY>
int launch_d(const AttnArgs& a, int D, cudaStream_t s) {
    return D == 64 ? launch<64, TY>(a, s) : D == 128 ? launch<128, TY>(a, s) : launch<256, TY>(a, s);
}

}  // namespace

size_t attn_ws_bytes(int D) {
    const size_t slots = 2 * (size_t)attn_blocks();
    return slots * ROWS * D * sizeof(float) + slots * ROWS * sizeof(float2) + slots / 2 * sizeof(Cut);
}

int attn_decode(const e0_kv_cache* c, const int32_t* table, int max_blocks, const int32_t* ctx, const int32_t* cu,
                int B, int max_q, const void* q, int dtype, int64_t q_ld, int Hq, float scale, int window, void* out,
                int64_t out_ld, float* lse, void* ws, uint32_t* st, cudaStream_t s) {
    AttnArgs a = {};
    a.k = c->k, a.v = c->v, a.ks = c->k_scale, a.vs = c->v_scale;
    a.table = table, a.ctx = ctx, a.cu = cu, a.q = q, a.out = out, a.lse = lse;
    a.blocks = attn_blocks();
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + 2 * (size_t)a.blocks * ROWS * c->D);
    a.cuts = reinterpret_cast<Cut*>(a.part_ml + 2 * (size_t)a.blocks * ROWS);
    a.st = st, a.q_ld = q_ld, a.out_ld = out_ld;
    a.B = B, a.max_blocks = max_blocks, a.n_blocks = c->n_blocks, a.Hq = Hq, a.Hkv = c->Hkv, a.max_q = max_q;
    a.window = window, a.scale = scale;
    while ((1 << a.shift) < c->block_tokens) ++a.shift;
    return dtype == E0_F32   ? launch_d<E0_F32>(a, c->D, s)
           : dtype == E0_F16 ? launch_d<E0_F16>(a, c->D, s)
                             : launch_d<E0_BF16>(a, c->D, s);
}

}  // namespace e0
