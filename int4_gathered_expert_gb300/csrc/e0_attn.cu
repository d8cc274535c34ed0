// Attention of decode queries over the paged 8-bit KV cache (e0_attn_decode).
#include <climits>
#include <cuda_runtime.h>

#include "e0_internal.h"
#include "e0_types.cuh"

namespace e0 {
namespace {

// out = softmax(scale q K^T) V in one pass over the context with the running
// maximum and sum.  A job is one (sequence, KV head, tile of query rows): the rows
// are the query heads of the group and the sequence's new tokens, token major.  A
// job's context is cut into units, and the units of all jobs, one after another,
// are dealt out evenly to the thread blocks: every block reads the same number
// of bytes whatever the lengths are.  A job that ends up on several blocks
// leaves one partial result (maximum, sum, unscaled output) on each, at most two
// a block, and k_attn_join adds them in order.
//
// A unit is one step of each of a block's warps.  Products run on the tensor
// cores (16 x 8 x 16, fp16 operands, fp32 accumulation); e4m3 codes widen to fp16
// exactly.  The 16 operand rows hold 8 query rows twice: rows 0..7 the fp16 part,
// rows 8..15 the rest of the value, so neither q nor the probabilities lose bits
// that matter (22 significant bits), at no cost: a decode step has few rows and
// the kernel is bound by reading the cache.  Where there are more than 8 rows and the
// outputs are bf16, the tile is WIDE: 16 query rows, q exact (8 bits of each row's
// power of two), probabilities rounded to fp16, an eighth of what the output's
// rounding is; a sequence is then read half as often.  (fp16 outputs would be 1.4
// times as far off with it, so they keep the rests.)
// A warp's codes come through its own ring in shared memory, copied some steps
// ahead, so warps never wait for one another inside a job.  Operand layouts are
// chosen so that every lane reads 16 bytes at a time: the order of D inside the
// first product and of the output columns in the second are permuted (the same
// permutation on both operands).
// The scale of a block of keys multiplies the scores; that of the values goes into
// the exponent: with t_j = score_j + log2(scale_j) and m the running maximum of
// t, the weights of the codes are 2^(t_j - m + 7), at most 2^15 because m follows
// only where t has grown by more than 8 (a row's output is then scaled once or
// twice in a job, not at every new maximum).  That fills fp16's range whatever the
// scales are: the rest of a weight goes in times 2^12, so weights down to 2^-43
// of the largest count.  The softmax's sum is that of the weights over their
// scales, times 2^-12: the weights are at most 2^15 and the scales at least 2^-100, so 2^25
// positions of zero values (2^30 with equal scores) stay inside fp32's range, and so
// does the inverse of the sum where the scales are the largest ones of finite values,
// 2^120, and the sum is 2^(7 - 120 - 12) or more.
//
// Measured (device time, GB300): 64 sequences of up to 16000 tokens, 32 query on 4
// KV heads of 128, 498 MB: 85.5 us, 5.8 TB/s, 86 % of the measured copy rate; what
// is missing is the first steps' latency (4 us), jobs' ends and the join (3 us).  One
// sequence of 32000, 16 on 2 heads of 256, 33 MB: 16.9 us, four steps a warp
// between the schedule and the join.  16 sequences of 16000, 32 on 2 heads of 256:
// 94.2 us in tiles of 8 rows, 73.8 in tiles of 16 (bf16); 32 of 8000, two queries
// each, 32 on 4 of 128: 46.2 and 43.0.
// What got it there, on the first of these: 166 us with loads straight into
// registers; 155 with the ring; 110 with steps of 32 positions, the hardware's
// widening of e4m3 (one instruction a pair; masks and shifts took three) and value
// scales in the exponent; 93 with the next job's copies started before a job's end
// and query loads without a branch between them; 86 with jobs' costs in the schedule.

constexpr int AT_WARPS = 4;
constexpr int MOST_ROWS = 16;

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
    // what a job costs beside its units (block ids, queries, result: 3 us, in which
    // the block's share of the memory's rate reads 64 KB), in units
    static constexpr int JOB_COST = 65536 / (AT_WARPS * BYTES);
};

// What a block leaves for the join: the job that it started and did not end, and
// the one that it went on with.
struct Cut {
    int parts, block;  // blocks that have a part (0: no job), the first of them
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
    float* part_o;    // [2 * blocks][rows][D]
    float2* part_ml;  // [2 * blocks][rows]
    Cut* cuts;        // [blocks][2]
    uint32_t* st;
    int64_t q_ld, out_ld;
    int B, max_blocks, n_blocks, shift, Hq, Hkv, max_q, window, blocks, unit, job_cost, rows;
    float scale;
};

// One sequence as the schedule sees it.
struct Seq {
    int row0, n, ctx, first;  // first query row, queries, cached tokens, first unit that anyone sees
    int units, tiles;         // units of context, tiles of query rows per KV head
    int low;                  // the first position that the first query sees
};

E0_DEV Seq seq_of(const AttnArgs& A, int b, bool tell) {
    Seq s;
    s.row0 = A.cu ? A.cu[b] : b;
    const long long n = A.cu ? (long long)A.cu[b + 1] - s.row0 : 1;  // of any two 32-bit numbers: not a 32-bit one
    s.n = (int)n;
    s.ctx = A.ctx[b];
    bool bad = false;
    if (s.row0 < 0 || n < 0 || n > A.max_q) bad = true, s.n = 0;
    if (s.ctx < 0 || (long long)s.ctx > ((long long)A.max_blocks << A.shift)) bad = true, s.ctx = 0;
    if (bad && tell) set_status(A.st, E0_ST_BAD_LENGTH);
    s.low = A.window > 0 ? max(s.ctx - s.n + 1 - A.window, 0) : 0;
    s.first = s.low / A.unit;
    s.units = (int)(((long long)s.ctx + A.unit - 1) / A.unit) - s.first;
    if (s.units < 1) s.units = 1;  // a job without context still writes its rows
    const int G = A.Hq / A.Hkv;
    s.tiles = (int)(((long long)s.n * G + A.rows - 1) / A.rows);
    return s;
}

// A schedule longer than this is not run (it would read for seconds).
constexpr uint32_t MOST_UNITS = 0x7FFFFFFFu;

E0_DEV uint32_t add_units(uint32_t a, uint32_t b) { return min(a + b, MOST_UNITS); }

// How the jobs are dealt out.  Even: every block the same share of the schedule, as
// many blocks as get one unit besides a job's cost.  Or, where there are no more jobs
// than blocks and the longest is not much longer than a share, a job a block: nothing
// to join, no block with the ends of two jobs (16 sequences of up to 500, 8 heads of
// 64: 10.0 us against 11.8, the join launched in both).  Or, where there are no more
// units than blocks, a unit a block (a sequence of 4096, 32 on 8 heads of 128: 10.0 us
// against 11.7; with two units a block where there are up to twice as many, a sequence
// of 8000, 8 heads of 64: 12.3 against 11.3).
struct Plan {
    uint32_t total;  // places in the schedule: units and jobs' costs, or jobs, or units
    uint32_t share;  // of a block
    uint32_t cost;   // places that a job takes beside its units
    bool whole;      // a job a block
};

// Every sequence's first place in the schedule goes to shared memory.
E0_DEV Plan schedule(const AttnArgs& A, uint32_t* first, uint32_t (*red)[3], bool tell) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (A.B + blockDim.x - 1) / blockDim.x, b0 = threadIdx.x * per;
    uint32_t sum = 0, jobs = 0, most = 0;
    for (int i = 0; i < per && b0 + i < A.B; ++i) {
        const Seq s = seq_of(A, b0 + i, tell);
        first[b0 + i] = sum;  // from the thread's own first sequence on, for now
        const unsigned long long k = (unsigned long long)s.tiles * A.Hkv, n = (s.units + A.job_cost) * k;
        sum = add_units(sum, n < MOST_UNITS ? (uint32_t)n : MOST_UNITS);
        jobs = add_units(jobs, k < MOST_UNITS ? (uint32_t)k : MOST_UNITS);
        if (k > 0) most = max(most, (uint32_t)s.units);
    }
    uint32_t inc = sum, inc_jobs = jobs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o), y = __shfl_up_sync(0xffffffffu, inc_jobs, o);
        if (lane >= o) inc = add_units(inc, x), inc_jobs = add_units(inc_jobs, y);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) red[warp][0] = inc, red[warp][1] = inc_jobs, red[warp][2] = most;
    __syncthreads();
    uint32_t base = 0, base_jobs = 0, total = 0, total_jobs = 0;
#pragma unroll
    for (int i = 0; i < AT_WARPS; ++i) {
        if (i < warp) base = add_units(base, red[i][0]), base_jobs = add_units(base_jobs, red[i][1]);
        total = add_units(total, red[i][0]), total_jobs = add_units(total_jobs, red[i][1]);
        most = max(most, red[i][2]);
    }
    Plan p;
    const uint32_t even = (total + A.blocks - 1) / A.blocks, units = total - total_jobs * A.job_cost;
    p.whole = total_jobs <= (uint32_t)A.blocks && most <= max(even, (uint32_t)A.job_cost + 2) + A.job_cost;
    p.total = total;
    p.share = max(even, (uint32_t)A.job_cost + 1);
    p.cost = A.job_cost;
    if (p.whole || (total < MOST_UNITS && units <= (uint32_t)A.blocks)) {
        p.total = p.whole ? total_jobs : units, p.share = 1, p.cost = 0;
        uint32_t at = base_jobs + inc_jobs - jobs;  // jobs before
        for (int i = 0; i < per && b0 + i < A.B; ++i) {
            first[b0 + i] = p.whole ? at : first[b0 + i] + (base + inc - sum) - at * A.job_cost;
            at += (uint32_t)seq_of(A, b0 + i, false).tiles * A.Hkv;
        }
    } else {
        for (int i = 0; i < per && b0 + i < A.B; ++i) first[b0 + i] = add_units(first[b0 + i], base + inc - sum);
        if (total >= MOST_UNITS) {
            if (tell && threadIdx.x == 0) set_status(A.st, E0_ST_BAD_LENGTH);
            p.total = 0;
        }
    }
    __syncthreads();
    return p;
}

// A block's part of a job: units c0..c1-1 of it (none where c1 <= c0).
struct Span {
    Seq s;
    int seq, head, tile, c0, c1;
    uint32_t first, end;  // the job's place in the schedule; where the part ends there
};

E0_DEV Span span_at(const AttnArgs& A, const Plan& p, const uint32_t* first, uint32_t u, uint32_t u1) {
    int lo = 0, hi = A.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= u) lo = mid; else hi = mid;
    }
    Span j;
    j.seq = lo;
    j.s = seq_of(A, lo, false);
    const uint32_t len = p.whole ? 1 : j.s.units + p.cost, k = (u - first[lo]) / len;
    j.head = k / j.s.tiles;
    j.tile = k % j.s.tiles;
    j.first = first[lo] + k * len;
    j.end = min(j.first + len, u1);
    j.c0 = max((int)(u - j.first) - (int)p.cost, 0);
    j.c1 = p.whole ? j.s.units : (int)(j.end - j.first) - (int)p.cost;
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
constexpr float LIFT = 7.f, SLACK = 8.f;                // weights are 2^(t - m + LIFT), t at most m + SLACK
constexpr float REST = 4096.f;                          // what the rests of the weights go in times
constexpr float SUM_LIFT = -12.f, SUM_UNIT = 1.f / 4096.f;  // sums are times 2^SUM_LIFT

// ln of the softmax's sum from the running maximum and sum.
E0_DEV float lse_of(float m, float l) {
    return l > 0.f || l != l ? (m - (LIFT + SUM_LIFT) + log2f(l)) * LN2 : -INFINITY;
}

template <int D>
struct AttnSmem {
    uint8_t ring[AT_WARPS][Tile<D>::STAGES][Tile<D>::BYTES];  // a warp's output at the end of a job
    uint32_t q[D / 16][32][4];
    float4 scales[AT_WARPS][Tile<D>::STAGES][2];  // of a piece: keys' scale (< 0: not seen), values' log2 and inverse
    float m[AT_WARPS][MOST_ROWS], l[AT_WARPS][MOST_ROWS];
    float f[MOST_ROWS];
    uint32_t red[AT_WARPS][3];
};

// Element d of row r (of 8) of a warp's output, in its ring's first stage; columns are
// permuted inside 32 so that what the lanes write at once has 32 banks.
template <int D>
E0_DEV float& warp_out(AttnSmem<D>& S, int w, int r, int d) {
    static_assert(Tile<D>::BYTES >= 8 * D * sizeof(float), "a stage holds a warp's output");
    const int key = D == 64 ? 4 * r + (d >> 4) : 4 * r + (d >> 5);
    return reinterpret_cast<float*>(S.ring[w])[r * D + (d ^ (key & 31))];
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

template <int D, int TY, bool WIDE>
__global__ void __launch_bounds__(AT_WARPS * 32) k_attn(AttnArgs A) {
    typedef typename Elem<TY>::T T;
    extern __shared__ __align__(128) char attn_sm[];
    AttnSmem<D>& S = *reinterpret_cast<AttnSmem<D>*>(attn_sm);
    uint32_t* first = reinterpret_cast<uint32_t*>(attn_sm + sizeof(AttnSmem<D>));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, t4 = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Plan plan = schedule(A, first, S.red, blockIdx.x == 0);
    uint32_t u = blockIdx.x * plan.share;
    const uint32_t u1 = min(u + plan.share, plan.total);
    const int G = A.Hq / A.Hkv, bs = 1 << A.shift;
    constexpr int RW = WIDE ? 2 : 1, ROWS = 8 * RW;  // rows of a lane (gid, gid + 8); of a tile
    constexpr int KC = D / 64;          // 16-byte chunks of a key row a lane reads
    constexpr int NT = D / 8;           // output tiles
    constexpr int VC = D >= 128 ? D / 128 : 1;  // 16-byte chunks of a value row
    constexpr int SUBS = Tile<D>::SUBS, STEP = Tile<D>::STEP, UNIT = Tile<D>::UNIT, STAGES = Tile<D>::STAGES;
    constexpr int AHEAD = 32 / SUBS;    // steps whose block ids the lanes hold
    Cut begun = {0, 0, 0, 0, 0, 0}, went_on = {0, 0, 0, 0, 0, 0};

    // the next part that has units
    Span j;
    const auto next = [&]() {
        while (u < u1) {
            j = span_at(A, plan, first, u, u1);
            u = j.end;
            if (j.c1 > j.c0) return true;
        }
        return false;
    };
    // block ids and scales of the next pieces, one a lane
    int my_id = -1;
    float4 my_sc;
    const auto look_up = [&](int c) {
        const int cc = c + lane / SUBS, pos = (j.s.first + cc) * UNIT + STEP * warp + 16 * (lane % SUBS);
        my_id = -1;
        my_sc = make_float4(-1.f, 0.f, 0.f, 0.f);
        if (cc < j.c1 && pos < j.s.ctx && pos + 16 > j.s.low) {
            my_id = A.table[(size_t)j.seq * A.max_blocks + (pos >> A.shift)];
            if (my_id >= 0 && my_id < A.n_blocks) {
                const size_t i = (size_t)my_id * A.Hkv + j.head;
                const float v = fmaxf(A.vs[i], LEAST_SCALE);
                my_sc = make_float4(A.ks[i], log2f(v), SUM_UNIT / v, 0.f);
            } else {
                my_id = -1;
                set_status(A.st, E0_ST_BAD_BLOCK);
            }
        }
    };
    int in_stage = 0, in_at = 0;  // where the next copy goes; its place among the lanes' ids
    const auto put_scales = [&](int at, int stage) {
        if (lane / SUBS == at) S.scales[warp][stage][lane % SUBS] = my_sc;
    };
    const auto issue = [&](int c, bool scales) {
        if (c < j.c1) {
            if (in_at == AHEAD) {
                look_up(c);
                in_at = 0;
            }
#pragma unroll
            for (int h = 0; h < SUBS; ++h) {
                const int from = in_at * SUBS + h;
                const int id = __shfl_sync(0xffffffffu, my_id, from);
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
            if (scales) put_scales(in_at, in_stage);
            ++in_at;
            if (++in_stage == STAGES) in_stage = 0;
        }
        copy_commit();
    };
    // the first steps of a part go to the stages but the first, which holds the
    // former part's output until it has been written; the codes' copies need the
    // block ids only and go ahead of the scales
    const auto begin = [&]() {
        in_stage = 1, in_at = 0;
#pragma unroll 1
        for (int i = 0; i < STAGES - 1; ++i) issue(j.c0 + i, false);
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) put_scales(i, i + 1);
    };
    // this lane's query row: 16 elements of each 64, as they are in memory; a row
    // beyond the tile's reads the tile's first and counts as zeros
    constexpr int RAW = TY == E0_F32 ? 4 : 2;
    uint4 raw[KC][RAW];
    const auto load_q = [&](int at) {  // row at of the tile
        const int row = j.tile * ROWS + (j.tile * ROWS + at < j.s.n * G ? at : 0);
        const T* p = reinterpret_cast<const T*>(A.q) + (size_t)(j.s.row0 + row / G) * A.q_ld +
                     (size_t)(j.head * G + row % G) * D + 16 * t4;
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int i = 0; i < RAW; ++i) raw[c][i] = __ldg(reinterpret_cast<const uint4*>(p + 64 * c) + i);
    };
    const auto q_of = [&](int c, int i) {  // element i of 16
        const uint4 u = raw[c][TY == E0_F32 ? i / 4 : i / 8];
        if constexpr (TY == E0_F32) {
            const uint32_t w = i % 4 == 0 ? u.x : i % 4 == 1 ? u.y : i % 4 == 2 ? u.z : u.w;
            return __uint_as_float(w);
        } else {
            const uint32_t w = i % 8 < 2 ? u.x : i % 8 < 4 ? u.y : i % 8 < 6 ? u.z : u.w;
            const float2 f = unpack16<TY>(w);
            return i % 2 ? f.y : f.x;
        }
    };

    bool more = next();
    if (more) {
        look_up(j.c0);
        load_q(gid);
        begin();
    }
    while (more) {
        // ---- the job's queries as operand fragments: every warp reads them all for the
        // rows' maxima and leaves its share of the fragments in shared memory
#pragma unroll
        for (int w = 0; w < RW; ++w) {
            if (w == 1) load_q(gid + 8);
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(q_of(c, i)) & 0x7FFFFFFFu);
            if (j.tile * ROWS + gid + 8 * w >= j.s.n * G) m = 0;
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            // rows go in times a power of two that brings the largest near 1
            int e = (int)(m >> 23);
            e = e < 27 ? 27 : e > 253 ? 253 : e;
            const float down = m == 0 ? 0.f : __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if ((4 * c + i) / KC != warp) continue;
                    uint32_t a[4];
                    split_half(q_of(c, 4 * i) * down, q_of(c, 4 * i + 1) * down, a[0], a[1]);
                    split_half(q_of(c, 4 * i + 2) * down, q_of(c, 4 * i + 3) * down, a[2], a[3]);
                    uint32_t* to = S.q[4 * c + i][lane];
                    if constexpr (WIDE)
                        to[w] = a[0], to[2 + w] = a[2];
                    else
                        *reinterpret_cast<uint4*>(to) = make_uint4(a[0], a[1], a[2], a[3]);
                }
            // what the product lacks: the power of two, the scale, log2 e
            if (warp == 0 && t4 == 0)
                S.f[gid + 8 * w] = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                                    : __uint_as_float((uint32_t)e << 23) * A.scale * LOG2E;
        }
        __syncthreads();  // and the former part's output and statistics have been read
        const Span cur = j;
        bool row_ok[RW];
        int last[RW], low[RW];  // the last and first positions that the row sees
        float f[RW];
#pragma unroll
        for (int w = 0; w < RW; ++w) {
            const int row = cur.tile * ROWS + gid + 8 * w;
            row_ok[w] = row < cur.s.n * G;
            last[w] = cur.s.ctx - cur.s.n + row / G;
            low[w] = A.window > 0 ? last[w] - A.window + 1 : 0;
            f[w] = S.f[gid + 8 * w];
        }
        // what every row of the tile sees
        const int last_all = cur.s.ctx - cur.s.n + cur.tile * ROWS / G;
        const int low_all = A.window > 0 ? cur.s.ctx - A.window : 0;
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
        float mx[RW], sum[RW];
#pragma unroll
        for (int w = 0; w < RW; ++w) mx[w] = -INFINITY, sum[w] = 0.f;

        int stage = 1;
        for (int c = cur.c0; c < cur.c1; ++c) {
            copy_wait<STAGES - 2>();
            __syncwarp();  // the step has arrived for all lanes, and all have read the one before it
            float4 sc[SUBS];
#pragma unroll
            for (int h = 0; h < SUBS; ++h) sc[h] = S.scales[warp][stage][h];
            const uint8_t* kp = S.ring[warp][stage];
            if (++stage == STAGES) stage = 0;
            issue(c + STAGES - 1, true);
            if (sc[0].x < 0.f && sc[SUBS - 1].x < 0.f) continue;
            const int pos = (cur.s.first + c) * UNIT + STEP * warp;
            // whether some row does not see all of the step: masks, and codes that may be anything
            const bool edge = pos + STEP - 1 > last_all || pos < low_all || sc[0].x < 0.f || sc[SUBS - 1].x < 0.f;
            const uint8_t* vp = kp + STEP * D;
            // four chains of products: pieces of 8 positions, or for few pieces also halves of D
            constexpr int CH = 2 / SUBS;
            float s[2 * SUBS][4], s2[CH == 2 ? 2 * SUBS : 1][4];
#pragma unroll
            for (int h = 0; h < 2 * SUBS; ++h) s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.f;
#pragma unroll
            for (int h = 0; h < (CH == 2 ? 2 * SUBS : 1); ++h) s2[h][0] = s2[h][1] = s2[h][2] = s2[h][3] = 0.f;
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
                        const uint32_t b0 = e4m3x2_to_half2((uint16_t)w), b1 = e4m3x2_to_half2((uint16_t)(w >> 16));
                        if (CH == 2 && (k & 1))
                            mma(s2[CH == 2 ? h : 0], a[0], a[1], a[2], a[3], b0, b1);
                        else
                            mma(s[h], a[0], a[1], a[2], a[3], b0, b1);
                    }
                }
            }
            // t (in units of log2); this lane: rows gid (+ 8), positions 8h + 2t, + 1
            float p[RW][2 * SUBS][2], top[RW];
#pragma unroll
            for (int h = 0; h < 2 * SUBS; ++h) {
                if constexpr (CH == 2) s[h][0] += s2[h][0], s[h][1] += s2[h][1], s[h][2] += s2[h][2], s[h][3] += s2[h][3];
                const float fk = f[0] * sc[h / 2].x;
                if constexpr (WIDE) {
                    const float fk1 = f[RW - 1] * sc[h / 2].x;
                    p[0][h][0] = fmaf(s[h][0], fk, sc[h / 2].y), p[0][h][1] = fmaf(s[h][1], fk, sc[h / 2].y);
                    p[RW - 1][h][0] = fmaf(s[h][2], fk1, sc[h / 2].y), p[RW - 1][h][1] = fmaf(s[h][3], fk1, sc[h / 2].y);
                } else {
                    p[0][h][0] = fmaf(s[h][0] + s[h][2], fk, sc[h / 2].y);
                    p[0][h][1] = fmaf(s[h][1] + s[h][3], fk, sc[h / 2].y);
                }
            }
            if (edge) {
#pragma unroll
                for (int w = 0; w < RW; ++w)
#pragma unroll
                    for (int h = 0; h < 2 * SUBS; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int at = pos + 8 * h + 2 * t4 + i;
                            const bool seen = row_ok[w] && at <= last[w] && at >= low[w] && !(sc[h / 2].x < 0.f);
                            if (!seen) p[w][h][i] = -INFINITY;
                        }
            }
            bool grows = false;
#pragma unroll
            for (int w = 0; w < RW; ++w) {
                top[w] = mx[w];
#pragma unroll
                for (int h = 0; h < 2 * SUBS; ++h) top[w] = fmaxf(top[w], fmaxf(p[w][h][0], p[w][h][1]));
                top[w] = quad_max(top[w]);
                grows |= top[w] > mx[w] + SLACK;
            }
            if (__any_sync(0xffffffffu, grows)) {
                float keep[RW];
#pragma unroll
                for (int w = 0; w < RW; ++w) {
                    if (!(top[w] > mx[w] + SLACK)) top[w] = mx[w];
                    keep[w] = mx[w] == top[w] ? 1.f : exp2_of(mx[w] - top[w]);
                    mx[w] = top[w];
                    sum[w] *= keep[w];
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[n][0] *= keep[0], acc[n][1] *= keep[0], acc[n][2] *= keep[RW - 1], acc[n][3] *= keep[RW - 1];
            }
            uint32_t ph[2 * SUBS], pl[2 * SUBS];  // the operand's rows 0..7 and 8..15
#pragma unroll
            for (int w = 0; w < RW; ++w) {
                const float base = (mx[w] == -INFINITY ? 0.f : mx[w]) - LIFT;
#pragma unroll
                for (int h = 0; h < 2 * SUBS; ++h) {
                    const float a = exp2_of(p[w][h][0] - base), b = exp2_of(p[w][h][1] - base);
                    sum[w] = fmaf(a + b, sc[h / 2].z, sum[w]);
                    if constexpr (WIDE)
                        (w ? pl : ph)[h] = half2_of(a, b);
                    else
                        split_half(a, b, ph[h], pl[h], REST);
                }
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
        // ---- the next part's copies start, then the warps' results come together
        more = next();
        if (more) {
            look_up(j.c0);
            load_q(gid);
        }
#pragma unroll
        for (int w = 0; w < RW; ++w) {
            sum[w] = quad_sum(sum[w]);
            if (t4 == 0) S.m[warp][gid + 8 * w] = mx[w], S.l[warp][gid + 8 * w] = sum[w];
        }
        // rows 0..7, then 8..15 of a wide tile, through the ring's first stage
        const auto put_out = [&](int w) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                // tile n, columns 2t and 2t+1: elements 16 * column + n % 16 of its 128 (8 * column + n of 64)
                const int d0 = D == 64 ? 16 * t4 + n : 128 * (n / 16) + 32 * t4 + n % 16;
                const float a = WIDE ? acc[n][2 * w] : fmaf(acc[n][2], 1.f / REST, acc[n][0]);
                const float b = WIDE ? acc[n][2 * w + 1] : fmaf(acc[n][3], 1.f / REST, acc[n][1]);
                warp_out<D>(S, warp, gid, d0) = a;
                warp_out<D>(S, warp, gid, d0 + (D == 64 ? 8 : 16)) = b;
            }
        };
        put_out(0);
        if (more) begin();
        __syncthreads();
        const bool whole = cur.c0 == 0 && cur.c1 == cur.s.units;
        const int slot = 2 * blockIdx.x + (cur.c0 == 0 ? 1 : 0);  // a job that began in a former block: the first slot
        const int rows = min(ROWS, cur.s.n * G - cur.tile * ROWS);
#pragma unroll
        for (int half = 0; half < RW; ++half) {
            if (half == 1) {
                __syncthreads();  // the first rows have been read
                put_out(1);
                __syncthreads();
            }
#pragma unroll 1
            for (int r = 8 * half + warp; r < min(rows, 8 * half + 8); r += AT_WARPS) {
                float m = S.m[0][r], l = 0.f, k[AT_WARPS];
#pragma unroll
                for (int w = 1; w < AT_WARPS; ++w) m = fmaxf(m, S.m[w][r]);
                const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int w = 0; w < AT_WARPS; ++w) {
                    k[w] = exp2_of(S.m[w][r] - base);
                    l += k[w] * S.l[w][r];
                }
                const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
                const int row = cur.tile * ROWS + r, head = cur.head * G + row % G;
                const size_t tok = (size_t)cur.s.row0 + row / G;
#pragma unroll
                for (int d = lane; d < D; d += 32) {
                    float o = 0.f;
#pragma unroll
                    for (int w = 0; w < AT_WARPS; ++w) o += k[w] * warp_out<D>(S, w, r & 7, d);
                    if (whole)
                        store_out<TY>(A, tok, head * D + d, o * SUM_UNIT * inv);
                    else
                        A.part_o[((size_t)slot * ROWS + r) * D + d] = o;
                }
                if (lane == 0) {
                    if (!whole)
                        A.part_ml[(size_t)slot * ROWS + r] = make_float2(m, l);
                    else if (A.lse)
                        A.lse[tok * A.Hq + head] = lse_of(m, l);
                }
            }
        }
        if (!whole) {
            const int b0 = (int)((cur.first + plan.cost) / plan.share);
            const int b1 = (int)((cur.first + plan.cost + cur.s.units - 1) / plan.share);
            (cur.c0 == 0 ? begun : went_on) = {b1 - b0 + 1, b0, cur.s.row0, cur.tile, cur.head, rows};
        }
    }
    if (threadIdx.x == 0) A.cuts[2 * blockIdx.x] = begun, A.cuts[2 * blockIdx.x + 1] = went_on;
}

// Join the parts of the jobs that several blocks have.  Few parts: the thread
// block that started the job takes all of it, a thread four columns of a row.
// Many: the thread blocks that have a part share its rows and quarters of rows; a
// thread adds four columns of every GROUPS-th part, then the groups' sums are
// added.  Either way in the same order in every run.
constexpr int JOIN_THREADS = 256;
constexpr int JOIN_FEW = 8;

template <int D, int TY>
__global__ void __launch_bounds__(JOIN_THREADS) k_attn_join(AttnArgs A) {
    constexpr int COLS = D / 4;                     // a quarter of a row
    constexpr int GROUPS = JOIN_THREADS / (COLS / 4);
    constexpr int BATCH = 4;  // a sequence of 32000, 8 on 1 head of 128: 12.1 us, 12.4 with 8
    __shared__ float part[GROUPS][COLS + 4];
    __shared__ float gm[GROUPS], gl[GROUPS];
    const int tid = threadIdx.x, G = A.Hq / A.Hkv;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
    const Cut begun = A.cuts[2 * blockIdx.x], went_on = A.cuts[2 * blockIdx.x + 1];
    const auto write = [&](const Cut& cut, int r, int d, float o, float m, float l) {
        const int row = cut.tile * A.rows + r, head = cut.head * G + row % G;
        const size_t tok = (size_t)cut.row0 + row / G;
        store_out<TY>(A, tok, head * D + d, l > 0.f || l != l ? o * SUM_UNIT / l : 0.f);
        if (A.lse && d == 0) A.lse[tok * A.Hq + head] = lse_of(m, l);
    };
    // the first block left its part in its second slot, the others in their first
    const auto slot_of = [&](const Cut& cut, int r, int i) { return ((size_t)2 * (cut.block + i) + (i == 0)) * A.rows + r; };
    if (begun.parts > 0 && begun.parts <= JOIN_FEW) {
        const int n = begun.parts, d4 = tid % (D / 4) * 4;
        for (int r = tid / (D / 4); r < begun.rows; r += JOIN_THREADS / (D / 4)) {
            float2 ml[JOIN_FEW];
            float4 x[JOIN_FEW];
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int i = 0; i < JOIN_FEW; ++i)
                if (i < n) {
                    ml[i] = A.part_ml[slot_of(begun, r, i)];
                    x[i] = *reinterpret_cast<const float4*>(A.part_o + slot_of(begun, r, i) * D + d4);
                }
#pragma unroll
            for (int i = 0; i < JOIN_FEW; ++i)
                if (i < n) m = fmaxf(m, ml[i].x);
            const float base = m == -INFINITY ? 0.f : m;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < JOIN_FEW; ++i)
                if (i < n) {
                    const float k = exp2_of(ml[i].x - base);
                    l += k * ml[i].y;
                    o.x += k * x[i].x, o.y += k * x[i].y, o.z += k * x[i].z, o.w += k * x[i].w;
                }
            write(begun, r, d4, o.x, m, l);
            write(begun, r, d4 + 1, o.y, m, l);
            write(begun, r, d4 + 2, o.z, m, l);
            write(begun, r, d4 + 3, o.w, m, l);
        }
    }
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const Cut cut = side ? went_on : begun;
        if (cut.parts <= JOIN_FEW) continue;
        const int n = cut.parts, g = tid / (COLS / 4), d4 = tid % (COLS / 4) * 4;
        for (int item = (int)blockIdx.x - cut.block; item < 4 * cut.rows; item += n) {
            const int r = item >> 2, col = (item & 3) * COLS;
            // BATCH parts a thread at a time, with the running maximum
            float m = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = g; i0 < n; i0 += BATCH * GROUPS) {
                float2 ml[BATCH];
                float4 x[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int i = i0 + k * GROUPS;
                    ml[k] = make_float2(-INFINITY, 0.f);
                    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < n) {
                        ml[k] = A.part_ml[slot_of(cut, r, i)];
                        x[k] = *reinterpret_cast<const float4*>(A.part_o + slot_of(cut, r, i) * D + col + d4);
                    }
                }
                float top = m;
#pragma unroll
                for (int k = 0; k < BATCH; ++k) top = fmaxf(top, ml[k].x);
                const float base = top == -INFINITY ? 0.f : top, keep = exp2_of(m - base);
                m = top;
                l *= keep;
                o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const float w = exp2_of(ml[k].x - base);
                    l += w * ml[k].y;
                    o.x += w * x[k].x, o.y += w * x[k].y, o.z += w * x[k].z, o.w += w * x[k].w;
                }
            }
            *reinterpret_cast<float4*>(&part[g][d4]) = o;
            if (d4 == 0) gm[g] = m, gl[g] = l;
            __syncthreads();
            if (tid < COLS) {
                float M = -INFINITY, v = 0.f;
                l = 0.f;
#pragma unroll
                for (int k = 0; k < GROUPS; ++k) M = fmaxf(M, gm[k]);
                const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int k = 0; k < GROUPS; ++k) {
                    const float w = exp2_of(gm[k] - base);
                    l += w * gl[k];
                    v += w * part[k][tid];
                }
                write(cut, r, col + tid, v, M, l);
            }
            __syncthreads();
        }
    }
}

constexpr int BLOCKS_PER_SM = 2;

int attn_blocks() { return num_sms() * BLOCKS_PER_SM; }

template <int D, int TY, bool WIDE>
int launch(AttnArgs a, cudaStream_t s) {
    a.rows = WIDE ? 16 : 8;
    a.unit = Tile<D>::UNIT;
    a.job_cost = Tile<D>::JOB_COST;
    const size_t sched = (size_t)a.B * sizeof(uint32_t);
    const size_t sm = sizeof(AttnSmem<D>) + sched;
    static std::atomic<uint64_t> asked{0};
    if (!allow_smem((const void*)k_attn<D, TY, WIDE>, sizeof(AttnSmem<D>) + E0_MAX_SEQS * sizeof(uint32_t), asked))
        return E0_ERR_CUDA;
    k_attn<D, TY, WIDE><<<a.blocks, AT_WARPS * 32, sm, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return E0_ERR_CUDA;
    // No join where every schedule is a job a block: no more jobs than blocks whatever the
    // sequences have, and no context so long that a share could be too short for it
    // (16 sequences of up to 500, 8 heads of 64: 8.7 us against 10.0).
    const long long tiles = ((long long)a.max_q * (a.Hq / a.Hkv) + a.rows - 1) / a.rows;
    const long long seen = a.window > 0 ? (long long)a.window + a.max_q + a.unit : LLONG_MAX;
    const long long most = min(seen, (long long)a.max_blocks << a.shift);
    if (a.B * tiles * a.Hkv <= a.blocks && (most + a.unit - 1) / a.unit <= 2 * a.job_cost + 2) return E0_OK;
    // the join's blocks start while those above still run and wait for all of them
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.blocks);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attn_join<D, TY>, a) == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

template <int TY, bool WIDE>
int launch_d(const AttnArgs& a, int D, cudaStream_t s) {
    return D == 64 ? launch<64, TY, WIDE>(a, s) : D == 128 ? launch<128, TY, WIDE>(a, s) : launch<256, TY, WIDE>(a, s);
}

}  // namespace

size_t attn_ws_bytes(int D) {
    const size_t slots = 2 * (size_t)attn_blocks();
    return slots * MOST_ROWS * D * sizeof(float) + slots * MOST_ROWS * sizeof(float2) + slots * sizeof(Cut);
}

int attn_decode(const e0_kv_cache* c, const int32_t* table, int max_blocks, const int32_t* ctx, const int32_t* cu,
                int B, int max_q, const void* q, int dtype, int64_t q_ld, int Hq, float scale, int window, void* out,
                int64_t out_ld, float* lse, void* ws, uint32_t* st, cudaStream_t s) {
    AttnArgs a = {};
    a.k = c->k, a.v = c->v, a.ks = c->k_scale, a.vs = c->v_scale;
    a.table = table, a.ctx = ctx, a.cu = cu, a.q = q, a.out = out, a.lse = lse;
    a.blocks = attn_blocks();
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + 2 * (size_t)a.blocks * MOST_ROWS * c->D);
    a.cuts = reinterpret_cast<Cut*>(a.part_ml + 2 * (size_t)a.blocks * MOST_ROWS);
    a.st = st, a.q_ld = q_ld, a.out_ld = out_ld;
    a.B = B, a.max_blocks = max_blocks, a.n_blocks = c->n_blocks, a.Hq = Hq, a.Hkv = c->Hkv, a.max_q = max_q;
    a.window = window, a.scale = scale;
    while ((1 << a.shift) < c->block_tokens) ++a.shift;
    if (dtype == E0_F32) return launch_d<E0_F32, false>(a, c->D, s);
    if (dtype == E0_F16) return launch_d<E0_F16, false>(a, c->D, s);
    const bool wide = (int64_t)max_q * (Hq / c->Hkv) > 8;
    return wide ? launch_d<E0_BF16, true>(a, c->D, s) : launch_d<E0_BF16, false>(a, c->D, s);
}

}  // namespace e0
