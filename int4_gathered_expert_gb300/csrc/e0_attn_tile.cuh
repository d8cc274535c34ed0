// Attention of many query rows over the paged 8-bit KV cache on the 5th-generation tensor
// cores: prompts of e0_attn_scored, and the shared prefix of e0_attn_shared.
#pragma once
#include "e0_attn.cuh"
#include "e0_umma.cuh"

namespace e0 {
namespace {

// One pass over the keys with the running maximum and sum, as in e0_attn.cuh, for tiles of
// many query rows.  A job is a (sequence, KV head, tile of query rows); its context is cut
// into units of KV positions, and the units of all jobs are dealt out evenly, one block an
// SM.  Every row sees one range of positions, so a job's units are those that some row of it
// sees, and masks are two comparisons.  Jobs that several blocks have are joined.
//
// A block's roles:
//   - four warps turn a unit's codes into fp16 operands in shared memory (keys and values in
//     the same order: 8 tokens x 8 elements are 128 bytes in a row, no swizzle; keys are then
//     K-major, values MN-major), the next unit's codes already in registers;
//   - one thread issues the products: S = Q K^T into tensor memory, O += P V with P from
//     tensor memory;
//   - four warps a half of the rows, a thread a row (so that maxima and sums need no
//     exchange), turn S into P where S was.
// With D up to 128 the tile has 256 rows in two halves, one half's products run under the other's
// exponentials, and both read the same operands; with D = 256 tensor memory holds one half
// and two S.
// fp16 operands: codes widen exactly; bf16 queries go in times a power of two of the
// row, fp16 ones as they are; the weights 2^(t - m + TILE_LIFT), at most 2^15, go in as an fp16 part and
// their rests, a product each: 22 bits for outputs of either type, as in e0_attn.cuh for up to 8 rows, so
// that a call's bits do not depend on its path beyond what fp32 sums in another order do.  (bf16 outputs
// without the rests: 116 us a call for 129, the documents below, and 61 for 66 behind a prefix of 16000, but
// one output in 25 rounded to the other side of a step.)
//
// Products are issued by one thread and done in its order: a unit's first products go where the
// weights of the unit before were as soon as that one's second products have been issued.
//
// Measured (device time, GB300; heads of 128, 32 on 4, bf16): 4096 tokens of five documents 126 us, 276 TFLOP/s of
// what is seen; the same tokens as one document 229 us, 600 TFLOP/s.  What bounds it, by the clock in a copy, in cycles
// a unit of 128 positions and 256 rows (5.9 thousand with one document, 6.8 with five): a half's softmax, 3.4 thousand
// of a thread's own instructions and their latencies, behind which its products have to wait, 2.5 thousand (3.2 with
// five), for there is room for one S a half.  The products by themselves would be 3.1 thousand, three of 1024 (S, O
// by the weights, O by their rests) at 8192 a cycle.  The end of a piece of a job costs 5 to 6 thousand, its start
// as much; of the documents' 126 us the schedule takes about 6 beside its launch, the join 8.
template <int D>
struct Geo {
    static constexpr int HALVES = D == 256 ? 1 : 2;
    static constexpr int ROWS = 128 * HALVES;
    static constexpr int KV = D == 256 ? 64 : 128;
    static constexpr int STAGES = D == 64 ? 3 : 2;
    static constexpr int OPERAND = KV * D * 2;
    static constexpr int SOFT = 4 * HALVES;  // softmax warps
    static constexpr int OPS = HALVES == 2 ? 2 : 1;  // operands of a converting warp: keys and values, or one of them
    static constexpr int TURN = 8 / OPS;             // converting warps
    static constexpr int THREADS = (SOFT + TURN + 4) * 32;  // of the last four, one issues the products
    // Registers of a softmax, a converting and another thread: together what was launched, 512 x 128.
    // With heads of 256, whose softmax has four warps, there is room for eight converting ones (20
    // times two queries over 6000 positions: 56 us with four, 52 with eight); with others it would be
    // 640 threads of 96, and softmax's and the operands' registers in local memory (4096 tokens of
    // documents, weights without rests: 113 us with four, 126 with eight).
    static constexpr int SOFT_REGS = HALVES == 2 ? 168 : 208, TURN_REGS = HALVES == 2 ? 112 : 88, OTHER_REGS = HALVES == 2 ? 64 : 128;
    static_assert(32 * (SOFT * SOFT_REGS + TURN * TURN_REGS + 4 * OTHER_REGS) == THREADS * 128 && THREADS == 512, "all of them come");
    static constexpr int O_COL = 2 * KV;  // tensor memory: two S, then the halves' O
    static constexpr int Q_BYTES = 128 * D * 2;             // of a half
    static constexpr int Q_BUFS = D == 256 ? 1 : 3;         // halves' Q in shared memory
    static constexpr int Q_WARPS = 3;                       // that bring it there
    static constexpr int LOADS = KV * D / (4 * 512);  // 16-byte loads of a converting lane for one operand
};
// Weights are 2^(t - m + TILE_LIFT) and m follows where t has grown by more than TILE_SLACK, so
// that fp16's 2^15 is not passed: the rows of a warp seldom need O scaled after their first
// scores, and every such time holds up both halves.  m's own weight is 2^3; what fp16 has no
// steps for is 2^-28 of that.
constexpr float TILE_LIFT = 3.f, TILE_SLACK = 12.f;
// What a job costs beside its units (its rows of Q, its result, two halves that start and
// stop), in units: 10 to 12 thousand cycles of about six.  Dealt out by units alone the blocks with
// the first rows of prompts, a unit a job, were twice as long as the others.
constexpr uint32_t TILE_JOB_COST = 2;
constexpr uint32_t TILE_TMEM = 512;
constexpr uint64_t TILE_WAIT_NS = 2000000000ull;  // 2 s

struct TileJob {
    int seq, mtile, unit0, units;  // the first unit, how many
    int k0[2], k1[2];              // of each half: its units, counted from unit0
    int lo, hi, full_lo, full_hi;  // positions that some row sees; that all rows see
    uint32_t start;                // place in the schedule of the first head's first unit
    int row0, rows, p0;            // query rows: the sequence's first; of this tile (heads x tokens); position of its token 0
};
struct TileCut {
    int parts, block, job, head;  // parts 0: none
};
struct TileHead {
    uint32_t total, share;
    int jobs, pad;
};

// No position: those of queries are -2^30 and more (a sequence may have more queries than tokens).
constexpr int NO_ROW = INT_MIN;

struct TileArgs {
    AttnArgs a;               // parts and cuts unused
    // A prefix (own.B > 0): `own` are the sequences whose rows are the one job's; their positions
    // behind the prefix go to own_at, NO_ROW where a row is no sequence's.
    AttnArgs own;
    int32_t* own_at;
    const float* own_o;       // merge: the sequences' own results, normed, and their lse
    const float* own_lse;
    bool merge;               // every piece of a job is a part; the join ends the rows with the own results
    float* part_o;            // [2 * blocks][ROWS][D]
    float2* part_ml;          // [2 * blocks][ROWS]
    TileCut* cuts;            // [blocks]: the job that the block began and left unfinished
    TileJob* jobs;
    int4* begin;              // [blocks]: job, head, unit
    TileHead* head;
    int blocks, most_jobs;
    uint32_t by_group;        // n / G = n * by_group >> 31 + by_shift for n below 2^31
    int by_shift;
    bool vec_out, out_16;     // rows of out start on 8 bytes, on 16
};

E0_DEV int div_group(const TileArgs& A, int n) { return (int)((unsigned long long)(uint32_t)n * A.by_group >> (31 + A.by_shift)); }

// The range of positions that a token of a sequence sees.
E0_DEV void range_of(const TileArgs& A, int seq, int row0, int p0, int ctx, int i, int& p, int& lo, int& hi) {
    p = !A.a.at ? p0 + i : A.a.window > 0 || A.a.slopes ? A.a.at[row0 + i] : 0;  // needed there alone
    hi = !A.a.at ? p + 1 : p == NO_ROW ? 0 : ctx;
    p = max(p, -(1 << 30));  // no distance from NO_ROW passes 32 bits
    if (A.a.open) hi = max(hi, A.a.open[seq]);
    hi = min(hi, ctx);
    lo = A.a.window > 0 ? max(p - A.a.window + 1, 0) : 0;
    if (A.a.first) lo = max(lo, A.a.first[row0 + i]);
}

// ---------------------------------------------------------------- the schedule

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_SHARED = 6144;  // jobs whose places are kept in shared memory

// One block, and chains of loads: 6 us beside the launch for 128 tiles of one sequence.
template <int D>
__global__ void __launch_bounds__(PLAN_THREADS) k_tile_plan(TileArgs A) {
    typedef Geo<D> G_;
    extern __shared__ uint32_t tiles_before[];  // [B + 1], then the jobs' units and places
    __shared__ uint32_t red[32];
    __shared__ uint32_t carry;
    __shared__ int all_rows;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = A.a.B, G = A.a.Hq / A.a.Hkv;
    uint32_t* place = tiles_before + B + 1;
    const auto block_scan = [&](uint32_t v, uint32_t& all) {  // exclusive
        const uint32_t own = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v = add_units(v, t);
        }
        __syncthreads();
        if (lane == 31) red[warp] = v;
        __syncthreads();
        uint32_t w = red[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w = add_units(w, t);
        }
        all = __shfl_sync(0xffffffffu, w, 31);
        const uint32_t before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
        return add_units(before, v - own);
    };
    if (tid == 0) all_rows = 0, carry = 0;
    if (A.own.B > 0) {
        for (int t = tid; t < A.own.limit; t += PLAN_THREADS) A.own_at[t] = NO_ROW;
        __syncthreads();
        const int before = prefix_of(*A.a.ctx, A.a.max_blocks, A.a.shift);
        for (int b = warp; b < A.own.B; b += PLAN_THREADS / 32) {
            const Seq s = seq_of<true>(A.own, b, false);
            for (int i = lane; i < s.n; i += 32) A.own_at[s.row0 + i] = before + s.ctx - s.n + i;
            if (lane == 0 && s.n > 0) atomicMax(&all_rows, s.row0 + s.n);
        }
        __syncthreads();
    }
    const auto sequence = [&](int b, bool tell) {
        if (A.own.B == 0) return seq_of<true>(A.a, b, tell);
        Seq s;
        const int given = *A.a.ctx;
        s.row0 = 0, s.n = all_rows, s.ctx = prefix_of(given, A.a.max_blocks, A.a.shift);
        if (s.ctx != given && tell && tid == 0) set_status(A.a.st, E0_ST_BAD_LENGTH);
        return s;
    };
    // tiles of query rows of each sequence
    uint32_t at = 0;
    for (int b0 = 0; b0 < B; b0 += PLAN_THREADS) {
        const int b = b0 + tid;
        uint32_t n = 0, all;
        if (b < B) n = (uint32_t)(((long long)sequence(b, true).n * G + G_::ROWS - 1) / G_::ROWS);
        const uint32_t before = block_scan(n, all);
        if (b < B) tiles_before[b] = at + before;
        at = add_units(at, all);
    }
    if (tid == 0) tiles_before[B] = at;
    __syncthreads();
    const int jobs = (int)min(at, (uint32_t)A.most_jobs);
    // a warp a job: what its rows see
    for (int j = warp; j < jobs; j += PLAN_THREADS / 32) {
        int b = 0, end = B;
        while (end - b > 1) {
            const int mid = (b + end) >> 1;
            if (tiles_before[mid] <= (uint32_t)j) b = mid; else end = mid;
        }
        while (tiles_before[b + 1] <= (uint32_t)j) ++b;  // sequences without rows share a place
        const Seq s = sequence(b, false);
        TileJob J;
        J.seq = b, J.mtile = j - (int)tiles_before[b], J.row0 = s.row0, J.p0 = s.ctx - s.n;
        const int r0 = J.mtile * G_::ROWS;
        J.rows = min(G_::ROWS, s.n * G - r0);
        J.lo = J.full_hi = INT_MAX, J.hi = J.full_lo = 0;
        int u0 = INT_MAX, u1 = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            J.k0[h] = J.k1[h] = 0;
            const int ra = r0 + 128 * h, rb = r0 + min(J.rows, 128 * (h + 1));
            if (h >= G_::HALVES || ra >= rb) continue;
            int lo = INT_MAX, hi = 0, most = 0, least = INT_MAX;
            for (int i = div_group(A, ra) + lane; i <= div_group(A, rb - 1); i += 32) {
                int p, l, e;
                range_of(A, b, s.row0, J.p0, s.ctx, i, p, l, e);
                if (l < e) lo = min(lo, l), hi = max(hi, e);
                most = max(most, l), least = min(least, e);
            }
            lo = __reduce_min_sync(0xffffffffu, lo), hi = __reduce_max_sync(0xffffffffu, hi);
            J.full_lo = max(J.full_lo, __reduce_max_sync(0xffffffffu, most));
            J.full_hi = min(J.full_hi, __reduce_min_sync(0xffffffffu, least));
            if (lo >= hi) continue;
            J.lo = min(J.lo, lo), J.hi = max(J.hi, hi);
            J.k0[h] = lo / G_::KV, J.k1[h] = (hi - 1) / G_::KV + 1;
            u0 = min(u0, J.k0[h]), u1 = max(u1, J.k1[h]);
        }
        if (u1 == 0) u0 = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (J.k1[h] > 0) J.k0[h] -= u0, J.k1[h] -= u0;
        J.unit0 = u0, J.units = max(u1 - u0, 1);  // a job without context still writes its rows
        J.start = 0;
        if (lane == 0) {
            A.jobs[j] = J;
            if (j < PLAN_SHARED) place[2 * j] = J.units;
        }
    }
    __syncthreads();
    // their places in the schedule
    for (int j0 = 0; j0 < jobs; j0 += PLAN_THREADS) {
        const int j = j0 + tid;
        uint32_t n = 0, all;
        if (j < jobs) {
            const unsigned long long u = (unsigned long long)((j < PLAN_SHARED ? (int)place[2 * j] : A.jobs[j].units) + TILE_JOB_COST) * A.a.Hkv;
            n = u < MOST_UNITS ? (uint32_t)u : MOST_UNITS;
        }
        const uint32_t before = block_scan(n, all);
        if (j < jobs) {
            const uint32_t start = add_units(carry, before);
            A.jobs[j].start = start;
            if (j < PLAN_SHARED) place[2 * j + 1] = start;
        }
        __syncthreads();
        if (tid == 0) carry = add_units(carry, all);
        __syncthreads();
    }
    uint32_t total = carry;
    if (total >= MOST_UNITS || at > (uint32_t)A.most_jobs) {
        if (tid == 0) set_status(A.a.st, E0_ST_BAD_LENGTH);
        total = 0;
    }
    const uint32_t share = max((total + A.blocks - 1) / A.blocks, TILE_JOB_COST + 1);
    if (tid == 0) *A.head = {total, share, jobs, 0};
    for (int c = tid; c < A.blocks; c += PLAN_THREADS) {
        const uint32_t u = c * share;
        int4 to = make_int4(-1, 0, 0, 0);
        if (u < total) {
            const auto start = [&](int j) { return j < PLAN_SHARED ? place[2 * j + 1] : A.jobs[j].start; };
            int lo = 0, hi = jobs;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (start(mid) <= u) lo = mid; else hi = mid;
            }
            const uint32_t rel = u - start(lo), len = (lo < PLAN_SHARED ? place[2 * lo] : A.jobs[lo].units) + TILE_JOB_COST;
            to = make_int4(lo, (int)(rel / len), (int)(rel % len), 0);
        }
        A.begin[c] = to;
    }
    // what went before may still be running: the kernels after this one wait for it through here
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------- a block's pieces of jobs

struct Piece {
    TileJob J;
    int job, head, k0, k1;  // units k0..k1-1 of the job
    // the units of the piece that half h has (no index that is not a constant: J stays in registers)
    E0_DEV int first(int h) const { return max(k0, h ? J.k0[1] : J.k0[0]); }
    E0_DEV int end(int h) const { return min(k1, h ? J.k1[1] : J.k1[0]); }
    E0_DEV bool all() const { return k0 == 0 && k1 == J.units; }
};

// The first jobs of a block's are in shared memory from the start.
constexpr int AT_HAND = 12;

struct Pieces {
    const TileArgs& A;
    const TileJob* near;
    int near0;
    uint32_t left;
    int job, head, k;
    E0_DEV Pieces(const TileArgs& args, const TileJob* at_hand) : A(args), near(at_hand), near0(0), left(0), job(-1), head(0), k(0) {
        const TileHead h = *A.head;
        const uint32_t u = blockIdx.x * h.share;
        if (u < h.total) {
            const int4 b = A.begin[blockIdx.x];
            job = near0 = b.x, head = b.y, k = b.z;
            left = min(h.share, h.total - u);
        }
    }
    E0_DEV bool next(Piece& p) {
        while (left > 0) {
            int4 a, b, c, d;
            if (job - near0 < AT_HAND) {
                const int4* from = reinterpret_cast<const int4*>(near + (job - near0));
                a = from[0], b = from[1], c = from[2], d = from[3];
            } else {
                const int4* from = reinterpret_cast<const int4*>(A.jobs + job);
                a = __ldcg(from), b = __ldcg(from + 1), c = __ldcg(from + 2), d = __ldcg(from + 3);
            }
            p.J = {a.x, a.y, a.z, a.w, {b.x, b.y}, {b.z, b.w}, c.x, c.y, c.z, c.w, (uint32_t)d.x, d.y, d.z, d.w};
            p.job = job, p.head = head;
            // places k .. of the job: its cost, then its units
            const int places = min(p.J.units + (int)TILE_JOB_COST - k, (int)left);
            p.k0 = max(k - (int)TILE_JOB_COST, 0);
            p.k1 = k + places - (int)TILE_JOB_COST;
            left -= places;
            k = 0;
            if (++head == A.a.Hkv) head = 0, ++job;
            if (p.k1 > p.k0) return true;  // otherwise a part of its cost: the units are the next block's
        }
        return false;
    }
};
static_assert(sizeof(TileJob) == 64, "four 16-byte loads");

// ---------------------------------------------------------------- operands

// Operand descriptor without swizzle: 8 x 16-byte blocks of 128 bytes, `lead` and `stride`
// bytes apart.  K-major: lead from 8 elements of k to the next, stride from 8 rows to the
// next; MN-major: lead from 8 elements of k to the next, stride from 8 elements of the other
// side to the next.  Low word: address and lead in 16-byte units; high word: stride, version 1.
E0_DEV uint32_t desc_low(uint32_t addr, uint32_t lead) { return ((addr >> 4) & 0x3FFFu) | (lead >> 4) << 16; }
constexpr uint32_t desc_high(uint32_t stride) { return (stride >> 4) | 1u << 14; }
// umma_f16 and umma_f16_ta with descriptors by their words: what changes from one product to
// the next is one 32-bit addition.
E0_DEV void umma_lo(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
E0_DEV void umma_ta_lo(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
E0_DEV bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
constexpr uint32_t B_MN_MAJOR = 1u << 16;  // of the instruction descriptor

E0_DEV void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
E0_DEV void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

template <int D>
struct TileSmem {
    uint8_t q[Geo<D>::Q_BUFS][Geo<D>::Q_BYTES];
    uint8_t k[Geo<D>::STAGES][Geo<D>::OPERAND];
    uint8_t v[Geo<D>::STAGES][Geo<D>::OPERAND];
    TileJob jobs[AT_HAND];
    float4 sc[Geo<D>::STAGES][Geo<D>::KV / 16];  // of 16 tokens: keys' scale, values' log2 and inverse, seen (1) or not
    uint64_t k_full[Geo<D>::STAGES], k_empty[Geo<D>::STAGES], v_full[Geo<D>::STAGES], v_empty[Geo<D>::STAGES];
    float qf[Geo<D>::Q_BUFS][128];               // of a row of Q: what its scores want
    uint64_t q_full[Geo<D>::Q_BUFS], q_empty[Geo<D>::Q_BUFS];
    uint64_t s_full[2], p_full[2][2], o_half[2], o_done[2], drained;
    uint32_t tmem, abort;
};

static_assert(sizeof(TileSmem<64>) <= 232448 && sizeof(TileSmem<128>) <= 232448 && sizeof(TileSmem<256>) <= 232448, "227 KB");

// 16 codes as 16 fp16: two 16-byte chunks.
E0_DEV void widen16(const uint4 c, uint4& a, uint4& b) {
    a = make_uint4(e4m3x2_to_half2((uint16_t)c.x), e4m3x2_to_half2((uint16_t)(c.x >> 16)), e4m3x2_to_half2((uint16_t)c.y),
                   e4m3x2_to_half2((uint16_t)(c.y >> 16)));
    b = make_uint4(e4m3x2_to_half2((uint16_t)c.z), e4m3x2_to_half2((uint16_t)(c.z >> 16)), e4m3x2_to_half2((uint16_t)c.w),
                   e4m3x2_to_half2((uint16_t)(c.w >> 16)));
}

// (a0 * f + c, a1 * f + c) and (s0 + a, s1 + b), a pair an instruction.
E0_DEV void fma2(float& r0, float& r1, float a0, float a1, float f, float c) {
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mov.b64 z, {%5, %5};\n"
        " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
        : "=f"(r0), "=f"(r1)
        : "f"(a0), "f"(a1), "f"(f), "f"(c));
}
E0_DEV void add2(float& s0, float& s1, float a, float b) {
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
        : "+f"(s0), "+f"(s1)
        : "f"(a), "f"(b));
}
E0_DEV void mul2(float& r0, float& r1, float a0, float a1, float f) {
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
        : "=f"(r0), "=f"(r1)
        : "f"(a0), "f"(a1), "f"(f));
}
// (a0 * b0 + c, a1 * b1 + c)
E0_DEV void fma2_by(float& r0, float& r1, float a0, float a1, float b0, float b1, float c) {
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %6};\n"
        " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
        : "=f"(r0), "=f"(r1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c));
}
// 16 bytes on their way to shared memory, zeros where there are none.
E0_DEV void copy16_or_zero(uint8_t* dst, const void* src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(have ? 16 : 0)
                 : "memory");
}
E0_DEV float inverse_of(float x) {  // a step of fp32 off
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// x = cap tanh(x / cap) of 64 scores: a polynomial where none of the warp's is beyond the cap,
// otherwise cap - 2 cap / (1 + e^(2 x / cap)), two steps of fp32 of cap off.
E0_DEV void cap_scores(float (&x)[64], float cap, float inv_cap) {
    float top[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        top[y] = fmaxf(fabsf(x[y]), fabsf(x[4 + y]));
#pragma unroll
        for (int j = 8; j < 64; j += 8) top[y] = fmaxf(fmaxf(top[y], fabsf(x[j + y])), fabsf(x[j + 4 + y]));
    }
    // A score takes the form that its own size asks for (NaN the polynomial, which keeps it): a row's result
    // knows nothing of what its neighbours, or places that nobody sees, hold.
    const auto below = [&](int j, float& p0, float& p1) {  // cap (x / cap) p of a pair
        float u0, u1, v0, v1;
        mul2(u0, u1, x[j], x[j + 1], inv_cap);
        fma2_by(v0, v1, u0, u1, u0, u1, 0.f);
        fma2(p0, p1, v0, v1, tanh_of(7), tanh_of(6));
#pragma unroll
        for (int i = 5; i >= 0; --i) fma2_by(p0, p1, p0, p1, v0, v1, tanh_of(i));
        fma2_by(p0, p1, x[j], x[j + 1], p0, p1, 0.f);
    };
    if (!__any_sync(0xffffffffu, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > cap)) {
#pragma unroll
        for (int j = 0; j < 64; j += 2) {
            float p[2];
            below(j, p[0], p[1]);
            x[j] = p[0], x[j + 1] = p[1];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 64; j += 2) {
            float p[2];
            below(j, p[0], p[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float e = exp2_of(fminf(x[j + i] * inv_cap * (2.f * LOG2E), 126.f));
                x[j + i] = fabsf(x[j + i]) > cap ? fmaf(-2.f * cap, inverse_of(1.f + e), cap) : p[i];
            }
        }
    }
}
// Bits 0 .. n-1, n any number.
E0_DEV uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1; }

// 32 columns of fp32 in tensor memory times `keep` of the row.
E0_DEV void scale32(uint32_t at, float keep) {
    uint32_t u[32];
    tmem_ld32(at, u);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * keep);
    tmem_st32(at, u);
}

// Where element `col` (a multiple of four) of a part's row is.
template <int D>
E0_DEV size_t part_at(int slot, int row, int col) {
    return (size_t)slot * Geo<D>::ROWS * D + (size_t)(row / 8) * (8 * D) + col * 8 + (row & 7) * 4;
}

template <int TY>
E0_DEV void put_row4(const AttnArgs& a, bool vec, size_t tok, int col, float x, float y, float z, float w) {
    if (a.raw) {
        *reinterpret_cast<float4*>(a.raw + tok * ((size_t)a.Hq * a.D) + col) = make_float4(x, y, z, w);
        return;
    }
    typedef typename Elem<TY>::T T;
    T* to = reinterpret_cast<T*>(a.out) + tok * a.out_ld + col;
    if (vec) {
        *reinterpret_cast<uint2*>(to) = make_uint2(pack16<TY>(x, y), pack16<TY>(z, w));
    } else {
        to[0] = Elem<TY>::put(x), to[1] = Elem<TY>::put(y), to[2] = Elem<TY>::put(z), to[3] = Elem<TY>::put(w);
    }
}

// Wait for a barrier's phase, 2 s at most or until *abort.  The barrier's own test sleeps until the
// phase ends or a while has passed; no sleep of a given length, which would go on after
// the phase's end, and the clock only now and then: of 36 million instructions 17 had been waiting.
E0_DEV bool arrived(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort) {
    uint64_t t0 = 0;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        const uint64_t t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > TILE_WAIT_NS) return false;
    }
}

// ---------------------------------------------------------------- the kernel

// TY: E0_F16 or E0_BF16.  RULES: scores are capped or lose with the distance.
template <int D, int TY, bool RULES>
__global__ void __launch_bounds__(Geo<D>::THREADS, 1) k_attn_tile(const __grid_constant__ TileArgs A) {
    typedef Geo<D> G_;
    typedef typename Elem<TY>::T T;
    constexpr int KV = G_::KV, STAGES = G_::STAGES, HALVES = G_::HALVES, CHUNKS = KV / 64;
    extern __shared__ __align__(1024) char tile_sm[];
    TileSmem<D>& S = *reinterpret_cast<TileSmem<D>*>(tile_sm);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = A.a.Hq / A.a.Hkv;
    volatile uint32_t* abort = &S.abort;
    const volatile uint32_t never = 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&S.k_full[s], 4), mbar_init(&S.v_full[s], 4);
            mbar_init(&S.k_empty[s], 1), mbar_init(&S.v_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&S.s_full[s], 1), mbar_init(&S.o_done[s], 1);
            mbar_init(&S.p_full[s][0], 4), mbar_init(&S.p_full[s][1], 4), mbar_init(&S.o_half[s], 1);
        }
        for (int s = 0; s < G_::Q_BUFS; ++s) mbar_init(&S.q_full[s], G_::Q_WARPS), mbar_init(&S.q_empty[s], 4);
        mbar_init(&S.drained, 1);
        S.abort = 0;
        mbar_fence_init();
    }
    if (warp == G_::SOFT + G_::TURN) tmem_alloc(&S.tmem, TILE_TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    const auto give_up = [&]() {
        *abort = 1;
        set_status(A.a.st, E0_ST_TIMEOUT);
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the schedule is there
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    {
        const int job0 = A.begin[blockIdx.x].x, i = threadIdx.x;  // -1: the block has nothing to do
        if (i < AT_HAND * 4 && job0 >= 0 && job0 + i / 4 < A.head->jobs)
            reinterpret_cast<int4*>(S.jobs)[i] = __ldcg(reinterpret_cast<const int4*>(A.jobs + job0) + i);
        __syncthreads();
    }
    Pieces pieces(A, S.jobs);

    if (warp < G_::SOFT) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G_::SOFT_REGS));
        // ---------------- softmax: a thread a row, half h of the tile
        const int h = warp >> 2, t = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t o_at = tmem + lanes + G_::O_COL + h * D;
        uint32_t n_s = 0;  // S of this half so far
        uint32_t gk = 0;   // units of the block before this piece
        uint32_t n_q = 0;  // halves with units before this piece
        bool ok = true;
        // The second products of this half's n-th S are done.  (A warp may be two units ahead of
        // another's P with one half: a barrier for even and one for odd units, so that a phase
        // is never mistaken for the one before the last.)
        const auto wait_o = [&](uint32_t n) {
            return HALVES == 2 ? arrived(&S.o_done[h], n & 1, abort)
                               : arrived(&S.o_done[n & 1], (n >> 1) & 1, abort);
        };
        Piece p;
        TileCut begun = {0, 0, 0, 0};
        while (ok && pieces.next(p)) {
            const TileJob& J = p.J;
            const int r = J.mtile * G_::ROWS + 128 * h + t;  // row of the sequence: token, head of the group
            const bool row_ok = 128 * h + t < J.rows;
            const int i = div_group(A, r), head = p.head * G + r - i * G;
            const size_t tok = (size_t)J.row0 + i;
            const int kf = p.first(h), ke = p.end(h);
            int pos = 0, lo = 0, hi = 0;
            if (row_ok) range_of(A, J.seq, J.row0, J.p0, J.hi, i, pos, lo, hi);
            float mx = -INFINITY, sum = 0.f, f = 0.f, slope = 0.f;
            // the number of this half's Q, of all that the block has had
            const uint32_t nq = n_q + (h && p.first(0) < p.end(0)), qb = nq % G_::Q_BUFS;
            n_q += (p.first(0) < p.end(0)) + (HALVES == 2 && p.first(1) < p.end(1));
            if (RULES && kf < ke && A.a.slopes && row_ok) slope = A.a.slopes[head] * LOG2E;
            // ---- units
            for (int k = kf; k < ke; ++k, ++n_s) {
                const uint32_t g = gk + (uint32_t)(k - p.k0), st = g % STAGES;
                const uint32_t slot = HALVES == 2 ? h : n_s & 1, use = HALVES == 2 ? n_s : n_s >> 1;
                const uint32_t s_at = tmem + lanes + slot * KV;
                // S first: a half without units in some pieces comes here well before the other, and
                // its S alone says that the other barriers are in the phases that are asked for
                ok = arrived(&S.s_full[slot], use & 1, abort) &&
                     arrived(&S.v_full[st], (g / STAGES) & 1, abort) &&
                     (k > kf || arrived(&S.q_full[qb], (nq / G_::Q_BUFS) & 1, abort));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (k == kf) f = S.qf[qb][t];
                const int at0 = (J.unit0 + k) * KV;
                bool edge = at0 < lo || at0 + KV > hi;
                if (lane < KV / 16) edge |= !(S.sc[st][lane].w > 0.f);
                edge = __any_sync(0xffffffffu, edge);
                const float away = (float)(pos - at0);
                float base = (mx == -INFINITY ? 0.f : mx) - TILE_LIFT;
#pragma unroll 1
                for (int c = 0; c < CHUNKS; ++c) {
                    uint32_t u[2][32];
                    tmem_ld32(s_at + 64 * c, u[0]);
                    tmem_ld32(s_at + 64 * c + 32, u[1]);
                    // x = t - base of 64 positions
                    float x[64], top[4];
                    float iv[4];  // of 16 positions: values' inverse
                    const float4* scales = &S.sc[st][4 * c];
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 sc = scales[q];
                        const float fk = f * sc.x, off = sc.y - base;
                        iv[q] = sc.z;
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float s0 = __uint_as_float(u[q / 2][16 * (q & 1) + j]);
                            const float s1 = __uint_as_float(u[q / 2][16 * (q & 1) + j + 1]);
                            if constexpr (RULES)
                                mul2(x[16 * q + j], x[16 * q + j + 1], s0, s1, fk);
                            else
                                fma2(x[16 * q + j], x[16 * q + j + 1], s0, s1, fk, off);
                        }
                    }
                    if constexpr (RULES) {
                        if (A.a.cap > 0.f) cap_scores(x, A.a.cap, A.a.inv_cap);
                        if (A.a.slopes) {
                            const float from = away - (float)(64 * c);
#pragma unroll
                            for (int j = 0; j < 64; ++j) x[j] = fmaf(-slope, fabsf(from - (float)j), x[j]);
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float off = scales[q].y - base;
#pragma unroll
                            for (int j = 0; j < 16; ++j) x[16 * q + j] += off;
                        }
                    }
                    if (edge) {
                        const int a = at0 + 64 * c;
                        uint32_t see[2] = {bits_below(hi - a) & ~bits_below(lo - a), bits_below(hi - a - 32) & ~bits_below(lo - a - 32)};
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (!(scales[q].w > 0.f)) see[q / 2] &= q & 1 ? 0xFFFFu : 0xFFFF0000u;
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (!(see[j / 32] & (1u << (j & 31)))) x[j] = -INFINITY;
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) {  // four chains of maxima, three operands each
                        top[y] = fmaxf(x[y], x[4 + y]);
#pragma unroll
                        for (int j = 8; j < 64; j += 8) top[y] = fmaxf(fmaxf(top[y], x[j + y]), x[j + 4 + y]);
                    }
                    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    // m follows where t has grown by more than TILE_SLACK; the first one is any
                    const bool grows = mx == -INFINITY ? most > -INFINITY : most > TILE_LIFT + TILE_SLACK;
                    if (__any_sync(0xffffffffu, grows)) {
                        const float now = grows ? most + base : mx, keep = mx == now ? 1.f : exp2_of(mx - now);
                        const float base_now = (now == -INFINITY ? 0.f : now) - TILE_LIFT, shift = base - base_now;
                        const bool had = grows && mx > -INFINITY;
                        mx = now, base = base_now;
                        sum *= keep;
#pragma unroll
                        for (int j = 0; j < 64; ++j) x[j] += shift;
                        // O of the units, or the positions, before, where a row had seen any (otherwise it is 0)
                        if ((k > kf || c > 0) && __any_sync(0xffffffffu, had)) {
                            ok = c > 0 ? arrived(&S.o_half[h], n_s & 1, abort) : wait_o(n_s - 1);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int y = 0; y < D / 32; ++y) scale32(o_at + 32 * y, keep);
                        }
                    }
                    float part[4];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t hi16[16], lo16[16];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float s0 = 0.f, s1 = 0.f;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float v = exp2_of(x[32 * b + 16 * q + 2 * j]), w = exp2_of(x[32 * b + 16 * q + 2 * j + 1]);
                                add2(s0, s1, v, w);
                                split_half(v, w, hi16[8 * q + j], lo16[8 * q + j]);
                            }
                            part[2 * b + q] = s0 + s1;
                        }
                        tmem_st16(s_at + 64 * c + 16 * b, hi16);
                        tmem_st16(s_at + 64 * c + 32 + 16 * b, lo16);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (iv[q] < INFINITY) sum = fmaf(part[q], iv[q], sum);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.p_full[slot][c]);
                }
                if (!ok) break;
            }
            if (!ok) break;
            gk += (uint32_t)(p.k1 - p.k0);
            // ---- the row's result, or its part: through shared memory, where Q was, COLS columns of
            // fp32 at a time, so that rows are written whole
            constexpr int COLS = D == 64 ? 32 : 64;
            static_assert(32 * COLS * 4 <= 32 * 2 * D, "the warp's rows of Q");
            const bool whole = p.all() && !A.merge;
            const int part = 2 * blockIdx.x + (p.k0 == 0 ? 1 : 0);
            if (kf < ke) {
                ok = wait_o(n_s - 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
            }
            if (kf >= ke) {  // nobody sees anything
                if (row_ok && whole)
                    for (int c = 0; c < D; c += 4) put_row4<TY>(A.a, A.vec_out, tok, head * D + c, 0.f, 0.f, 0.f, 0.f);
                if (row_ok && !whole)
                    for (int c = 0; c < D; c += 4)
                        *reinterpret_cast<float4*>(A.part_o + part_at<D>(part, 128 * h + t, c)) = make_float4(0.f, 0.f, 0.f, 0.f);
            } else if (!whole || A.a.raw) {
                // fp32: a part's columns stand by fours, eight rows of each together (part_at), so that a warp
                // writes whole lines
                const float inv = !whole ? 1.f : sum > 0.f || sum != sum ? SUM_UNIT / sum : 0.f;
                float* to = !whole ? A.part_o + part_at<D>(part, 128 * h + t, 0) : A.a.raw + (tok * A.a.Hq + head) * D;
                const int step = !whole ? 32 : 4;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t u[32];
                    tmem_ld32(o_at + 32 * c, u);
                    tmem_ld_wait();
                    if (row_ok)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4*>(to + (8 * c + j) * step) =
                                make_float4(__uint_as_float(u[4 * j]) * inv, __uint_as_float(u[4 * j + 1]) * inv,
                                            __uint_as_float(u[4 * j + 2]) * inv, __uint_as_float(u[4 * j + 3]) * inv);
                }
            } else {
                // through shared memory, where the warp's rows of Q were, so that rows are written whole
                constexpr int ROW = D / 8;  // chunks of 16 bytes, lanes of a row
                uint8_t* mine = S.q[qb] + 32 * (warp & 3) * (2 * D);
                const float inv = sum > 0.f || sum != sum ? SUM_UNIT / sum : 0.f;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t u[32];
                    tmem_ld32(o_at + 32 * c, u);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            w[z] = pack16<TY>(__uint_as_float(u[8 * j + 2 * z]) * inv, __uint_as_float(u[8 * j + 2 * z + 1]) * inv);
                        *reinterpret_cast<uint4*>(mine + lane * (2 * D) + (((4 * c + j) ^ (lane & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
                const int c = lane % ROW;
#pragma unroll 4
                for (int y = 0; y < ROW; ++y) {
                    const int row = y * (32 / ROW) + lane / ROW, in = 128 * h + 32 * (warp & 3) + row;
                    const uint4 v = *reinterpret_cast<const uint4*>(mine + row * (2 * D) + ((c ^ (row & 7)) << 4));
                    const int rr = J.mtile * G_::ROWS + in, ii = div_group(A, rr);
                    T* to = reinterpret_cast<T*>(A.a.out) + ((size_t)J.row0 + ii) * A.a.out_ld + (p.head * G + rr - ii * G) * D + 8 * c;
                    if (in >= J.rows) continue;
                    if (A.out_16) {
                        *reinterpret_cast<uint4*>(to) = v;
                    } else {
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            to[2 * z] = reinterpret_cast<const T*>(&w[z])[0];
                            to[2 * z + 1] = reinterpret_cast<const T*>(&w[z])[1];
                        }
                    }
                }
                __syncwarp();
            }
            tc_fence_before();  // O has been read before the next job's P is there
            __syncwarp();
            if (kf < ke && lane == 0) mbar_arrive(&S.q_empty[qb]);
            if (row_ok) {
                if (!whole)
                    A.part_ml[(size_t)part * G_::ROWS + 128 * h + t] = make_float2(mx, sum);
                else if (A.a.lse)
                    A.a.lse[tok * A.a.Hq + head] = lse_of(mx, sum, TILE_LIFT);
            }
            if (!whole && p.k0 == 0 && threadIdx.x == 0) {
                const uint32_t u0 = J.start + (uint32_t)p.head * (J.units + TILE_JOB_COST) + TILE_JOB_COST, share = A.head->share;
                const int b0 = (int)(u0 / share), b1 = (int)((u0 + J.units - 1) / share);
                begun = {b1 - b0 + 1, b0, p.job, p.head};
            }
        }
        if (!ok && lane == 0) give_up();
        if (threadIdx.x == 0) A.cuts[blockIdx.x] = begun;
    } else if (warp < G_::SOFT + G_::TURN) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G_::TURN_REGS));
        // ---------------- codes into operands, four warps an operand: block ids are read two units
        // ahead, codes and scales one
        const int cw = (warp - G_::SOFT) & 3, bs = 1 << A.a.shift;
        constexpr int OPS = G_::OPS;
        const int op0 = OPS == 2 ? 0 : (warp - G_::SOFT) >> 2;  // 0: keys (first), 1: values
        constexpr int L = G_::LOADS, PER = D / 64;  // loads; of 64 bytes a group of 8 tokens
        constexpr uint32_t NOWHERE = 0xFFFFFFFFu;
        constexpr int NOT_LOOKED_UP = INT_MIN;
        struct Unit {
            int at0, head, hi;
            int id;       // lane l < KV / 16: the block of its tokens 16 l ..., -1 for what is none; NOT_LOOKED_UP
            uint32_t at;  // ... and where they are, in 16 tokens; NOWHERE
            bool edge;    // some row does not see all of it: codes may be anything
        };
        Piece p;
        bool more = pieces.next(p);
        int k = more ? p.k0 : 0;
        const auto look_up = [&](Unit& u) {  // the next unit, if there is one
            if (!more) return false;
            const TileJob& J = p.J;
            u.at0 = (J.unit0 + k) * KV, u.head = p.head, u.hi = J.hi;
            u.edge = u.at0 < J.full_lo || u.at0 + KV > J.full_hi;
            const int at = u.at0 + 16 * lane;
            u.id = -1;
            if (lane < KV / 16 && at < J.hi && at + 16 > J.lo) u.id = max(A.a.table[(size_t)J.seq * A.a.max_blocks + (at >> A.a.shift)], -1);
            else if (lane < KV / 16) u.id = NOT_LOOKED_UP;
            if (++k == p.k1) {
                more = pieces.next(p);
                k = p.k0;
            }
            return true;
        };
        // the id's bounds, its scales
        const auto look_in = [&](Unit& u, float& ks, float& vs) {
            if (lane < KV / 16 && u.id != NOT_LOOKED_UP && (u.id < 0 || u.id >= A.a.n_blocks)) set_status(A.a.st, E0_ST_BAD_BLOCK);
            ks = vs = 0.f;
            u.at = NOWHERE;
            if (lane < KV / 16 && u.id >= 0 && u.id < A.a.n_blocks) {
                const size_t i = (size_t)u.id * A.a.Hkv + u.head;
                ks = A.a.ks[i], vs = A.a.vs[i];
                u.at = (uint32_t)(((i << A.a.shift) + ((u.at0 + 16 * lane) & (bs - 1))) >> 4);
            }
        };
        // load i: tokens 8 * group + lane % 8, 16 bytes of 64 of them
        const uint32_t in_group = (lane & 7) * D + 16 * (lane >> 3);
        const auto load = [&](const Unit& u, const uint8_t* from, uint4 (&to)[L]) {
            const int left = u.hi - u.at0 - (lane & 7);
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int n = 4 * i + cw, group = n / PER, part = n % PER;
                const uint32_t b = __shfl_sync(0xffffffffu, u.at, group >> 1);
                to[i] = make_uint4(0, 0, 0, 0);
                if (b != NOWHERE && 8 * group < left)
                    to[i] = __ldg(reinterpret_cast<const uint4*>(from + (size_t)b * (16 * D) + ((group & 1) * (8 * D) + part * 64 + in_group)));
            }
        };
        const auto store = [&](const uint4 (&from)[L], uint8_t* to, bool clean) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int n = 4 * i + cw, group = n / PER, part = n % PER;
                uint8_t* dst = to + group * (16 * D) + (8 * part + 2 * (lane >> 3)) * 128 + (lane & 7) * 16;
                uint4 c = from[i], a, b;
                if (clean) c.x = without_nan(c.x), c.y = without_nan(c.y), c.z = without_nan(c.z), c.w = without_nan(c.w);
                widen16(c, a, b);
                *reinterpret_cast<uint4*>(dst) = a;
                *reinterpret_cast<uint4*>(dst + 128) = b;
            }
        };
        Unit now, next, after;
        uint4 r[OPS][L];
        float ks, vs, ks1, vs1;
        bool have = look_up(now), have1 = look_up(next), ok = true;
        if (have) {
            look_in(now, ks, vs);
#pragma unroll
            for (int o = 0; o < OPS; ++o) load(now, op0 + o ? A.a.v : A.a.k, r[o]);
        }
        for (uint32_t g = 0; have; ++g) {
            const uint32_t st = g % STAGES, par = ((g / STAGES) + 1) & 1;
            const bool have2 = look_up(after);
            if (have1) look_in(next, ks1, vs1);
#pragma unroll
            for (int o = 0; o < OPS; ++o) {
                const bool values = op0 + o > 0;
                ok = __all_sync(0xffffffffu, arrived(values ? &S.v_empty[st] : &S.k_empty[st], par, abort));
                if (!ok) break;
                if (values && cw == 0 && lane < KV / 16) {
                    const float v = fmaxf(vs, LEAST_SCALE);
                    S.sc[st][lane] = now.at != NOWHERE ? make_float4(ks, log2f(v), SUM_UNIT / v, 1.f) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                store(r[o], values ? S.v[st] : S.k[st], values && now.edge);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(values ? &S.v_full[st] : &S.k_full[st]);
                if (have1) load(next, values ? A.a.v : A.a.k, r[o]);
            }
            if (!ok) break;
            now = next, next = after, ks = ks1, vs = vs1;
            have = have1, have1 = have2;
        }
        if (!ok && lane == 0) give_up();
    } else {
        // ---------------- products: the warp follows the schedule together, one lane issues
        if constexpr (G_::OTHER_REGS < 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G_::OTHER_REGS));
        if (warp == G_::SOFT + G_::TURN) {
            const uint32_t id_s = idesc_f16_f32(128, KV), id_o = idesc_f16_f32(128, D) | B_MN_MAJOR;
            // the operands' addresses, the low words of their descriptors: 16-byte units
            const uint32_t q_lo = desc_low(smem_u32(S.q), 128), k_lo = desc_low(smem_u32(S.k), 128), v_lo = desc_low(smem_u32(S.v), 16 * D);
            constexpr uint32_t QK_HI = desc_high(16 * D), V_HI = desc_high(128);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const bool leader = elect_one();
            uint32_t n_s0 = 0, n_s1 = 0, n_q = 0, gk = 0;
            bool ok = true, issued = false;
            Piece p;
            const auto q_there = [&](uint32_t n) {
                const bool there = __all_sync(0xffffffffu, arrived(&S.q_full[n % G_::Q_BUFS], (n / G_::Q_BUFS) & 1, abort));
                tc_fence_after();
                return there;
            };
            // S of half h, its n-th = Q K^T of the unit in stage st
            const auto first = [&](int h, uint32_t st, uint32_t n, uint32_t nq) {
                const uint32_t slot = HALVES == 2 ? h : n & 1, d = tm + slot * KV;
                const uint32_t a = q_lo + nq % G_::Q_BUFS * (uint32_t)(G_::Q_BYTES >> 4), b = k_lo + st * (uint32_t)(G_::OPERAND >> 4);
                if (leader) {
#pragma unroll
                    for (int s = 0; s < D / 16; ++s) umma_lo(d, a + 16 * s, QK_HI, b + 16 * s, QK_HI, id_s, s > 0);
                    umma_commit(&S.s_full[slot]);
                }
            };
            // O of half h += P V of the unit in stage st, the half's n-th; `more`: not the piece's first
            const auto second = [&](int h, uint32_t st, uint32_t n, uint32_t more) {
                const uint32_t slot = HALVES == 2 ? h : n & 1, use = HALVES == 2 ? n : n >> 1;
                const uint32_t p_at = tm + slot * KV, d = tm + G_::O_COL + h * D, b = v_lo + st * (uint32_t)(G_::OPERAND >> 4);
#pragma unroll
                for (int c = 0; c < CHUNKS; ++c) {  // the first positions' products run under the last ones' exponentials
                    if (!__all_sync(0xffffffffu, arrived(&S.p_full[slot][c], use & 1, abort))) return false;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int s = 4 * c; s < 4 * c + 4; ++s) {
                            const uint32_t a = p_at + 64 * c + 8 * (s % 4);
                            umma_ta_lo(d, a, b + s * 2 * D, V_HI, id_o, s > 0 ? 1 : more);
                            umma_ta_lo(d, a + 32, b + s * 2 * D, V_HI, id_o, 1);
                        }
                        umma_commit(c + 1 < CHUNKS ? &S.o_half[h] : &S.o_done[slot]);
                    }
                }
                return true;
            };
            while (ok && pieces.next(p)) {
                const int f0 = p.first(0), e0 = p.end(0), f1 = p.first(1), e1 = p.end(1), k0 = p.k0, k1 = p.k1;
                const uint32_t nq0 = n_q, nq1 = n_q + (f0 < e0);
                n_q = nq1 + (HALVES == 2 && f1 < e1);
                // one turn more than units: a unit's second products come with the next one's first
#pragma unroll 1
                for (int k = k0; ok && k <= k1; ++k) {
                    const uint32_t g = gk + (uint32_t)(k - k0), st = g % STAGES, last = (g - 1) % STAGES;
                    const bool now = k < k1, before = k > k0;
                    if (now) ok = arrived(&S.k_full[st], (g / STAGES) & 1, abort);
                    if (ok && before) ok = arrived(&S.v_full[last], ((g - 1) / STAGES) & 1, abort);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    issued = true;
                    const bool now0 = now && k >= f0 && k < e0, before0 = before && k - 1 >= f0 && k - 1 < e0;
                    if constexpr (HALVES == 2) {
                        const bool now1 = now && k >= f1 && k < e1, before1 = before && k - 1 >= f1 && k - 1 < e1;
                        if (before0) ok = second(0, last, n_s0 - 1, k - 1 > f0);
                        if (ok && now0 && k == f0) ok = q_there(nq0);  // a half's Q is waited for where it is wanted
                        if (ok && now0) first(0, st, n_s0++, nq0);
                        if (ok && before1) ok = second(1, last, n_s1 - 1, k - 1 > f1);
                        if (ok && now1 && k == f1) ok = q_there(nq1);
                        if (ok && now1) first(1, st, n_s1++, nq1);
                    } else {
                        const uint32_t n = n_s0;
                        if (now0 && k == f0) ok = q_there(nq0);
                        if (ok && now0) first(0, st, n_s0++, nq0);
                        if (ok && before0) ok = second(0, last, n - 1, k - 1 > f0);
                    }
                    if (!ok) break;
                    if (leader) {
                        if (now) umma_commit(&S.k_empty[st]);
                        if (before) umma_commit(&S.v_empty[last]);
                    }
                }
                gk += (uint32_t)(k1 - k0);
            }
            if (!ok && leader) give_up();
            if (issued) {  // the products have ended before tensor memory is freed
                if (leader) umma_commit(&S.drained);
                arrived(&S.drained, 0, &never);
            }
            __syncwarp();
        } else {
            // ---------------- Q: a warp eight rows at a time, a lane 16 bytes of every 64 of row lane % 8.
            // All of a warp's rows are copied to their places first, so that one latency is waited for, then
            // looked at and, bf16, turned into fp16 there.
            const int g0 = warp - G_::SOFT - G_::TURN - 1;
            constexpr int C = D / 32;
            uint32_t nq = 0;
            bool ok = true;
            Piece p;
            while (ok && pieces.next(p)) {
                const TileJob& J = p.J;
#pragma unroll 1
                for (int h = 0; h < HALVES; ++h) {
                    if (p.first(h) >= p.end(h)) continue;
                    const uint32_t qb = nq % G_::Q_BUFS;
                    ok = __all_sync(0xffffffffu, arrived(&S.q_empty[qb], ((nq / G_::Q_BUFS) + 1) & 1, abort));
                    if (!ok) break;
                    uint8_t* mine = S.q[qb] + (lane & 7) * 16 + (lane >> 3) * 128;
#pragma unroll 1
                    for (int g8 = g0; g8 < 16; g8 += G_::Q_WARPS) {
                        const int row = 128 * h + 8 * g8 + (lane & 7), rr = J.mtile * G_::ROWS + row, ii = div_group(A, rr);
                        const bool have = row < J.rows;
                        const T* src = reinterpret_cast<const T*>(A.a.q) + 8 * (lane >> 3) +
                                       (have ? ((size_t)J.row0 + ii) * A.a.q_ld + (size_t)(p.head * G + rr - ii * G) * D : 0);
#pragma unroll
                        for (int c = 0; c < C; ++c) copy16_or_zero(mine + g8 * (16 * D) + c * 512, src + 32 * c, have);
                    }
                    copy_commit();
                    copy_wait<0>();
#pragma unroll 1
                    for (int g8 = g0; g8 < 16; g8 += G_::Q_WARPS) {
                        uint4 u[C];
                        uint32_t m = 0;
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            u[c] = *reinterpret_cast<const uint4*>(mine + g8 * (16 * D) + c * 512);
                            m = __vmaxu2(__vmaxu2(__vmaxu2(m, u[c].x & 0x7FFF7FFFu), u[c].y & 0x7FFF7FFFu),
                                         __vmaxu2(u[c].z & 0x7FFF7FFFu, u[c].w & 0x7FFF7FFFu));
                        }
                        m = max(m & 0xFFFFu, m >> 16);
                        m = max(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        float fr;
                        if constexpr (TY == E0_F16) {
                            fr = m >= 0x7C00u ? __uint_as_float(0x7FC00000u) : A.a.scale * LOG2E;
                        } else {  // times a power of two that brings the largest near 1
                            const uint32_t b = m << 16;
                            int e = (int)(b >> 23);
                            e = e < 27 ? 27 : e > 253 ? 253 : e;
                            const float down = b == 0 ? 0.f : __uint_as_float((uint32_t)(254 - e) << 23);
                            fr = b >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                                  : __uint_as_float((uint32_t)e << 23) * A.a.scale * LOG2E;
#pragma unroll
                            for (int c = 0; c < C; ++c) {
                                const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
                                uint32_t x[4];
#pragma unroll
                                for (int z = 0; z < 4; ++z) {
                                    const float2 v = unpack16<E0_BF16>(w[z]);
                                    x[z] = half2_of(v.x * down, v.y * down);
                                }
                                *reinterpret_cast<uint4*>(mine + g8 * (16 * D) + c * 512) = make_uint4(x[0], x[1], x[2], x[3]);
                            }
                        }
                        if (lane < 8) S.qf[qb][8 * g8 + lane] = fr;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.q_full[qb]);
                    ++nq;
                }
            }
            if (!ok && lane == 0) give_up();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == G_::SOFT + G_::TURN) {
        tc_fence_after();
        tmem_dealloc(tmem, TILE_TMEM);
    }
}

// ---------------------------------------------------------------- jobs that several blocks have

constexpr int TILE_JOIN_THREADS = 256;
template <int D>
constexpr int TILE_JOIN_ROWS = TILE_JOIN_THREADS / (D / 4);  // of a block, as many as four columns a thread make

template <int D, int TY>
__global__ void __launch_bounds__(TILE_JOIN_THREADS) k_tile_join(TileArgs A) {
    typedef Geo<D> G_;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
    const TileCut cut = A.cuts[blockIdx.x];
    if (cut.parts == 0) return;
    const int4* from = reinterpret_cast<const int4*>(A.jobs + cut.job);
    const int mtile = from[0].y, row0 = from[3].y, rows = from[3].z;
    // a warp: eight rows, 16 columns; a thread: four
    constexpr int WIDE = D / 16;  // warps of eight rows
    const int lane = threadIdx.x & 31, warp = (blockIdx.y * TILE_JOIN_THREADS + threadIdx.x) >> 5;
    const int G = A.a.Hq / A.a.Hkv, d4 = 16 * (warp % WIDE) + 4 * (lane >> 3), r = 8 * (warp / WIDE) + (lane & 7);
    if (r >= rows) return;
    const int row = mtile * G_::ROWS + r, i_tok = div_group(A, row), head = cut.head * G + row - i_tok * G;
    const size_t tok = (size_t)row0 + i_tok, at = tok * A.a.Hq + head;
    if (A.merge && A.own_at[tok] == NO_ROW) return;  // no sequence's row
    const auto slot_of = [&](int i) { return 2 * (cut.block + i) + (i == 0); };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int BATCH = 8;
    for (int i0 = 0; i0 < cut.parts; i0 += BATCH) {
        float2 ml[BATCH];
        float4 x[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            ml[i] = make_float2(-INFINITY, 0.f);
            x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + i < cut.parts) {
                ml[i] = A.part_ml[(size_t)slot_of(i0 + i) * G_::ROWS + r];
                x[i] = *reinterpret_cast<const float4*>(A.part_o + part_at<D>(slot_of(i0 + i), r, d4));
            }
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) top = fmaxf(top, ml[i].x);
        const float base = top == -INFINITY ? 0.f : top, keep = exp2_of(m - base);
        m = top;
        l *= keep;
        o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const float w = exp2_of(ml[i].x - base);
            l += w * ml[i].y;
            o.x += w * x[i].x, o.y += w * x[i].y, o.z += w * x[i].z, o.w += w * x[i].w;
        }
    }
    const float inv = l > 0.f || l != l ? SUM_UNIT / l : 0.f;
    float lse = lse_of(m, l, TILE_LIFT);
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    if (A.merge) {
        const float4 x = *reinterpret_cast<const float4*>(A.own_o + at * D + d4);
        const Two two = two_of(lse, A.own_lse[at]);
        o.x = fmaf(two.f1, o.x, two.f2 * x.x), o.y = fmaf(two.f1, o.y, two.f2 * x.y);
        o.z = fmaf(two.f1, o.z, two.f2 * x.z), o.w = fmaf(two.f1, o.w, two.f2 * x.w);
        lse = two.lse;
    }
    put_row4<TY>(A.a, A.vec_out, tok, head * D + d4, o.x, o.y, o.z, o.w);
    if (A.a.lse && d4 == 0) A.a.lse[at] = lse;
}

// ---------------------------------------------------------------- host

inline int tile_blocks() { return num_sms(); }
inline long long tile_jobs(int B, int max_q, int G, int D) {
    const int rows = D == 256 ? 128 : 256;
    return (long long)B * (((long long)max_q * G + rows - 1) / rows);
}
inline size_t tile_ws_bytes(int B, int max_q, int G, int D) {
    const size_t rows = D == 256 ? 128 : 256, slots = 2 * (size_t)tile_blocks();
    return up256(slots * rows * D * sizeof(float)) + up256(slots * rows * sizeof(float2)) + up256(tile_blocks() * sizeof(TileCut)) +
           up256((size_t)tile_jobs(B, max_q, G, D) * sizeof(TileJob)) + up256(tile_blocks() * sizeof(int4)) + 256;
}

template <int D, int TY, bool RULES>
int tile_launch(const TileArgs& t, cudaStream_t s) {
    static std::atomic<uint64_t> asked{0};
    if (!allow_smem((const void*)k_attn_tile<D, TY, RULES>, sizeof(TileSmem<D>), asked)) return E0_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    // The schedule beside the kernel before it where that one is this library's own results, which
    // nothing here writes over; otherwise after all that went before.
    cfg.numAttrs = t.merge ? 1 : 0;
    cfg.stream = s;
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(PLAN_THREADS);
    const int kept = t.most_jobs < PLAN_SHARED ? t.most_jobs : PLAN_SHARED;
    cfg.dynamicSmemBytes = (size_t)(t.a.B + 1 + 2 * kept) * sizeof(uint32_t);
    static std::atomic<uint64_t> asked_plan{0};
    if (!allow_smem((const void*)k_tile_plan<D>, (size_t)(E0_MAX_SEQS + 1 + 2 * PLAN_SHARED) * sizeof(uint32_t), asked_plan))
        return E0_ERR_CUDA;
    if (cudaLaunchKernelEx(&cfg, k_tile_plan<D>, t) != cudaSuccess) return E0_ERR_CUDA;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(t.blocks);
    cfg.blockDim = dim3(Geo<D>::THREADS);
    cfg.dynamicSmemBytes = sizeof(TileSmem<D>);
    if (cudaLaunchKernelEx(&cfg, k_attn_tile<D, TY, RULES>, t) != cudaSuccess) return E0_ERR_CUDA;
    cfg.gridDim = dim3(t.blocks, Geo<D>::ROWS / TILE_JOIN_ROWS<D>);
    cfg.blockDim = dim3(TILE_JOIN_THREADS);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, k_tile_join<D, TY>, t) == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

template <int D>
int tile_launch_d(const TileArgs& t, int dtype, cudaStream_t s) {
    const bool rules = t.a.cap > 0.f || t.a.slopes;
    if (dtype == E0_F16) return rules ? tile_launch<D, E0_F16, true>(t, s) : tile_launch<D, E0_F16, false>(t, s);
    return rules ? tile_launch<D, E0_BF16, true>(t, s) : tile_launch<D, E0_BF16, false>(t, s);
}

// The arguments of the kernels above; `ws` of tile_ws_bytes.
inline TileArgs tile_args(const AttnArgs& a, const TilePrefix* prefix, int dtype, void* ws) {
    TileArgs t = {};
    t.a = a;
    if (prefix) {
        t.own = prefix->own, t.own_at = prefix->at, t.own_o = prefix->o, t.own_lse = prefix->lse, t.merge = prefix->merge;
        t.own.unit = 64;  // any
    }
    t.a.unit = a.D == 256 ? 64 : 128;
    const int G = a.Hq / a.Hkv;
    while ((1 << t.by_shift) < G) ++t.by_shift;
    t.by_group = (uint32_t)(((1ull << (31 + t.by_shift)) + G - 1) / G);
    t.blocks = tile_blocks();
    t.most_jobs = (int)tile_jobs(a.B, a.max_q, a.Hq / a.Hkv, a.D);
    const size_t rows = a.D == 256 ? 128 : 256, slots = 2 * (size_t)t.blocks;
    char* p = reinterpret_cast<char*>(ws);
    const auto take = [&](size_t n) {
        char* at = p;
        p += up256(n);
        return at;
    };
    t.part_o = reinterpret_cast<float*>(take(slots * rows * a.D * sizeof(float)));
    t.part_ml = reinterpret_cast<float2*>(take(slots * rows * sizeof(float2)));
    t.cuts = reinterpret_cast<TileCut*>(take(t.blocks * sizeof(TileCut)));
    t.jobs = reinterpret_cast<TileJob*>(take((size_t)t.most_jobs * sizeof(TileJob)));
    t.begin = reinterpret_cast<int4*>(take(t.blocks * sizeof(int4)));
    t.head = reinterpret_cast<TileHead*>(take(sizeof(TileHead)));
    t.out_16 = !((uintptr_t)a.out & 15) && (a.out_ld * type_size(dtype)) % 16 == 0;
    t.vec_out = a.raw || (!((uintptr_t)a.out & 7) && (a.out_ld * type_size(dtype)) % 8 == 0);
    return t;
}

}  // namespace
}  // namespace e0
