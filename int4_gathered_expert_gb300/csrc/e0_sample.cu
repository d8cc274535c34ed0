// The next tokens from the logits: temperature, top-k, top-p, min-p, one draw a row
// (e0_sample).
#include <cfloat>
#include <cuda_runtime.h>

#include "e0_internal.h"
#include "e0_types.cuh"

namespace e0 {
namespace {

// A row belongs to a cluster of up to eight thread blocks, which hold it in shared memory
// as fp32: it is read from memory once, and what bounds the kernel beyond that is instructions
// (a weight is thirty) and the cluster's meetings (a microsecond each; a block by itself has
// none).  Nothing is sorted.  The kept tokens are a beginning of the row in the order "larger
// logit, then lower token", so all there is to find is its last member:
//   - a histogram over bins of equal width in log2 of the weight (counts and weights' sums),
//     of the weights above 2^-16 first, says in which bin it is;
//   - where few tokens come up to that bin's end, one block takes them all and ends the row;
//   - otherwise the bin's members go to one block, which divides them again by the bits of
//     their logits; a bin of very many members is divided by all blocks.  What is left are
//     some tokens, or equal ones, whose order is that of the tokens.
// The draw then needs no order: the first token, by number, whose running sum of kept
// weights exceeds u times their total.  Each block's sum is in its histogram already unless
// min-p takes from it, and only the block of the draw looks for its place (all blocks adding up
// once more: 92 us for 85 below).
// 64 rows of 131071 fp32 logits, top-p 0.9: 85 us, two turns of 38 clusters of 13 us for the
// histogram (three additions in shared memory a token), 5 for the reading (of the 5 us in which
// memory alone could be read), 12 for meetings and searches, 8 for the draw.  Read from the L2
// cache in each pass instead of held, all rows would run at once, and take 98 us.  (Up to 149888
// tokens an SM has room for two blocks, beyond for one: 24 rows of 151936, not truncated, 23 us in two turns.)
//
// A draw over V tokens has V borders, and an error in the sums moves all of them: with fp32
// exponentials one row in a hundred would get another token than the definition gives.
// So a weight 2^-y, y = (largest - logit) log2 e / temperature, is a 64-bit integer, 2^44
// times its value, good to 2^-28 of itself or to one, whichever is more: y comes from a difference and
// a product that carry their rounding errors along (Dekker, Numer. Math. 18, 1971), its power of two from a
// table of 128 and the series of what is left.  Sums of integers are exact in any order, so
// equal calls give equal tokens.  Weights below 2^-44 of the largest count as nothing.
constexpr int SM_THREADS = 512, SM_WARPS = SM_THREADS / 32;
constexpr int MOST_BLOCKS = 8;
constexpr int BINS = 2048;
constexpr int FEW = 512;  // members of a bin that one block takes
constexpr int ALL = 256;  // tokens up to a bin's end that one block ends the row with
constexpr int WEIGHT_BITS = 44;
constexpr int BATCH = 4;
constexpr int STEPS_OF_ONE = 128;

typedef unsigned long long u64;

struct SampleArgs {
    const void* x;
    const float* u;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* token;
    float* logp;
    int32_t* kept;
    uint32_t* st;
    int64_t ld;
    int V, slice;
};

// What the blocks of a cluster tell one another; every block has a copy.
struct Told {
    u64 best[MOST_BLOCKS];            // the block's largest logit's order and token
    uint32_t odd[MOST_BLOCKS];        // whether it saw NaN or +infinity
    u64 mass[2][MOST_BLOCKS];         // of the block's bins, members or kept tokens
    uint32_t count[2][MOST_BLOCKS];
    uint32_t lo[2][MOST_BLOCKS], hi[2][MOST_BLOCKS];  // the least and the greatest order of a bin's members
    // from the block that found it
    uint32_t bin, key, index, members;
    u64 mass_before, mass_through;
    uint32_t count_before, count_through;
};

struct SampleSmem {
    uint32_t count[BINS], low[BINS], high[BINS];  // of this block's share of the row; a sum of weights is high : low
    u64 few[FEW];                                 // order : token of the last bin's members (the first block's)
    u64 few_w[FEW];
    u64 mine[FEW];                                // this block's own of them
    int2 steps[STEPS_OF_ONE];
    uint32_t n_few, n_mine, mine_at;
    uint32_t sub, sub_count;
    u64 sub_mass;
    uint32_t n_sub;
    uint16_t sub_list[FEW];
    Told told;
    u64 wsum[SM_WARPS];
    uint32_t wcount[SM_WARPS], wa[SM_WARPS], wb[SM_WARPS];
    // the row's rules
    float ch, cl;  // log2 e / temperature
    u64 least;     // weight of min_p
};

// ---------------------------------------------------------------- cluster

E0_DEV uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
E0_DEV uint32_t cluster_blocks() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// All threads of all the row's blocks; what they wrote to one another's memory is seen.
E0_DEV void meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Only once all the row's blocks have begun may one write to another's memory: each says so as its first
// act and waits for the others before its first such write, the reading of the row between the two.
E0_DEV void say_begun() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
E0_DEV void all_begun() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// A variable of block r's shared memory.
template <typename P>
E0_DEV uint32_t of_block(P* p, uint32_t r) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(r));
    return a;
}
E0_DEV void put(uint32_t a, uint32_t v) { asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
E0_DEV void put(uint32_t a, u64 v) { asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory"); }
E0_DEV uint32_t get32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
E0_DEV uint32_t add_to(uint32_t a, uint32_t v) {
    uint32_t was;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(was) : "r"(a), "r"(v) : "memory");
    return was;
}

// ---------------------------------------------------------------- order and weights

// Larger logits have larger orders (-0 and +0 the same one).
E0_DEV uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
E0_DEV float logit_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o); }

struct Scale {
    float most, ch, cl;
    const int2* steps;  // STEPS in shared memory
};

// y of a logit (>= 0) as fp32, monotone in the logit; and the exact one's rest.
E0_DEV float y_of(const Scale& s, float x) { return (s.most - x) * s.ch; }

// 2^(-i / STEPS_OF_ONE), times 2^30, from the power series at compile time.
struct Steps {
    int at[STEPS_OF_ONE];
};
constexpr double power_of_half(double y) {  // 2^-y, y in [0, 1)
    double term = 1, sum = 1;
    for (int k = 1; k < 30; ++k) term *= -0.69314718055994530942 * y / k, sum += term;
    return sum;
}
constexpr Steps steps_of() {
    Steps t = {};
    for (int i = 0; i < STEPS_OF_ONE; ++i) t.at[i] = (int)(power_of_half((double)i / STEPS_OF_ONE) * 1073741824.0 + 0.5);
    return t;
}
__constant__ const Steps STEPS = steps_of();

// 2^44 * 2^-y.  y = k / 128 + f with k a whole number and f at most 1/256 in size: T = 2^-(k % 128) / 128
// comes from a table, 2^-f = 1 + t from three terms of its series, and T + T t is summed as
// an integer: t's part of it is below 2^22, which fp32 holds to half a unit.  Adding 1.5 * 2^23 leaves a
// number's whole part in the low bits (1.5 * 2^16: its whole 128ths).  Nothing here is slower than
// an addition but the table's read (products of whole numbers would be eight times).
E0_DEV u64 weight_of(const Scale& s, float x) {
    const float d = s.most - x;
    const float back = d - s.most;
    const float dl = (s.most - (d - back)) - (x + back);  // d + dl is the difference
    const float p = __fmul_rn(d, s.ch);  // not to be joined with the subtraction below
    if (!(p < (float)(WEIGHT_BITS + 1))) return 0;
    const float e = fmaf(d, s.ch, -p) + fmaf(d, s.cl, dl * s.ch);
    constexpr float WHOLE = 12582912.f, WHOLE_STEPS = 12582912.f / STEPS_OF_ONE;
    const float near = __fadd_rn(p, WHOLE_STEPS);
    const int k = __float_as_int(near) - __float_as_int(WHOLE_STEPS);
    const float f = (p - __fadd_rn(near, -WHOLE_STEPS)) + e;  // the difference is exact
    const int2 step = s.steps[k & (STEPS_OF_ONE - 1)];
    constexpr float L1 = -0.69314718f, L2 = 0.24022651f, L3 = -0.055504109f;
    const float t = f * fmaf(f, fmaf(f, L3, L2), L1);
    const int g = step.x + (__float_as_int(fmaf(__int_as_float(step.y), t, WHOLE)) - __float_as_int(WHOLE));
    return ((u64)(uint32_t)g << (WEIGHT_BITS - 30)) >> (k / STEPS_OF_ONE);
}

// ln of a token's weight, from its logit: the whole number of a rare token has few bits.  Three steps of
// fp32 (the constant's, the product's, the sum's).
E0_DEV float ln_weight_of(const Scale& s, float x) {
    const float d = s.most - x, p = __fmul_rn(d, s.ch);
    return -0.6931471805599453f * (p + (fmaf(d, s.ch, -p) + d * s.cl));
}

// v of [0, 1) times 2^64, rounded down.
E0_DEV u64 fraction_of(float v) {
    const float up = v * 4294967296.f, whole = truncf(up);
    return (u64)__float2uint_rz(whole) << 32 | __float2uint_rz((up - whole) * 4294967296.f);
}

// ---------------------------------------------------------------- sums of a block

template <typename V>
E0_DEV V warp_total(V v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <typename V>
E0_DEV V warp_scan(V v) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V t = __shfl_up_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31) >= o) v += t;
    }
    return v;
}

// What the warps before this one have of a count and a sum, and what all have; every thread
// gives its own.
struct Before {
    uint32_t count, all_count;
    u64 sum, all_sum;
};
E0_DEV Before block_before(SampleSmem& S, uint32_t c, u64 m) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t ci = warp_scan(c);
    const u64 mi = warp_scan(m);
    __syncthreads();  // the former use is over
    if (lane == 31) S.wcount[warp] = ci, S.wsum[warp] = mi;
    __syncthreads();
    uint32_t wc = lane < SM_WARPS ? S.wcount[lane] : 0;
    u64 wm = lane < SM_WARPS ? S.wsum[lane] : 0;
    wc = warp_scan(wc), wm = warp_scan(wm);
    Before b;
    b.all_count = __shfl_sync(0xffffffffu, wc, 31), b.all_sum = __shfl_sync(0xffffffffu, wm, 31);
    const uint32_t bc = __shfl_sync(0xffffffffu, wc, warp - 1);
    const u64 bm = __shfl_sync(0xffffffffu, wm, warp - 1);
    b.count = ci - c + (warp ? bc : 0), b.sum = mi - m + (warp ? bm : 0);
    return b;
}

// ---------------------------------------------------------------- the last of the kept tokens

// A beginning of the row's order: the tokens of larger order than key, and those of that
// order up to index.
struct End {
    uint32_t key, index;
    uint32_t count;
    u64 mass;
    E0_DEV bool holds(uint32_t o, uint32_t i) const { return o > key || (o == key && i <= index); }
};

struct Row {
    SampleSmem& S;
    float* x;       // this block's share
    int n, from;    // its length, its first token
    uint32_t rank, blocks;
    Scale sc;
    float per_unit;  // bins of a unit of y: the first 16 units of y are looked at alone, or all of them
    // this block's share of what `find` found, where its histogram of weights says it
    bool known;
    uint32_t own_count, own_members;
    u64 own_mass;

    // Counts, and sums where they are wanted, of this block's tokens by bin (`bin_of` gives
    // BINS for none).  told[1]: every block's tokens in bins, and the sum of their weights, or of
    // all weights where `every` is set.
    template <typename F>
    E0_DEV void histogram(F bin_of, bool sums, bool every, bool clear = true) {
        if (clear) {
            for (int i = threadIdx.x; i < BINS; i += SM_THREADS) S.count[i] = S.low[i] = S.high[i] = 0;
            __syncthreads();
        }
        u64 m = 0;
        uint32_t c = 0;
        // BATCH tokens a thread at a time: their weights and the answers of the additions are
        // chains that run beside one another
        for (int i0 = 0; i0 < n; i0 += BATCH * SM_THREADS) {
            float v[BATCH];
            uint32_t b[BATCH];
            bool any = false;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int i = i0 + k * SM_THREADS + threadIdx.x;
                v[k] = i < n ? x[i] : -INFINITY;
                b[k] = bin_of(v[k]);
                any |= b[k] < BINS;
            }
            if (!every && !__any_sync(0xffffffffu, any)) continue;
            u64 w[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                w[k] = sums ? weight_of(sc, v[k]) : 0;
                m += every || b[k] < BINS ? w[k] : 0;
            }
            uint32_t was[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                was[k] = 0;
                if (b[k] < BINS) {
                    ++c;
                    atomicAdd(&S.count[b[k]], 1u);
                    if (sums) was[k] = atomicAdd(&S.low[b[k]], (uint32_t)w[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const uint32_t lo = (uint32_t)w[k], hi = (uint32_t)(w[k] >> 32) + (was[k] + lo < lo);
                if (b[k] < BINS && hi) atomicAdd(&S.high[b[k]], hi);
            }
        }
        const Before all = block_before(S, c, m);
        if (threadIdx.x < blocks) {
            put(of_block(&S.told.count[1][rank], threadIdx.x), all.all_count);
            put(of_block(&S.told.mass[1][rank], threadIdx.x), all.all_sum);
        }
        meet();
    }
    E0_DEV void totals(uint32_t& c, u64& m) const {
        c = 0, m = 0;
        for (uint32_t r = 0; r < blocks; ++r) c += S.told.count[1][r], m += S.told.mass[1][r];
    }

    // The bin in which the running count (of what stands before it and `count` before the
    // first bin) first reaches want_n, or the running sum want_w.  The blocks share the bins.
    // told.members is 0 where none does.
    E0_DEV void find_bin(bool by_count, uint32_t want_n, u64 want_w, uint32_t count0, u64 mass0) {
        if (threadIdx.x == 0) S.told.members = 0;
        const int per = BINS / blocks, mine = rank * per;
        const int each = (per + SM_THREADS - 1) / SM_THREADS;  // 4 where the block is alone
        uint32_t c[4];
        u64 m[4], mt = 0;
        uint32_t ct = 0;
        const int b0 = threadIdx.x * each;
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = 0, m[k] = 0;
        if (b0 < per) {
#pragma unroll 1
            for (uint32_t r0 = 0; r0 < blocks; r0 += 4) {
                uint32_t v[4][3];
                if (blocks >= 4) {  // a bin a thread: of four blocks at once
#pragma unroll
                    for (uint32_t r = 0; r < 4; ++r) {
                        v[r][0] = get32(of_block(&S.count[mine + b0], r0 + r));
                        v[r][1] = get32(of_block(&S.low[mine + b0], r0 + r));
                        v[r][2] = get32(of_block(&S.high[mine + b0], r0 + r));
                    }
#pragma unroll
                    for (uint32_t r = 0; r < 4; ++r) c[0] += v[r][0], m[0] += ((u64)v[r][2] << 32) + v[r][1];
                } else {  // two or four bins a thread: of a block at once
#pragma unroll 1
                    for (uint32_t r = 0; r < blocks; ++r) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int b = mine + min(b0 + k, per - 1);
                            v[k][0] = get32(of_block(&S.count[b], r));
                            v[k][1] = get32(of_block(&S.low[b], r));
                            v[k][2] = get32(of_block(&S.high[b], r));
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < each && b0 + k < per) c[k] += v[k][0], m[k] += ((u64)v[k][2] << 32) + v[k][1];
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) ct += c[k], mt += m[k];
        const Before mine_before = block_before(S, ct, mt);
        uint32_t cb = mine_before.count;
        u64 mb = mine_before.sum;
        if (threadIdx.x < blocks) {
            put(of_block(&S.told.count[0][rank], threadIdx.x), mine_before.all_count);
            put(of_block(&S.told.mass[0][rank], threadIdx.x), mine_before.all_sum);
        }
        meet();
        cb += count0, mb += mass0;
        for (uint32_t r = 0; r < rank; ++r) cb += S.told.count[0][r], mb += S.told.mass[0][r];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool here = by_count ? cb < want_n && want_n <= cb + c[k] : mb < want_w && want_w <= mb + m[k];
            if (here && k < each && b0 + k < per) {
                for (uint32_t r = 0; r < blocks; ++r) {
                    put(of_block(&S.told.bin, r), (uint32_t)(mine + b0 + k));
                    put(of_block(&S.told.members, r), c[k]);
                    put(of_block(&S.told.count_before, r), cb);
                    put(of_block(&S.told.mass_before, r), mb);
                }
            }
            cb += c[k], mb += m[k];
        }
        meet();
    }

    // The tokens with `in(logit)`, FEW in all at most, go to the first block, in any order: each block's
    // together, for an addition in another block's memory takes a microsecond to answer.  n_few and
    // n_mine are 0.  Returns how many are this block's, in S.mine.
    template <typename F>
    E0_DEV uint32_t gather(F in) {
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += SM_THREADS)
            if (in(x[i])) {
                const uint32_t at = atomicAdd(&S.n_mine, 1u);
                if (at < FEW) S.mine[at] = ((u64)order_of(x[i]) << 32) | (uint32_t)~(from + i);  // larger is earlier
            }
        __syncthreads();
        const uint32_t m = min(S.n_mine, (uint32_t)FEW);
        if (threadIdx.x == 0) S.mine_at = m ? add_to(of_block(&S.n_few, 0), m) : 0;
        __syncthreads();
        if (threadIdx.x == 0) S.n_mine = 0;
        const uint32_t at = S.mine_at + threadIdx.x;
        if (threadIdx.x < m && at < FEW) {
            const u64 me = S.mine[threadIdx.x];
            put(of_block(&S.few[at], 0), me);
            put(of_block(&S.few_w[at], 0), weight_of(sc, logit_of((uint32_t)(me >> 32))));
        }
        meet();
        return m;
    }

    // The first block: of the m tokens in S.few, after count0 others of sum mass0, the one with
    // which the count reaches want_n or the sum want_w.  They are divided by their orders' bits
    // (the histogram's place is free), so that each is compared with few others.
    E0_DEV void pick(int m, bool by_count, uint32_t want_n, u64 want_w, uint32_t count0, u64 mass0) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        const u64 me = tid < m ? S.few[tid] : 0, w = tid < m ? S.few_w[tid] : 0;
        static_assert(FEW <= SM_THREADS && BINS % SM_THREADS == 0, "a thread a token");
        const uint32_t o = (uint32_t)(me >> 32);
        uint32_t lo = __reduce_min_sync(0xffffffffu, tid < m ? o : 0xFFFFFFFFu), hi = __reduce_max_sync(0xffffffffu, o);
        if (lane == 0) S.wa[warp] = lo, S.wb[warp] = hi;
        if (tid == 0) S.n_sub = 0;
        for (int i = tid; i < BINS; i += SM_THREADS) S.count[i] = S.low[i] = S.high[i] = 0;
        __syncthreads();
        for (int i = 0; i < SM_WARPS; ++i) lo = min(lo, S.wa[i]), hi = max(hi, S.wb[i]);
        int shift = 0;
        while (((hi - lo) >> shift) >= BINS) ++shift;
        const uint32_t bin = (hi - o) >> shift;
        if (tid < m) {
            atomicAdd(&S.count[bin], 1u);
            const uint32_t l = (uint32_t)w, was = atomicAdd(&S.low[bin], l);
            const uint32_t h = (uint32_t)(w >> 32) + (was + l < l);
            if (h) atomicAdd(&S.high[bin], h);
        }
        __syncthreads();
        // sums of the bins before each thread's four
        constexpr int PER = BINS / SM_THREADS;
        uint32_t c[PER], ct = 0;
        u64 s[PER], st = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int b = tid * PER + k;
            c[k] = S.count[b], s[k] = ((u64)S.high[b] << 32) + S.low[b];
            ct += c[k], st += s[k];
        }
        const Before b4 = block_before(S, ct, st);
        uint32_t cb = count0 + b4.count;
        u64 sb = mass0 + b4.sum;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const bool here = by_count ? cb < want_n && want_n <= cb + c[k] : sb < want_w && want_w <= sb + s[k];
            if (here) S.sub = tid * PER + k, S.sub_count = cb, S.sub_mass = sb;
            cb += c[k], sb += s[k];
        }
        __syncthreads();
        const bool in_sub = tid < m && bin == S.sub;
        if (in_sub) S.sub_list[atomicAdd(&S.n_sub, 1u)] = (uint16_t)tid;
        __syncthreads();
        if (in_sub) {
            cb = S.sub_count, sb = S.sub_mass;
            const int n_sub = S.n_sub;
#pragma unroll 4
            for (int j = 0; j < n_sub; ++j) {
                const int at = S.sub_list[j];
                const bool before = S.few[at] > me;
                cb += before;
                sb += before ? S.few_w[at] : 0;
            }
            // by weight: members without weight pass nothing, so this is one member too
            if (by_count ? cb + 1 == want_n : sb < want_w && want_w <= sb + w)
                for (uint32_t r = 0; r < blocks; ++r) {
                    put(of_block(&S.told.key, r), o);
                    put(of_block(&S.told.index, r), ~(uint32_t)me);
                    put(of_block(&S.told.count_through, r), cb + 1);
                    put(of_block(&S.told.mass_through, r), sb + w);
                }
        }
    }

    // Of the tokens with `in(logit)`, `members` in all, after count0 tokens of sum mass0:
    // the one with which the count reaches want_n or the sum want_w.  One block takes them.
    template <typename F>
    E0_DEV End among_few(F in, bool by_count, uint32_t want_n, u64 want_w, uint32_t count0, u64 mass0) {
        own_members = gather(in);
        if (rank == 0) {
            pick(min((int)S.n_few, FEW), by_count, want_n, want_w, count0, mass0);
            if (threadIdx.x == 0) S.n_few = 0;
        }
        meet();
        return {S.told.key, S.told.index, S.told.count_through, S.told.mass_through};
    }

    // Of the tokens of one order: the nth (from 1) by number.
    E0_DEV uint32_t nth_of(uint32_t key, uint32_t nth) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int per = (n + SM_THREADS - 1) / SM_THREADS * 32, i0 = warp * per, i1 = min(n, i0 + per);
        uint32_t c = 0;
        for (int i = i0; i < i1; i += 32) c += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && order_of(x[i + lane]) == key));
        __syncthreads();
        if (lane == 0) S.wcount[warp] = c;
        __syncthreads();
        uint32_t all = 0, before = 0;
        for (int w = 0; w < SM_WARPS; ++w) all += S.wcount[w], before += w < warp ? S.wcount[w] : 0;
        if (threadIdx.x < blocks) put(of_block(&S.told.count[1][rank], threadIdx.x), all);
        meet();
        for (uint32_t r = 0; r < rank; ++r) before += S.told.count[1][r];
        if (before < nth && nth <= before + c)
            for (int i = i0; i < i1; i += 32) {
                const bool is = i + lane < i1 && order_of(x[i + lane]) == key;
                const uint32_t b = __ballot_sync(0xffffffffu, is);
                if (is && before + __popc(b & ((2u << lane) - 1)) == nth)
                    for (uint32_t r = 0; r < blocks; ++r) put(of_block(&S.told.index, r), (uint32_t)(from + i + lane));
                before += __popc(b);
            }
        meet();
        return S.told.index;
    }

    // The end of the kept tokens: the token with which their count reaches want_n, or
    // their sum want_w (> 0, at most the row's).  find_bin has found its bin by weight.
    E0_DEV End find(bool by_count, uint32_t want_n, u64 want_w, bool sums) {
        uint32_t bin = S.told.bin, members = S.told.members, count0 = S.told.count_before;
        u64 mass0 = S.told.mass_before;
        const Scale s = sc;
        const float per = per_unit;
        const auto in_first = [s, per, bin](float v) { return weight_bin(s, per, v) == bin; };
        known = sums && members <= FEW;
        if (members <= FEW) {
            // the bins before, and the bin's own members up to the end
            uint32_t c = 0;
            u64 m = 0;
            for (int b = threadIdx.x; known && b < (int)bin; b += SM_THREADS) c += S.count[b], m += ((u64)S.high[b] << 32) + S.low[b];
            const End end = among_few(in_first, by_count, want_n, want_w, count0, mass0);
            if (!known) return end;
            if (threadIdx.x < own_members) {
                const u64 me = S.mine[threadIdx.x];
                if (end.holds((uint32_t)(me >> 32), ~(uint32_t)me)) ++c, m += weight_of(sc, logit_of((uint32_t)(me >> 32)));
            }
            const Before own = block_before(S, c, m);
            own_count = own.all_count, own_mass = own.all_sum;
            return end;
        }
        // many: by the bits of their orders
        uint32_t lo = 0xFFFFFFFFu, hi = 0;
        for (int i = threadIdx.x; i < n; i += SM_THREADS)
            if (in_first(x[i])) lo = min(lo, order_of(x[i])), hi = max(hi, order_of(x[i]));
        lo = __reduce_min_sync(0xffffffffu, lo), hi = __reduce_max_sync(0xffffffffu, hi);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) S.wa[threadIdx.x >> 5] = lo, S.wb[threadIdx.x >> 5] = hi;
        __syncthreads();
        for (int w = 0; w < SM_WARPS; ++w) lo = min(lo, S.wa[w]), hi = max(hi, S.wb[w]);
        if (threadIdx.x < blocks) {
            put(of_block(&S.told.lo[0][rank], threadIdx.x), lo);
            put(of_block(&S.told.hi[0][rank], threadIdx.x), hi);
        }
        meet();
        for (uint32_t r = 0; r < blocks; ++r) lo = min(lo, S.told.lo[0][r]), hi = max(hi, S.told.hi[0][r]);
        // every turn leaves a range a 2048th as long, so three at most
        while (lo < hi && members > FEW) {
            int shift = 0;
            while (((hi - lo) >> shift) >= BINS) ++shift;
            const uint32_t top = hi, bottom = lo;
            histogram([=](float v) {
                const uint32_t o = order_of(v);
                return o >= bottom && o <= top ? (top - o) >> shift : (uint32_t)BINS;
            }, true, false);
            find_bin(by_count, want_n, want_w, count0, mass0);
            bin = S.told.bin, members = S.told.members, count0 = S.told.count_before, mass0 = S.told.mass_before;
            hi = top - (bin << shift);
            lo = hi - bottom >> shift ? hi - ((1u << shift) - 1) : bottom;  // the bin's other end, or the range's
        }
        const uint32_t top = hi, bottom = lo;
        if (lo < hi)
            return among_few([=](float v) { return order_of(v) >= bottom && order_of(v) <= top; }, by_count, want_n, want_w,
                             count0, mass0);
        const u64 w = weight_of(sc, logit_of(hi));
        const uint32_t nth = by_count ? want_n - count0 : (uint32_t)((want_w - mass0 + w - 1) / w);
        return {hi, nth_of(hi, nth), count0 + nth, mass0 + nth * w};
    }

    // The bin of a logit: 128 of a unit of y where only the first 16 units count (BINS beyond
    // them), or 32, the last bin for all of 63.97 and more.  -infinity has none.
    static constexpr float NEAR = BINS / 16, FAR = BINS / 64;
    static E0_DEV uint32_t weight_bin(const Scale& s, float per_unit, float v) {
        if (v == -INFINITY) return BINS;
        const float y = y_of(s, v) * per_unit;
        if (y < (float)(BINS - 1)) return (uint32_t)y;
        return per_unit == NEAR ? (y < (float)BINS ? BINS - 1 : BINS) : BINS - 1;
    }
};

// ---------------------------------------------------------------- the kernel

E0_DEV void put_token(const SampleArgs& A, const Scale& s, int row, int token, float x, uint32_t kept, u64 w, u64 total) {
    A.token[row] = token;
    if (A.kept) A.kept[row] = (int32_t)kept;
    if (A.logp) {
        // ln(w / total), by what is left of 1 where that is small (w has 43 bits and more then)
        const float rest = (float)(total - w) / (float)total;
        A.logp[row] = rest < 0.5f ? log1pf(-rest) : ln_weight_of(s, x) - logf((float)total * 0x1p-44f);
    }
}

template <int TY>
__global__ void __launch_bounds__(SM_THREADS, 2) k_sample(SampleArgs A) {
    typedef typename Elem<TY>::T T;
    extern __shared__ __align__(16) char sample_sm[];
    SampleSmem& S = *reinterpret_cast<SampleSmem*>(sample_sm);
    float* x = reinterpret_cast<float*>(sample_sm + sizeof(SampleSmem));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), blocks = cluster_blocks();
    say_begun();
    const int row = blockIdx.x / blocks;
    const int from = min(A.V, (int)rank * A.slice), n = min(A.V, from + A.slice) - from;
    const float temp = A.temperature ? A.temperature[row] : 1.f;
    const float u = A.u[row];
    const float top_p = A.top_p ? A.top_p[row] : 1.f, min_p = A.min_p ? A.min_p[row] : 0.f;
    const int top_k = A.top_k ? A.top_k[row] : 0;
    if (tid == 0) {
        // (beyond 2^116 the factor would lose bits below fp32's normal numbers, and differences that count pass its range)
        const double c = 1.4426950408889634 / (double)fminf(temp, 0x1p116f);
        S.ch = (float)c, S.cl = (float)(c - (double)S.ch);
        S.least = min_p > 0.f ? (u64)((double)fminf(min_p, 1.f) * 17592186044416.0) : 0;  // 2^44
    }
    if (tid == 0) S.n_few = S.n_mine = 0;
    if (tid < STEPS_OF_ONE) S.steps[tid] = make_int2(STEPS.at[tid], __float_as_int((float)STEPS.at[tid]));
    for (int i = tid; i < BINS; i += SM_THREADS) S.count[i] = S.low[i] = S.high[i] = 0;  // for the first histogram
    // ---- the row's share, its largest logit
    const T* p = reinterpret_cast<const T*>(A.x) + (size_t)row * A.ld + from;
    float top = -INFINITY;
    int top_at = 0;
    bool odd = false;
    const auto take = [&](int i, float v) {  // a thread's tokens come in order
        x[i] = v;
        odd |= !(v < INFINITY);
        if (v > top) top = v, top_at = i;
    };
    constexpr int VEC = 16 / sizeof(T);
    const int lead = min(n, (int)((16 - ((uintptr_t)p & 15)) & 15) / (int)sizeof(T));
    for (int i = tid; i < lead; i += SM_THREADS) take(i, Elem<TY>::get(p[i]));
    const int vecs = (n - lead) / VEC;
#pragma unroll 4
    for (int k = tid; k < vecs; k += SM_THREADS) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p + lead) + k);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (TY == E0_F32) {
                take(lead + 4 * k + j, __uint_as_float(w[j]));
            } else {
                const float2 f = unpack16<TY>(w[j]);
                take(lead + 8 * k + 2 * j, f.x);
                take(lead + 8 * k + 2 * j + 1, f.y);
            }
        }
    }
    for (int i = lead + vecs * VEC + tid; i < n; i += SM_THREADS) take(i, Elem<TY>::get(p[i]));
    u64 best = ((u64)order_of(top) << 32) | (uint32_t)~(from + top_at);
#pragma unroll
    for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    odd = __any_sync(0xffffffffu, odd);
    if (lane == 0) S.wsum[warp] = best, S.wcount[warp] = odd;
    __syncthreads();
    all_begun();
    if (tid < blocks) {
        uint32_t some = 0;
        for (int w = 0; w < SM_WARPS; ++w) best = max(best, S.wsum[w]), some |= S.wcount[w];
        put(of_block(&S.told.best[rank], tid), best);
        put(of_block(&S.told.odd[rank], tid), some);
    }
    meet();
    uint32_t some = 0;
    best = 0;
    for (uint32_t r = 0; r < blocks; ++r) best = max(best, S.told.best[r]), some |= S.told.odd[r];
    const float most = logit_of((uint32_t)(best >> 32));
    const bool refused = some || !(most > -INFINITY) || !(temp >= 0.f && temp < INFINITY) || !(u >= 0.f && u <= 1.f) ||
                         top_p != top_p || min_p != min_p;
    if (refused || temp < 7.8886090522101181e-31f || top_k == 1) {  // no token, or the first one
        if (rank == 0 && tid == 0) {
            A.token[row] = refused ? -1 : (int)~(uint32_t)best;
            if (A.logp) A.logp[row] = refused ? -INFINITY : 0.f;
            if (A.kept) A.kept[row] = refused ? 0 : 1;
            if (refused) set_status(A.st, E0_ST_NONFINITE);
        }
        return;  // every block of the row leaves here, and none reads another's memory after the meeting
    }
    Row R = {S, x, n, from, rank, blocks, {most, S.ch, S.cl, S.steps}, Row::NEAR, false, 0, 0, 0};
    // ---- the end of what top-k and top-p keep
    End end = {0, 0xFFFFFFFFu, 0, 0};
    const bool by_k = top_k > 0 && top_k < A.V, by_p = top_p < 1.f;
    const u64 part_p = fraction_of(fminf(fmaxf(top_p, 0.f), 0.99999994f));
    // the least whole sum that is not below top_p times m; at least the first token
    const auto wanted = [&](u64 m) { return max(__umul64hi(part_p, m) + (part_p * m != 0), 1ull); };
    if (by_k || by_p) {
        const auto bin_of = [&R](float v) { return Row::weight_bin(R.sc, R.per_unit, v); };
        // all weights' sum is needed where top-p is of all tokens
        R.histogram(bin_of, by_p, by_p && !by_k, false);
        uint32_t c;
        u64 m;
        R.totals(c, m);
        R.find_bin(by_k, top_k, wanted(m), 0, 0);
        if (S.told.members == 0) {  // not among the weights above 2^-16: all of them
            R.per_unit = Row::FAR;
            R.histogram(bin_of, by_p, false);
            R.totals(c, m);
            // top-k of more tokens than there are keeps all of them
            R.find_bin(by_k && (uint32_t)top_k < c, top_k, wanted(m), 0, 0);
        }
        const bool cut = by_k && (R.per_unit == Row::NEAR || (uint32_t)top_k < c);
        if ((cut || by_p) && S.told.count_before + S.told.members <= ALL) {
            // ---- few tokens: the first block ends the row
            const uint32_t bin = S.told.bin;
            R.gather([&](float v) { return bin_of(v) <= bin; });
            if (rank != 0) return;
            const int all = (int)S.n_few;
            const u64 me = tid < all ? S.few[tid] : 0, w = tid < all ? S.few_w[tid] : 0;
            uint32_t before = 0;
            u64 sum = 0;
            if (tid < all)
                for (int j = 0; j < all; ++j) {
                    const bool is = S.few[j] > me;
                    before += is;
                    sum += is ? S.few_w[j] : 0;
                }
            // those within top-k, and their sum
            const bool in_k = tid < all && (!cut || before < (uint32_t)top_k);
            u64 mine = warp_total(in_k ? w : 0);
            if (lane == 0) S.wsum[warp] = mine;
            __syncthreads();
            u64 of_k = 0;
            for (int i = 0; i < SM_WARPS; ++i) of_k += S.wsum[i];
            __syncthreads();
            if (!cut) of_k = m;
            const bool keep = in_k && (!by_p || sum < wanted(of_k)) && w >= S.least;
            // the draw: by number, which few_w's place gets in place of the order
            if (tid < all) S.few[tid] = keep ? ~(uint32_t)me : 0xFFFFFFFFull;
            const uint32_t kept = __popc(__ballot_sync(0xffffffffu, keep));
            mine = warp_total(keep ? w : 0);
            if (lane == 0) S.wsum[warp] = mine, S.wcount[warp] = kept;
            __syncthreads();
            u64 total = 0;
            uint32_t count = 0;
            for (int i = 0; i < SM_WARPS; ++i) total += S.wsum[i], count += S.wcount[i];
            if (!keep) return;
            u64 want = u < 1.f ? __umul64hi(fraction_of(u), total) : total;
            if (want >= total) want = total - 1;
            const uint32_t id = ~(uint32_t)me;
            u64 run = 0;
            for (int j = 0; j < all; ++j)
                if ((uint32_t)S.few[j] < id) run += S.few_w[j];
            if (run <= want && want < run + w) put_token(A, R.sc, row, (int)id, logit_of((uint32_t)(me >> 32)), count, w, total);
            return;
        }
        // of top-k, then of top-p within these
#pragma unroll 1
        for (bool by_count = cut; by_count || by_p;) {
            end = R.find(by_count, top_k, wanted(m), !by_count && S.least == 0);
            if (!by_count || !by_p) break;
            by_count = false;
            m = end.mass;
            R.per_unit = Row::NEAR;
            R.histogram(bin_of, true, false);
            R.find_bin(false, 0, wanted(m), 0, 0);
            if (S.told.members == 0) {  // their sum ends in another bin
                R.per_unit = Row::FAR;
                R.histogram(bin_of, true, false);
                R.find_bin(false, 0, wanted(m), 0, 0);
            }
        }
    }
    // ---- sums of the kept tokens' weights: a warp has consecutive tokens
    const int per = (n + SM_THREADS - 1) / SM_THREADS * 32, i0 = min(n, warp * per), i1 = min(n, i0 + per);
    const u64 least = S.least;
    // logits that cannot be kept are told by a comparison: the end's, and half a bit below min_p's
    const float floor = min_p > 0.f ? most - (0.5f - log2f(fminf(min_p, 1.f))) / S.ch : -FLT_MAX;
    const float lowest = fmaxf(end.key ? logit_of(end.key) : -FLT_MAX, fmaxf(floor, -FLT_MAX));
    const auto kept = [&](int i, u64& w) {  // i < n
        const float v = x[i];
        if (!(v >= lowest) || !end.holds(order_of(v), from + i)) return false;
        w = weight_of(R.sc, v);
        return w >= least;
    };
    u64 all = R.own_mass, before = 0, total = 0, want = 0;
    uint32_t total_count = R.own_count;
    // Where the histogram has said what the block has of them, only the block of the draw adds them up.
#pragma unroll 1
    for (bool here = false;;) {
        if (here || !R.known) {
            u64 sum = 0;
            uint32_t count = 0;
            for (int ib = i0; ib < i1; ib += BATCH * 32) {
                float v[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int i = ib + 32 * k + lane;
                    v[k] = i < i1 ? x[i] : -INFINITY;
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    if (!__any_sync(0xffffffffu, v[k] >= lowest)) continue;
                    const u64 w = weight_of(R.sc, v[k]);
                    if (v[k] >= lowest && end.holds(order_of(v[k]), from + ib + 32 * k + lane) && w >= least) sum += w, ++count;
                }
            }
            sum = warp_total(sum), count = warp_total(count);
            __syncthreads();
            if (lane == 0) S.wsum[warp] = sum, S.wcount[warp] = count;
            __syncthreads();
            if (here) break;
            for (int w = 0; w < SM_WARPS; ++w) all += S.wsum[w], total_count += S.wcount[w];
        }
        if (tid < blocks) {
            put(of_block(&S.told.mass[0][rank], tid), all);
            put(of_block(&S.told.count[0][rank], tid), total_count);
        }
        meet();  // the last one: each block goes on with its own memory
        total_count = 0;
        for (uint32_t r = 0; r < blocks; ++r) {
            if (r == rank) before = total;
            total += S.told.mass[0][r], total_count += S.told.count[0][r];
        }
        // the first token whose running sum exceeds u * total
        want = u < 1.f ? __umul64hi(fraction_of(u), total) : total;
        if (want >= total) want = total - 1;
        if (want < before || want >= before + all) return;
        if (!R.known) break;
        here = true;
    }
    int at = 0;  // the warp whose tokens it is among
    while (want >= before + S.wsum[at]) before += S.wsum[at++];
    // the block shares that warp's tokens, consecutive ones a thread
    const int j0 = at * per, j1 = min(n, j0 + per), each = (j1 - j0 + SM_THREADS - 1) / SM_THREADS;
    const int a0 = min(j1, j0 + tid * each), a1 = min(j1, a0 + each);
    u64 mine = 0;
    for (int i = a0; i < a1; ++i) {
        u64 w;
        if (kept(i, w)) mine += w;
    }
    const u64 inc = warp_scan(mine);
    __syncthreads();
    if (lane == 31) S.wsum[warp] = inc;
    __syncthreads();
    before += inc - mine;
    for (int w = 0; w < warp; ++w) before += S.wsum[w];
    if (want < before || want >= before + mine) return;
    for (int i = a0; i < a1; ++i) {
        u64 w;
        if (!kept(i, w)) continue;
        if (want < before + w) {
            put_token(A, R.sc, row, from + i, x[i], total_count, w, total);
            return;
        }
        before += w;
    }
}

template <int TY>
int launch(SampleArgs a, int T, cudaStream_t s) {
    static std::atomic<uint64_t> asked{0};
    const size_t most = sizeof(SampleSmem) + (size_t)(E0_MAX_VOCAB / MOST_BLOCKS) * sizeof(float);
    if (!allow_smem((const void*)k_sample<TY>, most, asked)) return E0_ERR_CUDA;
    // Blocks of a row: shares of 2048 tokens and less while there are more blocks to have (one row
    // of 32000: 13.6 us with eight, 15.5 with four, 23 with two, 32 with one).
    int blocks = 1;
    while (blocks < MOST_BLOCKS && (a.V + blocks - 1) / blocks > 2048) blocks *= 2;
    a.slice = ((a.V + blocks - 1) / blocks + 7) / 8 * 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)T * blocks);
    cfg.blockDim = dim3(SM_THREADS);
    cfg.dynamicSmemBytes = sizeof(SampleSmem) + (size_t)a.slice * sizeof(float);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_sample<TY>, a) == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

}  // namespace

int sample(const void* x, int dtype, int64_t ld, int T, int V, const e0_sampling* r, const float* u, int32_t* token,
           float* logp, int32_t* kept, uint32_t* st, cudaStream_t s) {
    SampleArgs a = {};
    a.x = x, a.u = u, a.token = token, a.logp = logp, a.kept = kept, a.st = st, a.ld = ld, a.V = V;
    if (r) a.temperature = r->temperature, a.top_k = r->top_k, a.top_p = r->top_p, a.min_p = r->min_p;
    switch (dtype) {
        case E0_F32: return launch<E0_F32>(a, T, s);
        case E0_F16: return launch<E0_F16>(a, T, s);
        default: return launch<E0_BF16>(a, T, s);
    }
}

}  // namespace e0
