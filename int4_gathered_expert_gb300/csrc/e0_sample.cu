// The next tokens from the logits: temperature, top-k, top-p, min-p, one draw a row
// (e0_sample).
#include <cuda_runtime.h>

#include "e0_internal.h"
#include "e0_types.cuh"

namespace e0 {
namespace {

// A row belongs to a cluster of up to eight thread blocks, which hold it in shared memory
// as fp32: it is read from memory once, and what bounds the kernel beyond that is the chain
// of passes over shared memory and meetings of the cluster.  Nothing is sorted.  The kept
// tokens are a beginning of the row in the order "larger logit, then lower token", so all
// there is to find is its last member:
//   - a histogram over bins of equal width in log2 of the weight (counts and weights' sums)
//     says in which bin it is;
//   - the bin's members, few as a rule, go to one block, where each adds up the members
//     before itself: the last one is that whose sum passes what is wanted;
//   - a bin of many members is divided again, by the bits of the logits, until few are left
//     or all that are left are equal, where the order is that of the tokens.
// The draw then needs no order: the first token, by number, whose running sum of kept
// weights exceeds u times their total.
//
// A draw over V tokens has V borders, and an error in the sums moves all of them: with fp32
// exponentials one row in a hundred would get another token than the definition gives.
// So a weight 2^-y, y = (largest - logit) log2 e / temperature, is a 64-bit integer, 2^44
// times its value, good to 2^-29 of itself: y comes from a difference and a product that
// carry their rounding errors along (Dekker, Numer. Math. 18, 1971), its fraction goes through the power
// series of 2^-f in 32-bit fixed point.  Sums of integers are exact in any order, so
// equal calls give equal tokens.  Weights below 2^-44 of the largest count as nothing.
constexpr int SM_THREADS = 512, SM_WARPS = SM_THREADS / 32;
constexpr int MOST_BLOCKS = 8;
constexpr int BINS = 2048;
constexpr int FEW = 1024;  // members of a bin that one block takes
constexpr int WEIGHT_BITS = 44;

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
    uint32_t n_few;
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
};

// y of a logit (>= 0) as fp32, monotone in the logit; and the exact one's rest.
E0_DEV float y_of(const Scale& s, float x) { return (s.most - x) * s.ch; }

constexpr long long fixed(double v) { return (long long)(v * 2147483648.0 + (v < 0 ? -0.5 : 0.5)); }

// 2^44 * 2^-y.  2^-f, f in [0, 1), is the series of 2^-1/2 * 2^-r around f = 1/2, r = f - 1/2:
// the ninth term is below 2^-32.
E0_DEV u64 weight_of(const Scale& s, float x) {
    const float d = s.most - x;
    const float back = d - s.most;
    const float dl = (s.most - (d - back)) - (x + back);  // d + dl is the difference
    const float p = __fmul_rn(d, s.ch);  // not to be joined with the subtraction below
    if (!(p < (float)(WEIGHT_BITS + 1))) return 0;
    const float e = fmaf(d, s.ch, -p) + fmaf(d, s.cl, dl * s.ch);
    const float whole = floorf(p);
    const long long y = ((long long)whole << 32) + (long long)__float2uint_rz((p - whole) * 4294967296.f) +
                        (long long)__float2int_rn(e * 4294967296.f);
    if (y <= 0) return 1ull << WEIGHT_BITS;
    const int r = (int)((uint32_t)y ^ 0x80000000u);  // (f - 1/2) 2^32
    constexpr double A = 0.70710678118654752, L = -0.69314718055994531;
    constexpr double A1 = A * L, A2 = A1 * L / 2, A3 = A2 * L / 3, A4 = A3 * L / 4, A5 = A4 * L / 5, A6 = A5 * L / 6,
                     A7 = A6 * L / 7, A8 = A7 * L / 8;
    int g = (int)fixed(A8);
    g = (int)fixed(A7) + __mulhi(g, r);
    g = (int)fixed(A6) + __mulhi(g, r);
    g = (int)fixed(A5) + __mulhi(g, r);
    g = (int)fixed(A4) + __mulhi(g, r);
    g = (int)fixed(A3) + __mulhi(g, r);
    g = (int)fixed(A2) + __mulhi(g, r);
    g = (int)fixed(A1) + __mulhi(g, r);
    g = (int)fixed(A) + __mulhi(g, r);  // 2^31 * 2^-f, at least 2^30
    return ((u64)(uint32_t)g << (WEIGHT_BITS - 31)) >> (int)(y >> 32);
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

    // Counts and sums of this block's tokens by bin (`bin_of` gives BINS for none) and, in
    // told[1], of every block's tokens in all.
    template <typename F>
    E0_DEV void histogram(F bin_of) {
        for (int i = threadIdx.x; i < BINS; i += SM_THREADS) S.count[i] = S.low[i] = S.high[i] = 0;
        __syncthreads();
        u64 m = 0;
        uint32_t c = 0;
#pragma unroll 2
        for (int i = threadIdx.x; i < n; i += SM_THREADS) {
            const uint32_t b = bin_of(x[i]);
            if (b >= BINS) continue;
            const u64 w = weight_of(sc, x[i]);
            ++c, m += w;
            atomicAdd(&S.count[b], 1u);
            const uint32_t lo = (uint32_t)w, was = atomicAdd(&S.low[b], lo);
            const uint32_t hi = (uint32_t)(w >> 32) + (was + lo < lo);
            if (hi) atomicAdd(&S.high[b], hi);
        }
        c = warp_total(c), m = warp_total(m);
        if ((threadIdx.x & 31) == 0) S.wcount[threadIdx.x >> 5] = c, S.wsum[threadIdx.x >> 5] = m;
        __syncthreads();
        if (threadIdx.x < blocks) {
            c = 0, m = 0;
            for (int w = 0; w < SM_WARPS; ++w) c += S.wcount[w], m += S.wsum[w];
            put(of_block(&S.told.count[1][rank], threadIdx.x), c);
            put(of_block(&S.told.mass[1][rank], threadIdx.x), m);
        }
        meet();
    }

    // The bin in which the running count (of what stands before it and `count` before the
    // first bin) first reaches want_n, or the running sum want_w.  The blocks share the bins.
    E0_DEV void find_bin(bool by_count, uint32_t want_n, u64 want_w, uint32_t count0, u64 mass0) {
        const int per = BINS / blocks, mine = rank * per;
        const int each = (per + SM_THREADS - 1) / SM_THREADS;  // 4 where the block is alone
        uint32_t c[4];
        u64 m[4], mt = 0;
        uint32_t ct = 0;
        const int b0 = threadIdx.x * each;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            c[k] = 0, m[k] = 0;
            const int b = b0 + k;
            if (k < each && b < per) {
                uint32_t v[MOST_BLOCKS][3];
#pragma unroll
                for (uint32_t r = 0; r < MOST_BLOCKS; ++r) {
                    v[r][0] = v[r][1] = v[r][2] = 0;
                    if (r < blocks) {
                        v[r][0] = get32(of_block(&S.count[mine + b], r));
                        v[r][1] = get32(of_block(&S.low[mine + b], r));
                        v[r][2] = get32(of_block(&S.high[mine + b], r));
                    }
                }
#pragma unroll
                for (uint32_t r = 0; r < MOST_BLOCKS; ++r) c[k] += v[r][0], m[k] += ((u64)v[r][2] << 32) + v[r][1];
            }
            ct += c[k], mt += m[k];
        }
        const uint32_t cs = warp_scan(ct);
        const u64 ms = warp_scan(mt);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 31) S.wcount[warp] = cs, S.wsum[warp] = ms;
        __syncthreads();
        uint32_t cb = cs - ct, call = 0;
        u64 mb = ms - mt, mall = 0;
        for (int w = 0; w < SM_WARPS; ++w) {
            if (w < warp) cb += S.wcount[w], mb += S.wsum[w];
            call += S.wcount[w], mall += S.wsum[w];
        }
        if (threadIdx.x < blocks) {
            put(of_block(&S.told.count[0][rank], threadIdx.x), call);
            put(of_block(&S.told.mass[0][rank], threadIdx.x), mall);
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

    // Of the tokens with `in(logit)`, `members` in all, after count0 tokens of sum mass0:
    // the one with which the count reaches want_n or the sum want_w.  One block takes them.
    template <typename F>
    E0_DEV End among_few(F in, bool by_count, uint32_t want_n, u64 want_w, uint32_t count0, u64 mass0) {
        if (threadIdx.x == 0) S.n_few = 0;
        meet();
        for (int i = threadIdx.x; i < n; i += SM_THREADS)
            if (in(x[i])) {
                const uint32_t at = add_to(of_block(&S.n_few, 0), 1u);
                if (at < FEW) {
                    put(of_block(&S.few[at], 0), ((u64)order_of(x[i]) << 32) | (uint32_t)~(from + i));  // larger is earlier
                    put(of_block(&S.few_w[at], 0), weight_of(sc, x[i]));
                }
            }
        meet();
        if (rank == 0) {
            const int m = min(S.n_few, (uint32_t)FEW);
            for (int i = threadIdx.x; i < m; i += SM_THREADS) {
                const u64 me = S.few[i], w = S.few_w[i];
                uint32_t cb = count0;
                u64 mb = mass0;
#pragma unroll 4
                for (int j = 0; j < m; ++j) {
                    const bool before = S.few[j] > me;
                    cb += before;
                    mb += before ? S.few_w[j] : 0;
                }
                // by weight: members without weight pass nothing, so this is one member too
                if (by_count ? cb + 1 == want_n : mb < want_w && want_w <= mb + w)
                    for (uint32_t r = 0; r < blocks; ++r) {
                        put(of_block(&S.told.key, r), (uint32_t)(me >> 32));
                        put(of_block(&S.told.index, r), ~(uint32_t)me);
                        put(of_block(&S.told.count_through, r), cb + 1);
                        put(of_block(&S.told.mass_through, r), mb + w);
                    }
            }
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
    // their sum want_w (> 0, at most the row's).  The histogram by weight is there; `again`
    // says whether its bins were needed for another.
    E0_DEV End find(bool by_count, uint32_t want_n, u64 want_w, bool& again) {
        again = false;
        find_bin(by_count, want_n, want_w, 0, 0);
        uint32_t bin = S.told.bin, members = S.told.members, count0 = S.told.count_before;
        u64 mass0 = S.told.mass_before;
        const Scale s = sc;
        const auto in_first = [s, bin](float v) { return weight_bin(s, v) == bin; };
        if (members <= FEW) return among_few(in_first, by_count, want_n, want_w, count0, mass0);
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
            again = true;
            while (((hi - lo) >> shift) >= BINS) ++shift;
            const uint32_t top = hi, bottom = lo;
            histogram([=](float v) {
                const uint32_t o = order_of(v);
                return o >= bottom && o <= top ? (top - o) >> shift : (uint32_t)BINS;
            });
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

    // Bins of 1/32 in y; the last holds all of 63.97 and more, but for -infinity.
    static E0_DEV uint32_t weight_bin(const Scale& s, float v) {
        if (v == -INFINITY) return BINS;
        const float y = y_of(s, v) * 32.f;
        return y < (float)(BINS - 1) ? (uint32_t)y : (uint32_t)(BINS - 1);
    }
};

// ---------------------------------------------------------------- the kernel

template <int TY>
__global__ void __launch_bounds__(SM_THREADS) k_sample(SampleArgs A) {
    typedef typename Elem<TY>::T T;
    extern __shared__ __align__(16) char sample_sm[];
    SampleSmem& S = *reinterpret_cast<SampleSmem*>(sample_sm);
    float* x = reinterpret_cast<float*>(sample_sm + sizeof(SampleSmem));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), blocks = cluster_blocks();
    const int row = blockIdx.x / blocks;
    const int from = min(A.V, (int)rank * A.slice), n = min(A.V, from + A.slice) - from;
    const float temp = A.temperature ? A.temperature[row] : 1.f;
    const float u = A.u[row];
    const float top_p = A.top_p ? A.top_p[row] : 1.f, min_p = A.min_p ? A.min_p[row] : 0.f;
    const int top_k = A.top_k ? A.top_k[row] : 0;
    if (tid == 0) {
        const double c = 1.4426950408889634 / (double)temp;
        S.ch = (float)c, S.cl = (float)(c - (double)S.ch);
        S.least = min_p > 0.f ? (u64)((double)fminf(min_p, 1.f) * 17592186044416.0) : 0;  // 2^44
    }
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
    Row R = {S, x, n, from, rank, blocks, {most, S.ch, S.cl}};
    // ---- the end of what top-k and top-p keep
    End end = {0, 0xFFFFFFFFu, 0, 0};
    const bool by_k = top_k > 0 && top_k < A.V, by_p = top_p < 1.f;
    if (by_k || by_p) {
        const Scale sc = R.sc;
        R.histogram([sc](float v) { return Row::weight_bin(sc, v); });
        // the row's tokens (without -infinity) and their sum
        uint32_t c = 0;
        u64 m = 0;
        for (uint32_t r = 0; r < blocks; ++r) c += S.told.count[1][r], m += S.told.mass[1][r];
        bool again = false;
        const bool cut = by_k && (uint32_t)top_k < c;
        if (cut) {
            end = R.find(true, top_k, 0, again);
            m = end.mass;
        }
        if (by_p) {
            // the least whole sum that is not below top_p times m; at least the first token
            const u64 part = fraction_of(fmaxf(top_p, 0.f));
            u64 w = __umul64hi(part, m) + (part * m != 0);
            if (w < 1) w = 1;
            if (again) R.histogram([sc](float v) { return Row::weight_bin(sc, v); });
            end = R.find(false, 0, w, again);
        }
    }
    // ---- sums of the kept tokens' weights: a warp has consecutive tokens
    const int per = (n + SM_THREADS - 1) / SM_THREADS * 32, i0 = min(n, warp * per), i1 = min(n, i0 + per);
    const u64 least = S.least;
    const auto kept = [&](int i, u64& w) {  // i < n
        const float v = x[i];
        if (!(v > -INFINITY) || !end.holds(order_of(v), from + i)) return false;
        w = weight_of(R.sc, v);
        return w >= least;
    };
    u64 sum = 0;
    uint32_t count = 0;
#pragma unroll 4
    for (int i = i0 + lane; i < i1; i += 32) {
        u64 w;
        if (kept(i, w)) sum += w, ++count;
    }
    sum = warp_total(sum), count = warp_total(count);
    __syncthreads();
    if (lane == 0) S.wsum[warp] = sum, S.wcount[warp] = count;
    __syncthreads();
    u64 all = 0, before = 0;
    uint32_t total_count = 0;
    for (int w = 0; w < SM_WARPS; ++w) all += S.wsum[w], total_count += S.wcount[w];
    if (tid < blocks) {
        put(of_block(&S.told.mass[0][rank], tid), all);
        put(of_block(&S.told.count[0][rank], tid), total_count);
    }
    meet();  // the last one: each block goes on with its own memory
    u64 total = 0;
    total_count = 0;
    for (uint32_t r = 0; r < blocks; ++r) {
        if (r == rank) before = total;
        total += S.told.mass[0][r], total_count += S.told.count[0][r];
    }
    // the first token whose running sum exceeds u * total
    u64 want = u < 1.f ? __umul64hi(fraction_of(u), total) : total;
    if (want >= total) want = total - 1;
    if (want < before || want >= before + all) return;
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
            A.token[row] = from + i;
            if (A.kept) A.kept[row] = total_count;
            if (A.logp) {
                // ln(w / total), by what is left of 1 where that is small
                const float rest = (float)(total - w) / (float)total;
                A.logp[row] = rest < 0.5f ? log1pf(-rest) : logf((float)w / (float)total);
            }
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
    // blocks of a row: shares of 2048 tokens and more
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
