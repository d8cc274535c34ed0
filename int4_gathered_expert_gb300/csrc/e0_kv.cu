// The paged 8-bit KV cache: block tables and slot maps from sequence lengths
// (e0_kv_plan, e0_kv_release) and writing keys and values (e0_kv_append).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "e0_internal.h"
#include "e0_types.cuh"

namespace cg = cooperative_groups;

namespace e0 {
namespace {

// ------------------------------------------------------------------ plan and release
//
// Both are a prefix sum over the sequences and then work on every new token or
// place of the table.  Every thread block computes the whole prefix sum by
// itself (B lengths, a few KB out of L2) and takes its share of the rest, so a plan
// is one launch without blocks waiting on one another.  Only new lengths and stack
// height written over the old ones must come after every block has read those: in
// the same block where there is one, else in a second launch.
// Bound by latency: a launch, the lengths' loads, two barriers, a search.  Measured
// (device time, GB300): 64 sequences, a token each, 3.4 us; 300 sequences, 73739
// tokens, 5.2 us.

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_ONE_BLOCK = 4096;  // tokens that one thread block takes

// What the lengths come to: sequence b's first token and first block, in
// shared memory, and the totals; ok false where the request cannot be met.
struct PlanSums {
    int32_t* tok;   // [B + 1]
    int32_t* blk;   // [B + 1]
    int32_t* ctx;   // [B]
    int total_tok, total_blk, height;
    bool ok;
};

// Inclusive sums over the block's threads of two values.
E0_DEV void block_scan2(long long& a, long long& b, long long (*red)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) a += x, b += y;
    }
    if (lane == 31) red[warp][0] = a, red[warp][1] = b;
    __syncthreads();
    long long sa = 0, sb = 0;
    for (int i = 0; i < warp; ++i) sa += red[i][0], sb += red[i][1];
    a += sa, b += sb;
}

struct PlanArgs {
    int32_t* table;
    const int32_t* ctx;
    int32_t* free_list;
    const int32_t* free_count;
    const int32_t* new_len;   // plan
    const uint8_t* mask;      // release
    int32_t* ctx_out;
    int32_t* free_out;
    int32_t* cu_q;
    int64_t* slots;
    int32_t* positions;
    int32_t* seq_ids;
    uint32_t* st;
    int B, max_blocks, shift, n_blocks, T_cap;
    bool fill, commit;        // plan: write slots and tables; write ctx_out and free_out
};

template <bool RELEASE>
E0_DEV PlanSums plan_sums(const PlanArgs& A, int32_t* sm) {
    __shared__ long long red[PLAN_THREADS / 32][2];
    PlanSums S;
    S.tok = sm, S.blk = sm + A.B + 1, S.ctx = sm + 2 * (A.B + 1);
    const int per = (A.B + blockDim.x - 1) / blockDim.x, b0 = threadIdx.x * per;
    const long long bs = 1ll << A.shift, room = (long long)A.max_blocks << A.shift;
    long long nt = 0, nb = 0;
    bool bad_len = false, full = false;
    for (int i = 0; i < per; ++i) {
        const int b = b0 + i;
        if (b >= A.B) break;
        const int c = A.ctx[b], n = RELEASE ? 0 : A.new_len[b];
        const bool on = RELEASE ? A.mask[b] != 0 : true;
        bad_len |= on && (c < 0 || n < 0 || (long long)c + n > room);
        if (on) {
            nt += n;
            nb += RELEASE ? ((c + bs - 1) >> A.shift) : ((c + n + bs - 1) >> A.shift) - ((c + bs - 1) >> A.shift);
        }
    }
    long long it = nt, ib = nb;
    block_scan2(it, ib, red);
    __shared__ long long tot[2];
    if (threadIdx.x == blockDim.x - 1) tot[0] = it, tot[1] = ib;
    __syncthreads();
    S.height = *A.free_count;
    full = tot[0] > A.T_cap;
    bad_len |= S.height < 0 || S.height > A.n_blocks;
    if (RELEASE)
        bad_len |= tot[1] > E0_MAX_ROWS;  // places, whether there is a block in them or not
    else
        full |= tot[1] > S.height;
    bad_len = __syncthreads_or(bad_len);
    S.ok = !bad_len && !full;
    if (!S.ok && blockIdx.x == 0 && threadIdx.x == 0)
        set_status(A.st, bad_len ? E0_ST_BAD_LENGTH : E0_ST_POOL_FULL);
    S.total_tok = S.ok ? (int)tot[0] : 0;
    S.total_blk = S.ok ? (int)tot[1] : 0;
    long long t = it - nt, k = ib - nb;
    for (int i = 0; i < per; ++i) {
        const int b = b0 + i;
        if (b >= A.B) break;
        const int c = A.ctx[b], n = RELEASE ? 0 : A.new_len[b];
        S.ctx[b] = c;
        S.tok[b] = S.ok ? (int)t : 0;
        S.blk[b] = S.ok ? (int)k : 0;
        if (S.ok && (!RELEASE || A.mask[b])) {
            t += n;
            k += RELEASE ? ((c + bs - 1) >> A.shift) : ((c + n + bs - 1) >> A.shift) - ((c + bs - 1) >> A.shift);
        }
    }
    if (threadIdx.x == 0) S.tok[A.B] = S.total_tok, S.blk[A.B] = S.total_blk;
    __syncthreads();
    return S;
}

// The last b < B with first[b] <= i.
E0_DEV int find_seq(const int32_t* first, int B, int i) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(PLAN_THREADS) k_kv_plan(PlanArgs A) {
    extern __shared__ int32_t plan_sm[];
    const PlanSums S = plan_sums<false>(A, plan_sm);
    const int bs = 1 << A.shift;
    if (A.fill) {
        const int n = gridDim.x * blockDim.x, at = blockIdx.x * blockDim.x + threadIdx.x;
        for (int i = at; i < S.total_blk; i += n) {
            const int b = find_seq(S.blk, A.B, i);
            const int id = A.free_list[S.height - 1 - i];
            const int j = ((S.ctx[b] + bs - 1) >> A.shift) + i - S.blk[b];
            A.table[(size_t)b * A.max_blocks + j] = id;
            if (id < 0 || id >= A.n_blocks) set_status(A.st, E0_ST_BAD_BLOCK);
        }
        for (int t = at; t < A.T_cap; t += n) {
            int64_t slot = -1;
            int pos = -1, b = -1;
            if (t < S.total_tok) {
                b = find_seq(S.tok, A.B, t);
                pos = S.ctx[b] + t - S.tok[b];
                const int held = (S.ctx[b] + bs - 1) >> A.shift, j = pos >> A.shift;
                const int id = j < held ? A.table[(size_t)b * A.max_blocks + j]
                                        : A.free_list[S.height - 1 - (S.blk[b] + j - held)];
                if (id >= 0 && id < A.n_blocks)
                    slot = ((int64_t)id << A.shift) + (pos & (bs - 1));
                else
                    set_status(A.st, E0_ST_BAD_BLOCK);
            }
            A.slots[t] = slot;
            if (A.positions) A.positions[t] = pos;
            if (A.seq_ids) A.seq_ids[t] = b;
        }
        if (blockIdx.x == 0)
            for (int b = threadIdx.x; b <= A.B; b += blockDim.x) A.cu_q[b] = S.tok[b];
    }
    // block 0 alone writes these; where they lie over the inputs it is the only block
    if (A.commit && blockIdx.x == 0) {
        for (int b = threadIdx.x; b < A.B; b += blockDim.x) A.ctx_out[b] = S.ctx[b] + (S.tok[b + 1] - S.tok[b]);
        if (threadIdx.x == 0) *A.free_out = S.height - S.total_blk;
    }
}

// Only ids of the pool go onto the stack, so how high it gets, and where an id goes, is
// known once all of them have been looked at.  The thread blocks of the cluster count
// their shares of the places, meet, and write theirs; they meet again before the first
// one writes what may lie over the lengths and the height.
// Measured (device time, GB300): 32 blocks of one sequence, 4.3 us; 6400 of 64 sequences, 7.7;
// 60000 of 300, 21 (as many independent thread blocks as SMs, which cannot know how many
// ids there are before theirs: 7.8 and a launch for the lengths in place).
__global__ void __launch_bounds__(PLAN_THREADS) k_kv_release(PlanArgs A) {
    extern __shared__ int32_t plan_sm[];
    __shared__ int32_t found, in_warp[PLAN_THREADS / 32];
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int ranks = gridDim.x, rank = blockIdx.x;
    if (tid == 0) found = 0;
    const PlanSums S = plan_sums<true>(A, plan_sm);
    const auto meet = [&]() {
        if (ranks > 1) cg::this_cluster().sync(); else __syncthreads();
    };
    const auto place = [&](int i) {
        const int b = find_seq(S.blk, A.B, i);
        return A.table + (size_t)b * A.max_blocks + (i - S.blk[b]);
    };
    const auto of_pool = [&](int id) { return id >= 0 && id < A.n_blocks; };
    const int share = (S.total_blk + ranks - 1) / ranks;
    const int i0 = min(rank * share, S.total_blk), i1 = min(i0 + share, S.total_blk);
    int n = 0;
#pragma unroll 4
    for (int i = i0 + tid; i < i1; i += nt) n += of_pool(*place(i));
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) atomicAdd(&found, n);
    meet();
    int before = 0, all = 0;
    for (int k = 0; k < ranks; ++k) {
        const int f = ranks > 1 ? *cg::this_cluster().map_shared_rank(&found, k) : found;
        all += f;
        if (k < rank) before += f;
    }
    const bool fits = (long long)S.height + all <= A.n_blocks;
    if (!fits && rank == 0 && tid == 0) set_status(A.st, E0_ST_BAD_LENGTH);
    if (fits && all == S.total_blk) {  // all places have a block
#pragma unroll 4
        for (int i = i0 + tid; i < i1; i += nt) {
            int32_t* p = place(i);
            A.free_list[S.height + i] = *p;
            *p = -1;
        }
    } else if (fits) {
        int at = S.height + before;
        for (int base = i0; base < i1; base += nt) {
            int id = -1;
            if (base + tid < i1) {
                int32_t* p = place(base + tid);
                id = *p;
                *p = -1;
                if (id != -1 && !of_pool(id)) set_status(A.st, E0_ST_BAD_BLOCK);
            }
            const uint32_t in = __ballot_sync(0xffffffffu, of_pool(id));
            if (lane == 0) in_warp[warp] = __popc(in);
            __syncthreads();
            int to = at + __popc(in & ((1u << lane) - 1));
            for (int w = 0; w < nt / 32; ++w) {
                if (w < warp) to += in_warp[w];
                at += in_warp[w];
            }
            if (of_pool(id)) A.free_list[to] = id;
            __syncthreads();  // in_warp has been read
        }
    }
    meet();  // every block has read the lengths, the height and the counts
    if (rank == 0) {
        for (int b = tid; b < A.B; b += nt) A.ctx_out[b] = S.ok && fits && A.mask[b] ? 0 : S.ctx[b];
        if (tid == 0) *A.free_out = S.height + (fits ? all : 0);
    }
}

constexpr size_t PLAN_MOST_SMEM = (3 * (size_t)E0_MAX_SEQS + 2) * sizeof(int32_t);
size_t plan_smem(int B) { return (3 * (size_t)B + 2) * sizeof(int32_t); }
int plan_threads(long long work, int B) { return work <= 256 && B <= 256 ? 256 : PLAN_THREADS; }

// Fill and commit in one launch where the outputs lie apart from the inputs or one
// thread block does it all, else one after the other.
int plan_launch(PlanArgs a, cudaStream_t s) {
    static std::atomic<uint64_t> asked{0};
    long long g = a.T_cap <= PLAN_ONE_BLOCK ? 1 : (a.T_cap + PLAN_THREADS - 1) / PLAN_THREADS;
    if (g > num_sms()) g = num_sms();
    const bool apart = a.ctx_out != a.ctx && a.free_out != a.free_count;
    a.fill = true;
    a.commit = g == 1 || apart;
    if (!allow_smem((const void*)k_kv_plan, PLAN_MOST_SMEM, asked)) return E0_ERR_CUDA;
    k_kv_plan<<<(int)g, plan_threads(a.T_cap, a.B), plan_smem(a.B), s>>>(a);
    if (!a.commit) {
        a.fill = false, a.commit = true;
        a.st = nullptr;  // said already
        k_kv_plan<<<1, PLAN_THREADS, plan_smem(a.B), s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

// A thread block, or a cluster of eight where the table has more places than that has threads.
int release_launch(const PlanArgs& a, cudaStream_t s) {
    static std::atomic<uint64_t> asked{0};
    const long long places = (long long)a.B * a.max_blocks;
    if (!allow_smem((const void*)k_kv_release, PLAN_MOST_SMEM, asked)) return E0_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3(places <= PLAN_THREADS ? 1 : 8);
    cfg.blockDim = dim3(plan_threads(places, a.B));
    cfg.dynamicSmemBytes = plan_smem(a.B);
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cfg.gridDim.x, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cfg.gridDim.x > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_kv_release, a) == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

PlanArgs plan_args(const e0_kv_state* k, int32_t* ctx_out, int32_t* free_out, uint32_t* st) {
    PlanArgs a = {};
    a.table = k->block_table, a.ctx = k->ctx_len, a.free_list = k->free_list, a.free_count = k->free_count;
    a.ctx_out = ctx_out, a.free_out = free_out, a.st = st;
    a.B = k->B, a.max_blocks = k->max_blocks, a.n_blocks = k->n_blocks;
    while ((1 << a.shift) < k->block_tokens) ++a.shift;
    return a;
}

// ------------------------------------------------------------------ append
//
// A run is the consecutive new tokens of one block of the cache; for a run, a head and
// keys or values the kernel finds the largest magnitude, settles the scale, rounds
// the older codes again if the scale grew, and writes the new ones.  A thread block
// finds the runs that begin among its `per` tokens.  Where a block of the cache is
// small, it has eight heads' keys or values and a warp for each; else it has one's and
// takes each run with all its warps or, where there are many (single tokens), one with
// each warp.  A lane has eight elements of a token, and some tokens stay in registers
// between the maximum and the codes, so most runs (up to 8192 elements by a thread
// block) are read once.  Scales are powers of two: x / s and code * old / new are then
// exact, so the only rounding is that to e4m3, and a scale that grows costs nothing
// but the codes that fall into e4m3's subnormals.  (A scale of max / 448 would round
// every older code again at each new maximum, and e4m3's relative precision gains
// nothing from it.)
// Measured (device time, GB300): 13013 tokens of 2 heads of 256 in fp16, 40 MB: 12.2 us,
// 3.3 TB/s: a run is a chain of slots, rows, a barrier and stores of 4 us, and an
// SM holds five thread blocks at a time; 64 single tokens of 8 heads of 128: 3.0 us.

constexpr int APP_WARPS = 8;

struct AppendArgs {
    const void* x[2];
    int64_t ld[2];
    uint8_t* codes[2];
    float* scale[2];
    const int64_t* slots;
    uint32_t* st;
    int T, Hkv, shift, n_blocks;
};

// The smallest 2^e >= 2^-100 with m / 448 (rounded) <= 2^e, for the bits of a finite m >= 0:
// 448 = 1.75 * 2^8, and the fp32 number after 1.75 * 2^k rounds to more than 2^(k - 8).
E0_DEV float pow2_scale(uint32_t m) {
    const int e = (int)(m >> 23) - 8 + ((m & 0x7FFFFFu) > 0x600000u);
    return __int_as_float(max(e, 27) << 23);
}

// A lane's eight elements of one token's head, as they are in memory.
template <int TY>
struct AppRaw {
    static constexpr int N = 8, WORDS = N * (TY == E0_F32 ? 4 : 2) / 4;
    uint32_t w[WORDS];
    E0_DEV void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0;
    }
    E0_DEV void load(const typename Elem<TY>::T* p, bool vec) {
        if (vec) {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
                w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
            }
        } else if constexpr (TY == E0_F32) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
        }
    }
    // The largest magnitude's bits with those of m: 16-bit types two at a time, each
    // half for itself until fp32_bits.
    E0_DEV uint32_t max_bits(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            m = TY == E0_F32 ? max(m, w[i] & 0x7FFFFFFFu) : __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        return m;
    }
    static E0_DEV uint32_t fp32_bits(uint32_t m) {
        if constexpr (TY == E0_F32) return m;
        const float2 f = unpack16<TY>(max(m & 0xFFFFu, m >> 16));
        return __float_as_uint(f.x);
    }
    E0_DEV void get(float (&v)[N]) const {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (TY == E0_F32) {
                v[i] = __uint_as_float(w[i]);
            } else {
                const float2 f = unpack16<TY>(w[i]);
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
            }
        }
    }
};

// Slots of the 64 tokens from `base`, two a lane; -1 behind the last one.
struct Slots {
    int64_t lo, hi;
    E0_DEV void load(const AppendArgs& A, long long base, int lane) {
        lo = base + lane < A.T ? A.slots[base + lane] : -1;
        hi = base + 32 + lane < A.T ? A.slots[base + 32 + lane] : -1;
    }
};

// The run that begins with token base + j, by the calling warp (TEAM 1) or by all warps
// of the thread block together.  HOLD: steps of the run that stay in registers.
template <int TY, int D, int TEAM, int HOLD>
E0_DEV void append_run(const AppendArgs& A, bool vec, int which, int head, int base, int j, const Slots& near,
                       uint32_t* most) {
    typedef typename Elem<TY>::T T;
    constexpr int N = 8, LANES = D / N, AT_ONCE = TEAM * 32 / LANES;  // tokens that the team reads in a step
    const int lane = threadIdx.x & 31, member = TEAM == 1 ? 0 : threadIdx.x >> 5;
    const int bs = 1 << A.shift, t0 = base + j, mine = (member * 32 + lane) / LANES, at = lane % LANES * N;
    const int64_t slot = __shfl_sync(0xffffffffu, near.lo, j);
    const int off = (int)(slot & (bs - 1));
    const int64_t blk = slot >> A.shift;
    if (blk >= A.n_blocks) {
        if (member == 0 && lane == 0) set_status(A.st, E0_ST_BAD_BLOCK);
        return;
    }
    float* scale = (which ? A.scale[1] : A.scale[0]) + (size_t)blk * A.Hkv + head;
    float old = off > 0 ? *scale : 0.f;
    // the run's length: tokens that follow with consecutive slots inside the block
    int n;
    {
        const int64_t first = slot - j + lane;
        const uint64_t follow = (uint64_t)__ballot_sync(0xffffffffu, near.hi == first + 32) << 32 |
                                __ballot_sync(0xffffffffu, near.lo == first);
        n = __ffsll(~(follow >> j)) - 1;  // j = 0 and all 64: -1
        if (n < 0) n = 64;
        if (n == 64 - j)
            for (;;) {
                const int i = n + lane;
                const bool in = off + i < bs && t0 + i < A.T && A.slots[t0 + i] == slot + i;
                const uint32_t out = ~__ballot_sync(0xffffffffu, in);
                n += out ? __ffs(out) - 1 : 32;
                if (out) break;
            }
        n = min(n, bs - off);
    }
    // the lane has a part of the tokens mine, mine + AT_ONCE, ...
    const int64_t ld = which ? A.ld[1] : A.ld[0];
    const T* x = reinterpret_cast<const T*>(which ? A.x[1] : A.x[0]) + (t0 + mine) * ld + (size_t)head * D + at;
    uint8_t* codes = (which ? A.codes[1] : A.codes[0]) + ((size_t)blk * A.Hkv + head) * ((size_t)D << A.shift);
    AppRaw<TY> held[HOLD];
    // batches of HOLD steps; a longer run is read again for its codes
    const bool once = n <= HOLD * AT_ONCE;
    const auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            if (i0 + mine + k * AT_ONCE < n)
                held[k].load(x + (i0 + k * AT_ONCE) * ld, vec);
            else
                held[k].zero();
    };
    load(0);
    // largest magnitude as bits: of the values, and of those that are finite
    uint32_t all = 0, m = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += HOLD * AT_ONCE) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int k = 0; k < HOLD; ++k) all = held[k].max_bits(all);
    }
    all = __reduce_max_sync(0xffffffffu, AppRaw<TY>::fp32_bits(all));
    const bool plain = all < 0x7F800000u;  // what this warp has is finite
    if (plain) {
        m = all;
    } else {
        if (lane == 0) set_status(A.st, E0_ST_NONFINITE);
#pragma unroll 1
        for (int i = 0; i < n - mine; i += AT_ONCE) {
            AppRaw<TY> r;
            r.load(x + i * ld, vec);
            float v[N];
            r.get(v);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint32_t a = __float_as_uint(v[j]) & 0x7FFFFFFFu;
                m = max(m, a < 0x7F800000u ? a : 0u);
            }
        }
        m = __reduce_max_sync(0xffffffffu, m);
    }
    if constexpr (TEAM > 1) {
        if (lane == 0) most[member] = m;
        __syncthreads();  // and the old scale has been read
#pragma unroll
        for (int w = 0; w < TEAM; ++w) m = max(m, most[w]);
        __syncthreads();  // most has been read
    } else {
        __syncwarp();
    }
    float s = pow2_scale(m);
    if (off > 0) {
        if (!(old > 0.f && old < 3.0e38f)) old = s;  // nothing a call of ours wrote: the codes stay as they are
        s = fmaxf(s, old);
        if (s > old) {
            const float ratio = old / s;
            uint4* c = reinterpret_cast<uint4*>(codes);
            const int words = off * D / 16;
#pragma unroll 4
            for (int i = member * 32 + lane; i < words; i += TEAM * 32) {
                const uint4 u = c[i];
                uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t r = 0;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 f = unpack16<E0_F16>(e4m3x2_to_half2((uint16_t)(w[k] >> (16 * h))));
                        r |= e4m3x2(f.x * ratio, f.y * ratio) << (16 * h);
                    }
                    w[k] = r;
                }
                c[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    if (member == 0 && lane == 0) *scale = s;
    const float inv = 1.f / s;  // a power of two
    uint8_t* to = codes + (size_t)(off + mine) * D + at;
    const auto write = [&](auto finite, uint8_t* p, const AppRaw<TY>& r) {
        float v[N];
        r.get(v);
        uint32_t c[2] = {};
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            float a = v[j] * inv, b = v[j + 1] * inv;
            if (!finite) a = fabsf(v[j]) < INFINITY ? a : 0.f, b = fabsf(v[j + 1]) < INFINITY ? b : 0.f;
            c[j / 4] |= e4m3x2(a, b) << (8 * (j & 2));
        }
        *reinterpret_cast<uint2*>(p) = make_uint2(c[0], c[1]);
    };
    const auto write_all = [&](auto finite) {
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += HOLD * AT_ONCE) {
            if (!once) load(i0);
#pragma unroll
            for (int k = 0; k < HOLD; ++k)
                if (i0 + mine + k * AT_ONCE < n) write(finite, to + (i0 + k * AT_ONCE) * D, held[k]);
        }
    };
    if (plain) write_all(std::true_type{}); else write_all(std::false_type{});
}

// per: tokens that a thread block looks for runs among, at most 32.  SMALL: a warp takes
// all runs among them for its keys or values of a head; else the thread block does.
template <int TY, int D, bool SMALL>
__global__ void __launch_bounds__(APP_WARPS * 32, SMALL || TY == E0_F32 ? 4 : 5)
    k_kv_append(AppendArgs A, bool vec, int per) {
    __shared__ uint32_t most[APP_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = SMALL ? blockIdx.y * APP_WARPS + warp : blockIdx.y, head = part >> 1, which = part & 1;
    if (SMALL && part >= 2 * A.Hkv) return;
    // the tokens that begin a run, the same for every warp
    const long long base = (long long)blockIdx.x * per;
    Slots near;
    const int64_t before0 = base > 0 && base < A.T ? A.slots[base - 1] : -2;
    near.load(A, base, lane);
    int64_t before = __shfl_up_sync(0xffffffffu, near.lo, 1);
    if (lane == 0) before = before0;
    const bool begins = lane < per && near.lo >= 0 && ((near.lo & ((1 << A.shift) - 1)) == 0 || before != near.lo - 1);
    uint32_t left = __ballot_sync(0xffffffffu, begins);
    if constexpr (SMALL) {
        // steps held: blocks of 16 x 128, 13.8 us with 8, 16.2 with 4; of 16 x 64, which
        // are four steps, 8.5 and 7.4; 8 of fp32 are too many registers
        constexpr int HOLD = TY == E0_F32 || D == 64 ? 4 : 8;
        for (; left; left &= left - 1)
            append_run<TY, D, 1, HOLD>(A, vec, which, head, (int)base, __ffs(left) - 1, near, most);
    } else if (__popc(left) > 2) {
        for (int k = 0; left; left &= left - 1, ++k)
            if (k % APP_WARPS == warp)
                append_run<TY, D, 1, 4>(A, vec, which, head, (int)base, __ffs(left) - 1, near, most);
    } else {
        for (; left; left &= left - 1)
            append_run<TY, D, APP_WARPS, 4>(A, vec, which, head, (int)base, __ffs(left) - 1, near, most);
    }
}

template <int TY, int D>
int append_launch(const AppendArgs& a, cudaStream_t s) {
    const int sz = type_size(TY);
    const uintptr_t bits = (uintptr_t)a.x[0] | (uintptr_t)a.x[1] | (uintptr_t)(a.ld[0] * sz) | (uintptr_t)(a.ld[1] * sz);
    // small: a thread block a run and head has too little to do (blocks of 16, 8 heads of 64,
    // 9300 tokens: 29.9 us against 7.4; of 32 x 128: 21.2 against 13.4), but one warp a
    // large run takes too long over it (32 x 256: 16.9 against 12.7).
    // per: about one run of a prompt (of two, one waits for the other; thread blocks that
    // find none are in the others' way: 16 tokens each against 32: blocks of 128, 22.4 us
    // against 18.5; of 32 x 256, 12.8 against 16.2), fewer where that leaves SMs without
    // a thread block, down to as many as there are warps for.
    const int most = a.shift > 5 ? 32 : 16;
    const bool small = D << a.shift <= 4096;
    const int parts = small ? (2 * a.Hkv + APP_WARPS - 1) / APP_WARPS : 2 * a.Hkv;
    int per = most;
    while (per > (small ? 1 : APP_WARPS) && (long long)a.T * parts < 4LL * per * num_sms()) per /= 2;
    const dim3 grid((a.T + per - 1) / per, parts);
    if (small)
        k_kv_append<TY, D, true><<<grid, APP_WARPS * 32, 0, s>>>(a, !(bits & 15), per);
    else
        k_kv_append<TY, D, false><<<grid, APP_WARPS * 32, 0, s>>>(a, !(bits & 15), per);
    return cudaGetLastError() == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

template <int TY>
int append_d(const AppendArgs& a, int D, cudaStream_t s) {
    return D == 64 ? append_launch<TY, 64>(a, s) : D == 128 ? append_launch<TY, 128>(a, s) : append_launch<TY, 256>(a, s);
}

}  // namespace

int kv_plan(const e0_kv_state* k, const int32_t* new_len, int T_cap, int32_t* ctx_out, int32_t* free_out,
            int32_t* cu_q, int64_t* slots, int32_t* positions, int32_t* seq_ids, uint32_t* st, cudaStream_t s) {
    PlanArgs a = plan_args(k, ctx_out, free_out, st);
    a.new_len = new_len, a.T_cap = T_cap, a.cu_q = cu_q, a.slots = slots, a.positions = positions, a.seq_ids = seq_ids;
    return plan_launch(a, s);
}

int kv_release(const e0_kv_state* k, const uint8_t* mask, int32_t* ctx_out, int32_t* free_out, uint32_t* st,
               cudaStream_t s) {
    PlanArgs a = plan_args(k, ctx_out, free_out, st);
    a.mask = mask;
    return release_launch(a, s);
}

int kv_append(const e0_kv_cache* c, const void* k, const void* v, int dtype, int64_t k_ld, int64_t v_ld,
              const int64_t* slots, int T, uint32_t* st, cudaStream_t s) {
    AppendArgs a = {{k, v}, {k_ld, v_ld}, {c->k, c->v}, {c->k_scale, c->v_scale}, slots, st, T, c->Hkv, 0, c->n_blocks};
    while ((1 << a.shift) < c->block_tokens) ++a.shift;
    return dtype == E0_F32   ? append_d<E0_F32>(a, c->D, s)
           : dtype == E0_F16 ? append_d<E0_F16>(a, c->D, s)
                             : append_d<E0_BF16>(a, c->D, s);
}

}  // namespace e0
