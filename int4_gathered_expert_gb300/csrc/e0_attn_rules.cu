// e0_attn_scored and e0_attn_shared: attention under score rules, and over a prefix that a
// batch shares.
#include "e0_attn.cuh"

namespace e0 {
namespace {

// Whether B times max_q queries of D can go through the tensor cores' tiles: enough rows of a KV head to
// fill a part of one (they hold one fp16 operand of Q, and fp32 queries need their rests, too), and a list
// of the tiles that might be that takes 256 MB at most.
bool has_tiles(int dtype, int64_t B, int64_t max_q, int64_t G, int D) {
    const int64_t rows = max_q * G, tile = D == 256 ? 128 : 256;
    return dtype != E0_F32 && rows >= 64 && B * ((rows + tile - 1) / tile) <= 1 << 22;
}

// Whether they do: the tiles' kernels take 17 to 25 us before a first product counts, the one
// for few rows 8 us and then 1 us for every 160 thousand pairs of a row and a position in fp16 with
// heads of 128 (a half of that with heads of 256, one and a half times as many in bf16).  Measured with 8
// heads on 2 (us, few rows / tiles; fp16, heads of 128): 200 queries behind 1000 tokens 14.8 / 29.6, 600
// queries alone 31.2 / 31.7, four times 600 85 / 36, 1500 behind 500 153 / 40.  The host knows what a
// sequence can hold, not what it does: no more than 8192 positions are counted on.  `rows`: of q in all,
// at most (0: any); a decode step of a batch, where any one sequence might have all of them, is not for tiles.
bool by_tiles(const AttnArgs& a, int dtype, int64_t pairs_worth, int64_t rows) {
    const int64_t G = a.Hq / a.Hkv, all = (int64_t)a.B * a.max_q, queries = rows > 0 && rows < all ? rows : all;
    if (!has_tiles(dtype, a.B, a.max_q, G, a.D) || queries * G < 64 * (int64_t)a.B) return false;
    int64_t seen = (int64_t)a.max_blocks << a.shift;
    if (a.window > 0 && !a.at) seen = seen < (int64_t)a.window + a.max_q ? seen : (int64_t)a.window + a.max_q;
    return queries * a.Hq * (seen < 8192 ? seen : 8192) >= pairs_worth;
}

int64_t prompt_pairs(int dtype, int D) {
    const int64_t n = dtype == E0_BF16 ? 4500000 : 3000000;
    return D == 256 ? n * 6 / 10 : n;
}
// (32 sequences behind 8000 tokens, 8 heads of 128 on 2, 2 million pairs: 37.1 / 34.8 us; behind 2000: 26.9 / 31.2.)
constexpr int64_t PREFIX_PAIRS = 1000000;

void put_rules(AttnArgs& a, const e0_attn_rules* r) {
    if (!r) return;
    a.window = r->window, a.slopes = r->slopes, a.first = r->first, a.open = r->open_len;
    if (r->cap > 0.f) {
        // between 2^-120 and 2^120 neither the cap nor its inverse leaves fp32's range; beyond, no score that fp32
        // holds beside others knows the difference
        a.cap = fminf(fmaxf(r->cap, 0x1p-120f), 0x1p120f) * LOG2E;
        a.inv_cap = 1.f / a.cap;
    }
}

// ---------------------------------------------------------------- the shared prefix

// For each row its position behind the prefix, and {0, rows} as the bounds of one sequence
// of them all; under a window then the first position that one of them sees.  `a` is of the sequences' own tokens,
// prefix_blocks of the prefix.
constexpr int ROWS_THREADS = 1024;
__global__ void __launch_bounds__(ROWS_THREADS) k_shared_rows(AttnArgs a, const int32_t* prefix_len, int prefix_blocks, int32_t* at,
                                                              int32_t* cu) {
    __shared__ int rows, least;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) rows = 0, least = INT_MAX;
    for (int t = threadIdx.x; t < a.limit; t += ROWS_THREADS) at[t] = 0;
    __syncthreads();
    const int before = prefix_of(*prefix_len, prefix_blocks, a.shift);
    for (int b = threadIdx.x >> 5; b < a.B; b += ROWS_THREADS / 32) {
        const Seq s = seq_of<true>(a, b, false);
        for (int i = lane; i < s.n; i += 32) at[s.row0 + i] = before + s.ctx - s.n + i;
        if (lane == 0 && s.n > 0) {
            atomicMax(&rows, s.row0 + s.n);
            if (a.window > 0) atomicMin(&least, before + s.ctx - s.n);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        cu[0] = 0, cu[1] = rows;
        if (a.window > 0) cu[2] = low_in(before, max(least - a.window + 1, 0));
    }
}

// out = (e^(l1 - m) o1 + e^(l2 - m) o2) / (e^(l1 - m) + e^(l2 - m)) of two normed results
// and their lse: a warp a row and head.
constexpr int MERGE_WARPS = 8;
template <int TY>
__global__ void __launch_bounds__(MERGE_WARPS * 32) k_shared_merge(AttnArgs a, const float* o1, const float* l1, const float* o2,
                                                                   const float* l2) {
    typedef typename Elem<TY>::T T;
    const int lane = threadIdx.x & 31;
    const Seq s = seq_of<true>(a, blockIdx.x, false);
    for (int item = blockIdx.y * MERGE_WARPS + (threadIdx.x >> 5); item < s.n * a.Hq; item += gridDim.y * MERGE_WARPS) {
        const size_t tok = (size_t)s.row0 + item / a.Hq, at = tok * a.Hq + item % a.Hq;
        const Two two = two_of(l1[at], l2[at]);
        T* to = reinterpret_cast<T*>(a.out) + tok * a.out_ld + (size_t)(item % a.Hq) * a.D;
        for (int d = lane; d < a.D; d += 32)
            to[d] = Elem<TY>::put(fmaf(two.f1, o1[at * a.D + d], two.f2 * o2[at * a.D + d]));
        if (a.lse && lane == 0) a.lse[at] = two.lse;
    }
}

size_t parts_bytes(int T, int Hq, int D) {  // a normed fp32 result and its lse
    return up256((size_t)T * Hq * D * sizeof(float)) + up256((size_t)T * Hq * sizeof(float));
}

}  // namespace

size_t attn_scored_ws_bytes(int B, int Hq, int Hkv, int D, int max_q) {
    const size_t few = attn_ws_bytes(D), many = attn_tile_ws_bytes(B, max_q, Hq / Hkv, D);
    return has_tiles(E0_F16, B, max_q, Hq / Hkv, D) && many > few ? many : few;
}

int attn_scored(const e0_kv_cache* c, const int32_t* table, int max_blocks, const int32_t* ctx, const int32_t* cu, int B,
                int max_q, const void* q, int dtype, int64_t q_ld, int Hq, float scale, const e0_attn_rules* rules,
                void* out, int64_t out_ld, float* lse, void* ws, uint32_t* st, cudaStream_t s) {
    AttnArgs a = args_of(c, table, max_blocks, ctx, cu, B, max_q, q, q_ld, Hq, scale, 0, out, out_ld, lse, ws, st);
    put_rules(a, rules);
    if (by_tiles(a, dtype, prompt_pairs(dtype, c->D), rules ? rules->rows : 0)) return attn_tile(a, nullptr, dtype, ws, s);
    return launch_t<true>(a, dtype, c->D, s);
}

size_t attn_shared_ws_bytes(int B, int T, int Hq, int Hkv, int D, int max_q) {
    // the tiles' schedule is made while the sequences' own attention runs: a place for each
    const size_t tiles = has_tiles(E0_F16, 1, T, Hq / Hkv, D) ? attn_tile_ws_bytes(1, T, Hq / Hkv, D) : 0;
    return up256((size_t)T * sizeof(int32_t)) + 256 + 2 * parts_bytes(T, Hq, D) + up256(attn_ws_bytes(D)) + tiles;
}

int attn_shared(const e0_kv_cache* c, const int32_t* prefix_table, int prefix_blocks, const int32_t* prefix_len,
                const int32_t* table, int max_blocks, const int32_t* ctx, const int32_t* cu, int B, int T, int max_q,
                const void* q, int dtype, int64_t q_ld, int Hq, float scale, const e0_attn_rules* rules, void* out,
                int64_t out_ld, float* lse, void* ws, uint32_t* st, cudaStream_t s) {
    char* p = reinterpret_cast<char*>(ws);
    const auto take = [&](size_t n) {
        char* at = p;
        p += up256(n);
        return at;
    };
    int32_t* at = reinterpret_cast<int32_t*>(take((size_t)T * sizeof(int32_t)));
    int32_t* cu2 = reinterpret_cast<int32_t*>(take(3 * sizeof(int32_t)));
    float* o[2];
    float* l[2];
    for (int i = 0; i < 2; ++i) {
        o[i] = reinterpret_cast<float*>(take((size_t)T * Hq * c->D * sizeof(float)));
        l[i] = reinterpret_cast<float*>(take((size_t)T * Hq * sizeof(float)));
    }
    char* tiles = p + up256(attn_ws_bytes(c->D));
    AttnArgs mine = args_of(c, table, max_blocks, ctx, cu, B, max_q, q, q_ld, Hq, scale, 0, out, out_ld, l[1], p, st);
    put_rules(mine, rules);
    mine.raw = o[1], mine.limit = T;
    mine.unit = 64;  // any: the kernels set their own
    // the prefix, as one sequence whose queries are all rows
    AttnArgs front = args_of(c, prefix_table, prefix_blocks, prefix_len, cu2, 1, T, q, q_ld, Hq, scale, 0, out, out_ld, l[0], p, st);
    put_rules(front, rules);
    front.limit = T, front.at = at, front.at_low = front.window > 0 ? cu2 + 2 : nullptr;
    // what the sequences have of their own comes first: the prefix' last kernel adds it where it can
    int rc = launch_t<true>(mine, dtype, c->D, s);
    if (rc != E0_OK) return rc;
    if (by_tiles(front, dtype, PREFIX_PAIRS, 0)) {
        const TilePrefix prefix = {mine, at, o[1], l[1], attn_tile_merges(front)};
        if (prefix.merge) {
            front.lse = lse;
            return attn_tile(front, &prefix, dtype, tiles, s);
        }
        front.raw = o[0];
        rc = attn_tile(front, &prefix, dtype, tiles, s);
    } else {
        k_shared_rows<<<1, ROWS_THREADS, 0, s>>>(mine, prefix_len, prefix_blocks, at, cu2);
        if (cudaGetLastError() != cudaSuccess) return E0_ERR_CUDA;
        front.raw = o[0];
        rc = launch_t<true>(front, dtype, c->D, s);
    }
    if (rc != E0_OK) return rc;
    mine.lse = lse;
    const long long items = (long long)max_q * Hq;
    const dim3 grid(B, (unsigned)((items + MERGE_WARPS - 1) / MERGE_WARPS < 64 ? (items + MERGE_WARPS - 1) / MERGE_WARPS : 64));
    switch (dtype) {
        case E0_F32: k_shared_merge<E0_F32><<<grid, MERGE_WARPS * 32, 0, s>>>(mine, o[0], l[0], o[1], l[1]); break;
        case E0_F16: k_shared_merge<E0_F16><<<grid, MERGE_WARPS * 32, 0, s>>>(mine, o[0], l[0], o[1], l[1]); break;
        default: k_shared_merge<E0_BF16><<<grid, MERGE_WARPS * 32, 0, s>>>(mine, o[0], l[0], o[1], l[1]); break;
    }
    return cudaGetLastError() == cudaSuccess ? E0_OK : E0_ERR_CUDA;
}

}  // namespace e0
