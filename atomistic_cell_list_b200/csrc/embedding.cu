// Species embedding: out[n,0,:] = scale table[token_n,:] (higher degrees zero),
// and its gradient, grad_table[v,:] = scale sum_{n: token_n = v} grad_out[n,0,:].
//
// The gradient sums runs of equal tokens in sorted order. A block takes a tile of
// T tokens; teams of lanes sum equal parts of the tile, run by run; the runs that
// cross parts are added in the block, those that cross tiles by a second kernel.
//   Tables of up to 256 rows (species): each tile is sorted by itself, in shared
//   memory. A block writes a sum for each of its distinct tokens, and two launches
//   do it all (one for a single tile).
//   100,000 tokens of two species, C = 128: 51 MB in 20 us, 63 us with a global sort and
//   a join of 64-token chunks; latency bounds it (the sort of a tile, its rows 8 at a time).
//   Larger tables: a stable radix sort of all tokens first, 8 bits a pass. 65,536
//   tokens of 32,003, C = 512: 200 MB in 70 us, half of it the sort's six kernels.
// Every sum has one fixed order and no atomics, so results repeat bit for bit.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "feature_io.cuh"
#include "launch.cuh"

namespace e2f {
namespace {

constexpr int kMaxEmbedC = 16384;
constexpr int kSortTile = 1024;  // tokens of a sorting block (256 threads, 4 each)
constexpr int kLocalTokens = 256;  // largest table whose tiles are sorted one by one
constexpr int kMaxTile = 2048;
constexpr int64_t kMostTiles = 296;  // two an SM, as long as tiles can grow
constexpr int64_t kMostBlocks = 4 * kMostTiles;  // of all columns, in small tables
constexpr int64_t kPartBytes = 16 << 20;

struct EmbedWs {
    size_t o_status, o_hist, o_tot, o_key[2], o_idx[2], o_part, bytes;
    int64_t sort_tiles, tiles;
    int tile, passes, V, TL;
};

EmbedWs embed_layout(int64_t n, const e2f_embed_cfg& c) {
    EmbedWs w{};
    size_t o = 0;
    auto take = [&](size_t b) { size_t r = o; o = align_up(o + b, 256); return r; };
    w.V = c.C % 4 == 0 ? 4 : 1;
    w.TL = 1;
    while (w.TL < 32 && w.TL * w.V < c.C) w.TL *= 2;
    // up to two tiles per SM, 8 tokens a team at least; what one block sorts fast goes to one block
    const bool local = c.n_tokens <= kLocalTokens;
    w.tile = std::max(64, 8 * (256 / w.TL));
    // Small tables: every tile writes sums for n_tokens rows of C values. Many blocks of columns leave room for fewer
    // tiles: kMostBlocks blocks in all. Where the tiles' sums take more than kPartBytes, a tile has at least n_tokens
    // tokens, so that the sums are no more than what they are made of. 19,000 tokens of 256 rows, C = 8,192: 251 us
    // in 151 MB, 454 us in 1.2 GB without either; 18,900 of 256, C = 128: 13 and 17 us. Sums of fewer bytes come
    // faster from small tiles: 6,000 tokens of 256 rows, C = 128, 12 MB: 9 us, in tiles of 256 tokens 12 us.
    int64_t most = kMostTiles, cheap = INT64_MAX;
    if (local) {
        most = std::max<int64_t>(1, std::min(most, kMostBlocks * w.TL * w.V / c.C));
        cheap = kPartBytes / (4ll * c.n_tokens * c.C);
    }
    int no_less = w.tile;  // the tile that holds n_tokens tokens
    while (local && no_less < c.n_tokens) no_less *= 2;
    // Where a tile grows there are fewer of them. The workspace has room for the most that n or fewer tokens have,
    // so that one made for the largest batch serves every smaller one.
    const auto tiles_of = [n](int tile) { return (n + tile - 1) / tile; };
    const int64_t room = local && n <= 512 ? 1 : std::max(tiles_of(kMaxTile),
        std::min({tiles_of(w.tile), most, std::max(cheap, tiles_of(no_less))}));
    while (w.tile < kMaxTile && (tiles_of(w.tile) > most || (w.tile < no_less && tiles_of(w.tile) > cheap))) w.tile *= 2;
    if (local && n <= 512) w.tile = std::max(w.tile, 512);
    w.tiles = tiles_of(w.tile);
    w.o_status = take(256);  // first: e2f_attention_status reads it
    if (local) {
        w.o_hist = take((size_t)room * (c.n_tokens + 1));  // which tokens a tile has, whether one is beyond the table
        w.o_part = take(room > 1 ? 4 * (size_t)room * c.n_tokens * c.C : 0);
    } else {
        w.passes = 1;
        while (w.passes < 4 && ((int64_t)c.n_tokens >> (8 * w.passes))) ++w.passes;
        w.sort_tiles = (n + kSortTile - 1) / kSortTile;
        w.o_hist = take(4 * 256 * (size_t)w.sort_tiles);
        w.o_tot = take(4 * 256);
        for (int k = 0; k < 2; ++k) {
            w.o_key[k] = take(4 * (size_t)n);
            w.o_idx[k] = take(4 * (size_t)n);
        }
        w.o_part = take(8 * (size_t)room * c.C);
    }
    w.bytes = o;
    return w;
}

// V = 1, 4 or 8 values from an index that is a multiple of V
template <int T, int V>
__device__ __forceinline__ void load_row(const void* p, int64_t i, float (&v)[V]) {
    if constexpr (V == 8) load8<T>(p, i / 8, v);
    else load_vec<T, V>(p, i, v);
}
template <int T, int V>
__device__ __forceinline__ void store_row(void* p, int64_t i, const float (&v)[V]) {
    if constexpr (V == 8) store8<T>(p, i / 8, v);
    else store_vec<T, V>(p, i, v);
}

// 16 bytes of values: 8 of bf16, 4 of fp32
template <int T>
constexpr int kWide = T == kBF16 ? 8 : 4;

// One group of `lanes` lanes (a power of two) per node: its first C values from
// the table, zeros behind them. V values a store; the write of the output bounds it:
// 100,000 atoms, L = 4, C = 128 in bf16, 640 MB in 94 us (6.8 TB/s; with a division
// per 8 bytes it was 222 us); C = 132, which no 16 bytes divide, value by value: 660 MB in 123 us.
template <int TT, int YT, int V>
__global__ void __launch_bounds__(256) k_embed(const int32_t* tok, int64_t n, const void* table, int n_tokens, int K,
                                               int C, float scale, int lanes, void* out, int* status) {
    const int t = threadIdx.x & (lanes - 1), head = C / V, all = K * head;
    const int64_t step = (int64_t)gridDim.x * (256 / lanes);
    for (int64_t node = (int64_t)blockIdx.x * (256 / lanes) + threadIdx.x / lanes; node < n; node += step) {
        const int token = tok[node];
        const bool ok = token >= 0 && token < n_tokens;
        if (token >= n_tokens && status && t == 0) *status = E2F_ERR_INVALID_ARG;
        const int64_t row = (int64_t)token * C, base = node * all;
        for (int j = t; j < head; j += lanes) {
            float v[V] = {};
            if (ok) {
                load_row<TT, V>(table, row + j * V, v);
                for (int k = 0; k < V; ++k) v[k] *= scale;
            }
            store_row<YT, V>(out, (base + j) * V, v);
        }
        const float zero[V] = {};
#pragma unroll 4
        for (int j = head + t; j < all; j += lanes) store_row<YT, V>(out, (base + j) * V, zero);
    }
}

// sort key of a token: padding and tokens outside the table go behind the last token
__device__ __forceinline__ uint32_t sort_key(int t, int n_tokens) {
    return t < 0 || t >= n_tokens ? (uint32_t)n_tokens : (uint32_t)t;
}

// What the kernels of the sort do beside it: zeros for the whole table, a share
// in each kernel, by blocks behind those that sort. The sort is bound by latency,
// the zeros by the memory.
struct Zeros {
    float* to;
    int64_t from, n;  // values; from is a multiple of 4
};
constexpr int kZeroBlocks = 148;
// true in the blocks behind the first `blocks`, which write their part of the zeros
__device__ __forceinline__ bool zero_blocks(const Zeros& z, int64_t blocks) {
    if ((int64_t)blockIdx.x < blocks) return false;
    after_previous();
    const int64_t t = (blockIdx.x - blocks) * 256 + threadIdx.x;
    float4* to = reinterpret_cast<float4*>(z.to + z.from);
    for (int64_t i = t; i < z.n / 4; i += kZeroBlocks * 256) to[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < z.n % 4) z.to[z.from + z.n / 4 * 4 + t] = 0.f;
    return true;
}

// digit counts of one tile: hist[digit][tile]
template <bool FIRST>
__global__ void __launch_bounds__(256) k_sort_count(const void* keys, int64_t n, int n_tokens, int shift,
                                                    int64_t tiles, uint32_t* hist, int* status, Zeros z) {
    if (zero_blocks(z, tiles)) return;
    __shared__ uint32_t cnt[256];
    after_previous();
    if (FIRST && blockIdx.x == 0 && threadIdx.x == 0) *status = E2F_OK;  // k_sort_place reports
    cnt[threadIdx.x] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kSortTile;
    for (int j = 0; j < kSortTile / 256; ++j) {
        const int64_t p = base + j * 256 + threadIdx.x;
        if (p >= n) break;
        uint32_t k;
        if constexpr (FIRST) {
            k = sort_key(static_cast<const int*>(keys)[p], n_tokens);
        } else {
            k = static_cast<const uint32_t*>(keys)[p];
        }
        atomicAdd(&cnt[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    hist[threadIdx.x * tiles + blockIdx.x] = cnt[threadIdx.x];
}

// block d: exclusive prefix over the tiles of digit d, in place; its total
__global__ void __launch_bounds__(256) k_sort_scan(uint32_t* hist, int64_t tiles, uint32_t* total, Zeros z) {
    if (zero_blocks(z, 256)) return;
    after_previous();
    __shared__ uint32_t ws[8];
    uint32_t* h = hist + blockIdx.x * tiles;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint32_t carry = 0;
    for (int64_t b = 0; b < tiles; b += 256) {
        const int64_t i = b + threadIdx.x;
        const uint32_t v = i < tiles ? h[i] : 0u;
        uint32_t inc = v;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) ws[w] = inc;
        __syncthreads();
        uint32_t before = 0, all = 0;
        for (int k = 0; k < 8; ++k) {
            if (k < w) before += ws[k];
            all += ws[k];
        }
        if (i < tiles) h[i] = carry + before + inc - v;
        carry += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) total[blockIdx.x] = carry;
}

// places one tile's (key, index) pairs, equal digits in their order
template <bool FIRST>
__global__ void __launch_bounds__(256) k_sort_place(const void* keys, const int* idx, int64_t n, int n_tokens,
                                                    int shift, int64_t tiles, const uint32_t* hist,
                                                    const uint32_t* total, uint32_t* keys_out, int* idx_out,
                                                    int* status, Zeros z) {
    if (zero_blocks(z, tiles)) return;
    constexpr int J = kSortTile / 256;
    __shared__ uint32_t wc[8][256];
    __shared__ uint32_t ws[8];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int k = 0; k < 8; ++k) wc[k][threadIdx.x] = 0;
    __syncthreads();
    after_previous();
    const int64_t base = (int64_t)blockIdx.x * kSortTile + w * (32 * J);
    uint32_t key[J], rank[J];
    for (int j = 0; j < J; ++j) {
        const int64_t p = base + j * 32 + lane;
        const bool ok = p < n;
        key[j] = 0;
        if (ok) {
            if constexpr (FIRST) {
                const int t = static_cast<const int*>(keys)[p];
                if (t >= n_tokens) *status = E2F_ERR_INVALID_ARG;
                key[j] = sort_key(t, n_tokens);
            } else key[j] = static_cast<const uint32_t*>(keys)[p];
        }
        const uint32_t d = ok ? (key[j] >> shift) & 255u : 256u;
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        const uint32_t below = __popc(same & ((1u << lane) - 1u));
        rank[j] = ok ? wc[w][d] + below : 0u;
        __syncwarp();
        if (ok && below == 0) wc[w][d] += __popc(same);
        __syncwarp();
    }
    // digit d's place in the output: totals of the smaller digits + this digit's earlier tiles + earlier warps
    const uint32_t v = total[threadIdx.x];
    uint32_t inc = v;
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    if (lane == 31) ws[w] = inc;
    __syncthreads();
    uint32_t at = inc - v + hist[threadIdx.x * tiles + blockIdx.x];
    for (int k = 0; k < w; ++k) at += ws[k];
    for (int k = 0; k < 8; ++k) {
        const uint32_t c = wc[k][threadIdx.x];
        wc[k][threadIdx.x] = at;
        at += c;
    }
    __syncthreads();
    for (int j = 0; j < J; ++j) {
        const int64_t p = base + j * 32 + lane;
        if (p >= n) break;
        const uint32_t to = wc[w][(key[j] >> shift) & 255u] + rank[j];
        keys_out[to] = key[j];
        idx_out[to] = FIRST ? (int)p : idx[p];
    }
}

// Sorts the tile's tokens in shared memory, equal ones in their order; cnt holds
// how often each occurs. 256 threads; a warp takes a contiguous part of the tile.
// Returns, in every thread, whether a token lies beyond the table.
__device__ __forceinline__ bool sort_tile(const int32_t* tok, int64_t base, int n, int tile, int n_tokens,
                                          uint32_t* keys, int* idx, uint32_t (*wc)[257], uint32_t* cnt) {
    bool beyond = false;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, part = tile / 8;
    for (int k = threadIdx.x; k < 8 * 257; k += 256) wc[0][k] = 0;
    __syncthreads();
    // two sweeps over the warp's part: counts, then places (the second repeats the ranks)
    for (int sweep = 0; sweep < 2; ++sweep) {
        for (int j = 0; j < part; j += 32) {
            const int p = w * part + j + lane;
            const bool ok = j + lane < part && p < n;
            uint32_t key = 0;
            if (ok) {
                const int t = tok[base + p];
                beyond |= t >= n_tokens;
                key = sort_key(t, n_tokens);
            }
            const uint32_t same = __match_any_sync(0xffffffffu, ok ? key : 0xffffffffu);
            const uint32_t below = __popc(same & ((1u << lane) - 1u));
            const uint32_t at = ok ? wc[w][key] + below : 0u;
            __syncwarp();
            if (ok && below == 0) wc[w][key] += __popc(same);
            __syncwarp();
            if (sweep == 1 && ok) {
                keys[at] = key;
                idx[at] = (int)(base + p);
            }
        }
        __syncthreads();
        if (sweep == 0) {
            // token k's places: smaller tokens, then the warps before (thread k; key 256 by thread 255)
            __shared__ uint32_t ws[8];
            uint32_t all = 0;
            for (int q = 0; q < 8; ++q) all += wc[q][threadIdx.x];
            cnt[threadIdx.x] = all;
            uint32_t inc = all;
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 31) ws[w] = inc;
            __syncthreads();
            uint32_t at = inc - all;
            for (int q = 0; q < w; ++q) at += ws[q];
            for (int q = 0; q < 8; ++q) {
                const uint32_t c = wc[q][threadIdx.x];
                wc[q][threadIdx.x] = at;
                at += c;
            }
            __syncthreads();
            if (threadIdx.x == 255)  // key 256: padding of a table of 256 rows
                for (int q = 0; q < 8; ++q) {
                    const uint32_t c = wc[q][256];
                    wc[q][256] = at;
                    at += c;
                }
            __syncthreads();
        }
    }
    return __syncthreads_or(beyond);
}

struct RunArgs {
    const float* g;
    int64_t row_stride, n;
    int C, n_tokens, tile, TL;
    float scale;
    float* grad;
    float* part;
    // tables of up to 256 rows
    const int32_t* tok;
    uint8_t* has;
    int* status;
    // larger tables: all tokens sorted
    const uint32_t* keys;
    const int* idx;
};

// One tile, TL V columns. LOCAL: sorts the tile and writes its sums by token to
// part[tile][token] (to the table itself when there is one tile). Otherwise runs
// inside the tile are final; one that begins here and goes on is the tile's open
// sum (part[2 tile + 1]), one that came in from the tile before its carry
// (part[2 tile]).
template <int V, bool LOCAL>
__global__ void __launch_bounds__(256) k_run_sum(RunArgs a) {
    extern __shared__ uint32_t sm[];  // [tile] keys, [tile] indexes, then LOCAL: [8][257] counts, [256] totals
    __shared__ __align__(16) float ent[256 * 2 * V];  // [team][first, last run][TL V]
    __shared__ uint32_t ent_key[256][2];
    uint32_t* keys = sm;
    int* idx = reinterpret_cast<int*>(sm + a.tile);
    const int64_t base = (int64_t)blockIdx.x * a.tile;
    const int n = (int)min((int64_t)a.tile, a.n - base);
    const uint32_t none = 0xffffffffu, n_tokens = (uint32_t)a.n_tokens;
    if constexpr (LOCAL) {
        uint32_t (*wc)[257] = reinterpret_cast<uint32_t (*)[257]>(sm + 2 * a.tile);
        uint32_t* cnt = sm + 2 * a.tile + 8 * 257;
        const bool beyond = sort_tile(a.tok, base, n, a.tile, a.n_tokens, keys, idx, wc, cnt);
        const int k = threadIdx.x;
        if (gridDim.x > 1) {
            uint8_t* has = a.has + (int64_t)blockIdx.x * (a.n_tokens + 1);  // by token, then `beyond`
            if (k < a.n_tokens) has[k] = cnt[k] != 0;
            if (k == 0) has[a.n_tokens] = beyond;
        } else if (k == 0) {
            *a.status = beyond ? E2F_ERR_INVALID_ARG : E2F_OK;
        }
    } else {
        after_previous();
        for (int p = threadIdx.x; p < n; p += 256) {
            keys[p] = a.keys[base + p];
            idx[p] = a.idx[base + p];
        }
        __syncthreads();
    }
    const int team = threadIdx.x / a.TL, teams = 256 / a.TL, t = threadIdx.x % a.TL;
    const int c = (blockIdx.y * a.TL + t) * V, per = a.tile / teams;
    const bool in = c < a.C;
    const int p0 = min(team * per, n), p1 = min(p0 + per, n);
    float* row_out = LOCAL ? (gridDim.x > 1 ? a.part + (int64_t)blockIdx.x * a.n_tokens * a.C : a.grad) : a.grad;
    const float f = LOCAL && gridDim.x > 1 ? 1.f : a.scale;
    auto final_row = [&](uint32_t key, const float (&v)[V]) {
        if (key >= n_tokens || !in) return;
        float o[V];
        for (int k = 0; k < V; ++k) o[k] = v[k] * f;
        store_vec<kF32, V>(row_out, (int64_t)key * a.C + c, o);
    };
    // this team's part
    {
        uint32_t cur = p0 < p1 ? keys[p0] : none;
        bool first = true;
        float acc[V] = {};
        constexpr int U = 8;
        for (int p = p0; p < p1; p += U) {
            uint32_t key[U];
            float v[U][V];
            // every load is made, so that all are in flight: what lies behind the part reads the batch's first row,
            // lanes beyond the columns the first column, padding its own row, and none of it counts
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int at = p + j < p1 ? p + j : p;
                key[j] = keys[at];
                load_vec<kF32, V>(a.g, idx[at] * a.row_stride + (in ? c : 0), v[j]);
            }
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (key[j] >= n_tokens)
                    for (int k = 0; k < V; ++k) v[j][k] = 0.f;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (p + j >= p1) break;
                if (key[j] != cur) {
                    if (first) {
                        for (int k = 0; k < V; ++k) ent[(team * 2 * a.TL + t) * V + k] = acc[k];
                        if (t == 0) ent_key[team][0] = cur;
                        first = false;
                    } else {
                        final_row(cur, acc);
                    }
                    cur = key[j];
                    for (int k = 0; k < V; ++k) acc[k] = 0.f;
                }
                for (int k = 0; k < V; ++k) acc[k] += v[j][k];
            }
        }
        const int e = first ? 0 : 1;
        for (int k = 0; k < V; ++k) ent[((team * 2 + e) * a.TL + t) * V + k] = acc[k];
        if (t == 0) {
            ent_key[team][e] = cur;
            if (e == 0) ent_key[team][1] = none;
        }
    }
    __syncthreads();
    // the tile's first and last runs of all parts, in order
    if (team == 0) {
        bool begins = LOCAL || base == 0 || a.keys[base - 1] != keys[0];
        uint32_t cur = keys[0];
        float acc[V] = {};
        auto flush = [&](bool ends) {
            if (begins && ends) return final_row(cur, acc);
            if (cur < n_tokens && in)
                store_vec<kF32, V>(a.part, (2 * (int64_t)blockIdx.x + (begins ? 1 : 0)) * a.C + c, acc);
        };
        for (int q = 0; q < 2 * ((n + per - 1) / per); ++q) {  // the teams that had tokens
            const uint32_t key = ent_key[q >> 1][q & 1];
            if (key == none) continue;
            if (key != cur) {
                flush(true);
                begins = true;
                cur = key;
                for (int k = 0; k < V; ++k) acc[k] = 0.f;
            }
            for (int k = 0; k < V; ++k) acc[k] += ent[(q * a.TL + t) * V + k];
        }
        flush(LOCAL || base + n == a.n || a.keys[base + n] != cur);
    }
    if constexpr (LOCAL)
        if (gridDim.x == 1) {  // rows of tokens that do not occur
            const uint32_t* cnt = sm + 2 * a.tile + 8 * 257;
            const float zero[V] = {};
            for (int k = team; k < a.n_tokens; k += teams)
                if (cnt[k] == 0 && in) store_vec<kF32, V>(a.grad, (int64_t)k * a.C + c, zero);
        }
}

constexpr int kJoinWarps = 16;

// sum of the block's warps, in order, by its first warp; true there
template <int V>
__device__ __forceinline__ bool join_warps(float (&v)[V]) {
    __shared__ float sh[kJoinWarps][32][V];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int k = 0; k < V; ++k) sh[w][lane][k] = v[k];
    __syncthreads();
    if (w) return false;
    for (int q = 1; q < kJoinWarps; ++q)
        for (int k = 0; k < V; ++k) v[k] += sh[q][lane][k];
    return true;
}

// Block (token, 32 V columns): adds the tiles' sums of the token.
template <int V>
__global__ void __launch_bounds__(32 * kJoinWarps) k_token_join(RunArgs a, int64_t tiles) {
    const int key = blockIdx.x, c = (blockIdx.y * 32 + (threadIdx.x & 31)) * V;
    float acc[V] = {};
    after_previous();
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        bool beyond = false;
        for (int64_t b = threadIdx.x; b < tiles; b += blockDim.x) beyond |= a.has[b * (a.n_tokens + 1) + a.n_tokens];
        beyond = __syncthreads_or(beyond);
        if (threadIdx.x == 0) *a.status = beyond ? E2F_ERR_INVALID_ARG : E2F_OK;
    }
    constexpr int U = 8;  // tiles whose sums are loaded together; those without the token are loaded and not used
    for (int64_t b0 = threadIdx.x >> 5; b0 < tiles; b0 += U * kJoinWarps) {
        bool has[U];
        bool any = false;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t b = b0 + j * kJoinWarps;
            has[j] = a.has[min(b, tiles - 1) * (a.n_tokens + 1) + key] && b < tiles;
            any |= has[j];
        }
        if (!any || c >= a.C) continue;
        float v[U][V];
#pragma unroll
        for (int j = 0; j < U; ++j)
            load_vec<kF32, V>(a.part, (min(b0 + j * kJoinWarps, tiles - 1) * a.n_tokens + key) * a.C + c, v[j]);
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (has[j])
                for (int k = 0; k < V; ++k) acc[k] += v[j][k];
    }
    if (!join_warps<V>(acc) || c >= a.C) return;
    for (int k = 0; k < V; ++k) acc[k] *= a.scale;
    store_vec<kF32, V>(a.grad, (int64_t)key * a.C + c, acc);
}

// Block (tile, 32 V columns): if a run opened in the tile, adds the carries of the tiles it reaches.
template <int V>
__global__ void __launch_bounds__(32 * kJoinWarps) k_run_join(RunArgs a, int64_t tiles) {
    const int64_t s = blockIdx.x, p0 = s * a.tile, p1 = p0 + a.tile;
    after_previous();
    if (p1 >= a.n) return;
    const uint32_t key = a.keys[p1 - 1];
    if (key >= (uint32_t)a.n_tokens || a.keys[p1] != key) return;        // nothing goes on
    if (p0 > 0 && a.keys[p0] == key && a.keys[p0 - 1] == key) return;  // it did not begin here
    const int w = threadIdx.x >> 5, c = (blockIdx.y * 32 + (threadIdx.x & 31)) * V;
    float acc[V] = {}, v[V];
    if (c < a.C) {
        if (w == 0) load_vec<kF32, V>(a.part, (2 * s + 1) * a.C + c, acc);
#pragma unroll 4
        for (int64_t j = s + 1 + w; j < tiles && a.keys[j * a.tile] == key; j += kJoinWarps) {
            load_vec<kF32, V>(a.part, 2 * j * a.C + c, v);
            for (int k = 0; k < V; ++k) acc[k] += v[k];
        }
    }
    if (!join_warps<V>(acc) || c >= a.C) return;
    for (int k = 0; k < V; ++k) acc[k] *= a.scale;
    store_vec<kF32, V>(a.grad, (int64_t)key * a.C + c, acc);
}

template <int TT, int YT>
cudaError_t launch_embed(const e2f_embed_cfg& f, const int32_t* tok, int64_t n, const void* table, void* out,
                         int* status, cudaStream_t s) {
    const int K = (f.L + 1) * (f.L + 1);
    const bool wide = f.C % kWide<YT> == 0;
    const int V = wide ? kWide<YT> : 1;
    int lanes = 1;  // a warp a node at most, no lanes without a value
    while (lanes < 32 && lanes * V < K * f.C) lanes *= 2;
    const unsigned grid = (unsigned)std::min<int64_t>((n + 256 / lanes - 1) / (256 / lanes), 148 * 32);
    count_launch();
    if (wide)
        k_embed<TT, YT, kWide<YT>><<<grid, 256, 0, s>>>(tok, n, table, f.n_tokens, K, f.C, f.scale, lanes, out, status);
    else
        k_embed<TT, YT, 1><<<grid, 256, 0, s>>>(tok, n, table, f.n_tokens, K, f.C, f.scale, lanes, out, status);
    return cudaGetLastError();
}

template <int V>
cudaError_t run_embed_bwd(const e2f_embed_cfg& f, const int32_t* tok, int64_t n, const float* g, float* grad, char* ws,
                          const EmbedWs& w, cudaStream_t s) {
    const int K = (f.L + 1) * (f.L + 1);
    int* status = reinterpret_cast<int*>(ws + w.o_status);
    RunArgs a{g, (int64_t)K * f.C, n, f.C, f.n_tokens, w.tile, w.TL, f.scale, grad,
              reinterpret_cast<float*>(ws + w.o_part)};
    const dim3 grid((unsigned)w.tiles, (unsigned)((f.C + w.TL * V - 1) / (w.TL * V)));
    if (f.n_tokens <= kLocalTokens) {
        a.tok = tok;
        a.has = reinterpret_cast<uint8_t*>(ws + w.o_hist);
        a.status = status;
        k_run_sum<V, true><<<grid, 256, 4 * (2 * w.tile + 8 * 257 + 256), s>>>(a);
        count_launch();
        if (w.tiles > 1) {
            cudaError_t e = launch_after(k_token_join<V>, dim3(f.n_tokens, (f.C + 32 * V - 1) / (32 * V)), 32 * kJoinWarps,
                                         0, s, a, w.tiles);
            if (e != cudaSuccess) return e;
        }
        return cudaGetLastError();
    }
    uint32_t* hist = reinterpret_cast<uint32_t*>(ws + w.o_hist);
    uint32_t* total = reinterpret_cast<uint32_t*>(ws + w.o_tot);
    uint32_t* key[2];
    int* idx[2];
    for (int k = 0; k < 2; ++k) {
        key[k] = reinterpret_cast<uint32_t*>(ws + w.o_key[k]);
        idx[k] = reinterpret_cast<int*>(ws + w.o_idx[k]);
    }
    const unsigned tiles = (unsigned)w.sort_tiles;
    // equal shares for the sort's kernels, in whole 4,096s, both divisions rounded up: together no less than `values`
    const int64_t values = (int64_t)f.n_tokens * f.C, kernels = 3 * w.passes;
    const int64_t share = ((values + kernels - 1) / kernels + 4095) / 4096 * 4096;
    int64_t zeroed = 0;
    auto zeros = [&]() {  // the next share; the last ones may be shorter or empty
        const Zeros z{grad, zeroed, std::min(share, values - zeroed)};
        zeroed += z.n;
        return z;
    };
    cudaError_t e = cudaSuccess;
    auto next = [&](auto kernel, unsigned blocks, auto... args) {
        if (e == cudaSuccess) e = launch_after(kernel, dim3(blocks + kZeroBlocks), 256, 0, s, args..., zeros());
    };
    for (int p = 0; p < w.passes; ++p) {
        const int to = p & 1, from = to ^ 1;
        if (p == 0) {
            k_sort_count<true><<<tiles + kZeroBlocks, 256, 0, s>>>(tok, n, f.n_tokens, 0, w.sort_tiles, hist, status,
                                                                   zeros());
            count_launch();
            next(k_sort_scan, 256, hist, w.sort_tiles, total);
            next(k_sort_place<true>, tiles, tok, nullptr, n, f.n_tokens, 0, w.sort_tiles, hist, total, key[to], idx[to],
                 status);
        } else {
            next(k_sort_count<false>, tiles, key[from], n, f.n_tokens, 8 * p, w.sort_tiles, hist, nullptr);
            next(k_sort_scan, 256, hist, w.sort_tiles, total);
            next(k_sort_place<false>, tiles, key[from], idx[from], n, f.n_tokens, 8 * p, w.sort_tiles, hist, total,
                 key[to], idx[to], nullptr);
        }
    }
    a.keys = key[(w.passes - 1) & 1];
    a.idx = idx[(w.passes - 1) & 1];
    if (e == cudaSuccess) e = launch_after(k_run_sum<V, false>, grid, 256, 8 * w.tile, s, a);
    if (e == cudaSuccess && w.tiles > 1)
        e = launch_after(k_run_join<V>, dim3((unsigned)w.tiles, (f.C + 32 * V - 1) / (32 * V)), 32 * kJoinWarps, 0, s, a,
                         w.tiles);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

e2f_status check_embed_cfg(const e2f_embed_cfg* c) {
    if (!c) return E2F_ERR_INVALID_ARG;
    if (c->L < 0 || c->C <= 0 || c->n_tokens <= 0 || !std::isfinite(c->scale)) return E2F_ERR_INVALID_ARG;
    if (c->table_dtype != E2F_F32 && c->table_dtype != E2F_BF16) return E2F_ERR_UNSUPPORTED;
    if (c->out_dtype != E2F_F32 && c->out_dtype != E2F_BF16) return E2F_ERR_UNSUPPORTED;
    if (c->L > kMaxL || c->C > kMaxEmbedC) return E2F_ERR_UNSUPPORTED;
    return E2F_OK;
}

}  // namespace
}  // namespace e2f

using namespace e2f;

extern "C" e2f_status e2f_embedding(const e2f_embed_cfg* cfg, const int32_t* tokens, int64_t n_atoms,
                                    const void* table, void* out, void* workspace, size_t ws_bytes, void* stream) {
    e2f_status st = check_embed_cfg(cfg);
    if (st != E2F_OK) return st;
    if (n_atoms < 0 || n_atoms > INT32_MAX) return E2F_ERR_INVALID_ARG;
    if (workspace && ws_bytes < 256) return E2F_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) % 256) return E2F_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n_atoms > 0 && (!tokens || !table || !out)) return E2F_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(table) % 16 || reinterpret_cast<uintptr_t>(out) % 16) return E2F_ERR_ALIGNMENT;
    int* status = static_cast<int*>(workspace);
    if (status) E2F_CUDA_TRY(cudaMemsetAsync(status, 0, sizeof(int), s));
    if (n_atoms == 0) return E2F_OK;
    const bool tb = cfg->table_dtype == E2F_BF16, yb = cfg->out_dtype == E2F_BF16;
    E2F_CUDA_TRY(tb ? (yb ? launch_embed<kBF16, kBF16>(*cfg, tokens, n_atoms, table, out, status, s)
                          : launch_embed<kBF16, kF32>(*cfg, tokens, n_atoms, table, out, status, s))
                    : (yb ? launch_embed<kF32, kBF16>(*cfg, tokens, n_atoms, table, out, status, s)
                          : launch_embed<kF32, kF32>(*cfg, tokens, n_atoms, table, out, status, s)));
    return E2F_OK;
}

extern "C" size_t e2f_embedding_backward_workspace_size(int64_t n_atoms, const e2f_embed_cfg* cfg) {
    if (check_embed_cfg(cfg) != E2F_OK || n_atoms < 0 || n_atoms > INT32_MAX) return 0;
    return embed_layout(n_atoms, *cfg).bytes;
}

extern "C" e2f_status e2f_embedding_backward(const e2f_embed_cfg* cfg, const int32_t* tokens, int64_t n_atoms,
                                             const float* grad_out, float* grad_table, void* workspace,
                                             size_t ws_bytes, void* stream) {
    e2f_status st = check_embed_cfg(cfg);
    if (st != E2F_OK) return st;
    if (n_atoms < 0 || n_atoms > INT32_MAX) return E2F_ERR_INVALID_ARG;
    if (!grad_table || !workspace || (n_atoms > 0 && (!tokens || !grad_out))) return E2F_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) % 256 || reinterpret_cast<uintptr_t>(grad_out) % 16 ||
        reinterpret_cast<uintptr_t>(grad_table) % 16)
        return E2F_ERR_ALIGNMENT;
    const EmbedWs w = embed_layout(n_atoms, *cfg);
    if (ws_bytes < w.bytes) return E2F_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n_atoms == 0) {
        E2F_CUDA_TRY(cudaMemsetAsync(workspace, 0, sizeof(int), s));
        E2F_CUDA_TRY(cudaMemsetAsync(grad_table, 0, 4 * (size_t)cfg->n_tokens * cfg->C, s));
        return E2F_OK;
    }
    char* ws = static_cast<char*>(workspace);
    E2F_CUDA_TRY(w.V == 4 ? run_embed_bwd<4>(*cfg, tokens, n_atoms, grad_out, grad_table, ws, w, s)
                          : run_embed_bwd<1>(*cfg, tokens, n_atoms, grad_out, grad_table, ws, w, s));
    return E2F_OK;
}
