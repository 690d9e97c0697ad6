// Species embedding: out[n,0,:] = scale table[token_n,:] (higher degrees zero),
// and its gradient, grad_table[v,:] = scale sum_{n: token_n = v} grad_out[n,0,:].
//
// The gradient sorts the tokens (a stable radix sort, 8 bits a pass, so equal
// tokens keep their order) and sums runs of equal tokens over fixed chunks of
// the sorted order; a run that crosses chunks is joined from its chunks' sums.
// Every sum has one fixed order and no atomics, so results repeat bit for bit.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "feature_io.cuh"

namespace e2f {
namespace {

constexpr int kMaxEmbedC = 16384;
constexpr int kSortTile = 1024;  // tokens of a sorting block (256 threads, 4 each)
constexpr int kRunChunk = 64;    // sorted tokens summed by one team of lanes

struct EmbedWs {
    size_t o_status, o_hist, o_tot, o_key[2], o_idx[2], o_part, bytes;
    int64_t tiles, chunks;
    int passes;
};

EmbedWs embed_layout(int64_t n, const e2f_embed_cfg& c) {
    EmbedWs w{};
    size_t o = 0;
    auto take = [&](size_t b) { size_t r = o; o = align_up(o + b, 256); return r; };
    w.passes = 1;
    while (w.passes < 4 && ((int64_t)c.n_tokens >> (8 * w.passes))) ++w.passes;
    w.tiles = (n + kSortTile - 1) / kSortTile;
    w.chunks = (n + kRunChunk - 1) / kRunChunk;
    w.o_status = take(256);  // first: e2f_attention_status reads it
    w.o_hist = take(4 * 256 * (size_t)w.tiles);
    w.o_tot = take(4 * 256);
    for (int k = 0; k < 2; ++k) {
        w.o_key[k] = take(4 * (size_t)n);
        w.o_idx[k] = take(4 * (size_t)n);
    }
    w.o_part = take(8 * (size_t)w.chunks * c.C);
    w.bytes = o;
    return w;
}

template <int TT, int YT, int V>
__global__ void __launch_bounds__(256) k_embed(const int32_t* tok, int64_t n, const void* table, int n_tokens, int K,
                                               int C, float scale, void* out, int* status) {
    const int cv = C / V;
    const int64_t total = n * K * cv, step = (int64_t)gridDim.x * 256;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += step) {
        const int64_t row = i / cv, node = row / K;
        const int c = (int)(i - row * cv) * V;
        float v[V] = {};
        if (row == node * K) {
            const int t = tok[node];
            if (t >= 0 && t < n_tokens) {
                load_vec<TT, V>(table, (int64_t)t * C + c, v);
                for (int k = 0; k < V; ++k) v[k] *= scale;
            } else if (t >= n_tokens && status) {
                *status = E2F_ERR_INVALID_ARG;
            }
        }
        store_vec<YT, V>(out, row * C + c, v);
    }
}

// sort key of a token: padding and tokens outside the table go behind the last token
__device__ __forceinline__ uint32_t sort_key(int t, int n_tokens) {
    return t < 0 || t >= n_tokens ? (uint32_t)n_tokens : (uint32_t)t;
}

// digit counts of one tile: hist[digit][tile]
template <bool FIRST>
__global__ void __launch_bounds__(256) k_sort_count(const void* keys, int64_t n, int n_tokens, int shift,
                                                    int64_t tiles, uint32_t* hist, int* status) {
    __shared__ uint32_t cnt[256];
    cnt[threadIdx.x] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kSortTile;
    for (int j = 0; j < kSortTile / 256; ++j) {
        const int64_t p = base + j * 256 + threadIdx.x;
        if (p >= n) break;
        uint32_t k;
        if constexpr (FIRST) {
            const int t = static_cast<const int*>(keys)[p];
            if (t >= n_tokens && status) *status = E2F_ERR_INVALID_ARG;
            k = sort_key(t, n_tokens);
        } else {
            k = static_cast<const uint32_t*>(keys)[p];
        }
        atomicAdd(&cnt[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    hist[threadIdx.x * tiles + blockIdx.x] = cnt[threadIdx.x];
}

// block d: exclusive prefix over the tiles of digit d, in place; its total
__global__ void __launch_bounds__(256) k_sort_scan(uint32_t* hist, int64_t tiles, uint32_t* total) {
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
                                                    const uint32_t* total, uint32_t* keys_out, int* idx_out) {
    constexpr int J = kSortTile / 256;
    __shared__ uint32_t wc[8][256];
    __shared__ uint32_t ws[8];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int k = 0; k < 8; ++k) wc[k][threadIdx.x] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kSortTile + w * (32 * J);
    uint32_t key[J], rank[J];
    for (int j = 0; j < J; ++j) {
        const int64_t p = base + j * 32 + lane;
        const bool ok = p < n;
        key[j] = 0;
        if (ok) {
            if constexpr (FIRST) key[j] = sort_key(static_cast<const int*>(keys)[p], n_tokens);
            else key[j] = static_cast<const uint32_t*>(keys)[p];
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

// A team of lanes sums one chunk of the sorted tokens, run by run. A run that
// begins and ends in the chunk is final; one that begins here and goes on is
// the chunk's open sum (part[2 chunk + 1]); one that came in from the chunk
// before is its carry (part[2 chunk]).
template <int V>
__global__ void __launch_bounds__(256) k_run_sum(const float* g, int64_t row_stride, int C, const uint32_t* keys,
                                                 const int* idx, int64_t n, uint32_t n_tokens, float scale, int team,
                                                 float* grad, float* part) {
    const int64_t chunk = (blockIdx.x * 256ll + threadIdx.x) / team;
    const int c = (blockIdx.y * team + threadIdx.x % team) * V;
    const int64_t p0 = chunk * kRunChunk, p1 = min(p0 + kRunChunk, n);
    if (p0 >= n || c >= C) return;
    float acc[V] = {};
    uint32_t cur = keys[p0];
    bool begins = p0 == 0 || keys[p0 - 1] != cur;
    auto flush = [&](bool ends) {
        if (cur >= n_tokens) return;
        float v[V];
        for (int k = 0; k < V; ++k) v[k] = acc[k] * (begins && ends ? scale : 1.f);
        if (begins && ends) store_vec<kF32, V>(grad, (int64_t)cur * C + c, v);
        else store_vec<kF32, V>(part, (2 * chunk + (begins ? 1 : 0)) * C + c, v);
    };
    constexpr int U = 8;
    for (int64_t p = p0; p < p1; p += U) {
        uint32_t key[U];
        float v[U][V];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            key[j] = p + j < p1 ? keys[p + j] : n_tokens;
            for (int k = 0; k < V; ++k) v[j][k] = 0.f;
            if (p + j < p1 && key[j] < n_tokens) load_vec<kF32, V>(g, idx[p + j] * row_stride + c, v[j]);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (p + j >= p1) break;
            if (key[j] != cur) {
                flush(true);
                cur = key[j];
                begins = true;
                for (int k = 0; k < V; ++k) acc[k] = 0.f;
            }
            for (int k = 0; k < V; ++k) acc[k] += v[j][k];
        }
    }
    flush(p1 == n || keys[p1] != cur);
}

// Block (chunk, 32 columns): if a run opened in the chunk, adds the carries of the chunks it reaches.
__global__ void __launch_bounds__(1024) k_run_join(const float* part, int C, const uint32_t* keys, int64_t n,
                                                   uint32_t n_tokens, int64_t chunks, float scale, float* grad) {
    __shared__ float sh[32][33];
    const int64_t s = blockIdx.x, p0 = s * kRunChunk, p1 = p0 + kRunChunk;
    if (p1 >= n) return;
    const uint32_t key = keys[p1 - 1];
    if (key >= n_tokens || keys[p1] != key) return;              // nothing goes on
    if (p0 > 0 && keys[p0] == key && keys[p0 - 1] == key) return;  // it did not begin here
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.y * 32 + lane;
    float sum = w == 0 && c < C ? part[(2 * s + 1) * C + c] : 0.f;
    for (int64_t j = s + 1 + w; j < chunks && keys[j * kRunChunk] == key; j += 32)
        if (c < C) sum += part[2 * j * C + c];
    sh[w][lane] = sum;
    __syncthreads();
    if (w == 0 && c < C) {
        for (int k = 1; k < 32; ++k) sum += sh[k][lane];
        grad[(int64_t)key * C + c] = scale * sum;
    }
}

template <int TT, int YT>
cudaError_t launch_embed(const e2f_embed_cfg& f, const int32_t* tok, int64_t n, const void* table, void* out,
                         int* status, cudaStream_t s) {
    const int K = (f.L + 1) * (f.L + 1);
    auto grid = [&](int v) { return (unsigned)std::min<int64_t>((n * K * (f.C / v) + 255) / 256, 148 * 64); };
    count_launch();
    if (f.C % 4 == 0)
        k_embed<TT, YT, 4><<<grid(4), 256, 0, s>>>(tok, n, table, f.n_tokens, K, f.C, f.scale, out, status);
    else
        k_embed<TT, YT, 1><<<grid(1), 256, 0, s>>>(tok, n, table, f.n_tokens, K, f.C, f.scale, out, status);
    return cudaGetLastError();
}

cudaError_t run_embed_bwd(const e2f_embed_cfg& f, const int32_t* tok, int64_t n, const float* g, float* grad, char* ws,
                          const EmbedWs& w, cudaStream_t s) {
    const int K = (f.L + 1) * (f.L + 1);
    int* status = reinterpret_cast<int*>(ws + w.o_status);
    uint32_t* hist = reinterpret_cast<uint32_t*>(ws + w.o_hist);
    uint32_t* total = reinterpret_cast<uint32_t*>(ws + w.o_tot);
    uint32_t* key[2];
    int* idx[2];
    for (int k = 0; k < 2; ++k) {
        key[k] = reinterpret_cast<uint32_t*>(ws + w.o_key[k]);
        idx[k] = reinterpret_cast<int*>(ws + w.o_idx[k]);
    }
    float* part = reinterpret_cast<float*>(ws + w.o_part);
    cudaError_t e = cudaMemsetAsync(grad, 0, 4 * (size_t)f.n_tokens * f.C, s);
    if (e != cudaSuccess) return e;
    const unsigned tiles = (unsigned)w.tiles;
    for (int p = 0; p < w.passes; ++p) {
        const int to = p & 1, from = to ^ 1;
        if (p == 0) {
            k_sort_count<true><<<tiles, 256, 0, s>>>(tok, n, f.n_tokens, 0, w.tiles, hist, status);
            k_sort_scan<<<256, 256, 0, s>>>(hist, w.tiles, total);
            k_sort_place<true><<<tiles, 256, 0, s>>>(tok, nullptr, n, f.n_tokens, 0, w.tiles, hist, total, key[to],
                                                     idx[to]);
        } else {
            k_sort_count<false><<<tiles, 256, 0, s>>>(key[from], n, f.n_tokens, 8 * p, w.tiles, hist, nullptr);
            k_sort_scan<<<256, 256, 0, s>>>(hist, w.tiles, total);
            k_sort_place<false><<<tiles, 256, 0, s>>>(key[from], idx[from], n, f.n_tokens, 8 * p, w.tiles, hist, total,
                                                      key[to], idx[to]);
        }
        count_launch(3);
    }
    const int at = (w.passes - 1) & 1;
    const int V = f.C % 4 == 0 ? 4 : 1;
    int team = 1;
    while (team < 32 && team * V < f.C) team *= 2;
    const dim3 grid((unsigned)((w.chunks * team + 255) / 256), (unsigned)((f.C + team * V - 1) / (team * V)));
    if (V == 4)
        k_run_sum<4><<<grid, 256, 0, s>>>(g, (int64_t)K * f.C, f.C, key[at], idx[at], n, (uint32_t)f.n_tokens, f.scale,
                                          team, grad, part);
    else
        k_run_sum<1><<<grid, 256, 0, s>>>(g, (int64_t)K * f.C, f.C, key[at], idx[at], n, (uint32_t)f.n_tokens, f.scale,
                                          team, grad, part);
    count_launch();
    if (w.chunks > 1) {
        k_run_join<<<dim3((unsigned)w.chunks, (unsigned)((f.C + 31) / 32)), 1024, 0, s>>>(
            part, f.C, key[at], n, (uint32_t)f.n_tokens, w.chunks, f.scale, grad);
        count_launch();
    }
    return cudaGetLastError();
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
    E2F_CUDA_TRY(cudaMemsetAsync(workspace, 0, sizeof(int), s));
    if (n_atoms == 0) {
        E2F_CUDA_TRY(cudaMemsetAsync(grad_table, 0, 4 * (size_t)cfg->n_tokens * cfg->C, s));
        return E2F_OK;
    }
    E2F_CUDA_TRY(run_embed_bwd(*cfg, tokens, n_atoms, grad_out, grad_table, static_cast<char*>(workspace), w, s));
    return E2F_OK;
}
