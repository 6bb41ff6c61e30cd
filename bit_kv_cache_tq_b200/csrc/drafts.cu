// The accepted path of a tree of drafted tokens moved to the front of the
// drafted slots, in every layer, and the sequence lengths advanced.
//
// Sequence b's drafts sit in slots base[b] .. base[b] + n - 1; draft path[b][i]
// goes to slot base[b] + i for i < path_lens[b].  Rows are carried over byte
// for byte, so what they stand for does not change.

#include <cuda_runtime.h>

#include "device_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tq {
namespace drafts {

constexpr int MAX_PATH = 64;
constexpr int LAYERS_PER_LAUNCH = 64;
constexpr int THREADS = 256;

struct Layer {
    uint8_t* k_codes;
    uint8_t* v_codes;
    uint16_t* k_norms;
    uint16_t* v_norms;
    uint32_t* k_qjl;
    uint16_t* k_gamma;
    int32_t k_units, v_units, qjl_words;  // 16-byte units of a code row; 32-bit words of a sketch row
    int32_t hkv;
    int32_t row0;      // index of the layer's first (sequence, kv head) block
    int32_t capacity;  // slots of a sequence, or of a block of the pool
    int32_t num_blocks;
};

struct Args {
    Layer layers[LAYERS_PER_LAUNCH];
    int n_layers, batch, max_path, advance;
    int max_blocks;            // paged: entries per sequence (0: contiguous)
    const int32_t* table;
    const int32_t* path;       // [batch][max_path]
    const int32_t* path_lens;  // [batch]
    const int32_t* base;       // [batch]
    int32_t* new_lens;         // [batch] or null
    uint32_t* err;
};

// Up to N units of one array per thread, read before the barrier, written after it.
template <typename T, int N>
struct Held {
    T v[N];
};

template <typename T, int N>
__device__ __forceinline__ void load_rows(Held<T, N>& h, const T* base, const long long* from, int units, int total) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int u = threadIdx.x + i * THREADS;
        if (u < total) {
            const long long row = from[u / units];
            if (row >= 0) h.v[i] = base[row * units + u % units];
        }
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_rows(const Held<T, N>& h, T* base, const long long* from, const long long* to,
                                           int units, int total) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int u = threadIdx.x + i * THREADS;
        if (u < total && from[u / units] >= 0) base[to[u / units] * units + u % units] = h.v[i];
    }
}

// One block per (layer, sequence, kv head): all the path's rows are read
// before any is written, so the path may name the drafts in any order.
__global__ void __launch_bounds__(THREADS) commit_kernel(const __grid_constant__ Args a) {
    __shared__ long long from[MAX_PATH], to[MAX_PATH];
    __shared__ int bad;
    int l = 0;
    const int blk = static_cast<int>(blockIdx.x);
    while (l + 1 < a.n_layers && blk >= a.layers[l + 1].row0) ++l;
    const Layer& y = a.layers[l];
    const int b = (blk - y.row0) / y.hkv, head = (blk - y.row0) % y.hkv;
    const int tid = threadIdx.x;
    const int n = a.path_lens[b], base = a.base[b];
    const long long room = a.table ? static_cast<long long>(a.max_blocks) * y.capacity : y.capacity;
    const bool fits = n >= 0 && n <= a.max_path && base >= 0 && base + static_cast<long long>(n) <= room;
    const bool first = a.advance && blk == y.row0 + b * y.hkv && l == 0;
    if (tid == 0) bad = fits ? 0 : TQ_DEVERR_POSITION;
    __syncthreads();
    if (fits && tid < n) {
        const int p = a.path[static_cast<size_t>(b) * a.max_path + tid];
        if (p < 0 || p >= MAX_PATH || base + static_cast<long long>(p) >= room) {
            atomicOr(&bad, TQ_DEVERR_POSITION);
        } else {
            auto row = [&](int slot) -> long long {
                if (!a.table) return (static_cast<long long>(b) * y.hkv + head) * y.capacity + slot;
                const int pg = a.table[static_cast<size_t>(b) * a.max_blocks + slot / y.capacity];
                if (pg < 0 || pg >= y.num_blocks) {
                    atomicOr(&bad, TQ_DEVERR_PAGE);
                    return -1;
                }
                return (static_cast<long long>(pg) * y.hkv + head) * y.capacity + slot % y.capacity;
            };
            to[tid] = row(base + tid);
            from[tid] = p == tid ? -1 : row(base + p);  // (a row that is already in place is left alone)
        }
    }
    __syncthreads();
    if (bad) {
        if (tid == 0 && a.err) atomicOr(a.err, static_cast<uint32_t>(bad));
        if (first && tid == 0 && a.new_lens) a.new_lens[b] = base;
        return;
    }
    if (first && tid == 0 && a.new_lens) a.new_lens[b] = base + n;
    Held<uint4, 4> kc, vc;
    Held<uint16_t, 1> kn, vn, kg;
    Held<uint32_t, 2> kq;
    load_rows(kc, reinterpret_cast<const uint4*>(y.k_codes), from, y.k_units, n * y.k_units);
    load_rows(vc, reinterpret_cast<const uint4*>(y.v_codes), from, y.v_units, n * y.v_units);
    load_rows(kn, y.k_norms, from, 1, n);
    load_rows(vn, y.v_norms, from, 1, n);
    if (y.qjl_words) {
        load_rows(kq, y.k_qjl, from, y.qjl_words, n * y.qjl_words);
        load_rows(kg, y.k_gamma, from, 1, n);
    }
    __syncthreads();
    store_rows(kc, reinterpret_cast<uint4*>(y.k_codes), from, to, y.k_units, n * y.k_units);
    store_rows(vc, reinterpret_cast<uint4*>(y.v_codes), from, to, y.v_units, n * y.v_units);
    store_rows(kn, y.k_norms, from, to, 1, n);
    store_rows(vn, y.v_norms, from, to, 1, n);
    if (y.qjl_words) {
        store_rows(kq, y.k_qjl, from, to, y.qjl_words, n * y.qjl_words);
        store_rows(kg, y.k_gamma, from, to, 1, n);
    }
}

static tq_status commit(int32_t n_layers, const tq_params* params, const tq_cache* caches, const tq_block_table* table,
                        const int32_t* d_path, int32_t max_path, const int32_t* d_path_lens,
                        const int32_t* d_base_lens, int32_t* d_new_lens, uint32_t* d_error, void* stream) {
    if (n_layers < 1 || !params || !caches || !d_path || !d_path_lens || !d_base_lens) return TQ_ERR_INVALID_ARG;
    if (max_path < 1 || max_path > MAX_PATH) return TQ_ERR_INVALID_ARG;
    if (d_new_lens && (d_new_lens == d_base_lens || d_new_lens == d_path_lens)) return TQ_ERR_INVALID_ARG;
    int batch = 0;
    for (int i = 0; i < n_layers; ++i) {
        tq_status st = validate_params(params + i);
        if (st != TQ_OK) return st;
        PageMap pm;
        st = table ? validate_pages(params[i], caches + i, table, &pm) : validate_cache(params[i], caches + i);
        if (st != TQ_OK) return st;
        const int n = table ? table->batch : caches[i].batch;
        if (i && (n != batch || caches[i].capacity != caches[0].capacity || caches[i].batch != caches[0].batch))
            return TQ_ERR_INVALID_ARG;
        batch = n;
    }
    for (int at = 0; at < n_layers; at += LAYERS_PER_LAUNCH) {
        Args a{};
        a.n_layers = n_layers - at < LAYERS_PER_LAUNCH ? n_layers - at : LAYERS_PER_LAUNCH;
        long long blocks = 0;
        for (int i = 0; i < a.n_layers; ++i) {
            const tq_params& p = params[at + i];
            const tq_cache& c = caches[at + i];
            Layer& y = a.layers[i];
            y.k_codes = c.k_codes;
            y.v_codes = c.v_codes;
            y.k_norms = c.k_norms;
            y.v_norms = c.v_norms;
            y.k_qjl = reinterpret_cast<uint32_t*>(c.k_qjl);
            y.k_gamma = c.k_gamma;
            y.k_units = vector_bytes(p.k_mode, p.k_bits, p.head_dim) / 16;
            y.v_units = vector_bytes(p.v_mode, p.v_bits, p.head_dim) / 16;
            y.qjl_words = p.qjl_dims / 32;
            y.hkv = p.num_kv_heads;
            y.row0 = static_cast<int32_t>(blocks);
            y.capacity = c.capacity;
            y.num_blocks = c.batch;
            blocks += static_cast<long long>(batch) * p.num_kv_heads;
            if (blocks > INT32_MAX) return TQ_ERR_INVALID_ARG;
        }
        a.batch = batch;
        a.max_path = max_path;
        a.advance = at == 0;
        a.max_blocks = table ? table->max_blocks : 0;
        a.table = table ? table->d_table : nullptr;
        a.path = d_path;
        a.path_lens = d_path_lens;
        a.base = d_base_lens;
        a.new_lens = d_new_lens;
        a.err = d_error;
        commit_kernel<<<static_cast<unsigned>(blocks), THREADS, 0, static_cast<cudaStream_t>(stream)>>>(a);
        if (cudaGetLastError() != cudaSuccess) return TQ_ERR_CUDA;
    }
    return TQ_OK;
}

}  // namespace drafts
}  // namespace tq

// =================================================================== C ABI
extern "C" {

tq_status tq_commit_drafts(int32_t n_layers, const tq_params* params, const tq_cache* caches, const int32_t* d_path,
                           int32_t max_path, const int32_t* d_path_lens, const int32_t* d_base_lens,
                           int32_t* d_new_lens, uint32_t* d_error, void* stream) {
    return tq::drafts::commit(n_layers, params, caches, nullptr, d_path, max_path, d_path_lens, d_base_lens,
                              d_new_lens, d_error, stream);
}

tq_status tq_commit_drafts_paged(int32_t n_layers, const tq_params* params, const tq_cache* pools,
                                 const tq_block_table* table, const int32_t* d_path, int32_t max_path,
                                 const int32_t* d_path_lens, const int32_t* d_base_lens, int32_t* d_new_lens,
                                 uint32_t* d_error, void* stream) {
    if (!table) return TQ_ERR_INVALID_ARG;
    return tq::drafts::commit(n_layers, params, pools, table, d_path, max_path, d_path_lens, d_base_lens, d_new_lens,
                              d_error, stream);
}

}  // extern "C"
