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

constexpr int HEADS = 2;  // kv heads of one block

struct Layer {
    uint8_t* k_codes;
    uint8_t* v_codes;
    uint16_t* k_norms;
    uint16_t* v_norms;
    uint32_t* k_qjl;
    uint16_t* k_gamma;
    int32_t k_bytes, v_bytes, qjl_words;  // of one row
    int32_t hkv;
};

struct Args {
    Layer layers[LAYERS_PER_LAUNCH];
    int batch, max_path, advance, groups;  // groups: blocks per sequence (of HEADS heads), for the layer with most
    int capacity;              // slots of a sequence, or of a block of the pool
    int num_blocks, max_blocks;  // paged: blocks of a pool, entries per sequence
    const int32_t* table;
    const int32_t* path;       // [batch][max_path]
    const int32_t* path_lens;  // [batch]
    const int32_t* base;       // [batch]
    int32_t* new_lens;         // [batch] or null
    uint32_t* err;
};

// The rows of one array that a block moves, as units of T: thread t takes unit
// t % lanes of every THREADS / lanes-th row, lanes being the units of a row
// rounded up to a power of two (no division).  All of a head's rows are read
// before any is written.
template <typename T, int N>
struct Mover {
    T v[HEADS][N];
    int unit, row0, shift, units;
    __device__ __forceinline__ Mover(int row_bytes) {
        units = row_bytes / static_cast<int>(sizeof(T));
        shift = units <= 1 ? 0 : 32 - __clz(units - 1);
        unit = threadIdx.x & ((1 << shift) - 1);
        row0 = threadIdx.x >> shift;
    }
    // f(i, head, row, unit) over this thread's units
    template <typename F>
    __device__ __forceinline__ void each(int n, int heads, F f) {
        const int step = THREADS >> shift;
        if (unit >= units) return;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = row0 + i * step;
            if (r < n) {
#pragma unroll
                for (int h = 0; h < HEADS; ++h)
                    if (h < heads) f(i, h, r);
            }
        }
    }
    __device__ __forceinline__ void load(const void* base, const long long* from, int n, int heads, long long head) {
        each(n, heads, [&](int i, int h, int r) {
            if (from[r] >= 0) v[h][i] = static_cast<const T*>(base)[(from[r] + h * head) * units + unit];
        });
    }
    __device__ __forceinline__ void store(void* base, const long long* from, const long long* to, int n, int heads,
                                          long long head) {
        each(n, heads, [&](int i, int h, int r) {
            if (from[r] >= 0) static_cast<T*>(base)[(to[r] + h * head) * units + unit] = v[h][i];
        });
    }
};

// Rows of codes in 16-byte units, or 8-byte ones (d = 64 at 3 bits: 24 bytes).
template <typename T, int N>
__device__ __forceinline__ void move_codes(const Layer& y, const long long* from, const long long* to, int n, int heads,
                                           long long row, long long head) {
    Mover<T, N> k(y.k_bytes), v(y.v_bytes);
    uint8_t* kc = y.k_codes + row * y.k_bytes;
    uint8_t* vc = y.v_codes + row * y.v_bytes;
    k.load(kc, from, n, heads, head);
    v.load(vc, from, n, heads, head);
    __syncthreads();
    k.store(kc, from, to, n, heads, head);
    v.store(vc, from, to, n, heads, head);
}

// Block (sequence and two heads, layer).  It is latency: a chain of length,
// path, row and write; two heads a block share the chain's start, and six
// blocks an SM cover one another's.  (48 sequences x 32 layers x 8 heads, up to
// 64 rows of 116 bytes each: 27 us, 3.3 TB/s.  Its 6144 blocks each walk the
// chain anew, barriers being the first stall; of the 64 MB it reads, 44 are the
// rows, the rest mostly the second halves of 48-byte rows' sectors and sectors
// written in part; norms, next to each other, are 5%.  27.5 us with four heads a
// block and four blocks an SM, 42 with one head, 67 with one head and divisions
// in the row index.)
// SMALL: every layer's rows are of at most 64 bytes, in 16-byte units; SKETCH:
// some layer has one (the larger rows' and the sketches' registers would cost
// the others their blocks per SM).  One layer with wider rows sends a launch's
// layers all to the wide instance: the same call with four int8 layers takes 83
// us in place of 30 (caches flushed).
template <bool SMALL, bool SKETCH>
__global__ void __launch_bounds__(THREADS, SMALL ? (SKETCH ? 3 : 6) : 1) commit_kernel(const __grid_constant__ Args a) {
    __shared__ long long from[MAX_PATH], to[MAX_PATH];  // cache rows of head 0 (from: -1, a row that stays)
    __shared__ int bad;
    const Layer& y = a.layers[blockIdx.y];
    const int b = static_cast<int>(blockIdx.x) / a.groups, h0 = static_cast<int>(blockIdx.x) % a.groups * HEADS;
    if (h0 >= y.hkv) return;
    const int tid = threadIdx.x, heads = min(HEADS, y.hkv - h0);
    const int n = a.path_lens[b], base = a.base[b];
    const int p = tid < min(n, a.max_path) ? a.path[static_cast<size_t>(b) * a.max_path + tid] : 0;
    const long long room = a.table ? static_cast<long long>(a.max_blocks) * a.capacity : a.capacity;
    const bool fits = n >= 0 && n <= a.max_path && base >= 0 && base + static_cast<long long>(n) <= room;
    const bool first = a.advance && h0 == 0 && blockIdx.y == 0;
    if (tid == 0) bad = fits ? 0 : TQ_DEVERR_POSITION;
    __syncthreads();
    if (fits && tid < n) {
        if (p < 0 || p >= MAX_PATH || base + static_cast<long long>(p) >= room) {
            atomicOr(&bad, TQ_DEVERR_POSITION);
        } else {
            auto row = [&](int slot) -> long long {
                if (!a.table) return static_cast<long long>(b) * y.hkv * a.capacity + slot;
                const int pg = a.table[static_cast<size_t>(b) * a.max_blocks + slot / a.capacity];
                if (pg < 0 || pg >= a.num_blocks) {
                    atomicOr(&bad, TQ_DEVERR_PAGE);
                    return -1;
                }
                return static_cast<long long>(pg) * y.hkv * a.capacity + slot % a.capacity;
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
    const long long head = a.capacity, row = h0 * head;  // rows between heads; the block's first head
    Mover<uint16_t, 1> kn(2), vn(2), kg(2);
    Mover<uint32_t, 2> kq(4 * y.qjl_words);
    kn.load(y.k_norms + row, from, n, heads, head);
    vn.load(y.v_norms + row, from, n, heads, head);
    if (SKETCH && y.qjl_words) {
        kq.load(y.k_qjl + row * y.qjl_words, from, n, heads, head);
        kg.load(y.k_gamma + row, from, n, heads, head);
    }
    // (the codes' barrier stands between these loads and their stores too)
    if constexpr (SMALL) {
        move_codes<uint4, 1>(y, from, to, n, heads, row, head);
    } else if (((y.k_bytes | y.v_bytes) & 15) == 0) {
        move_codes<uint4, 4>(y, from, to, n, heads, row, head);
    } else {
        move_codes<uint2, 2>(y, from, to, n, heads, row, head);
    }
    kn.store(y.k_norms + row, from, to, n, heads, head);
    vn.store(y.v_norms + row, from, to, n, heads, head);
    if (SKETCH && y.qjl_words) {
        kq.store(y.k_qjl + row * y.qjl_words, from, to, n, heads, head);
        kg.store(y.k_gamma + row, from, to, n, heads, head);
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
        st = table ? validate_pages(params[i], caches + i, table, &pm, true) : validate_cache(params[i], caches + i, true);
        if (st != TQ_OK) return st;
        const int n = table ? table->batch : caches[i].batch;
        if (i && (n != batch || caches[i].capacity != caches[0].capacity || caches[i].batch != caches[0].batch))
            return TQ_ERR_INVALID_ARG;
        batch = n;
    }
    for (int at = 0; at < n_layers; at += LAYERS_PER_LAUNCH) {
        Args a{};
        bool small = true, sketch = false;
        const int count = n_layers - at < LAYERS_PER_LAUNCH ? n_layers - at : LAYERS_PER_LAUNCH;
        for (int i = 0; i < count; ++i) {
            const tq_params& p = params[at + i];
            const tq_cache& c = caches[at + i];
            Layer& y = a.layers[i];
            y.k_codes = c.k_codes;
            y.v_codes = c.v_codes;
            y.k_norms = c.k_norms;
            y.v_norms = c.v_norms;
            y.k_qjl = reinterpret_cast<uint32_t*>(c.k_qjl);
            y.k_gamma = c.k_gamma;
            y.k_bytes = vector_bytes(p.k_mode, p.k_bits, p.head_dim);
            y.v_bytes = vector_bytes(p.v_mode, p.v_bits, p.head_dim);
            y.qjl_words = p.qjl_dims / 32;
            sketch = sketch || y.qjl_words;
            small = small && y.k_bytes <= 64 && y.v_bytes <= 64 && ((y.k_bytes | y.v_bytes) & 15) == 0;
            y.hkv = p.num_kv_heads;
            const int groups = (p.num_kv_heads + HEADS - 1) / HEADS;
            if (groups > a.groups) a.groups = groups;
        }
        if (static_cast<long long>(batch) * a.groups > INT32_MAX) return TQ_ERR_INVALID_ARG;
        a.batch = batch;
        a.capacity = caches[0].capacity;
        a.num_blocks = caches[0].batch;
        a.max_path = max_path;
        a.advance = at == 0;
        a.max_blocks = table ? table->max_blocks : 0;
        a.table = table ? table->d_table : nullptr;
        a.path = d_path;
        a.path_lens = d_path_lens;
        a.base = d_base_lens;
        a.new_lens = d_new_lens;
        a.err = d_error;
        const dim3 grid(static_cast<unsigned>(batch) * a.groups, static_cast<unsigned>(count));
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
        if (!small) commit_kernel<false, true><<<grid, THREADS, 0, cs>>>(a);
        else if (sketch) commit_kernel<true, true><<<grid, THREADS, 0, cs>>>(a);
        else commit_kernel<true, false><<<grid, THREADS, 0, cs>>>(a);
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
