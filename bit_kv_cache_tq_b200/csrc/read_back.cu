// Ranges of several sequences read back from the cache in 16 or 32 bits.
//
// Mathematics (as tq_dequantize): turbo vectors are
//   x = n16 R^-1(c[code] + gamma16 sqrt(pi/2)/m S^T (2z - 1)),  R^-1 = diag(s) H / sqrt(d),
// the sketch term only for keys with one; int8 vectors are scale16 * q.

#include <cuda_runtime.h>

#include <cmath>

#include "device_common.cuh"
#include "encode.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tq {
namespace read_back {

struct Args {
    QuantSide side[2];
    void* out[2];             // [batch][max_count][hkv][d]
    const int32_t* starts;    // [batch]
    const int32_t* counts;    // [batch]
    uint32_t* err;
    int batch, max_count, hkv, capacity;
    const int32_t* table;
    int max_blocks, block_size, num_blocks;
    uint32_t signs[8];
};

template <int DTYPE>
__device__ __forceinline__ void store8(void* base, size_t off, const float* x) {
    if constexpr (DTYPE == 0) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + off);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DTYPE == 1) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                w[i] = ptx::pack_half2(x[2 * i], x[2 * i + 1]);
            }
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Grid: (blocks, batch, side).  A vector on d/32 lanes, as the encoders.
template <int D, int DTYPE>
__global__ void __launch_bounds__(256) read_back_kernel(const __grid_constant__ Args a) {
    constexpr int LPV = D / 32, VPW = 32 / LPV;
    const QuantSide& s = a.side[blockIdx.z];
    void* out = a.out[blockIdx.z];
    if (!out) return;  // (the whole block: one side per block)
    __shared__ float scen[16];
    if (threadIdx.x < 16) scen[threadIdx.x] = s.centroids[threadIdx.x];
    __syncthreads();
    const int b = static_cast<int>(blockIdx.y);
    const int start = a.starts[b], count = a.counts[b];
    if (start < 0 || count < 0 || count > a.max_count || start > a.capacity - count) {
        if (a.err && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, TQ_DEVERR_POSITION);
        return;
    }
    const int lane = threadIdx.x & 31, sub = lane % LPV, grp = lane / LPV;
    const long long total = static_cast<long long>(count) * a.hkv;
    const long long nwarps = static_cast<long long>(gridDim.x) * (blockDim.x / 32);
    for (long long base = (static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32) * VPW;
         base < total; base += nwarps * VPW) {
        const long long v = base + grp;
        bool valid = v < total;
        const int h = valid ? static_cast<int>(v % a.hkv) : 0;
        const int t = valid ? static_cast<int>(v / a.hkv) : 0;
        size_t slot = 0;
        if (a.table) {
            const int at = start + t;
            const int blk = valid ? a.table[static_cast<size_t>(b) * a.max_blocks + at / a.block_size] : 0;
            if (blk < 0 || blk >= a.num_blocks) {
                if (a.err && sub == 0) atomicOr(a.err, TQ_DEVERR_PAGE);
                valid = false;
            }
            if (valid) slot = (static_cast<size_t>(blk) * a.hkv + h) * a.block_size + at % a.block_size;
        } else {
            slot = (static_cast<size_t>(b) * a.hkv + h) * a.capacity + (valid ? start + t : 0);
        }
        float x[32];
        const float norm = valid ? half_bits_to_float(s.norms[slot]) : 0.0f;
        if (s.mode == TQ_MODE_INT8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint2 w = valid ? *reinterpret_cast<const uint2*>(s.codes + slot * D + 8 * (sub + LPV * k))
                                      : make_uint2(0, 0);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t word = e < 4 ? w.x : w.y;
                    x[8 * k + e] = norm * static_cast<float>(static_cast<int8_t>((word >> (8 * (e & 3))) & 0xffu));
                }
            }
        } else {
            const uint32_t* words = reinterpret_cast<const uint32_t*>(s.codes + slot * static_cast<size_t>(s.vbytes));
            const uint32_t mask = (1u << s.bits) - 1u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t chunk =
                    valid ? stream_bits(words, s.vbytes / 4, 8 * s.bits * (sub + LPV * k), 8 * s.bits) : 0u;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[8 * k + e] = scen[(chunk >> (s.bits * e)) & mask];
            }
            if (s.m > 0 && valid) {
                const float coef = half_bits_to_float(s.gamma[slot]) * sqrtf(0.5f * 3.14159265358979f) / s.m;
                const uint32_t* z = reinterpret_cast<const uint32_t*>(s.qjl + slot * static_cast<size_t>(s.m / 8));
                for (int r = 0; r < s.m; ++r) {
                    const float w = (z[r >> 5] >> (r & 31)) & 1u ? coef : -coef;
                    const float* row = s.sketch + static_cast<size_t>(r) * D;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            x[8 * k + e] = fmaf(w, __ldg(row + 8 * (sub + LPV * k) + e), x[8 * k + e]);
                }
            }
            fwht_registers(x);
            fwht_lanes<32, LPV>(x, sub);
            const float scale = norm / sqrtf(static_cast<float>(D));
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[8 * k + e] = flip_sign(x[8 * k + e] * scale, sign_bit(a.signs, 8 * (sub + LPV * k) + e));
        }
        if (valid) {
            const size_t dst = ((static_cast<size_t>(b) * a.max_count + t) * a.hkv + h) * D;
#pragma unroll
            for (int k = 0; k < 4; ++k) store8<DTYPE>(out, dst + 8 * (sub + LPV * k), &x[8 * k]);
        }
    }
}

template <int D>
static void launch(const Args& a, int dtype, dim3 grid, cudaStream_t s) {
    switch (dtype) {
        case TQ_F32: read_back_kernel<D, 0><<<grid, 256, 0, s>>>(a); break;
        case TQ_BF16: read_back_kernel<D, 1><<<grid, 256, 0, s>>>(a); break;
        default: read_back_kernel<D, 2><<<grid, 256, 0, s>>>(a); break;
    }
}

static tq_status read(const tq_params* params, const tq_codebook* kcb, const tq_codebook* vcb, const tq_cache* cache,
                      const PageMap* pm, const int32_t* d_starts, const int32_t* d_counts, int32_t max_count,
                      tq_dtype dtype, void* k_out, void* v_out, uint32_t* d_error, void* stream) {
    tq_status st = validate_params(params);
    if (st != TQ_OK) return st;
    const tq_params& p = *params;
    if ((st = validate_cache(p, cache)) != TQ_OK) return st;
    if (!d_starts || !d_counts || max_count < 1 || (!k_out && !v_out)) return TQ_ERR_INVALID_ARG;
    if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16) return TQ_ERR_INVALID_ARG;
    if (!aligned16(k_out) || !aligned16(v_out)) return TQ_ERR_ALIGNMENT;
    if (k_out && p.k_mode == TQ_MODE_TURBO && (st = validate_codebook(kcb, p.head_dim, p.k_bits)) != TQ_OK) return st;
    if (v_out && p.v_mode == TQ_MODE_TURBO && (st = validate_codebook(vcb, p.head_dim, p.v_bits)) != TQ_OK) return st;
    Args a{};
    if (k_out) fill_side(a.side[0], p.k_mode, p.k_bits, p.head_dim, kcb);
    if (v_out) fill_side(a.side[1], p.v_mode, p.v_bits, p.head_dim, vcb);
    a.side[0].codes = cache->k_codes;
    a.side[0].norms = cache->k_norms;
    a.side[0].qjl = cache->k_qjl;
    a.side[0].gamma = cache->k_gamma;
    a.side[0].sketch = cache->qjl_matrix;
    a.side[0].m = p.qjl_dims;
    a.side[1].codes = cache->v_codes;
    a.side[1].norms = cache->v_norms;
    a.out[0] = k_out;
    a.out[1] = v_out;
    a.starts = d_starts;
    a.counts = d_counts;
    a.err = d_error;
    a.batch = pm ? pm->batch : cache->batch;
    a.max_count = max_count;
    a.hkv = p.num_kv_heads;
    a.capacity = pm ? pm->max_blocks * pm->block_size : cache->capacity;
    if (pm) {
        a.table = pm->table;
        a.max_blocks = pm->max_blocks;
        a.block_size = pm->block_size;
        a.num_blocks = pm->num_blocks;
    }
    if (a.batch > 65535) return TQ_ERR_INVALID_ARG;
    rotation_sign_bits(p.seed, p.head_dim, a.signs);
    const long long warps = (static_cast<long long>(max_count) * p.num_kv_heads * (p.head_dim / 32) + 31) / 32;
    long long blocks = (warps + 7) / 8;
    const long long cap = (148ll * 8 + a.batch - 1) / a.batch;
    if (blocks > cap) blocks = cap;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(a.batch), 2);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (p.head_dim) {
        case 64: launch<64>(a, dtype, grid, s); break;
        case 128: launch<128>(a, dtype, grid, s); break;
        default: launch<256>(a, dtype, grid, s); break;
    }
    return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace read_back
}  // namespace tq

// =================================================================== C ABI
extern "C" {

tq_status tq_read_back(const tq_params* params, const tq_codebook* kcb, const tq_codebook* vcb, const tq_cache* cache,
                       const int32_t* d_starts, const int32_t* d_counts, int32_t max_count, tq_dtype out_dtype,
                       void* d_k_out, void* d_v_out, uint32_t* d_error, void* stream) {
    return tq::read_back::read(params, kcb, vcb, cache, nullptr, d_starts, d_counts, max_count, out_dtype, d_k_out,
                               d_v_out, d_error, stream);
}

tq_status tq_read_back_paged(const tq_params* params, const tq_codebook* kcb, const tq_codebook* vcb,
                             const tq_cache* pool, const tq_block_table* table, const int32_t* d_starts,
                             const int32_t* d_counts, int32_t max_count, tq_dtype out_dtype, void* d_k_out,
                             void* d_v_out, uint32_t* d_error, void* stream) {
    if (!params) return TQ_ERR_INVALID_ARG;
    tq::PageMap pm;
    const tq_status st = tq::validate_pages(*params, pool, table, &pm);
    if (st != TQ_OK) return st;
    return tq::read_back::read(params, kcb, vcb, pool, &pm, d_starts, d_counts, max_count, out_dtype, d_k_out, d_v_out,
                               d_error, stream);
}

}  // extern "C"
