// Rotary positions fused with the append: a step's queries and keys are
// turned by their positions, the keys and values quantised into the cache.
//
// Mathematics: coordinate pair i of the first r coordinates of a head is
// turned by the angle pos * f_i, scaled by a magnitude g:
//   (a, b) -> g (a cos - b sin, b cos + a sin).
// The pairs are (i, i + r/2) in the half layout and (2i, 2i + 1) in the
// interleaved one.  Angles are counted in turns, as 64-bit fractions: the
// host rounds f_i / (2 pi) to a multiple of 2^-64 and the product with the
// position wraps modulo one whole turn by itself, so no position is too far
// for an exact reduction (an fp32 product pos * f loses the angle past a few
// ten thousand positions).  The remaining fraction, in [-1/2, 1/2), goes to
// fp32 (error below 2^-25 of a turn) and to sincospif.  The turned key stays
// in fp32 until its norm and codes are taken: nothing is rounded between the
// rotation and the quantiser.
//
// It is bound by instructions where it quantises and by memory where it turns
// queries, so blocks of the three kinds of work alternate.  8192 tokens of
// 32 + 8 + 8 heads, K4/V3, bf16: 54 us (176 MB, 3.3 TB/s), quantising alone
// 24.  (The kinds share one register limit, 80 for three blocks an SM, at which
// the encoders spill 284 bytes.  With cold caches: 62 us, int8 sides 50, keys with
// 64 sketch rows 193, whose search and sketch are scalar; rotary_dims other than d
// and d/2 in the half layout cost 45 us more, the partners being read again one by
// one.)

#include <cuda_runtime.h>

#include <cmath>
#include <limits>

#include "device_common.cuh"
#include "encode.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tq {
namespace rope {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int MAX_TOKENS = 8;  // tokens of one block's table of cosines and sines

struct Args {
    QuantSide side[2];            // 0 = K, 1 = V (src unused: the sources have strides)
    const void* src[3];           // K, V, Q: [batch * n_new] tokens, `stride` elements apart, [heads][d] each
    long long stride[3];
    void* q_out;                  // [batch * n_new][hq][d]
    const int32_t* positions;     // [batch]: first slot
    const int32_t* rope_positions;  // [batch][n_new], or null: the slot
    uint32_t* err;
    int tokens, n_new, hq, hkv, capacity;
    int chunk, chunks, kinds;     // tokens per block, blocks per kind, kinds (3, or 2 without queries)
    uint64_t hq_magic, hkv_magic, n_new_magic;
    const int32_t* table;
    int max_blocks, block_size, num_blocks;
    int rotary, layout;
    float magnitude;
    uint32_t signs[8];
    uint64_t turns[128];          // 2^64ths of a turn a position adds to pair i
};

// What a block keeps of its tokens.
template <int D>
struct Shared {
    uint32_t grid[128];
    float2 cs[MAX_TOKENS][D / 2];      // (g cos, g sin) of pair i (the rows' stride keeps 16-byte alignment)
    long long slot[MAX_TOKENS];        // cache row of head 0, or -1: not written
};

// Turn the lane's 32 coordinates (chunks sub + LPV k of the vector at `row`).
template <int D, int DTYPE>
__device__ __forceinline__ void turn(const Args& a, const float2* cs, const void* base, size_t off, float (&x)[32],
                                     int sub) {
    constexpr int LPV = D / 32;
    const int r = a.rotary;
    if (a.layout == TQ_ROPE_INTERLEAVED) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i0 = 8 * (sub + LPV * k);
            if (i0 < r) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 t = i0 + e < r ? cs[(i0 + e) / 2] : make_float2(1.f, 0.f);
                    const float u = x[8 * k + e], w = x[8 * k + e + 1];
                    x[8 * k + e] = u * t.x - w * t.y;
                    x[8 * k + e + 1] = w * t.x + u * t.y;
                }
            }
        }
        return;
    }
    if (r == D || r == D / 2) {
        // the partner coordinate i + r/2 is in this lane too: chunk k + 2 (r = D) or k + 1 (r = D/2)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (r == D / 2 && k == 1) break;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 t = cs[8 * (sub + LPV * k) + e];
                if (r == D) {
                    const float u = x[8 * k + e], w = x[8 * (k + 2) + e];
                    x[8 * k + e] = u * t.x - w * t.y;
                    x[8 * (k + 2) + e] = w * t.x + u * t.y;
                } else {
                    const float u = x[e], w = x[8 + e];
                    x[e] = u * t.x - w * t.y;
                    x[8 + e] = w * t.x + u * t.y;
                }
            }
        }
        return;
    }
    // any other even r: the partners are other lanes' coordinates, read again from the source (the line is in L1)
    const int h = r / 2;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = 8 * (sub + LPV * k) + e;
            if (i < r) {
                const bool low = i < h;
                const float2 t = cs[low ? i : i - h];
                const float p = load_scalar(base, off + (low ? i + h : i - h), DTYPE);
                x[8 * k + e] = low ? x[8 * k + e] * t.x - p * t.y : x[8 * k + e] * t.x + p * t.y;
            }
        }
    }
}

// A lane's 32 coordinates as they are in memory.
template <int D, int DTYPE>
struct Raw {
    static constexpr int LPV = D / 32, N = DTYPE == 0 ? 2 : 1;
    uint4 w[4 * N];
    __device__ __forceinline__ void load(const void* src, size_t off, int sub) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(src) + off * (DTYPE == 0 ? 4 : 2));
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) w[N * k + i] = __ldcs(p + N * (sub + LPV * k) + i);
    }
    __device__ __forceinline__ void values(float (&x)[32]) const {
#pragma unroll
        for (int k = 0; k < 4 * N; ++k) {
            const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DTYPE == 0) {
                    x[4 * k + i] = __uint_as_float(u[i]);
                } else if constexpr (DTYPE == 1) {  // bf16: the upper half of an fp32
                    x[8 * k + 2 * i] = __uint_as_float(u[i] << 16);
                    x[8 * k + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                    x[8 * k + 2 * i] = f.x;
                    x[8 * k + 2 * i + 1] = f.y;
                }
            }
        }
    }
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

// KIND 0: keys (turned, quantised), 1: values (quantised), 2: queries (turned, stored).
template <int D, int DTYPE, int KIND>
__device__ __forceinline__ void run_kind(const Args& a, Shared<D>& sh, int chunk) {
    constexpr int LPV = D / 32, VPW = 32 / LPV;
    const QuantSide& s = a.side[KIND == 1];
    // (Not for sketched keys: the grid's boundaries lose a few bits, and a code that
    // turns over at one changes the residual and with it several of its signs:
    // a tenth of the vector, where the code alone moves it by a fiftieth.)
    const bool grid_path = KIND < 2 && s.mode == TQ_MODE_TURBO && s.grid_inv_w > 0.0f && s.m == 0;
    const int tid = threadIdx.x;
    if (grid_path && tid < 128) sh.grid[tid] = s.grid[tid];
    const int tok0 = chunk * a.chunk, ntok = min(a.chunk, a.tokens - tok0);
    const int lane = tid & 31, sub = lane % LPV, grp = lane / LPV;
    const int heads = KIND == 2 ? a.hq : a.hkv;
    const uint64_t magic = KIND == 2 ? a.hq_magic : a.hkv_magic;
    const void* src = a.src[KIND == 2 ? 2 : KIND];
    const long long stride = a.stride[KIND == 2 ? 2 : KIND];
    const uint32_t total = static_cast<uint32_t>(ntok) * heads;
    ptx::wait_prerequisites();
    ptx::launch_dependents();  // (after the wait, as the append kernel does: see quantize_side)
    // the first vectors are on their way while the table is made, and the next
    // queries while a pass's are turned
    Raw<D, DTYPE> raw;
    auto fetch = [&](uint32_t v) {
        if (v < total) {
            const uint32_t t = div_magic(v, magic), h = v - t * heads;
            raw.load(src, static_cast<size_t>(tok0 + t) * stride + static_cast<size_t>(h) * D, sub);
        }
    };
    uint32_t base = (tid / 32) * VPW;
    fetch(base + grp);
    // positions, slots, cosines and sines of the block's tokens
    if (KIND < 2 && tid < ntok) {
        const uint32_t tok = static_cast<uint32_t>(tok0 + tid), b = div_magic(tok, a.n_new_magic);
        const int t = static_cast<int>(tok - b * static_cast<uint32_t>(a.n_new));
        const int pos = a.positions[b];
        long long slot = -1;
        if (pos < 0 || pos > a.capacity - a.n_new) {
            if (KIND == 0 && a.err) atomicOr(a.err, TQ_DEVERR_POSITION);
        } else if (a.table) {
            const int at = pos + t, blk = a.table[static_cast<size_t>(b) * a.max_blocks + at / a.block_size];
            if (blk < 0 || blk >= a.num_blocks) {
                if (KIND == 0 && a.err) atomicOr(a.err, TQ_DEVERR_PAGE);
            } else {
                slot = static_cast<long long>(blk) * a.hkv * a.block_size + at % a.block_size;
            }
        } else {
            slot = static_cast<long long>(b) * a.hkv * a.capacity + pos + t;
        }
        sh.slot[tid] = slot;
    }
    if (KIND != 1) {
        const int half = a.rotary / 2;
        for (int i = tid; i < ntok * (D / 2); i += THREADS) {
            const int t = i / (D / 2), c = i % (D / 2);
            if (c < half) {
                const uint32_t tok = static_cast<uint32_t>(tok0 + t);
                const uint32_t b = div_magic(tok, a.n_new_magic);
                const long long pos = a.rope_positions ? a.rope_positions[tok]
                                                       : static_cast<long long>(a.positions[b]) + (tok - b * a.n_new);
                const long long frac = static_cast<long long>(static_cast<uint64_t>(pos) * a.turns[c]);
                float sn, cn;
                sincospif(__ll2float_rn(frac) * 0x1.0p-63f, &sn, &cn);  // (half turns)
                sh.cs[t][c] = make_float2(cn * a.magnitude, sn * a.magnitude);
            }
        }
    }
    __syncthreads();
    const uint32_t smask = KIND < 2 ? lane_sign_mask<D>(a.signs, sub) : 0u;
    const long long hstride = a.table ? a.block_size : a.capacity;  // cache rows between heads
    for (; base < total; base += WARPS * VPW) {
        const uint32_t v = base + grp;
        const bool in = v < total;
        const uint32_t t = in ? div_magic(v, magic) : 0u, h = in ? v - t * heads : 0u;
        const size_t off = static_cast<size_t>(tok0 + t) * stride + static_cast<size_t>(h) * D;
        float x[32];
        if (in) {
            raw.values(x);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 0.0f;
        }
        // (the encoders need the registers)
        if (KIND == 2 && base + WARPS * VPW < total) fetch(v + WARPS * VPW);
        if (KIND != 1 && in) turn<D, DTYPE>(a, sh.cs[t], src, off, x, sub);
        if constexpr (KIND == 2) {
            // (the output may be the input: every lane of the vector has read it before any writes)
            __syncwarp();
            if (in) {
                const size_t dst = (static_cast<size_t>(tok0 + t) * heads + h) * D;
#pragma unroll
                for (int k = 0; k < 4; ++k) store8<DTYPE>(a.q_out, dst + 8 * (sub + LPV * k), &x[8 * k]);
            }
        } else {
            const long long slot0 = in ? sh.slot[t] : -1;
            const bool valid = slot0 >= 0;
            const size_t slot = static_cast<size_t>(valid ? slot0 + h * hstride : 0);
            if (s.mode == TQ_MODE_INT8) {
                int8_encode<D>(s, x, sub, slot, valid);
            } else if (grid_path) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    x[j] = __uint_as_float(__float_as_uint(x[j]) ^ ((smask << (31 - j)) & 0x80000000u));
                if (s.bits == 4) turbo_encode_grid<D, 4>(s, sh.grid, x, sub, slot, valid);
                else if (s.bits == 3) turbo_encode_grid<D, 3>(s, sh.grid, x, sub, slot, valid);
                else turbo_encode_grid<D, 2>(s, sh.grid, x, sub, slot, valid);
            } else if (s.bits == 4) {
                turbo_encode<D, 4>(s, x, sub, slot, valid, smask);
            } else if (s.bits == 3) {
                turbo_encode<D, 3>(s, x, sub, slot, valid, smask);
            } else {
                turbo_encode<D, 2>(s, x, sub, slot, valid, smask);
            }
            if (base + WARPS * VPW < total) fetch(v + WARPS * VPW);
        }
    }
}

template <int D, int DTYPE>
__global__ void __launch_bounds__(THREADS, 3) rope_append_kernel(const __grid_constant__ Args a) {
    __shared__ Shared<D> sh;
    // (the kinds alternate: encoding is bound by instructions, turning queries by memory)
    const int kind = static_cast<int>(blockIdx.x) % a.kinds, chunk = static_cast<int>(blockIdx.x) / a.kinds;
    if (kind == 0) run_kind<D, DTYPE, 0>(a, sh, chunk);
    else if (kind == 1) run_kind<D, DTYPE, 1>(a, sh, chunk);
    else run_kind<D, DTYPE, 2>(a, sh, chunk);
}

template <int D, int DTYPE>
static cudaError_t launch(const Args& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.chunks) * a.kinds);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_append_kernel<D, DTYPE>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
static cudaError_t launch_dtype(const Args& a, int dtype, cudaStream_t stream) {
    switch (dtype) {
        case TQ_F32: return launch<D, 0>(a, stream);
        case TQ_BF16: return launch<D, 1>(a, stream);
        default: return launch<D, 2>(a, stream);
    }
}

// Tokens per block: as few as let the blocks of all three kinds run at once
// (three an SM), up to MAX_TOKENS; a block of one token leaves most of its
// warps without keys.  (464 tokens of 32 + 8 + 8 heads, the read-back that
// follows included: 18.8 us of device time with 1 a block, 11.9 us with this
// rule's 4.)
static int tokens_per_block(long long tokens, int sms) {
    int c = 1;
    while (c < MAX_TOKENS && (tokens + c - 1) / c > sms) c *= 2;
    return c;
}

static tq_status append(const tq_params* params, const tq_codebook* kcb, const tq_codebook* vcb, const tq_rope* rope,
                        const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
                        int64_t v_stride, int dtype, int32_t n_new, const int32_t* d_positions,
                        const int32_t* d_rope_positions, const tq_cache* cache, const PageMap* pm, void* q_out,
                        uint32_t* d_error, void* stream) {
    tq_status st = validate_params(params);
    if (st != TQ_OK) return st;
    const tq_params& p = *params;
    if ((st = validate_cache(p, cache)) != TQ_OK) return st;
    if (!rope || !k_new || !v_new || !d_positions || n_new < 1 || (q == nullptr) != (q_out == nullptr))
        return TQ_ERR_INVALID_ARG;
    if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16) return TQ_ERR_INVALID_ARG;
    if (rope->rotary_dims < 2 || rope->rotary_dims > p.head_dim || rope->rotary_dims % 2) return TQ_ERR_INVALID_ARG;
    if (rope->layout != TQ_ROPE_HALF && rope->layout != TQ_ROPE_INTERLEAVED) return TQ_ERR_INVALID_ARG;
    const float magnitude = static_cast<float>(rope->magnitude);
    if (!(std::isfinite(magnitude) && magnitude > 0.0f)) return TQ_ERR_INVALID_ARG;
    const long long kv_row = static_cast<long long>(p.num_kv_heads) * p.head_dim;
    const long long q_row = static_cast<long long>(p.num_q_heads) * p.head_dim;
    if (!k_stride) k_stride = kv_row;
    if (!v_stride) v_stride = kv_row;
    if (!q_stride) q_stride = q_row;
    if (k_stride < kv_row || v_stride < kv_row || q_stride < q_row) return TQ_ERR_INVALID_ARG;
    if (q && q == q_out && q_stride != q_row) return TQ_ERR_INVALID_ARG;
    const int size = dtype == TQ_F32 ? 4 : 2;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(q) || !aligned16(q_out) || k_stride * size % 16 ||
        v_stride * size % 16 || q_stride * size % 16)
        return TQ_ERR_ALIGNMENT;
    const int capacity = pm ? pm->max_blocks * pm->block_size : cache->capacity;
    if (n_new > capacity) return TQ_ERR_CAPACITY;
    if (p.k_mode == TQ_MODE_TURBO && (st = validate_codebook(kcb, p.head_dim, p.k_bits)) != TQ_OK) return st;
    if (p.v_mode == TQ_MODE_TURBO && (st = validate_codebook(vcb, p.head_dim, p.v_bits)) != TQ_OK) return st;
    const long long tokens = static_cast<long long>(pm ? pm->batch : cache->batch) * n_new;
    if (tokens > INT32_MAX / 4) return TQ_ERR_INVALID_ARG;
    const int sms = num_sms_current();
    if (sms <= 0) return TQ_ERR_CUDA;
    Args a{};
    fill_side(a.side[0], p.k_mode, p.k_bits, p.head_dim, kcb, true);
    fill_side(a.side[1], p.v_mode, p.v_bits, p.head_dim, vcb, true);
    a.side[0].codes = cache->k_codes;
    a.side[0].norms = cache->k_norms;
    a.side[0].qjl = cache->k_qjl;
    a.side[0].gamma = cache->k_gamma;
    a.side[0].sketch = cache->qjl_matrix;
    a.side[0].m = p.qjl_dims;
    a.side[1].codes = cache->v_codes;
    a.side[1].norms = cache->v_norms;
    a.src[0] = k_new;
    a.src[1] = v_new;
    a.src[2] = q;
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    a.stride[2] = q_stride;
    a.q_out = q_out;
    a.positions = d_positions;
    a.rope_positions = d_rope_positions;
    a.err = d_error;
    a.tokens = static_cast<int>(tokens);
    a.n_new = n_new;
    a.hq = p.num_q_heads;
    a.hkv = p.num_kv_heads;
    a.capacity = capacity;
    a.chunk = tokens_per_block(tokens, sms);
    a.chunks = (a.tokens + a.chunk - 1) / a.chunk;
    a.kinds = q ? 3 : 2;
    a.hq_magic = quotient_magic(static_cast<uint32_t>(p.num_q_heads));
    a.hkv_magic = quotient_magic(static_cast<uint32_t>(p.num_kv_heads));
    a.n_new_magic = quotient_magic(static_cast<uint32_t>(n_new));
    if (pm) {
        a.table = pm->table;
        a.max_blocks = pm->max_blocks;
        a.block_size = pm->block_size;
        a.num_blocks = pm->num_blocks;
    }
    a.rotary = rope->rotary_dims;
    a.layout = rope->layout;
    a.magnitude = magnitude;
    for (int i = 0; i < rope->rotary_dims / 2; ++i) a.turns[i] = rope->turns[i];
    rotation_sign_bits(p.seed, p.head_dim, a.signs);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (p.head_dim) {
        case 64: e = launch_dtype<64>(a, dtype, s); break;
        case 128: e = launch_dtype<128>(a, dtype, s); break;
        default: e = launch_dtype<256>(a, dtype, s); break;
    }
    return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace rope
}  // namespace tq

// =================================================================== C ABI
extern "C" {

tq_status tq_rope_init(int32_t rotary_dims, int32_t layout, double base, int32_t scaling, double factor, double low,
                       double high, double trained_len, double magnitude, tq_rope* out) {
    if (!out || rotary_dims < 2 || rotary_dims > 256 || rotary_dims % 2) return TQ_ERR_INVALID_ARG;
    if (layout != TQ_ROPE_HALF && layout != TQ_ROPE_INTERLEAVED) return TQ_ERR_INVALID_ARG;
    if (!(std::isfinite(base) && base > 1.0)) return TQ_ERR_INVALID_ARG;
    if (scaling < TQ_ROPE_SCALE_NONE || scaling > TQ_ROPE_SCALE_RAMP) return TQ_ERR_INVALID_ARG;
    if (!(std::isfinite(magnitude) && magnitude >= 0.0)) return TQ_ERR_INVALID_ARG;
    if (scaling != TQ_ROPE_SCALE_NONE && !(std::isfinite(factor) && factor > 0.0)) return TQ_ERR_INVALID_ARG;
    const bool banded = scaling == TQ_ROPE_SCALE_WAVELENGTH || scaling == TQ_ROPE_SCALE_RAMP;
    if (banded && !(std::isfinite(low) && std::isfinite(high) && low > 0.0 && high > low &&
                    std::isfinite(trained_len) && trained_len > 0.0))
        return TQ_ERR_INVALID_ARG;
    // The frequencies in 64-bit significands: a table entry is right to about
    // its last bit, 2^-64 of a turn, and its product with any int32 position to
    // 2^-32 (a double's would be off by 2^-25 there).
    using wide = long double;
    static_assert(std::numeric_limits<wide>::digits >= 64, "a table entry needs 64 bits");
    const double r = rotary_dims, two_pi = 2.0 * M_PI;
    const wide turn = 6.28318530717958647692528676655900577L;
    wide b = base;
    if (scaling == TQ_ROPE_SCALE_BASE && rotary_dims > 2) b *= std::pow(wide(factor), wide(r) / (r - 2.0));
    double lo = 0.0, hi = 0.0;
    if (scaling == TQ_ROPE_SCALE_RAMP) {
        // the pairs that turn `high` and `low` times within the trained length
        lo = std::fmax(0.0, std::floor(r * std::log(trained_len / (two_pi * high)) / (2.0 * std::log(base))));
        hi = std::fmin(r - 1.0, std::ceil(r * std::log(trained_len / (two_pi * low)) / (2.0 * std::log(base))));
    }
    tq_rope t{};
    t.rotary_dims = rotary_dims;
    t.layout = layout;
    t.magnitude = magnitude > 0.0 ? magnitude
                  : scaling == TQ_ROPE_SCALE_RAMP ? std::fmax(1.0, 0.1 * std::log(factor) + 1.0) : 1.0;
    for (int i = 0; i < rotary_dims / 2; ++i) {
        wide f = std::pow(b, wide(-2.0) * i / r);
        if (scaling == TQ_ROPE_SCALE_LINEAR) {
            f /= factor;
        } else if (scaling == TQ_ROPE_SCALE_WAVELENGTH) {
            const wide s = std::fmin(wide(1), std::fmax(wide(0), (trained_len * f / turn - low) / (wide(high) - low)));
            f = (1.0L - s) * f / factor + s * f;
        } else if (scaling == TQ_ROPE_SCALE_RAMP) {
            const wide s = std::fmin(wide(1), std::fmax(wide(0), wide(i - lo) / std::fmax(hi - lo, 0.001)));
            f = s * f / factor + (1.0L - s) * f;
        }
        if (!std::isfinite(static_cast<double>(f))) return TQ_ERR_INVALID_ARG;
        // turns per position, modulo one, in 2^-64ths
        wide turns = f / turn;
        turns -= std::floor(turns);
        const wide hi32 = std::floor(std::ldexp(turns, 32));
        const wide rest = std::nearbyint(std::ldexp(std::ldexp(turns, 32) - hi32, 32));
        t.turns[i] = (static_cast<uint64_t>(hi32) << 32) + static_cast<uint64_t>(rest);
    }
    *out = t;
    return TQ_OK;
}

tq_status tq_rope_append(const tq_params* params, const tq_codebook* kcb, const tq_codebook* vcb, const tq_rope* rope,
                         const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
                         int64_t v_stride, tq_dtype dtype, int32_t n_new, const int32_t* d_positions,
                         const int32_t* d_rope_positions, const tq_cache* cache, void* q_out, uint32_t* d_error,
                         void* stream) {
    return tq::rope::append(params, kcb, vcb, rope, q, q_stride, k_new, k_stride, v_new, v_stride, dtype, n_new,
                            d_positions, d_rope_positions, cache, nullptr, q_out, d_error, stream);
}

tq_status tq_rope_append_paged(const tq_params* params, const tq_codebook* kcb, const tq_codebook* vcb,
                               const tq_rope* rope, const void* q, int64_t q_stride, const void* k_new,
                               int64_t k_stride, const void* v_new, int64_t v_stride, tq_dtype dtype, int32_t n_new,
                               const int32_t* d_positions, const int32_t* d_rope_positions, const tq_cache* pool,
                               const tq_block_table* table, void* q_out, uint32_t* d_error, void* stream) {
    if (!params) return TQ_ERR_INVALID_ARG;
    tq::PageMap pm;
    const tq_status st = tq::validate_pages(*params, pool, table, &pm);
    if (st != TQ_OK) return st;
    return tq::rope::append(params, kcb, vcb, rope, q, q_stride, k_new, k_stride, v_new, v_stride, dtype, n_new,
                            d_positions, d_rope_positions, pool, &pm, q_out, d_error, stream);
}

}  // extern "C"
