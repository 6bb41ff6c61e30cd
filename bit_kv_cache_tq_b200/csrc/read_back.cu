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
    float scale[2];           // of the fp16 centroids
    int copies_log2;          // copies of a code table
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

// ------------------------------------------------- turbo vectors, no sketch
// The inverse rotation on the tensor cores: x = diag(s) H c n / sqrt(d) for 16
// vectors a warp.  H is a Kronecker product over the bits of the channel
// index, so the sum over four of them is one m16n8k16 product with a constant
// +-1 operand (16 x 16, in four registers) and the other bits are butterflies
// between a lane's own accumulators.  Channel bits, for a lane t = lane % 4:
//   0, 1  element i of the lane's four operand values
//   2     which half of the 8 codes it looked up (s)
//   3, 4  the lane t
//   5 ..  its group of 8 channels (j)
// The product runs over bits 0, 1, 3, 4; s and j are butterflies; the result's
// fragment gives lane t the channels 32 j + 8 t .. + 7, whole 16-byte stores.
// Centroids are fp16 at the codebook's scale (2^-11 at most); fp32 outputs add
// a second term with what the rounding left.  (2 x 32768 tokens x 8 heads, K4
// and V2 to bf16: 68 us, 4.6 TB/s; 132 us with all butterflies in lanes and
// shuffles, bound by issue.)
constexpr int THREADS = 256;

template <int BITS, bool LO>
struct Table {
    // Pairs of codes to pairs of fp16 centroids (and their remainders), a copy
    // for every lane: lookups of a warp never share a bank.
    uint32_t hi[1 << (2 * BITS)][32];
    uint32_t lo[LO ? 1 << (2 * BITS) : 1][32];
};

template <int D, int DTYPE, int BITS, bool TOUCH>
__device__ __forceinline__ void read_turbo(const Args& a, int side) {
    constexpr bool LO = DTYPE == 0;
    constexpr int J = D / 32;  // groups of 8 channels of a lane
    // The next tile's rows are loaded ahead where the registers allow it (d = 64:
    // 53.5 -> 51.4 us for 64000 tokens x 8 heads; d = 256: 101 -> 80 us for 32000).
    // At d = 128 that spills (77 -> 89 us for 65536 tokens): there they are only
    // touched (TOUCH, 68 us), for 16-bit outputs of a contiguous cache (a
    // table's lookup or the second term's work cost more than it gives: 87 -> 93
    // and 115 -> 127 us for 64000 tokens).
    constexpr bool AHEAD = D != 128;
    extern __shared__ __align__(16) uint8_t rb_smem[];
    Table<BITS, LO>& tab = *reinterpret_cast<Table<BITS, LO>*>(rb_smem);
    const QuantSide& s = a.side[side];
    void* out = a.out[side];
    // (blocks with little to do make four copies: their lookups may collide)
    const int copies = 1 << a.copies_log2;
    for (int i = threadIdx.x; i < copies << (2 * BITS); i += THREADS) {
        const int e = i >> a.copies_log2, l = i & (copies - 1);
        const float c0 = s.centroids[e & ((1 << BITS) - 1)] * a.scale[side], c1 = s.centroids[e >> BITS] * a.scale[side];
        const uint32_t h = ptx::pack_half2(c0, c1);
        tab.hi[e][l] = h;
        if constexpr (LO) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            tab.lo[e][l] = ptx::pack_half2(c0 - f.x, c1 - f.y);
        }
    }
    __syncthreads();
    const int b = static_cast<int>(blockIdx.x);
    const int start = a.starts[b], count = a.counts[b];
    if (start < 0 || count < 0 || count > a.max_count || start > a.capacity - count) {
        if (a.err && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(a.err, TQ_DEVERR_POSITION);
        return;
    }
    const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2, copy = lane & (copies - 1);
    // +-1 operand: row k (a lane's element: k = 2 t + i, or 2 t + 8 + i - 2),
    // column n: bit 0 of n is channel bit 0, bits 1, 2 are 3, 4, the tile is bit 1
    uint32_t hb[2][2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int kt = t, ki = 2 * q + e;  // the operand's lane and element
                const int par = __popc((kt & (g >> 1)) ^ 0) + ((ki & 1) & (g & 1)) + ((ki >> 1) & nt);
                w |= (par & 1 ? 0xBC00u : 0x3C00u) << (16 * e);
            }
            hb[nt][q] = w;
        }
    // signs of the lane's channels 32 j + 8 t + e, as bit 8 j + e
    uint32_t sg[(J + 3) / 4] = {};
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) sg[j / 4] |= sign_bit(a.signs, 32 * j + 8 * t + e) << (8 * (j % 4) + e);
    const float factor = rsqrtf(static_cast<float>(D)) / a.scale[side];
    const int runs = count / 16 + (count % 16 != 0);
    const long long tiles = static_cast<long long>(runs) * a.hkv;
    const int nwarps = gridDim.y * (THREADS / 32);
    size_t h = 0;
    int t0 = 0;
    bool ok[2];
    uint16_t nraw[2];
    uint32_t lo[2][J], hi[2][BITS == 3 ? J : 1];  // the lane's codes of group j (3 bits: in two words)
    auto touch = [&](uint32_t w) {  // the rows of such a tile to L1
        const uint32_t hw = w / static_cast<uint32_t>(runs);
        const int first = static_cast<int>(w - hw * runs) * 16;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int at = start + min(first + g + 8 * r, count - 1);
            const size_t slot = (static_cast<size_t>(b) * a.hkv + hw) * a.capacity + at;
            if (32 * t < D * BITS / 8) asm volatile("prefetch.global.L1 [%0];" ::"l"(s.codes + slot * (D * BITS / 8) + 32 * t));
            if (t == 3) asm volatile("prefetch.global.L1 [%0];" ::"l"(s.norms + slot));
        }
    };
    auto fetch = [&](uint32_t w) {  // 16 tokens of one head
        const uint32_t hw = w / static_cast<uint32_t>(runs);
        h = hw;
        t0 = static_cast<int>(w - hw * runs) * 16;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int tok = t0 + g + 8 * r;
            ok[r] = tok < count;
            size_t slot = (static_cast<size_t>(b) * a.hkv + h) * a.capacity + start + (ok[r] ? tok : 0);
            if (a.table) {
                const int at = start + (ok[r] ? tok : 0);
                const int blk = a.table[static_cast<size_t>(b) * a.max_blocks + at / a.block_size];
                if (blk < 0 || blk >= a.num_blocks) {
                    if (ok[r] && a.err && t == 0) atomicOr(a.err, TQ_DEVERR_PAGE);
                    ok[r] = false;
                }
                slot = (static_cast<size_t>(ok[r] ? blk : 0) * a.hkv + h) * a.block_size + at % a.block_size;
            }
            const uint8_t* row = s.codes + slot * (D * BITS / 8);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if constexpr (BITS == 4) {
                    lo[r][j] = __ldg(reinterpret_cast<const uint32_t*>(row) + 4 * j + t);
                } else if constexpr (BITS == 2) {
                    lo[r][j] = __ldg(reinterpret_cast<const uint16_t*>(row) + 4 * j + t);
                } else {  // 24 bits from byte 3 (4 j + t)
                    const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + 3 * j;
                    const int first = (3 * t) >> 2;
                    lo[r][j] = __ldg(p + first);
                    hi[r][j] = __ldg(p + (t == 3 ? 2 : first + (t > 0)));
                }
            }
            nraw[r] = s.norms[slot];
        }
    };
    long long w = static_cast<long long>(blockIdx.y) * (THREADS / 32) + threadIdx.x / 32;
    if (AHEAD && w < tiles) fetch(static_cast<uint32_t>(w));
    for (; w < tiles; w += nwarps) {
        if (!AHEAD) {
            fetch(static_cast<uint32_t>(w));
            if (TOUCH && w + nwarps < tiles) touch(static_cast<uint32_t>(w + nwarps));
        }
        float norm[2];
        bool live[2];
        uint32_t code[2][J];  // the 8 codes of group j, from bit 0
        size_t dst[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            live[r] = ok[r];
            norm[r] = ok[r] ? half_bits_to_float(nraw[r]) * factor : 0.f;
            dst[r] = ((static_cast<size_t>(b) * a.max_count + t0 + g + 8 * r) * a.hkv + h) * D + 8 * t;
#pragma unroll
            for (int j = 0; j < J; ++j) code[r][j] = BITS == 3 ? __funnelshift_r(lo[r][j], hi[r][BITS == 3 ? j : 0], 24 * t) : lo[r][j];
        }
        // acc[j][s]: channels 32 j + 8 t' + 4 s + .. before the butterflies
        float acc[J][2][2][4];
        constexpr uint32_t M = (1u << (2 * BITS)) - 1u;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int sx = 0; sx < 2; ++sx) {
                // (rows g and g + 8) x (codes 0, 1 and 2, 3 of the half)
                uint32_t f[4];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    f[q] = (code[q][j] >> (4 * BITS * sx)) & M;
                    f[2 + q] = (code[q][j] >> (4 * BITS * sx + 2 * BITS)) & M;
                }
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[j][sx][nt][q] = 0.f;
                {
                    const uint32_t x0 = tab.hi[f[0]][copy], x1 = tab.hi[f[1]][copy], x2 = tab.hi[f[2]][copy],
                                   x3 = tab.hi[f[3]][copy];
                    ptx::mma_16816(acc[j][sx][0], x0, x1, x2, x3, hb[0][0], hb[0][1]);
                    ptx::mma_16816(acc[j][sx][1], x0, x1, x2, x3, hb[1][0], hb[1][1]);
                }
                if constexpr (LO) {
                    const uint32_t x0 = tab.lo[f[0]][copy], x1 = tab.lo[f[1]][copy], x2 = tab.lo[f[2]][copy],
                                   x3 = tab.lo[f[3]][copy];
                    ptx::mma_16816(acc[j][sx][0], x0, x1, x2, x3, hb[0][0], hb[0][1]);
                    ptx::mma_16816(acc[j][sx][1], x0, x1, x2, x3, hb[1][0], hb[1][1]);
                }
            }
        // the next tile's rows are on their way during the butterflies and the stores
        if (AHEAD && w + nwarps < tiles) fetch(static_cast<uint32_t>(w + nwarps));
        // butterflies over s and the bits of j
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
                float2 v[2 * J];
#pragma unroll
                for (int k = 0; k < 2 * J; ++k) v[k] = make_float2(acc[k >> 1][k & 1][nt][q], acc[k >> 1][k & 1][nt][q + 1]);
#pragma unroll
                for (int m = 1; m < 2 * J; m <<= 1)
#pragma unroll
                    for (int k = 0; k < 2 * J; ++k)
                        if (!(k & m)) {
                            const float2 x = v[k], y = v[k + m];
                            v[k] = ptx::fadd2(x, y);
                            v[k + m] = ptx::fsub2(x, y);
                        }
#pragma unroll
                for (int k = 0; k < 2 * J; ++k) {
                    acc[k >> 1][k & 1][nt][q] = v[k].x;
                    acc[k >> 1][k & 1][nt][q + 1] = v[k].y;
                }
            }
        // lane t of row g + 8 r: channels 32 j + 8 t + (4 s + 2 nt + e)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = flip_sign(acc[j][e >> 2][(e >> 1) & 1][2 * r + (e & 1)] * norm[r],
                                     (sg[j / 4] >> (8 * (j % 4) + e)) & 1u);
                if (live[r]) store8<DTYPE>(out, dst[r] + 32 * j, x);
            }
        }
    }
}

// ------------------------------------------- int8 sides and sketched keys
// A vector on d/32 lanes, as the encoders.  (2 x 32768 tokens x 8 heads to bf16,
// d = 128: both sides int8 124 us, bound by its chain of loads with nothing ahead;
// keys with 64 sketch rows 767 us alone, 64 x 32 scalar multiply-adds a lane.  The
// tensor-core path takes 73 for both sides.)
template <int D, int DTYPE>
__device__ __forceinline__ void read_other(const Args& a, int side) {
    constexpr int LPV = D / 32, VPW = 32 / LPV;
    const QuantSide& s = a.side[side];
    void* out = a.out[side];
    __shared__ float scen[16];
    if (threadIdx.x < 16) scen[threadIdx.x] = s.centroids[threadIdx.x];
    __syncthreads();
    const int b = static_cast<int>(blockIdx.x);
    const int start = a.starts[b], count = a.counts[b];
    if (start < 0 || count < 0 || count > a.max_count || start > a.capacity - count) {
        if (a.err && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(a.err, TQ_DEVERR_POSITION);
        return;
    }
    const int lane = threadIdx.x & 31, sub = lane % LPV, grp = lane / LPV;
    const long long total = static_cast<long long>(count) * a.hkv;
    const long long nwarps = static_cast<long long>(gridDim.y) * (blockDim.x / 32);
    for (long long base = (static_cast<long long>(blockIdx.y) * (blockDim.x / 32) + threadIdx.x / 32) * VPW;
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

// Grid: (batch, blocks of a sequence, side).
// TOUCH: see read_turbo.
template <int D, int DTYPE, bool TOUCH>
__global__ void __launch_bounds__(THREADS, D == 256 ? 1 : 2) read_back_kernel(const __grid_constant__ Args a) {
    const int side = static_cast<int>(blockIdx.z);
    const QuantSide& s = a.side[side];
    if (!a.out[side]) return;
    if (s.mode != TQ_MODE_TURBO || s.m > 0) read_other<D, DTYPE>(a, side);
    else if (s.bits == 4) read_turbo<D, DTYPE, 4, TOUCH>(a, side);
    else if (s.bits == 3) read_turbo<D, DTYPE, 3, TOUCH>(a, side);
    else read_turbo<D, DTYPE, 2, TOUCH>(a, side);
}

template <int D, int DTYPE>
static cudaError_t launch_typed(Args& a, int sms, cudaStream_t s) {
    int bytes = 0;
    for (int side = 0; side < 2; ++side) {
        const QuantSide& q = a.side[side];
        if (!a.out[side] || q.mode != TQ_MODE_TURBO || q.m > 0) continue;
        const int n = static_cast<int>(q.bits == 4   ? sizeof(Table<4, DTYPE == 0>)
                                       : q.bits == 3 ? sizeof(Table<3, DTYPE == 0>)
                                                     : sizeof(Table<2, DTYPE == 0>));
        if (n > bytes) bytes = n;
    }
    // (the largest table's for every call: another thread's call may set it between this line and the launch)
    auto kernel = read_back_kernel<D, DTYPE, false>;
    if constexpr (D == 128 && DTYPE != 0)
        if (!a.table) kernel = read_back_kernel<D, DTYPE, true>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(sizeof(Table<4, DTYPE == 0>)));
    if (e != cudaSuccess) return e;
    // eight warps a block and 16 vectors a warp, two blocks an SM and side, shared by the sequences
    const long long want = ((a.max_count / 16 + 1ll) * a.hkv + 7) / 8;
    const long long most = (2ll * sms + a.batch - 1) / a.batch;
    const dim3 grid(static_cast<unsigned>(a.batch), static_cast<unsigned>(want < most ? want : most), 2);
    a.copies_log2 = want <= most ? 2 : 5;
    kernel<<<grid, THREADS, bytes, s>>>(a);
    return cudaGetLastError();
}

template <int D>
static cudaError_t launch(Args& a, int dtype, int sms, cudaStream_t s) {
    switch (dtype) {
        case TQ_F32: return launch_typed<D, 0>(a, sms, s);
        case TQ_BF16: return launch_typed<D, 1>(a, sms, s);
        default: return launch_typed<D, 2>(a, sms, s);
    }
}

// One side's kernel arguments (no code grid: nothing is encoded here).
static void fill(QuantSide& s, float& scale, int mode, int bits, int d, const tq_codebook* cb) {
    s.mode = mode;
    s.bits = mode == TQ_MODE_INT8 ? 8 : bits;
    s.vbytes = vector_bytes(mode, bits, d);
    if (mode != TQ_MODE_TURBO) return;
    for (int j = 0; j < 1 << bits; ++j) s.centroids[j] = static_cast<float>(cb->centroids[j]);
    scale = static_cast<float>(cb->fp16_scale > 0.0 ? cb->fp16_scale : std::sqrt(static_cast<double>(d)));
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
    if (k_out) fill(a.side[0], a.scale[0], p.k_mode, p.k_bits, p.head_dim, kcb);
    if (v_out) fill(a.side[1], a.scale[1], p.v_mode, p.v_bits, p.head_dim, vcb);
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
    rotation_sign_bits(p.seed, p.head_dim, a.signs);
    const int sms = num_sms_current();
    if (sms <= 0) return TQ_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (p.head_dim) {
        case 64: e = launch<64>(a, dtype, sms, s); break;
        case 128: e = launch<128>(a, dtype, sms, s); break;
        default: e = launch<256>(a, dtype, sms, s); break;
    }
    return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
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
