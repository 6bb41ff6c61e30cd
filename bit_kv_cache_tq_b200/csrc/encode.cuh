// The encoding of one head vector (turbo codes, QJL sketch, int8) as device
// code, shared by the kernels that write the cache: quantise-append and the
// rotary append.
//
// Work layout: a head vector of d coordinates is held by d/32 lanes, 32
// coordinates each.  The vector is read as 16-byte chunks of 8 elements;
// lane j of the vector's lane group holds chunks j, j + d/32, j + 2d/32,
// j + 3d/32, so every load instruction of a warp covers whole 32-byte
// sectors.  The Walsh-Hadamard transform then runs 5 butterfly stages in
// registers and log2(d/32) stages across lanes (warp shuffles).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "device_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tq {

struct QuantSide {
    const void* src;        // [batch][n_new][Hkv][d]
    uint8_t* codes;         // [batch][Hkv][capacity][vbytes]
    uint16_t* norms;        // [batch][Hkv][capacity]
    uint8_t* qjl;           // [batch][Hkv][capacity][m/8] or null
    uint16_t* gamma;        // [batch][Hkv][capacity] or null
    const float* sketch;    // [m][d] or null
    int mode, bits, vbytes, m;
    float centroids[16];
    float pos_boundaries[8];  // boundaries above zero, ascending (2^(bits-1) - 1 of them)
    // Code grid (turbo mode; grid_inv_w = 0 when the table cannot hold the
    // codebook): the rotated unit coordinate y is cut into cells of width w
    // (no wider than the narrowest code cell, so a grid cell holds at most one
    // boundary), cell c = round(y / w) covering [(c - 0.5) w, (c + 0.5) w).
    // Entry c & 127 is the fp32 bit pattern of the boundary inside the cell,
    // in cells, with its 4 low mantissa bits replaced by the number of
    // boundaries below the cell (the boundary moves by at most 15 ulps); a
    // cell without a boundary holds +inf's pattern, a NaN once those bits are
    // set, so it never compares below y.  The code of y is the count plus
    // (y / w > the boundary).  |y| <= 1 keeps c within +-63.
    float grid_inv_w;
    uint32_t grid[128];
};

template <int BITS>
__device__ __forceinline__ void store_chunk_codes(uint8_t* row, int chunk, uint32_t packed) {
    if constexpr (BITS == 4) {
        *reinterpret_cast<uint32_t*>(row + 4 * chunk) = packed;
    } else if constexpr (BITS == 2) {
        *reinterpret_cast<uint16_t*>(row + 2 * chunk) = static_cast<uint16_t>(packed);
    } else {
        row[3 * chunk] = static_cast<uint8_t>(packed);
        row[3 * chunk + 1] = static_cast<uint8_t>(packed >> 8);
        row[3 * chunk + 2] = static_cast<uint8_t>(packed >> 16);
    }
}

// Code of the rotated coordinate x = y * sqrt(d) * ||x|| against the
// boundaries scaled the same way (ts[k] = t_k sqrt(d) ||x||, ascending): the
// count of boundaries below y, found with a binary search over the positive
// half (the table is odd-symmetric, its middle boundary is 0).  Deciding on x
// against scaled boundaries instead of on y = x / (sqrt(d) ||x||) moves a
// decision only when y is within a few ulp of a boundary.
template <int BITS>
__device__ __forceinline__ uint32_t code_scaled(float x, const float (&ts)[7]) {
    constexpr int half = 1 << (BITS - 1);
    const float a = fabsf(x);
    int m;
    if constexpr (BITS == 4) {
        const bool p2 = a > ts[3];
        const bool p1 = a > (p2 ? ts[5] : ts[1]);
        const float w = p1 ? (p2 ? ts[6] : ts[2]) : (p2 ? ts[4] : ts[0]);
        m = 4 * p2 + 2 * p1 + (a > w);
    } else if constexpr (BITS == 3) {
        const bool p1 = a > ts[1];
        m = 2 * p1 + (a > (p1 ? ts[2] : ts[0]));
    } else {
        m = a > ts[0];
    }
    return x > 0.0f ? static_cast<uint32_t>(half + m) : static_cast<uint32_t>(half - 1 - m);
}

// n / d for n < 2^32 as the high word of n * M, M = ceil(2^64 / d) (exact:
// the product overshoots n / d by less than n / 2^64 < 1 / d); M = 0 stands
// for d = 1.
__device__ __forceinline__ uint32_t div_magic(uint32_t n, uint64_t m) {
    return m == 0 ? n : static_cast<uint32_t>(__umul64hi(static_cast<uint64_t>(n), m));
}

// Walsh-Hadamard butterflies over a lane's 32 values, the stages of span 2
// and more as packed fp32 pairs (the same additions, in the same order).
__device__ __forceinline__ void fwht32_pairs(float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float a = v[i], b = v[i + 1];
        v[i] = a + b;
        v[i + 1] = a - b;
    }
#pragma unroll
    for (int h = 2; h < 32; h <<= 1)
#pragma unroll
        for (int i = 0; i < 32; i += 2)
            if (!(i & h)) {
                const float2 a = make_float2(v[i], v[i + 1]), b = make_float2(v[i + h], v[i + h + 1]);
                const float2 s = ptx::fadd2(a, b), d = ptx::fsub2(a, b);
                v[i] = s.x;
                v[i + 1] = s.y;
                v[i + h] = d.x;
                v[i + h + 1] = d.y;
            }
}

// fwht_lanes with the fused multiply-adds in packed pairs.
template <int SPAN>
__device__ __forceinline__ void fwht_lanes_pairs(float (&v)[32], int sub) {
#pragma unroll
    for (int m = 1; m < SPAN; m <<= 1) {
        const float sg = (sub & m) ? -1.0f : 1.0f;  // upper lane: p - v, lower lane: v + p
        const float2 sg2 = make_float2(sg, sg);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float2 p = make_float2(__shfl_xor_sync(kFullMask, v[i], m), __shfl_xor_sync(kFullMask, v[i + 1], m));
            const float2 r = ptx::ffma2(make_float2(v[i], v[i + 1]), sg2, p);
            v[i] = r.x;
            v[i + 1] = r.y;
        }
    }
}

// Turbo encode through the code grid (shared copy `grid`); x holds the
// lane's 32 coordinates with the rotation signs already applied.
template <int D, int BITS>
__device__ __forceinline__ void turbo_encode_grid(const QuantSide& s, const uint32_t* grid, float (&x)[32], int sub,
                                                  size_t slot, bool valid) {
    constexpr int LPV = D / 32;
    float sumsq = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) sumsq = fmaf(x[j], x[j], sumsq);
    fwht32_pairs(x);
    fwht_lanes_pairs<LPV>(x, sub);
    sumsq = group_sum<LPV>(sumsq);
    const float n = sqrtf(sumsq);
    const float scale = sqrtf(static_cast<float>(D)) * n;  // y_i = x_i / scale
    const float inv = n > 0.0f ? s.grid_inv_w / scale : 0.0f;  // grid cells per unit of x
    uint32_t packed[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t acc = 0;
#pragma unroll
        for (int e = 7; e >= 0; --e) {
            const float g = x[8 * k + e] * inv;
            // round(g) in the low mantissa bits of g + 1.5 * 2^23 (|g| < 64)
            const uint32_t cell = grid[__float_as_uint(g + 12582912.0f) & 127u];
            const uint32_t code = (cell & ((1u << BITS) - 1u)) + (g > __uint_as_float(cell) ? 1u : 0u);
            acc = acc * (1u << BITS) + code;
        }
        packed[k] = acc;
    }
    if (valid) {
        uint8_t* row = s.codes + slot * static_cast<size_t>(s.vbytes);
#pragma unroll
        for (int k = 0; k < 4; ++k) store_chunk_codes<BITS>(row, sub + LPV * k, packed[k]);
        if (sub == 0) s.norms[slot] = float_to_half_bits(n);
    }
    if (s.m > 0) {  // QJL residual sketch (keys only)
        const float rinv = n > 0.0f ? 1.0f / scale : 0.0f;
        float g2 = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t code = (packed[i >> 3] >> (BITS * (i & 7))) & ((1u << BITS) - 1u);
            x[i] = x[i] * rinv - s.centroids[code];  // residual r_i = y_i - c[code_i]
            g2 = fmaf(x[i], x[i], g2);
        }
        g2 = group_sum<LPV>(g2);
        uint32_t word = 0;
        for (int r = 0; r < s.m; ++r) {
            const float* row = s.sketch + static_cast<size_t>(r) * D;
            float acc = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 a = __ldg(reinterpret_cast<const float4*>(row + 8 * (sub + LPV * k)));
                const float4 b = __ldg(reinterpret_cast<const float4*>(row + 8 * (sub + LPV * k) + 4));
                acc = fmaf(a.x, x[8 * k + 0], acc); acc = fmaf(a.y, x[8 * k + 1], acc);
                acc = fmaf(a.z, x[8 * k + 2], acc); acc = fmaf(a.w, x[8 * k + 3], acc);
                acc = fmaf(b.x, x[8 * k + 4], acc); acc = fmaf(b.y, x[8 * k + 5], acc);
                acc = fmaf(b.z, x[8 * k + 6], acc); acc = fmaf(b.w, x[8 * k + 7], acc);
            }
            acc = group_sum<LPV>(acc);
            word |= static_cast<uint32_t>(acc >= 0.0f) << (r & 31);
            if ((r & 31) == 31) {
                if (valid && sub == 0)
                    reinterpret_cast<uint32_t*>(s.qjl + slot * static_cast<size_t>(s.m / 8))[r >> 5] = word;
                word = 0;
            }
        }
        if (valid && sub == 0) s.gamma[slot] = float_to_half_bits(sqrtf(g2));
    }
}

// Rotation signs of this lane's 32 coordinates 8 (sub + LPV k) + e, as bit
// 8 k + e of one word (built once per thread).
template <int D>
__device__ __forceinline__ uint32_t lane_sign_mask(const uint32_t* signs, int sub) {
    constexpr int LPV = D / 32;
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i0 = 8 * (sub + LPV * k);
        m |= ((signs[i0 >> 5] >> (i0 & 31)) & 0xFFu) << (8 * k);
    }
    return m;
}

template <int D, int BITS>
__device__ __forceinline__ void turbo_encode(const QuantSide& s, float (&x)[32], int sub, size_t slot, bool valid,
                                             uint32_t smask) {
    constexpr int LPV = D / 32;
    float sumsq = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        sumsq = fmaf(x[j], x[j], sumsq);
        x[j] = __uint_as_float(__float_as_uint(x[j]) ^ ((smask << (31 - j)) & 0x80000000u));
    }
    fwht_registers(x);
    fwht_lanes<32, LPV>(x, sub);
    sumsq = group_sum<LPV>(sumsq);
    const float n = sqrtf(sumsq);
    const float scale = sqrtf(static_cast<float>(D)) * n;  // y_i = x_i / scale
    float ts[7];
#pragma unroll
    for (int k = 0; k < 7; ++k) ts[k] = s.pos_boundaries[k] * scale;
    uint32_t codes[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) codes[i] = code_scaled<BITS>(x[i], ts);
    if (valid) {
        uint8_t* row = s.codes + slot * static_cast<size_t>(s.vbytes);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t packed = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) packed |= codes[8 * k + e] << (BITS * e);
            store_chunk_codes<BITS>(row, sub + LPV * k, packed);
        }
        if (sub == 0) s.norms[slot] = float_to_half_bits(n);
    }
    if (s.m > 0) {  // QJL residual sketch (keys only)
        const float inv = n > 0.0f ? 1.0f / scale : 0.0f;
        float g2 = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            x[i] = x[i] * inv - s.centroids[codes[i]];  // residual r_i = y_i - c[code_i]
            g2 = fmaf(x[i], x[i], g2);
        }
        g2 = group_sum<LPV>(g2);
        uint32_t word = 0;
        for (int r = 0; r < s.m; ++r) {
            const float* row = s.sketch + static_cast<size_t>(r) * D;
            float acc = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 a = __ldg(reinterpret_cast<const float4*>(row + 8 * (sub + LPV * k)));
                const float4 b = __ldg(reinterpret_cast<const float4*>(row + 8 * (sub + LPV * k) + 4));
                acc = fmaf(a.x, x[8 * k + 0], acc); acc = fmaf(a.y, x[8 * k + 1], acc);
                acc = fmaf(a.z, x[8 * k + 2], acc); acc = fmaf(a.w, x[8 * k + 3], acc);
                acc = fmaf(b.x, x[8 * k + 4], acc); acc = fmaf(b.y, x[8 * k + 5], acc);
                acc = fmaf(b.z, x[8 * k + 6], acc); acc = fmaf(b.w, x[8 * k + 7], acc);
            }
            acc = group_sum<LPV>(acc);
            word |= static_cast<uint32_t>(acc >= 0.0f) << (r & 31);
            if ((r & 31) == 31) {
                if (valid && sub == 0)
                    reinterpret_cast<uint32_t*>(s.qjl + slot * static_cast<size_t>(s.m / 8))[r >> 5] = word;
                word = 0;
            }
        }
        if (valid && sub == 0) s.gamma[slot] = float_to_half_bits(sqrtf(g2));
    }
}

template <int D>
__device__ __forceinline__ void int8_encode(const QuantSide& s, const float (&x)[32], int sub, size_t slot,
                                            bool valid) {
    constexpr int LPV = D / 32;
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = group_max<LPV>(amax);
    const __half scale16 = __float2half_rn(__fdiv_rn(amax, 127.0f));
    const float scale = __half2float(scale16);
    const float recip = (scale > 0.0f && scale < INFINITY) ? __frcp_rn(scale) : 0.0f;
    if (!valid) return;
    uint8_t* row = s.codes + slot * static_cast<size_t>(D);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = fminf(fmaxf(rintf(__fmul_rn(x[8 * k + e], recip)), -127.0f), 127.0f);
            const uint32_t byte = static_cast<uint32_t>(static_cast<int32_t>(q)) & 0xffu;
            if (e < 4) lo |= byte << (8 * e);
            else hi |= byte << (8 * (e - 4));
        }
        *reinterpret_cast<uint2*>(row + 8 * (sub + LPV * k)) = make_uint2(lo, hi);
    }
    if (sub == 0) s.norms[slot] = __half_as_ushort(scale16);
}

// Host: one side of the kernel arguments from its mode, width and codebook.
// tight: a grid cell gives up only the bits its code takes and rounds its
// boundary to the nearest such pattern (off by at most 2, 4 or 8 ulp at 2, 3 and
// 4 bits; by up to 15 otherwise).
inline void fill_side(QuantSide& s, int mode, int bits, int d, const tq_codebook* cb, bool tight = false) {
    s.mode = mode;
    s.bits = mode == TQ_MODE_INT8 ? 8 : bits;
    s.vbytes = vector_bytes(mode, bits, d);
    for (int j = 0; j < 16; ++j) s.centroids[j] = 0.0f;
    for (int j = 0; j < 8; ++j) s.pos_boundaries[j] = INFINITY;
    s.grid_inv_w = 0.0f;
    if (mode == TQ_MODE_TURBO) {
        const int n = 1 << bits, half = n / 2;
        for (int j = 0; j < n; ++j) s.centroids[j] = static_cast<float>(cb->centroids[j]);
        for (int k = 0; k < half - 1; ++k) s.pos_boundaries[k] = static_cast<float>(cb->boundaries[half + k]);
        // the code grid: cells no wider than the narrowest code cell; used
        // only when |y| <= 1 stays within 62.5 cells of zero (else the binary
        // search below serves)
        double w = INFINITY;
        for (int j = 0; j + 1 < n - 1; ++j) w = std::min(w, cb->boundaries[j + 1] - cb->boundaries[j]);
        if (n == 2) w = 1.0;  // (not a width the codebooks produce: one boundary, at zero)
        w *= 1.0 - 1e-6;
        bool ok = 1.0 / w < 62.5;
        for (int c = -64, j = 0; ok && c < 64; ++c) {  // (cells and boundaries ascend together)
            const double lo = (c - 0.5) * w, hi = (c + 0.5) * w;
            while (j < n - 1 && cb->boundaries[j] < lo) ++j;
            const uint32_t below = static_cast<uint32_t>(j);
            const bool inside = j < n - 1 && cb->boundaries[j] < hi;
            if (inside && j + 1 < n - 1 && cb->boundaries[j + 1] < hi) ok = false;  // two boundaries in a cell
            const float bnd = inside ? static_cast<float>(cb->boundaries[j] / w) : INFINITY;
            uint32_t bits32;
            std::memcpy(&bits32, &bnd, 4);
            const uint32_t field = tight ? static_cast<uint32_t>(n) : 16u;
            uint32_t cell = (bits32 & ~(field - 1u)) | below;
            if (tight && inside) {
                if (cell + field / 2 < bits32) cell += field;
                else if (cell > bits32 + field / 2 && cell >= field) cell -= field;
            }
            s.grid[c & 127] = cell;
        }
        if (ok) s.grid_inv_w = static_cast<float>(1.0 / w);
    }
}

// ceil(2^64 / d) for the quotients of div_magic; 0 for d = 1.
inline uint64_t quotient_magic(uint32_t d) { return d <= 1 ? 0 : UINT64_MAX / d + 1; }

}  // namespace tq
