// What the tree-attention kernels share: their arguments, the visibility rule,
// addresses and stores.
//
// Query row (t, g) of unit (sequence b, kv head) is draft t with head g of
// the kv head's group.  It sees the L = base[b] slots before the tree, and
// slot L + j where bit j of mask[b][t] is set and j is below the sequence's
// draft count.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "device_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tq {
namespace tree {

constexpr int MAX_DRAFTS = 64;  // bits of a mask word

struct Args {
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const uint16_t* k_norms;
    const uint16_t* v_norms;
    const uint8_t* k_qjl;
    const uint16_t* k_gamma;
    const float* sketch;
    const void* q;               // [batch][n_draft][hq][d]
    const uint64_t* mask;        // [batch][n_draft]
    const int32_t* base;         // [batch] slots before the tree
    const int32_t* draft_lens;   // [batch] or null: n_draft for all
    void* out;                   // [batch][n_draft][hq][d]
    uint32_t* err;
    float* parts;                // partial results (see the kernels)
    uint32_t* sched;             // [units + 1] (tensor-memory kernel)
    uint8_t* prep;               // prepared queries
    float* row_factor;           // [units][rows] what their scores are multiplied by (see row_exponent)
    const int32_t* table;        // paged, or null
    int max_blocks, block_size, num_blocks;
    uint64_t block_magic;        // ceil(2^64 / block_size): t / block_size is the high word of t times it
    int q_dtype, out_dtype, batch, hq, hkv, group, capacity, n_draft;
    int k_bits, v_bits, qjl_dims;  // 8 bits: an int8 side
    int staged_norms;              // rows of norms are 16-byte aligned every 8 slots
    int tok_per_tile, qtiles, units, n_split, spread;
    int wave;                             // (general kernel) blocks that run at once
    int pair, terms, part_rows;           // (tensor-memory kernel) two row blocks a unit; fp16 terms of a query; rows of a slot
    float score_scale, out_scale, key_scale;
    uint32_t signs[8];
    uint16_t kcent[16], vcent[16];  // fp16 centroids (tensor-memory kernel)
    float kcent32[16], vcent32[16];
};

// A row's softmax reference before it has seen a key: below every score, but
// finite, so that masked scores (-inf) weigh 2^-inf = 0 against it and a NaN
// score stays NaN.
constexpr float NOTHING = -0x1p127f;
// What a piece leaves as its reference: -inf marks rows without a weight.
__device__ __forceinline__ float piece_reference(float m, float l) { return m <= NOTHING && l == 0.f ? -INFINITY : m; }

// Value rows enter the products in fp16 as 2^-e times their norm, e one number
// per key tile that brings the tile's largest norm to [2^14, 2^15): norms near
// 65504 do not leave the fp16 range (int8 values enter as q / 128, turbo
// centroids below one), and small ones keep their bits (2^-e is at most 2^15,
// which makes the smallest norm fp16 holds, 2^-24, a normal number).  The
// weights take the factor back, in the exponent they are made of: a row's
// reference follows score + e, and sums of weights are counted without it.
// (Turbo values of the tensor-memory kernel: e = 0.)
constexpr int VALUE_E_MIN = -15;
__device__ __forceinline__ int value_exponent(float largest_norm) {
    return max(static_cast<int>(__float_as_uint(largest_norm) >> 23) - (127 + 14), VALUE_E_MIN);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Prepared queries are fp16 terms of 2^-k times the row, k = 0 for rows whose
// largest entry lies in [2^-2, 2^15) (entries 2^-23 of it and below are lost, no
// more than two terms hold) and else the exponent of that entry: no query is
// cut, none loses its bits.  The scores are multiplied by 2^k in fp32.
__device__ __forceinline__ int row_exponent(float largest) {
    if (!(largest > 0.f && largest < INFINITY) || (largest >= 0.25f && largest < 32768.f)) return 0;
    return min(max(static_cast<int>(__float_as_uint(largest) >> 23) - 127, -126), 126);
}

// One unit: a run of query rows of one (sequence, kv head).
struct Unit {
    int qt, kv, b, tok0, base, drafts, ntok, kend, ntiles;
    bool bad;
};

template <int BK>
__device__ __forceinline__ Unit unit_of(const Args& a, int u) {
    Unit x;
    x.qt = u % a.qtiles;
    const int bk = u / a.qtiles;
    x.kv = bk % a.hkv;
    x.b = bk / a.hkv;
    x.tok0 = x.qt * a.tok_per_tile;
    x.base = a.base[x.b];
    x.drafts = a.draft_lens ? a.draft_lens[x.b] : a.n_draft;
    x.bad = x.drafts < 0 || x.drafts > a.n_draft || x.base < 0 || x.base > a.capacity - x.drafts;
    x.ntok = x.bad ? 0 : max(0, min(a.tok_per_tile, x.drafts - x.tok0));
    x.kend = x.ntok > 0 ? x.base + x.drafts : 0;
    x.ntiles = static_cast<int>((static_cast<uint32_t>(x.kend) + BK - 1) / BK);
    return x;
}

// Visible keys of a row among slots key0 .. key0 + 63, as bits: those before
// `base`, and draft j = slot - base where bit j of m is set (m holds no bit
// at or past the draft count).
__device__ __forceinline__ uint64_t visible(uint64_t m, int key0, int base) {
    const int before = base - key0;  // slots of the tile before the tree
    if (before >= 64) return ~0ull;
    if (before >= 0) return ((1ull << before) - 1ull) | (m << before);
    return before > -64 ? m >> -before : 0ull;
}

__device__ __forceinline__ uint64_t row_mask(const Args& a, const Unit& x, int t) {
    const uint64_t m = a.mask[static_cast<size_t>(x.b) * a.n_draft + t];
    return x.drafts >= 64 ? m : m & ((1ull << x.drafts) - 1ull);
}

// Cache row (in units of one vector) of slot t of (b, kv).  An entry outside
// the pool sets TQ_DEVERR_PAGE and block 0 is read in its place.
__device__ __forceinline__ size_t cache_row(const Args& a, int b, int kv, int t) {
    if (!a.table) return (static_cast<size_t>(b) * a.hkv + kv) * a.capacity + t;
    const int page = static_cast<int>(__umul64hi(static_cast<uint64_t>(t), a.block_magic));
    int blk = a.table[static_cast<size_t>(b) * a.max_blocks + page];
    if (blk < 0 || blk >= a.num_blocks) {
        if (a.err) atomicOr(a.err, TQ_DEVERR_PAGE);
        blk = 0;
    }
    return (static_cast<size_t>(blk) * a.hkv + kv) * a.block_size + (t - page * a.block_size);
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int dtype) {
    if (dtype == TQ_F16) return ptx::pack_half2(lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// N consecutive values (N = 2, 4 or 8) in any of the three output types.
template <int N>
__device__ __forceinline__ void store_row(void* base, size_t off, const float (&e)[N], int dtype) {
    if (dtype == TQ_F32) {
        float* p = static_cast<float*>(base) + off;
#pragma unroll
        for (int i = 0; i < N; i += 2) *reinterpret_cast<float2*>(p + i) = make_float2(e[i], e[i + 1]);
    } else {
        uint32_t* p = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(base) + off);
        if constexpr (N == 2) {
            *p = pack16(e[0], e[1], dtype);
        } else if constexpr (N == 4) {
            *reinterpret_cast<uint2*>(p) = make_uint2(pack16(e[0], e[1], dtype), pack16(e[2], e[3], dtype));
        } else {
            *reinterpret_cast<uint4*>(p) = make_uint4(pack16(e[0], e[1], dtype), pack16(e[2], e[3], dtype),
                                                      pack16(e[4], e[5], dtype), pack16(e[6], e[7], dtype));
        }
    }
}

}  // namespace tree
}  // namespace tq
