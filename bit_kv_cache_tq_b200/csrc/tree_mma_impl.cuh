// Tree attention on the 5th-generation tensor cores: d = 128, turbo or int8
// keys and values without a sketch.
//
// The work is a sequence of key tiles (64 slots) of units (sequence, kv head,
// up to 128 query rows); every block takes an equal run of it, so a unit may
// be cut between blocks, whose pieces the merge kernel joins.
//
// A block runs two streams of online softmax, each with its own scores,
// reference, sum and output accumulator in tensor memory; while one stream's
// softmax runs, the tensor cores work for the other.  Units of up to 128 rows:
// the tiles alternate between the streams, which are joined at the end of a
// unit's run (a row's two accumulators lie in one tensor-memory lane).  Units
// of up to 256 rows (`pair`): each stream has half of the rows and both read
// every tile, so a dequantised tile serves twice the rows.
//
// Queries enter as fp16 terms (a.terms): two for fp16 and fp32 outputs, so
// that a score keeps about 22 bits of its query; one for bf16 outputs, whose
// rounding (2^-8) hides that of the queries (2^-11 of each coordinate).  The
// second term's tensor memory then holds the second row block's queries (pair)
// or the weights, which otherwise overwrite the scores (overlay) and hold the
// stream's next scores back until they are used.
//
// The queries come from a small kernel before this one (tree_prep_kernel):
// rotated once, scaled, as fp16 terms in the order a block's threads load them.
//
// Roles (20 warps):
//  * producer (1 warp): bulk copies of packed codes and norms into a ring (and
//    2 warps that load the norms where a cache's rows of norms are not 16-byte
//    aligned);
//  * dequantisers (8 warps): codes to fp16 operand tiles (128-byte swizzle),
//    keys (a tile ahead of values) as centroids, values as centroids times
//    norms (int8: see value_exponent; turbo values keep one factor, at which a
//    norm of 65504 fits fp16 and rounding adds at most 2^-26 to a coordinate,
//    which shows in rows of values whose norms are below 2^-13.  An exponent for
//    each tile costs time in the dequantisers, which nothing hides: 113 -> 121 us
//    for 16 sequences of 2048 to 8192 tokens, 13 drafts, K3/V2);
//  * MMA issuer (1 warp): S = (Qhi + Qlo) K~^T (M = 128, N = 64, K = 128) and O += P V~
//    (M = 128, N = 128, K = 64), the queries and the weights as A operands in
//    tensor memory;
//  * softmax (2 x 4 warps, one query row a thread): the queries are scaled by
//    the softmax scale (log2 units), so a weight is 2^(S n - reference), n the
//    key's norm (int8 values: 2^(S n + e - reference), e the exponent of the
//    tile's values).  There is no pass for the maximum: a row's reference is
//    raised only when the tile's sum of weights shows that one of them may pass
//    the fp16 range (always on a stream's first tile), and the tile is then done
//    again.
//
// What bounds it is the shared-memory and tensor-memory data path: a tile of
// 64 keys moves, in 128-byte passes, 256 for the scores, 128 for the weights
// and 128 for the norms of every 128 rows, and 256 for the operand tiles, 256
// for the table lookups and 100 for codes once; hence the pairing of row
// blocks.  (The norm inside K~ would save the norms' passes, but its fp16
// rounding grows with the scores: 6e-3 of a row's output at score deviations
// of ten.)  A pair of row blocks takes about 3400 cycles a tile, of which the
// tensor cores work 1020: the chain scores, softmax, weights, P V of a stream
// is longer than the other stream can cover.  64 drafts of 32 heads over 32768
// tokens (K4/V2, 8 kv heads, bf16): 89 us, 385 TFLOP/s; 16 sequences of 2048 to
// 8192 tokens in pages, 13 drafts each (K3/V2): 113 us; 2 x 131072 tokens, 25
// drafts of 64 heads (K4/V4, fp16, two terms): 507 to 516 us.
// Units of few rows are bound elsewhere: with 52 rows a stream's softmax is two
// warps, and both streams' are on the same two of the SM's four sub-partitions
// (the busiest one issues 2.5 times the instructions of the idlest, 39% of the
// slots on average), at 2700 cycles a tile of which the MMAs, half of their rows
// empty, take 600.
//
// What is rounded to fp16, and why that is enough: the key table (at the scale
// that rounds it best, 6e-5 of an entry), a value row (table times norm, 2^-12.3
// rms), a weight (the same), the queries in one or two terms.  Products and sums
// are fp32.  Together 4.5e-4 of a row over 131072 tokens, fp16 outputs' own
// rounding of 2.1e-4 included.
//
// Every mbarrier wait is bounded (about a second, then TQ_DEVERR_TIMEOUT; the
// block stops issuing copies and MMAs, waits for those under way, and its other
// warps run to the end of their tiles without waiting).
#pragma once

#include <type_traits>

#include "tcgen05.cuh"
#include "tree_common.cuh"

namespace tq {
namespace tree {
namespace mma {

constexpr int D = 128, BM = 128, BK = 64, NS = 4;
constexpr int SOFTMAX_WARPS = 8, DEQ_WARPS = 8;
constexpr int DEQ0 = SOFTMAX_WARPS * 32, LIGHT0 = DEQ0 + DEQ_WARPS * 32;
constexpr int PRODUCER_WARP = LIGHT0 / 32, MMA_WARP = PRODUCER_WARP + 1, NORM_WARP = MMA_WARP + 1;
constexpr int NTHREADS = LIGHT0 + 128;
// Registers a thread: launched at 96, the dequantisers and the last warpgroup
// give up what the softmax warpgroups take (32 scores, 32 packed weights and the
// loads ahead: fewer spill).
constexpr int REGS_LAUNCH = 96, REGS_SOFTMAX = 136, REGS_DEQ = 64, REGS_LIGHT = 72;
static_assert(SOFTMAX_WARPS * 32 * REGS_SOFTMAX + DEQ_WARPS * 32 * REGS_DEQ + 128 * REGS_LIGHT <=
                  NTHREADS * REGS_LAUNCH,
              "the register split draws on what the block was launched with");
// tensor-memory columns (32-bit; fp16 operands take two elements a column)
constexpr uint32_t TM_Q = 0;     // scaled queries, fp16 [128][128]; then their second term, or (pair) the second row
                                 // block's, or the weights, 2 x fp16 [128][64]
constexpr uint32_t TM_S = 128;   // 2 x fp32 scores [128][64]; (overlay) the weights over their first half
constexpr uint32_t TM_O = 256;   // 2 x fp32 accumulators [128][128]
constexpr uint32_t TMEM_COLS = 512;
constexpr long long WAIT_LIMIT = 2000000000ll;  // clock cycles (~1 s)
// Weights are 2^(s + e - reference + WSHIFT): 2^6 for a score at the reference,
// normal fp16 numbers down to 2^-20 of that.  The reference moves when a
// tile's sum passes WLIMIT, below which no single weight leaves the fp16 range.
constexpr float WSHIFT = 6.0f, WLIMIT = 32768.0f, WMOST = 15.5f;
// The key table is 2^-8 of the codebook's fp16 scale (int8 keys: q / 128), so
// that ordinary queries, which carry the inverse, need no factor of their own.
constexpr double KEY_SHIFT = 1.0 / 256.0;

// Prepared queries of a unit: per fp16 term, 16 chunks of 8 channels of every
// row, the rows of a chunk next to each other.
__host__ __device__ constexpr size_t prep_bytes(int rows, int terms) { return static_cast<size_t>(rows) * D * 2 * terms; }

__host__ __device__ constexpr int row_bytes(int bits) { return bits == 8 ? D : D * bits / 8; }
// Shared memory (offsets from a 1024-byte aligned base).
__host__ __device__ constexpr uint32_t lut_bytes(int bits) { return bits == 8 ? 0u : 32u * 4u * (1u << (2 * bits)); }
// A lookup address is made of the code word by a shift and one logic
// operation (the field in bits 7 and up, the lane's offset below), or, for
// 4-bit keys, whose table has 256-byte rows, by one byte permute; the load's
// immediate offset holds the table's shared-window address (dynamic shared
// memory begins at window address SMEM_WINDOW, which the host checks).
constexpr uint32_t SMEM_WINDOW = 1024;
__host__ __device__ constexpr bool wide(int kb) { return kb == 4; }
__host__ __device__ constexpr uint32_t klut_bytes(int kb) { return wide(kb) ? 65536u : lut_bytes(kb); }
constexpr int SCHED_MAX = 4096;                             // most units the shared schedule holds
constexpr uint32_t SM_K = 0;                                // 2 x fp16 K~ [64][128]
constexpr uint32_t SM_V = SM_K + 2 * BK * D * 2;            // 2 x fp16 V~ [64][128]
constexpr uint32_t SM_KNR = SM_V + 2 * BK * D * 2;          // fp16 key norms of the last four tiles
constexpr uint32_t SM_ML = SM_KNR + 4 * BK * 2;             // float [2][2][2][128]: the streams' references and sums
constexpr uint32_t SM_CENT = SM_ML + 8 * BM * 4;            // fp16 centroids, keys then values
constexpr uint32_t SM_VEXP = SM_CENT + 64;                  // (int8 values) float2 (e, 2^-e) of the last four tiles
constexpr uint32_t SM_FACTOR = SM_VEXP + 4 * 8;             // float [256]: the softmax threads' row factors
constexpr uint32_t SM_BAR = SM_FACTOR + SOFTMAX_WARPS * 32 * 4;
constexpr int B_FULL = 0, B_EMPTY = NS, B_KFULL = 2 * NS, B_KEMPTY = B_KFULL + 2, B_VFULL = B_KEMPTY + 2,
              B_VEMPTY = B_VFULL + 2, B_PV = B_VEMPTY + 2, B_SFULL = B_PV + 2, B_SEMPTY = B_SFULL + 2, B_PFULL = B_SEMPTY + 2, B_QREADY = B_PFULL + 2,
              B_FINAL = B_QREADY + 1, NBARS = B_FINAL + 1;
constexpr uint32_t SM_TMEM = SM_BAR + NBARS * 8;
constexpr uint32_t SM_FLAG = SM_TMEM + 4;
constexpr uint32_t SM_SEG = (SM_FLAG + 4 + 15) & ~15u;      // uint32 [5]: g0, g1, the end for empty units, C, first unit
constexpr uint32_t SM_SCAN = SM_SEG + 32;
constexpr uint32_t SM_SCHED = SM_SCAN + NTHREADS * 4;       // uint32 [units + 1]: tiles before each unit
constexpr uint32_t SM_KLUT = (SM_SCHED + (SCHED_MAX + 1) * 4 + 127) & ~127u;
__host__ __device__ constexpr uint32_t sm_vlut(int kb) { return SM_KLUT + klut_bytes(kb); }
__host__ __device__ constexpr uint32_t sm_stage(int kb, int vb) { return sm_vlut(kb) + lut_bytes(vb); }
__host__ __device__ constexpr uint32_t stage_bytes(int kb, int vb) {
    return BK * (row_bytes(kb) + row_bytes(vb) + 4);  // K codes, V codes, K norms, V norms
}
__host__ __device__ constexpr uint32_t sm_alloc(int kb, int vb) {
    return sm_stage(kb, vb) + NS * stage_bytes(kb, vb) + 1024;
}
static_assert(sm_alloc(4, 4) <= 227u * 1024u && sm_alloc(4, 8) <= 227u * 1024u && sm_alloc(8, 8) <= 227u * 1024u,
              "the largest layouts fit a block's shared memory");

__device__ __forceinline__ float lds_f32(uint32_t addr) { return __uint_as_float(ptx::lds32(addr)); }
__device__ __forceinline__ uint32_t pack2(uint16_t lo, uint16_t hi) { return lo | (static_cast<uint32_t>(hi) << 16); }

// ------------------------------------------------------------ the schedule
struct Segment {
    int u, j0, j1;
};

// The block's share of the tile sequence as segments (unit, tiles [j0, j1)):
// P[u] tiles come before unit u, block c of C takes [c total / C,
// (c + 1) total / C); a unit without tiles belongs to the block whose range
// holds its start.  Without a schedule block c is unit c, whole.
__device__ __forceinline__ bool next_segment(const Args& a, const uint8_t* smem, int& it, Segment& s) {
    const volatile uint32_t* seg = reinterpret_cast<const volatile uint32_t*>(smem + SM_SEG);
    if (it < 0) it = static_cast<int>(seg[4]);
    if (it >= a.units) return false;
    s.u = it;
    if (!a.spread) {
        if (it != static_cast<int>(blockIdx.x)) return false;
        s.j0 = 0;
        s.j1 = unit_of<BK>(a, it).ntiles;
    } else {
        const volatile uint32_t* P = reinterpret_cast<const volatile uint32_t*>(smem + SM_SCHED);
        const uint32_t pu = P[it], pn = P[it + 1], g0 = seg[0], g1 = seg[1];
        if (pu >= seg[2]) return false;
        s.j0 = static_cast<int>((pu > g0 ? pu : g0) - pu);
        s.j1 = static_cast<int>((pn < g1 ? pn : g1) - pu);
    }
    ++it;
    return true;
}

// The same walk tile by tile.
struct Tiles {
    int it = -1, gi = -1, j = 0, kend = 0;
    Segment s{0, 0, 0};
    __device__ __forceinline__ int keys() const { return min(BK, kend - j * BK); }
    __device__ __forceinline__ bool next(const Args& a, const uint8_t* smem) {
        if (++j >= s.j1) {
            do {
                if (!next_segment(a, smem, it, s)) return false;
            } while (s.j1 <= s.j0);
            j = s.j0;
            kend = unit_of<BK>(a, s.u).kend;
        }
        ++gi;
        return true;
    }
};

// The block whose range holds global tile g (g < total).
__device__ __forceinline__ int block_of(uint32_t g, uint32_t total, uint32_t nblocks) {
    return static_cast<int>(((static_cast<uint64_t>(g) + 1) * nblocks - 1) / total);
}
// A block holds at most two pieces of cut units: the head of the unit its
// range starts (slot 2c + 1) and a piece of a unit begun earlier (slot 2c).
// A slot is 32 chunks of 4 channels of every row, fp32, the rows of a chunk
// next to each other; then the rows' m and l.
__host__ __device__ constexpr size_t part_floats(int rows) { return static_cast<size_t>(rows) * (D + 2); }
__device__ __forceinline__ int part_slot(int block, int first_block) { return 2 * block + (block == first_block); }

// --------------------------------------------------------------- dequantise
template <int BITS, int ROW = 32>
__device__ void build_lut(uint32_t* lut, const uint16_t* cent, int t, int nthreads) {
    constexpr int n = 32 << (2 * BITS), m = (1 << BITS) - 1;
    for (int i = t; i < n; i += nthreads) {
        const int e = i >> 5;
        lut[e * ROW + (i & 31)] = pack2(cent[e & m], cent[e >> BITS]);
    }
}

// Four int8 bytes q as two fp16 pairs q / 128: the byte with its top bit
// flipped is the mantissa of 8, 9 + q / 128; subtracting 9 is exact.
__device__ __forceinline__ uint2 int8_to_half(uint32_t b) {
    const uint32_t x = b ^ 0x80808080u, k = 0x48484848u;
    const __half2 off = __halves2half2(__ushort_as_half(0x4880), __ushort_as_half(0x4880));
    uint32_t lo = __byte_perm(x, k, 0x4140), hi = __byte_perm(x, k, 0x4342);
    const __half2 p = __hsub2(*reinterpret_cast<__half2*>(&lo), off), q = __hsub2(*reinterpret_cast<__half2*>(&hi), off);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
}

// Lookup j of a code word through a table with 128-byte rows at TABLE: the
// field of 2 BITS bits at bit 2 BITS j moves to bit 7.
template <int BITS, uint32_t TABLE, int J>
__device__ __forceinline__ uint32_t lookup(uint32_t c, uint32_t l4) {
    constexpr int SH = 2 * BITS * J - 7;
    constexpr uint32_t M = ((1u << (2 * BITS)) - 1u) << 7;
    uint32_t x;
    if constexpr (SH > 0) x = c >> SH;
    else x = c << -SH;
    return ptx::lds32_imm<TABLE>((x & M) | l4);
}

// One operand tile [64 slots][128 channels] from a stage's rows by THREADS
// threads: this one takes channel group dt % 16 (8 channels) of slots
// dt / 16 + (THREADS / 16) i.  SCALE: values, times the slot's fp16 norm (and,
// int8, the tile's factor, a pair).  Slots at or past nk are zeros.
template <int BITS, bool SCALE, bool WIDE, uint32_t TABLE, int THREADS>
__device__ __forceinline__ void dequant_tile(uint32_t tile, uint32_t codes, uint32_t snorms, uint32_t factor,
                                             int dt, int nk) {
    constexpr int RB = row_bytes(BITS), IT = BK * (D / 8) / THREADS, KS = THREADS / 16, B = 4;
    static_assert(IT % B == 0, "whole batches");
    const int cg = dt & 15, k0 = dt >> 4;
    const uint32_t l4 = 4u * static_cast<uint32_t>(dt & 31);
    // (in batches of four slots, whose loads go out together)
#pragma unroll
    for (int b = 0; b < IT; b += B) {
        uint4 v[B];
        if constexpr (BITS == 8) {
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const uint32_t at = codes + (k0 + KS * (b + i)) * RB + 8 * cg;
                const uint2 p = int8_to_half(ptx::lds32(at)), q = int8_to_half(ptx::lds32(at + 4));
                v[i] = make_uint4(p.x, p.y, q.x, q.y);
            }
        } else {
            uint32_t c8[B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const uint32_t row = codes + (k0 + KS * (b + i)) * RB;
                if constexpr (BITS == 4) {
                    c8[i] = ptx::lds32(row + 4 * cg);
                } else if constexpr (BITS == 2) {
                    c8[i] = ptx::lds16(row + 2 * cg);
                } else {  // 24 bits from bit 24 cg: may straddle two words
                    const int bit = 24 * cg, w = bit >> 5, sh = bit & 31;
                    const uint32_t lo = ptx::lds32(row + 4 * w), hi = ptx::lds32(row + 4 * min(w + 1, RB / 4 - 1));
                    c8[i] = __funnelshift_r(lo, hi, sh);
                }
            }
#pragma unroll
            for (int i = 0; i < B; ++i) {
                if constexpr (WIDE) {
                    v[i].x = ptx::lds32_imm<TABLE>(__byte_perm(c8[i], l4, 0x7604));
                    v[i].y = ptx::lds32_imm<TABLE>(__byte_perm(c8[i], l4, 0x7614));
                    v[i].z = ptx::lds32_imm<TABLE>(__byte_perm(c8[i], l4, 0x7624));
                    v[i].w = ptx::lds32_imm<TABLE>(__byte_perm(c8[i], l4, 0x7634));
                } else {
                    v[i].x = lookup<BITS, TABLE, 0>(c8[i], l4);
                    v[i].y = lookup<BITS, TABLE, 1>(c8[i], l4);
                    v[i].z = lookup<BITS, TABLE, 2>(c8[i], l4);
                    v[i].w = lookup<BITS, TABLE, 3>(c8[i], l4);
                }
            }
        }
        if constexpr (SCALE) {
#pragma unroll
            for (int i = 0; i < B; ++i) {
                uint32_t nb = ptx::lds16(snorms + 2 * (k0 + KS * (b + i)));
                // (a norm that is not finite: the row is zeros, its key's score NaN)
                if ((nb & 0x7C00u) == 0x7C00u) nb = 0u;
                const uint32_t n2 = nb | (nb << 16);
                __half2 f = *reinterpret_cast<const __half2*>(&n2);
                if constexpr (BITS == 8) f = __hmul2(f, *reinterpret_cast<const __half2*>(&factor));
                __half2* h = reinterpret_cast<__half2*>(&v[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = __hmul2(h[e], f);
            }
        }
        if (nk < BK) {  // the last, partial tile only
#pragma unroll
            for (int i = 0; i < B; ++i)
                if (k0 + KS * (b + i) >= nk) v[i] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < B; ++i) ptx::sts128(tile + tc::sw128_offset(k0 + KS * (b + i), 8 * cg, BK), v[i]);
    }
}

// The exponent e of a tile's values (see value_exponent) from its nk staged
// fp16 norms, by the whole warp.  (A norm that is not finite counts as 2^16.)
__device__ __forceinline__ int tile_exponent(uint32_t snorms, int lane, int nk) {
    uint32_t w = ptx::lds32(snorms + 4 * lane) & 0x7FFF7FFFu;
    if (nk < BK) w = 2 * lane + 1 < nk ? w : 2 * lane < nk ? w & 0xFFFFu : 0u;
    return max(static_cast<int>(__reduce_max_sync(kFullMask, max(w & 0xFFFFu, w >> 16)) >> 10) - 29, VALUE_E_MIN);
}

__device__ __forceinline__ float2 half2_float2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// 8 consecutive fp32 columns of this thread's tensor-memory lane.
__device__ __forceinline__ void ld_8cols(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

template <int KB, int VB>
__global__ void __launch_bounds__(NTHREADS, 1) tree_mma_kernel(const __grid_constant__ Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bars = sbase + SM_BAR;
    auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM_FLAG);
    auto fail = [&]() {
        if (!*abort_flag && a.err) atomicOr(a.err, TQ_DEVERR_TIMEOUT);
        *abort_flag = 1;
    };
    // A wait that runs out sets the flag, and once it is set no wait waits: the
    // warps go on through their tiles as they would have (on data that is not
    // valid), so no lane leaves its warp, nor a warp the block, at a collective
    // instruction.  Only what would start new work stops: the producer and the
    // MMA issuer (which alone uses the answer).
    auto lane_wait = [&](int i, uint32_t parity) -> bool {
        const uint32_t b = bar(i);
        if (ptx::mbar_try_wait(b, parity)) return true;
        const long long start = clock64();
        while (!*abort_flag) {
#pragma unroll 1
            for (int k = 0; k < 8; ++k)
                if (ptx::mbar_try_wait(b, parity)) return true;
            if (clock64() - start > WAIT_LIMIT) fail();
        }
        return false;
    };
    auto wait = [&](int i, uint32_t parity) { lane_wait(i, parity); };
    // for warps that wait most of the time (polling would take issue slots from the working ones)
    auto wait_asleep = [&](int i, uint32_t parity) {
        if (!*abort_flag && !ptx::mbar_wait_bounded_sleep(bar(i), parity, WAIT_LIMIT, 64)) fail();
    };
    const int G = a.group;
    const bool pair = a.pair, two_terms = a.terms == 2, overlay = pair || two_terms;
    // softmax warps that own query rows, of each stream
    const int rows = a.tok_per_tile * G;
    const int aw0 = (min(BM, rows) + 31) / 32, aw1 = pair ? (rows - BM + 31) / 32 : aw0;
    const int soft_threads = 32 * (aw0 + aw1);

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            ptx::mbar_init(bar(B_FULL + i), a.staged_norms ? 1 : 2);
            ptx::mbar_init(bar(B_EMPTY + i), DEQ_WARPS);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(B_KFULL + i), DEQ_WARPS);
            ptx::mbar_init(bar(B_KEMPTY + i), 1);
            ptx::mbar_init(bar(B_VFULL + i), DEQ_WARPS);
            ptx::mbar_init(bar(B_VEMPTY + i), 1);
            ptx::mbar_init(bar(B_PV + i), 1);
            ptx::mbar_init(bar(B_SFULL + i), 1);
            ptx::mbar_init(bar(B_SEMPTY + i), i ? aw1 : aw0);
            ptx::mbar_init(bar(B_PFULL + i), i ? aw1 : aw0);
        }
        ptx::mbar_init(bar(B_QREADY), aw0 + aw1);
        ptx::mbar_init(bar(B_FINAL), 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (tid < 32) reinterpret_cast<uint16_t*>(smem + SM_CENT)[tid] = tid < 16 ? a.kcent[tid] : a.vcent[tid - 16];
    if (warp == MMA_WARP) {
        tc::tmem_alloc(sbase + SM_TMEM, TMEM_COLS);
        tc::tmem_relinquish();
    }
    __syncthreads();
    if (warp >= DEQ0 / 32 && warp < LIGHT0 / 32) {
        constexpr int N = LIGHT0 - DEQ0;
        const uint16_t* kcent = reinterpret_cast<const uint16_t*>(smem + SM_CENT);
        if constexpr (KB < 8) build_lut<KB, wide(KB) ? 64 : 32>(reinterpret_cast<uint32_t*>(smem + SM_KLUT), kcent, tid - DEQ0, N);
        if constexpr (VB < 8) build_lut<VB>(reinterpret_cast<uint32_t*>(smem + sm_vlut(KB)), kcent + 16, tid - DEQ0, N);
    }
    // everything above overlaps the end of the kernel before; nothing of the
    // caller's memory has been read or written yet
    ptx::wait_prerequisites();
    ptx::launch_dependents();

    // ---- the schedule: P[u] = tiles of the units before u
    uint32_t* P = reinterpret_cast<uint32_t*>(smem + SM_SCHED);
    uint32_t* scan = reinterpret_cast<uint32_t*>(smem + SM_SCAN);
    const int U = a.units;
    if (a.spread) {
        const int per = (U + NTHREADS - 1) / NTHREADS, u0 = min(U, tid * per), u1 = min(U, u0 + per);
        uint32_t sum = 0;
        for (int u = u0; u < u1; ++u) sum += static_cast<uint32_t>(unit_of<BK>(a, u).ntiles);
        scan[tid] = sum;
        __syncthreads();
        if (warp == 0) {
            constexpr int PER_LANE = NTHREADS / 32;
            uint32_t t = 0;
            for (int i = 0; i < PER_LANE; ++i) t += scan[lane * PER_LANE + i];
            uint32_t incl = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(kFullMask, incl, o);
                if (lane >= o) incl += y;
            }
            uint32_t run = incl - t;
            for (int i = 0; i < PER_LANE; ++i) {
                const uint32_t v = scan[lane * PER_LANE + i];
                scan[lane * PER_LANE + i] = run;
                run += v;
            }
            if (lane == 31) P[U] = run;
        }
        __syncthreads();
        uint32_t run = scan[tid];
        for (int u = u0; u < u1; ++u) {
            P[u] = run;
            run += static_cast<uint32_t>(unit_of<BK>(a, u).ntiles);
        }
        __syncthreads();
        if (blockIdx.x == 0)  // (for the merge kernel)
            for (int u = tid; u <= U; u += NTHREADS) a.sched[u] = P[u];
    }
    if (tid == 0) {
        uint32_t* seg = reinterpret_cast<uint32_t*>(smem + SM_SEG);
        const uint32_t c = blockIdx.x;
        if (a.spread) {
            const uint32_t total = P[U];
            // no more sharing blocks than tiles, so that each one's range holds at least one
            const uint32_t C = gridDim.x > total ? (total > 0 ? total : 1u) : gridDim.x;
            const uint32_t g0 = static_cast<uint32_t>(static_cast<uint64_t>(c) * total / C);
            const uint32_t g1 = static_cast<uint32_t>(static_cast<uint64_t>(c + 1) * total / C);
            int lo = 0, hi = U;
            if (c >= C) {
                lo = U;
            } else {  // first u with P[u + 1] > g0 or P[u] >= g0
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (P[mid + 1] > g0 || P[mid] >= g0) hi = mid;
                    else lo = mid + 1;
                }
            }
            seg[0] = g0;
            seg[1] = g1;
            seg[2] = c == C - 1 ? total + 1 : g1;
            seg[3] = C;
            seg[4] = static_cast<uint32_t>(lo);
        } else {
            seg[4] = c;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + SM_TMEM);
    constexpr int kbytes = row_bytes(KB), vbytes = row_bytes(VB);
    constexpr uint32_t STAGE = sm_stage(KB, VB), STAGE_BYTES = stage_bytes(KB, VB);
    constexpr uint32_t ST_VC = BK * kbytes, ST_KN = ST_VC + BK * vbytes, ST_VN = ST_KN + BK * 2;

    // Every role walks the same segments; tile gi (counted over the block's
    // run) is in ring stage gi % NS and operand buffers gi % 2.  A stream's
    // steps are its tiles: all of them (pair), or tile gi is step gi / 2 of
    // stream gi % 2.
    if (warp >= LIGHT0 / 32) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_LIGHT));
        if (warp == PRODUCER_WARP) {
            // -------------------------------------------------------- producer
            const bool leader = tc::elect_one();
            int gi = 0, it = -1;
            Segment s;
            while (next_segment(a, smem, it, s)) {
                const Unit x = unit_of<BK>(a, s.u);
                for (int j = s.j0; j < s.j1; ++j, ++gi) {
                    const int st = gi % NS;
                    if (gi >= NS) {
                        wait_asleep(B_EMPTY + st, ((gi - NS) / NS) & 1);
                        if (__any_sync(kFullMask, *abort_flag)) goto produced;
                    }
                    if (leader) {
                        const int key0 = j * BK, nk = min(BK, x.kend - key0), n8 = (nk + 7) & ~7;
                        const uint32_t dst = sbase + STAGE + st * STAGE_BYTES, full = bar(B_FULL + st);
                        ptx::mbar_arrive_expect_tx(full, nk * (kbytes + vbytes) + (a.staged_norms ? n8 * 4 : 0));
                        // one run of slots, or one per block of the pool
                        for (int k = 0; k < nk;) {
                            const int n = a.table ? min(nk - k, a.block_size - (key0 + k) % a.block_size) : nk;
                            const size_t row = cache_row(a, x.b, x.kv, key0 + k);
                            ptx::bulk_copy_g2s(dst + k * kbytes, a.k_codes + row * kbytes, n * kbytes, full);
                            ptx::bulk_copy_g2s(dst + ST_VC + k * vbytes, a.v_codes + row * vbytes, n * vbytes, full);
                            if (a.staged_norms) {  // (runs of norms move in 16-byte pieces)
                                const int m8 = (n + 7) & ~7;
                                ptx::bulk_copy_g2s(dst + ST_KN + 2 * k, a.k_norms + row, m8 * 2, full);
                                ptx::bulk_copy_g2s(dst + ST_VN + 2 * k, a.v_norms + row, m8 * 2, full);
                            }
                            k += n;
                        }
                    }
                    __syncwarp();
                }
            }
        produced:
            // every copy issued must land before the block may exit
            for (int k = max(0, gi - NS); k < gi; ++k)
                ptx::mbar_wait_bounded(bar(B_FULL + k % NS), (k / NS) & 1, WAIT_LIMIT);
        } else if (warp >= NORM_WARP) {
            // ---------------------------------------- norms that are not staged
            if (!a.staged_norms) {
                int gi = 0, it = -1;
                Segment s;
                while (next_segment(a, smem, it, s)) {
                    const Unit x = unit_of<BK>(a, s.u);
                    const size_t row0 = (static_cast<size_t>(x.b) * a.hkv + x.kv) * a.capacity;
                    for (int j = s.j0; j < s.j1; ++j, ++gi) {
                        if ((gi & 1) != warp - NORM_WARP) continue;
                        const int st = gi % NS, nk = min(BK, x.kend - j * BK);
                        const size_t row = row0 + static_cast<size_t>(j) * BK;
                        uint16_t n[4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int k = lane + 32 * h;
                            n[h] = k < nk ? a.k_norms[row + k] : uint16_t(0);
                            n[2 + h] = k < nk ? a.v_norms[row + k] : uint16_t(0);
                        }
                        if (gi >= NS) wait_asleep(B_EMPTY + st, ((gi - NS) / NS) & 1);
                        uint16_t* kn = reinterpret_cast<uint16_t*>(smem + STAGE + st * STAGE_BYTES + ST_KN);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            kn[lane + 32 * h] = n[h];
                            kn[BK + lane + 32 * h] = n[2 + h];
                        }
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bar(B_FULL + st));
                    }
                }
            }
        } else if (warp == MMA_WARP) {
            // ----------------------------------------------------- MMA issuer
            // (no collective instruction before the end of the role: after a wait
            // that ran out, lanes may leave the loops one by one)
            const bool leader = tc::elect_one();
            const uint32_t idesc_s = tc::idesc_f16(BM, BK), idesc_o = tc::idesc_f16_bmn(BM, D);
            const uint64_t kdesc0 = tc::sw128_desc(sbase + SM_K);
            const uint64_t vdesc0 = tc::sw128_mn_desc(sbase + SM_V, BK * 128, 1024);
            // scores of stream g from tile gi; the tile's last reader frees it
            // (false: a wait ran out somewhere, nothing is issued any more)
            auto issue_s = [&](int gi, int g, bool last) -> bool {
                const int bf = gi & 1;
                if (!lane_wait(B_KFULL + bf, (gi >> 1) & 1)) return false;
                tc::fence_after_sync();
                if (leader) {
                    const uint64_t kd = kdesc0 + static_cast<uint64_t>(bf * (BK * D * 2) >> 4);
                    const uint32_t sd = tmem + TM_S + BK * g, qd = tmem + TM_Q + (pair ? 64 * g : 0);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint64_t bd = kd + static_cast<uint64_t>(((ks >> 2) * (BK * 128) + (ks & 3) * 32) >> 4);
                        tc::mma_f16_ts(sd, qd + 8 * ks, bd, idesc_s, ks > 0);
                        if (two_terms) tc::mma_f16_ts(sd, qd + 64 + 8 * ks, bd, idesc_s, true);
                    }
                    tc::commit(bar(B_SFULL + g));
                    if (last) tc::commit(bar(B_KEMPTY + bf));
                }
                return true;
            };
            // output of stream g's step q from tile gi
            auto issue_pv = [&](int gi, int g, int q, bool first, bool last) -> bool {
                const int bf = gi & 1;
                if (!lane_wait(B_PFULL + g, q & 1)) return false;
                if (!lane_wait(B_VFULL + bf, (gi >> 1) & 1)) return false;
                tc::fence_after_sync();
                if (leader) {
                    const uint64_t vd = vdesc0 + static_cast<uint64_t>(bf * (BK * D * 2) >> 4);
                    const uint32_t pd = tmem + (overlay ? TM_S + BK * g : TM_Q + 64 + (BK / 2) * g);
#pragma unroll
                    for (int ks = 0; ks < BK / 16; ++ks)
                        tc::mma_f16_ts(tmem + TM_O + D * g, pd + 8 * ks,
                                       vd + static_cast<uint64_t>(ks * 2048 >> 4), idesc_o, !first || ks > 0);
                    tc::commit(bar(B_PV + g));
                    if (last) tc::commit(bar(B_VEMPTY + bf));
                }
                return true;
            };
            int gi = 0, qs = 0, it = -1;
            Segment s;
            while (next_segment(a, smem, it, s)) {
                if (s.j1 <= s.j0) continue;
                // the queries are in tensor memory, and the segment before has left it
                if (!lane_wait(B_QREADY, qs & 1)) break;
                ++qs;
                const int gfirst = gi, gend = gi + (s.j1 - s.j0);
                // (overlay: a stream's weights lie in its score buffer, so its
                // P V is waited for before the buffer is written again)
                if (pair) {
                    if (!issue_s(gi, 0, false) || !issue_s(gi, 1, true)) break;
                    for (; gi < gend; ++gi) {
#pragma unroll 1
                        for (int g = 0; g < 2; ++g) {
                            if (!issue_pv(gi, g, gi, gi == gfirst, g == 1)) goto issued;
                            if (gi + 1 < gend) {
                                if (!lane_wait(B_PV + g, gi & 1)) goto issued;
                                if (!issue_s(gi + 1, g, g == 1)) goto issued;
                            }
                        }
                    }
                } else {
                    if (!issue_s(gi, gi & 1, true)) break;
                    if (gi + 1 < gend && !issue_s(gi + 1, (gi + 1) & 1, true)) break;
                    for (; gi < gend; ++gi) {
                        const int g = gi & 1, q = gi >> 1;
                        if (!overlay && gi + 2 < gend) {
                            if (!lane_wait(B_SEMPTY + g, q & 1)) goto issued;
                            if (!issue_s(gi + 2, g, true)) goto issued;
                        }
                        if (!issue_pv(gi, g, q, gi < gfirst + 2, true)) goto issued;
                        if (overlay && gi + 2 < gend) {
                            if (!lane_wait(B_PV + g, q & 1)) goto issued;
                            if (!issue_s(gi + 2, g, true)) goto issued;
                        }
                    }
                }
            }
        issued:
            if (leader) {
                tc::commit(bar(B_FINAL));
                ptx::mbar_wait_bounded(bar(B_FINAL), 0, WAIT_LIMIT);
            }
            __syncwarp();
        }
    } else if (warp >= DEQ0 / 32) {
        // ------------------------------------------------------ dequantisers
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_DEQ));
        const int dt = tid - DEQ0;
        // (keys run a tile ahead of values: K~(gi + 1) waits for the scores of
        // tile gi - 1 only, V~(gi) for the P V of tile gi - 2)
        Tiles k, v;
        int vexp = 0;  // (int8 values) the exponent of the keys' tile
        for (;;) {
            const int e = vexp;  // and of the values' tile, the one before (at the end, the last)
            const bool more = k.next(a, smem);
            if (more) {
                const int gi = k.gi, st = gi % NS, bf = gi & 1, nk = k.keys();
                const uint32_t sst = sbase + STAGE + st * STAGE_BYTES;
                wait(B_FULL + st, (gi / NS) & 1);
                if (gi >= 2) wait(B_KEMPTY + bf, ((gi - 2) >> 1) & 1);
                if (dt < BK) {
                    // the tile's key norms, for the softmax (which is through
                    // with tile gi - 4: the scores of tile gi - 2 followed it)
                    const uint16_t kn = ptx::lds16(sst + ST_KN + 2 * dt), vn = ptx::lds16(sst + ST_VN + 2 * dt);
                    reinterpret_cast<uint16_t*>(smem + SM_KNR)[(gi & 3) * BK + dt] =
                        dt >= nk ? uint16_t(0) : (vn & 0x7C00u) == 0x7C00u ? uint16_t(0x7E00) : kn;
                }
                if constexpr (VB == 8) {
                    vexp = tile_exponent(sst + ST_VN, lane, nk);
                    if (dt == 0)
                        reinterpret_cast<float2*>(smem + SM_VEXP)[gi & 3] =
                            make_float2(static_cast<float>(vexp), power_of_two(-vexp));
                }
                dequant_tile<KB, false, wide(KB), SMEM_WINDOW + SM_KLUT, DEQ_WARPS * 32>(
                    sbase + SM_K + bf * (BK * D * 2), sst, 0u, 0u, dt, nk);
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(B_KFULL + bf));
            }
            if (v.gi < (more ? k.gi - 1 : k.gi)) {
                v.next(a, smem);
                const int gi = v.gi, st = gi % NS, bf = gi & 1;
                const uint32_t sst = sbase + STAGE + st * STAGE_BYTES;
                if (gi >= 2) wait(B_VEMPTY + bf, ((gi - 2) >> 1) & 1);
                dequant_tile<VB, true, false, SMEM_WINDOW + sm_vlut(KB), DEQ_WARPS * 32>(
                    sbase + SM_V + bf * (BK * D * 2), sst + ST_VC, sst + ST_VN,
                    static_cast<uint32_t>(15 - e) * 0x04000400u, dt, v.keys());
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(bar(B_VFULL + bf));
                    ptx::mbar_arrive(bar(B_EMPTY + st));
                }
            }
            if (!more) break;
        }
    } else {
        // ---------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        const int g = warp >> 2, r = tid & 127;  // stream, its tensor-memory lane
        const int ur = pair ? BM * g + r : r;    // query row of the unit
        const int rt = ur / G, rh = ur % G;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        constexpr float rsqrt_d = 0.08838834764831845f;
        // (two of them in turn: a stream without a tile in a segment does not wait for the other one's reads)
        float* ml = reinterpret_cast<float*>(smem + SM_ML);
        int ml_next = 4 * BM;
        int gi = 0, it = -1;
        Segment s;
        if ((warp & 3) >= (g ? aw1 : aw0)) it = U;  // no rows: the warp takes no part
        while (next_segment(a, smem, it, s)) {
            const Unit x = unit_of<BK>(a, s.u);
            const bool row_ok = rt < x.ntok;
            const size_t qoff = ((static_cast<size_t>(x.b) * a.n_draft + x.tok0 + rt) * a.hq + x.kv * G + rh) * D;
            // this thread's 64-channel halves of the row: both, or (two streams over the same rows) its stream's
            const int h0 = pair ? 0 : g, h1 = pair ? 2 : g + 1;
            if (s.j1 <= s.j0) {
                // no tiles: a refused sequence, or one without drafts in this unit
                if (x.bad) {
                    if (x.qt == 0 && x.kv == 0 && tid == 0 && a.err) atomicOr(a.err, TQ_DEVERR_SEQLEN);
                    if (rt < min(a.tok_per_tile, a.n_draft - x.tok0)) {
                        const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                        for (int c = 64 * h0; c < 64 * h1; c += 8) store_row<8>(a.out, qoff + c, z, a.out_dtype);
                    }
                }
                continue;
            }
            // ---- queries: the warps of a stream move its row block's (pair),
            // one of two terms, or every second group of four chunks
            {
                const uint4* src = reinterpret_cast<const uint4*>(a.prep + static_cast<size_t>(s.u) * prep_bytes(a.part_rows, a.terms)) +
                                   (two_terms ? static_cast<size_t>(g) * 16 * a.part_rows : 0) + ur;
                const uint32_t dst = tmem + lanes + TM_Q + (overlay ? 64 * g : 0);
                const int step = overlay ? 4 : 8;
#pragma unroll 2
                for (int c = overlay ? 0 : 4 * g; c < 16; c += step) {
                    uint4 w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = src[static_cast<size_t>(c + i) * a.part_rows];
                    const uint32_t v[16] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w,
                                            w[2].x, w[2].y, w[2].z, w[2].w, w[3].x, w[3].y, w[3].z, w[3].w};
                    tc::st_16cols_u(dst + 4 * c, v);
                }
            }
            // a warp with a row whose scores are multiplied by a factor, or pass
            // 2^22, takes the masked path for all its tiles
            int careful_from = x.base - BK;
            {
                const float f = a.row_factor[static_cast<size_t>(s.u) * a.part_rows + ur];
                *reinterpret_cast<float*>(smem + SM_FACTOR + 4 * tid) = f;
                if (__any_sync(kFullMask, f != 1.f)) careful_from = -1;
            }
            tc::st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_QREADY));
            const uint64_t mask = row_ok ? row_mask(a, x, x.tok0 + rt) : 0ull;
            float mref = NOTHING, l = 0.f;
            bool first = true;
            const int gfirst = gi, gend = gi + (s.j1 - s.j0), inc = pair ? 1 : 2;
            if (!pair) gi += (gi & 1) != g;  // the stream's first tile of the segment
            for (; gi < gend; gi += inc, first = false) {
                const int q = pair ? gi : gi >> 1;
                wait(B_SFULL + g, q & 1);
                tc::fence_after_sync();
                const uint32_t kn = sbase + SM_KNR + (gi & 3) * BK * 2, ve = sbase + SM_VEXP + (gi & 3) * 8;
                const int key0 = (s.j0 + gi - gfirst) * BK;
                uint32_t pw[BK / 2];
                float sum;
                // the tile's weights against the present reference, and their
                // sum (one straight run of code without the mask's test and the
                // rows' factors)
                auto weigh = [&](auto with_mask) {
                    const float f = decltype(with_mask)::value ? lds_f32(sbase + SM_FACTOR + 4 * tid) : 1.f;
                    const uint64_t seen = decltype(with_mask)::value ? visible(mask, key0, x.base) : 0ull;
                    const uint32_t vis[2] = {static_cast<uint32_t>(seen), static_cast<uint32_t>(seen >> 32)};
                    const float shift = (VB == 8 ? WSHIFT + lds_f32(ve) : WSHIFT) - mref;
                    const float2 nm2 = make_float2(shift, shift);
                    float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
                    float sc[32];
                    uint4 k8;
#pragma unroll
                    for (int i = 0; i < BK; i += 4) {
                        if (i % 32 == 0) {
                            tc::ld_32cols(tmem + lanes + TM_S + BK * g + i, sc);
                            tc::ld_wait();
                        }
                        if (i % 8 == 0) k8 = ptx::lds128(kn + 2 * i);  // the norms of 8 keys
                        const int e = i % 32;
                        const float2 n0 = half2_float2(i % 8 ? k8.z : k8.x), n1 = half2_float2(i % 8 ? k8.w : k8.y);
                        const float2 s0 = make_float2(sc[e], sc[e + 1]), s1 = make_float2(sc[e + 2], sc[e + 3]);
                        float2 t0, t1;
                        if constexpr (!decltype(with_mask)::value) {
                            t0 = ptx::ffma2(s0, n0, nm2);
                            t1 = ptx::ffma2(s1, n1, nm2);
                        } else {
                            // (scores rounded as the reference was, in single operations
                            // that are not fused, and weights that fit fp16, however large
                            // the scores; NaN stays)
                            auto shifted = [&](float x, float n) {
                                const float t = __fadd_rn(__fmul_rn(__fmul_rn(x, f), n), shift);
                                return t > WMOST ? WMOST : t;
                            };
                            t0 = make_float2(shifted(s0.x, n0.x), shifted(s0.y, n0.y));
                            t1 = make_float2(shifted(s1.x, n1.x), shifted(s1.y, n1.y));
                            const uint32_t v = vis[i / 32] >> e;
                            if (!(v & 1u)) t0.x = -INFINITY;
                            if (!(v & 2u)) t0.y = -INFINITY;
                            if (!(v & 4u)) t1.x = -INFINITY;
                            if (!(v & 8u)) t1.y = -INFINITY;
                        }
                        const float2 p0 = make_float2(ptx::ex2(t0.x), ptx::ex2(t0.y));
                        const float2 p1 = make_float2(ptx::ex2(t1.x), ptx::ex2(t1.y));
                        acc0 = ptx::fadd2(acc0, p0);
                        acc1 = ptx::fadd2(acc1, p1);
                        pw[i / 2] = ptx::pack_half2(p0.x, p0.y);
                        pw[i / 2 + 1] = ptx::pack_half2(p1.x, p1.y);
                    }
                    sum = (acc0.x + acc0.y) + (acc1.x + acc1.y);
                };
#pragma unroll 1
                for (bool again = false;; again = true) {
                    // (a tile with drafts: the tree's mask; key0 + BK may pass int32)
                    const bool careful = key0 > careful_from;
                    if (careful) weigh(std::true_type());
                    else weigh(std::false_type());
                    if (again || !__any_sync(kFullMask, !(sum <= WLIMIT))) break;
                    // a weight may leave the fp16 range (or is NaN): raise the
                    // reference to the row's largest score, rescale, again
                    float m = -INFINITY;
                    const float f = lds_f32(sbase + SM_FACTOR + 4 * tid);
                    const uint64_t seen = careful ? visible(mask, key0, x.base) : ~0ull;
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
                        float sc[16];
                        tc::ld_16cols(tmem + lanes + TM_S + BK * g + 16 * h, sc);
                        tc::ld_wait();
                        const uint32_t v = static_cast<uint32_t>(seen >> (16 * h));
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float n = half_bits_to_float(ptx::lds16(kn + 2 * (16 * h + i)));
                            if ((v >> i) & 1u) m = fmaxf(m, __fmul_rn(__fmul_rn(sc[i], f), n));
                        }
                    }
                    const float mnew = fmaxf(VB == 8 ? m + lds_f32(ve) : m, mref), c = ptx::ex2(mref - mnew);
                    // (past 2^22 a fused product would differ from the reference by more than a bit)
                    if (__any_sync(kFullMask, fabsf(mnew) > 0x1p22f && mnew > NOTHING)) careful_from = -1;
                    if (!first) {
                        // the accumulator is complete (overlay: this step's scores came after the stream's last P V)
                        if (!overlay) {
                            wait(B_PV + g, (q - 1) & 1);
                            tc::fence_after_sync();
                        }
#pragma unroll 1
                        for (int q8 = 0; q8 < 8; ++q8) {
                            float ov[16];
                            tc::ld_16cols(tmem + lanes + TM_O + D * g + 16 * q8, ov);
                            tc::ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) ov[i] *= c;
                            tc::st_16cols(tmem + lanes + TM_O + D * g + 16 * q8, ov);
                        }
                    }
                    l *= c;
                    mref = mnew;
                }
                l += VB == 8 ? sum * lds_f32(ve + 4) : sum;
                uint32_t pd = tmem + lanes + TM_S + BK * g;
                if (!overlay) {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(B_SEMPTY + g));  // the scores have been read
                    if (!first) {  // the weights' columns are free when the stream's last P V is done
                        wait(B_PV + g, (q - 1) & 1);
                        tc::fence_after_sync();
                    }
                    pd = tmem + lanes + TM_Q + 64 + (BK / 2) * g;
                }
                tc::st_16cols_u(pd, *reinterpret_cast<const uint32_t (*)[16]>(&pw[0]));
                tc::st_16cols_u(pd + 16, *reinterpret_cast<const uint32_t (*)[16]>(&pw[16]));
                tc::st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(B_PFULL + g));
            }
            // ---- the segment's end: the stream's last P V; two streams over
            // the same rows are joined
            {
                const int last = pair ? gend - 1 : gend - 1 - ((gend - 1 - g) & 1);  // the stream's last tile, if any
                if (last >= gfirst) wait(B_PV + g, (pair ? last : last >> 1) & 1);
                gi = gend;
                ml += ml_next;
                ml_next = -ml_next;
                ml[g * BM + r] = mref;
                ml[(2 + g) * BM + r] = l;
            }
            ptx::named_barrier(2, soft_threads);
            tc::fence_after_sync();
            {
                float M = mref, L = l, w0 = 1.f, w1 = 0.f;
                uint32_t o0 = tmem + lanes + TM_O + D * g, o1 = o0;  // this row's accumulators and their weights
                const bool two = !pair && s.j1 - s.j0 > 1;           // (with one tile the other stream has nothing)
                if (!pair) {
                    const float mo = ml[(1 - g) * BM + r], lo = ml[(3 - g) * BM + r];
                    M = fmaxf(mref, mo);
                    w0 = ptx::ex2(mref - M);
                    w1 = ptx::ex2(mo - M);
                    L = l * w0 + lo * w1;
                    o1 = tmem + lanes + TM_O + D * (1 - g);
                    if (!two && (gfirst & 1) != g) {
                        o0 = o1;
                        w0 = w1;
                    }
                }
                // 8 joined channels from column c
                auto joined = [&](int c, float (&v)[8]) {
                    float u[8];
                    ld_8cols(o0 + c, v);
                    if (two) ld_8cols(o1 + c, u);
                    tc::ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = two ? v[i] * w0 + u[i] * w1 : v[i] * w0;
                };
                const volatile uint32_t* seg = reinterpret_cast<const volatile uint32_t*>(smem + SM_SEG);
                const bool cut = a.spread && (P[s.u] < seg[0] || P[s.u + 1] > seg[1]);
                if (cut) {
                    const int cb = static_cast<int>(blockIdx.x), ca = block_of(P[s.u], P[U], seg[3]);
                    float* mine = a.parts + static_cast<size_t>(part_slot(cb, ca)) * part_floats(a.part_rows);
#pragma unroll 1
                    for (int c = 64 * h0; c < 64 * h1; c += 8) {
                        float v[8];
                        joined(c, v);
                        if (row_ok) {
                            float4* p = reinterpret_cast<float4*>(mine) + static_cast<size_t>(c / 4) * a.part_rows + ur;
                            p[0] = make_float4(v[0], v[1], v[2], v[3]);
                            p[a.part_rows] = make_float4(v[4], v[5], v[6], v[7]);
                        }
                        __syncwarp();
                    }
                    if (row_ok && (pair || g == 0)) {
                        mine[a.part_rows * D + ur] = piece_reference(M, L);
                        mine[a.part_rows * (D + 1) + ur] = L;
                    }
                } else {
                    const float inv = (L == 0.f ? 0.f : a.out_scale / L) * (VB < 8 ? rsqrt_d : 1.f);
#pragma unroll 1
                    for (int h = h0; h < h1; ++h) {
                        float o[64];
                        if constexpr (VB < 8) {
#pragma unroll
                            for (int c = 0; c < 64; c += 8) {
                                float v[8], u[8];
                                joined(c, v);
                                joined(64 + c, u);
#pragma unroll
                                for (int i = 0; i < 8; ++i) o[c + i] = h ? v[i] - u[i] : v[i] + u[i];
                            }
                            fwht_registers(o);
                        } else {
#pragma unroll
                            for (int c = 0; c < 64; c += 8) {
                                float v[8];
                                joined(64 * h + c, v);
#pragma unroll
                                for (int i = 0; i < 8; ++i) o[c + i] = v[i];
                            }
                        }
                        if (row_ok) {
#pragma unroll
                            for (int c = 0; c < 64; c += 8) {
                                float y[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const int i = c + e;
                                    y[e] = o[i] * inv;
                                    if constexpr (VB < 8) y[e] = flip_sign(y[e], (a.signs[2 * h + (i >> 5)] >> (i & 31)) & 1u);
                                }
                                store_row<8>(a.out, qoff + 64 * h + c, y, a.out_dtype);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            tc::fence_before_sync();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <typename... PP, typename... T>
static cudaError_t launch_dependent(void (*kernel)(PP...), dim3 grid, dim3 block, uint32_t smem_bytes, cudaStream_t s,
                                    T&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem_bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<T&&>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int KB, int VB>
cudaError_t launch_typed(const Args& a, int blocks, cudaStream_t s) {
    constexpr uint32_t bytes = sm_alloc(KB, VB);
    const cudaError_t e = cudaFuncSetAttribute(tree_mma_kernel<KB, VB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(bytes));
    if (e != cudaSuccess) return e;
    return launch_dependent(tree_mma_kernel<KB, VB>, dim3(static_cast<unsigned>(blocks)), dim3(NTHREADS), bytes, s, a);
}

}  // namespace mma

// The tensor-memory kernel for keys of 2, 3, 4 bits or int8 (one source file each).
cudaError_t launch_mma_k2(int vb, const Args& a, int blocks, cudaStream_t s);
cudaError_t launch_mma_k3(int vb, const Args& a, int blocks, cudaStream_t s);
cudaError_t launch_mma_k4(int vb, const Args& a, int blocks, cudaStream_t s);
cudaError_t launch_mma_k8(int vb, const Args& a, int blocks, cudaStream_t s);

}  // namespace tree
}  // namespace tq
