// Attention of a tree of drafted tokens over the cache: the general kernel,
// the merge kernels and the C entry points (the tensor-memory kernel, which
// d = 128 layers without a sketch take, is in tree_mma_impl.cuh).
//
// For draft t of sequence b and query head h (kv head h / (Hq / Hkv)):
//   s_i = sm_scale <q, k_hat_i>,  p = softmax over the slots the draft sees,
//   out = sum_i p_i v_hat_i,
// where the draft sees the base[b] slots before the tree and the drafts its
// mask names.  Turbo keys score in the rotated domain, n_i <R q, c[code]>, and
// turbo values are summed there, with one inverse rotation at the end; int8
// sides stay in the original domain.  A key's sketch enters the score product
// as m more channels: the key row carries +-gamma in them, the query row
// sqrt(pi/2)/m (S R q).
//
// The general kernel takes every configuration: 64 query rows (16 a warp) of
// one (sequence, kv head) against tiles of BK keys, dequantised to fp16 in
// shared memory; warp-level MMAs (m16n8k16, fp32 accumulation); the online
// softmax in registers; the next tile's packed rows are loaded while a tile is
// worked on.  Queries enter as fp16 terms: two, so that a score keeps
// about 22 bits of its query, or one for bf16 outputs (see the other kernel).  The key axis is split between blocks and the
// merge kernel joins the pieces.  It is bound by the latency of that chain with
// three blocks an SM (two at d = 256): 2800 instructions a warp and tile of 32
// keys at d = 256, in 27% of the issue slots, 1500 a tile of 64 in 35% at d = 64;
// the first stalls are fixed latencies and instruction fetch.  16 drafts of 32
// heads over 6000 tokens take 68 us at d = 256 and 55 at d = 128 with a sketch; 4
// sequences of 777 to 4001 tokens, 17 drafts of 16 heads, int8, d = 64: 34 us.

#include "tree_common.cuh"
#include "tree_mma_impl.cuh"

namespace tq {
namespace tree {

constexpr int GEN_ROWS = 64, GEN_THREADS = 128;
// weights are held as 2^(s + e - m + PSHIFT) <= 2^12 in fp16 (e: value_exponent):
// those 2^26 times smaller than the largest are still normal numbers
constexpr float PSHIFT = 12.0f;

template <int D>
constexpr int GEN_BK = D == 256 ? 32 : 64;

// Rows of halves padded by 8, so that the 8 rows of a fragment load fall in different banks.
__host__ __device__ constexpr int gen_qk_stride(int d, int m) { return d + m + 8; }
constexpr size_t gen_smem(int d, int m, int terms) {
    const size_t bk = d == 256 ? GEN_BK<256> : GEN_BK<128>;
    return (static_cast<size_t>(terms) * GEN_ROWS + bk) * gen_qk_stride(d, m) * 2 + bk * (d + 8) * 2 + bk * 8 + 128;
}
// Blocks an SM holds: what the launch bounds allow the registers, and shared memory.
constexpr int gen_bound(int d) { return d == 256 ? 2 : 3; }
static int gen_resident(int d, int m, int terms) {
    const int n = static_cast<int>(227 * 1024 / (gen_smem(d, m, terms) + 1024));
    return n < gen_bound(d) ? n : gen_bound(d);
}

__device__ __forceinline__ void ldmatrix_x2_trans(uint32_t& r0, uint32_t& r1, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr));
}

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The general kernel's queries, once a call: rotated (turbo keys), times the
// softmax scale in log2 units (and a power of two: see row_exponent), the
// sketch's projections appended, as two fp16 terms: per unit [2][64 rows][d + m].  A row on d / 32 lanes; blockIdx.y
// takes PREP_SKETCH of the sketch's rows (the first also the rotated row).
constexpr int PREP_THREADS = 128, PREP_SKETCH = 8;
template <int D>
__global__ void __launch_bounds__(PREP_THREADS) tree_general_prep_kernel(const __grid_constant__ Args a) {
    constexpr int LPV = D / 32, VPW = 32 / LPV;
    ptx::wait_prerequisites();
    ptx::launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane % LPV, m = a.qjl_dims, KD = D + m, G = a.group;
    const long long row = (static_cast<long long>(blockIdx.x) * (PREP_THREADS / 32) + (threadIdx.x >> 5)) * VPW + lane / LPV;
    const int u = static_cast<int>(row / GEN_ROWS), r = static_cast<int>(row % GEN_ROWS);
    if (u >= a.units) return;  // (whole warps)
    const int rt = r / G, rh = r % G;
    const int qt = u % a.qtiles, kv = (u / a.qtiles) % a.hkv, b = u / a.qtiles / a.hkv, t = qt * a.tok_per_tile + rt;
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.f;
    if (rt < a.tok_per_tile && t < a.n_draft) {
        const size_t off = ((static_cast<size_t>(b) * a.n_draft + t) * a.hq + kv * G + rh) * D;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const size_t at = off + 8 * (sub + LPV * k);
            load4(a.q, at, a.q_dtype, *reinterpret_cast<float (*)[4]>(&v[8 * k]));
            load4(a.q, at + 4, a.q_dtype, *reinterpret_cast<float (*)[4]>(&v[8 * k + 4]));
        }
    }
    __syncwarp();
    float scale = a.score_scale;
    if (a.k_bits != 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * k + e] = flip_sign(v[8 * k + e], sign_bit(a.signs, 8 * (sub + LPV * k) + e));
        fwht_registers(v);
        fwht_lanes<32, LPV>(v, sub);
        scale *= rsqrtf(static_cast<float>(D));
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(v[i]));
    const int k2 = row_exponent(group_max<LPV>(top) * scale);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = v[i] * scale * power_of_two(-k2);
    __half* hi = reinterpret_cast<__half*>(a.prep + static_cast<size_t>(u) * (GEN_ROWS * 4) * KD) + static_cast<size_t>(r) * KD;
    __half* lo = hi + static_cast<size_t>(GEN_ROWS) * KD;
    if (blockIdx.y == 0) {
        if (sub == 0) a.row_factor[row] = power_of_two(k2);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v0 = v[8 * k + 2 * e], v1 = v[8 * k + 2 * e + 1];
                hw[e] = ptx::pack_half2(v0, v1);
                const float2 h = mma::half2_float2(hw[e]);
                lw[e] = ptx::pack_half2(v0 - h.x, v1 - h.y);
            }
            *reinterpret_cast<uint4*>(hi + 8 * (sub + LPV * k)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            *reinterpret_cast<uint4*>(lo + 8 * (sub + LPV * k)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        }
    }
    // a key's sketch channels hold +-gamma, its others centroids times
    // key_scale (which score_scale takes out): the projections put it back
    const float coef = m ? sqrtf(0.5f * 3.14159265358979f) / m * a.key_scale : 0.f;
    const int s0 = static_cast<int>(blockIdx.y) * PREP_SKETCH;
#pragma unroll 2
    for (int j = s0; j < min(m, s0 + PREP_SKETCH); ++j) {
        const float4* srow = reinterpret_cast<const float4*>(a.sketch + static_cast<size_t>(j) * D);
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 p = __ldg(srow + 2 * (sub + LPV * k)), q = __ldg(srow + 2 * (sub + LPV * k) + 1);
            y = fmaf(p.x, v[8 * k], y);
            y = fmaf(p.y, v[8 * k + 1], y);
            y = fmaf(p.z, v[8 * k + 2], y);
            y = fmaf(p.w, v[8 * k + 3], y);
            y = fmaf(q.x, v[8 * k + 4], y);
            y = fmaf(q.y, v[8 * k + 5], y);
            y = fmaf(q.z, v[8 * k + 6], y);
            y = fmaf(q.w, v[8 * k + 7], y);
        }
        y = group_sum<LPV>(y) * coef;
        if (sub == 0) {
            const __half h = __float2half_rn(y);
            hi[D + j] = h;
            lo[D + j] = __float2half_rn(y - __half2float(h));
        }
    }
}

// Tiles of one block's piece of unit x: pieces of equal length over all the
// call's units (ragged sequences), as long as lets the pieces be one wave of
// blocks (each unit may end in a short one), and no unit has more than n_split.
// The whole warp calls it.
template <int BK>
__device__ __forceinline__ int piece_tiles(const Args& a, const Unit& x) {
    if (a.batch == 1 || a.n_split == 1) return max(1, (x.ntiles + a.n_split - 1) / a.n_split);
    long long total = 0;
    for (int b = threadIdx.x & 31; b < a.batch; b += 32) {
        const int base = a.base[b], drafts = a.draft_lens ? a.draft_lens[b] : a.n_draft;
        if (drafts < 1 || drafts > a.n_draft || base < 0 || base > a.capacity - drafts) continue;
        const uint32_t tiles = (static_cast<uint32_t>(base + drafts) + BK - 1) / BK;
        total += static_cast<long long>(tiles) * ((drafts + a.tok_per_tile - 1) / a.tok_per_tile);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFullMask, total, o);
    total *= a.hkv;
    const int room = a.wave - a.units;  // (above zero: n_split is 1 otherwise)
    const long long even = (total + room - 1) / room;
    const int most = (x.ntiles + a.n_split - 1) / a.n_split;
    return max(1, even < x.ntiles ? max(static_cast<int>(even), most) : x.ntiles);
}

template <int D>
__global__ void __launch_bounds__(GEN_THREADS, gen_bound(D)) tree_general_kernel(const __grid_constant__ Args a) {
    constexpr int BK = GEN_BK<D>;
    extern __shared__ __align__(16) uint8_t gsm[];
    const int m = a.qjl_dims, KD = D + m, KS = gen_qk_stride(D, m), VS = D + 8;
    __half* qh = reinterpret_cast<__half*>(gsm);
    __half* ql = qh + GEN_ROWS * KS;  // (two terms)
    __half* ks = qh + a.terms * GEN_ROWS * KS;
    __half* vs = ks + BK * KS;
    float* kn = reinterpret_cast<float*>(vs + BK * VS);
    float* vnorm = kn + BK;
    float* cent = vnorm + BK;  // key centroids (key_scale c), then value centroids (sqrt(d)/4 c)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < 32) cent[tid] = tid < 16 ? a.kcent32[tid] : a.vcent32[tid - 16];
    ptx::wait_prerequisites();
    ptx::launch_dependents();
    const Unit x = unit_of<BK>(a, static_cast<int>(blockIdx.x));
    const int G = a.group, split = static_cast<int>(blockIdx.y);
    float* mine = a.parts + (static_cast<size_t>(blockIdx.x) * a.n_split + split) * (GEN_ROWS * (D + 2));
    const int per = piece_tiles<BK>(a, x);
    const long long start = static_cast<long long>(per) * split;
    const int j0 = static_cast<int>(start < x.ntiles ? start : x.ntiles), j1 = x.ntiles - j0 > per ? j0 + per : x.ntiles;
    if (x.bad && x.qt == 0 && x.kv == 0 && split == 0 && tid == 0 && a.err) atomicOr(a.err, TQ_DEVERR_SEQLEN);
    if (j1 <= j0) return;  // (the unit has fewer pieces)
    // ---- queries, prepared by tree_general_prep_kernel
    {
        const uint4* src = reinterpret_cast<const uint4*>(a.prep + static_cast<size_t>(blockIdx.x) * (GEN_ROWS * 4) * KD);
        const int per_row = KD / 8;
        for (int r = warp; r < a.terms * GEN_ROWS; r += GEN_THREADS / 32)  // (rows of the first term, then of the second)
            for (int c = lane; c < per_row; c += 32)
                copy16_async(ptx::smem_addr(qh + r * KS + 8 * c), src + r * per_row + c);
    }
    const int r0 = warp * 16 + lane / 4, r1 = r0 + 8;  // the lane's two rows
    const bool idle = warp * 16 >= x.ntok * G;         // a warp without rows only dequantises
    const bool two_terms = a.terms == 2;
    const uint64_t mk0 = r0 / G < x.ntok ? row_mask(a, x, x.tok0 + r0 / G) : 0ull;
    const uint64_t mk1 = r1 / G < x.ntok ? row_mask(a, x, x.tok0 + r1 / G) : 0ull;
    // what the lane's rows' scores are multiplied by
    const float* factors = a.row_factor + static_cast<size_t>(blockIdx.x) * GEN_ROWS;
    const float g0 = factors[r0], g1 = factors[r1];
    float o[D / 8][4], m0 = NOTHING, m1 = NOTHING, l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) o[i][q] = 0.f;
    const int kbytes = a.k_bits == 8 ? D : D * a.k_bits / 8, vbytes = a.v_bits == 8 ? D : D * a.v_bits / 8;

    // A tile's packed rows come through registers, a tile ahead: this thread
    // takes channel group cg (8 channels) of keys ck + KPP i.
    constexpr int CH = D / 8, KPP = GEN_THREADS / CH, N = BK / KPP;
    const int cg = tid % CH, ck = tid / CH;
    uint2 kraw[N], vraw[N];
    uint16_t knraw = 0, vnraw = 0, graw[2] = {0, 0};
    uint32_t zraw[2] = {0u, 0u};
    const int zw = m / 32;  // sketch words of a key
    auto raw8 = [&](const uint8_t* row, int bits) -> uint2 {
        if (bits == 8) return __ldg(reinterpret_cast<const uint2*>(row) + cg);
        if (bits == 4) return make_uint2(__ldg(reinterpret_cast<const uint32_t*>(row) + cg), 0u);
        if (bits == 2) return make_uint2(__ldg(reinterpret_cast<const uint16_t*>(row) + cg), 0u);
        // 24 bits from byte 3 cg, in one or two words of the row
        const uint32_t* w = reinterpret_cast<const uint32_t*>(row) + ((3 * cg) >> 2);
        return make_uint2(__ldg(w), (3 * cg) & 3 ? __ldg(w + (((3 * cg) & 3) > 1)) : 0u);
    };
    auto fetch = [&](int j) {
        const int key0 = j * BK, nk = min(BK, x.kend - key0);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int key = ck + KPP * i;
            kraw[i] = vraw[i] = make_uint2(0u, 0u);
            if (key < nk) {
                const size_t row = cache_row(a, x.b, x.kv, key0 + key);
                kraw[i] = raw8(a.k_codes + row * kbytes, a.k_bits);
                vraw[i] = raw8(a.v_codes + row * vbytes, a.v_bits);
            }
        }
        if (tid < BK) {
            knraw = vnraw = 0;
            if (tid < nk) {
                const size_t row = cache_row(a, x.b, x.kv, key0 + tid);
                knraw = a.k_norms[row];
                vnraw = a.v_norms[row];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = tid + GEN_THREADS * i;
            zraw[i] = 0u;
            graw[i] = 0;
            if (at < BK * zw && at / zw < nk) {
                const size_t row = cache_row(a, x.b, x.kv, key0 + at / zw);
                zraw[i] = reinterpret_cast<const uint32_t*>(a.k_qjl + row * (m / 8))[at % zw];
                graw[i] = a.k_gamma[row];
            }
        }
    };
    // eight values of a packed group, as fp16 pairs
    auto values = [&](uint2 raw, int bits, const float* ct, float n) -> uint4 {
        float y[8];
        if (bits == 8) {  // (exact as fp16; times a norm, fp16 too, one rounding)
            const uint2 p = mma::int8_to_half(raw.x), q = mma::int8_to_half(raw.y);
            uint4 v = make_uint4(p.x, p.y, q.x, q.y);
            const __half2 n2 = __float2half2_rn(n);
            __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = __hmul2(h[e], n2);
            return v;
        }
        const uint32_t codes = bits == 3 ? __funnelshift_r(raw.x, raw.y, 8 * ((3 * cg) & 3)) : raw.x;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = n * ct[(codes >> (bits * e)) & ((1u << bits) - 1u)];
        return make_uint4(ptx::pack_half2(y[0], y[1]), ptx::pack_half2(y[2], y[3]), ptx::pack_half2(y[4], y[5]),
                          ptx::pack_half2(y[6], y[7]));
    };
    fetch(j0);
    asm volatile("cp.async.wait_all;" ::: "memory");  // (the queries: the loop's first barrier shares them)
    for (int j = j0; j < j1; ++j) {
        const int key0 = j * BK, nk = min(BK, x.kend - key0);
        // ---- the tile to fp16: keys as centroids (norms multiply the fp32
        // scores), values times their norms and 2^-e; slots past the end are zeros.
        // (A value row that is not finite is left out of V~, where a zero
        // weight would turn it into NaN for rows that do not see it; its key's
        // score is NaN instead, for those that do.)
        if (tid < BK) {
            const float vn = half_bits_to_float(vnraw);
            const bool fine = fabsf(vn) < INFINITY;
            kn[tid] = fine ? half_bits_to_float(knraw) : NAN;
            vnorm[tid] = fine ? vn : 0.f;
        }
        __syncthreads();
        const float vtop = BK == 64 ? fmaxf(fabsf(vnorm[lane]), fabsf(vnorm[(lane + 32) % BK])) : fabsf(vnorm[lane]);
        const int ve = value_exponent(__uint_as_float(__reduce_max_sync(kFullMask, __float_as_uint(vtop))));
        const float vfactor = power_of_two(-ve);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int key = ck + KPP * i;
            uint4 k8 = values(kraw[i], a.k_bits, cent, 1.f);
            uint4 v8 = values(vraw[i], a.v_bits, cent + 16, vnorm[key] * vfactor);
            if (key >= nk) k8 = v8 = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(ks + key * KS + 8 * cg) = k8;
            *reinterpret_cast<uint4*>(vs + key * VS + 8 * cg) = v8;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // the sketch's channels: +-gamma
            const int at = tid + GEN_THREADS * i;
            if (at < BK * zw) {
                uint32_t* dst = reinterpret_cast<uint32_t*>(ks + (at / zw) * KS + D + 32 * (at % zw));
                const uint32_t gm = graw[i];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const uint32_t lo = gm ^ (((zraw[i] >> e) & 1u) ? 0u : 0x8000u);
                    const uint32_t hi = gm ^ (((zraw[i] >> (e + 1)) & 1u) ? 0u : 0x8000u);
                    dst[e / 2] = lo | (hi << 16);
                }
            }
        }
        __syncthreads();
        if (j + 1 < j1) fetch(j + 1);
        if (idle) {
            __syncthreads();
            continue;
        }
        // ---- scores
        float s[BK / 8][4];
#pragma unroll
        for (int n = 0; n < BK / 8; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) s[n][q] = 0.f;
        for (int c = 0; c < KD; c += 16) {
            const int cc = c + 2 * (lane & 3);
            auto w32 = [](const __half* p) { return *reinterpret_cast<const uint32_t*>(p); };
            const uint32_t h0 = w32(qh + r0 * KS + cc), h1 = w32(qh + r1 * KS + cc), h2 = w32(qh + r0 * KS + cc + 8),
                           h3 = w32(qh + r1 * KS + cc + 8);
            uint32_t y0 = 0u, y1 = 0u, y2 = 0u, y3 = 0u;
            if (two_terms) {
                y0 = w32(ql + r0 * KS + cc), y1 = w32(ql + r1 * KS + cc);
                y2 = w32(ql + r0 * KS + cc + 8), y3 = w32(ql + r1 * KS + cc + 8);
            }
#pragma unroll
            for (int n = 0; n < BK / 8; ++n) {
                const __half* kp = ks + (8 * n + lane / 4) * KS + cc;
                const uint32_t b0 = w32(kp), b1 = w32(kp + 8);
                ptx::mma_16816(s[n], h0, h1, h2, h3, b0, b1);
                if (two_terms) ptx::mma_16816(s[n], y0, y1, y2, y3, b0, b1);
            }
        }
        // ---- online softmax, in log2 units
        const uint64_t v0 = visible(mk0, key0, x.base), v1 = visible(mk1, key0, x.base);
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int n = 0; n < BK / 8; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int key = 8 * n + 2 * (lane & 3) + e;
                const float kk = kn[key];
                s[n][e] = key < nk && ((v0 >> key) & 1u) ? __fmul_rn(s[n][e] * g0, kk) : -INFINITY;
                s[n][2 + e] = key < nk && ((v1 >> key) & 1u) ? __fmul_rn(s[n][2 + e] * g1, kk) : -INFINITY;
                t0 = fmaxf(t0, s[n][e]);
                t1 = fmaxf(t1, s[n][2 + e]);
            }
#pragma unroll
        for (int q = 1; q < 4; q <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(kFullMask, t0, q));
            t1 = fmaxf(t1, __shfl_xor_sync(kFullMask, t1, q));
        }
        const float n0 = fmaxf(m0, t0 + ve), n1 = fmaxf(m1, t1 + ve);
        const float c0 = ptx::ex2(m0 - n0), c1 = ptx::ex2(m1 - n1);
        const float f0 = PSHIFT + ve - n0, f1 = PSHIFT + ve - n1;
        m0 = n0;
        m1 = n1;
        float u0 = 0.f, u1 = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= c0;
            o[i][1] *= c0;
            o[i][2] *= c1;
            o[i][3] *= c1;
        }
#pragma unroll
        for (int n = 0; n < BK / 8; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // (scores past 2^25 leave more than the four bits between the largest weight and fp16's)
                const float x0 = __fadd_rn(s[n][e], f0), x1 = __fadd_rn(s[n][2 + e], f1);
                s[n][e] = ptx::ex2(x0 > 15.5f ? 15.5f : x0);  // (NaN stays)
                s[n][2 + e] = ptx::ex2(x1 > 15.5f ? 15.5f : x1);
                u0 += s[n][e];
                u1 += s[n][2 + e];
            }
        l0 = fmaf(l0, c0, u0 * vfactor);
        l1 = fmaf(l1, c1, u1 * vfactor);
        // ---- O += P V
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
            const uint32_t a0 = ptx::pack_half2(s[2 * kk][0], s[2 * kk][1]), a1 = ptx::pack_half2(s[2 * kk][2], s[2 * kk][3]);
            const uint32_t a2 = ptx::pack_half2(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                           a3 = ptx::pack_half2(s[2 * kk + 1][2], s[2 * kk + 1][3]);
            const uint32_t vrow = ptx::smem_addr(vs + (16 * kk + (lane & 15)) * VS);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                uint32_t b0, b1;
                ldmatrix_x2_trans(b0, b1, vrow + 16 * i);
                ptx::mma_16816(o[i], a0, a1, a2, a3, b0, b1);
            }
        }
        __syncthreads();
    }
    if (idle) return;
#pragma unroll
    for (int q = 1; q < 4; q <<= 1) {
        l0 += __shfl_xor_sync(kFullMask, l0, q);
        l1 += __shfl_xor_sync(kFullMask, l1, q);
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        *reinterpret_cast<float2*>(mine + r0 * D + 8 * i + 2 * (lane & 3)) = make_float2(o[i][0], o[i][1]);
        *reinterpret_cast<float2*>(mine + r1 * D + 8 * i + 2 * (lane & 3)) = make_float2(o[i][2], o[i][3]);
    }
    if ((lane & 3) == 0) {
        mine[GEN_ROWS * D + r0] = piece_reference(m0, l0);
        mine[GEN_ROWS * D + r1] = piece_reference(m1, l1);
        mine[GEN_ROWS * (D + 1) + r0] = l0;
        mine[GEN_ROWS * (D + 1) + r1] = l1;
    }
}

// The general kernel's output: block (unit, 2 rows), four warps a row.  Each
// of them adds every fourth piece (so a call's few rows still keep many loads
// in flight), the first joins the four and applies the inverse rotation.
constexpr int GM_ROWS = 2, GM_WARPS = 4, GM_THREADS = GM_ROWS * GM_WARPS * 32, GM_BATCH = 4;
template <int D>
__global__ void __launch_bounds__(GM_THREADS) tree_general_merge_kernel(const __grid_constant__ Args a) {
    constexpr int N = D / 32;
    __shared__ float sums[GM_ROWS][GM_WARPS][D];
    __shared__ float total[GM_ROWS][GM_WARPS];
    ptx::wait_prerequisites();
    ptx::launch_dependents();
    const Unit x = unit_of<GEN_BK<D>>(a, static_cast<int>(blockIdx.x));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mr = warp / GM_WARPS, part = warp % GM_WARPS;
    const int r = static_cast<int>(blockIdx.y) * GM_ROWS + mr, G = a.group, t = r / G, g = r % G;
    // rows past the sequence's drafts are left as they are (all n_draft rows of a refused sequence are zeros)
    const int rows = x.bad ? min(a.tok_per_tile, a.n_draft - x.tok0) : x.ntok;
    const bool live = t < rows;
    const int per = piece_tiles<GEN_BK<D>>(a, x), np = x.bad || !live ? 0 : (x.ntiles - 1) / per + 1;
    const float* first = a.parts + static_cast<size_t>(blockIdx.x) * a.n_split * (GEN_ROWS * (D + 2));
    auto piece = [&](int j) { return first + static_cast<size_t>(j) * (GEN_ROWS * (D + 2)); };
    float M = -INFINITY;
    for (int j = lane; j < np; j += 32) M = fmaxf(M, __ldcg(piece(j) + GEN_ROWS * D + r));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
    float L = 0.f, e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = 0.f;
    for (int j0 = part; j0 < np; j0 += GM_WARPS * GM_BATCH) {
        float v[GM_BATCH][N], w[GM_BATCH];
#pragma unroll
        for (int k = 0; k < GM_BATCH; ++k) {
            const int j = j0 + GM_WARPS * k;
            w[k] = 0.f;
            float m = -INFINITY;
            if (j < np) m = __ldcg(piece(j) + GEN_ROWS * D + r);
            if (m > -INFINITY) {
                w[k] = ptx::ex2(m - M);
                L = fmaf(__ldcg(piece(j) + GEN_ROWS * (D + 1) + r), w[k], L);
            }
            const float* p = piece(w[k] != 0.f ? j : 0) + r * D + lane * N;
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float2 y = w[k] != 0.f ? __ldcg(reinterpret_cast<const float2*>(p + i)) : make_float2(0.f, 0.f);
                v[k][i] = y.x;
                v[k][i + 1] = y.y;
            }
        }
#pragma unroll
        for (int k = 0; k < GM_BATCH; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) e[i] = fmaf(v[k][i], w[k], e[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) sums[mr][part][lane * N + i] = e[i];
    if (lane == 0) total[mr][part] = L;
    __syncthreads();
    if (part != 0 || !live) return;
    L = 0.f;
#pragma unroll
    for (int k = 0; k < GM_WARPS; ++k) L += total[mr][k];
    const float inv = L == 0.f ? 0.f : a.out_scale / L;  // (NaN stays NaN)
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < GM_WARPS; ++k) y += sums[mr][k][lane * N + i];
        e[i] = y * inv;
    }
    if (a.v_bits != 8) {
        fwht_registers(e);
        fwht_lanes<N, 32>(e, lane);
        const float rs = rsqrtf(static_cast<float>(D));
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = flip_sign(e[i] * rs, sign_bit(a.signs, lane * N + i));
    }
    store_row<N>(a.out, ((static_cast<size_t>(x.b) * a.n_draft + x.tok0 + t) * a.hq + x.kv * G + g) * D + lane * N, e,
                 a.out_dtype);
}

// The queries of the tensor-memory kernel, once a call: rotated (turbo keys),
// times the softmax scale and the inverse key-table scale in log2 units (and a
// power of two: see row_exponent), as one or two fp16 terms in the order its
// threads load them.  A row on 4 lanes,
// 32 channels each (the chunks of the encoders), 8 rows a warp.
__global__ void __launch_bounds__(256) tree_prep_kernel(const __grid_constant__ Args a) {
    constexpr int D = mma::D, LPV = D / 32;
    ptx::wait_prerequisites();
    ptx::launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane % LPV;
    const long long row = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * 8 + lane / LPV;
    const int u = static_cast<int>(row / a.part_rows), ur = static_cast<int>(row % a.part_rows);
    if (u >= a.units) return;  // (whole warps: part_rows is a multiple of 32)
    const int G = a.group, rt = ur / G, rh = ur % G;
    const int qt = u % a.qtiles, kv = (u / a.qtiles) % a.hkv, b = u / a.qtiles / a.hkv, t = qt * a.tok_per_tile + rt;
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = 0.f;
    if (rt < a.tok_per_tile && t < a.n_draft) {
        const size_t off = ((static_cast<size_t>(b) * a.n_draft + t) * a.hq + kv * G + rh) * D;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const size_t at = off + 8 * (sub + LPV * k);
            load4(a.q, at, a.q_dtype, *reinterpret_cast<float (*)[4]>(&x[8 * k]));
            load4(a.q, at + 4, a.q_dtype, *reinterpret_cast<float (*)[4]>(&x[8 * k + 4]));
        }
    }
    __syncwarp();
    float scale = a.score_scale;
    if (a.k_bits != 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[8 * k + e] = flip_sign(x[8 * k + e], sign_bit(a.signs, 8 * (sub + LPV * k) + e));
        fwht_registers(x);
        fwht_lanes<32, LPV>(x, sub);
        scale *= 0.08838834764831845f;  // 1 / sqrt(128)
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(x[i]));
    const int k2 = row_exponent(group_max<LPV>(top) * scale);
    const float shrink = power_of_two(-k2);
    if (sub == 0) a.row_factor[row] = power_of_two(k2);
    uint4* dst = reinterpret_cast<uint4*>(a.prep + static_cast<size_t>(u) * mma::prep_bytes(a.part_rows, a.terms)) + ur;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float v0 = x[8 * k + 2 * e] * scale * shrink, v1 = x[8 * k + 2 * e + 1] * scale * shrink;
            hi[e] = ptx::pack_half2(v0, v1);
            const float2 h = mma::half2_float2(hi[e]);
            lo[e] = ptx::pack_half2(v0 - h.x, v1 - h.y);
        }
        const size_t c = static_cast<size_t>(sub + LPV * k) * a.part_rows;
        dst[c] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (a.terms == 2) dst[16 * static_cast<size_t>(a.part_rows) + c] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// The rows of the units that the tensor-memory kernel cut between blocks (it
// wrote the others' outputs itself): block (unit, 8 rows).  A warp per row
// finds the pieces' weights 2^(m - M) / sum; then thread (row, 4 channels)
// adds its channels over the pieces, whose rows lie next to each other, and a
// warp per row applies the inverse rotation.
constexpr int MM_ROWS = 8, MM_THREADS = 256, MM_BATCH = 8;
__global__ void __launch_bounds__(MM_THREADS) tree_mma_merge_kernel(const __grid_constant__ Args a, int nblocks) {
    extern __shared__ float mm_smem[];  // weights [pieces][8], then rows [8][128 + 4]
    ptx::wait_prerequisites();  // launched as a programmatic dependent of the attention kernel
    ptx::launch_dependents();
    const int u = static_cast<int>(blockIdx.x);
    const uint32_t total = a.sched[a.units], pu = a.sched[u], pn = a.sched[u + 1];
    if (pn <= pu) return;
    const uint32_t C = static_cast<uint32_t>(nblocks) > total ? total : static_cast<uint32_t>(nblocks);
    const int ca = mma::block_of(pu, total, C), cz = mma::block_of(pn - 1, total, C);
    if (ca == cz) return;
    const Unit x = unit_of<mma::BK>(a, u);
    const int G = a.group, r0 = static_cast<int>(blockIdx.y) * MM_ROWS;
    if (r0 / G >= x.ntok) return;
    const int np = cz - ca + 1, R = a.part_rows, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float* wts = mm_smem;
    float* rows = mm_smem + ((np * MM_ROWS + 3) & ~3);
    const size_t slot = mma::part_floats(R);
    auto piece = [&](int j) { return a.parts + static_cast<size_t>(mma::part_slot(ca + j, ca)) * slot; };
    {
        const int r = r0 + warp;
        const bool in = r / G < x.ntok;  // (other rows hold nothing)
        float M = -INFINITY, L = 0.f;
        for (int j = lane; j < np; j += 32) {
            const float m = in ? __ldcg(piece(j) + R * mma::D + r) : -INFINITY;
            wts[j * MM_ROWS + warp] = m;
            M = fmaxf(M, m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
        for (int j = lane; j < np; j += 32) {
            const float m = wts[j * MM_ROWS + warp];
            float w = 0.f;
            if (m > -INFINITY) {
                w = ptx::ex2(m - M);
                L = fmaf(__ldcg(piece(j) + R * (mma::D + 1) + r), w, L);
            }
            wts[j * MM_ROWS + warp] = w;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(kFullMask, L, o);
        const float inv = L == 0.f ? 0.f : a.out_scale / L;  // (NaN stays NaN)
        for (int j = lane; j < np; j += 32) wts[j * MM_ROWS + warp] *= inv;
    }
    __syncthreads();
    {
        const int r = tid & 7, chunk = tid >> 3;
        const size_t at = (static_cast<size_t>(chunk) * R + r0 + r) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j0 = 0; j0 < np; j0 += MM_BATCH) {
            float4 v[MM_BATCH];
            float w[MM_BATCH];
#pragma unroll
            for (int k = 0; k < MM_BATCH; ++k) {
                w[k] = j0 + k < np ? wts[(j0 + k) * MM_ROWS + r] : 0.f;
                // (rows that were never written, or weigh nothing, are not read)
                v[k] = w[k] != 0.f ? __ldcg(reinterpret_cast<const float4*>(piece(j0 + k) + at))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < MM_BATCH; ++k) {
                acc.x = fmaf(v[k].x, w[k], acc.x);
                acc.y = fmaf(v[k].y, w[k], acc.y);
                acc.z = fmaf(v[k].z, w[k], acc.z);
                acc.w = fmaf(v[k].w, w[k], acc.w);
            }
        }
        *reinterpret_cast<float4*>(rows + r * (mma::D + 4) + 4 * chunk) = acc;
    }
    __syncthreads();
    const int r = r0 + warp, t = r / G, g = r % G;
    if (t >= x.ntok) return;
    const float4 y = *reinterpret_cast<const float4*>(rows + warp * (mma::D + 4) + 4 * lane);
    float e[4] = {y.x, y.y, y.z, y.w};
    if (a.v_bits != 8) {
        fwht_registers(e);
        fwht_lanes<4, 32>(e, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = flip_sign(e[i] * 0.08838834764831845f, sign_bit(a.signs, 4 * lane + i));
    }
    store_row<4>(a.out, ((static_cast<size_t>(x.b) * a.n_draft + x.tok0 + t) * a.hq + x.kv * G + g) * mma::D + 4 * lane, e,
                 a.out_dtype);
}

// Work layout of a call.  general: up to n_split blocks per unit of GEN_ROWS rows.
// Tensor-memory kernel: units of up to 128 rows, or (pair) 256 where a kv head
// has more than 128 (its drafts spread evenly over its units), the
// tile sequence shared by one block per SM (spread) or, past SCHED_MAX units,
// a block per unit; workspace: the prepared queries, then (spread) the schedule
// and two partial outputs per block.
struct Plan {
    long long units;
    int tok_per_tile, qtiles, n_split, wave, spread, blocks, pair, terms, part_rows;
    size_t prep_bytes, factor_bytes, sched_bytes, bytes;  // (the rows' factors end the prepared queries)
};

static bool mma_supported(const tq_params& p) { return p.head_dim == mma::D && p.qjl_dims == 0; }

static Plan mma_plan(const tq_params& p, int batch, int n_draft, int sms, bool one_term) {
    Plan pl{};
    const int group = p.num_q_heads / p.num_kv_heads;
    pl.terms = one_term ? 1 : 2;
    pl.pair = one_term && n_draft > mma::BM / group;
    const int most = (pl.pair ? 2 * mma::BM : mma::BM) / group;
    pl.qtiles = (n_draft + most - 1) / most;
    pl.tok_per_tile = (n_draft + pl.qtiles - 1) / pl.qtiles;
    pl.pair = pl.pair && pl.tok_per_tile * group > mma::BM;
    pl.part_rows = (pl.tok_per_tile * group + 31) / 32 * 32;
    pl.units = static_cast<long long>(batch) * p.num_kv_heads * pl.qtiles;
    pl.spread = pl.units <= mma::SCHED_MAX;
    pl.blocks = pl.spread ? sms : static_cast<int>(pl.units);
    pl.factor_bytes = static_cast<size_t>(pl.units) * pl.part_rows * sizeof(float);
    pl.prep_bytes = static_cast<size_t>(pl.units) * mma::prep_bytes(pl.part_rows, pl.terms) + pl.factor_bytes;
    pl.bytes = pl.prep_bytes;
    if (pl.spread) {
        pl.sched_bytes = (static_cast<size_t>(pl.units + 1) * 4 + 255) / 256 * 256;
        pl.bytes += pl.sched_bytes + 2ull * pl.blocks * mma::part_floats(pl.part_rows) * sizeof(float);
    }
    return pl;
}

static Plan general_plan(const tq_params& p, int batch, int n_draft, int sms, bool one_term) {
    Plan pl{};
    pl.terms = one_term ? 1 : 2;
    pl.tok_per_tile = GEN_ROWS / (p.num_q_heads / p.num_kv_heads);
    pl.qtiles = (n_draft + pl.tok_per_tile - 1) / pl.tok_per_tile;
    pl.units = static_cast<long long>(batch) * p.num_kv_heads * pl.qtiles;
    // The pieces that one wave of blocks gives each unit (a second wave of a few
    // blocks costs as much as the first: 87 against 63 us for 16 drafts over 6000
    // tokens at d = 256), or one where the units alone fill the wave.  The longest
    // sequences of a batch may take twice their share (see piece_tiles: 8
    // sequences of 600 to 6000 tokens, d = 128 with a sketch, 16-token pages: 214
    // -> 152 us), which costs one sequence alone 2 us and is left out there.
    pl.wave = gen_resident(p.head_dim, p.qjl_dims, pl.terms) * sms;
    const long long n = pl.wave <= pl.units ? 1 : (batch == 1 ? 1ll : 2ll) * pl.wave / pl.units;
    pl.n_split = static_cast<int>(n > 256 ? 256 : n);
    pl.factor_bytes = static_cast<size_t>(pl.units) * GEN_ROWS * sizeof(float);
    pl.prep_bytes = static_cast<size_t>(pl.units) * (GEN_ROWS * 4) * (p.head_dim + p.qjl_dims) + pl.factor_bytes;
    pl.bytes = pl.prep_bytes + static_cast<size_t>(pl.units) * pl.n_split * GEN_ROWS * (p.head_dim + 2) * sizeof(float);
    return pl;
}

template <int D>
static cudaError_t launch_general(const Args& a, cudaStream_t s) {
    const size_t smem = gen_smem(D, a.qjl_dims, a.terms);
    // (the widest sketch's for every call: another thread's call may set it between this line and the launch)
    cudaError_t e = cudaFuncSetAttribute(tree_general_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(gen_smem(D, D, 2)));
    if (e != cudaSuccess) return e;
    constexpr int per_block = PREP_THREADS / 32 * (32 / (D / 32));
    const long long prep = (static_cast<long long>(a.units) * GEN_ROWS + per_block - 1) / per_block;
    e = mma::launch_dependent(tree_general_prep_kernel<D>, dim3(static_cast<unsigned>(prep), a.qjl_dims ? (a.qjl_dims + PREP_SKETCH - 1) / PREP_SKETCH : 1),
                              dim3(PREP_THREADS), 0u, s, a);
    if (e != cudaSuccess) return e;
    e = mma::launch_dependent(tree_general_kernel<D>, dim3(static_cast<unsigned>(a.units), static_cast<unsigned>(a.n_split)),
                              dim3(GEN_THREADS), static_cast<uint32_t>(smem), s, a);
    if (e != cudaSuccess) return e;
    return mma::launch_dependent(tree_general_merge_kernel<D>, dim3(static_cast<unsigned>(a.units), GEN_ROWS / GM_ROWS),
                                 dim3(GM_THREADS), 0u, s, a);
}

static cudaError_t launch_mma(const Args& a, const Plan& pl, cudaStream_t s) {
    const long long warps = pl.units * a.part_rows / 8;
    cudaError_t e = mma::launch_dependent(tree_prep_kernel, dim3(static_cast<unsigned>((warps + 7) / 8)), dim3(256), 0u, s, a);
    if (e != cudaSuccess) return e;
    switch (a.k_bits) {
        case 2: e = launch_mma_k2(a.v_bits, a, pl.blocks, s); break;
        case 3: e = launch_mma_k3(a.v_bits, a, pl.blocks, s); break;
        case 4: e = launch_mma_k4(a.v_bits, a, pl.blocks, s); break;
        default: e = launch_mma_k8(a.v_bits, a, pl.blocks, s); break;
    }
    if (e != cudaSuccess || !pl.spread) return e;
    const int rows = (a.tok_per_tile * a.group + MM_ROWS - 1) / MM_ROWS;
    const uint32_t smem = (pl.blocks * MM_ROWS + 4 + MM_ROWS * (mma::D + 4)) * 4u;
    return mma::launch_dependent(tree_mma_merge_kernel, dim3(static_cast<unsigned>(a.units), static_cast<unsigned>(rows)),
                                 dim3(MM_THREADS), smem, s, a, pl.blocks);
}

static Plan plan_of(const tq_params& p, int batch, int n_draft, int sms, int out_dtype) {
    return mma_supported(p) ? mma_plan(p, batch, n_draft, sms, out_dtype == TQ_BF16)
                            : general_plan(p, batch, n_draft, sms, out_dtype == TQ_BF16);
}

static tq_status attend(const tq_params* params, const tq_codebook* kcb, const tq_codebook* vcb, const void* d_q,
                        tq_dtype q_dtype, int32_t n_draft, const uint64_t* d_mask, const int32_t* d_base,
                        const int32_t* d_draft_lens, const tq_cache* cache, const PageMap* pm, void* d_out,
                        tq_dtype out_dtype, void* d_workspace, size_t workspace_bytes, uint32_t* d_error,
                        void* stream) {
    tq_status st = validate_params(params);
    if (st != TQ_OK) return st;
    const tq_params& p = *params;
    if ((st = validate_cache(p, cache)) != TQ_OK) return st;
    if (!d_q || !d_out || !d_mask || !d_base || n_draft < 1) return TQ_ERR_INVALID_ARG;
    for (const tq_dtype t : {q_dtype, out_dtype})
        if (t != TQ_F32 && t != TQ_BF16 && t != TQ_F16) return TQ_ERR_INVALID_ARG;
    if (n_draft > MAX_DRAFTS) return TQ_ERR_UNSUPPORTED;
    if (!aligned16(d_q) || !aligned16(d_out) || reinterpret_cast<uintptr_t>(d_mask) % 8) return TQ_ERR_ALIGNMENT;
    if (p.k_mode == TQ_MODE_TURBO && (st = validate_codebook(kcb, p.head_dim, p.k_bits)) != TQ_OK) return st;
    if (p.v_mode == TQ_MODE_TURBO && (st = validate_codebook(vcb, p.head_dim, p.v_bits)) != TQ_OK) return st;
    const int batch = pm ? pm->batch : cache->batch;
    const int sms = num_sms_current();
    if (sms <= 0) return TQ_ERR_CUDA;
    const int capacity = pm ? pm->max_blocks * pm->block_size : cache->capacity;
    const bool mm = mma_supported(p);
    Plan pl = plan_of(p, batch, n_draft, sms, out_dtype);
    if (pl.units > INT32_MAX) return TQ_ERR_INVALID_ARG;
    if (mm && pl.spread && pl.units * (capacity / mma::BK + 1ll) >= (1ll << 31)) {
        // the shared tile sequence is counted in 32 bits: a block per unit instead
        pl.spread = 0;
        pl.blocks = static_cast<int>(pl.units);
        pl.bytes = pl.prep_bytes;
    }
    if (!d_workspace) return TQ_ERR_INVALID_ARG;
    if (workspace_bytes < pl.bytes) return TQ_ERR_CAPACITY;
    if (!aligned16(d_workspace)) return TQ_ERR_ALIGNMENT;
    if (mm) {  // (the code tables' lookups carry their shared-window addresses)
        int reserved = 0, dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess)
            return TQ_ERR_CUDA;
        if (static_cast<uint32_t>(reserved) != mma::SMEM_WINDOW) return TQ_ERR_UNSUPPORTED;
    }
    Args a{};
    a.k_codes = cache->k_codes;
    a.v_codes = cache->v_codes;
    a.k_norms = cache->k_norms;
    a.v_norms = cache->v_norms;
    a.k_qjl = cache->k_qjl;
    a.k_gamma = cache->k_gamma;
    a.sketch = cache->qjl_matrix;
    a.q = d_q;
    a.mask = d_mask;
    a.base = d_base;
    a.draft_lens = d_draft_lens;
    a.out = d_out;
    a.err = d_error;
    a.prep = static_cast<uint8_t*>(d_workspace);
    a.row_factor = reinterpret_cast<float*>(a.prep + pl.prep_bytes - pl.factor_bytes);
    a.sched = reinterpret_cast<uint32_t*>(a.prep + pl.prep_bytes);
    a.parts = reinterpret_cast<float*>(a.prep + pl.prep_bytes + pl.sched_bytes);
    a.capacity = capacity;
    if (pm) {
        a.table = pm->table;
        a.max_blocks = pm->max_blocks;
        a.block_size = pm->block_size;
        a.num_blocks = pm->num_blocks;
        a.block_magic = UINT64_MAX / static_cast<uint32_t>(pm->block_size) + 1;  // (block_size is 16 or more)
    }
    a.q_dtype = q_dtype;
    a.out_dtype = out_dtype;
    a.batch = batch;
    a.hq = p.num_q_heads;
    a.hkv = p.num_kv_heads;
    a.group = p.num_q_heads / p.num_kv_heads;
    a.n_draft = n_draft;
    a.k_bits = p.k_mode == TQ_MODE_INT8 ? 8 : p.k_bits;
    a.v_bits = p.v_mode == TQ_MODE_INT8 ? 8 : p.v_bits;
    a.qjl_dims = p.qjl_dims;
    a.tok_per_tile = pl.tok_per_tile;
    a.qtiles = pl.qtiles;
    a.units = static_cast<int>(pl.units);
    a.n_split = pl.n_split;
    a.wave = pl.wave;
    a.spread = pl.spread;
    a.pair = pl.pair;
    a.terms = pl.terms;
    a.part_rows = pl.part_rows;
    a.staged_norms = pm || capacity % 8 == 0;
    const double rd = std::sqrt(static_cast<double>(p.head_dim));
    const double sm = p.sm_scale > 0.0f ? static_cast<double>(p.sm_scale) : 1.0 / rd;
    // key centroids enter at the codebook's fp16 scale, which rounds the table
    // best; the values' as sqrt(d)/4 c or q / 128, below one (times a norm they stay
    // below the fp16 range)
    double ak = 1.0 / 128.0;
    if (a.k_bits < 8) {
        ak = kcb->fp16_scale > 0.0 ? kcb->fp16_scale : rd;
        int e;
        if (mm) ak = std::frexp(ak, &e) * 16.0 * mma::KEY_SHIFT;  // (a caller's scale brought to [8, 16) too)
    }
    a.key_scale = static_cast<float>(ak);
    a.score_scale = static_cast<float>(sm * 1.4426950408889634 / ak);
    // (the tensor-memory kernel rounds the value table itself to fp16: at its codebook's scale too)
    const double av = a.v_bits == 8 ? 1.0 / 128.0 : 0.25 * (mm && vcb->fp16_scale > 0.0 ? vcb->fp16_scale : rd);
    a.out_scale = static_cast<float>(1.0 / av);
    for (int j = 0; j < 16; ++j) {
        a.kcent32[j] = a.k_bits < 8 && j < (1 << a.k_bits) ? static_cast<float>(kcb->centroids[j] * ak) : 0.f;
        a.vcent32[j] = a.v_bits < 8 && j < (1 << a.v_bits) ? static_cast<float>(vcb->centroids[j] * av) : 0.f;
        a.kcent[j] = __half_as_ushort(__float2half_rn(a.kcent32[j]));
        a.vcent[j] = __half_as_ushort(__float2half_rn(a.vcent32[j]));
    }
    rotation_sign_bits(p.seed, p.head_dim, a.signs);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (mm) e = launch_mma(a, pl, s);
    else switch (p.head_dim) {
        case 64: e = launch_general<64>(a, s); break;
        case 128: e = launch_general<128>(a, s); break;
        default: e = launch_general<256>(a, s); break;
    }
    return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace tree
}  // namespace tq

// =================================================================== C ABI
extern "C" {

tq_status tq_tree_workspace_bytes(const tq_params* params, int32_t batch, int32_t n_draft, size_t* bytes) {
    using namespace tq;
    const tq_status st = validate_params(params);
    if (st != TQ_OK) return st;
    if (!bytes || batch < 1 || n_draft < 1) return TQ_ERR_INVALID_ARG;
    if (n_draft > tree::MAX_DRAFTS) return TQ_ERR_UNSUPPORTED;
    const int sms = num_sms_current();
    if (sms <= 0) return TQ_ERR_CUDA;
    // (for every output type)
    const size_t a = tree::plan_of(*params, batch, n_draft, sms, TQ_BF16).bytes;
    const size_t b = tree::plan_of(*params, batch, n_draft, sms, TQ_F32).bytes;
    *bytes = a > b ? a : b;
    return TQ_OK;
}

tq_status tq_tree_attention(const tq_params* params, const tq_codebook* kcb, const tq_codebook* vcb, const void* d_q,
                            tq_dtype q_dtype, int32_t n_draft, const uint64_t* d_mask, const int32_t* d_base_lens,
                            const int32_t* d_draft_lens, const tq_cache* cache, void* d_out, tq_dtype out_dtype,
                            void* d_workspace, size_t workspace_bytes, uint32_t* d_error, void* stream) {
    return tq::tree::attend(params, kcb, vcb, d_q, q_dtype, n_draft, d_mask, d_base_lens, d_draft_lens, cache, nullptr,
                            d_out, out_dtype, d_workspace, workspace_bytes, d_error, stream);
}

tq_status tq_tree_attention_paged(const tq_params* params, const tq_codebook* kcb, const tq_codebook* vcb,
                                  const void* d_q, tq_dtype q_dtype, int32_t n_draft, const uint64_t* d_mask,
                                  const int32_t* d_base_lens, const int32_t* d_draft_lens, const tq_cache* pool,
                                  const tq_block_table* table, void* d_out, tq_dtype out_dtype, void* d_workspace,
                                  size_t workspace_bytes, uint32_t* d_error, void* stream) {
    if (!params) return TQ_ERR_INVALID_ARG;
    tq::PageMap pm;
    const tq_status st = tq::validate_pages(*params, pool, table, &pm);
    if (st != TQ_OK) return st;
    return tq::tree::attend(params, kcb, vcb, d_q, q_dtype, n_draft, d_mask, d_base_lens, d_draft_lens, pool, &pm,
                            d_out, out_dtype, d_workspace, workspace_bytes, d_error, stream);
}

}  // extern "C"
