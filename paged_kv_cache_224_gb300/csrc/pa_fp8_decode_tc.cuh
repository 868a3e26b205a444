// Device code of the tensor-core decode over an 8-bit cache (head_dim 128); see
// pa_fp8_decode_tc.cu for the design.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "pa_decode_tc.cuh"
#include "pa_fp8.cuh"

namespace pa {
namespace tc8 {

using tcd::sts128;

constexpr int kD = 128;                  // head_dim: a row of codes is one 128-byte swizzle row
constexpr int kKeys = 128;               // keys per tile (M of the QK^T MMA)
constexpr int kSlot = kKeys * kD;        // 16 KB: one K or V tile
constexpr int kThreads = 192;
constexpr float kRescale = 8.0f;         // log2 units a maximum may lag behind
constexpr float kLift = 7.0f;            // weights are 2^(z - M + kLift), at most 2^15
constexpr int kQPieces = 3, kPPieces = 4;

// G heads of a kv head take GP rows a piece; the MMAs' N is the four pieces' rows.
template <int G, int S_>
struct Lay {
    static constexpr int S = S_;
    static constexpr int GP = G <= 4 ? 4 : 8;
    static constexpr int N = 4 * GP;
    static constexpr uint32_t kCols = N == 16 ? 64 : 128;   // TMEM: S^T x 2 buffers, O^T
    static constexpr uint32_t kColO = 2 * N;
    static constexpr int kOffQ = S * kSlot;
    static constexpr int kOffP = kOffQ + N * 128;
    static constexpr int kOffBar = kOffP + 2 * N * 128;
    static constexpr int kOffXch = kOffBar + 256;           // [2][4 warps][GP] maxima, [4 warps][GP] sums, [GP] query scales
    static constexpr int kUsed = kOffXch + (2 * 4 * GP + 4 * GP + GP) * 4;
    static constexpr int kAlloc = kUsed + 1024;             // room to align the base to 1 KB
    static_assert((2 * S + 7) * 8 + 8 <= 256, "barrier area");
};

// kind::f8f6f4, fp32 accumulator: A e4m3, B e4m3 or e5m2.
__host__ __device__ constexpr uint32_t instr_desc8(bool b_e5m2, bool a_mn_major, int m, int n) {
    return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn_major ? 1u : 0u) << 15) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// 2-D tensor copy global -> shared of the box at (0, row), completing bytes on `bar`.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *map, int row, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void sts8(uint32_t addr, unsigned v) {
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, unsigned a, unsigned b) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// Two values as e5m2 codes, and what those stand for: e5m2 is the upper byte of an fp16.
__device__ __forceinline__ unsigned e5m2x2(float a, float b) {
    return (unsigned)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E5M2);
}
__device__ __forceinline__ float2 from_e5m2x2(unsigned two) {
    const unsigned w = __byte_perm(two, 0u, 0x1404);
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Reduce G values of every lane across the warp; lane l ends with the result for
// value l / (32 / G).
template <bool kMax, int G>
__device__ __forceinline__ float warp_scatter(const float (&v)[G], int lane) {
    auto op = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
    float a[G];
#pragma unroll
    for (int i = 0; i < G; ++i) a[i] = v[i];
    int m = 16;
#pragma unroll
    for (int n = G; n > 1; n >>= 1, m >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int k = 0; k < n / 2; ++k) {
            const float keep = up ? a[k + n / 2] : a[k], send = up ? a[k] : a[k + n / 2];
            a[k] = op(keep, __shfl_xor_sync(kFull, send, m));
        }
    }
#pragma unroll
    for (; m > 0; m >>= 1) a[0] = op(a[0], __shfl_xor_sync(kFull, a[0], m));
    return a[0];
}

struct Unit {
    int part, s, kvh, tok0, ntok, ntiles;
    bool skip;    // a partition past the sequence's end
    bool direct;  // the whole sequence
};

__device__ __forceinline__ Unit unit_of(const DecodeParams &p, int unit, int bs, bool speaks) {
    Unit u;
    const int per_part = p.num_seqs * p.num_kv_heads;
    u.part = unit / per_part;
    const int rem = unit - u.part * per_part;
    u.s = rem / p.num_kv_heads;
    u.kvh = rem - u.s * p.num_kv_heads;
    int L = p.context_lens[u.s];
    const int cap = min(p.max_context_len, p.max_blocks_per_seq * bs);
    if (L < 0 || L > cap) {
        if (speaks && u.part == 0 && u.kvh == 0) flag_error(p.d_err, PA_DEVERR_CONTEXT_RANGE);
        L = L < 0 ? 0 : cap;
    }
    const int pt = p.partition_tokens;
    const int nparts = L > 0 ? (L + pt - 1) / pt : 1;
    u.skip = u.part >= nparts;
    u.tok0 = u.part * pt;
    u.ntok = u.skip ? 0 : min(L, u.tok0 + pt) - u.tok0;
    u.ntiles = (u.ntok + kKeys - 1) / kKeys;
    u.direct = nparts == 1;
    return u;
}

// A unit without keys: zeros, or an empty partial.
template <typename T, int G>
__device__ __forceinline__ void empty_unit(const DecodeParams &p, const Unit &u, int tid) {
    if (tid >= G * 16) return;
    const int h = tid >> 4, c = tid & 15;
    const size_t row = (size_t)u.s * p.num_heads + (size_t)u.kvh * G + h;
    if (u.direct) {
        *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + row * kD + c * 8) = make_uint4(0, 0, 0, 0);
    } else {
        const size_t at = row * p.slots + u.part;
        float4 *dst = reinterpret_cast<float4 *>(p.ws_acc + at * kD + c * 8);
        dst[0] = dst[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c == 0) p.ws_ml[at] = make_float2(kEmptyMax, 0.f);
    }
}

// One unit with keys, by the CTA's six warps.
template <typename T, int BS, int G, int S>
__device__ __forceinline__ void run_unit(const Fp8DecodeParams &fp, const CUtensorMap *tmk, const CUtensorMap *tmv,
                                         const Unit &u, unsigned char *smem, uint32_t sb, uint32_t tmem) {
    using L = Lay<G, S>;
    constexpr int GP = L::GP, N = L::N;
    constexpr int kBPT = kKeys / BS;  // blocks per tile
    static_assert(kKeys % BS == 0 && BS % 8 == 0 && 32 % kBPT == 0, "block_size");
    const DecodeParams &p = fp.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ntiles = u.ntiles, ntok = u.ntok, kvh = u.kvh;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kOffBar);  // [S] TMA -> MMA
    uint64_t *empty = full + S;                                        // [S] MMA -> TMA
    uint64_t *q_full = empty + S;                                      // softmax threads -> MMA (Q^T written)
    uint64_t *s_full = q_full + 1;                                     // [2] MMA -> softmax (S^T of a tile ready)
    uint64_t *p_full = s_full + 2;                                     // [2] softmax -> MMA (P^T written, O rescaled)
    uint64_t *pv_done = p_full + 2;                                    // [2] MMA -> softmax (PV of a tile complete)
    float *xmax = reinterpret_cast<float *>(smem + L::kOffXch);
    float *xsum = xmax + 2 * 4 * GP, *qscale = xsum + 4 * GP;
    // ring items in consumption order: K(0), then K(j), V(j-1) for j >= 1, then V(last)
    auto item_k = [](int j) { return j == 0 ? 0 : 2 * j - 1; };
    auto item_v = [ntiles](int j) { return j + 1 < ntiles ? 2 * j + 2 : 2 * j + 1; };
    const int32_t *table = p.block_tables + (size_t)u.s * p.table_stride + u.tok0 / BS;

    if (warp == 0) {
        // ============================================================ producer
        const int nblk = (ntok + BS - 1) / BS;
        const int oob = p.num_blocks * p.num_kv_heads * BS;  // first row past the pool: zero fill
        const uint64_t pol = policy_evict_first();
        constexpr int kTilesPerChunk = 32 / kBPT;
        // table entries 32 at a time, one per lane, a chunk ahead of use
        auto chunk = [&](int c) { return c * 32 + lane < nblk ? table[c * 32 + lane] : -1; };
        int ent_cur = chunk(0), ent_nxt = chunk(1);
        int item = 0;
        auto load = [&](const CUtensorMap *map, int y) {
            const int sl = item % S;
            if (lane == 0) {
                if (item >= S) wait_or_flag(&empty[sl], (uint32_t)(item / S - 1) & 1u, p.d_err);
                mbar_arrive_expect_tx(&full[sl], (uint32_t)kSlot);
            }
            __syncwarp();
            if (lane < kBPT) tma_rows(sb + sl * kSlot + lane * (BS * kD), map, y, &full[sl], pol);
            ++item;
        };
        int y_prev = oob;
        for (int j = 0; j < ntiles; ++j) {
            if (j > 0 && j % kTilesPerChunk == 0) {
                ent_cur = ent_nxt;
                ent_nxt = chunk(j / kTilesPerChunk + 1);
            }
            const int e = __shfl_sync(kFull, ent_cur, (j % kTilesPerChunk) * kBPT + (lane % kBPT));
            int y = oob;
            if (lane < kBPT && j * kBPT + lane < nblk) {
                if (e >= 0 && e < p.num_blocks) y = (e * p.num_kv_heads + kvh) * BS;
                else flag_error(p.d_err, PA_DEVERR_BLOCK_RANGE);
            }
            load(tmk, y);
            if (j >= 1) load(tmv, y_prev);
            y_prev = y;
        }
        load(tmv, y_prev);
    } else if (warp == 1) {
        // ============================================================ MMA issuer
        if (lane == 0) {
            constexpr uint32_t id_qk = instr_desc8(false, false, kKeys, N);
            constexpr uint32_t id_pv = instr_desc8(true, true, kD, N);
            constexpr uint32_t hi = desc_hi(1024);       // 8-row (8-key) groups 1 KB apart everywhere
            const uint32_t kv_lo0 = desc_lo(sb, 16);     // one swizzle row wide: leading offset unused
            const uint32_t q_lo = desc_lo(sb + L::kOffQ, 16);
            const uint32_t p_lo0 = desc_lo(sb + L::kOffP, 16);
            wait_or_flag(q_full, 0u, p.d_err);
            tc_fence_after();
            for (int j = 0; j <= ntiles; ++j) {
                if (j < ntiles) {
                    // S^T(j) = K(j) Q^T into buffer j & 1 (its previous tile's
                    // softmax finished before the PV issued last iteration)
                    const int it = item_k(j), sl = it % S;
                    wait_or_flag(&full[sl], (uint32_t)(it / S) & 1u, p.d_err);
                    tc_fence_after();
                    const uint32_t k_lo = kv_lo0 + ((uint32_t)(sl * kSlot) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8(tmem + (j & 1) * N, desc_of(k_lo + kk * 2, hi), desc_of(q_lo + kk * 2, hi), id_qk, kk > 0);
                    mma_commit(&s_full[j & 1]);
                    mma_commit(&empty[sl]);
                }
                if (j >= 1) {
                    // O^T += V^T(j-1) P^T(j-1)
                    const int jj = j - 1;
                    wait_or_flag(&p_full[jj & 1], (uint32_t)(jj >> 1) & 1u, p.d_err);
                    const int it = item_v(jj), sl = it % S;
                    wait_or_flag(&full[sl], (uint32_t)(it / S) & 1u, p.d_err);
                    tc_fence_after();
                    const uint32_t v_lo = kv_lo0 + ((uint32_t)(sl * kSlot) >> 4);
                    const uint32_t p_lo = p_lo0 + ((uint32_t)((jj & 1) * N * 128) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8(tmem + L::kColO, desc_of(v_lo + kk * 256, hi), desc_of(p_lo + kk * 2, hi), id_pv, jj > 0 || kk > 0);
                    mma_commit(&pv_done[jj & 1]);
                    mma_commit(&empty[sl]);
                }
            }
        }
    } else {
        // ============================================================ softmax
        const int quarter = warp & 3;         // TMEM lanes 32*quarter .. +31
        const int t = quarter * 32 + lane;    // key of the tile (S^T row) and dimension (O^T row)
        const int sw = warp - 2;              // index among the softmax warps
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const size_t row0 = (size_t)u.s * p.num_heads + (size_t)kvh * G;
        {
            // Q^T: each head over a power of two that brings its largest element to
            // 128 .. 256, as three e4m3 pieces, each the residual of those before
            // times 2^4: 12 bits, as many as fp16 has, and the products are exact
            const int h = t >> 4, c = t & 15;  // 16 threads a head, 8 dimensions each
            float x[8];
            unpack8<T>(h < G ? *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.query) + (row0 + h) * kD + c * 8)
                             : make_uint4(0, 0, 0, 0), x);
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, counted(x[i]));
#pragma unroll
            for (int m = 8; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, m));
            const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100) - 7;
            const float f = __uint_as_float((unsigned)(127 - e) << 23);
            if (h < G) {
                if (c == 0) qscale[h] = __uint_as_float((unsigned)(127 + e) << 23) * p.scale_log2;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = fabsf(x[i]) <= 3.402823466e38f ? x[i] * f : __uint_as_float(0x7fc00000u);
#pragma unroll
                for (int pc = 0; pc < kQPieces; ++pc) {
                    const unsigned lo = codes4(x[0], x[1], x[2], x[3]), hi = codes4(x[4], x[5], x[6], x[7]);
                    const int n = pc * GP + h;
                    sts64(sb + L::kOffQ + n * 128 + (((c >> 1) ^ (n & 7)) << 4) + (c & 1) * 8, lo, hi);
                    const float2 a = values2(lo & 0xffffu), b = values2(lo >> 16), d = values2(hi & 0xffffu), g = values2(hi >> 16);
                    x[0] = (x[0] - a.x) * 16.f, x[1] = (x[1] - a.y) * 16.f, x[2] = (x[2] - b.x) * 16.f, x[3] = (x[3] - b.y) * 16.f;
                    x[4] = (x[4] - d.x) * 16.f, x[5] = (x[5] - d.y) * 16.f, x[6] = (x[6] - g.x) * 16.f, x[7] = (x[7] - g.y) * 16.f;
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive1(q_full);
            named_bar_sync(1, 128);  // qscale
        }
        float qf[G], m_run[G], l_part[G];
#pragma unroll
        for (int h = 0; h < G; ++h) {
            qf[h] = qscale[h];
            m_run[h] = -INFINITY;
            l_part[h] = 0.f;
        }
        // this key's block, and its scales, a tile ahead of use (two for the block)
        auto entry = [&](int j) { return j * kKeys + t < ntok ? table[(j * kKeys + t) / BS] : -1; };
        auto in_pool = [&](int ent) { return ent >= 0 && ent < p.num_blocks; };
        int ent = entry(0), ent_nx = entry(1);
        unsigned kb = 127u, vb = 127u;
        if (in_pool(ent)) {
            kb = fp.k_scales[(size_t)ent * p.num_kv_heads + kvh];
            vb = fp.v_scales[(size_t)ent * p.num_kv_heads + kvh];
        }
        for (int j = 0; j < ntiles; ++j) {
            const int b = j & 1;
            const bool valid = in_pool(ent);
            const int ent_n2 = entry(j + 2);
            unsigned kb_nx = 127u, vb_nx = 127u;
            if (in_pool(ent_nx)) {
                kb_nx = fp.k_scales[(size_t)ent_nx * p.num_kv_heads + kvh];
                vb_nx = fp.v_scales[(size_t)ent_nx * p.num_kv_heads + kvh];
            }
            wait_or_flag(&s_full[b], (uint32_t)(j >> 1) & 1u, p.d_err);
            tc_fence_after();
            float z[G];
            {
                const float ks = scale_of(kb), ev = log_scale_of(vb);
                float s0[16];
                tmem_ld16(tmem + lane_off + b * N, s0);
                if constexpr (GP == 4) {
#pragma unroll
                    for (int h = 0; h < G; ++h) z[h] = fmaf(fmaf(s0[8 + h], 0.0625f, s0[4 + h]), 0.0625f, s0[h]);
                } else {
                    float s1[8];
                    tmem_ld8(tmem + lane_off + b * N + 16, s1);
#pragma unroll
                    for (int h = 0; h < G; ++h) z[h] = fmaf(fmaf(s1[h], 0.0625f, s0[8 + h]), 0.0625f, s0[h]);
                }
#pragma unroll
                for (int h = 0; h < G; ++h) z[h] = valid ? fmaf(z[h], ks * qf[h], ev) : -INFINITY;
            }
            // each head's maximum over the tile's 128 keys
            const float wmax = warp_scatter<true, G>(z, lane);
            if ((lane & (32 / G - 1)) == 0) xmax[(b * 4 + sw) * GP + lane / (32 / G)] = wmax;
            named_bar_sync(1, 128);
            float tmax[GP];
            {
                const float4 *x = reinterpret_cast<const float4 *>(xmax + b * 4 * GP);
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int k = 0; k < GP / 4; ++k) {
                        const float4 v = x[w * (GP / 4) + k];
                        tmax[4 * k] = w ? fmaxf(tmax[4 * k], v.x) : v.x;
                        tmax[4 * k + 1] = w ? fmaxf(tmax[4 * k + 1], v.y) : v.y;
                        tmax[4 * k + 2] = w ? fmaxf(tmax[4 * k + 2], v.z) : v.z;
                        tmax[4 * k + 3] = w ? fmaxf(tmax[4 * k + 3], v.w) : v.w;
                    }
            }
            // rescale when a maximum has grown by more than 2^8 (the same decision in every thread)
            bool grow = false;
            float alpha[GP];
#pragma unroll
            for (int h = 0; h < GP; ++h) alpha[h] = 1.f;
#pragma unroll
            for (int h = 0; h < G; ++h) {
                const float nm = tmax[h] > m_run[h] + kRescale ? tmax[h] : m_run[h];
                alpha[h] = m_run[h] == -INFINITY ? 0.f : fast_exp2(m_run[h] - nm);
                grow |= nm != m_run[h];
                m_run[h] = nm;
            }
            if (grow && j > 0) {
                // O must hold the PV of tile j-1 before it is scaled
                wait_or_flag(&pv_done[(j - 1) & 1], (uint32_t)((j - 1) >> 1) & 1u, p.d_err);
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < N; q += 16) {
                    float o[16];
                    tmem_ld16(tmem + lane_off + L::kColO + q, o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] *= alpha[(q + i) % GP];
                    tmem_st16(tmem + lane_off + L::kColO + q, o);
                }
#pragma unroll
                for (int h = 0; h < G; ++h) l_part[h] *= alpha[h];
            }
            float pr[G + (G & 1)];
            if constexpr (G & 1) pr[G] = 0.f;
            const float per = vb == 255u ? __uint_as_float(0x7fc00000u) : scale_of(254u - vb);  // 2^(-ev)
#pragma unroll
            for (int h = 0; h < G; ++h) {
                pr[h] = valid ? fast_exp2(z[h] - m_run[h] + kLift) : 0.f;  // no NaN while every key so far is left out
                l_part[h] = fmaf(pr[h], valid ? per : 0.f, l_part[h]);
            }
            // P^T buffer b is free once the PV of tile j-2 completed
            if (j >= 2) wait_or_flag(&pv_done[b], (uint32_t)((j - 2) >> 1) & 1u, p.d_err);
            {
                // each weight as four e5m2 pieces, each the rounded residual of those
                // before times 2^3: 12 bits from 2^15 down, and never coarser than 2^-26
                const uint32_t pb = sb + L::kOffP + b * N * 128 + (t & 15);
                const int ch = t >> 4;
#pragma unroll
                for (int pc = 0; pc < kPPieces; ++pc) {
#pragma unroll
                    for (int h = 0; h < G; h += 2) {
                        const unsigned two = e5m2x2(pr[h], pr[h + 1]);
                        const int n = pc * GP + h;
                        sts8(pb + n * 128 + ((ch ^ (n & 7)) << 4), two);
                        if (h + 1 < G) sts8(pb + (n + 1) * 128 + ((ch ^ ((n + 1) & 7)) << 4), two >> 8);
                        if (pc + 1 < kPPieces) {
                            const float2 a = from_e5m2x2(two);
                            pr[h] = (pr[h] - a.x) * 8.f;
                            pr[h + 1] = (pr[h + 1] - a.y) * 8.f;
                        }
                    }
                }
            }
            if (j == ntiles - 1 && j * kKeys + t >= ntok) {
                // this key's V row holds whatever the pool has past the context
                // (possibly NaN, and 0 * NaN poisons O): zero it
                const int it = item_v(j), sl = it % S;
                wait_or_flag(&full[sl], (uint32_t)(it / S) & 1u, p.d_err);
                const uint32_t vr = sb + sl * kSlot + t * kD;
                const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < 8; ++c) sts128(vr + c * 16, zero);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive1(&p_full[b]);
            ent = ent_nx, ent_nx = ent_n2, kb = kb_nx, vb = vb_nx;
        }

        // row sums over the 128 key lanes, then the four warps
        const float wsum = warp_scatter<false, G>(l_part, lane);
        if ((lane & (32 / G - 1)) == 0) xsum[sw * GP + lane / (32 / G)] = wsum;
        named_bar_sync(1, 128);
        const int last = ntiles - 1;
        wait_or_flag(&pv_done[last & 1], (uint32_t)(last >> 1) & 1u, p.d_err);
        tc_fence_after();
        float o[N];
#pragma unroll
        for (int q = 0; q < N; q += 16) tmem_ld16(tmem + lane_off + L::kColO + q, *reinterpret_cast<float(*)[16]>(&o[q]));
#pragma unroll
        for (int h = 0; h < G; ++h) {
            const float lsum = (xsum[h] + xsum[GP + h]) + (xsum[2 * GP + h] + xsum[3 * GP + h]);
            const float v = fmaf(fmaf(fmaf(o[3 * GP + h], 0.125f, o[2 * GP + h]), 0.125f, o[GP + h]), 0.125f, o[h]);
            const size_t row = row0 + h;
            if (u.direct) {
                static_cast<T *>(p.out)[row * kD + t] = (T)(lsum != 0.f ? v / lsum : 0.f);
            } else {
                const size_t at = row * p.slots + u.part;
                p.ws_acc[at * kD + t] = v;
                if (t == h) p.ws_ml[at] = make_float2(m_run[h] == -INFINITY ? kEmptyMax : m_run[h], lsum);
            }
        }
    }
    // copies still in flight (only after a timeout) land before the CTA ends
    if (threadIdx.x == 0)
        for (int i = max(0, 2 * ntiles - S); i < 2 * ntiles; ++i) mbar_wait(&full[i % S], (uint32_t)(i / S) & 1u);
}

}  // namespace tc8
}  // namespace pa
