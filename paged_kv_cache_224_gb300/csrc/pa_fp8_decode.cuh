// Device code of the decode over an 8-bit cache; see pa_fp8_decode.cu for the design.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "pa_fp8.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace d8 {

constexpr int kKeys = 128;               // keys per tile (M of the QK^T MMA)
constexpr int kThreads = 224;            // producer, MMA issuer, four softmax warps, scales
constexpr int kScaleRing = 8;            // tiles whose blocks' scales are held
constexpr int kLens = 256;               // context lengths held from the first sequence on
// A maximum may lag 2^kRescale behind and weights are 2^(z - M + kLift), at most 2^15.  The
// last row of a weight ends at 2^-26, whatever the lift: a shorter lag is more bits for
// small weights.  (Lags of 8 and 4 take the same time.)
constexpr float kRescale = 4.0f;
constexpr float kLift = 11.0f;
constexpr float kLowest = -110.0f;       // log2 of the least weight for O; 2^-ev brings it up to 2^64 higher in l
constexpr int kQPieces = 4, kPPieces = 4;
constexpr float kQStep = 32.0f;          // from one piece of a query to the next

// G heads of a kv head take GP rows a piece; N is the four pieces' rows.  At
// head_dim 64 a 128-byte row of V holds two keys: O^T has the sums over the even
// keys in its first 64 rows and over the odd ones in the others, each of them right in
// that half of the columns whose weights are its keys'.
template <int D, int G>
struct Lay {
    static constexpr int kPar = 128 / D;                    // keys in a 128-byte row of V
    static constexpr int GP = G <= 4 ? 4 : 8;
    static constexpr int N = 4 * GP, NO = N * kPar;         // columns of S^T and of O^T
    static constexpr uint32_t kCols = 2 * N + NO <= 64 ? 64 : 128;  // TMEM: S^T x 2 buffers, O^T
    static constexpr uint32_t kColO = 2 * N;
    static constexpr int kSlot = kKeys * D;                 // one K or V tile
    static constexpr int kCtas = ctas_per_sm(D, G);
    static constexpr int S = GP == 8 ? 5 * kPar : 6;        // ring slots: 80 KB, else 96 KB (48 KB at head_dim 64)
    static constexpr int kRowP = kKeys / kPar;              // bytes of a row of P^T: a tile's keys of one parity
    static constexpr int kOffQ = S * kSlot;
    static constexpr int kQ = N * D;
    static constexpr int kOffP = kOffQ + 2 * kQ;            // 2 x [N][D], then 2 x [NO][kRowP]
    static constexpr int kP = NO * kRowP;
    static constexpr int kOffSc = kOffP + 2 * kP;           // [kScaleRing][16 blocks] of float4
    static constexpr int kOffBar = kOffSc + kScaleRing * 16 * 16;
    static constexpr int kBars = 2 * S + 10 + 2 * kScaleRing;
    static constexpr int kOffLen = kOffBar + (kBars * 8 + 8 + 15) / 16 * 16;
    // [4 warps][GP] maxima, [4][GP] sums, [2][GP] query scales, [G][64] sums of odd keys, [2] of Cut
    static constexpr int kOffXch = kOffLen + kLens * 4 + 64;
    static constexpr int kUsed = kOffXch + (4 * GP + 4 * GP + 2 * GP + (kPar == 2 ? G * 64 : 0)) * 4 + 2 * 32;
    static constexpr int kAlloc = kUsed + 1024;             // room to align the base to 1 KB
    // (what a merge keeps goes where the tiles were; two units' weights never do together)
    static_assert((kThreads / 32 * G * D + G + kFp8MaxCtas * G) * 4 <= S * kSlot, "the merge's sums and weights");
};

// kind::f8f6f4, fp32 accumulator: A e4m3, B e4m3 or e5m2.
__host__ __device__ constexpr uint32_t instr_desc8(bool b_e5m2, bool a_mn_major, int m, int n) {
    return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn_major ? 1u : 0u) << 15) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}
// As desc_hi, for 64-byte swizzling (value 4 at bit 61).
__host__ __device__ constexpr uint32_t desc_hi64(uint32_t sbo) { return ((sbo >> 4) & 0x3FFFu) | (1u << 14) | (4u << 29); }

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
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// wait_or_flag with the polling out of line: the roles' code has to stay in the
// instruction cache together, and most waits find their phase complete.
static __device__ __noinline__ void poll_or_flag(uint64_t *bar, uint32_t parity, int *d_err) {
    for (uint32_t i = 0; i < kMaxPolls; ++i)
        if (mbar_try_wait(bar, parity)) return;
    flag_error(d_err, PA_DEVERR_TIMEOUT);
}
__device__ __forceinline__ void await(uint64_t *bar, uint32_t parity, int *d_err) {
    if (!mbar_test(bar, parity)) poll_or_flag(bar, parity, d_err);
}

// Barrier `id` over `count` threads, which all learn whether any of them came with `mine`.
__device__ __forceinline__ bool bar_any(int id, int count, bool mine) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
        "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(id), "r"(count), "r"((uint32_t)mine)
        : "memory");
    return any != 0;
}

// Byte `at` of row `row` in rows of W bytes, swizzled over W bytes (W = 64 or 128).
template <int W>
__device__ __forceinline__ uint32_t swizzled(int row, int at) {
    const int x = W == 128 ? row & 7 : (row >> 1) & 3;
    return row * W + ((((at >> 4) ^ x) << 4) | (at & 15));
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

// The call's `total` key tiles lie end to end, sequence by sequence and kv head by kv
// head; CTA c of n (n <= total, so that each has one) has those from share(c) to
// share(c + 1), and owner(t) is the CTA that has tile t.
__device__ __forceinline__ long long share(long long total, int n, int c) { return total * c / n; }
__device__ __forceinline__ int owner(long long total, int n, long long t) { return (int)(((t + 1) * n - 1) / total); }

// A CTA's tiles of one (sequence, kv head).  `slot`: where its partial goes, -1 if it
// is the whole; a CTA's first piece has slot 2c, a last one that is not its first 2c + 1.
struct Piece {
    int s, kvh;
    int tile, n;      // first tile within the sequence, tiles
    int ntok;         // tokens from the first tile on
    int slot;
    long long at;     // first tile within the call
    int whole;        // tiles of the (sequence, kv head)
};

// Walks a CTA's pieces; every role of the CTA has one and sees the same.
struct Walk {
    long long at, end, total;  // the next tile of the call, the CTA's end, all tiles
    int ctas;                  // CTAs that have tiles
    int s, kvh, tile, len;
    int s0;                    // sequence whose length is lens[0]
    bool first;
};

__device__ __forceinline__ int tiles_of(int len) { return (len + kKeys - 1) / kKeys; }

__device__ __forceinline__ int clamped_len(const DecodeParams &p, int s) {
    const int cap = min(p.max_context_len, p.max_blocks_per_seq * p.block_size);
    return min(max(p.context_lens[s], 0), cap);
}

__device__ __forceinline__ bool next_piece(const DecodeParams &p, const int *lens, Walk &w, Piece &q) {
    if (w.at >= w.end) return false;
    while (w.len == 0) {  // (tiles are left, so a sequence with some follows, unless the lengths changed meanwhile)
        if (++w.s >= p.num_seqs) {
            w.at = w.end;
            return false;
        }
        w.len = w.s - w.s0 < kLens ? lens[w.s - w.s0] : clamped_len(p, w.s);
        w.kvh = w.tile = 0;
    }
    const int whole = tiles_of(w.len);
    q.s = w.s;
    q.kvh = w.kvh;
    q.tile = w.tile;
    q.n = (int)min((long long)(whole - w.tile), w.end - w.at);
    q.ntok = min(w.len - w.tile * kKeys, q.n * kKeys);
    q.slot = q.n == whole ? -1 : 2 * (int)blockIdx.x + (w.first ? 0 : 1);
    q.at = w.at;
    q.whole = whole;
    w.first = false;
    w.at += q.n;
    w.tile += q.n;
    if (w.tile == whole) {
        w.tile = 0;
        if (++w.kvh == p.num_kv_heads) {
            w.kvh = 0;
            w.len = 0;
        }
    }
    return true;
}

// The walk's start, by all threads: a scan of the sequences' tiles, the CTA's share of
// them, and the sequence that it begins in.  Sequences without tokens get their zeros here.
template <typename T>
__device__ __forceinline__ Walk begin(const Fp8DecodeParams &fp, int head_dim, int *lens, long long *scan) {
    const DecodeParams &p = fp.d;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (p.num_seqs + kThreads - 1) / kThreads;
    const int a = min(tid * per, p.num_seqs), b = min(a + per, p.num_seqs);
    long long mine = 0;
    for (int s = a; s < b; ++s) {
        const int len = clamped_len(p, s);
        if (blockIdx.x == 0 && len != p.context_lens[s]) flag_error(p.d_err, PA_DEVERR_CONTEXT_RANGE);
        mine += tiles_of(len);
    }
    long long upto = mine;  // inclusive
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(kFull, upto, m);
        if (lane >= m) upto += o;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    long long before = upto - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const long long x = scan[w];
        if (w < warp) before += x;
        total += x;
    }
    __syncthreads();
    total *= p.num_kv_heads;
    Walk w;
    w.total = total;
    w.ctas = (int)min((long long)gridDim.x, total);
    const bool has = (int)blockIdx.x < w.ctas;
    const long long t0 = w.at = has ? share(total, w.ctas, blockIdx.x) : 0;
    w.end = has ? share(total, w.ctas, blockIdx.x + 1) : 0;
    int *start = reinterpret_cast<int *>(scan);  // sequence, kv head, tile
    if (has && t0 >= before * p.num_kv_heads && t0 < (before + mine) * p.num_kv_heads) {
        for (int s = a; s < b; ++s) {
            const int n = tiles_of(clamped_len(p, s));
            if (t0 < (before + n) * p.num_kv_heads) {
                const long long rest = t0 - before * p.num_kv_heads;
                start[0] = s;
                start[1] = (int)(rest / n);
                start[2] = (int)(rest % n);
                break;
            }
            before += n;
        }
    }
    for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x) {
        if (clamped_len(p, s) > 0) continue;
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (size_t)s * p.num_heads * head_dim);
        for (int i = tid; i < p.num_heads * head_dim / 8; i += kThreads) dst[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    w.first = true;
    w.s = w.s0 = has ? start[0] : 0;
    w.kvh = has ? start[1] : 0;
    w.tile = has ? start[2] : 0;
    if (has)
        for (int i = tid; i < kLens && w.s0 + i < p.num_seqs; i += kThreads) lens[i] = clamped_len(p, w.s0 + i);
    __syncthreads();
    w.len = has ? lens[0] : 0;
    return w;
}

// A unit (sequence, kv head) that the shares cut, as a CTA that has a piece of it sees it.
struct Cut {
    long long from;  // its first tile within the call
    int whole;  // its tiles
    int row0;   // its first row of the output
    int lead;   // CTA that has its first piece; piece i is of CTA lead + i
    int n;      // pieces; 0: no such unit
    int first;  // slot of the first piece (piece i > 0 has the even slot of its CTA); -1 once another CTA merges it
    int pad;
};

// Log-sum-exp merge of a unit's pieces by all warps:
//   M = max m_i,  w_i = 2^(m_i - M),  out = sum w_i acc_i / sum w_i l_i.
// A warp has a head for the weights, a lane a piece; then a warp has every kWarps-th
// piece, whole, and the warps' sums are added up.  `work`: the ring, which has served.
// (Loads go past L1, which may hold what an earlier call left.  Inlined: with this and
// merge_few out of line 256 contexts of 2048 tokens, 64/8 heads of 64, took 138 us, not 131.)
template <typename T, int D, int G>
__device__ __forceinline__ void merge_many(const DecodeParams &p, const Cut &c, float *work) {
    using V = typename std::conditional<D == 128, float4, float2>::type;
    constexpr int kWarps = kThreads / 32, kN = D / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *sums = work, *total = sums + kWarps * G * D, *weight = total + G;  // [kWarps][G][D], [G], [n][G]
    auto slot = [&](int i) { return (size_t)(i ? 2 * (c.lead + i) : c.first) * G; };
#pragma unroll 1
    for (int h = warp; h < G; h += kWarps) {
        float M = kEmptyMax, l = 0.f;
        for (int i = lane; i < c.n; i += 32) {
            const float2 ml = __ldcg(&p.ws_ml[slot(i) + h]);
            const float top = fmaxf(M, ml.x);
            l = moved(l, M - top) + moved(ml.y, ml.x - top);
            M = top;
            weight[i * G + h] = ml.x;
        }
        float top = M;
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
        l = moved(l, M - top);
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) l += __shfl_xor_sync(kFull, l, x);
        for (int i = lane; i < c.n; i += 32) weight[i * G + h] = fast_exp2(weight[i * G + h] - top);
        if (lane == 0) total[h] = l;
    }
    __syncthreads();
    if (warp < c.n) {
        float o[G][kN] = {};
#pragma unroll (16 / G)
        for (int i = warp; i < c.n; i += kWarps) {
            const V *src = reinterpret_cast<const V *>(p.ws_acc + slot(i) * D) + lane;
#pragma unroll
            for (int h = 0; h < G; ++h) {
                const V v = __ldcg(src + h * 32);
                const float w = weight[i * G + h];
#pragma unroll
                for (int k = 0; k < kN; ++k) o[h][k] = fmaf(w, reinterpret_cast<const float *>(&v)[k], o[h][k]);
            }
        }
#pragma unroll
        for (int h = 0; h < G; ++h)
            *reinterpret_cast<V *>(sums + (warp * G + h) * D + lane * kN) = *reinterpret_cast<const V *>(o[h]);
    }
    __syncthreads();
    for (int e = tid; e < G * D / 2; e += kThreads) {
        float2 x = make_float2(0.f, 0.f);
        for (int w = 0; w < min(c.n, kWarps); ++w) {
            const float2 y = reinterpret_cast<const float2 *>(sums)[w * (G * D / 2) + e];
            x.x += y.x, x.y += y.y;
        }
        const float l = total[e / (D / 2)];
        reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + (size_t)c.row0 * D)[e] = l != 0.f ? Elem<T>::pack2(x.x / l, x.y / l) : 0u;
    }
    __syncthreads();  // (the next unit's weights and sums go to the same place)
}

// The same of up to kFew pieces by single threads, four dimensions each, with everything
// loaded at once: most cuts in a large batch are in two.  (32 contexts of 700 tokens, 32/8
// heads: 17.0 us by merge_many alone, 15.0 by both.)
constexpr int kFew = 4;
template <typename T, int D, int G>
__device__ __forceinline__ void merge_few(const DecodeParams &p, const Cut *cuts) {
#pragma unroll 1
    for (int e = threadIdx.x; e < 2 * G * (D / 4); e += kThreads) {
        const int k = e >= G * (D / 4), f = e - k * G * (D / 4), h = f / (D / 4);
        const Cut c = cuts[k];
        if (c.n == 0 || c.n > kFew || c.first < 0) continue;
        float2 ml[kFew];
        float4 v[kFew];
        float M = kEmptyMax, l = 0.f;
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
            ml[i] = make_float2(kEmptyMax, 0.f);
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < c.n) {
                const size_t at = (size_t)(i ? 2 * (c.lead + i) : c.first) * G;
                ml[i] = __ldcg(&p.ws_ml[at + h]);
                v[i] = __ldcg(reinterpret_cast<const float4 *>(p.ws_acc + at * D) + f);
            }
        }
#pragma unroll
        for (int i = 0; i < kFew; ++i) M = fmaxf(M, ml[i].x);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
            const float w = fast_exp2(ml[i].x - M);
            l += moved(ml[i].y, ml[i].x - M);
            o.x = fmaf(w, v[i].x, o.x), o.y = fmaf(w, v[i].y, o.y);
            o.z = fmaf(w, v[i].z, o.z), o.w = fmaf(w, v[i].w, o.w);
        }
        uint2 out = make_uint2(0u, 0u);
        if (l != 0.f) out = make_uint2(Elem<T>::pack2(o.x / l, o.y / l), Elem<T>::pack2(o.z / l, o.w / l));
        reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (size_t)c.row0 * D)[f] = out;
    }
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kThreads, Lay<D, G>::kCtas)
    decode_fp8_kernel(const __grid_constant__ Fp8DecodeParams fp, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv) {
    using L = Lay<D, G>;
    constexpr int S = L::S, GP = L::GP, N = L::N, NO = L::NO;
    const DecodeParams &p = fp.d;
    extern __shared__ unsigned char smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw = smem_addr(smem_raw), sb = (raw + 1023u) & ~1023u;  // swizzle atoms start on 1 KB
    unsigned char *smem = smem_raw + (sb - raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kOffBar);  // [S] TMA -> MMA
    uint64_t *empty = full + S;                                        // [S] MMA -> TMA
    uint64_t *q_full = empty + S;                                      // [2] helper -> MMA, softmax (Q^T written)
    uint64_t *q_empty = q_full + 2;                                    // [2] MMA, softmax -> helper
    uint64_t *s_full = q_empty + 2;                                    // [2] MMA -> softmax (S^T of a tile ready)
    uint64_t *p_full = s_full + 2;                                     // [2] softmax -> MMA (P^T written, O rescaled)
    uint64_t *pv_done = p_full + 2;                                    // [2] MMA -> softmax (PV of a tile complete)
    uint64_t *sc_full = pv_done + 2;                                   // [kScaleRing] helper -> softmax
    uint64_t *sc_empty = sc_full + kScaleRing;                         // [kScaleRing] softmax -> helper
    volatile uint32_t *holder = reinterpret_cast<volatile uint32_t *>(sc_empty + kScaleRing);
    int *lens = reinterpret_cast<int *>(smem + L::kOffLen);
    float4 *scales = reinterpret_cast<float4 *>(smem + L::kOffSc);
    float *xmax = reinterpret_cast<float *>(smem + L::kOffXch);
    float *xsum = xmax + 4 * GP, *qscale = xsum + 4 * GP, *odd = qscale + 2 * GP;
    Cut *cuts = reinterpret_cast<Cut *>(odd + (L::kPar == 2 ? G * 64 : 0));  // [2], of the pieces with slots 2c and 2c + 1
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * S; ++i) mbar_init(&full[i], 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&q_full[b], 1);
            mbar_init(&q_empty[b], 1 + 4);  // the MMA thread's commit and the softmax warps
            mbar_init(&s_full[b], 1);
            mbar_init(&p_full[b], 128);
            mbar_init(&pv_done[b], 1);
        }
        for (int i = 0; i < kScaleRing; ++i) {
            mbar_init(&sc_full[i], 1);
            mbar_init(&sc_empty[i], 4);
        }
        fence_barrier_init();
        cuts[0].n = cuts[1].n = cuts[0].whole = cuts[1].whole = 0;
    }
    pdl_wait();     // the kernel before this one on the stream (e.g. the cache write) has finished
    // (not before the wait: a kernel that is still to allocate tensor memory on this SM
    // would wait for this one, and this one for that)
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(const_cast<uint32_t *>(holder))),
                     "r"(L::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_trigger();  // what follows may be placed; it waits for these writes
    Walk walk = begin<T>(fp, D, lens, reinterpret_cast<long long *>(lens + kLens));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;
    const int shift = __ffs(p.block_size) - 1;  // block_size is a power of two, 8 .. 128
    const int per_tile = kKeys >> shift;        // blocks per tile
    Piece q;

    if (warp == 0) {
        // ============================================================ producer
        const int oob = p.num_blocks * p.num_kv_heads * p.block_size;  // first row past the pool: zero fill
        const uint64_t pol = policy_evict_first();
        const int per_chunk = 32 / per_tile;  // tiles of 32 table entries
        int item = 0;
        auto load = [&](const CUtensorMap *map, int y) {
            const int sl = item % S;
            if (lane == 0) {
                if (item >= S) await(&empty[sl], (uint32_t)(item / S - 1) & 1u, p.d_err);
                mbar_arrive_expect_tx(&full[sl], (uint32_t)L::kSlot);
            }
            __syncwarp();
            if (lane < per_tile) tma_rows(sb + sl * L::kSlot + lane * p.block_size * D, map, y, &full[sl], pol);
            ++item;
        };
        // ring items in consumption order, whatever piece a tile is of: K(0), then K(g),
        // V(g-1) for g >= 1, then V(last)
        int y_prev = -1;
        while (next_piece(p, lens, walk, q)) {
            const int32_t *table = p.block_tables + (size_t)q.s * p.table_stride + q.tile * per_tile;
            const int nblk = (q.ntok + p.block_size - 1) >> shift;
            // table entries 32 at a time, one per lane, a chunk ahead of use
            auto chunk = [&](int c) { return c * 32 + lane < nblk ? table[c * 32 + lane] : -1; };
            int ent_cur = chunk(0), ent_nxt = chunk(1);
            for (int j = 0; j < q.n; ++j) {
                const int in = j & (per_chunk - 1);
                if (j > 0 && in == 0) {
                    ent_cur = ent_nxt;
                    ent_nxt = chunk(j / per_chunk + 1);
                }
                const int e = __shfl_sync(kFull, ent_cur, in * per_tile + (lane & (per_tile - 1)));
                int y = oob;
                if (lane < per_tile && j * per_tile + lane < nblk) {
                    if (e >= 0 && e < p.num_blocks) y = (e * p.num_kv_heads + q.kvh) << shift;
                    else flag_error(p.d_err, PA_DEVERR_BLOCK_RANGE);
                }
                load(&tmk, y);
                if (y_prev >= 0) load(&tmv, y_prev / L::kPar);
                y_prev = y;
            }
        }
        if (y_prev >= 0) load(&tmv, y_prev / L::kPar);
        // copies still in flight (only after a timeout) land before the CTA ends
        if (lane == 0)
            for (int i = max(0, item - S); i < item; ++i) mbar_wait(&full[i % S], (uint32_t)(i / S) & 1u);
    } else if (warp == 1) {
        // ============================================================ MMA issuer
        if (lane == 0) {
            constexpr uint32_t id_qk = instr_desc8(false, false, kKeys, N);
            constexpr uint32_t id_pv = instr_desc8(true, true, 128, NO);
            constexpr uint32_t hi_v = desc_hi(1024);  // 128-byte rows: groups of 8 are 1 KB apart
            constexpr uint32_t hi = D == 128 ? hi_v : desc_hi64(512);  // K, Q^T, P^T: rows of D, D and kRowP = D bytes
            static_assert(L::kRowP == D, "P^T is swizzled like K and Q^T");
            // one swizzle row wide: the leading offset is unused
            const uint32_t kv_lo0 = desc_lo(sb, 16), q_lo = desc_lo(sb + L::kOffQ, 16), p_lo0 = desc_lo(sb + L::kOffP, 16);
            // O^T (+)= V^T(g) P^T(g); `item`: V's place in the ring
            auto pv = [&](int g, int item, bool first) {
                const int b = g & 1, sl = item % S;
                await(&p_full[b], (uint32_t)(g >> 1) & 1u, p.d_err);
                await(&full[sl], (uint32_t)(item / S) & 1u, p.d_err);
                tc_fence_after();
                const uint32_t v_lo = kv_lo0 + ((uint32_t)(sl * L::kSlot) >> 4);
                const uint32_t p_lo = p_lo0 + ((uint32_t)(b * L::kP) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                    mma_f8(tmem + L::kColO, desc_of(v_lo + kk * 256, hi_v), desc_of(p_lo + kk * 2, hi), id_pv, !first || kk > 0);
                mma_commit(&pv_done[b]);
                mma_commit(&empty[sl]);
            };
            int g = 0, pieces = 0;  // tiles and pieces so far
            bool first = false;     // whether tile g - 1 is its piece's first
            while (next_piece(p, lens, walk, q)) {
                const int qb = pieces & 1;
                await(&q_full[qb], (uint32_t)(pieces >> 1) & 1u, p.d_err);
                tc_fence_after();
                for (int j = 0; j < q.n; ++j, ++g) {
                    // S^T(g) = K(g) Q^T into buffer g & 1 (its previous tile's softmax
                    // finished before the PV issued last iteration)
                    const int it = g == 0 ? 0 : 2 * g - 1, sl = it % S, b = g & 1;
                    await(&full[sl], (uint32_t)(it / S) & 1u, p.d_err);
                    tc_fence_after();
                    const uint32_t k_lo = kv_lo0 + ((uint32_t)(sl * L::kSlot) >> 4);
                    const uint32_t qq = q_lo + ((uint32_t)(qb * L::kQ) >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk)
                        mma_f8(tmem + b * N, desc_of(k_lo + kk * 2, hi), desc_of(qq + kk * 2, hi), id_qk, kk > 0);
                    mma_commit(&s_full[b]);
                    mma_commit(&empty[sl]);
                    if (j == q.n - 1) mma_commit(&q_empty[qb]);
                    if (g > 0) pv(g - 1, 2 * g, first);
                    first = j == 0;
                }
                ++pieces;
            }
            if (g > 0) pv(g - 1, 2 * g - 1, first);
        }
    } else if (warp == 6) {
        // ============================================================ helper
        // Q^T of each piece, a piece ahead, and of every block of a tile (2^ek, ev,
        // 2^(-ev)), up to kScaleRing tiles ahead; a block outside the pool has (0, -inf,
        // 0), so that its keys (zeros) weigh nothing
        int g = 0, pieces = 0;
        while (next_piece(p, lens, walk, q)) {
            const int32_t *table = p.block_tables + (size_t)q.s * p.table_stride + q.tile * per_tile;
            const int nblk = (q.ntok + p.block_size - 1) >> shift;
            const int per_chunk = 32 / per_tile;
            auto entry = [&](int c) { return c * 32 + lane < nblk ? table[c * 32 + lane] : -1; };
            auto fetch = [&](int e, unsigned &kb, unsigned &vb) {
                kb = vb = 256u;
                if (e >= 0 && e < p.num_blocks) {
                    const size_t at = (size_t)e * p.num_kv_heads + q.kvh;
                    kb = fp.k_scales[at];
                    vb = fp.v_scales[at];
                }
            };
            // entries two chunks ahead, scales one
            unsigned kb, vb, kn, vn;
            const int e0 = entry(0);
            int e1 = entry(1), e2 = entry(2);
            fetch(e0, kb, vb);
            // Q^T: each head over a power of two that brings its largest element to
            // 128 .. 256, as four e4m3 pieces, each the residual of those before times
            // 2^5 (of up to 8, so up to 256): the last one's step is 2^-24.  fp16 elements
            // are exact down to 2^-21 of the largest one's power of two, bf16 down to
            // 2^-24, what is smaller to 2^-32 of it, and the products are exact
            const int qb = pieces & 1;
            if (pieces >= 2) {
                if (lane == 0) await(&q_empty[qb], (uint32_t)((pieces >> 1) - 1) & 1u, p.d_err);
                __syncwarp();
            }
            {
                // (rolled up: what runs once a piece should not push the tiles' code out of
                // the instruction cache, and the second reads come from L1)
                constexpr int kLanes = 32 / G;  // of a head, four dimensions at a time
                const int h = lane / kLanes, d0 = lane % kLanes * 4;
                const T *src = static_cast<const T *>(p.query) + ((size_t)q.s * p.num_heads + (size_t)q.kvh * G + h) * D;
                float x[4], amax = 0.f;
                auto four = [&](int d) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(src + d);
                    Elem<T>::unpack2(u.x, x[0], x[1]);
                    Elem<T>::unpack2(u.y, x[2], x[3]);
                };
#pragma unroll 4
                for (int d = d0; d < D; d += 4 * kLanes) {
                    four(d);
                    amax = fmaxf(amax, fmaxf(fmaxf(counted(x[0]), counted(x[1])), fmaxf(counted(x[2]), counted(x[3]))));
                }
#pragma unroll
                for (int m = kLanes / 2; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, m));
                const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100) - 7;
                const float f = __uint_as_float((unsigned)(127 - e) << 23);
                if (d0 == 0) qscale[qb * GP + h] = __uint_as_float((unsigned)(127 + e) << 23) * p.scale_log2;
#pragma unroll 1
                for (int d = d0; d < D; d += 4 * kLanes) {
                    four(d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = fabsf(x[i]) <= 3.402823466e38f ? x[i] * f : __uint_as_float(0x7fc00000u);
#pragma unroll
                    for (int pc = 0; pc < kQPieces; ++pc) {
                        const unsigned lo = codes2(x[0], x[1]), hi2 = codes2(x[2], x[3]);
                        const float2 v0 = values2(lo), v1 = values2(hi2);
                        x[0] = (x[0] - v0.x) * kQStep, x[1] = (x[1] - v0.y) * kQStep;
                        x[2] = (x[2] - v1.x) * kQStep, x[3] = (x[3] - v1.y) * kQStep;
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(sb + L::kOffQ + qb * L::kQ + swizzled<D>(pc * GP + h, d)),
                                     "r"(lo | hi2 << 16)
                                     : "memory");
                    }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive1(&q_full[qb]);
            ++pieces;
            if (q.slot >= 0 && lane == 0) {
                Cut &c = cuts[q.slot & 1];
                c.from = q.at - q.tile;
                c.whole = q.whole;
                c.row0 = q.s * p.num_heads + q.kvh * G;
            }
            for (int j = 0; j < q.n; ++j, ++g) {
                const int in = j & (per_chunk - 1);
                if (in == 0) {
                    if (j > 0) kb = kn, vb = vn;
                    fetch(e1, kn, vn);
                    e1 = e2;
                    e2 = entry(j / per_chunk + 3);
                }
                const int r = g % kScaleRing;
                if (g >= kScaleRing) {
                    if (lane == 0) await(&sc_empty[r], (uint32_t)(g / kScaleRing - 1) & 1u, p.d_err);
                    __syncwarp();
                }
                if (lane / per_tile == in) {
                    float4 v = make_float4(0.f, -INFINITY, 0.f, 0.f);
                    if (kb < 256u) v = make_float4(scale_of(kb), log_scale_of(vb), vb == 255u ? scale_of(255u) : scale_of(254u - vb), 0.f);
                    scales[r * 16 + (lane & (per_tile - 1))] = v;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive1(&sc_full[r]);
            }
        }
        // (here and not with its piece: the divisions are a lot of code)
        __syncwarp();
        if (lane < 2 && cuts[lane].whole > 0) {
            Cut &c = cuts[lane];
            c.lead = owner(walk.total, walk.ctas, c.from);
            c.n = owner(walk.total, walk.ctas, c.from + c.whole - 1) - c.lead + 1;
            c.first = share(walk.total, walk.ctas, c.lead) == c.from ? 2 * c.lead : 2 * c.lead + 1;
        }
    } else {
        // ============================================================ softmax
        const int quarter = warp & 3;         // TMEM lanes 32*quarter .. +31
        const int t = quarter * 32 + lane;    // key of the tile (S^T row), row of O^T
        const int sw = warp - 2;              // index among the softmax warps
        const int par = t / D, d = t % D;     // parity of the keys whose sums, and dimension that, O^T's row has
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t col_o = L::kColO + par * N;
        int g0 = 0, pieces = 0;
        while (next_piece(p, lens, walk, q)) {
            const size_t row0 = (size_t)q.s * p.num_heads + (size_t)q.kvh * G;
            const int qb = pieces & 1;
            await(&q_full[qb], (uint32_t)(pieces >> 1) & 1u, p.d_err);
            float qf[G], m_run[G], l_part[G];
#pragma unroll
            for (int h = 0; h < G; ++h) {
                qf[h] = qscale[qb * GP + h];
                m_run[h] = kEmptyMax;
                l_part[h] = 0.f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive1(&q_empty[qb]);
            ++pieces;
            for (int j = 0; j < q.n; ++j) {
                const int g = g0 + j, b = g & 1, r = g % kScaleRing;
                const bool valid = j * kKeys + t < q.ntok;
                await(&sc_full[r], (uint32_t)(g / kScaleRing) & 1u, p.d_err);
                const float4 sc = scales[r * 16 + (t >> shift)];
                __syncwarp();
                if (lane == 0) mbar_arrive1(&sc_empty[r]);
                await(&s_full[b], (uint32_t)(g >> 1) & 1u, p.d_err);
                tc_fence_after();
                float z[G];
                {
                    float s0[16];
                    tmem_ld16(tmem + lane_off + b * N, s0);
                    auto join = [](float a, float b, float c, float d) {
                        return fmaf(fmaf(fmaf(d, 1 / kQStep, c), 1 / kQStep, b), 1 / kQStep, a);
                    };
                    if constexpr (GP == 4) {
#pragma unroll
                        for (int h = 0; h < G; ++h) z[h] = join(s0[h], s0[4 + h], s0[8 + h], s0[12 + h]);
                    } else {
                        float s1[16];
                        tmem_ld16(tmem + lane_off + b * N + 16, s1);
#pragma unroll
                        for (int h = 0; h < G; ++h) z[h] = join(s0[h], s0[8 + h], s1[h], s1[8 + h]);
                    }
#pragma unroll
                    for (int h = 0; h < G; ++h) z[h] = valid ? fmaf(z[h], sc.x * qf[h], sc.y) : -INFINITY;
                }
                // The maxima that weights are relative to move only when some key is more
                // than 2^kRescale above them (and at a piece's first keys): one barrier tells
                // every thread whether any has seen that.
                bool over = false;
#pragma unroll
                for (int h = 0; h < G; ++h) over |= z[h] > m_run[h] + kRescale;
                if (bar_any(1, 128, over)) {
                    const float wmax = warp_scatter<true, G>(z, lane);
                    if ((lane & (32 / G - 1)) == 0) xmax[sw * GP + lane / (32 / G)] = wmax;
                    named_bar_sync(1, 128);
                    float alpha[GP];
#pragma unroll
                    for (int h = 0; h < GP; ++h) alpha[h] = 1.f;
#pragma unroll
                    for (int h = 0; h < G; ++h) {
                        const float tmax = fmaxf(fmaxf(xmax[h], xmax[GP + h]), fmaxf(xmax[2 * GP + h], xmax[3 * GP + h]));
                        const float nm = tmax > m_run[h] + kRescale ? tmax : m_run[h];
                        alpha[h] = fast_exp2(m_run[h] - nm);
                        l_part[h] = moved(l_part[h], m_run[h] - nm);
                        m_run[h] = nm;
                    }
                    if (j > 0) {
                        // O must hold the PV of tile g-1 before it is scaled
                        await(&pv_done[(g - 1) & 1], (uint32_t)((g - 1) >> 1) & 1u, p.d_err);
                        tc_fence_after();
#pragma unroll
                        for (int i0 = 0; i0 < N; i0 += 16) {
                            float o[16];
                            tmem_ld16(tmem + lane_off + col_o + i0, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= alpha[(i0 + i) % GP];
                            tmem_st16(tmem + lane_off + col_o + i0, o);
                        }
                        tmem_wait_st();
                    }
                }
                float pr[G + (G & 1)];
                bool low = false;
                if constexpr (G & 1) pr[G] = 0.f;
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    const float x = z[h] - m_run[h] + kLift;
                    low |= x < kLowest;
                    pr[h] = x < kLowest ? 0.f : fast_exp2(x);
                    l_part[h] = fmaf(pr[h], valid ? sc.z : 0.f, l_part[h]);
                }
                // A key whose values' scale is far below the largest one's may weigh
                // nothing for O and count for l all the same: 2^(x - ev) in one step.
                // (2^60, so that the smallest are not flushed to zero.)
                if (low) {
#pragma unroll
                    for (int h = 0; h < G; ++h) {
                        const float x = z[h] - m_run[h] + kLift;
                        if (x < kLowest && z[h] > -INFINITY) l_part[h] = fmaf(fast_exp2(x - sc.y + 60.f), 0x1p-60f, l_part[h]);
                    }
                }
                // P^T buffer b is free once the PV of tile j-2 completed
                if (j >= 2) await(&pv_done[b], (uint32_t)((g - 2) >> 1) & 1u, p.d_err);
                {
                    // each weight as four e5m2 pieces, each the rounded residual of those
                    // before times 2^3: off by 2^-12 of itself or 2^-26, the greater: 12
                    // bits down to 2^-25 of a weight at the maximum, and 2^-37 of that below
                    const uint32_t pb = sb + L::kOffP + b * L::kP;
                    const int kp = t % L::kPar, at = t / L::kPar;  // the key's parity, and its place among that parity's
#pragma unroll
                    for (int pc = 0; pc < kPPieces; ++pc) {
#pragma unroll
                        for (int h = 0; h < G; h += 2) {
                            const unsigned two = e5m2x2(pr[h], pr[h + 1]);
                            const int n = kp * N + pc * GP + h;
                            sts8(pb + swizzled<L::kRowP>(n, at), two);
                            if (h + 1 < G) sts8(pb + swizzled<L::kRowP>(n + 1, at), two >> 8);
                            if (pc + 1 < kPPieces) {
                                const float2 a = from_e5m2x2(two);
                                pr[h] = (pr[h] - a.x) * 8.f;
                                pr[h + 1] = (pr[h + 1] - a.y) * 8.f;
                            }
                        }
                    }
                }
                if (j == q.n - 1 && !valid) {
                    // this key's V row holds whatever the pool has past the context
                    // (possibly NaN, and 0 * NaN poisons O): zero it
                    const int it = walk.at >= walk.end ? 2 * g + 1 : 2 * g + 2, sl = it % S;  // (the CTA's last V is the last item)
                    await(&full[sl], (uint32_t)(it / S) & 1u, p.d_err);
                    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int c = 0; c < D / 16; ++c)
                        sts128(sb + sl * L::kSlot + swizzled<128>(t / L::kPar, (t % L::kPar) * D + c * 16), zero);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_before();
                mbar_arrive1(&p_full[b]);
            }
            g0 += q.n;

            // row sums over the 128 key lanes, then the four warps
            const float wsum = warp_scatter<false, G>(l_part, lane);
            if ((lane & (32 / G - 1)) == 0) xsum[sw * GP + lane / (32 / G)] = wsum;
            const int gl = g0 - 1;
            await(&pv_done[gl & 1], (uint32_t)(gl >> 1) & 1u, p.d_err);
            tc_fence_after();
            float v[G];
            {
                float o[N];
#pragma unroll
                for (int i0 = 0; i0 < N; i0 += 16)
                    tmem_ld16(tmem + lane_off + col_o + i0, *reinterpret_cast<float(*)[16]>(&o[i0]));
#pragma unroll
                for (int h = 0; h < G; ++h)
                    v[h] = fmaf(fmaf(fmaf(o[3 * GP + h], 0.125f, o[2 * GP + h]), 0.125f, o[GP + h]), 0.125f, o[h]);
            }
            tc_fence_before();  // the next piece's first PV overwrites O
            if constexpr (L::kPar == 2) {
                if (par) {
#pragma unroll
                    for (int h = 0; h < G; ++h) odd[h * 64 + d] = v[h];
                }
            }
            named_bar_sync(1, 128);
            if (par == 0) {
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    if constexpr (L::kPar == 2) v[h] += odd[h * 64 + d];
                    const float lsum = (xsum[h] + xsum[GP + h]) + (xsum[2 * GP + h] + xsum[3 * GP + h]);
                    if (q.slot < 0) {
                        static_cast<T *>(p.out)[(row0 + h) * D + d] = (T)(lsum != 0.f ? __fdividef(v[h], lsum) : 0.f);
                    } else {
                        const size_t at = (size_t)q.slot * G + h;
                        p.ws_acc[at * D + d] = v[h];
                        if (d == h) p.ws_ml[at] = make_float2(m_run[h], lsum);
                    }
                }
            }
            // (the next piece's sums go to xsum and odd after its own tiles' barriers)
        }
    }
    tc_fence_before();
    __threadfence();  // the partials, before the counts below
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols) : "memory");
    }
    if (cuts[0].n == 0 && cuts[1].n == 0) return;
    // The last CTA to get here of those that have a unit's pieces merges them.  Which that
    // is does not change the result: the sums are the same.
    if (threadIdx.x < 2) {
        Cut &c = cuts[threadIdx.x];
        // (counts to n - 1 and then from 0 again: nothing is left for the next call)
        if (c.n > 0 && atomicInc(fp.counters + c.lead, (unsigned)(c.n - 1)) != (unsigned)(c.n - 1)) c.first = -1;
        __threadfence();
    }
    __syncthreads();
    merge_few<T, D, G>(p, cuts);
#pragma unroll 1
    for (int k = 0; k < 2; ++k)
        if (cuts[k].n > kFew && cuts[k].first >= 0) merge_many<T, D, G>(p, cuts[k], reinterpret_cast<float *>(smem));
}

// ---- host side -------------------------------------------------------------

// The pool as rows of `width` bytes, a block of a kv head one box of `rows` of them.
inline bool make_rows_map(CUtensorMap *map, const void *pool, long long all_rows, int width, int rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)all_rows};
    const cuuint64_t strides[1] = {(cuuint64_t)width};
    const cuuint32_t box[2] = {(cuuint32_t)width, (cuuint32_t)rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int G>
int launch_t(const Fp8DecodeParams &p, cudaStream_t stream) {
    auto kern = decode_fp8_kernel<T, D, G>;
    using L = Lay<D, G>;
    static std::atomic<uint64_t> attr_done{0};
    if (ensure_smem_attr(kern, L::kAlloc, attr_done) != PA_OK) return PA_ERR_CUDA;
    const long long rows = (long long)p.d.num_blocks * p.d.num_kv_heads * p.d.block_size;
    CUtensorMap tmk, tmv;
    if (!make_rows_map(&tmk, p.d.k_cache, rows, D, p.d.block_size) ||
        !make_rows_map(&tmv, p.d.v_cache, rows / L::kPar, 128, p.d.block_size / L::kPar))
        return PA_ERR_CUDA;
    return launch_pdl(kern, dim3(p.ctas), dim3(kThreads), L::kAlloc, stream, p, tmk, tmv) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <typename T, int D>
int launch_group(int group, const Fp8DecodeParams &p, cudaStream_t stream) {
    return group == 1   ? launch_t<T, D, 1>(p, stream)
           : group == 2 ? launch_t<T, D, 2>(p, stream)
           : group == 4 ? launch_t<T, D, 4>(p, stream)
                        : launch_t<T, D, 8>(p, stream);
}

template <typename T>
int launch_dtype(int head_dim, int group, const Fp8DecodeParams &p, cudaStream_t stream) {
    return head_dim == 128 ? launch_group<T, 128>(group, p, stream) : launch_group<T, 64>(group, p, stream);
}

}  // namespace d8
}  // namespace pa
