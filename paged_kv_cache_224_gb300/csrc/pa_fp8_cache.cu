// Writing and reading back an 8-bit cache.
//
// store_fp8_kernel: one CTA per block that the call's tokens write to, and up to
// kHeadsPerCta kv heads of it.  The CTA of the first token that names a block finds
// all the call's tokens for it (the later one where two name the same slot),
// normalises and rotates their keys, and then decides the scale of each head:
//   need = the least e with amax <= 448 * 2^e, over the written rows
//   e    = need where the block's first row is among them (the block starts afresh),
//          else max(the old e, need)
// Rows that were there before are moved to a scale that grew, code by code.
// The values are computed twice, once for the amax and once for the codes: the rows
// come from L1 or L2 the second time, and nothing is kept per row.
#include <algorithm>
#include <type_traits>

#include "pa_fp8.cuh"
#include "pa_internal.h"
#include "pa_rotary.cuh"

namespace pa {
namespace {

constexpr int kStoreThreads = 256;
constexpr int kStoreWarps = kStoreThreads / 32;
constexpr int kHeadsPerCta = 16;
constexpr int kChunkRows = 16;  // rows whose angles are held at a time

template <typename T, bool kInterleaved, bool kNorm>
__global__ void __launch_bounds__(kStoreThreads) store_fp8_kernel(const __grid_constant__ RotaryParams p) {
    __shared__ int s_tok[kStoreMaxBlock];   // token of each row, -1: not written
    __shared__ int s_row[kStoreMaxBlock];   // the written rows
    __shared__ int s_rows, s_late;
    __shared__ float2 s_cs[kChunkRows][kRotaryMaxDim / 2];
    __shared__ float s_amax[2][kHeadsPerCta];
    __shared__ float s_w[kNorm ? kRotaryMaxDim : 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bs = p.block_size, D = p.head_dim;
    const int head0 = blockIdx.y * kHeadsPerCta, heads = min(kHeadsPerCta, p.num_kv_heads - head0);

    pdl_wait();
    pdl_trigger();  // what follows may be placed; it waits for these writes

    const int t0 = blockIdx.x;
    const long long slot = p.slots[t0];
    if (slot < 0) return;
    if (slot >= (long long)p.num_blocks * bs) {
        if (tid == 0 && blockIdx.y == 0) flag_error(p.d_err, PA_DEVERR_SLOT_RANGE);
        return;
    }
    const long long blk = slot / bs, base = blk * bs;
    // a token that follows another of its block is not the block's first
    if (t0 > 0 && (unsigned long long)(p.slots[t0 - 1] - base) < (unsigned long long)bs) return;
    for (int i = tid; i < bs; i += kStoreThreads) s_tok[i] = -1;
    if (tid == 0) s_late = 0;
    __syncthreads();
    for (int t = tid; t < p.num_tokens; t += kStoreThreads) {
        const unsigned long long r = (unsigned long long)(p.slots[t] - base);
        if (r < (unsigned long long)bs) {
            if (t < t0) s_late = 1;
            atomicMax(&s_tok[(int)r], t);
        }
    }
    __syncthreads();
    if (s_late) return;
    if (warp == 0) {
        int n = 0;
        for (int i = 0; i < bs; i += 32) {
            const bool has = i + lane < bs && s_tok[i + lane] >= 0;
            const unsigned m = __ballot_sync(kFull, has);
            if (has) s_row[n + __popc(m & ((1u << lane) - 1u))] = i + lane;
            n += __popc(m);
        }
        if (lane == 0) s_rows = n;
    }
    if constexpr (kNorm)
        for (int i = tid; i < D; i += kStoreThreads) s_w[i] = to_float(static_cast<const T *>(p.key_norm)[i]);
    __syncthreads();
    const int nrows = s_rows, chunks = (nrows + kChunkRows - 1) / kChunkRows;
    const bool fresh = s_tok[0] >= 0;

    const int upr = D / 16, half = p.rot_dim / 2, lanes = norm_lanes(upr);
    const int c = lane % lanes, per_warp = 32 / lanes;
    const bool active = c < upr, turned = c < p.rot_dim / 16;
    const int e0 = turned && !kInterleaved ? c * 8 : c * 16;
    const int e1 = turned && !kInterleaved ? half + c * 8 : e0 + 8;
    const float per_dim = 1.f / (float)D;

    auto angles = [&](int chunk) {
        const int n = min(kChunkRows, nrows - chunk * kChunkRows);
        for (int i = tid; i < n * half; i += kStoreThreads) {
            const int k = i / half, pair = i - k * half;
            const float f = p.inv_freq[pair];
            float sn, cs;
            turn_sincos(turn_fraction(f),
                        p.positions[(long long)p.pair_axis[pair] * p.num_tokens + s_tok[s_row[chunk * kChunkRows + k]]], sn, cs);
            if (!isfinite(f)) sn = cs = __int_as_float(0x7fc00000);
            s_cs[k][pair] = make_float2(cs, sn);
        }
    };
    // the unit of row k of the chunk, of head h's key or value, as it is to be held
    auto unit = [&](int which, int h, int chunk, int k, float (&a)[8], float (&b)[8]) {
        const int t = s_tok[s_row[chunk * kChunkRows + k]];
        const T *src = which ? static_cast<const T *>(p.value) + t * p.value_stride : static_cast<const T *>(p.key) + t * p.key_stride;
        src += (long long)(head0 + h) * D;
        uint4 va = make_uint4(0, 0, 0, 0), vb = va;
        if (active) {
            va = *reinterpret_cast<const uint4 *>(src + e0);
            vb = *reinterpret_cast<const uint4 *>(src + e1);
        }
        unpack8<T>(va, a);
        unpack8<T>(vb, b);
        if (which == 0) {
            if constexpr (kNorm) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
                for (int m = lanes >> 1; m > 0; m >>= 1) sum += __shfl_xor_sync(kFull, sum, m);
                const float r = __frsqrt_rn(fmaf(sum, per_dim, p.eps));
                if (active) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a[i] *= r * s_w[e0 + i];
                        b[i] *= r * s_w[e1 + i];
                    }
                }
            }
            if (turned) {
                const float2 *q = s_cs[k] + c * 8;
                if (kInterleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
                        a[2 * i] = fmaf(x, q[i].x, -(y * q[i].y));
                        a[2 * i + 1] = fmaf(y, q[i].x, x * q[i].y);
                        b[2 * i] = fmaf(z, q[4 + i].x, -(w * q[4 + i].y));
                        b[2 * i + 1] = fmaf(w, q[4 + i].x, z * q[4 + i].y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float x = a[i], y = b[i];
                        a[i] = fmaf(x, q[i].x, -(y * q[i].y));
                        b[i] = fmaf(y, q[i].x, x * q[i].y);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = holdable<T>(a[i]);
            b[i] = holdable<T>(b[i]);
        }
    };

    // ---- the largest magnitudes; a (key or value, head) belongs to one warp throughout
    for (int j = warp; j < 2 * heads; j += kStoreWarps)
        if (lane == 0) s_amax[j / heads][j % heads] = 0.f;
    __syncwarp();
    for (int ch = 0; ch < chunks; ++ch) {
        __syncthreads();
        angles(ch);
        __syncthreads();
        const int n = min(kChunkRows, nrows - ch * kChunkRows);
        for (int j = warp; j < 2 * heads; j += kStoreWarps) {
            const int which = j / heads, h = j % heads;
            float amax = 0.f;
            for (int k0 = 0; k0 < n; k0 += per_warp) {
                const int k = min(k0 + lane / lanes, n - 1);  // lanes past the rows look at the last one again
                float a[8], b[8];
                unit(which, h, ch, k, a, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(counted(a[i]), counted(b[i])));
            }
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, m));
            if (lane == 0) s_amax[which][h] = fmaxf(s_amax[which][h], amax);
            __syncwarp();
        }
    }
    // ---- the codes
    for (int ch = chunks - 1; ch >= 0; --ch) {
        if (chunks > 1) {
            __syncthreads();
            angles(ch);
            __syncthreads();
        }
        const int n = min(kChunkRows, nrows - ch * kChunkRows);
        for (int j = warp; j < 2 * heads; j += kStoreWarps) {
            const int which = j / heads, h = j % heads;
            uint8_t *scale = (which ? p.v_scales : p.k_scales) + blk * p.num_kv_heads + head0 + h;
            uint8_t *tile = static_cast<uint8_t *>(which ? p.v_cache : p.k_cache) + (blk * p.num_kv_heads + head0 + h) * bs * D;
            const int need = scale_exponent(s_amax[which][h]);
            int e = need;
            if (ch == chunks - 1) {
                // (of several chunks the first one to come here moves the old rows and leaves the new scale)
                const int old = (int)*scale - 127;
                if (!fresh) e = max(old, need);
                __syncwarp();
                if (lane == 0) *scale = (uint8_t)(e + 127);
                if (!fresh && e > old) {
                    const float down = __uint_as_float((unsigned)(max(old - e, -32) + 127) << 23);
                    for (int i = lane; i < bs * upr; i += 32) {
                        const int r = i / upr;
                        if (s_tok[r] >= 0) continue;
                        uint4 *q = reinterpret_cast<uint4 *>(tile) + i;
                        float f[16];
                        values16(*q, f);
#pragma unroll
                        for (int x = 0; x < 16; ++x) f[x] *= down;
                        *q = make_uint4(codes4(f[0], f[1], f[2], f[3]), codes4(f[4], f[5], f[6], f[7]),
                                        codes4(f[8], f[9], f[10], f[11]), codes4(f[12], f[13], f[14], f[15]));
                    }
                }
                __syncwarp();
            } else if (!fresh) {
                e = (int)*scale - 127;
            }
            const float up = __uint_as_float((unsigned)(127 - e) << 23);
            for (int k0 = 0; k0 < n; k0 += per_warp) {
                const int k = min(k0 + lane / lanes, n - 1);
                float a[8], b[8];
                unit(which, h, ch, k, a, b);
                if (active && k0 + lane / lanes < n) {
                    uint8_t *row = tile + s_row[ch * kChunkRows + k] * D;
                    uint2 x, y;
                    x = make_uint2(codes4(a[0] * up, a[1] * up, a[2] * up, a[3] * up), codes4(a[4] * up, a[5] * up, a[6] * up, a[7] * up));
                    y = make_uint2(codes4(b[0] * up, b[1] * up, b[2] * up, b[3] * up), codes4(b[4] * up, b[5] * up, b[6] * up, b[7] * up));
                    *reinterpret_cast<uint2 *>(row + e0) = x;
                    *reinterpret_cast<uint2 *>(row + e1) = y;
                }
            }
        }
    }
}

// ---- reading back ------------------------------------------------------------

// One CTA per block of the laid-out sequences: every thread turns vectors of 16
// codes into two vectors of 16-bit values.
template <typename T>
__global__ void __launch_bounds__(256) expand_fp8_kernel(const __grid_constant__ Fp8ExpandParams p) {
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    const int at = blockIdx.x;
    for (long long i = (long long)at * blockDim.x + tid; i < p.num_zero; i += (long long)gridDim.x * blockDim.x) p.zero[i] = 0u;
    int lo = 0, hi = p.num_seqs;  // first[lo] <= at < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.first[mid] <= at) lo = mid;
        else hi = mid;
    }
    const int blk = p.tables[lo][at - p.first[lo]];
    const bool ok = blk >= 0 && blk < p.num_blocks;
    if (tid == 0) {
        p.table[at] = ok ? at : -1;
        if (!ok) flag_error(p.d_err, PA_DEVERR_BLOCK_RANGE);
    }
    if (!ok) return;
    const int per_head = p.block_size * p.head_dim / 16, n = p.num_kv_heads * per_head;
    const size_t src0 = (size_t)blk * n, dst0 = (size_t)at * n;
    for (int i = tid; i < 2 * n; i += blockDim.x) {
        const bool is_v = i >= n;
        const int j = is_v ? i - n : i;
        const uint4 u = reinterpret_cast<const uint4 *>(is_v ? p.v_cache : p.k_cache)[src0 + j];
        const float s = scale_of((is_v ? p.v_scales : p.k_scales)[(size_t)blk * p.num_kv_heads + j / per_head]);
        float f[16];
        values16(u, f);
        float a[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            a[k] = f[k] * s;
            b[k] = f[8 + k] * s;
        }
        uint4 *dst = reinterpret_cast<uint4 *>(is_v ? p.v_out : p.k_out) + (dst0 + j) * 2;
        dst[0] = pack8<T>(a);
        dst[1] = pack8<T>(b);
    }
}

template <typename T, bool kInterleaved>
cudaError_t store_t(const RotaryParams &p, cudaStream_t stream) {
    const dim3 grid((unsigned)p.num_tokens, (unsigned)((p.num_kv_heads + kHeadsPerCta - 1) / kHeadsPerCta));
    return p.key_norm ? launch_pdl(store_fp8_kernel<T, kInterleaved, true>, grid, dim3(kStoreThreads), 0, stream, p)
                      : launch_pdl(store_fp8_kernel<T, kInterleaved, false>, grid, dim3(kStoreThreads), 0, stream, p);
}

}  // namespace

int launch_store_fp8(pa_dtype dt, const RotaryParams &p, cudaStream_t stream) {
    const cudaError_t e = dt == PA_BF16 ? (p.interleaved ? store_t<__nv_bfloat16, true>(p, stream) : store_t<__nv_bfloat16, false>(p, stream))
                                        : (p.interleaved ? store_t<__half, true>(p, stream) : store_t<__half, false>(p, stream));
    if (e != cudaSuccess) return PA_ERR_CUDA;
    if (p.num_heads == 0) return PA_OK;
    RotaryParams q = p;
    q.num_kv_heads = 0;
    return launch_rotary(dt, q, stream);
}

int launch_expand_fp8(pa_dtype dt, const Fp8ExpandParams &p, cudaStream_t stream) {
    const int blocks = p.first[p.num_seqs];
    if (blocks == 0) return PA_OK;
    const cudaError_t e = dt == PA_BF16 ? launch_pdl(expand_fp8_kernel<__nv_bfloat16>, dim3(blocks), dim3(256), 0, stream, p)
                                        : launch_pdl(expand_fp8_kernel<__half>, dim3(blocks), dim3(256), 0, stream, p);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
