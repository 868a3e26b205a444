// Writing and reading back an 8-bit cache.
//
// store_fp8_kernel: a CTA has the blocks that up to 16 of the call's tokens are the first
// to name, and up to kHeadsPerCta kv heads of them, a warp for each.  For each block it
// finds all the call's tokens (the later one where two name the same slot), normalises
// and rotates their keys, and then decides the scale of each head:
//   need = the least e with amax <= 448 * 2^e, over the written rows
//   e    = need where the block's first row is among them (the block starts afresh),
//          else max(the old e, need)
// Rows that were there before are moved to a scale that grew, code by code.
//
// HBM-bound for prompts, latency-bound for steps of single tokens.  A warp has all of
// its rows' loads under way at once (16 rows of 128 values, keys and values) while the
// angles are computed, and keeps the values in registers between the maximum and the
// codes; only blocks with more rows than that are read twice.  To find a block's tokens
// every CTA reads the whole slot mapping, 8 bytes a token from L2 (8192 tokens: 64 KB
// beside the 64 KB of keys and values that eight heads of 16 tokens have).
// With the queries' kernel, which it starts beside: 8192 tokens of 64/8 heads of 128,
// bf16, 64.5 us, 73% of the copy rate (the queries alone take 45); 1021 of 40/40 heads,
// fp16, 20; a step of 256 tokens 8 on the device.  Rows read a second time for the codes
// took 108 and 51 us; a CTA per token, of which most had nothing to do, 114 and 38; a warp
// for keys and one for values, four heads to a CTA, 74 and 24; the rows computed before
// the slots are looked through 80 and 33 (every later run of a block does so in vain); two
// warps to a head's keys 81 and 28.  Looking through the slots costs 3 us of the 64.5, and
// grows with the square of the tokens: without rotation, 8 kv heads of 128, blocks of 16,
// bf16, 8192 tokens 15.2 us, 32768 84, 131072 648 (floors 7.4, 29.6, 118.5); with 40 kv heads
// 74, 380, 3193; blocks of 8 half as much again to twice; every fourth token padding 26, 178,
// 1894.  8192 tokens in blocks of their own 151 (1 kv head 160: a single warp looks).
#include <algorithm>
#include <type_traits>

#include "pa_fp8.cuh"
#include "pa_internal.h"
#include "pa_rotary.cuh"

namespace pa {
namespace {

constexpr int kHeadsPerCta = 8;
constexpr int kStoreThreads = 32 * kHeadsPerCta;  // at most

// kPasses: rows that a lane holds at a time.
template <typename T, bool kInterleaved, bool kNorm, int kPasses>
__global__ void __launch_bounds__(kStoreThreads, kPasses == 1 ? 4 : 2) store_fp8_kernel(const __grid_constant__ RotaryParams p) {
    __shared__ int s_tok[kStoreMaxBlock];   // token of each row, -1: not written
    __shared__ int s_row[kStoreMaxBlock];   // the written rows
    __shared__ int s_rows, s_late;
    __shared__ unsigned s_heads;            // tokens that may be the first of their block
    // [rows of a chunk][4 planes][units]: cosines of pairs 8c .. 8c+3, 8c+4 .. 8c+7, then
    // the sines alike, so that a row's lanes read side by side
    __shared__ float4 s_cs[kPasses * 32 * 4];
    __shared__ long long s_frac[kRotaryMaxDim / 2];  // turns per position, 2^-64
    __shared__ bool s_odd[kRotaryMaxDim / 2];        // whose frequency is not finite
    __shared__ uint8_t s_axis[kRotaryMaxDim / 2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bs = p.block_size, D = p.head_dim, shift = __ffs(bs) - 1;
    const int head0 = blockIdx.y * kHeadsPerCta, heads = min(kHeadsPerCta, p.num_kv_heads - head0);

    // (a launch beside this call's own query kernel reads nothing that one writes, and
    // waits for it at the end; any other launch starts when what was before it is done)
    // Of this CTA's tokens, those that do not follow another one of their block:
    const int first = blockIdx.x * p.tokens_per_cta;
    const int upr = D / 16, half = p.rot_dim / 2, lanes = norm_lanes(upr);
    if (warp == 0) {
        const int t = first + lane;
        bool head = lane < p.tokens_per_cta && t < p.num_tokens;
        if (head) {
            const long long slot = p.slots[t], prev = t > 0 ? p.slots[t - 1] : -1;
            head = slot >= 0;
            if (head && slot >= (long long)p.num_blocks * bs) {
                if (blockIdx.y == 0) flag_error(p.d_err, PA_DEVERR_SLOT_RANGE);
                head = false;
            }
            if (head && (unsigned long long)(prev - (slot >> shift << shift)) < (unsigned long long)bs) head = false;
        }
        const unsigned m = __ballot_sync(kFull, head);
        if (lane == 0) s_heads = m;
    }
    for (int i = tid; i < half; i += blockDim.x) {
        const float f = p.inv_freq[i];
        s_odd[i] = !isfinite(f);
        s_frac[i] = turn_fraction(f);
        s_axis[i] = p.one_axis ? 0 : p.pair_axis[i];
    }
    __syncthreads();
    for (unsigned heads_left = s_heads; heads_left; heads_left &= heads_left - 1) {
        const int t0 = first + __ffs(heads_left) - 1;
        const long long slot = p.slots[t0], blk = slot >> shift, base = blk << shift;
        // this warp's head (the last heads' CTA may have idle warps), its tiles and scales
        const bool busy = warp < heads;
        const int h = head0 + (busy ? warp : 0);
        const long long at = blk * p.num_kv_heads + h;
        auto tile_of = [&](int which) { return static_cast<uint8_t *>(which ? p.v_cache : p.k_cache) + at * bs * D; };
        auto scale_at = [&](int which) { return (which ? p.v_scales : p.k_scales) + at; };
        const int old_k = (int)*scale_at(0) - 127, old_v = (int)*scale_at(1) - 127;
        // rows that may have to move: on their way while the slots are looked through
        if (busy && slot != base)
            for (int i = lane * 128; i < 2 * bs * D; i += 32 * 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(i < bs * D ? tile_of(0) + i : tile_of(1) + (i - bs * D)));
        __syncthreads();  // what the block before left in shared memory is read
        for (int i = tid; i < bs; i += blockDim.x) s_tok[i] = -1;
        if (tid == 0) s_late = 0;
        __syncthreads();
        auto look = [&](long long at, int t) {
            const unsigned long long r = (unsigned long long)(at - base);
            if (r < (unsigned long long)bs) {
                if (t < t0) s_late = 1;
                atomicMax(&s_tok[(int)r], t);
            }
        };
        const int odd = (int)(reinterpret_cast<uintptr_t>(p.slots) >> 3 & 1u);  // slots before the first 16-byte boundary
        const longlong2 *pairs = reinterpret_cast<const longlong2 *>(p.slots + odd);
        const int npairs = (p.num_tokens - odd) / 2;
#pragma unroll 8
        for (int i = tid; i < npairs; i += blockDim.x) {
            const longlong2 v = pairs[i];
            look(v.x, odd + 2 * i);
            look(v.y, odd + 2 * i + 1);
        }
        if (tid == 0 && odd) look(p.slots[0], 0);
        if (tid == 0 && odd + 2 * npairs < p.num_tokens) look(p.slots[p.num_tokens - 1], p.num_tokens - 1);
        __syncthreads();
        if (s_late) continue;
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
        __syncthreads();
        const int c = lane % lanes, k0 = lane / lanes, per_warp = 32 / lanes;  // rows k0, + per_warp, ... are this lane's
        const int per_chunk = kPasses * per_warp;
        const int nrows = s_rows, chunks = (nrows + per_chunk - 1) / per_chunk;
        const bool fresh = s_tok[0] >= 0;
        const bool turned = c < p.rot_dim / 16;
        const int e0 = turned && !kInterleaved ? c * 8 : c * 16;
        const int e1 = turned && !kInterleaved ? half + c * 8 : e0 + 8;
        const float per_dim = 1.f / (float)D;
        uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
        if (kNorm && c < upr) {
            w0 = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.key_norm) + e0);
            w1 = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.key_norm) + e1);
        }

        auto rows_of = [&](int ch) { return min(per_chunk, nrows - ch * per_chunk); };
        // the units of this lane's rows of a chunk, of keys or values
        auto load = [&](int which, int ch, uint4(&va)[kPasses], uint4(&vb)[kPasses]) {
            const int n = rows_of(ch);
            const T *src = (which ? static_cast<const T *>(p.value) : static_cast<const T *>(p.key)) + (long long)h * D;
            const long long stride = which ? p.value_stride : p.key_stride;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int k = k0 + i * per_warp;
                va[i] = vb[i] = make_uint4(0, 0, 0, 0);
                if (busy && k < n && c < upr) {
                    const T *row = src + s_tok[s_row[ch * per_chunk + k]] * stride;
                    va[i] = *reinterpret_cast<const uint4 *>(row + e0);
                    vb[i] = *reinterpret_cast<const uint4 *>(row + e1);
                }
            }
        };
        // the angles of a chunk's rows, by all warps
        auto angles = [&](int ch) {
            if (half == 0) return;
            const int n = rows_of(ch);
            __syncthreads();  // the angles of the chunk before are read
            const int by_row = blockDim.x / half, by_pair = blockDim.x - by_row * half;
            int k = tid / half, pair = tid - k * half;
            while (k < n) {
                float sn, cs;
                turn_sincos(s_frac[pair], p.positions[(long long)s_axis[pair] * p.num_tokens + s_tok[s_row[ch * per_chunk + k]]], sn, cs);
                if (s_odd[pair]) sn = cs = __int_as_float(0x7fc00000);
                float *q = reinterpret_cast<float *>(s_cs) + k * 2 * half + (pair >> 2 & 1) * (half / 2) + (pair >> 3) * 4 + (pair & 3);
                q[0] = cs;
                q[half] = sn;
                k += by_row;
                pair += by_pair;
                if (pair >= half) pair -= half, ++k;
            }
            __syncthreads();
        };
        float a[kPasses][8], b[kPasses][8];  // the units of this lane's rows, as they are to be held
        // returns the largest magnitude among them (0 for lanes without a row)
        auto compute = [&](int which, int ch, const uint4(&va)[kPasses], const uint4(&vb)[kPasses]) {
            const int n = rows_of(ch);
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                unpack8<T>(va[i], a[i]);
                unpack8<T>(vb[i], b[i]);
                if (which == 0) {
                    if constexpr (kNorm) norm_unit<T>(a[i], b[i], lanes, per_dim, p.eps, w0, w1);
                    const int k = k0 + i * per_warp;
                    if (turned && k < n) {
                        float cs[8], sn[8];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float4 u = s_cs[k * (half / 2) + x * (half / 8) + c], v = s_cs[k * (half / 2) + (2 + x) * (half / 8) + c];
                            cs[4 * x] = u.x, cs[4 * x + 1] = u.y, cs[4 * x + 2] = u.z, cs[4 * x + 3] = u.w;
                            sn[4 * x] = v.x, sn[4 * x + 1] = v.y, sn[4 * x + 2] = v.z, sn[4 * x + 3] = v.w;
                        }
                        turn_unit<kInterleaved>(a[i], b[i], cs, sn);
                    }
                }
            }
            // (the bits of magnitudes order as they do, infinities and NaN above all)
            unsigned top = 0u;
#pragma unroll
            for (int i = 0; i < kPasses; ++i)
                if (k0 + i * per_warp < n && c < upr) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        top = max(top, max(__float_as_uint(a[i][x]) & 0x7fffffffu, __float_as_uint(b[i][x]) & 0x7fffffffu));
                }
            if (__any_sync(kFull, top > top_held<T>())) {  // rare: what cannot be held as it is
                float most = 0.f;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const bool on = k0 + i * per_warp < n && c < upr;
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        a[i][x] = holdable<T>(a[i][x]);
                        b[i][x] = holdable<T>(b[i][x]);
                        if (on) most = fmaxf(most, fmaxf(counted(a[i][x]), counted(b[i][x])));
                    }
                }
                return most;
            }
            return __uint_as_float(top);
        };
        // the scale that the lanes' largest magnitudes ask for, and the rows that it moves;
        // returns what brings values to codes
        auto settle = [&](int which, float amax, int old) {
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, m));
            const int need = scale_exponent(amax), e = fresh ? need : max(old, need);
            if (busy && lane == 0) *scale_at(which) = (uint8_t)(e + 127);
            if (busy && !fresh && e > old) {
                const float down = __uint_as_float((unsigned)(max(old - e, -32) + 127) << 23);
                for (int i = lane; i < bs * upr; i += 32) {
                    if (s_tok[i / upr] >= 0) continue;
                    uint4 *q = reinterpret_cast<uint4 *>(tile_of(which)) + i;
                    float f[16];
                    values16(*q, f);
#pragma unroll
                    for (int x = 0; x < 16; ++x) f[x] *= down;
                    *q = make_uint4(codes4(f[0], f[1], f[2], f[3]), codes4(f[4], f[5], f[6], f[7]),
                                    codes4(f[8], f[9], f[10], f[11]), codes4(f[12], f[13], f[14], f[15]));
                }
            }
            return scale_of(min((unsigned)(127 - e), 255u));  // (2^-127 beside a scale of 2^127, NaN beside NaN)
        };
        // the codes of the units that are held
        auto put = [&](int which, int ch, float up) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int k = k0 + i * per_warp;
                if (busy && k < rows_of(ch) && c < upr) {
                    uint8_t *row = tile_of(which) + s_row[ch * per_chunk + k] * D;
                    const float(&x)[8] = a[i], (&y)[8] = b[i];
                    *reinterpret_cast<uint2 *>(row + e0) =
                        make_uint2(codes4(x[0] * up, x[1] * up, x[2] * up, x[3] * up), codes4(x[4] * up, x[5] * up, x[6] * up, x[7] * up));
                    *reinterpret_cast<uint2 *>(row + e1) =
                        make_uint2(codes4(y[0] * up, y[1] * up, y[2] * up, y[3] * up), codes4(y[4] * up, y[5] * up, y[6] * up, y[7] * up));
                }
            }
        };
        uint4 ka[kPasses], kb[kPasses], va[kPasses], vb[kPasses];
        if (chunks == 1) {
            load(0, 0, ka, kb);
            load(1, 0, va, vb);
            angles(0);
            put(0, 0, settle(0, compute(0, 0, ka, kb), old_k));
            put(1, 0, settle(1, compute(1, 0, va, vb), old_v));
        } else {
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                float amax = 0.f;
#pragma unroll 1
                for (int step = 0; step < 2 * chunks - 1; ++step) {
                    // chunks upwards for the largest magnitude, then down again for the codes, the last one once
                    const int ch = step < chunks ? step : 2 * chunks - 2 - step;
                    load(which, ch, va, vb);
                    if (which == 0) angles(ch);
                    const float most = compute(which, ch, va, vb);
                    if (step < chunks) amax = fmaxf(amax, most);
                    if (step == chunks - 1) amax = settle(which, amax, which ? old_v : old_k);
                    if (step >= chunks - 1) put(which, ch, amax);
                }
            }
        }
    }

    pdl_wait();
    pdl_trigger();
}

// ---- reading back ------------------------------------------------------------

// CTA (b, piece): piece of block b of the laid-out sequences, four vectors of 8 codes a
// thread, all on their way together, each into one vector of 16-bit values, side by side
// with its neighbours' (vectors of 16 codes, whose two halves are stored 32 bytes apart
// from lane to lane, cost a chunk after 8192 tokens 3 us more, eight of those 9).
constexpr int kExpandVectors = 4;
template <typename T>
__global__ void __launch_bounds__(256) expand_fp8_kernel(const __grid_constant__ Fp8ExpandParams p) {
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    const int at = blockIdx.x;
    if (blockIdx.y == 0)
        for (long long i = (long long)at * blockDim.x + tid; i < p.num_zero; i += (long long)gridDim.x * blockDim.x) p.zero[i] = 0u;
    int lo = 0, hi = p.num_seqs;  // first[lo] <= at < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.first[mid] <= at) lo = mid;
        else hi = mid;
    }
    const int blk = p.tables[lo][at - p.first[lo]];
    const bool ok = blk >= 0 && blk < p.num_blocks;
    const int parts = p.block_size / kExpandRows;
    if (blockIdx.y == 0) {
        for (int i = tid; i < parts; i += 256) p.table[at * parts + i] = ok ? at * parts + i : -1;
        if (tid == 0 && !ok) flag_error(p.d_err, PA_DEVERR_BLOCK_RANGE);
    }
    if (!ok) return;
    // vectors of a head's block and of a part of it: powers of two, like block_size and head_dim
    const int head_bits = __ffs(p.block_size * p.head_dim / 8) - 1, part_bits = __ffs(kExpandRows * p.head_dim / 8) - 1;
    const int n = p.num_kv_heads << head_bits;
    const size_t src0 = (size_t)blk * n, dst0 = (size_t)at * n;
    const int i0 = blockIdx.y * (256 * kExpandVectors) + tid;
    uint2 u[kExpandVectors];
#pragma unroll
    for (int k = 0; k < kExpandVectors; ++k) {
        const int i = i0 + k * 256, j = i >= n ? i - n : i;
        if (i < 2 * n) u[k] = reinterpret_cast<const uint2 *>(i >= n ? p.v_cache : p.k_cache)[src0 + j];
    }
    // the greatest scales of the tile that this block is in, of the heads whose values these are
    constexpr bool kOver = std::is_same<T, __nv_bfloat16>::value;
    __shared__ int s_top[256 * kExpandVectors / 128 + 1];  // (a head has 128 vectors at least)
    const int from = max((int)blockIdx.y * 256 * kExpandVectors - n, 0);
    const int to = min((int)(blockIdx.y + 1) * 256 * kExpandVectors, 2 * n) - n;  // (none: <= 0)
    const int head0 = from >> head_bits;
    if (kOver && to > 0) {
        const int heads = ((to - 1) >> head_bits) - head0 + 1, blocks = p.first[lo + 1] - p.first[lo];
        const int per_tile = kExpandTile / p.block_size, b = ((at - p.first[lo]) & -per_tile) + (tid & 7);
        // eight lanes a head, one of them a block of the tile
        for (int h = tid >> 3; h - (tid >> 3) < heads; h += 32) {
            unsigned byte = 0u;
            if (h < heads && (tid & 7) < per_tile && b < blocks) {
                const int blk2 = p.tables[lo][b];
                if (blk2 >= 0 && blk2 < p.num_blocks) byte = p.v_scales[(size_t)blk2 * p.num_kv_heads + head0 + h];
            }
            if (byte == 255u) byte = 0u;
#pragma unroll
            for (int m = 4; m > 0; m >>= 1) byte = max(byte, __shfl_xor_sync(kFull, byte, m));
            if (h < heads && (tid & 7) == 0) s_top[h] = (int)byte;
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kExpandVectors; ++k) {
        const int i = i0 + k * 256, j = i >= n ? i - n : i;
        if (i >= 2 * n) continue;
        const bool is_v = i >= n;
        const int head = j >> head_bits, rest = j & ((1 << head_bits) - 1);
        const unsigned byte = (is_v ? p.v_scales : p.k_scales)[(size_t)blk * p.num_kv_heads + head];
        float f = scale_of(byte);
        if (kOver && is_v) {
            // (exact down to 2^-22 of the greatest scale, nothing below 2^-41)
            const int e = (int)byte - s_top[head - head0] + kValueLift + 127;
            f = byte == 255u ? f : e > 0 ? scale_of((unsigned)e) : 0.f;
        }
        const float2 a = values2(u[k].x & 0xffffu), b = values2(u[k].x >> 16), c = values2(u[k].y & 0xffffu), d = values2(u[k].y >> 16);
        const float x[8] = {a.x * f, a.y * f, b.x * f, b.y * f, c.x * f, c.y * f, d.x * f, d.y * f};
        const int dst = ((((rest >> part_bits) * p.num_kv_heads) + head) << part_bits) + (rest & ((1 << part_bits) - 1));
        reinterpret_cast<uint4 *>(is_v ? p.v_out : p.k_out)[dst0 + dst] = kOver && is_v ? pack8<__half>(x) : pack8<T>(x);
    }
}

// After this call's query kernel (`beside`) it may start while that one runs; else not
// before everything that was queued has ended.
template <typename T, bool kInterleaved, bool kNorm, int kPasses>
cudaError_t store_t(const RotaryParams &p, bool beside, cudaStream_t stream) {
    const unsigned splits = (unsigned)((p.num_kv_heads + kHeadsPerCta - 1) / kHeadsPerCta);
    const dim3 grid((unsigned)((p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta), splits);
    const dim3 block(32 * std::min(kHeadsPerCta, p.num_kv_heads));
    auto kern = store_fp8_kernel<T, kInterleaved, kNorm, kPasses>;
    if (beside) return launch_pdl(kern, grid, block, 0, stream, p);
    kern<<<grid, block, 0, stream>>>(p);
    return cudaPeekAtLastError();
}

template <typename T, bool kInterleaved, bool kNorm>
cudaError_t store_passes(const RotaryParams &p, bool beside, cudaStream_t stream) {
    return p.tokens_per_cta == 1 ? store_t<T, kInterleaved, kNorm, 1>(p, beside, stream)
                                 : store_t<T, kInterleaved, kNorm, 4>(p, beside, stream);
}

template <typename T>
cudaError_t store_dtype(const RotaryParams &p, bool beside, cudaStream_t stream) {
    if (p.key_norm)
        return p.interleaved ? store_passes<T, true, true>(p, beside, stream) : store_passes<T, false, true>(p, beside, stream);
    return p.interleaved ? store_passes<T, true, false>(p, beside, stream) : store_passes<T, false, false>(p, beside, stream);
}

}  // namespace

int launch_store_fp8(pa_dtype dt, const RotaryParams &p, cudaStream_t stream) {
    if (p.num_heads > 0) {
        RotaryParams q = p;
        q.num_kv_heads = 0;
        const int rc = q.query_norm ? launch_norm_rotary(dt, q, stream) : launch_rotary(dt, q, stream);
        if (rc != PA_OK) return rc;
    }
    const bool beside = p.num_heads > 0;
    // One token to a CTA while that gives no more than four CTAs to an SM, up to 16 beyond
    // (a prompt, where one of 16 begins a block).  With one token, the variant that holds one
    // row a lane, of half the registers, leaves room for all CTAs at once: right for a step
    // of single tokens; a block's rows it reads twice, in chunks.  Both sides (the host does
    // not see the slots), bf16, heads of 128, replayed, us, one row / four rows a lane:
    //                                        step        run of one sequence
    //   without rotation, 256 tokens, 2 kv   4.2 / 5.4     9.0 / 5.7
    //                     256         8      4.5 / 5.5    10.9 / 7.1
    //                     600         8      6.2 / 9.9    13.8 / 7.5
    //   norms, rotation,  256         8      8.8 / 9.9    16.7 / 11.0
    RotaryParams q = p;
    const long long all = (long long)p.num_tokens * ((p.num_kv_heads + kHeadsPerCta - 1) / kHeadsPerCta);
    q.tokens_per_cta = (int)std::min(16LL, std::max(1LL, all / (2LL * sm_count())));
    const cudaError_t e = dt == PA_BF16 ? store_dtype<__nv_bfloat16>(q, beside, stream) : store_dtype<__half>(q, beside, stream);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int launch_expand_fp8(pa_dtype dt, const Fp8ExpandParams &p, cudaStream_t stream) {
    const int blocks = p.first[p.num_seqs];
    if (blocks == 0) return PA_OK;
    const long long vectors = 2LL * p.num_kv_heads * p.block_size * p.head_dim / 8;
    const long long pieces = (vectors + 256 * kExpandVectors - 1) / (256 * kExpandVectors);
    if (pieces > 65535) return PA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks, (unsigned)pieces);
    const cudaError_t e = dt == PA_BF16 ? launch_pdl(expand_fp8_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, p)
                                        : launch_pdl(expand_fp8_kernel<__half>, grid, dim3(256), 0, stream, p);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
