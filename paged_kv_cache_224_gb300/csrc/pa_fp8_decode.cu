// Paged decode attention over an 8-bit cache on the tensor cores (tcgen05,
// kind::f8f6f4).
//
// With k_j = code * 2^(ek_j), v_j = code * 2^(ev_j) of key j's block, and scores in
// log2 units (scale * log2(e) in the query's factor), the sums that are kept run over
//     z_j = s_j + ev_j,   o = sum_j 2^(z_j - M) * (codes of v_j),
//     l = sum_j 2^(z_j - M) * 2^(-ev_j),   M the running maximum of z,
// and out = o / l: the scales of the values only move exponents, and however far the
// scales of two blocks are apart, the terms of o are as exact as their weights.  The
// terms of l are 2^(s_j - M) in one step where 2^(z_j - M) would be too small for fp32
// (scales from 2^-64 to 2^120 occur), and l is moved from one M to another in two halves.
//
// The codes go to the MMAs as they lie in memory, with keys as the M dimension:
//   S^T[128 keys][N] = K[128 keys][D] . Q^T
//   O^T[128][NO] += V^T[128][keys] . P^T    (V read in place, MN-major)
// An 8-bit operand on the other side would leave a query or a weight 3 or 4 bits, so
// each goes in as several rows of N, every one the rounded residual of those before
// times a power of two: queries as four e4m3 rows (16 bits, and for elements below the
// head's largest 2^-32 of that: scores are as exact as fp32 sums unless the keys meet a
// query's largest elements with next to nothing; with three rows an element of 10^4 beside
// N(0, 0.02^2) took the small ones' scores off by 1%), weights as four e5m2 rows (12
// bits down to 2^-25 of the largest weight, off by 2^-37 of that below; e5m2 for its
// range: a long context may hold very many small weights, all rounded alike).  N is padded to 16 by the
// MMA anyway (32 for eight heads).
//
// HBM-bound: every code is read once, and 128 keys of a kv head are 32 KB.  The call's
// tiles of 128 keys lie end to end and every CTA, two to an SM, takes an equal share of
// them, whatever the lengths are: one start per CTA, no tail, and no more than two
// partials per CTA, which the last CTA to finish one of a unit's pieces merges.  A CTA is
//   warp 0    TMA producer: one copy per (block, K or V) into a ring of 96 KB, tiles in
//             the order that the MMAs take them, running on from one sequence to the next;
//   warp 1    MMA issuer (one thread): QK^T of tile j into one of two S buffers, then
//             O += P V of tile j-1;
//   warps 2-5 softmax, one thread per key (= TMEM lane): scores, maxima over the tile,
//             O rescaled only when a maximum has grown by 2^4, weights to shared memory;
//             at a piece's end one thread per dimension writes the output or the partial;
//   warp 6    the next piece's queries, and the scales of each tile's blocks up to eight
//             tiles ahead.
// At head_dim 64, where a tile is 16 KB, three CTAs to an SM (two with eight heads).
//
// Measured (bf16, us, share of the copy rate): 256 contexts of up to 4096 tokens, 32/8
// heads of 128, 177, 94%; eight of 32768 to 131072, 64/8 heads, 209, 97%; 256 of 2048, 32/8
// heads of 64, 91.5, 86%, 64/8 heads of 64, 132, 60% (bound by the softmax warps).  On the
// way (the first two cases): on the CUDA cores 1088 and 2367; one unit (sequence, kv head,
// 1024 tokens) a CTA 203 and 228; equal shares 196 and 216.  What runs once a piece was
// kept small after 256 contexts of 2048 tokens with 64/8 heads had taken 234, not 168: the
// roles' code did not stay in the instruction cache together.  A vote instead of every
// tile's maxima: 1024 contexts of 512 tokens, 64/8 heads, 197 -> 188.  The merge at the end of
// this kernel, not in one behind it: 188 -> 183, one context of 4096, 32/8 heads, 15.1 -> 11.5.
// All waits are bounded; a wait that gives up flags PA_DEVERR_TIMEOUT.
#include <algorithm>
#include <cmath>

#include "pa_internal.h"

namespace pa {

int launch_decode_fp8_bf16(int head_dim, int group, const Fp8DecodeParams &p, cudaStream_t stream);
int launch_decode_fp8_f16(int head_dim, int group, const Fp8DecodeParams &p, cudaStream_t stream);

// As many CTAs as the SMs hold, but at most 4 sqrt(tiles) to a (sequence, kv head) of the
// greatest length: its pieces are merged by one CTA, and with p pieces that takes as long
// as p grows, the pieces themselves as tiles / p does.  One context of 131072 tokens, 8/1
// heads: 35 us by all 304 CTAs (1024 tiles), 28.6 by up to 6 sqrt(tiles), 25.2 by 4 or 3,
// 27.5 by 2; of 16384: 20.0, 16.3, 15.1, 15.4.  64/8 heads reach all 304 either way.
int fp8_decode_ctas(int num_seqs, int num_kv_heads, int group, int head_dim, int max_context_len) {
    const long long units = (long long)num_seqs * num_kv_heads, tiles = ((long long)max_context_len + 127) / 128;
    const long long pieces = std::min(tiles, (long long)std::ceil(4.0 * std::sqrt((double)tiles)));
    const long long most = std::min((long long)d8::ctas_per_sm(head_dim, group) * sm_count(), (long long)kFp8MaxCtas);
    return (int)std::max(1LL, std::min(most, units * pieces));
}

int launch_decode_fp8(pa_dtype dt, int head_dim, int group, const Fp8DecodeParams &p, cudaStream_t stream) {
    return dt == PA_BF16 ? launch_decode_fp8_bf16(head_dim, group, p, stream) : launch_decode_fp8_f16(head_dim, group, p, stream);
}

}  // namespace pa
