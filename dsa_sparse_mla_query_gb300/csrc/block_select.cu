// block_select.cu -- blocks of keys for every query and key head, chosen by an
// upper bound of their scores (sm_103a).
//
// Per block and head the bounds lo_d <= k_d <= hi_d of its keys, in whole steps
// of a power of two s (lo rounded down, hi up, -127 .. 127), say for any query
//   q . k <= s sum_d max(q_d lo_d, q_d hi_d) = s (max(q, 0) . hi + min(q, 0) . lo).
// With q in whole steps too (-127 .. 127, one step for a token's group of heads)
// the sums are whole numbers below 2^22: exact in fp32 in any order, in the
// tensor cores as well, so the order of the blocks depends on nothing but the
// inputs, and ties are ties.
//
// - block_bounds_kernel: minimum and maximum over the keys of the blocks that new
//   tokens touch, a warp per block and head, keys read once.
// - block_score_kernel: the sums on the warp-level matrix instruction, 16 blocks
//   by 8 query rows, k-steps over lo with min(q, 0), then over hi with max(q, 0).
//   A warp holds 16 blocks' bounds as f16 fragments straight from global memory
//   (the order of the dims within a k-step is the same for both operands and free
//   otherwise, so a thread's 16 bytes make whole fragments) and walks the query
//   rows, which lie in shared memory as fragments.  With one token a sequence it
//   reads 2 D bytes a block once: HBM.  With a prompt's tokens a product of
//   [tokens heads] x [blocks]: the matrix instruction.
// - block_pick_kernel: the nsel best of a row by a histogram over the keys' range
//   (order-preserving codes), one CTA per query and key head.
#include <algorithm>

#include "gqa_common.cuh"
#include "segments.cuh"

namespace dsa {
namespace gqa {
namespace {

// ---------------------------------------------------------------------------
// bounds
constexpr int kBoundThreads = 256;

struct BoundArgs {
    const uint8_t* k;  // the cache, bytes
    const float* k_scale;
    int8_t* bounds;    // [blocks][hkv][2][D]
    float* steps;      // [blocks][hkv]
    dsa_seqs s;
    int64_t stride;    // bytes between rows
    int32_t* d_status;
    int32_t num_q, hkv, shift, scale_shift;
};

template <int D, bool FP8>
__global__ void __launch_bounds__(kBoundThreads) block_bounds_kernel(const __grid_constant__ BoundArgs a) {
    constexpr int V = FP8 ? 16 : 8;    // dims per lane
    constexpr int L = D / V;           // lanes per row
    constexpr int R = 32 / L;          // rows per access
    __shared__ Pieces<kBoundThreads> pieces;
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int li = lane % L, sub = lane / L;
    int64_t before = 0;
    for (int c0 = 0; c0 < a.s.num_seqs; c0 += Pieces<kBoundThreads>::kChunk) {
        const int left = min(Pieces<kBoundThreads>::kChunk, a.s.num_seqs - c0);
        const int total = pieces.scan(c0, a.s.num_seqs, [&](int b) {
            const NewTokens n = new_tokens(a.s, b, a.num_q);
            if (n.bad && blockIdx.x == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
            return blocks_touched(n, a.shift);
        });
        // warps take (block, head) pairs
        const int64_t tasks = (int64_t)total * a.hkv;
        const int64_t all = (int64_t)gridDim.x * (kBoundThreads / 32);
        for (int64_t x = ((int64_t)blockIdx.x * (kBoundThreads / 32) + warp + all - before % all) % all; x < tasks;
             x += all) {
            const int piece = (int)(x / a.hkv), h = (int)(x - (int64_t)piece * a.hkv);
            const int i = pieces.find(piece, left);
            const NewTokens nt = new_tokens(a.s, c0 + i, a.num_q);
            const int64_t first = (int64_t)((nt.p0 >> a.shift) + (piece - pieces.first[i])) << a.shift;
            const int n = (int)min((int64_t)1 << a.shift, (int64_t)nt.p0 + nt.nq - first);  // its keys
            const int64_t row0 = phys_row(a.s, c0 + i, first);
            if (row0 < 0 || (row0 & ((1 << a.shift) - 1)) || row0 + n > a.s.num_rows || nt.p0 + (int64_t)nt.nq > nt.ctx) {
                if (lane == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
                continue;
            }
            float lo[V], hi[V], top = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) lo[e] = INFINITY, hi[e] = -INFINITY;
            const uint8_t* src = a.k + row0 * a.stride + h * (FP8 ? D : 2 * D) + 16 * li;
            for (int r0 = 0; r0 < n; r0 += 4 * R) {
                uint4 z[4];
                float f[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int r = min(r0 + u * R + sub, n - 1);  // the last key again behind the last
                    z[u] = __ldg(reinterpret_cast<const uint4*>(src + r * a.stride));
                    f[u] = FP8 ? __ldg(a.k_scale + ((row0 + r) >> a.scale_shift) * a.hkv + h) : 1.f;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t w[4] = {z[u].x, z[u].y, z[u].z, z[u].w};
                    float v[V];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (FP8) {
                            uint32_t p, q;
                            e4m3x4_to_f16(w[e], p, q);
                            const float2 x0 = __half22float2(*reinterpret_cast<__half2*>(&p));
                            const float2 x1 = __half22float2(*reinterpret_cast<__half2*>(&q));
                            v[4 * e % V] = x0.x * f[u], v[(4 * e + 1) % V] = x0.y * f[u];
                            v[(4 * e + 2) % V] = x1.x * f[u], v[(4 * e + 3) % V] = x1.y * f[u];
                        } else {
                            v[2 * e] = __uint_as_float(w[e] << 16);
                            v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float m = fabsf(v[e]);
                        top = fmaxf(top, m < INFINITY ? m : 0.f);
                        // NaN may be anything
                        lo[e] = fminf(lo[e], v[e] == v[e] ? v[e] : -INFINITY);
                        hi[e] = fmaxf(hi[e], v[e] == v[e] ? v[e] : INFINITY);
                    }
                }
            }
#pragma unroll
            for (int o = L; o < 32; o <<= 1)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
                    hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
                }
            top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
            // |v| <= 127 steps; 127 = 1.984375 2^6
            const int e2 = top > 0.f ? scale_exponent(top, 6, 0x7E0000u) : 0;
            const float up = two_to(-e2 > 127 ? 127 : -e2);
            uint32_t cl[V / 4], ch[V / 4];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                // (a product that vanishes still lies below, or above, 0)
                const float x = lo[e] * up, y = hi[e] * up;
                const int l = (int)fmaxf(-127.f, fminf(127.f, x == 0.f && lo[e] < 0.f ? -1.f : floorf(x)));
                const int g = (int)fmaxf(-127.f, fminf(127.f, y == 0.f && hi[e] > 0.f ? 1.f : ceilf(y)));
                const int sh = 8 * (e & 3);
                cl[e / 4] = (e & 3 ? cl[e / 4] : 0u) | (uint32_t)(l & 0xFF) << sh;
                ch[e / 4] = (e & 3 ? ch[e / 4] : 0u) | (uint32_t)(g & 0xFF) << sh;
            }
            const int64_t at = (row0 >> a.shift) * a.hkv + h;
            if (sub == 0) {
                uint32_t* dst = reinterpret_cast<uint32_t*>(a.bounds + at * (2 * D) + V * li);
#pragma unroll
                for (int e = 0; e < V / 4; ++e) dst[e] = cl[e], dst[D / 4 + e] = ch[e];
            }
            if (lane == 0) a.steps[at] = two_to(e2);
        }
        before += tasks;
        __syncthreads();  // the chunk's counts are no longer read
    }
}

// ---------------------------------------------------------------------------
// scores
constexpr int kScoreThreads = 256, kScoreWarps = kScoreThreads / 32;
constexpr int kScoreBlocks = 16 * kScoreWarps;  // blocks per CTA
constexpr int kScoreTiles = 32;                 // 8-row query tiles per CTA

struct ScoreArgs {
    const __nv_bfloat16* q;
    const int8_t* bounds;
    const float* steps;
    float* scores;  // [num_q][hkv][ld]
    dsa_seqs s;
    int64_t q_stride;
    int32_t* d_status;
    int32_t num_q, group, hkv, shift, ld;
    int32_t pad;     // a token's rows: a power of two of them in one tile, or 8
    int32_t npt;     // tiles per token (1 where pad < 8)
    int32_t tokens;  // per CTA
    int32_t xt;      // CTAs along the blocks
    int32_t direct;  // slot = sequence
};

template <int D>
__global__ void __launch_bounds__(kScoreThreads, 2) block_score_kernel(const __grid_constant__ ScoreArgs a) {
    constexpr int KS = D / 16;  // k-steps over lo, and over hi
    extern __shared__ __align__(16) uint4 q_sh[];  // [tile][KS / 2][lane]: two k-steps' fragments
    __shared__ Pieces<kScoreThreads> pieces;
    __shared__ int own_sh[kScoreWarps];  // the last block that a query sees
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = lane >> 2, t = lane & 3;
    const int xtile = blockIdx.x % a.xt;
    const int rest = blockIdx.x / a.xt;
    const int kvh = rest % a.hkv, slot = rest / a.hkv;
    // ---- the CTA's tokens: [t0, t0 + n) of sequence b
    int b = slot, skip = 0;
    if (!a.direct) {
        int before = 0;
        b = -1;
        for (int c0 = 0; c0 < a.s.num_seqs; c0 += Pieces<kScoreThreads>::kChunk) {
            const int total = pieces.scan(c0, a.s.num_seqs, [&](int i) {
                const Seq q = load_seq(a.s, i, a.num_q);
                if (!q.ok && blockIdx.x == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
                return q.ok ? (q.nq + a.tokens - 1) / a.tokens : 0;
            });
            if (slot < before + total) {
                const int i = pieces.find(slot - before, min(Pieces<kScoreThreads>::kChunk, a.s.num_seqs - c0));
                b = c0 + i;
                skip = (slot - before - pieces.first[i]) * a.tokens;
                break;
            }
            before += total;
            __syncthreads();
        }
        if (b < 0) return;
    }
    const Seq sq = load_seq(a.s, b, a.num_q);
    if (!sq.ok) {
        if (threadIdx.x == 0 && xtile == 0 && kvh == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
        return;
    }
    const int n = min(a.tokens, sq.nq - skip);
    if (n <= 0) return;
    const int t0 = sq.q0 + skip;
    int most = -1;
    for (int i = threadIdx.x; i < n; i += kScoreThreads) {
        const int p = __ldg(a.s.q_pos + t0 + i);
        const int o = p >= 0 && p < sq.ctx ? p >> a.shift : -1;
        most = max(most, o);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) own_sh[warp] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kScoreWarps; ++w) most = max(most, own_sh[w]);
    if (xtile * kScoreBlocks > most) return;  // no query sees these blocks

    // ---- this warp's bounds: rows col and col + 8 of its 16 blocks
    const int blk0 = xtile * kScoreBlocks + warp * 16;
    int64_t at = -1;  // the lane's block (lanes 0 .. 15)
    if (blk0 + (lane & 15) <= most) {
        const int64_t row = phys_row(a.s, b, (int64_t)(blk0 + (lane & 15)) << a.shift);
        if (row < 0 || (row & ((1 << a.shift) - 1))) {
            if (kvh == 0 && lane < 16) report(a.d_status, DSA_ERR_BAD_INPUT);
        } else {
            at = (row >> a.shift) * a.hkv + kvh;
        }
    }
    const int64_t at0 = __shfl_sync(0xffffffffu, at, col), at1 = __shfl_sync(0xffffffffu, at, col + 8);
    uint4 raw[2][D / 32];  // [row][lo's chunks, hi's]
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        raw[0][c] = raw[1][c] = make_uint4(0u, 0u, 0u, 0u);
        if (at0 >= 0) raw[0][c] = __ldg(reinterpret_cast<const uint4*>(a.bounds + at0 * (2 * D) + c * 64) + t);
        if (at1 >= 0) raw[1][c] = __ldg(reinterpret_cast<const uint4*>(a.bounds + at1 * (2 * D) + c * 64) + t);
    }
    const float step0 = at0 >= 0 ? __ldg(a.steps + at0) : 0.f, step1 = at1 >= 0 ? __ldg(a.steps + at1) : 0.f;

    // ---- the queries in whole steps, as fragments
    const int tpt = 8 / a.pad;  // tokens per tile (npt = 1)
    const int groups = (n + tpt - 1) / tpt;
    for (int gu = warp; gu < groups; gu += kScoreWarps) {
        const int tok = gu * tpt + col / a.pad;
        const bool live = tok < n;
        auto load = [&](int j, int c, uint4& x, uint4& y) {
            const int head = min(j * 8 + col % a.pad, a.group - 1);  // a group's last head again behind it
            const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(t0 + tok) * a.q_stride +
                                                              (int64_t)(kvh * a.group + head) * D + c * 64 + t * 16);
            x = live ? __ldg(src) : make_uint4(0u, 0u, 0u, 0u);
            y = live ? __ldg(src + 1) : make_uint4(0u, 0u, 0u, 0u);
        };
        float top = 0.f;
        for (int j = 0; j < a.npt; ++j)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint4 x, y;
                load(j, c, x, y);
                const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = fabsf(__uint_as_float(w[e] << 16)), v = fabsf(__uint_as_float(w[e] & 0xFFFF0000u));
                    top = fmaxf(top, fmaxf(u < INFINITY ? u : 0.f, v < INFINITY ? v : 0.f));
                }
            }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        for (int o = 1; o < a.pad; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4 * o));
        const int e2 = top > 0.f ? scale_exponent(top, 6, 0x7E0000u) : 0;
        const float up = two_to(-e2 > 127 ? 127 : -e2);
        auto whole = [&](uint32_t w) {  // two bf16 -> whole steps, f16
            float u = __uint_as_float(w << 16), v = __uint_as_float(w & 0xFFFF0000u);
            u = u == u ? fmaxf(-127.f, fminf(127.f, rintf(u * up))) : 0.f;
            v = v == v ? fmaxf(-127.f, fminf(127.f, rintf(v * up))) : 0.f;
            return pack_f16(u, v);
        };
        for (int j = 0; j < a.npt; ++j)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint4 x, y;
                load(j, c, x, y);
                uint4* dst = q_sh + ((gu * a.npt + j) * (KS / 2) + 2 * c) * 32 + lane;
                dst[0] = make_uint4(whole(x.x), whole(x.y), whole(x.z), whole(x.w));
                dst[32] = make_uint4(whole(y.x), whole(y.y), whole(y.z), whole(y.w));
            }
    }
    __syncthreads();
    if (blk0 > most) return;

    // bounds to f16 fragments: a byte + 128 under the exponent of 1024
    uint32_t lo[KS][4], hi[KS][4];
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t w[4] = {raw[r][c].x, raw[r][c].y, raw[r][c].z, raw[r][c].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t u = w[e] ^ 0x80808080u;
                uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
                const __half2 xh = __hsub2(*reinterpret_cast<__half2*>(&x), bias);
                const __half2 yh = __hsub2(*reinterpret_cast<__half2*>(&y), bias);
                auto& f = c < D / 64 ? lo : hi;
                const int k = (c % (D / 64)) * 4 + e;
                f[k][r] = *reinterpret_cast<const uint32_t*>(&xh);
                f[k][2 + r] = *reinterpret_cast<const uint32_t*>(&yh);
            }
        }
    auto mma = [](float (&d)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
    };
    auto below = [](uint32_t x) {
        const __half2 v = __hmin2(*reinterpret_cast<__half2*>(&x), __half2half2(__ushort_as_half(0)));
        return *reinterpret_cast<const uint32_t*>(&v);
    };
    auto above = [](uint32_t x) {
        const __half2 v = __hmax2(*reinterpret_cast<__half2*>(&x), __half2half2(__ushort_as_half(0)));
        return *reinterpret_cast<const uint32_t*>(&v);
    };
    for (int gu = 0; gu < groups; ++gu) {
        float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        for (int j = 0; j < a.npt; ++j) {
            float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
            const uint4* src = q_sh + (gu * a.npt + j) * (KS / 2) * 32 + lane;
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
                const uint4 z = src[(k / 2) * 32];
                mma(x, lo[k], below(z.x), below(z.y));
                mma(y, hi[k], above(z.x), above(z.y));
                mma(x, lo[k + 1], below(z.z), below(z.w));
                mma(y, hi[k + 1], above(z.z), above(z.w));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], x[e] + y[e]);
        }
        // the best of a token's heads: columns 2t, 2t + 1 of rows col and col + 8
        if (a.pad >= 2) m[0] = m[1] = fmaxf(m[0], m[1]), m[2] = m[3] = fmaxf(m[2], m[3]);
        for (int o = 2; o < a.pad; o <<= 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], o / 2));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = 2 * t + e;
            const int tok = gu * tpt + c / a.pad;
            if (c % a.pad || tok >= n) continue;
            float* dst = a.scores + ((int64_t)(t0 + tok) * a.hkv + kvh) * a.ld + blk0 + col;
            // (a step below 2^-126 / 2^22 of nothing, above 2^105 overflows to equal scores)
            if (blk0 + col < a.ld) dst[0] = m[e] * step0;
            if (blk0 + col + 8 < a.ld) dst[8] = m[2 + e] * step1;
        }
    }
}

// ---------------------------------------------------------------------------
// the best blocks of a row
constexpr int kPickThreads = 256, kBins = 1024;

struct PickArgs {
    const float* scores;
    int32_t *blocks, *len;
    dsa_seqs s;
    int32_t* d_status;
    int32_t num_q, hkv, shift, ld, nsel, first, local;
};

__global__ void __launch_bounds__(kPickThreads) block_pick_kernel(const __grid_constant__ PickArgs a) {
    extern __shared__ uint32_t key[];
    __shared__ int hist[kBins];
    __shared__ int red[kPickThreads / 32 + 1];
    __shared__ uint32_t range[2];
    __shared__ int found[2], pos_sh;
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31;
    const int t = blockIdx.x / a.hkv, kvh = blockIdx.x - t * a.hkv;
    if (tid < 32) {
        const int b = warp_seq_of(a.s.q_start, a.s.num_seqs, t);
        const Seq sq = load_seq(a.s, b, a.num_q);
        if (lane == 0) {
            int pos = __ldg(a.s.q_pos + t);
            if (t >= sq.q0 + sq.nq || t < sq.q0)
                pos = -3;  // behind the last sequence
            else if (!sq.ok || pos < -1 || pos >= sq.ctx)
                pos = -2;
            pos_sh = pos;
            range[0] = 0xFFFFFFFFu;
            range[1] = 0u;
        }
    }
    __syncthreads();
    const int pos = pos_sh;
    if (pos < -1) {  // left as it was
        if (pos == -2 && tid == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
        return;
    }
    const int n = pos < 0 ? 0 : (pos >> a.shift) + 1;
    int32_t* out = a.blocks + (int64_t)blockIdx.x * a.nsel;
    if (tid == 0)
        a.len[blockIdx.x] = n == 0 ? 0 : ((min(n, a.nsel) - 1) << a.shift) + (pos & ((1 << a.shift) - 1)) + 1;
    if (n <= a.nsel) {  // all of them
        for (int i = tid; i < a.nsel; i += kPickThreads) out[i] = i < n ? i : -1;
        return;
    }
    // [0, first) and [hi, n) for sure, `want` of [first, hi)
    const int hi = n - a.local;
    int want = a.nsel - a.first - a.local;
    const float* row = a.scores + (int64_t)blockIdx.x * a.ld;
    uint32_t least = 0xFFFFFFFFu, best = 0u;
    for (int i = a.first + tid; i < hi; i += kPickThreads) {
        const float s = row[i];
        const uint32_t u = __float_as_uint(s == 0.f ? 0.f : s);
        const uint32_t k = u & 0x80000000u ? ~u : u | 0x80000000u;
        key[i] = k;
        least = min(least, k);
        best = max(best, k);
    }
    least = __reduce_min_sync(0xffffffffu, least);
    best = __reduce_max_sync(0xffffffffu, best);
    if (lane == 0) {
        atomicMin(&range[0], least);
        atomicMax(&range[1], best);
    }
    __syncthreads();
    // the want-th largest key: bins over the range that is left, until a bin is one key or is taken whole
    uint32_t low = range[0], width = range[1] - range[0];
    uint32_t cut = 0xFFFFFFFFu;  // keys above are taken, and `ties` of those equal
    int ties = 0;
    while (want > 0) {
        const int sh = max(0, 22 - __clz(width | 1));  // width >> sh < 1024
        for (int i = tid; i < kBins; i += kPickThreads) hist[i] = 0;
        __syncthreads();
        for (int i = a.first + tid; i < hi; i += kPickThreads) {
            const uint32_t d = key[i] - low;
            if (key[i] >= low && d <= width) atomicAdd(&hist[d >> sh], 1);
        }
        __syncthreads();
        // from the top: the thread with the bin where the count passes `want`
        const int b0 = kBins - 1 - 4 * tid;
        const int h0 = hist[b0], h1 = hist[b0 - 1], h2 = hist[b0 - 2], h3 = hist[b0 - 3];
        int all;
        const int above = cta_scan<kPickThreads>(h0 + h1 + h2 + h3, red, all);
        if (above < want && above + h0 + h1 + h2 + h3 >= want) {
            int c = above, z = 0;
            if (c + h0 < want) {
                c += h0, z = 1;
                if (c + h1 < want) {
                    c += h1, z = 2;
                    if (c + h2 < want) c += h2, z = 3;
                }
            }
            found[0] = b0 - z;
            found[1] = want - c;
        }
        __syncthreads();
        const int bin = found[0], need = found[1], has = hist[bin];
        low += (uint32_t)bin << sh;
        __syncthreads();
        if (sh == 0 || (need == has && low > 0)) {
            cut = sh == 0 ? low : low - 1;
            ties = sh == 0 ? need : 0;
            break;
        }
        want = need;
        width = (1u << sh) - 1;
    }
    // in order: a run of blocks per thread
    const int per = (n + kPickThreads - 1) / kPickThreads;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    int sure = 0, equal = 0;
    for (int i = i0; i < i1; ++i) {
        if (i < a.first || i >= hi || key[i] > cut) ++sure;
        else if (key[i] == cut) ++equal;
    }
    uint32_t total;
    uint32_t* ured = reinterpret_cast<uint32_t*>(red);
    const uint32_t before = cta_scan<kPickThreads, uint32_t>((uint32_t)sure | (uint32_t)equal << 16, ured, total);
    int eq = (int)(before >> 16);
    int at = (int)(before & 0xFFFFu) + min(eq, ties);
    for (int i = i0; i < i1; ++i) {
        bool take = i < a.first || i >= hi || key[i] > cut;
        if (!take && key[i] == cut) take = eq++ < ties;
        if (take && at < a.nsel) out[at++] = i;
    }
}

}  // namespace

size_t select_ld(const dsa_seqs& s, int block) { return ((size_t)s.max_ctx + block - 1) / block; }

size_t select_workspace(const dsa_gqa_shape& sh, const dsa_seqs& s, int num_q, int block) {
    return (size_t)num_q * sh.num_kv_heads * select_ld(s, block) * 4;
}

cudaError_t launch_bounds(const dsa_gqa_shape& sh, const void* k, const float* k_scale, const dsa_seqs& s, int num_q,
                          int block, void* bounds, float* steps, int32_t* d_status, cudaStream_t stream) {
    BoundArgs a;
    a.k = static_cast<const uint8_t*>(k);
    a.k_scale = k_scale;
    a.bounds = static_cast<int8_t*>(bounds);
    a.steps = steps;
    a.s = s;
    a.stride = sh.k_stride * (sh.kv_dtype == DSA_BF16 ? 2 : 1);
    a.d_status = d_status;
    a.num_q = num_q;
    a.hkv = sh.num_kv_heads;
    a.shift = 31 - __builtin_clz((unsigned)block);
    a.scale_shift = scale_shift(sh);
    const int64_t blocks = std::min<int64_t>(num_q, (num_q >> a.shift) + 2 * (int64_t)s.num_seqs);
    const int64_t ctas = (blocks * sh.num_kv_heads + kBoundThreads / 32 - 1) / (kBoundThreads / 32);
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(ctas, kPlanSms * 6));
    auto go = [&](auto kern) { return launch_pdl(kern, dim3(grid), dim3(kBoundThreads), 0, stream, 1, a); };
    if (sh.head_dim == 64)
        return sh.kv_dtype == DSA_BF16 ? go(block_bounds_kernel<64, false>) : go(block_bounds_kernel<64, true>);
    return sh.kv_dtype == DSA_BF16 ? go(block_bounds_kernel<128, false>) : go(block_bounds_kernel<128, true>);
}

cudaError_t launch_select(const dsa_gqa_shape& sh, const void* q, const void* bounds, const float* steps,
                          const dsa_seqs& s, int num_q, int block, int nsel, int first, int local, int32_t* blocks,
                          int32_t* len, void* workspace, int32_t* d_status, cudaStream_t stream) {
    const int shift = 31 - __builtin_clz((unsigned)block);
    ScoreArgs a;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.bounds = static_cast<const int8_t*>(bounds);
    a.steps = steps;
    a.scores = static_cast<float*>(workspace);
    a.s = s;
    a.q_stride = sh.q_stride;
    a.d_status = d_status;
    a.num_q = num_q;
    a.group = sh.num_heads / sh.num_kv_heads;
    a.hkv = sh.num_kv_heads;
    a.shift = shift;
    a.ld = (int32_t)select_ld(s, block);
    a.pad = 1;
    while (a.pad < a.group && a.pad < 8) a.pad *= 2;
    a.npt = (a.group + 7) / 8;
    const int tpt = 8 / a.pad;
    a.tokens = std::min(s.max_q_per_seq, kScoreTiles / a.npt * tpt);
    a.direct = s.max_q_per_seq <= a.tokens;
    a.xt = (a.ld + kScoreBlocks - 1) / kScoreBlocks;
    const int64_t slots = a.direct ? s.num_seqs : std::min<int64_t>(num_q, num_q / a.tokens + s.num_seqs);
    const int64_t grid = slots * a.hkv * a.xt;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)((a.tokens + tpt - 1) / tpt) * a.npt * (sh.head_dim / 32) * 512;
    auto go = [&](auto d) {
        auto kern = block_score_kernel<decltype(d)::value>;
        static OncePerDevice once;
        const cudaError_t e = once.run([&] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kScoreTiles * (decltype(d)::value / 32) * 512);
        });
        return e != cudaSuccess ? e : launch_pdl(kern, dim3((unsigned)grid), dim3(kScoreThreads), smem, stream, 1, a);
    };
    cudaError_t e = sh.head_dim == 64 ? go(std::integral_constant<int, 64>()) : go(std::integral_constant<int, 128>());
    if (e != cudaSuccess) return e;
    PickArgs p;
    p.scores = a.scores;
    p.blocks = blocks;
    p.len = len;
    p.s = s;
    p.d_status = d_status;
    p.num_q = num_q;
    p.hkv = a.hkv;
    p.shift = shift;
    p.ld = a.ld;
    p.nsel = nsel;
    p.first = first;
    p.local = local;
    static OncePerDevice once;
    e = once.run([] {
        return cudaFuncSetAttribute(block_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    DSA_GQA_MAX_BLOCKS * 4);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(block_pick_kernel, dim3((unsigned)(num_q * a.hkv)), dim3(kPickThreads), (size_t)a.ld * 4, stream,
                      1, p);
}

}  // namespace gqa
}  // namespace dsa
