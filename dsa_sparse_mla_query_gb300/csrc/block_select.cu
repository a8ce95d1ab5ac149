// block_select.cu -- blocks of keys for every query and key head, chosen by a
// score from bounds of their keys (sm_103a).
//
// Per block and head the bounds lo_d <= k_d <= hi_d of its keys, in whole steps
// of a power of two s (lo rounded down, hi up, -127 .. 127), say for any query
//   q . k <= s sum_d max(q_d lo_d, q_d hi_d) = s (max(q, 0) . hi + min(q, 0) . lo).
// With q in whole steps too (-127 .. 127, one step for a token's group of heads: the
// bound is then the rounded query's, and an estimate of the query's own)
// the sums are whole numbers below 2^22: exact in fp32 in any order, in the
// tensor cores as well, so the order of the blocks depends on nothing but the
// inputs, and ties are ties.
//
// - block_bounds_kernel: minimum and maximum over the keys of the blocks that new
//   tokens touch, four warps per block and head, keys read once; and over older
//   blocks whose codes the new tokens' scale changed.
// - block_score_few_kernel: few tokens a sequence read 2 D bytes a block once:
//   HBM.  The sums on the warp-level matrix instruction, 16 blocks by 8 query
//   rows, straight from global memory (the order of the dims within a k-step is
//   the same for both operands and free otherwise, so a thread's 16 bytes make
//   whole fragments).
// - block_score_wide_kernel: a prompt's tokens, a product of [blocks] x [tokens
//   heads] on tcgen05.
// - block_pick_kernel, block_pick_row_kernel: the nsel best of a row by a
//   histogram over the keys' range (order-preserving codes) or, many rows, by
//   halving it, a warp a row.
//
// Measured, 64/8 heads of 128, blocks of 64 keys, with the host's calls and the new
// keys' bounds: 64 tokens over 32,768 keys 28.7 us, 3 over 524,288 30 us (HBM 36%
// busy while the bounds are read: two or three rounds of loads a warp, then the
// choice); 2,048 of 65,536 138 us: the scores 96 (the CTA's own warps turn the
// bounds into f16 operands: the tensor cores are 33% busy), the choice 39 (69% of
// the issue slots), the bounds 5.
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
    int32_t num_q, hkv, shift, scale_shift, page_shift;
};

// two packed values: f16 (e4m3 codes, converted), or bf16
template <bool FP8>
__device__ __forceinline__ uint32_t packed_min(uint32_t x, uint32_t y) {  // NaN if either is
    if (FP8) {
        const __half2 r = __hmin2_nan(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<__nv_bfloat162*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <bool FP8>
__device__ __forceinline__ uint32_t packed_max(uint32_t x, uint32_t y) {
    if (FP8) {
        const __half2 r = __hmax2_nan(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<__nv_bfloat162*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <bool FP8>
__device__ __forceinline__ float2 packed_floats(uint32_t x) {
    if (FP8) return __half22float2(*reinterpret_cast<__half2*>(&x));
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}

// One over the step of values up to `top`, and the step
__device__ __forceinline__ float step_up(float top, float& step) {
    const int e = top > 0.f ? scale_exponent(top, 6, 0x7E0000u) : 0;  // 127 = 1.984375 2^6
    step = two_to(e);
    return two_to(-e);
}
// bounds in whole steps (a product that vanishes still lies below, or above, 0)
__device__ __forceinline__ uint32_t low_code(float v, float up) {
    const float x = v * up;
    return (uint32_t)(int)fmaxf(-127.f, fminf(127.f, x == 0.f && v < 0.f ? -1.f : floorf(x))) & 0xFFu;
}
__device__ __forceinline__ uint32_t high_code(float v, float up) {
    const float x = v * up;
    return (uint32_t)(int)fmaxf(-127.f, fminf(127.f, x == 0.f && v > 0.f ? 1.f : ceilf(x))) & 0xFFu;
}

// May a sequence's new tokens (from position p0) have raised the scale of the scale block that p0
// lies in, so that its older tokens' codes are others than before?  A scale grows by a power of two
// to the least one that holds the new tokens: afterwards one of their codes is 224 or more, and every
// older one 224 or less.  (Where that holds and nothing grew, the older blocks get the bounds that they
// have.)  A warp, over the codes of one head: src its row of the scale block's first token, `older`
// of its `all` rows before p0.
template <int D>
__device__ __forceinline__ bool scale_raised(const uint8_t* src, int64_t stride, int older, int all) {
    constexpr int kLanes = D / 16, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31;
    uint32_t held = 0, fresh = 0;  // largest magnitudes of older and of new codes
    for (int r = lane / kLanes; r < all; r += kRows) {
        const uint4 z = __ldg(reinterpret_cast<const uint4*>(src + r * stride) + lane % kLanes);
        const uint32_t w[4] = {z.x, z.y, z.z, z.w};
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t x = w[e] & 0x7F7F7F7Fu;
            m = __vmaxu4(m, x & ~__vcmpeq4(x, 0x7F7F7F7Fu));  // NaN has no say
        }
        held = __vmaxu4(held, r < older ? m : 0u);
        fresh = __vmaxu4(fresh, r < older ? 0u : m);
    }
    auto most = [](uint32_t y) {
        const uint32_t x = __vmaxu2(y & 0x00FF00FFu, (y >> 8) & 0x00FF00FFu);
        return __reduce_max_sync(0xffffffffu, max(x & 0xFFu, x >> 16));
    };
    constexpr uint32_t k224 = 0x76;  // 1.75 2^7
    return most(held) <= k224 && most(fresh) >= k224;
}

// Four warps take a block and head, its rows among them: minima and maxima as
// they lie in the cache (pairs of f16 or bf16: exact), converted at the end.
// Rows with scales of their own, negative scales and blocks with values that are
// not finite take the long way in fp32, by one warp.
template <int D, bool FP8>
__global__ void __launch_bounds__(kBoundThreads) block_bounds_kernel(const __grid_constant__ BoundArgs a) {
    constexpr int V = FP8 ? 16 : 8;    // dims per lane
    constexpr int L = D / V;           // lanes per row
    constexpr int R = 32 / L;          // rows per access
    constexpr int P = V / 2;           // pairs per lane
    constexpr int kChunk = Pieces<kBoundThreads>::kChunk;
    constexpr int kParts = 4, kHeads = kBoundThreads / 32 / kParts;
    __shared__ Pieces<kBoundThreads> pieces;
    __shared__ int4 seq_sh[kChunk];    // first position, tokens, context
    __shared__ uint32_t ends[kHeads][kParts][2][D / 2];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = warp % kParts, slot = warp / kParts;
    const int li = lane % L, sub = lane / L;
    const int big = max(a.shift, a.scale_shift);
    int64_t before = 0;
    for (int c0 = 0; c0 < a.s.num_seqs; c0 += kChunk) {
        const int left = min(kChunk, a.s.num_seqs - c0);
        const int total = pieces.scan(c0, a.s.num_seqs, [&](int b) {
            const NewTokens n = new_tokens(a.s, b, a.num_q);
            if (n.bad && blockIdx.x == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
            // scale blocks of more than a block: from the first new token's scale block on
            const int start = n.nq ? n.p0 >> big << (big - a.shift) : 0;
            seq_sh[b - c0] = make_int4(n.p0, n.nq, n.ctx, start);
            return n.nq ? blocks_touched(n, a.shift) + (n.p0 >> a.shift) - start : 0;
        });
        // CTAs take kHeads heads of a block at a time
        const int per = (a.hkv + kHeads - 1) / kHeads;
        const int64_t tasks = (int64_t)total * per;
        for (int64_t x = (int64_t)((gridDim.x + blockIdx.x - before % gridDim.x) % gridDim.x); x < tasks; x += gridDim.x) {
            const int piece = (int)((uint64_t)x >> 32 ? x / per : (uint32_t)x / (uint32_t)per);
            const int h = (int)(x - (int64_t)piece * per) * kHeads + slot;
            const int i = pieces.find(piece, left);
            const int4 nt = seq_sh[i];
            const int64_t first = (int64_t)(nt.w + (piece - pieces.first[i])) << a.shift;
            const int n = (int)min((int64_t)1 << a.shift, (int64_t)nt.x + nt.y - first);  // its keys
            const int64_t row0 = row_at(a.s, a.page_shift, c0 + i, first);
            // a block of older tokens alone (what is wrong with the sequence is reported with the others)
            const bool older = FP8 && first + n <= nt.x;
            const int64_t big0 = older ? first & -((int64_t)1 << big) : 0;  // its scale block's first token
            const int64_t big_row = row0 - (first - big0);
            if (older && (row0 < 0 || (big_row & ((1 << big) - 1)) || row0 + n > a.s.num_rows || nt.x + (int64_t)nt.y > nt.z))
                continue;
            if (row0 < 0 || (row0 & ((1 << a.shift) - 1)) || row0 + n > a.s.num_rows || nt.x + (int64_t)nt.y > nt.z) {
                if (threadIdx.x == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
                continue;
            }
            bool live = h < a.hkv;
            const uint8_t* src = a.k + row0 * a.stride + (int64_t)(live ? h : 0) * (FP8 ? D : 2 * D) + 16 * li;
            if (FP8 && older && live && part == 0)  // (the warp that writes)
                live = scale_raised<D>(a.k + big_row * a.stride + (int64_t)h * D, a.stride, (int)(nt.x - big0),
                                       (int)min((int64_t)1 << big, min((int64_t)nt.x + nt.y - big0, a.s.num_rows - big_row)));
            const int64_t at = (row0 >> a.shift) * a.hkv + h;
            const bool even = !FP8 || a.scale_shift >= a.shift;  // one scale for the block
            float scale = 1.f;
            bool odd = !even;
            if (even) {
                if (FP8 && live && part == 0) scale = __ldg(a.k_scale + (row0 >> a.scale_shift) * a.hkv + h);
                uint32_t lo[P], hi[P];
                // this warp's rows: every fourth access of R rows, the last key again behind the last
#pragma unroll
                for (int d = 0; d < P; ++d) lo[d] = hi[d] = 0;
                for (int r0 = part * R; r0 == part * R || r0 < n; r0 += 4 * kParts * R) {
                    uint4 z[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        z[u] = __ldg(reinterpret_cast<const uint4*>(src + min(r0 + u * kParts * R + sub, n - 1) * a.stride));
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t w[4] = {z[u].x, z[u].y, z[u].z, z[u].w};
                        const bool start = u == 0 && r0 == part * R;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t p[2] = {w[e], 0u};
                            if (FP8) e4m3x4_to_f16(w[e], p[0], p[1]);
#pragma unroll
                            for (int y = 0; y < P / 4; ++y) {
                                const int d = e * (P / 4) + y;
                                lo[d] = start ? p[y] : packed_min<FP8>(lo[d], p[y]);
                                hi[d] = start ? p[y] : packed_max<FP8>(hi[d], p[y]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int o = L; o < 32; o <<= 1)
#pragma unroll
                    for (int d = 0; d < P; ++d) {
                        lo[d] = packed_min<FP8>(lo[d], __shfl_xor_sync(0xffffffffu, lo[d], o));
                        hi[d] = packed_max<FP8>(hi[d], __shfl_xor_sync(0xffffffffu, hi[d], o));
                    }
                if (sub == 0)
#pragma unroll
                    for (int d = 0; d < P; ++d) ends[slot][part][0][li * P + d] = lo[d], ends[slot][part][1][li * P + d] = hi[d];
                __syncthreads();
                if (part == 0 && live) {
                    // D / 64 pairs of dims a lane
                    float top = 0.f;
                    odd = !(scale >= 0.f);  // (turned around by a negative one)
                    float2 l[D / 64], g[D / 64];
#pragma unroll
                    for (int y = 0; y < D / 64; ++y) {
                        const int d = lane * (D / 64) + y;
                        uint32_t x0 = ends[slot][0][0][d], x1 = ends[slot][0][1][d];
#pragma unroll
                        for (int z = 1; z < kParts; ++z) {
                            x0 = packed_min<FP8>(x0, ends[slot][z][0][d]);
                            x1 = packed_max<FP8>(x1, ends[slot][z][1][d]);
                        }
                        l[y] = packed_floats<FP8>(x0), g[y] = packed_floats<FP8>(x1);
                        l[y].x *= scale, l[y].y *= scale, g[y].x *= scale, g[y].y *= scale;
                        const float m = fmaxf(fmaxf(fabsf(l[y].x), fabsf(l[y].y)), fmaxf(fabsf(g[y].x), fabsf(g[y].y)));
                        // (fmaxf leaves NaN out)
                        odd = odd || !(m < INFINITY) || l[y].x != l[y].x || l[y].y != l[y].y || g[y].x != g[y].x || g[y].y != g[y].y;
                        top = fmaxf(top, m);
                    }
                    odd = __any_sync(0xffffffffu, odd);
                    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
                    if (!odd) {
                        float step;
                        const float up = step_up(top, step);
                        uint32_t cl = 0, ch = 0;
#pragma unroll
                        for (int y = 0; y < D / 64; ++y) {
                            cl |= (low_code(l[y].x, up) | low_code(l[y].y, up) << 8) << (16 * y);
                            ch |= (high_code(g[y].x, up) | high_code(g[y].y, up) << 8) << (16 * y);
                        }
                        int8_t* dst = a.bounds + at * (2 * D) + lane * (D / 32);
                        if (D == 128) {
                            *reinterpret_cast<uint32_t*>(dst) = cl;
                            *reinterpret_cast<uint32_t*>(dst + D) = ch;
                        } else {
                            *reinterpret_cast<uint16_t*>(dst) = (uint16_t)cl;
                            *reinterpret_cast<uint16_t*>(dst + D) = (uint16_t)ch;
                        }
                        if (lane == 0) a.steps[at] = step;
                    }
                }
                __syncthreads();  // the halves' ends are no longer read
            }
            if (!odd || part != 0 || !live) continue;
            float lo[V], hi[V], top = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) lo[e] = INFINITY, hi[e] = -INFINITY;
            for (int r0 = 0; r0 < n; r0 += 2 * R) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int r = min(r0 + u * R + sub, n - 1);
                    const uint4 z = __ldg(reinterpret_cast<const uint4*>(src + r * a.stride));
                    const float f = FP8 ? __ldg(a.k_scale + ((row0 + r) >> a.scale_shift) * a.hkv + h) : 1.f;
                    const uint32_t w[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t p[2] = {w[e], 0u};
                        if (FP8) e4m3x4_to_f16(w[e], p[0], p[1]);
#pragma unroll
                        for (int y = 0; y < P / 4; ++y) {
                            const float2 v2 = packed_floats<FP8>(p[y]);
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int d = (e * (P / 4) + y) * 2 + c;
                                const float v = (c ? v2.y : v2.x) * f, m = fabsf(v);
                                top = fmaxf(top, m < INFINITY ? m : 0.f);
                                // NaN may be anything
                                lo[d] = fminf(lo[d], v == v ? v : -INFINITY);
                                hi[d] = fmaxf(hi[d], v == v ? v : INFINITY);
                            }
                        }
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
            float step;
            const float up = step_up(top, step);
            if (sub == 0) {
                uint32_t* dst = reinterpret_cast<uint32_t*>(a.bounds + at * (2 * D) + V * li);
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    dst[e / 4] = low_code(lo[e], up) | low_code(lo[e + 1], up) << 8 | low_code(lo[e + 2], up) << 16 |
                                 low_code(lo[e + 3], up) << 24;
                    dst[D / 4 + e / 4] = high_code(hi[e], up) | high_code(hi[e + 1], up) << 8 |
                                         high_code(hi[e + 2], up) << 16 | high_code(hi[e + 3], up) << 24;
                }
            }
            if (lane == 0) a.steps[at] = step;
        }
        before += tasks;
        __syncthreads();  // the chunk's counts are no longer read
    }
}

// ---------------------------------------------------------------------------
// the choice among a row's scores
constexpr int kBins = 1024;

struct PickArgs {
    const float* scores;
    int32_t *blocks, *len;
    dsa_seqs s;
    int32_t* d_status;
    int32_t num_q, hkv, shift, ld, nsel, first, local;
};

// keys that a query at `pos` sees in its m blocks (the last one its own)
__device__ __forceinline__ int seen_keys(int pos, int m, int shift) {
    return pos < 0 ? 0 : ((m - 1) << shift) + (pos & ((1 << shift) - 1)) + 1;
}

// what a CTA needs to choose among a row's keys
template <int T>
struct PickShared {
    static constexpr int W = T / 32;
    int hist[kBins];
    int red[W + 1];
    uint32_t ends[2][W], names[T], codes[T];
    int2 sums[W];
    int found[2], count;
};
// an order-preserving code of a score, 1 at least and infinity's at most (NaN, of a step that was never
// written: last)
__device__ __forceinline__ uint32_t score_code(float s) {
    const uint32_t u = __float_as_uint(s + 0.f);  // (-0 as 0)
    return s != s ? 1u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Of the n blocks of a row those in [0, first) and [hi, n), and the `want` with
// the largest keys in [first, hi): into `out`, ascending.  A CTA; sh.ends holds
// the warps' least and largest keys, sh.hist zeros, sh.count 0, a barrier behind
// them.  nsel = the number taken.
template <int T>
__device__ __forceinline__ void pick(PickShared<T>& sh, uint32_t* key, int n, int first, int hi, int want, int nsel,
                                     int32_t* out) {
    constexpr int W = T / 32, kPer = kBins / T;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t least = 0xFFFFFFFFu, best = 0u;
#pragma unroll
    for (int w = 0; w < W; ++w) least = min(least, sh.ends[0][w]), best = max(best, sh.ends[1][w]);
    // The want-th largest key: bins over the range that is left, until a bin is taken whole, holds few
    // enough keys to rank each against the others, or is one key.
    uint32_t low = least, width = best - least;
    uint32_t cut = 0xFFFFFFFFu;  // keys above are taken, and the first `ties` of those equal
    int ties = 0;
    while (want > 0) {
        const int bits = max(0, 22 - __clz(width | 1));  // width >> bits < kBins
        for (int i = first + tid; i < hi; i += T) {
            const uint32_t k = key[i];
            if (k >= low && k - low <= width) atomicAdd(&sh.hist[(k - low) >> bits], 1);
        }
        __syncthreads();
        // from the top: the thread with the bin where the count passes `want`
        int h[kPer], mine = 0;
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            h[y] = tid < kBins / kPer ? sh.hist[kBins - 1 - kPer * tid - y] : 0;
            mine += h[y];
        }
        int all;
        int c = cta_scan<T>(mine, sh.red, all);
        if (c < want && c + mine >= want) {
#pragma unroll
            for (int y = 0; y < kPer; ++y) {
                if (c < want && c + h[y] >= want) {
                    sh.found[0] = kBins - 1 - kPer * tid - y;
                    sh.found[1] = want - c;
                }
                c += h[y];
            }
        }
        __syncthreads();
        const int bin = sh.found[0], need = sh.found[1], has = sh.hist[bin];
        low += (uint32_t)bin << bits;
        width = (1u << bits) - 1;
        if (need == has && low > 0) {
            cut = low - 1;
            break;
        }
        if (has <= T) {
            for (int i = first + tid; i < hi; i += T) {
                const uint32_t k = key[i];
                if (k >= low && k - low <= width) {
                    const int at = atomicAdd(&sh.count, 1);
                    sh.names[at] = i;
                    sh.codes[at] = k;
                }
            }
            __syncthreads();
            if (tid < has) {
                const uint32_t k = sh.codes[tid], me = sh.names[tid];
                int rank = 0;
                for (int y = 0; y < has; ++y) rank += sh.codes[y] > k || (sh.codes[y] == k && sh.names[y] < me);
                if (rank < need) key[me] = 0xFFFFFFFFu;  // above any score's code
            }
            cut = low + width;
            __syncthreads();
            break;
        }
        if (bits == 0) {
            cut = low;
            ties = need;
            break;
        }
        want = need;
        __syncthreads();
        for (int i = tid; i < kBins; i += T) sh.hist[i] = 0;
        __syncthreads();
    }
    // in order: a run of blocks per warp, counted, then written
    const int run = (n + T - 1) / T * 32, i0 = min(n, warp * run), i1 = min(n, i0 + run);
    int sure = 0, equal = 0;
    for (int i = i0 + lane; i < i1 + lane; i += 32) {
        const bool in = i < i1, fix = i < first || i >= hi;
        sure += __popc(__ballot_sync(0xffffffffu, in && (fix || key[i] > cut)));
        if (ties) equal += __popc(__ballot_sync(0xffffffffu, in && !fix && key[i] == cut));
    }
    if (lane == 0) sh.sums[warp] = make_int2(sure, equal);
    __syncthreads();
    int at = 0, eq = 0;
    for (int w = 0; w < warp; ++w) at += sh.sums[w].x, eq += sh.sums[w].y;
    const uint32_t under = (1u << lane) - 1;
    for (int i = i0 + lane; i < i1 + lane; i += 32) {
        const bool in = i < i1, fix = i < first || i >= hi;
        const bool yes = in && (fix || key[i] > cut), tie = in && !fix && ties && key[i] == cut;
        const uint32_t y = __ballot_sync(0xffffffffu, yes), e = __ballot_sync(0xffffffffu, tie);
        const int rank = eq + __popc(e & under);
        const int place = at + __popc(y & under) + min(rank, ties);
        if ((yes || (tie && rank < ties)) && place < nsel) out[place] = i;
        at += __popc(y);
        eq += __popc(e);
    }
}

// ---------------------------------------------------------------------------
// scores
struct ScoreArgs {
    const __nv_bfloat16* q;
    const int8_t* bounds;
    const float* steps;
    float* scores;  // [num_q][hkv][ld]
    dsa_seqs s;
    int64_t q_stride;
    int32_t* d_status;
    int32_t num_q, group, hkv, shift, ld, page_shift;
    int32_t pad;     // a token's rows, a power of two of them (up to 8 in the 8-row tiles of few rows)
    int32_t npt;     // tiles per token there (1 where pad < 8)
    int32_t tokens;  // per CTA
    int32_t xt;      // CTAs that share the blocks
    int32_t items, tiles;  // many rows: (sequence's tokens, key head)s, and tiles of blocks of the longest context
    int32_t direct;  // slot = sequence
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}
// four signed bytes as f16: a byte + 128 under the exponent of 1024, less 1152
__device__ __forceinline__ void bytes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));
    const __half2 xh = __hsub2(*reinterpret_cast<__half2*>(&x), bias);
    const __half2 yh = __hsub2(*reinterpret_cast<__half2*>(&y), bias);
    lo = *reinterpret_cast<const uint32_t*>(&xh);
    hi = *reinterpret_cast<const uint32_t*>(&yh);
}

// Scores are kept 2^15 times smaller: a sum (below 2^21) times a step, 2^-126 to 2^122, is then a
// multiple of 2^-141 below 2^128, exact in fp32 at either end (subnormal at the lower one).
constexpr float kStepDown = 0x1p-15f;

__device__ __forceinline__ float whole_steps(float v, float up) {
    return v == v ? fmaxf(-127.f, fminf(127.f, rintf(v * up))) : 0.f;
}

// A few query rows a sequence (up to 4 tiles): a CTA of four warps takes a
// (sequence, key head), or a share of its blocks.  Every warp keeps two tiles of
// 16 blocks on their way, and the pages of two more; a thread's 16 bytes of a
// block become fragments of whole k-steps as they meet the products (f16:
// as 8-bit integers, which need no conversion and half as many products, 3 x 8,192
// blocks of 8 heads took 39 us, 30 so).  Where
// (sequence, key head)s alone fill the GPU (PICK) their scores stay in shared
// memory, and the CTA chooses among them: no second launch.
constexpr int kFewThreads = 128, kFewWarps = kFewThreads / 32, kFewTiles = 4;
constexpr int kFewScores = 6144;  // of a CTA's tokens, in shared memory

template <int D, int NT, bool PICK>
__global__ void __launch_bounds__(kFewThreads, PICK ? 4 : 5)
    block_score_few_kernel(const __grid_constant__ ScoreArgs a, const __grid_constant__ PickArgs k) {
    extern __shared__ uint32_t keys[];  // PICK: [token][ld]
    __shared__ __align__(16) uint4 q_sh[NT * (D / 32) * 64];  // [tile][lo, hi][D / 64][2][lane]: two k-steps each
    __shared__ uint32_t top_sh[8 * kFewTiles];                    // largest of a token's queries
    __shared__ int pos_sh[8 * kFewTiles];
    __shared__ PickShared<kFewThreads> pick_sh;
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col = lane >> 2, t = lane & 3;
    const int kvh = blockIdx.x % a.hkv, rest = blockIdx.x / a.hkv;
    const int share = rest % a.xt, b = rest / a.xt;
    if (tid < 8 * kFewTiles) top_sh[tid] = 0;
    const Seq sq = load_seq(a.s, b, a.num_q);
    if (!sq.ok) {
        if (tid == 0 && share == 0 && kvh == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
        return;
    }
    const int n = sq.nq;
    if (n == 0) return;
    // places of tile i's blocks (lanes 0 .. 15) among the cache's, by the context; those that no query
    // sees may lie anywhere
    const int64_t base = first_row(a.s, b);
    auto page_of = [&](int i) {
        const int64_t tok = (int64_t)(i * 16 + (lane & 15)) << a.shift;
        return tok < sq.ctx ? page_at(a.s, a.page_shift, b, tok) : 0;
    };
    auto place = [&](int i, int page) -> int {
        const int64_t tok = (int64_t)(i * 16 + (lane & 15)) << a.shift;
        if (tok >= sq.ctx) return -1;
        const int64_t row = row_in(a.s, a.page_shift, page, base, tok);
        return row < 0 || (row & ((1 << a.shift) - 1)) ? -2 : (int)(row >> a.shift);
    };
    struct Tile {
        uint4 x[2][D / 32];
        float step[2];
    };
    const int8_t* bounds = a.bounds + (int64_t)kvh * (2 * D) + 16 * t;
    auto fetch = [&](int at, Tile& z) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int p = __shfl_sync(0xffffffffu, at, col + 8 * r);
            const uint4* src = reinterpret_cast<const uint4*>(bounds + (int64_t)max(p, 0) * (a.hkv * 2 * D));
#pragma unroll
            for (int c = 0; c < D / 32; ++c) z.x[r][c] = p >= 0 ? __ldg(src + 4 * c) : make_uint4(0u, 0u, 0u, 0u);
            z.step[r] = p >= 0 ? __ldg(a.steps + (int64_t)p * a.hkv + kvh) : 0.f;
        }
    };
    const int stride = a.xt * kFewWarps;
    int i = share * kFewWarps + warp;
    int page = page_of(i), then_page = page_of(i + stride);
    if (tid < n) pos_sh[tid] = __ldg(a.s.q_pos + sq.q0 + tid);
    // ---- the queries in whole steps: a thread's 16 dims of a row, twice for more than two tiles
    constexpr int kSets = (NT * 8 * (D / 16) + kFewThreads - 1) / kFewThreads;
    const int tpt = 8 >> (31 - __clz(a.pad));
    uint4 raw[kSets][2];
#pragma unroll
    for (int y = 0; y < kSets; ++y) {
        const int x = y * kFewThreads + tid, row = x / (D / 16), c = x % (D / 16);
        const int j = row >> 3, cl = row & 7;
        const int tok = a.npt > 1 ? j / a.npt : j * tpt + cl / a.pad;
        const int head = min(a.npt > 1 ? j % a.npt * 8 + cl : cl % a.pad, a.group - 1);  // the last again behind it
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(sq.q0 + tok) * a.q_stride +
                                                          (int64_t)(kvh * a.group + head) * D + 16 * c);
        raw[y][0] = raw[y][1] = make_uint4(0u, 0u, 0u, 0u);
        if (j < NT && tok < n) raw[y][0] = __ldg(src), raw[y][1] = __ldg(src + 1);
    }
    Tile cur;
    int at = place(i, page);
    fetch(at, cur);
    page = then_page;
    then_page = page_of(i + 2 * stride);
    __syncthreads();
    auto token = [&](int y) {
        const int row = (y * kFewThreads + tid) / (D / 16);
        return a.npt > 1 ? (row >> 3) / a.npt : (row >> 3) * tpt + (row & 7) / a.pad;
    };
#pragma unroll
    for (int y = 0; y < kSets; ++y) {
        const uint32_t w[8] = {raw[y][0].x, raw[y][0].y, raw[y][0].z, raw[y][0].w,
                               raw[y][1].x, raw[y][1].y, raw[y][1].z, raw[y][1].w};
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = fabsf(__uint_as_float(w[e] << 16)), v = fabsf(__uint_as_float(w[e] & 0xFFFF0000u));
            top = fmaxf(top, fmaxf(u < INFINITY ? u : 0.f, v < INFINITY ? v : 0.f));
        }
        if (top > 0.f) atomicMax(&top_sh[token(y)], __float_as_uint(top));
    }
    int most = -1;
    for (int y = 0; y < n; ++y) {
        const int p = pos_sh[y];
        if (p >= 0 && p < sq.ctx) most = max(most, p >> a.shift);
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < kSets; ++y) {
        const int x = y * kFewThreads + tid, row = x / (D / 16), c = x % (D / 16);
        if (row >= NT * 8) break;
        const float top = __uint_as_float(top_sh[min(token(y), 8 * kFewTiles - 1)]);
        float step;
        const float up = step_up(top, step);
        const uint32_t w[8] = {raw[y][0].x, raw[y][0].y, raw[y][0].z, raw[y][0].w,
                               raw[y][1].x, raw[y][1].y, raw[y][1].z, raw[y][1].w};
        // dims 16 c ..: chunk c / 4, thread c % 4 of the row's four
        uint4* dst = q_sh + ((row >> 3) * (D / 32) + c / 4) * 64 + (row & 7) * 4 + c % 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t z = w[4 * h + e];
                const float u = whole_steps(__uint_as_float(z << 16), up), v = whole_steps(__uint_as_float(z & 0xFFFF0000u), up);
                lo[e] = pack_f16(fminf(u, 0.f), fminf(v, 0.f));
                hi[e] = pack_f16(fmaxf(u, 0.f), fmaxf(v, 0.f));
            }
            dst[32 * h] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            dst[(D / 64) * 64 + 32 * h] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        }
    }
    __syncthreads();
    const int groups = (n + tpt - 1) / tpt;
    const uint4* qf = q_sh + lane;
    // (divisions take longer than a tile's products: out of the loop)
    const int sh = 31 - __clz(a.pad);
    bool leads[NT];   // a token's first tile
    int group_of[NT], put[2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        group_of[j] = j / a.npt;
        leads[j] = group_of[j] * a.npt == j && group_of[j] < groups;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) put[e] = (2 * t + e) & (a.pad - 1) ? -1 : (2 * t + e) >> sh;  // token of the group
    bool lost = false;
    for (; i * 16 <= most; i += stride) {
        lost = lost || (at == -2 && i * 16 + (lane & 15) <= most);
        Tile then;
        at = place(i + stride, page);
        fetch(at, then);
        page = then_page;
        then_page = page_of(i + 3 * stride);
        float acc[NT][4], odd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {  // lo's chunks, hi's
            const uint4 r0 = cur.x[0][c], r1 = cur.x[1][c];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t f[2][4];
                bytes_to_f16(h ? r0.z : r0.x, f[0][0], f[0][2]);
                bytes_to_f16(h ? r1.z : r1.x, f[0][1], f[0][3]);
                bytes_to_f16(h ? r0.w : r0.y, f[1][0], f[1][2]);
                bytes_to_f16(h ? r1.w : r1.y, f[1][1], f[1][3]);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 z = qf[(j * (D / 32) + c) * 64 + 32 * h];
                    mma_f16(acc[j], f[0], z.x, z.y);
                    mma_f16(NT == 1 ? odd : acc[j], f[1], z.z, z.w);
                }
            }
        }
        if (NT == 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[0][e] += odd[e];
        // the best of a token's heads, and its scores of blocks blk and blk + 8
        const int blk = i * 16 + col;
        const float step0 = kStepDown * cur.step[0], step1 = kStepDown * cur.step[1];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (!leads[j]) continue;
            float m[4] = {acc[j][0], acc[j][1], acc[j][2], acc[j][3]};
#pragma unroll
            for (int z = j + 1; z < NT; ++z)
                if (z < j + a.npt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], acc[z][e]);
            if (a.pad >= 2) m[0] = m[1] = fmaxf(m[0], m[1]), m[2] = m[3] = fmaxf(m[2], m[3]);
            for (int o = 2; o < a.pad; o <<= 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], o / 2));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = group_of[j] * tpt + put[e];
                if (put[e] < 0 || tok >= n) continue;
                const float s0 = m[e] * step0, s1 = m[2 + e] * step1;
                if (PICK) {
                    if (blk <= most) keys[tok * a.ld + blk] = score_code(s0);
                    if (blk + 8 <= most) keys[tok * a.ld + blk + 8] = score_code(s1);
                } else {
                    float* dst = a.scores + ((int64_t)(sq.q0 + tok) * a.hkv + kvh) * a.ld + blk;
                    if (blk < a.ld) dst[0] = s0;
                    if (blk + 8 < a.ld) dst[8] = s1;
                }
            }
        }
        cur = then;
    }
    if (lost && kvh == 0 && lane < 16) report(a.d_status, DSA_ERR_BAD_INPUT);
    if (!PICK) return;
    __syncthreads();
    for (int tok = 0; tok < n; ++tok) {
        const int pos = pos_sh[tok];
        if (pos < -1 || pos >= sq.ctx) {  // left as it was
            if (tid == 0 && kvh == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
            continue;
        }
        const int64_t row = (int64_t)(sq.q0 + tok) * a.hkv + kvh;
        const int m = pos < 0 ? 0 : (pos >> a.shift) + 1;
        int32_t* out = k.blocks + row * k.nsel;
        if (tid == 0) k.len[row] = seen_keys(pos, min(m, k.nsel), a.shift);
        if (m <= k.nsel) {
            for (int x = tid; x < k.nsel; x += kFewThreads) out[x] = x < m ? x : -1;
            continue;
        }
        uint32_t* key = keys + tok * a.ld;
        const int hi = m - k.local;
        uint32_t least = 0xFFFFFFFFu, best = 0u;
        for (int x = k.first + tid; x < hi; x += kFewThreads) {
            least = min(least, key[x]);
            best = max(best, key[x]);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        best = __reduce_max_sync(0xffffffffu, best);
        __syncthreads();  // the last token's choice is made
        if (lane == 0) pick_sh.ends[0][warp] = least, pick_sh.ends[1][warp] = best;
        for (int x = tid; x < kBins; x += kFewThreads) pick_sh.hist[x] = 0;
        if (tid == 0) pick_sh.count = 0;
        __syncthreads();
        pick<kFewThreads>(pick_sh, key, m, k.first, hi, k.nsel - k.first - k.local, k.nsel, out);
    }
}

// Many query rows a sequence: [128 blocks] x [256 (token, head) columns] on the
// tensor cores, K = 2 D: min(q, 0) beside lo, max(q, 0) beside hi, whole numbers
// in f16 (sums below 2^22: exact).  Blocks are the rows, so that a token's heads
// are columns, and their maximum one thread's, and a warp stores 32 neighbouring
// scores of a token.  An item is a head of up to 256 / pad tokens, and its tiles of
// blocks behind a start that takes some three tiles' time (15,000 cycles, the last
// maxima among them, a tile 4,500): its columns are laid out in shared memory (a
// warp owns a token, so its step is a warp's maximum).  A CTA an SM has an even
// share of all items' tiles and starts, in a row.
// Eight warps turn the bounds into f16, 64 dims at a time, ahead of the products,
// which one thread issues, and eight warps take the maxima of the last tile out
// of TMEM.  The bounds on their way are asynchronous copies, each lane's its own:
// loads into registers are waited for by the fence behind every chunk (1,250
// cycles a chunk, 640 so).  As an operand in TMEM they bound the products at some
// 150 cycles each, whatever their columns, and leave no second accumulator.
constexpr int kWideCols = 256, kWideHalf = 128, kWideRows = 128;  // a warp's maxima: half of the columns
constexpr int kWideRing = 3, kWideStart = 3;
constexpr int kWideLay = 512, kWideThreads = kWideLay + 32;
constexpr int kTagSelect = 8;

template <int D>
struct Wide {
    static constexpr int kChunks = D / 32;              // of 64 dims: lo's, then hi's
    static constexpr int kB = kChunks * kWideCols * 128, kA = kWideRing * kWideRows * 128;
    static constexpr int kStage = kWideRows * 2 * D;    // bounds of the next tile
    static constexpr int kSmem = kB + kA + kStage + 1024 + 64 + 256;
};

template <int D>
__global__ void __launch_bounds__(kWideThreads, 1) block_score_wide_kernel(const __grid_constant__ ScoreArgs a) {
    using C = Wide<D>;
    extern __shared__ uint8_t wide_sh[];
    uint8_t* bsh = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(wide_sh) + 1023) & ~(uintptr_t)1023);
    uint8_t* ash = bsh + C::kB;
    uint8_t* stage = ash + C::kA;
    int* most_sh = reinterpret_cast<int*>(stage + C::kStage);  // [warps] last block that a token sees
    uint64_t* afull = reinterpret_cast<uint64_t*>(most_sh + 16);
    uint64_t *aempty = afull + kWideRing, *tfull = aempty + kWideRing, *tempty = tfull + 2;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tempty + 2);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 3);
    __shared__ Pieces<kWideThreads> pieces;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < kWideRing; ++i) {
            ptx::mbar_init(afull + i, 8);
            ptx::mbar_init(aempty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(tfull + i, 1);
            ptx::mbar_init(tempty + i, 8);
        }
        abort_flag[0] = 0;
        abort_flag[1] = kTagSelect;
        ptx::fence_mbar_init();
    }
    if (warp == kWideLay / 32) {
        ptx::tmem_alloc(tmem_slot, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_enter();
    // every malformed sequence is reported, whatever rows it has: a share per CTA, by the products' warp, which
    // waits for the columns anyway
    if (warp == kWideLay / 32)
        for (int64_t i = (int64_t)blockIdx.x * 32 + lane; i < a.s.num_seqs; i += gridDim.x * 32)
            if (!load_seq(a.s, (int)i, a.num_q).ok) report(a.d_status, DSA_ERR_BAD_INPUT);

    bool ok = true;
    int tile = 0;            // tiles so far
    Cursor<kWideRing> ring;  // the products' and the bounds' place among the chunks
    bool lap = false;        // every place has been used
    const int quarter = warp & 3, part = (warp >> 2) & 1;  // rows, and maxima: half; bounds: lo or hi
    const int units = kWideStart + a.tiles;
    const int64_t all = (int64_t)a.items * units;
    int64_t unit = all * blockIdx.x / gridDim.x;
    const int64_t end = all * (blockIdx.x + 1) / gridDim.x;
    while (unit < end && __syncthreads_and(ok)) {
        const int item = (int)(unit / units), u0 = (int)(unit - (int64_t)item * units);
        const int u1 = (int)min((int64_t)units, u0 + (end - unit));
        unit += u1 - u0;
        const int x0 = max(u0 - kWideStart, 0);  // the CTA's tiles of the item: [x0, x1)
        if (u1 - kWideStart <= x0) continue;
        const int kvh = item % a.hkv, slot = item / a.hkv;
        // ---- the CTA's tokens: [t0, t0 + n) of sequence b
        int b = slot, skip = 0;
        if (!a.direct) {
            auto tiles_of_seq = [&](int i) {
                const Seq q = load_seq(a.s, i, a.num_q);
                return q.ok ? (q.nq + a.tokens - 1) / a.tokens : 0;
            };
            b = -1;
            if (a.s.num_seqs <= 32) {  // a warp's sums: no barrier
                const int mine = lane < a.s.num_seqs ? tiles_of_seq(lane) : 0;
                int incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                const uint32_t hit = __ballot_sync(0xffffffffu, slot >= incl - mine && slot < incl);
                if (hit) {
                    b = __ffs(hit) - 1;
                    skip = (slot - __shfl_sync(0xffffffffu, incl - mine, b)) * a.tokens;
                }
            } else {
                int before = 0;
                for (int c0 = 0; c0 < a.s.num_seqs; c0 += Pieces<kWideThreads>::kChunk) {
                    const int total = pieces.scan(c0, a.s.num_seqs, tiles_of_seq);
                    if (slot < before + total) {
                        const int i = pieces.find(slot - before, min(Pieces<kWideThreads>::kChunk, a.s.num_seqs - c0));
                        b = c0 + i;
                        skip = (slot - before - pieces.first[i]) * a.tokens;
                        break;
                    }
                    before += total;
                    __syncthreads();
                }
            }
        }
        Seq sq{0, 0, 0, false};
        if (b >= 0) sq = load_seq(a.s, b, a.num_q);
        const int n = sq.ok ? min(a.tokens, sq.nq - skip) : 0;
        const int t0 = sq.q0 + skip;
        // a context that ends before these tiles (max_ctx may be far longer): nothing to lay out
        if (n <= 0 || ((int64_t)x0 * kWideRows << a.shift) >= sq.ctx) continue;
        // ---- the bounds' warps: a lane's 16 bytes of a chunk's row, four lanes a row, 16 rows a warp; on
        // their way beside the queries
        const bool bounds_warp = warp >= 8 && warp < 16;
        const int li = lane & 3, row0 = (warp - 8) * 16 + (lane >> 2);
        // block of row (warp - 8) 16 + lane, by the context (-1 none, -2 lost), from its page
        auto token_of = [&](int x) { return (int64_t)(x * kWideRows + (warp & 7) * 16 + (lane & 15)) << a.shift; };
        const int64_t base = first_row(a.s, b);
        auto page_of_tile = [&](int x) {
            return token_of(x) < sq.ctx ? page_at(a.s, a.page_shift, b, token_of(x)) : 0;
        };
        auto place = [&](int x, int page) -> int {
            if (token_of(x) >= sq.ctx) return -1;
            const int64_t r = row_in(a.s, a.page_shift, page, base, token_of(x));
            return r < 0 || (r & ((1 << a.shift) - 1)) ? -2 : (int)(r >> a.shift);
        };
        const uint4* bounds = reinterpret_cast<const uint4*>(a.bounds + (int64_t)kvh * (2 * D)) + li;
        // a lane's copies are its own: nobody else waits for them
        uint8_t* mine = stage + (warp & 7) * (C::kStage / 8) + lane * 16;
        auto fetch = [&](int at, int c) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int p = __shfl_sync(0xffffffffu, at, u * 8 + (lane >> 2));
                copy16(mine + (2 * c + u) * 512, bounds + (int64_t)max(p, 0) * (a.hkv * (D / 8)) + 4 * c, p >= 0);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int at = -1;
        int page = 0;  // of the next tile
        if (bounds_warp) {
            at = place(x0, page_of_tile(x0));
            page = page_of_tile(x0 + 1);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) fetch(at, c);
        }
        // ---- the queries in whole steps: a warp takes a token's columns (of 8 columns' tokens, where they
        // are several), four columns at a time, 16 dims a lane (D = 64: eight columns)
        if (tid < kWideLay) {
            constexpr int kLanes = D / 16, kSet = 32 / kLanes;  // lanes per column, columns per set
            const int pad = a.pad, sh = 31 - __clz(pad);
            const int unit = max(pad, 8);       // columns a warp takes at a time
            // (eight lanes next to each other: four of two columns, so that their stores meet no bank twice)
            const int c = (lane & 3) | (D == 128 ? lane >> 4 << 2 : 0), lane_col = (lane >> 2) & (kSet - 1);
            auto query = [&](int col, uint32_t (&w)[8]) {
                const int tok = col >> sh, head = min(col & (pad - 1), a.group - 1);  // the last again behind it
                const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(t0 + tok) * a.q_stride +
                                                                  (int64_t)(kvh * a.group + head) * D + 16 * c);
                uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u;
                if (tok < n) u = __ldg(src), v = __ldg(src + 1);
                w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
            };
            // largest magnitude, as it is; what is not finite leaves by hand
            auto top_of = [&](const uint32_t (&w)[8]) {
                uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
                for (int e = 1; e < 8; ++e) m = packed_max<false>(m, w[e] & 0x7FFF7FFFu);
                const float2 m2 = packed_floats<false>(m);
                float top = fmaxf(m2.x, m2.y);
                if (!(m2.x < INFINITY && m2.y < INFINITY)) {
                    top = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float u = fabsf(__uint_as_float(w[e] << 16)), v = fabsf(__uint_as_float(w[e] & 0xFFFF0000u));
                        top = fmaxf(top, fmaxf(u < INFINITY ? u : 0.f, v < INFINITY ? v : 0.f));
                    }
                }
                return top;
            };
            // over a column's lanes, and over the columns of its token among the set's
            auto over_token = [&](float top) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if (D == 128) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
#pragma unroll
                for (int o = 1; o < kSet; o <<= 1) {
                    const float y = __shfl_xor_sync(0xffffffffu, top, 4 * o);
                    if (o < pad) top = fmaxf(top, y);
                }
                return top;
            };
            auto lay = [&](int col, const uint32_t (&w)[8], float top) {
                float step;
                const float up = step_up(top, step);
                // rounded by adding 1.5 2^23 (a value times a power of two is exact); what is not finite by hand
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = packed_max<false>(m, w[e] & 0x7FFF7FFFu);
                const float2 m2 = packed_floats<false>(m);
                const bool plain = m2.x < INFINITY && m2.y < INFINITY;
                const uint64_t up2 = f32x2(up, up), magic = f32x2(0x1.8p23f, 0x1.8p23f), back = f32x2(-0x1.8p23f, -0x1.8p23f);
                const __half2 zero = __half2half2(__ushort_as_half(0));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t lo[4], hi[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t q2 = w[4 * h + e];
                        float u = __uint_as_float(q2 << 16), v = __uint_as_float(q2 & 0xFFFF0000u);
                        if (plain) {
                            unpack2(add2(fma2(f32x2(u, v), up2, magic), back), u, v);
                        } else {
                            u = whole_steps(u, up);
                            v = whole_steps(v, up);
                        }
                        uint32_t z2 = pack_f16(u, v);
                        const __half2 l2 = __hmin2(*reinterpret_cast<__half2*>(&z2), zero);
                        const __half2 h2 = __hmax2(*reinterpret_cast<__half2*>(&z2), zero);
                        lo[e] = *reinterpret_cast<const uint32_t*>(&l2);
                        hi[e] = *reinterpret_cast<const uint32_t*>(&h2);
                    }
                    uint8_t* dst = bsh + (c / 4) * (kWideCols * 128) + col * 128 + (((c % 4 * 2 + h) ^ (col & 7)) << 4);
                    *reinterpret_cast<uint4*>(dst) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    *reinterpret_cast<uint4*>(dst + C::kChunks / 2 * (kWideCols * 128)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                }
            };
            if (unit == 8) {  // all of the warp's columns on their way at once
                constexpr int kSets = kWideCols / (kWideLay / 32) / kSet;
                uint32_t w[kSets][8];
                float top[kSets];
                const int c0 = warp * (kWideCols / (kWideLay / 32)) + lane_col;
#pragma unroll
                for (int y = 0; y < kSets; ++y) query(c0 + y * kSet, w[y]);
#pragma unroll
                for (int y = 0; y < kSets; ++y) top[y] = over_token(top_of(w[y]));
#pragma unroll
                for (int y = 0; y < kSets; ++y)
                    lay(c0 + y * kSet, w[y], kSet == 4 && pad == 8 ? fmaxf(top[y], top[y ^ 1]) : top[y]);
            } else {
                // tokens of 16 columns or more: read twice
                for (int c0 = warp * unit; c0 < kWideCols; c0 += kWideLay / 32 * unit) {
                    float top = 0.f;
                    for (int y = 0; y < unit; y += kSet) {
                        uint32_t w[8];
                        query(c0 + y + lane_col, w);
                        top = fmaxf(top, top_of(w));
                    }
                    top = over_token(top);
                    for (int y = 0; y < unit; y += kSet) {
                        uint32_t w[8];
                        query(c0 + y + lane_col, w);
                        lay(c0 + y + lane_col, w, top);
                    }
                }
            }
            int most = -1;
            for (int i = tid; i < n; i += kWideLay) {
                const int p = __ldg(a.s.q_pos + t0 + i);
                if (p >= 0 && p < sq.ctx) most = max(most, p >> a.shift);
            }
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0) most_sh[warp] = most;
            ptx::fence_proxy_async_smem();
        }
        __syncthreads();
        int most = -1;
#pragma unroll
        for (int w = 0; w < kWideLay / 32; ++w) most = max(most, most_sh[w]);
        const int cols = (n * a.pad + 15) & ~15;
        const int x1 = min(u1 - kWideStart, (most + kWideRows) / kWideRows);  // (none where no query sees a block)

        if (warp == kWideLay / 32) {
            // ---- the products
            if (lane == 0) {
                const uint32_t idesc = ptx::idesc_f16_m128(cols, false);
                const uint64_t da = ptx::sdesc_sw128(smem_u32(ash)), db = ptx::sdesc_sw128(smem_u32(bsh));
                for (int x = x0; x < x1 && ok; ++x, ++tile) {
                    const int buf = tile & 1;
                    if (tile >= 2) ok = quick_wait(tempty + buf, ((tile >> 1) - 1) & 1, abort_flag, a.d_status);
                    for (int c = 0; c < C::kChunks && ok; ++c, ring.move(1)) {
                        ok = quick_wait(afull + ring.st, ring.ph, abort_flag, a.d_status);
                        if (!ok) break;
                        ptx::tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ptx::mma_ss(tmem + buf * kWideCols,
                                        da + (uint32_t)(ring.st * (kWideRows * 128 / 16) + k * 2),
                                        db + (uint32_t)(c * (kWideCols * 128 / 16) + k * 2), idesc,
                                        c > 0 || k > 0 ? 1u : 0u);
                        ptx::mma_commit(aempty + ring.st);
                        if (c == C::kChunks - 1) ptx::mma_commit(tfull + buf);
                    }
                }
            }
            __syncwarp();
        } else if (bounds_warp) {
            // ---- bounds to f16
            for (int x = x0; x < x1 && ok; ++x) {
                if (at == -2 && lane < 16 && x * kWideRows + (warp - 8) * 16 + lane <= most && kvh == 0)
                    report(a.d_status, DSA_ERR_BAD_INPUT);
                at = place(x + 1, page);
                page = page_of_tile(x + 2);
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c) {
                    if (lap) ok = ok && quick_wait(aempty + ring.st, ring.ph ^ 1u, abort_flag, a.d_status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    // (the oldest group: as many are on their way as a tile has chunks)
                    asm volatile("cp.async.wait_group %0;" ::"n"(C::kChunks - 1) : "memory");
                    uint4 z[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) z[u] = *reinterpret_cast<const uint4*>(mine + (2 * c + u) * 512);
                    fetch(at, c);  // the next tile's, beside this one's products
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int row = row0 + u * 8;
                        uint32_t f[8];
                        bytes_to_f16(z[u].x, f[0], f[1]);
                        bytes_to_f16(z[u].y, f[2], f[3]);
                        bytes_to_f16(z[u].z, f[4], f[5]);
                        bytes_to_f16(z[u].w, f[6], f[7]);
                        uint8_t* dst = ash + ring.st * (kWideRows * 128) + row * 128;
                        *reinterpret_cast<uint4*>(dst + (((li * 2) ^ (row & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
                        *reinterpret_cast<uint4*>(dst + (((li * 2 + 1) ^ (row & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(afull + ring.st);
                    ring.move(1);
                    lap = lap || ring.st == 0;
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");  // the next item's take the same places
        } else {
            // ---- maxima: this thread's block, 32 of its half of the columns at a time
            const int from = part * kWideHalf, to = min(cols, from + kWideHalf);
            // the step of its block: the page's load two tiles ahead, the step's one
            auto page_of = [&](int x) {
                const int blk = x * kWideRows + quarter * 32 + lane;
                return blk <= most ? page_at(a.s, a.page_shift, b, (int64_t)blk << a.shift) : -1;
            };
            auto step_at = [&](int x, int page) {
                const int blk = x * kWideRows + quarter * 32 + lane;
                const int64_t r = blk <= most ? row_in(a.s, a.page_shift, page, base, (int64_t)blk << a.shift) : -1;
                return r >= 0 && (r & ((1 << a.shift) - 1)) == 0 ? __ldg(a.steps + (r >> a.shift) * a.hkv + kvh) : 0.f;
            };
            const int64_t next = (int64_t)a.hkv * a.ld;  // to the next token's row
            float ahead = step_at(x0, page_of(x0));
            int far = page_of(x0 + 1);
            for (int x = x0; x < x1 && ok; ++x, ++tile) {
                const int buf = tile & 1, blk = x * kWideRows + quarter * 32 + lane;
                const float step = kStepDown * ahead;
                ahead = step_at(x + 1, far);
                far = page_of(x + 2);
                ok = __all_sync(0xffffffffu, quick_wait(tfull + buf, (tile >> 1) & 1, abort_flag, a.d_status));
                if (!ok) break;
                ptx::tc_fence_after();
                auto give_back = [&] {  // every column is read
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(tempty + buf);
                };
                if (from >= to) give_back();
                const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + buf * kWideCols;
                const int lim = blk <= most ? n : 0;  // tokens that this thread stores
                int tok = from / a.pad;
                float* dst = a.scores + ((int64_t)(t0 + tok) * a.hkv + kvh) * a.ld + blk;
                float last = -INFINITY;  // pad 64: of the first half of a token's columns
                auto store = [&](float m) {
                        if (tok < lim) *dst = m * step;
                    ++tok;
                    dst += next;
                };
                auto put = [&](auto pad, const uint32_t (&v)[32], int c) {
                    constexpr int P = decltype(pad)::value;
                    if constexpr (P <= 32) {
#pragma unroll
                        for (int y = 0; y < 32; y += P) {
                            float m = __uint_as_float(v[y]);
#pragma unroll
                            for (int e = 1; e + 1 < P; e += 2)
                                m = fmaxf(fmaxf(m, __uint_as_float(v[y + e])), __uint_as_float(v[y + e + 1]));
                            if (P > 1) m = fmaxf(m, __uint_as_float(v[y + P - 1]));
                            store(m);
                        }
                    } else {
                        float m = __uint_as_float(v[0]);
#pragma unroll
                        for (int e = 1; e < 32; ++e) m = fmaxf(m, __uint_as_float(v[e]));
                        if (c & 32) store(fmaxf(m, last));
                        else last = m;
                    }
                };
                auto walk = [&](auto pad) {
#pragma unroll 1
                    for (int c = from; c < to; c += 32) {
                        uint32_t v[32];
                        ptx::tmem_ld32_async(src + c, v);
                        ptx::tmem_wait_ld32(v);
                        if (c + 32 >= to) give_back();
                        put(pad, v, c);
                    }
                };
                using std::integral_constant;
                if (a.pad == 8) walk(integral_constant<int, 8>());
                else if (a.pad == 4) walk(integral_constant<int, 4>());
                else if (a.pad == 16) walk(integral_constant<int, 16>());
                else if (a.pad == 1) walk(integral_constant<int, 1>());
                else if (a.pad == 2) walk(integral_constant<int, 2>());
                else if (a.pad == 32) walk(integral_constant<int, 32>());
                else walk(integral_constant<int, 64>());
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kWideLay / 32) ptx::tmem_dealloc(tmem, 512);
}

// A warp per row of up to 32 K blocks: the keys stay in registers, and the cut
// is found by halving their range (counts by a warp's sums, no barrier; it ends
// when exactly `want` lie above).
constexpr int kRowsPerCta = 4, kKept = 128;

template <int K>
__global__ void __launch_bounds__(32 * kRowsPerCta) block_pick_row_kernel(const __grid_constant__ PickArgs a) {
    __shared__ uint32_t kept[kRowsPerCta][2][kKept];
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kRowsPerCta + (threadIdx.x >> 5);
    if (r >= (int64_t)a.num_q * a.hkv) return;
    const int t = (int)(r / a.hkv);
    const int pos = __ldg(a.s.q_pos + t);  // checked beside the scores' loads
    const int n = min(a.ld, pos < 0 ? 0 : (pos >> a.shift) + 1);
    const bool choose = n > a.nsel;
    const int hi = n - a.local;
    int want = a.nsel - a.first - a.local;
    const int i0 = lane * K;  // the lane's blocks: neighbours, so that the lanes' order is theirs
    uint32_t key[K];
    if (choose) {
        const float* row = a.scores + r * a.ld;
#pragma unroll
        for (int k = 0; k < K; k += 4) {
            const int i = i0 + k;
            const float4 f = i < a.ld ? *reinterpret_cast<const float4*>(row + i) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)  // 0: none, below any score's code
                key[k + e] = (uint32_t)(i + e - a.first) < (uint32_t)(hi - a.first) ? score_code(v[e]) : 0u;
        }
    }
    const int b = warp_seq_of(a.s.q_start, a.s.num_seqs, t);
    const Seq sq = load_seq(a.s, b, a.num_q);
    if (t >= sq.q0 + sq.nq || t < sq.q0) return;  // behind the last sequence: left as it was
    if (!sq.ok || pos < -1 || pos >= sq.ctx) {
        if (lane == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
        return;
    }
    int32_t* out = a.blocks + r * a.nsel;
    if (lane == 0)
        a.len[r] = seen_keys(pos, min(n, a.nsel), a.shift);
    if (!choose) {
        for (int i = lane; i < a.nsel; i += 32) out[i] = i < n ? i : -1;
        return;
    }
    // the largest `cut` with at least `want` keys at or above it, until exactly `want` are, or few enough
    // for four a lane
    uint32_t cut = 0xFFFFFFFFu;
    int ties = 0;
    const uint32_t under = (1u << lane) - 1;
    auto before = [&](int x) {  // sum over the lanes before
        int incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        return incl - x;
    };
    if (want > 0) {
        uint32_t least = 0xFFFFFFFFu, best = 0u;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            least = min(least, key[k] ? key[k] : 0xFFFFFFFFu);
            best = max(best, key[k]);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        best = __reduce_max_sync(0xffffffffu, best);
        int have = hi - a.first;  // keys at or above `least`
        while (least < best && have != want && have > kKept) {
            const uint32_t mid = least + (best - least + 1) / 2;
            int c = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) c += key[k] >= mid;
            c = __reduce_add_sync(0xffffffffu, c);
            if (c >= want) least = mid, have = c; else best = mid - 1;
        }
        if (have <= kKept) {
            // those, in order, with their blocks: the rest of the search is theirs alone
            uint32_t* codes = kept[threadIdx.x >> 5][0];
            uint32_t* names = kept[threadIdx.x >> 5][1];
            uint32_t mine = 0;  // the lane's keys that stay
#pragma unroll
            for (int k = 0; k < K; ++k) mine |= key[k] >= least ? 1u << k : 0u;
            int at = before(__popc(mine));
#pragma unroll
            for (int k = 0; k < K; ++k)
                if ((mine >> k) & 1) {
                    codes[at] = key[k];
                    names[at++] = i0 + k;
                }
            __syncwarp();
            uint32_t c4[kKept / 32];
#pragma unroll
            for (int y = 0; y < kKept / 32; ++y) c4[y] = y * 32 + lane < have ? codes[y * 32 + lane] : 0u;
            int left = have;
            while (least < best && left != want) {
                const uint32_t mid = least + (best - least + 1) / 2;
                int c = 0;
#pragma unroll
                for (int y = 0; y < kKept / 32; ++y) c += __popc(__ballot_sync(0xffffffffu, c4[y] >= mid));
                if (c >= want) least = mid, left = c; else best = mid - 1;
            }
            int over = 0;
#pragma unroll
            for (int y = 0; y < kKept / 32; ++y) over += __popc(__ballot_sync(0xffffffffu, c4[y] > least));
            int eq = 0, to = a.first;
#pragma unroll
            for (int y = 0; y < kKept / 32; ++y) {
                const bool yes = c4[y] > least, tie = c4[y] == least;  // (0, none, is below any)
                const uint32_t e = __ballot_sync(0xffffffffu, tie);
                const int rank = eq + __popc(e & under);
                const uint32_t in = __ballot_sync(0xffffffffu, yes || (tie && rank < want - over));
                if ((in >> lane) & 1) out[to + __popc(in & under)] = names[y * 32 + lane];
                to += __popc(in);
                eq += __popc(e);
            }
            for (int i = lane; i < a.first; i += 32) out[i] = i;
            for (int i = lane; i < a.local; i += 32) out[a.nsel - a.local + i] = hi + i;
            return;
        }
        cut = least;
        if (have == want) {
            --cut;
        } else {
            int c = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) c += key[k] > cut;
            ties = want - __reduce_add_sync(0xffffffffu, c);
        }
    }
    int sure = 0, same = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = i0 + k;
        const bool fix = i < n && (i < a.first || i >= hi);
        sure += fix || key[k] > cut;
        same += !fix && key[k] == cut && ties > 0;
    }
    int at = before(sure), eq = before(same);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = i0 + k;
        const bool fix = i < n && (i < a.first || i >= hi);
        const bool yes = fix || key[k] > cut, tie = !fix && key[k] == cut && ties > 0;
        const int place = at + min(eq, ties);
        if ((yes || (tie && eq < ties)) && place < a.nsel) out[place] = i;
        at += yes;
        eq += tie;
    }
}

template <int T>
__global__ void __launch_bounds__(T) block_pick_kernel(const __grid_constant__ PickArgs a) {
    extern __shared__ uint32_t key[];
    __shared__ PickShared<T> sh;
    __shared__ int bad_sh;
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = blockIdx.x / a.hkv;
    const int pos = __ldg(a.s.q_pos + t);  // checked beside the scores' loads
    const int n = min(a.ld, pos < 0 ? 0 : (pos >> a.shift) + 1);
    if (warp == 0) {
        const int b = warp_seq_of(a.s.q_start, a.s.num_seqs, t);
        const Seq sq = load_seq(a.s, b, a.num_q);
        // 1: behind the last sequence, 2: bad
        if (lane == 0)
            bad_sh = t >= sq.q0 + sq.nq || t < sq.q0 ? 1 : !sq.ok || pos < -1 || pos >= sq.ctx ? 2 : 0;
    }
    const bool choose = n > a.nsel;
    const int hi = n - a.local;
    if (choose) {
        uint32_t least = 0xFFFFFFFFu, best = 0u;
        const float* row = a.scores + (int64_t)blockIdx.x * a.ld;
#pragma unroll 8
        for (int i = a.first + tid; i < hi; i += T) {
            const uint32_t k = score_code(row[i]);
            key[i] = k;
            least = min(least, k);
            best = max(best, k);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        best = __reduce_max_sync(0xffffffffu, best);
        if (lane == 0) sh.ends[0][warp] = least, sh.ends[1][warp] = best;
        for (int i = tid; i < kBins; i += T) sh.hist[i] = 0;
        if (tid == 0) sh.count = 0;
    }
    __syncthreads();
    if (bad_sh) {  // left as it was
        if (bad_sh == 2 && tid == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
        return;
    }
    int32_t* out = a.blocks + (int64_t)blockIdx.x * a.nsel;
    if (tid == 0) a.len[blockIdx.x] = seen_keys(pos, min(n, a.nsel), a.shift);
    if (!choose) {  // all of them
        for (int i = tid; i < a.nsel; i += T) out[i] = i < n ? i : -1;
        return;
    }
    pick<T>(sh, key, n, a.first, hi, a.nsel - a.first - a.local, a.nsel, out);
}

}  // namespace

// scores of a row: whole 16 bytes
size_t select_ld(const dsa_seqs& s, int block) { return (((size_t)s.max_ctx + block - 1) / block + 3) & ~(size_t)3; }

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
    a.page_shift = page_shift_of(s);
    int64_t blocks = std::min<int64_t>(num_q, (num_q >> a.shift) + 2 * (int64_t)s.num_seqs);
    if (a.scale_shift > a.shift)  // and the older ones of a scale block, once per sequence
        blocks += std::min<int64_t>(num_q, s.num_seqs) * ((1 << (a.scale_shift - a.shift)) - 1);
    const int64_t ctas = blocks * ((sh.num_kv_heads + 1) / 2);  // two heads of a block at a time
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(ctas, kPlanSms * 8));
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
    a.page_shift = page_shift_of(s);
    a.ld = (int32_t)select_ld(s, block);
    a.pad = 1;
    while (a.pad < a.group && a.pad < 8) a.pad *= 2;
    a.npt = (a.group + 7) / 8;
    const int tpt = 8 / a.pad;
    PickArgs p;
    p.scores = a.scores;
    p.blocks = blocks;
    p.len = len;
    p.s = s;
    p.d_status = d_status;
    p.num_q = num_q;
    p.hkv = sh.num_kv_heads;
    p.shift = shift;
    p.ld = a.ld;
    p.nsel = nsel;
    p.first = first;
    p.local = local;
    // up to four tiles of query rows per sequence and head: as many CTAs as fit at once, in shares of
    // the blocks (four tiles of 16 at least)
    const int64_t tiles = ((int64_t)s.max_q_per_seq + tpt - 1) / tpt * a.npt;
    cudaError_t e;
    if (s.max_q_per_seq <= kFewTiles * tpt && tiles <= kFewTiles) {
        a.tokens = s.max_q_per_seq;
        a.direct = 1;
        const int64_t pairs = (int64_t)s.num_seqs * a.hkv, most = (a.ld + 16 * kFewWarps - 1) / (16 * kFewWarps);
        // (sequence, key head)s that make two CTAs an SM choose for themselves: with fewer the scores take
        // longer than the second kernel (one token, 8 key heads, L2 flushed, without the bounds, a second kernel
        // and not: 8 sequences of 512 blocks 29.2 us and 32.2, of 2,048 41.7 and 71.4; 24 33.0 and 33.2, 61.8
        // and 78.9; 38 37.0 and 34.6, 75.3 and 81.9; 48 43.8 and 36.4, 97.7 and 85.1; 150 71.4 and 66.1,
        // 179 and 165; of 32 blocks 21 and 18 with any number up to 64)
        const bool own = pairs >= 2 * kPlanSms && (int64_t)s.max_q_per_seq * a.ld <= kFewScores;
        a.xt = own ? 1 : (int32_t)std::max<int64_t>(1, std::min<int64_t>(most, kPlanSms * 5 / pairs));
        const int64_t grid = pairs * a.xt;
        if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
        const size_t smem = own ? (size_t)s.max_q_per_seq * a.ld * 4 : 0;
        auto go = [&](auto kern) {
            return launch_pdl(kern, dim3((unsigned)grid), dim3(kFewThreads), smem, stream, 1, a, p);
        };
        auto by_tiles = [&](auto d, auto o) {
            constexpr int D = decltype(d)::value;
            constexpr bool O = decltype(o)::value;
            return tiles == 1   ? go(block_score_few_kernel<D, 1, O>)
                   : tiles == 2 ? go(block_score_few_kernel<D, 2, O>)
                                : go(block_score_few_kernel<D, 4, O>);
        };
        using std::integral_constant;
        if (sh.head_dim == 64)
            e = own ? by_tiles(integral_constant<int, 64>(), std::true_type())
                    : by_tiles(integral_constant<int, 64>(), std::false_type());
        else
            e = own ? by_tiles(integral_constant<int, 128>(), std::true_type())
                    : by_tiles(integral_constant<int, 128>(), std::false_type());
        if (e != cudaSuccess || own) return e;
    } else {
        a.pad = 1;
        while (a.pad < a.group) a.pad *= 2;
        a.tokens = std::min(s.max_q_per_seq, kWideCols / a.pad);
        a.direct = s.max_q_per_seq <= a.tokens;
        const int64_t slots = a.direct ? s.num_seqs : std::min<int64_t>(num_q, num_q / a.tokens + s.num_seqs);
        const int64_t items = slots * a.hkv;
        a.tiles = (a.ld + kWideRows - 1) / kWideRows;
        if (items > INT32_MAX) return cudaErrorInvalidConfiguration;
        a.items = (int32_t)items;
        const unsigned grid = (unsigned)std::min<int64_t>(items * a.tiles, num_sms());
        auto go = [&](auto d) {
            constexpr int D = decltype(d)::value;
            auto kern = block_score_wide_kernel<D>;
            static OncePerDevice once;
            const cudaError_t r = once.run(
                [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Wide<D>::kSmem); });
            if (r != cudaSuccess) return r;
            return launch_pdl(kern, dim3(grid), dim3(kWideThreads), Wide<D>::kSmem, stream, 1, a);
        };
        e = sh.head_dim == 64 ? go(std::integral_constant<int, 64>()) : go(std::integral_constant<int, 128>());
    }
    if (e != cudaSuccess) return e;
    // a row's keys by 128 threads (many rows at once), or 1,024 where they are many
    auto go = [&](auto threads) {
        constexpr int T = decltype(threads)::value;
        static OncePerDevice once;
        const cudaError_t r = once.run([] {
            return cudaFuncSetAttribute(block_pick_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        DSA_GQA_MAX_BLOCKS * 4);
        });
        if (r != cudaSuccess) return r;
        return launch_pdl(block_pick_kernel<T>, dim3((unsigned)(num_q * a.hkv)), dim3(T), (size_t)a.ld * 4, stream, 1,
                          p);
    };
    // or by a warp, where the rows are eight CTAs of four an SM (with the scores, L2 flushed, a CTA a row and a warp:
    // 2,432 rows of 256 blocks 37.1 us and 35.6, of 1,024 51.1 and 47.5; 4,864 51.9 and 43.6, 74.9 and 64.5;
    // 16,384 107 and 76, 185 and 142; level at 512, 31.0 and 30.6, 37.2 and 38.3)
    const unsigned ctas = (unsigned)(((int64_t)num_q * a.hkv + kRowsPerCta - 1) / kRowsPerCta);
    auto rows = [&](auto kern) { return launch_pdl(kern, dim3(ctas), dim3(32 * kRowsPerCta), 0, stream, 1, p); };
    if ((int64_t)num_q * a.hkv >= 8 * kPlanSms * kRowsPerCta) {
        if (a.ld <= 256) return rows(block_pick_row_kernel<8>);
        if (a.ld <= 512) return rows(block_pick_row_kernel<16>);
        if (a.ld <= 1024) return rows(block_pick_row_kernel<32>);
    }
    return a.ld <= 2048 ? go(std::integral_constant<int, 128>()) : go(std::integral_constant<int, 1024>());
}

}  // namespace gqa
}  // namespace dsa
