// gqa_decode.cu -- dense attention of a few new tokens per sequence over a
// long K/V cache with grouped heads (sm_103a), split over the cache and joined.
//
//   s_j = sm_scale * q_h . k_j,  p = softmax over j <= pos,  out = sum_j p_j v_j
//
// One pass over the keys with a running reference m (in log2 units) and sum l
// per query row: p_j = 2^(x_j - m), x_j = s_j log2 e, l and the output
// accumulators rescaled when a row's maximum passes m by more than 8 (so a
// weight stays below 2^8).  Partial results (m, l, O) of pieces of a row's
// keys combine exactly: M = max m, weights 2^(m - M).
//
// What bounds it: the cache is read once, 2 (G T) / 2 flop a byte (G query
// heads a key head, T new tokens): HBM.  So the products run on the warp-level
// matrix instruction straight from shared memory (8 columns wide: no padding
// of a group of 8), which leaves the accumulators in registers and the
// issue slots mostly idle, and everything else serves the stream of loads:
// - A CTA owns a contiguous piece of the space (lane = key head x row chunk,
//   sequence, 64-key tile), balanced over the tiles that exist, and CTAs of
//   neighbouring lanes walk the same keys at the same time, so a token's heads
//   (256 or 512 bytes apart) are read from the same DRAM pages together.
// - One warp loads: TMA boxes of whole pages (or of a tile) into a ring of
//   stages; the computing warps take 16 keys of each tile, each with its own
//   softmax state, and meet only at the end of a sequence.  Up to 8 query rows:
//   four of them, two CTAs per SM.  Up to 32 rows (drafts to verify): eight
//   that hold all the rows each, so that a key is read and converted once.
// - A sequence cut by CTA borders leaves one partial per CTA, which a second
//   kernel joins in a fixed order.
// - Few and short sequences are bound by latency, and the second kernel alone
//   takes 4 us: there a cluster of CTAs shares a (lane, sequence) and joins its
//   partials through distributed shared memory.
//
// Measured, 64/8 heads of 128: 64 x 32,768 bf16 1,230 us, 7.0 TB/s (a copy: 6.8);
// 1 x 524,288 e4m3 170 to 173 us, 6.4 TB/s; 128 x 4 tokens over 61 to 16,381 e4m3 566 us,
// 3.9 TB/s: there 32 rows make 64 products, 64 conversions and 480 instructions of
// a warp's 16 keys, and two warps a scheduler leave 62% of its issue slots unused
// (the rows split over 16 warps: 699, a key is then converted twice).
#include <type_traits>

#include "gqa_common.cuh"

namespace dsa {
namespace gqa {
namespace {

constexpr int kTagDecode = 6;
constexpr int kMaxCluster = 16;
constexpr float kLazy = 8.f;  // a row's reference moves when its maximum passes it by 2^8
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -3e38f;  // the reference of a row that has seen no key (its sum is 0)

// NT: 8-row tiles of query rows; KS: computing warps, 16 keys of a tile each
template <int D, bool FP8, int NT, int KS>
struct Cfg {
    static constexpr int kRows = 8 * NT;     // query rows per chunk
    static constexpr int kTile = 16 * KS;    // keys per tile
    static constexpr bool kSplitRegs = KS == 8;  // three warpgroups, the registers given to the computing two
    static constexpr int kThreads = kSplitRegs ? 384 : 32 * (KS + 1);
    static constexpr int kOcc = KS == 8 ? 1 : 2;  // CTAs per SM
    static constexpr int kHeadBytes = D * (FP8 ? 1 : 2);
    static constexpr int kHalf = kTile * kHeadBytes;  // K or V of a stage
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kScaleBytes = FP8 ? 2 * kTile * 4 : 0;
    static constexpr int kScratch = 4 * 8 * D * 4;  // four key slices' outputs of 8 rows
    static constexpr int kMl = KS * kRows * 8;
    // What a sequence's start and end cost, in tiles.  (Left out of the deal, the CTA with the most
    // sequences ended 14% after the average; with twice these 128 x 4 tokens over 61 to 16,381 take 2% longer.)
    static constexpr int kStart = KS == 8 ? 6 : 3;
    static constexpr bool kQShared = NT > 2;        // query fragments in shared memory, else in registers
    static constexpr int kQBytes = kQShared ? (D / 16) * NT * 32 * 8 : 0;
    static constexpr int kMisc = 256 + kRows * 24;
    static constexpr int kFixed = kScratch + kMl + kQBytes + kMisc;
    static constexpr int kBudget = (kOcc == 2 ? 115712 : 232448) - kFixed;
    static constexpr int kFit = kBudget / (kStage + kScaleBytes);
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr int kSmem = kStages * (kStage + kScaleBytes) + kFixed;
    static_assert(kStages >= 3, "a ring of at least three stages");
};

struct Args {
    const __nv_bfloat16* q;
    const float *k_scale, *v_scale;
    __nv_bfloat16* out;
    float* lse;
    float* part_o;   // [2 grid][rows][D]
    float2* part_ml; // [2 grid][rows]
    int4* desc;      // [grid]: {parts, q0, nq, lane} of the cut sequence that the CTA is the second of
    dsa_seqs s;
    int64_t q_stride;
    int32_t* d_status;
    float scale_log2;
    int32_t num_q, group, hkv, lanes, hl, parts;  // hl: lanes side by side; parts: CTAs per lane column
    int32_t cluster;  // > 0: a cluster of this many CTAs per (lane, sequence) instead
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void lds128(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void lds64(uint32_t (&r)[2], uint32_t addr) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
    return r;
}
__device__ __forceinline__ void bar_sync(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// two floats to a shared-memory address of the cluster's CTA `rank`
__device__ __forceinline__ void st_cluster(uint32_t addr, int rank, float2 v) {
    asm volatile(
        "{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %0, %1;\n st.shared::cluster.v2.f32 [r], {%2, %3};\n}\n" ::"r"(
            addr),
        "r"(rank), "f"(v.x), "f"(v.y)
        : "memory");
}
// two dims of a row times 1 / sum; a row that sees no key (inv = 0) is 0 beside any values
__device__ __forceinline__ uint32_t pack_row(float a, float b, float inv) {
    return inv == 0.f ? 0u : pack_bf16(a * inv, b * inv);
}
__device__ __forceinline__ float warp_max_all(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// byte address of 16-byte chunk `c` of a tile's row in the layout TMA wrote
// (128-byte pieces of a tile's rows, 128-byte swizzle; a 64-byte head row:
// 64-byte swizzle)
template <int HB, int TILE>
__device__ __forceinline__ uint32_t chunk_addr(uint32_t base, int row, int c) {
    if (HB == 64) return base + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
    return base + (c >> 3) * (TILE * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

template <int TILE>
__device__ __forceinline__ int tiles_of(const Seq& q) {
    return q.ok && q.nq > 0 ? max(1, (q.ctx + TILE - 1) / TILE) : 0;
}

// The walk over a CTA's pieces: each begin() gives a run of tiles [i0, i1) of
// one (lane, sequence).  Every warp of the CTA walks alike.
struct Piece {
    int lane, b, i0, i1;
    Seq q;
    bool front, back;        // cut by the border before / after this CTA
    int row0, tok0, ntok;    // chunk's first row, first token and tokens
    int limit;               // keys that some query of the chunk sees
    int64_t base;            // first row of a contiguous sequence
};

// The tiles of all lanes of a column in a row, before each sequence's START
// units for what its start and end cost, dealt to the column's CTAs in pieces
// of `each` units, the first `more` CTAs one more.
struct Deal {
    int64_t total, each;
    int more;
    __device__ __forceinline__ void set(int64_t n, int parts) {
        total = n;
        const int p = (int)min((int64_t)parts, n);
        if (n <= 0x7FFFFFFF) {  // a 32-bit division is several times faster
            each = p ? (uint32_t)n / (uint32_t)p : 0;
        } else {
            each = n / p;
        }
        more = (int)(n - each * p);
    }
    __device__ __forceinline__ int64_t first(int c) const { return each * c + min(c, more); }
    // the CTA that has unit x
    __device__ __forceinline__ int owner(int64_t x) const {
        const int64_t big = (each + 1) * more;
        if (x < big) return (int)(x / (each + 1));
        return more + (int)((x - big) / each);
    }
};

template <int TILE, int ROWS, int START, bool KEEP>
struct Walk {
    Deal deal;
    int64_t r0, left;
    int u, b, i;  // the place in the walk: tile i of sequence b, from -START
    Seq kept;     // of the lane's of the 32 sequences around b
    int kept_of;
    __device__ __forceinline__ int units_of(const Seq& q) const {
        const int n = tiles_of<TILE>(q);
        return n ? n + START : 0;
    }
    __device__ __forceinline__ void init(const Args& a) {
        const int lane = threadIdx.x & 31;
        const int B = a.s.num_seqs;
        kept_of = -1;
        if (a.cluster) {
            // the cluster's (lane, sequence), this CTA's share of its tiles
            const int seg = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
            u = seg % a.lanes;
            b = seg / a.lanes;
            const Seq q = load_seq(a.s, b, a.num_q);
            const int cnt = tiles_of<TILE>(q);
            if (!q.ok && rank == 0 && u == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
            i = (int)((int64_t)cnt * rank / a.cluster);
            left = cnt ? max(1, (int)((int64_t)cnt * (rank + 1) / a.cluster) - i) : 0;
            return;
        }
        const int c = blockIdx.x / a.hl;
        const int units = a.lanes / a.hl;
        // every lane a run of sequences: their tiles, then a scan over the lanes
        const int per = (B + 31) / 32;
        int64_t mine = 0;
        for (int k = 0; k < per; k += 4) {
            int v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int bb = lane * per + k + x;
                v[x] = 0;
                if (k + x < per && bb < B) {
                    const Seq q = load_seq(a.s, bb, a.num_q);
                    v[x] = units_of(q);
                    if (!q.ok && blockIdx.x == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
                }
            }
            mine += v[0] + v[1] + v[2] + v[3];
        }
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const int64_t sum = __shfl_sync(0xffffffffu, incl, 31);
        deal.set(sum * units, a.parts);
        left = 0;
        u = b = i = 0;
        r0 = 0;
        if (c >= a.parts || c >= deal.total) return;  // fewer tiles than CTAs
        r0 = deal.first(c);
        left = deal.first(c + 1) - r0;
        int64_t rem = r0;
        if (units > 1) {
            u = deal.total <= 0x7FFFFFFF ? (int)((uint32_t)r0 / (uint32_t)sum) : (int)(r0 / sum);
            rem -= u * sum;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, rem >= incl - mine && rem < incl);
        const int l = __ffs(hit) - 1;
        int64_t off = rem - __shfl_sync(0xffffffffu, incl - mine, l);
        if (per == 1) {
            b = l;
            i = (int)off - START;
            return;
        }
        // within that lane's run
        for (int k0 = 0; k0 < per; k0 += 32) {
            const int bb = l * per + k0 + lane;
            int v = 0;
            if (k0 + lane < per && bb < B) v = units_of(load_seq(a.s, bb, a.num_q));
            int in = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, in, o);
                if (lane >= o) in += y;
            }
            const uint32_t h = __ballot_sync(0xffffffffu, off >= in - v && off < in);
            if (h) {
                const int x = __ffs(h) - 1;
                b = l * per + k0 + x;
                i = (int)(off - __shfl_sync(0xffffffffu, in - v, x)) - START;
                break;
            }
            off -= __shfl_sync(0xffffffffu, in, 31);
        }
    }
    // sequence b's counts, from those that the lanes hold (whole warp); a CTA that
    // shares its SM has no registers for them, and another's work to hide the loads
    __device__ __forceinline__ Seq seq(const Args& a) {
        if (!KEEP) return load_seq(a.s, b, a.num_q);
        if (kept_of != b >> 5) {
            kept_of = b >> 5;
            const int bb = (b & ~31) + (threadIdx.x & 31);
            kept = bb < a.s.num_seqs ? load_seq(a.s, bb, a.num_q) : Seq{0, 0, 0, false};
            if (!kept.ok) kept.nq = 0;
        }
        Seq q;
        q.ctx = __shfl_sync(0xffffffffu, kept.ctx, b & 31);
        q.q0 = __shfl_sync(0xffffffffu, kept.q0, b & 31);
        q.nq = __shfl_sync(0xffffffffu, kept.nq, b & 31);
        q.ok = q.nq > 0;
        return q;
    }
    // the next piece, without its limit: `pos` is the lane's share of that
    __device__ __forceinline__ bool begin(const Args& a, Piece& p, int& pos) {
        while (left > 0) {
            if (b == a.s.num_seqs) {
                b = 0;
                ++u;
            }
            const Seq q = seq(a);
            const int cnt = tiles_of<TILE>(q);
            if (cnt == 0) {
                ++b;
                i = -START;
                continue;
            }
            int take = (int)min((int64_t)(cnt - i), left);
            left -= take;
            take += min(i, 0);  // the tiles among them
            i = max(i, 0);
            if (take <= 0) return false;  // the deal ends before the sequence's first tile
            p.lane = a.cluster ? u : blockIdx.x % a.hl + a.hl * u;
            p.b = b;
            p.q = q;
            p.front = i > 0;
            p.back = i + take < cnt;
            // (a cluster's CTA without tiles still has a share of nothing)
            if (a.cluster && (int64_t)cnt * (blockIdx.x % a.cluster + 1) / a.cluster == i) take = 0;
            p.i0 = i;
            p.i1 = i + take;
            i = -START;
            ++b;
            p.row0 = p.lane / a.hkv * ROWS;
            const int64_t rows = (int64_t)q.nq * a.group;
            if (p.row0 >= rows) continue;  // fewer queries than the longest sequence's
            p.tok0 = p.row0 / a.group;
            const int last = (int)min((int64_t)p.row0 + ROWS, rows) - 1;
            p.ntok = last / a.group - p.tok0 + 1;
            // keys that the chunk's queries see (at most ROWS <= 32 tokens)
            pos = -1;
            const int lane = threadIdx.x & 31;
            if (lane < p.ntok) pos = __ldg(a.s.q_pos + q.q0 + p.tok0 + lane);
            p.base = a.s.page_table ? 0 : __ldg(a.s.seq_base + p.b);
            return true;
        }
        return false;
    }
    __device__ __forceinline__ void finish(Piece& p, int pos) const {
        if (pos < -1 || pos >= p.q.ctx) pos = -1;
        p.limit = __reduce_max_sync(0xffffffffu, pos) + 1;
    }
};

template <int D, bool FP8, int NT, int KS>
__global__ void __launch_bounds__(Cfg<D, FP8, NT, KS>::kThreads, Cfg<D, FP8, NT, KS>::kOcc)
    gqa_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ Args a) {
    using C = Cfg<D, FP8, NT, KS>;
    constexpr int HB = C::kHeadBytes, kTile = C::kTile;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* ring = smem;
    float* ring_scale = reinterpret_cast<float*>(smem + C::kStages * C::kStage);
    float* scratch = reinterpret_cast<float*>(smem + C::kStages * (C::kStage + C::kScaleBytes));
    float2* ml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(scratch) + C::kScratch);
    uint8_t* q_sh = reinterpret_cast<uint8_t*>(ml) + C::kMl;  // [D / 16][NT / 2][lane] two tiles' fragments
    float* fac_sh = reinterpret_cast<float*>(q_sh + C::kQBytes);  // [rows]
    int* pos_sh = reinterpret_cast<int*>(fac_sh + C::kRows);      // [rows]
    float2* total = reinterpret_cast<float2*>(pos_sh + C::kRows);   // [rows] reference and sum of all slices
    int64_t* at_sh = reinterpret_cast<int64_t*>(total + C::kRows);  // [rows] row of out and lse
    uint64_t* full = reinterpret_cast<uint64_t*>(at_sh + C::kRows);
    uint64_t* empty = full + C::kStages;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + C::kStages);
    float* vref_sh = reinterpret_cast<float*>(empty + C::kStages + 1);  // [slices] e4m3
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            ptx::mbar_init(full + i, FP8 ? 33 : 1);
            ptx::mbar_init(empty + i, KS);
        }
        abort_flag[0] = 0;
        abort_flag[1] = kTagDecode;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&kmap);
        ptx::prefetch_tmap(&vmap);
    }
    __syncthreads();
    pdl_enter();

    Walk<kTile, C::kRows, C::kStart, C::kOcc == 1> w;
    Piece p;
    bool had = false;  // a computing warp had a piece

    if (warp >= KS) {
        if (C::kSplitRegs) reg_dec<72>();
        if (warp == KS) {
            w.init(a);
            // ---- the loading warp: a lane per TMA box of a 32-box window of the page table
            const int R = a.s.page_table ? min(a.s.page_size, kTile) : kTile;  // rows per box
            const int nbox = kTile / R;
            const int shift = 31 - __clz(R);
            Cursor<C::kStages> c;
            bool lap = false;  // every stage has been used
            bool ok = true;
            int pos;
            while (ok && w.begin(a, p, pos)) {
                const int kvh = p.lane % a.hkv;
                // physical row of a box's first token among the sequence's, num_rows: outside the
                // cache, -1: none; its load goes out before the queries' positions have arrived
                auto row_of = [&](int box) -> int {
                    const int64_t j = (int64_t)box << shift;
                    if (j >= p.q.ctx) return -1;
                    int64_t row = a.s.page_table ? phys_row(a.s, p.b, j) : p.base + j;
                    if (row < 0 || row >= a.s.num_rows) row = a.s.num_rows;
                    return (int)row;
                };
                // -1 for a box that no query sees.  Rows outside the cache are loaded as zeros (TMA's fill),
                // and reported where a query sees one.
                auto seen = [&](int row, int box) -> int {
                    const int64_t j = (int64_t)box << shift;
                    if (j >= p.limit) return -1;
                    if (row + (min(j + R, (int64_t)p.limit) - j) > a.s.num_rows) report(a.d_status, DSA_ERR_BAD_INPUT);
                    return row;
                };
                int w0 = p.i0 * nbox;
                int cur = row_of(w0 + lane), nxt = row_of(w0 + 32 + lane);
                // the computing warps' queries, on their way to L2 before those ask for them (608 x 1
                // token over 64 of 128 dims, e4m3: 86 -> 81 us; 64 dims and 8 rows: 320 -> 328, so not there)
                if ((KS == 8 || D == 128) && lane < C::kRows) {
                    const int f = p.row0 + lane, tok = f / a.group;
                    if (tok < p.q.nq) {
                        const __nv_bfloat16* src =
                            a.q + (int64_t)(p.q.q0 + tok) * a.q_stride + (int64_t)(kvh * a.group + f - tok * a.group) * D;
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
                        if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64));
                    }
                }
                w.finish(p, pos);
                const int end = min(p.i1, (p.limit + kTile - 1) / kTile);
                if (p.i0 < end) cur = seen(cur, w0 + lane);
                for (int i = p.i0; i < end && ok; ++i) {
                    const int st = c.st;
                    if (i * nbox >= w0 + 32) {
                        w0 += 32;
                        cur = seen(nxt, w0 + lane);
                        nxt = row_of(w0 + 32 + lane);
                    }
                    if (lap) {
                        ok = ptx::mbar_wait(empty + st, c.ph ^ 1u, abort_flag, a.d_status);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                    }
                    c.move(1);
                    lap = lap || c.st == 0;
                    uint8_t* kd = ring + st * C::kStage;
                    uint8_t* vd = kd + C::kHalf;
                    const int l = i * nbox - w0;  // window lane of the tile's first box
                    const uint32_t have = __ballot_sync(0xffffffffu, cur >= 0 && lane >= l && lane < l + nbox);
                    if (lane == 0) ptx::mbar_expect_tx(full + st, (uint32_t)__popc(have) * 2u * R * HB);
                    __syncwarp();
                    if ((have >> lane) & 1) {
                        const int x = lane - l;
                        constexpr int PB = HB < 128 ? HB : 128;
                        if (HB <= 128 || nbox == 1) {
                            tma_load_4d(kd + x * R * PB, &kmap, 0, cur, 0, kvh, full + st);
                            tma_load_4d(vd + x * R * PB, &vmap, 0, cur, 0, kvh, full + st);
                        } else {
                            // two 128-byte pieces, each a block of the tile's rows: a smaller box is one piece
                            for (int h = 0; h < HB / 128; ++h) {
                                tma_load_4d(kd + h * (kTile * 128) + x * R * 128, &kmap, 0, cur, h, kvh, full + st);
                                tma_load_4d(vd + h * (kTile * 128) + x * R * 128, &vmap, 0, cur, h, kvh, full + st);
                            }
                        }
                    }
                    if (FP8) {
                        float* sd = ring_scale + st * (C::kScaleBytes / 4);
#pragma unroll
                        for (int h = 0; h < kTile / 32; ++h) {
                            const int x = h * 32 + lane;
                            const int row = __shfl_sync(0xffffffffu, cur, l + (x >> shift));
                            const int64_t at = ((int64_t)row + (x & (R - 1))) * a.hkv + kvh;
                            if (row >= 0 && (int64_t)i * kTile + x < p.limit) {
                                const bool in = (int64_t)row + (x & (R - 1)) < a.s.num_rows;
                                ptx::cp_async4_or_zero(sd + x, a.k_scale + (in ? at : 0), in);
                                ptx::cp_async4_or_zero(sd + kTile + x, a.v_scale + (in ? at : 0), in);
                            }
                        }
                        ptx::cp_async_arrive_noinc(full + st);
                    }
                }
            }
            if (!ok) {
                // after an abort: let the copies in flight land before the CTA ends
                for (int st = 0; st < C::kStages; ++st)
                    if (lap || st < c.st) ptx::mbar_drain(full + st, st < c.st ? c.ph : c.ph ^ 1u);
            }
        }
        if (a.cluster > 1) {  // the computing warps' two meetings
            cluster_arrive();
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
        return;
    }

    // ---- the computing warps: key slice ks of every tile
    if (C::kSplitRegs) reg_inc<216>();
    w.init(a);
    const int ks = warp;
    const int g = lane >> 2, t = lane & 3;
    constexpr int KK = D / 16;  // k-steps of q.k, and 16-dim tiles of the output
    constexpr int NQ = C::kQShared ? 1 : NT;
    const uint32_t ring_u = smem_u32(ring), q_u = smem_u32(q_sh);
    Cursor<C::kStages> c;
    bool ok = true;
    int4 join = make_int4(0, 0, 0, 0);
    const int share = C::kRows * D / 2 / max(1, a.cluster);  // pairs of dims that a cluster's CTA joins
    int seen;
    while (w.begin(a, p, seen)) {
        had = true;
        const int kvh = p.lane % a.hkv;
        // query fragments: this thread's of row g of 8-row tile n, 2^-e of a scaled row
        auto fragments = [&](int n, uint32_t (&qf)[KK][2], float& down) {
            const int f = p.row0 + n * 8 + g;
            const int tok = f / a.group, head = f - tok * a.group;
            const bool live = tok < p.q.nq;
            const __nv_bfloat16* src =
                a.q + (int64_t)(p.q.q0 + tok) * a.q_stride + (int64_t)(kvh * a.group + head) * D;
            down = 1.f;
            if (!FP8) {
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    const uint32_t* s32 = reinterpret_cast<const uint32_t*>(src + k * 16 + 2 * t);
                    qf[k][0] = live ? __ldg(s32) : 0u;
                    qf[k][1] = live ? __ldg(s32 + 4) : 0u;
                }
            } else {
                // dims (D/4) t .. + D/4 - 1: k-step k takes 4 of them.  f16 after an
                // exact power-of-two scaling of the row to [2^14, 2^15): only values
                // 2^28 below the row's largest lose bits.
                float v[D / 4];
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(src + (D / 4) * t) + k)
                                         : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[8 * k + 2 * e] = __uint_as_float(xs[e] << 16);
                        v[8 * k + 2 * e + 1] = __uint_as_float(xs[e] & 0xFFFF0000u);
                        top = fmaxf(top, fmaxf(fabsf(v[8 * k + 2 * e]), fabsf(v[8 * k + 2 * e + 1])));
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = top > 0.f && top < INFINITY ? ilogbf(top) : 14;
                const int sh = min(14 - e, 126);  // a row below 2^-112 stays below 2^14
                const float up = __int_as_float((127 + sh) << 23);
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    qf[k][0] = pack_f16(v[4 * k] * up, v[4 * k + 1] * up);
                    qf[k][1] = pack_f16(v[4 * k + 2] * up, v[4 * k + 3] * up);
                }
                down = __int_as_float((127 - sh) << 23);
            }
        };
        uint32_t qf[NQ][KK][2];  // (loaded beside the positions)
        if (C::kQShared) {
            if (ks < NT) {
                float down;
                fragments(ks, qf[0], down);
#pragma unroll
                for (int k = 0; k < KK; ++k)
                    *reinterpret_cast<uint2*>(q_sh + (((k * (NT / 2) + (ks >> 1)) * 32 + lane) * 2 + (ks & 1)) * 8) =
                        make_uint2(qf[0][k][0], qf[0][k][1]);
                if (t == 0) fac_sh[ks * 8 + g] = down;
            }
        } else {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float down;
                fragments(n, qf[n], down);
                if (ks == 0 && t == 0) fac_sh[n * 8 + g] = down;
            }
        }
        w.finish(p, seen);
        // the rows' positions; -2: not to be written
        if (threadIdx.x < C::kRows) {
            const int f = p.row0 + (int)threadIdx.x, tok = f / a.group;
            int pos = __shfl_sync(C::kRows >= 32 ? 0xffffffffu : (1u << (C::kRows & 31)) - 1, seen, (tok - p.tok0) & 31);
            if (tok >= p.q.nq) {
                pos = -2;
            } else if (pos < -1 || pos >= p.q.ctx) {
                if (p.i0 == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
                pos = -2;
            }
            pos_sh[threadIdx.x] = pos;
            at_sh[threadIdx.x] = (int64_t)(p.q.q0 + tok) * (a.hkv * a.group) + kvh * a.group + (f - tok * a.group);
        }
        const int end = min(p.i1, (p.limit + kTile - 1) / kTile);
        bar_sync(1, 32 * KS);
        int cpos[NQ][2];
        float qfac[NQ][2];
        int minpos = 0x7FFFFFFF;
        for (int r = lane; r < C::kRows; r += 32) {
            const int pos = pos_sh[r];
            if (pos >= -1) minpos = min(minpos, pos);
        }
        minpos = __reduce_min_sync(0xffffffffu, minpos);
        if (!C::kQShared) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    cpos[n][c] = pos_sh[n * 8 + 2 * t + c];
                    qfac[n][c] = fac_sh[n * 8 + 2 * t + c];
                }
        }

        float o[NT][KK][4];
        float m[NT][2];  // references: far below any score until a key is seen
        uint64_t l[NT];  // sums of the weights, a pair of columns
        // FP8: weights take V's scales along, relative to vref, a power of two above every scale so far, times
        // 2^7: below 2^15 with the lazy reference.  f16 rounds such a product by 2^-11 of itself or 2^-25,
        // which is 2^-32 vref, and a row's largest product is at least its weight of 1 times the least scale.
        // So while vref stays below 2^span that scale, all of the slice's products that vanish in f16 are
        // together less than 2^-8 of the largest; beyond it (wide) weights are rounded to bf16 (2^-8 of
        // each), which reaches down to 2^-126 of vref.  (128 x 4 tokens over 61 to 16,381: 566 us, 1,300
        // wide; 1 x 524,288: 173 and 303.  With f16 and a power of two per row and 16 keys, 1,570, dims
        // that the row's largest product leaves 0 lost the others.)
        float vref = 0x1p-119f, vinv = 0x1p126f;
        uint32_t vlow = 0xFFFFFFFFu;  // bits of a power of two below every scale so far but 0, less 1
        bool wide = false;
        const int span = 25 - (32 - __clz(16 * max(1, p.i1 - p.i0) - 1));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = kNone;
            l[n] = 0ull;
#pragma unroll
            for (int k = 0; k < KK; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }

        for (int i = p.i0; i < end; ++i, c.move(1)) {
            ok = ok && __all_sync(0xffffffffu, quick_wait(full + c.st, c.ph, abort_flag, a.d_status));
            if (!ok) continue;  // keep to the walk, so that the slices still meet at its barriers
            const uint32_t kb = ring_u + c.st * C::kStage, vb = kb + C::kHalf;
            const int r0 = ks * 16;                // this warp's first key within the tile
            const int j0 = i * kTile + r0;         // and its position
            const bool edge = j0 + 16 > p.limit;   // rows past the last key that is seen
            if (edge) {
                // whatever lies there must not reach the products: its weights are 0, but 0 * inf is not
                uint8_t* vrow = ring + c.st * C::kStage + C::kHalf;
                for (int x = lane; x < 16 * (HB / 16); x += 32) {
                    const int row = r0 + x / (HB / 16), ch = x % (HB / 16);
                    if (i * kTile + row >= p.limit)
                        *reinterpret_cast<uint4*>(vrow + (chunk_addr<HB, kTile>(0u, row, ch))) = make_uint4(0u, 0u, 0u, 0u);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
            }
            // S^T = K Q^T: 16 keys x 8 rows per tile
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            // few tiles: two sums each, for shorter chains of products
            constexpr int N2 = NT <= 2 ? NT : 1;
            float s2[N2][4];
#pragma unroll
            for (int n = 0; n < N2; ++n) s2[n][0] = s2[n][1] = s2[n][2] = s2[n][3] = 0.f;
            auto dot = [&](int k, const uint32_t (&af)[4]) {
                if (C::kQShared) {
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t y[4];
                        lds128(y, q_u + ((k * (NT / 2) + (n >> 1)) * 32 + lane) * 16);
                        mma16816<FP8>(s[n], af, y[0], y[1]);
                        if (n + 1 < NT) mma16816<FP8>(s[n + 1], af, y[2], y[3]);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        mma16816<FP8>((k & 1) && N2 == NT ? s2[n < N2 ? n : 0] : s[n], af, qf[n][k][0], qf[n][k][1]);
                }
            };
            if (!FP8) {
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    uint32_t af[4];
                    ldsm4(af, chunk_addr<HB, kTile>(kb, r0 + (lane & 15), 2 * k + (lane >> 4)));
                    dot(k, af);
                }
            } else {
                uint32_t x0[D / 16], x1[D / 16];  // rows g and g + 8: the thread's D / 4 dims
#pragma unroll
                for (int e = 0; e < D / 64; ++e) {
                    uint32_t y[4];
                    lds128(y, chunk_addr<HB, kTile>(kb, r0 + g, (D / 64) * t + e));
                    x0[4 * e] = y[0], x0[4 * e + 1] = y[1], x0[4 * e + 2] = y[2], x0[4 * e + 3] = y[3];
                    lds128(y, chunk_addr<HB, kTile>(kb, r0 + g + 8, (D / 64) * t + e));
                    x1[4 * e] = y[0], x1[4 * e + 1] = y[1], x1[4 * e + 2] = y[2], x1[4 * e + 3] = y[3];
                }
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    uint32_t af[4];
                    e4m3x4_to_f16(x0[k], af[0], af[2]);
                    e4m3x4_to_f16(x1[k], af[1], af[3]);
                    dot(k, af);
                }
            }
            // scores in log2 units, masked: pairs of columns, keys g and g + 8
            float fk0 = 1.f, fk1 = 1.f, fv0 = 1.f, fv1 = 1.f;
            if (FP8) {
                const float* sd = ring_scale + c.st * (C::kScaleBytes / 4);
                fk0 = sd[r0 + g] * a.scale_log2, fk1 = sd[r0 + g + 8] * a.scale_log2;
                fv0 = j0 + g < p.limit ? sd[kTile + r0 + g] : 0.f;
                fv1 = j0 + g + 8 < p.limit ? sd[kTile + r0 + g + 8] : 0.f;
            }
            const uint64_t k0 = f32x2(FP8 ? fk0 : a.scale_log2, FP8 ? fk0 : a.scale_log2);
            const uint64_t k1 = f32x2(FP8 ? fk1 : a.scale_log2, FP8 ? fk1 : a.scale_log2);
            const bool masked = j0 + 15 > minpos;
            bool move = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint64_t x0 = f32x2(s[n][0], s[n][1]), x1 = f32x2(s[n][2], s[n][3]);
                if (N2 == NT) {
                    x0 = add2(x0, f32x2(s2[n < N2 ? n : 0][0], s2[n < N2 ? n : 0][1]));
                    x1 = add2(x1, f32x2(s2[n < N2 ? n : 0][2], s2[n < N2 ? n : 0][3]));
                }
                if (FP8) {
                    const uint64_t f = C::kQShared ? *reinterpret_cast<const uint64_t*>(fac_sh + n * 8 + 2 * t)
                                                   : f32x2(qfac[n < NQ ? n : 0][0], qfac[n < NQ ? n : 0][1]);
                    x0 = mul2(x0, f);
                    x1 = mul2(x1, f);
                }
                unpack2(mul2(x0, k0), s[n][0], s[n][1]);
                unpack2(mul2(x1, k1), s[n][2], s[n][3]);
                if (masked) {
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int pos = C::kQShared ? pos_sh[n * 8 + 2 * t + z] : cpos[n < NQ ? n : 0][z];
                        s[n][z] = j0 + g <= pos ? s[n][z] : -INFINITY;
                        s[n][2 + z] = j0 + g + 8 <= pos ? s[n][2 + z] : -INFINITY;
                    }
                }
#pragma unroll
                for (int z = 0; z < 2; ++z) move = move || fmaxf(s[n][z], s[n][2 + z]) > m[n][z] + kLazy;
            }
            // the bytes of two words (keys) that hold the dims of the z-th of two 16-dim tiles, a dim's side by side
            auto pick_dim = [](int z) { return z ? 0x7362u : 0x5140u; };
            auto above0 = [](float x) { return (__float_as_uint(x) & 0x7FFFFFFFu) - 1u; };  // 0: none
            if (FP8)
                move = move || fmaxf(fabsf(fv0), fabsf(fv1)) > vref || min(above0(fv0), above0(fv1)) < vlow || wide;
            if (__any_sync(0xffffffffu, move)) {
                // rare: the rows' maxima over the slice's keys, and everything relative to them
                float fv = 1.f;
                if (FP8) {
                    // a row of zeros may have any scale (1 as a rule): it has no say in the references
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        uint32_t any = 0;
#pragma unroll
                        for (int e = 0; e < D / 64; ++e) {
                            uint32_t y[4];
                            lds128(y, chunk_addr<HB, kTile>(vb, r0 + g + 8 * z, (D / 64) * t + e));
                            any |= y[0] | y[1] | y[2] | y[3];
                        }
                        any &= 0x7F7F7F7Fu;
                        any |= __shfl_xor_sync(0xffffffffu, any, 1);
                        any |= __shfl_xor_sync(0xffffffffu, any, 2);
                        float& f = z ? fv1 : fv0;
                        f = any || fabsf(f) == INFINITY ? f : 0.f;
                    }
                    const float vtop = warp_max_all(fmaxf(fabsf(fv0), fabsf(fv1)));
                    if (vtop > vref) {
                        // the next power of two (the largest finite one for an infinite scale)
                        const float nref = __uint_as_float(
                            min((__float_as_uint(vtop) & 0x7F800000u) + 0x00800000u, 0x7E800000u));
                        fv = vref * (1.f / nref);
                        vref = nref;
                        vinv = 0x1p7f / nref;
                    }
                    const uint32_t least = __reduce_min_sync(0xffffffffu, min(above0(fv0), above0(fv1)));
                    if (least < vlow) vlow = max((least + 1u) & 0x7F800000u, 1u) - 1u;
                    wide = (int)(__float_as_uint(vref) >> 23) - (int)((vlow + 1u) >> 23) > span && vlow != 0xFFFFFFFFu;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float al[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        float mx = fmaxf(s[n][z], s[n][2 + z]);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float mn = fmaxf(m[n][z], mx);
                        al[z] = mn == m[n][z] ? 1.f : fast_exp2(m[n][z] - mn);
                        m[n][z] = mn;
                    }
                    l[n] = mul2(l[n], f32x2(al[0], al[1]));
#pragma unroll
                    for (int k = 0; k < KK; ++k) {
                        o[n][k][0] *= al[0] * fv;
                        o[n][k][1] *= al[1] * fv;
                        o[n][k][2] *= al[0] * fv;
                        o[n][k][3] *= al[1] * fv;
                    }
                }
                if (FP8 && wide) {
                    // rare: the products with bf16 weights, whose exponents suffice, and bf16 codes
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float w00 = fast_exp2(s[n][0] - m[n][0]), w01 = fast_exp2(s[n][1] - m[n][1]);
                        const float w10 = fast_exp2(s[n][2] - m[n][0]), w11 = fast_exp2(s[n][3] - m[n][1]);
                        l[n] = add2(l[n], add2(f32x2(w00, w01), f32x2(w10, w11)));
                        const float u0 = fv0 * vinv, u1 = fv1 * vinv;
                        const uint32_t p0 = movm_t(pack_bf16(w00 * u0, w01 * u0));
                        const uint32_t p1 = movm_t(pack_bf16(w10 * u1, w11 * u1));
#pragma unroll
                        for (int e = 0; e < KK / 2; ++e) {
                            __syncwarp();  // keeps later loads behind these products: registers
                            uint32_t x[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const int at = (D / 8) * g + 4 * e;  // the row's byte
                                x[z] = lds32(chunk_addr<HB, kTile>(vb, r0 + 2 * t + (z & 1) + ((z >> 1) << 3), at >> 4) + (at & 15));
                            }
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                uint32_t af[4];
                                e4m3x4_to_bf16(__byte_perm(x[0], x[1], pick_dim(z)), af[0], af[1]);
                                e4m3x4_to_bf16(__byte_perm(x[2], x[3], pick_dim(z)), af[2], af[3]);
                                mma16816<false>(o[n][2 * e + z], af, p0, p1);
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = -INFINITY;  // done
                }
            }
            // weights, as the B operand of O^T = V^T P^T (two 8x8 transposes per tile)
            const uint64_t v0 = f32x2(fv0 * vinv, fv0 * vinv), v1 = f32x2(fv1 * vinv, fv1 * vinv);
            uint32_t pf[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float w00 = fast_exp2(s[n][0] - m[n][0]), w01 = fast_exp2(s[n][1] - m[n][1]);
                const float w10 = fast_exp2(s[n][2] - m[n][0]), w11 = fast_exp2(s[n][3] - m[n][1]);
                uint64_t w0 = f32x2(w00, w01), w1 = f32x2(w10, w11);
                l[n] = add2(l[n], add2(w0, w1));
                if (FP8) {
                    w0 = mul2(w0, v0);
                    w1 = mul2(w1, v1);
                }
                float x, y, u, v;
                unpack2(w0, x, y);
                unpack2(w1, u, v);
                // bf16 rounds a weight by up to 2^-8 of itself, f16 by 2^-11 or 2^-25 (see vref)
                pf[n][0] = movm_t(FP8 ? pack_f16(x, y) : pack_bf16(x, y));
                pf[n][1] = movm_t(FP8 ? pack_f16(u, v) : pack_bf16(u, v));
            }
            if (!FP8) {
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    uint32_t af[4];
                    ldsm4t(af, chunk_addr<HB, kTile>(vb, r0 + ((lane >> 4) << 3) + (lane & 7), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16816<false>(o[n][k], af, pf[n][0], pf[n][1]);
                }
            } else {
                // keys 2t, 2t+1, 2t+8, 2t+9 of the thread's D / 8 dims (D/8) g ..; a 16-dim
                // tile takes two of them: rows g and g + 8 of tile k are dims (D/8) g + 2k, + 1
                uint32_t x[4][D / 32];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int row = r0 + 2 * t + (z & 1) + ((z >> 1) << 3);
                    if (D == 128) {
                        uint32_t y[4];
                        lds128(y, chunk_addr<HB, kTile>(vb, row, g));
#pragma unroll
                        for (int e = 0; e < D / 32; ++e) x[z][e] = y[e];
                    } else {
                        uint32_t y[2];
                        lds64(y, chunk_addr<HB, kTile>(vb, row, g >> 1) + ((g & 1) << 3));
#pragma unroll
                        for (int e = 0; e < D / 32; ++e) x[z][e] = y[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < KK / 2; ++e) {
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        uint32_t af[4];
                        e4m3x4_to_f16(__byte_perm(x[0][e], x[1][e], pick_dim(z)), af[0], af[1]);
                        e4m3x4_to_f16(__byte_perm(x[2][e], x[3][e], pick_dim(z)), af[2], af[3]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816<true>(o[n][2 * e + z], af, pf[n][0], pf[n][1]);
                    }
                }
            }
            // The stage's next contents come through the async proxy: without the fence they were
            // seen to overtake this warp's reads (wrong values of a few keys of e4m3 caches, whenever
            // the loads were waited for: a different result in each of twenty runs).
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty + c.st);
        }

        if (a.cluster > 1) {
            __syncwarp();
            cluster_arrive();  // this warp reads the ring no more
        }
        // ---- the key slices meet
        {
            float x[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) unpack2(l[n], x[n][0], x[n][1]);
#pragma unroll
            for (int y = 4; y < 32; y <<= 1)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int z = 0; z < 2; ++z) x[n][z] += __shfl_xor_sync(0xffffffffu, x[n][z], y);
            if (g == 0)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int z = 0; z < 2; ++z) ml[ks * C::kRows + n * 8 + 2 * t + z] = make_float2(m[n][z], x[n][z]);
        }
        if (FP8 && lane == 0) vref_sh[ks] = vref * 0x1p-7f;
        const bool cut = !a.cluster && (p.front || p.back), shared = a.cluster > 1;
        const int64_t slot = (int64_t)blockIdx.x * 2 + (p.front ? 0 : 1);
        const int rank = shared ? blockIdx.x % a.cluster : 0;
        bar_sync(1, 32 * KS);
        // a row's reference and sum over the slices, and what each slice's outputs are multiplied by
        if (threadIdx.x < C::kRows * KS) {
            const int r = threadIdx.x / KS, y = threadIdx.x % KS;
            const float2 v = ml[y * C::kRows + r];
            float mm = v.x;
#pragma unroll
            for (int z = 1; z < KS; z <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, z));
            const float f = fast_exp2(v.x - mm);
            float sum = f * v.y;
#pragma unroll
            for (int z = 1; z < KS; z <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, z);
            ml[y * C::kRows + r].x = FP8 ? f * vref_sh[y] : f;
            if (y == 0) {
                const bool write = ok && pos_sh[r] >= -1;
                // a sum of -1: a row that is not to be written
                const float2 tot = make_float2(mm, write ? sum : -1.f);
                total[r] = tot;
                if (cut) a.part_ml[slot * C::kRows + r] = tot;
                else if (!shared && write && a.lse) a.lse[at_sh[r]] = sum == 0.f ? -INFINITY : (mm + log2f(sum)) * kLn2;
            }
        }
        bar_sync(1, 32 * KS);
        constexpr int kDims = D / (4 * KS);  // dims per thread of the sum: 8 rows x 4 KS threads
        const int hr = threadIdx.x / (4 * KS);
        const int d0 = threadIdx.x % (4 * KS) * kDims;
        if (shared) cluster_wait();  // every CTA's ring is at rest: partials may go there
        // [key slice][8 rows][D], a row's dims turned so that a warp's stores meet no bank twice
        auto turn = [](int row, int d) {  // rows 2t, 2t + 1 alike
            return FP8 ? (row >> 1) | ((d >> 5) << 2) : (row >> 1) << 3;
        };
        float4* mine = reinterpret_cast<float4*>(scratch) + (ks & 3) * (KK * 32) + lane;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int col = n * 8 + 2 * t;
            const uint64_t f = f32x2(ml[ks * C::kRows + col].x, ml[ks * C::kRows + col + 1].x);
#pragma unroll
            for (int k = 0; k < KK; ++k) {
                unpack2(mul2(f32x2(o[n][k][0], o[n][k][1]), f), o[n][k][0], o[n][k][1]);
                unpack2(mul2(f32x2(o[n][k][2], o[n][k][3]), f), o[n][k][2], o[n][k][3]);
            }
            if (KS == 8) {
                // the upper four slices hand theirs to the lower four, lane to lane
                if (ks >= 4) {
#pragma unroll
                    for (int k = 0; k < KK; ++k)
                        mine[k * 32] = make_float4(o[n][k][0], o[n][k][1], o[n][k][2], o[n][k][3]);
                }
                bar_sync(1, 32 * KS);
                if (ks < 4) {
                    float4 x[KK];
#pragma unroll
                    for (int k = 0; k < KK; ++k) x[k] = mine[k * 32];
#pragma unroll
                    for (int k = 0; k < KK; ++k) {
                        o[n][k][0] += x[k].x, o[n][k][1] += x[k].y;
                        o[n][k][2] += x[k].z, o[n][k][3] += x[k].w;
                    }
                    __syncwarp();
                }
            }
            if (ks < 4) {
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int d = FP8 ? (D / 8) * g + 2 * k + y : 16 * k + g + 8 * y;
                        float* dst = scratch + (ks * 8 + 2 * t) * D + (d ^ turn(2 * t, d));
                        dst[0] = o[n][k][2 * y];
                        dst[D] = o[n][k][2 * y + 1];
                    }
            }
            bar_sync(1, 32 * KS);
            const int r = n * 8 + hr;
            const float2 tot = total[r];
            const bool write = tot.y != -1.f;
            const float inv = tot.y == 0.f ? 0.f : 1.f / tot.y;
            __nv_bfloat16* dst = a.out + at_sh[r] * D + d0;
#pragma unroll
            for (int e = 0; e < kDims; e += 2) {
                float2 v = make_float2(0.f, 0.f);
                const int x = turn(hr, d0 + e);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float2 z =
                        *reinterpret_cast<const float2*>(scratch + (y * 8 + hr) * D + ((d0 + e) ^ (x & ~1)));
                    v.x += x & 1 ? z.y : z.x, v.y += x & 1 ? z.x : z.y;
                }
                if (cut)
                    *reinterpret_cast<float2*>(a.part_o + (slot * C::kRows + r) * D + d0 + e) = v;
                else if (shared) {
                    // pair x of the rows' dims belongs to CTA x / share, which gets it from every rank;
                    // the first pair of a row, or of a share, brings the row's reference and sum
                    const int pair = (r * D + d0 + e) >> 1;
                    const int own = pair / share, at2 = pair % share;
                    st_cluster(ring_u + (rank * share + at2) * 8, own, v);
                    if (at2 % min(share, D / 2) == 0)
                        st_cluster(ring_u + C::kRows * D * 4 + (rank * C::kRows + r) * 8, own, tot);
                } else if (write)
                    *reinterpret_cast<uint32_t*>(dst + e) = pack_row(v.x, v.y, inv);
            }
            bar_sync(1, 32 * KS);
        }
        // the first CTA behind a cut tells the joining kernel what to join
        if (p.front && !a.cluster) {
            const int c = blockIdx.x / a.hl;
            const int64_t s0 = w.r0 - p.i0, s1 = s0 + tiles_of<kTile>(p.q);
            if (s0 >= w.deal.first(c - 1)) join = make_int4(w.deal.owner(s1 - 1) - c + 2, p.q.q0, p.q.nq, p.lane);
        }
    }
    if (threadIdx.x == 0 && !a.cluster) a.desc[blockIdx.x] = join;
    if (a.cluster <= 1) return;

    // ---- a cluster's partials meet: every CTA joins its share of the rows' dims,
    // in the order of the ranks
    if (!had) {  // the same in all of the cluster's CTAs
        cluster_arrive();
        cluster_wait();
    }
    cluster_arrive();
    cluster_wait();
    if (!had) return;
    const int rank = blockIdx.x % a.cluster;
    for (int y = threadIdx.x; y < share; y += 32 * KS) {
        const int pair = rank * share + y;
        const int r = pair / (D / 2), d0 = pair % (D / 2) * 2;
        const float2* from = reinterpret_cast<const float2*>(ring) + y;
        const float2* from_ml = reinterpret_cast<const float2*>(ring + C::kRows * D * 4) + r;
        float top = kNone;
        bool write = true;
        for (int z = 0; z < a.cluster; ++z) {
            const float2 v = from_ml[z * C::kRows];
            top = fmaxf(top, v.x);
            write = write && v.y != -1.f;
        }
        float sum = 0.f;
        float2 acc = make_float2(0.f, 0.f);
        for (int z = 0; z < a.cluster; ++z) {
            const float2 v = from_ml[z * C::kRows], q = from[z * share];
            const float f = fast_exp2(v.x - top);
            sum = fmaf(f, v.y, sum);
            acc.x = fmaf(f, q.x, acc.x);
            acc.y = fmaf(f, q.y, acc.y);
        }
        if (!write) continue;
        const int f = p.row0 + r;
        const int tok = f / a.group, head = f - tok * a.group;
        const int64_t at = (int64_t)(p.q.q0 + tok) * (a.hkv * a.group) + p.lane % a.hkv * a.group + head;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint32_t*>(a.out + at * D + d0) = pack_row(acc.x, acc.y, inv);
        if (d0 == 0 && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

// Joins the partials of one cut (lane, sequence), a CTA per row: its four
// warps take every fourth part.  Weights 2^(m_i - M), in the parts' order.
constexpr int kJoinParts = 2 * kPlanSms + 8;  // parts of one sequence: at most the CTAs of a lane column

template <int D>
__global__ void __launch_bounds__(128) gqa_join_kernel(const __grid_constant__ Args a, int rows) {
    __shared__ float weight[kJoinParts];
    __shared__ float red[4][D];
    __shared__ float sums[4], tops[4];
    pdl_enter();
    const int r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int4 d = a.desc[blockIdx.x];
    const int n = d.x;
    if (n == 0) return;
    const int f = d.w / a.hkv * rows + r;
    const int tok = f / a.group, head = f - tok * a.group;
    if (tok >= d.z) return;
    // part i: CTA blockIdx.x + (i - 1) hl; the first one's sequence is cut behind it, the others' before
    auto slot = [&](int i) -> int64_t {
        return ((int64_t)blockIdx.x + (int64_t)(i - 1) * a.hl) * 2 + (i == 0 ? 1 : 0);
    };
    constexpr int E = D / 32;
    constexpr int kFly = 8;  // loads in flight
    auto load = [&](int i0, float4 (&x)[kFly]) {
#pragma unroll
        for (int y = 0; y < kFly; ++y) {
            const int i = i0 + 4 * y;
            x[y] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n) {
                const float* src = a.part_o + (slot(i) * rows + r) * D + lane * E;
                if (E == 4) {
                    x[y] = __ldcg(reinterpret_cast<const float4*>(src));
                } else {
                    const float2 z = __ldcg(reinterpret_cast<const float2*>(src));
                    x[y].x = z.x, x[y].y = z.y;
                }
            }
        }
    };
    float2 v[(kJoinParts + 127) / 128];
#pragma unroll
    for (int k = 0; k < (kJoinParts + 127) / 128; ++k) {
        const int i = k * 128 + threadIdx.x;
        v[k] = i < n ? a.part_ml[slot(i) * rows + r] : make_float2(kNone, 0.f);
    }
    float4 x[kFly];
    load(warp, x);  // beside the references and sums
    float top = kNone;
    bool skip = false;
#pragma unroll
    for (int k = 0; k < (kJoinParts + 127) / 128; ++k) {
        skip = skip || v[k].y == -1.f;
        top = fmaxf(top, v[k].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) tops[warp] = top;
    if (__syncthreads_or(skip)) return;
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < (kJoinParts + 127) / 128; ++k) {
        const int i = k * 128 + threadIdx.x;
        const float w = fast_exp2(v[k].x - top);
        if (i < n) weight[i] = w;
        sum = fmaf(w, v[k].y, sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int i0 = warp; i0 < n; i0 += 4 * kFly) {
        if (i0 != warp) load(i0, x);
#pragma unroll
        for (int y = 0; y < kFly; ++y) {
            const int i = i0 + 4 * y;
            const float w = i < n ? weight[i] : 0.f;
            acc[0] = fmaf(w, x[y].x, acc[0]);
            acc[1] = fmaf(w, x[y].y, acc[1]);
            if (E == 4) {
                acc[E - 2] = fmaf(w, x[y].z, acc[E - 2]);
                acc[E - 1] = fmaf(w, x[y].w, acc[E - 1]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) red[warp][lane * E + e] = acc[e];
    __syncthreads();
    const int64_t at = (int64_t)(d.y + tok) * (a.hkv * a.group) + d.w % a.hkv * a.group + head;
    if (threadIdx.x < D / 2) {
        const int e = 2 * threadIdx.x;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float x0 = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
        const float x1 = (red[0][e + 1] + red[1][e + 1]) + (red[2][e + 1] + red[3][e + 1]);
        reinterpret_cast<uint32_t*>(a.out + at * D)[threadIdx.x] = pack_row(x0, x1, inv);
    }
    if (a.lse && threadIdx.x == 0) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// ---------------------------------------------------------------------------
// host side
struct Plan {
    int nt, tile, rows, chunks, lanes, hl, parts, grid, cluster;
    size_t o_bytes, ml_bytes, desc_bytes;
};

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

Plan make_plan(const dsa_gqa_shape& sh, const dsa_seqs& s) {
    Plan p;
    const int group = sh.num_heads / sh.num_kv_heads;
    const int64_t rows = (int64_t)s.max_q_per_seq * group;
    // 8, 16 or 32 query rows a chunk; more than 8 take a CTA of eight computing
    // warps with an SM to itself (their accumulators need the registers)
    p.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    p.rows = 8 * p.nt;
    p.tile = p.nt == 1 ? 64 : 128;
    p.chunks = (int)((rows + p.rows - 1) / p.rows);
    p.lanes = sh.num_kv_heads * p.chunks;
    const int n = kPlanSms * (p.nt == 1 ? 2 : 1);
    const int64_t tiles = std::max<int64_t>(1, ((int64_t)s.max_ctx + p.tile - 1) / p.tile);
    // Clusters where all (lane, sequence)s fit at once and an estimate from the
    // longest sequence says that they are faster: a CTA takes at least tile_ns a
    // tile (latency), all together no less than the bytes at 6.8 TB/s, and the
    // joining kernel join_ns.  Larger clusters leave room: their CTAs have to
    // find place in one part of the GPU.  Clusters against the joining kernel,
    // launch included (64/8 heads of 128, one token, bf16 where not said): 8 x 8,192
    // 47.7 us and 53.3; 16 x 4,096 48.4 and 54.2; 32 x 8,192 156.7 and 167.5, e4m3
    // 92.7 and 100; four tokens over e4m3, 2 x 4,000 22.8 and 24.4, 19 x 4,000 50.5
    // and 57.5; level at 4 x 65,536, 165 and 164; and where the estimate chooses the
    // other: 3 x 30,000 70.8 and 66.7, 3 x up to 9,000 with 32/8 heads of 64 18.7 and 15.1.
    p.cluster = 0;
    const int64_t segs = (int64_t)p.lanes * s.num_seqs;
    if (segs <= n) {
        int c = 1;
        auto room = [&](int size) { return size >= 16 ? n / 2 : size >= 8 ? n * 5 / 8 : n * 7 / 8; };
        while (c < kMaxCluster && segs * 2 * c <= room(2 * c) && 2 * c <= tiles) c *= 2;
        const int64_t tile_ns = p.tile == 64 ? 600 : 1200, join_ns = p.nt == 1 ? 4000 : p.nt == 2 ? 6000 : 8000;
        const int64_t bytes = (int64_t)2 * p.tile * sh.head_dim * (sh.kv_dtype == DSA_BF16 ? 2 : 1);
        const int64_t with = (tiles + c - 1) / c * std::max(tile_ns, segs * c * bytes / 6800);
        const int64_t without = std::max(segs * tiles * bytes / 6800, segs * tiles * tile_ns / n) + join_ns;
        if (with <= without) {
            p.cluster = c;
            p.grid = (int)segs * c;
            p.hl = p.parts = 1;  // not used
            p.o_bytes = p.ml_bytes = p.desc_bytes = 0;
            return p;
        }
    }
    // lanes side by side: a divisor of the lanes that leaves few CTAs idle, the
    // largest such (its lanes' rows are neighbours in memory)
    int best = 0;
    p.hl = p.lanes;
    if (p.lanes > n || n / p.lanes * p.lanes * 32 < n * 31)
        for (int d = 1; d <= p.lanes && d <= n; ++d)
            if (p.lanes % d == 0) {
                const int used = n / d * d;
                if (used * 32 >= best * 31) p.hl = d;
                best = std::max(best, used);
            }
    p.parts = (int)std::min<int64_t>(n / p.hl, (int64_t)(p.lanes / p.hl) * s.num_seqs * tiles);
    p.grid = p.parts * p.hl;
    const size_t slots = (size_t)2 * p.grid;
    p.o_bytes = up256(slots * p.rows * sh.head_dim * 4);
    p.ml_bytes = up256(slots * p.rows * 8);
    p.desc_bytes = up256((size_t)p.grid * 16);
    return p;
}

template <int D, bool FP8, int NT, int KS>
cudaError_t launch_one(const CUtensorMap& km, const CUtensorMap& vm, const Args& a, int grid, cudaStream_t stream) {
    using C = Cfg<D, FP8, NT, KS>;
    auto kern = gqa_decode_kernel<D, FP8, NT, KS>;
    static OncePerDevice once;
    const cudaError_t e = once.run([&] {
        const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        return r != cudaSuccess ? r : cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(C::kThreads), C::kSmem, stream, a.cluster, km, vm, a);
}

}  // namespace

// For any call: two partials of 8, 16 or 32 rows per CTA, of two CTAs per SM with 8.
size_t decode_workspace(const dsa_gqa_shape& sh) {
    const size_t rows = (size_t)2 * kPlanSms * 32;
    return up256(rows * sh.head_dim * 4) + up256(rows * 8) + up256((size_t)2 * kPlanSms * 16);
}

cudaError_t launch_decode(const dsa_gqa_shape& sh, const void* q, const void* k, const void* v, const float* k_scale,
                          const float* v_scale, const dsa_seqs& s, int num_q, float sm_scale, void* out, float* lse,
                          void* workspace, int32_t* d_status, cudaStream_t stream) {
    const Plan p = make_plan(sh, s);
    const bool fp8 = sh.kv_dtype == DSA_FP8_E4M3_ROWSCALE;
    const int box = s.page_table ? std::min(s.page_size, p.tile) : p.tile;
    CUtensorMap km, vm;
    cudaError_t e = cache_map(&km, fp8, k, sh.num_kv_heads, sh.head_dim, sh.k_stride, s.num_rows, box, box == p.tile);
    if (e == cudaSuccess)
        e = cache_map(&vm, fp8, v, sh.num_kv_heads, sh.head_dim, sh.v_stride, s.num_rows, box, box == p.tile);
    if (e != cudaSuccess) return e;
    Args a;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    a.part_o = reinterpret_cast<float*>(w);
    a.part_ml = reinterpret_cast<float2*>(w + p.o_bytes);
    a.desc = reinterpret_cast<int4*>(w + p.o_bytes + p.ml_bytes);
    a.s = s;
    a.q_stride = sh.q_stride;
    a.d_status = d_status;
    a.scale_log2 = sm_scale * 1.4426950408889634f;
    a.num_q = num_q;
    a.group = sh.num_heads / sh.num_kv_heads;
    a.hkv = sh.num_kv_heads;
    a.lanes = p.lanes;
    a.hl = p.hl;
    a.parts = p.parts;
    a.cluster = p.cluster;
    auto by_rows = [&](auto d, auto f8) {
        constexpr int D = decltype(d)::value;
        constexpr bool F = decltype(f8)::value;
        return p.nt == 4   ? launch_one<D, F, 4, 8>(km, vm, a, p.grid, stream)
               : p.nt == 2 ? launch_one<D, F, 2, 8>(km, vm, a, p.grid, stream)
                           : launch_one<D, F, 1, 4>(km, vm, a, p.grid, stream);
    };
    using std::integral_constant;
    if (sh.head_dim == 64)
        e = fp8 ? by_rows(integral_constant<int, 64>(), std::true_type())
                : by_rows(integral_constant<int, 64>(), std::false_type());
    else
        e = fp8 ? by_rows(integral_constant<int, 128>(), std::true_type())
                : by_rows(integral_constant<int, 128>(), std::false_type());
    if (e != cudaSuccess || p.cluster || p.parts == 1) return e;
    auto join = sh.head_dim == 64 ? gqa_join_kernel<64> : gqa_join_kernel<128>;
    return launch_pdl(join, dim3(p.grid, p.rows), dim3(128), 0, stream, 1, a, p.rows);
}

}  // namespace gqa
}  // namespace dsa
