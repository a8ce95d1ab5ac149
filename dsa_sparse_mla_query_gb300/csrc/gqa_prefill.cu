// gqa_prefill.cu -- dense causal attention of whole prompts with grouped heads
// over packed or paged sequences (sm_103a, tcgen05).
//
//   s_j = sm_scale * q_h . k_j,  p = softmax over j <= pos,  out = sum_j p_j v_j
//
// A 128-row tile holds 128 / G tokens x the G query heads of one key head, so
// that every key and value tile is read once for the whole group, and a
// prompt of few tokens still fills its rows.  An item is two such tiles; both
// run over the same keys, 64 at a time:
//   S = Q K^T (tcgen05, Q and K by TMA in shared memory, S in TMEM),
//   one pass with a running reference m and sum l per row (a thread per row):
//   p = 2^(x - m), the weights below 2^8 because O is rescaled only when a
//   row's maximum passes m by more than 8,
//   O += P V (P from TMEM as bf16, V in shared memory, O in TMEM).
// Bound by the tensor cores: 4 D flop a visible (query, key) pair.  A thread's
// softmax of a step is a chain far longer than the step's products (TMEM load,
// maximum, exponentials, TMEM store and two hand-overs), so each tile has two
// buffers of S: the scores of step j + 1 are made while step j's weights are
// computed, and the products wait for neither.  (Steps of 128 keys with one
// buffer: the two tiles' chains alone left the tensor cores idle half the
// time, 1,083 TFLOP/s on 16,384 tokens, 64/8 heads of 128.)
//
// Roles (one CTA per SM, persistent): two warpgroups of softmax (one per tile,
// each also writes its tile's output), four warps that issue the products (a
// tile's scores, its outputs), and one warp each that loads, clears the rows
// behind the last key, and walks the items.  Items go longest first, dealt to
// the CTAs in turn, back and forth.  Where few items leave CTAs idle, each is
// split into ranges of keys, whose partial results a second kernel joins.
//
// Measured, 64/8 heads of 128, bf16: 16,384 tokens 1,540 to 1,590 TFLOP/s (the
// chip at its power cap, as a library matrix product is at 1,700 sustained), a
// step 1,340 cycles of the 1,280 that its products take; 24 packed prompts of 17 to
// 4,095 tokens 1,200 to 1,240, where an item's start and end are 4,000 cycles of
// 30,000 to 90,000.
#include "gqa_common.cuh"

namespace dsa {
namespace gqa {
namespace {

constexpr int kTagPrefill = 7;
constexpr int kKeys = 128;  // keys per stage of the ring
constexpr int kStep = 64;   // keys per step of the products
constexpr int kIssueWarp = 8, kLoadWarp = 12, kClearWarp = 13, kWalkWarp = 14;  // then an idle one
constexpr int kConvertWarp = 16, kConverters = 8;  // e4m3 caches only
constexpr float kLazy = 8.f;  // a row's reference moves when its maximum passes it by 2^8
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kItemSlots = 2;

template <int D, bool FP8>
struct Cfg {
    static constexpr int kThreads = FP8 ? 768 : 512;
    // registers per thread of the softmax warpgroups and of the others, which
    // together take what the CTA is launched with
    static constexpr int kSoftRegs = FP8 ? 144 : 192, kOtherRegs = FP8 ? 48 : 64;
    // warps that read an item: softmax, issuers, loader, and the clearer or the converters
    static constexpr int kItemReaders = 13 + (FP8 ? kConverters : 1);
    static constexpr int kHalves = D / 64;                   // 128-byte pieces of a head row
    static constexpr int kQTile = 128 * D * 2;               // bytes
    static constexpr int kStage = kKeys * D * 2;             // a K or a V tile
    static constexpr int kStages = FP8 ? (D == 128 ? 3 : 5) : (D == 128 ? 4 : 8);  // (five and ten bf16: no faster)
    // e4m3: tiles as they are in the cache, before their conversion, and the scales of
    // a stage's keys.  Those of stage i + slots are written once the values
    // of stage i have been used: by then no softmax reads the scales of stage i.
    static constexpr int kCodeStage = FP8 ? kKeys * D : 0;
    static constexpr int kScaleSlots = (kStages + 2) / 2;
    static constexpr int kScaleBytes = FP8 ? (kScaleSlots + 1) * 2 * kKeys * 4 : 0;  // and those beside the codes
    // outputs leave through shared memory: so many dims of a warp's 32 rows at a time
    static constexpr int kOutDims = FP8 ? 32 : 64;
    static constexpr int kOutWarp = 32 * kOutDims * 2;
    static constexpr int kSmem = 2 * kQTile + kStages * kStage + 2 * kCodeStage + 8 * kOutWarp + kScaleBytes + 1024;
    static_assert(kSmem <= 232448, "a CTA's shared memory");
    // TMEM columns: two buffers of S per tile, then O; P takes the place of its S
    static constexpr uint32_t kO = 256;
    static constexpr uint32_t s_col(int x, int buf) { return x * 128 + buf * kStep; }
};

struct Item {
    int n;       // stages of keys (0: no key is seen; -1: no more items)
    int key0;    // the first stage's first key
    int limit;   // keys that some query sees, up to the last stage's end
    int steps[2];// steps of either tile (0: the tile sees no key, or has no query)
    int part;    // which of the key ranges that the call is split into
    int b, kvh;
    int q0;      // first query row
    int ntok;    // tokens from there to the sequence's end (may exceed the item)
    int ctx;
    int64_t base;
};

struct Args {
    __nv_bfloat16* out;
    float* lse;
    dsa_seqs s;
    int32_t* d_status;
    float scale_log2;  // > 0: masked scores are -inf before they are scaled
    int32_t num_q, group, hkv, tpt;  // tpt: tokens per tile
    int32_t splits;   // key ranges per item; more than one: partial results
    const float *k_scale, *v_scale;  // e4m3: [rows >> scale_shift][hkv]
    int32_t scale_shift;
    float* part_o;    // [splits][num_q heads][D]
    float2* part_ml;  // [splits][num_q heads]
};

// Shared-memory matrix descriptors as a low word, which holds the address and
// the leading stride, and the high word they share (8-row groups 1024 bytes
// apart, 128-byte swizzle)
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
    return ((addr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}
__device__ __forceinline__ uint64_t make_desc(uint32_t lo) {
    constexpr uint64_t hi = (uint64_t)(1024 >> 4) | ((uint64_t)1 << 14) | ((uint64_t)2 << 29);
    return (hi << 32) | lo;
}
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}

// Walks the items of this CTA, longest first: item y of the order is the one
// with the y-th largest level, level = item index within the sequence plus the
// items' worth of tokens before its first query.  With more sequences than a
// warp holds in registers, the search for a level would take longer than an
// item: there the order is that of the sequences, each one's longest first, and
// the walk goes through them once.  Whole warp.
struct Schedule {
    static constexpr int kKept = 4;  // sequences per lane held in registers
    int n[kKept], p[kKept];
    int64_t total;
    int top;
    int group;       // many sequences: the 32 that the walk has come to,
    int64_t before;  // and the items before them
    __device__ __forceinline__ void get(const Args& a, int b, int& nn, int& pp, bool report_errors) const {
        nn = pp = 0;
        if (b >= a.s.num_seqs) return;
        const Seq q = load_seq(a.s, b, a.num_q);
        if (!q.ok) {
            if (report_errors) report(a.d_status, DSA_ERR_BAD_INPUT);
            return;
        }
        const int per = 2 * a.tpt;
        nn = (q.nq + per - 1) / per;
        pp = nn ? max(q.ctx - q.nq, 0) / per : 0;
    }
    __device__ __forceinline__ void pair(const Args& a, int g, int& nn, int& pp) const {
        if (g >= kKept) {
            get(a, g * 32 + (threadIdx.x & 31), nn, pp, false);
            return;
        }
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            if (g == k) nn = n[k], pp = p[k];
    }
    // items at this level or above
    __device__ __forceinline__ int64_t above(const Args& a, int level) const {
        int64_t c = 0;
        for (int g = 0; g * 32 < a.s.num_seqs; ++g) {
            int nn = 0, pp = 0;
            pair(a, g, nn, pp);
            c += __reduce_add_sync(0xffffffffu, (unsigned)min(max(nn + pp - level, 0), nn));
        }
        return c;
    }
    __device__ __forceinline__ void init(const Args& a) {
        const int lane = threadIdx.x & 31;
        int t = 0;
        for (int g = 0; g * 32 < a.s.num_seqs; ++g) {
            int nn, pp;
            get(a, g * 32 + lane, nn, pp, blockIdx.x == 0);
#pragma unroll
            for (int k = 0; k < kKept; ++k)
                if (g == k) n[k] = nn, p[k] = pp;
            t = max(t, nn + pp);
        }
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            if (k * 32 >= a.s.num_seqs) n[k] = p[k] = 0;
        top = __reduce_max_sync(0xffffffffu, t);
        group = 0;
        before = 0;
        total = above(a, 0) * a.hkv * a.splits;
    }
    // item f of the order (f < total)
    __device__ __forceinline__ Item find(const Args& a, int64_t f) {
        const int lane = threadIdx.x & 31;
        int part = 0;
        if (a.splits > 1) {
            part = (int)(f % a.splits);
            f /= a.splits;
        }
        const int64_t y = f <= 0x7FFFFFFF ? (int64_t)((uint32_t)f / (uint32_t)a.hkv) : f / a.hkv;
        Item it;
        it.kvh = (int)(f - y * a.hkv);
        it.b = 0;
        int tile = 0;
        if (a.s.num_seqs <= 32 * kKept) {
            int lo = 0, hi = top - 1;  // the largest level with above(level) > y
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (above(a, mid) > y) lo = mid; else hi = mid - 1;
            }
            int64_t z = y - above(a, lo + 1);  // place among the level's items
            for (int g = 0; g * 32 < a.s.num_seqs; ++g) {
                int nn = 0, pp = 0;
                pair(a, g, nn, pp);
                const bool in = pp <= lo && lo < pp + nn;
                const uint32_t m = __ballot_sync(0xffffffffu, in);
                if (z < __popc(m)) {
                    const int l =
                        __ffs(__ballot_sync(0xffffffffu, in && __popc(m & ((1u << lane) - 1)) == (int)z)) - 1;
                    it.b = g * 32 + l;
                    tile = lo - __shfl_sync(0xffffffffu, pp, l);
                    break;
                }
                z -= __popc(m);
            }
        } else {
            for (;; ++group) {  // y only grows from call to call
                int nn = 0, pp = 0;
                get(a, group * 32 + lane, nn, pp, false);
                int in = nn;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, in, o);
                    if (lane >= o) in += v;
                }
                const int z = (int)(y - before);  // place among the group's items
                const uint32_t m = __ballot_sync(0xffffffffu, z < in);
                if (m) {
                    const int l = __ffs(m) - 1;
                    it.b = group * 32 + l;
                    tile = __shfl_sync(0xffffffffu, in, l) - 1 - z;
                    break;
                }
                before += __shfl_sync(0xffffffffu, in, 31);
                if (group * 32 >= a.s.num_seqs) break;  // (not reached: y < total)
            }
        }
        const Seq q = load_seq(a.s, it.b, a.num_q);
        const int tok = tile * 2 * a.tpt;
        it.q0 = q.q0 + tok;
        it.ntok = q.nq - tok;
        it.ctx = q.ctx;
        it.base = a.s.page_table ? 0 : __ldg(a.s.seq_base + it.b);
        int pos[2] = {-1, -1};
        for (int i = lane; i < min(2 * a.tpt, it.ntok); i += 32) {
            const int x = __ldg(a.s.q_pos + it.q0 + i);
            if (x < q.ctx) {
                if (i < a.tpt) pos[0] = max(pos[0], x);
                else pos[1] = max(pos[1], x);
            }
        }
        it.limit = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int lim = max(0, __reduce_max_sync(0xffffffffu, pos[x]) + 1);
            it.steps[x] = (lim + kStep - 1) / kStep;
            it.limit = max(it.limit, lim);
        }
        it.n = (it.limit + kKeys - 1) / kKeys;
        it.key0 = 0;
        it.part = part;
        if (a.splits > 1) {
            const int first = (int)((int64_t)it.n * part / a.splits), last = (int)((int64_t)it.n * (part + 1) / a.splits);
            it.n = last - first;
            it.key0 = first * kKeys;
            it.limit = min(it.limit, last * kKeys);
#pragma unroll
            for (int x = 0; x < 2; ++x)
                it.steps[x] = min(max(it.steps[x] - first * (kKeys / kStep), 0), it.n * (kKeys / kStep));
        }
        return it;
    }
};

struct Shared {
    Item item[kItemSlots];
    uint64_t item_full[kItemSlots], item_empty[kItemSlots];
    uint64_t q_full[2], q_empty[2];
    uint64_t kv_full[10], kv_empty[10], tail_full[10], c_full[2], c_empty[2];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], o_full[2], o_empty[2];
    uint64_t drain[4];
    int abort_flag[2];
    uint32_t tmem;
};
static_assert(sizeof(Shared) <= 1024, "the barriers' page");

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads, 1)
    gqa_prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a) {
    using C = Cfg<D, FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* qs = smem;
    uint8_t* ring = smem + 2 * C::kQTile;
    uint8_t* codes = ring + C::kStages * C::kStage;
    uint8_t* stage_out = codes + 2 * C::kCodeStage;
    float* scales = reinterpret_cast<float*>(stage_out + 8 * C::kOutWarp);  // [slot][keys', values'][kKeys]
    float* code_scales = scales + C::kScaleSlots * 2 * kKeys;               // [keys', values'][kKeys]
    Shared& sh = *reinterpret_cast<Shared*>(stage_out + 8 * C::kOutWarp + C::kScaleBytes);
    volatile int* abort_flag = sh.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 8) {
        ptx::tmem_alloc(&sh.tmem, 512);
        ptx::tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kItemSlots; ++i) {
            ptx::mbar_init(sh.item_full + i, 1);
            ptx::mbar_init(sh.item_empty + i, C::kItemReaders);
        }
        for (int i = 0; i < C::kStages; ++i) {
            ptx::mbar_init(sh.kv_full + i, FP8 ? kConverters : 1);
            ptx::mbar_init(sh.kv_empty + i, 2);
            ptx::mbar_init(sh.tail_full + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(sh.c_full + i, 33);  // the codes' bytes, and every lane's scales
            ptx::mbar_init(sh.c_empty + i, kConverters);
        }
        for (int x = 0; x < 2; ++x) {
            ptx::mbar_init(sh.q_full + x, 1);
            ptx::mbar_init(sh.q_empty + x, 1);
            for (int b = 0; b < 2; ++b) {
                ptx::mbar_init(&sh.s_full[x][b], 1);
                ptx::mbar_init(&sh.p_full[x][b], 4);
                ptx::mbar_init(&sh.pv_done[x][b], 1);
            }
            ptx::mbar_init(sh.o_full + x, 1);
            ptx::mbar_init(sh.o_empty + x, 4);
        }
        for (int i = 0; i < 4; ++i) ptx::mbar_init(sh.drain + i, 1);
        abort_flag[0] = 0;
        abort_flag[1] = kTagPrefill;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&qmap);
        ptx::prefetch_tmap(&kmap);
        ptx::prefetch_tmap(&vmap);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);
    pdl_enter();

    auto wait = [&](uint64_t* bar, uint32_t parity) { return quick_wait(bar, parity & 1, abort_flag, a.d_status); };
    // the next item, read by a whole warp; false at the end or after an abort
    int item_no = 0;
    auto next_item = [&](Item& it) -> bool {
        const int sl = item_no % kItemSlots;
        const bool ok = wait(sh.item_full + sl, item_no / kItemSlots);
        if (!__all_sync(0xffffffffu, ok)) return false;
        it = sh.item[sl];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(sh.item_empty + sl);
        ++item_no;
        return it.n >= 0;
    };

    if (warp >= 8) {
        reg_dec<C::kOtherRegs>();
        if (warp == kWalkWarp) {
            // ------------------------------------------------------------ walks the items
            Schedule sc;
            sc.init(a);
            bool ok = true;
            int64_t k = 0;
            for (;; ++k) {
                const int64_t f = k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                Item it;
                it.n = -1;
                if (f < sc.total) it = sc.find(a, f);
                const int sl = (int)(k % kItemSlots);
                if (k >= kItemSlots) {
                    ok = wait(sh.item_empty + sl, (uint32_t)(k / kItemSlots) - 1);
                    if (!__all_sync(0xffffffffu, ok)) break;
                }
                if (lane == 0) {
                    sh.item[sl] = it;
                    ptx::mbar_arrive(sh.item_full + sl);
                }
                __syncwarp();
                if (it.n < 0) break;  // every later round's item lies past the end too
            }
        } else if (!FP8 && warp == kClearWarp) {
            // ------------------------------------------------------------ clears V's rows behind the last key
            // whatever lies there must not reach the products: its weights are 0, but 0 * inf is not
            Item it;
            uint32_t phases = 0;
            int c = 0;  // the item's first stage
            while (next_item(it)) {
                if (it.n > 0 && it.limit % kKeys) {
                    const int st = (c + 2 * it.n - 1) % C::kStages;
                    const bool ok = wait(sh.tail_full + st, (phases >> st) & 1);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    phases ^= 1u << st;
                    const int r0 = it.limit % kKeys;
                    for (int h = 0; h < C::kHalves; ++h) {
                        uint4* dst = reinterpret_cast<uint4*>(ring + st * C::kStage + h * (kKeys * 128));
                        for (int i = r0 * 8 + lane; i < kKeys * 8; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(sh.kv_full + st);
                }
                c = (c + 2 * it.n) % C::kStages;
            }
        } else if (warp == kLoadWarp) {
            // ------------------------------------------------------------ loads
            const int R = a.s.page_table ? min(a.s.page_size, kKeys) : kKeys;  // rows per box
            const int nbox = kKeys / R;
            const int shift = 31 - __clz(R);
            Item it;
            constexpr int N = FP8 ? 2 : C::kStages;  // e4m3: into the code stages
            Cursor<N> c;
            bool lap = false;      // every stage has been used
            int uses[2] = {0, 0};  // Q loads per tile
            bool ok = true;
            uint32_t tails = 0;    // stages whose last load goes to tail_full
            uint32_t tail_phase = 0;
            while (ok && next_item(it)) {
                if (it.n == 0) continue;
                // physical row of a box's first token, -1 for a box that no query sees.  Rows outside the cache
                // are loaded as zeros (TMA's fill) and reported.
                auto row_of = [&](int box) -> int {
                    const int64_t j = (int64_t)box << shift;
                    if (j >= it.limit) return -1;
                    int64_t row = a.s.page_table ? phys_row(a.s, it.b, j) : it.base + j;
                    if (row < 0 || row >= a.s.num_rows) row = a.s.num_rows;
                    if (row + (min(j + R, (int64_t)it.limit) - j) > a.s.num_rows) report(a.d_status, DSA_ERR_BAD_INPUT);
                    return (int)row;
                };
                const int b0 = it.key0 >> shift;  // the item's first box
                int w0 = b0;
                int cur = row_of(w0 + lane), nxt = row_of(w0 + 32 + lane);
                auto load = [&](const CUtensorMap* map, int i, bool tail) -> bool {
                    const int st = c.st;
                    if (lap) {
                        const bool free = wait((FP8 ? sh.c_empty : sh.kv_empty) + st, c.ph ^ 1u);
                        if (!__all_sync(0xffffffffu, free)) return false;
                    }
                    c.move(1);
                    lap = lap || c.st == 0;
                    uint64_t* bar = FP8 ? sh.c_full + st : tail ? sh.tail_full + st : sh.kv_full + st;
                    if (tail) tails |= 1u << st, tail_phase ^= 1u << st;
                    else tails &= ~(1u << st);
                    const int l = b0 + i * nbox - w0;
                    const uint32_t have = __ballot_sync(0xffffffffu, cur >= 0 && lane >= l && lane < l + nbox);
                    if (lane == 0) ptx::mbar_expect_tx(bar, (uint32_t)__popc(have) * R * D * (FP8 ? 1 : 2));
                    __syncwarp();
                    if ((have >> lane) & 1) {
                        constexpr int PB = FP8 && D == 64 ? 64 : 128;  // bytes of a row's piece
                        uint8_t* dst = (FP8 ? codes + st * C::kCodeStage : ring + st * C::kStage) + (lane - l) * R * PB;
                        if (FP8 || C::kHalves == 1 || nbox == 1)
                            tma_load_4d(dst, map, 0, cur, 0, it.kvh, bar);
                        else
                            for (int h = 0; h < C::kHalves; ++h)
                                tma_load_4d(dst + h * (kKeys * 128), map, 0, cur, h, it.kvh, bar);
                    }
                    if (FP8) {
                        // both scales come with the keys: the weights take the values' before the values' turn
                        if (map == &kmap)
#pragma unroll
                            for (int y = 0; y < kKeys / 32; ++y) {
                                const int key = y * 32 + lane;
                                const int row = __shfl_sync(0xffffffffu, cur, l + (key >> shift));
                                if (row >= 0 && it.key0 + i * kKeys + key < it.limit) {
                                    const int64_t at = (int64_t)row + (key & (R - 1));
                                    const bool in = at < a.s.num_rows;
                                    const int64_t off = in ? (at >> a.scale_shift) * a.hkv + it.kvh : 0;
                                    ptx::cp_async4_or_zero(code_scales + key, a.k_scale + off, in);
                                    ptx::cp_async4_or_zero(code_scales + kKeys + key, a.v_scale + off, in);
                                }
                            }
                        ptx::cp_async_arrive_noinc(bar);
                    }
                    return true;
                };
                for (int i = 0; ok && i < it.n; ++i) {
                    if (b0 + i * nbox >= w0 + 32) {
                        w0 += 32;
                        cur = nxt;
                        nxt = row_of(w0 + 32 + lane);
                    }
                    ok = load(&kmap, i, false);
                    if (ok && i == 0) {
                        for (int x = 0; ok && x < 2; ++x) {
                            if (it.steps[x] == 0) continue;
                            if (uses[x] > 0) ok = __all_sync(0xffffffffu, wait(sh.q_empty + x, uses[x] - 1));
                            if (!ok) break;
                            if (lane == 0) {
                                const int rows = a.group * a.tpt;
                                ptx::mbar_expect_tx(sh.q_full + x, (uint32_t)rows * D * 2);
                                for (int h = 0; h < C::kHalves; ++h)
                                    tma_load_4d(qs + x * C::kQTile + h * (128 * 128), &qmap, 0, it.kvh * a.group,
                                                it.q0 + x * a.tpt, h, sh.q_full + x);
                            }
                            __syncwarp();
                            ++uses[x];
                        }
                    }
                    if (ok) ok = load(&vmap, i, !FP8 && i + 1 == it.n && it.limit % kKeys);
                }
            }
            if (abort_flag[0] && lane == 0) {
                // after an abort: let the copies in flight land before the CTA ends
                for (int st = 0; st < N; ++st) {
                    if (!lap && st >= c.st) break;
                    if (FP8) ptx::mbar_drain(sh.c_full + st, st < c.st ? c.ph : c.ph ^ 1u);
                    else if ((tails >> st) & 1) ptx::mbar_drain(sh.tail_full + st, ((tail_phase >> st) & 1) ^ 1);
                    else ptx::mbar_drain(sh.kv_full + st, st < c.st ? c.ph : c.ph ^ 1u);
                }
                for (int x = 0; x < 2; ++x)
                    if (uses[x]) ptx::mbar_drain(sh.q_full + x, (uses[x] - 1) & 1);
            }
        } else if (FP8 && warp >= kConvertWarp) {
            // ------------------------------------------------------------ converts e4m3 tiles
            // Codes to bf16, exactly, in the layout that TMA gives a bf16 tile: the keys' scales go
            // to the scores, the values' to the weights.  Rows behind the last key become
            // zeros: whatever lies there must not reach the products, where 0 * inf is not 0.
            // 2,048 tokens behind 30,000, 64/8 heads of 128: 944 TFLOP/s.  A tile takes 2,300
            // cycles, the 1,300 that a step's products take twice over, most of them waits and
            // latencies (without the conversion instructions 1,004 TFLOP/s; four warps 729; four
            // for the keys and four for the values 833; a ring of seven stages of 64 keys 781, and
            // with the warps so divided 844; all loads ahead of the ring's wait 913).
            const int tid = threadIdx.x - kConvertWarp * 32;
            constexpr int kChunks = D / 16;                      // 16-code chunks of a row
            constexpr int kRowsAt = 32 * kConverters / kChunks;  // rows that the warps take at once
            Item it;
            Cursor<2> cc;
            Cursor<C::kStages> c;
            bool lap = false;  // every stage has been used
            int slot = 0;
            bool ok = true;
            while (ok && next_item(it)) {
                for (int i = 0; ok && i < 2 * it.n; ++i) {
                    const int what = i & 1;  // 0: keys, 1: values
                    const int rows = min(kKeys, it.limit - it.key0 - (i >> 1) * kKeys);
                    if (lap) ok = __all_sync(0xffffffffu, wait(sh.kv_empty + c.st, c.ph ^ 1u));
                    ok = ok && __all_sync(0xffffffffu, wait(sh.c_full + cc.st, cc.ph));
                    if (!ok) break;
                    const uint8_t* src = codes + cc.st * C::kCodeStage;
                    uint8_t* dst = ring + c.st * C::kStage;
                    if (what == 0) {
                        // this slot's last stage has been used: its values' place in the ring, or a later one,
                        // is the one that has just been waited for (see Cfg)
                        if (tid < kKeys) {
                            scales[slot * 2 * kKeys + tid] = tid < rows ? code_scales[tid] * a.scale_log2 : 0.f;
                            scales[slot * 2 * kKeys + kKeys + tid] = tid < rows ? code_scales[kKeys + tid] : 0.f;
                        }
                        slot = slot + 1 == C::kScaleSlots ? 0 : slot + 1;
                    }
#pragma unroll
                    for (int z = 0; z < kKeys / kRowsAt; ++z) {
                        const int row = z * kRowsAt + tid / kChunks, ch = tid % kChunks;
                        const int from = D == 128 ? row * 128 + ((ch ^ (row & 7)) << 4)
                                                  : row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
                        uint4 x = *reinterpret_cast<const uint4*>(src + from);
                        if (row >= rows) x = make_uint4(0u, 0u, 0u, 0u);
                        uint32_t y[8];
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) e4m3x4_to_bf16(xs[e], y[2 * e], y[2 * e + 1]);
                        uint8_t* to = dst + (ch >> 2) * (kKeys * 128) + row * 128;
                        const int c16 = (ch & 3) * 2;
                        *reinterpret_cast<uint4*>(to + ((c16 ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                        *reinterpret_cast<uint4*>(to + (((c16 + 1) ^ (row & 7)) << 4)) =
                            make_uint4(y[4], y[5], y[6], y[7]);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::mbar_arrive(sh.c_empty + cc.st);
                        ptx::mbar_arrive(sh.kv_full + c.st);
                    }
                    cc.move(1);
                    c.move(1);
                    lap = lap || c.st == 0;
                }
            }
        } else if (warp < kLoadWarp) {
            // ------------------------------------------------------------ issue the products
            // The whole warp walks and waits, on values broadcast from lane 0, and
            // one elected lane issues: descriptors then stay in uniform registers.
            // An issue blocks until the tensor cores take it and a wait costs a few
            // hundred cycles even when its phase is over (the products keep shared
            // memory busy), so each tile has a warp for its scores and one for its
            // outputs: one waits while the others' products run.  (Two warps, one
            // per tile: 1,320 TFLOP/s; one for both: 836; one lane of it: 660.)
            const int role = __shfl_sync(0xffffffffu, warp, 0) - kIssueWarp;
            const int x = role & 1;
            constexpr uint32_t idesc_s = ptx::idesc_f16(128, kStep, true);
            constexpr uint32_t idesc_o = ptx::idesc_f16(128, D, true, false, true);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t t_s = tm + C::s_col(x, 0), t_o = tm + C::kO + x * D;
            auto all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
            Item it;
            Cursor<C::kStages> c;        // the next stage of keys, or of values
            uint32_t items = 0, no = 0;  // the tile's items and steps so far: buffer no & 1
            bool ok = true;
            auto release = [&]() {
                if (elect_one()) ptx::mma_commit(sh.kv_empty + c.st);
                __syncwarp();
                c.move(2);
            };
            if (role >= 2) c.move(1);
            while (ok && next_item(it)) {
                const int n = __shfl_sync(0xffffffffu, it.steps[x], 0), stages = __shfl_sync(0xffffffffu, it.n, 0);
                if (n > 0 && role < 2) {
                    const uint32_t qd = desc_lo(smem_u32(qs) + x * C::kQTile, 16), k_lo = desc_lo(smem_u32(ring), 16);
                    ok = all(sh.q_full + x, items);
                    for (int j = 0; ok && j < n; ++j, ++no) {
                        const int buf = no & 1;
                        if ((j & 1) == 0) ok = all(sh.kv_full + c.st, c.ph);
                        // the buffer's last weights have been used
                        if (ok && no >= 2) ok = all(&sh.pv_done[x][buf], (no >> 1) - 1);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint32_t kd = k_lo + ((c.st * C::kStage + (j & 1) * (kStep * 128)) >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint32_t off = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
                                ptx::mma_ss(t_s + buf * kStep, make_desc(qd + off), make_desc(kd + off), idesc_s,
                                            k > 0 ? 1u : 0u);
                            }
                            ptx::mma_commit(&sh.s_full[x][buf]);
                            if (j + 1 == n) ptx::mma_commit(sh.q_empty + x);
                        }
                        __syncwarp();
                        if ((j & 1) || j + 1 == n) release();
                    }
                    ++items;
                } else if (n > 0) {
                    const uint32_t v_lo = desc_lo(smem_u32(ring), kKeys * 128);
                    if (items > 0) ok = all(sh.o_empty + x, items - 1);
                    for (int j = 0; ok && j < n; ++j, ++no) {
                        const int buf = no & 1;
                        if ((j & 1) == 0) ok = all(sh.kv_full + c.st, c.ph);
                        ok = ok && all(&sh.p_full[x][buf], no >> 1);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint32_t vd = v_lo + ((c.st * C::kStage + (j & 1) * (kStep * 128)) >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < kStep / 16; ++k)
                                ptx::mma_ts(t_o, t_s + buf * kStep + k * 8, make_desc(vd + ((k * 2048) >> 4)), idesc_o,
                                            k > 0 ? 1u : (j > 0 ? 1u : 0u));
                            ptx::mma_commit(&sh.pv_done[x][buf]);
                            if (j + 1 == n) ptx::mma_commit(sh.o_full + x);
                        }
                        __syncwarp();
                        if ((j & 1) || j + 1 == n) release();
                    }
                    ++items;
                }
                // stages that only the other tile reads
                for (int i = (n + 1) / 2; ok && i < stages; ++i) {
                    ok = all(sh.kv_full + c.st, c.ph);
                    if (ok && lane == 0) ptx::mbar_arrive(sh.kv_empty + c.st);
                    __syncwarp();
                    c.move(2);
                }
            }
            if (abort_flag[0]) {
                if (elect_one()) {
                    ptx::mma_commit(sh.drain + role);
                    ptx::mbar_drain(sh.drain + role, 0);
                }
                __syncwarp();
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax: a row per thread
        reg_inc<C::kSoftRegs>();
        const int x = warp >> 2;
        const int r = threadIdx.x & 127;
        const int tok = r / a.group, head = r - tok * a.group;
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // 32 lanes a warp, lane in bits 16..
        const uint32_t to = tmem + lane_base + C::kO + x * D;
        Item it;
        uint32_t no = 0, o_use = 0;  // steps so far (buffer no & 1), outputs
        bool ok = true;
        const uint64_t sc2 = f32x2(a.scale_log2, a.scale_log2);
        int slot = 0;  // e4m3: of the item's first scales
        while (ok && next_item(it)) {
            const int t = x * a.tpt + tok;  // token within the item
            int sl = slot;
            if (FP8) slot = (slot + it.n) % C::kScaleSlots;
            if (x == 1 && it.ntok <= a.tpt) continue;
            bool live = tok < a.tpt && t < it.ntok;
            int pos = 0x7FFFFFFF;  // unused rows: no mask, no output
            if (live) {
                pos = __ldg(a.s.q_pos + it.q0 + t);
                if (pos < -1 || pos >= it.ctx) {
                    report(a.d_status, DSA_ERR_BAD_INPUT);
                    live = false;
                    pos = -1;
                }
            }
            const int n = it.steps[x];
            float m = -INFINITY;
            uint64_t l2[2] = {0ull, 0ull};  // two pairs of fp32 sums
            for (int j = 0; j < n; ++j, ++no) {
                const int buf = no & 1;
                ok = __all_sync(0xffffffffu, wait(&sh.s_full[x][buf], no >> 1));
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t ts = tmem + lane_base + C::s_col(x, buf);
                uint32_t s[2][32];
                ptx::tmem_ld32_async(ts, s[0]);
                ptx::tmem_ld32_async(ts + 32, s[1]);
                ptx::tmem_wait_ld32(s[0]);
                ptx::tmem_wait_ld32(s[1]);
                const float* sc = scales + sl * 2 * kKeys + (j & 1) * kStep;  // e4m3: the step's keys' (times log2 e)
                if (FP8) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(sc + 32 * k + e);
                            uint32_t* y = s[k] + e;
                            const uint64_t u = mul2(f32x2(__uint_as_float(y[0]), __uint_as_float(y[1])), f.x);
                            const uint64_t w = mul2(f32x2(__uint_as_float(y[2]), __uint_as_float(y[3])), f.y);
                            y[0] = (uint32_t)u, y[1] = (uint32_t)(u >> 32);
                            y[2] = (uint32_t)w, y[3] = (uint32_t)(w >> 32);
                        }
                }
                const int lim = pos - it.key0 - j * kStep;  // the step's last key that the row sees
                if (__any_sync(0xffffffffu, lim < kStep - 1)) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * k + e > lim) s[k][e] = 0xFF800000u;
                }
                float mx[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mx[k] = __uint_as_float(s[k >> 1][16 * (k & 1)]);
#pragma unroll
                    for (int e = 1; e < 16; ++e) mx[k] = fmaxf(mx[k], __uint_as_float(s[k >> 1][16 * (k & 1) + e]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * (FP8 ? 1.f : a.scale_log2);
                const bool move = top > m + kLazy;
                if (__any_sync(0xffffffffu, move)) {
                    const float mn = move ? top : m;
                    const float al = move ? fast_exp2(m - mn) : 1.f;
                    m = mn;
                    const uint64_t al2 = f32x2(al, al);
                    l2[0] = fma2(l2[0], al2, 0ull);
                    l2[1] = fma2(l2[1], al2, 0ull);
                    if (j > 0) {
                        // O is at rest once the last step's product is done (the one before it is: this
                        // step's scores waited for it) and until this step's weights are handed over
                        ok = __all_sync(0xffffffffu, wait(&sh.pv_done[x][buf ^ 1], (no - 1) >> 1));
                        if (!ok) break;
                        ptx::tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < D / 32; ++k) {
                            float o[32];
                            ptx::tmem_ld32(to + 32 * k, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= al;
                            ptx::tmem_st32(to + 32 * k, o);
                        }
                    }
                }
                const float mm = m == -INFINITY ? 0.f : -m;
                const uint64_t nm2 = f32x2(mm, mm);
                uint32_t pk[32];
                ulonglong2 vs = make_ulonglong2(0, 0);
                uint64_t step[2];  // the step's sums: 16 additions each, and one to the row's
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        uint64_t v = f32x2(__uint_as_float(s[k][e]), __uint_as_float(s[k][e + 1]));
                        v = FP8 ? add2(v, nm2) : fma2(v, sc2, nm2);
                        float p0, p1;
                        unpack2(v, p0, p1);
                        p0 = fast_exp2(p0);
                        p1 = fast_exp2(p1);
                        uint64_t& sum = step[(e >> 1) & 1];
                        sum = k == 0 && e < 4 ? f32x2(p0, p1) : add2(sum, f32x2(p0, p1));
                        if (FP8) {
                            if ((e & 2) == 0) vs = *reinterpret_cast<const ulonglong2*>(sc + kKeys + 32 * k + e);
                            unpack2(mul2(f32x2(p0, p1), e & 2 ? vs.y : vs.x), p0, p1);
                        }
                        // a weight (times its value's scale) rounded to bf16 is off by up to 2^-8 of itself;
                        // the sum keeps fp32
                        pk[16 * k + e / 2] = pack_bf16(p0, p1);
                    }
                l2[0] = add2(l2[0], step[0]);
                l2[1] = add2(l2[1], step[1]);
                if (FP8 && (j & 1)) sl = sl + 1 == C::kScaleSlots ? 0 : sl + 1;
                ptx::tmem_st32_nowait(ts, pk);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sh.p_full[x][buf]);
            }
            if (!ok) break;
            float la, lb, lc, ld;
            unpack2(l2[0], la, lb);
            unpack2(l2[1], lc, ld);
            const float l = (la + lb) + (lc + ld);
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int64_t at = (int64_t)(it.q0 + t) * (a.hkv * a.group) + it.kvh * a.group + head;
            if (a.splits > 1) {
                // a partial result: O as it is, its reference and its sum (0: O is not read)
                const int64_t row = (int64_t)it.part * a.num_q * (a.hkv * a.group) + at;
                if (live) a.part_ml[row] = make_float2(m, l);
                if (n == 0) continue;
                ok = __all_sync(0xffffffffu, wait(sh.o_full + x, o_use));
                if (!ok) break;
                ++o_use;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    float o[32];
                    ptx::tmem_ld32(to + 32 * k, o);
                    if (live) {
                        float4* dst = reinterpret_cast<float4*>(a.part_o + row * D + 32 * k);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sh.o_empty + x);
                continue;
            }
            if (n > 0) {
                ok = __all_sync(0xffffffffu, wait(sh.o_full + x, o_use));
                if (!ok) break;
                ++o_use;
                ptx::tc_fence_after();
                // kOutDims at a time: a thread's row into the warp's 32 rows (16-byte pieces turned by
                // the row: no bank conflicts), then whole lines of 128 (or 64) bytes a store
                constexpr int OD = C::kOutDims, kPieces = OD / 8;  // 16-byte pieces of a row
                constexpr int kAtOnce = 32 / kPieces;              // rows a store
                uint8_t* mine = stage_out + warp * C::kOutWarp;
                auto piece = [&](int row, int c) {
                    return row * OD * 2 + ((c ^ (OD == 64 ? row & 7 : (row >> 1) & 3)) << 4);
                };
                const uint32_t alive = __ballot_sync(0xffffffffu, live);
                const uint64_t inv2 = f32x2(inv, inv);
                const int part = lane % kPieces, first = lane / kPieces;
                __nv_bfloat16* to_row[kPieces];
#pragma unroll
                for (int y = 0; y < kPieces; ++y)
                    to_row[y] = a.out + __shfl_sync(0xffffffffu, at, kAtOnce * y + first) * D + 8 * part;
#pragma unroll 1
                for (int k = 0; k < D / OD; ++k) {
                    uint32_t o[OD / 32][32];
#pragma unroll
                    for (int z = 0; z < OD / 32; ++z) ptx::tmem_ld32_async(to + OD * k + 32 * z, o[z]);
#pragma unroll
                    for (int z = 0; z < OD / 32; ++z) ptx::tmem_wait_ld32(o[z]);
                    if (l == 0.f) {  // no key: whatever O holds
#pragma unroll
                        for (int e = 0; e < OD; ++e) o[e >> 5][e & 31] = 0u;
                    }
#pragma unroll
                    for (int e = 0; e < kPieces; ++e) {
                        uint32_t y[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const uint32_t* w = &o[e >> 2][8 * (e & 3) + 2 * z];
                            float p, q;
                            unpack2(mul2(f32x2(__uint_as_float(w[0]), __uint_as_float(w[1])), inv2), p, q);
                            y[z] = pack_bf16(p, q);
                        }
                        *reinterpret_cast<uint4*>(mine + piece(lane, e)) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                    __syncwarp();
                    uint4 v[kPieces];
#pragma unroll
                    for (int y = 0; y < kPieces; ++y)
                        v[y] = *reinterpret_cast<const uint4*>(mine + piece(kAtOnce * y + first, part));
                    __syncwarp();
#pragma unroll
                    for (int y = 0; y < kPieces; ++y)
                        if ((alive >> (kAtOnce * y + first)) & 1) *reinterpret_cast<uint4*>(to_row[y] + OD * k) = v[y];
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sh.o_empty + x);
            } else if (live) {
                uint4* dst = reinterpret_cast<uint4*>(a.out + at * D);
#pragma unroll
                for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
            }
            if (live && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Joins the partial results of a row (query, head), a warp per row: weights
// 2^(m_i - M), in the ranges' order.  Rows that no valid query owns stay.
constexpr int kMaxSplits = 16;
constexpr int kMostPieces = 4 * kPlanSms;  // (item, key range) pairs of a call that is split
template <int D>
__global__ void __launch_bounds__(128) gqa_prefill_join_kernel(const __grid_constant__ Args a) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int heads = a.hkv * a.group;
    const int64_t rows = (int64_t)a.num_q * heads;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int t = (int)(row / heads);
    const int b = seq_of(a.s.q_start, a.s.num_seqs, t);
    const Seq q = load_seq(a.s, b, a.num_q);
    if (!q.ok || t < q.q0 || t >= q.q0 + q.nq) return;
    const int pos = __ldg(a.s.q_pos + t);
    if (pos < -1 || pos >= q.ctx) return;
    float2 v = make_float2(-INFINITY, 0.f);
    if (lane < a.splits) v = a.part_ml[lane * rows + row];
    float top = v.y == 0.f ? -INFINITY : v.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float w = v.y == 0.f ? 0.f : fast_exp2(v.x - top);
    float sum = w * v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    constexpr int E = D / 32;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = 0; i < a.splits; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        if (__shfl_sync(0xffffffffu, v.y, i) == 0.f) continue;  // nothing was written
        const float* src = a.part_o + (i * rows + row) * D + lane * E;
        if (E == 4) {
            const float4 x = __ldcs(reinterpret_cast<const float4*>(src));
            acc[0] = fmaf(wi, x.x, acc[0]), acc[1] = fmaf(wi, x.y, acc[1]);
            acc[E - 2] = fmaf(wi, x.z, acc[E - 2]), acc[E - 1] = fmaf(wi, x.w, acc[E - 1]);
        } else {
            const float2 x = __ldcs(reinterpret_cast<const float2*>(src));
            acc[0] = fmaf(wi, x.x, acc[0]), acc[1] = fmaf(wi, x.y, acc[1]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    if (a.lse && lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// ---------------------------------------------------------------------------
// host side: Q [num_q, heads, d] with rows `stride` elements apart, a box of
// `tokens` x `group` heads x 64 dims
cudaError_t query_map(CUtensorMap* m, const void* q, int heads, int d, int64_t stride, int num_q, int group, int tokens) {
    auto enc = tmap_encoder();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[4] = {64, (cuuint64_t)heads, (cuuint64_t)num_q, (cuuint64_t)d / 64};
    cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2, 128};
    cuuint32_t box[4] = {64, (cuuint32_t)group, (cuuint32_t)tokens, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, bool FP8>
cudaError_t launch_one(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const Args& a, int grid,
                       cudaStream_t stream) {
    using C = Cfg<D, FP8>;
    auto kern = gqa_prefill_kernel<D, FP8>;
    static OncePerDevice once;
    const cudaError_t e = once.run(
        [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(C::kThreads), C::kSmem, stream, 1, qm, km, vm, a);
}

struct Plan {
    int splits;
    size_t o_bytes, ml_bytes;
};

// Key ranges per item, from the sizes that the host knows: one, unless an
// estimate gains 15% with more, then the fewest within 2% of the best.  Items of
// equal length fill the GPU in rounds (512 items over 152 CTAs: four rounds, the
// last for a third of them); items of many lengths, longest first, even out by
// themselves.  In steps of 64 keys: six of an item's own start and end, a
// partial result two more, the join at 6.8 TB/s.  Idle SMs leave the others
// power, so a smaller gain is none.  Split against not: 720 and 360 tokens
// behind 25,728, 16/2 heads of 128, 183 us and 308; up to 64 tokens of four
// sequences behind 4,000, 64/8 heads, 46 and 58; and where the estimate says no:
// 1,867 tokens behind 18,711, 16/2 heads, 256 and 244; 4,000 from the start 61
// and 56; 2,048 behind 63,488, 64/8 heads, 2,974 and 2,998.
Plan make_plan(const dsa_gqa_shape& sh, const dsa_seqs& s, int num_q) {
    const int group = sh.num_heads / sh.num_kv_heads, per = 2 * (128 / group);
    const double rows = (double)std::max(num_q, 1) * sh.num_heads;
    const double items = std::max<double>((num_q + per - 1) / per, std::min(num_q, s.num_seqs)) * sh.num_kv_heads;
    const double mean = (s.max_ctx - 0.5 * std::min(s.max_q_per_seq, s.max_ctx)) / kStep;
    const bool even = s.max_q_per_seq < s.max_ctx / 4;
    double t[kMaxSplits + 1], best = 1e30;
    int most = 0;
    for (int n = 1; n <= kMaxSplits; ++n) {
        if (n > 1 && (mean / n < 8 || items * n > kMostPieces)) break;
        const double piece = mean / n + (n > 1 ? 8 : 6), work = items * n * piece / kPlanSms;
        t[n] = items * n >= 8 * kPlanSms ? work : std::ceil(items * n / kPlanSms) * piece;
        if (!even) t[n] = std::max(work, (double)s.max_ctx / kStep / n + 6);
        if (n > 1) t[n] += 6 + rows * (n * 2.0 * (sh.head_dim * 4 + 8) + sh.head_dim * 2) / 6.8e6 / 0.7;
        best = std::min(best, t[n]);
        most = n;
    }
    Plan p{1, 0, 0};
    if (best < 0.85 * t[1])
        while (p.splits < most && t[p.splits] > 1.02 * best) ++p.splits;
    if (p.splits > 1) {
        p.o_bytes = ((size_t)rows * p.splits * sh.head_dim * 4 + 255) & ~(size_t)255;
        p.ml_bytes = ((size_t)rows * p.splits * 8 + 255) & ~(size_t)255;
    }
    return p;
}

}  // namespace

// For any call of up to num_q queries: an item has at most 256 rows, and at
// most kMostPieces pieces of items leave partial results.
size_t prefill_workspace(const dsa_gqa_shape& sh, int num_q) {
    const size_t rows = std::min((size_t)num_q * sh.num_heads * kMaxSplits, (size_t)kMostPieces * 256);
    return rows * (sh.head_dim * 4 + 8) + 512;
}

cudaError_t launch_prefill(const dsa_gqa_shape& sh, const void* q, const void* k, const void* v,
                           const float* k_scale, const float* v_scale, const dsa_seqs& s, int num_q, float sm_scale,
                           void* out, float* lse, void* workspace, int32_t* d_status, cudaStream_t stream) {
    const Plan p = make_plan(sh, s, num_q);
    Args a;
    a.splits = p.splits;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.o_bytes);
    a.group = sh.num_heads / sh.num_kv_heads;
    a.hkv = sh.num_kv_heads;
    a.tpt = 128 / a.group;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.s = s;
    a.d_status = d_status;
    a.num_q = num_q;
    a.scale_log2 = sm_scale * 1.4426950408889634f;
    const int box = s.page_table ? std::min(s.page_size, kKeys) : kKeys;
    const bool fp8 = sh.kv_dtype != DSA_BF16;
    a.scale_shift = scale_shift(sh);
    CUtensorMap qm, km, vm;
    cudaError_t e = query_map(&qm, q, sh.num_heads, sh.head_dim, sh.q_stride, num_q, a.group, a.tpt);
    if (e == cudaSuccess)
        e = cache_map(&km, fp8, k, sh.num_kv_heads, sh.head_dim, sh.k_stride, s.num_rows, box, box == kKeys);
    if (e == cudaSuccess)
        e = cache_map(&vm, fp8, v, sh.num_kv_heads, sh.head_dim, sh.v_stride, s.num_rows, box, box == kKeys);
    if (e != cudaSuccess) return e;
    const int64_t items = ((int64_t)num_q / (2 * a.tpt) + s.num_seqs) * a.hkv * a.splits;  // at most
    const int grid = (int)std::min<int64_t>(num_sms(), items);
    e = sh.head_dim == 64 ? (fp8 ? launch_one<64, true>(qm, km, vm, a, grid, stream)
                                 : launch_one<64, false>(qm, km, vm, a, grid, stream))
                          : (fp8 ? launch_one<128, true>(qm, km, vm, a, grid, stream)
                                 : launch_one<128, false>(qm, km, vm, a, grid, stream));
    if (e != cudaSuccess || a.splits == 1) return e;
    const int64_t rows = (int64_t)num_q * sh.num_heads;
    auto join = sh.head_dim == 64 ? gqa_prefill_join_kernel<64> : gqa_prefill_join_kernel<128>;
    return launch_pdl(join, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, 1, a);
}

}  // namespace gqa
}  // namespace dsa
