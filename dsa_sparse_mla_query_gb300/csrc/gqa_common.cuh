// gqa_common.cuh -- pieces shared by the dense grouped-head attention kernels
// (gqa_decode.cu, gqa_prefill.cu): sequences' counts, tensor maps, paired fp32
// arithmetic, e4m3 codes, ring places and waits.
#pragma once

#include <atomic>

#include "indexer_common.cuh"

namespace dsa {
namespace gqa {

constexpr int kPlanSms = 152;  // GB300's SMs: sizes that the host alone has to know are planned for them

// A sequence's counts, checked: queries [q0, q0 + nq) over `ctx` tokens.
struct Seq {
    int ctx, q0, nq;
    bool ok;
};
__device__ __forceinline__ Seq load_seq(const dsa_seqs& s, int b, int num_q) {
    Seq r;
    r.ctx = __ldg(s.ctx_len + b);
    r.q0 = __ldg(s.q_start + b);
    const int qe = __ldg(s.q_start + b + 1);
    r.nq = qe - r.q0;
    r.ok = r.ctx >= 0 && r.ctx <= s.max_ctx && r.q0 >= 0 && qe >= r.q0 && qe <= num_q && r.nq <= s.max_q_per_seq;
    return r;
}

// Tensor map over a cache [rows, heads, d] whose rows lie `stride` elements
// apart: dimensions (128 bytes of a head's row, rows, the row's 128-byte
// pieces, heads), so that a box of R rows lands in shared memory as one
// [R][128 B] swizzled block per piece (all of a row's pieces, or one).  A
// head row of 64 bytes (e4m3, d = 64) is one piece of 64 bytes.
inline cudaError_t cache_map(CUtensorMap* m, bool bytes, const void* base, int heads, int d, int64_t stride,
                             int64_t rows, int box_rows, bool all_pieces) {
    auto enc = tmap_encoder();
    if (!enc) return cudaErrorNotSupported;
    const uint64_t el = bytes ? 1 : 2;
    const uint64_t piece = std::min<uint64_t>(128, d * el);
    cuuint64_t dims[4] = {piece / el, (cuuint64_t)rows, d * el / piece, (cuuint64_t)heads};
    cuuint64_t strides[3] = {(cuuint64_t)stride * el, piece, d * el};
    cuuint32_t box[4] = {(cuuint32_t)(piece / el), (cuuint32_t)box_rows,
                         all_pieces ? (cuuint32_t)(d * el / piece) : 1u, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    const CUresult r = enc(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                           const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           piece == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// two fp32 values in one register pair, and arithmetic on both at once
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// four e4m3 codes (low byte first) -> two f16x2, exact
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}
// four e4m3 codes (low byte first) as two bf16 pairs, exact
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t x, uint32_t& lo, uint32_t& hi) {
    uint32_t a, b;
    e4m3x4_to_f16(x, a, b);
    const float2 u = __half22float2(*reinterpret_cast<__half2*>(&a)), v = __half22float2(*reinterpret_cast<__half2*>(&b));
    lo = pack_bf16(u.x, u.y);
    hi = pack_bf16(v.x, v.y);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// A place in the ring of N stages: the stage and the parity of its use.  (A
// 64-bit remainder for every stage held the issuing thread for longer than a
// step's products take.)
template <int N>
struct Cursor {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void move(int by) {
        st += by;
        if (st >= N) {
            st -= N;
            ph ^= 1u;
        }
    }
};

// A warpgroup's registers per thread, from those that the CTA was launched with
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// mbar_wait for waits that are short as a rule: several hardware-timed probes
// before the first read of the timer, which takes longer than a probe.
__device__ __forceinline__ bool quick_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                           int32_t* d_status) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (ptx::mbar_try_wait(bar, parity)) return true;
    return ptx::mbar_wait(bar, parity, abort_flag, d_status);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

// A kernel's attributes, set once on each device that launches it (they belong
// to the device's own copy of the kernel, and setting them takes longer than
// the rest of a launch's preparation).
struct OncePerDevice {
    std::atomic<uint64_t> done{0};
    template <typename F>
    cudaError_t run(F set) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
        if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
        const cudaError_t r = set();
        if (r == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
        return r;
    }
};

}  // namespace gqa
}  // namespace dsa
