// gqa_decode.cu -- dense attention of a few new tokens per sequence: the kernels
// of gqa_decode.cuh over all of a sequence's keys.
#include "gqa_decode.cuh"

namespace dsa {
namespace gqa {

constexpr int kDecodeOcc = 2;

size_t decode_workspace(const dsa_gqa_shape& sh) { return plan_workspace(sh, kDecodeOcc); }

cudaError_t launch_decode(const dsa_gqa_shape& sh, const void* q, const void* k, const void* v, const float* k_scale,
                          const float* v_scale, const dsa_seqs& s, int num_q, float sm_scale, void* out, float* lse,
                          void* workspace, int32_t* d_status, cudaStream_t stream) {
    const Plan p = make_plan(sh, s, kDecodeOcc, false);
    const int box = s.page_table ? std::min(s.page_size, p.tile) : p.tile;
    return launch_all<false>(p, sh, q, k, v, k_scale, v_scale, s, num_q, sm_scale, out, lse, workspace, d_status,
                             stream, kDecodeOcc, box, nullptr, nullptr, 0, 0);
}

}  // namespace gqa
}  // namespace dsa
