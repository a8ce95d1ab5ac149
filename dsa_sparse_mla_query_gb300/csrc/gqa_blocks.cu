// gqa_blocks.cu -- attention over blocks of keys that are listed for each token
// and key head: the kernels of gqa_decode.cuh, every token a sequence of its own.
#include "gqa_decode.cuh"

namespace dsa {
namespace gqa {

static int listed_occ(const dsa_gqa_shape& sh) { return sh.kv_dtype == DSA_BF16 ? 2 : kListedOcc; }

size_t attend_workspace(const dsa_gqa_shape& sh) { return plan_workspace(sh, listed_occ(sh)); }

cudaError_t launch_attend(const dsa_gqa_shape& sh, const void* q, const void* k, const void* v, const float* k_scale,
                          const float* v_scale, const dsa_seqs& s, int num_q, const int32_t* blocks,
                          const int32_t* len, int block, int nsel, float sm_scale, void* out, float* lse,
                          void* workspace, int32_t* d_status, cudaStream_t stream) {
    dsa_seqs each = s;
    each.num_seqs = num_q;
    each.max_q_per_seq = 1;
    each.max_ctx = nsel * block;
    const Plan p = make_plan(sh, each, listed_occ(sh), true);
    return launch_all<true>(p, sh, q, k, v, k_scale, v_scale, s, num_q, sm_scale, out, lse, workspace, d_status,
                            stream, listed_occ(sh), std::min(block, p.tile), blocks, len, nsel, block);
}

}  // namespace gqa
}  // namespace dsa
