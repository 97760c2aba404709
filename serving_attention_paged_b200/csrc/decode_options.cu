// Runs of the CUDA-core decode kernel with options (pa_run_options): capped
// scores and distance bias over 16-bit pools, 8-bit pools with block scales,
// and either with rotary positions.  The kernel template is decode_kernel.cuh
// (kExt); this file only instantiates it.  Which options apply is a launch
// argument; so is the index check on the fp32 path, as without options.
#include <cuda_runtime.h>

#include "decode_kernel.cuh"

namespace pa {
namespace {

template <typename Tag, typename KV>
cudaError_t dispatch_rope(bool rope, int group, const dec::DecodeArgs& a, int64_t n,
                          cudaStream_t s) {
  return rope ? dec::dispatch_group<Tag, KV, dec::kRuntimeCheck, true, true>(group, a, n, s)
              : dec::dispatch_group<Tag, KV, dec::kRuntimeCheck, false, true>(group, a, n, s);
}

template <typename Tag>
cudaError_t dispatch_kv(pa_dtype kv, bool rope, int group, const dec::DecodeArgs& a, int64_t n,
                        cudaStream_t s) {
  using dec::KV16;
  if (kv == PA_E4M3) return dispatch_rope<Tag, dec::E4M3>(rope, group, a, n, s);
  if (kv == PA_E5M2) return dispatch_rope<Tag, dec::E5M2>(rope, group, a, n, s);
  if (rope) return dec::dispatch_group<Tag, KV16, dec::kRuntimeCheck, true, true>(group, a, n, s);
  return a.check ? dec::dispatch_group<Tag, KV16, dec::kChecked, false, true>(group, a, n, s)
                 : dec::dispatch_group<Tag, KV16, dec::kNoCheck, false, true>(group, a, n, s);
}

}  // namespace

int launch_decode_options(const pa_plan_s& plan, const RunPointers& p, void* stream) {
  const pa_problem& pr = plan.prob;
  dec::DecodeArgs a;
  fill_decode_args(plan, p, &a);
  a.k_scales = p.options->k_scales;
  a.v_scales = p.options->v_scales;
  while ((1 << a.log2_block) < p.options->scale_block) ++a.log2_block;
  set_score_args(*p.options, &a.score, &a.score_scale);
  const int64_t n = int64_t(plan.cta_indptr.size()) - 1;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const pa_dtype kv = kv_is_8bit(pr) ? pr.kv_dtype : pr.dtype;
  const bool rope = pr.rope_theta > 0.f;
  return int(pr.dtype == PA_BF16 ? dispatch_kv<BF16>(kv, rope, plan.group, a, n, s)
                                 : dispatch_kv<F16>(kv, rope, plan.group, a, n, s));
}

}  // namespace pa
