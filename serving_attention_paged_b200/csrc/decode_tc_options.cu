// The tensor-core decode kernel's launches with options (pa_run_options): block
// scales of an 8-bit pool, capped scores, distance bias.
#include "decode_tc_kernel.cuh"

namespace pa {
namespace {

template <typename Tag, int KV8>
cudaError_t dispatch_check(bool check, int group, const TcArgs& a, int64_t n, cudaStream_t s) {
  return check ? dispatch_tc<Tag, KV8, kTcOptionsChecked>(group, a, n, s)
               : dispatch_tc<Tag, KV8, kTcOptions>(group, a, n, s);
}

template <typename Tag>
cudaError_t dispatch_kv(pa_dtype kv, bool check, int group, const TcArgs& a, int64_t n,
                        cudaStream_t s) {
  if (kv == PA_E4M3) return dispatch_check<Tag, 1>(check, group, a, n, s);
  if (kv == PA_E5M2) return dispatch_check<Tag, 2>(check, group, a, n, s);
  return dispatch_check<Tag, 0>(check, group, a, n, s);
}

}  // namespace

int launch_decode_tc_options(const pa_plan_s& plan, const RunPointers& p, void* stream) {
  const pa_problem& pr = plan.prob;
  TcArgs a = make_tc_args(plan, p);
  a.kv_len = reinterpret_cast<const int32_t*>(p.ws + plan.ws.kv_len);
  a.k_scales = p.options->k_scales;
  a.v_scales = p.options->v_scales;
  while ((1 << a.log2_block) < p.options->scale_block) ++a.log2_block;
  set_score_args(*p.options, &a.score, &a.score_scale);
  const int64_t n = int64_t(plan.cta_indptr.size()) - 1;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const pa_dtype kv = kv_is_8bit(pr) ? pr.kv_dtype : pr.dtype;
  const bool check = (pr.flags & PA_FLAG_CHECK_INDICES) != 0;
  return int(pr.dtype == PA_BF16 ? dispatch_kv<BF16>(kv, check, plan.group, a, n, s)
                                 : dispatch_kv<F16>(kv, check, plan.group, a, n, s));
}

}  // namespace pa
