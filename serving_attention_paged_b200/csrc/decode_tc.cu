// The tensor-core decode kernel's plain launches (decode_tc_kernel.cuh holds
// the kernel and its design; runs with options are decode_tc_options.cu's).
#include "decode_tc_kernel.cuh"

namespace pa {
namespace {

template <typename Tag, int KV8>
cudaError_t dispatch_tc_check(bool check, int group, const TcArgs& a, int64_t n, cudaStream_t s) {
  return check ? dispatch_tc<Tag, KV8, kTcChecked>(group, a, n, s)
               : dispatch_tc<Tag, KV8, kTcPlain>(group, a, n, s);
}

template <typename Tag>
cudaError_t dispatch_tc_kv(pa_dtype kv, bool check, int group, const TcArgs& a, int64_t n,
                           cudaStream_t s) {
  if (kv == PA_E4M3) return dispatch_tc_check<Tag, 1>(check, group, a, n, s);
  if (kv == PA_E5M2) return dispatch_tc_check<Tag, 2>(check, group, a, n, s);
  return dispatch_tc_check<Tag, 0>(check, group, a, n, s);
}

}  // namespace

bool decode_tc_supported(int32_t group, pa_dtype dtype) {
  return (group == 1 || group == 2 || group == 4 || group == 8) &&
         (dtype == PA_F16 || dtype == PA_BF16);
}

int decode_tc_ctas_per_sm(int32_t group, pa_dtype dtype, int32_t* out) {
  // one CTA per SM whatever the shape: the kernels hold ~200 KB of shared memory
  (void)group;
  (void)dtype;
  auto kern = paged_decode_tc_kernel<F16, 0, 8, kTcPlain>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Off<false, false>::kSmemBytes);
  int n = 0;
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kThreads,
                                                      Off<false, false>::kSmemBytes);
  *out = n;
  return int(e);
}

int launch_decode_tc(const pa_plan_s& plan, const RunPointers& p, void* stream) {
  const pa_problem& pr = plan.prob;
  if (p.options) return launch_decode_tc_options(plan, p, stream);
  const TcArgs a = make_tc_args(plan, p);
  const bool kv8 = kv_is_8bit(pr);
  const bool check = (pr.flags & PA_FLAG_CHECK_INDICES) != 0;
  const int64_t n = int64_t(plan.cta_indptr.size()) - 1;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const pa_dtype kv = kv8 ? pr.kv_dtype : pr.dtype;
  const cudaError_t e = pr.dtype == PA_BF16 ? dispatch_tc_kv<BF16>(kv, check, plan.group, a, n, s)
                                            : dispatch_tc_kv<F16>(kv, check, plan.group, a, n, s);
  return int(e);
}

}  // namespace pa
