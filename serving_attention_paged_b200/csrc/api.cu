// C-ABI entry points of libpagedattn.so that touch the device: workspace
// upload, the run stage, cascade run, prefill run, cache write and read,
// merge_state, the index check and the scheduling defaults.  Argument checking happens here, on the
// host, before anything is enqueued; pointers must be device pointers
// (16-byte aligned for q, o and the pools).
#include <cuda_runtime.h>

#include "pa_internal.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

pa_status from_cuda(int e) { return e == 0 ? PA_OK : PA_ERR_CUDA; }

int launch_decode_any(const pa_plan_s& plan, const pa::RunPointers& p, void* stream) {
  return pa::decode_uses_tensor_cores(plan.prob) ? pa::launch_decode_tc(plan, p, stream)
                                                 : pa::launch_decode(plan, p, stream);
}

pa_status check_run_args(pa_plan_t plan, const void* q, const void* k_pool, const void* v_pool,
                         const int32_t* kv_indices, void* o, void* ws, size_t ws_bytes) {
  if (!plan || !ws) return PA_ERR_INVALID_ARG;
  if (ws_bytes < plan->ws.total) return PA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(ws) || (reinterpret_cast<uintptr_t>(ws) & (pa::kAlign - 1)))
    return PA_ERR_INVALID_ARG;
  if (plan->prob.batch == 0) return PA_OK;
  if (!q || !o || !aligned16(q) || !aligned16(o)) return PA_ERR_INVALID_ARG;
  const bool has_pages = plan->kv_indptr.back() > 0 || plan->prefix_len > 0;
  if (has_pages && (!k_pool || !v_pool || !aligned16(k_pool) || !aligned16(v_pool)))
    return PA_ERR_INVALID_ARG;
  if (plan->kv_indptr.back() > 0 && !kv_indices) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

// What a run asks for: the options if they ask for anything, else null.
const pa_attention_options* asked(const pa_attention_options* o) {
  if (!o) return nullptr;
  const bool nothing = !o->k_scales && !o->v_scales && o->logit_cap == 0.f && !o->alibi_slopes;
  return nothing && o->scale_block == 0 ? nullptr : o;
}

pa_status check_options(const pa_plan_s& plan, const pa_attention_options& o) {
  const pa_problem& pr = plan.prob;
  if (o.logit_cap != 0.f && !(o.logit_cap >= 0x1p-20f && o.logit_cap <= 0x1p20f))
    return PA_ERR_INVALID_ARG;  // NaN too
  if (!aligned4(o.k_scales) || !aligned4(o.v_scales) || !aligned4(o.alibi_slopes))
    return PA_ERR_INVALID_ARG;
  if (o.k_scales || o.v_scales || o.scale_block != 0) {
    if (plan.prefill) return PA_ERR_UNSUPPORTED;
    if (!pa::kv_is_8bit(pr) || !o.k_scales || !o.v_scales ||
        !pa::scale_block_valid(o.scale_block, pr.page_size) || pr.k_scale != 1.f ||
        pr.v_scale != 1.f)
      return PA_ERR_INVALID_ARG;
  }
  if (plan.prefill && !plan.causal && o.alibi_slopes) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// Rows of k / v: 16-byte vectors, consecutive rows at least a row apart.
bool rows_valid(const pa_plan_s& plan, const void* x, int64_t stride) {
  return x && aligned16(x) && stride % 8 == 0 &&
         stride >= int64_t(plan.prob.num_kv_heads) * plan.prob.head_dim;
}

pa_status check_kv_args(pa_plan_t plan, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, const void* k_pool, const void* v_pool,
                        const float* k_scales, const float* v_scales, const int32_t* kv_indices,
                        void* ws, size_t ws_bytes) {
  if (!plan || !plan->kv_cache || !ws) return PA_ERR_INVALID_ARG;
  if (ws_bytes < plan->ws.total) return PA_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(ws) & (pa::kAlign - 1)) return PA_ERR_INVALID_ARG;
  if (plan->total_q == 0) return PA_OK;
  if (!rows_valid(*plan, k, k_stride) || !rows_valid(*plan, v, v_stride))
    return PA_ERR_INVALID_ARG;
  if (!k_pool || !v_pool || !aligned16(k_pool) || !aligned16(v_pool) || !k_scales || !v_scales ||
      !kv_indices || !aligned4(k_scales) || !aligned4(v_scales) || !aligned4(kv_indices))
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_plan_upload(pa_plan_t plan, void* d_workspace, size_t workspace_bytes,
                         void* stream) {
  if (!plan || !d_workspace) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->ws.total) return PA_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(d_workspace) & (pa::kAlign - 1)) return PA_ERR_INVALID_ARG;
  // one copy of the plan's image of the workspace head (work list, offsets,
  // zeroed counters, cleared status words)
  const std::vector<uint8_t>& img = plan->upload_image;
  const cudaError_t e = cudaMemcpyAsync(d_workspace, img.data(), img.size(),
                                        cudaMemcpyHostToDevice, static_cast<cudaStream_t>(stream));
  return from_cuda(int(e));
}

pa_status pa_run(pa_plan_t plan, const void* q, const void* k_pool, const void* v_pool,
                 const int32_t* d_kv_indices, void* o, float* lse, void* d_workspace,
                 size_t workspace_bytes, void* stream) {
  return pa_run_options(plan, nullptr, q, k_pool, v_pool, d_kv_indices, o, lse, d_workspace,
                        workspace_bytes, stream);
}

pa_status pa_run_options(pa_plan_t plan, const pa_attention_options* options, const void* q,
                         const void* k_pool, const void* v_pool, const int32_t* d_kv_indices,
                         void* o, float* lse, void* d_workspace, size_t workspace_bytes,
                         void* stream) {
  pa_status st =
      check_run_args(plan, q, k_pool, v_pool, d_kv_indices, o, d_workspace, workspace_bytes);
  if (st != PA_OK) return st;
  // other plans run through pa_cascade_run, pa_prefill_run, pa_kv_append / pa_kv_read
  if (plan->cascade || plan->prefill || plan->kv_cache) return PA_ERR_INVALID_ARG;
  pa::RunPointers p{q, k_pool, v_pool, d_kv_indices, nullptr, o, lse,
                    static_cast<uint8_t*>(d_workspace), asked(options)};
  if (p.options) st = check_options(*plan, *p.options);
  if (st != PA_OK) return st;
  return from_cuda(launch_decode_any(*plan, p, stream));
}

pa_status pa_cascade_run(pa_plan_t plan, const void* q, const void* k_pool,
                         const void* v_pool, const int32_t* d_prefix_indices,
                         const int32_t* d_kv_indices, void* o, float* lse, void* d_workspace,
                         size_t workspace_bytes, void* stream) {
  pa_status st =
      check_run_args(plan, q, k_pool, v_pool, d_kv_indices, o, d_workspace, workspace_bytes);
  if (st != PA_OK) return st;
  if (!plan->cascade) return PA_ERR_INVALID_ARG;
  if (plan->prefix_chunks > 0 && !d_prefix_indices) return PA_ERR_INVALID_ARG;
  pa::RunPointers p{q, k_pool, v_pool, d_kv_indices, d_prefix_indices, o, lse,
                    static_cast<uint8_t*>(d_workspace)};
  if (plan->prefix_chunks > 0) {
    int e = pa::launch_cascade_prefix(*plan, p, stream);
    if (e == int(cudaErrorNotSupported)) return PA_ERR_UNSUPPORTED;
    if (e) return PA_ERR_CUDA;
  }
  return from_cuda(launch_decode_any(*plan, p, stream));
}

pa_status pa_prefill_run(pa_plan_t plan, const void* q, const void* k_pool, const void* v_pool,
                         const int32_t* d_kv_indices, void* o, float* lse, void* d_workspace,
                         size_t workspace_bytes, void* stream) {
  return pa_prefill_run_options(plan, nullptr, q, k_pool, v_pool, d_kv_indices, o, lse,
                                d_workspace, workspace_bytes, stream);
}

pa_status pa_prefill_run_options(pa_plan_t plan, const pa_attention_options* options,
                                 const void* q, const void* k_pool, const void* v_pool,
                                 const int32_t* d_kv_indices, void* o, float* lse,
                                 void* d_workspace, size_t workspace_bytes, void* stream) {
  pa_status st =
      check_run_args(plan, q, k_pool, v_pool, d_kv_indices, o, d_workspace, workspace_bytes);
  if (st != PA_OK) return st;
  if (!plan->prefill) return PA_ERR_INVALID_ARG;
  pa::RunPointers p{q, k_pool, v_pool, d_kv_indices, nullptr, o, lse,
                    static_cast<uint8_t*>(d_workspace), asked(options)};
  if (p.options) st = check_options(*plan, *p.options);
  if (st != PA_OK) return st;
  return from_cuda(pa::launch_prefill(*plan, p, stream));
}

pa_status pa_kv_append(pa_plan_t plan, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, void* k_pool, void* v_pool, float* k_scales,
                       float* v_scales, const int32_t* d_kv_indices, void* d_workspace,
                       size_t workspace_bytes, void* stream) {
  const pa_status st = check_kv_args(plan, k, k_stride, v, v_stride, k_pool, v_pool, k_scales,
                                     v_scales, d_kv_indices, d_workspace, workspace_bytes);
  if (st != PA_OK) return st;
  const pa::KvPointers p{const_cast<void*>(k), const_cast<void*>(v), k_stride, v_stride,
                         k_pool, v_pool, k_scales, v_scales, d_kv_indices, nullptr, 0,
                         static_cast<uint8_t*>(d_workspace)};
  return from_cuda(pa::launch_kv_append(*plan, p, stream));
}

pa_status pa_kv_read(pa_plan_t plan, const void* k_pool, const void* v_pool,
                     const float* k_scales, const float* v_scales, const int32_t* d_kv_indices,
                     void* k, int64_t k_stride, void* v, int64_t v_stride,
                     const int32_t* d_out_indices, int64_t num_out_pages, void* d_workspace,
                     size_t workspace_bytes, void* stream) {
  const pa_status st = check_kv_args(plan, k, k_stride, v, v_stride, k_pool, v_pool, k_scales,
                                     v_scales, d_kv_indices, d_workspace, workspace_bytes);
  if (st != PA_OK) return st;
  if (d_out_indices) {
    const int64_t row = int64_t(plan->prob.num_kv_heads) * plan->prob.head_dim;
    if (k_stride != row || v_stride != row || num_out_pages < 0 || !aligned4(d_out_indices))
      return PA_ERR_INVALID_ARG;
    // pool rows are 32-bit indices inside the kernel
    if (num_out_pages > int64_t(UINT32_MAX) / plan->prob.page_size) return PA_ERR_UNSUPPORTED;
  }
  const pa::KvPointers p{k, v, k_stride, v_stride, const_cast<void*>(k_pool),
                         const_cast<void*>(v_pool), const_cast<float*>(k_scales),
                         const_cast<float*>(v_scales), d_kv_indices, d_out_indices,
                         num_out_pages, static_cast<uint8_t*>(d_workspace)};
  return from_cuda(pa::launch_kv_read(*plan, p, stream));
}

pa_status pa_merge_state(const void* o_a, const float* lse_a, const void* o_b,
                         const float* lse_b, void* o, float* lse, int64_t rows,
                         int32_t head_dim, pa_dtype dtype, void* stream) {
  if (rows < 0 || head_dim <= 0) return PA_ERR_INVALID_ARG;
  if (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_F32) return PA_ERR_INVALID_ARG;
  if (rows == 0) return PA_OK;
  if (!o_a || !lse_a || !o_b || !lse_b || !o) return PA_ERR_INVALID_ARG;
  return from_cuda(
      pa::launch_merge_state(o_a, lse_a, o_b, lse_b, o, lse, rows, head_dim, dtype, stream));
}

pa_status pa_plan_check(pa_plan_t plan, void* d_workspace, int64_t* bad_position,
                        void* stream) {
  if (!plan || !d_workspace) return PA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  unsigned long long words[2] = {0, 0};
  cudaError_t e = cudaMemcpyAsync(words, ws + plan->ws.error, sizeof words,
                                  cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemsetAsync(ws + plan->ws.error, 0xff, sizeof(uint64_t), s);
  if (e == cudaSuccess)
    e = cudaMemsetAsync(ws + plan->ws.error + sizeof(uint64_t), 0, sizeof(uint64_t), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return PA_ERR_CUDA;
  const unsigned long long word = words[0];
  if (bad_position) *bad_position = word == ~0ull ? -1 : int64_t(word);
  if (words[1]) return PA_ERR_DEVICE_TIMEOUT;
  if (word == ~0ull) {
    if (bad_position) *bad_position = -1;
    return PA_OK;
  }
  if (bad_position) *bad_position = int64_t(word);
  return PA_ERR_DEVICE_CHECK;
}

pa_status pa_default_schedule(int32_t device, int32_t num_qo_heads, int32_t num_kv_heads,
                              pa_dtype dtype, uint32_t flags, int32_t* num_sms,
                              int32_t* ctas_per_sm) {
  if (!num_sms || !ctas_per_sm || num_kv_heads <= 0 || num_qo_heads % num_kv_heads)
    return PA_ERR_INVALID_ARG;
  const int32_t group = num_qo_heads / num_kv_heads;
  if (!pa::decode_group_supported(group)) return PA_ERR_UNSUPPORTED;
  int prev = 0;
  cudaError_t e = cudaGetDevice(&prev);
  if (e == cudaSuccess) e = cudaSetDevice(device);
  int sms = 0;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  int32_t k = 0;
  pa_problem shape{};
  shape.num_qo_heads = num_qo_heads;
  shape.num_kv_heads = num_kv_heads;
  shape.dtype = dtype;
  shape.flags = flags;
  if (e == cudaSuccess)
    e = cudaError_t(pa::decode_uses_tensor_cores(shape) ? pa::decode_tc_ctas_per_sm(group, dtype, &k)
                                                        : pa::decode_ctas_per_sm(group, dtype, &k));
  cudaSetDevice(prev);
  if (e != cudaSuccess) return PA_ERR_CUDA;
  *num_sms = sms;
  *ctas_per_sm = k;
  return PA_OK;
}

pa_status pa_problem_schedule(const pa_problem* problem, int32_t device, int32_t* num_sms,
                              int32_t* ctas_per_sm) {
  if (!problem || !num_sms || !ctas_per_sm || problem->num_kv_heads <= 0 ||
      problem->num_qo_heads % problem->num_kv_heads)
    return PA_ERR_INVALID_ARG;
  const int32_t group = problem->num_qo_heads / problem->num_kv_heads;
  if (!pa::decode_group_supported(group)) return PA_ERR_UNSUPPORTED;
  if (pa::decode_uses_tensor_cores(*problem) || !pa::decode_f32_path(*problem))
    return pa_default_schedule(device, problem->num_qo_heads, problem->num_kv_heads,
                               problem->dtype, problem->flags | (pa::decode_uses_tensor_cores(*problem)
                                                                     ? PA_FLAG_TENSOR_CORES
                                                                     : 0u),
                               num_sms, ctas_per_sm);
  int prev = 0;
  cudaError_t e = cudaGetDevice(&prev);
  if (e == cudaSuccess) e = cudaSetDevice(device);
  int sms = 0;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  int32_t k = 0;
  if (e == cudaSuccess) e = cudaError_t(pa::decode_f32_ctas_per_sm(*problem, &k));
  cudaSetDevice(prev);
  if (e != cudaSuccess) return PA_ERR_CUDA;
  *num_sms = sms;
  *ctas_per_sm = k;
  return PA_OK;
}

}  // extern "C"
