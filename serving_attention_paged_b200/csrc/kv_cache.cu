// Writing an 8-bit paged KV cache with a scale for each block of tokens and
// kv head (pa_kv_append), and reading it back (pa_kv_read).
//
// FlashInfer README, core feature 3 (attention over a compressed KV-Cache)
// names the compressed cache and no more; the format is this library's: E4M3
// or E5M2 codes in the NHD pools, value = scale * code, one fp32 scale per
// scale_block consecutive pool rows and kv head.
//
// Quantisation.  With a the largest finite |x| of a block's new tokens,
// scale = the smallest power of two with a <= MAX * scale.  A power of two
// costs an FP8 format nothing (its relative step is the same at every
// exponent) and makes every step exact: MAX is 0.875 * 2^9 (E4M3) or
// 0.875 * 2^16 (E5M2), so the exponent is read off a's bits; x / scale is one
// exact product; codes of earlier tokens move to a grown scale by an exact
// power of two (rounded only where a code becomes subnormal); and a value read
// back into bf16 is exact.  The only rounding is the code itself (rn,
// saturating).
//
// Work.  Spans of max(16, scale_block) tokens (the plan's), one unit per
// (span, K or V, kv head), heads fastest, so neighbouring units touch
// neighbouring 256-byte rows.  Blocks of up to 16 tokens: a warp per unit,
// 16 lanes per row, eight 16-byte loads per lane in flight, the row kept in
// registers between the maximum and the rounding: each byte is read once.
// Larger blocks: a CTA per unit, up to 128 rows at a time in registers (rows of
// a longer block are read a second time for the rounding, out of L2).
// Both are bound by HBM; a decode step's few tokens by the launch and the
// chain span -> page index -> row.  No atomics on results: a block's scale is
// decided by one warp or CTA.
// Measured (one B200, 8 kv heads; launches replayed from a graph on inputs that
// rotate past L2): 66,934 tokens in 64-token blocks 75 us (411 MB, 5.5 TB/s), in
// 1,024-token blocks, read twice, 102 us; 8,192 in 16-token blocks 13.7 us (50
// MB, 3.7 TB/s; 1,024 CTAs where 592 are resident at a time); 128 single tokens
// 4.8 us after a flush of L2; 98,277 tokens read back 103 us (604 MB, 5.9 TB/s).
#include <cuda_runtime.h>

#include "common.cuh"
#include "decode_kernel.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

using dec::E4M3;
using dec::E5M2;

constexpr int D = kHeadDim;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kSteps = 8;                      // row pairs a warp holds: 16 tokens
constexpr uint32_t kNoRow = 0xffffffffu;       // pool rows are < 2^32 - 1

struct KvArgs {
  uint16_t* x[2];        // K and V rows
  int64_t stride[2];     // elements between rows
  uint8_t* pool[2];
  float* scales[2];
  const int32_t* kv_indices;
  const int32_t* out_indices;
  const KvSpan* spans;
  unsigned long long* error_pos;
  int64_t num_pages, num_out_pages;
  uint32_t n_units;  // the plan keeps it below 2^31
  uint32_t num_kv_heads;
  int32_t log2_page, log2_block;
  bool check;
  bool zero_bad;  // reads into rows: zeros for tokens on a bad page, which are else left alone
};

template <typename F> struct Format;
template <> struct Format<E4M3> { static constexpr int kMaxExp = 9; };   // MAX = 0.875 * 2^9
template <> struct Format<E5M2> { static constexpr int kMaxExp = 16; };  // MAX = 0.875 * 2^16

__device__ __forceinline__ uint32_t fp8x2(E4M3, float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}
__device__ __forceinline__ uint32_t fp8x2(E5M2, float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;\n" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}
template <typename F>
__device__ __forceinline__ uint2 fp8x8(const float (&y)[8]) {
  return make_uint2(fp8x2(F{}, y[0], y[1]) | (fp8x2(F{}, y[2], y[3]) << 16),
                    fp8x2(F{}, y[4], y[5]) | (fp8x2(F{}, y[6], y[7]) << 16));
}
template <typename F>
__device__ __forceinline__ void from_fp8x8(const uint2& u, float (&y)[8]) {
  float2 f[4];
  dec::fp8x4_to_f32(F{}, u.x, f);
  dec::fp8x4_to_f32(F{}, u.y, f + 2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = f[i].x;
    y[2 * i + 1] = f[i].y;
  }
}

// Largest |x| of a run of 16-bit values, as its bits without the sign: they
// order as the values do, two to a register, so 8 values take 4 masks and 2
// three-way maxima.  Infinities and NaN order above every finite value; only
// where one turns up is the maximum taken again without them (finite_amax).
template <typename Tag> struct Half;
template <> struct Half<F16> { static constexpr uint32_t kInf = 0x7c00u; };
template <> struct Half<BF16> { static constexpr uint32_t kInf = 0x7f80u; };
__device__ __forceinline__ uint32_t amax2(const uint4& u, uint32_t m) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  return __vimax3_u16x2(__vimax3_u16x2(m, u.x & kAbs, u.y & kAbs), u.z & kAbs, u.w & kAbs);
}
__device__ __forceinline__ uint32_t fold2(uint32_t m) { return max(m & 0xffffu, m >> 16); }
template <typename Tag>
__device__ __forceinline__ uint32_t finite_amax(const uint4& u, uint32_t m) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
    m = max(m, max(lo < Half<Tag>::kInf ? lo : 0u, hi < Half<Tag>::kInf ? hi : 0u));
  }
  return m;
}
template <typename Tag>
__device__ __forceinline__ uint32_t as_fp32(uint32_t bits) {
  return __float_as_uint(to_float(Tag{}, uint16_t(bits)));
}

// The smallest power of two s in [2^-60, 2^60] with a <= MAX * s, a given by
// its fp32 bits.  Writing
// a = (1 + f) 2^e: a <= 1.75 * 2^(kMaxExp - 1) s holds for s = 2^(e - kMaxExp
// + 1) if 1 + f <= 1.75, else for twice that.  (A subnormal or zero a clamps.)
template <typename F>
__device__ __forceinline__ float scale_for(uint32_t a) {
  const int k = int(a >> 23) - 127 - (Format<F>::kMaxExp - 1) + ((a & 0x7fffffu) > 0x600000u);
  return __int_as_float((min(max(k, -60), 60) + 127) << 23);
}

// x / s for 8 values: by the exact reciprocal of a power of two, else by
// rounded division (a scale that another writer chose).
template <typename Tag, typename F>
__device__ __forceinline__ uint2 quantise(const uint4& u, float s, float inv, bool pow2) {
  float f[8];
  to_float8(Tag{}, u, f);
  if (pow2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= inv;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __fdiv_rn(f[e], s);
  }
  return fp8x8<F>(f);
}
__device__ __forceinline__ bool is_pow2(float s) {
  return (__float_as_uint(s) & 0x7fffffu) == 0;  // normal, mantissa zero
}

// Pool row of request token t, kNoRow if its page is negative or the bounds
// check rejects it.
__device__ __forceinline__ uint32_t pool_row(const KvArgs& a, const int32_t* indices,
                                             int64_t num_pages, int page_begin, int t) {
  const int pos = page_begin + (t >> a.log2_page);
  const int page = __ldg(indices + pos);
  if (page < 0 || (a.check && int64_t(page) >= num_pages)) {
    if (a.check) atomicMin(a.error_pos, (unsigned long long)pos);
    return kNoRow;
  }
  return (uint32_t(page) << a.log2_page) | (uint32_t(t) & ((1u << a.log2_page) - 1u));
}

// Byte offset of row r of head h in a pool (8-bit codes).
__device__ __forceinline__ int64_t code_offset(const KvArgs& a, uint32_t r, int h) {
  return (int64_t(r) * a.num_kv_heads + h) * D;
}
__device__ __forceinline__ int64_t scale_index(const KvArgs& a, uint32_t r, int h) {
  return int64_t(r >> a.log2_block) * a.num_kv_heads + h;
}

// 8 codes of an earlier token, moved to the block's new scale.
template <typename F>
__device__ __forceinline__ void rescale8(uint8_t* p, float ratio) {
  uint2* q = reinterpret_cast<uint2*>(p);
  float y[8];
  from_fp8x8<F>(*q, y);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] *= ratio;
  *q = fp8x8<F>(y);
}

// Blocks of 2^kLB <= 16 tokens: a warp per (span of 16 tokens, K or V, head).
template <typename Tag, typename F, int kLB>
__global__ void __launch_bounds__(kThreads, 4) kv_append_warp_kernel(const KvArgs a) {
  const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (unit >= a.n_units) return;
  const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
  const uint32_t rest = unit / a.num_kv_heads;
  const int h = int(unit - rest * a.num_kv_heads), kv = int(rest & 1);
  const KvSpan sp = a.spans[rest >> 1];

  const uint16_t* x0 = a.x[kv] + h * D + c * 8;
  const int64_t stride = a.stride[kv];
  uint4 x[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int t = sp.start + 2 * i + half;
    x[i] = t >= sp.begin && t < sp.end
               ? __ldg(reinterpret_cast<const uint4*>(x0 + (sp.row + int64_t(t - sp.begin)) * stride))
               : make_uint4(0, 0, 0, 0);
  }
  // lane j < 16 holds the pool row of token start + j, from the first block's
  // earlier tokens on
  const int held = sp.begin & ~((1 << kLB) - 1);  // start of the first block
  uint32_t rows = kNoRow;
  {
    const int t = sp.start + c;
    if (t >= held && t < sp.end) rows = pool_row(a, a.kv_indices, a.num_pages, sp.page_begin, t);
  }
  float s_old = 0.f;
  uint32_t first_row = __shfl_sync(0xffffffffu, rows, sp.begin - sp.start);
  const bool has_old = held < sp.begin && first_row != kNoRow;
  float* scales = a.scales[kv];
  if (has_old) s_old = scales[scale_index(a, first_row, h)];

  // the scale of each step's row pair (kLB = 0: of this half's row)
  constexpr int kPer = kLB == 0 ? 1 : 1 << (kLB - 1);  // steps per block
  uint32_t m[kSteps / kPer], most = 0;
#pragma unroll
  for (int j = 0; j < kSteps / kPer; ++j) {
    m[j] = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m[j] = amax2(x[j * kPer + i], m[j]);
    m[j] = fold2(m[j]);
    most = max(most, m[j]);
  }
  if (__any_sync(0xffffffffu, most >= Half<Tag>::kInf)) {
#pragma unroll
    for (int j = 0; j < kSteps / kPer; ++j) {
      m[j] = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) m[j] = finite_amax<Tag>(x[j * kPer + i], m[j]);
    }
  }
  if constexpr (kLB == 0) {  // over the 16 lanes of a row, two rows' 16-bit maxima at a time
#pragma unroll
    for (int j = 0; j < kSteps; j += 2) {
      uint32_t v = m[j] | (m[j + 1] << 16);
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) v = __vmaxu2(v, __shfl_xor_sync(0xffffffffu, v, off));
      m[j] = v & 0xffffu;
      m[j + 1] = v >> 16;
    }
  }
  float s[kSteps / kPer];
  float s_first = 0.f;
#pragma unroll
  for (int j = 0; j < kSteps / kPer; ++j) {
    uint32_t mj = m[j];
    if constexpr (kLB > 0) mj = __reduce_max_sync(0xffffffffu, mj);
    s[j] = scale_for<F>(as_fp32<Tag>(mj));
    // the block's tokens are [b0, b0 + 2^kLB); those written start at w0
    const int b0 = sp.start + 2 * kPer * j + (kLB == 0 ? half : 0);
    const int w0 = max(b0, sp.begin);
    if (kLB > 0 && has_old && b0 == held) {
      s[j] = fmaxf(s[j], s_old);
      s_first = s[j];
    }
    const uint32_t r = __shfl_sync(0xffffffffu, rows, min(w0 - sp.start, 15));
    if (w0 < min(b0 + (1 << kLB), sp.end) && r != kNoRow && (kLB == 0 ? c == 0 : lane == 0))
      scales[scale_index(a, r, h)] = s[j];
  }
  uint8_t* pool = a.pool[kv] + c * 8;
  if (kLB > 0 && has_old && s_first > s_old) {
    const float ratio = __fdiv_rn(s_old, s_first);
#pragma unroll
    for (int i = 0; i < (1 << kLB) / 2; ++i) {
      const int t = held + 2 * i + half;
      const uint32_t r = __shfl_sync(0xffffffffu, rows, (t - sp.start) & 15);
      if (t < sp.begin && r != kNoRow) rescale8<F>(pool + code_offset(a, r, h), ratio);
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int t = sp.start + 2 * i + half;
    const uint32_t r = __shfl_sync(0xffffffffu, rows, 2 * i + half);
    const float si = s[i / kPer];
    if (t >= sp.begin && t < sp.end && r != kNoRow)
      *reinterpret_cast<uint2*>(pool + code_offset(a, r, h)) =
          quantise<Tag, F>(x[i], si, __frcp_rn(si), is_pow2(si));
  }
}

// Blocks of 32 to 1024 tokens: a CTA per (block, K or V, head), of a warp per 16
// tokens but at most 8, so that every thread has its eight loads in flight
// whatever the block (64-token blocks: 8 warps of four loads each moved 3.9
// TB/s, 4 warps of eight 5.7).  The block divides the page, so its rows are
// consecutive.
template <typename Tag, typename F, int kW>
__global__ void __launch_bounds__(32 * kW) kv_append_block_kernel(const KvArgs a) {
  constexpr int kChunk = 2 * kSteps * kW;  // rows held at a time
  __shared__ uint32_t warp_max[kW];
  const uint32_t unit = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
  const uint32_t rest = unit / a.num_kv_heads;
  const int h = int(unit - rest * a.num_kv_heads), kv = int(rest & 1);
  const KvSpan sp = a.spans[rest >> 1];

  const uint16_t* x0 = a.x[kv] + h * D + c * 8;
  const int64_t stride = a.stride[kv];
  const int q0 = (sp.begin - sp.start) / kChunk, q1 = (sp.end - 1 - sp.start) / kChunk;
  uint4 x[kSteps];
  auto load = [&](int q) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int t = sp.start + q * kChunk + (i * kW + warp) * 2 + half;
      x[i] = t >= sp.begin && t < sp.end
                 ? __ldg(reinterpret_cast<const uint4*>(x0 + (sp.row + int64_t(t - sp.begin)) * stride))
                 : make_uint4(0, 0, 0, 0);
    }
  };
  load(q0);  // in flight while the page is looked up
  const uint32_t row0 = pool_row(a, a.kv_indices, a.num_pages, sp.page_begin, sp.start);
  if (row0 == kNoRow) return;  // the whole CTA: its block lies on one page

  float* scale = a.scales[kv] + scale_index(a, row0, h);
  const bool has_old = sp.start < sp.begin;
  const float s_old = has_old ? *scale : 0.f;
  uint32_t m = 0;
  for (int q = q0; q <= q1; ++q) {
    if (q > q0) load(q);
    uint32_t mq = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) mq = amax2(x[i], mq);
    mq = fold2(mq);
    if (__any_sync(0xffffffffu, mq >= Half<Tag>::kInf)) {
      mq = 0;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) mq = finite_amax<Tag>(x[i], mq);
    }
    m = max(m, mq);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) warp_max[warp] = m;
  __syncthreads();  // every thread has read the old scale, too
#pragma unroll
  for (int w = 0; w < kW; ++w) m = max(m, warp_max[w]);
  float s = scale_for<F>(as_fp32<Tag>(m));
  if (has_old) s = fmaxf(s, s_old);
  if (threadIdx.x == 0) *scale = s;

  uint8_t* pool = a.pool[kv] + c * 8;
  if (has_old && s > s_old) {
    const float ratio = __fdiv_rn(s_old, s);
    for (int t = sp.start + warp * 2 + half; t < sp.begin; t += 2 * kW)
      rescale8<F>(pool + code_offset(a, row0 + uint32_t(t - sp.start), h), ratio);
  }
  const float inv = __frcp_rn(s);
  const bool pow2 = is_pow2(s);
  for (int q = q1; q >= q0; --q) {  // the last chunk is still in registers
    if (q < q1) load(q);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int t = sp.start + q * kChunk + (i * kW + warp) * 2 + half;
      if (t >= sp.begin && t < sp.end)
        *reinterpret_cast<uint2*>(pool + code_offset(a, row0 + uint32_t(t - sp.start), h)) =
            quantise<Tag, F>(x[i], s, inv, pow2);
    }
  }
}

__device__ __forceinline__ uint32_t pack16(F16, float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack16(BF16, float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A warp per (16 tokens, K or V, head): scale * code, rounded once.
template <typename Tag, typename F>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvArgs a) {
  const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (unit >= a.n_units) return;
  const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
  uint32_t rest = unit / a.num_kv_heads;
  const int h = int(unit - rest * a.num_kv_heads), kv = int(rest & 1);
  rest >>= 1;
  // 16-token pieces of a longer span
  const int log2_pieces = max(a.log2_block - 4, 0);
  const int piece = int(rest & ((1 << log2_pieces) - 1));
  const KvSpan sp = a.spans[rest >> log2_pieces];
  const int t0 = sp.start + piece * kKvSpanTokens;
  const int begin = max(t0, sp.begin), end = min(t0 + kKvSpanTokens, sp.end);
  if (begin >= end) return;
  uint32_t rows = kNoRow, out_rows = kNoRow;
  if (t0 + c >= begin && t0 + c < end) {
    rows = pool_row(a, a.kv_indices, a.num_pages, sp.page_begin, t0 + c);
    out_rows = a.out_indices
                   ? pool_row(a, a.out_indices, a.num_out_pages, sp.page_begin, t0 + c)
                   : 0u;
    if (out_rows == kNoRow) rows = kNoRow;
  }
  uint2 x[kSteps];
  float s[kSteps];
  const uint8_t* pool = a.pool[kv] + c * 8;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint32_t r = __shfl_sync(0xffffffffu, rows, 2 * i + half);
    x[i] = make_uint2(0, 0);
    s[i] = 0.f;
    if (r != kNoRow) {
      x[i] = __ldg(reinterpret_cast<const uint2*>(pool + code_offset(a, r, h)));
      s[i] = __ldg(a.scales[kv] + scale_index(a, r, h));
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint32_t r = __shfl_sync(0xffffffffu, rows, 2 * i + half);
    const uint32_t ro = __shfl_sync(0xffffffffu, out_rows, 2 * i + half);
    const int t = t0 + 2 * i + half;
    if (r == kNoRow && !(a.zero_bad && t >= begin && t < end)) continue;  // bad page: 0 * 0
    float y[8];
    from_fp8x8<F>(x[i], y);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack16(Tag{}, s[i] * y[2 * e], s[i] * y[2 * e + 1]);
    const int64_t out = a.out_indices
                            ? int64_t(ro) * a.num_kv_heads * D
                            : (sp.row + int64_t(t - sp.begin)) * a.stride[kv];
    *reinterpret_cast<uint4*>(a.x[kv] + out + h * D + c * 8) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

KvArgs make_args(const pa_plan_s& plan, const KvPointers& p) {
  const pa_problem& pr = plan.prob;
  KvArgs a{};
  a.x[0] = static_cast<uint16_t*>(p.k);
  a.x[1] = static_cast<uint16_t*>(p.v);
  a.stride[0] = p.k_stride;
  a.stride[1] = p.v_stride;
  a.pool[0] = static_cast<uint8_t*>(p.k_pool);
  a.pool[1] = static_cast<uint8_t*>(p.v_pool);
  a.scales[0] = p.k_scales;
  a.scales[1] = p.v_scales;
  a.kv_indices = p.kv_indices;
  a.out_indices = p.out_indices;
  a.spans = reinterpret_cast<const KvSpan*>(p.ws + plan.ws.kv_spans);
  a.error_pos = reinterpret_cast<unsigned long long*>(p.ws + plan.ws.error);
  a.num_pages = pr.num_pages;
  a.num_out_pages = p.num_out_pages;
  a.n_units = uint32_t(plan.kv_spans.size()) * 2u * uint32_t(pr.num_kv_heads);
  a.num_kv_heads = pr.num_kv_heads;
  a.log2_page = plan.log2_page;
  while ((1 << a.log2_block) < plan.scale_block) ++a.log2_block;
  a.check = (pr.flags & PA_FLAG_CHECK_INDICES) != 0;
  return a;
}

template <typename Tag, typename F>
void launch_append(const KvArgs& a, cudaStream_t s) {
  const unsigned ctas = (a.n_units + kWarps - 1) / kWarps;
  switch (a.log2_block) {
    case 0: kv_append_warp_kernel<Tag, F, 0><<<ctas, kThreads, 0, s>>>(a); break;
    case 1: kv_append_warp_kernel<Tag, F, 1><<<ctas, kThreads, 0, s>>>(a); break;
    case 2: kv_append_warp_kernel<Tag, F, 2><<<ctas, kThreads, 0, s>>>(a); break;
    case 3: kv_append_warp_kernel<Tag, F, 3><<<ctas, kThreads, 0, s>>>(a); break;
    case 4: kv_append_warp_kernel<Tag, F, 4><<<ctas, kThreads, 0, s>>>(a); break;
    case 5: kv_append_block_kernel<Tag, F, 2><<<a.n_units, 64, 0, s>>>(a); break;
    case 6: kv_append_block_kernel<Tag, F, 4><<<a.n_units, 128, 0, s>>>(a); break;
    default: kv_append_block_kernel<Tag, F, 8><<<a.n_units, 256, 0, s>>>(a);
  }
}

}  // namespace

int launch_kv_append(const pa_plan_s& plan, const KvPointers& p, void* stream) {
  const KvArgs a = make_args(plan, p);
  if (a.n_units == 0) return 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = plan.prob.kv_dtype == PA_E4M3;
  if (plan.prob.dtype == PA_BF16)
    e4m3 ? launch_append<BF16, E4M3>(a, s) : launch_append<BF16, E5M2>(a, s);
  else
    e4m3 ? launch_append<F16, E4M3>(a, s) : launch_append<F16, E5M2>(a, s);
  return int(cudaGetLastError());
}

int launch_kv_read(const pa_plan_s& plan, const KvPointers& p, void* stream) {
  KvArgs a = make_args(plan, p);
  if (a.n_units == 0) return 0;
  a.zero_bad = !p.out_indices && p.num_out_pages == PA_KV_ZERO_BAD_ROWS;
  if (a.log2_block > 4) a.n_units <<= a.log2_block - 4;  // 16-token pieces of a span
  const unsigned ctas = (a.n_units + kWarps - 1) / kWarps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = plan.prob.kv_dtype == PA_E4M3;
  if (plan.prob.dtype == PA_BF16)
    e4m3 ? kv_read_kernel<BF16, E4M3><<<ctas, kThreads, 0, s>>>(a)
         : kv_read_kernel<BF16, E5M2><<<ctas, kThreads, 0, s>>>(a);
  else
    e4m3 ? kv_read_kernel<F16, E4M3><<<ctas, kThreads, 0, s>>>(a)
         : kv_read_kernel<F16, E5M2><<<ctas, kThreads, 0, s>>>(a);
  return int(cudaGetLastError());
}

}  // namespace pa
