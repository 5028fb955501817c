// add_rmsnorm and quantize_rows: the row kernels in front of the linears.
//
// add_rmsnorm: r = x + residual, p = r * w, h = fp16(p / sqrt(mean r^2 + eps)),
// and the same row in 8 bits: with A = max |p|, q = rint(p * f), f = 127 * (1 / A), and
// q_scale = A / (127 * sqrt(mean r^2 + eps)). The norm's factor scales p and A
// alike and so cancels in q: a code depends on single IEEE operations on one
// element and on A, never on the order of the sum of squares. quantize_rows: the same codes of an fp16 row.
//
// A row that holds NaN or an infinity, or whose sum of squares leaves fp32,
// has no 8-bit form: its codes are 0 and its scale is NaN, so that the
// products that use it show it.
#include "pbg_device.hpp"
#include "pbg_internal.hpp"

namespace pbg {
namespace {

constexpr float kTiny = 0x1p-100f;  // rows below this have codes 0 and scale 0 (1 / A stays finite)
constexpr uint32_t kInfBits = 0x7F800000u;

// Sum of s and maximum of t over the workgroup's W waves; every thread gets both.
template <int W>
__device__ __forceinline__ void block_sum_max(float& s, uint32_t& t) {
  __shared__ float ps[W];
  __shared__ uint32_t pt[W];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    s += __shfl_xor(s, d);
    const uint32_t o = __shfl_xor(t, d);
    t = o > t ? o : t;
  }
  if constexpr (W > 1) {
    const int wave = threadIdx.x / kWave;
    if ((threadIdx.x & (kWave - 1)) == 0) {
      ps[wave] = s;
      pt[wave] = t;
    }
    __syncthreads();
    s = ps[0];
    t = pt[0];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      s += ps[w];
      t = pt[w] > t ? pt[w] : t;
    }
  }
}

// Bits of |v|: ordered like the magnitudes, with infinities and NaN on top.
__device__ __forceinline__ uint32_t mag(float v) { return as_u32(v) & 0x7FFFFFFFu; }

// Factor f of the codes (0 for a row of nothing or without an 8-bit
// form) and the row's scale, from the bits of A and the factor of the norm.
__device__ __forceinline__ float code_factor(uint32_t top, float norm, float& scale) {
  const float a = as_f32(top);
  const bool bad = top >= kInfBits || !(norm < __builtin_inff());
  const bool some = !bad && a >= kTiny;
  scale = bad ? __builtin_nanf("") : some ? a * norm / 127.0f : 0.0f;
  return some ? 127.0f * (1.0f / a) : 0.0f;
}

// The caller passes f = 0 with p possibly non-finite: that row's codes are 0.
__device__ __forceinline__ int code_of(float p, float f) { return f == 0.0f ? 0 : static_cast<int>(rintf(p * f)); }

__device__ __forceinline__ uint32_t half_bits(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

// Norm factor 1 / sqrt(mean + eps); NaN where the sum of squares is not finite.
__device__ __forceinline__ float norm_factor(float sum, int64_t k, float eps) {
  if (!(sum < __builtin_inff())) return __builtin_nanf("");
  return 1.0f / sqrtf(sum / static_cast<float>(k) + eps);
}

// Any k and alignment: one workgroup a row, the row read twice. The second
// pass reads r back from residual_out where it is given (it may be the
// buffer of x or residual); a thread reads only what it wrote itself.
constexpr int kAnyThreads = 256;

__global__ __launch_bounds__(kAnyThreads) void add_rmsnorm_any_kernel(const float* x, const float* residual,
                                                                      const float* __restrict__ weight, float eps,
                                                                      int64_t k, int64_t kp, float* residual_out,
                                                                      uint16_t* __restrict__ h, int8_t* __restrict__ q,
                                                                      float* __restrict__ q_scale) {
  const int64_t row = blockIdx.x;
  const int64_t base = row * k;
  float sum = 0.0f;
  uint32_t top = 0;
  for (int64_t j = threadIdx.x; j < k; j += kAnyThreads) {
    float r = x[base + j];
    if (residual) r += residual[base + j];
    if (residual_out) residual_out[base + j] = r;
    sum += r * r;
    const uint32_t b = mag(r * weight[j]);
    top = b > top ? b : top;
  }
  block_sum_max<kAnyThreads / kWave>(sum, top);
  const float norm = norm_factor(sum, k, eps);
  float scale;
  const float f = code_factor(top, norm, scale);
  for (int64_t j = threadIdx.x; j < (q ? kp : k); j += kAnyThreads) {
    if (j < k) {
      float r;
      if (residual_out) {
        r = residual_out[base + j];
      } else {
        r = x[base + j];
        if (residual) r += residual[base + j];
      }
      const float p = r * weight[j];
      if (h) h[base + j] = static_cast<uint16_t>(half_bits(p * norm));
      if (q) q[row * kp + j] = static_cast<int8_t>(code_of(p, f));
    } else {
      q[row * kp + j] = 0;
    }
  }
  if (q && threadIdx.x == 0) q_scale[row] = scale;
}

__global__ __launch_bounds__(kAnyThreads) void quantize_rows_any_kernel(const uint16_t* __restrict__ x, int64_t k,
                                                                        int64_t kp, int8_t* __restrict__ q,
                                                                        float* __restrict__ q_scale) {
  const int64_t row = blockIdx.x;
  float none = 0.0f;
  uint32_t top = 0;
  for (int64_t j = threadIdx.x; j < k; j += kAnyThreads) {
    const uint32_t b = mag(static_cast<float>(__builtin_bit_cast(_Float16, x[row * k + j])));
    top = b > top ? b : top;
  }
  block_sum_max<kAnyThreads / kWave>(none, top);
  float scale;
  const float f = code_factor(top, 1.0f, scale);
  for (int64_t j = threadIdx.x; j < kp; j += kAnyThreads) {
    const float p = j < k ? static_cast<float>(__builtin_bit_cast(_Float16, x[row * k + j])) : 0.0f;
    q[row * kp + j] = static_cast<int8_t>(code_of(p, f));
  }
  if (threadIdx.x == 0) q_scale[row] = scale;
}

}  // namespace

hipError_t launch_add_rmsnorm(const float* x, const float* residual, const float* weight, float eps, int64_t m,
                              int64_t k, float* residual_out, uint16_t* h, int8_t* q, float* q_scale,
                              hipStream_t stream) {
  hipLaunchKernelGGL(add_rmsnorm_any_kernel, dim3(static_cast<unsigned>(m)), dim3(kAnyThreads), 0, stream, x, residual,
                     weight, eps, k, q8_row_bytes(k), residual_out, h, q, q_scale);
  return hipGetLastError();
}

hipError_t launch_quantize_rows(const uint16_t* x, int64_t m, int64_t k, int8_t* q, float* q_scale,
                                hipStream_t stream) {
  hipLaunchKernelGGL(quantize_rows_any_kernel, dim3(static_cast<unsigned>(m)), dim3(kAnyThreads), 0, stream, x, k,
                     q8_row_bytes(k), q, q_scale);
  return hipGetLastError();
}

}  // namespace pbg
