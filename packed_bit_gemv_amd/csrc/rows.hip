// add_rmsnorm and quantize_rows: the row kernels in front of the linears.
//
// add_rmsnorm: r = x + residual, p = r * w, h = fp16(p / sqrt(mean r^2 + eps)),
// and the same row in 8 bits: with A = max |p|, q = rint(p * f), f = 127 * (1 / A), and
// q_scale = A / (127 * sqrt(mean r^2 + eps)). The norm's factor scales p and A
// alike and so cancels in q: a code depends on single IEEE operations on one
// element and on A, never on the order of the sum of squares. quantize_rows: the same codes of an fp16 row.
//
// A row whose r or p holds NaN or an infinity, or whose sum of squares leaves
// fp32, has no 8-bit form: its codes are 0 and its scale is NaN, so that the
// products that use it show it. With r or the sum, its h is NaN too.
#include "pbg_device.hpp"
#include "pbg_internal.hpp"

namespace pbg {
namespace {

constexpr float kTiny = 0x1p-100f;  // rows below this have codes 0 and scale 0 (1 / A stays finite)
constexpr uint32_t kInfBits = 0x7F800000u;
// From here on small workgroups, several of them on a CU, beat one large workgroup a row: 1,024 rows of 4,096 columns
// normed in 12.5 against 15.8 us, 4,096 rows of 8,192 quantized in 18.2 against 21.6; below it a large one ends a row
// sooner: one row 3.2 against 3.5 us, 256 rows 5.75 against 6.0, one row of 12,288 quantized 2.8 against 3.3.
constexpr int64_t kManyRows = 1024;

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Sum of s and maximum of t over the workgroup's W waves; every thread gets
// both, summed in one fixed order. Row rotates and lane swaps inside a wave,
// one pass through LDS between the waves.
template <int W>
__device__ __forceinline__ void block_sum_max(float& s, uint32_t& t) {
  s = row_sum16(s);
  t = max_u32(t, as_u32(row_ror<8>(as_f32(t))));
  t = max_u32(t, as_u32(row_ror<4>(as_f32(t))));
  t = max_u32(t, as_u32(row_ror<2>(as_f32(t))));
  t = max_u32(t, as_u32(row_ror<1>(as_f32(t))));
  auto s16 = __builtin_amdgcn_permlane16_swap(as_u32(s), as_u32(s), false, false);
  auto t16 = __builtin_amdgcn_permlane16_swap(t, t, false, false);
  s = as_f32(s16[0]) + as_f32(s16[1]);
  t = max_u32(t16[0], t16[1]);
  auto s32 = __builtin_amdgcn_permlane32_swap(as_u32(s), as_u32(s), false, false);
  auto t32 = __builtin_amdgcn_permlane32_swap(t, t, false, false);
  s = as_f32(s32[0]) + as_f32(s32[1]);
  t = max_u32(t32[0], t32[1]);
  if constexpr (W > 1) {
    __shared__ float ps[W];
    __shared__ uint32_t pt[W];
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
      t = max_u32(t, pt[w]);
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

typedef float f32x4_t __attribute__((ext_vector_type(4)));
// The same at the alignment of their elements: the hardware takes vector loads and stores at any address.
typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(2)));

// Four fp32 elements from column c, 0 from column k on.
__device__ __forceinline__ f32x4_t load4(const float* row, int c, int k) {
  f32x4_t v = {};
  if (c + 4 <= k) {
    v = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any_t*>(row + c));
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (c + e < k) v[e] = row[c + e];
  }
  return v;
}

// Four codes as bytes.
__device__ __forceinline__ uint32_t codes4(f32x4_t p, float f) {
  return static_cast<uint32_t>(code_of(p[0], f) & 0xFF) | static_cast<uint32_t>(code_of(p[1], f) & 0xFF) << 8 |
         static_cast<uint32_t>(code_of(p[2], f) & 0xFF) << 16 | static_cast<uint32_t>(code_of(p[3], f)) << 24;
}

// One workgroup of T threads a row, the row read once and held in registers
// (V groups of four columns a thread), both reductions in one pass. Bound by
// the bytes, each of x, residual and the outputs crossing HBM once: 4,096 rows
// of 4,096 with every output take 47-49 us, 5.1-5.4 TB/s, above what a copy
// reaches. One row is bound by its launch and one trip to memory (3.0 us).
template <int T, int V>
__global__ __launch_bounds__(T) void add_rmsnorm_kernel(const float* x, const float* residual,
                                                        const float* __restrict__ weight, float eps, int k, int kp,
                                                        float* residual_out, uint16_t* __restrict__ h,
                                                        int8_t* __restrict__ q, float* __restrict__ q_scale) {
  const int64_t row = blockIdx.x;
  const int64_t base = row * k;
  f32x4_t p[V], w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] = load4(x + base, 4 * (threadIdx.x + i * T), k);
  if (residual) {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] += load4(residual + base, 4 * (threadIdx.x + i * T), k);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = 4 * (threadIdx.x + i * T);
    w[i] = f32x4_t{};
    if (c + 4 <= k) {
      w[i] = *reinterpret_cast<const f32x4_any_t*>(weight + c);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (c + e < k) w[i][e] = weight[c + e];
    }
  }
  float sum = 0.0f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = 4 * (threadIdx.x + i * T);
    if (residual_out) {
      if (c + 4 <= k) {
        *reinterpret_cast<f32x4_any_t*>(residual_out + base + c) = p[i];
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (c + e < k) residual_out[base + c + e] = p[i][e];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += p[i][e] * p[i][e];
    p[i] *= w[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max_u32(top, mag(p[i][e]));
  }
  block_sum_max<T / kWave>(sum, top);
  const float norm = norm_factor(sum, k, eps);
  if (h) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = 4 * (threadIdx.x + i * T);
      uint32_t b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = half_bits(p[i][e] * norm);
      if (c + 4 <= k) {
        u32x2_any_t two = {b[0] | b[1] << 16, b[2] | b[3] << 16};
        *reinterpret_cast<u32x2_any_t*>(h + base + c) = two;
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (c + e < k) h[base + c + e] = static_cast<uint16_t>(b[e]);
      }
    }
  }
  if (q) {
    float scale;
    const float f = code_factor(top, norm, scale);
    uint32_t* qr = reinterpret_cast<uint32_t*>(q + row * kp);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int g = threadIdx.x + i * T;
      if (4 * g < k) qr[g] = codes4(p[i], f);  // columns past k hold 0
    }
    const int pad = (k + 3) / 4 + threadIdx.x;
    if (pad < kp / 4) qr[pad] = 0;
    if (threadIdx.x == 0) q_scale[row] = scale;
  }
}

// The same for fp16 rows, V groups of eight columns a thread: 2,048 rows of
// 12,288 take 14.0-14.3 us, 5.3 TB/s.
template <int T, int V>
__global__ __launch_bounds__(T) void quantize_rows_kernel(const uint16_t* __restrict__ x, int k, int kp,
                                                          int8_t* __restrict__ q, float* __restrict__ q_scale) {
  const int64_t row = blockIdx.x;
  const uint16_t* xr = x + row * k;
  u32x4_t v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = 8 * (threadIdx.x + i * T);
    v[i] = u32x4_t{};
    if (c + 8 <= k) {
      v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any_t*>(xr + c));
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (c + e < k) v[i][e / 2] |= static_cast<uint32_t>(xr[c + e]) << (16 * (e & 1));
    }
  }
  // fp16 magnitudes order like their bits: the maximum is taken on both halves of a word
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo = max_u32(lo, v[i][e] & 0x7FFFu);
      hi = max_u32(hi, v[i][e] & 0x7FFF0000u);
    }
  const uint16_t both = static_cast<uint16_t>(max_u32(lo, hi >> 16));
  uint32_t top = mag(static_cast<float>(__builtin_bit_cast(_Float16, both)));
  float none = 0.0f;
  block_sum_max<T / kWave>(none, top);
  float scale;
  const float f = code_factor(top, 1.0f, scale);
  uint64_t* qr = reinterpret_cast<uint64_t*>(q + row * kp);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int g = threadIdx.x + i * T;
    float c[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t word = v[i][e];
      const half2_t two = __builtin_bit_cast(half2_t, word);
      c[2 * e] = static_cast<float>(two[0]);
      c[2 * e + 1] = static_cast<float>(two[1]);
    }
    const f32x4_t a = {c[0], c[1], c[2], c[3]}, b = {c[4], c[5], c[6], c[7]};
    if (8 * g < k) qr[g] = codes4(a, f) | static_cast<uint64_t>(codes4(b, f)) << 32;
  }
  const int pad = (k + 7) / 8 + threadIdx.x;
  if (pad < kp / 8) qr[pad] = 0;
  if (threadIdx.x == 0) q_scale[row] = scale;
}

// Rows too long for registers: one workgroup a row, the row read twice. The second
// pass reads r back from residual_out where it is given (it may be the
// buffer of x or residual); a thread reads only what it wrote itself. Single
// elements a load, so far from the row kernels: 256 rows of 20,000 columns with
// every output take 65 us (256 of 16,384 in registers 12.1), one row 39 (5.7);
// 256 rows of 40,000 quantized 70 us (256 of 32,768 6.1), one row 43 (3.9).
constexpr int kLongThreads = 256;

__global__ __launch_bounds__(kLongThreads) void add_rmsnorm_long_kernel(const float* x, const float* residual,
                                                                      const float* __restrict__ weight, float eps,
                                                                      int64_t k, int64_t kp, float* residual_out,
                                                                      uint16_t* __restrict__ h, int8_t* __restrict__ q,
                                                                      float* __restrict__ q_scale) {
  const int64_t row = blockIdx.x;
  const int64_t base = row * k;
  float sum = 0.0f;
  uint32_t top = 0;
  for (int64_t j = threadIdx.x; j < k; j += kLongThreads) {
    float r = x[base + j];
    if (residual) r += residual[base + j];
    if (residual_out) residual_out[base + j] = r;
    sum += r * r;
    const uint32_t b = mag(r * weight[j]);
    top = b > top ? b : top;
  }
  block_sum_max<kLongThreads / kWave>(sum, top);
  const float norm = norm_factor(sum, k, eps);
  float scale;
  const float f = code_factor(top, norm, scale);
  for (int64_t j = threadIdx.x; j < (q ? kp : k); j += kLongThreads) {
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

__global__ __launch_bounds__(kLongThreads) void quantize_rows_long_kernel(const uint16_t* __restrict__ x, int64_t k,
                                                                        int64_t kp, int8_t* __restrict__ q,
                                                                        float* __restrict__ q_scale) {
  const int64_t row = blockIdx.x;
  float none = 0.0f;
  uint32_t top = 0;
  for (int64_t j = threadIdx.x; j < k; j += kLongThreads) {
    const uint32_t b = mag(static_cast<float>(__builtin_bit_cast(_Float16, x[row * k + j])));
    top = b > top ? b : top;
  }
  block_sum_max<kLongThreads / kWave>(none, top);
  float scale;
  const float f = code_factor(top, 1.0f, scale);
  for (int64_t j = threadIdx.x; j < kp; j += kLongThreads) {
    const float p = j < k ? static_cast<float>(__builtin_bit_cast(_Float16, x[row * k + j])) : 0.0f;
    q[row * kp + j] = static_cast<int8_t>(code_of(p, f));
  }
  if (threadIdx.x == 0) q_scale[row] = scale;
}

}  // namespace

namespace {

template <int T, int V>
void launch_norm(const float* x, const float* residual, const float* weight, float eps, int64_t m, int64_t k,
                 float* residual_out, uint16_t* h, int8_t* q, float* q_scale, hipStream_t stream) {
  hipLaunchKernelGGL((add_rmsnorm_kernel<T, V>), dim3(static_cast<unsigned>(m)), dim3(T), 0, stream, x, residual,
                     weight, eps, static_cast<int>(k), static_cast<int>(q8_row_bytes(k)), residual_out, h, q, q_scale);
}

template <int T, int V>
void launch_quant(const uint16_t* x, int64_t m, int64_t k, int8_t* q, float* q_scale, hipStream_t stream) {
  hipLaunchKernelGGL((quantize_rows_kernel<T, V>), dim3(static_cast<unsigned>(m)), dim3(T), 0, stream, x,
                     static_cast<int>(k), static_cast<int>(q8_row_bytes(k)), q, q_scale);
}

}  // namespace

hipError_t launch_add_rmsnorm(const float* x, const float* residual, const float* weight, float eps, int64_t m,
                              int64_t k, float* residual_out, uint16_t* h, int8_t* q, float* q_scale,
                              hipStream_t stream) {
  const int64_t groups = (k + 3) / 4;
  if (groups > 4096) {
    hipLaunchKernelGGL(add_rmsnorm_long_kernel, dim3(static_cast<unsigned>(m)), dim3(kLongThreads), 0, stream, x,
                       residual, weight, eps, k, q8_row_bytes(k), residual_out, h, q, q_scale);
    return hipGetLastError();
  }
#define PBG_NORM(T, V) launch_norm<T, V>(x, residual, weight, eps, m, k, residual_out, h, q, q_scale, stream)
  if (groups <= 256) PBG_NORM(256, 1);
  else if (m >= kManyRows && groups <= 512) PBG_NORM(256, 2);
  else if (m >= kManyRows && groups <= 1024) PBG_NORM(256, 4);
  else if (groups <= 512) PBG_NORM(512, 1);
  else if (groups <= 1024) PBG_NORM(1024, 1);
  else if (groups <= 2048) PBG_NORM(1024, 2);
  else PBG_NORM(1024, 4);
#undef PBG_NORM
  return hipGetLastError();
}

hipError_t launch_quantize_rows(const uint16_t* x, int64_t m, int64_t k, int8_t* q, float* q_scale,
                                hipStream_t stream) {
  const int64_t groups = (k + 7) / 8;
  if (groups > 4096) {
    hipLaunchKernelGGL(quantize_rows_long_kernel, dim3(static_cast<unsigned>(m)), dim3(kLongThreads), 0, stream, x, k,
                       q8_row_bytes(k), q, q_scale);
    return hipGetLastError();
  }
#define PBG_QUANT(T, V) launch_quant<T, V>(x, m, k, q, q_scale, stream)
  if (groups <= 256) PBG_QUANT(256, 1);
  else if (m >= kManyRows && groups <= 512) PBG_QUANT(256, 2);
  else if (m >= kManyRows && groups <= 1024) PBG_QUANT(256, 4);
  else if (m >= kManyRows && groups <= 2048) PBG_QUANT(256, 8);
  else if (groups <= 512) PBG_QUANT(512, 1);
  else if (groups <= 1024) PBG_QUANT(1024, 1);
  else if (groups <= 2048) PBG_QUANT(1024, 2);
  else PBG_QUANT(1024, 4);
#undef PBG_QUANT
  return hipGetLastError();
}

}  // namespace pbg
