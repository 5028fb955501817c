// penalize_logits: penalties for repeated tokens, biases and grammar masks on logits, and the greedy token.
#include "pbg_device.hpp"
#include "pbg_internal.hpp"

namespace pbg {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));

constexpr uint32_t kGiven = 0x80000000u;  // the prompt holds the token; the low bits count the output's

__device__ __forceinline__ unsigned long long max_u64(unsigned long long a, unsigned long long b) {
  return a > b ? a : b;
}

__device__ __forceinline__ uint32_t min_u32(uint32_t a, uint32_t b) { return a < b ? a : b; }

// Key of the largest value over the workgroup's W waves, for every thread: each brings its own largest and the place
// of the first that is as large, kNowhere where it has none above -infinity. Inside a wave the value first and then
// the lowest place of it, by row rotates and lane swaps (as 64-bit keys through shuffles one row takes 7.2 us, so 7.0,
// and 64 rows 25.8 and 25.2).
constexpr uint32_t kNowhere = 0xFFFFFFFFu;

template <int W>
__device__ __forceinline__ unsigned long long block_best(float high, uint32_t at, int64_t base) {
  float top = high;
  top = fmaxf(top, row_ror<8>(top));
  top = fmaxf(top, row_ror<4>(top));
  top = fmaxf(top, row_ror<2>(top));
  top = fmaxf(top, row_ror<1>(top));
  const auto t16 = __builtin_amdgcn_permlane16_swap(as_u32(top), as_u32(top), false, false);
  top = fmaxf(as_f32(t16[0]), as_f32(t16[1]));
  const auto t32 = __builtin_amdgcn_permlane32_swap(as_u32(top), as_u32(top), false, false);
  top = fmaxf(as_f32(t32[0]), as_f32(t32[1]));
  uint32_t place = high == top ? at : kNowhere;
  place = min_u32(place, as_u32(row_ror<8>(as_f32(place))));
  place = min_u32(place, as_u32(row_ror<4>(as_f32(place))));
  place = min_u32(place, as_u32(row_ror<2>(as_f32(place))));
  place = min_u32(place, as_u32(row_ror<1>(as_f32(place))));
  const auto p16 = __builtin_amdgcn_permlane16_swap(place, place, false, false);
  place = min_u32(p16[0], p16[1]);
  const auto p32 = __builtin_amdgcn_permlane32_swap(place, place, false, false);
  place = min_u32(p32[0], p32[1]);
  __shared__ unsigned long long part[W];
  if ((threadIdx.x & (kWave - 1)) == 0)
    part[threadIdx.x / kWave] = place == kNowhere ? 0 : argmax_key(top, base + place);
  __syncthreads();
  unsigned long long key = part[0];
#pragma unroll
  for (int w = 1; w < W; ++w) key = max_u64(key, part[w]);
  return key;
}

struct LogitsArgs {
  const float* logits;
  const int32_t* request;
  const int32_t* tokens;
  int64_t tokens_width;
  const int32_t* prompt_length;
  const int32_t* length;
  const float* repetition;
  const float* frequency;
  const float* presence;
  int requests;
  const int32_t* drafts;
  const int32_t* row_start;
  const uint64_t* ancestors;
  const int32_t* bias_start;
  const int32_t* bias_token;
  const float* bias_value;
  int64_t bias_entries;
  const uint32_t* grammar;
  const int32_t* grammar_row;
  int64_t states;
  int64_t m, n;
  float* out;
  unsigned long long* best;  // [m][slices], or null
};

typedef __attribute__((address_space(4))) int32_t const_int_t;  // read through the scalar cache
typedef __attribute__((address_space(4))) float const_float_t;
typedef __attribute__((address_space(4))) uint64_t const_u64_t;

template <typename C, typename P>
__device__ __forceinline__ C* scalars(P* p) {
  return (C*)p;
}

// A workgroup of T threads takes a slice of 4 V T tokens of one row: it counts
// the row's tokens that fall into the slice in LDS, then makes one pass over
// the slice's logits, which were loaded before. Everything that the row's
// request says is loaded together, and the history several loads at a time.
// The results are stored past the caches, the logits, which the head has just
// written, are read through them (64 rows: 22.2 us; 23.5 with ordinary stores, 22.6
// with loads past the caches too).
template <int T, int V>
__global__ __launch_bounds__(T) void penalize_kernel(LogitsArgs a, int slices) {
  constexpr int kSlice = 4 * V * T;
  constexpr int kAhead = 8;
  __shared__ __attribute__((aligned(16))) uint32_t count[kSlice];
  const int64_t row = blockIdx.x / static_cast<unsigned>(slices);
  const int slice = blockIdx.x % static_cast<unsigned>(slices);
  const int i = scalars<const const_int_t>(a.request)[row];
  const uint64_t anc = a.drafts ? scalars<const const_u64_t>(a.ancestors)[row] : 0;
  const int64_t state = a.grammar ? scalars<const const_int_t>(a.grammar_row)[row] : -1;
  if (i < 0 || i >= a.requests) return;
  const int tid = threadIdx.x;
  const int64_t base = static_cast<int64_t>(slice) * kSlice;
  const int len = static_cast<int>(a.n - base < kSlice ? a.n - base : kSlice);
  const float* x = a.logits + row * a.n + base;
  f32x4_t v[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = 4 * (tid + k * T);
    v[k] = f32x4_t{};
    if (c + 4 <= len) {
      v[k] = *reinterpret_cast<const f32x4_any_t*>(x + c);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (c + e < len) v[k][e] = x[c + e];
    }
  }
  const int64_t held = scalars<const const_int_t>(a.length)[i], width = a.tokens_width;
  const int used = static_cast<int>(held < 0 ? 0 : held < width ? held : width);
  const int prompt = scalars<const const_int_t>(a.prompt_length)[i];
  const float rep = scalars<const const_float_t>(a.repetition)[i], freq = scalars<const const_float_t>(a.frequency)[i];
  const float pres = scalars<const const_float_t>(a.presence)[i];
  const int64_t draft_at = a.drafts ? scalars<const const_int_t>(a.row_start)[i] : 0;
  int64_t from = 0, to = 0;
  if (a.bias_start) {
    from = scalars<const const_int_t>(a.bias_start)[i];
    to = scalars<const const_int_t>(a.bias_start)[i + 1];
    if (from < 0) from = 0;
    if (to > a.bias_entries) to = a.bias_entries;
  }
  const bool masks = state >= 0 && state < a.states;
  uint32_t allowed[V];
  if (masks) {
    const uint32_t* words = a.grammar + state * ((a.n + 31) / 32) + base / 32;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = 4 * (tid + k * T);
      allowed[k] = c < len ? words[c / 32] >> (c % 32) : 0u;
    }
  }
  auto clear = [&]() {
#pragma unroll
    for (int k = 0; k < V; ++k) *reinterpret_cast<uint4*>(&count[4 * (tid + k * T)]) = make_uint4(0, 0, 0, 0);
    __syncthreads();
  };
  if (used > 0 || anc) {
    clear();
    const int32_t* said = a.tokens + i * width;
    const uint32_t lo = static_cast<uint32_t>(base);
    for (int j0 = 0; j0 < used; j0 += kAhead * T) {
      int32_t token[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) token[k] = said[min(j0 + k * T + tid, used - 1)];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int j = j0 + k * T + tid;
        const uint32_t u = static_cast<uint32_t>(token[k]) - lo;
        if (j < used && u < static_cast<uint32_t>(len)) {
          if (j < prompt) atomicOr(&count[u], kGiven);
          else atomicAdd(&count[u], 1u);
        }
      }
    }
    if (tid < 64 && (anc >> tid & 1)) {
      const int64_t r = draft_at + tid;
      if (r >= 0 && r < a.m) {
        const uint32_t u = static_cast<uint32_t>(a.drafts[r]) - lo;
        if (u < static_cast<uint32_t>(len)) atomicAdd(&count[u], 1u);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const uint4 n4 = *reinterpret_cast<const uint4*>(&count[4 * (tid + k * T)]);
      const uint32_t n[4] = {n4.x, n4.y, n4.z, n4.w};
      // few groups of four hold a token that was said
      if (n4.x | n4.y | n4.z | n4.w)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // every step a rounding of its own, selected afterwards: branches around single elements cost 200 registers
        // here
#pragma clang fp contract(off)
        const float y = v[k][e];
        const float z = y > 0.0f ? y / rep : y * rep;
        const uint32_t times = n[e] & ~kGiven;
        const float f = freq * static_cast<float>(times);
        const float g = z - f;
        const float h = g - pres;
        v[k][e] = n[e] ? times ? h : z : y;
      }
    }
  }
  if (from < to) {
    // the last entry of a token, plus one
    __syncthreads();
    clear();
    for (int64_t j = from + tid; j < to; j += T) {
      const uint32_t u = static_cast<uint32_t>(a.bias_token[j]) - static_cast<uint32_t>(base);
      if (u < static_cast<uint32_t>(len)) atomicMax(&count[u], static_cast<uint32_t>(j - from) + 1u);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const uint4 n4 = *reinterpret_cast<const uint4*>(&count[4 * (tid + k * T)]);
      const uint32_t n[4] = {n4.x, n4.y, n4.z, n4.w};
      if (n4.x | n4.y | n4.z | n4.w)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float add = a.bias_value[from + (n[e] ? n[e] - 1 : 0)];
        v[k][e] = n[e] ? v[k][e] + add : v[k][e];
      }
    }
  }
  if (masks) {
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[k][e] = allowed[k] >> e & 1 ? v[k][e] : -__builtin_inff();
  }
  float* o = a.out + row * a.n + base;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = 4 * (tid + k * T);
    if (c + 4 <= len) {
      __builtin_nontemporal_store(v[k], reinterpret_cast<f32x4_any_t*>(o + c));
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (c + e < len) o[c + e] = v[k][e];
    }
  }
  if (a.best) {
    // the thread's largest value, the first of equal ones: its elements' places grow with k and e
    float high = -__builtin_inff();
    uint32_t at = kNowhere;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = 4 * (tid + k * T) + e;
        const bool more = c < len && v[k][e] > high;
        high = more ? v[k][e] : high;
        at = more ? static_cast<uint32_t>(c) : at;
      }
    const unsigned long long key = block_best<T / kWave>(high, at, base);
    if (tid == 0) a.best[row * slices + slice] = key;
  }
}

// The best of a row's slices: one wave a row.
__global__ __launch_bounds__(kWave) void logits_best_kernel(const unsigned long long* __restrict__ best, int slices,
                                                            const int32_t* __restrict__ request, int requests,
                                                            int32_t* __restrict__ token, float* __restrict__ top) {
  const int64_t row = blockIdx.x;
  const int i = request[row];
  if (i < 0 || i >= requests) return;
  unsigned long long key = 0;
  for (int s = threadIdx.x; s < slices; s += kWave) key = max_u64(key, best[row * slices + s]);
#pragma unroll
  for (int d = kWave / 2; d > 0; d /= 2) key = max_u64(key, __shfl_xor(key, d));
  if (threadIdx.x == 0) {
    token[row] = key ? argmax_key_row(key) : -1;
    top[row] = key ? argmax_key_logit(key) : -__builtin_inff();
  }
}

}  // namespace

hipError_t launch_penalize_logits(const float* logits, const int32_t* request, const int32_t* tokens,
                                  int64_t tokens_width, const int32_t* prompt_length, const int32_t* length,
                                  const float* repetition, const float* frequency, const float* presence,
                                  int64_t requests, const int32_t* drafts, const int32_t* row_start,
                                  const uint64_t* ancestors, const int32_t* bias_start, const int32_t* bias_token,
                                  const float* bias_value, int64_t bias_entries, const uint32_t* grammar,
                                  const int32_t* grammar_row, int64_t states, int64_t m, int64_t n, float* out,
                                  int32_t* token, float* top, uint64_t* workspace, hipStream_t stream) {
  const LogitsArgs a = {logits,    request,  tokens,     tokens_width, prompt_length, length,    repetition,
                        frequency, presence, static_cast<int>(requests), drafts, row_start, ancestors, bias_start,
                        bias_token, bias_value, bias_entries, grammar, grammar_row, states, m, n, out,
                        token ? reinterpret_cast<unsigned long long*>(workspace) : nullptr};
  // 4,096 tokens a workgroup: 64 rows of 151,936 (histories of 2,000, biases, grammars) take 22.2 us and one row
  // (8,000) 7.0; with 2,048 of 256 threads 21.8 and 7.5, of 512 30.2 and 6.7, with 4,096 of 1,024 threads 32.4 and
  // 6.8, of 256 threads 22.6 and 9.4, with 8,192 of 512 threads 23.3 and 8.3
  constexpr int kT = 512, kV = 2;
  const int64_t slices = (n + 4 * kV * kT - 1) / (4 * kV * kT);
  hipLaunchKernelGGL((penalize_kernel<kT, kV>), dim3(static_cast<unsigned>(m * slices)), dim3(kT), 0, stream, a,
                     static_cast<int>(slices));
  if (token)
    hipLaunchKernelGGL(logits_best_kernel, dim3(static_cast<unsigned>(m)), dim3(kWave), 0, stream, a.best,
                       static_cast<int>(slices), request, static_cast<int>(requests), token, top);
  return hipGetLastError();
}

}  // namespace pbg
