// cache_plan and rotary_qkv: the tables of a step over the paged cache, and the
// step's queries, keys and values from the q|k|v linear's output.
#include "pbg_device.hpp"
#include "pbg_internal.hpp"
#include "pbg_scan.hpp"

namespace pbg {
namespace {

constexpr int kPlanRows = 256;                    // rows a workgroup writes
constexpr int kTree = 64;                         // rows of one request that a tree can have
constexpr int kPlanThreads = kPlanRows + kTree;   // the rows before them hold their ancestors
constexpr int kPlanWaves = kPlanThreads / kWave;
constexpr int kMaxRequests = 4096;

// Every workgroup adds up all requests again (their two numbers come from the
// caches), so that one launch needs no second pass, and then writes
// its own rows. An entry of the table is read only for pages that the request
// held before (page index < have) and written only from there on, by the row
// that stands first in the page, so that no workgroup waits for another.
// Bound by its launch and the chain of loads: a request's numbers, then
// the table or the stack.
__global__ __launch_bounds__(kPlanThreads) void cache_plan_kernel(
    const int32_t* __restrict__ lengths, const int32_t* __restrict__ added, int requests, int32_t* table, int width,
    const int32_t* __restrict__ free_pages, int64_t free_capacity, const int32_t* __restrict__ free_count,
    int64_t pages, int shift, const int32_t* __restrict__ parents, int m, int32_t* __restrict__ row_start,
    int32_t* __restrict__ request, int32_t* __restrict__ position, int64_t* __restrict__ slot,
    uint64_t* __restrict__ ancestors, int32_t* __restrict__ free_left) {
  __shared__ int start[kMaxRequests + 1];
  __shared__ int opened[kMaxRequests + 1];  // pages that the requests before open
  __shared__ int64_t waves[kPlanWaves];
  __shared__ uint64_t mask[kPlanThreads];
  __shared__ int16_t up[kPlanThreads];
  __shared__ int8_t steps[kPlanThreads];
  const int tid = threadIdx.x;
  const int per = (requests + kPlanThreads - 1) / kPlanThreads;
  const int first = min(tid * per, requests), last = min(first + per, requests);
  // rows before each request, ending at the m-th; up to 2^32 in sum before that
  int64_t rows = 0, total;
  for (int i = first; i < last; ++i) rows += min(max(added[i], 0), m);
  int64_t at = block_scan<kPlanWaves>(rows, waves, total);
  int64_t open = 0;
  for (int i = first; i < last; ++i) {
    const int s = static_cast<int>(min(at, static_cast<int64_t>(m)));
    at += min(max(added[i], 0), m);
    const int n = static_cast<int>(min(at, static_cast<int64_t>(m))) - s;
    const int64_t len = max(lengths[i], 0), round = (1 << shift) - 1;
    const int64_t have = (len + round) >> shift;
    const int64_t want = min((len + n + round) >> shift, static_cast<int64_t>(width));
    start[i] = s;
    opened[i] = static_cast<int>(max(want - have, static_cast<int64_t>(0)));
    open += opened[i];
  }
  const int end = static_cast<int>(min(total, static_cast<int64_t>(m)));
  int64_t opens;
  int64_t before = block_scan<kPlanWaves>(open, waves, opens);
  for (int i = first; i < last; ++i) {
    const int o = opened[i];
    opened[i] = static_cast<int>(before);
    before += o;
  }
  if (tid == 0) start[requests] = end;
  __syncthreads();
  const int64_t free = min(max(static_cast<int64_t>(free_count[0]), static_cast<int64_t>(0)), free_capacity);
  if (blockIdx.x == 0) {
    for (int i = tid; i <= requests; i += kPlanThreads) row_start[i] = start[i];
    if (tid == 0) free_left[0] = static_cast<int32_t>(max(free - opens, static_cast<int64_t>(0)));
  }

  const int row = static_cast<int>(blockIdx.x) * kPlanRows + tid - kTree;
  const bool live = row >= 0 && row < end;
  int i = 0, c = 0;
  if (live) {
    // the last request that starts at the row or before it and has rows
    int lo = 0, hi = requests;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (start[mid + 1] > row) hi = mid;
      else lo = mid + 1;
    }
    i = lo;
    c = row - start[i];
  }
  // Ancestors by doubling: after k rounds mask holds the 2^k nearest rows on the way up and `up` the next one.
  uint64_t bits = 0;
  int depth = c;
  if (parents) {
    int next = -1;
    if (live && c < kTree) {
      bits = 1ull << c;
      const int p = parents[row];
      next = p >= 0 && p < c ? tid - (c - p) : -1;
    }
    int way = next >= 0;
    mask[tid] = bits;
    up[tid] = static_cast<int16_t>(next);
    steps[tid] = static_cast<int8_t>(way);
    __syncthreads();
#pragma unroll
    for (int k = 1; k < kTree; k *= 2) {
      uint64_t more = 0;
      int further = -1, longer = 0;
      if (next >= 0) {
        more = mask[next];
        further = up[next];
        longer = steps[next];
      }
      __syncthreads();
      bits |= more;
      way += longer;
      next = further;
      mask[tid] = bits;
      up[tid] = static_cast<int16_t>(next);
      steps[tid] = static_cast<int8_t>(way);
      __syncthreads();
    }
    depth = way;
  } else if (live) {
    bits = c >= kTree - 1 ? ~0ull : (2ull << c) - 1;
  }
  if (tid < kTree || row >= m) return;
  const bool stands = live && !(parents && c >= kTree);
  const int64_t len = live ? max(lengths[i], 0) : 0;
  const int64_t t = len + c, page = t >> shift, have = (len + (1 << shift) - 1) >> shift;
  int64_t number = -1;
  if (live && page < width) {
    if (page < have) {
      number = table[static_cast<int64_t>(i) * width + page];
    } else {
      const int64_t j = free - 1 - (opened[i] + (page - have));
      if (j >= 0) number = free_pages[j];
    }
    if (number < 0 || number >= pages) number = -1;
    if (page >= have && (t & ((1 << shift) - 1)) == 0)
      table[static_cast<int64_t>(i) * width + page] = static_cast<int32_t>(number);
  }
  request[row] = live ? i : -1;
  position[row] = stands ? static_cast<int32_t>(min(len + depth, static_cast<int64_t>(0x7FFFFFFF))) : -1;
  slot[row] = stands && number >= 0 ? (number << shift) + (t & ((1 << shift) - 1)) : -1;
  if (ancestors) ancestors[row] = stands ? bits : 0;
}

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4_t load4(const float* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const f32x4_any_t*>(p));
}

struct RotaryArgs {
  const float* qkv;
  const int32_t* position;
  const int64_t* slot;
  const double* inv_freq;
  const float* q_weight;
  const float* k_weight;
  float eps, amplitude;
  int m, heads, kv_heads, d, rot;
  uint16_t* q;
  uint16_t* k_cache;
  uint16_t* v_cache;
  int64_t slots;
  int shift;
};

// LPH lanes hold a head, eight elements a lane: four pairs, of which the
// halves layout takes two pieces of four elements, the interleaved one and
// elements past the turned ones one piece of eight. A pair and its angle stay
// in one lane. A wave takes U times 64 / LPH heads of one row, so that the
// angles (64-bit products, reduced to a part of a turn before they are rounded to fp32)
// are made once for them.
template <int LPH, bool INTER, int U>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
  constexpr int kHeads = kWave / LPH;  // heads a wave takes at once
  const int lane = threadIdx.x & (kWave - 1);
  const int all = a.heads + 2 * a.kv_heads;
  const int pieces = (all + U * kHeads - 1) / (U * kHeads);
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / kWave;
  const int64_t row = w / pieces;
  if (row >= a.m) return;
  const int piece = static_cast<int>(w - row * pieces);
  const int pos = a.position[row];
  if (pos < 0) return;
  const int part = lane % LPH, d = a.d, rot = a.rot;
  const bool mine = 8 * part < d;
  const bool turns = 8 * part < rot;
  // the lane's two pieces of four elements
  const int e0 = !INTER && turns ? 4 * part : 8 * part;
  const int e1 = !INTER && turns ? 4 * part + rot / 2 : 8 * part + 4;
  f32x4_t x0[U], x1[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int head = (piece * U + u) * kHeads + lane / LPH;
    x0[u] = f32x4_t{};
    x1[u] = f32x4_t{};
    if (mine && head < all) {
      // values are cast, not turned: two pieces side by side
      const bool v = head >= a.heads + a.kv_heads;
      const float* p = a.qkv + (row * all + head) * d;
      x0[u] = load4(p + (v ? 8 * part : e0));
      x1[u] = load4(p + (v ? 8 * part + 4 : e1));
    }
  }
  const int64_t slot = a.slot[row];
  float c[4], s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    c[j] = 1.0f;
    s[j] = 0.0f;
    if (turns) {
      const double turn = pos * a.inv_freq[4 * part + j] * 0.15915494309189533577;  // 1 / (2 pi)
      float sine, cosine;
      sincospif(static_cast<float>(2.0 * (turn - rint(turn))), &sine, &cosine);
      c[j] = cosine * a.amplitude;
      s[j] = sine * a.amplitude;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int head = (piece * U + u) * kHeads + lane / LPH;
    const bool is_q = head < a.heads, is_v = head >= a.heads + a.kv_heads;
    const float* weight = is_q ? a.q_weight : a.k_weight;
    f32x4_t y0 = x0[u], y1 = x1[u];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += y0[j] * y0[j] + y1[j] * y1[j];
#pragma unroll
    for (int k = LPH / 2; k > 0; k /= 2) sum += __shfl_xor(sum, k);
    float eps = a.eps;
    if (__any(sum > __FLT_MAX__)) {
      // Squares that leave fp32: such a head is taken times 2^-70, which its norm takes out again. (An infinite element
      // stays infinite.)
      const bool large = sum > __FLT_MAX__ && weight && !is_v;
      const float down = large ? 0x1p-70f : 1.0f;
      y0 *= down;
      y1 *= down;
      float less = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) less += y0[j] * y0[j] + y1[j] * y1[j];
#pragma unroll
      for (int k = LPH / 2; k > 0; k /= 2) less += __shfl_xor(less, k);
      if (large) sum = less;
      eps *= down * down;
    }
    if (head >= all || !mine) continue;
    if (!is_v) {
      if (weight) {
        const float norm = 1.0f / sqrtf(sum / static_cast<float>(d) + eps);
        const f32x4_t w0 = *reinterpret_cast<const f32x4_any_t*>(weight + e0);
        const f32x4_t w1 = *reinterpret_cast<const f32x4_any_t*>(weight + e1);
        y0 *= w0 * norm;
        y1 *= w1 * norm;
      }
      if (turns) {
        if constexpr (INTER) {
          const f32x4_t z0 = y0, z1 = y1;
          y0[0] = z0[0] * c[0] - z0[1] * s[0];
          y0[1] = z0[1] * c[0] + z0[0] * s[0];
          y0[2] = z0[2] * c[1] - z0[3] * s[1];
          y0[3] = z0[3] * c[1] + z0[2] * s[1];
          y1[0] = z1[0] * c[2] - z1[1] * s[2];
          y1[1] = z1[1] * c[2] + z1[0] * s[2];
          y1[2] = z1[2] * c[3] - z1[3] * s[3];
          y1[3] = z1[3] * c[3] + z1[2] * s[3];
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p = y0[j], r = y1[j];
            y0[j] = p * c[j] - r * s[j];
            y1[j] = r * c[j] + p * s[j];
          }
        }
      }
    }
    uint16_t* out;
    if (is_q) {
      out = a.q + (row * a.heads + head) * d;
    } else {
      if (slot < 0 || slot >= a.slots) continue;
      const int h = head - a.heads - (is_v ? a.kv_heads : 0);
      const int64_t page = slot >> a.shift, off = slot & ((int64_t{1} << a.shift) - 1);
      out = (is_v ? a.v_cache : a.k_cache) + (((page * a.kv_heads + h) << a.shift) + off) * d;
    }
    half4_t* out0 = reinterpret_cast<half4_t*>(out + (is_v ? 8 * part : e0));
    half4_t* out1 = reinterpret_cast<half4_t*>(out + (is_v ? 8 * part + 4 : e1));
    if constexpr (U > 1) {
      __builtin_nontemporal_store(__builtin_convertvector(y0, half4_t), out0);
      __builtin_nontemporal_store(__builtin_convertvector(y1, half4_t), out1);
    } else {
      *out0 = __builtin_convertvector(y0, half4_t);
      *out1 = __builtin_convertvector(y1, half4_t);
    }
  }
}

template <int LPH, int U>
void launch_rotary(const RotaryArgs& a, bool interleaved, hipStream_t stream) {
  const int all = a.heads + 2 * a.kv_heads;
  const int64_t pieces = (all + U * (kWave / LPH) - 1) / (U * (kWave / LPH));
  const dim3 grid(static_cast<unsigned>((pieces * a.m + 3) / 4));
  if (interleaved) hipLaunchKernelGGL((rotary_kernel<LPH, true, U>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((rotary_kernel<LPH, false, U>), grid, dim3(256), 0, stream, a);
}

template <int LPH>
void launch_rotary_rows(const RotaryArgs& a, bool interleaved, hipStream_t stream) {
  // Two groups of heads a wave share its angles: 4,096 rows of 48 heads take 32.1 us, with one 39.0, with three 31.8,
  // with four 35.1; 1,000 rows 11.0 and 12.7. One group ends sooner where there are waves to spare: one row 3.4 and
  // 3.9 us, 333 rows of 18 heads 3.6 and 3.9. From there on the results are stored past the caches: 4,096 rows 30.5
  // us, 1,000 rows 10.7, 400 rows 5.9 against 6.1; 333 rows of 18 heads would take 4.0 with such stores, 3.6 without.
  if (static_cast<int64_t>(a.m) * (a.heads + 2 * a.kv_heads) >= 16384) launch_rotary<LPH, 2>(a, interleaved, stream);
  else launch_rotary<LPH, 1>(a, interleaved, stream);
}

}  // namespace

int page_shift(int64_t page_size) { return __builtin_ctzll(static_cast<unsigned long long>(page_size)); }

hipError_t launch_cache_plan(const int32_t* lengths, const int32_t* added, int64_t requests, int32_t* table,
                             int64_t table_width, const int32_t* free_pages, int64_t free_capacity,
                             const int32_t* free_count, int64_t pages, int64_t page_size, const int32_t* parents,
                             int64_t m, int32_t* row_start, int32_t* request, int32_t* position, int64_t* slot,
                             uint64_t* ancestors, int32_t* free_left, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((m + kPlanRows - 1) / kPlanRows));
  hipLaunchKernelGGL(cache_plan_kernel, grid, dim3(kPlanThreads), 0, stream, lengths, added,
                     static_cast<int>(requests), table, static_cast<int>(table_width), free_pages, free_capacity,
                     free_count, pages, page_shift(page_size), parents, static_cast<int>(m), row_start,
                     request, position, slot, ancestors, free_left);
  return hipGetLastError();
}

hipError_t launch_rotary_qkv(const float* qkv, const int32_t* position, const int64_t* slot, const double* inv_freq,
                             const float* q_weight, const float* k_weight, float eps, float amplitude,
                             bool interleaved, int64_t m, int heads, int kv_heads, int head_dim, int rotary_dim,
                             uint16_t* q, uint16_t* k_cache, uint16_t* v_cache, int64_t pages, int64_t page_size,
                             hipStream_t stream) {
  const RotaryArgs a = {qkv,  position, slot,  inv_freq, q_weight, k_weight, eps,  amplitude, static_cast<int>(m),
                        heads, kv_heads, head_dim, rotary_dim, q, k_cache, v_cache, pages * page_size,
                        page_shift(page_size)};
  if (head_dim <= 64) launch_rotary_rows<8>(a, interleaved, stream);
  else if (head_dim <= 128) launch_rotary_rows<16>(a, interleaved, stream);
  else launch_rotary_rows<32>(a, interleaved, stream);
  return hipGetLastError();
}

}  // namespace pbg
