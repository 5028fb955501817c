// tree_attention: attention of a step's rows over a paged cache.
//
// out = sum_t w_t v_t / sum_t w_t, w_t = exp(scale q . k_t), in one pass over the tokens with a
// running maximum: w_t is held relative to the largest score so far, and the sums are scaled
// down whenever it grows.
#include "pbg_device.hpp"
#include "pbg_internal.hpp"

namespace pbg {
namespace {

constexpr int kTree = 64;
constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kStep = 32;                // tokens a wave takes at once
constexpr int kTokens = kWaves * kStep;  // tokens of a unit of work
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -__builtin_inff();

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4_t lds_short4_t;

struct AttnArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t pages;
  int shift;
  const int32_t* table;
  int width;
  const int32_t* lengths;
  const int32_t* row_start;
  int requests;
  const uint64_t* ancestors;
  int m, heads, kv_heads, d;
  float scale;  // times log2(e)
  uint16_t* out;
  // heads of a key head that a tile takes, such groups of a key head, rows of a tile
  int group, chunks, rows;
  int4* parts;    // [workgroups]: first row, first head, rows and pieces of the work that a workgroup leaves to others
  float* states;  // [workgroups][2] tiles: outputs, then maxima and sums
};

// Request i: its rows, its tokens and its units of work.
struct Request {
  int first, rows, length, tokens;
  int64_t tiles, steps, units;  // tiles of rows, units of a tile, units in all
};

__device__ __forceinline__ Request request_of(const AttnArgs& a, int i) {
  Request r;
  const int s = min(max(a.row_start[i], 0), a.m), e = min(max(a.row_start[i + 1], 0), a.m);
  r.first = s;
  r.rows = max(e - s, 0);
  r.length = max(a.lengths[i], 0);
  const int64_t room = static_cast<int64_t>(a.width) << a.shift;
  r.tokens = static_cast<int>(min(static_cast<int64_t>(r.length) + r.rows, room));
  r.tiles = (r.rows + a.rows - 1) / a.rows;
  r.steps = (static_cast<int64_t>(r.tokens) + kTokens - 1) / kTokens;
  // a request without a token to look at still has its zeros to write
  if (r.steps == 0) r.steps = 1;
  r.units = r.tiles * r.steps * a.kv_heads * a.chunks;
  return r;
}

template <int D>
__device__ __forceinline__ int swizzled(int token, int chunk) {
  if constexpr (D == 64) return chunk ^ (((token >> 1) & 3) << 1);
  else return chunk ^ ((token & 7) << 1);
}

__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }

// Maximum over the four 16-lane groups of a wave, lane by lane.
__device__ __forceinline__ float groups_max(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
  v = fmaxf(as_f32(a[0]), as_f32(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
  return fmaxf(as_f32(b[0]), as_f32(b[1]));
}

__device__ __forceinline__ float groups_sum(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
  v = as_f32(a[0]) + as_f32(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
  return as_f32(b[0]) + as_f32(b[1]);
}

// Halves of w that are an infinity or NaN, as a mask of 16 bits each.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & 0x7C00u) == 0x7C00u ? 0xFFFFu : 0u) | ((w & 0x7C000000u) == 0x7C000000u ? 0xFFFF0000u : 0u);
}

// Scale of a state with maximum m next to one with maximum `top`.
__device__ __forceinline__ float weight_of(float m, float top) { return m == kNone ? 0.0f : exp2_of(m - top); }

// D: head_dim rounded up to 64, 128 or 256. QB: blocks of 16 query rows (a
// query row is one head of one row of the step; the heads of a key
// head share its keys).
//
// The units of work (one tile of query rows over 128 tokens) of all requests
// stand in one line, which the workgroups share evenly, so that requests
// of any lengths fill the chip; a tile that ends up with several workgroups is
// joined by the second kernel.
//
// A wave takes 32 tokens of a unit for all query rows, on its own: S^T = K Q^T
// with keys straight from memory as the first operand, so that a lane
// holds one query row's scores (its maximum and sum need two lane swaps), and
// the weights are then the second operand of O^T = V^T W^T as they are. V^T comes out
// of LDS with transposing reads.
template <int D, int QB>
__global__ __launch_bounds__(kThreads) void attention_kernel(AttnArgs a) {
  constexpr int J = D / 32;       // products of 32 columns in a score
  constexpr int DB = D / 16;      // blocks of 16 columns of the output
  constexpr int kRow = D + 4;     // floats of a row where waves meet
  constexpr int kStage = kStep * D * 2;
  constexpr int kMeet = 16 * kRow * 4;
  constexpr int kSlice = kStage > kMeet ? kStage : kMeet;
  __shared__ __attribute__((aligned(16))) char lds[kWaves * kSlice];
  __shared__ float meet_max[kWaves][QB * 16], meet_sum[kWaves][QB * 16];
  __shared__ int64_t scan[kWaves];
  __shared__ int64_t found[2];
  __shared__ int found_request;

  const int tid = threadIdx.x, lane = tid & (kWave - 1), li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int64_t groups = gridDim.x;
  const int64_t me = blockIdx.x;

  // ---- the share of the line
  const int per = (a.requests + kThreads - 1) / kThreads;
  const int i0 = min(tid * per, a.requests), i1 = min(i0 + per, a.requests);
  int64_t mine = 0;
  for (int i = i0; i < i1; ++i) mine += request_of(a, i).units;
  int64_t sum = mine;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int64_t o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == kWave - 1) scan[wave] = sum;
  if (tid == 0) found_request = -1;
  __syncthreads();
  int64_t before = sum - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += scan[w];
    total += scan[w];
  }
  const int64_t share = (total + groups - 1) / groups;
  const int64_t begin = min(me * share, total), end = min(begin + share, total);
  if (begin >= before && begin < before + mine) {
    int i = i0;
    for (; i < i1; ++i) {
      const int64_t u = request_of(a, i).units;
      if (begin < before + u) break;
      before += u;
    }
    found_request = i;
    found[0] = before;
  }
  __syncthreads();
  if (tid == 0) a.parts[me] = make_int4(0, 0, 0, 0);
  if (begin >= end) return;
  int request = found_request;
  int64_t base = found[0];
  Request r = request_of(a, request);

  for (int64_t at = begin; at < end;) {
    while (at >= base + r.units) {
      base += r.units;
      r = request_of(a, ++request);
    }
    const int64_t in = at - base, tile_units = r.steps;
    const int64_t head_units = r.tiles * tile_units;
    const int vhead = static_cast<int>(in / head_units);
    const int64_t in_head = in - vhead * head_units;
    const int tile = static_cast<int>(in_head / tile_units);
    const int64_t step0 = in_head - tile * tile_units;
    const int64_t step1 = min(step0 + (end - at), tile_units);
    const int kvh = vhead / a.chunks, chunk = vhead - kvh * a.chunks;
    const int ratio = a.heads / a.kv_heads;
    const int head0 = kvh * ratio + chunk * a.group;
    const int tile_heads = min(a.group, ratio - chunk * a.group);
    const int row0 = r.first + tile * a.rows;
    const int tile_rows = min(a.rows, r.rows - tile * a.rows);

    // ---- queries: block b's row li is query row 16 b + li: row / group, head % group
    mfma_half8_t q[QB][J];
    uint64_t sees[QB];
    int upto[QB];  // last token seen without a tree
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      const int n = 16 * b + li, rr = n / a.group, hh = n - rr * a.group;
      const bool fine = rr < tile_rows && hh < tile_heads;
      const int row = row0 + rr;
      sees[b] = fine && a.ancestors ? a.ancestors[row] : 0;
      upto[b] = fine && !a.ancestors ? r.length + (row - r.first) : r.length - 1;
      const uint16_t* p = a.q + (static_cast<int64_t>(row) * a.heads + head0 + hh) * a.d;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = 8 * (4 * j + lg);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (fine && c < a.d) w = *reinterpret_cast<const uint4*>(p + c);
        q[b][j] = __builtin_bit_cast(mfma_half8_t, w);
      }
    }
    float top[QB], part[QB];
    f32x4_t o[QB][DB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      top[b] = kNone;
      part[b] = 0.0f;
#pragma unroll
      for (int e = 0; e < DB; ++e) o[b][e] = f32x4_t{};
    }

    const int32_t* table = a.table + static_cast<int64_t>(request) * a.width;
    const int64_t page_bytes = (static_cast<int64_t>(a.kv_heads) << a.shift) * a.d;  // in elements
    const int64_t head_at = (static_cast<int64_t>(kvh) << a.shift) * a.d;
    char* slice = lds + wave * kSlice;
    // where a token lies in k and v (in elements), or -1
    auto place = [&](int t) -> int64_t {
      if (t >= r.tokens) return -1;
      const int page = table[t >> a.shift];
      if (page < 0 || page >= a.pages) return -1;
      return page * page_bytes + head_at + static_cast<int64_t>(t & ((1 << a.shift) - 1)) * a.d;
    };

    for (int64_t s = step0; s < step1; ++s) {
      const int t0 = static_cast<int>(s) * kTokens + wave * kStep;
      if (t0 >= r.tokens) continue;
      const int64_t at0 = place(t0 + li), at1 = place(t0 + 16 + li);
      // tokens that have a place, one bit each
      const uint32_t held = static_cast<uint32_t>(__ballot(at0 >= 0) & 0xFFFFu) |
                            static_cast<uint32_t>(__ballot(at1 >= 0) & 0xFFFFu) << 16;
      uint4 kr[2][J], vr[2][J];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int64_t p = b ? at1 : at0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int c = 8 * (4 * j + lg);
          kr[b][j] = make_uint4(0, 0, 0, 0);
          vr[b][j] = make_uint4(0, 0, 0, 0);
          if (p >= 0 && c < a.d) {
            kr[b][j] = *reinterpret_cast<const uint4*>(a.k + p + c);
            vr[b][j] = *reinterpret_cast<const uint4*>(a.v + p + c);
          }
        }
      }
      // whether any row may not see a token of these, and values that must reach only rows that see them
      const bool masked = t0 + kStep > r.length || held != 0xFFFFFFFFu;
      uint32_t wild = 0;
      if (masked) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t any = 0;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            uint4& w = vr[b][j];
            const uint4 n = make_uint4(not_finite(w.x), not_finite(w.y), not_finite(w.z), not_finite(w.w));
            any |= n.x | n.y | n.z | n.w;
            w = make_uint4(w.x & ~n.x, w.y & ~n.y, w.z & ~n.z, w.w & ~n.w);
          }
          const uint64_t lanes = __ballot(any != 0);
          const uint32_t tokens = static_cast<uint32_t>((lanes | lanes >> 16 | lanes >> 32 | lanes >> 48) & 0xFFFFu);
          wild |= tokens << (16 * b);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int t = 16 * b + li;
#pragma unroll
        for (int j = 0; j < J; ++j)
          *reinterpret_cast<uint4*>(slice + t * (D * 2) + swizzled<D>(t, 4 * j + lg) * 16) = vr[b][j];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

      mfma_half8_t w[QB];
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        mfma_float4_t x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[h] = mfma_float4_t{};
#pragma unroll
          for (int j = 0; j < J; ++j)
            x[h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(mfma_half8_t, kr[h][j]), q[b][j], x[h], 0, 0, 0);
        }
        if (masked) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int n = 16 * h + 4 * lg + e, t = t0 + n, late = t - r.length;
              const bool seen = t <= upto[b] || (late >= 0 && late < kTree && (sees[b] >> late & 1));
              if (!seen || !(held >> n & 1)) x[h][e] = kNone;
            }
        }
        float high = kNone;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) high = fmaxf(high, x[h][e]);
        high = groups_max(high) * a.scale;
        const float now = fmaxf(top[b], high);
        const float shift = now == kNone ? 0.0f : now;
        const float keep = weight_of(top[b], shift);
        top[b] = now;
        float p[8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) p[4 * h + e] = exp2_of(__builtin_fmaf(x[h][e], a.scale, -shift));
        // the sum is that of the rounded weights, so that their rounding does not change the weights' total
        float add = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[b][e] = static_cast<_Float16>(p[e]);
          add += static_cast<float>(w[b][e]);
        }
        part[b] = part[b] * keep + add;
#pragma unroll
        for (int e = 0; e < DB; ++e) o[b][e] *= keep;
      }
      // ---- O^T += V^T W^T
#pragma unroll
      for (int e = 0; e < DB; ++e) {
        mfma_half8_t v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = 16 * h + 4 * lg + li / 4, c = 2 * e + (li & 3) / 2;
          const auto v4 = __builtin_bit_cast(half4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_short4_t*)(slice + t * (D * 2) + swizzled<D>(t, c) * 16 + (li & 1) * 8)));
#pragma unroll
          for (int x = 0; x < 4; ++x) v[4 * h + x] = v4[x];
        }
#pragma unroll
        for (int b = 0; b < QB; ++b) o[b][e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w[b], o[b][e], 0, 0, 0);
      }
      // infinities and NaN among values that some rows may not see: added for the rows that do
      while (wild) {
        const int n = __builtin_ctz(wild);
        wild &= wild - 1;
        const int t = t0 + n, late = t - r.length;
        const int64_t p = place(t);
        const int at_lane = li + 16 * ((n & 15) >> 2), at_elem = (n >> 4) * 4 + (n & 3);
#pragma unroll
        for (int b = 0; b < QB; ++b) {
          float x = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) x = e == at_elem ? static_cast<float>(w[b][e]) : x;
          x = __shfl(x, at_lane);
          const bool seen = t <= upto[b] || (late >= 0 && late < kTree && (sees[b] >> late & 1));
          if (seen && p >= 0) {
#pragma unroll
            for (int e = 0; e < DB; ++e)
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int c = 16 * e + 4 * lg + y;
                const uint16_t bits = c < a.d ? a.v[p + c] : 0;
                if ((bits & 0x7C00u) == 0x7C00u) o[b][e][y] += x * static_cast<float>(__builtin_bit_cast(_Float16, bits));
              }
          }
        }
      }
    }

    // ---- the four waves' states meet
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      const float s = groups_sum(part[b]);
      if (lg == 0) {
        meet_max[wave][16 * b + li] = top[b];
        meet_sum[wave][16 * b + li] = s;
      }
    }
    __syncthreads();
    const bool starts = step0 == 0, ends = step1 == tile_units;
    float* state = a.states + (me * 2 + (starts ? 1 : 0)) * (QB * 16) * (D + 2);
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      const int n = 16 * b + li;
      float high = meet_max[0][n];
#pragma unroll
      for (int x = 1; x < kWaves; ++x) high = fmaxf(high, meet_max[x][n]);
      const float keep = weight_of(top[b], high);
      float* to = reinterpret_cast<float*>(slice) + li * kRow;
#pragma unroll
      for (int e = 0; e < DB; ++e) *reinterpret_cast<f32x4_t*>(to + 16 * e + 4 * lg) = o[b][e] * keep;
      __syncthreads();
      for (int x = tid; x < 16 * (D / 4); x += kThreads) {
        const int nn = x / (D / 4), c = 4 * (x % (D / 4));
        const int qr = 16 * b + nn, rr = qr / a.group, hh = qr - rr * a.group;
        if (rr >= tile_rows || hh >= tile_heads) continue;
        float most = meet_max[0][qr];
#pragma unroll
        for (int y = 1; y < kWaves; ++y) most = fmaxf(most, meet_max[y][qr]);
        float total_w = 0.0f;
        f32x4_t acc = {};
#pragma unroll
        for (int y = 0; y < kWaves; ++y) {
          total_w += meet_sum[y][qr] * weight_of(meet_max[y][qr], most);
          acc += *reinterpret_cast<const f32x4_t*>(lds + y * kSlice + (nn * kRow + c) * 4);
        }
        if (starts && ends) {
          if (c < a.d) {
            const float inv = total_w == 0.0f ? 0.0f : 1.0f / total_w;
            if (total_w == 0.0f) acc = f32x4_t{};
            uint16_t* to_out = a.out + (static_cast<int64_t>(row0 + rr) * a.heads + head0 + hh) * a.d + c;
            *reinterpret_cast<half4_t*>(to_out) = __builtin_convertvector(acc * inv, half4_t);
          }
        } else {
          *reinterpret_cast<f32x4_t*>(state + qr * D + c) = acc;
          if (c == 0) {
            state[QB * 16 * D + 2 * qr] = most;
            state[QB * 16 * D + 2 * qr + 1] = total_w;
          }
        }
      }
      __syncthreads();
    }
    if (starts && !ends && tid == 0) {
      // the pieces after this one: whole shares of the workgroups that follow
      const int64_t tile_end = at + tile_units;
      a.parts[me] = make_int4(row0, head0, tile_heads << 16 | tile_rows, static_cast<int>((tile_end - 1) / share - me + 1));
    }
    at += step1 - step0;
  }
}

// Joins the pieces of a tile that several workgroups had: one workgroup for
// four query rows, their pieces shared by the waves.
template <int D, int QB>
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttnArgs a) {
  constexpr int kState = QB * 16 * (D + 2);
  constexpr int kPer = D / kWave;  // columns a lane
  __shared__ float acc_at[kWaves][4][D];
  __shared__ float top_at[kWaves][4], sum_at[kWaves][4];
  const int64_t me = blockIdx.x;
  const int4 part = a.parts[me];
  if (part.w == 0) return;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int tile_rows = part.z & 0xFFFF, tile_heads = part.z >> 16;
  const int first = blockIdx.y * 4;
  if (first / a.group >= tile_rows) return;
  for (int x = 0; x < 4; ++x) {
    const int n = first + x;
    float top = kNone, sum = 0.0f, acc[kPer] = {};
    for (int p = wave; p < part.w; p += kWaves) {
      const float* s = a.states + ((me + p) * 2 + (p == 0 ? 1 : 0)) * kState;
      const float high = s[QB * 16 * D + 2 * n], w = s[QB * 16 * D + 2 * n + 1];
      const float now = fmaxf(top, high);
      const float keep = weight_of(top, now), add = weight_of(high, now);
      top = now;
      sum = sum * keep + w * add;
#pragma unroll
      for (int c = 0; c < kPer; ++c) acc[c] = acc[c] * keep + s[n * D + lane + kWave * c] * add;
    }
    if (lane == 0) {
      top_at[wave][x] = top;
      sum_at[wave][x] = sum;
    }
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc_at[wave][x][lane + kWave * c] = acc[c];
  }
  __syncthreads();
  const int n = first + wave, rr = n / a.group, hh = n - rr * a.group;
  if (rr >= tile_rows || hh >= tile_heads) return;
  float top = top_at[0][wave];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) top = fmaxf(top, top_at[w][wave]);
  float sum = 0.0f, scale[kWaves];
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    scale[w] = weight_of(top_at[w][wave], top);
    sum += sum_at[w][wave] * scale[w];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    const int col = lane + kWave * c;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += acc_at[w][wave][col] * scale[w];
    if (sum == 0.0f) v = 0.0f;
    if (col < a.d)
      a.out[(static_cast<int64_t>(part.x + rr) * a.heads + part.y + hh) * a.d + col] =
          __builtin_bit_cast(uint16_t, static_cast<_Float16>(v * inv));
  }
}

// Workgroups of a launch: as many as the chip holds at once.
constexpr int kGroups = 768;
constexpr int kWideGroups = 256;  // tiles of more than 16 query rows

template <int D, int QB>
hipError_t launch_tiles(AttnArgs a, void* ws, hipStream_t stream) {
  const int ratio = a.heads / a.kv_heads;
  a.group = ratio < QB * 16 ? ratio : QB * 16;
  a.chunks = (ratio + a.group - 1) / a.group;
  a.rows = QB * 16 / a.group;
  const int groups = QB == 1 ? kGroups : kWideGroups;
  a.parts = static_cast<int4*>(ws);
  a.states = reinterpret_cast<float*>(static_cast<char*>(ws) + kGroups * sizeof(int4));
  hipLaunchKernelGGL((attention_kernel<D, QB>), dim3(groups), dim3(kThreads), 0, stream, a);
  hipLaunchKernelGGL((attention_join_kernel<D, QB>), dim3(groups, QB * 4), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

int64_t attention_workspace_bytes(int head_dim) {
  const int64_t d = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
  const int64_t wide = d == 256 ? 32 : 64;
  const int64_t narrow = kGroups * 2 * 16 * (d + 2) * 4, many = kWideGroups * 2 * wide * (d + 2) * 4;
  return kGroups * 16 + (narrow > many ? narrow : many);
}

hipError_t launch_tree_attention(const uint16_t* q, const uint16_t* k_cache, const uint16_t* v_cache, int64_t pages,
                                 int64_t page_size, const int32_t* table, int64_t table_width, const int32_t* lengths,
                                 const int32_t* row_start, int64_t requests, const uint64_t* ancestors, int64_t m,
                                 int heads, int kv_heads, int head_dim, float scale, uint16_t* out, void* workspace,
                                 hipStream_t stream) {
  const AttnArgs a = {q, k_cache, v_cache, pages, page_shift(page_size), table, static_cast<int>(table_width), lengths,
                      row_start, static_cast<int>(requests), ancestors, static_cast<int>(m), heads, kv_heads, head_dim,
                      scale * kLog2e, out, 0, 0, 0, nullptr, nullptr};
  // query rows of a key head that a request has on average
  const bool few = m * (heads / kv_heads) <= 16 * requests;
  if (head_dim <= 64) return few ? launch_tiles<64, 1>(a, workspace, stream) : launch_tiles<64, 4>(a, workspace, stream);
  if (head_dim <= 128)
    return few ? launch_tiles<128, 1>(a, workspace, stream) : launch_tiles<128, 4>(a, workspace, stream);
  return few ? launch_tiles<256, 1>(a, workspace, stream) : launch_tiles<256, 2>(a, workspace, stream);
}

}  // namespace pbg
