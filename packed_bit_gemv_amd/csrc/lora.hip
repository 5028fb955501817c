// lora_add: out_i = y_i + s_a B_a (A_a x_i) with a = ids[i], the adapters of
// many requests at once beside a shared projection; rows without an adapter
// are passed through.
//
// v_i = A_a x_i on the f16 matrix cores (fp16 products are exact in its fp32
// sums), then the product with B_a added to y. Between the two each v keeps 22
// bits or more: a power of two brings the row's largest |v| to [2^13, 2^14),
// and v = hi + 2^-11 lo in two fp16 parts, the 2^11 giving lo the range of hi,
// so that B_a stays fp16 on the matrix cores, with a sum for each part. That
// holds for |v| down to 2^-27 of the row's largest. Rows with a smaller one (not
// 0), and outputs that meet an infinity or NaN, are taken from the fp32 matrix
// cores, an eighth of the f16 rate, on v itself: 1,531 rows at rank 64, n =
// 12,288, that are all of this kind take 78 us against 58. (Those cores for
// every row take 66.9 us against 61.9 of ordinary rows, at rank 128 110 against 98.)
//
// Rows come in any order. A workgroup takes a block of R rows, sorts them by
// adapter in LDS and cuts the sorted list into groups of at most 16 rows of
// one adapter, which is what a matrix instruction takes: an adapter's weights
// are read once per group, not once per row, and only for its own rows, so
// that NaN in one adapter cannot reach another's rows. Where many adapters
// share many rows, a launch before sorts those rows by adapter.
#include "pbg_device.hpp"
#include "pbg_internal.hpp"

namespace pbg {
namespace {

constexpr int kRows = 16;       // rows of a group
constexpr int kWaves = 4;
constexpr int kMaxSlices = 16;  // slices of K
constexpr int kSliced = 16384;  // rows times slices of K
constexpr int64_t kSortBytes = 160 << 20;  // of adapters that mixed rows would read again

// Up to 16 rows are one block whose second launch adds the slices itself.
bool lora_one_block(int64_t m) { return m <= kRows; }

// Slices of K: 16 for one block, else 8 up to 2,048 rows, then as many as keep
// rows times slices at kSliced, down to 2.
int lora_slices(int64_t m) {
  if (lora_one_block(m)) return kMaxSlices;
  const int64_t s = kSliced / m;
  return static_cast<int>(s < 2 ? 2 : s > 8 ? 8 : s);
}

int rank_padded(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// The groups of R places from m0 on: rows m0 .. m0 + R - 1, or perm of them
// with their ids. Built by the first R threads (R <= 64: one wave); group g is
// the rows row[start[g]] .. row[start[g + 1] - 1]. Rows without an adapter
// come last, in groups with id -1; places past m are left out.
template <int R>
struct Groups {
  int key[R];         // adapter of a row, `adapters` for none, INT_MAX past m
  int row[R];         // rows by key
  int16_t start[R + 1];
  int id[R];          // adapter of a group
  int count;

  __device__ void build(const int32_t* __restrict__ ids, const int32_t* __restrict__ perm, int64_t m0, int64_t m,
                        int adapters) {
    static_assert(R <= kWave, "one wave sorts");
    const int i = threadIdx.x;
    if (i < kWave) {
      int k = 0x7FFFFFFF, of = 0;
      if (i < R && m0 + i < m) {
        of = perm ? perm[m0 + i] : static_cast<int>(m0 + i);
        const int t = ids[m0 + i];
        k = t >= 0 && t < adapters ? t : adapters;
      }
      int place = 0;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int o = __builtin_amdgcn_readlane(k, j);
        place += o < k || (o == k && j < i);
      }
      if (i < R) {
        key[place] = k;
        row[place] = of;
      }
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const int mine = i < R ? key[i] : 0x7FFFFFFF;
      const bool live = mine != 0x7FFFFFFF;
      const bool first = live && (i % kRows == 0 || key[i - 1] != mine);
      const uint64_t firsts = __ballot(first), lives = __ballot(live);
      if (first) {
        const int g = __popcll(firsts & ((1ull << i) - 1));
        start[g] = static_cast<int16_t>(i);
        id[g] = mine < adapters ? mine : -1;
      }
      if (i == 0) {
        count = __popcll(firsts);
        start[count] = static_cast<int16_t>(__popcll(lives));
      }
    }
    __syncthreads();
  }
};

// Where many adapters mix in a prompt, a block of 64 rows holds few rows of
// each. Then the rows are put in the order of their adapters first: perm, by a
// counting sort of kChunk rows in a workgroup, and the ids in that order. Only
// the grouping depends on it, no result does: rows of one adapter come in the
// order of their atomics, and ids that share a bin are told apart by the
// groups.
constexpr int kChunk = 4096;
constexpr int kBins = 1024;  // the last one for rows without an adapter

__global__ __launch_bounds__(kBins) void lora_sort_kernel(const int32_t* __restrict__ ids, int64_t m, int adapters,
                                                          int32_t* __restrict__ sorted, int32_t* __restrict__ perm) {
  __shared__ int bin[kBins];
  __shared__ int before[kBins / kWave];
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kChunk;
  int id[kChunk / kBins], of[kChunk / kBins], at[kChunk / kBins];
  bin[t] = 0;
#pragma unroll
  for (int u = 0; u < kChunk / kBins; ++u) {
    const int64_t row = c0 + t + u * kBins;
    id[u] = row < m ? ids[row] : 0;
    of[u] = id[u] >= 0 && id[u] < adapters ? id[u] % (kBins - 1) : kBins - 1;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kChunk / kBins; ++u)
    at[u] = c0 + t + u * kBins < m ? atomicAdd(&bin[of[u]], 1) : 0;
  __syncthreads();
  int sum = bin[t];
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int other = __shfl_up(sum, d);
    sum += lane >= d ? other : 0;
  }
  if (lane == kWave - 1) before[t / kWave] = sum;
  __syncthreads();
  int start = sum - bin[t];
#pragma unroll
  for (int w = 0; w < kBins / kWave; ++w) start += w < t / kWave ? before[w] : 0;
  bin[t] = start;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kChunk / kBins; ++u) {
    const int64_t row = c0 + t + u * kBins;
    if (row < m) {
      const int64_t place = c0 + bin[of[u]] + at[u];
      sorted[place] = id[u];
      perm[place] = static_cast<int32_t>(row);
    }
  }
}

template <int N>
using half_t = _Float16 __attribute__((ext_vector_type(N)));
// The same at the alignment of an element (an alias template would drop the attribute).
template <int N>
struct HalfAny;
template <>
struct HalfAny<4> {
  typedef _Float16 type __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct HalfAny<8> {
  typedef _Float16 type __attribute__((ext_vector_type(8), aligned(2)));
};
static_assert(alignof(HalfAny<4>::type) == 2 && alignof(HalfAny<8>::type) == 2, "element alignment");

// N (4 or 8) fp16 elements from column c, a multiple of N, zero from column k on. FAST: p
// 16-byte aligned and k a multiple of 8; otherwise one load at any alignment, and
// single elements at the end of a row only. The second does everything, the
// first is faster: 900 rows of 12 adapters at rank 32, k = 6,000, take 27.9
// against 32.4 us, 300 rows of 40 at rank 16 20.9 against 23.6.
template <int N, bool FAST>
__device__ __forceinline__ half_t<N> load_halves(const uint16_t* __restrict__ p, int64_t c, int64_t k) {
  if constexpr (FAST) {
    half_t<N> v = {};
    if (c < k) v = *reinterpret_cast<const half_t<N>*>(p + c);
    return v;
  } else {
    if (c + N <= k) return *reinterpret_cast<const typename HalfAny<N>::type*>(p + c);
    half_t<N> v;
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = c + e < k ? __builtin_bit_cast(_Float16, p[c + e]) : static_cast<_Float16>(0.0f);
    return v;
  }
}

// First product: v[slice][row][rank] for the row block blockIdx.x, the slice
// of K blockIdx.y and the groups blockIdx.z, + gridDim.z, ... The waves take
// 32-column steps in turn, U steps of loads in flight. A group alone is bound
// by the latency of its loads, so K is sliced until the launch fills the chip:
// 1,531 rows at rank 64, k = 4,096 take 13 us with 8 slices, 24 unsliced.
template <int R, int RT, bool FAST>
__global__ __launch_bounds__(kWaves* kWave) void lora_down_kernel(const uint16_t* __restrict__ x,
                                                                  const int32_t* __restrict__ ids,
                                                                  const int32_t* __restrict__ perm,
                                                                  const uint16_t* __restrict__ a, int64_t m, int64_t k,
                                                                  int adapters, int rank, int64_t k_slice,
                                                                  float* __restrict__ v) {
  constexpr int U = RT >= 8 ? 2 : 4;
  __shared__ Groups<R> groups;
  __shared__ mfma_float4_t part[kWaves - 1][RT][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int li = lane & 15, lg = lane >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * R;
  groups.build(ids, perm, m0, m, adapters);
  const int64_t k0 = blockIdx.y * k_slice;
  const int64_t k1 = k0 + k_slice < k ? k0 + k_slice : k;
  const int count = __builtin_amdgcn_readfirstlane(groups.count);
  for (int g = blockIdx.z; g < count; g += gridDim.z) {
    const int ad = __builtin_amdgcn_readfirstlane(groups.id[g]);
    if (ad < 0) break;  // the groups without an adapter are the last ones
    const int p0 = groups.start[g], p1 = groups.start[g + 1];
    const uint16_t* xr = x + static_cast<int64_t>(groups.row[p0 + li < p1 ? p0 + li : p0]) * k;
    const uint16_t* ar[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int j = 16 * t + li;
      ar[t] = a + (static_cast<int64_t>(ad) * rank + (j < rank ? j : rank - 1)) * k;
    }
    mfma_float4_t acc[RT] = {};
#pragma unroll 1
    for (int64_t c0 = k0 + 32 * wave; c0 < k1; c0 += 32 * kWaves * U) {
      mfma_half8_t xv[U], av[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + 32 * kWaves * u + 8 * lg;
        xv[u] = load_halves<8, FAST>(xr, c, k1);
#pragma unroll
        for (int t = 0; t < RT; ++t) av[u][t] = load_halves<8, FAST>(ar[t], c, k1);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < RT; ++t)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[u], av[u][t], acc[t], 0, 0, 0);
    }
    __syncthreads();
    if (wave > 0) {
#pragma unroll
      for (int t = 0; t < RT; ++t) part[wave - 1][t][lane] = acc[t];
    }
    __syncthreads();
    if (wave > 0) continue;
    // lane: v[4 lg + e][16 t + li] of the group's rows
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
      for (int w = 0; w < kWaves - 1; ++w) acc[t] += part[w][t][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = p0 + 4 * lg + e;
        if (at < p1 && 16 * t + li < rank)
          v[(blockIdx.y * m + groups.row[at]) * rank + 16 * t + li] = acc[t][e];
      }
    }
  }
}

// Power of two (as its exponent) that brings a row's largest |v| to [2^13, 2^14).
// A finite v is a multiple of 2^-48 below 2^50, so this and its negative are
// within fp32's exponents.
__device__ __forceinline__ int exponent_of(float top) {
  return top > 0.0f && top < __builtin_inff() ? 13 - ilogbf(top) : 0;
}

__device__ __forceinline__ float row_max16(float v) {
  v = fmaxf(v, row_ror<8>(v));
  v = fmaxf(v, row_ror<4>(v));
  v = fmaxf(v, row_ror<2>(v));
  return fmaxf(v, row_ror<1>(v));
}

// v of one row on the 16 lanes of a DPP row, the slices added in order: its two
// fp16 parts to hi and lo [16 RT], and the factor that undoes the power of two,
// times the adapter's scale; v itself to sum[0 .. width), 0 past the rank (sum
// may be the first slice, which one wave has read by then). The factor is NaN, which asks for the fp32 form of
// the second product, where the parts do not hold every v to 2^-22 or the
// factor is no normal number. With w in hi's normal range, w - hi is at most
// 2^-11 |w|, and lo holds it, 2^11 times, to 2^-11 of itself or 2^-25: in w
// 2^-22 |w| or less.
template <int RT>
__device__ __forceinline__ void join_row(const float* v, int64_t slice_stride, int slices, int rank, float scale,
                                         float* sum, int width, _Float16* hi, _Float16* lo, float* factor) {
  const int li = threadIdx.x & 15;
  float s[RT], top = 0.0f;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int j = 16 * t + li;
    float p[kMaxSlices];
#pragma unroll
    for (int q = 0; q < kMaxSlices; ++q) p[q] = q < slices ? v[q * slice_stride + (j < rank ? j : 0)] : 0.0f;
    s[t] = 0.0f;
#pragma unroll
    for (int q = 0; q < kMaxSlices; ++q) s[t] += p[q];
    if (j >= rank) s[t] = 0.0f;
    top = fmaxf(top, fabsf(s[t]));
  }
  const int ex = exponent_of(row_max16(top));
  bool wide = false;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const float w = ldexpf(s[t], ex);
    const _Float16 h = static_cast<_Float16>(w);
    wide |= w != 0.0f && !(fabsf(w) >= 0x1p-14f && fabsf(w) < __builtin_inff());
    if (16 * t + li < width) sum[16 * t + li] = s[t];
    hi[16 * t + li] = h;
    lo[16 * t + li] = static_cast<_Float16>(0x1p11f * (w - static_cast<float>(h)));
  }
  const float f = ldexpf(scale, -ex);
  wide |= scale != 0.0f && !(fabsf(f) >= 0x1p-126f && fabsf(f) < __builtin_inff());
  const uint64_t any = __ballot(wide) >> (threadIdx.x & 48) & 0xFFFF;
  if (li == 0) *factor = any ? __builtin_nanf("") : f;
}

// The same for every row with an adapter, v to the first slice, parts [m][2][16
// RT] and factors [m] to memory; 16 rows a workgroup.
template <int RT>
__global__ __launch_bounds__(256) void lora_join_kernel(const int32_t* __restrict__ ids,
                                                        const float* __restrict__ scale, int64_t m, int adapters,
                                                        int rank, int slices, float* v,
                                                        _Float16* __restrict__ parts, float* __restrict__ factors) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 16 + threadIdx.x / 16;
  if (row >= m) return;
  const int id = ids[row];
  if (id < 0 || id >= adapters) return;
  _Float16* hi = parts + row * (32 * RT);
  float* vr = v + row * rank;
  join_row<RT>(vr, m * rank, slices, rank, scale[id], vr, rank, hi, hi + 16 * RT, factors + row);
}

__device__ __forceinline__ mfma_float4_t multiply(half_t<8> a, half_t<8> b, mfma_float4_t d) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, d, 0, 0, 0);
}
__device__ __forceinline__ mfma_float4_t multiply(half_t<4> a, half_t<4> b, mfma_float4_t d) {
  return __builtin_amdgcn_mfma_f32_16x16x16f16(a, b, d, 0, 0, 0);
}

typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));

// Four elements p[c .. c + 3], zero from column k on.
__device__ __forceinline__ mfma_float4_t load_floats(const float* __restrict__ p, int c, int k) {
  mfma_float4_t v = {};
  if (c + 4 <= k) {
    v = *reinterpret_cast<const f32x4_any_t*>(p + c);
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (c + e < k) v[e] = p[c + e];
  }
  return v;
}

// Waves a SIMD that the second product's registers must leave room for: as many
// as its ordinary path alone would, where the compiler would give the fp32 form
// registers past that (1,531 rows of n = 12,288 at rank 128 98 against 104 us, at
// rank 32 45.5 against 47.3; 64 rows at rank 64 26.0 against 26.9; 300 rows of n
// = 4,097 at rank 20 33.5 against 36.1). Elsewhere a bound costs: 1,531 mixed
// rows of 64 adapters at rank 64 104.0 us with room for 4 waves against 100.2.
constexpr int up_waves(int rt, int c, bool join, bool fast) {
  if (join) return 1;
  if (c == 4) return rt == 8 ? 3 : rt == 2 && fast ? 5 : 1;
  return rt == 2 ? 8 : rt == 4 && fast ? 7 : 1;
}

// out = y + s_a 2^-e B_a (hi + 2^-11 lo) for a row block and 16 C columns of
// each wave, the groups blockIdx.y, + gridDim.y, ... of the block. B_a is the
// row operand of the matrix instruction, so a lane gets four consecutive
// outputs of one row; an instruction takes 32 of the rank (16 up to rank 16),
// hi and lo on one load of B_a. Outputs that come out infinite or NaN, as those
// of a row marked by its factor do, are taken from the fp32 form, on v itself:
// fp16 parts of an infinity, and a part of 0 against one in B_a, would make NaN
// of it. Whether an output takes that form depends on its own operands only.
// Bound by y and out, which a wave reads and writes in pieces of 64 C bytes a
// row: the product goes through LDS to that order. JOIN: the workgroup adds the
// slices of its groups' v itself. 1,531 rows at rank 64, n = 12,288: 45 us, 3.4
// TB/s of y and out (pieces of 64 bytes, straight from the product's layout: 73
// us).
template <int R, int RT, int C, bool JOIN, bool FAST>
__global__ __launch_bounds__(kWaves* kWave, up_waves(RT, C, JOIN, FAST)) void lora_up_kernel(
    const float* y, const int32_t* __restrict__ ids, const int32_t* __restrict__ perm, const uint16_t* __restrict__ b,
    const float* __restrict__ scale, int64_t m, int64_t n, int adapters, int rank, int slices, int64_t n_blocks,
    const float* __restrict__ v, const _Float16* __restrict__ parts, const float* __restrict__ factors, float* out) {
  constexpr int KT = RT > 1 ? RT / 2 : 1;  // loads of B_a per column tile
  constexpr int kPer = RT > 1 ? 8 : 4;     // of the rank in one of them
  constexpr int RP = 16 * RT;
  constexpr int kTile = 16 * C;            // columns of a wave
  constexpr int kGroup = kTile / 4;        // lanes on one row of y
  constexpr int kPieces = 16 * kGroup / kWave;
  __shared__ Groups<R> groups;
  __shared__ __align__(16) _Float16 own[JOIN ? kRows : 1][2][RP + 8];
  __shared__ float own_factor[kRows];
  __shared__ __align__(16) float own_v[JOIN ? kRows : 1][RP + 4];
  __shared__ __align__(16) float turn[kWaves][kRows][kTile + 4];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int li = lane & 15, lg = lane >> 4;
  const int64_t m0 = blockIdx.x / n_blocks * R;
  groups.build(ids, perm, m0, m, adapters);
  const int64_t n0 = (blockIdx.x % n_blocks * kWaves + wave) * kTile;
  const int count = __builtin_amdgcn_readfirstlane(groups.count);
  const int pc = 4 * (lane % kGroup);  // this lane's columns of y and out, rows lane / kGroup + i (64 / kGroup)
  const int64_t r0 = n0 + pc;
  for (int g = blockIdx.y; g < count; g += gridDim.y) {
    const int ad = __builtin_amdgcn_readfirstlane(groups.id[g]);
    if (ad < 0 && y == out) break;  // nothing left to copy
    const int p0 = groups.start[g], p1 = groups.start[g + 1];
    // y and B first, so that they are in flight while v is made
    mfma_float4_t base[kPieces];
    int64_t row[kPieces];
    bool in[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = p0 + lane / kGroup + i * (kWave / kGroup);
      in[i] = at < p1;
      row[i] = groups.row[in[i] ? at : p0] * n;
      base[i] = mfma_float4_t{};
      if (in[i] && r0 + 4 <= n) {
        base[i] = *reinterpret_cast<const f32x4_any_t*>(y + row[i] + r0);
      } else if (in[i]) {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (r0 + e < n) base[i][e] = y[row[i] + r0 + e];
      }
    }
    if (ad >= 0) {
      half_t<kPer> bv[C][KT];
      const uint16_t* ba = b + static_cast<int64_t>(ad) * n * rank;
      auto load_b = [&](int c, int t) {
        const int64_t r = n0 + 16 * c + li;
        return load_halves<kPer, FAST>(ba + (r < n ? r : n - 1) * rank, kPer * (4 * t + lg), rank);
      };
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int t = 0; t < KT; ++t) bv[c][t] = load_b(c, t);
      // operand of the rows: lane (li, lg) holds kPer values of row li for each load
      const int64_t mine = groups.row[p0 + li < p1 ? p0 + li : p0];
      const _Float16* src;
      float back;
      if constexpr (JOIN) {
        const int i = threadIdx.x >> 4;
        __syncthreads();
        join_row<RT>(v + static_cast<int64_t>(groups.row[p0 + i < p1 ? p0 + i : p0]) * rank, m * rank, slices, rank,
                     scale[ad], own_v[i], RP, own[i][0], own[i][1], own_factor + i);
        __syncthreads();
        src = own[li][0];
        back = own_factor[li];
      } else {
        src = parts + mine * (2 * RP);
        back = factors[mine];
      }
      constexpr int kLo = JOIN ? RP + 8 : RP;  // from hi to lo
      half_t<kPer> hi[KT], lo[KT];
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        hi[t] = *reinterpret_cast<const half_t<kPer>*>(src + kPer * (4 * t + lg));
        lo[t] = *reinterpret_cast<const half_t<kPer>*>(src + kLo + kPer * (4 * t + lg));
      }
      mfma_float4_t d[C];
      float none = 0.0f;  // NaN once an output is infinite or NaN
#pragma unroll
      for (int c = 0; c < C; ++c) {
        mfma_float4_t low = {};
        d[c] = mfma_float4_t{};
#pragma unroll
        for (int t = 0; t < KT; ++t) low = multiply(bv[c][t], lo[t], low);
#pragma unroll
        for (int t = 0; t < KT; ++t) d[c] = multiply(bv[c][t], hi[t], d[c]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // both parts under the row's factor
          d[c][e] = back * (d[c][e] + 0x1p-11f * low[e]);
          none += 0.0f * d[c][e];
        }
      }
      if (__any(none != none)) {
        // an instruction takes four of the rank, element e of each lane's kPer; B_a is read again (kept, its registers
        // cost the ordinary path: 1,531 rows at rank 128 106 against 98 us)
        mfma_float4_t f[C] = {};
#pragma unroll 1
        for (int t = 0; t < KT; ++t) {
          mfma_float4_t vf[kPer / 4];
          half_t<kPer> bf[C];
#pragma unroll
          for (int c = 0; c < C; ++c) bf[c] = load_b(c, t);
#pragma unroll
          for (int u = 0; u < kPer / 4; ++u) {
            const int j = kPer * (4 * t + lg) + 4 * u;
            if constexpr (JOIN) vf[u] = *reinterpret_cast<const mfma_float4_t*>(own_v[li] + j);
            else vf[u] = load_floats(v + mine * rank, j, rank);
          }
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < kPer; ++e)
              f[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(static_cast<float>(bf[c][e]), vf[e / 4][e % 4], f[c], 0, 0, 0);
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) d[c][e] = fabsf(d[c][e]) < __builtin_inff() ? d[c][e] : scale[ad] * f[c][e];
      }
#pragma unroll
      for (int c = 0; c < C; ++c) *reinterpret_cast<mfma_float4_t*>(&turn[wave][li][16 * c + 4 * lg]) = d[c];
      // one wave writes and reads its own part: LDS is in order within a wave
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        base[i] += *reinterpret_cast<const mfma_float4_t*>(&turn[wave][lane / kGroup + i * (kWave / kGroup)][pc]);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (in[i] && r0 + 4 <= n) {
        // not kept in the caches, where B_a is: 61.7 against 66.3 us for the prompt below
        __builtin_nontemporal_store(f32x4_any_t(base[i]), reinterpret_cast<f32x4_any_t*>(out + row[i] + r0));
      } else if (in[i]) {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (r0 + e < n) out[row[i] + r0 + e] = base[i][e];
      }
    }
  }
}

// Columns of one slice: whole steps of four waves.
int64_t slice_columns(int64_t k, int slices) {
  return ((k + slices - 1) / slices + 127) / 128 * 128;
}

struct Args {
  const float* y;
  const uint16_t* x;
  const int32_t* ids;
  const uint16_t* a;
  const uint16_t* b;
  const float* scale;
  int64_t m, n, k;
  int adapters, rank;
  float* out;
  const int32_t* perm;  // with ids in its order; null: rows as they come
  void* ws;
  hipStream_t stream;
};

// Workspace: the slices' sums [slices][m][rank], then, 16-byte aligned, the
// parts [m][2][padded rank] and the factors [m], then, for more rows than a
// block, the sorted ids and perm [m].
int64_t sums_bytes(int64_t m, int rank) { return (4 * m * rank * lora_slices(m) + 15) / 16 * 16; }
int64_t parts_bytes(int64_t m, int rank) { return 4 * m * (rank_padded(rank) + 1); }

template <int R, int RT, bool FAST>
void launch_down(const Args& g, int slices, int64_t k_slice, int64_t z) {
  hipLaunchKernelGGL((lora_down_kernel<R, RT, FAST>),
                     dim3(static_cast<unsigned>((g.m + R - 1) / R), slices, static_cast<unsigned>(z)),
                     dim3(kWaves * kWave), 0, g.stream, g.x, g.ids, g.perm, g.a, g.m, g.k, g.adapters, g.rank, k_slice,
                     static_cast<float*>(g.ws));
}

template <int R, int RT, int C, bool JOIN, bool FAST>
void launch_up(const Args& g, int slices, int64_t z) {
  const int64_t blocks = (g.m + R - 1) / R, nb = (g.n + 16 * C * kWaves - 1) / (16 * C * kWaves);
  const _Float16* parts = reinterpret_cast<const _Float16*>(static_cast<char*>(g.ws) + sums_bytes(g.m, g.rank));
  hipLaunchKernelGGL((lora_up_kernel<R, RT, C, JOIN, FAST>),
                     dim3(static_cast<unsigned>(blocks * nb), static_cast<unsigned>(z)), dim3(kWaves * kWave), 0,
                     g.stream, g.y, g.ids, g.perm, g.b, g.scale, g.m, g.n, g.adapters, g.rank, slices, nb,
                     static_cast<const float*>(g.ws), parts, reinterpret_cast<const float*>(parts + g.m * 32 * RT),
                     g.out);
}

template <int RT, bool FAST>
void launch(Args g) {
  const int64_t ks = slice_columns(g.k, lora_slices(g.m));
  const int slices = static_cast<int>((g.k + ks - 1) / ks);
  if (lora_one_block(g.m)) {
    launch_down<16, RT, FAST>(g, slices, ks, g.m);
    launch_up<16, RT, 1, true, FAST>(g, slices, g.m);
    return;
  }
  // A block of 64 rows has 4 groups or a few more where rows come in runs, and up to one for each adapter (and 4 more)
  // where they mix; z workgroups share them. A workgroup without a group costs its sort, one with many takes them one
  // after another, so z fills the chip and no more, and is at least 3: 1,531 rows of 3 adapters in runs (rank 64, n =
  // 12,288) take 66 us with 4 and 2 in the two launches against 72 with 16 and 4, and 60.8 against 61.2 us with 3 and
  // 2 in the second; 64 mixed rows of 24 adapters 13.5 with 28 against 15.4 with 16. (One launch less, with the first
  // product unsliced on 16 waves and its parts finished in place, is slower: 15.9 us for the 64 rows, 80 against 37 at
  // rank 64 and n = 12,288.)
  const int64_t blocks = (g.m + 63) / 64;
  const int32_t* by_row = g.ids;
  int64_t most = g.adapters < 59 ? g.adapters + 5 : 64;
  // In a prompt of mixed rows every block reads its part of nearly all the adapters, and sorted rows read each about
  // once; the sort costs 4 us, which rows that come in runs pay for nothing. At n = 12,288, k = 4,096, rank 64, 1,531
  // mixed rows of 64 / 24 / 8 / 3 adapters take 101 / 84 / 75 / 68 us sorted, 321 / 201 / 116 / 79 not, and in runs of
  // 24 / 3 82 / 65.5 and 77 / 61.5; at n = 4,096 and rank 16, 1,000 rows of 16 take 25 and 29 us, 256 rows of 16 18.0
  // and 16.6. So it runs from the bytes on at which mixed rows gain about four times its cost.
  if ((blocks - 1) * (g.adapters < 60 ? g.adapters : 60) * (32 * RT) * (g.n + g.k) >= kSortBytes) {
    int32_t* sorted = reinterpret_cast<int32_t*>(static_cast<char*>(g.ws) + sums_bytes(g.m, g.rank) +
                                                 parts_bytes(g.m, g.rank));
    hipLaunchKernelGGL(lora_sort_kernel, dim3(static_cast<unsigned>((g.m + kChunk - 1) / kChunk)), dim3(kBins), 0,
                       g.stream, g.ids, g.m, g.adapters, sorted, sorted + g.m);
    g.ids = sorted;
    g.perm = sorted + g.m;
    const int64_t few = 6 + g.adapters / (blocks < 64 ? blocks : 64);
    most = few < most ? few : most;
  }
  auto share = [&](int64_t workgroups, int64_t fill) {
    const int64_t z = fill / workgroups < 3 ? 3 : fill / workgroups;
    return z < most ? z : most;
  };
  launch_down<64, RT, FAST>(g, slices, ks, share(blocks * slices, 768));
  if constexpr (RT == 1) {
    // One block and few columns: each workgroup adds the slices of its groups again, which costs less than a launch
    // (64 rows of 24 adapters, rank 16: 11.7 against 13.5 us at n = 4,096, 14.4 against 14.0 at n = 8,192).
    if (blocks == 1 && g.n <= 6144) {
      launch_up<64, RT, 2, true, FAST>(g, slices, share((g.n + 32 * kWaves - 1) / (32 * kWaves), 2048));
      return;
    }
  }
  _Float16* parts = reinterpret_cast<_Float16*>(static_cast<char*>(g.ws) + sums_bytes(g.m, g.rank));
  hipLaunchKernelGGL((lora_join_kernel<RT>), dim3(static_cast<unsigned>((g.m + 15) / 16)), dim3(256), 0, g.stream,
                     by_row, g.scale, g.m, g.adapters, g.rank, slices, static_cast<float*>(g.ws), parts,
                     reinterpret_cast<float*>(parts + g.m * 32 * RT));
  // 64 columns of a wave need the workgroups to fill the chip: at n = 4,096 1,000 rows of 16 adapters take 29.1 us with
  // them and 25.9 with 32, 512 rows 22.5 and 19.8; at n = 12,288 1,531 rows of 3 61.6 and 64.5.
  const int64_t wide = blocks * ((g.n + 64 * kWaves - 1) / (64 * kWaves));
  if (wide >= 384) launch_up<64, RT, 4, false, FAST>(g, slices, share(wide, 2048));
  else launch_up<64, RT, 2, false, FAST>(g, slices, share(2 * wide, 2048));
}

template <bool FAST>
void launch_rank(const Args& g) {
  switch (rank_padded(g.rank)) {
    case 16: return launch<1, FAST>(g);
    case 32: return launch<2, FAST>(g);
    case 64: return launch<4, FAST>(g);
    default: return launch<8, FAST>(g);
  }
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace

// No less than for fewer rows: what one call needs falls where its slices do,
// after 16 rows and after the last row count with each number of slices.
int64_t lora_workspace_bytes(int64_t m, int rank) {
  auto call = [&](int64_t rows) {
    return sums_bytes(rows, rank) + (lora_one_block(rows) ? 0 : parts_bytes(rows, rank)) + (rows > 64 ? 8 * rows : 0);
  };
  int64_t most = call(m);
  for (int64_t last : {kRows, kSliced / 8, kSliced / 7, kSliced / 6, kSliced / 5, kSliced / 4, kSliced / 3}) {
    const int64_t b = call(last < m ? last : m);
    most = b > most ? b : most;
  }
  return most;
}

hipError_t launch_lora_add(const float* y, const uint16_t* x, const int32_t* ids, const uint16_t* a, const uint16_t* b,
                           const float* scale, int64_t m, int64_t n, int64_t k, int adapters, int rank, float* out,
                           void* ws, hipStream_t stream) {
  const Args g{y, x, ids, a, b, scale, m, n, k, adapters, rank, out, nullptr, ws, stream};
  if (k % 8 == 0 && rank % 8 == 0 && !off16(x) && !off16(a) && !off16(b)) launch_rank<true>(g);
  else launch_rank<false>(g);
  return hipGetLastError();
}

}  // namespace pbg
