// lora_add: out_i = y_i + s_a B_a (A_a x_i) with a = ids[i], the adapters of
// many requests at once beside a shared projection; rows without an adapter
// are passed through.
//
// Two launches. The first forms v_i = A_a x_i on the f16 matrix cores (fp16
// products are exact in its fp32 sums), K split over the waves of a workgroup
// and, for few rows, over workgroups; the slices' sums go to the workspace.
// The second adds the slices in order and multiplies by B_a: v stays fp32 in
// effect, split into two fp16 parts, so that B_a can stay fp16 on the matrix
// cores.
//
// Both take 16 rows at a time and run once for each different adapter among
// them; a row takes the result of its own adapter by a select, so infinities
// or NaN in another request's adapter never reach it.
#include "pbg_device.hpp"
#include "pbg_internal.hpp"

namespace pbg {
namespace {

constexpr int kRows = 16;
constexpr int kWaves = 4;

// ids of a 16-row tile, -1 for rows past m and rows without an adapter (lane
// l of every wave holds row l % 16).
__device__ __forceinline__ int tile_id(const int32_t* __restrict__ ids, int64_t row, int64_t m, int adapters) {
  const int id = row < m ? ids[row] : -1;
  return id >= 0 && id < adapters ? id : -1;
}

// Bit i (0..15): row i is the tile's first one with its adapter.
__device__ __forceinline__ uint32_t first_rows(int id) {
  const int li = threadIdx.x & 15;
  bool first = id >= 0;
#pragma unroll
  for (int j = 0; j < 15; ++j) first &= !(j < li && __builtin_amdgcn_readlane(id, j) == id);
  return static_cast<uint32_t>(__ballot(first)) & 0xFFFFu;
}

// Eight fp16 elements p[c .. c + 7], zero from column k on; FAST: 16-byte
// aligned and k a multiple of 8.
template <bool FAST>
__device__ __forceinline__ mfma_half8_t load8(const uint16_t* __restrict__ p, int64_t c, int64_t k) {
  if constexpr (FAST) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c < k) v = *reinterpret_cast<const uint4*>(p + c);
    return __builtin_bit_cast(mfma_half8_t, v);
  } else {
    mfma_half8_t v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < k ? __builtin_bit_cast(_Float16, p[c + e]) : static_cast<_Float16>(0.0f);
    return v;
  }
}

// v[slice][row][rank] for one 16-row tile (blockIdx.x) and one slice of K
// (blockIdx.y); blockIdx.z is the first of the tile's adapters (stepping by
// gridDim.z). The waves take 32-column steps in turn, U steps of loads in
// flight; K is cut into slices until the launch fills the chip, since a tile
// alone is bound by the latency of its loads.
template <int RT, bool FAST>
__global__ __launch_bounds__(kWaves* kWave) void lora_down_kernel(const uint16_t* __restrict__ x,
                                                                  const int32_t* __restrict__ ids,
                                                                  const uint16_t* __restrict__ a, int64_t m, int64_t k,
                                                                  int adapters, int rank, int64_t k_slice,
                                                                  float* __restrict__ v) {
  constexpr int U = RT >= 8 ? 2 : RT >= 4 ? 4 : 8;
  __shared__ mfma_float4_t part[kWaves - 1][RT][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int li = lane & 15, lg = lane >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kRows;
  const int id = tile_id(ids, m0 + li, m, adapters);
  const int64_t k0 = blockIdx.y * k_slice;
  const int64_t k1 = k0 + k_slice < k ? k0 + k_slice : k;
  const uint16_t* xr = x + (m0 + li < m ? m0 + li : m - 1) * k;
  uint32_t todo = first_rows(id);
  for (int d = 0; todo; ++d) {
    const int f = __builtin_ctz(todo);
    todo &= todo - 1;
    if (d % gridDim.z != blockIdx.z) continue;
    const int ad = __builtin_amdgcn_readlane(id, f);
    const uint16_t* ar[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int j = 16 * t + li;
      ar[t] = a + (static_cast<int64_t>(ad) * rank + (j < rank ? j : rank - 1)) * k;
    }
    mfma_float4_t acc[RT] = {};
    for (int64_t c0 = k0 + 32 * wave; c0 < k1; c0 += 32 * kWaves * U) {
      mfma_half8_t xv[U], av[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + 32 * kWaves * u + 8 * lg;
        xv[u] = load8<FAST>(xr, c, k1);
#pragma unroll
        for (int t = 0; t < RT; ++t) av[u][t] = load8<FAST>(ar[t], c, k1);
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
    if (wave == 0) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int w = 0; w < kWaves - 1; ++w) acc[t] += part[w][t][lane];
        const int j = 16 * t + li;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 4 * lg + e;  // row of the tile
          const int idi = __shfl(id, i);
          if (j < rank && idi == ad) v[(blockIdx.y * m + m0 + i) * rank + j] = acc[t][e];
        }
      }
    }
  }
}

typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));

// out = y + (s_a 2^-e) B_a (hi + lo) for one 16-row tile and 16 C kWaves
// columns. First the tile's v: the slices' sums in order, then a power of two
// that brings the row's largest |v| to [2^13, 2^14), then two fp16 parts,
// which hold v to 2^-22 of itself (2^-38 of the row's largest). One matrix
// instruction takes 16 of the rank with both parts: its 32 columns are
// [hi | lo] against [B_a | B_a]. With B_a as the row operand a lane ends up
// with four consecutive outputs of one row. Bound by y and out; the C column
// tiles of a wave are loaded together.
template <int RT, int C, bool FAST>
__global__ __launch_bounds__(kWaves* kWave) void lora_up_kernel(const float* y, const int32_t* __restrict__ ids,
                                                                const uint16_t* __restrict__ b,
                                                                const float* __restrict__ scale, int64_t m, int64_t n,
                                                                int adapters, int rank, int slices, int64_t n_blocks,
                                                                const float* __restrict__ v, float* out) {
  constexpr int RP = 16 * RT;
  __shared__ _Float16 parts[2][kRows][RP + 8];
  __shared__ float back[kRows];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int li = lane & 15, lg = lane >> 4;
  const int64_t m0 = blockIdx.x / n_blocks * kRows;
  const int id = tile_id(ids, m0 + li, m, adapters);
  {
    const int i = threadIdx.x >> 4;  // row of the tile, on the 16 lanes of a DPP row
    const int idi = __shfl(id, i);
    float s[RT], top = 0.0f;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int j = 16 * t + li;
      s[t] = 0.0f;
      if (idi >= 0 && j < rank)
        for (int p = 0; p < slices; ++p) s[t] += v[(p * m + m0 + i) * rank + j];
      top = fmaxf(top, fabsf(s[t]));
    }
    top = fmaxf(top, row_ror<8>(top));
    top = fmaxf(top, row_ror<4>(top));
    top = fmaxf(top, row_ror<2>(top));
    top = fmaxf(top, row_ror<1>(top));
    const int e = top > 0.0f && top < __builtin_inff() ? 13 - ilogbf(top) : 0;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float w = ldexpf(s[t], e);
      const _Float16 hi = static_cast<_Float16>(w);
      parts[0][i][16 * t + li] = hi;
      parts[1][i][16 * t + li] = static_cast<_Float16>(w - static_cast<float>(hi));
    }
    if (li == 0) back[i] = idi >= 0 ? ldexpf(scale[idi], -e) : 0.0f;
  }
  __syncthreads();
  mfma_half8_t vf[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
    vf[t] = *reinterpret_cast<const mfma_half8_t*>(&parts[lg >> 1][li][16 * t + 8 * (lg & 1)]);
  const float bk = back[li];
  const int64_t n0 = (blockIdx.x % n_blocks * kWaves + wave) * (16 * C);
  if (n0 >= n) return;
  const bool in = m0 + li < m;
  const float* yr = y + (m0 + li) * n;
  float* o = out + (m0 + li) * n;
  mfma_float4_t base[C], acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t r = n0 + 16 * c + 4 * lg;
    acc[c] = mfma_float4_t{};
    base[c] = mfma_float4_t{};
    if (in && r + 4 <= n) {
      base[c] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any_t*>(yr + r));
    } else if (in) {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (r + e < n) base[c][e] = yr[r + e];
    }
  }
  for (uint32_t todo = first_rows(id); todo; todo &= todo - 1) {
    const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const uint16_t* ba = b + static_cast<int64_t>(ad) * n * rank;
    mfma_half8_t bv[C][RT];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t r = n0 + 16 * c + li;
#pragma unroll
      for (int t = 0; t < RT; ++t) bv[c][t] = load8<FAST>(ba + (r < n ? r : n - 1) * rank, 16 * t + 8 * (lg & 1), rank);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      mfma_float4_t d = {};
#pragma unroll
      for (int t = 0; t < RT; ++t) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(bv[c][t], vf[t], d, 0, 0, 0);
      if (id == ad) acc[c] = d;
    }
  }
  if (!in) return;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t r = n0 + 16 * c + 4 * lg;
    if (id >= 0) base[c] += bk * acc[c];
    if (r + 4 <= n) {
      *reinterpret_cast<f32x4_any_t*>(o + r) = base[c];
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (r + e < n) o[r + e] = base[c][e];
    }
  }
}

// Columns of one slice: whole steps of the down kernel's four waves.
int64_t slice_columns(int64_t k, int slices) {
  const int64_t step = 32 * kWaves;
  return ((k + slices - 1) / slices + step - 1) / step * step;
}

template <int RT, bool FAST>
void launch(const float* y, const uint16_t* x, const int32_t* ids, const uint16_t* a, const uint16_t* b,
            const float* scale, int64_t m, int64_t n, int64_t k, int adapters, int rank, float* out, float* ws,
            hipStream_t stream) {
  const int64_t tiles = (m + kRows - 1) / kRows;
  const int64_t ks = slice_columns(k, lora_slices(m));
  const int slices = static_cast<int>((k + ks - 1) / ks);
  // few tiles: their adapters go to workgroups of their own
  const unsigned dz = tiles <= 32 ? (m < 16 ? static_cast<unsigned>(m) : 16) : 1;
  hipLaunchKernelGGL((lora_down_kernel<RT, FAST>), dim3(static_cast<unsigned>(tiles), slices, dz),
                     dim3(kWaves * kWave), 0, stream, x, ids, a, m, k, adapters, rank, ks, ws);
  constexpr int C = RT >= 8 ? 2 : 4;
  if (tiles * n >= 16 * 4096) {
    const int64_t nb = (n + 16 * C * kWaves - 1) / (16 * C * kWaves);
    hipLaunchKernelGGL((lora_up_kernel<RT, C, FAST>), dim3(static_cast<unsigned>(nb * tiles)), dim3(kWaves * kWave), 0,
                       stream, y, ids, b, scale, m, n, adapters, rank, slices, nb, ws, out);
  } else {
    const int64_t nb = (n + 16 * kWaves - 1) / (16 * kWaves);
    hipLaunchKernelGGL((lora_up_kernel<RT, 1, FAST>), dim3(static_cast<unsigned>(nb * tiles)), dim3(kWaves * kWave), 0,
                       stream, y, ids, b, scale, m, n, adapters, rank, slices, nb, ws, out);
  }
}

template <bool FAST>
void launch_rank(const float* y, const uint16_t* x, const int32_t* ids, const uint16_t* a, const uint16_t* b,
                 const float* scale, int64_t m, int64_t n, int64_t k, int adapters, int rank, float* out, float* ws,
                 hipStream_t stream) {
  if (rank <= 16) launch<1, FAST>(y, x, ids, a, b, scale, m, n, k, adapters, rank, out, ws, stream);
  else if (rank <= 32) launch<2, FAST>(y, x, ids, a, b, scale, m, n, k, adapters, rank, out, ws, stream);
  else if (rank <= 64) launch<4, FAST>(y, x, ids, a, b, scale, m, n, k, adapters, rank, out, ws, stream);
  else launch<8, FAST>(y, x, ids, a, b, scale, m, n, k, adapters, rank, out, ws, stream);
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace

// Enough slices of K to fill the chip with 16-row tiles.
int lora_slices(int64_t m) {
  const int64_t tiles = (m + kRows - 1) / kRows;
  const int64_t s = 1024 / tiles;
  return static_cast<int>(s < 2 ? 2 : s > 16 ? 16 : s);
}

hipError_t launch_lora_add(const float* y, const uint16_t* x, const int32_t* ids, const uint16_t* a, const uint16_t* b,
                           const float* scale, int64_t m, int64_t n, int64_t k, int adapters, int rank, float* out,
                           float* ws, hipStream_t stream) {
  if (k % 8 == 0 && rank % 8 == 0 && !off16(x) && !off16(a) && !off16(b))
    launch_rank<true>(y, x, ids, a, b, scale, m, n, k, adapters, rank, out, ws, stream);
  else
    launch_rank<false>(y, x, ids, a, b, scale, m, n, k, adapters, rank, out, ws, stream);
  return hipGetLastError();
}

}  // namespace pbg
