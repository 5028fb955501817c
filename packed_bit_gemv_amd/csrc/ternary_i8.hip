// ternary_gemm_i8 and ternary_swiglu_gate_up_i8: packed ternary matrices times
// 8-bit activation rows, any number of rows.
//
// y[i][r] = q_scale_i * s_r * sum_j c_rj q_ij. Codes are decoded in registers
// to bytes 64 * c and multiplied on the i8 matrix cores; the int32 sums are
// exact (64 * 128 * 2^17 = 2^30), so any split of K gives the same bits.
#include "pbg_device.hpp"
#include "pbg_internal.hpp"

namespace pbg {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

constexpr uint32_t kByteMask = 0xC0C0C0C0u;
constexpr int kCodeShift = 6;  // decoded bytes are 64 * c

// The 16 codes of a word as bytes 64 * c in column order. Code 2t + h is the
// field at bits 16h + 14 - 2t: bytes 1 and 3 of the word hold codes 0..7
// (even and odd ones), bytes 0 and 2 codes 8..15, highest field first. One
// permute per half pairs the two bytes with themselves shifted by one field;
// a shift by two fields then gives the next four codes, and the mask drops
// what was carried across bytes (it stays below each byte's top field).
__device__ __forceinline__ i32x4_t word_bytes(uint32_t w) {
  const uint32_t s = w << 2;
  const uint32_t lo = __builtin_amdgcn_perm(s, w, 0x07050301u);
  const uint32_t hi = __builtin_amdgcn_perm(s, w, 0x06040200u);
  const uint64_t next = shl64<4>(static_cast<uint64_t>(hi) << 32 | lo);
  i32x4_t o;
  o[0] = static_cast<int>(lo & kByteMask);
  o[1] = static_cast<int>(static_cast<uint32_t>(next) & kByteMask);
  o[2] = static_cast<int>(hi & kByteMask);
  o[3] = static_cast<int>(static_cast<uint32_t>(next >> 32) & kByteMask);
  return o;
}

// Chunk c of a row (the last one past its end, for the caller to mask).
__device__ __forceinline__ i32x4_t load_chunk(const uint4* __restrict__ row, int64_t c, int64_t chunks) {
  return *reinterpret_cast<const i32x4_t*>(row + (c < chunks ? c : chunks - 1));
}

// Matrix product of few activation rows: a workgroup owns T tiles of 16
// weight rows (of gate and of up each with SWIGLU) against MT tiles of 16
// activation rows and streams the weights. Its SK waves share K in units of
// 256 columns, the next unit's loads in flight under a unit's products: lane
// (i, g) = (l % 16, l / 16) holds the 16-byte chunk 4u + g (64 codes) of
// weight row i, and step w of a unit multiplies word w of the chunk with bytes
// 16w .. 16w + 15 of chunk 4u + g of the activations. Those are loaded 256
// consecutive bytes of a row on 16 lanes and turned through LDS that only this
// wave uses, without a barrier (piece p of row i at place p ^ i: every bank
// once in 16 lanes): read directly, 16 lanes would touch 16 lines. The waves
// add their int32 sums in LDS (exact in any order). Bound by the weight stream
// and the launch: 8 rows by 12,288 x 4,096 take 6.1 us, 7 rows by 4,096 x
// 12,288 6.3-6.5, gate and up for 8 rows 8.6 (25.5 MB, 3.0 TB/s).
template <int MT, int T, int SK, bool SWIGLU>
__global__ __launch_bounds__(SK* kWave) void gemm_i8_stream_kernel(
    const uint4* __restrict__ packed, const float* __restrict__ scale, const uint4* __restrict__ packed2,
    const float* __restrict__ scale2, int64_t n, int64_t chunks, const int8_t* __restrict__ q,
    const float* __restrict__ q_scale, int64_t m, int64_t n_blocks, float* __restrict__ y, uint16_t* __restrict__ h) {
  constexpr int TT = SWIGLU ? 2 * T : T;
  constexpr int kThreads = SK * kWave;
  __shared__ __align__(16) int sums[MT * TT][4][kWave];  // element e of a lane's four sums of a tile
  __shared__ __align__(16) float scales[(MT + TT) * 16];  // of the rows, then of the columns
  const float* row_scale = scales;
  const float* col_scale = scales + MT * 16;
  __shared__ i32x4_t turn[SK][MT][256];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int li = lane & 15, lg = lane >> 4;
  const int64_t n0 = (blockIdx.x % n_blocks) * (16 * T);
  const int64_t m0 = (blockIdx.x / n_blocks) * (16 * MT);
  const int64_t kp = chunks * 64;
  const int64_t units = (chunks + 3) / 4;
  // Addresses are a uniform pointer, moved from unit to unit, plus 32-bit offsets that stay (a row holds at most
  // 131,072 codes, so the rows of a workgroup span less than 2^31 bytes).
  const int64_t row_bytes = chunks * 16;
  uint32_t wo[T], xo[MT][4];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int64_t r = n0 + 16 * t + li < n ? 16 * t + li : n - 1 - n0;
    wo[t] = static_cast<uint32_t>(r * row_bytes + lg * 16);
  }
  // load e of a tile: rows 4e + lg, piece li of the unit
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t r = m0 + 16 * a + 4 * e + lg < m ? 16 * a + 4 * e + lg : m - 1 - m0;
      xo[a][e] = static_cast<uint32_t>(r * kp + li * 16);
    }
  const char* wb[2] = {reinterpret_cast<const char*>(packed) + n0 * row_bytes,
                       SWIGLU ? reinterpret_cast<const char*>(packed2) + n0 * row_bytes : nullptr};
  const char* xb = reinterpret_cast<const char*>(q) + m0 * kp;
  const int rows_in = static_cast<int>(m - m0 < 16 * MT ? m - m0 : 16 * MT);  // rows past m are left out four at a time
  i32x4_t wv[TT], xv[MT][4];
  auto load = [&](int64_t u) {
    // the last unit may hold fewer than four chunks: the others read the row's last one, their codes are masked below
    const int over = 4 * u + 4 > chunks ? static_cast<int>(4 * u + 4 - chunks) : 0;
    uint32_t wback = 0, xback = 0;
    if (over > 0) {
      wback = lg > 3 - over ? 16 * (lg - 3 + over) : 0;
      xback = (li >> 2) > 3 - over ? 64 * ((li >> 2) - 3 + over) : 0;
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
      wv[t] = __builtin_nontemporal_load(reinterpret_cast<const i32x4_t*>(wb[t / T] + u * 64 + (wo[t % T] - wback)));
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (16 * a + 4 * e < rows_in)
          xv[a][e] = *reinterpret_cast<const i32x4_t*>(xb + u * 256 + (xo[a][e] - xback));
  };
  i32x4_t acc[MT][TT] = {};
  // The scales are loaded ahead of everything else (loads return in order), one a thread, and stored to LDS with the
  // zero sums while the first units' loads are on their way.
  static_assert((MT + TT) * 16 <= kThreads, "one scale a thread");
  float one_scale = 0.0f;
  {
    const int i = threadIdx.x, c = i - MT * 16;
    const int64_t r = n0 + c % (16 * T);
    if (i < MT * 16) one_scale = q_scale[m0 + i < m ? m0 + i : m - 1];
    else if (c < TT * 16) one_scale = (c < 16 * T ? scale : scale2)[r < n ? r : n - 1];
  }
  __builtin_amdgcn_sched_barrier(0);
  int64_t u = wave;
  if (u < units) load(u);
  __builtin_amdgcn_sched_barrier(0);
  for (int i = threadIdx.x; i < MT * TT * kWave; i += kThreads) reinterpret_cast<i32x4_t*>(sums)[i] = i32x4_t{};
  if (threadIdx.x < (MT + TT) * 16) scales[threadIdx.x] = one_scale;
  __syncthreads();
  while (u < units) {
    i32x4_t w[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) w[t] = wv[t];
    if (4 * u + 4 > chunks) {
#pragma unroll
      for (int t = 0; t < TT; ++t) w[t] &= 4 * u + lg < chunks ? -1 : 0;
    }
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e) turn[wave][a][(4 * e + lg) * 16 + (li ^ (4 * e + lg))] = xv[a][e];
    u += SK;
    if (u < units) load(u);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      i32x4_t x[MT];
#pragma unroll
      for (int a = 0; a < MT; ++a) x[a] = turn[wave][a][li * 16 + ((4 * lg + s) ^ li)];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const i32x4_t b = word_bytes(static_cast<uint32_t>(w[t][s]));
#pragma unroll
        for (int a = 0; a < MT; ++a) acc[a][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[a], b, acc[a][t], 0, 0, 0);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }

#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        __hip_atomic_fetch_add(&sums[a * TT + t][e][lane], acc[a][t][e], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_WORKGROUP);
  __syncthreads();
  // the tiles in turn to the waves: column li, activation rows 4 lg + e
#pragma unroll
  for (int i = 0; i < (MT * T + SK - 1) / SK; ++i) {
    const int tile = wave + i * SK;
    if (tile >= MT * T) break;
    const int a = tile / T, t = tile % T;
    const int64_t r = n0 + 16 * t + li;
    const mfma_float4_t qs = *reinterpret_cast<const mfma_float4_t*>(row_scale + 16 * a + 4 * lg);
    const float s1 = col_scale[16 * t + li], s2 = SWIGLU ? col_scale[16 * (T + t) + li] : 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t row = m0 + 16 * a + 4 * lg + e;
      if (row >= m || r >= n) continue;
      const float v = static_cast<float>(sums[a * TT + t][e][lane] >> kCodeShift) * qs[e] * s1;
      if constexpr (SWIGLU) {
        const float v2 = static_cast<float>(sums[a * TT + T + t][e][lane] >> kCodeShift) * qs[e] * s2;
        h[row * n + r] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(silu(v) * v2));
      } else {
        y[row * n + r] = v;
      }
    }
  }
}

template <int MT, int T, int SK, bool SWIGLU>
void launch_stream(const uint32_t* p1, const float* s1, const uint32_t* p2, const float* s2, int64_t n, int64_t k,
                   const int8_t* q, const float* q_scale, int64_t m, float* y, uint16_t* h, hipStream_t stream) {
  const int64_t nb = (n + 16 * T - 1) / (16 * T), mb = (m + 16 * MT - 1) / (16 * MT);
  hipLaunchKernelGGL((gemm_i8_stream_kernel<MT, T, SK, SWIGLU>), dim3(static_cast<unsigned>(nb * mb)),
                     dim3(SK * kWave), 0, stream, reinterpret_cast<const uint4*>(p1), s1,
                     reinterpret_cast<const uint4*>(p2), s2, n, words_per_row(k) / 4, q, q_scale, m, nb, y, h);
}

// Tile of a workgroup. Workgroups go round the 8 XCDs, each with its own L2:
// an XCD gets a run of consecutive tiles, ordered by groups of kGroupM row
// blocks under one column block, so that the tiles in flight on an XCD share
// both operands.
constexpr int kXcds = 8;
constexpr int kGroupM = 4;

__device__ __forceinline__ void tile_of_block(int m_blocks, int n_blocks, int& mb, int& nb) {
  const int total = m_blocks * n_blocks;
  const int xcd = blockIdx.x % kXcds, at = blockIdx.x / kXcds;
  const int each = total / kXcds, over = total % kXcds;
  const int id = xcd * each + (xcd < over ? xcd : over) + at;
  const int group = id / (kGroupM * n_blocks);
  const int rows = m_blocks - group * kGroupM < kGroupM ? m_blocks - group * kGroupM : kGroupM;
  const int in = id - group * kGroupM * n_blocks;
  mb = group * kGroupM + in % rows;
  nb = in / rows;
}

// Up to M activation rows, K of at most 64 CPL chunks: a wave owns R weight
// rows (of gate and of up each with SWIGLU), lane l the chunks l, l + 64, ...
// of every row, so that each load of a wave is 1 KiB of one row. The
// activations are loaded first, before a barrier that nothing waits for
// behind it, so that they return first; they go through LDS (piece p of chunk
// 64 j + l at (4 j + p) 64 + l) and meet the decoded bytes in dot products of
// four: 8 + 4 M vector instructions a word. The lanes' sums are multiples of
// 64 below 2^30, so the transposed fp32 reduction adds them exactly. Bound by
// the launch and the first bytes, as ternary_gemv is: gate at one row 4.3 us,
// down 4.4, gate and up 6.4 (5.5, 5.5 and 8.2 for the streaming kernel, whose
// loads are 64 bytes of 16 rows).
template <int M, int CPL, int G, int R, bool SWIGLU>
__global__ __launch_bounds__(G* kWave) void gemv_i8_kernel(const uint4* __restrict__ packed,
                                                           const float* __restrict__ scale,
                                                           const uint4* __restrict__ packed2,
                                                           const float* __restrict__ scale2, int64_t n, int64_t chunks,
                                                           const int8_t* q, const float* __restrict__ q_scale, int m,
                                                           float* __restrict__ y, uint16_t* __restrict__ h) {
  constexpr int RR = SWIGLU ? 2 * R : R;  // row i of the wave: weight row i / 2 of gate (even) or up (odd) with SWIGLU
  constexpr int kSums = M * RR;           // sum of activation row a and weight row i at a RR + i
  constexpr int kRed = (kSums + 3) / 4;
  static_assert(!SWIGLU || kSums % 2 == 0, "a gate sum and its up sum in one reduction");
  constexpr int kThreads = G * kWave;
  constexpr int kPieces = CPL * kWave * 4;
  constexpr int kXPer = (M * kPieces + kThreads - 1) / kThreads;
  __shared__ i32x4_t xs[M][kPieces];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * G + wave) * R;
  const int pieces = static_cast<int>(chunks) * 4;
  const i32x4_t* xg = reinterpret_cast<const i32x4_t*>(q);

  i32x4_t xv[kXPer];
#pragma unroll
  for (int i = 0; i < kXPer; ++i) {
    const int at = threadIdx.x + i * kThreads, a = at / kPieces, p = at % kPieces;
    xv[i] = xg[a < m && p < pieces ? a * pieces + p : 0];
  }
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");  // order, not wait: the loads stay in flight across it
  __builtin_amdgcn_sched_barrier(0);

  i32x4_t w[RR][CPL];
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const int64_t c = lane + kWave * j;
    const int64_t cc = c < chunks ? c : chunks - 1;
#pragma unroll
    for (int i = 0; i < RR; ++i) {
      const int64_t r = row0 + (SWIGLU ? i / 2 : i);
      const uint4* base = SWIGLU && (i & 1) ? packed2 : packed;
      w[i][j] = __builtin_nontemporal_load(reinterpret_cast<const i32x4_t*>(base + (r < n ? r : n - 1) * chunks + cc));
    }
  }
  // the sums that this lane gets: slot i of each reduction
  const int slot = reduce4_slot(lane);
  float row_s[kRed], col_s[kRed];  // applied one after the other, as the other kernels do
#pragma unroll
  for (int e = 0; e < kRed; ++e) {
    const int idx = 4 * e + (slot < 0 ? 0 : slot), a = idx / RR, i = idx % RR;
    const int64_t r = row0 + (SWIGLU ? i / 2 : i);
    row_s[e] = q_scale[a < m ? a : m - 1];
    col_s[e] = (SWIGLU && (i & 1) ? scale2 : scale)[r < n ? r : n - 1];
  }
  __builtin_amdgcn_sched_barrier(0);

  // chunks past the row hold 0 activations
#pragma unroll
  for (int i = 0; i < kXPer; ++i) {
    const int at = threadIdx.x + i * kThreads, a = at / kPieces, p = at % kPieces, c = p >> 2;
    if (a < M) xs[a][((c >> 6) * 4 + (p & 3)) * kWave + (c & (kWave - 1))] = xv[i] & (p < pieces ? -1 : 0);
  }
  __syncthreads();
  int acc[4 * kRed] = {};
#pragma unroll
  for (int j = 0; j < CPL; ++j)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      i32x4_t x[M];
#pragma unroll
      for (int a = 0; a < M; ++a) x[a] = xs[a][(4 * j + s) * kWave + lane];
#pragma unroll
      for (int i = 0; i < RR; ++i) {
        const i32x4_t b = word_bytes(static_cast<uint32_t>(w[i][j][s]));
#pragma unroll
        for (int a = 0; a < M; ++a)
#pragma unroll
          for (int d = 0; d < 4; ++d) acc[a * RR + i] = __builtin_amdgcn_sdot4(b[d], x[a][d], acc[a * RR + i], false);
      }
    }
#pragma unroll
  for (int e = 0; e < kRed; ++e) {
    const float red = wave_reduce4(static_cast<float>(acc[4 * e]), static_cast<float>(acc[4 * e + 1]),
                                   static_cast<float>(acc[4 * e + 2]), static_cast<float>(acc[4 * e + 3]));
    const float v = red * (1.0f / (1 << kCodeShift)) * row_s[e] * col_s[e];
    const int idx = 4 * e + slot, a = idx / RR, i = idx % RR;
    const int64_t r = row0 + (SWIGLU ? i / 2 : i);
    const bool in = slot >= 0 && idx < kSums && a < m && r < n;
    if constexpr (SWIGLU) {
      const float u = __shfl_xor(v, 32);  // slots 0 and 1, 2 and 3 are 32 lanes apart
      if (in && (slot & 1) == 0) h[a * n + r] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(silu(v) * u));
    } else {
      if (in) y[a * n + r] = v;
    }
  }
}

template <int M, int CPL, int G, int R, bool SWIGLU>
void launch_gemv(const uint32_t* p1, const float* s1, const uint32_t* p2, const float* s2, int64_t n, int64_t k,
                 const int8_t* q, const float* q_scale, int64_t m, float* y, uint16_t* h, hipStream_t stream) {
  hipLaunchKernelGGL((gemv_i8_kernel<M, CPL, G, R, SWIGLU>), dim3(static_cast<unsigned>((n + G * R - 1) / (G * R))),
                     dim3(G * kWave), 0, stream, reinterpret_cast<const uint4*>(p1), s1,
                     reinterpret_cast<const uint4*>(p2), s2, n, words_per_row(k) / 4, q, q_scale, static_cast<int>(m),
                     y, h);
}

// Order of one word's work: the next word's operand reads first, then its
// decode in shares between the matrix instructions, which cover both.
template <int TM, int TN>
__device__ __forceinline__ void interleave() {
  __builtin_amdgcn_sched_group_barrier(0x100, TM, 0);  // LDS reads
#pragma unroll
  for (int i = 0; i < TM * TN; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one matrix instruction
    __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);  // vector instructions
  }
  __builtin_amdgcn_sched_barrier(0);
}

// Matrix product of many activation rows: a workgroup of WM x WN waves owns
// 32 TM WM rows by 32 TN WN columns, a wave TM x TN tiles of the 32x32x32 i8
// matrix instruction, whose A operand is activations and B operand decoded
// codes. K goes in steps of two chunks (128 columns), four words a lane. The
// activations go through LDS, double-buffered with one barrier a step: a step
// starts by storing the next step's activations, which were loaded during the
// step before, into the buffer that every wave has read by then, and reaches
// the barrier with only its last word's products left, whose operands are in
// registers; they run while the first operands of the next step are read.
// 16-byte piece c of row i sits at place c ^ (i / 2 % 8) of its 128 bytes, so
// that 16 lanes of a store or an operand read touch each of the 64 banks once.
// Bound by the matrix cores at the clock that the power allows: 4,096 x 4,096
// x 12,288 takes 156-165 us, 2.5-2.65e15 operations/s (3.13e15 on zeros, the
// matrix cores then busy 62 % of the cycles).
// Loads are issued D steps ahead (one for the largest tile, whose step is
// longer than a load; four for small tiles, whose steps are short). The
// packed words come straight to registers (lane (i, g) = (l % 32, l / 32) the
// chunk 2u + g of column i) and are decoded once for all TM row tiles, which
// is what pays for the decode: 8 vector instructions a word against TM matrix
// instructions of 32 cycles.
template <int WM, int WN, int TM, int TN, int D, bool SWIGLU>
__global__ __launch_bounds__(WM* WN* kWave) void gemm_i8_tile_kernel(
    const uint4* __restrict__ packed, const float* __restrict__ scale, const uint4* __restrict__ packed2,
    const float* __restrict__ scale2, int64_t n, int64_t chunks, const int8_t* __restrict__ q,
    const float* __restrict__ q_scale, int64_t m, int m_blocks, int n_blocks, float* __restrict__ y,
    uint16_t* __restrict__ h) {
  static_assert(D == 1 || D % 2 == 0, "the buffers of a step are known at compile time");
  static_assert(!SWIGLU || TN % 2 == 0, "a wave holds as many gate tiles as up tiles");
  constexpr int kThreads = WM * WN * kWave;
  constexpr int BM = 32 * TM * WM;
  constexpr int TC = SWIGLU ? TN / 2 : TN;  // column tiles of a wave
  constexpr int BN = 32 * TC * WN;
  constexpr int kLoads = BM * 8 / kThreads;
  static_assert(BM * 8 % kThreads == 0, "whole loads");
  __shared__ i32x4_t xs[2][BM * 8];
  __shared__ __align__(16) float row_scale[BM];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int li = lane & 31, lg = lane >> 5;
  const int wm = wave / WN, wn = wave % WN;
  int mb, nb;
  tile_of_block(m_blocks, n_blocks, mb, nb);
  const int64_t m0 = static_cast<int64_t>(mb) * BM;
  const int64_t n0 = static_cast<int64_t>(nb) * BN + wn * (32 * TC);
  const int64_t kp = chunks * 64;
  const int64_t steps = (chunks + 1) / 2;

  const uint4* wp[TN];
#pragma unroll
  for (int t = 0; t < TN; ++t) {
    const int64_t r = n0 + 32 * (t % TC) + li;
    wp[t] = (t < TC ? packed : packed2) + (r < n ? r : n - 1) * chunks;
  }
  const int8_t* xp[kLoads];  // this thread's pieces: row (threadIdx.x + i kThreads) / 8, piece threadIdx.x % 8
  int xo[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = (threadIdx.x + i * kThreads) >> 3, c = threadIdx.x & 7;
    const int64_t r = m0 + row;
    xp[i] = q + (r < m ? r : m - 1) * kp + 16 * c;
    xo[i] = row * 8 + (c ^ (row >> 1 & 7));
  }
  float s1[TN];
#pragma unroll
  for (int t = 0; t < TN; ++t) {
    const int64_t r = n0 + 32 * (t % TC) + li;
    s1[t] = (t < TC ? scale : scale2)[r < n ? r : n - 1];
  }
  for (int i = threadIdx.x; i < BM; i += kThreads) row_scale[i] = q_scale[m0 + i < m ? m0 + i : m - 1];
  const int half = (threadIdx.x & 7) >> 2;  // chunk of the step that this thread's pieces belong to
  i32x4_t xv[D][kLoads], wv[D][TN], w[TN], a[2][TM], b[2][TN];
  // Steps past the last one read it again, chunks past the row (the last step of an odd count) the row's last one:
  // activations as they are, codes 0 (masked when used, so that nothing waits for the load before its step).
  auto load_x = [&](int64_t u, int slot) {
    const int64_t v = u < steps ? u : steps - 1;
    const int64_t at = v * 128 - (2 * v + half < chunks ? 0 : 64);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) xv[slot][i] = *reinterpret_cast<const i32x4_t*>(xp[i] + at);
  };
  auto load_w = [&](int64_t u, int slot) {
#pragma unroll
    for (int t = 0; t < TN; ++t) wv[slot][t] = load_chunk(wp[t], 2 * u + lg, chunks);
  };
  auto store_x = [&](int buffer, int slot) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) xs[buffer][xo[i]] = xv[slot][i];
  };
  auto take_w = [&](int64_t u, int slot) {
#pragma unroll
    for (int t = 0; t < TN; ++t) w[t] = wv[slot][t] & (2 * u + lg < chunks ? -1 : 0);
  };
  const int row8 = (wm * TM * 32 + li) * 8;
  auto operands = [&](int buffer, int s) {
#pragma unroll
    for (int i = 0; i < TM; ++i) a[s & 1][i] = xs[buffer][row8 + i * 256 + ((4 * lg + s) ^ (li >> 1 & 7))];
#pragma unroll
    for (int t = 0; t < TN; ++t) b[s & 1][t] = word_bytes(static_cast<uint32_t>(w[t][s]));
  };
  i32x16_t acc[TM][TN] = {};
  auto multiply = [&](int s) {
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int i = 0; i < TM; ++i)
        acc[i][t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[s & 1][i], b[s & 1][t], acc[i][t], 0, 0, 0);
  };

  load_x(0, 0);
  load_w(0, 0);
  store_x(0, 0);
  take_w(0, 0);
#pragma unroll
  for (int d = 1; d <= D; ++d) load_x(d, d % D);
#pragma unroll
  for (int d = 1; d < D; ++d) load_w(d, d);
  __syncthreads();
  operands(0, 0);
  // steps past the last one (to a whole number of D) multiply codes 0
  for (int64_t u0 = 0; u0 < steps; u0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int64_t u = u0 + d;
      const int here = D > 1 ? d & 1 : static_cast<int>(u & 1), next = here ^ 1;
      store_x(next, (d + 1) % D);
      load_w(u + D, d);
      load_x(u + 1 + D, (d + 1) % D);
      __builtin_amdgcn_sched_barrier(0);
      operands(here, 1);
      multiply(0);
      interleave<TM, TN>();
      operands(here, 2);
      multiply(1);
      interleave<TM, TN>();
      operands(here, 3);
      multiply(2);
      interleave<TM, TN>();
      __syncthreads();
      take_w(u + 1, (d + 1) % D);
      operands(next, 0);
      multiply(3);
      interleave<TM, TN>();
    }
  }

  // lane: column li of a tile, rows 8 g + 4 lg + e; whole tiles store without a check
  const bool whole = m0 + BM <= m && n0 + 32 * TC <= n;
  auto store = [&](int64_t at, int i, int t, int e, float qs) {
    const float v = static_cast<float>(acc[i][t][e] >> kCodeShift) * qs * s1[t];
    if constexpr (SWIGLU) {
      const float v2 = static_cast<float>(acc[i][TC + t][e] >> kCodeShift) * qs * s1[TC + t];
      h[at] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(silu(v) * v2));
    } else {
      y[at] = v;
    }
  };
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int row = (wm * TM + i) * 32 + 8 * g + 4 * lg;
      const mfma_float4_t qs = *reinterpret_cast<const mfma_float4_t*>(row_scale + row);
      const int64_t at = (m0 + row) * n + n0 + li;
      if (whole) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int t = 0; t < TC; ++t) store(at + e * n + 32 * t, i, t, 4 * g + e, qs[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int t = 0; t < TC; ++t)
            if (m0 + row + e < m && n0 + 32 * t + li < n) store(at + e * n + 32 * t, i, t, 4 * g + e, qs[e]);
      }
    }
}

template <int WM, int WN, int TM, int TN, int D, bool SWIGLU>
void launch_tile(const uint32_t* p1, const float* s1, const uint32_t* p2, const float* s2, int64_t n, int64_t k,
                 const int8_t* q, const float* q_scale, int64_t m, float* y, uint16_t* h, hipStream_t stream) {
  constexpr int BM = 32 * TM * WM, BN = 32 * (SWIGLU ? TN / 2 : TN) * WN;
  const int64_t nb = (n + BN - 1) / BN, mb = (m + BM - 1) / BM;
  hipLaunchKernelGGL((gemm_i8_tile_kernel<WM, WN, TM, TN, D, SWIGLU>), dim3(static_cast<unsigned>(nb * mb)),
                     dim3(WM * WN * kWave), 0, stream, reinterpret_cast<const uint4*>(p1), s1,
                     reinterpret_cast<const uint4*>(p2), s2, n, words_per_row(k) / 4, q, q_scale, m,
                     static_cast<int>(mb), static_cast<int>(nb), y, h);
}

// Rows and columns of a workgroup, and the time of a round of 256 of them (one
// a CU) in us.
struct Shape {
  int rows, columns;
  double round;
};

// The shape that takes the least rounds x time of a round.
template <int N>
int pick_shape(const Shape (&shapes)[N], int64_t m, int64_t columns) {
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < N; ++i) {
    const Shape& s = shapes[i];
    const int64_t groups = (m + s.rows - 1) / s.rows * ((columns + s.columns - 1) / s.columns);
    const double t = static_cast<double>((groups + 255) / 256) * s.round;
    if (i == 0 || t < least) {
      best = i;
      least = t;
    }
  }
  return best;
}

// The kernels of one to eight rows whose loads are whole pieces of one row (us
// against the best streaming shape, k = 4,096 unless stated): one row n =
// 1,024 / 4,096 / 6,144 / 12,288 2.3 / 2.9 / 3.3 / 4.3 against 3.2 / 3.9 / 4.6
// / 5.5, k = 12,288 4.4 against 5.5; two rows 2.5 / 3.2 / 3.7 / 4.7 against
// 3.7 / 4.0 / 4.7 / 5.7; three and four rows below n = 8,192 2.7 / 3.5 / 4.1
// against 3.9 / 4.1 / 4.9 (12,288: 6.1 against 5.8); up to eight rows at n <=
// 2,048 3.2 against 4.1 (4,096: 4.8 against 4.3). Two weight rows a wave from
// n = 8,192 on (4.28 against 4.8 us for one), below it one (3.27 against 3.38
// at 6,144), for K of several chunks a lane two from n = 4,096 on.
bool launch_gemv_rows(const uint32_t* packed, const float* scale, int64_t n, int64_t k, const int8_t* q,
                      const float* q_scale, int64_t m, float* y, hipStream_t stream) {
#define PBG_GEMV(...) \
  (launch_gemv<__VA_ARGS__, false>(packed, scale, nullptr, nullptr, n, k, q, q_scale, m, y, nullptr, stream), true)
  const int64_t cpl = (words_per_row(k) / 4 + kWave - 1) / kWave;  // chunks a lane
  if (m == 1) {
    switch (cpl) {
      case 1: return n >= 8192 ? PBG_GEMV(1, 1, 4, 2) : PBG_GEMV(1, 1, 4, 1);
      case 2: return n >= 4096 ? PBG_GEMV(1, 2, 4, 2) : PBG_GEMV(1, 2, 4, 1);
      case 3: return n >= 4096 ? PBG_GEMV(1, 3, 4, 2) : PBG_GEMV(1, 3, 4, 1);
      case 4: return n >= 4096 ? PBG_GEMV(1, 4, 4, 2) : PBG_GEMV(1, 4, 4, 1);
      default: return false;
    }
  }
  if (m == 2) {
    switch (cpl) {
      case 1: return n >= 4096 ? PBG_GEMV(2, 1, 4, 2) : PBG_GEMV(2, 1, 4, 1);
      case 2: return PBG_GEMV(2, 2, 4, 2);
      case 3: return PBG_GEMV(2, 3, 4, 2);
      default: return false;
    }
  }
  if (m <= 4 && cpl == 1 && n < 8192) return PBG_GEMV(4, 1, 8, 1);
  if (m <= 8 && cpl == 1 && n <= 2048) return PBG_GEMV(8, 1, 4, 1);
#undef PBG_GEMV
  return false;
}

// The same for gate and up: one row 6.4 us against 8.2 (d_ff = 12,288, k =
// 4,096; two pairs for two waves, 6.9 for four), two rows 7.3 against 8.4.
bool launch_gemv_gate_up(const uint32_t* gate, const float* gate_scale, const uint32_t* up, const float* up_scale,
                         int64_t d_model, int64_t d_ff, const int8_t* q, const float* q_scale, int64_t m, uint16_t* h,
                         hipStream_t stream) {
#define PBG_GEMV(...)                                                                                                 \
  (launch_gemv<__VA_ARGS__, true>(gate, gate_scale, up, up_scale, d_ff, d_model, q, q_scale, m, nullptr, h, stream), \
   true)
  const int64_t cpl = (words_per_row(d_model) / 4 + kWave - 1) / kWave;
  if (m == 1) {
    switch (cpl) {
      case 1: return PBG_GEMV(1, 1, 2, 2);
      case 2: return PBG_GEMV(1, 2, 4, 1);
      case 3: return PBG_GEMV(1, 3, 4, 1);
      case 4: return PBG_GEMV(1, 4, 4, 1);
      default: return false;
    }
  }
  if (m == 2 && cpl == 1) return PBG_GEMV(2, 1, 4, 1);
#undef PBG_GEMV
  return false;
}

}  // namespace

// Streaming shapes up to 48 x 64, tiles from 32 x 128 on. The times of a round
// are those of 128 to 256 workgroups at k = 4,096 on MI355X; at k = 12,288 all
// grow alike (by 2.0 to 2.4); below 4,096, where the fixed part of a round
// weighs more, they are not measured. Where it picks a shape, that shape was within 5
// % of the fastest of 24 (m x n at k = 4,096, us against the runner-up of
// another size): 8 x 4,096 4.2 / 5.0, 32 x 4,096 5.3 / 6.1, 64 x 4,096 6.6 /
// 7.4, 100 x 4,096 8.2 / 8.7, 160 x 4,096 10.1 / 11.2, 64 x 12,288 11.5 /
// 16.6, 100 x 12,288 14.3 / 17.2, 256 x 12,288 18.9 / 21.5, 512 x 12,288 31.9
// / 33.2, 1,024 x 12,288 51.1 / 54.2.
hipError_t launch_ternary_gemm_i8(const uint32_t* packed, const float* scale, int64_t n, int64_t k, const int8_t* q,
                                  const float* q_scale, int64_t m, float* y, hipStream_t stream) {
  if (launch_gemv_rows(packed, scale, n, k, q, q_scale, m, y, stream)) return hipGetLastError();
  static const Shape shapes[] = {{16, 16, 4.3}, {16, 32, 5.2}, {16, 48, 6.3},   {16, 64, 6.5},   {32, 32, 6.3},
                                 {32, 48, 8.0}, {32, 64, 8.3}, {48, 48, 9.6},   {48, 64, 10.0},  {32, 128, 11.5},
                                 {64, 128, 14}, {64, 256, 20}, {128, 256, 32.0}, {256, 256, 51.0}};
#define PBG_TILE(...) \
  launch_tile<__VA_ARGS__, false>(packed, scale, nullptr, nullptr, n, k, q, q_scale, m, y, nullptr, stream)
#define PBG_STREAM(...) \
  launch_stream<__VA_ARGS__, false>(packed, scale, nullptr, nullptr, n, k, q, q_scale, m, y, nullptr, stream)
  switch (pick_shape(shapes, m, n)) {
    case 0: PBG_STREAM(1, 1, 16); break;
    case 1: PBG_STREAM(1, 2, 8); break;
    case 2: PBG_STREAM(1, 3, 8); break;
    case 3: PBG_STREAM(1, 4, 8); break;
    case 4: PBG_STREAM(2, 2, 8); break;
    case 5: PBG_STREAM(2, 3, 8); break;
    case 6: PBG_STREAM(2, 4, 8); break;
    case 7: PBG_STREAM(3, 3, 8); break;
    case 8: PBG_STREAM(3, 4, 8); break;
    case 9: PBG_TILE(1, 4, 1, 1, 4); break;
    case 10: PBG_TILE(1, 4, 2, 1, 4); break;
    case 11: PBG_TILE(1, 8, 2, 1, 2); break;
    case 12: PBG_TILE(2, 4, 2, 2, 2); break;
    default: PBG_TILE(2, 4, 4, 2, 1); break;
  }
#undef PBG_TILE
#undef PBG_STREAM
  return hipGetLastError();
}

// The same with d_ff columns of gate and of up in a workgroup (8 x 4,096 5.4
// us against 5.7, 32 x 4,096 7.2 / 7.9, 64 x 4,096 9.1 / 9.9, 32 x 12,288 11.8
// / 12.8, 64 x 12,288 16.4 / 21.3, 256 x 12,288 31.6 / 33.3).
hipError_t launch_swiglu_gate_up_i8(const uint32_t* gate, const float* gate_scale, const uint32_t* up,
                                    const float* up_scale, int64_t d_model, int64_t d_ff, const int8_t* q,
                                    const float* q_scale, int64_t m, uint16_t* h, hipStream_t stream) {
  if (launch_gemv_gate_up(gate, gate_scale, up, up_scale, d_model, d_ff, q, q_scale, m, h, stream))
    return hipGetLastError();
  static const Shape shapes[] = {{16, 16, 5.3},  {16, 32, 7.2},  {16, 48, 9.0},   {32, 32, 9.0},   {32, 48, 11.8},
                                 {48, 48, 13.9}, {32, 128, 16.0}, {64, 128, 21.0}, {128, 128, 32.0}, {256, 128, 51.0}};
#define PBG_TILE(...) \
  launch_tile<__VA_ARGS__, true>(gate, gate_scale, up, up_scale, d_ff, d_model, q, q_scale, m, nullptr, h, stream)
#define PBG_STREAM(...) \
  launch_stream<__VA_ARGS__, true>(gate, gate_scale, up, up_scale, d_ff, d_model, q, q_scale, m, nullptr, h, stream)
  switch (pick_shape(shapes, m, d_ff)) {
    case 0: PBG_STREAM(1, 1, 16); break;
    case 1: PBG_STREAM(1, 2, 8); break;
    case 2: PBG_STREAM(1, 3, 8); break;
    case 3: PBG_STREAM(2, 2, 8); break;
    case 4: PBG_STREAM(2, 3, 8); break;
    case 5: PBG_STREAM(3, 3, 8); break;
    case 6: PBG_TILE(1, 4, 1, 2, 4); break;
    case 7: PBG_TILE(1, 4, 2, 2, 2); break;
    case 8: PBG_TILE(2, 4, 2, 2, 2); break;
    default: PBG_TILE(2, 4, 4, 2, 1); break;
  }
#undef PBG_TILE
#undef PBG_STREAM
  return hipGetLastError();
}

}  // namespace pbg
