// tree_attention: attention of a step's rows over a paged cache.
//
// out = sum_t w_t v_t / sum_t w_t, w_t = exp(scale q . k_t), in one pass over the tokens with a
// running maximum: w_t is held relative to the largest score so far, and the sums are scaled
// down whenever it grows.
#include "pbg_device.hpp"
#include "pbg_internal.hpp"
#include "pbg_scan.hpp"

namespace pbg {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kMinPage = 8;  // tokens
constexpr int kParts = 8;  // of the chip; workgroups go to them in turn
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -__builtin_inff();
// Weights are rounded to fp16 for the second product, to half a step each (2^-11), independent of one another and no
// more than the output's own rounding; their sum is that of the unrounded ones (of the rounded ones the wide kernel is
// 13 % slower). They are held relative to 2^-lift of the row's running maximum, so that light ones keep their bits
// beside a token that has nearly all the weight: what the second product loses of one is 2^-(25 + lift) of the largest
// at most, 2^-40 in the kernel for few rows and 2^-33 in the others. (Without a lift 3,000 tokens of 2^-25.2 each
// added to 0 above and not below.)
// The maximum is raised when a score passes it by more than the slack (in powers of two), and with both the weights
// reach 2^15, still inside fp16. Without a slack the largest weights are exactly 2^15, and both roundings together are
// 1.09 times the output's own against 64 bits; with one of 7 or 8 they are 1.38 times. The kernel for few rows, which
// waits for its reads, has none (64 tokens 218 us either way, 7 rows 43.4 -> 44.2); in the others the sums would be
// scaled in most units (chunk 778 -> 825 us, trees 90.8 -> 96.1).
constexpr float kFewLift = 15.0f;
constexpr float kWideLift = 8.0f, kWideSlack = 7.0f;

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) short4_t lds_short4_t;
typedef __attribute__((address_space(4))) int32_t const_int_t;  // read through the scalar cache

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
  int least, most;  // requests with fewer or more rows are not this launch's
  int4* parts;    // [workgroups]: first row, first head, rows and pieces of the work that a workgroup leaves to others
  float* states;  // [workgroups][2] tiles: outputs, then maxima and sums
};

// Request i: its rows and tokens, and its units of work. A unit is one tile of
// query rows over T tokens. Every tile of a tree looks at all tokens; tile n of
// rows that follow one another needs ceil((length + (n + 1) rows) / T) units,
// counted as first + more * ceil(n / 2^every), at most one unit too many.
struct Request {
  int begin, rows, length, tokens, tiles;
  int64_t first, units;  // units of the first tile, of all heads and tiles
  int more, every;
};

// a / b with a short division where both fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Units of the first n tiles of one head.
__device__ __forceinline__ int64_t units_before(const Request& r, int n) {
  if (n == 0) return 0;
  const int64_t k = n - 1, q = k >> r.every, rest = k & ((1 << r.every) - 1);
  return r.first * n + r.more * (((q * (q + 1) / 2) << r.every) + rest * (q + 1));
}

template <int T>
__device__ __forceinline__ Request request_of(const AttnArgs& a, int i) {
  Request r;
  const const_int_t* row_start = (const const_int_t*)a.row_start;
  const const_int_t* lengths = (const const_int_t*)a.lengths;
  const int s = min(max(row_start[i], 0), a.m), e = min(max(row_start[i + 1], 0), a.m);
  const int64_t room = static_cast<int64_t>(a.width) << a.shift;
  r.begin = s;
  r.rows = max(e - s, 0);
  if (r.rows < a.least || r.rows > a.most) r.rows = 0;
  // tokens past the table have no place, so that no sum of these leaves 32 bits
  r.length = static_cast<int>(min(static_cast<int64_t>(max(lengths[i], 0)), room));
  const int64_t tokens = min(static_cast<int64_t>(r.length) + r.rows, room);
  r.tokens = static_cast<int>(tokens);
  r.tiles = (r.rows + a.rows - 1) / a.rows;
  r.more = 0;
  r.every = 0;
  int64_t seen = tokens;
  if (!a.ancestors && r.tiles > 1) {
    seen = min(static_cast<int64_t>(r.length) + a.rows, room);
    // rows is a power of two where there is more than one tile
    if (a.rows >= T) r.more = a.rows / T;
    else r.more = 1, r.every = __builtin_ctz(T / a.rows);
  }
  // a request without a token to look at still has its zeros to write
  r.first = max((seen + T - 1) / T, static_cast<int64_t>(1));
  r.units = units_before(r, r.tiles) * a.kv_heads * a.chunks;
  return r;
}

// Tile n of head group v of a request, from unit `step` of it on.
struct Place {
  int head, tile;
  int64_t step, steps;
};

__device__ __forceinline__ Place place_of(const Request& r, int64_t in) {
  Place p;
  if (r.tiles == 1) {
    p.head = static_cast<int>(quotient(in, r.first));
    p.tile = 0;
    p.step = in - p.head * r.first;
    p.steps = r.first;
    return p;
  }
  const int64_t each = units_before(r, r.tiles);
  p.head = static_cast<int>(quotient(in, each));
  in -= p.head * each;
  int lo = 0, hi = r.tiles - 1;  // the last tile that begins at `in` or before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (units_before(r, mid) <= in) lo = mid;
    else hi = mid - 1;
  }
  p.tile = lo;
  p.step = in - units_before(r, lo);
  p.steps = units_before(r, lo + 1) - units_before(r, lo);
  return p;
}

// The workgroup's share of the line of all requests' units, [begin, end), and
// the request r that begin lies in, with the units before it, for 2^G
// workgroups of W waves. The lengths are on the GPU only: every workgroup adds
// them up, which takes it about 1 us for up to 64 requests (2 us with a scan
// by the whole workgroup).
struct Share {
  int64_t begin, end, share, base;
  int request;
};

__device__ __forceinline__ int from_lane(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

__device__ __forceinline__ int64_t from_lane(int64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(v), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(v >> 32), lane);
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

template <int T, int W, int G>
__device__ __forceinline__ Share share_of(const AttnArgs& a, int64_t me, Request& r) {
  __shared__ int64_t scan[W];
  __shared__ int64_t found_base;
  __shared__ int found_request;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  Share s;
  if (a.requests <= kWave) {
    // every wave by itself, a request a lane
    const Request mine = request_of<T>(a, min(lane, a.requests - 1));
    const int64_t units = lane < a.requests ? mine.units : 0;
    int64_t sum = units;
    for (int d = 1; d < a.requests; d *= 2) {
      const int64_t o = __shfl_up(sum, d);
      if (lane >= d) sum += o;
    }
    const int64_t total = from_lane(sum, a.requests - 1), before = sum - units;
    s.share = (total + ((1 << G) - 1)) >> G;
    s.begin = min(me * s.share, total);
    s.end = min(s.begin + s.share, total);
    const uint64_t where = __ballot(s.begin >= before && s.begin < before + units);
    const int at = where ? __builtin_ctzll(where) : 0;
    s.request = at;
    s.base = from_lane(before, at);
    r.begin = from_lane(mine.begin, at);
    r.rows = from_lane(mine.rows, at);
    r.length = from_lane(mine.length, at);
    r.tokens = from_lane(mine.tokens, at);
    r.tiles = from_lane(mine.tiles, at);
    r.first = from_lane(mine.first, at);
    r.units = from_lane(mine.units, at);
    r.more = from_lane(mine.more, at);
    r.every = from_lane(mine.every, at);
    return s;
  }
  const int per = (a.requests + W * kWave - 1) / (W * kWave);
  const int i0 = min(tid * per, a.requests), i1 = min(i0 + per, a.requests);
  int64_t mine = 0;
  for (int i = i0; i < i1; ++i) mine += request_of<T>(a, i).units;
  int64_t sum = mine;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int64_t o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == kWave - 1) scan[wave] = sum;
  if (tid == 0) found_request = 0, found_base = 0;
  __syncthreads();
  int64_t before = sum - mine, total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < wave) before += scan[w];
    total += scan[w];
  }
  s.share = (total + ((1 << G) - 1)) >> G;
  s.begin = min(me * s.share, total);
  s.end = min(s.begin + s.share, total);
  if (s.begin >= before && s.begin < before + mine) {
    int i = i0;
    for (; i < i1; ++i) {
      const int64_t u = request_of<T>(a, i).units;
      if (s.begin < before + u) break;
      before += u;
    }
    found_request = i;
    found_base = before;
  }
  __syncthreads();
  s.request = __builtin_amdgcn_readfirstlane(found_request);
  s.base = from_lane(found_base, 0);
  r = request_of<T>(a, s.request);
  return s;
}

// Places of a token's 16-byte pieces in LDS, such that 16 lanes that read the same piece of 16 tokens, and 32 lanes
// that read 64 bytes of each of four tokens across, touch every bank once.
template <int D>
__device__ __forceinline__ int key_piece(int token, int piece) {
  if constexpr (D == 64) return piece ^ ((token >> 1) & 7);
  else return piece ^ (token & 15);
}

template <int D>
__device__ __forceinline__ int value_piece(int token, int piece) {
  if constexpr (D == 64) return piece ^ (((token >> 1) & 1) << 2);
  else return piece ^ ((token & 3) << 2);
}

// The same for 32 bytes of each of eight tokens.
template <int D>
__device__ __forceinline__ int narrow_piece(int token, int piece) {
  if constexpr (D == 64) return piece ^ (((token >> 1) & 3) << 1);
  else return piece ^ ((token & 7) << 1);
}

// Scores, in powers of two, from which on their rounding matters. The maximum is a rounded product; a score that is
// held against it by a product and difference in one has no such rounding, and the difference, up to 2^-25 of the
// score, is a power of two of its own (at a score of 2^30 the largest weight was anything from 2^-32 to 2^32). Rows
// whose maximum is that far from 0 have every score rounded first, and no lift, behind a branch that lies out of the
// way: with the lift it takes 4,096 rows over 8,192 tokens from 747 to 752 us (758 where it lies in the way), 16 trees
// from 88 to 89. The kernel for few rows always rounds, which takes it no longer.
constexpr float kFar = 0x1p20f;

__device__ __forceinline__ float rounded_product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

__device__ __forceinline__ bool is_far(float top) { return fabsf(top) > kFar && top != kNone; }

// Score x of a row whose maximum is far, less that maximum and before the scale; x itself in other rows, whose bits are
// the same beside any others. (A scale that lets scores get that far has a reciprocal.)
__device__ __forceinline__ float over_far(float x, float scale, float top) {
  return is_far(top) ? (rounded_product(x, scale) - top) * __builtin_amdgcn_rcpf(scale) : x;
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

// x where bit n of mask is set, else -infinity.
__device__ __forceinline__ float seen_or_none(float x, uint32_t mask, int n) {
  const uint32_t keep = static_cast<uint32_t>(static_cast<int32_t>(mask << (31 - n)) >> 31);
  return as_f32((as_u32(x) & keep) | (0xFF800000u & ~keep));
}

// 16 bytes at a wave's address and a lane's offset.
__device__ __forceinline__ uint4 load16(const uint16_t* p, uint32_t bytes) {
  return *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) + bytes);
}

// Scale of a state with maximum m next to one with maximum `top`.
__device__ __forceinline__ float weight_of(float m, float top) { return m == kNone ? 0.0f : exp2_of(m - top); }

// Which of the 32 or 64 tokens from t0 on a query row sees, one bit each: all up to the row itself (`upto`, the last of
// them), or with a tree those before the step and its ancestors.
__device__ __forceinline__ uint64_t ones_below(int n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }

__device__ __forceinline__ uint64_t seen_from(int t0, int length, int upto, uint64_t tree) {
  const int n = t0 - length;  // tokens of the step before t0
  const uint64_t branch = n >= 64 ? 0 : n >= 0 ? tree >> n : n > -64 ? tree << -n : 0;
  return ones_below(upto - t0 + 1) | branch;
}

// o += y v for those of the four values at column c that are an infinity or NaN.
__device__ __forceinline__ void add_wild(f32x4_t& o, const uint16_t* v, int c, int d, float y) {
  __builtin_amdgcn_sched_barrier(0);  // one piece at a time: this path is rare and must not cost registers
  if (c >= d) return;
  const uint2 two = *reinterpret_cast<const uint2*>(v + c);
  const uint32_t bits[4] = {two.x & 0xFFFFu, two.x >> 16, two.y & 0xFFFFu, two.y >> 16};
#pragma unroll
  for (int z = 0; z < 4; ++z) {
    const float add = y * static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits[z])));
    o[z] = (bits[z] & 0x7C00u) == 0x7C00u ? o[z] + add : o[z];
  }
}

// ---- few query rows

constexpr int kStep = 32;                // tokens a wave takes at once
constexpr int kTokens = kWaves * kStep;  // tokens of a unit of work

// Workgroups that a compute unit holds, and the launch's (as many as the chip holds), a power of two.
constexpr int few_blocks(int d, int qb) { return d == 256 || (d == 128 && qb > 1) ? 1 : 2; }
constexpr int few_bits(int d, int qb) { return few_blocks(d, qb) == 1 ? 8 : 9; }

// D: head_dim rounded up to 64, 128 or 256. QB: blocks of 16 query rows (a
// query row is one head of one row of the step; the heads of a key
// head share its keys).
//
// The units of work of all requests stand in one line, which the workgroups
// share evenly, so that requests of any lengths fill the chip; a tile that ends
// up with several workgroups is joined by a second kernel.
//
// A wave takes 32 tokens of a unit for all query rows, on its own: S^T = K Q^T,
// so that a lane holds one query row's scores (its maximum and sum need two
// lane swaps), and the weights are then the second operand of O^T = V^T W^T as
// they are; V^T comes out of LDS with transposing reads. Keys and values are
// loaded 1 KiB of consecutive bytes at a time and pass through LDS that only
// the wave uses; the loads of the next unit are issued before the products of
// this one.
//
// Bound by the reads of the cache: 64 requests of 820 to 8,192 tokens, one row
// each (32 heads over 8 of 128, 1.18 GB), take 217 us, 5.4 TB/s; the loads
// alone take as long, a pure read of as many consecutive bytes 174. 7 rows over
// 40,953 tokens (168 MB) take 38 us and 5 for the join, of which the reads are
// 28. One token over 1,000 takes 8 us and 3, four loads that wait for one
// another.
template <int D, int QB>
__global__ __launch_bounds__(kThreads, few_blocks(D, QB)) void attention_kernel(AttnArgs a) {
  constexpr int J = D / 32;       // products of 32 columns in a score
  constexpr int DB = D / 16;      // blocks of 16 columns of the output
  constexpr int kRow = D + 4;     // floats of a row where waves meet
  constexpr int kChunks = D / 8;             // 16-byte pieces of a token's keys
  constexpr int kGroup = kWave / kChunks;    // tokens that a wave loads at once
  constexpr int kLoads = kStep / kGroup, kPages = kStep / kMinPage;
  constexpr int kStage = kStep * D * 2;
  constexpr int kMeet = 16 * kRow * 4;
  constexpr int kSlice = 2 * kStage;
  static_assert(kSlice >= kMeet && kMinPage % kGroup == 0, "room for a state, whole pages");
  __shared__ __attribute__((aligned(16))) char lds[kWaves * kSlice];
  __shared__ __attribute__((aligned(16))) _Float16 weights[kWaves][QB][kWave][8];  // for the rare path only
  __shared__ float meet_max[kWaves][QB * 16], meet_sum[kWaves][QB * 16];

  const int tid = threadIdx.x, lane = tid & (kWave - 1), li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int64_t me = blockIdx.x;
  Request r;
  const Share line = share_of<kTokens, kWaves, few_bits(D, QB)>(a, me, r);
  if (tid == 0) a.parts[me] = make_int4(0, 0, 0, 0);
  if (line.begin >= line.end) return;
  int request = line.request;
  int64_t base = line.base;

  for (int64_t at = line.begin; at < line.end;) {
    while (at >= base + r.units) {
      base += r.units;
      r = request_of<kTokens>(a, ++request);
    }
    const Place here = place_of(r, at - base);
    const int step0 = static_cast<int>(here.step);
    const int step1 = static_cast<int>(min(here.step + (line.end - at), here.steps));
    const int kvh = here.head / a.chunks, chunk = here.head - kvh * a.chunks;
    const int ratio = a.heads / a.kv_heads;
    const int head0 = kvh * ratio + chunk * a.group;
    const int tile_heads = min(a.group, ratio - chunk * a.group);
    const int row0 = r.begin + here.tile * a.rows;
    const int tile_rows = min(a.rows, r.rows - here.tile * a.rows);

    const const_int_t* table = (const const_int_t*)(a.table + static_cast<int64_t>(request) * a.width);
    const int64_t page_elements = (static_cast<int64_t>(a.kv_heads) << a.shift) * a.d;
    const int64_t head_at = (static_cast<int64_t>(kvh) << a.shift) * a.d;
    const int page_mask = (1 << a.shift) - 1;
    char* key_slice = lds + wave * kSlice;
    char* value_slice = key_slice + kStage;
    // Eight tokens that follow one another are of one page, so that page numbers and addresses are the wave's, not a
    // lane's. Columns past head_dim are loaded as column 0 and made zero in the keys; tokens without a page are loaded
    // from the first page and made zero.
    const int load_t = lane / kChunks, load_c = lane % kChunks;
    const uint32_t lane_at = 2 * (load_t * a.d + (8 * load_c < a.d ? 8 * load_c : 0));  // in bytes
    int page[kPages], page_next[kPages];
    uint4 kr[kLoads], vr[kLoads];
    auto fetch_pages = [&](int s) {
#pragma unroll
      for (int g = 0; g < kPages; ++g) {
        const int t = s * kTokens + wave * kStep + g * kMinPage;
        const int found = table[static_cast<uint32_t>(min(t >> a.shift, a.width - 1))];
        page_next[g] = t < r.tokens && static_cast<uint32_t>(found) < static_cast<uint32_t>(a.pages) ? found : -1;
      }
    };
    auto fetch = [&](int s) {
#pragma unroll
      for (int g = 0; g < kPages; ++g) {
        page[g] = page_next[g];
        const int t = s * kTokens + wave * kStep + g * kMinPage;
        const int64_t from = max(page[g], 0) * page_elements + head_at + (t & page_mask) * a.d;
#pragma unroll
        for (int i = 0; i < kLoads / kPages; ++i) {
          const int64_t at = from + i * kGroup * a.d;
          kr[g * (kLoads / kPages) + i] = load16(a.k + at, lane_at);
          vr[g * (kLoads / kPages) + i] = load16(a.v + at, lane_at);
        }
      }
    };
    fetch_pages(step0);

    // ---- queries: block b's row li is query row 16 b + li: row / group, head % group
    mfma_half8_t q[QB][J];
    uint64_t tree[QB];
    int upto[QB];  // last token seen without a tree
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      const int n = 16 * b + li, rr = n / a.group, hh = n - rr * a.group;
      const bool fine = rr < tile_rows && hh < tile_heads;
      const int row = row0 + rr;
      tree[b] = fine && a.ancestors ? a.ancestors[row] : 0;
      upto[b] = fine && !a.ancestors ? r.length + (row - r.begin) : r.length - 1;
      const uint16_t* p = a.q + (static_cast<int64_t>(row) * a.heads + head0 + hh) * a.d;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = 8 * (4 * j + lg);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (fine && c < a.d) w = *reinterpret_cast<const uint4*>(p + c);
        q[b][j] = __builtin_bit_cast(mfma_half8_t, w);
      }
    }
    fetch(step0);
    fetch_pages(step0 + 1);
    float top[QB], part[QB];
    f32x4_t o[QB][DB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      top[b] = kNone;
      part[b] = 0.0f;
#pragma unroll
      for (int e = 0; e < DB; ++e) o[b][e] = f32x4_t{};
    }

    for (int s = step0; s < step1; ++s) {
      const int t0 = s * kTokens + wave * kStep;
      if (t0 >= r.tokens) break;
      uint32_t held = 0;  // tokens that have a place, one bit each
#pragma unroll
      for (int g = 0; g < kPages; ++g) held |= page[g] >= 0 ? 0xFFu << (8 * g) : 0u;
      // whether any row may not see a token of these, and values that must reach only rows that see them
      const bool masked = t0 + kStep > r.length || held != 0xFFFFFFFFu;
      uint32_t wild = 0;
      if (masked) {
        held &= static_cast<uint32_t>(ones_below(r.tokens - t0));
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
          __builtin_amdgcn_sched_barrier(0);  // one after the other, for the registers' sake
          uint4& w = vr[n];
          if (page[n / (kLoads / kPages)] < 0) kr[n] = w = make_uint4(0, 0, 0, 0);
          const uint4 x = make_uint4(not_finite(w.x), not_finite(w.y), not_finite(w.z), not_finite(w.w));
          const uint64_t lanes = __ballot((x.x | x.y | x.z | x.w) != 0);
          w = make_uint4(w.x & ~x.x, w.y & ~x.y, w.z & ~x.z, w.w & ~x.w);
#pragma unroll
          for (int t = 0; t < kGroup; ++t)
            if (lanes >> (t * kChunks) & ones_below(kChunks)) wild |= 1u << (n * kGroup + t);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int n = 0; n < kLoads; ++n) {
        const int t = n * kGroup + load_t;
        if (a.d != D && 8 * load_c >= a.d) kr[n] = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(key_slice + t * (D * 2) + key_piece<D>(t, load_c) * 16) = kr[n];
        *reinterpret_cast<uint4*>(value_slice + t * (D * 2) + narrow_piece<D>(t, load_c) * 16) = vr[n];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // the registers are free from here on
      if (s + 1 < step1) {
        fetch(s + 1);
        fetch_pages(s + 2);
      }

      mfma_float4_t x[QB][2];
#pragma unroll
      for (int b = 0; b < QB; ++b) x[b][0] = x[b][1] = mfma_float4_t{};
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = 16 * h + li;
          const char* piece = key_slice + t * (D * 2) + key_piece<D>(t, 4 * j + lg) * 16;
          const auto k = *reinterpret_cast<const mfma_half8_t*>(piece);
#pragma unroll
          for (int b = 0; b < QB; ++b) x[b][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[b][j], x[b][h], 0, 0, 0);
        }
      mfma_half8_t w[QB];
      uint32_t seen[QB];
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        if (masked) {
          seen[b] = static_cast<uint32_t>(seen_from(t0, r.length, upto[b], tree[b])) & held;
          const uint32_t mine = seen[b] >> (4 * lg);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[b][h][e] = seen_or_none(x[b][h][e], mine, 16 * h + e);
        }
        float high = kNone;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[b][h][e] = rounded_product(x[b][h][e], a.scale);
            high = fmaxf(high, x[b][h][e]);
          }
        high = groups_max(high);
        if (!is_far(high)) high -= kFewLift;
        if (__any(high > top[b])) {
          const float now = fmaxf(top[b], high), keep = weight_of(top[b], now);
          top[b] = now;
          part[b] *= keep;
#pragma unroll
          for (int e = 0; e < DB; ++e) o[b][e] *= keep;
        }
        const float less = top[b] == kNone ? 0.0f : top[b];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = exp2_of(x[b][h][e] - less);
            part[b] += p;
            w[b][4 * h + e] = static_cast<_Float16>(p);
          }
      }
      // ---- O^T += V^T W^T
#pragma unroll
      for (int e = 0; e < DB; ++e) {
        mfma_half8_t v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = 16 * h + 4 * lg + li / 4, c = 2 * e + (li & 3) / 2;
          const auto v4 = __builtin_bit_cast(half4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_short4_t*)(value_slice + t * (D * 2) + narrow_piece<D>(t, c) * 16 + (li & 1) * 8)));
#pragma unroll
          for (int y = 0; y < 4; ++y) v[4 * h + y] = v4[y];
        }
#pragma unroll
        for (int b = 0; b < QB; ++b) o[b][e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w[b], o[b][e], 0, 0, 0);
      }
      // infinities and NaN among values that some rows may not see: added for the rows that do
      if (wild) {
#pragma unroll
        for (int b = 0; b < QB; ++b) *reinterpret_cast<mfma_half8_t*>(weights[wave][b][lane]) = w[b];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      while (wild) {
        const int n = __builtin_ctz(wild);
        wild &= wild - 1;
        const int t = t0 + n;
        const int64_t p = table[static_cast<uint32_t>(t >> a.shift)] * page_elements + head_at + (t & page_mask) * a.d;
#pragma unroll
        for (int b = 0; b < QB; ++b) {
          // element (n / 16) * 4 + n % 4 of the lane that holds the token
          const float y = static_cast<float>(
              weights[wave][b][li + 16 * ((n & 15) >> 2)][(n >> 4) * 4 + (n & 3)]);
          if (seen[b] >> n & 1) {
#pragma unroll
            for (int e = 0; e < DB; ++e) add_wild(o[b][e], a.v + p, 16 * e + 4 * lg, a.d, y);
          }
        }
      }
    }

    // ---- the four waves' states meet
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      const float sum = groups_sum(part[b]);
      if (lg == 0) {
        meet_max[wave][16 * b + li] = top[b];
        meet_sum[wave][16 * b + li] = sum;
      }
    }
    __syncthreads();
    const bool starts = here.step == 0, ends = step1 == here.steps;
    float* state = a.states + (me * 2 + (starts ? 1 : 0)) * (QB * 16) * (D + 2);
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      const int n = 16 * b + li;
      float high = meet_max[0][n];
#pragma unroll
      for (int y = 1; y < kWaves; ++y) high = fmaxf(high, meet_max[y][n]);
      const float keep = weight_of(top[b], high);
      float* to = reinterpret_cast<float*>(key_slice) + li * kRow;
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
        float sum = 0.0f;
        f32x4_t acc = {};
#pragma unroll
        for (int y = 0; y < kWaves; ++y) {
          sum += meet_sum[y][qr] * weight_of(meet_max[y][qr], most);
          acc += *reinterpret_cast<const f32x4_t*>(lds + y * kSlice + (nn * kRow + c) * 4);
        }
        if (starts && ends) {
          if (c < a.d) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            if (sum == 0.0f) acc = f32x4_t{};
            uint16_t* to_out = a.out + (static_cast<int64_t>(row0 + rr) * a.heads + head0 + hh) * a.d + c;
            *reinterpret_cast<half4_t*>(to_out) = __builtin_convertvector(acc * inv, half4_t);
          }
        } else {
          *reinterpret_cast<f32x4_t*>(state + qr * D + c) = acc;
          if (c == 0) {
            state[QB * 16 * D + 2 * qr] = most;
            state[QB * 16 * D + 2 * qr + 1] = sum;
          }
        }
      }
      __syncthreads();
    }
    // the pieces after this one: whole shares of the workgroups that follow
    if (starts && !ends && tid == 0)
      a.parts[me] = make_int4(row0, head0, tile_heads << 16 | tile_rows,
                              static_cast<int>(quotient(at + here.steps - 1, line.share) - me + 1));
    at += step1 - step0;
  }
}

// ---- many query rows

// What scores are held against. Half of the lift is in the maximum already: a whole one there or here takes a constant
// more, and 1.5 % of the time. Finite where the row has seen nothing, so that its weights are 0.
__device__ __forceinline__ float lifted(float top) { return fmaxf(top, -__FLT_MAX__) - kWideLift / 2; }

constexpr int kWide = 64;  // tokens of a unit of work
constexpr int kWideBits = 8;  // one workgroup on each compute unit

// NB: blocks of 32 query rows a wave; the W waves have rows of their own and
// share the tokens, 64 at a time, through LDS, with the next 64 on their way in
// registers. The products are turned as in the kernel for few rows
// (S^T = K Q^T, O^T = V^T W^T), on 32 x 32 tiles: a lane holds one query row's
// scores, half of its tokens.
//
// A unit has two turns, with a barrier behind each: the matrix products (O^T of
// the unit before, S^T of this one), then everything else (weights, loads). The
// two waves of a SIMD are half a unit apart, so that one's products run beside
// the other's exponentials. The waves that come second write their part of a
// unit's keys and values one turn early; K(s) is read in turns 2 s and 2 s + 1,
// V(s) in 2 s + 2 and 2 s + 3, so keys need two buffers and values three.
//
// 4,096 rows over 8,192 tokens and themselves (32 heads over 8 of 128) take 752
// us, 914 TFLOP/s: a unit takes 2.3 us, of which its products are 0.9, its
// exponentials and the rest of the vector instructions 1.0 and its LDS reads
// 0.9, each on units of their own. Without the loads it would be 670, without
// the exponentials 690.
template <int D>
__global__ __launch_bounds__(512) void attention_wide_kernel(AttnArgs a) {
  constexpr int W = 8, NB = 1;         // two blocks a wave do not fit the registers
  constexpr int KS = D / 16;           // products of 16 columns in a score
  constexpr int DB = D / 32;           // blocks of 32 columns of the output
  constexpr int kChunks = D / 8;       // 16-byte pieces of a token's keys
  constexpr int kGroup = kWave / kChunks;  // tokens that a wave loads at once
  constexpr int kMine = kWide / W;         // tokens of a unit that it loads
  constexpr int kPasses = kMine / kGroup;
  constexpr int kPages = kMine / kMinPage;
  static_assert(kPages * kMinPage == kMine && kMinPage % kGroup == 0, "whole pages");
  constexpr int kAhead = 4;            // pieces of keys or values read before they are needed
  constexpr int kRows = W * NB * 32;
  constexpr int kTile = kWide * D * 2;
  constexpr int kValueTiles = 3;
  __shared__ __attribute__((aligned(16))) char keys[2][kTile];
  __shared__ __attribute__((aligned(16))) char values[kValueTiles][kTile];
  __shared__ __attribute__((aligned(16))) _Float16 weights[W][NB][4][kWave][8];  // for the rare path only
  __shared__ uint32_t flags[4][4];  // tokens without a page, and with values that are infinite or NaN

  const int tid = threadIdx.x, lane = tid & (kWave - 1), li = lane & 31, lh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  // neighbours in the line, which read the same keys and values, on one of the chip's eight parts, each with its own
  // cache
  const int64_t me = (blockIdx.x % kParts) * (gridDim.x / kParts) + blockIdx.x / kParts;
  Request r;
  const Share line = share_of<kWide, W, kWideBits>(a, me, r);
  if (tid == 0) a.parts[me] = make_int4(0, 0, 0, 0);
  if (line.begin >= line.end) return;
  int request = line.request;
  int64_t base = line.base;

  // The end of a tile that another workgroup began comes last: all then walk the tokens from the first on at about the
  // same time, and find the keys that they share in the cache (771 -> 750 us of the above when it was done).
  const Place begun = place_of(r, line.begin - base);
  const int64_t begun_end = begun.step == 0 ? line.begin : min(line.begin + begun.steps - begun.step, line.end);
  int64_t stop = line.end;
  bool done = begun_end == line.begin;  // with that end
  for (int64_t at = begun_end;;) {
    if (at == stop) {
      if (done) break;
      done = true;
      at = line.begin;
      stop = begun_end;
      request = line.request;
      base = line.base;
      r = request_of<kWide>(a, request);
    }
    while (at >= base + r.units) {
      base += r.units;
      r = request_of<kWide>(a, ++request);
    }
    const Place here = place_of(r, at - base);
    const int step0 = static_cast<int>(here.step);
    const int step1 = static_cast<int>(min(here.step + (stop - at), here.steps));
    const int kvh = here.head / a.chunks, chunk = here.head - kvh * a.chunks;
    const int ratio = a.heads / a.kv_heads;
    const int head0 = kvh * ratio + chunk * a.group;
    const int tile_heads = min(a.group, ratio - chunk * a.group);
    const int row0 = r.begin + here.tile * a.rows;
    const int tile_rows = min(a.rows, r.rows - here.tile * a.rows);
    // the first token that some row of the tile does not see, and the end of those that any row sees
    const int edge = a.ancestors ? r.length : r.length + here.tile * a.rows + 1;
    const int ending = a.ancestors ? r.tokens : min(r.tokens, r.length + here.tile * a.rows + tile_rows);
    const int last = min(step1, (ending + kWide - 1) / kWide);

    const const_int_t* table = (const const_int_t*)(a.table + static_cast<int64_t>(request) * a.width);
    const int64_t page_elements = (static_cast<int64_t>(a.kv_heads) << a.shift) * a.d;
    const int64_t head_at = (static_cast<int64_t>(kvh) << a.shift) * a.d;
    const int page_mask = (1 << a.shift) - 1;
    // A wave loads kMine tokens of a unit that follow one another, eight of them always of one page, so that page
    // numbers and addresses are the wave's, not a lane's. Columns past head_dim are loaded as column 0 and
    // made zero in the keys; tokens without a page are loaded from the first page and made zero.
    const int load_t = lane / kChunks, load_c = lane % kChunks;
    const uint32_t lane_at = 2 * (load_t * a.d + (8 * load_c < a.d ? 8 * load_c : 0));  // in bytes
    int page[kPages], page_next[kPages];
    uint4 kr[kPasses], vr[kPasses];
    auto fetch_pages = [&](int s) {
#pragma unroll
      for (int g = 0; g < kPages; ++g) {
        const int t = s * kWide + wave * kMine + g * kMinPage;
        const int found = table[static_cast<uint32_t>(min(t >> a.shift, a.width - 1))];
        page_next[g] = t < r.tokens && static_cast<uint32_t>(found) < static_cast<uint32_t>(a.pages) ? found : -1;
      }
    };
    auto fetch = [&](int s) {
#pragma unroll
      for (int g = 0; g < kPages; ++g) {
        page[g] = page_next[g];
        const int t = s * kWide + wave * kMine + g * kMinPage;
        const int64_t from = max(page[g], 0) * page_elements + head_at + (t & page_mask) * a.d;
#pragma unroll
        for (int i = 0; i < kPasses / kPages; ++i) {
          const int64_t at = from + i * kGroup * a.d;
          kr[g * (kPasses / kPages) + i] = load16(a.k + at, lane_at);
          vr[g * (kPasses / kPages) + i] = load16(a.v + at, lane_at);
        }
      }
    };
    // the loaded tokens of unit s to its buffers
    auto store = [&](int s, char* key_to, char* value_to) {
      const bool edges = (s + 1) * kWide > edge;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int t = wave * kMine + i * kGroup + load_t;
        uint32_t* flag = &flags[s & 3][t / 32];
        if (page[i / (kPasses / kPages)] < 0) {
          __builtin_amdgcn_sched_barrier(0);  // a branch
          kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
          if (load_c == 0) atomicOr(flag, 1u << (t % 32));
        }
        if (a.d != D && 8 * load_c >= a.d) kr[i] = make_uint4(0, 0, 0, 0);
        if (edges) {
          __builtin_amdgcn_sched_barrier(0);
          uint4& w = vr[i];
          const uint4 n = make_uint4(not_finite(w.x), not_finite(w.y), not_finite(w.z), not_finite(w.w));
          if (n.x | n.y | n.z | n.w) atomicOr(flag + 2, 1u << (t % 32));
          w = make_uint4(w.x & ~n.x, w.y & ~n.y, w.z & ~n.z, w.w & ~n.w);
        }
        *reinterpret_cast<uint4*>(key_to + t * (D * 2) + key_piece<D>(t, load_c) * 16) = kr[i];
        *reinterpret_cast<uint4*>(value_to + t * (D * 2) + value_piece<D>(t, load_c) * 16) = vr[i];
      }
    };

    // ---- queries: block b's row li is query row 32 (wave NB + b) + li: row / group, head % group
    mfma_half8_t q[NB][KS];
    uint64_t tree[NB];
    int upto[NB];
    const int wave_n = wave * NB * 32;
    const bool busy = wave_n / a.group < tile_rows;
    // the last token that any row of the wave sees
    const int wave_rows = (wave_n + NB * 32 - 1) / a.group + 1;
    const int wave_end = a.ancestors ? ending : min(ending, r.length + here.tile * a.rows + wave_rows);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int n = wave_n + 32 * b + li, rr = n / a.group, hh = n - rr * a.group;
      const bool fine = rr < tile_rows && hh < tile_heads;
      const int row = row0 + rr;
      tree[b] = fine && a.ancestors ? a.ancestors[row] : 0;
      upto[b] = fine && !a.ancestors ? r.length + (row - r.begin) : r.length - 1;
      const uint16_t* p = a.q + (static_cast<int64_t>(row) * a.heads + head0 + hh) * a.d;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const int c = 8 * (2 * j + lh);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (fine && c < a.d) w = *reinterpret_cast<const uint4*>(p + c);
        q[b][j] = __builtin_bit_cast(mfma_half8_t, w);
      }
    }
    float top[NB], part[NB];
    f32x16_t o[NB][DB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      top[b] = kNone;
      part[b] = 0.0f;
#pragma unroll
      for (int e = 0; e < DB; ++e) o[b][e] = f32x16_t{};
    }

    const int turn = wave / (W / 2);  // a SIMD has a wave of either
    __syncthreads();  // the last tile's buffers and flags
    if (tid < 16) flags[tid / 4][tid % 4] = 0;
    __syncthreads();
    fetch_pages(step0);
#pragma unroll
    for (int n = 0; n < 2; ++n)
      if (n <= turn && step0 + n < last) {
        fetch(step0 + n);
        fetch_pages(step0 + n + 1);
        store(step0 + n, keys[(step0 + n) & 1], values[n]);
      }
    if (step0 + 1 + turn < last) {
      fetch(step0 + 1 + turn);
      fetch_pages(step0 + 2 + turn);
    }
    __syncthreads();
    if (turn) __syncthreads();

    mfma_half8_t w[NB][4];
    f32x16_t x[NB][2];
    uint64_t seen[NB];
    bool masked = false;
    bool far[NB];  // the maximum of some row of the wave is far from 0
#pragma unroll
    for (int b = 0; b < NB; ++b) seen[b] = 0, far[b] = false;
    // values of units s - 1 and of the one that is stored next
    int value_read = (kValueTiles - 1) * kTile, value_store = (1 + turn) * kTile;
    for (int s = step0; s <= last; ++s) {
      const uint64_t gaps = flags[s & 3][0] | static_cast<uint64_t>(flags[s & 3][1]) << 32;
      // ---- the matrix products' turn: O^T += V^T W^T of unit s - 1, S^T = K Q^T of unit s
      const bool scores = busy && s < last && s * kWide < wave_end;
      if (busy && s > step0 && (s - 1) * kWide < wave_end) {
        const char* vs = values[0] + value_read;
        auto value = [&](int n) {  // columns 32 (n % DB) on of tokens 16 (n / DB) on
          mfma_half8_t v;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int t = 16 * (n / DB) + 8 * y + 4 * lh + (lane & 15) / 4;
            const int c = 4 * (n % DB) + 2 * ((lane >> 4) & 1) + (lane & 3) / 2;
            const auto v4 = __builtin_bit_cast(half4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_short4_t*)(vs + t * (D * 2) + value_piece<D>(t, c) * 16 + (lane & 1) * 8)));
#pragma unroll
            for (int z = 0; z < 4; ++z) v[4 * y + z] = v4[z];
          }
          return v;
        };
        mfma_half8_t vf[kAhead];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kAhead; ++n) vf[n] = value(n);
#pragma unroll
        for (int n = 0; n < 4 * DB; ++n) {
          const mfma_half8_t v = vf[n % kAhead];
#pragma unroll
          for (int b = 0; b < NB; ++b)
            o[b][n % DB] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, w[b][n / DB], o[b][n % DB], 0, 0, 0);
          if (n + kAhead < 4 * DB) vf[n % kAhead] = value(n + kAhead);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * kAhead, 0);  // LDS reads
#pragma unroll
        for (int n = 0; n < 4 * DB - kAhead; ++n) {
          __builtin_amdgcn_sched_group_barrier(0x008, NB, 0);  // matrix instructions
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, NB * kAhead, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (masked) {
          // infinities and NaN among values that some rows may not see: added for the rows that do
          const int t0 = (s - 1) * kWide;
          uint64_t wild = flags[(s - 1) & 3][2] | static_cast<uint64_t>(flags[(s - 1) & 3][3]) << 32;
          if (wild) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int j = 0; j < 4; ++j) *reinterpret_cast<mfma_half8_t*>(weights[wave][b][j][lane]) = w[b][j];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          }
          while (wild) {
            const int n = __builtin_ctzll(wild);
            wild &= wild - 1;
            const int t = t0 + n, number = table[static_cast<uint32_t>(t >> a.shift)];
            const int64_t p = number * page_elements + head_at + (t & page_mask) * a.d;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              // element (n / 8) * 4 + n % 4 of the lane that holds the token
              const _Float16* mine = weights[wave][b][n >> 4][li + 32 * ((n >> 2) & 1)];
              const float y = static_cast<float>(mine[((n >> 3) & 1) * 4 + (n & 3)]);
              if (seen[b] >> n & 1) {
#pragma unroll
                for (int e = 0; e < DB; ++e)
#pragma unroll
                  for (int z = 0; z < 4; ++z) {
                    f32x4_t part_o = {o[b][e][4 * z], o[b][e][4 * z + 1], o[b][e][4 * z + 2], o[b][e][4 * z + 3]};
                    add_wild(part_o, a.v + p, 32 * e + 8 * z + 4 * lh, a.d, y);
#pragma unroll
                    for (int u = 0; u < 4; ++u) o[b][e][4 * z + u] = part_o[u];
                  }
              }
            }
          }
        }
      }
      if (scores) {
        const char* ks = keys[s & 1];
        auto key = [&](int n) {
          const int t = 32 * (n & 1) + li;
          return *reinterpret_cast<const mfma_half8_t*>(ks + t * (D * 2) + key_piece<D>(t, (n & ~1) + lh) * 16);
        };
        mfma_half8_t kf[kAhead];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kAhead; ++n) kf[n] = key(n);
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n) {
          const mfma_half8_t k = kf[n % kAhead];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const f32x16_t before = n < 2 ? f32x16_t{} : x[b][n & 1];
            x[b][n & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[b][n / 2], before, 0, 0, 0);
          }
          if (n + kAhead < 2 * KS) kf[n % kAhead] = key(n + kAhead);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int n = 0; n < 2 * KS - kAhead; ++n) {
          __builtin_amdgcn_sched_group_barrier(0x008, NB, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, NB * kAhead, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();

      // ---- the other instructions' turn: loads, and the weights of unit s
      const int next = s + 1 + turn;
      if (next < last) store(next, keys[next & 1], values[0] + value_store);
      value_store = value_store == (kValueTiles - 1) * kTile ? 0 : value_store + kTile;
      value_read = value_read == (kValueTiles - 1) * kTile ? 0 : value_read + kTile;
      if (next + 1 < last) {
        fetch(next + 1);
        fetch_pages(next + 2);
      }
      // last read two units before it, written from the next turn on
      if (tid < 4) flags[(s + 2) & 3][tid] = 0;
      if (scores) {
        const int t0 = s * kWide;
        masked = t0 + kWide > edge || gaps != 0;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (masked) {
            __builtin_amdgcn_sched_barrier(0);  // a branch, not a selection in every unit
            seen[b] = seen_from(t0, r.length, upto[b], tree[b]) & ~gaps & ones_below(r.tokens - t0);
            const uint64_t mine = seen[b] >> (4 * lh);
            const uint32_t half[2] = {static_cast<uint32_t>(mine), static_cast<uint32_t>(mine >> 32)};
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                x[b][h][e] = seen_or_none(x[b][h][e], half[h], 8 * (e / 4) + e % 4);
          }
          float high = kNone;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 16; ++e) high = fmaxf(high, x[b][h][e]);
          auto both = __builtin_amdgcn_permlane32_swap(as_u32(high), as_u32(high), false, false);
          const float most = fmaxf(as_f32(both[0]), as_f32(both[1]));
          high = __builtin_fmaf(most, a.scale, -kWideLift / 2);
          if (__any(high > top[b] + kWideSlack)) {
            // of the rows that pass it: what other rows see does not change a row's bits
            const bool passes = high > top[b] + kWideSlack;
            if (is_far(high)) high = rounded_product(most, a.scale);
            const float now = passes ? high : top[b], keep = weight_of(top[b], now);
            top[b] = now;
            part[b] *= keep;
#pragma unroll
            for (int e = 0; e < DB; ++e) o[b][e] *= keep;
            far[b] = __any(is_far(now));
          }
          float less = lifted(top[b]);
          if (__builtin_expect(far[b], 0)) {
            __builtin_amdgcn_sched_barrier(0);  // a branch
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 16; ++e) x[b][h][e] = over_far(x[b][h][e], a.scale, top[b]);
            less = is_far(top[b]) ? 0.0f : less;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              p[e] = exp2_of(__builtin_fmaf(x[b][j / 2][8 * (j & 1) + e], a.scale, -less));
              w[b][j][e] = static_cast<_Float16>(p[e]);
            }
            part[b] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
          }
        }
      }
      __syncthreads();
    }
    if (!turn) __syncthreads();

    const bool starts = here.step == 0, ends = step1 == here.steps;
    float* state = a.states + (me * 2 + (starts ? 1 : 0)) * kRows * (D + 2);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int n = wave_n + 32 * b + li, rr = n / a.group, hh = n - rr * a.group;
      auto both = __builtin_amdgcn_permlane32_swap(as_u32(part[b]), as_u32(part[b]), false, false);
      const float sum = as_f32(both[0]) + as_f32(both[1]);
      if (rr >= tile_rows || hh >= tile_heads) continue;
      if (starts && ends) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint16_t* to = a.out + (static_cast<int64_t>(row0 + rr) * a.heads + head0 + hh) * a.d;
#pragma unroll
        for (int e = 0; e < DB; ++e)
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int c = 32 * e + 8 * z + 4 * lh;
            f32x4_t y = {o[b][e][4 * z], o[b][e][4 * z + 1], o[b][e][4 * z + 2], o[b][e][4 * z + 3]};
            if (sum == 0.0f) y = f32x4_t{};
            if (c < a.d) *reinterpret_cast<half4_t*>(to + c) = __builtin_convertvector(y * inv, half4_t);
          }
      } else {
#pragma unroll
        for (int e = 0; e < DB; ++e)
#pragma unroll
          for (int z = 0; z < 4; ++z)
            *reinterpret_cast<f32x4_t*>(state + n * D + 32 * e + 8 * z + 4 * lh) =
                f32x4_t{o[b][e][4 * z], o[b][e][4 * z + 1], o[b][e][4 * z + 2], o[b][e][4 * z + 3]};
        if (lh == 0) {
          state[kRows * D + 2 * n] = top[b];
          state[kRows * D + 2 * n + 1] = sum;
        }
      }
    }
    if (starts && !ends && tid == 0)
      a.parts[me] = make_int4(row0, head0, tile_heads << 16 | tile_rows,
                              static_cast<int>(quotient(at + here.steps - 1, line.share) - me + 1));
    at += step1 - step0;
  }
}

// ---- many query rows of wide heads

// What is made of v is made again in every unit: held over the loop, addresses and masks of the branches alone spill
// registers, whose loads then wait for the keys and values on their way.
__device__ __forceinline__ int afresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The same for heads of 256 columns, whose outputs and queries would not fit the registers of two waves on a SIMD
// (one wave with all of them spills, and nothing runs beside its products): two waves share 32 query rows. Each
// makes the scores of half of a unit's tokens and the output of half of the columns, so that both read keys and
// values once between them. They meet in LDS: each half's largest scores at the end of the products' turn, the
// weights at the end of the other. Both then raise the same maximum.
//
// There is room for two buffers of values, so that a wave stores its values one unit after its keys: in the turn behind
// the products of unit s the waves that come first store K(s + 1) and V(s), the others K(s + 2) and V(s + 1). K(s) is
// read in turns 2 s and 2 s + 1, V(s) in 2 s + 2 and 2 s + 3.
//
// 4,096 rows over 8,192 tokens and themselves (16 heads over 4) take 900 us, 764 TFLOP/s (one wave with 32 rows of its
// own 2,144); 16 trees of 31 to 61 rows over 2,050 to 4,100 tokens 105 (266). Matrix cores busy 34 % of the cycles,
// vector units 42 %, LDS 31 %, where the other kernel has 44, 48 and 28: the weights' way through LDS and the addresses
// made again are what is longer.
constexpr int kPairRows = 128;  // query rows of a tile: four pairs of waves

__global__ __launch_bounds__(512) void attention_pairs_kernel(AttnArgs a) {
  constexpr int D = 256, W = 8;
  constexpr int KS = D / 16;           // products of 16 columns in a score
  constexpr int DB = D / 64;           // blocks of 32 columns of a wave's half of the output
  constexpr int kChunks = D / 8;       // 16-byte pieces of a token's keys
  constexpr int kGroup = kWave / kChunks;  // tokens that a wave loads at once
  constexpr int kMine = kWide / W;         // tokens of a unit that it loads, of one page
  constexpr int kPasses = kMine / kGroup;
  static_assert(kMine == kMinPage, "whole pages");
  constexpr int kAhead = 4;            // pieces of keys or values read before they are needed
  constexpr int kTile = kWide * D * 2;
  __shared__ __attribute__((aligned(16))) char keys[2][kTile];
  __shared__ __attribute__((aligned(16))) char values[2][kTile];
  __shared__ __attribute__((aligned(16))) _Float16 weights[W / 2][4][kWave][8];
  __shared__ float meet[W / 2][2][32];  // largest scores, at the end the sums of weights
  __shared__ uint32_t flags[4][4];      // tokens without a page, and with values that are infinite or NaN

  const int tid = threadIdx.x, lane = tid & (kWave - 1), li = lane & 31, lh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave), pair = wave / 2, half = wave % 2;
  const int turn = wave / (W / 2);  // a SIMD has a wave of either
  const int64_t me = (blockIdx.x % kParts) * (gridDim.x / kParts) + blockIdx.x / kParts;
  Request r;
  const Share line = share_of<kWide, W, kWideBits>(a, me, r);
  if (tid == 0) a.parts[me] = make_int4(0, 0, 0, 0);
  if (line.begin >= line.end) return;
  int request = line.request;
  int64_t base = line.base;

  const Place begun = place_of(r, line.begin - base);
  const int64_t begun_end = begun.step == 0 ? line.begin : min(line.begin + begun.steps - begun.step, line.end);
  int64_t stop = line.end;
  bool done = begun_end == line.begin;
  for (int64_t at = begun_end;;) {
    if (at == stop) {
      if (done) break;
      done = true;
      at = line.begin;
      stop = begun_end;
      request = line.request;
      base = line.base;
      r = request_of<kWide>(a, request);
    }
    while (at >= base + r.units) {
      base += r.units;
      r = request_of<kWide>(a, ++request);
    }
    const Place here = place_of(r, at - base);
    const int step0 = static_cast<int>(here.step);
    const int step1 = static_cast<int>(min(here.step + (stop - at), here.steps));
    const int kvh = here.head / a.chunks, chunk = here.head - kvh * a.chunks;
    const int ratio = a.heads / a.kv_heads;
    const int head0 = kvh * ratio + chunk * a.group;
    const int tile_heads = min(a.group, ratio - chunk * a.group);
    const int row0 = r.begin + here.tile * a.rows;
    const int tile_rows = min(a.rows, r.rows - here.tile * a.rows);
    const int edge = a.ancestors ? r.length : r.length + here.tile * a.rows + 1;
    const int ending = a.ancestors ? r.tokens : min(r.tokens, r.length + here.tile * a.rows + tile_rows);
    const int last = min(step1, (ending + kWide - 1) / kWide);

    const const_int_t* table = (const const_int_t*)(a.table + static_cast<int64_t>(request) * a.width);
    const int64_t page_elements = (static_cast<int64_t>(a.kv_heads) << a.shift) * a.d;
    const int64_t head_at = (static_cast<int64_t>(kvh) << a.shift) * a.d;
    const int page_mask = (1 << a.shift) - 1;
    const int load_t = lane / kChunks, load_c = lane % kChunks;
    const uint32_t lane_at = 2 * (load_t * a.d + (8 * load_c < a.d ? 8 * load_c : 0));  // in bytes
    int key_page = -1, value_page = -1, page_next = -1;
    uint4 kr[kPasses], vr[kPasses];
    auto fetch_page = [&](int s) {
      const int t = s * kWide + wave * kMine;
      const int found = table[static_cast<uint32_t>(min(t >> a.shift, a.width - 1))];
      page_next = t < r.tokens && static_cast<uint32_t>(found) < static_cast<uint32_t>(a.pages) ? found : -1;
    };
    auto place = [&](int s, int page) {
      return max(page, 0) * page_elements + head_at + ((s * kWide + wave * kMine) & page_mask) * a.d;
    };
    // keys of unit s, and the page of the next
    auto fetch_keys = [&](int s) {
      key_page = page_next;
      const int64_t from = place(s, key_page);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) kr[i] = load16(a.k + from + i * kGroup * a.d, lane_at);
      fetch_page(s + 1);
    };
    // values of unit s, whose keys were the last to be loaded, and the keys after those
    auto fetch = [&](int s) {
      if (s < last) {
        value_page = key_page;
        const int64_t from = place(s, value_page);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) vr[i] = load16(a.v + from + i * kGroup * a.d, lane_at);
      }
      if (s + 1 < last) fetch_keys(s + 1);
    };
    auto store_keys = [&](int s) {
      char* to = keys[s & 1];
      const int lane_now = afresh(lane), load_t = lane_now / kChunks, load_c = lane_now % kChunks;
      if (key_page < 0) {
        __builtin_amdgcn_sched_barrier(0);  // a branch
        if (lane == 0) atomicOr(&flags[s & 3][wave / 4], 0xFFu << (wave % 4 * 8));
#pragma unroll
        for (int i = 0; i < kPasses; ++i) kr[i] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int t = wave * kMine + i * kGroup + load_t;
        if (a.d != D && 8 * load_c >= a.d) kr[i] = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(to + t * (D * 2) + key_piece<D>(t, load_c) * 16) = kr[i];
      }
    };
    auto store_values = [&](int s) {
      char* to = values[s & 1];
      const int lane_now = afresh(lane), load_t = lane_now / kChunks, load_c = lane_now % kChunks;
      const bool edges = (s + 1) * kWide > edge;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int t = wave * kMine + i * kGroup + load_t;
        if (value_page < 0) {
          __builtin_amdgcn_sched_barrier(0);
          vr[i] = make_uint4(0, 0, 0, 0);
        }
        if (edges) {
          __builtin_amdgcn_sched_barrier(0);
          uint4& w = vr[i];
          const uint4 n = make_uint4(not_finite(w.x), not_finite(w.y), not_finite(w.z), not_finite(w.w));
          if (n.x | n.y | n.z | n.w) atomicOr(&flags[s & 3][2 + t / 32], 1u << (t % 32));
          w = make_uint4(w.x & ~n.x, w.y & ~n.y, w.z & ~n.z, w.w & ~n.w);
        }
        *reinterpret_cast<uint4*>(to + t * (D * 2) + value_piece<D>(t, load_c) * 16) = vr[i];
      }
    };

    // ---- queries: row li is query row 32 pair + li: row / group, head % group
    const int n = 32 * pair + li, rr = n / a.group, hh = n - rr * a.group;
    const bool fine = rr < tile_rows && hh < tile_heads;
    const bool busy = 32 * pair / a.group < tile_rows;
    // the last token that any row of the pair sees
    const int pair_rows = (32 * pair + 31) / a.group + 1;
    const int pair_end = a.ancestors ? ending : min(ending, r.length + here.tile * a.rows + pair_rows);
    const uint64_t tree = fine && a.ancestors ? a.ancestors[row0 + rr] : 0;
    const int upto = fine && !a.ancestors ? r.length + (row0 + rr - r.begin) : r.length - 1;
    mfma_half8_t q[KS];
    {
      const uint16_t* p = a.q + (static_cast<int64_t>(row0 + rr) * a.heads + head0 + hh) * a.d;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const int c = 8 * (2 * j + lh);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (fine && c < a.d) w = *reinterpret_cast<const uint4*>(p + c);
        q[j] = __builtin_bit_cast(mfma_half8_t, w);
      }
    }
    float top = kNone, part = 0.0f;
    f32x16_t o[DB];
#pragma unroll
    for (int e = 0; e < DB; ++e) o[e] = f32x16_t{};

    __syncthreads();  // the last tile's buffers and flags
    if (tid < 16) flags[tid / 4][tid % 4] = 0;
    __syncthreads();
    if (step0 < last) {
      fetch_page(step0);
      fetch_keys(step0);
      store_keys(step0);
      fetch(step0);
      if (turn) {
        if (step0 + 1 < last) store_keys(step0 + 1);
        store_values(step0);
        fetch(step0 + 1);
      }
    }
    __syncthreads();
    if (turn) __syncthreads();

    f32x16_t x;
    uint64_t seen = 0;
    bool masked = false, far = false;  // far: the maximum of some row of the pair is far from 0
    for (int s = step0; s <= last; ++s) {
      // ---- the matrix products' turn: O^T += V^T W^T of unit s - 1, S^T = K Q^T of unit s
      const bool scores = busy && s < last && s * kWide < pair_end;
      if (busy && s > step0 && (s - 1) * kWide < pair_end) {
        const char* vs = values[(s - 1) & 1];
        const int lane_now = afresh(lane), lh = lane_now >> 5;
        mfma_half8_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const mfma_half8_t*>(weights[pair][j][lane_now]);
        auto value = [&](int y) {  // columns 32 (y % DB) of the half on of tokens 16 (y / DB) on
          mfma_half8_t v;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int t = 16 * (y / DB) + 8 * z + 4 * lh + (lane_now & 15) / 4;
            const int c = 16 * half + 4 * (y % DB) + 2 * ((lane_now >> 4) & 1) + (lane_now & 3) / 2;
            const auto v4 = __builtin_bit_cast(half4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_short4_t*)(vs + t * (D * 2) + value_piece<D>(t, c) * 16 + (lane_now & 1) * 8)));
#pragma unroll
            for (int u = 0; u < 4; ++u) v[4 * z + u] = v4[u];
          }
          return v;
        };
        mfma_half8_t vf[kAhead];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int y = 0; y < kAhead; ++y) vf[y] = value(y);
#pragma unroll
        for (int y = 0; y < 4 * DB; ++y) {
          const mfma_half8_t v = vf[y % kAhead];
          o[y % DB] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, w[y / DB], o[y % DB], 0, 0, 0);
          if (y + kAhead < 4 * DB) vf[y % kAhead] = value(y + kAhead);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * kAhead, 0);  // LDS reads
#pragma unroll
        for (int y = 0; y < 4 * DB - kAhead; ++y) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix instructions
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (masked) {
          // infinities and NaN among values that some rows may not see: added for the rows that do
          uint64_t wild = flags[(s - 1) & 3][2] | static_cast<uint64_t>(flags[(s - 1) & 3][3]) << 32;
          const int li = afresh(lane) & 31, lh = afresh(lane) >> 5;
          while (wild) {
            const int y = __builtin_ctzll(wild);
            wild &= wild - 1;
            const int t = (s - 1) * kWide + y, number = table[static_cast<uint32_t>(t >> a.shift)];
            const int64_t p = number * page_elements + head_at + (t & page_mask) * a.d;
            // element (y / 8) * 4 + y % 4 of the lane that holds the token
            const _Float16* mine = weights[pair][y >> 4][li + 32 * ((y >> 2) & 1)];
            const float add = static_cast<float>(mine[((y >> 3) & 1) * 4 + (y & 3)]);
            if (seen >> y & 1) {
#pragma unroll
              for (int e = 0; e < DB; ++e)
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  f32x4_t part_o = {o[e][4 * z], o[e][4 * z + 1], o[e][4 * z + 2], o[e][4 * z + 3]};
                  add_wild(part_o, a.v + p, 128 * half + 32 * e + 8 * z + 4 * lh, a.d, add);
#pragma unroll
                  for (int u = 0; u < 4; ++u) o[e][4 * z + u] = part_o[u];
                }
            }
          }
        }
      }
      if (scores) {
        const char* ks = keys[s & 1];
        const int lane_now = afresh(lane), li = lane_now & 31, lh = lane_now >> 5;
        auto key = [&](int y) {
          const int t = 32 * half + li;
          return *reinterpret_cast<const mfma_half8_t*>(ks + t * (D * 2) + key_piece<D>(t, 2 * y + lh) * 16);
        };
        mfma_half8_t kf[kAhead];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int y = 0; y < kAhead; ++y) kf[y] = key(y);
#pragma unroll
        for (int y = 0; y < KS; ++y) {
          const mfma_half8_t k = kf[y % kAhead];
          x = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[y], y == 0 ? f32x16_t{} : x, 0, 0, 0);
          if (y + kAhead < KS) kf[y % kAhead] = key(y + kAhead);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int y = 0; y < KS - kAhead; ++y) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
        __builtin_amdgcn_sched_barrier(0);
        const int t0 = s * kWide;
        const uint64_t gaps = flags[s & 3][0] | static_cast<uint64_t>(flags[s & 3][1]) << 32;
        masked = t0 + kWide > edge || gaps != 0;
        if (masked) {
          __builtin_amdgcn_sched_barrier(0);  // a branch, not a selection in every unit
          seen = seen_from(t0, r.length, upto, tree) & ~gaps & ones_below(r.tokens - t0);
          const uint32_t mine = static_cast<uint32_t>(seen >> (32 * half + 4 * lh));
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = seen_or_none(x[e], mine, 8 * (e / 4) + e % 4);
        }
        float high = kNone;
#pragma unroll
        for (int e = 0; e < 16; ++e) high = fmaxf(high, x[e]);
        auto both = __builtin_amdgcn_permlane32_swap(as_u32(high), as_u32(high), false, false);
        if (lh == 0) meet[pair][half][li] = fmaxf(as_f32(both[0]), as_f32(both[1]));
      }
      __syncthreads();

      // ---- the other instructions' turn: loads, and the weights of unit s
      const int next = s + 1 + turn;
      if (next < last) store_keys(next);
      if (next - 1 < last) store_values(next - 1);
      fetch(next);
      // last read two units before it, written from the next turn on
      if (tid < 4) flags[(s + 2) & 3][tid] = 0;
      if (scores) {
        const float most = fmaxf(meet[pair][0][li], meet[pair][1][li]);
        float high = __builtin_fmaf(most, a.scale, -kWideLift / 2);
        if (__any(high > top + kWideSlack)) {
          const bool passes = high > top + kWideSlack;
          if (is_far(high)) high = rounded_product(most, a.scale);
          const float now = passes ? high : top, keep = weight_of(top, now);
          top = now;
          part *= keep;
#pragma unroll
          for (int e = 0; e < DB; ++e) o[e] *= keep;
          far = __any(is_far(now));
        }
        float less = lifted(top);
        if (__builtin_expect(far, 0)) {
          __builtin_amdgcn_sched_barrier(0);  // a branch
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = over_far(x[e], a.scale, top);
          less = is_far(top) ? 0.0f : less;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float p[8];
          mfma_half8_t w;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            p[e] = exp2_of(__builtin_fmaf(x[8 * j + e], a.scale, -less));
            w[e] = static_cast<_Float16>(p[e]);
          }
          part += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
          *reinterpret_cast<mfma_half8_t*>(weights[pair][2 * half + j][lane]) = w;
        }
      }
      __syncthreads();
    }
    if (!turn) __syncthreads();

    auto both = __builtin_amdgcn_permlane32_swap(as_u32(part), as_u32(part), false, false);
    if (lh == 0) meet[pair][half][li] = as_f32(both[0]) + as_f32(both[1]);
    __syncthreads();
    const float sum = meet[pair][0][li] + meet[pair][1][li];
    const bool starts = here.step == 0, ends = step1 == here.steps;
    if (fine && starts && ends) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      uint16_t* to = a.out + (static_cast<int64_t>(row0 + rr) * a.heads + head0 + hh) * a.d;
#pragma unroll
      for (int e = 0; e < DB; ++e)
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int c = 128 * half + 32 * e + 8 * z + 4 * lh;
          f32x4_t y = {o[e][4 * z], o[e][4 * z + 1], o[e][4 * z + 2], o[e][4 * z + 3]};
          if (sum == 0.0f) y = f32x4_t{};
          if (c < a.d) *reinterpret_cast<half4_t*>(to + c) = __builtin_convertvector(y * inv, half4_t);
        }
    } else if (fine) {
      float* state = a.states + (me * 2 + (starts ? 1 : 0)) * kPairRows * (D + 2);
#pragma unroll
      for (int e = 0; e < DB; ++e)
#pragma unroll
        for (int z = 0; z < 4; ++z)
          *reinterpret_cast<f32x4_t*>(state + n * D + 128 * half + 32 * e + 8 * z + 4 * lh) =
              f32x4_t{o[e][4 * z], o[e][4 * z + 1], o[e][4 * z + 2], o[e][4 * z + 3]};
      if (lh == 0 && half == 0) {
        state[kPairRows * D + 2 * n] = top;
        state[kPairRows * D + 2 * n + 1] = sum;
      }
    }
    if (starts && !ends && tid == 0)
      a.parts[me] = make_int4(row0, head0, tile_heads << 16 | tile_rows,
                              static_cast<int>(quotient(at + here.steps - 1, line.share) - me + 1));
    at += step1 - step0;
  }
}

// Joins the pieces of the tiles of R query rows that several of N workgroups had. Every workgroup counts the jobs,
// four query rows of a tile each, and takes its share of them (a workgroup for each that could be, most of them with
// nothing to do, took 9 us for 4,096). A wave has 16 lanes a row and merges pieces as they come, the loads of AHEAD
// in flight. With SHARE the workgroup's waves share the pieces of the same four rows (few rows, many pieces),
// otherwise each has rows of its own.
template <int D, int R, int N, bool SHARE, int AHEAD>
__device__ __forceinline__ void join(const AttnArgs& a, int block, int blocks) {
  constexpr int64_t kState = R * (D + 2);
  constexpr int V = D / 64;  // groups of four columns a lane
  constexpr int kAhead = AHEAD;
  constexpr int kEach = N / kThreads;
  __shared__ __attribute__((aligned(16))) float acc_at[SHARE ? kWaves : 1][4][D];
  __shared__ float top_at[kWaves][4], sum_at[kWaves][4];
  // tiles of 16 query rows have a job or two each: a workgroup each, with no need to count
  constexpr bool kCounts = R > 16;
  __shared__ int ends[kCounts ? N : 1], waves[kWaves];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), li = lane & 15, lg = lane >> 4, wave = tid / kWave;
  auto jobs_of = [&](const int4& part) { return part.w == 0 ? 0 : ((part.z & 0xFFFF) * a.group + 3) / 4; };
  int jobs;
  if constexpr (kCounts) {
    int count[kEach], mine = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      count[i] = jobs_of(a.parts[tid * kEach + i]);
      mine += count[i];
    }
    int before = block_scan<kWaves>(mine, waves, jobs);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      before += count[i];
      ends[tid * kEach + i] = before;
    }
    __syncthreads();
  } else {
    jobs = jobs_of(a.parts[block]);
  }
  const int step = !kCounts ? 1 : SHARE ? blocks : blocks * kWaves;
  for (int job = !kCounts ? 0 : SHARE ? block : block * kWaves + wave; job < jobs; job += step) {
    int64_t me = block;
    int n = job * 4 + lg;
    if constexpr (kCounts) {
      int lo = 0, hi = N - 1;  // the first workgroup whose jobs end behind this one
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (ends[mid] > job) hi = mid;
        else lo = mid + 1;
      }
      me = __builtin_amdgcn_readfirstlane(lo);
      n -= me == 0 ? 0 : ends[me - 1] * 4;
    }
    const int4 part = a.parts[me];
    const int rr = n / a.group, hh = n - rr * a.group;
    const bool fine = rr < (part.z & 0xFFFF) && hh < part.z >> 16;
    // the first piece is the second state of its workgroup
    const float* states = a.states + me * 2 * kState;
    float top = kNone, sum = 0.0f;
    f32x4_t acc[V] = {};
    auto merge = [&](float high, float w, const f32x4_t (&x)[V]) {
      const float now = fmaxf(top, high), keep = weight_of(top, now), add = weight_of(high, now);
      top = now;
      sum = sum * keep + w * add;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = acc[v] * keep + x[v] * add;
    };
    const int first = SHARE ? wave : 0, by = SHARE ? kWaves : 1;
    if (fine) {
      for (int p = first; p < part.w; p += kAhead * by) {
        float high[kAhead], w[kAhead];
        f32x4_t x[kAhead][V];
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
          const int piece = min(p + y * by, part.w - 1);
          const float* s = states + piece * 2 * kState + (piece == 0 ? kState : 0);
          high[y] = s[R * D + 2 * n];
          w[y] = s[R * D + 2 * n + 1];
#pragma unroll
          for (int v = 0; v < V; ++v) x[y][v] = *reinterpret_cast<const f32x4_t*>(s + n * D + 64 * v + 4 * li);
        }
#pragma unroll
        for (int y = 0; y < kAhead; ++y)
          if (p + y * by < part.w) merge(high[y], w[y], x[y]);
      }
    }
    if constexpr (SHARE) {
#pragma unroll
      for (int v = 0; v < V; ++v) *reinterpret_cast<f32x4_t*>(&acc_at[wave][lg][64 * v + 4 * li]) = acc[v];
      if (li == 0) {
        top_at[wave][lg] = top;
        sum_at[wave][lg] = sum;
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int y = 1; y < kWaves; ++y) {
          f32x4_t x[V];
#pragma unroll
          for (int v = 0; v < V; ++v) x[v] = *reinterpret_cast<const f32x4_t*>(&acc_at[y][lg][64 * v + 4 * li]);
          merge(top_at[y][lg], sum_at[y][lg], x);
        }
      }
      __syncthreads();
    }
    if (fine && (!SHARE || wave == 0)) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      uint16_t* to = a.out + (static_cast<int64_t>(part.x + rr) * a.heads + part.y + hh) * a.d;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 64 * v + 4 * li;
        if (sum == 0.0f) acc[v] = f32x4_t{};
        if (c < a.d) *reinterpret_cast<half4_t*>(to + c) = __builtin_convertvector(acc[v] * inv, half4_t);
      }
    }
  }
}

template <int D, int R, int N, bool SHARE>
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttnArgs a) {
  join<D, R, N, SHARE, SHARE ? 1024 / D : 4>(a, blockIdx.x, gridDim.x);
}

// For both kernels at once: the first N workgroups join tiles of 16 query rows, the others those of R.
template <int D, int N, int R, int M>
__global__ __launch_bounds__(kThreads) void attention_join_both_kernel(AttnArgs few, AttnArgs wide) {
  if (blockIdx.x < N) join<D, 16, N, true, 4>(few, blockIdx.x, N);
  else join<D, R, M, false, 4>(wide, blockIdx.x - N, gridDim.x - N);
}

// Workgroups of a launch: as many as the chip holds at once.
constexpr int kGroups = 1 << few_bits(64, 1);
constexpr int kWideGroups = 1 << kWideBits;
constexpr int kJoinGroups = 256;

constexpr int wide_rows(int d) { return d == 256 ? kPairRows : 256; }

// The sizes of tiles of R query rows, and their part of the workspace.
AttnArgs with_tiles(AttnArgs a, int r, void* ws) {
  const int ratio = a.heads / a.kv_heads;
  a.group = ratio < r ? ratio : r;
  a.chunks = (ratio + a.group - 1) / a.group;
  a.rows = 1 << (31 - __builtin_clz(r / a.group));
  a.parts = static_cast<int4*>(ws);
  a.states = reinterpret_cast<float*>(static_cast<char*>(ws) + kGroups * sizeof(int4));
  return a;
}

constexpr int64_t workspace_of(int groups, int r, int d) {
  return kGroups * sizeof(int4) + static_cast<int64_t>(groups) * 2 * r * (d + 2) * sizeof(float);
}

template <int D, int QB>
hipError_t launch_few(const AttnArgs& args, void* ws, hipStream_t stream) {
  constexpr int groups = 1 << few_bits(D, QB);
  const AttnArgs a = with_tiles(args, QB * 16, ws);
  hipLaunchKernelGGL((attention_kernel<D, QB>), dim3(groups), dim3(kThreads), 0, stream, a);
  hipLaunchKernelGGL((attention_join_kernel<D, QB * 16, groups, true>), dim3(QB == 1 ? groups : kJoinGroups),
                     dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

// Without a tree, requests with at most 16 query rows a key head go through the kernel for few rows, also here:
// single tokens beside a prompt. 63 tokens of requests of 4,096 beside a prompt of 1,024 rows take 256 us, all
// through the wide kernel 422. Where there are none the launch costs 7 us with its part of the join (of 771 for 4,096
// rows over 8,192 tokens), which calls with a tree do not pay (16 trees of 30 to 61 rows: 87 us, 94 with it; single
// tokens among them take the wide kernel), nor does one request, nor heads of which more than 16 share a key head.
template <int D>
hipError_t launch_wide(const AttnArgs& args, void* ws, hipStream_t stream) {
  constexpr int R = wide_rows(D), groups = 1 << few_bits(D, 1);
  AttnArgs few = with_tiles(args, 16, ws);
  AttnArgs wide = with_tiles(args, R, static_cast<char*>(ws) + workspace_of(groups, 16, D));
  const int ratio = args.heads / args.kv_heads;
  const bool both = !args.ancestors && args.requests > 1 && ratio <= 16;
  if (both) {
    few.most = 16 / ratio;
    wide.least = few.most + 1;
    hipLaunchKernelGGL((attention_kernel<D, 1>), dim3(groups), dim3(kThreads), 0, stream, few);
  }
  if constexpr (D == 256) hipLaunchKernelGGL(attention_pairs_kernel, dim3(kWideGroups), dim3(512), 0, stream, wide);
  else hipLaunchKernelGGL((attention_wide_kernel<D>), dim3(kWideGroups), dim3(512), 0, stream, wide);
  if (both)
    hipLaunchKernelGGL((attention_join_both_kernel<D, groups, R, kWideGroups>), dim3(groups + 8 * kJoinGroups),
                       dim3(kThreads), 0, stream, few, wide);
  else
    hipLaunchKernelGGL((attention_join_kernel<D, R, kWideGroups, false>), dim3(8 * kJoinGroups), dim3(kThreads), 0,
                       stream, wide);
  return hipGetLastError();
}

// Which kernel, by the query rows of a key head that a request has on average, which is what the host knows; rows
// behind the last request and requests without rows count like others. It suits requests that are alike, and a prompt
// that an average hides among many tokens is slow in small tiles: 255 tokens over 1,000 with a prompt of 512 rows over
// 8,192 take 724 us, in calls of their own 197 and 108. Eight requests of up to 8,192 tokens
// at head_dim 128: 20 rows take 74.5 us in tiles of 16, 61.7 in tiles of 32 and 62.5 in the wide kernel; 28 rows
// 90.1, 62.4 and 63.0; 48 rows 93.9 in tiles of 48, 128.6 in tiles of 64 and 67.4 in the wide kernel. One row each of
// 64 requests: 217 us in tiles of 16, 291 in tiles of 32, 829 wide. At head_dim 256, where a tile of 32 does not fit
// the registers, the kernel of pairs takes over: 16 trees of 24 query rows over 2,050 to 4,100 tokens take 71 us there
// and 99 in tiles of 16, 40 rows 75 and 143; 8 requests of 32 rows 43.6 and 46.0, one of 32 rows over 2,000 tokens
// 25.5 and 24.3.
template <int D>
hipError_t launch_rows(const AttnArgs& a, int64_t rows, void* ws, hipStream_t stream) {
  if (rows <= 16) return launch_few<D, 1>(a, ws, stream);
  if constexpr (D < 256) {
    if (rows <= 32) return launch_few<D, 2>(a, ws, stream);
  }
  return launch_wide<D>(a, ws, stream);
}

}  // namespace

// For heads of this width and narrower ones.
int64_t attention_workspace_bytes(int head_dim) {
  int64_t most = 0;
  for (int d = 64; d <= 256 && (d == 64 || d < 2 * head_dim); d *= 2) {
    const int64_t two = d == 256 ? 0 : workspace_of(1 << few_bits(d, 2), 32, d);
    const int64_t both = workspace_of(1 << few_bits(d, 1), 16, d) + workspace_of(kWideGroups, wide_rows(d), d);
    most = most > two ? most : two;
    most = most > both ? most : both;
  }
  return most;
}

hipError_t launch_tree_attention(const uint16_t* q, const uint16_t* k_cache, const uint16_t* v_cache, int64_t pages,
                                 int64_t page_size, const int32_t* table, int64_t table_width, const int32_t* lengths,
                                 const int32_t* row_start, int64_t requests, const uint64_t* ancestors, int64_t m,
                                 int heads, int kv_heads, int head_dim, float scale, uint16_t* out, void* workspace,
                                 hipStream_t stream) {
  const AttnArgs a = {q, k_cache, v_cache, pages, page_shift(page_size), table, static_cast<int>(table_width), lengths,
                      row_start, static_cast<int>(requests), ancestors, static_cast<int>(m), heads, kv_heads, head_dim,
                      scale * kLog2e, out, 0, 0, 0, 0, 0x7FFFFFFF, nullptr, nullptr};
  // query rows of a key head that a request has on average
  const int64_t rows = (m * (heads / kv_heads) + requests - 1) / requests;
  if (head_dim <= 64) return launch_rows<64>(a, rows, workspace, stream);
  if (head_dim <= 128) return launch_rows<128>(a, rows, workspace, stream);
  return launch_rows<256>(a, rows, workspace, stream);
}

}  // namespace pbg
