// sgmv_matmul.h -- gfx950 device helpers of the shared projection with
// adapters and of the grouped products: which tile a workgroup runs, which
// adapter each of its rows has, and the result's last steps.  Internal to
// libsgmv.
#pragma once

#include "sgmv_common.h"
#include "sgmv_matmul_launch.h"

namespace sgmv {
namespace dev {

// Kernel modes: dense, grouped, grouped with the SiLU gate, dense with adapters.
enum { kDense = 0, kGrouped = 1, kGated = 2, kAdapted = 3 };

// make_rsrc of a wave-uniform range, said so (the compiler otherwise loops over
// the lanes' descriptors at every load).
__device__ __forceinline__ rsrc_t uniform_rsrc(const char* base, int64_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint64_t u = (uint64_t)(uint32_t)uniform((int)(b >> 32)) << 32 | (uint32_t)uniform((int)b);
  return make_rsrc(reinterpret_cast<const void*>(u), uniform(bytes <= 0 ? 0 : (int)bytes));
}

// ---------------------------------------------------------------------------
// Tiles.
// ---------------------------------------------------------------------------

// A workgroup's rows [row, end) of out with weight matrix `e`, and its
// column tile; row < 0: nothing to do.
struct TileLoc {
  int32_t row, end, e, col;
};

// Position of workgroup `id` in the (row tile, column tile) grid.  Workgroups
// go round-robin to the 8 XCDs, so XCD x = id mod 8 takes a contiguous eighth
// of the order; in that order kGroupRows row tiles sweep the column tiles
// together, so that the tiles an XCD runs at one time share a few weight and
// input rows in its L2.
constexpr uint32_t kGroupRows = 8;
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t row_tiles, uint32_t col_tiles,
                                        int32_t* rt, int32_t* ct) {
  const uint32_t U = row_tiles * col_tiles;
  const uint32_t x = id & 7, j = id >> 3, share = U >> 3, extra = U & 7;
  const uint32_t u = x * share + (x < extra ? x : extra) + j;
  if (j >= share + (x < extra ? 1u : 0u)) {
    *rt = -1;
    *ct = 0;
    return;
  }
  const uint32_t per_group = kGroupRows * col_tiles;
  const uint32_t g = u / per_group, in = u - g * per_group;
  const uint32_t left = row_tiles - g * kGroupRows;
  const uint32_t rows = left < kGroupRows ? left : kGroupRows;
  *ct = (int32_t)(in / rows);
  *rt = (int32_t)(g * kGroupRows + in % rows);
}

// Row range and weight matrix of grouped segment b; tiles of `tile_rows`
// rows it takes (0: inactive -- index out of range, empty, or outside
// [0, T)).
__device__ __forceinline__ int32_t read_group(const MatmulParams& p, int32_t b, int32_t tile_rows,
                                              int32_t* row, int32_t* end, int32_t* e) {
  const int64_t st = p.start[b], ln = p.lens[b];
  const int64_t a = p.idx ? p.idx[b] : b;
  const bool active = a >= 0 && a < p.L && ln > 0 && st >= 0 && st <= p.T - ln;
  *row = active ? (int32_t)st : 0;
  *end = active ? (int32_t)(st + ln) : 0;
  *e = active ? (int32_t)a : 0;
  return active ? (int32_t)((ln + tile_rows - 1) / tile_rows) : 0;
}

// The tile of this workgroup (all NT threads take part; `sh` holds
// NT / 64 + 4 words of LDS).  Grouped: every workgroup counts the segments'
// tiles (a block scan over contiguous runs of segments, so the order of
// tiles is the order of segments), and the thread whose run holds the tile
// looks it up.  None may have it where segments overlap, a broken
// precondition, and their tiles' sum passes 32 bits.
template <int NT>
__device__ __forceinline__ TileLoc find_tile(const MatmulParams& p, int32_t tile_rows,
                                             int32_t* sh) {
  TileLoc loc;
  int32_t rt;
  if (!p.grouped) {
    tile_of(blockIdx.x, (uint32_t)p.row_tiles, (uint32_t)p.col_tiles, &rt, &loc.col);
    loc.e = 0;
    loc.row = rt < 0 ? -1 : rt * tile_rows;
    const int64_t e = (int64_t)loc.row + tile_rows;
    loc.end = (int32_t)(e < p.T ? e : p.T);
    return loc;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t per = (p.batches + NT - 1) / NT;
  const int32_t b0 = tid * per, b1 = b0 + per < p.batches ? b0 + per : p.batches;
  int32_t row = 0, end = 0, e = 0, mine = 0;
  for (int32_t b = b0; b < b1; ++b) mine += read_group(p, b, tile_rows, &row, &end, &e);
  const int32_t incl = wave_inclusive_sum(mine);
  if (lane == 63) sh[wave] = incl;
  if (tid == 0) sh[NT / 64] = -1;  // no tile, should none of the threads below have it
  __syncthreads();
  int32_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    before += w < wave ? sh[w] : 0;
    total += sh[w];
  }
  total = uniform(total);
  tile_of(blockIdx.x, (uint32_t)total, (uint32_t)p.col_tiles, &rt, &loc.col);
  loc.row = -1;
  loc.end = loc.e = 0;
  if (rt < 0) return loc;  // the same in every thread of the workgroup
  int32_t at = before + incl - mine;
  if (rt >= at && rt < at + mine) {
    for (int32_t b = b0; b < b1; ++b) {
      const int32_t n = read_group(p, b, tile_rows, &row, &end, &e);
      if (rt < at + n) {
        const int32_t r = row + (rt - at) * tile_rows;
        sh[NT / 64] = r;
        sh[NT / 64 + 1] = end - r > tile_rows ? r + tile_rows : end;
        sh[NT / 64 + 2] = e;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  loc.row = uniform(sh[NT / 64]);
  loc.end = uniform(sh[NT / 64 + 1]);
  loc.e = uniform(sh[NT / 64 + 2]);
  return loc;
}

// ---------------------------------------------------------------------------
// Adapters of a tile's rows.
// ---------------------------------------------------------------------------

// Fill list[0 .. *count) with the distinct adapters of rows row0 .. end and
// row_pos[0 .. ROWS) with the place of row row0 + i's adapter in it (-1: none)
// (all NT threads take part, NT >= ROWS; `segs` holds adapter_words<ROWS>()
// words, `count` two; `mine` from read_segment, which a caller can issue
// earlier).  The segments meet in an order that changes from run to run.
// ORDERED lists the adapters in order of their first row, for the kernel whose
// rounding goes by an adapter's place (few rows); in the others an adapter's
// products meet zeros, whatever stands beside them, and the order by rows
// would cost 1% of a large prefill (256 rows, gate/up 2998 -> 3033 us).
// Segments are disjoint, so at most ROWS of them meet the tile; more (a broken
// precondition) are dropped.
struct Segment {
  int64_t start, len, a;
};
__device__ __forceinline__ Segment read_segment(const MatmulParams& p, int32_t b) {
  return b < p.batches ? Segment{p.start[b], p.lens[b], p.idx[b]} : Segment{0, 0, -1};
}

// Words of LDS in which tile_adapters keeps the segments it meets.
template <int ROWS>
constexpr int adapter_words() { return 3 * ROWS + (ROWS + 31) / 32; }

template <int NT, int ROWS, bool ORDERED>
__device__ __forceinline__ void tile_adapters(const MatmulParams& p, Segment seg, int32_t row0,
                                              int32_t end, int32_t* row_pos, int32_t* list,
                                              int32_t* count, int32_t* segs) {
  static_assert(NT >= ROWS, "one row per thread");
  constexpr int kHeads = (ROWS + 31) / 32;
  int32_t* heads = segs + 3 * ROWS;  // a bit for every row that is some adapter's first
  const int tid = threadIdx.x;
  if (tid < 2) count[tid] = 0;
  if (ORDERED && tid < kHeads) heads[tid] = 0;
  __syncthreads();
  for (int32_t b = tid; b < p.batches; b += NT) {
    if (b >= NT) seg = read_segment(p, b);
    const int64_t st = seg.start, ln = seg.len, a = seg.a;
    if (a < 0 || a >= p.L || ln <= 0 || st < 0 || st > p.T - ln) continue;
    if (st >= end || st + ln <= row0) continue;
    const int i = atomicAdd(&count[1], 1);
    if (i >= ROWS) continue;
    segs[i] = (int32_t)(st > row0 ? st - row0 : 0);
    segs[ROWS + i] = (int32_t)((st + ln < end ? st + ln : end) - row0);
    segs[2 * ROWS + i] = (int32_t)a;
  }
  __syncthreads();
  const int n = count[1] < ROWS ? count[1] : ROWS;
  int32_t head = -1;  // of the adapter that this thread lists
  if (tid < ROWS) {
    int32_t mine = -1;  // the row's adapter
    // Thread i also has segment i: its adapter is listed at its first segment here.
    const int32_t a = tid < n ? segs[2 * ROWS + tid] : -1, row = tid < n ? segs[tid] : 0;
    bool first = tid < n;
    for (int i = 0; i < n; ++i) {
      const int32_t si = segs[i], ai = segs[2 * ROWS + i];
      mine = si <= tid && tid < segs[ROWS + i] ? ai : mine;
      first = first && (ai != a || si >= row);
    }
    row_pos[tid] = mine;
    if (first && !ORDERED) list[atomicAdd(&count[0], 1)] = a;
    if (first && ORDERED) {
      head = row;
      atomicOr(&heads[row >> 5], (int32_t)(1u << (row & 31)));
    }
  }
  if (ORDERED) __syncthreads();
  if (ORDERED && (tid == 0 || head >= 0)) {
    int32_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const uint32_t h = (uint32_t)heads[i];
      const int below = head - 32 * i;  // rows of this word ahead of this thread's
      const uint32_t mask = below <= 0 ? 0u : below >= 32 ? ~0u : (1u << below) - 1u;
      before += __builtin_popcount(h & mask);
      all += __builtin_popcount(h);
    }
    if (head >= 0) list[before] = segs[2 * ROWS + tid];
    if (tid == 0) count[0] = all;
  }
  __syncthreads();
  if (tid < ROWS) {
    const int32_t mine = row_pos[tid], adapters = count[0];
    int32_t pos = -1;
    for (int i = 0; i < adapters; ++i) pos = mine >= 0 && list[i] == mine ? i : pos;
    row_pos[tid] = pos;
  }
  __syncthreads();
}

// Slice i's descriptor, read from the kernel's argument memory: a variable
// index into the argument itself makes the compiler copy all of it to scratch
// memory and read every field from there.  MatmulParams is the kernels' only
// argument.
__device__ __forceinline__ AdapterDesc adapter_desc(int i) {
  typedef const __attribute__((address_space(4))) MatmulParams* Args;
  const Args args = (Args)__builtin_amdgcn_kernarg_segment_ptr();
  const auto& d = args->s[i];
  return AdapterDesc{d.b, d.v, d.n, d.offset};
}

// Eight finite float32 values as packed operands of the 16-bit weight dtype:
// one rounding to the weights' dtype would leave the adapters' share of a
// float32 result with an error of 2^-9 or 2^-12.  v = hi + lo to 16 (bfloat16)
// or 22 (float16) bits; what bfloat16 leaves, third_operand, makes it exact
// and is multiplied where results are float32 (half as many matrix
// instructions again, invisible after a rounding to 16 bits).  float16 has its
// bits from 2^-2 to 2^15 only (lo ends at 2^-24, hi at 65504): see
// split_exponent.  Values that would round up to an infinity of bfloat16 leave
// more to the lower parts instead; the parts are added from the lowest on, so
// that hi + lo, which may round up too, is no step of an exact sum.
constexpr float kLargestBf16 = 3.38953139e38f;  // 2^128 - 2^120
template <int WD>
__device__ __forceinline__ uint32_t high_pair(float v0, float v1) {
  if constexpr (WD == BF16) {
    v0 = __builtin_amdgcn_fmed3f(v0, -kLargestBf16, kLargestBf16);
    v1 = __builtin_amdgcn_fmed3f(v1, -kLargestBf16, kLargestBf16);
  }
  return pack2<WD>(v0, v1);
}

template <int WD>
__device__ __forceinline__ void split_operand(const float* v, u32x4* hi, u32x4* lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = high_pair<WD>(v[2 * i], v[2 * i + 1]);
    (*hi)[i] = h;
    (*lo)[i] = pack2<WD>(v[2 * i] - widen<WD>(h & 0xFFFFu), v[2 * i + 1] - widen<WD>(h >> 16));
  }
}

// What hi + lo leave of eight values, at most seven bits each: exact.
__device__ __forceinline__ u32x4 third_operand(const float* v) {
  u32x4 third;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = high_pair<BF16>(v[2 * i], v[2 * i + 1]);
    const float r0 = v[2 * i] - widen<BF16>(h & 0xFFFFu), r1 = v[2 * i + 1] - widen<BF16>(h >> 16);
    const uint32_t l = pack2<BF16>(r0, r1);
    third[i] = pack2<BF16>(r0 - widen<BF16>(l & 0xFFFFu), r1 - widen<BF16>(l >> 16));
  }
  return third;
}

// float16: the e for which a row's values times 2^e have 22 bits of the largest
// in two parts, from the bits of its magnitude.  0 where they have them as they
// are, which is the usual case; else the largest comes to lie at 2^14, or, of
// values below 2^-26, 2^40 times higher.  The products are multiplied by 2^-e
// again, both exact.
__device__ __forceinline__ int split_exponent(uint32_t largest) {
  const int x = (int)(largest >> 23) - 127;
  return largest == 0 || (x >= -2 && x < 15) ? 0 : x < -26 ? 40 : 14 - x;
}

// Bits of the largest magnitude of eight values.
__device__ __forceinline__ uint32_t largest_of(const float* v) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    most = m > most ? m : most;
  }
  return most;
}

// The largest of lanes l, l + 16, l + 32 and l + 48 in all of them: two swaps of
// rows of 16 and of halves, of a register with its copy.
__device__ __forceinline__ uint32_t quarters_max(uint32_t v) {
  auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = r[0] > r[1] ? r[0] : r[1];
  r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return r[0] > r[1] ? r[0] : r[1];
}

// Eight values times 2^e.
__device__ __forceinline__ void scale_values(float* v, int e) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = ldexpf(v[i], e);
}

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int dtype) {
  if (dtype == F32) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == BF16 ? widen<BF16>(h) : widen<F16>(h);
}

// Projected values and weights that are not finite.  The two parts of a value
// times an infinity may be infinities of both signs, or zero times it; one
// request's weights must not reach another's rows, nor a slice's values the
// columns outside its window, through zeros.  The kernels multiply with what
// is not finite replaced by zeros, and what its products add (an infinity or
// NaN) is added to the results they belong to at the end (odd_products).

// Whether any of eight packed 16-bit values is an infinity or NaN: its
// exponent's bits are all ones, so that one more carries into the sign's place.
template <int WD>
__device__ __forceinline__ bool any_odd(u32x4 v) {
  constexpr uint32_t kExp = WD == BF16 ? 0x7F807F80u : 0x7C007C00u;
  constexpr uint32_t kOne = WD == BF16 ? 0x00800080u : 0x04000400u;
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) t |= (v[i] & kExp) + kOne;
  return (t & 0x80008000u) != 0;
}

// Those values replaced by zero.
template <int WD>
__device__ __forceinline__ u32x4 drop_odd(u32x4 v) {
  constexpr uint32_t kExp = WD == BF16 ? 0x7F80u : 0x7C00u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (v[i] & kExp) == kExp ? 0u : v[i] & 0xFFFFu;
    const uint32_t hi = (v[i] & kExp << 16) == kExp << 16 ? 0u : v[i] & 0xFFFF0000u;
    v[i] = hi | lo;
  }
  return v;
}

// The same for eight float32 values.
constexpr uint32_t kOddBits = 0x7F800000u;  // the least magnitude's that is not finite
__device__ __forceinline__ bool any_odd(const float* v) { return largest_of(v) >= kOddBits; }
__device__ __forceinline__ void drop_odd(float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __builtin_isfinite(v[i]) ? v[i] : 0.f;
}

// What the products that are not finite, of row `row`'s values with the weights
// of adapter a (-1: none), add to out[row][n]: 0, an infinity or NaN.
template <int WD>
__device__ __forceinline__ float odd_products(const MatmulParams& p, int row, int a, int n) {
  float sum = 0.f;
  for (int s = 0; s < p.num_slices && a >= 0; ++s) {
    const AdapterDesc d = adapter_desc(s);
    if (n < d.offset || n >= d.offset + d.n) continue;
    for (int k = 0; k < p.K; ++k) {
      const float b = load_elem(d.b, ((int64_t)a * d.n + n - d.offset) * p.K + k, WD);
      const float v = d.v[(int64_t)row * p.v_stride + k];
      if (!__builtin_isfinite(b) || !__builtin_isfinite(v)) sum += v * b;
    }
  }
  return sum;
}

// silu(g) * u = g u / (1 + exp(-g)).  For g -> -inf exp overflows to +inf and
// the quotient is -0; g = -inf itself gives NaN, as -inf * 0 does.
__device__ __forceinline__ float gate(float g, float u) {
  return g / (1.f + __expf(-g)) * u;
}

__device__ __forceinline__ void store_elem(void* p, int64_t i, int dtype, float v) {
  if (dtype == F32) {
    static_cast<float*>(p)[i] = v;
  } else {
    const uint32_t h = dtype == BF16 ? pack2<BF16>(v, 0.f) : pack2<F16>(v, 0.f);
    static_cast<uint16_t*>(p)[i] = (uint16_t)h;
  }
}

}  // namespace dev
}  // namespace sgmv
