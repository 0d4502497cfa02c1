// Expert routing and the sum of a token's expert rows.
//
// route_select: the k largest logits of every token and their softmax
// weights.  16 lanes hold a token's logits (64 lanes above 256 experts) in
// registers and take the largest k times: each lane's own largest, then a
// butterfly over the lanes (row rotations, no LDS), ties to the lowest
// expert.  A workgroup then ranks its choices by expert: each wave compares
// the expert numbers of 64 choices bit by bit with ballots, so a choice's
// rank among equal ones is the count of lower lanes in its match mask --
// in order of (token, choice), with no atomic whose order could change it.
// route_place: every workgroup adds up the counts of the ones before it and
// writes each choice's slot and each slot's token.
// Calls of one workgroup place their choices in route_select itself.
//
// Bound by the latency of its passes over registers and LDS, not by memory:
// 16384 tokens, 128 experts, 8 choices 13 us + 7 us for 7.9 MB; 32 tokens of 64
// experts 5.6 us in one launch.  16 lanes a token keep the butterfly within the
// rotations of a row; up to 256 workgroups keep the counts that every one of
// them reads to 256 rows (reading them one at a time cost 19 us instead of 7).
#include "sgmv_matmul.h"
#include "sgmv_route_launch.h"

namespace sgmv {
namespace dev {

__device__ __forceinline__ int32_t row_ror(int32_t v, int n) {
  // rotation within each row of 16 lanes; n must fold to a constant
  switch (n) {
    case 1: return __builtin_amdgcn_update_dpp(0, v, 0x121, 0xf, 0xf, false);
    case 2: return __builtin_amdgcn_update_dpp(0, v, 0x122, 0xf, 0xf, false);
    case 4: return __builtin_amdgcn_update_dpp(0, v, 0x124, 0xf, 0xf, false);
    default: return __builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, false);
  }
}

// Largest (value, lowest expert) over the LPT lanes of a token, in all of them.
template <int LPT>
__device__ __forceinline__ void reduce_best(float* v, int32_t* e) {
#pragma unroll
  for (int d = 1; d < LPT; d <<= 1) {
    float ov;
    int32_t oe;
    if (d < 16) {
      ov = __int_as_float(row_ror(__float_as_int(*v), d));
      oe = row_ror(*e, d);
    } else {
      ov = __shfl_xor(*v, d);
      oe = __shfl_xor(*e, d);
    }
    const bool take = ov > *v || (ov == *v && oe < *e);
    *v = take ? ov : *v;
    *e = take ? oe : *e;
  }
}

template <int LPT>
__device__ __forceinline__ float reduce_sum(float v) {
#pragma unroll
  for (int d = 1; d < LPT; d <<= 1)
    v += d < 16 ? __int_as_float(row_ror(__float_as_int(v), d)) : __shfl_xor(v, d);
  return v;
}

// exp(x - m) for x <= m; 1 at x = m, also where both are +inf.
__device__ __forceinline__ float exp_below(float x, float m) {
  return x == m ? 1.f : __expf(x - m);
}

// Logits e0 .. e0 + V of a row; past E and NaN: -inf, never chosen.
template <int V>
__device__ __forceinline__ void load_logits(const char* row, int e0, int E, int dtype, bool vec,
                                            float* x) {
  if (V >= 4 && vec) {  // E is a multiple of V and rows are aligned for these loads
    if (dtype == F32) {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const float4 q = e0 < E ? *reinterpret_cast<const float4*>(row + (e0 + v) * 4)
                                : float4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        x[v] = q.x, x[v + 1] = q.y, x[v + 2] = q.z, x[v + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        uint2 q = e0 < E ? *reinterpret_cast<const uint2*>(row + (e0 + v) * 2) : uint2{0u, 0u};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t h = (i < 2 ? q.x : q.y) >> (16 * (i & 1)) & 0xFFFFu;
          x[v + i] = e0 >= E ? -INFINITY : dtype == BF16 ? widen<BF16>(h) : widen<F16>(h);
        }
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      x[v] = e0 + v < E ? load_elem(row, e0 + v, dtype) : -INFINITY;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = x[v] == x[v] ? x[v] : -INFINITY;
}

// First slot of every expert from its total in `start` (in place), and the
// number of all choices; all threads take part.
__device__ __forceinline__ int32_t starts_of(int32_t* start, int E, int32_t* sh) {
  __syncthreads();
  return block_exclusive_scan<kRouteThreads>(start, E, sh);
}

// Slots past the last choice have no token.
__device__ __forceinline__ void clear_rows(const RouteParams& p, int32_t used) {
  const int64_t n = (int64_t)p.T * p.k;
  for (int64_t i = used + (int64_t)blockIdx.x * kRouteThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kRouteThreads)
    p.rows[i] = -1;
}

template <int LPT, int V>
__global__ __launch_bounds__(kRouteThreads) void route_select(RouteParams p) {
  constexpr int kW = kRouteThreads / 64;
  extern __shared__ int32_t lds[];
  int32_t* hist = lds;                 // [E] choices of the rounds so far
  int32_t* cnt = hist + p.E;           // [kW][E] choices of a wave's 64 entries
  __shared__ int32_t ent[kRouteEntries];
  __shared__ int32_t sh[kW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int sub = lane & (LPT - 1);
  const int32_t t0 = blockIdx.x * p.block_tokens;
  const int32_t t1 = t0 + p.block_tokens < p.T ? t0 + p.block_tokens : p.T;
  for (int e = tid; e < p.E; e += kRouteThreads) hist[e] = 0;

  for (int32_t r0 = t0; r0 < t1; r0 += p.round_tokens) {
    const int32_t r1 = r0 + p.round_tokens < t1 ? r0 + p.round_tokens : t1;
    for (int e = tid; e < kW * p.E; e += kRouteThreads) cnt[e] = 0;
    // Selection, a token per LPT lanes (uniform trip count per wave: idle
    // groups repeat the last token and store nothing).
    for (int32_t base = r0; base < r1; base += kRouteThreads / LPT) {
      const int32_t t = base + tid / LPT;
      const bool live = t < r1;
      const char* row = static_cast<const char*>(p.logits) +
                        (int64_t)(live ? t : r1 - 1) * p.logits_row_bytes;
      float x[V];  // experts sub V ..: consecutive, so that a whole lane's take one or two loads
      load_logits<V>(row, sub * V, p.E, p.dtype, p.vec, x);
      float top = 0.f, over = 0.f;
      float w0 = 0.f, w1 = 0.f;      // this lane's choices: j = sub and j = sub + LPT
      int32_t e0 = -1, e1 = -1;
      for (int j = 0; j < p.k; ++j) {
        float best = -INFINITY;
        int32_t e = 0x7fffffff;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const bool take = x[v] > best;
          best = take ? x[v] : best;
          e = take ? sub * V + v : e;
        }
        reduce_best<LPT>(&best, &e);
        const bool none = best == -INFINITY;
        if (j == 0) {
          top = best;
          if (!p.renormalize) {
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) s += none ? 0.f : exp_below(x[v], top);
            over = reduce_sum<LPT>(s);
          }
        }
        const float w = none ? 0.f : exp_below(best, top);
        if (p.renormalize) over += w;
        if (j == sub) {
          w0 = w;
          e0 = none ? -1 : e;
        } else if (j == sub + LPT) {
          w1 = w;
          e1 = none ? -1 : e;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = e == sub * V + v ? -INFINITY : x[v];
      }
      if (live) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = sub + LPT * i;
          if (j < p.k) {
            const int64_t at = (int64_t)t * p.k + j;
            const int32_t e = i ? e1 : e0;
            p.weights[at] = e < 0 ? 0.f : (i ? w1 : w0) / over;
            p.experts[at] = e;
            ent[(t - r0) * p.k + j] = e;
          }
        }
      }
    }
    __syncthreads();
    // Rank of entry `tid` among the round's entries of its expert.
    const int n = (r1 - r0) * p.k;
    const int32_t e = tid < n ? ent[tid] : -1;
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; (1 << b) < p.E; ++b) {
      const uint64_t m = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? m : ~m;
    }
    int32_t rank = __builtin_popcountll(same & ((1ull << lane) - 1));
    if (e >= 0 && rank == 0) cnt[wave * p.E + e] = __builtin_popcountll(same);
    __syncthreads();
    if (e >= 0) {
      rank += hist[e];
      for (int w = 0; w < wave; ++w) rank += cnt[w * p.E + e];
    }
    if (tid < n) p.slots[(int64_t)r0 * p.k + tid] = e < 0 ? -1 : rank;  // within this workgroup
    __syncthreads();
    for (int i = tid; i < p.E; i += kRouteThreads) {
      int32_t s = hist[i];
      for (int w = 0; w < kW; ++w) s += cnt[w * p.E + i];
      hist[i] = s;
    }
    __syncthreads();
  }

  if (p.blocks > 1) {
    for (int e = tid; e < p.E; e += kRouteThreads)
      p.counts[(int64_t)blockIdx.x * p.E + e] = hist[e];
    return;
  }
  for (int e = tid; e < p.E; e += kRouteThreads) {
    cnt[e] = hist[e];
    p.lens[e] = hist[e];
  }
  const int32_t used = starts_of(cnt, p.E, sh);
  for (int e = tid; e < p.E; e += kRouteThreads) p.start[e] = cnt[e];
  for (int32_t i = tid; i < p.T * p.k; i += kRouteThreads) {
    const int32_t e = (int32_t)p.experts[i];
    if (e < 0) continue;
    const int64_t slot = cnt[e] + p.slots[i];
    p.slots[i] = slot;
    p.rows[slot] = i / p.k;
  }
  clear_rows(p, used);
}

__global__ __launch_bounds__(kRouteThreads) void route_place(RouteParams p) {
  extern __shared__ int32_t lds[];
  int32_t* total = lds;           // [E] choices of an expert, then its first slot
  int32_t* before = lds + p.E;    // [E] choices in the workgroups before this one
  __shared__ int32_t sh[kRouteThreads / 64];
  const int tid = threadIdx.x;
  for (int e = tid; e < 2 * p.E; e += kRouteThreads) lds[e] = 0;
  __syncthreads();
  // The counts' rows are dealt to as many groups of E threads as there are;
  // whole numbers, so the order of the adds does not matter.
  const int groups = p.E < kRouteThreads ? kRouteThreads / p.E : 1;
  const int g = p.E < kRouteThreads ? tid / p.E : 0;
  // The first choices of this workgroup (often all of them) are read meanwhile.
  const int32_t i0 = (int32_t)blockIdx.x * p.block_tokens * p.k;
  const int32_t end = p.T * p.k;
  const int32_t i1 = end - i0 > p.block_tokens * p.k ? i0 + p.block_tokens * p.k : end;
  int32_t e1 = -1, s1 = 0;
  if (i0 + tid < i1) {
    e1 = (int32_t)p.experts[i0 + tid];
    s1 = (int32_t)p.slots[i0 + tid];
  }
  if (g < groups) {
    for (int e = p.E < kRouteThreads ? tid % p.E : tid; e < p.E; e += kRouteThreads) {
      int32_t all = 0, mine = 0;
      constexpr int kAtOnce = 8;  // loads in flight
      for (int b = g; b < p.blocks; b += groups * kAtOnce) {
        int32_t c[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int at = b + j * groups;
          c[j] = p.counts[(int64_t)(at < p.blocks ? at : b) * p.E + e];
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int at = b + j * groups;
          all += at < p.blocks ? c[j] : 0;
          mine += at < (int)blockIdx.x ? c[j] : 0;
        }
      }
      if (all) atomicAdd(&total[e], all);
      if (mine) atomicAdd(&before[e], mine);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = tid; e < p.E; e += kRouteThreads) p.lens[e] = total[e];
  const int32_t used = starts_of(total, p.E, sh);
  if (blockIdx.x == 0)
    for (int e = tid; e < p.E; e += kRouteThreads) p.start[e] = total[e];
  for (int32_t i = i0 + tid; i < i1; i += kRouteThreads) {
    const bool first = i == i0 + tid;
    const int32_t e = first ? e1 : (int32_t)p.experts[i];
    if (e < 0) continue;
    const int32_t slot = total[e] + before[e] + (first ? s1 : (int32_t)p.slots[i]);
    p.slots[i] = slot;
    p.rows[slot] = i / p.k;
  }
  clear_rows(p, used);
}

// out[t] = (add ? out[t] : 0) + sum_j weights[t][j] rows[slots[t][j]]: eight
// columns a thread, the k rows in order, sums in float32, one rounding.
// Bound by memory: every row is read once (16384 tokens, 8 rows of 2048 each,
// bfloat16: 123 us, 4.8 TB/s; a large copy here runs at 5.1).
template <int D>
__global__ __launch_bounds__(kCombineThreads) void combine(CombineParams p) {
  const int64_t blocks8 = (p.H + 7) / 8;
  const int64_t total = p.T * blocks8;
  for (int64_t i = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kCombineThreads) {
    const int64_t t = i / blocks8, c = (i - t * blocks8) * 8;
    const int cnt = clamp8(p.H - c);
    float y[8] = {};
    for (int j = 0; j < p.k; ++j) {
      const int64_t slot = p.slots[t * p.k + j];
      if (slot < 0 || slot >= p.R) continue;
      const float w = p.weights[t * p.k + j];
      u32x4 raw[raw_vecs<D>()];
      load_any8<D>(static_cast<const char*>(p.rows) + slot * p.rows_row_bytes, c, cnt, p.vec, raw);
      float v[8];
      out_values<D>(raw, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] += w * v[q];
    }
    char* orow = static_cast<char*>(p.out) + t * p.out_row_bytes;
    if (p.add) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < cnt) y[q] += load_elem(orow, c + q, p.out_dtype);
    }
    if (p.out_dtype == F32) store_any8<F32>(orow, c, cnt, p.vec, y);
    else if (p.out_dtype == BF16) store_any8<BF16>(orow, c, cnt, p.vec, y);
    else store_any8<F16>(orow, c, cnt, p.vec, y);
  }
}

}  // namespace dev

const void* route_select_kernel(int experts) {
  using namespace dev;
  if (experts <= 16) return (const void*)route_select<16, 1>;
  if (experts <= 32) return (const void*)route_select<16, 2>;
  if (experts <= 64) return (const void*)route_select<16, 4>;
  if (experts <= 128) return (const void*)route_select<16, 8>;
  if (experts <= 256) return (const void*)route_select<16, 16>;
  if (experts <= 512) return (const void*)route_select<64, 8>;
  return (const void*)route_select<64, 16>;
}

int route_lane_experts(int experts) {
  const int lanes = experts <= 256 ? 16 : 64;
  int v = 1;
  while (lanes * v < experts) v <<= 1;
  return v;
}

const void* route_place_kernel() { return (const void*)dev::route_place; }

const void* combine_kernel(int dtype) {
  using namespace dev;
  if (dtype == F16) return (const void*)combine<F16>;
  if (dtype == BF16) return (const void*)combine<BF16>;
  return (const void*)combine<F32>;
}

}  // namespace sgmv
