// sgmv_matmul_api.cpp -- libsgmv C entry points of the shared projection
// with the adapters of many requests (sgmv_lora_linear) and of the products
// grouped by expert (sgmv_grouped_gemm): argument checks, kernel choice, grid
// sizing and launch.  No allocation, no synchronisation, no device-to-host
// traffic.
#include <stdint.h>

#include "sgmv.h"
#include "sgmv_host.h"
#include "sgmv_limits.h"
#include "sgmv_matmul_launch.h"

namespace {

using namespace sgmv::host;

sgmv_status check_inputs(const sgmv_matrix& x, const sgmv_matrix& out) {
  if (!known_dtype(x.dtype)) return fail(SGMV_ERR_INVALID_ARGUMENT, "unknown inputs dtype %d", x.dtype);
  if (!known_dtype(out.dtype)) return fail(SGMV_ERR_INVALID_ARGUMENT, "unknown output dtype %d", out.dtype);
  if (x.rows < 0 || x.cols < 1 || x.row_stride < x.cols)
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "inputs shape (%lld, %lld) with row stride %lld is invalid", (long long)x.rows,
                (long long)x.cols, (long long)x.row_stride);
  if (out.rows < 0 || out.cols < 0 || out.row_stride < out.cols)
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "output shape (%lld, %lld) with row stride %lld is invalid", (long long)out.rows,
                (long long)out.cols, (long long)out.row_stride);
  if (x.rows > INT32_MAX || out.rows > INT32_MAX)
    return fail(SGMV_ERR_UNSUPPORTED, "more than 2^31-1 rows");
  if (x.cols > INT32_MAX - 4096 || out.cols > INT32_MAX / 2 - 4096)
    return fail(SGMV_ERR_UNSUPPORTED, "more than 2^31-1 columns");
  return SGMV_OK;
}

sgmv_status check_segments(int64_t batches, int64_t max_seq_len) {
  if (batches < 0) return fail(SGMV_ERR_INVALID_ARGUMENT, "batches must be >= 0");
  if (batches > SGMV_MAX_BATCHES)
    return fail(SGMV_ERR_UNSUPPORTED, "batches %lld exceeds %d", (long long)batches,
                SGMV_MAX_BATCHES);
  if (max_seq_len < 0) return fail(SGMV_ERR_INVALID_ARGUMENT, "max_seq_len must be >= 0");
  return SGMV_OK;
}

// The kernel that p's sizes, types and alignment take, its tile and its grid.
struct Plan {
  const void* kernel;
  int rows, cols, threads;
  int64_t row_tiles, col_tiles;
};

int64_t tiles(int64_t n, int64_t of) { return (n + of - 1) / of; }

// Whether the tiled kernels' 16-byte blocks and 32-bit offsets fit: hidden a
// multiple of eight, aligned rows, and less than 2 GiB from the first to the
// last row of a tile (gathered inputs: of all of them); adapters of ranks that are
// multiples of eight, aligned and less than 2 GiB each.
bool tiled_fits(const sgmv::MatmulParams& p) {
  const int64_t most = int64_t(1) << 31, rows = 256;
  for (int i = 0; i < p.num_slices; ++i)
    if (p.K % 8 != 0 || !aligned16(p.s[i].b) || p.s[i].n * p.K * 2 >= most) return false;
  return p.H % 8 == 0 && aligned16(p.x) && aligned16(p.w) && p.x_row_bytes % 16 == 0 &&
         p.w_row_bytes % 16 == 0 && p.w_mat_bytes % 16 == 0 && rows * p.w_row_bytes < most && rows * p.out_row_bytes < most &&
         (p.rows ? p.X : rows) * p.x_row_bytes < most;
}

// 256 x 256 tiles, one workgroup per compute unit, or 128 x 128 tiles, two:
// whichever ends first, by the rounds of workgroups that each takes.  A round
// of large tiles is taken as 100; of medium ones as 34 with one workgroup per
// compute unit, 57 with two, and 75 past two rounds, where their twice as
// many bytes per product bind.  Measured, large and medium, bfloat16, weights
// from memory: dense, hidden 4096, 4096 columns, 4096 rows 99 and 132 us (256
// large tiles, 1024 medium ones), 2048 rows 81 and 70, 512 rows 79 and 46;
// grouped, 8 experts x 1024 rows, hidden 14336, 4096 columns 703 and 1031 us,
// 64 experts x 32 rows, hidden 2048, 2 x 1408 columns 180 and 167.  Where they
// are near each other (32 experts x 188 rows of the same, 124 and 121 us) it
// may miss by 5%.  A segment fills half of its last tile on average.
sgmv::TiledKernel pick_tiled(const sgmv::MatmulParams& p, int wd, int mode, int cus) {
  const sgmv::TiledKernel l = sgmv::matmul_tiled_large(wd, mode);
  const sgmv::TiledKernel m = sgmv::matmul_tiled_medium(wd, mode);
  auto count = [&](const sgmv::TiledKernel& k) {
    const int64_t rows = p.grouped ? (2 * p.T + p.batches * k.rows) / (2 * k.rows) : tiles(p.T, k.rows);
    return rows * tiles(p.N, k.cols);
  };
  const int64_t nl = count(l), nm = count(m);
  const int64_t tl = 100 * tiles(nl, cus);
  const int64_t tm = nm <= cus ? 34 : nm <= 4 * cus ? 57 * tiles(nm, 2 * cus) : 75 * nm / (2 * cus);
  return tl < tm ? l : m;
}

sgmv_status make_plan(const sgmv::MatmulParams& p, int wd, bool gated, Plan* plan) {
  using namespace sgmv;
  const int mode = gated ? 2 : p.grouped ? 1 : p.num_slices > 0 ? 3 : 0;
  if (tiled_fits(p)) {
    int cus = 0;
    const hipError_t e = device_compute_units(&cus);
    if (e != hipSuccess)
      return fail(SGMV_ERR_HIP, "device query failed: %s", hipGetErrorString(e));
    // The kernel for few rows where there would be few tiles: dense calls of
    // up to 32 rows (64 with adapters, whose share its waves divide), and
    // segments of up to 16 rows whose 128 x 128 tiles leave half of the compute
    // units idle.  It reads the rows again for every 16 or 32 columns, which
    // costs more than 128 x 128 tiles do once it has many workgroups of more
    // than 16 rows.  Measured, few-row kernel and 128 x 128 tiles, bfloat16,
    // hidden 4096, weights from memory, us.  Dense: 1 row, 4096 and 28672 columns
    // 10 and 37, 41 and 52; 16 rows 12 and 38, 60 and 53; 32 rows, 4096, 10240
    // and 14336 columns 15 and 38, 38 and 40, 50 and 42.  Rank 16, 32 adapters:
    // 32 rows, 6144, 14336 and 28672 columns 43 and 69, 73 and 73, 127 and 85;
    // 64 rows 50 and 74, 91 and 78, 170 and 90 (4 adapters 45 and 59, 80 and
    // 64, 150 and 76; 64 adapters of rank 64, 14336 columns 129 and 192).
    // Segments of 4 rows: 4 experts, hidden 2048, 2 x 1408 columns 17 and 23, 2
    // experts, hidden 14336, 4096 columns 49 and 125; past half of the units
    // 13 experts, 2 x 1408 columns 36 and 45, but hidden 1408, 2048 columns 24
    // and 19, 32 experts x 8 rows 54 and 36.
    const TiledKernel m = matmul_tiled_medium(wd, mode);
    const bool adapted = p.num_slices > 0;
    const TiledKernel f = p.grouped || p.T <= 16 ? matmul_skinny_16(wd, mode)
                          : p.T <= 32           ? matmul_skinny_32(wd, adapted)
                                                : matmul_skinny_64_adapted(wd);
    const int64_t used = p.batches < p.T ? p.batches : p.T;
    const bool few = p.grouped ? tiles(p.T, p.batches) <= 16 && 2 * used * tiles(p.N, m.cols) <= cus
                               : p.T <= 16 || (p.T <= (adapted ? 64 : 32) &&
                                               f.rows * tiles(p.N, f.cols) <= (adapted ? 160 : 80) * (int64_t)cus);
    const TiledKernel k = few ? f : pick_tiled(p, wd, mode, cus);
    *plan = Plan{k.kernel, k.rows, k.cols, k.threads, 0, 0};
  } else {
    *plan = Plan{matmul_generic_kernel(wd, gated), kGenericRows, kGenericCols, kThreads, 0, 0};
  }
  if (!plan->kernel) return fail(SGMV_ERR_UNSUPPORTED, "no kernel for this dtype combination");
  // Grouped: at most ceil(T / rows) + min(batches, T) row tiles.
  plan->row_tiles = tiles(p.T, plan->rows) + (p.grouped ? (p.batches < p.T ? p.batches : p.T) : 0);
  plan->col_tiles = tiles(p.N, plan->cols);
  // A launch holds fewer than 2^32 threads: refused here, ahead of the adapters'
  // own launch (64 x 64 tiles reach it at 2^36 results).
  if (plan->row_tiles * plan->col_tiles > (int64_t)UINT32_MAX / plan->threads)
    return fail(SGMV_ERR_UNSUPPORTED, "more than 2^32-1 threads (%lld tiles of %d x %d)",
                (long long)(plan->row_tiles * plan->col_tiles), plan->rows, plan->cols);
  return SGMV_OK;
}

sgmv_status launch(const Plan& plan, sgmv::MatmulParams& p, hipStream_t stream) {
  p.row_tiles = (int32_t)plan.row_tiles;
  p.col_tiles = (int32_t)plan.col_tiles;
  p.vec_out = aligned16(p.out) && p.out_row_bytes % 16 == 0 && p.N % 8 == 0;
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(plan.kernel, dim3((unsigned)(plan.row_tiles * plan.col_tiles)),
                                       dim3((unsigned)plan.threads), args, 0, stream);
  if (e != hipSuccess) return fail(SGMV_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  g_error.clear();
  return SGMV_OK;
}

// Row stride (floats) of the projected rows of one slice in the workspace:
// whole 32-byte blocks, as the projection's vector stores want them.
int64_t projected_stride(int64_t rank) { return (rank + 7) / 8 * 8; }
int64_t projected_bytes(int64_t tokens, int64_t rank) {
  return (tokens * projected_stride(rank) * 4 + 255) / 256 * 256;
}

}  // namespace

extern "C" {

sgmv_status sgmv_lora_linear_workspace_bytes(int64_t tokens, int num_slices, int64_t rank,
                                             size_t* bytes) {
  if (!bytes) return fail(SGMV_ERR_INVALID_ARGUMENT, "bytes pointer is null");
  if (tokens < 0 || num_slices < 0 || num_slices > SGMV_MAX_SLICES || rank < 0)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "tokens, num_slices (<= %d) and rank must be >= 0",
                SGMV_MAX_SLICES);
  if (tokens > INT32_MAX || rank > SGMV_MAX_RANK)
    return fail(SGMV_ERR_UNSUPPORTED, "tokens exceed 2^31-1 or the rank %d", SGMV_MAX_RANK);
  *bytes = (size_t)(num_slices * projected_bytes(tokens, rank));
  g_error.clear();
  return SGMV_OK;
}

sgmv_status sgmv_lora_linear(sgmv_matrix inputs, sgmv_matrix weight, const void* bias,
                             const sgmv_fused_slice* slices, int num_slices, sgmv_matrix out,
                             const int64_t* b_seq_start_loc, const int64_t* seq_lens,
                             const int64_t* lora_indices, int64_t batches, int64_t max_seq_len,
                             float scale, int add_inputs, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  using namespace sgmv;
  if (num_slices < 0 || num_slices > SGMV_MAX_SLICES)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "num_slices must be in 0..%d, got %d", SGMV_MAX_SLICES,
                num_slices);
  if (num_slices > 0 && !slices) return fail(SGMV_ERR_INVALID_ARGUMENT, "slices pointer is null");
  const sgmv_matrix& x = inputs;
  sgmv_status st = check_inputs(x, out);
  if (st != SGMV_OK) return st;
  if (out.rows != x.rows)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "output must have the inputs' %lld rows",
                (long long)x.rows);
  if (!known_dtype(weight.dtype))
    return fail(SGMV_ERR_INVALID_ARGUMENT, "unknown weight dtype %d", weight.dtype);
  if (weight.dtype == SGMV_F32 || x.dtype != weight.dtype)
    return fail(SGMV_ERR_UNSUPPORTED, "inputs and weight must share one 16-bit dtype");
  if (weight.cols != x.cols || weight.rows != out.cols || weight.row_stride < weight.cols)
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "weight (%lld, %lld) with row stride %lld must be (output columns %lld, hidden %lld)",
                (long long)weight.rows, (long long)weight.cols, (long long)weight.row_stride,
                (long long)out.cols, (long long)x.cols);
  st = check_segments(batches, max_seq_len);
  if (st != SGMV_OK) return st;

  int64_t K = 0, L = 0;
  for (int i = 0; i < num_slices; ++i) {
    const sgmv_fused_slice& s = slices[i];
    if (!known_dtype(s.lora_a.dtype) || !known_dtype(s.lora_b.dtype))
      return fail(SGMV_ERR_INVALID_ARGUMENT, "slice %d: unknown dtype", i);
    if (s.lora_a.dtype != weight.dtype || s.lora_b.dtype != weight.dtype)
      return fail(SGMV_ERR_UNSUPPORTED, "slice %d: lora_a and lora_b must have the weight's dtype",
                  i);
    if (s.lora_a.num < 0 || s.lora_a.rows < 1 || s.lora_a.cols != x.cols)
      return fail(SGMV_ERR_INVALID_ARGUMENT, "slice %d: lora_a must be (lora_num, rank, %lld)", i,
                  (long long)x.cols);
    if (s.lora_b.num != s.lora_a.num || s.lora_b.cols != s.lora_a.rows || s.lora_b.rows < 0)
      return fail(SGMV_ERR_INVALID_ARGUMENT,
                  "slice %d: lora_b must be (lora_num, slice_size, rank) with lora_a's "
                  "lora_num and rank", i);
    if (s.slice_offset < 0 || s.slice_offset > out.cols - s.lora_b.rows)
      return fail(SGMV_ERR_INVALID_ARGUMENT,
                  "slice %d: window [%lld, %lld) is outside the %lld output columns", i,
                  (long long)s.slice_offset, (long long)(s.slice_offset + s.lora_b.rows),
                  (long long)out.cols);
    if (i == 0) {
      K = s.lora_a.rows;
      L = s.lora_a.num;
    } else if (s.lora_a.rows != K || s.lora_a.num != L) {
      return fail(SGMV_ERR_INVALID_ARGUMENT, "slice %d: rank and lora_num must match slice 0", i);
    }
    for (int q = 0; q < i; ++q) {
      const sgmv_fused_slice& o = slices[q];
      if (s.lora_b.rows > 0 && o.lora_b.rows > 0 &&
          s.slice_offset < o.slice_offset + o.lora_b.rows &&
          o.slice_offset < s.slice_offset + s.lora_b.rows)
        return fail(SGMV_ERR_INVALID_ARGUMENT, "slices %d and %d overlap", q, i);
    }
  }
  if (L > INT32_MAX) return fail(SGMV_ERR_UNSUPPORTED, "lora_num exceeds 2^31-1");
  if (K > SGMV_MAX_RANK)
    return fail(SGMV_ERR_UNSUPPORTED, "rank %lld exceeds %d", (long long)K, SGMV_MAX_RANK);
  if (x.rows == 0 || out.cols == 0) {
    g_error.clear();
    return SGMV_OK;  // nothing to do
  }
  if (!x.data || !out.data || !weight.data)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "null data pointer");
  const bool adapters = num_slices > 0 && batches > 0 && L > 0;
  if (adapters) {
    if (!b_seq_start_loc || !seq_lens || !lora_indices)
      return fail(SGMV_ERR_INVALID_ARGUMENT, "segment metadata pointer is null");
    for (int i = 0; i < num_slices; ++i)
      if (!slices[i].lora_a.data || (slices[i].lora_b.rows > 0 && !slices[i].lora_b.data))
        return fail(SGMV_ERR_INVALID_ARGUMENT, "slice %d: null data pointer", i);
    const size_t need = (size_t)(num_slices * projected_bytes(x.rows, K));
    if (!workspace || workspace_bytes < need || !aligned16(workspace))
      return fail(SGMV_ERR_INVALID_ARGUMENT,
                  "workspace must be 16-byte aligned and hold %zu bytes, got %zu", need,
                  workspace ? workspace_bytes : (size_t)0);
  }

  MatmulParams p{};
  p.x = x.data;
  p.w = weight.data;
  p.bias = bias;
  p.out = out.data;
  p.x_row_bytes = x.row_stride * 2;
  p.w_row_bytes = weight.row_stride * 2;
  p.out_row_bytes = out.row_stride * elem_bytes(out.dtype);
  p.T = p.X = x.rows;
  p.H = (int32_t)x.cols;
  p.N = (int32_t)out.cols;
  p.out_dtype = out.dtype;
  p.add = add_inputs != 0;
  sgmv_shrink_slice down[SGMV_MAX_SLICES];
  if (adapters) {
    p.start = b_seq_start_loc;
    p.lens = seq_lens;
    p.idx = lora_indices;
    p.batches = (int32_t)batches;
    p.L = (int32_t)L;
    p.K = (int32_t)K;
    p.v_stride = (int32_t)projected_stride(K);
    for (int i = 0; i < num_slices; ++i) {
      if (slices[i].lora_b.rows == 0) continue;  // no column (and maybe no data)
      const int j = p.num_slices++;
      float* v = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                          j * projected_bytes(x.rows, K));
      down[j].lora_a = slices[i].lora_a;
      down[j].out = sgmv_matrix{v, SGMV_F32, x.rows, K, p.v_stride};
      p.s[j] = AdapterDesc{slices[i].lora_b.data, v, slices[i].lora_b.rows, slices[i].slice_offset};
    }
  }
  Plan plan;
  st = make_plan(p, weight.dtype, false, &plan);
  if (st != SGMV_OK) return st;
  if (p.num_slices > 0) {
    // First the projections onto the adapters' rank, kept in float32.
    st = sgmv_shrink_multi_slice(inputs, down, p.num_slices, b_seq_start_loc, seq_lens, lora_indices,
                                 batches, max_seq_len, scale, nullptr, 0, stream);
    if (st != SGMV_OK) return st;
  }
  return launch(plan, p, stream);
}

sgmv_status sgmv_grouped_gemm(sgmv_matrix inputs, sgmv_stack weights, sgmv_matrix out,
                              const int64_t* row_indices, const int64_t* b_seq_start_loc,
                              const int64_t* seq_lens, const int64_t* expert_indices,
                              int64_t batches, int64_t max_seq_len, int gated,
                              hipStream_t stream) {
  using namespace sgmv;
  const sgmv_matrix& x = inputs;
  sgmv_status st = check_inputs(x, out);
  if (st != SGMV_OK) return st;
  if (!known_dtype(weights.dtype))
    return fail(SGMV_ERR_INVALID_ARGUMENT, "unknown weights dtype %d", weights.dtype);
  if (weights.dtype == SGMV_F32 || x.dtype != weights.dtype)
    return fail(SGMV_ERR_UNSUPPORTED, "inputs and weights must share one 16-bit dtype");
  if (weights.num < 0 || weights.cols != x.cols ||
      weights.rows != (gated ? 2 * out.cols : out.cols))
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "weights must be (experts, %lld, %lld), got (%lld, %lld, %lld)",
                (long long)(gated ? 2 * out.cols : out.cols), (long long)x.cols,
                (long long)weights.num, (long long)weights.rows, (long long)weights.cols);
  if (!row_indices && x.rows != out.rows)
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "output must have the inputs' %lld rows without row_indices", (long long)x.rows);
  if (weights.num > INT32_MAX) return fail(SGMV_ERR_UNSUPPORTED, "experts exceed 2^31-1");
  st = check_segments(batches, max_seq_len);
  if (st != SGMV_OK) return st;
  if (batches == 0 || out.rows == 0 || out.cols == 0 || weights.num == 0) {
    g_error.clear();
    return SGMV_OK;  // nothing to do
  }
  if ((!x.data && x.rows > 0) || !out.data || !weights.data)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "null data pointer");
  if (!b_seq_start_loc || !seq_lens)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "segment metadata pointer is null");

  MatmulParams p{};
  p.x = x.data;
  p.w = weights.data;
  p.out = out.data;
  p.start = b_seq_start_loc;
  p.lens = seq_lens;
  p.idx = expert_indices;
  p.rows = row_indices;
  p.x_row_bytes = x.row_stride * 2;
  p.w_row_bytes = weights.cols * 2;
  p.w_mat_bytes = weights.rows * weights.cols * 2;
  p.out_row_bytes = out.row_stride * elem_bytes(out.dtype);
  p.T = out.rows;
  p.X = x.rows;
  p.H = (int32_t)x.cols;
  p.N = (int32_t)out.cols;
  p.batches = (int32_t)batches;
  p.L = (int32_t)weights.num;
  p.grouped = 1;
  p.out_dtype = out.dtype;
  Plan plan;
  st = make_plan(p, weights.dtype, gated != 0, &plan);
  if (st != SGMV_OK) return st;
  return launch(plan, p, stream);
}

}  // extern "C"
