// sgmv_matmul_api.cpp -- libsgmv C entry points of the shared projection
// with the adapters of many requests (sgmv_lora_linear) and of the products
// grouped by expert (sgmv_grouped_gemm), and of both with microscaled 4-bit
// weights (sgmv_mx_*): argument checks, kernel choice, grid
// sizing and launch.  No allocation, no synchronisation, no device-to-host
// traffic.
#include <stdint.h>

#include "sgmv.h"
#include "sgmv_host.h"
#include "sgmv_limits.h"
#include "sgmv_matmul_launch.h"
#include "sgmv_mx_host.h"
#include "sgmv_mx_launch.h"

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
  bool quantises = false;  // microscaled: the kernel takes the 16-bit inputs
  int strips = 0;          // microscaled, few rows: workgroups wanted
};

int64_t tiles(int64_t n, int64_t of) { return (n + of - 1) / of; }

// Whether the tiled kernels' 16-byte blocks and 32-bit offsets fit: hidden a
// multiple of eight, aligned rows, and less than 2 GiB from the first to the
// last row of a tile (gathered inputs: of all of them); adapters of ranks that are
// multiples of eight, aligned and less than 2 GiB each.  Microscaled rows are
// aligned as they are; their scales have the same bounds on far shorter rows,
// but whatever stride a caller gives them.
bool tiled_fits(const sgmv::MatmulParams& p) {
  const int64_t most = int64_t(1) << 31, rows = 256;
  for (int i = 0; i < p.num_slices; ++i)
    if (p.K % 8 != 0 || !aligned16(p.s[i].b) || p.s[i].n * p.K * 2 >= most) return false;
  return p.H % 8 == 0 && aligned16(p.x) && aligned16(p.w) && p.x_row_bytes % 16 == 0 &&
         p.w_row_bytes % 16 == 0 && p.w_mat_bytes % 16 == 0 && rows * p.w_row_bytes < most && rows * p.out_row_bytes < most &&
         (p.rows ? p.X : rows) * p.x_row_bytes < most && rows * p.ws_row_bytes < most;
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

// The same for microscaled operands, in tenths of a microsecond, by the steps
// of 256 along the contraction: a round of large tiles takes 13 us and 1.84 a
// step (6 and 1.6 with few of them), medium ones 6 and 0.75 a step with one workgroup
// per compute unit, else 3.5 and for each round of two 4.5 and 1.25 a step (1.35
// where many rounds bind at the L2); adapters add 13 and 5.5 us a round.  Measured,
// large and medium, us, 4096 columns: hidden 2048, 512, 2048 and 4096 rows 21 and
// 11, 24 and 17, 28 and 30; hidden 4096, 512, 2048 and 4096 rows 32 and 16, 36 and 28,
// 43 and 49; hidden 8192, 2048 rows 60 and 46; 2048 rows with 16 adapters 49 and 33;
// 2501 rows, hidden 2056, 5000 columns, float32 results 55 and 48; 64 experts of
// 94 rows 83 and 69; 8 of 128 rows, hidden 4096, 2 x 14336 columns 165 and 172.
sgmv::TiledKernel pick_mx_tiled(const sgmv::MatmulParams& p, int wd, int mode, int cus) {
  const sgmv::TiledKernel l = sgmv::mx_tiled_large(wd, mode);
  const sgmv::TiledKernel m = sgmv::mx_tiled_medium(wd, mode);
  auto count = [&](const sgmv::TiledKernel& k) {
    const int64_t rows = p.grouped ? (2 * p.T + p.batches * k.rows) / (2 * k.rows) : tiles(p.T, k.rows);
    return (double)(rows > 0 ? rows : 1) * tiles(p.N, k.cols) / cus;
  };
  const double steps = tiles(p.H, 64), nl = count(l), nm = count(m) / 2;
  const double full = (double)(int64_t)nl, part = nl - full;
  const double adapted = p.num_slices > 0 ? 1 : 0;
  const double tl = full * (130 + 18.4 * steps + 130 * adapted) +
                    (part > 0 ? 60 + 16 * steps + part * (70 + 2.4 * steps + 130 * adapted) : 0);
  const double tm = nm <= 0.5 ? 60 + 7.5 * steps + 55 * adapted
                              : 35 + (nm < 1 ? 1 : nm) * (45 + (nm > 4 ? 13.5 : 12.5) * steps + 55 * adapted);
  return tl < tm ? l : m;
}

// The kernel for few rows of a microscaled call (x: its 16-bit inputs), or none;
// *quantises: whether it does that with the inputs itself (16 rows).
// Measured, us, few-row kernel and 128 x 128 tiles (which take a quantisation
// of 3-4 besides), bfloat16, hidden 4096.  Dense: one row, 4096 and 28672
// columns 6.8 and 12.5, 15.4 and 16.5; 16 rows 8.7 and 12.6, 17.7 and 16.1; 64 rows,
// 4096, 8192 and 28672 columns 9.0 and 13.4, 12.6 and 13.8, 22.9 and 19.9.
// Rank 16, 32 adapters, 6144 columns: 64 rows 12.7 and 36.9, 128 rows 18.8 and 52.4,
// 256 rows 29.4 and 50.3; 4 adapters 14.0 and 19.0, 19.5 and 20.9, 30.6 and 18.6;
// rank 64, 28672 columns 73 and 90, 131 and 112, 232 and 119.  Experts: 16 used
// by a row each, hidden 2048, 2 x 1408 columns 14.5 and 14.9, 64 of 4 rows 46.9 and
// 50.9, of 16 rows 66 and 54; hidden 14336, 4096 columns, 8 of one row 124 and 54
// (the inputs are quantised again for every tile).  Up to 16 rows take it whatever
// their adapters.  Both with all of a call's launches, ranks 16, 64, 128 and 256, 4096
// columns: one row 10.5 and 20.0, 11.9 and 21.1, 12.4 and 23.4, 14.3 and 28.1, 16 rows of as
// many adapters 13.7 and 28.9, 17.1 and 54.7, 20.6 and 86.9, 27.4 and 150.5; 28672 columns:
// one row 25.6 and 25.4, 30.0 and 26.2, 36.8 and 28.8, 51.4 and 34.2, 16 rows of one adapter
// 29.5 and 28.8, 38.8 and 28.6, 50.2 and 31.4, 72.6 and 38.9, of 16 adapters 31.3 and 35.7,
// 42.9 and 56.6, 59.0 and 89.5, 93.5 and 154.6: it loses where a wide projection's rows
// share few adapters of rank 64 and more.
sgmv::TiledKernel mx_few(const sgmv::MatmulParams& p, const sgmv_matrix& x, int mode, int cus,
                         bool* quantises) {
  using namespace sgmv;
  const bool fits = x.cols % 8 == 0 && aligned16(x.data) && x.row_stride % 8 == 0 &&
                    (p.rows ? p.X : 256) * x.row_stride * 2 < int64_t(1) << 31;
  const int64_t groups = p.H / 32;
  *quantises = true;
  if (p.grouped) {
    // Few experts of up to 16 rows: 128 x 128 tiles read more experts' weights faster.
    const int64_t used = p.batches < p.T ? p.batches : p.T;
    if (fits && tiles(p.T, p.batches) <= 16 && used * tiles(p.N, 16) <= 6 * cus && groups <= 64)
      return mx_skinny(x.dtype, mode, 16, groups);
    return TiledKernel{};
  }
  if (fits && p.T <= 16) return mx_skinny(x.dtype, mode, 16, groups);
  *quantises = false;
  // Tiles of 16 columns a compute unit takes, with rows in 32s and in 64s.
  const int64_t by32 = tiles(p.T, 32) * tiles(p.N, 16) / cus, by64 = tiles(p.T, 64) * tiles(p.N, 16) / cus;
  bool few = p.T <= 32 || (p.T <= 64 && by64 <= 3);
  if (p.num_slices > 0 && p.T <= 256) {
    // A few-row workgroup's tile costs 2 us and 0.12 a rank; 128 x 128 tiles a
    // round of 14 us and 3 for every 64 of their adapters' ranks (at least 8 each).
    const int64_t row_tiles = tiles(p.T, 128), most = p.batches < p.T ? p.batches : p.T;
    const int64_t near = tiles(most, row_tiles), seen = near < p.L ? near : p.L;  // adapters of a row tile
    const int64_t rounds = tiles(seen * (p.K < 8 ? 8 : p.K), 64);
    const int64_t launch = tiles(row_tiles * tiles(p.N, 128), 2 * cus);
    few = 800 + by64 * (200 + 12 * p.K) <= launch * 1400 + rounds * 300;
  }
  if (!few) return TiledKernel{};
  return mx_skinny(x.dtype, mode, p.T <= 32 || by32 <= 3 ? 32 : 64, groups);
}

sgmv_status make_plan(const sgmv::MatmulParams& p, int wd, bool gated, Plan* plan,
                      const sgmv_matrix* mx_inputs = nullptr) {
  using namespace sgmv;
  const int mode = gated ? 2 : p.grouped ? 1 : p.num_slices > 0 ? 3 : 0;
  *plan = Plan{};
  if (mx_inputs && tiled_fits(p)) {
    int cus = 0;
    const hipError_t e = device_compute_units(&cus);
    if (e != hipSuccess)
      return fail(SGMV_ERR_HIP, "device query failed: %s", hipGetErrorString(e));
    bool quantises = false;
    TiledKernel k = mx_few(p, *mx_inputs, mode, cus, &quantises);
    const bool few = k.kernel != nullptr;
    if (!few) k = pick_mx_tiled(p, wd, mode, cus);
    // Grouped: the row tiles below are a bound, about twice those there are.
    *plan = Plan{k.kernel, k.rows, k.cols, k.threads, 0, 0, few && quantises, !few ? 0 : p.grouped ? 2 * cus : cus};
  } else if (tiled_fits(p)) {
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
    *plan = Plan{matmul_generic_kernel(wd, gated, p.ws != nullptr), kGenericRows, kGenericCols, kThreads, 0, 0};
  }
  if (!plan->kernel) return fail(SGMV_ERR_UNSUPPORTED, "no kernel for this dtype combination");
  // Grouped: at most ceil(T / rows) + min(batches, T) row tiles.
  plan->row_tiles = tiles(p.T, plan->rows) + (p.grouped ? (p.batches < p.T ? p.batches : p.T) : 0);
  plan->col_tiles = tiles(p.N, plan->cols);
  // The few-row kernel on microscaled weights walks over its column tiles: one
  // workgroup a compute unit (two: 28672 columns and 16 rows 25.1 against 17.8
  // us, one row 17.7 against 15.6), each with (nearly) as many of them.
  if (plan->strips > 0) {
    const int64_t strips = plan->strips / plan->row_tiles > 0 ? plan->strips / plan->row_tiles : 1;
    plan->col_tiles = tiles(plan->col_tiles, tiles(plan->col_tiles, strips));
  }
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


// The adapter slices of a projection of `x` (weights of dtype wd) into `out`:
// their rank and number of adapters.
sgmv_status check_slices(const sgmv_fused_slice* slices, int num_slices, const sgmv_matrix& x,
                         const sgmv_matrix& out, int wd, int64_t* rank, int64_t* lora_num) {
  int64_t K = 0, L = 0;
  for (int i = 0; i < num_slices; ++i) {
    const sgmv_fused_slice& s = slices[i];
    if (!known_dtype(s.lora_a.dtype) || !known_dtype(s.lora_b.dtype))
      return fail(SGMV_ERR_INVALID_ARGUMENT, "slice %d: unknown dtype", i);
    if (s.lora_a.dtype != wd || s.lora_b.dtype != wd)
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
  *rank = K;
  *lora_num = L;
  return SGMV_OK;
}

sgmv_status check_num_slices(const sgmv_fused_slice* slices, int num_slices) {
  if (num_slices < 0 || num_slices > SGMV_MAX_SLICES)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "num_slices must be in 0..%d, got %d", SGMV_MAX_SLICES,
                num_slices);
  if (num_slices > 0 && !slices) return fail(SGMV_ERR_INVALID_ARGUMENT, "slices pointer is null");
  return SGMV_OK;
}

// The pointers that adapters need.
sgmv_status check_adapters(const sgmv_fused_slice* slices, int num_slices, const int64_t* start,
                           const int64_t* lens, const int64_t* idx) {
  if (!start || !lens || !idx)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "segment metadata pointer is null");
  for (int i = 0; i < num_slices; ++i)
    if (!slices[i].lora_a.data || (slices[i].lora_b.rows > 0 && !slices[i].lora_b.data))
      return fail(SGMV_ERR_INVALID_ARGUMENT, "slice %d: null data pointer", i);
  return SGMV_OK;
}

sgmv_status check_workspace(const void* workspace, size_t workspace_bytes, size_t need) {
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "workspace must be 16-byte aligned and hold %zu bytes, got %zu", need,
                workspace ? workspace_bytes : (size_t)0);
  return SGMV_OK;
}

// The adapters as p's further factors and as the slices of their projection
// (down), whose rows lie in `workspace`.
void attach_adapters(sgmv::MatmulParams& p, const sgmv_fused_slice* slices, int num_slices, int64_t K,
                     int64_t L, const int64_t* start, const int64_t* lens, const int64_t* idx,
                     int64_t batches, void* workspace, sgmv_shrink_slice* down) {
  p.start = start;
  p.lens = lens;
  p.idx = idx;
  p.batches = (int32_t)batches;
  p.L = (int32_t)L;
  p.K = (int32_t)K;
  p.v_stride = (int32_t)projected_stride(K);
  for (int i = 0; i < num_slices; ++i) {
    if (slices[i].lora_b.rows == 0) continue;  // no column (and maybe no data)
    const int j = p.num_slices++;
    float* v = reinterpret_cast<float*>(static_cast<char*>(workspace) + j * projected_bytes(p.T, K));
    down[j].lora_a = slices[i].lora_a;
    down[j].out = sgmv_matrix{v, SGMV_F32, p.T, K, p.v_stride};
    p.s[j] = sgmv::AdapterDesc{slices[i].lora_b.data, v, slices[i].lora_b.rows, slices[i].slice_offset};
  }
}

// Rows quantised in a workspace: their codes, then their scales.
struct Quantised {
  int64_t code_stride, scale_stride, scales_at, bytes;
};
Quantised quantised(int64_t rows, int64_t cols) {
  const int64_t g = sgmv::limits::mx_groups(cols);
  Quantised q;
  q.code_stride = g * sgmv::limits::kMxCodeBytes;
  q.scale_stride = g * sgmv::limits::kMxScaleBytes;
  q.scales_at = (rows * q.code_stride + 255) / 256 * 256;
  q.bytes = q.scales_at + (rows * q.scale_stride + 255) / 256 * 256;
  return q;
}

// Rows and columns that a workspace is sized for: as many as the quantisation
// of a call's inputs takes.
sgmv_status check_quantised(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "rows must be >= 0 and hidden >= 1");
  if (cols > INT32_MAX - 4096 || rows > sgmv::kMxMaxItems / sgmv::limits::mx_groups(cols))
    return fail(SGMV_ERR_UNSUPPORTED, "more than 2^28 groups of 128 inputs");
  return SGMV_OK;
}

// p's factors as microscaled rows: the weights' (checked) and the inputs',
// which lie quantised in `workspace`.
void attach_mx(sgmv::MatmulParams& p, const sgmv_mx_stack& w, const Quantised& q, void* workspace) {
  p.x = workspace;
  p.xs = static_cast<char*>(workspace) + q.scales_at;
  p.x_row_bytes = q.code_stride;
  p.xs_row_bytes = q.scale_stride;
  p.w = w.codes;
  p.ws = w.scales;
  p.w_row_bytes = w.code_stride;
  p.ws_row_bytes = w.scale_stride;
  p.w_mat_bytes = w.rows * w.code_stride;
  p.H = (int32_t)(q.code_stride / 2);
}

// The inputs into the workspace, or handed to the kernel that quantises them.
sgmv_status quantise_inputs(sgmv::MatmulParams& p, const Plan& plan, const sgmv_matrix& x,
                            const Quantised& q, void* workspace, hipStream_t stream) {
  if (!plan.quantises)
    return sgmv::launch_mx_quantize(x, workspace, q.code_stride,
                                    static_cast<char*>(workspace) + q.scales_at, q.scale_stride, stream);
  p.x = x.data;
  p.x_row_bytes = x.row_stride * 2;
  p.mx_hidden = (int32_t)x.cols;
  return SGMV_OK;
}

// Whether the adapters' projections of a call run token by token: for few rows
// of inputs and lora_A rows (64 MiB of them with each token's read for itself).
bool projects_by_token(const sgmv::MatmulParams& p, const sgmv_shrink_slice* down, const sgmv_matrix& x) {
  if (x.cols % 8 != 0 || !aligned16(x.data) || x.row_stride % 8 != 0 || p.T > 64 ||
      p.T * p.num_slices * p.K * x.cols * 2 > int64_t(64) << 20)
    return false;
  for (int i = 0; i < p.num_slices; ++i)
    if (!aligned16(down[i].lora_a.data)) return false;
  return true;
}

// Whether the few-row kernel's workgroups each do all of these projections, which saves a launch.
// Measured, us a call, that and a launch of their own, hidden 4096: rank 16, 4096
// columns, one token 11.7 and 13.6, two 11.5 and 13.5, four 16.5 and 13.6; QKV,
// one token 14.9 and 17.3, two 18.2 and 17.3; rank 64 16.6 and 13.7; hidden
// 14336, rank 16 22.7 and 25.9.
bool projects_itself(const sgmv::MatmulParams& p, const Plan& plan, const sgmv_matrix& x) {
  const int64_t rows = p.T * p.num_slices * p.K;
  return plan.quantises && rows <= sgmv::kMxProjectMost && rows * x.cols <= 1 << 18;
}

// Those projections and, unless the kernel does that itself, the inputs' codes and scales.
sgmv_status project_by_token(sgmv::MatmulParams& p, const Plan& plan, const sgmv_shrink_slice* down,
                             const sgmv_matrix& x, const Quantised& q, void* workspace, float scale,
                             hipStream_t stream) {
  using namespace sgmv;
  MxProjectParams m{};
  m.x = x.data;
  m.x_row_bytes = x.row_stride * 2;
  if (plan.quantises) {
    quantise_inputs(p, plan, x, q, workspace, stream);
  } else {
    m.codes = workspace;
    m.scales = static_cast<char*>(workspace) + q.scales_at;
  }
  m.code_stride = q.code_stride;
  m.scale_stride = q.scale_stride;
  m.start = p.start;
  m.lens = p.lens;
  m.idx = p.idx;
  m.T = p.T;
  m.H = (int32_t)x.cols;
  m.K = p.K;
  m.L = p.L;
  m.batches = p.batches;
  m.parts = (p.K + kMxProjectRows - 1) / kMxProjectRows;
  m.v_stride = p.v_stride;
  m.scale = scale;
  for (int i = 0; i < p.num_slices; ++i) {
    m.a[i] = down[i].lora_a.data;
    m.v[i] = static_cast<float*>(down[i].out.data);
  }
  void* args[] = {&m};
  const hipError_t e = hipLaunchKernel(mx_project_kernel(x.dtype),
                                       dim3((unsigned)(m.parts * p.num_slices), (unsigned)p.T),
                                       dim3(64 * kMxProjectWaves), args, 0, stream);
  if (e != hipSuccess) return fail(SGMV_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return SGMV_OK;
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
  const sgmv_matrix& x = inputs;
  sgmv_status st = check_num_slices(slices, num_slices);
  if (st != SGMV_OK) return st;
  st = check_inputs(x, out);
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
  st = check_slices(slices, num_slices, x, out, weight.dtype, &K, &L);
  if (st != SGMV_OK) return st;
  if (x.rows == 0 || out.cols == 0) {
    g_error.clear();
    return SGMV_OK;  // nothing to do
  }
  if (!x.data || !out.data || !weight.data)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "null data pointer");
  const bool adapters = num_slices > 0 && batches > 0 && L > 0;
  if (adapters) {
    st = check_adapters(slices, num_slices, b_seq_start_loc, seq_lens, lora_indices);
    if (st != SGMV_OK) return st;
    st = check_workspace(workspace, workspace_bytes, (size_t)(num_slices * projected_bytes(x.rows, K)));
    if (st != SGMV_OK) return st;
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
  if (adapters)
    attach_adapters(p, slices, num_slices, K, L, b_seq_start_loc, seq_lens, lora_indices, batches,
                    workspace, down);
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

sgmv_status sgmv_mx_lora_linear_workspace_bytes(int64_t tokens, int64_t hidden, int num_slices,
                                                int64_t rank, size_t* bytes) {
  size_t adapters = 0;
  sgmv_status st = sgmv_lora_linear_workspace_bytes(tokens, num_slices, rank, bytes ? &adapters : nullptr);
  if (st != SGMV_OK) return st;
  st = check_quantised(tokens, hidden);
  if (st != SGMV_OK) return st;
  *bytes = (size_t)quantised(tokens, hidden).bytes + adapters;
  g_error.clear();
  return SGMV_OK;
}

sgmv_status sgmv_mx_lora_linear(sgmv_matrix inputs, sgmv_mx_stack weight, const void* bias,
                                const sgmv_fused_slice* slices, int num_slices, sgmv_matrix out,
                                const int64_t* b_seq_start_loc, const int64_t* seq_lens,
                                const int64_t* lora_indices, int64_t batches, int64_t max_seq_len,
                                float scale, int add_inputs, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  using namespace sgmv;
  const sgmv_matrix& x = inputs;
  sgmv_status st = check_num_slices(slices, num_slices);
  if (st != SGMV_OK) return st;
  st = check_inputs(x, out);
  if (st != SGMV_OK) return st;
  if (out.rows != x.rows)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "output must have the inputs' %lld rows",
                (long long)x.rows);
  if (x.dtype == SGMV_F32) return fail(SGMV_ERR_UNSUPPORTED, "inputs must have a 16-bit dtype");
  st = check_mx(weight, x.cols, "weight");
  if (st != SGMV_OK) return st;
  if (weight.num != 1 || weight.rows != out.cols)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "weight must be one matrix of %lld rows, got %lld of %lld",
                (long long)out.cols, (long long)weight.num, (long long)weight.rows);
  st = check_segments(batches, max_seq_len);
  if (st != SGMV_OK) return st;
  int64_t K = 0, L = 0;
  st = check_slices(slices, num_slices, x, out, x.dtype, &K, &L);
  if (st != SGMV_OK) return st;
  st = check_quantised(x.rows, x.cols);
  if (st != SGMV_OK) return st;
  if (x.rows == 0 || out.cols == 0) {
    g_error.clear();
    return SGMV_OK;  // nothing to do
  }
  if (!x.data || !out.data || !weight.codes || !weight.scales)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "null data pointer");
  const bool adapters = num_slices > 0 && batches > 0 && L > 0;
  if (adapters) {
    st = check_adapters(slices, num_slices, b_seq_start_loc, seq_lens, lora_indices);
    if (st != SGMV_OK) return st;
  }
  const Quantised q = quantised(x.rows, x.cols);
  st = check_workspace(workspace, workspace_bytes,
                       (size_t)(q.bytes + (adapters ? num_slices * projected_bytes(x.rows, K) : 0)));
  if (st != SGMV_OK) return st;

  MatmulParams p{};
  p.bias = bias;
  p.out = out.data;
  p.out_row_bytes = out.row_stride * elem_bytes(out.dtype);
  p.T = p.X = x.rows;
  p.N = (int32_t)out.cols;
  p.out_dtype = out.dtype;
  p.add = add_inputs != 0;
  attach_mx(p, weight, q, workspace);
  sgmv_shrink_slice down[SGMV_MAX_SLICES];
  if (adapters)
    attach_adapters(p, slices, num_slices, K, L, b_seq_start_loc, seq_lens, lora_indices, batches,
                    static_cast<char*>(workspace) + q.bytes, down);
  Plan plan;
  st = make_plan(p, x.dtype, false, &plan, &x);
  if (st != SGMV_OK) return st;
  if (p.num_slices > 0 && projects_by_token(p, down, x)) {
    if (projects_itself(p, plan, x)) {
      quantise_inputs(p, plan, x, q, workspace, stream);
      p.projects = 1;
      p.scale = scale;
      for (int i = 0; i < p.num_slices; ++i) p.s[i].v = static_cast<const float*>(down[i].lora_a.data);
      return launch(plan, p, stream);
    }
    st = project_by_token(p, plan, down, x, q, workspace, scale, stream);
    if (st != SGMV_OK) return st;
    return launch(plan, p, stream);
  }
  st = quantise_inputs(p, plan, x, q, workspace, stream);
  if (st != SGMV_OK) return st;
  if (p.num_slices > 0) {
    // The adapters' projections read the inputs themselves, not their 4-bit values.
    st = sgmv_shrink_multi_slice(inputs, down, p.num_slices, b_seq_start_loc, seq_lens, lora_indices,
                                 batches, max_seq_len, scale, nullptr, 0, stream);
    if (st != SGMV_OK) return st;
  }
  return launch(plan, p, stream);
}

sgmv_status sgmv_mx_grouped_gemm_workspace_bytes(int64_t input_rows, int64_t hidden, size_t* bytes) {
  if (!bytes) return fail(SGMV_ERR_INVALID_ARGUMENT, "bytes pointer is null");
  const sgmv_status st = check_quantised(input_rows, hidden);
  if (st != SGMV_OK) return st;
  *bytes = (size_t)quantised(input_rows, hidden).bytes;
  g_error.clear();
  return SGMV_OK;
}

sgmv_status sgmv_mx_grouped_gemm(sgmv_matrix inputs, sgmv_mx_stack weights, sgmv_matrix out,
                                 const int64_t* row_indices, const int64_t* b_seq_start_loc,
                                 const int64_t* seq_lens, const int64_t* expert_indices,
                                 int64_t batches, int64_t max_seq_len, int gated, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  using namespace sgmv;
  const sgmv_matrix& x = inputs;
  sgmv_status st = check_inputs(x, out);
  if (st != SGMV_OK) return st;
  if (x.dtype == SGMV_F32) return fail(SGMV_ERR_UNSUPPORTED, "inputs must have a 16-bit dtype");
  st = check_mx(weights, x.cols, "weights");
  if (st != SGMV_OK) return st;
  if (weights.rows != (gated ? 2 * out.cols : out.cols))
    return fail(SGMV_ERR_INVALID_ARGUMENT, "weights must have %lld rows each, got %lld",
                (long long)(gated ? 2 * out.cols : out.cols), (long long)weights.rows);
  if (!row_indices && x.rows != out.rows)
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "output must have the inputs' %lld rows without row_indices", (long long)x.rows);
  if (weights.num > INT32_MAX) return fail(SGMV_ERR_UNSUPPORTED, "experts exceed 2^31-1");
  st = check_segments(batches, max_seq_len);
  if (st != SGMV_OK) return st;
  st = check_quantised(x.rows, x.cols);
  if (st != SGMV_OK) return st;
  if (batches == 0 || out.rows == 0 || out.cols == 0 || weights.num == 0) {
    g_error.clear();
    return SGMV_OK;  // nothing to do
  }
  if ((!x.data && x.rows > 0) || !out.data || !weights.codes || !weights.scales)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "null data pointer");
  if (!b_seq_start_loc || !seq_lens)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "segment metadata pointer is null");
  const Quantised q = quantised(x.rows, x.cols);
  if (x.rows > 0) {
    st = check_workspace(workspace, workspace_bytes, (size_t)q.bytes);
    if (st != SGMV_OK) return st;
  }

  MatmulParams p{};
  p.out = out.data;
  p.start = b_seq_start_loc;
  p.lens = seq_lens;
  p.idx = expert_indices;
  p.rows = row_indices;
  p.out_row_bytes = out.row_stride * elem_bytes(out.dtype);
  p.T = out.rows;
  p.X = x.rows;
  p.N = (int32_t)out.cols;
  p.batches = (int32_t)batches;
  p.L = (int32_t)weights.num;
  p.grouped = 1;
  p.out_dtype = out.dtype;
  attach_mx(p, weights, q, workspace);
  Plan plan;
  st = make_plan(p, x.dtype, gated != 0, &plan, &x);
  if (st != SGMV_OK) return st;
  if (x.rows > 0) {
    st = quantise_inputs(p, plan, x, q, workspace, stream);
    if (st != SGMV_OK) return st;
  }
  return launch(plan, p, stream);
}

}  // extern "C"
