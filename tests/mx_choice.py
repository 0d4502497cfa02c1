"""Which kernels the products with microscaled weights launch for given sizes:
their entry points compiled for the host, with kernels that print their names."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <string>
#include <vector>
#include "sgmv_host.cpp"
#include "sgmv_matmul_api.cpp"
#include "sgmv_mx_api.cpp"

static const char* const kModes[] = {"dense", "grouped", "gated", "adapted"};
static const void* name(const std::string& s) { return strdup(s.c_str()); }
static std::string of(const char* what, int mode) { return std::string(what) + "_" + kModes[mode]; }

namespace sgmv {
TiledKernel mx_tiled_large(int, int mode) { return {name(of("large", mode)), 256, mode == 2 ? 128 : 256, 256}; }
TiledKernel mx_tiled_medium(int, int mode) { return {name(of("medium", mode)), 128, mode == 2 ? 64 : 128, 256}; }
TiledKernel mx_skinny(int, int mode, int rows, int64_t) {
  return {name(of("few", mode) + std::to_string(rows)), rows, 16, 64 * kMxSkinnyWaves};
}
const void* matmul_generic_kernel(int, bool gated, bool mx) { return name(gated ? "generic_gated" : "generic"); }
TiledKernel matmul_tiled_large(int, int) { abort(); }
TiledKernel matmul_tiled_medium(int, int) { abort(); }
TiledKernel matmul_skinny_16(int, int) { abort(); }
TiledKernel matmul_skinny_32(int, bool) { abort(); }
TiledKernel matmul_skinny_64_adapted(int) { abort(); }
const void* mx_project_kernel(int) { return name("project"); }
const void* mx_quantize_kernel(int) { return name("quantize"); }
const void* mx_dequantize_kernel(int) { return name("dequantize"); }
}  // namespace sgmv

extern "C" sgmv_status sgmv_shrink_multi_slice(sgmv_matrix, const sgmv_shrink_slice*, int, const int64_t*, const int64_t*,
                                               const int64_t*, int64_t, int64_t, float, void*, size_t, hipStream_t) {
  printf("shrink ");
  return SGMV_OK;
}
extern "C" {
hipError_t hipLaunchKernel(const void* f, dim3, dim3, void**, size_t, hipStream_t) {
  printf("%s ", (const char*)f);
  return hipSuccess;
}
const char* hipGetErrorString(hipError_t) { return "error"; }
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* n, hipDeviceAttribute_t, int) { *n = 256; return hipSuccess; }
hipError_t hipOccupancyMaxActiveBlocksPerMultiprocessor(int*, const void*, int, size_t) { abort(); }
}

int main() {
  void* const p = (void*)0x10000;
  const size_t any = size_t(1) << 60;
  char kind;
  long long T, H, K, L, B, X, gated, stride, out_stride, n;
  while (scanf(" %c %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", &kind, &T, &H, &K, &L, &B, &X, &gated, &stride, &out_stride, &n) == 11) {
    std::vector<long long> w(n);
    long long N = 0;
    for (auto& v : w) { if (scanf("%lld", &v) != 1) return 1; N += v; }
    const int64_t G = (H + 127) / 128;
    const sgmv_matrix x{p, SGMV_BF16, kind == 'l' || !X ? T : X, H, stride}, out{p, SGMV_BF16, T, N, out_stride ? out_stride : N};
    sgmv_status st;
    if (kind == 'l') {
      std::vector<sgmv_fused_slice> s;
      long long at = 0;
      for (long long v : w) {
        s.push_back(sgmv_fused_slice{{p, SGMV_BF16, L, K, H}, {p, SGMV_BF16, L, v, K}, at});
        at += v;
      }
      st = sgmv_mx_lora_linear(x, sgmv_mx_stack{p, p, 1, N, H, 64 * G, 4 * G}, nullptr, s.data(), K ? (int)n : 0, out, (int64_t*)p,
                               (int64_t*)p, (int64_t*)p, B, T, 1.f, 0, p, any, nullptr);
    } else {
      st = sgmv_mx_grouped_gemm(x, sgmv_mx_stack{p, p, L, gated ? 2 * N : N, H, 64 * G, 4 * G}, out, X ? (int64_t*)p : nullptr, (int64_t*)p,
                                (int64_t*)p, nullptr, B, T, (int)gated, p, any, nullptr);
    }
    printf("%s\n", st == SGMV_OK ? "" : sgmv::host::g_error.c_str());
  }
}
"""


def linear(T, H, widths, K=0, L=0, B=0, stride=0, out_stride=0):
    """A call of sgmv_mx_lora_linear (K 0: without adapters) with the inputs' and results' row strides (0: their columns)."""
    return f"l {T} {H} {K} {L} {B} 0 0 {stride or H} {out_stride} {len(widths)} {' '.join(map(str, widths))}"


def grouped(T, H, N, experts, gated=False, gathered=0, stride=0, out_stride=0):
    """A call of sgmv_mx_grouped_gemm over T rows of results, gathered from `gathered` input rows (0: none)."""
    return f"g {T} {H} 0 {experts} {experts} {gathered} {int(gated)} {stride or H} {out_stride} 1 {N}"


def launches(tmp_path, calls):
    """The kernels of each of the calls, in order."""
    src, exe = tmp_path / "choice.cpp", str(tmp_path / "choice")
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{os.path.join(ROOT, 'include')}",
                    f"-I{os.path.join(ROOT, 'segmented_gather_gemm_amd', 'csrc')}", str(src), "-o", exe], check=True)
    out = subprocess.run([exe], input="\n".join(calls), check=True, capture_output=True, text=True).stdout
    return [line.split() for line in out.splitlines()]
