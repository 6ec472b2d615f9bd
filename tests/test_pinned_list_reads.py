"""What the host-merged transfers of spax_tiered_gemv_pinned read of a caller's column lists:
csrc/pinned.cpp built for the host, with the runtime's copies replaced by checked ones.  A list may
end with its last entry and the counts with the second."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "activation_sparse_tiered_amd", "csrc")

PROGRAM = r"""
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include "common.h"

// "Device" buffers that may be read: the lists and the counts.
static struct { const char* p; size_t bytes; } readable[3];
static bool bad;

extern "C" {
hipError_t hipMemcpyAsync(void* dst, const void* src, size_t n, hipMemcpyKind kind, hipStream_t) {
  const char* s = (const char*)src;
  if (kind == hipMemcpyDeviceToHost) {
    bool inside = false;
    for (auto& r : readable) inside |= s >= r.p && s + n <= r.p + r.bytes;
    if (!inside) { bad = true; printf("a read of %zu bytes outside the lists\n", n); return hipErrorInvalidValue; }
  }
  memcpy(dst, src, n);
  return hipSuccess;
}
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipEventSynchronize(hipEvent_t) { return hipSuccess; }
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipSuccess; }
hipError_t hipEventCreateWithFlags(hipEvent_t* e, unsigned) { *e = (hipEvent_t)1; return hipSuccess; }
hipError_t hipHostMalloc(void** p, size_t n, unsigned) { *p = calloc(1, n); return hipSuccess; }
hipError_t hipHostFree(void* p) { free(p); return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "refused"; }
}

namespace spax {
int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vprintf(fmt, ap);
  va_end(ap);
  return status;
}
int hip_fail(hipError_t, const char* what) { printf("%s\n", what); return SPAX_ERR_HIP; }
GemvPlan gemv_plan(const spax_layout*) { return GemvPlan{}; }
int launch_merge_and_gather(const spax_layout*, const void*, void*, const int32_t*, const int32_t*,
                            const int32_t*, int32_t, uint32_t*, uint32_t*, int32_t*, int32_t*,
                            int32_t*, hipStream_t) { return SPAX_OK; }
static const uint32_t *staged_full, *staged_approx;
int launch_tiered_gemv(const spax_layout*, const GemvPlan&, const void*, const uint16_t*,
                       const int32_t* f, const int32_t* a, const int32_t*, float*, bool, hipStream_t,
                       Lists, float*) {
  staged_full = (const uint32_t*)f;
  staged_approx = (const uint32_t*)a;
  return SPAX_OK;
}
}  // namespace spax

// argv: d_in, FULL and APPROX entries, transfer
int main(int, char** argv) {
  using namespace spax;
  const int d = atoi(argv[1]), n[2] = {atoi(argv[2]), atoi(argv[3])}, transfer = atoi(argv[4]);
  spax_layout L{};
  L.d_in = d;
  L.stride_F = L.stride_A = 128;
  L.off_A = 128 * (int64_t)d;
  L.total_bytes = 256 * (int64_t)d;
  uint8_t* packed = (uint8_t*)calloc(1, (size_t)L.total_bytes);
  void* ws = calloc(1, pinned_workspace_bytes(&L));
  int32_t* list[2];
  for (int i = 0; i < 2; ++i) {
    list[i] = (int32_t*)malloc(4 * (size_t)(n[i] ? n[i] : 1));
    for (int e = 0; e < n[i]; ++e) list[i][e] = (int32_t)((int64_t)e * d / n[i]);
    readable[i].p = (const char*)list[i];
    readable[i].bytes = 4 * (size_t)n[i];
  }
  int32_t* counts = (int32_t*)malloc(8);
  counts[0] = n[0];
  counts[1] = n[1];
  readable[2].p = (const char*)counts;
  readable[2].bytes = 8;
  spax_move_stats st{};
  const int rc = tiered_gemv_pinned(&L, packed, packed, nullptr, list[0], list[1], counts, nullptr, 0,
                                    transfer, ws, &st, nullptr);
  if (rc || bad) return printf(" status %d\n", rc), 1;
  if (st.n_full != n[0] || st.n_approx != n[1]) return printf("counts %d %d\n", st.n_full, st.n_approx), 1;
  const uint32_t* staged[2] = {staged_full, staged_approx};
  for (int i = 0; i < 2; ++i)
    for (int e = 0; e < n[i]; ++e)
      if ((int)(staged[i][e] >> 16) != list[i][e]) return printf("entry %d of list %d\n", e, i), 1;
  return 0;
}
"""


@pytest.fixture(scope="module")
def move(tmp_path_factory):
    d = tmp_path_factory.mktemp("pinned_reads")
    src, exe = d / "move.cpp", d / "move"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-D__HIP_PLATFORM_AMD__",
                    "-I/opt/rocm/include", f"-I{CSRC}", f"-I{os.path.join(ROOT, 'include')}",
                    str(src), os.path.join(CSRC, "pinned.cpp"), "-o", str(exe)],
                   check=True, capture_output=True)
    return lambda *a: subprocess.run([str(exe), *map(str, a)], capture_output=True, text=True,
                                     timeout=60)


@pytest.mark.parametrize("transfer", [0, 2])
@pytest.mark.parametrize("d_in,n", [(333, (84, 118)), (1000, (0, 0)), (1000, (1, 0)), (1000, (0, 1)),
                                    (64, (64, 0)), (32768, (9000, 20000))])
def test_no_entry_past_the_counts(move, d_in, n, transfer):
    r = move(d_in, *n, transfer)
    assert r.returncode == 0, r.stdout
