"""Which tile shape a forward product of the ragged kernel takes: the launch code is compiled for the host alone, with
the runtime's launch replaced by one that names the kernel."""
import os
import re
import subprocess

import pytest

from moe_w4a16_grouped_amd import build

SOURCE = """#include "ragged_gemm.h"
#include <cstdio>
#include <cstdlib>
static struct { const void* host; const char* name; } known[256];
static int count;
extern "C" void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  known[count++] = {host, name};
}
extern "C" hipError_t hipLaunchKernel(const void* f, dim3, dim3, void**, size_t, hipStream_t) {
  for (int i = 0; i < count; ++i) if (known[i].host == f) puts(known[i].name);
  return hipSuccess;
}
extern "C" hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
extern "C" hipError_t __hipPopCallConfiguration(dim3*, dim3*, size_t*, hipStream_t*) { return hipSuccess; }
extern "C" void** __hipRegisterFatBinary(const void*) { static void* p; return &p; }
extern "C" void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
extern "C" void __hipUnregisterFatBinary(void**) {}
extern "C" hipError_t hipGetLastError() { return hipSuccess; }
int main(int, char** v) {
  static int32_t offsets[1];
  moe::RaggedArgs a{};
  a.R = atoi(v[1]), a.E = atoi(v[2]), a.N = atoi(v[3]), a.K = atoi(v[4]), a.a_row_div = 1;
  a.offsets = a.E > 1 ? offsets : nullptr;
  (void)moe::launch_ragged_fwd<moe::ElemI8, MOE_EPI_NONE>(a, nullptr);
  (void)moe::launch_ragged_fwd<moe::ElemI8, MOE_EPI_SILU_MUL>(a, nullptr);
  (void)moe::launch_ragged_fwd<moe::ElemBF16, MOE_EPI_NONE>(a, nullptr);
  (void)moe::launch_ragged_fwd<moe::ElemBF16, MOE_EPI_SILU_MUL>(a, nullptr);
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.hip").write_text(SOURCE)
    subprocess.run([build.HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O0", "-std=c++17", "-fPIC", "-I", build.INCLUDE,
                    "-I", build.CSRC, "-c", str(d / "choice.hip"), "-o", str(d / "choice.o")], check=True, timeout=300)
    subprocess.run(["g++", str(d / "choice.o"), "-o", str(d / "choice"), "-Wl,--unresolved-symbols=ignore-all"], check=True, timeout=300)

    def shapes(R, E, N, K):
        """[rows, columns, ..., weights past the L2] of the highest tiles, for int8 and bf16, without and with SiLU*mul."""
        out = subprocess.run([str(d / "choice"), *map(str, (R, E, N, K))], check=True, capture_output=True, text=True, timeout=60).stdout
        return [[int(x) for x in re.findall(r"L[ib](\d+)E", n)] for n in re.findall(r"TileShapeI((?:L[ib]\d+E)+)E", out)]

    return shapes


def test_weights_pass_the_l2_only_for_groups_of_one_tile(choose):
    """Groups of more than 16 rows on 16-row tiles read their weights more than once."""
    for R, E, N in ((64, 128, 1536), (1024, 64, 2048), (16, 1, 28672)):
        assert all(s[0] == 16 and s[-1] == 1 for s in choose(R, E, N, 2048)), (R, E, N)
    for R, E, N in ((200, 1, 1024), (300, 1, 1536), (400, 1, 1024), (600, 1, 1024), (200, 4, 1024), (200, 8, 1024), (1025, 64, 2048)):
        shapes = choose(R, E, N, 2048)
        assert len(shapes) == 4 and all(s[-1] == 0 for s in shapes), (R, E, N, shapes)


def test_weight_rows_that_share_lines_stay_in_the_l2(choose):
    assert [s[-1] for s in choose(64, 128, 1536, 2064)] == [0] * 4
