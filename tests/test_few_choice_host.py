"""What the launches of the layer for a few tokens choose: the launch code is compiled for the host alone, with the runtime's
launch replaced by one that checks what its kernels rely on, over all token counts and a sweep of the other sizes."""
import os
import subprocess

import pytest

from moe_w4a16_grouped_amd import build

SOURCE = """#include "few.hip"
#include <cstdio>
#include <cstdlib>
#include <cstring>
static struct { const void* host; const char* name; } known[256];
static int count;
static size_t shared;
static long launches, bad, most_units;
extern "C" void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  known[count++] = {host, name};
}
static void need(bool ok, const char* what, const moe::FewArgs& p) {
  if (!ok && ++bad <= 20) printf("%s: T %d, E %d, k %d, H %d, I %d, shift %d, groups %d\\n", what, p.T, p.E, p.k, p.H, p.I, p.pieces_shift, p.groups);
}
extern "C" hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t lds, hipStream_t) {
  const char* name = "";
  for (int i = 0; i < count; ++i) if (known[i].host == f) name = known[i].name;
  if (strstr(name, "few_join")) return hipSuccess;
  const moe::FewArgs& p = *static_cast<const moe::FewArgs*>(args[0]);
  const int R = p.T * p.k, waves = block.x / 64;
  ++launches;
  need(grid.x >= 1 && block.x == 64u * waves, "launch", p);
  need(lds <= 160 << 10 && (lds <= 64 << 10 || shared == lds), "LDS", p);
  if (const char* at = strstr(name, "few_down_kernel")) {
    int cols = 0, super = 0, tok = 0;
    need(sscanf(strstr(at, "ELi"), "ELi%dELi%dELi%dE", &cols, &super, &tok) == 3, "name", p);
    const int pieces = 1 << p.pieces_shift, supers = (p.I + super - 1) / super, workers = waves * p.groups;
    // an entry holds a row at least, so R bounds the entries
    const int units = (R * pieces + workers - 1) / workers;
    most_units = units > most_units ? units : most_units;
    need(units <= 64, "a wave's units, one a lane", p);
    need(pieces <= supers, "a super-chunk for every piece", p);
    need(p.entry_rows >= 1 && p.entry_rows <= tok && (p.T > 1 || p.entry_rows == 1) && (p.T == 1 || p.entry_rows >= 4), "rows of an entry", p);
    need(p.cols >= 1 && p.cols <= cols && (int)grid.x == (p.H + p.cols - 1) / p.cols && (int)grid.y == p.groups, "columns", p);
    need(cols * p.T <= (int)block.x, "a thread for each y", p);
    need(p.groups >= 1 && p.groups <= moe::kFewGroups && (p.groups == 1 || p.H <= moe::kFewGroupsH), "groups, whose parts the workspace holds", p);
  }
  return hipSuccess;
}
extern "C" hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int value) { shared = value; return hipSuccess; }
static struct { dim3 grid, block; size_t lds; hipStream_t s; } call;
extern "C" hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t s) { call = {grid, block, lds, s}; return hipSuccess; }
extern "C" hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
  *grid = call.grid, *block = call.block, *lds = call.lds, *s = call.s;
  return hipSuccess;
}
extern "C" void** __hipRegisterFatBinary(const void*) { static void* p; return &p; }
extern "C" void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
extern "C" void __hipUnregisterFatBinary(void**) {}
extern "C" hipError_t hipGetLastError() { return hipSuccess; }
int main() {
  const int Hs[] = {16, 32, 48, 64, 128, 240, 256, 272, 496, 512, 528, 592, 768, 784, 1008, 1024, 1040, 1536, 1760, 2032, 2048, 2064, 2304,
                    4080, 4096, 4112, 7168, 8192, 16384, 32768, 65536};
  const int Is[] = {16, 48, 240, 256, 272, 496, 512, 528, 1024, 1040, 1536, 2064, 4112, 5280, 7168, 8192, 13712, 14336, 32768, 131072};
  const int Es[] = {1, 2, 3, 4, 5, 7, 8, 10, 12, 16, 18, 20, 24, 28, 32, 40, 48, 56, 60, 64, 68, 72, 80, 90, 96, 100, 112, 118, 120, 126, 127, 128, 129, 160,
                    200, 256, 257, 300, 384, 512, 513, 1024};
  for (int T = 1; T <= 16; ++T)
    for (int k = 1; k <= 16; ++k)
      for (int E : Es)
        for (int H : Hs)
          for (int I : Is)
            if (k <= E && T * H <= 65536)
              for (int i8 = 0; i8 < 2; ++i8) {
                moe::FewArgs a{};
                a.T = T, a.H = H, a.I = I, a.E = E, a.k = k;
                (void)moe::launch_ffn_few(a, i8, nullptr);
              }
  printf("%ld launches, %ld bad, at most %ld units a wave\\n", launches, bad, most_units);
  return bad || !launches;
}
"""


def test_choices_keep_what_the_kernels_rely_on(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    (tmp_path / "choice.hip").write_text(SOURCE)
    subprocess.run([build.HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-I", build.INCLUDE,
                    "-I", build.CSRC, "-c", str(tmp_path / "choice.hip"), "-o", str(tmp_path / "choice.o")], check=True, timeout=300)
    subprocess.run(["g++", str(tmp_path / "choice.o"), "-o", str(tmp_path / "choice"), "-Wl,--unresolved-symbols=ignore-all"], check=True, timeout=300)
    run = subprocess.run([str(tmp_path / "choice")], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout + run.stderr
