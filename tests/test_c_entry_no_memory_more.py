"""tc_linear and tc_attend_shared where host memory cannot be had (CPU): a return code, and no exception that leaves
the entry."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

PROGRAM = r"""
#include <dlfcn.h>
#include <cstdio>
#include <cstdlib>
#include <new>
#include "tcd_linear.h"

static bool none = false;
void* operator new(std::size_t n) {
  void* p = none ? nullptr : std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

#define GET(name) auto name##_ = reinterpret_cast<decltype(&name)>(dlsym(lib, #name))
static int bad = 0;
static void want(const char* what, int got, int code) {
  if (got != code) std::printf("%s: %d, not %d\n", what, got, code), ++bad;
}

int main(int, char** argv) {
  void* lib = dlopen(argv[1], RTLD_NOW);
  if (!lib) return std::printf("%s\n", dlerror()), 2;
  GET(tc_linear); GET(tc_attend_shared); GET(tc_attend_shared_workspace);
  alignas(64) static char memory[64];
  int32_t status = 0;
  int64_t bytes = 0;
  tc_linear_t layer{};
  tc_linear_call_t call{};
  tc_kv_t kv{};
  tc_tokens_t tokens{};
  tc_attend_t args{};
  tc_shared_t shared{};
  none = true;
  want("linear, NULL", tc_linear_(nullptr, nullptr, nullptr, nullptr), TC_ERR_INVALID_ARG);
  want("linear, empty", tc_linear_(&layer, &call, &status, nullptr), TC_ERR_INVALID_ARG);
  layer.in_features = layer.out_features = 8;
  layer.dtype = 7;
  want("linear, type", tc_linear_(&layer, &call, &status, nullptr), TC_ERR_UNSUPPORTED);
  layer.dtype = TC_DT_F16;
  layer.weight = memory;
  layer.weight_stride = 8;
  call.n_tokens = TC_LINEAR_MAX_TOKENS + 1;
  want("linear, tokens", tc_linear_(&layer, &call, &status, nullptr), TC_ERR_CAPACITY);
  call.n_tokens = 0;
  want("linear, none", tc_linear_(&layer, &call, &status, nullptr), TC_OK);
  call.n_tokens = 1;
  want("linear, x", tc_linear_(&layer, &call, &status, nullptr), TC_ERR_INVALID_ARG);
  want("shared, NULL", tc_attend_shared_(&kv, 0, &tokens, &args, nullptr, memory, 64, &status, nullptr),
       TC_ERR_INVALID_ARG);
  want("shared, cache", tc_attend_shared_(&kv, 0, &tokens, &args, &shared, memory, 64, &status, nullptr),
       TC_ERR_INVALID_ARG);
  want("workspace", tc_attend_shared_workspace_(&kv, 1, 1, &bytes), TC_ERR_INVALID_ARG);
  none = false;
  return bad;
}
"""


def test_no_exception_leaves_a_c_entry(tcd, tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "entries.cpp", tmp_path / "entries"
    src.write_text(PROGRAM)
    # (-rdynamic: the library's allocations come to this program's operator new)
    subprocess.run([cxx, "-std=c++17", "-O1", "-rdynamic", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe),
                    "-ldl"], check=True)
    r = subprocess.run([str(exe), tcd.LIB_PATH], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
