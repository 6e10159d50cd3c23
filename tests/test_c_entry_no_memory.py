"""The paged cache's C entries where host memory cannot be had (CPU): a return
code, and no exception that leaves the entry and ends the process."""
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
#include "tcd_cache.h"

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
  GET(tc_attend); GET(tc_attend_workspace); GET(tc_kv_append); GET(tc_kv_compact); GET(tc_kv_copy_pages);
  GET(tc_tree_masks); GET(tc_pages_create); GET(tc_pages_open); GET(tc_pages_reserve); GET(tc_pages_fork);
  GET(tc_pages_trim); GET(tc_pages_close); GET(tc_pages_row); GET(tc_pages_destroy); GET(tc_pages_free_count);
  int word = 0, seq = -1, n = 0, src = 0, dst = 0;
  int64_t bytes = 0;
  tc_kv_t kv{};
  kv.pool = aligned_alloc(64, 64);
  kv.layers = kv.pages = kv.kv_heads = 1;
  kv.page_size = 24;
  kv.head_dim = 64;
  tc_tokens_t few{}, many{};
  many.batch = TC_KV_MAX_BATCH + 1;
  many.ctx_lens = many.cu_tokens = &word;
  tc_pages* pages = nullptr;
  want("create", tc_pages_create_(200, 16, &pages), TC_OK);
  want("open", tc_pages_open_(pages, &seq), TC_OK);
  none = true;
  // refused arguments: the message cannot be written
  want("workspace", tc_attend_workspace_(nullptr, &bytes), TC_ERR_INVALID_ARG);
  want("workspace, page size", tc_attend_workspace_(&kv, &bytes), TC_ERR_UNSUPPORTED);
  want("append", tc_kv_append_(&kv, 0, nullptr, nullptr, nullptr, nullptr), TC_ERR_UNSUPPORTED);
  want("attend", tc_attend_(nullptr, 0, nullptr, nullptr, nullptr, 0, nullptr, nullptr), TC_ERR_INVALID_ARG);
  want("copy", tc_kv_copy_pages_(&kv, nullptr, nullptr, 1, nullptr, nullptr), TC_ERR_UNSUPPORTED);
  kv.page_size = 16;
  want("attend, tokens", tc_attend_(&kv, 0, &few, nullptr, nullptr, 0, nullptr, nullptr), TC_ERR_INVALID_ARG);
  want("compact, batch", tc_kv_compact_(&kv, &many, nullptr, 1, nullptr, nullptr, nullptr, nullptr), TC_ERR_CAPACITY);
  want("masks, batch", tc_tree_masks_(&many, nullptr, 1, nullptr, nullptr, nullptr, nullptr), TC_ERR_CAPACITY);
  // pages: nothing has changed afterwards
  tc_pages* other = nullptr;
  want("create, none", tc_pages_create_(200, 16, &other), TC_ERR_OOM);
  want("reserve, none", tc_pages_reserve_(pages, seq, 0, 1600, &src, &dst, &n), TC_ERR_OOM);
  int second = -1;
  want("open, none", tc_pages_open_(pages, &second), TC_ERR_OOM);
  want("row, NULL", tc_pages_row_(pages, 7, nullptr, 0, &n), TC_ERR_INVALID_ARG);
  none = false;
  want("free", tc_pages_free_count_(pages, &n), TC_OK);
  want("pages free", n, 200);
  want("reserve", tc_pages_reserve_(pages, seq, 0, 1600, &src, &dst, &n), TC_OK);
  none = true;
  want("fork, none", tc_pages_fork_(pages, seq, 1600, &second), TC_ERR_OOM);
  want("trim", tc_pages_trim_(pages, seq, 100), TC_OK);
  want("close", tc_pages_close_(pages, seq), TC_OK);
  none = false;
  want("free", tc_pages_free_count_(pages, &n), TC_OK);
  want("pages free", n, 200);
  tc_pages_destroy_(pages);
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
