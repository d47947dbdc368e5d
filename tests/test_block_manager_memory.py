"""pa_bm_prepare_eviction when host memory runs out at any of its allocations:
an error, and the manager as it was (a small C++ program around the manager's
source, with an operator new that fails at a chosen call; no GPU)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <new>
#include <vector>

#include "pa.h"

static long left = -1;  // allocations until one fails; negative: none does
void* operator new(std::size_t n) {
  if (left == 0) throw std::bad_alloc();
  if (left > 0) --left;
  void* p = std::malloc(n ? n : 1);
  if (p == nullptr) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

struct State {
  std::vector<int32_t> v;
  explicit State(pa_block_manager* bm) {
    v.push_back(pa_bm_num_free_blocks(bm));
    for (int b = 0; b < 1200; ++b) v.push_back(pa_bm_ref_count(bm, b));
    for (int s = 0; s < 4; ++s) {
      std::vector<int32_t> t(400);
      int32_t blocks = -1, tokens = -1;
      pa_bm_table(bm, s, t.data(), 400, &blocks, &tokens);
      v.push_back(blocks);
      v.push_back(tokens);
      v.insert(v.end(), t.begin(), t.begin() + (blocks > 0 ? blocks : 0));
    }
  }
};

int main() {
  std::vector<int32_t> reference;
  int failures = 0;
  for (long fail = -1; fail < 400; ++fail) {
    pa_block_manager* bm = pa_bm_create(1200, 8);
    pa_bm_add(bm, 0, 8 * 300);
    pa_bm_add(bm, 1, 8 * 350 + 3);
    pa_bm_fork(bm, 0, 2);
    pa_bm_add(bm, 3, 8 * 100);
    const State before(bm);
    const int64_t ids[4] = {0, 1, 2, 3};
    const int32_t budgets[4] = {17, 9, 8 * 40, -1};
    std::vector<int32_t> tables(4 * 400), lens(4), dst(4 * 400);
    left = fail;
    const int rc = pa_bm_prepare_eviction(bm, ids, budgets, 4, 400, tables.data(), lens.data(), dst.data());
    left = -1;
    const State after(bm);
    if (rc == PA_OK) {
      // the free set is whole: every block that is handed out now is another one
      std::vector<int32_t> now(after.v);
      const int32_t free_blocks = pa_bm_num_free_blocks(bm);
      if (pa_bm_add(bm, 9, 8 * free_blocks) != PA_OK) return std::printf("free set\n"), 1;
      for (int b = 0; b < 1200; ++b) {
        if (pa_bm_ref_count(bm, b) != 1) return std::printf("block %d\n", b), 1;
      }
      if (reference.empty()) reference = now;
      if (reference != now) return std::printf("another result\n"), 1;
      pa_bm_destroy(bm);
      if (fail >= 0) return std::printf("%d failures\n", failures), 0;
      continue;
    }
    ++failures;
    if (after.v != before.v) return std::printf("changed at allocation %ld\n", fail), 1;
    pa_bm_destroy(bm);
  }
  return std::printf("never succeeded\n"), 1;
}
"""


def test_prepare_eviction_out_of_memory(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "bm.cpp", tmp_path / "bm"
    src.write_text(PROGRAM)
    manager = os.path.join(ROOT, "paged_kv_cache_357_b200", "csrc", "pa_block_manager.cpp")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), str(src), manager, "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout.split()[0]) >= 5, r.stdout
