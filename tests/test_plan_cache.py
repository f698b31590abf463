"""The cache of launch plans (plan_cache.h): bounded, and no exception leaves it, so
that none crosses a C entry point when host memory runs out."""
import os
import re
import subprocess

import memory_bound_normalization_rmsnorm_gb300 as gb

CSRC = os.path.join(os.path.dirname(gb.__file__), "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <new>
#include "plan_cache.h"
static bool g_full = false;
void *operator new(std::size_t n) {
  if (g_full) throw std::bad_alloc();
  return std::malloc(n);
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
int main() {
  gbn::PlanCache<int, int> c(3);
  int v = 0;
  for (int i = 0; i < 3; ++i) c.keep(i, 10 * i);
  if (!c.find(2, &v) || v != 20 || c.find(3, &v)) return 1;
  c.keep(3, 30);                               // the fourth: the cache starts anew
  if (c.find(0, &v) || !c.find(3, &v) || v != 30) return 2;
  g_full = true;
  c.keep(4, 40);                               // no memory for a new entry
  c.keep(3, 31);                               // none needed for one that is there
  if (c.find(4, &v) || !c.find(3, &v) || v != 31) return 3;
  g_full = false;
  c.keep(4, 40);
  return c.find(4, &v) && v == 40 ? 0 : 4;
}
"""


def test_bounded_and_quiet_without_host_memory(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe), "-pthread"], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_the_linear_layer_keeps_nothing_elsewhere():
    """Containers that grow in a call: plans only, and the set of prepared kernels,
    whose insertion is guarded too."""
    with open(os.path.join(CSRC, "linear.cu")) as f:
        text = f.read()
    assert not re.search(r"std::(map|set|vector|string|unordered_\w+)<", text)
    with open(os.path.join(CSRC, "api.cu")) as f:
        ready = re.search(r"norm_status_t prepare_function.*?\n\}\n", f.read(), re.S).group(0)
    assert re.search(r"try \{\s+g_attr_done\.insert\(\{dev, fn\}\);\s+\} catch \(\.\.\.\)", ready)
