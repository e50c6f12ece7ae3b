"""The table of shared-memory limits (ensure_smem in csrc/abi.cu), compiled from its
source against fakes of the two CUDA calls it makes: a limit is raised when a launch
needs more than before, never lowered, and the table has one entry for a function and
device, so that sizes which grow step by step neither fill it nor set the function's
attribute again once it is there. And the launches whose size follows the batch ask
once, for the largest batch."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "learned_token_pruning_gemm_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <map>
#include <mutex>
#include <utility>
enum cudaError_t { cudaSuccess = 0 };
enum { cudaFuncAttributeMaxDynamicSharedMemorySize = 8 };
static int g_dev = 0, g_sets = 0;
static std::map<std::pair<int, const void*>, int> g_limit;
static std::mutex g_mu;
static cudaError_t cudaGetDevice(int* d) { *d = g_dev; return cudaSuccess; }
static cudaError_t cudaFuncSetAttribute(const void* f, int, int bytes) {
  ++g_sets;
  g_limit[{g_dev, f}] = bytes;
  return cudaSuccess;
}
%s
static int bad = 0;
static void ask(const char* f, int bytes) {
  if (!ensure_smem(f, bytes) || g_limit[{g_dev, f}] < bytes) ++bad;
}
int main() {
  const char f[300] = {};   // functions: one address each
  for (int bytes = 1; bytes <= 1000; ++bytes) ask(f, bytes);         // grows step by step
  for (int bytes = 1000; bytes > 0; --bytes) ask(f, bytes);          // and back
  const int grown = g_sets;
  for (int i = 1; i < 200; ++i) ask(f + i, 50 + i);                  // others still find room
  const int others = g_sets - grown;
  for (int k = 0; k < 10; ++k)
    for (int i = 0; i < 200; ++i) ask(f + i, 50);
  const int again = g_sets - grown - others;
  g_dev = 1;
  ask(f, 1000);
  ask(f, 10);
  std::printf("%%d %%d %%d %%d %%d\n", grown, others, again, g_sets - grown - others - again, bad);
}
"""


def test_limits_grow_in_place(tmp_path):
    src = open(os.path.join(CSRC, "abi.cu")).read()
    body = re.search(r"^bool ensure_smem\(.*?^}\n", src, re.S | re.M).group(0)
    cpp, exe = tmp_path / "t.cpp", tmp_path / "t"
    cpp.write_text(PROGRAM % body)
    subprocess.run(["g++", "-std=c++17", "-o", str(exe), str(cpp)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    grown, others, again, other_device, bad = map(int, out)
    assert bad == 0 and grown == 1000 and others == 199
    assert again == 0, "a limit that is there was set again"
    assert other_device == 1


def test_sizes_by_the_batch_are_asked_for_once():
    src = open(os.path.join(CSRC, "tree_rows.cu")).read()
    asked = re.findall(r"ensure_smem\((.*?)\)\)\s*\n?\s*return", src, re.S)
    assert len(asked) == 1 and "kTreeMaxBatch" in asked[0] and "a.batch" not in asked[0]
