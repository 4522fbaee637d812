"""Host-side rules of the operators around the routed experts (no GPU)."""
import shutil
import subprocess

import pytest

from moe_routing_precision_gb300 import _build


@pytest.fixture(scope="module")
def L():
    _build.build()
    from moe_routing_precision_gb300 import ops
    return ops.lib()


@pytest.mark.parametrize("T,E,S,table", [
    (16384, 1, 1, True), (5461, 3, 1, True), (963, 17, 1, True), (496, 33, 1, True),
    (16384, 1, 4, True), (963, 17, 100, True),       # too long for any one block
    (64, 16, 1, False), (64, 256, 1, False), (128, 17, 1, False), (129, 17, 1, True),
    (496, 33, 4, False), (513, 17, 4, True), (16, 1024, 1, False), (17, 1024, 1, True),
    # eight passes with 16-byte aligned rows, 64 without: the table's size is named
    (1024, 16, 1, True), (128, 16, 1, False)])
def test_balance_loss_workspace_follows_the_passes_of_a_block(L, T, E, S, table):
    """One block walks a sequence's tokens 16 warps at a time (4 to 32 lanes a token):
    beyond eight passes for each of up to four sequences the table is faster."""
    assert (L.moe_balance_loss_workspace_bytes(T, E, S) > 0) == table


KNOWN = r"""
#include <cstdio>
#include <thread>
#include <utility>
#include <vector>
#include "known.cuh"

int main() {
  // a width known on one device is not known on another
  moe::Known<std::pair<int, int>, int> per_sm;
  int v = -1;
  if (per_sm.find({0, 9000}, &v)) return 1;
  per_sm.put({0, 9000}, 2);
  if (per_sm.find({1, 9000}, &v) || per_sm.find({0, 9001}, &v)) return 2;
  per_sm.put({1, 9000}, 3);
  if (!per_sm.find({0, 9000}, &v) || v != 2) return 3;
  if (!per_sm.find({1, 9000}, &v) || v != 3) return 4;
  // and any number of keys is kept, from several threads
  moe::Known<const void*, int> caps;
  static char kernels[2000];
  std::vector<std::thread> t;
  for (int i = 0; i < 4; ++i)
    t.emplace_back([&] { for (int k = 0; k < 2000; ++k) caps.put(kernels + k, k); });
  for (auto& x : t) x.join();
  for (int k = 0; k < 2000; ++k)
    if (!caps.find(kernels + k, &v) || v != k) return 5;
  std::puts("OK");
}
"""


def test_known_values_by_key(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    src, exe = tmp_path / "known.cpp", tmp_path / "known"
    src.write_text(KNOWN)
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", f"-I{_build.CSRC}",
                        str(src), "-pthread", "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "OK", (r.returncode, r.stderr)
