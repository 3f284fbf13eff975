"""CPU check of the staging buffers' order (csrc/store_ring.h): whenever a buffer is taken for writing, the wait in
front of it (at most N - 1 store groups pending, the newest ones) covers the last store that read that buffer, over
several tiles of any number of stores."""
import pathlib
import shutil
import subprocess

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "mla_latent_kv_27_b200" / "csrc"

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "store_ring.h"

// the first (tile, store) whose buffer a pending group may still read, or none
template <int N>
int walk(int stores, int tiles) {
  mla::StoreRing<N> ring;
  std::vector<int> groups;  // buffers of the committed groups, oldest first
  for (int t = 0; t < tiles; ++t)
    for (int s = 0; s < stores; ++s) {
      const int buf = ring.take();
      if (buf < 0 || buf >= N) return 2;
      const int pending = (int)groups.size() < N - 1 ? (int)groups.size() : N - 1;
      for (int k = 0; k < pending; ++k)
        if (groups[groups.size() - 1 - k] == buf) {
          std::printf("N %d, %d stores a tile: tile %d store %d\n", N, stores, t, s);
          return 1;
        }
      groups.push_back(buf);
    }
  return 0;
}

int main() {
  for (int stores = 1; stores <= 12; ++stores)
    if (walk<1>(stores, 9) || walk<2>(stores, 9) || walk<4>(stores, 9) || walk<8>(stores, 9)) return 1;
  return 0;
}
"""


def run(tmp_path, program):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(program)
    subprocess.run([cxx, "-std=c++17", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True)


def test_a_buffer_is_not_written_under_its_last_store(tmp_path):
    r = run(tmp_path, PROGRAM)
    assert r.returncode == 0, r.stdout


def test_the_walk_sees_turns_that_start_again_with_a_tile(tmp_path):
    """The same walk with a count that begins at buffer 0 in every tile fails for 5 stores and 2 or 4 buffers."""
    again = PROGRAM.replace("const int buf = ring.take();", "const int buf = s % N;")
    assert again != PROGRAM
    r = run(tmp_path, again)
    assert r.returncode == 1 and "stores a tile" in r.stdout


def test_the_kernel_takes_its_buffers_from_the_ring():
    text = (CSRC / "proj_fp8.cu").read_text()
    assert "StoreRing<NBUF>" in text and "ring.take()" in text and "bulk_wait_group_read<NBUF - 1>" in text
