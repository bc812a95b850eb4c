"""Positions given to an append, as its kernels look them up (compiled for the host): those of
rows of no sequence are not read."""
import os
import shutil
import subprocess

from test_paged_cpu import CSRC


def test_rows_of_no_sequence_have_none(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    src, out = tmp_path / "at.cu", str(tmp_path / "at")
    # (an address that nothing may be read from)
    src.write_text('''#include "paged.cuh"
int main() {
  const int32_t given[3] = {5, -7, 11};
  mha::RopeArgs a{};
  if (mha::append_angle(a, 2, 0, 40) != 40 || mha::append_angle(a, 2, -1, 0) != 0) return 1;
  a.positions = given;
  for (int t = 0; t < 3; ++t)
    if (mha::append_angle(a, t, 4, 40) != given[t]) return 2;
  a.positions = reinterpret_cast<const int32_t *>(64);
  for (int t = 0; t < 3; ++t)
    if (mha::append_angle(a, t, -1, 0) != 0) return 3;
  return 0;
}
''')
    subprocess.run([nvcc, "-O1", "-std=c++17", "-I", CSRC, "-o", out, str(src)], check=True,
                   capture_output=True)
    assert subprocess.run([out]).returncode == 0
    # and it is how both kernels that append find their angles
    code = open(os.path.join(CSRC, "qk_rope.cu")).read()
    assert code.count("append_angle(") == 1 and code.count("ang.at(cells.angle(a, t), col)") == 2
