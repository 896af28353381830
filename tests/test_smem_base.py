"""The host's check of where a kernel's dynamic shared memory starts (no GPU): what would not start on 1024 bytes is refused
with an error, so that no launch returns GTP_OK and leaves its output as it was."""
import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]
CSRC = ROOT / "param_buffers_gb300" / "csrc"

PROGRAM = r"""
#include <cstdio>
#include "smem_base.h"
extern "C" const char *gtp_last_error(void);
int main() {
  const size_t cases[][2] = {{1024, 0}, {0, 0}, {1024, 2048}, {1024, 16}, {512, 0}, {1040, 0}, {512, 512}};
  for (const auto &c : cases) {
    gtp::clear_error();
    const gtp_status s = gtp::check_dynamic_base("kernel", c[0], c[1], 1024);
    std::printf("%d %s\n", int(s), gtp_last_error());
  }
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_a_base_off_1024_bytes_is_refused(tmp_path):
    (tmp_path / "main.cpp").write_text(PROGRAM)
    exe = tmp_path / "check"
    subprocess.run(["g++", "-std=c++17", f"-I{ROOT / 'include'}", f"-I{CSRC}", str(tmp_path / "main.cpp"),
                    str(CSRC / "status.cpp"), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    assert [int(v.split()[0]) != 0 for v in lines] == [False, False, False, True, True, True, True]
    assert all("shared memory" in v for v in lines[3:])


def test_the_kernel_without_room_goes_through_the_check():
    """MXFP4's products are the one kernel that does not align its shared memory itself."""
    src = (CSRC / "gemm_blockscaled.cu").read_text()
    assert "F::SLACK == 0 ? configure_unpadded(" in src and "check_dynamic_base(what" in src
