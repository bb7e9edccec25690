"""Index arithmetic and plans of the device code, run on the CPU: the kernels' own headers compiled
for the host (tests/host), so that sizes no GPU test can hold are walked through too."""
import os
import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]
HOST = ROOT / "tests" / "host"


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    """program(name): the built tests/host/<name>.cpp."""
    out, built = tmp_path_factory.mktemp("host"), {}

    def get(name):
        if name not in built:
            from entropy_gated_kv_gb300 import build as B

            cuda = Path(os.path.realpath(B.nvcc())).parents[1] / "include"
            cxx = shutil.which("g++") or "c++"
            cmd = [cxx, "-std=c++20", "-O2", "-Wno-unknown-pragmas", "-pthread", f"-I{HOST}", f"-I{cuda}", f"-I{B.INCLUDE}",
                   f"-I{B.CSRC}", str(HOST / f"{name}.cpp"), "-o", str(out / name)]
            r = subprocess.run(cmd, capture_output=True, text=True)
            assert r.returncode == 0, r.stderr
            built[name] = out / name
        return built[name]

    return get


def run(exe, *args):
    r = subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, timeout=120)
    return r.returncode, r.stdout + r.stderr


MAX_ROWS = 2**31 - 2  # 2 L Hkv, an even number below 2^31


@pytest.mark.parametrize("rows,piece,ctas", [(0, 256, 8), (1, 128, 1), (1000, 128, 3), (131072, 256, 1216), (MAX_ROWS, 128, 1216),
                                             (MAX_ROWS, 256, 1216), (MAX_ROWS, 256, 1), (MAX_ROWS - 254, 256, 1184)])
def test_every_row_of_a_line_falls_to_one_cta(program, rows, piece, ctas):
    assert run(program("pieces"), rows, piece, ctas) == (0, "ok\n")


def test_a_signed_counter_would_leave_the_line(program):
    # what the test above must notice, planted in the oracle's copy of the loop
    assert run(program("pieces"), 1000, 128, 3, "signed") == (0, "ok\n")
    code, out = run(program("pieces"), MAX_ROWS, 256, 1216, "signed")
    assert code == 1 and "row -" in out
