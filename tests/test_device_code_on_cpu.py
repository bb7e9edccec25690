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


def plan(exe, B, L, Hq, Hkv, Rs, lens=None, Lp=0, scope=0, ctas=152, slots=1280, *args):
    """Runs the plan of a call with these sizes and checks it; (mode, prefix tiles, own tiles, units)."""
    text = f"{B} {L} {scope or L} {Lp} {Hkv} {Hq // Hkv} {ctas} {slots} {int(lens is not None)}\n"
    text += " ".join(map(str, Rs)) + "\n" + " ".join(map(str, lens or [])) + "\n"
    r = subprocess.run([str(exe), *args], input=text, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    mode, *n = r.stdout.split()
    return (mode, *map(int, n))


PLANS = [
    # B, L, Hq, Hkv, rows, lengths, Lp, mode
    (1, 1, 1, 1, [1], [0], 0, "whole"),
    (1, 1024, 32, 32, [95], None, 0, "separate"),
    (1, 32768, 32, 32, [95], None, 0, "separate"),
    (8, 2048, 28, 4, [95, 89, 83, 78, 72, 66, 60, 54], [2048 - 128 * b for b in range(8)], 0, "whole"),
    (3, 300, 6, 2, [5, 0, 300], [300, 17, 129], 0, "whole"),
    (40, 70, 2, 1, [(7 * b) % 5 for b in range(40)], [(11 * b) % 71 for b in range(40)], 0, "whole"),
    (4, 640, 16, 16, [640] * 4, [640, 5, 333, 640], 0, "separate"),
    (4, 50, 4, 2, [5, 51, 7, -1], [50, 50, 51, 3], 200, "whole"),
    (32, 256, 28, 4, [1] * 32, None, 1792, "shared"),
    (8, 256, 32, 32, [32 - 2 * b for b in range(8)], [256 - 16 * b for b in range(8)], 3840, "shared"),
    (16, 256, 28, 4, [31 - b for b in range(16)], [256 - 8 * b for b in range(16)], 32512, "shared"),
    (37, 9, 14, 2, [b % 4 for b in range(37)], [(5 * b) % 10 for b in range(37)], 700, "shared"),
    (5, 40, 6, 3, [3, 0, 40, 17, 1], [40, 3, 0, 17, 39], 640, "shared"),
    (2, 384, 4, 4, [384, 256], None, 512, "separate"),  # 20 tiles of 10 units: a share is 2
    (16, 64, 32, 4, [1] * 16, list(range(0, 64, 4)), 3000, "shared"),
    (7, 500, 24, 8, [90, 128, 1, 0, 300, 500, 17], [500, 1, 500, 400, 0, 333, 499], 1000, None),
]


@pytest.mark.parametrize("B,L,Hq,Hkv,Rs,lens,Lp,mode", PLANS)
@pytest.mark.parametrize("ctas", [152, 148, 7])
def test_a_plan_covers_every_block_once_and_leaves_every_record(program, B, L, Hq, Hkv, Rs, lens, Lp, mode, ctas):
    got = plan(program("plan"), B, L, Hq, Hkv, Rs, lens, Lp, ctas=ctas)
    assert mode is None or ctas != 152 or got[0] == mode, got


def test_a_tile_without_a_record_is_noticed(program):
    with pytest.raises(AssertionError, match="no record after giving up"):
        plan(program("plan"), 32, 256, 28, 4, [1] * 32, None, 1792, 0, 152, 1280, "lost")


def slots(B, L, Hq, Hkv):
    """Tiles whose partial rows the workspace of ec_prefix_attention holds."""
    g = Hq // Hkv
    return max(320, min(Hkv * -(-B * L * g // 128) + B * Hkv * -(-L * g // 128) + 160, 1280))


@pytest.mark.parametrize("Hkv,last", [(32, 34), (8, 139), (4, 279)])
def test_where_the_prefix_stops_being_shared(program, Hkv, last):
    # the interface's own figures: one row per sequence and head, as many sequences as the workspace has places for
    for B, mode in ((last, "shared"), (last + 1, "separate")):
        got = plan(program("plan"), B, 8, Hkv, Hkv, [1] * B, None, 700, slots=slots(B, 8, Hkv, Hkv))
        assert got[0] == mode, (B, got)


@pytest.mark.parametrize("B,L,Hq,Hkv,Rs,lens,Lp,mode", [
    # the sizes of the GPU tests that are meant for one mode of the plan
    (34, 8, 32, 32, [1 + b % 2 for b in range(34)], [b % 9 for b in range(34)], 700, "shared"),
    (36, 8, 32, 32, [1 + b % 2 for b in range(36)], [b % 9 for b in range(36)], 700, "separate"),
    (5, 130, 28, 28, [128, 120, 128, 101, 128], [130, 0, 59, 2, 128], 700, "whole"),
    (3, 260, 80, 40, [64, 50, 33], [260, 129, 7], 1000, "whole"),
])
def test_the_mode_that_a_gpu_test_is_meant_for(program, B, L, Hq, Hkv, Rs, lens, Lp, mode):
    assert plan(program("plan"), B, L, Hq, Hkv, Rs, lens, Lp, slots=slots(B, L, Hq, Hkv))[0] == mode
