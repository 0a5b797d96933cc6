"""The tile that a Newton-Schulz product gets, without a GPU: the estimates against times measured on an MI355X (us), and that the
choice is near the fastest."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

# batch, M, N, symmetric, steps: measured on tiles of 64, 128, 128 in pairs and 256
MEASURED = {(1, 256, 256, 1, 16): (7.5, 14.4, 13.8, 20.6), (1, 256, 256, 1, 4): (5.5, 10.2, 8.6, 15.6),
            (1, 256, 1024, 0, 4): (4.9, 7.8, 6.6, 11.6), (1, 1000, 1000, 1, 32): (9.8, 22.2, 23.8, 38.6),
            (1, 1000, 2001, 0, 16): (12.2, 14.7, 15.0, 23.1), (1, 512, 512, 1, 8): (6.4, 10.1, 10.3, 17.2),
            (1, 1024, 1024, 1, 64): (15.3, 33.2, 40.8, 66.2), (1, 1024, 4096, 0, 16): (19.6, 15.4, 16.4, 24.8),
            (1, 2048, 2048, 1, 32): (23.6, 21.5, 24.9, 40.1), (1, 2048, 2048, 0, 32): (36.1, 24.1, 26.6, 40.0),
            (1, 1536, 1536, 1, 64): (26.3, 33.8, 41.6, 67.1), (1, 1536, 4096, 0, 24): (37.8, 34.2, 27.2, 34.6),
            (8, 512, 512, 1, 16): (10.0, 13.3, 14.1, 24.7), (8, 1024, 1024, 1, 32): (34.4, 39.3, 31.9, 41.7),
            (8, 1024, 2048, 0, 16): (62.4, 52.0, 39.7, 34.8), (1, 4096, 4096, 1, 64): (162.1, 110.5, 97.4, 78.3),
            (1, 4096, 4096, 0, 64): (298.9, 166.4, 127.7, 102.7), (8, 2048, 7168, 0, 32): (None, 689.7, 550.1, 390.1)}


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("ortho") / "driver")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-I",
                        os.path.join(ROOT, "fp8_fine_grained_amax_amd", "csrc"), os.path.join(ROOT, "tests", "ortho_shape_driver.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(problems):
        text = "".join(" ".join(map(str, [*p, 0][:6])) + "\n" for p in problems)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60, env=dict(os.environ, ASAN_OPTIONS="verify_asan_link_order=0"))
        assert r.returncode == 0 and "runtime error" not in r.stderr, r.stderr
        lines = [line.split() for line in r.stdout.splitlines()]
        return [(int(v[0]), [float(x) for x in v[3:]], (int(v[1]), int(v[2]))) for v in lines]
    return run


def test_estimates_and_choices(ask):
    for (problem, measured), (choice, us, _) in zip(MEASURED.items(), ask(list(MEASURED))):
        for m, e in zip(measured, us):
            assert m is None or 0.65 < e / m < 1.5, (problem, measured, us)
        fastest = min(m for m in measured if m is not None)
        assert choice < 4 and measured[choice] <= 1.1 * fastest, (problem, choice, measured)


def test_rest_of_a_round(ask):
    # 288 tiles of 256: one round, and 32 tiles in quarters; 256 and 136 tiles have no whole round with a rest
    (tail, *_), (even, *_), (few, *_) = ask([(8, 2048, 2048, 1, 112), (1, 4096, 4096, 0, 64), (1, 4096, 4096, 1, 64)])
    assert (tail, even, few) == (4, 3, 3)


# Whole updates (us, five steps; batch, m, n) whose A has one workgroup a tile, and several on tiles of 64, 128 and 256
SPLITS = {(1, 64, 4096): (106, 84, 98, None), (1, 64, 16384): (221, 92, 108, None), (2, 76, 16200): (245, 135, 161, None),
          (1, 256, 2048): (105, 100, 114, None), (1, 256, 8192): (188, 110, 126, None), (1, 309, 4853): (160, 120, 144, None),
          (1, 512, 4096): (152, 139, 155, None), (1, 512, 16384): (317, 190, 208, None), (2, 496, 3973): (174, 167, 204, None),
          (1, 640, 10240): (291, 194, 223, None), (1, 768, 16384): (384, 286, 292, None), (1, 856, 11323): (376, 311, 310, None),
          (1, 1024, 4096): (191, None, 217, None), (1, 1024, 16384): (446, None, 387, 407), (1, 1280, 16384): (599, None, 577, 563),
          (1, 1536, 4096): (328, None, 329, None), (1, 1536, 8192): (530, None, 445, 484), (1, 1536, 16384): (996, None, 755, 724),
          (1, 1900, 18432): (1536, None, 1264, 1179), (1, 2048, 4096): (470, None, None, 470), (1, 2048, 8192): (725, None, None, 706),
          (1, 2048, 16384): (1321, None, None, 1106), (1, 2560, 2560): (476, None, None, 475), (1, 2560, 8192): (967, None, None, 1029),
          (1, 3000, 18432): (2721, None, None, 2416), (2, 1024, 8192): (458, None, 414, 428), (2, 2048, 8192): (1305, None, None, 1172),
          (4, 512, 8192): (281, None, 287, None), (4, 1024, 4096): (439, None, 438, 457)}


def test_shared_contractions(ask):
    def problem(b, m, n):
        return b, m, m, 1, (n + 63) // 64, 2 * (b if m % 64 == 0 else 1) * m * ((n + 63) // 64 * 64)
    for (size, measured), (_, _, (side, parts)) in zip(SPLITS.items(), ask([problem(*k) for k in SPLITS])):
        us = measured[{0: 0, 64: 1, 128: 2, 256: 3}[side]]
        assert (side == 0) == (parts == 1) and us is not None and us <= 1.08 * min(m for m in measured if m), (size, side, parts)
    # no part of fewer than eight steps, no more parts than the room holds or the CUs take
    for b, m, n, room in ((1, 64, 16384, 16384 * 3), (1, 64, 16384, 16383), (1, 64, 1000, 1 << 40), (300, 64, 16384, 1 << 40)):
        (_, _, (side, parts)), = ask([(b, m, m, 1, (n + 63) // 64, room)])
        assert parts <= max(1, min(room // 16384, (n + 63) // 512, 256 // b)), (b, m, n, room, parts)


def test_every_size_has_a_choice(ask):
    sides = (1, 2, 63, 64, 65, 129, 500, 1000, 3000, 8191, 20000, 65536)
    problems = [(b, m, n, int(m == n), (n + 63) // 64) for b in (1, 7, 300, 65535) for m in sides for n in sides
                if m <= n and b * ((m + 63) // 64) * ((n + 63) // 64) < 1 << 24]
    for problem, (choice, us, (_, parts)) in zip(problems, ask([(*p, 1 << 40) for p in problems])):
        assert 0 <= choice <= 4 and all(u > 0 for u in us) and 1 <= parts <= 256, problem
