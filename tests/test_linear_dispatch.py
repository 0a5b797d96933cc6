"""The Linear's choice between its two kernels, and the sizes it refuses, without a GPU (the launchers are stubs)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, SHAPE = 0, 2

pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                                reason="needs g++ and the HIP headers")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("linear") / "driver")
    csrc = os.path.join(ROOT, "fp8_fine_grained_amax_amd", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
                        os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "ffn_api.cpp"),
                        os.path.join(ROOT, "tests", "linear_dispatch_driver.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(stream_us, tiles_us, M, N, K, tile=None):
        env = {k: v for k, v in os.environ.items() if k != "FG_GEMM_TILE"}
        if tile:
            env["FG_GEMM_TILE"] = tile
        r = subprocess.run([exe], input=f"{stream_us} {tiles_us} {M} {N} {K}\n", capture_output=True, text=True, timeout=60, env=env)
        assert r.returncode == 0, r.stderr
        status, launched = r.stdout.split()
        return int(status), launched
    return ask


@pytest.mark.parametrize("M,N,K,fits", [
    (1 << 31, 1, 0, False),                            # 2^24 workgroups of 256 threads
    ((1 << 31) - 128, 1, 0, True),
    ((1 << 31) - 127, 128, 128, False),
    (1, 1 << 31, 128, False),
    (128, (1 << 31) - 128, 128, True),
    (1 << 31, 1 << 31, 128, False),
    (5592405 * 256, 192, 0, False),                    # two columns of 128x128
    (5592405 * 256 + 1, 129, 0, False),
    (5592405 * 256 + 1, 128, 0, True),                 # one column
    (1 << 62, 1, 128, False),
    (1, 1 << 62, 0, False),
])
def test_launches_past_32_bits_of_threads_are_refused(driver, M, N, K, fits):
    assert driver(2, 1, M, N, K) == ((OK, "tiles") if fits else (SHAPE, "-"))


def test_a_forced_tile_is_held_to_its_own_threads(driver):
    M = 5592405 * 256 + 1
    assert driver(2, 0, M, 128, 0, tile="256x192") == (SHAPE, "-")
    assert driver(2, 0, M - 1, 128, 0, tile="256x192") == (OK, "tiles")


@pytest.mark.parametrize("M", [1, 4096, 4097, 8192, 100000, 65535 * 16])
def test_the_estimates_choose_at_any_number_of_rows(driver, M):
    assert driver(1, 2, M, 64, 7168) == (OK, "stream")
    assert driver(2, 1, M, 64, 7168) == (OK, "tiles")


@pytest.mark.parametrize("M,N", [(1, 18432), (4096, 18432), (4096, 257), (4097, 257), (8192, 512)])
def test_many_rows_and_columns_go_to_the_tiles(driver, M, N):
    assert driver(1, 2, M, N, 2048) == (OK, "stream" if M <= 4096 else "tiles")


def test_rows_past_a_grid_go_to_the_tiles(driver):
    assert driver(1, 2, 65535 * 16 + 1, 64, 7168) == (OK, "tiles")


@pytest.fixture(scope="module")
def estimates(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("estimates") / "driver")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "fp8_fine_grained_amax_amd", "csrc"),
                        os.path.join(ROOT, "tests", "stream_estimate_driver.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return lambda *sizes: subprocess.run([exe, *map(str, sizes)], capture_output=True, text=True, timeout=60)


def test_no_estimate_beats_the_memory(estimates):
    r = estimates()
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("M,N,K,us", [
    (8192, 1024, 128, 15.5), (16384, 512, 128, 15.5), (65536, 256, 128, 29.4), (512, 5952, 256, 9.0), (512, 5952, 512, 10.5),
    (1024, 5952, 512, 17.2), (4096, 2944, 512, 30.1), (16384, 256, 2048, 31.2), (8192, 512, 7168, 85.6),     # 64x32
    (4096, 8, 16384, 14.3), (8192, 16, 7168, 12.7), (16384, 8, 16384, 48.9)])                                # narrow outputs
def test_estimates_near_measured_times(estimates, M, N, K, us):
    """Times of the kernel on an MI355X; boxes and runs differ by up to a tenth, the estimates' steps are as coarse again."""
    assert 0.8 * us <= float(estimates(M, N, K).stdout) <= 1.25 * us
