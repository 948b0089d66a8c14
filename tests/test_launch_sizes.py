"""CPU: whatever sizes the checks accept can be launched.  A driver
(tests/launch/launch_driver.cpp) calls the library at the ends of them with a
hipLaunchKernel of its own that records the grid and launches nothing."""
import ctypes as C
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "gated_deltanet_decode_amd")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = tmp_path_factory.mktemp("launch") / "launch_driver"
    # -rdynamic: the program's hipLaunchKernel is found before the runtime's
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-rdynamic", "-I", os.path.join(ROOT, "include"),
                           os.path.join(ROOT, "tests", "launch", "launch_driver.cpp"), os.path.join(LIB, "libgdn.so"),
                           f"-Wl,-rpath,{LIB}", "-Wl,-rpath,/opt/rocm/lib", "-Wl,-rpath-link,/opt/rocm/lib", "-o", str(exe)])
    return str(exe)


def fits(driver, which):
    r = subprocess.run([driver, which], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "every launch fits" in r.stdout, r.stdout[-500:] + r.stderr[-3000:]


def test_recurrent_layer(driver):
    fits(driver, "lru")


def test_norms(driver):
    fits(driver, "norms")


def test_the_largest_workspaces_serve_smaller_calls():
    """Where the gradient goes from one tile to another near the limit, its workspace's size still does not fall."""
    lib = C.CDLL(os.path.join(LIB, "libgdn.so"))
    size = lib.gdn_lru_backward_workspace_bytes
    size.restype, size.argtypes = C.c_size_t, [C.c_void_p, C.c_int32]
    room = lambda B, W, T, act: size((C.c_int32 * 3)(B, W, act), T)
    r, most = random.Random(5), 0
    for _ in range(20000):
        W, T = 8 * r.choice([1, 8, 9, 16, 17, 24, 25, 33, 40, 512, r.randint(1, 200)]), int(2 ** r.uniform(0, 22))
        B = int(((1 << 23) - 1) / (-(-W // 64) * -(-T // 64)) / 2 ** r.uniform(0, 2))
        if B < 2:
            continue
        for act in (0, 1):
            now = room(B, W, T, act)
            assert now
            most = max(most, now)
            for less in ((B - 1, W, T), (B // 2, W, T), (B, W - 8, T), (B, W // 16 * 8, T), (B, W, T - 1), (B, W, T // 2)):
                if min(less):
                    assert room(*less, act) <= now, ((B, W, T), less)
    assert most > 1 << 33
