"""The library's own buffer of the linear-layer calls, followed on the CPU through stand-ins for
the HIP runtime's allocation calls (tests/hip_alloc_shim.c): a graph captured on it replays into
the address that it had at the capture, so that has to stay allocated until ozaki2_release."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# acquire the sizes in turn through oz2::acquire_linear_workspace, then release
PROGRAM = """
import ctypes, sys
lib = ctypes.CDLL(sys.argv[1])
acquire = lib._ZN3oz224acquire_linear_workspaceEmPPc
acquire.argtypes = [ctypes.c_size_t, ctypes.POINTER(ctypes.c_void_p)]
for need in map(int, sys.argv[2:]):
    base = ctypes.c_void_p()
    print("need", need, acquire(need, ctypes.byref(base)), hex(base.value or 0), flush=True)
print("release", lib.ozaki2_release(), flush=True)
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("shim") / "shim.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", out, os.path.join(ROOT, "tests", "hip_alloc_shim.c")], check=True)
    return out


def followed(shim, *needs, limit=1 << 40):
    from fp64_gemm_emulation_amd.build import LIB_PATH
    env = dict(os.environ, SHIM_LIMIT=str(limit))
    # something may be preloaded already
    env["LD_PRELOAD"] = " ".join(filter(None, [shim, env.get("LD_PRELOAD")]))
    out = subprocess.run([sys.executable, "-c", PROGRAM, LIB_PATH, *map(str, needs)], env=env, capture_output=True,
                         text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    return [line.split() for line in out.stdout.splitlines()]


def test_outgrown_buffers_stay_until_release(shim):
    log = followed(shim, 1000, 800, 5000, 6000, 100, 1 << 20)
    release = next(i for i, line in enumerate(log) if line[:2] == ["release", "0"])
    frees = [i for i, line in enumerate(log) if line[0] == "free"]
    allocs = [line[1] for line in log if line[0] == "alloc"]
    assert min(frees) > max(i for i, line in enumerate(log) if line[0] == "need")
    # everything is freed by the release, once
    assert sorted(log[i][1] for i in frees) == sorted(allocs) and max(frees) < release
    # every call got a buffer that holds it, and one that was large enough already was used again
    size = {line[1]: int(line[2]) for line in log if line[0] == "alloc"}
    got = [line for line in log if line[0] == "need"]
    assert all(line[2] == "0" and size[line[3]] >= int(line[1]) for line in got)
    assert got[0][3] == got[1][3] and got[3][3] == got[4][3]


def test_outgrown_buffers_do_not_add_up(shim):
    """A thousand calls, each a little larger: few buffers, together less than twice the last."""
    log = followed(shim, *range(100000, 1100000, 1000))
    sizes = [int(line[2]) for line in log if line[0] == "alloc"]
    assert len(sizes) <= 6 and sum(sizes[:-1]) <= sizes[-1] and sizes[-1] <= 2 * 1099000


def test_memory_runs_out(shim):
    log = followed(shim, 600, 1000, 2000, 900, limit=1100)
    got = [(line[2], line[3]) for line in log if line[0] == "need"]
    # twice 600 cannot be had, 1000 can; 2000 cannot, and what is there stays in use
    assert [rc for rc, _ in got] == ["0", "0", "3", "0"] and got[1][1] == got[3][1]
