"""No C++ exception leaves an entry point: host tables that cannot be allocated are an error code (CPU, in a child process)."""
from __future__ import annotations

import subprocess
import sys

from muon_newton_schulz_07_b200 import binding as B

CHILD = """
import ctypes, resource, sys
sys.path.insert(0, {root!r})
from muon_newton_schulz_07_b200 import binding as B
L = B.lib()
shapes = B._shapes([(256 + i, 300) for i in range(4096)])
out, problems = ctypes.c_size_t(0), ctypes.c_int64(0)
check = L.muon_check_plan
check.argtypes = [ctypes.POINTER(B.Shape), ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]
check.restype = ctypes.c_int
assert L.muon_workspace_size(shapes, 4096, 0, 0, ctypes.byref(out)) == B.MUON_OK and out.value > 0
with open("/proc/self/statm") as f:
    used = int(f.read().split()[0]) * 4096
resource.setrlimit(resource.RLIMIT_AS, (used + (1 << 20), resource.RLIM_INFINITY))
codes = [L.muon_workspace_size(shapes, 4096, 0, mode, ctypes.byref(out)) for mode in (0, 1, 2)]
codes.append(check(shapes, 4096, 5, 148, ctypes.byref(problems)))
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
codes.append(L.muon_workspace_size(shapes, 4096, 0, 0, ctypes.byref(out)))
print(codes)
"""


def test_memory_that_runs_out_is_an_error_code():
    root = B.LIB_PATH.rsplit("/", 2)[0]
    child = subprocess.run([sys.executable, "-c", CHILD.format(root=root)], capture_output=True, text=True, timeout=120,
                           env={"MALLOC_TRIM_THRESHOLD_": "0", "MALLOC_MMAP_THRESHOLD_": "65536", "PATH": "/usr/bin"})
    assert child.returncode == 0, child.stderr[-500:]
    codes = eval(child.stdout)
    assert codes[:4] == [B.MUON_ERR_INVALID_ARG] * 4 and codes[4] == B.MUON_OK
