"""A pool that the host has no memory for is refused; no exception leaves the C entry (CPU, in a
process of its own whose address space is bounded)."""
import os
import subprocess
import sys

import pytest

CHILD = """
import ctypes, resource, sys
lib = ctypes.CDLL(sys.argv[1])
lib.carat_pool_create.restype = ctypes.c_void_p
lib.carat_pool_create.argtypes = [ctypes.c_int, ctypes.c_int]
lib.carat_pool_destroy.argtypes = [ctypes.c_void_p]
held = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (held + (1 << 30),) * 2)
# bytes a page: 1 and 4, and 5 for a block of one
for pages, ring in ((2 ** 31 - 1, 1), (2 ** 31 - 1, 2 ** 30), (3 * 10 ** 8, 1), (15 * 10 ** 7, 1)):
    print(lib.carat_pool_create(pages, ring))
pool = lib.carat_pool_create(1000, 4)
print(pool is not None)
lib.carat_pool_destroy(pool)
"""


def test_no_memory_for_a_pool():
    from sliding_window_gqa_ring_gb300 import build, carat
    if not os.path.exists(carat.LIBRARY):
        build.build()
    if not os.path.exists("/proc/self/statm"):
        pytest.skip("no /proc")
    got = subprocess.run([sys.executable, "-c", CHILD, carat.LIBRARY], capture_output=True,
                         text=True, timeout=120)
    assert got.returncode == 0, got.stderr
    assert got.stdout.split() == ["None"] * 4 + ["True"]
