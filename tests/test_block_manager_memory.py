"""The host block manager when memory runs out: a status code, no exception across the C entry."""
import os
import subprocess
import sys

import pytest

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_store_gb300",
                   "libpkvd.so")

CHILD = """
import ctypes, resource, sys
lib = ctypes.CDLL(sys.argv[1])
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (1 << 29), resource.RLIM_INFINITY))
out = ctypes.c_void_p(1)
# the arrays of 2^31 - 1 blocks alone, then those of the names of 2^24
for n in (2 ** 31 - 1, 2 ** 24):
    assert lib.pkvd_bm_create(n, 16, ctypes.byref(out)) == 6 and out.value is None, n
assert lib.pkvd_bm_create(8, 16, ctypes.byref(out)) == 0 and out.value
lib.pkvd_bm_destroy(out)
"""


def test_a_pool_larger_than_memory_is_refused():
    if not os.path.exists(LIB):
        pytest.skip("library not built")
    r = subprocess.run([sys.executable, "-c", CHILD, LIB], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
