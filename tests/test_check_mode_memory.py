"""Check mode copies index arrays to the host: where the host has no memory for them the call is answered, the process
lives on.  No GPU: the copies' space is asked for first."""
import subprocess
import sys

import pytest

SCRIPT = """
import ctypes, resource, sys
from paged_kv_cache_116_gb300 import _binding
lib = _binding.lib()
lib.pa_set_check_mode(1)
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (1 << 30), used + (1 << 30)))
P, BIG = ctypes.c_void_p, 2 ** 31 - 1
one, to = P(16), P(32)
ws = (one, 1 << 62, None)
def rope(): return lib.pa_rope_write_kv(to, one, one, one, 1024, 256, 256, one, 1, one, None, 128, 0, one, BIG, one, one,
                                        10, 16, 8, 2, 128, 1, None)
def decode(): return lib.pa_decode_weights(one, one, 64, one, one, one, one, 4, one, BIG, 8, 2, 128, 10, 16, 64, 1.0, 1,
                                           *ws)
def prompt(): return lib.pa_prompt_weights(one, 64, one, one, one, 4, one, one, BIG, 8, 6, 8, 2, 128, 10, 16, 64, 0, 1.0,
                                           1, 1, *ws)
def plain(): return lib.pa_decode(one, one, one, one, one, 4, one, BIG, 8, 2, 128, 10, 16, 64, 1.0, 1, *ws)
def varlen(): return lib.pa_varlen(one, one, one, one, one, 4, one, one, BIG, 8, 6, 8, 2, 128, 10, 16, 64, 1.0, 1, 1, *ws)
def write(): return lib.pa_write_kv(one, one, one, BIG, one, one, 10, 16, 2, 128, 1, None)
print(locals()[sys.argv[1]](), lib.pa_last_error().decode())
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_116_gb300 import build

    build.build()


@pytest.mark.parametrize("call", ["rope", "decode", "prompt", "plain", "varlen", "write"])
def test_no_host_memory_for_the_indices(call):
    r = subprocess.run([sys.executable, "-c", SCRIPT, call], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-500:]
    assert r.stdout.startswith("1 ") and "host memory" in r.stdout, r.stdout
