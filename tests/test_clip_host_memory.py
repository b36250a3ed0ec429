"""sv_clip_gradients where the host has no memory for its table (no GPU needed)."""
import os
import subprocess
import sys

from speculative_decoding_verification_71_gb300 import build as svbuild

CODE = """
import ctypes, resource
import speculative_decoding_verification_71_gb300 as svp
lib = svp.load_library()
n = 4_000_000                                     # a table of 192 MB
at = (ctypes.c_void_p * n)(*range(1 << 20, (1 << 20) + 64 * n, 64))
sizes, dtypes = (ctypes.c_longlong * n)(*[16] * n), (ctypes.c_int * n)()
held = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (held + (32 << 20), resource.getrlimit(resource.RLIMIT_AS)[1]))
# norm and work overlap: with the memory at hand the answer would be INVALID_ARG, and nothing launched
st = lib.sv_clip_gradients(n, at, sizes, dtypes, 0, 1.0, None, None, ctypes.c_void_p(64), ctypes.c_void_p(64), None)
print("status", st)
"""


def test_no_host_memory_is_not_a_bad_argument():
    svbuild.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300, cwd=root)
    assert "status 6" in out.stdout, (out.stdout, out.stderr[-2000:])       # SV_ERR_CUDA
