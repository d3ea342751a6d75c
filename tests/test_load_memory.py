"""A load that the host has no memory for is an error code: no C++ exception
leaves the C entry point.  Each attempt runs in a process of its own with a
little more address space than the last one; without a GPU, where a load that
gets through ends with TOK_ECUDA."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import ctypes, resource, sys
import numpy as np
import exact_bpe_tokenization_utf_gb300 as pkg
L = pkg.lib()
n = 60_000
ids = np.arange(n - 256)
toks = np.zeros((n - 256, 12), np.uint8)
for k in range(12):
    toks[:, k] = 97 + (ids >> (2 * k)) % 4
blob = np.concatenate([np.arange(256, dtype=np.uint8), toks.reshape(-1)])
off = np.concatenate([np.arange(256), 256 + 12 * np.arange(n - 256 + 1)]).astype(np.uint64)
h = ctypes.c_void_p()
args = (blob.ctypes.data_as(ctypes.POINTER(ctypes.c_uint8)), off.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)), n, None, 0,
        pkg.PATTERN_GPT2, ctypes.byref(h))
size = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (size + int(sys.argv[1]), resource.RLIM_INFINITY))
rc = L.tok_load(*args)
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
print("rc", rc, bool(h.value))
"""


def test_a_load_without_memory_is_an_error_code():
    import torch
    if torch.cuda.is_available():
        pytest.skip("with a GPU the limit would be that of CUDA itself too")
    from exact_bpe_tokenization_utf_gb300 import TOK_ECUDA, TOK_ENOMEM, _build
    _build.build()
    codes = []
    for more in (0, 1 << 20, 3 << 20, 6 << 20, 9 << 20, 12 << 20, 1 << 30):
        r = subprocess.run([sys.executable, "-c", CHILD, str(more)], capture_output=True, text=True, timeout=120,
                           cwd=ROOT, env={**os.environ, "PYTHONPATH": ROOT})
        assert r.returncode == 0, (more, r.returncode, r.stderr[-500:])
        word, code, handle = r.stdout.split()
        assert word == "rc" and handle == "False"
        codes.append(int(code))
    assert codes[0] == TOK_ENOMEM and codes[-1] == TOK_ECUDA and set(codes) == {TOK_ENOMEM, TOK_ECUDA}, codes
