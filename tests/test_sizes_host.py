"""The sizing helpers refuse sizes that no call takes, instead of overflowing on them. CPU only; each call in a process of
its own, so that one that ends the process fails its test alone."""
import ctypes
import subprocess
import sys

import pytest

BIG, HALF = (1 << 31) - 1, 1 << 30
CALLS = [
    ("fa_cross_num_splits", (HALF, HALF, 4096, 1000)),       # 2^64 work units
    ("fa_cross_num_splits", (1 << 16, 1 << 16, 1, 1)),
    ("fa_cross_num_splits", (1, 1 << 20, BIG, 1)),
    ("fa_kvq8_num_parts", (4, 1 << 28, 1, 16, 1000, 128)),   # 2^32 rows to a K/V head
    ("fa_kvq8_num_parts", (1 << 20, 1 << 12, 1, 1, 1000, 64)),
    ("fa_kvq8_num_parts", (4, 8, 8, 1, BIG, 128)),           # more positions than a cache has
    ("fa_kvq8_num_parts", (HALF, HALF, HALF, 16, 1000, 128)),
    ("fa_kvq8_num_parts", (1 << 14, 1 << 10, 1 << 10, 1, HALF, 64)),
    ("fa_kvq8_workspace_bytes", (1 << 28, 1, 16, 128, 4)),
    ("fa_kvq8_workspace_bytes", (8, 8, 1, 128, (1 << 20) + 1)),
    ("fa_bwd_cross_workspace_bytes", (HALF, HALF, HALF, HALF, HALF, 64)),
    ("fa_bwd_cross_workspace_bytes", (1 << 14, 64, 64, 5, HALF, 64)),
]


@pytest.mark.parametrize("name,args", CALLS)
def test_sizes_that_no_call_takes_are_refused(name, args):
    from io_aware_exact_13_gb300 import build

    lib = build.build()
    code = (f"import ctypes; f = ctypes.CDLL({lib!r}).{name}; f.restype = ctypes.c_longlong; "
            f"print(f(*[ctypes.c_int(a) for a in {args!r}]))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert ctypes.c_int(int(r.stdout)).value == -3  # FA_ERR_SHAPE
