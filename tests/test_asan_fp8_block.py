"""The host-side argument validation of the block-scaled FP8 entry points under
AddressSanitizer (CPU only, no GPU touched), as test_asan_host.py does for the others:
the sources that hold them, host half instrumented, linked with
tests/asan/fp8_block_driver.cpp.  The build is cached and redone when a source, a header,
the driver or the flags change."""

import concurrent.futures
import glob
import hashlib
import os
import subprocess

import pytest

host = pytest.importorskip("tests.test_asan_host")

DRIVER = os.path.join(host.ROOT, "tests", "asan", "fp8_block_driver.cpp")
OUT = os.path.join(host.OUT, "fp8_block")
SOURCES = [os.path.join(host.PKG, "csrc", f) for f in ("norm_fp8.hip", "gemm_block8.hip", "status.hip")]


def _build():
    headers = sorted(glob.glob(os.path.join(host.PKG, "csrc", "*.h")) +
                     glob.glob(os.path.join(host.ROOT, "include", "*.h")))
    h = hashlib.sha256(" ".join(host.FLAGS).encode())
    for f in SOURCES + headers + [DRIVER]:
        h.update(f.encode())
        h.update(open(f, "rb").read())
    exe, stamp = os.path.join(OUT, "driver"), os.path.join(OUT, "stamp")
    if os.path.exists(exe) and os.path.exists(stamp) and open(stamp).read() == h.hexdigest():
        return exe
    os.makedirs(OUT, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(OUT, os.path.basename(src) + ".o")
        r = subprocess.run([host.HIPCC] + host.FLAGS + ["-c", src, "-o", obj], capture_output=True,
                           text=True)
        assert r.returncode == 0, f"{src}:\n{r.stderr[-3000:]}"
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_one, SOURCES + [DRIVER]))
    link = [a for a in host.FLAGS if "sanitize" in a or a.startswith("--offload")]
    link = [b for a in link for b in (("-Xarch_host", a) if "sanitize" in a else (a,))]
    r = subprocess.run([host.HIPCC] + link + objs + ["-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    open(stamp, "w").write(h.hexdigest())
    return exe


def test_validation_under_address_sanitizer():
    if not os.path.exists(host.HIPCC):
        pytest.skip("hipcc not available")
    exe = _build()
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    assert r.returncode == 0 and " 0 failures" in r.stdout, r.stdout + r.stderr[-4000:]
