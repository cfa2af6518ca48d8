"""The host side of the cache operators (argument checks, sizes, cuts) built
with AddressSanitizer and UndefinedBehaviorSanitizer, host code only, linked
with the sanitized objects of the rest of the library and run through the host
ABI tests (CPU only)."""
import os
import subprocess
import sys

from tests import host_sanitize as h

OUT = os.path.join(h.ROOT, "_build", "host_asan_kv")
LIB = os.path.join(OUT, "libsvdq.so")


def _build():
    others = [os.path.join(h.OUT, n + ".o") for n in ("svdq_kernels", "svdq_probe", "svdq_pack", "svdq_svd")]
    if not all(os.path.exists(o) for o in others):
        h.build()
    os.makedirs(OUT, exist_ok=True)
    objs = []
    for name in ("svdq_kv_rows", "svdq_kv_attn"):
        objs.append(os.path.join(OUT, name + ".o"))
        subprocess.run([h.HIPCC, "--offload-arch=gfx950", "-ffp-contract=off"] + h.COMMON + h.HOST_SAN +
                       ["-c", os.path.join(h.CSRC, name + ".hip"), "-o", objs[-1]], check=True, capture_output=True)
    subprocess.run([h.CLANGXX, "-shared", "-fPIC", "-shared-libsan", "-Xarch_host", "-fsanitize=address,undefined", "-o", LIB]
                   + objs + others + ["-L" + os.path.join(h.ROCM, "lib"), "-lamdhip64", "-lpthread"], check=True, capture_output=True)


def test_cache_operators_host_code_under_asan_and_ubsan():
    _build()
    env = dict(os.environ, SVDQ_LIBRARY=LIB, LD_PRELOAD=h.asan_runtime(),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0:exitcode=23",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1:exitcode=24")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-s", "-p", "no:cacheprovider", "tests/test_kv_host.py"], cwd=h.ROOT, env=env,
                       capture_output=True, text=True)
    assert r.returncode == 0, f"sanitized host tests failed (exit {r.returncode}):\n{r.stdout[-1500:]}\n{r.stderr[-4000:]}"
    assert " passed" in r.stdout and " failed" not in r.stdout
