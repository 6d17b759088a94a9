"""The block operators' argument checks under AddressSanitizer and UndefinedBehaviorSanitizer.

Builds as test_abi_sanitize.py does: api.hip with both sanitizers on its host code
only, linked with the library's other objects, and a C driver
(block_ops_sanitize_main.c) whose calls all end before the device."""
import os
import subprocess

from tests.conftest import ROOT
from tests.test_abi_sanitize import CLANG, HIPCC, SAN, objects  # noqa: F401  (a fixture)


def test_block_ops_under_asan_and_ubsan(objects, tmp_path):  # noqa: F811
    b, objs = objects
    api_obj, lib, exe = (str(tmp_path / n) for n in ("api_san.o", "libmoe_w4_san.so", "check"))
    subprocess.run([HIPCC, *b.CFLAGS, *SAN, "-c", os.path.join(b.CSRC, "api.hip"), "-o", api_obj],
                   check=True, capture_output=True, text=True)
    others = [o for o in objs if not o.endswith(os.sep + "api.o")]
    subprocess.run([HIPCC, f"--offload-arch={b.ARCH}", "-mcode-object-version=5", "-shared", "-fPIC", *SAN,
                    "-o", lib, api_obj, *others], check=True, capture_output=True, text=True)
    flags = [f for f in SAN if f != "-Xarch_host"]
    subprocess.run([CLANG, *flags, os.path.join(ROOT, "tests", "block_ops_sanitize_main.c"),
                    "-I", os.path.join(ROOT, "include"), "-o", exe, lib, f"-Wl,-rpath,{tmp_path}"],
                   check=True, capture_output=True, text=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "ok" in r.stdout
