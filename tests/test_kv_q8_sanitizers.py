"""The 8-bit cache's and the step tables' argument checks under clang's AddressSanitizer and UndefinedBehaviorSanitizer
(host code only, no GPU), as test_kv_sanitizers does it for the other caches."""
from __future__ import annotations

import glob
import os
import subprocess
import tempfile

import pytest

from lora_bgmv_shrink_amd import build as hb
from test_sanitizers import _run


def test_argument_checks_under_asan_ubsan():
    rt = glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so")
    if not rt:
        pytest.skip("clang's AddressSanitizer runtime is not installed")
    objs = [os.path.join(hb.BUILD_DIR, os.path.splitext(s)[0] + ".o") for s in hb.SOURCES]
    if not all(os.path.exists(o) for o in objs):
        hb.build()
    with tempfile.TemporaryDirectory() as d:
        san = ("-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
               "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer")
        checked = hb._compile("kv_api.hip", False, d, san)
        objs = [checked if os.path.basename(o) == "kv_api.o" else o for o in objs]
        lib = os.path.join(d, "liblora_san.so")
        r = subprocess.run([hb.HIPCC, "--offload-arch=" + hb.ARCH, "-shared", "-fPIC", *san, *objs, "-o", lib],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        print(_run(["tests/test_kv_q8_abi.py"], {"LORA_MI355X_LIB": lib, "LD_PRELOAD": rt[0]})[-300:])
