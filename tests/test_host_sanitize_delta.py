"""The host code of libfalcon_block under AddressSanitizer and UndefinedBehaviorSanitizer:
its C layer and the host parts of the kernels' files (plans, workspaces, launch shapes), with
tests/host_sanitize_delta_driver.cpp.  Only host code is compiled here; on a machine without a
GPU every launch reports FALCON_ERR_HIP.
"""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "weight_recurrent_memory_amd", "csrc")
INCLUDE = os.path.join(ROOT, "include")
DRIVER = os.path.join(ROOT, "tests", "host_sanitize_delta_driver.cpp")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
SKIP_EXIT = 77          # the driver's exit status where a GPU is present


def _run(cmd, **kw):
    res = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert res.returncode == 0, "%s\n%s\n%s" % (" ".join(cmd), res.stdout[-3000:], res.stderr[-3000:])
    return res.stdout


def test_every_entry_point_is_called():
    with open(os.path.join(INCLUDE, "falcon_block.h")) as f:
        declared = set(re.findall(r"\b(falcon_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)))
    with open(DRIVER) as f:
        called = set(re.findall(r"\b(falcon_\w+)\s*\(", re.sub(r"//.*", "", f.read())))
    assert len(declared) >= 7 and declared <= called, declared - called


def test_host_code_under_asan_and_ubsan(tmp_path):
    if not os.path.exists(HIPCC) or not all(shutil.which(x) for x in ("g++", "nm")):
        pytest.skip("hipcc, g++ or nm not available")
    from weight_recurrent_memory_amd import build_lib
    objs, fatbins = [], set()
    for src in build_lib.BLOCK_SOURCES:
        obj = str(tmp_path / (src + ".o"))
        _run([HIPCC, "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950", "--offload-host-only",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I" + INCLUDE, "-I" + CSRC]
             + "-Xarch_host -fsanitize=address -Xarch_host -fsanitize=undefined "
               "-Xarch_host -fno-omit-frame-pointer".split()
             + ["-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj])
        objs.append(obj)
        fatbins |= set(re.findall(r"U (__hip_fatbin_\w+)", _run(["nm", obj])))
    drv, exe = str(tmp_path / "driver.o"), str(tmp_path / "driver")
    sanitize = ["-fsanitize=address,undefined", "-fno-omit-frame-pointer"]
    _run(["g++", "-O1", "-g", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + INCLUDE]
         + sanitize + ["-c", DRIVER, "-o", drv])
    _run(["g++"] + sanitize + ["-o", exe, drv] + objs
         + ["-Wl,--defsym=%s=no_device_code" % f for f in sorted(fatbins)]
         + ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = res.stdout + res.stderr
    if res.returncode == SKIP_EXIT:
        pytest.skip("a GPU is present: the driver's stand-in pointers are host memory")
    print(out[-2000:])
    assert "AddressSanitizer" not in out and "runtime error" not in out
    assert res.returncode == 0 and " 0 failures" in out
