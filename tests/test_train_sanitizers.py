"""The argument checks of include/hq_train.h under the host AddressSanitizer and
UndefinedBehaviorSanitizer: hq_train_api.cpp with stand-ins for the kernel launchers, under
tests/test_train_abi.py (CPU only, no GPU code)."""
import os
import subprocess

import pytest

from test_sanitizers import CSRC, LIBASAN, ROOT, SAN, _run_pytest

pytestmark = pytest.mark.skipif(LIBASAN is None, reason="gcc's libasan is not available")


def test_train_abi_checks_under_sanitizers(tmp_path):
    objs = []
    for src in (os.path.join(CSRC, "hq_api.cpp"), os.path.join(CSRC, "hq_profile.cpp"),
                os.path.join(CSRC, "hq_train_api.cpp"),
                os.path.join(ROOT, "tests", "sanitize", "launcher_stubs.cpp"),
                os.path.join(ROOT, "tests", "sanitize", "train_launcher_stubs.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        subprocess.run(["g++", "-std=c++17", "-w", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                        "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include")] + SAN +
                       ["-c", src, "-o", obj], check=True)
        objs.append(obj)
    lib = str(tmp_path / "libhq_train_san.so")
    subprocess.run(["g++", "-shared"] + SAN + objs +
                   ["-L/opt/rocm/lib", "-lamdhip64", "-o", lib], check=True)
    _run_pytest({"HQ_LIB_PATH": lib, "HQ_TRAIN_LIB_PATH": lib}, [os.path.join("tests", "test_train_abi.py")])
