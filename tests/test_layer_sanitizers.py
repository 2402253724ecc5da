"""The history layer's host side under the host sanitizers (CPU only): emb_layer.cpp, with its buckets' whole-number
arithmetic, and emb_seq.cpp are compiled with AddressSanitizer and UndefinedBehaviorSanitizer (g++, host code only),
linked with launches that are counted instead of made, and driven over their arguments' whole range by a C harness. Any
report, leak or unexpected result fails the test."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dlrm_sparse_embedding_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "sanitize")
HIP_INCLUDE = "/opt/rocm/include"


@pytest.mark.skipif(shutil.which("g++") is None or shutil.which("gcc") is None or
                    not os.path.isdir(HIP_INCLUDE), reason="needs gcc/g++ and the HIP headers")
def test_layer_arguments_under_asan_ubsan(tmp_path):
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", HIP_INCLUDE, "-D__HIP_PLATFORM_AMD__"]
    objs = []
    for path in [os.path.join(CSRC, n) for n in ("emb_layer.cpp", "emb_seq.cpp", "emb_api.cpp", "emb_plan.cpp")] + \
                [os.path.join(HERE, n) for n in ("device_stubs.cpp", "layer_stubs.cpp", "layer_harness.c")]:
        obj = str(tmp_path / (os.path.basename(path) + ".o"))
        cc = ["g++", "-std=c++17"] if path.endswith(".cpp") else ["gcc", "-std=c11"]
        r = subprocess.run(cc + san + inc + ["-c", path, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        objs.append(obj)
    exe = str(tmp_path / "layer_harness")
    r = subprocess.run(["g++"] + san + objs + ["-lm", "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, f"harness failed ({r.returncode}):\n{r.stdout}\n{r.stderr}"
    assert "layer harness ok" in r.stdout
    assert "runtime error" not in r.stderr and "ERROR: AddressSanitizer" not in r.stderr, r.stderr
