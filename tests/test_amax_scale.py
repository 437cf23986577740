"""The checkpoints' group scale and its reciprocal, which the kernels work out in nine operations
instead of two divisions, have to be the correctly rounded quotients: on them rests that packed
bytes are the quantiser's. The function is taken out of csrc/block.hpp and compiled for the host,
where it is run over every float that a group's largest magnitude can be. No GPU involved."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
BLOCK = os.path.join(os.path.dirname(HERE), "blockwise_fp8_gemm_x128_amd", "csrc", "block.hpp")


def function():
    text = open(BLOCK).read()
    found = re.findall(r"^__device__ __forceinline__ void amax_scale\(.*?^}\n", text,
                       flags=re.S | re.M)
    assert len(found) == 1
    return "AMAX_SCALE " + found[0]


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    if " fma " not in open("/proc/cpuinfo").read():
        pytest.skip("no fused multiply-add on this host")
    tmp = tmp_path_factory.mktemp("amax")

    def make(text, name):
        (tmp / "amax_scale.inc").write_text(text)
        exe = str(tmp / name)
        subprocess.check_call([cxx, "-std=c++17", "-O3", "-Wall", "-mavx2", "-mfma", "-pthread",
                               "-ffp-contract=off", "-fno-fast-math", "-I" + str(tmp),
                               os.path.join(HERE, "amax_scale_check.cpp"), "-o", exe])
        return lambda lo, hi: subprocess.run([exe, str(lo), str(hi)], capture_output=True,
                                             text=True, timeout=110)
    return make


def test_every_scale_is_the_rounded_quotient(run):
    res = run(function(), "check")(-119, 128)
    assert res.returncode == 0 and res.stdout == "0 wrong of 247 binades\n", res.stdout + res.stderr


def test_the_check_finds_a_dropped_step(run):
    """Without the remainder's step a tenth of the quotients and more would be an ulp off."""
    text = function()
    plain = re.sub(r"s = __builtin_fmaf\(__builtin_fmaf\(-448\.0f, q, a\), c, q\);", "s = q;", text)
    assert plain != text
    res = run(plain, "dropped")(0, 1)
    assert res.returncode == 1 and int(res.stdout.split()[0]) > 3 * (1 << 23) // 10, res.stdout
