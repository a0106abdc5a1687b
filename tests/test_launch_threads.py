"""The launches' host side from two threads at once, under ThreadSanitizer and without a GPU
(see _launch_threads.cu)."""

import concurrent.futures as cf
import os
import subprocess

import pytest

from moe_expert_ffn_scan_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))
TSAN = ["-Xcompiler", "-fsanitize=thread,-g"]


def _run(cmd, **kw):
    return subprocess.run(cmd, capture_output=True, text=True, timeout=600, **kw)


@pytest.fixture(scope="module")
def sanitizer(tmp_path_factory):
    """A folder to build in, where the sanitizer works."""
    d = tmp_path_factory.mktemp("threads")
    (d / "probe.cpp").write_text("int main() { return 0; }\n")
    r = _run(["g++", "-fsanitize=thread", str(d / "probe.cpp"), "-o", str(d / "probe")])
    if r.returncode or _run([str(d / "probe")]).returncode:
        pytest.skip("ThreadSanitizer does not run here")
    return d


def test_first_calls_of_two_threads(sanitizer):
    d = sanitizer
    flags = ["-gencode", "arch=compute_103a,code=compute_103a", *build.FLAGS, "-I" + build.CSRC]
    sources = [*[os.path.join(build.CSRC, s) for s in
                 ("linear.cu", "norm.cu", "balance.cu", "gemm.cu", "gemm_nv.cu", "router.cu")],
               os.path.join(HERE, "_launch_threads.cu")]
    objs = [str(d / os.path.basename(s)) + ".o" for s in sources]
    with cf.ThreadPoolExecutor(len(sources)) as ex:
        for r in ex.map(lambda so: _run([build.nvcc(), *flags, *TSAN, "-c", so[0], "-o", so[1]]),
                        zip(sources, objs)):
            assert r.returncode == 0, r.stderr
    cc = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=thread"]
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    objs.append(str(d / "fake.o"))
    r = _run([*cc, "-I" + cuda, "-c", os.path.join(HERE, "_fake_cudart.cpp"), "-o", objs[-1]])
    assert r.returncode == 0, r.stderr
    exe = str(d / "threads")
    r = _run([*cc, *objs, "-o", exe, "-lpthread"])
    assert r.returncode == 0, r.stderr
    r = _run([exe])
    assert r.returncode == 0, r.stdout + r.stderr[:4000]
