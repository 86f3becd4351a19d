"""The per-stream scratch on the host: csrc/stream_context.cu compiled as plain C++ with
stand-ins for the CUDA calls it makes (stream_context_check.cpp), so that what is
allocated, kept and freed, and which calls wait for which, can be counted."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "gated_deltanet_linear_chunked_b200", "csrc")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("stream_context") / "check")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-g", "-Wno-deprecated-declarations", "-I", CSRC,
                    "-I", os.path.join(ROOT, "include"), "-isystem", cuda, "-x", "c++",
                    os.path.join(CSRC, "stream_context.cu"), os.path.join(HERE, "stream_context_check.cpp"), "-o", path,
                    "-lpthread"], check=True)
    return path


@pytest.mark.parametrize("check", ["creeping", "graphs", "release", "failures", "threads"])
def test_stream_context(program, check):
    r = subprocess.run([program, check], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
