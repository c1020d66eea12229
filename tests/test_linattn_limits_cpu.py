"""The linear-attention calls at the ends of what their arguments can name, on
the host: plans, limits and the kernels that a call can reach, built with g++
and the host sanitizers against stand-in launchers."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "structured_sparse_state_pdssm_amd", "csrc")
SAN = os.path.join(ROOT, "tests", "sanitize")
HIP_INC = "/opt/rocm/include"
pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(HIP_INC),
                                reason="needs g++ and the HIP headers")


def run(tmp_path, name, *more, std="c++17"):
    """Build tests/sanitize/<name>.cpp (with the C ABI where asked for) and run it; its output."""
    exe = str(tmp_path / name)
    cmd = ["g++", f"-std={std}", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", f"-I{HIP_INC}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", *more,
           os.path.join(SAN, name + ".cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok: 0 failures" in r.stdout, r.stdout + r.stderr
    return r.stdout


API = os.path.join(CSRC, "pdscan_linattn_api.cpp")


def test_workspace_queries_of_extreme_sizes(tmp_path):
    """Jobs, slabs and heads multiply past 32 bits: refused, not divided by what is left of the product."""
    run(tmp_path, "linattn_sizes", API)


def test_segment_table_of_any_offsets(tmp_path):
    """The table's kernel lane by lane: entries of offsets in order, and nothing written outside the table where the
    offsets ask for more segments than 32 bits count."""
    run(tmp_path, "linattn_table", "-pthread", std="c++20")


def test_grids_of_the_largest_calls(tmp_path):
    """No launch of 2^32 threads along an axis, whatever the sizes; query and call agree; what is refused is refused
    before its first launch."""
    run(tmp_path, "linattn_grids", API)


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
def test_every_kernel_built_is_reached(tmp_path):
    """The library holds the product and state kernels that some call launches, and no others."""
    import re

    from tests._libutil import ensure_built
    reached = {ln for ln in run(tmp_path, "linattn_reached", API).splitlines() if "kernel<" in ln}
    names = subprocess.run(["nm", "-C", ensure_built()], capture_output=True, text=True, timeout=60).stdout
    built = {re.sub(r"pdscan::", "", m) for m in re.findall(r"__device_stub__pdssm_linattn_((?:state_)?kernel<(?:pdscan::La)[^>]*>)", names)}
    assert built == reached, (sorted(built - reached), sorted(reached - built))
