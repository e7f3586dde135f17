"""What the 4-bit products do when a wait runs out: nothing of theirs is under way any more when a CTA leaves, and a warp that
works as one gives up as one."""
import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "matrix_orthogonalizing_optimizer_gb300", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("ring") / "ring_model")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, os.path.join(HERE, "ring_model.cc"), "-o", out], check=True)
    return out


def test_loads_have_landed_when_a_group_leaves(model):
    r = subprocess.run([model], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout


def test_without_the_last_wait_loads_are_in_flight(model):
    r = subprocess.run([model, "0"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 1 and "in flight" in r.stdout


def test_the_kernel_settles_before_it_frees_its_memory():
    text = re.sub(r"//.*", "", open(os.path.join(CSRC, "fp4_gemm.cu")).read())
    kernel = text[text.index("fp4_gemm_kernel(const"):text.index("PFN_cuTensorMapEncodeTiled_v12000 encoder")]
    assert 0 < kernel.index("settle_ring(") < kernel.index("tmem_dealloc")
    # the MMA issuer and the epilogue are whole warps: only the producer, one lane, waits by itself
    alone = re.findall(r"(?<!_)fp4_wait\(&(\w+)", text)
    assert alone == ["empty"], alone
    assert sorted(re.findall(r"fp4_warp_wait\(&(\w+)", text)) == ["cbar", "full", "tempty", "tfull"]
