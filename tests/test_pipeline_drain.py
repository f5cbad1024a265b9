"""How the products wait for their loads in flight after a wait has run out, on
the CPU: the arithmetic that the kernels compile (csrc/pipeline_drain.h) in a
model of their rings, with random interleavings and waits that give up at
random."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fp8_microscaling_quantization_b200", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("drain") / "pipeline_drain_model")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-Wall", "-I", CSRC, "-o", exe,
                           os.path.join(HERE, "pipeline_drain_model.cpp")])

    def run(*args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout + r.stderr
        w = r.stdout.split()
        return int(w[2]), int(w[-1])

    return run


# CTAs, roles that store in each, stages: the block-scaled product's single
# CTAs and pairs, the dequantizing product's
RINGS = [(1, 1, 7), (1, 1, 3), (2, 1, 4), (2, 1, 5), (1, 16, 4), (2, 16, 4)]


@pytest.mark.parametrize("ring", RINGS)
def test_no_load_is_in_flight_after_the_drain(model, ring):
    gave_up, left = model(*ring, 20000, 1)
    assert gave_up > 2000 and left == 0


@pytest.mark.parametrize("ring", RINGS)
def test_a_drain_that_goes_by_the_load_role_alone_leaves_loads_in_flight(model, ring):
    gave_up, left = model(*ring, 20000, 0)
    assert gave_up > 2000 and left > 0


@pytest.mark.parametrize("name", ["scaled_mm.cu", "grouped_mm.cu"])
def test_the_products_drain_by_the_counts(name):
    """A kernel decides on the drain when its roles have joined (the CTA's last
    barrier but one), by the arithmetic that the model checks."""
    with open(os.path.join(CSRC, name)) as f:
        src = f.read()
    assert '#include "pipeline_drain.h"' in src and "phase_debt(" in src and "drain_first(" in src
    assert src.rindex("drain_loads<") > src.rindex("mbar_wait(sh.drain")
