"""The host's fractions of a turn (rotary_phase.h, compiled by itself) against exact fractions."""
import ctypes
import math
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from oracle.serving import TWO_PI

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_28_gb300", "csrc")


@pytest.fixture(scope="module")
def phase(tmp_path_factory):
    where = tmp_path_factory.mktemp("phase")
    (where / "phase.cpp").write_text('#include "rotary_phase.h"\n'
                                     'extern "C" uint64_t phase(double f) { return fa::rotary_phase(f); }\n')
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, str(where / "phase.cpp"), "-o",
                    str(where / "phase.so")], check=True)
    lib = ctypes.CDLL(str(where / "phase.so"))
    lib.phase.restype, lib.phase.argtypes = ctypes.c_uint64, [ctypes.c_double]
    return lib.phase


def off(phase, f):
    """Distance of the phase from f / (2 pi), modulo a turn, in units of 2^-64."""
    d = (phase(f) - Fraction(f) / TWO_PI * 2 ** 64) % 2 ** 64
    return float(min(d, 2 ** 64 - d))


@pytest.mark.parametrize("base,rot", [(500000.0, 128), (10000.0, 128), (10000.0, 64), (100.0, 48), (1e6, 16)])
def test_phases_of_a_base_are_the_nearest(phase, base, rot):
    # half a unit, and what the sum's own unit of 2^-96 leaves open
    assert max(off(phase, base ** (-2.0 * c / rot)) for c in range(rot // 2)) <= 0.5 + 2.0 ** -20


def test_phases_of_any_frequency_are_the_nearest(phase):
    rng = np.random.default_rng(3)
    some = np.concatenate([rng.uniform(-10, 10, 500), 2.0 ** rng.uniform(-80, 40, 500), -(2.0 ** rng.uniform(-80, 40, 500)),
                           [0.0, -0.0, math.pi, 2 * math.pi, -math.pi / 2, 1000.25, 1e-9, 2.0 ** 40, 5e-324]])
    # TWO_PI's 50 digits are good to 2^-160, the largest frequency's turns to 2^-120
    assert max(off(phase, float(f)) for f in some) <= 0.5 + 2.0 ** -20


def test_phases_of_huge_frequencies_are_numbers(phase):
    for f in (1e300, -1e308, 2.0 ** 1023):
        assert 0 <= phase(f) < 2 ** 64
