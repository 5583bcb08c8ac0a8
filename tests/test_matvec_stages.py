"""The stages in which rows of x come to LDS (csrc/qcast_stages.h), compiled here
for the CPU: the kernel's loop over them ends, and reads what it holds."""
import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "precision_quantization_amd", "csrc")
KB = 1024


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("stages")
    (d / "s.cpp").write_text('#include "qcast_stages.h"\nextern "C" {\n'
                             "uint32_t units(uint32_t l, uint32_t r, uint32_t b, uint32_t o, uint32_t u) "
                             "{ return qcast::stage_units(l, r, b, o, u); }\n"
                             "uint32_t waves(uint32_t l, uint32_t r, uint32_t b, uint32_t u, uint32_t w) "
                             "{ return qcast::stage_waves(l, r, b, u, w); }\n}\n")
    so = d / "s.so"
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "s.cpp"), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    for f in (lib.units, lib.waves):
        f.argtypes, f.restype = [ctypes.c_uint32] * 5, ctypes.c_uint32
    return lib


def test_a_stage_is_whole_rounds_that_fit(lib):
    for lds in (0, 15, 16, 600, 17 * KB, 48 * KB, 112 * KB):
        for rows in range(1, 17):
            for unit in (512, 520, 544):
                fits = [u for u in range(1, 230) if rows * (u * unit + 16) <= lds]
                for rnd in (1, 2, 4, 8, 16, 32, 64):
                    for units in (1, 2, 3, rnd, rnd + 1, 57, 221, 65535):
                        got = lib.units(lds, rows, unit, rnd, units)
                        if units in fits:
                            assert got == units
                        else:
                            assert got == max([u for u in fits if u % rnd == 0], default=0) < units


def walk(stage, units):
    """The kernel's loop: units that have been there, stage by stage."""
    u0 = steps = 0
    while u0 < units:
        assert stage > 0, "no end"
        u0 += min(units - u0, stage)
        steps += 1
    return steps


@pytest.mark.parametrize("lds", [48 * KB, 112 * KB])
@pytest.mark.parametrize("most,units_of_wave", [(4, 4), (16, 2)])      # rows of a pass; units a wave has in flight
@pytest.mark.parametrize("unit", [512, 520, 544])
def test_every_launch_has_a_stage(lib, lds, most, units_of_wave, unit):
    for rows in range(1, most + 1):
        for waves in (1, 2, 4, 8, 16):
            w = lib.waves(lds, rows, unit, units_of_wave, waves)
            assert 1 <= w <= waves and waves % w == 0
            assert w == waves or lib.units(lds, rows, unit, 2 * w * units_of_wave, 65536) == 0
            for units in (1, 5, 64, 145, 65536):
                for held in range(1, rows + 1):            # the last pass may have fewer rows
                    walk(lib.units(lds, held, unit, w * units_of_wave, units), units)


def test_sixteen_rows_in_48_kb_do_not_take_four_waves(lib):
    """16 rows with 8 scales a unit leave 5 units of room: a round of four waves
    with two units each would be none at all."""
    assert lib.units(48 * KB, 16, 544, 4 * 2, 64) == 0
    assert lib.waves(48 * KB, 16, 544, 2, 4) == 2 and lib.units(48 * KB, 16, 544, 2 * 2, 64) == 4
