"""Where a wave of beam search's selection keeps its lists in LDS (csrc/beam_lds.h):
every wave's candidates begin at a multiple of the 16 bytes that they are written by,
for odd numbers of beams too, and no list lies over the next."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_graph_recurrent_amd", "csrc")
PACK, WAVES = 8, 16     # logits an access; waves of a workgroup, at most


@pytest.fixture(scope="module")
def layouts(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("beam_lds") / "driver")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", exe,
                    os.path.join(ROOT, "tests", "beam_lds_driver.cpp")], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    return [tuple(map(int, ln.split())) for ln in out.strip().split("\n")]


def test_every_wave_of_every_number_of_beams_is_aligned(layouts):
    assert [row[0] for row in layouts] == list(range(1, 33))
    for K, packs, above, above_at, level_at, places_at, size in layouts:
        for wave in range(WAVES):
            at = wave * size
            for pack in range(packs):
                assert (at + pack * PACK * 4) % 16 == 0, (K, wave)
            assert (at + above_at) % 8 == 0 and (at + level_at) % 8 == 0, (K, wave)
            assert (at + places_at) % 4 == 0, (K, wave)
        assert above_at >= packs * PACK * 4 and level_at >= above_at + 8 * above
        assert places_at >= level_at + 8 * K and size >= places_at + 4 * packs
