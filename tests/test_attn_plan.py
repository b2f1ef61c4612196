"""Layout of single tokens over workgroups (CPU, tests/attn_plan_check.cpp): a
long sequence is never left whole to one workgroup for the number of the others."""
import os
import subprocess

import pytest

import test_attn_build as base
from lse_weighted_merge_dcp_amd.csrc import build as hip_build


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("plan")
    fatbin = tmp / "empty.fatbin"
    fatbin.write_bytes(b"")
    sources = [os.path.join(base.CSRC, "attn.hip"), os.path.join(base.CSRC, "attn_mass.hip"),
               os.path.join(base.ROOT, "tests", "attn_plan_check.cpp")]
    running = [subprocess.Popen([base._hipcc(), "-x", "hip", "--cuda-host-only", "-std=c++20", "-O1", "-w",
                                 "-I" + os.path.join(base.ROOT, "include"), "-Xclang", "-fcuda-include-gpubinary", "-Xclang",
                                 str(fatbin), "-c", s, "-o", str(tmp / (os.path.basename(s) + ".o"))]) for s in sources]
    assert [p.wait() for p in running] == [0] * len(running)
    clangxx = os.path.join(base.ROCM, "lib", "llvm", "bin", "clang++")
    if not os.path.exists(clangxx):
        pytest.skip("ROCm's clang++ is not here")
    exe = str(tmp / "attn_plan_check")
    subprocess.check_call([clangxx, "-o", exe] + [str(tmp / (os.path.basename(s) + ".o")) for s in sources])

    def run(*pairs):
        out = subprocess.check_output([exe] + [str(x) for p in pairs for x in p], text=True)
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def test_there_is_room_to_split(plan):
    """A sequence that holds all the keys there are gets at least half as many workgroups as the chip runs of a key
    head, as long as the sequences do not fill the chip four times over by themselves."""
    pairs = [(B, Hkv) for Hkv in (1, 3, 8, 64) for B in (1, 2, 7, 63, 64, 65, 100, 127, 128, 129, 300, 511) if B * Hkv < 4096]
    for (B, Hkv), (slots, share, tiles, units, ws, w_slots, w_share, w_units, w_ws) in zip(pairs, plan(*pairs)):
        each = -(-1024 // Hkv)
        assert tiles == B and units == slots and w_units == w_slots and w_ws == 0
        assert ws == units * Hkv * 32 * 129 * 4
        for n, s in ((slots, share), (w_slots, w_share)):
            # key ranges: no longer than 1 / s of all keys, n - B of them at least beside one to a sequence
            assert n - B >= each // 2 and each // 2 <= s <= max(each, n)
            assert n <= max(each, B + each // 2 + 1)


def test_small_batches_are_laid_out_as_ever_and_large_ones_stay_whole(plan):
    got = plan((32, 8), (64, 4), (512, 8), (4096, 1), (5000, 8))
    assert [g[0] for g in got] == [128, 256, 0, 0, 0] and [g[5] for g in got] == [128, 256, 0, 0, 0]
    assert [g[4] for g in got[2:]] == [0, 0, 0] and [g[3] for g in got[2:]] == [512, 4096, 5000]
