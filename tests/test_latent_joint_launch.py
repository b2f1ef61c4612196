"""dcpa_latent_attn on the host alone, under sanitizers (tests/latent_joint_check.cpp)."""
import os
import subprocess

import pytest

import test_attn_build as base
from lse_weighted_merge_dcp_amd.csrc import build as hip_build


def test_launches_under_asan_and_ubsan(tmp_path):
    clangxx = os.path.join(base.ROCM, "lib", "llvm", "bin", "clang++")
    if not os.path.exists(clangxx):
        pytest.skip("ROCm's clang++ is not here")
    fatbin = tmp_path / "empty.fatbin"
    fatbin.write_bytes(b"")
    host_only = [base._hipcc(), "-x", "hip", "--cuda-host-only", "-std=c++20", "-O1", "-g", "-w",
                 "-I" + os.path.join(base.ROOT, "include"), "-Xarch_host", "-fsanitize=address,undefined", "-Xarch_host",
                 "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer", "-Xclang",
                 "-fcuda-include-gpubinary", "-Xclang", str(fatbin), "-c"]
    sources = [os.path.join(base.CSRC, f + (".cpp" if f == "attn_api" else ".hip")) for f in hip_build.OBJECTS[hip_build.ATTN_LIB]]
    sources.append(os.path.join(base.ROOT, "tests", "latent_joint_check.cpp"))
    running = [subprocess.Popen(host_only + [s, "-o", str(tmp_path / (os.path.basename(s) + ".o"))]) for s in sources]
    assert [p.wait() for p in running] == [0] * len(running)
    exe = str(tmp_path / "latent_joint_check")
    subprocess.check_call([clangxx, "-fsanitize=address,undefined", "-o", exe] +
                          [str(tmp_path / (os.path.basename(s) + ".o")) for s in sources])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    for seed in (1, 2, 3):
        r = subprocess.run([exe, "30000", str(seed)], capture_output=True, text=True, timeout=300, env=env)
        assert r.returncode == 0 and r.stdout.startswith("ok "), (r.stdout, r.stderr[-3000:])
        calls, accepted, launches, _ = map(int, r.stdout.split()[1:5])
        assert calls == 30000 and accepted > 5000 and launches > accepted, r.stdout
