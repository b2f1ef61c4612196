"""What can be said of libdcpattn's code without a GPU: the compiled latent
kernel's use of the registers it names, and the host side (checks, plans,
launches) under sanitizers."""
import os
import re
import subprocess

import pytest

from lse_weighted_merge_dcp_amd.csrc import build as hip_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lse_weighted_merge_dcp_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def _hipcc():
    try:
        return hip_build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc is not here")


@pytest.fixture(scope="module")
def latent(tmp_path_factory):
    """The assembly of attn_latent.hip: kernel -> [(instruction, operands, written by hand)]."""
    out = str(tmp_path_factory.mktemp("asm") / "latent.s")
    subprocess.check_call([_hipcc(), "-x", "hip", os.path.join(CSRC, "attn_latent.hip"), "-o", out, "--cuda-device-only",
                           "-S", "-w"] + [f for f in hip_build.HIP_FLAGS if f not in ("-Wall", "-Wextra")])
    kernels, now, by_hand = {}, None, False
    for line in open(out):
        m = re.match(r"^(_Z\w*attn_latent\w*):", line)
        if m:
            now = kernels.setdefault(m.group(1), [])
        elif line.startswith(".Lfunc_end"):
            now = None
        if "#ASMSTART" in line or "#ASMEND" in line:
            by_hand = "#ASMSTART" in line
        text = line.split(";")[0].strip()
        if now is not None and text and not text.startswith(".") and not text.endswith(":"):
            now.append((text.split()[0], text[len(text.split()[0]):].strip(), by_hand))
    assert len(kernels) == 8, sorted(kernels)
    return kernels


def registers(text, kind="v"):
    got = set()
    for a, b, c in re.findall(r"\b%s(?:(\d+)\b|\[(\w+):(\w+)\])" % kind, text):
        got |= {int(a)} if a else set(range(int(b, 0), int(c, 0) + 1))
    return got


def test_latent_outputs_have_their_registers_alone(latent):
    """a0 .. a255 hold the outputs by name: no instruction of the compiler's may touch one."""
    for name, code in latent.items():
        stray = [op + " " + args for op, args, by_hand in code if not by_hand and registers(args, "a")]
        assert not stray, (name, stray[:5])
        assert registers(" ".join(args for _, args, by_hand in code if by_hand), "a") == set(range(256))


def test_latent_products_read_settled_operands(latent):
    """No vector instruction writes an operand of a matrix instruction in the two states before it (the compiler does
    not see that the asm is one, and adds no wait)."""
    for name, code in latent.items():
        for i, (op, args, _) in enumerate(code):
            if not op.startswith("v_mfma"):
                continue
            _, a, b = args.replace(", ", ",").split(",")[:3]
            use, states = registers(a) | registers(b), 0
            for before, where, _ in reversed(code[max(0, i - 3):i]):
                if states >= 2:
                    break
                writes = before.startswith("v_") and not before.startswith(("v_mfma", "v_cmp"))
                assert not (writes and registers(where.split(",")[0]) & use), (name, before, where, args)
                states += 1 + int(where) if before == "s_nop" else 1


def test_latent_scores_are_read_when_they_are_there(latent):
    """An 8-pass product's result may be read 11 states later; a later product takes 8 of them."""
    for name, code in latent.items():
        pending = {}
        for op, args, _ in code:
            if op.startswith("v_mfma"):
                pending = {r: n - 8 for r, n in pending.items() if n > 8}
                for r in registers(args.split(",")[0]):
                    pending[r] = 11
                continue
            assert not any(r in pending for r in registers(args)), (name, op, args)
            gone = 1 + int(args) if op == "s_nop" else 1
            pending = {r: n - gone for r, n in pending.items() if n > gone}


def test_no_packed_fp32(latent):
    for name, code in latent.items():
        assert not [op for op, _, _ in code if re.match(r"v_pk_(add|mul|fma)_f32", op)], name


def test_attn_launches_under_asan_and_ubsan(tmp_path):
    """tests/attn_launch_check.cpp: random calls through the real checks and launchers under ASan and UBSan; every
    launch within 2^31 work-items, and a workspace of the size that the query gives is enough, a byte less refused."""
    clangxx = os.path.join(ROCM, "lib", "llvm", "bin", "clang++")
    if not os.path.exists(clangxx):
        pytest.skip("ROCm's clang++ is not here")
    fatbin = tmp_path / "empty.fatbin"
    fatbin.write_bytes(b"")
    host_only = [_hipcc(), "-x", "hip", "--cuda-host-only", "-std=c++20", "-O1", "-g", "-w", "-I" + os.path.join(ROOT, "include"),
                 "-Xarch_host", "-fsanitize=address,undefined", "-Xarch_host", "-fno-sanitize-recover=all",
                 "-Xarch_host", "-fno-omit-frame-pointer", "-Xclang", "-fcuda-include-gpubinary", "-Xclang", str(fatbin), "-c"]
    sources = [os.path.join(CSRC, f + (".cpp" if f == "attn_api" else ".hip")) for f in hip_build.OBJECTS[hip_build.ATTN_LIB]]
    sources.append(os.path.join(ROOT, "tests", "attn_launch_check.cpp"))
    running = [(subprocess.Popen(host_only + [src, "-o", str(tmp_path / (os.path.basename(src) + ".o"))])) for src in sources]
    assert [p.wait() for p in running] == [0] * len(running)
    exe = str(tmp_path / "attn_launch_check")
    subprocess.check_call([clangxx, "-fsanitize=address,undefined", "-o", exe] +
                          [str(tmp_path / (os.path.basename(src) + ".o")) for src in sources])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    for seed in (1, 2, 3):
        r = subprocess.run([exe, "30000", str(seed)], capture_output=True, text=True, timeout=300, env=env)
        assert r.returncode == 0 and r.stdout.startswith("ok "), (r.stdout, r.stderr[-3000:])
        calls, accepted, launches, grid = map(int, r.stdout.split()[1:5])
        assert calls == 30000 and accepted > 5000 and launches > accepted // 2 and grid > 1 << 20, r.stdout
