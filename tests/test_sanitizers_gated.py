"""The host code of the gated products, the 8-bit checkpoints and the gradients from
codes and stacks under AddressSanitizer and UndefinedBehaviorSanitizer
(tests/sanitize/gated_driver.c), linked with the objects that the ABI driver's test
builds."""
import os
import subprocess


def test_gated_host_code_under_sanitizers():
    import torch

    import test_sanitizers as base
    base._build_abi_driver()
    objs = [os.path.join(base.OUT, n) for n in sorted(os.listdir(base.OUT)) if n.endswith(".hip.o")]
    clang = "/opt/rocm/llvm/bin/clang"
    drv = os.path.join(base.OUT, "gated_driver.o")
    exe = os.path.join(base.OUT, "gated_driver")
    base.run([clang, "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
              "-I", base.B.INCLUDE, "-c", os.path.join(base.HERE, "gated_driver.c"), "-o", drv])
    base.run([base.B.hipcc(), f"--offload-arch={base.B.ARCH}", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
              "-fsanitize=undefined", drv, *objs, "-o", exe])
    args = [exe] + (["gpu"] if torch.cuda.is_available() else [])
    r = subprocess.run(args, env=dict(base.ENV, ASAN_OPTIONS="detect_leaks=0"), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "gated driver: ok" in r.stdout
