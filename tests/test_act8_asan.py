"""The host code of the entry points that hold activations in 8 bits under AddressSanitizer (CPU only,
nothing is launched): tests/asan/act8_driver.cpp with the library's sources as test_host_asan builds them."""
import glob
import os
import subprocess


def test_entry_points_under_address_sanitizer():
    import test_host_asan as base
    base._build()
    driver = os.path.join(os.path.dirname(base.DRIVER), "act8_driver.cpp")
    exe, obj = os.path.join(base.OUT, "act8_asan"), os.path.join(base.OUT, "act8_driver.o")
    objs = sorted(glob.glob(os.path.join(base.OUT, "*.hip.o")))
    assert objs
    from grouped_expert_gemm_amd import build as b
    if not os.path.exists(exe) or any(os.path.getmtime(p) > os.path.getmtime(exe) for p in [driver, *objs]):
        base._run([b.HIPCC, f"--offload-arch={b.ARCH}", "-x", "hip", "-O1", "-std=c++17", "-I", b.INCLUDE, *base.SAN, "-c",
                   driver, "-o", obj])
        base._run([b.HIPCC, f"--offload-arch={b.ARCH}", *base.SAN, "-o", exe + ".tmp", obj, *objs])
        os.replace(exe + ".tmp", exe)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out, out[-6000:]
    assert r.returncode == 0 and "ok: 0 failure(s)" in r.stdout, out[-3000:]
