"""AddressSanitizer and UndefinedBehaviorSanitizer build of the host side of the
rotation's and Muon's entry points (CPU only), driven by
tests/sanitize/host_attention.cpp. No call reaches a HIP launch."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

base = pytest.importorskip("test_sanitizers")
CSRC, ENV, HIPCC, HOST_SAN, INC, SAN, run = (
    base.CSRC, base.ENV, base.HIPCC, base.HOST_SAN, base.INC, base.SAN, base.run)


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_attention_validation_under_asan_ubsan(tmp_path):
    common = ["-O1", "-g", "-std=c++17", *HOST_SAN, *INC]
    device = ["--offload-arch=gfx950", "-fPIC", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    jobs = [(os.path.join(CSRC, f), device) for f in sorted(os.listdir(CSRC)) if f.endswith(".hip")]
    jobs.append((os.path.join(SAN, "host_attention.cpp"), ["--offload-host-only", "-x", "hip"]))

    def compile_one(job):
        src, flags = job
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        rc, out = run([HIPCC, *flags, *common, "-c", src, "-o", obj])
        assert rc == 0, out
        return obj

    with ThreadPoolExecutor(8) as ex:
        objs = list(ex.map(compile_one, jobs))
    exe = str(tmp_path / "host_attention")
    rc, out = run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-o", exe, *objs])
    assert rc == 0, out
    rc, out = run([exe], env=ENV, timeout=300)
    assert rc == 0 and "ok" in out, out
