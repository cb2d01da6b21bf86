"""AddressSanitizer / UndefinedBehaviorSanitizer build of the host code of the block-128 and Muon units (CPU
only), driven by tests/sanitize/block128_muon_asan.cpp.  Any report fails the run (-fno-sanitize-recover)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CSRC = os.path.join(ROOT, "moe_grouped_gemm_mxq_amd", "csrc")
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all"]


def run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
    return r


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_block128_and_muon_entry_points_under_asan_ubsan(tmp_path):
    common = ["--offload-arch=gfx950", "-std=c++17", "-g", "-O1", *SAN, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    procs, objs = [], []
    for src in ("mxq_api.hip", "qdq_mxfp4.hip", "quant128.hip", "gemm128.hip", "muon.hip"):
        objs.append(str(tmp_path / (src + ".o")))
        procs.append((src, subprocess.Popen([HIPCC, *common, "-c", os.path.join(CSRC, src), "-o", objs[-1]],
                                            stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    for src, p in procs:
        out = p.communicate()[0]
        assert p.returncode == 0, f"{src}\n{out}"
    drv, exe = str(tmp_path / "drv.o"), str(tmp_path / "block128_muon_asan")
    run([HIPCC, *common, "-x", "hip", "-c", os.path.join(ROOT, "tests", "sanitize", "block128_muon_asan.cpp"), "-o", drv])
    run([HIPCC, "--offload-arch=gfx950", "-fno-gpu-sanitize", "-fsanitize=address,undefined", *objs, drv, "-o", exe])
    r = run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0", HIP_VISIBLE_DEVICES=""))
    assert r.stdout.strip() == "ok"
