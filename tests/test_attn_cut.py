"""How the attention's work is cut into pieces, on the CPU: the header that its kernels include, compiled
for the host."""
import os
import re
import subprocess

from mxfp4_routed_expert_e2m1_amd.build import HIPCC

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_piece_has_a_workgroup_and_workspace(tmp_path):
    """Texts of up to 2^30 tokens, batches of up to 900 of them: work far past 2^31 steps."""
    exe = str(tmp_path / "attn_cut_check")
    r = subprocess.run([HIPCC, "-O2", "-std=c++17", "-x", "hip", "--offload-host-only",
                        os.path.join(HERE, "attn_cut_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe, "300000"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-2000:]
    found = re.match(r"ok (\d+) cut calls", r.stdout)
    assert found and int(found[1]) > 10000, r.stdout
