"""The scored router's selection at 513 to 1,024 experts is bound by how many of its wavefronts a SIMD holds: of 512 registers, four
with at most 128 each, three with one more (32,768 tokens, d 1024: 1,024 experts 292 us a call against 298, 600 experts 204
against 210).  The compiler's own count, from the assembly of the source (no GPU)."""
import os
import re
import subprocess

from mixture_experts_layer_33_amd import build as libbuild


def test_four_wavefronts_of_the_selection_fit_a_simd(tmp_path):
    out = str(tmp_path / "score.s")
    subprocess.run([libbuild.HIPCC, *libbuild.FLAGS, "--offload-device-only", "-S", os.path.join(libbuild.CSRC, "score.hip"), "-o", out],
                   check=True, timeout=600, capture_output=True)
    with open(out) as f:
        text = f.read()
    name = "_ZN3moe19score_select_kernelILi16ELi1EEEvNS_10SelectArgsEi"
    meta = re.search(r"\.name:\s+" + name + r"\n.*?\.private_segment_fixed_size:\s+(\d+).*?\.vgpr_count:\s+(\d+)\s+\.vgpr_spill_count:\s+(\d+)",
                     text, re.S)
    scratch, registers, spilled = (int(v) for v in meta.groups())
    assert registers <= 128 and scratch == 0 and spilled == 0, (registers, scratch, spilled)
