"""The machine code of the kernels that copy to LDS and count what is in flight, and of their
neighbours, checked on the host (hipcc cross-compiles for gfx950): no scratch memory and no
vector register spilled, and in the attention kernel every stage's copies are as many as its
wait counts: a step starts with the copies of the next stage and waits until only those are
outstanding."""
import os
import re
import subprocess

import pytest

from tests.test_kernel_asm import ROOT, _hipcc, _kernel_meta

CSRC = os.path.join(ROOT, "weight_activation_quantized_amd", "csrc")


def assembly(name, tmp):
    out = tmp / (name + ".s")
    subprocess.run([_hipcc(), "-x", "hip", "-std=c++17", "-O3", "-ffp-contract=off", "-fno-fast-math",
                    f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "--offload-arch=gfx950", "-Xclang", "-target-feature",
                    "-Xclang", "-packed-fp32-ops", "--offload-device-only", "-S", os.path.join(CSRC, name + ".hip"), "-o", str(out)],
                   check=True, capture_output=True, timeout=600)
    return out.read_text().split("\n")


@pytest.fixture(scope="module")
def attention(tmp_path_factory):
    return assembly("mixllm_kv4_attention", tmp_path_factory.mktemp("asm"))


def test_no_scratch(attention, tmp_path_factory):
    tmp = tmp_path_factory.mktemp("asm2")
    for lines in (attention, assembly("mixllm_kv4", tmp), assembly("mixllm_norm", tmp)):
        meta = _kernel_meta(lines)
        assert meta
        for name, m in meta.items():
            if "norm_kernelILi1024ELi8E" in name:  # rows of more than 32768: 64 values a thread, of which some spill
                continue
            assert m["private_segment_fixed_size"] == 0 and m["vgpr_spill_count"] == 0, (name, m)


def test_waits_count_a_stage(attention):
    """kLoads: per run 2 x (D = 64: 2 dword copies, 128: 1, 256: 2 of 16 bytes) + the parameters'
    (D = 256: 2); 2 runs a step where rows fill the columns or D = 256, else 4."""
    text = "\n".join(attention)
    found = 0
    for m in re.finditer(r"^(_Z\S*kv4_attention_kernelILi(\d+)ELi(\d)ELi\d\S*):(.*?)\.end_amdhsa_kernel", text, re.M | re.S):
        d, v, body = int(m[2]), int(m[3]), m[4]
        per_run = {64: 5, 128: 3, 256: 6}[d]
        loads = (2 if v == 1 or d == 256 else 4) * per_run
        lines = [x.strip() for x in body.split("\n")]
        stages = 0
        for i, x in enumerate(lines):
            if not re.fullmatch(r"s_waitcnt vmcnt\(\d+\)", x):
                continue
            # back from the wait: the copies after anything that waits or branches, and no read
            # of what they bring
            copies = reads = 0
            for y in reversed(lines[:i]):
                if y.startswith(("s_waitcnt vmcnt", ".LBB", "s_cbranch", "s_branch")):
                    break
                copies += y.startswith("buffer_load") and y.endswith("lds")
                reads += y.startswith("ds_read")
            if copies and f"vmcnt({loads})" in x:
                assert copies == loads and reads == 0, (m[1], copies, reads)
                stages += 1
            elif copies:
                assert x == "s_waitcnt vmcnt(0)", (m[1], x)
        assert stages == 2, m[1]
        found += 1
    assert found >= 16
