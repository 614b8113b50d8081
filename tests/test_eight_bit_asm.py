"""The machine code of the 8-bit kernels, checked on the host (hipcc cross-compiles for gfx950): no
scratch memory and no vector register spilled; and in the product's tiles no wait of the
compiler's own for the copies in flight, whose counts the kernel's waits rely on."""
import re

import pytest

from tests.test_kernel_asm import _kernel_meta
from tests.test_serving_asm import assembly


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("asm8")
    return {name: assembly(name, tmp) for name in ("mixllm_gemm8", "mixllm_rotate", "mixllm_kv8", "mixllm_kv8_attention")}


def test_no_scratch(code):
    for name, lines in code.items():
        meta = _kernel_meta(lines)
        assert meta
        for kernel, m in meta.items():
            assert m["private_segment_fixed_size"] == 0, (kernel, m)
            if "kv8_many_kernelILi256E" not in kernel:  # which keeps a few in accumulation registers
                assert m["vgpr_spill_count"] == 0, (kernel, m)


def test_tiles_wait_only_for_the_stage_they_read(code):
    """The whole stages' loop: from its first barrier's wait on, every wait that names vmcnt is one
    before a barrier, for all copies (the last stages) or for those of ST - 2 stages."""
    text, found = "\n".join(code["mixllm_gemm8"]), 0
    for m in re.finditer(r"^(_Z\S*tile_kernelI\S*?TileShapeILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)\S*):(.*?)"
                         r"\.end_amdhsa_kernel", text, re.M | re.S):
        bm, bn, wm, wn, ks, bk, st = (int(m[i]) for i in range(2, 9))
        loads = (bm + bn) * bk // 1024 // (wm * wn * ks)
        lines = [x.strip().split(";")[0].strip() for x in m[9].split("\n")]
        lines = [x for x in lines if x and not x.startswith(".")]
        last = max(i for i, x in enumerate(lines) if x.startswith("v_mfma"))
        counted = 0
        for i, x in enumerate(lines[:last]):
            w = re.match(r"s_waitcnt .*vmcnt\((\d+)\)", x)
            if not w:
                continue
            assert lines[i + 1] == "s_barrier", (m[1], x, lines[i + 1])
            assert int(w[1]) in (0, (st - 2) * loads), (m[1], x)
            counted += int(w[1]) == (st - 2) * loads
        assert counted, m[1]
        found += 1
    assert found == 14
