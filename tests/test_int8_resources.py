"""CPU check of the int8 kernels' compiled resources (device assembly built
here, no GPU): a tile that spills its accumulators to scratch, or whose
registers keep a second workgroup off the CU, still computes the right thing,
several times slower."""
import os
import re
import tempfile

import pytest


@pytest.mark.parametrize("source,kernel,count", [("entq_int8_gemm.hip", "int8_tiles", 12),
                                                 ("entq_int8_grad.hip", "grad_tiles", 6),
                                                 ("entq_int8_few.hip", "int8_few", 18)])
def test_no_spills_and_the_intended_residency(source, kernel, count):
    from entropy_coded_weight_amd import build
    with tempfile.TemporaryDirectory() as d:
        txt = open(build.asm(os.path.join(d, "k.s"), source)).read()
    seen = 0
    for m in re.finditer(r"\.amdhsa_kernel (\S+)", txt):
        if kernel not in m.group(1):
            continue
        seen += 1
        seg = txt[m.end():]
        get = lambda p: int(re.search(p, seg).group(1))  # noqa: E731
        assert get(r"ScratchSize: (\d+)") == 0, m.group(1)
        lds, vgprs = get(r"group_segment_fixed_size (\d+)"), get(r"amdhsa_next_free_vgpr (\d+)")
        assert lds <= 160 * 1024, m.group(1)
        if kernel != "int8_few" and lds <= 80 * 1024:  # two workgroups of 4 waves on a CU
            assert vgprs <= 256, m.group(1)
    assert seen == count


def test_the_small_kernels_do_not_spill():
    from entropy_coded_weight_amd import build
    with tempfile.TemporaryDirectory() as d:
        txt = open(build.asm(os.path.join(d, "k.s"), "entq_int8.hip")).read()
    kernels = re.findall(r"\.amdhsa_kernel (\S+)", txt)
    assert sum("narrow_rows" in k for k in kernels) == 4 and sum("quantize_rows" in k for k in kernels) == 12
    assert [int(n) for n in re.findall(r"ScratchSize: (\d+)", txt)] == [0] * len(kernels)
