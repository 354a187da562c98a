"""CPU check of the compiled resources (device assembly built here, no GPU) of
the kernels around a block: rows and accumulators are meant to stay in
registers, and as many waves on a CU as their comments count on."""
import os
import re
import tempfile

import pytest


def kernels(source):
    from entropy_coded_weight_amd import build
    with tempfile.TemporaryDirectory() as d:
        txt = open(build.asm(os.path.join(d, "k.s"), source)).read()
    for m in re.finditer(r"\.amdhsa_kernel (\S+)", txt):
        seg = txt[m.end():]
        get = lambda p: int(re.search(p, seg).group(1))  # noqa: B023, E731
        yield m.group(1), get(r"amdhsa_next_free_vgpr (\d+)"), get(r"ScratchSize: (\d+)")


@pytest.mark.parametrize("source", ["entq_norm.hip", "entq_moe.hip"])
def test_no_spills(source):
    seen = list(kernels(source))
    assert len(seen) >= 20 and [n for n, _, scratch in seen if scratch] == []
    # a strip of the norms' backward pass keeps its rows: two waves on a SIMD
    assert all(v <= 256 for _, v, _ in seen)


def test_distillation_rows_stay_in_registers():
    seen = {re.search(r"distill_rowsILi\d+ELi\d+ELi(\d+)ELi(\d+)", n).groups() + (n,): (v, scratch)
            for n, v, scratch in kernels("entq_distill.hip")}
    assert len(seen) >= 30
    for (pieces, waves, name), (v, scratch) in seen.items():
        if (pieces, waves) == ("7", "15"):
            # held to 64 registers for two workgroups of 16 waves on a CU: the
            # entries' wave keeps a few words in scratch
            assert v <= 64 and scratch <= 32, name
        else:
            assert scratch == 0 and v <= 128, name
