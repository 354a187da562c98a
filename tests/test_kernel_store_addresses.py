"""CPU check of compiled kernels (device assembly built here, no GPU): on every
way through a kernel the vector registers of an address are written before
they are used, for every kind of access (loads, stores and atomics of global
memory, reads, writes and atomics of LDS) and for the 64-bit arithmetic that
addresses come from. A comparison writes no vector register, and an atomic
without a result none either."""
import os
import re
import tempfile

import pytest

from test_kernel_addresses import _registers

# 64-bit sums, products and shifts: what addresses are made of
ARITHMETIC = ("v_lshl_add_u64", "v_add_co_u32", "v_addc_co_u32", "v_mad_u64_u32", "v_mad_i64_i32", "v_lshlrev_b64")


def operands(op, rest):
    """(registers written, registers that an address needs) of an instruction."""
    regs = _registers(rest)
    first = rest.split(",")[0].strip()
    no_result = (op.startswith(("global_store", "flat_store", "buffer_store", "scratch_store", "ds_write", "s_cbranch", "s_cmp",
                                "s_bitcmp"))
                 or (op.startswith(("global_atomic", "flat_atomic")) and " sc0" not in rest)
                 or (op.startswith("ds_") and "rtn" not in op and not op.startswith(("ds_read", "ds_bpermute", "ds_permute",
                                                                                       "ds_swizzle"))))
    written = [] if no_result or not regs or not re.match(r"[vs](\d+|\[\d+:\d+\])$", first) else regs[0]
    need = []
    if op.startswith(("global_", "flat_", "buffer_", "ds_")) and not op.startswith("ds_swizzle"):
        at = 0 if no_result else 1
        need = regs[at] if len(regs) > at else []
    elif op.startswith("v_mad_u64_u32"):
        # (of the addend its low half, where the product only fills a pair's high one)
        need = [r for r in sum(regs[1:], []) if r[0] == "v"]
        last = [r for r in regs[-1] if r[0] == "v"]
        if len(last) == 2:
            need = [r for r in need if r != last[1]] + [r for g in regs[1:-1] for r in g if r == last[1]]
    elif op.startswith(ARITHMETIC):
        need = [r for group in regs[1:] for r in group]
    return set(written), [r for r in need if r[0] == "v"]


def unset_addresses(lines):
    ins, at = [], {}
    for line in lines:
        line = line.split(";")[0].rstrip()
        label = re.match(r"(\.LBB\S+):", line)
        if label:
            at[label.group(1)] = len(ins)
        elif line.startswith("\t") and not line.strip().startswith("."):
            ins.append(line.strip())
    follow, written, used = [], [], []
    for i, line in enumerate(ins):
        op, *rest = line.split(None, 1)
        rest = rest[0] if rest else ""
        nxt = [i + 1] if i + 1 < len(ins) and op not in ("s_endpgm", "s_branch") else []
        if op == "s_branch" or op.startswith("s_cbranch"):
            nxt.append(at[rest.strip()])
        follow.append(nxt)
        w, u = operands(op, rest)
        written.append(w)
        used.append(u)
    state = [None] * len(ins)
    state[0] = {("v", 0)}  # the thread's index
    todo = [0]
    while todo:
        i = todo.pop()
        out = state[i] | written[i]
        for j in follow[i]:
            new = out if state[j] is None else state[j] & out
            if new != state[j]:
                state[j] = set(new)
                todo.append(j)
    return [ins[i] for i in range(len(ins)) if state[i] is not None and any(r not in state[i] for r in used[i])]


def branched(last, *before):
    """A kernel with v[2:3] and v4 set on one of two ways, and a last access."""
    return ["\tv_mov_b32_e32 v3, 0", "\tv_mov_b32_e32 v6, 0", "\tv_mov_b32_e32 v7, 0", "\ts_cbranch_scc0 .LBB0_2",
            "\tv_mov_b32_e32 v2, 1", "\tv_mov_b32_e32 v4, 1", "\ts_branch .LBB0_3", ".LBB0_2:", *before, ".LBB0_3:",
            "\t" + last, "\ts_endpgm"]


@pytest.mark.parametrize("last", [
    "global_load_dword v6, v[2:3], off", "global_load_dwordx4 v[8:11], v2, s[4:5]", "global_store_dword v[2:3], v6, off",
    "global_store_short v2, v6, s[4:5] offset:2", "global_store_dwordx4 v[2:3], v[8:11], off nt",
    "global_atomic_or_x2 v[2:3], v[6:7], off", "global_atomic_add v8, v[2:3], v6, off sc0", "ds_write_b32 v4, v6",
    "ds_write2_b64 v4, v[6:7], v[6:7] offset1:1", "ds_read_b32 v8, v4", "ds_or_rtn_b32 v8, v4, v6", "ds_add_u32 v4, v6",
    "ds_bpermute_b32 v8, v4, v6", "v_lshl_add_u64 v[8:9], v[2:3], 2, s[4:5]", "v_add_co_u32_e32 v8, vcc, s4, v2",
    "v_addc_co_u32_e32 v8, vcc, 0, v2, vcc", "v_mad_u64_u32 v[8:9], s[4:5], v4, s6, v[6:7]", "v_lshlrev_b64 v[8:9], 2, v[2:3]"])
def test_the_check_finds_an_unset_address(last):
    assert unset_addresses(branched(last)) == [last]
    both = ("\tv_mov_b32_e32 v2, 2", "\tv_mov_b32_e32 v4, 2")
    assert unset_addresses(branched(last, *both)) == []
    # what reads a register does not write it
    for reads in ("\tv_cmp_lt_u32_e32 vcc, v2, v4", "\tglobal_store_dword v[6:7], v2, off", "\tds_write_b32 v6, v4",
                  "\tglobal_atomic_or_x2 v[6:7], v[2:3], off"):
        assert last in unset_addresses(branched(last, reads))


@pytest.mark.parametrize("source,count", [("entq_norm.hip", 40), ("entq_distill.hip", 30), ("entq_moe.hip", 20)])
def test_addresses_are_written_on_every_way(source, count):
    from entropy_coded_weight_amd import build
    with tempfile.TemporaryDirectory() as d:
        lines = open(build.asm(os.path.join(d, "k.s"), source)).read().split("\n")
    starts = [n for n, line in enumerate(lines) if re.match(r"_Z\S+:\s+; @", line)]
    assert len(starts) >= count
    for s in starts:
        end = next(n for n in range(s, len(lines)) if ".Lfunc_end" in lines[n])
        assert unset_addresses(lines[s + 1:end]) == [], lines[s].split(":")[0]
