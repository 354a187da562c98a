"""CPU check of compiled kernels (device assembly built here, no GPU): on every
way through a kernel the registers of a 64-bit address are written before they
are used. The compiler shares parts of addresses between branches; where a
branch was chosen by a type at run time, a shared offset has stayed unset on
the way of another type, which no test of the other types shows and which
reads anywhere. Two conditions that go together (one branch sets what a later
one on the same condition uses) are not told from that: kernels are written so
that neither occurs."""
import os
import re
import tempfile

import pytest


def _registers(operands):
    """Per operand, the registers it names: ("v" or "s", number)."""
    out = []
    for m in re.finditer(r"(?<![\w\[])([vs])(?:\[(\d+):(\d+)\]|(\d+))(?![\w\]])", operands):
        a, b = int(m.group(2) or m.group(4)), int(m.group(3) or m.group(4))
        out.append([(m.group(1), i) for i in range(a, b + 1)])
    return out


def unset_addresses(lines):
    """Instructions of one kernel that take a vector register into an address
    which some path has not written."""
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
        regs = _registers(rest[0]) if rest else []
        nxt = [i + 1] if i + 1 < len(ins) and op not in ("s_endpgm", "s_branch") else []
        if op == "s_branch" or op.startswith("s_cbranch"):
            nxt.append(at[rest[0].strip()])
        follow.append(nxt)
        silent = op.startswith(("global_store", "ds_write", "buffer_store", "s_cbranch", "s_cmp"))
        written.append(set(regs[0]) if regs and not silent else set())
        take = []
        if op.startswith("global_load"):
            take = regs[1] if len(regs) > 1 else []
        elif op.startswith("v_lshl_add_u64"):
            take = [r for group in regs[1:] for r in group]
        used.append([r for r in take if r[0] == "v"])
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


def test_the_check_finds_an_unset_address():
    good = ["\tv_mov_b32_e32 v3, 0", "\ts_cbranch_scc0 .LBB0_2", "\tv_mov_b32_e32 v2, 1", "\ts_branch .LBB0_3", ".LBB0_2:",
            "\tv_mov_b32_e32 v2, 2", ".LBB0_3:", "\tv_lshl_add_u64 v[4:5], v[2:3], 2, s[4:5]", "\tglobal_load_dword v6, v[4:5], off",
            "\ts_endpgm"]
    assert unset_addresses(good) == []
    bad = [line for line in good if "v2, 2" not in line]
    assert unset_addresses(bad) == ["v_lshl_add_u64 v[4:5], v[2:3], 2, s[4:5]"]


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
