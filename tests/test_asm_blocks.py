"""Instruction order of the hand-written VALU blocks, from the sources, on the host: the compiler inserts no
wait states inside an asm statement, so each block has to keep the gfx9 hazards by its order alone.  The rules
are those above step_readout1 in ssm_device.hpp."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_61_amd", "csrc")
FILES = ["ssm_device.hpp", "scan_packed.hpp", "scan_bwd_rows.hpp"]
STRING = re.compile(r'"((?:[^"\\]|\\.)*)"')


def blocks(text):
    """The instruction lists of the asm statements of a source: the string literals before the first colon
    that is not in one."""
    for m in re.finditer(r"\basm(?:\s+volatile)?\s*\(", text):
        at, out = m.end(), ""
        while text[at] not in ":)":
            s = STRING.match(text, at)
            if s:
                out, at = out + s.group(1), s.end()
            else:  # blanks, and the macros that name a row broadcast (their arguments in parentheses)
                w = re.match(r"\s+|\w+(\(\d+\))?", text[at:])
                out, at = out + (" row_newbcast " if not w.group(0).isspace() else ""), at + w.end()
        code = [line.strip() for line in out.replace("\\t", "").split("\\n") if line.strip()]
        if code:
            yield code


def operands(line):
    """(mnemonic, register read, registers written) of one instruction."""
    op, regs = line.split()[0], re.findall(r"%\[(\w+)\]", line)
    regs = [r for r in regs if not re.fullmatch(r"k[bc]?", r)]  # lane selectors are immediates
    if op == "s_nop":
        return op, [], []
    return op, regs[0 if op.startswith("v_fmac") else 1:], regs[:1]


def faults(code):
    """Violations of the rules: a DPP instruction reads what was written fewer than three wait states before
    it (or comes first of all, where the compiler may just have written what it reads), a v_exp_f32 result is
    read by the next instruction."""
    written, at, bad = {}, 0, []
    for line in code:
        op, reads, writes = operands(line)
        if op == "s_nop":
            at += int(line.split()[1]) + 1
            continue
        for r in reads:
            by, when = written.get(r, (None, -1))
            if op.endswith("_dpp") and at - when < 3:
                bad.append(f"{line}: {r} is {at - when} old")
            if by == "v_exp_f32" and at - when < 2:
                bad.append(f"{line}: {r} is the last exponential")
        for r in writes:
            written[r] = (op, at)
        at += 1
    return bad


def all_blocks():
    for f in FILES:
        with open(os.path.join(CSRC, f), encoding="utf-8") as h:
            for i, code in enumerate(blocks(h.read())):
                yield pytest.param(code, id=f"{f}-{i}")


@pytest.mark.parametrize("code", all_blocks())
def test_a_block_waits_for_what_it_reads(code):
    assert not faults(code)


def test_the_rules_see_a_fault():
    """A planted mistake of each kind, and the same instructions in order."""
    mul, dpp = "v_mul_f32 %[a], %[x], %[y]", "v_mul_f32_dpp %[s], %[b], %[a] row_newbcast:%[kb]"
    mac, exp = "v_fmac_f32_dpp %[s], %[c], %[g] row_newbcast:%[kc]", "v_exp_f32 %[e], %[x]"
    assert faults([dpp]) and faults([mul, exp, dpp]) and not faults([mul, exp, "s_nop 0", dpp])
    assert not faults(["s_nop 1", dpp])
    assert faults(["s_nop 1", dpp, exp, mac]) and not faults(["s_nop 1", dpp, exp, "s_nop 0", mac])
    use = "v_mul_f32 %[a], %[e], %[y]"
    assert faults([exp, use]) and not faults([exp, mac.replace("_dpp", ""), use])


def test_every_block_is_found():
    """As many lists as the sources have asm statements with instructions."""
    for f in FILES:
        with open(os.path.join(CSRC, f), encoding="utf-8") as h:
            text = h.read()
        assert len(list(blocks(text))) == len(re.findall(r'\basm(?:\s+volatile)?\s*\("[vs]_', text)) > 0
