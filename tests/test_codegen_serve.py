"""What the compiler makes of the serving operators' kernels: no register may be
spilled, nor an accumulation register written, while a branch of some lanes has
the others switched off. The compiler has lost the other lanes' values in both:
a spill stood in the block where such a branch joins, before the lanes come
back, and of a tuple of accumulation registers of which a branch set one
element the other three were overwritten. So such branches stay out of the code
that has no registers to spare, and this reads the assembly for it."""
import os
import re
import shutil
import subprocess

import pytest

from int4_weight_only_block_amd import build as q4build

PAIR = r"(s\[\d+:\d+\]|vcc)"


def functions(asm):
    name, body = None, []
    for line in asm.splitlines():
        start = re.match(r"(_Z\w+):", line)
        if start:
            name, body = start[1], []
        elif line.startswith(".Lfunc_end") and name:
            yield name, body
            name = None
        elif name:
            body.append(line)


def blocks_of(body):
    out = [["entry", []]]
    for line in body:
        label = re.match(r"(\.LBB\w+):", line) or re.match(r"; (%bb\.\d+):", line)
        if label:
            out.append([label[1], []])
        elif line.strip() and not line.strip().startswith((";", ".")):
            out[-1][1].append(line.strip())
    return out


def step(text, stack, held):
    """`stack`: the masks saved where lanes were switched off, outermost first; `held`: registers that hold exec."""
    def back_to(mask):
        return stack[:len(stack) - 1 - stack[::-1].index(mask)] if mask in stack else stack

    if m := re.match(rf"s_(and|or|andn2|xor)_saveexec_b64 {PAIR}, {PAIR}", text):
        if m[1] != "and":  # the other side of a branch begins: back to before it, then narrowed again
            stack = back_to(m[3])
        return stack + [m[2]]
    if m := re.match(rf"s_mov_b64 {PAIR}, exec", text):
        held.add(m[1])
    elif m := re.match(rf"s_(?:and|andn2|xor)_b64 {PAIR}, {PAIR}, {PAIR}", text):
        held.discard(m[1])
        if m[2] in held:  # (a mask formed from exec, for the move below)
            held.discard(m[2])
            held.add((m[1], m[2]))
    if m := re.match(rf"s_mov_b64 exec, {PAIR}", text):
        saved = [h[1] for h in held if isinstance(h, tuple) and h[0] == m[1]]
        return stack + [saved[0]] if saved else back_to(m[1])
    if m := re.match(rf"s_or_b64 exec, exec, {PAIR}", text):
        return back_to(m[1]) if m[1] in stack else stack[:-1] if stack[-1:] == ["loop"] else stack
    if m := re.match(rf"s_xor_b64 {PAIR}, exec, {PAIR}", text):
        return stack[:-1] + [m[1]] if stack[-1:] == [m[2]] else stack
    if text.startswith("s_andn2_b64 exec, exec"):  # lanes that leave a loop
        return stack if stack[-1:] == ["loop"] else stack + ["loop"]
    return stack


def hazards(body):
    """(block, instruction) of every spill and accumulation write with lanes switched off; and how many branches of
    some lanes there are."""
    blocks = blocks_of(body)
    at = {b[0]: i for i, b in enumerate(blocks)}
    seen, todo, found, branches = {0: []}, [0], [], 0
    while todo:
        i = todo.pop()
        stack, held, goes_on = seen[i], set(), True
        targets = []
        for text in blocks[i][1]:
            branches += "_saveexec_" in text
            if stack and ("Folded Spill" in text and "writelane" not in text or text.startswith("v_accvgpr_write")):
                found.append((blocks[i][0], text))
            stack = step(text, stack, held)
            if m := re.match(r"s_c?branch\w* (\.LBB\w+)", text):
                targets.append((at[m[1]], stack))
            if text.startswith(("s_branch", "s_endpgm", "s_setpc")):
                goes_on = False
        if goes_on and i + 1 < len(blocks):
            targets.append((i + 1, stack))
        for j, s in targets:
            if j not in seen:
                seen[j] = s
                todo.append(j)
    return found, branches


def test_reader_finds_what_it_is_for():
    outside = """
        s_and_saveexec_b64 s[2:3], vcc
        s_cbranch_execz .LBB0_2
; %bb.1:
        global_store_dword v0, v1, s[8:9]
.LBB0_2:
        s_or_b64 exec, exec, s[2:3]
        scratch_store_dword off, v4, off ; 4-byte Folded Spill
        s_endpgm"""
    assert hazards(outside.splitlines()) == ([], 1)
    lines = [x for x in outside.splitlines() if "Folded" not in x]
    join = lines.index(".LBB0_2:")
    spill = "        scratch_store_dword off, v4, off ; 4-byte Folded Spill"
    assert len(hazards(lines[:join + 1] + [spill] + lines[join + 1:])[0]) == 1
    assert len(hazards(lines[:join] + ["        v_accvgpr_write_b32 a1, v2"] + lines[join:])[0]) == 1
    # a mask moved into exec by hand, a loop that lanes leave one by one, and the other side of a branch
    by_hand = ["s_mov_b64 s[6:7], exec", "s_and_b64 s[8:9], s[6:7], vcc", "s_mov_b64 exec, s[8:9]", spill,
               "s_or_b64 exec, exec, s[6:7]", spill, "s_endpgm"]
    assert len(hazards(by_hand)[0]) == 1
    loop = ["s_mov_b64 s[10:11], 0", ".LBB0_1:", "s_or_b64 s[10:11], vcc, s[10:11]", "s_andn2_b64 exec, exec, s[10:11]",
            "s_cbranch_execnz .LBB0_1", "; %bb.2:", "s_or_b64 exec, exec, s[10:11]", spill, "s_endpgm"]
    assert hazards(loop)[0] == []
    other = ["s_and_saveexec_b64 s[2:3], vcc", "s_xor_b64 s[2:3], exec, s[2:3]", "s_cbranch_execz .LBB0_1", "; %bb.1:",
             "v_mov_b32_e32 v0, 0", ".LBB0_1:", "s_or_saveexec_b64 s[4:5], s[2:3]", "s_xor_b64 exec, exec, s[4:5]",
             "s_cbranch_execz .LBB0_3", "; %bb.2:", spill, ".LBB0_3:", "s_or_b64 exec, exec, s[4:5]", spill, "s_endpgm"]
    assert len(hazards(other)[0]) == 1


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"), reason="no hipcc")
@pytest.mark.parametrize("source", ["paged_attention.hip", "sample_logits.hip", "kv_append.hip"])
def test_no_spill_with_lanes_switched_off(source, tmp_path):
    out = str(tmp_path / "kernels.s")
    flags = q4build.HIPCC_FLAGS + q4build.FILE_FLAGS.get(source, [])
    subprocess.run([q4build.hipcc(), *flags, "--cuda-device-only", "-S", os.path.join(q4build.CSRC, source), "-o", out],
                   check=True, capture_output=True, timeout=600)
    with open(out) as f:
        kernels = dict(functions(f.read()))
    results = {name: hazards(body) for name, body in kernels.items()}
    assert len(kernels) >= 4 and sum(n for _, n in results.values()) > 0  # it has been read
    bad = {name: found for name, (found, _) in results.items() if found}
    assert not bad, bad
