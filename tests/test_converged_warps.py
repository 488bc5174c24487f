"""CPU check of the expert products' sources: instructions that a whole warp
has to execute together (tensor memory's loads and stores, stmatrix) are not
reached again by a warp whose lanes parted on the way round a loop."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_block_scaled_route_b200", "csrc")
ALIGNED = re.compile(r"\b(tmem_\w+|stmatrix_\w+|add_columns|own|sum_tile)\s*(<\w+>)?\s*\(")
MEETS = re.compile(r"__syncwarp\(\)|__all_sync\(|__shfl_sync\(|mbar_wait_warp\(|mbar_wait_moving\(|store_box\(")
# the condition of an `if` that names the lane (or a value that differs between lanes)
PARTS = re.compile(r"\bif \(([^;{}]*\b(?:lane|cols)\b[^;{}]*)\)")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def loops(text):
    """(start, end) of the braced body of every loop."""
    for m in re.finditer(r"\b(?:for|while) \(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        if text[i:i + 2] == " {":
            start, depth, i = i + 2, 1, i + 2
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            yield start, i


@pytest.mark.parametrize("name", ["moe_grouped.cu", "moe_wgrad.cu"])
def test_lanes_meet_before_aligned_instructions(name):
    text = code(name)
    epilogue = text.index("else if (warp >= 4)")
    seen = 0
    for start, end in loops(text):
        body = text[start:end]
        if start < epilogue or not ALIGNED.search(body):
            continue
        for m in PARTS.finditer(body):
            seen += 1
            # from there to the end of the body, and round again up to its first aligned instruction
            way = body[m.end():] + "\n" + body[:ALIGNED.search(body).start()]
            nxt = ALIGNED.search(way)
            way = way[:nxt.start()] if nxt else way
            assert MEETS.search(way), (name, m.group(0), text[:start + m.start()].count("\n") + 1)
            after = body[m.end():m.end() + 40]
            assert not re.match(r"\s*\{?\s*continue;", after), (name, m.group(0))
    assert seen >= 4, seen


def test_lanes_meet_behind_stores_of_fp32_results():
    """The stores of an 8-bit product into fp32 go by each lane's feature and row; the step after them reads tensor memory."""
    text = code("moe_grouped.cu")
    step = text[text.index("if (m < p.M && c + 1 < left) y[p.ldy] = b;"):]
    step = step[step.index("stmatrix_x4_trans("):]
    assert re.match(r"[^}]*}\s*__syncwarp\(\);\s*if \(p.out_type == MOE_DT_FP32\) continue;", step), step[:200]
