"""How the elementwise warps of the dq kernel leave after a wait that gave up.

Sixteen warps meet at a barrier twice an item (the sums of a row), and that
barrier has no limit: a warp that left before it, while another went on to the
next item, would hold the other there for good.  Waits are decided warp by warp
(one may look just before a barrier completes, another just after), so a failed
wait alone must not take a warp out of the item loop: only the barrier's own
answer, which is the same for all of them, may.  Checked by reading, since the
fault itself would hang a GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lora_linear_fine_b200", "csrc")


def _item_loop():
    """(condition, statements of the body with their depth) of the elementwise
    role's item loop in attn_dq_kernel."""
    with open(os.path.join(CSRC, "lora_attention_bwd.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    text = text[text.index("attn_dq_kernel(const __grid_constant__"):]
    text = text[text.index("regs_raise<kAttnBwdRegsHigh>"):]
    head = re.search(r"while \(([^{]*)\) \{", text)
    depth, at, body = 1, head.end(), []
    start = at
    while depth > 0:
        c = text[at]
        if c in "{};":
            piece = " ".join(text[start:at].split())
            if piece:
                body.append((depth, piece))
            start = at + 1
            depth += (c == "{") - (c == "}")
        at += 1
    return head.group(1), body


def test_the_item_loop_is_left_by_all_warps_or_none():
    condition, body = _item_loop()
    assert "whole_row" in " ".join(s for _, s in body)
    assert condition == "items.advance()", "the loop's condition depends on the warp"
    leaves = [k for k, (depth, s) in enumerate(body) if depth == 1 and re.search(r"\b(break|return)$", s)]
    assert leaves
    for k in leaves:
        assert re.match(r"ok = whole_row\(", body[k - 1][1]), f"`{body[k][1]}` after `{body[k - 1][1]}`"


def test_every_item_meets_at_the_barrier():
    """From the item's start to its first meeting no warp may go round it, but
    for items that have none; waits before it keep an earlier failure."""
    _, body = _item_loop()
    first = next(k for k, (depth, s) in enumerate(body) if depth == 1 and s.startswith("ok = whole_row("))
    before = body[:first]
    skips = [k for k, (_, s) in enumerate(before) if s.endswith("continue")]
    assert len(skips) == 1
    assert any("items.behind()" in s for _, s in before[:skips[0]])
    for _, s in before:
        if re.search(r"\bok = ", s):
            assert re.search(r"ok = ok && ", s), s
