"""What the prompt-side kernels do when a bounded wait runs out, read from their sources (no GPU).

A wait gives up per thread.  A warp that then left its loop while the others of its group met at a named barrier would
leave them there for good, and lanes that gave up one by one would leave a vote or a tensor-memory load without them.
The first part follows the epilogue warps of every INT8 matmul kernel through their barriers and waits, in the order
in which the source has them, for every choice of which warp's waits run out: all warps must come to the end."""
import itertools
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "group_wise_weight_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def block(text, start):
    """The text from `start` (an index at or before a '{') to the brace that closes it."""
    i = text.index("{", start)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i:j + 1]
    raise AssertionError("unbalanced braces")


def role(kernel, marker):
    """The body of a kernel's branch that begins with the comment `marker`."""
    text = source("wq_gemm_i8.cu") if kernel.startswith("gemm_i8") else source("wq_prompt_attn.cu")
    body = block(text, text.index(")\n{", text.index(kernel + "(const __grid_constant__")))
    at = body.index("--- " + marker)
    return block(body, body.rindex("{", 0, at))


EVENTS = re.compile(r"(?P<bar>named_bar_(?:sync|and)\()|(?P<leave>if \(!wait\(&b\.d_full[^\n]*break)"
                    r"|(?P<keep>ok = ok && warp_wait\(&b\.d_full)|(?P<skip>if \(!ok\) continue;)")


def events(text):
    return [m.lastgroup + ("_and" if m.group().startswith("named_bar_and") else "") for m in EVENTS.finditer(text)]


def warp(loop, join, tiles, fails):
    """One epilogue warp: yields `ok` at each barrier it meets and is sent what named_bar_and answers."""
    ok = True
    for t in range(tiles):
        for e in loop:
            if e.startswith("bar"):
                all_ok = yield ok
                ok = all_ok if e == "bar_and" else ok
            elif e == "leave" and t >= fails:
                ok = False
                break
            elif e == "keep":
                ok = ok and t < fails
            elif e == "skip" and not ok:
                break
        if "leave" in loop and not ok:
            break
    if join and ok:
        for _ in join:
            yield ok


def ends(loop, join, tiles, fails):
    """Whether warps whose waits run out from tile fails[i] on all end."""
    warps = [warp(loop, join, tiles, f) for f in fails]
    at = [next(w, None) for w in warps]
    while any(a is not None for a in at):
        if any(a is None for a in at):
            return False  # some wait at a barrier that another never meets
        together = all(at)
        for i, w in enumerate(warps):
            try:
                at[i] = w.send(together)
            except StopIteration:
                at[i] = None
    return True


@pytest.mark.parametrize("kernel,split", [("gemm_i8_pair_kernel", False), ("gemm_i8_rows_kernel", False),
                                          ("gemm_i8_stream_kernel", False), ("gemm_i8_stream_kernel", True)])
def test_epilogue_warps_all_end_whichever_wait_runs_out(kernel, split):
    body = role(kernel, "epilogue")
    loop = block(body, body.index("{", body.index("for (int")))
    rest = body[body.index(loop) + len(loop):]
    first, join = events(loop), [e for e in events(rest) if e.startswith("bar")] if split else []
    assert "keep" in first or "leave" in first
    if not split and kernel == "gemm_i8_stream_kernel":
        # whole tiles: what a CTA with a part does is left out, the tokens' scales are loaded for each tile
        part = block(loop, loop.index("if (count > 1)"))
        first = events(loop.replace(part, ""))
    assert any(e.startswith("bar") for e in first)
    tiles = 1 if split else 3
    for fails in itertools.product(range(tiles + 1), repeat=3):
        assert ends(first, join, tiles, fails), (kernel, fails)


@pytest.mark.parametrize("kernel", ["gemm_i8_pair_kernel", "gemm_i8_rows_kernel", "gemm_i8_stream_kernel"])
def test_epilogue_lanes_get_one_answer(kernel):
    body = role(kernel, "epilogue")
    assert not re.search(r"(?<![_\w])(?:wait|mbar_wait)\(", body)
    assert "warp_wait(" in body
    helper = source("wq_prompt.cuh")
    assert "__all_sync(0xffffffffu, mbar_wait(" in block(helper, helper.index("bool warp_wait("))


@pytest.mark.parametrize("marker", ["items and copies", "softmax, one row per thread", "output, both tiles in turn", "Q of tile x"])
def test_attention_roles_of_whole_warps_get_one_answer(marker):
    """Votes, shuffles and tensor-memory loads follow the waits of these roles."""
    text = source("wq_prompt_attn.cu")
    body = block(text, text.index(")\n{", text.index("prompt_attn_kernel(const __grid_constant__")))
    kind = re.search(r"const (\w+) wait\{", body).group(1)  # the kernel's; a role may have its own
    own = role("prompt_attn_kernel", marker)
    kind = m.group(1) if (m := re.search(r"const (\w+) wait\{", own)) else kind
    assert "wait(" in own and "mbar_wait(" not in own
    assert "return warp_wait(bar, parity, status, abort);" in block(text, text.index(f"struct {kind} "))


def test_attention_role_of_one_thread_votes_with_nobody():
    own = role("prompt_attn_kernel", "MMAs: one thread")
    at = own.index("if (elect_one())")
    kind = re.search(r"const (\w+) wait\{", block(own, at)).group(1)
    text = source("wq_prompt_attn.cu")
    assert "return mbar_wait(bar, parity, status, abort);" in block(text, text.index(f"struct {kind} "))
    assert "wait(" not in own[:at]


def test_attention_fences_after_every_wait_for_an_mma():
    """tcgen05 loads and stores are ordered behind an MMA's completion by a fence after the wait for it, not by the wait
    alone: in the softmax and output roles each wait on a barrier that a commit arrives on is followed by one before
    any tensor-memory access."""
    text = source("wq_prompt_attn.cu")
    committed = set(re.findall(r"tc_commit\(&b\.(\w+)", text))
    assert {"s_full", "pv_done"} <= committed
    access = re.compile(r"tmem_(?:ld|st)\d+\(|tc_fence_after\(\)")
    for marker in ("softmax, one row per thread", "output, both tiles in turn"):
        own = role("prompt_attn_kernel", marker)
        waits = [m for m in re.finditer(r"wait\(&b\.(\w+)", own) if m.group(1) in committed]
        assert waits
        for m in waits:
            # the function that holds a wait at its end returns to a caller that touches tensor memory next
            follows = access.search(own, m.end())
            assert follows and follows.group().startswith("tc_fence_after"), own[m.start():m.start() + 200]
