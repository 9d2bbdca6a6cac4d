"""What kernels do after a bounded wait gave up, read from their source: a warp takes one decision for all
of its lanes (its MMAs, shuffles and tensor-memory loads need them), and no barrier that several warps
count on lies behind a decision that they take separately.  A kernel that breaks either rule may never
end, so this is not tried out on a GPU."""
import os
import re

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "block_quant_gemv_b200", "csrc")
BARRIERS = ("ml_consumers_sync(", "ml_list_sync(", "bar.sync", "__syncthreads(", "cluster_sync(")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def closing(text, at, pair):
    """The place behind the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += {pair[0]: 1, pair[1]: -1}.get(text[i], 0)
        if depth == 0:
            return i + 1
    raise AssertionError("no closing bracket")


HEAD = re.compile(r"(?:if|while|for) (?:constexpr )?\(")


def statement(text, at):
    """The statement that starts at or behind `at`, as (start, end)."""
    start = at + len(text[at:]) - len(text[at:].lstrip())
    if text[start] == "{":
        return start, closing(text, start, "{}")
    head = HEAD.match(text, start)
    if head:
        return start, statement(text, closing(text, head.end() - 1, "()"))[1]
    return start, text.index(";", start)


def branches(text):
    """(condition, body) of every `if`, `while` and `for`."""
    for m in re.finditer(r"\b" + HEAD.pattern, text):
        end = closing(text, m.end() - 1, "()")
        start, stop = statement(text, end)
        yield text[m.end():end - 1], text[start:stop]


def single_thread(cond):
    return re.search(r"\b(tid|threadIdx\.x|lane) == \w+", cond) is not None


def test_no_barrier_behind_the_abort_word():
    for cond, body in branches(source("moe_layer.cuh")):
        if "abort" in cond and not single_thread(cond):
            assert not any(b in body for b in BARRIERS), cond


def waits(text, names):
    """Every call of a bounded wait outside the code of single threads, with the text before it."""
    alone = [body for cond, body in branches(text) if single_thread(cond)]
    for m in re.finditer(r"\b(?:%s)\(" % "|".join(names), text):
        before, line = text[:m.start()], text[text.rfind("\n", 0, m.start()) + 1:text.find("\n", m.start())]
        if "__device__" in line or single_thread(line) or any(line in body for body in alone):
            continue
        yield before, line


@pytest.mark.parametrize("name,vote", [("moe_layer.cuh", "ml_all("), ("i8.cuh", "__all_sync(0xffffffffu, ")])
def test_a_warp_decides_as_a_whole(name, vote):
    seen = 0
    for before, line in waits(source(name), ("mbar_wait", "ml_wait_seq")):
        if before.rstrip().endswith((";", "{", ")")):  # a wait whose answer nobody uses
            continue
        seen += 1
        assert before.endswith(vote), line
    assert seen > 0


def test_storing_warps_leave_their_loop_together():
    """The int8 products' storing warps meet at a barrier in every tile: none of them leaves the loop but by
    that barrier's own answer, which is the same for all."""
    text = source("i8.cuh")
    assert "bar.sync" not in text
    alone = [body for cond, body in branches(text) if single_thread(cond)]
    loops = [body for cond, body in branches(text) if "it_all_go_on<" in body and not any(body in a for a in alone)
             and re.match(r"long long i = ", cond)]
    assert len(loops) == 2
    for loop in loops:
        leaves = [cond for cond, body in branches(loop) if re.search(r"\b(break|return)\b", body)]
        assert len(leaves) == len(re.findall(r"\b(?:break|return)\b", loop)) == 1
        assert leaves[0].startswith("!it_all_go_on<")


def test_no_wait_lasts_as_long_as_the_product():
    """The second CTA of a pair issues no MMAs: it waits for the last of them only once its storing warps are
    through, since a bounded wait over a whole long product would give up."""
    text = source("i8.cuh")
    kernel = text[text.index("k_i8_gemm_pair("):]
    kernel = kernel[:closing(kernel, kernel.index("{"), "{}")]
    assert kernel.count("mbar_wait(done") == 1
    wait = kernel.index("mbar_wait(done")
    assert kernel.index("it_store_tile(") < kernel.rindex("__syncthreads()", 0, wait) < wait


@pytest.mark.parametrize("name,drain,kernels", [("i8.cuh", r"mbar_wait\(&full\[q %", 2),
                                                ("moe_layer.cuh", r"mbar_wait\(&S\.full\[k %", 1)])
def test_copies_in_flight_are_waited_for_whoever_gave_up(name, drain, kernels):
    """The copying thread waits for its last copies in every case: the warps that use them may have given up
    without it."""
    text = source(name)
    assert len(re.findall(drain, text)) == kernels
    for cond, body in branches(text):
        if re.search(r"\bok\b|abort", cond) and ";" not in cond:
            assert not re.search(drain, body), cond
