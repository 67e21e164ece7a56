"""The kernels' cluster-barrier protocol, read from their source (no GPU).

A cluster's barrier has one phase at a time: a thread that has arrived waits
before it arrives again.  Breaking that is undefined without having to give a
wrong result, so no run can show it; the order of the operations in the source
does.
"""
import itertools
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "video_vae_decode_b200", "csrc")
OPS = re.compile(r"cluster_sync\(\)|cluster_arrive\(\)|cluster_wait\(\)|barrier\.cluster\.(?:arrive|wait)")


def source(name):
    """A file's text without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def closing(text, at, pair="{}"):
    """Where the bracket that opens at `at` closes."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if not depth:
            return i
    raise AssertionError("unbalanced source")


def body(text, function):
    """The braces of a function's definition: behind the parameter list that follows its name."""
    at = text.index("(", text.index(function))
    at = text.index("{", closing(text, at, "()"))
    return text[at + 1:closing(text, at)]


def statement(text, at):
    """(statement's text, position behind it) of what stands at `at`: a block or up to a semicolon."""
    at += len(text[at:]) - len(text[at:].lstrip())
    end = closing(text, at) if text[at] == "{" else text.index(";", at)
    return text[at:end + 1], end + 1


def operations(text, flags):
    """'A' (arrive) and 'W' (wait) in the order in which a thread meets them, the conditions on `flags` decided.  Any
    other condition may differ from warp to warp: there may be none under it."""
    out, at = [], 0
    while at < len(text):
        branch, op = re.compile(r"\b(if|for|while)\s*(?:constexpr\s*)?\(").search(text, at), OPS.search(text, at)
        if not op:
            break
        if not branch or op.start() < branch.start():
            out += ["A", "W"] if "sync" in op.group() else ["A"] if "arrive" in op.group() else ["W"]
            at = op.end()
            continue
        opened = text.index("(", branch.start())
        end = closing(text, opened, "()")
        condition = text[opened + 1:end]
        then, at = statement(text, end + 1)
        other = ""
        if branch.group(1) == "if" and re.match(r"\s*else\b", text[at:]):
            other, at = statement(text, at + re.match(r"\s*else\b", text[at:]).end())
            if re.match(r"if\b", other):     # else if: the rest of the chain is one statement
                start = at - len(other)
                end = closing(text, text.index("(", start), "()")
                _, at = statement(text, end + 1)
                while re.match(r"\s*else\b", text[at:]):
                    after = at + re.match(r"\s*else\b", text[at:]).end()
                    inner = re.match(r"\s*if\s*", text[after:])
                    after = closing(text, after + inner.end(), "()") + 1 if inner else after
                    _, at = statement(text, after)
                other = text[start:at]
        if branch.group(1) == "if" and set(re.findall(r"\w+", condition)) <= set(flags):
            value = eval(condition.replace("&&", " and ").replace("||", " or ").replace("!", " not "), {}, dict(flags))
            out += operations(then if value else other, flags)
        else:
            assert not OPS.search(then) and not OPS.search(other), f"a cluster barrier under `{condition}`"
    return out


@pytest.mark.parametrize("name,function,flags", [("fp8.cuh", "linear_fp8_kernel", ("kPair", "split")),
                                                 ("conv.cuh", "conv3d_body", ("kPair",))])
def test_every_arrive_has_its_wait_before_the_next(name, function, flags):
    text = body(source(name), function)
    for values in itertools.product((False, True), repeat=len(flags)):
        on = dict(zip(flags, values))
        ops = operations(text, on)
        assert ops == ["A", "W"] * (len(ops) // 2), (on, ops)
        assert bool(ops) == any(values), (on, ops)


def test_the_reader_of_the_source_sees_two_arrives():
    text = "if (split) { cluster_sync(); cluster_arrive(); } if (kPair) { cluster_sync(); } else { __syncthreads(); } if (split) cluster_wait();"
    assert operations(text, {"split": True, "kPair": True}) == ["A", "W", "A", "A", "W", "W"]
    assert operations(text, {"split": True, "kPair": False}) == ["A", "W", "A", "W"]
    with pytest.raises(AssertionError):
        operations("if (warp == 1) { cluster_sync(); }", {"split": True})


def test_signals_between_the_ctas_of_a_linear_pair_are_at_cluster_scope():
    # barriers that the partner's threads arrive on: scale words in place, accumulator read
    text, ptx = body(source("fp8.cuh"), "linear_fp8_kernel"), source("ptx.cuh")
    assert "mbar_arrive_remote" not in text                              # (CTA scope)
    arrive = body(ptx, "void mbar_arrive_cluster_relaxed")
    assert "mbarrier.arrive.relaxed.cluster.shared::cluster" in arrive
    assert "mbarrier.try_wait.parity.relaxed.cluster" in body(ptx, "bool mbar_try_wait_cluster_relaxed")
    signalled = re.findall(r"mbar_arrive_cluster_relaxed\((?:map_to_cta\()?(\w+)", text)
    assert sorted(signalled) == ["empty_leader", "sf_full"]
    assert re.search(r"empty_leader = kPair \? map_to_cta\(acc_empty, lead_cta\)", text)
    waits = re.findall(r"(\w+)\((sf_full|acc_empty) \+", text)
    waits = [w for w in waits if w[0] != "mbar_init" and w[0] != "map_to_cta" and w[0] != "mbar_arrive"]
    assert sorted(waits) == [("wait_tmem", "acc_empty"), ("wait_tmem", "sf_full")]
    assert "mbar_wait_warp<kPair>" in text[text.index("auto wait_tmem"):text.index("auto commit")]
    # each stands behind its fence, and the waits in front of theirs
    for name in ("sf_full", "empty_leader"):
        at = text.index("mbar_arrive_cluster_relaxed(" + ("map_to_cta(" if name == "sf_full" else "") + name)
        assert "tc_fence_before();" in text[at - 300:at], name
    assert "tc_fence_after();" in text[text.index("wait_tmem(sf_full"):][:250]
