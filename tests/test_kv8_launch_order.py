"""What the kernels of the paged 8-bit cache do before they wait for the work ahead of them.

They are launched while the kernel ahead still runs (programmatic dependent launches), and
an attention's first kernel lets its second one start before it ends. A kernel knows the
work ahead to be complete behind its griddepcontrol.wait alone, or where the kernel ahead
lets it start (griddepcontrol.launch_dependents) behind a wait of its own, what came before
that one. Else lengths and boundaries may be those of before an append. So: nothing of
device memory is read before the wait, unless the kernel ahead triggers behind its own; then
lengths and boundaries, which that kernel does not write, may be. Read from the source: on
the GPU the mistake shows only when the kernels happen to overlap."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sequence_long_context_gb300", "csrc")
WAIT = re.compile(r"griddepcontrol\.wait|grid_dependency_wait\(\)")
TRIGGER = re.compile(r"griddepcontrol\.launch_dependents|grid_dependency_launch\(\)")
# Reads of what kernels ahead write (arguments by value, and a tensor map's prefetch, are
# none): by a call, or of the attention's own results
INPUTS = re.compile(r"__ldg|\bseq_of\b|\bseq_line\b|\bline_ends\b|\bfind_run\b|\btokens_of\b|"
                    r"\blens\b|P\.(a\.)?cu\[")
PARTIALS = re.compile(r"\bspan_of\b|P\.(span|rec|ml_part|o_part|lse|out)\b|\bpage_of\b")


def kernels(text):
    """(name, body) of every kernel that waits."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", text):
        at = text.index("{", m.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        body = text[at:end]
        if WAIT.search(body):
            yield m.group(1), body


def before_waits(body):
    """The text ahead of the first wait, and between a block that ends behind a wait of its
    own and the next one."""
    out = body
    while True:
        first = WAIT.search(out)
        # a block "{ .. wait .. return; }" is passed over: what follows it has not waited
        m = re.search(r"\{[^{}]*$", out[: first.start()])
        end = block_end(out, m.start()) if m and m.start() > 0 else len(out)
        if end < len(out) and WAIT.search(out, end) and "return;" in out[first.end(): end]:
            out = out[: first.start()] + out[end:]
        else:
            return out[: first.start()]


def block_end(text, at):
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return i + 1
    return len(text)


def late(body, own=False):
    """Does a kernel let the next one start behind its own wait alone? (own: in its form
    without a second kernel.)"""
    text = body.replace("if constexpr (%skOwn) grid_dependency_launch();" % ("!" if own else ""), "")
    t = TRIGGER.search(text)
    return t is None or t.start() > WAIT.search(text).start()


def mistakes(body, ahead=None):
    """What a kernel reads too early; ahead: the body of the kernel that lets it start."""
    text = before_waits(body)
    bad = [m.group(0) for m in PARTIALS.finditer(text)]
    if ahead is None or not late(ahead):
        bad += [m.group(0) for m in INPUTS.finditer(text)]
    return bad


FOUND = {name: body for f in ("attn_kv8.cu", "attn_kv8_tc.cu", "kv8_cache.cu")
         for name, body in kernels(open(os.path.join(CSRC, f)).read())}
# what an attention's second kernel follows; the others follow anything
AHEAD = {"attn_kv8_merge_kernel": "attn_kv8_kernel", "attn_kv8_tc_merge_kernel": "attn_kv8_tc_kernel"}


def test_every_dependent_kernel_is_looked_at():
    assert sorted(FOUND) == ["append_lens_kernel", "attn_kv8_kernel", "attn_kv8_merge_kernel",
                             "attn_kv8_tc_kernel", "attn_kv8_tc_merge_kernel"]


@pytest.mark.parametrize("name", sorted(FOUND))
def test_nothing_is_read_before_it_may(name):
    assert not mistakes(FOUND[name], FOUND.get(AHEAD.get(name))), name


FIRST = "__global__ void first_kernel(P p) {\n  %s\n  init();\n  %s\n  use(__ldg(P.cu));\n}\n"
SECOND = "__global__ void second_kernel(P p) {\n  if (pad) {\n    const int e = __ldg(P.cu);\n" \
         "    grid_dependency_wait();\n    return;\n  }\n  %s\n  grid_dependency_wait();\n" \
         "  span_of(P, 0);\n}\n"


def test_the_rule_on_planted_kernels():
    one = lambda text: next(kernels(text))[1]  # noqa: E731
    wait, launch = "grid_dependency_wait();", "grid_dependency_launch();"
    early, good = one(FIRST % (launch, wait)), one(FIRST % (wait, launch))
    assert not mistakes(early) and not mistakes(good)
    assert late(good) and not late(early)
    second = one(SECOND % "const Seq q = seq_of(P, b);")
    assert mistakes(second) and mistakes(second, early) and not mistakes(second, good)
    assert mistakes(one(SECOND % "x = P.o_part[0];"), good)
    assert mistakes(one(FIRST % ("n = P.c.lens[b];", wait)))
    assert "seq_of" in mistakes(second, early) and "__ldg" in mistakes(second, early)
    # a comment is no wait
    assert mistakes(one(FIRST % ("// grid_dependency_wait();\n n = __ldg(P.cu);", wait)))
