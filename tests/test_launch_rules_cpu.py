"""Rules of programmatic dependent launch, checked on the kernels' text (no
device).  A kernel that may be scheduled before its predecessor has ended is
what the rest of the stream waits for: it has to wait itself, in a CTA of every
launch at least, and before it ends."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "bit_quantization_b200", "csrc")


def _kernels():
    """(name, body without comments) of every __global__ function."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            code = "\n".join(line.split("//", 1)[0] for line in f.read().splitlines())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?"
                             r"(\w+)\s*\(", code):
            start = code.index("{", m.end())
            depth, i = 0, start
            while True:
                depth += (code[i] == "{") - (code[i] == "}")
                i += 1
                if depth == 0:
                    break
            yield m.group(1), code[start:i]


def _returns_before_the_wait(body):
    """Whether a return of the kernel itself (not of a lambda) stands before
    its first wait."""
    head = body[:body.index("pdl_wait()")]
    head = re.sub(r"\[&\]\s*(\([^()]*\))?\s*\{[^{}]*\}", "", head)
    return re.search(r"\breturn\b", head) is not None


# Its CTAs for the weights leave early where their tokens are behind the
# sequence; those that merge (one in every launch at least) all wait.
LEAVES_EARLY = {"kv8_finish_kernel"}


def test_no_kernel_returns_before_it_waits():
    seen = set()
    for name, body in _kernels():
        if "pdl_wait()" in body:
            seen.add(name)
            assert _returns_before_the_wait(body) == (name in LEAVES_EARLY), name
    assert {"kv8_append_kernel", "kv8_append_step_kernel", "kv8_advance_kernel",
            "kv8_decode_kernel", "kv8_finish_kernel", "kv8_select_kernel", "kv8_gather_kernel",
            "lin_digits_kernel", "linear_kernel", "amax_partial_kernel"} <= seen


def test_the_rule_sees_an_early_return():
    assert _returns_before_the_wait("{ if (x) return; pdl_wait(); }")
    assert not _returns_before_the_wait("{ pdl_wait(); if (x) return; }")
    assert not _returns_before_the_wait("{ auto f = [&](int a) { return a; }; pdl_wait(); }")


def test_the_quantiser_reads_x_behind_the_wait():
    """The first kernel of a call waits for what may have written x before it
    loads any of it, and lets the next be scheduled only after that; the second
    may load x ahead of its own wait, the first having waited."""
    body = dict(_kernels())
    first = body["amax_partial_kernel"]
    assert first.index("pdl_wait()") < first.index("load_raw(")
    assert first.index("pdl_wait()") < first.index("pdl_trigger()")
    rows = body["quant_rows_kernel"]
    given = re.search(r"if \(scale_given\) pdl_wait\(\);", rows)
    assert given and given.end() < rows.index("load_raw(")
    cols = body["quant_cols_kernel"]
    assert cols.index("quant_tensor_scale(") < cols.index("__ldg(x")
