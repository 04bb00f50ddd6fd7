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
    """Every kernel of a call waits for what may have written x before it loads
    any of it, and the first lets the next be scheduled only after that."""
    body = dict(_kernels())
    for name in ("amax_partial_kernel", "quant_rows_kernel"):
        wait = re.search(r"\n  pdl_wait\(\);", body[name])  # of every thread, on every path
        assert wait and wait.start() < body[name].index("load_raw("), name
        assert wait.start() < body[name].index("pdl_trigger()"), name
    cols = body["quant_cols_kernel"]
    assert cols.index("quant_tensor_scale(") < cols.index("ld_behind_l2(x")


# Read-only loads of the call's inputs alone (weights' scales, the tensor scale;
# the cache's scales and weights), which are final before the call's first
# kernel, having waited, lets these start.
READ_ONLY_LOADS = {"linear_kernel", "kv8_gather_kernel"}


def test_what_the_kernel_before_may_have_written_is_not_loaded_as_read_only():
    """A read-only load says that nothing writes the memory while the kernel
    exists: of a kernel that is scheduled early that is not so, and the load
    may be moved ahead of the wait."""
    for name, body in _kernels():
        if "pdl_wait()" in body or "quant_tensor_scale(" in body:
            assert bool(re.search(r"__ldg\(", body)) == (name in READ_ONLY_LOADS), name
            assert "__ldcg(" not in body, name
    for name in ("kv8.cuh", "linear.cuh", "tc.cuh"):
        with open(os.path.join(CSRC, name)) as f:
            assert "ld.global.nc" not in f.read(), name
    with open(os.path.join(CSRC, "quant_kernels.cuh")) as f:
        raw = re.search(r"void load_raw\(.*?\n\}", f.read(), re.S).group(0)
    assert raw.count("ld_behind(") == 2 and "__ldg" not in raw
    with open(os.path.join(CSRC, "kv8.cuh")) as f:
        geom = re.search(r"struct Kv8Geom \{.*?\n\};", f.read(), re.S).group(0)
    assert "ld_behind(lens + b)" in geom and "__ldg" not in geom


def test_loads_behind_a_wait_stay_there():
    """Each is volatile, as the wait is: neither passes the other."""
    with open(os.path.join(CSRC, "tc.cuh")) as f:
        text = f.read()
    loads = re.findall(r"asm(?: volatile)?\(\"ld\.global[^\"]*", text)
    assert len(loads) >= 4 and all(x.startswith("asm volatile") for x in loads)
    assert 'asm volatile("griddepcontrol.wait;" ::: "memory")' in text
