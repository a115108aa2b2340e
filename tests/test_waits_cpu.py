"""Kernels that are launched while the stream's previous kernel still runs: before their wait they touch nothing that
it may have written. Only declarations and arithmetic on indices and on the parameters' plain numbers stand there."""

import re

import pytest

from test_dependent_sources_cpu import CSRC, SOURCES

CALLS = {"min", "max", "cta_rank", "cluster_ctas"}
WAIT = re.compile(r"\b(begin_dependent|wait_for_previous_kernel)\(\)")


def kernels(text):
    """Name and body of each kernel of a source without its comments."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\((?:[^(){}]|\([^()]*\))*\)\s*\{(.*?)\n\}", text, re.S):
        yield m.group(1), m.group(2)


def touched(body):
    """What a kernel does before its wait that could read or write memory."""
    m = WAIT.search(body)
    assert m, "no wait"
    found = []
    for line in body[:m.start()].split(";"):
        line = " ".join(line.split())
        if re.match(r"(extern )?__shared__ [^=]*$", line):
            continue
        found += [line] if "[" in line or "->" in line else []
        found += [line] if re.search(r"(?:^|[=(,&|?:<>+\-!~{}]|\breturn)\s*\*", line) else []
        found += [line for f in re.findall(r"([A-Za-z_]\w*)\s*(?:<[^<>;]*>)?\s*\(", line) if f not in CALLS]
        found += [line for _ in re.findall(r"(?:^|\s)[A-Za-z_][\w:]*(?:<[^<>;]*>)?\s+\w+\{", line)]
    return found


@pytest.mark.parametrize("name", [s for s in SOURCES if s.endswith(".cu")])
def test_nothing_is_touched_before_the_wait(name):
    found = dict(kernels((CSRC / name).read_text()))
    assert found and (CSRC / name).read_text().count("__global__") == len(found)
    for kernel, body in found.items():
        assert touched(body) == [], kernel


@pytest.mark.parametrize("line", [
    "const int n = p.num_draft[b];", "const int64_t s = p.slot_map[t];", "int64_t nf = *p.num_free;", "if (lane == 0) *p.ticket = 0u;",
    "const int n = drafts_of(p, b);", "const int x = __ldcg(p.seq_lens + b);", "const float was = *scale;",
    "const QueryLane<128> ql(p, lane);", "atomicOr(p.err, 1u);", "const F fmt{p, lane};", "stream_split<F, NT, MOD>(fp);",
    "const int y = min(p.q_len, *p.num_free);", "auto v = reinterpret_cast<const int4 *>(p.k)[lane];", "prefetch_l2(p.q, 256);",
    "const int *q = p.num_draft; const int n = q[b];", "const int n = -*p.num_free;"])
@pytest.mark.parametrize("name", ["verify.cu", "cache_blocks.cu", "tables.cu", "fp4_split.cu"])
def test_a_load_ahead_of_the_wait_is_seen(name, line):
    for kernel, body in kernels((CSRC / name).read_text()):
        at = WAIT.search(body).start()
        assert touched(body[:at] + line + "\n  " + body[at:]) != [], kernel
