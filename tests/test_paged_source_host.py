"""The barriers of the softmax warps of the bf16 attention over pages, read from the source of its kernel and
walked through on the host."""
import itertools
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "lsh_sampled_sparse_gb300", "csrc")


def _softmax_loop():
    """The softmax warps' loop over tiles, without comments."""
    with open(os.path.join(CSRC, "mp_paged_tc.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    loop = code[code.index("for (int it = 0; total > 0; ++it)"):code.index("} else if (warp == 4)")]
    return loop


def _events():
    """[(kind, condition)] of a pass in the order of the source: the barriers among the softmax warps, and
    what is written to and read from the array of the warps' sums. The condition is that of the innermost
    `if` that tells passes apart."""
    found = []
    block = [None]                               # a condition a brace; None: always
    token = re.compile(r"if \((more|it > 0|!fresh|fresh|!more)\) (softmax_sync\(\);|\{)|\} else \{|\{|\}|"
                       r"softmax_sync\(\);|sums\[[^\]]*\] = |sums\[h\]")
    closed = None
    for m in token.finditer(_softmax_loop()):
        t = m.group(0)
        if m.group(1) and m.group(2) == "{":
            block.append(m.group(1))
        elif m.group(1):
            found.append(("barrier", [*filter(None, block), m.group(1)]))
        elif t == "} else {":
            closed = block.pop()
            block.append("fresh" if closed == "!fresh" else None)
        elif t == "{":
            block.append(None)
        elif t == "}":
            if len(block) > 1:
                block.pop()
        else:
            kind = "barrier" if t.startswith("softmax") else ("write" if t.endswith("= ") else "read")
            found.append((kind, list(filter(None, block))))
    return found


def _walk(units):
    """The barriers and accesses of a warp over a run of units of so many tiles each, in order."""
    tests = {"more": lambda more, fresh, it: more, "!more": lambda more, fresh, it: not more,
             "fresh": lambda more, fresh, it: fresh, "!fresh": lambda more, fresh, it: not fresh,
             "it > 0": lambda more, fresh, it: it > 0}
    events, total, it, ends = _events(), sum(units), 0, set(itertools.accumulate(units)) | {0}
    for it in range(total + 1):
        more, fresh = it < total, it in ends
        for kind, conditions in events:
            if all(tests[c](more, fresh, it) for c in conditions):
                yield kind


def test_the_events_of_a_pass_are_found():
    assert [k for k, _ in _events()].count("write") == 1
    assert [k for k, _ in _events()].count("read") == 1
    assert [k for k, _ in _events()].count("barrier") >= 2


@pytest.mark.parametrize("units", [[1], [5], [1, 1], [3, 1], [1, 3], [1, 1, 1, 1], [4, 1, 2, 1], [2, 2], [7, 1]])
def test_no_warp_writes_the_sums_while_another_may_read_the_last_ones(units):
    """Between an access of the sums and the next one of the other kind stands a barrier of the four warps:
    else a warp that lags would read the sums of another unit."""
    since, last, writes = 0, None, 0
    for kind in _walk(units):
        if kind == "barrier":
            since += 1
            continue
        writes += kind == "write"
        if last is not None and last != kind:
            assert since > 0, (units, last, kind)
        last, since = kind, 0
    assert writes == len(units)


def test_no_capacity_is_rounded_up_in_32_bits():
    """A capacity may be 2^31 - 1: n + 1023 wraps there, and the blocks a head has would be negative."""
    found = []
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        found += [(name, m.group(0)) for m in
                  re.finditer(r"[^\n;(]*\S+ \+ kKeysPerBlock - 1\) / kKeysPerBlock", code)
                  if "static_cast<size_t>" not in m.group(0) and not m.group(0).startswith("n) +")]
    assert not found


def test_blocks_of_the_largest_capacities(tmp_path):
    """The product's own count, compiled for the host."""
    import subprocess
    from lsh_sampled_sparse_gb300.build import NVCC_FLAGS, nvcc
    src = tmp_path / "blocks.cu"
    src.write_text('#include <cstdio>\n#include "mp_internal.cuh"\nint main() {\n'
                   "    for (int n : {1, 2, 1023, 1024, 1025, 1 << 30, 2147483647 - 1024, 2147483647 - 1023,\n"
                   "                  2147483647 - 1022, 2147483647})\n"
                   '        printf("%d %d\\n", n, mp::key_blocks(n));\n}\n')
    exe = tmp_path / "blocks"
    subprocess.run([nvcc(), *NVCC_FLAGS, str(src), "-o", str(exe)], check=True)
    rows = [tuple(map(int, line.split())) for line in
            subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    assert len(rows) == 10 and all(b == -(-n // 1024) for n, b in rows)


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_workspace_and_the_table_are_reached_behind_index_checks_only():
    """What the header says the checks build checks: partial states and beginnings of runs against the
    workspace, slots against the table, code words against the codes."""
    shared = _code("mp_paged.cuh")
    assert shared.count("a.begin[") == shared.count("begin_there(a, ") == 4
    for name in ("mp_paged.cu", "mp_paged_tc.cu", "mp_paged_mma.cu"):
        code = _code(name)
        stores = re.findall(r"(\S[^\n]*)\n\s*float\* p = part_of\(", code)
        assert len(stores) == 1 and all("part_there(a, blockIdx.x, " in s for s in stores), name
        # every entry by page_in, or (an append's) by paged_row, whose tokens were held against the table
        assert not re.search(r"table\[|slots\[", code), name
        assert "page_in(" in code
    join = re.search(r"__global__[^\n]* paged_join_kernel.*?\n}\n", _code("mp_paged.cu"), re.S).group(0)
    assert join.index("begin_there") < join.index("__ldcg")
    assert join.count("a.part +") == 1 and "part_there(a, s, s == c0, hc)" in join
    assert shared.count("slots[") == 1 and "kSitePagedRow) ? slots[slot] : -1" in shared
    decode = _code("mp_decode.cu")
    assert decode.count("slots[") == 1 and "a.pages.n_slots, kSitePagedRow) ? slots[slot0 + i] : -1" in decode
    at = re.search(r"encode_rows_at_kernel\(const AtArgs.*?\n}\n", _code("mp_append.cu"), re.S).group(0)
    assert at.count("mp_check(") == 2 and at.index("a.cblk * a.C * kWordsPerBlock") < at.index("atomicOr")
