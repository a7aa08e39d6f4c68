"""Every kernel that uses mbarriers orders their initialisation before their
first use (CPU only; read from the sources).

An arrival that came before another thread's initialisation of the same barrier
would be erased by it, and the wait for it would run out.  So between the last
`mbar_init` of a kernel and the first call that arrives on a barrier, waits on
one or gives one to a copy or a product, there has to be a barrier of all the
threads that take part: the block's, or in kernels of one warp the warp's."""
import glob
import os
import re

import pytest

from paged_kv_cache_468_b200 import build

USE = re.compile(r"\b(?:mbar_arrive\w*|mbar_wait\w*|mbar_try_wait|tma_load_\w+|bulk_load|tc_commit)\s*\(")
WARP = {"compact_long_kernel", "bounded_wait_selftest_kernel", "counted_wait_selftest_kernel"}   # kernels of one warp


def _code(text):
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return re.sub(r"//[^\n]*", " ", text)


def _body(text, at):
    """The braces' text that opens at or after `at`."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError("unbalanced braces")


def _functions():
    """(name, body) of the device functions that initialise barriers."""
    found = {}
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))):
        text = _code(open(path).read())
        for m in re.finditer(r"__(?:global|device)__[^;{}]*?\b(\w+)\s*\(", text):
            # the function's own name: the last word before its argument list
            head = text[m.start():text.index("{", m.end())]
            if ";" in head:
                continue
            names = [n for n in re.findall(r"\b(\w+)\s*\(", head) if n not in ("__launch_bounds__", "asm")]
            if not names:
                continue
            body = _body(text, m.end())
            if "mbar_init(" in body:
                found[names[0]] = body
    return found


FOUND = _functions()


def test_all_kernels_with_barriers_are_seen():
    sources = "".join(_code(open(p).read()) for p in glob.glob(os.path.join(build.CSRC, "*.cu*")))
    calls = len(re.findall(r"\bmbar_init\s*\(", sources)) - 1                # (its definition)
    assert sum(len(re.findall(r"\bmbar_init\s*\(", b)) for b in FOUND.values()) == calls
    assert {"tree_attend_kernel", "tree_rows_kernel", "compact_long_kernel", "paged_decode_kernel"} <= set(FOUND)


@pytest.mark.parametrize("name", sorted(FOUND))
def test_initialisation_comes_before_the_first_use(name):
    body = FOUND[name]
    last = [m.end() for m in re.finditer(r"\bmbar_init\s*\(", body)][-1]
    use = USE.search(body, last)
    assert use, "barriers that nobody uses"
    between = body[last:use.start()]
    assert "fence_mbar_init()" in between
    barrier = r"__syncthreads\(\)|__syncwarp\(\)" if name in WARP else r"__syncthreads\(\)"
    assert re.search(barrier, between), f"{name}: {use.group(0)} before a barrier"
