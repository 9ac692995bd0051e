"""The bounded waits of the cache's kernels: none gives up unheard.  A wait that runs out cannot be made to on a sound
GPU without a kernel that is broken on purpose, so the sources are looked at: each wait's result is used, or put aside
by name, and what follows a wait in kq_kv_append stands behind the abort flag that it raises."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kronecker_factored_transforms_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["kq_kv_append.cu", "kq_kv_attention.cu", "kq_kv_tile.cu"])
def test_no_wait_is_dropped(name):
    """A call that is a whole statement, alone or behind an if, drops its result."""
    text = source(name)
    assert re.search(r"\bwait(_all)?\(", text)
    dropped = re.findall(r"(?:[;{}]|\bif \([^;{}]*\)|\belse)\s+((?:tc::)?(?:wait|wait_all|wait_bounded_err)\([^;]*;)", text)
    assert not dropped, dropped


def test_append_leaves_when_a_wait_gave_up():
    text = source("kq_kv_append.cu")
    # products are issued, and rows stored, only where no wait has given up
    assert re.search(r"elect_one\(\) && ok && !\*s_abort", text)
    assert re.search(r"if \(!wait\(ready, [^;]*\) \|\| __any_sync\(0xffffffffu, \*s_abort != 0\)\) break;", text)
