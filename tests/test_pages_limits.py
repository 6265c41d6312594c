"""CPU checks of sizes near 2^31 in the calls for pages that several requests hold and in attention over
shared prefixes: refused before anything is launched."""
import pytest

from fp8_paged_kv_attn_gb300 import kvq
from test_pages_refusals import INVALID, WORKSPACE, call

LIMIT, MOST = 1 << 30, 2 ** 31 - 1


@pytest.mark.parametrize("op,names", [("fork", ("pages", "B", "n")), ("release", ("pages", "B", "n")),
                                      ("compact", ("pages", "B", "cap"))])
def test_sizes_beyond_a_limit(op, names):
    for name in names:
        for size in (LIMIT + 1, MOST - 65535, MOST):
            more = {"cap": MOST} if op == "compact" and name == "pages" else {}
            assert call(op, **{name: size, **more}) == INVALID, (name, size)
    more = {"cap": LIMIT} if op == "compact" else {"n": LIMIT}
    assert call(op, pages=LIMIT, B=LIMIT, wsb=0, **more) == WORKSPACE  # the largest that are taken


def test_workspace_of_sizes_beyond_a_limit():
    f = kvq.kvq_pages_workspace_size
    assert f(LIMIT + 1, 1) == f(1, LIMIT + 1) == f(MOST, MOST) == 0
    assert f(LIMIT, LIMIT) >= 3 * 4 * LIMIT
