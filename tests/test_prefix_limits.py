"""CPU checks of attention over shared prefixes: numbers of requests and groups near 2^31."""
from test_prefix_refusals import INVALID, call

MOST = 2 ** 31 - 1


def test_requests_and_groups_beyond_a_limit():
    for kw in (dict(groups=MOST), dict(groups=MOST - 1023), dict(B=MOST), dict(groups=1 << 29, B=(1 << 29) + 1),
               dict(groups=1 << 30)):
        assert call(**kw) == INVALID, kw
    assert call(groups=1 << 29, B=1 << 29, n=0, ts=None) == INVALID  # (rows without tok_start are one a request)
    assert call(groups=1 << 29, B=1 << 29, n=0) == 0
