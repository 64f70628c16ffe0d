"""Attention calls without queries or without batch entries against keys of
any number (no GPU needed).  Each call runs in a child process, where a signal
is a failure like any other, with a stand-in for the runtime's launch loaded
ahead of it that starts nothing."""
import json

import pytest
from test_attention_limits_cpu import launches  # noqa: F401  (the fixture)
from test_launch_limits_cpu import check

KEYS = [0, 1, 127, 128, 255, 256, 300, 1000, 4096, 1 << 20]


@pytest.mark.parametrize("dim", [1, 33, 64, 72, 128])
@pytest.mark.parametrize("dt", [0, 1])
def test_no_queries_or_no_batch(launches, dim, dt):  # noqa: F811
    """All four entry points take them (the sizes and both passes); what is
    launched is the zeros of the keys' and λ's gradients."""
    calls = [["attention", b, q, k, h, kv, dim, 0, causal, dt] for b, q in ((1, 0), (3, 0), (0, 5), (0, 0)) for k in KEYS
             for h, kv in ((4, 2), (28, 4)) for causal in (0, 1)]
    calls += [["attention", 1, 0, 0, 4, 2, dim, n, 1, dt] for n in (1, 5000)]  # a packed batch of no tokens
    found = launches(calls)
    assert len(found) == len(calls)
    check({c: ls for c, (ls, _) in found.items()}, least=1)
    for c, (ls, _) in found.items():
        _, b, _, k, h, _, _, seqs, *_ = json.loads(c)
        if b * k == 0 and not seqs:  # λ's gradient alone
            assert [g for g, _ in ls] == [[h, 1, 1]], c
