"""Outputs and workspaces of cross attention and shared prefixes that share memory with an input (nothing is launched)."""

import pytest

from tests.test_ragged_capi_cpu import LSE, OUT, P, WS, _cross, _shared

# what each input takes: 64 pages of 8 heads x 16 keys x 128 dims, a scale or one a row, tables of 8 (4) columns
CACHE, ROWS = 64 * 8 * 16 * 128, 64 * 8 * 16 * 4


def _cases(out_bytes, lse_bytes, inputs):
    for name, size, over in inputs:
        for at, span in ((OUT, out_bytes), (LSE, lse_bytes)):
            yield {name: at, **over}
            if size >= 32:  # its last bytes are the output's first ones, and the other way round
                yield {name: at - size + 16, **over}
            yield {name: at + span - 16 if name in ("kc", "vc") or over else at + span - 4, **over}
        yield {name: WS, **over}
        yield {name: WS + 256, **over}


COMMON = [("kc", CACHE, {}), ("vc", CACHE, {}), ("ks", 4, {}), ("vs", 4, {}), ("ks", ROWS, dict(rows=1)),
          ("vs", ROWS, dict(rows=1)), ("bt", 2 * 8 * 4, {})]
CROSS = [*_cases(10 * 4096 * 2, 10 * 32 * 4, [*COMMON, ("starts", 12, {}), ("kl", 8, {})])]
SHARED = [*_cases(2 * 4096 * 2, 2 * 32 * 4, [*COMMON, ("sl", 8, {}), ("pt", 2 * 4 * 4, {}), ("pl", 8, {}), ("ps", 12, {}),
                                            ("mask", 2, {}), ("sinks", 32 * 4, {})])]


def _text(over):
    return ",".join(f"{k}={v - P if isinstance(v, int) and v >= P else v}" for k, v in over.items())


@pytest.mark.parametrize("over", CROSS, ids=_text)
def test_cross(over):
    assert _cross(**over) == 1


@pytest.mark.parametrize("over", SHARED, ids=_text)
def test_shared(over):
    assert _shared(**over) == 1
