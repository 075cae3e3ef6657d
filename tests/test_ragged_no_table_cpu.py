"""Tables without columns: taken where they have no memory, refused where a pointer comes with no columns."""

import pytest

from tests.test_ragged_capi_cpu import P, _cross, _shared


@pytest.mark.parametrize("call,over", [(_cross, dict(mb=0, bt=None)), (_shared, dict(mb=0, bt=None)),
                                       (_shared, dict(pb=0, pt=None)), (_shared, dict(mb=0, bt=None, pb=0, pt=None))])
def test_no_columns(call, over):
    assert call(**over, wsb=64) == 3  # the next refusal: the workspace
    assert call(**over, **{("kl" if call is _cross else "sl"): None}) == 1  # lengths are there all the same


@pytest.mark.parametrize("call,over", [(_cross, dict(mb=-1)), (_cross, dict(mb=-1, bt=None)), (_shared, dict(mb=-1, bt=None)),
                                       (_shared, dict(pb=-1, pt=None)), (_shared, dict(pb=0, pt=P))])
def test_refused(call, over):
    assert call(**over) == 1
