"""Batches none of whose sequences has a key: tables without columns."""

import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from tests import ragged_inputs as inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("bs", [0, 3, 400])
@pytest.mark.parametrize("of_a_view", [False, True])
def test_cross(bs, of_a_view):
    pool = inputs.Pool(1, [[20]], 2, 64, 16, False)
    k, v, _, ks, vs = pool.device(DEV)
    q = pool.queries(2 * bs + 1, 4).to(DEV)
    table = torch.zeros((bs, 3), dtype=torch.int32, device=DEV)[:, :0].contiguous() if of_a_view else \
        torch.zeros((bs, 0), dtype=torch.int32, device=DEV)
    starts = torch.arange(0, 2 * bs + 1, 2, dtype=torch.int32, device=DEV)
    lens = torch.zeros(bs, dtype=torch.int32, device=DEV)
    out, lse = fm.paged_cross_attention(q, k, v, table, lens, ks, vs, q_starts=starts)
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    out, lse = fm.paged_cross_attention(q[:bs], k, v, table, lens, ks, vs)
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    assert fm.last_device_error() == 0
    if bs:  # a length that such a table cannot hold
        lens[bs // 2] = 1
        out, lse = fm.paged_cross_attention(q[:bs], k, v, table, lens, ks, vs)
        assert fm.last_device_error() == fm.DEV_BAD_SEQLEN and bool((out == 0).all())


@pytest.mark.parametrize("q_len", [1, 3])
def test_shared(q_len):
    """Either table without columns, and both, where only sinks are left."""
    lens = [40, 7, 3]
    pool, q, m, s, want = inputs.shared_case(2, [50], [0, 2], lens, 2, 2, 128, 16, True, q_len=q_len, sinks=True)
    k, v, prefixes, own, ks, vs = pool.device(DEV)
    kw = dict(softmax_scale=pool.softmax_scale, sinks=torch.from_numpy(s).to(DEV))
    none = torch.zeros((3, 0), dtype=torch.int32, device=DEV)
    shared = inputs.ragged.shared
    rest = (*pool.scale, pool.softmax_scale, None, s)
    for p_table, p_len, table, own_lens in ((prefixes, 50, none, [0, 0, 0]), (none[:1], 0, own, lens),
                                            (none[:1], 0, none, [0, 0, 0])):
        got = fm.paged_gqa_decode_shared(q.to(DEV), k, v, p_table, _i32(p_len), _i32(0, 2), table, _i32(*own_lens), ks, vs,
                                         **kw)
        want = shared(q, *pool.cache, pool.tables[0], [p_len], [0, 2], pool.tables[1], own_lens, *rest)
        wrong = inputs.within(*got, want, 100)
        assert wrong is None, wrong
    assert fm.last_device_error() == 0
