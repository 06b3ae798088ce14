"""Arguments of drafted trees and eviction that share memory where a call reads one while it writes the other:
refused before any work (no GPU)."""
import ctypes

import pytest

import __graft_entry__

P, OK, INVALID = 1 << 20, 0, 1       # P: an aligned address that is never read


@pytest.fixture(scope="module")
def pk():
    __graft_entry__.build()
    import paged_kv_decode_store_gb300 as pk
    return pk


def select(pk, counts, ctx, seqs=3, **kw):
    a = dict(w_out=None, s_seq=800, s_head=100, length=100, heads=8)
    a.update(kw)
    return pk.lib().pkvd_evict_select(64 * P, counts, a["w_out"], 32 * P, a["s_seq"], a["s_head"], a["length"], ctx, seqs,
                                      a["heads"], 10, 2, 8, None, None)


@pytest.mark.parametrize("off", [0, 4, 8, -4, -8])
def test_counts_over_context_lens(pk, off):
    """The rows of other heads, and the order by length, still read a length that is a count already."""
    assert select(pk, P + off, P) == INVALID
    assert select(pk, P, P, seqs=0) == OK
