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


@pytest.mark.parametrize("off", [0, 16, 256, 20 * 48 * 128 * 2 - 16, -16, -(20 * 48 * 128 * 2 - 16)])
def test_tree_outputs_over_queries(pk, off):
    """A CTA reads a row of q, for another KV head or part of its keys, after others have written theirs."""
    from paged_kv_decode_store_gb300 import _capi
    c = _capi.PkvdCache(P, P, 2, 16, 64, 8, 128, 16 * 8 * 128, 8 * 128, 128)
    q = 64 * P
    assert pk.lib().pkvd_tree_attention(q + off, q, ctypes.byref(c), P, 8, P, P, P, 2, 20, 9, 48, 0.1, 0, None, None, 0, None,
                                        None, 0) == INVALID
