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


ROWS = [  # sequences, heads, their strides: rows of 100 words that meet
    (2, 2, 100, 100), (2, 3, 250, 200), (5, 2, 100, 400), (3, 3, 299, 200), (2, 2, 101, 200), (65535, 4, 150, 65534 * 150),
]


@pytest.mark.parametrize("seqs,heads,s_seq,s_head", ROWS)
def test_rows_of_weights_that_meet(pk, seqs, heads, s_seq, s_head):
    """Two of them would be written to the same words."""
    used = set()
    if seqs < 100:
        for i in range(seqs):
            for h in range(heads):
                row = set(range(i * s_seq + h * s_head, i * s_seq + h * s_head + 100))
                met = bool(used & row)
                used |= row
                if met:
                    break
            if met:
                break
        assert met
    assert select(pk, 16 * P, 8 * P, seqs=seqs, heads=heads, s_seq=s_seq, s_head=s_head, w_out=32 * P) == INVALID
