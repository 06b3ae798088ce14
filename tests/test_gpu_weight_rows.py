"""Rows of counted weights in layouts of every kind: sequence by sequence, head by head, and between one another."""
import pytest
import torch

from gpu_helpers import require_gpu
from test_gpu_score_mod import cache_of
from test_gpu_tree import ints

pytestmark = pytest.mark.gpu
DEV = "cuda"
N, H, L = 3, 2, 100


def rows(s_seq, s_head, start=1):
    """A view of N x H rows of L words in a buffer of -1, and the buffer."""
    buf = torch.full((start + (N - 1) * s_seq + (H - 1) * s_head + L + 5,), -1.0, device=DEV)
    return buf.as_strided((N, H, L), (s_seq, s_head, 1), start), buf


LAYOUTS = [(H * L, L), (H * L + 7, L + 3), (L, N * L), (L + 1, N * L + 9), (2 * L, L), (2 * L, 3 * L), (150, 3 * 150)]
# (the last but one: rows of the next sequence lie between this one's)


@pytest.mark.parametrize("s_seq,s_head", LAYOUTS)
def test_layouts(s_seq, s_head):
    pk = require_gpu()
    ctx = ints([100, 31, 77])
    g = torch.Generator().manual_seed(1)
    plain = torch.rand(N, H, L, generator=g).to(DEV)
    w, buf = rows(s_seq, s_head)
    w.copy_(plain)
    kc, vc, tables, _ = cache_of([100, 31, 77], H, 64, 16, torch.float32, 2)
    q = torch.randn(N, 4, 64, generator=g).to(DEV)
    a, _ = pk.paged_decode_attention_weights(q, kc, vc, tables, ctx, L, 0.1, plain)
    b, _ = pk.paged_decode_attention_weights(q, kc, vc, tables, ctx, L, 0.1, w)
    assert torch.equal(a, b) and torch.equal(w, plain)
    pos, counts = pk.evict_select(plain, ctx, 40, sink=2, recent=5, weights_out=plain)
    got = pk.evict_select(w, ctx, 40, sink=2, recent=5, weights_out=w)
    assert torch.equal(got[0], pos) and torch.equal(got[1], counts) and torch.equal(w, plain)
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided((N, H, L), (s_seq, s_head, 1), 1).fill_(False)
    assert torch.all(buf[mask] == -1)


@pytest.mark.parametrize("s_seq,s_head", [(100, 100), (250, 200), (101, 200)])
def test_rows_that_meet(s_seq, s_head):
    """Refused where they are written; a selection alone may read them."""
    pk = require_gpu()
    w, buf = rows(s_seq, s_head)
    buf.uniform_()
    apart, ctx = w.contiguous(), ints([100, 31, 77])
    before = buf.clone()
    kc, vc, tables, _ = cache_of([100, 31, 77], H, 64, 16, torch.float32, 3)
    with pytest.raises(pk.PkvdError):
        pk.paged_decode_attention_weights(torch.zeros(N, 4, 64, device=DEV), kc, vc, tables, ctx, L, 0.1, w)
    with pytest.raises(pk.PkvdError):
        pk.evict_select(w, ctx, 40, weights_out=w)
    assert torch.equal(buf, before)
    a, b = pk.evict_select(w, ctx, 40, sink=1, recent=3), pk.evict_select(apart, ctx, 40, sink=1, recent=3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
