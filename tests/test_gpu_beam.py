"""Beam search selection on the GPU against the float64 oracle: ids and parents
equal, scores within fp32 rounding; ties, ended, dead and masked beams."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def check(got, logits, scores, keep, finished=None, eos=-1):
    """Ids and parents, and scores rounded once (2^-24) after a normaliser off by
    at most NORM = 2^-20: the terms of its sum are fp32 exponentials, each off
    by at most 2^-22 and by the rounding of its argument (2^-24 of up to 6 for
    the terms that matter), so the sum's logarithm by less than 2^-20.

    A normaliser shifts all continuations of its beam alike, so the order
    within a beam is exact (the lowest id among equal logits), and continuations
    of different beams may only change places where their exact values are
    within 2 NORM of each other."""
    NORM = 2.0 ** -20
    s, p, t = (x.cpu().numpy() for x in got)
    n, b = scores.shape
    x = logits.double().cpu().numpy().reshape(n, b, -1)
    for r in range(n):
        fin = None if finished is None else finished[r].cpu().numpy()
        sc = scores[r].double().cpu().numpy()
        ws, wp, wt = oracle.beam.step(x[r], sc, keep, fin, eos)
        have = list(zip(p[r].tolist(), t[r].tolist()))
        value = ws
        if have != list(zip(wp, wt)):
            value, taken = [], {}
            for q, tok in have:
                taken.setdefault(q, []).append(tok)
            own = {q: oracle.beam.step(x[r, q:q + 1], sc[q:q + 1], keep, None if fin is None else fin[q:q + 1], eos)
                   for q in taken if q >= 0}
            for q, toks in taken.items():          # each beam's first ones, in its own order
                assert q >= 0 and toks == own[q][2][:len(toks)], (r, q, toks)
            count = {q: 0 for q in taken}
            for k, (q, tok) in enumerate(have):
                value.append(own[q][0][count[q]])
                count[q] += 1
                assert abs(value[k] - ws[k]) <= 2 * NORM, (r, k, have[k], value[k], ws[k])
        for a, w in zip(s[r], value):
            assert a == w or abs(float(a) - w) <= abs(w) * 2.0 ** -24 + NORM, (r, a, w)


def draw(n, b, V, dt, seed, std=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = (std * torch.randn(n * b, V, generator=g)).to(dt)
    scores = -5 * torch.rand(n, b, generator=g)
    return logits.to(DEV), scores.to(DEV)


SHAPES = [(1, 1, 1, 1), (1, 4, 1000, 4), (3, 2, 37, 5), (2, 5, 16384, 10), (2, 3, 16385, 6), (1, 8, 65537, 16),
          (2, 1, 151936, 64), (5, 4, 8191, 1), (1, 64, 513, 64), (1, 2, 40000, 33)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_beam_step(shape, dt):
    pk = require_gpu()
    n, b, V, keep = shape
    logits, scores = draw(n, b, V, DT[dt], 1)
    check(pk.beam_search_step(logits, scores, keep), logits, scores, keep)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("off", [1, 3, 8])
def test_strided_rows_at_any_alignment(dt, off):
    """Rows that start inside a 16-byte vector; what lies around them is NaN."""
    pk = require_gpu()
    V = 20001
    logits, scores = draw(2, 3, V, DT[dt], 2)
    wide = torch.full((6, V + 21), float("nan"), dtype=DT[dt], device=DEV)
    wide[:, off:off + V] = logits
    got = pk.beam_search_step(wide[:, off:off + V], scores, 6)
    check(got, logits, scores, 6)
    want = pk.beam_search_step(logits, scores, 6)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("keep", [1, 8, 64])
def test_equal_logits_go_to_the_lowest_index(dt, keep):
    """All equal (every id ties), a few levels, and a plateau wider than the list of candidates."""
    pk = require_gpu()
    V = 50000
    flat = torch.zeros(4, V, dtype=DT[dt], device=DEV)
    scores = torch.zeros(2, 2, device=DEV)
    check(pk.beam_search_step(flat, scores, keep), flat, scores, keep)
    steps = (torch.arange(V, device=DEV) % 7).to(DT[dt]).repeat(4, 1)
    check(pk.beam_search_step(steps, scores, keep), steps, scores, keep)
    plateau = flat.clone()
    plateau[1:, 123::2] = 3.0
    plateau[0, 49999] = 5.0
    plateau[2, 7] = 4.0
    signed = torch.zeros(4, V, dtype=DT[dt], device=DEV)
    signed[:, ::3] = -0.0                               # zeros of both signs are equal
    for x in (plateau, signed):
        check(pk.beam_search_step(x, scores, keep), x, scores, keep)


def test_ended_dead_masked_and_broken_beams():
    pk = require_gpu()
    logits, _ = draw(4, 4, 30000, torch.bfloat16, 3)
    inf = float("inf")
    scores = torch.tensor([[-1.0, -2.0, -inf, -0.5], [-1.0, -1.0, -1.0, -1.0], [0.0, -inf, -inf, -inf],
                           [float("nan"), inf, -3.0, -4.0]], device=DEV)
    ended = torch.tensor([[1, 0, 1, 0], [1, 1, 1, 1], [0, 0, 0, 0], [0, 1, 0, 1]], dtype=torch.uint8, device=DEV)
    logits[1] = float("nan")
    logits[3, 77] = float("nan")                        # one NaN, one +inf, and a row without any id
    logits[8, ::2] = -inf
    logits[14, 5] = inf
    logits[4:8] = float("nan")                          # ended beams' logits are not read
    for keep in (1, 4, 8):
        for fin in (ended, ended.bool()):
            check(pk.beam_search_step(logits, scores, keep, finished=fin, eos_id=29999), logits, scores, keep, ended,
                  29999)
    logits[8] = -inf
    logits[8, 12345] = -7.0
    got = pk.beam_search_step(logits, scores, 8)
    check(got, logits, scores, 8)
    assert got[2][2].tolist() == [12345] + [-1] * 7 and got[0][2, 0].item() == 0.0
    logits[8] = -inf
    assert pk.beam_search_step(logits, scores, 8)[1][2].tolist() == [-1] * 8


@pytest.mark.parametrize("dt", list(DT))
def test_rows_of_large_numbers_and_masks_of_the_lowest_value(dt):
    """Rows around +-2048, 30000 and (where the type has them) 10^30, ids masked
    with the type's lowest value, and rows of nothing else: those continue with
    every id at score - log vocab."""
    pk = require_gpu()
    lowest, V = torch.finfo(DT[dt]).min, 20001
    logits, scores = draw(3, 4, V, DT[dt], 6)
    x = logits.float()
    far = [2040.0, -2047.0, 2049.0, -2100.0, 30000.0, -30000.0, 1e30 if dt != "f16" else 60000.0, 0.0]
    x[:8] += torch.tensor(far, device=DEV).view(-1, 1)
    x = x.to(DT[dt])
    x[7, ::3] = lowest
    x[8] = lowest
    x[9, 100:] = lowest
    x[10] = lowest
    x[10, 77] = 3.0
    scores[2, 0] = 9.0                                  # the masked row's beam is the best one
    for keep in (4, 64):
        check(pk.beam_search_step(x, scores, keep), x, scores, keep)


def test_few_ids_left_in_every_slice_and_many_candidates():
    """Masks that leave a few ids a slice (fewer than keep), and slices whose best ids crowd together."""
    pk = require_gpu()
    V = 200000
    logits, scores = draw(2, 4, V, torch.float16, 4)
    keepers = torch.zeros(V, dtype=torch.bool)
    keepers[torch.arange(0, V, 4001)] = True
    masked = logits.masked_fill(~keepers.to(DEV), float("-inf"))
    for keep in (8, 64):
        check(pk.beam_search_step(masked, scores, keep), masked, scores, keep)
    crowd = logits.clamp(max=0)
    crowd[:, 3000:5500] = 9.0                           # 2500 equal ones in a slice
    check(pk.beam_search_step(crowd, scores, 64), crowd, scores, 64)
    same = logits[:1].repeat(8, 1)                      # identical beams: the lower one first
    check(pk.beam_search_step(same, torch.zeros_like(scores), 64), same, torch.zeros_like(scores), 64)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("V", [1, 7, 511, 513, 33333])
def test_equal_beams_tie_exactly_whatever_their_alignment(V, dt):
    """Rows of the same logits that start at every offset of a 16-byte vector: the lowest beam first, always."""
    pk = require_gpu()
    one = draw(1, 1, V, DT[dt], 7)[0]
    x = one.repeat(9, 1)
    wide = torch.zeros(9, V + 2 - V % 2 + 1, dtype=DT[dt], device=DEV)      # odd row stride
    wide[:, :V] = x
    zero = torch.zeros(1, 9, device=DEV)
    want = oracle.beam.step(x.double().cpu().numpy(), np.zeros(9), 20)
    for rows in (x, wide[:, :V]):
        s, p, t = pk.beam_search_step(rows, zero, 20)
        assert p[0].tolist() == want[1] and t[0].tolist() == want[2]
        assert s[0].tolist() == sorted(s[0].tolist(), reverse=True)


def test_a_merge_of_more_candidates_than_its_list():
    """64 beams of one level each: every slice offers 64 equal ids, all tie in the merge."""
    pk = require_gpu()
    x = torch.zeros(64, 40000, device=DEV)
    s = torch.zeros(1, 64, device=DEV)
    check(pk.beam_search_step(x, s, 64), x, s, 64)
    x[63, 5] = 1e-3
    check(pk.beam_search_step(x, s, 64), x, s, 64)


def test_scores_in_place_another_stream_and_a_replayed_graph():
    pk = require_gpu()
    logits, scores = draw(3, 4, 33000, torch.bfloat16, 5)
    want = pk.beam_search_step(logits, scores, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = pk.beam_search_step(logits, scores, 4, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    state = scores.clone()
    out = (state, torch.empty(3, 4, dtype=torch.int32, device=DEV), torch.empty(3, 4, dtype=torch.int32, device=DEV))
    ws = torch.empty(pk.beam_workspace_bytes(3, 4, 33000, torch.bfloat16, 4), dtype=torch.uint8, device=DEV)
    ret = pk.beam_search_step(logits, state, 4, out=out, workspace=ws)
    assert ret[0] is state and all(torch.equal(a, b) for a, b in zip(ret, want))
    state.copy_(scores)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.beam_search_step(logits, state, 4, out=out, workspace=ws)
    before = scores.clone()
    for _ in range(3):                                  # each replay continues from the last one's scores
        g.replay()
        torch.cuda.synchronize()
        check(out, logits, before, 4)
        before = state.clone()


def test_empty_and_refused_calls():
    pk = require_gpu()
    logits, scores = draw(2, 3, 100, torch.float32, 6)
    assert [tuple(x.shape) for x in pk.beam_search_step(logits[:0], scores[:0], 5)] == [(0, 5)] * 3
    ok = dict(logits=logits, scores=scores, keep=3)
    for bad in (dict(scores=scores.half()), dict(scores=scores[0]), dict(scores=scores.cpu()), dict(logits=logits[:5]),
                dict(logits=logits.t()), dict(logits=logits[:, ::2]), dict(finished=scores),
                dict(finished=torch.zeros(2, 2, dtype=torch.uint8, device=DEV), eos_id=1),
                dict(out=(scores, scores, scores)), dict(workspace=torch.zeros(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            pk.beam_search_step(**{**ok, **bad})
    with pytest.raises(TypeError):
        pk.beam_search_step(logits.double(), scores, 3)
    fin = torch.zeros(2, 3, dtype=torch.uint8, device=DEV)
    for bad in (dict(keep=0), dict(keep=65), dict(finished=fin), dict(finished=fin, eos_id=100),
                dict(workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(pk.PkvdError):
            pk.beam_search_step(**{**ok, **bad})
