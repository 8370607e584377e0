"""The selection of beams against fp64.

Tolerances: a candidate is score + x - lse in fp64, so its error is that of the
sum of exponentials, whose terms are 2^-22 off each at the most (the hardware's
exponential to a unit, and the rounded argument: 2^-24 of a distance of which
those beyond 2^5 do not count), less 32 + 6 additions in fp32 a lane of
positive terms: 2^-19 of the sum in the worst case; and the output's rounding
to fp32, 2^-24 of its value.  Which candidates are chosen is compared where the
fp64 values around a place differ by more than twice that or are equal."""
import math

import numpy as np
import pytest
import torch

import quantized_matmul_quantize_amd as qmm
from gpu_util import note

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
OFF = 2.0 ** -19


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def reference(x, scores, k, finished=None, pad=0):
    """Candidates in falling order, their flat places; x fp64 [seqs, beams, vocabulary]."""
    x = np.where(np.isnan(x), -np.inf, x)
    seqs, beams, vocabulary = x.shape
    most = x.max(-1)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        lse = most + np.log(np.exp(x - most[..., None]).sum(-1))
        value = scores.astype(np.float64)[..., None] + x - lse[..., None]
    dead = ~(np.isfinite(scores) & np.isfinite(most))
    if finished is not None:
        value[finished] = -np.inf
        value[finished, pad] = scores[finished]
        dead = np.where(finished, ~np.isfinite(scores), dead)
    value[dead] = -np.inf
    value = value.reshape(seqs, -1)
    at = np.argsort(-value, axis=1, kind="stable")[:, :k + 1]
    return np.take_along_axis(value, at, 1), at


def check(logits, scores, k, finished=None, pad=0):
    seqs, beams = scores.shape
    vocabulary = logits.shape[1]
    x = logits.double().cpu().numpy().reshape(seqs, beams, vocabulary)
    got, tokens, parents = qmm.beam_select(logits.cuda(), scores.cuda(), k,
                                           None if finished is None else finished.cuda(), pad)
    assert got.dtype == F32 and tokens.dtype == parents.dtype == torch.int64
    want, at = reference(x, scores.numpy(), k, None if finished is None else finished.numpy(), pad)
    got, tokens, parents = got.cpu().numpy(), tokens.cpu().numpy(), parents.cpu().numpy()
    for s in range(seqs):
        for i in range(k):
            if i >= want.shape[1] or want[s, i] == -np.inf:
                assert got[s, i] == -np.inf and tokens[s, i] == -1 and parents[s, i] == i % beams, (s, i)
                continue
            off = OFF + 2.0 ** -24 * abs(want[s, i])
            assert abs(got[s, i] - want[s, i]) <= off, (s, i, got[s, i], want[s, i])
            near = [want[s, j] for j in (i - 1, i + 1) if 0 <= j < want.shape[1]]
            if all(v == want[s, i] or abs(v - want[s, i]) > 2 * OFF for v in near):
                assert (parents[s, i], tokens[s, i]) == divmod(at[s, i], vocabulary), (s, i)
    return got, tokens, parents


def logits_of(g, rows, vocabulary, dtype, spread=2.0, padded=0):
    x = g.standard_normal((rows, vocabulary + padded)) * spread
    return torch.from_numpy(x.astype(np.float32)).to(dtype)[:, :vocabulary]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("seqs,beams,vocabulary,k", [
    (1, 1, 1, 1), (2, 3, 1, 5), (1, 4, 7, 4), (3, 2, 9, 18), (2, 5, 1000, 10), (1, 1, 8191, 64), (2, 2, 8192, 3),
    (1, 3, 8193, 7), (4, 4, 32003, 8), (1, 16, 50001, 32), (3, 8, 131072, 16), (1, 64, 5003, 64), (40, 2, 300, 4)])
def test_sizes(dtype, seqs, beams, vocabulary, k):
    note(f"beam_select {seqs} x {beams} of {vocabulary}, k={k} {dtype}")
    g = rng(vocabulary + k)
    scores = torch.from_numpy((-5 * g.random((seqs, beams))).astype(np.float32))
    check(logits_of(g, seqs * beams, vocabulary, dtype), scores, k)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
def test_rows_apart_and_of_any_alignment(dtype):
    g = rng(2)
    for padded in (1, 3, 64):
        x = logits_of(g, 6, 9001, dtype, padded=padded)
        scores = torch.from_numpy((-g.random((3, 2))).astype(np.float32))
        whole = torch.zeros((6, 9001 + padded), dtype=dtype, device="cuda")
        whole.fill_(math.inf)                               # what lies between the rows is not read
        whole[:, :9001] = x.cuda()
        a = qmm.beam_select(whole[:, :9001], scores.cuda(), 5)
        b = qmm.beam_select(x.contiguous().cuda(), scores.cuda(), 5)
        assert all(torch.equal(u, v) for u, v in zip(a, b))
        check(x, scores, 5)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("vocabulary", [33, 8200, 40001])
def test_equal_candidates_go_to_the_lowest_index(dtype, vocabulary):
    """All logits equal; few values; the same row in every beam with the same score."""
    g = rng(vocabulary)
    for x in (np.zeros((6, vocabulary)), g.integers(0, 3, (6, vocabulary)).astype(float), -0.0 * g.integers(-1, 2, (6, vocabulary)),
              np.tile(g.integers(-2, 9, (1, vocabulary)).astype(float), (6, 1))):
        logits = torch.from_numpy(x.astype(np.float32)).to(dtype)
        for k in (1, 4, 33):
            _, tokens, parents = check(logits, torch.zeros((2, 3)), k)
            flat = parents * vocabulary + tokens
            want, at = reference(logits.double().numpy().reshape(2, 3, -1), np.zeros((2, 3), np.float32), k)
            same = np.abs(np.diff(want[:, :k], axis=1)) == 0
            assert (np.diff(flat, axis=1)[same] > 0).all()
            assert np.array_equal(flat, at[:, :k])          # sums of equal rows are equal to the last bit


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
def test_banned_tokens_nan_infinities_and_dead_beams(dtype):
    g = rng(5)
    vocabulary, beams = 20001, 6
    x = logits_of(g, 2 * beams, vocabulary, dtype)
    x[0, torch.from_numpy(g.integers(0, vocabulary, 15000))] = -math.inf
    x[1] = -math.inf
    x[1, 17000] = 3.0                                       # one candidate alone
    x[2, 5], x[2, 9000], x[2, 20000] = math.nan, -math.nan, math.nan
    x[3] = -math.inf                                        # none
    x[4, 77] = math.inf
    x[7] = math.nan
    if dtype != F32:                                        # signalling ones
        x.view(torch.int16)[8, 100:200] = 0x7F81 if dtype == BF16 else 0x7C01
    else:
        x.view(torch.int32)[8, 100:200] = 0x7F800001
    scores = torch.from_numpy((-g.random((2, beams))).astype(np.float32))
    scores[1, 0], scores[1, 3], scores[1, 4] = -math.inf, math.nan, math.inf
    for k in (1, 6, 40):
        check(x, scores, k)


def test_fewer_candidates_than_asked_for():
    x = torch.full((4, 9000), -math.inf)
    x[1, 8999], x[3, 0] = 0.5, 0.25
    got, tokens, parents = check(x, torch.zeros((2, 2)), 5)
    assert got[0].tolist() == [0.0] + [-math.inf] * 4 and tokens[0].tolist() == [8999, -1, -1, -1, -1]
    assert parents.tolist() == [[1, 1, 0, 1, 0], [1, 1, 0, 1, 0]]
    check(torch.full((4, 9000), math.nan), torch.zeros((2, 2)), 3)


@pytest.mark.parametrize("pad", [0, 1, 30000])
def test_finished_beams_have_one_candidate(pad):
    g = rng(7)
    beams = 5
    x = logits_of(g, 3 * beams, 30001, BF16)
    x[0] = math.nan                                         # a finished beam's logits do not matter
    scores = torch.from_numpy((-4 * g.random((3, beams))).astype(np.float32))
    finished = torch.zeros((3, beams), dtype=torch.bool)
    finished[0, 0] = finished[0, 3] = finished[2, :] = True
    scores[2, 1] = -math.inf
    for k in (1, 5, 10):
        check(x, scores, k, finished, pad)


def test_peaked_rows_and_large_logits():
    """One token that has nearly all of the row; logits of any size."""
    g = rng(9)
    x = logits_of(g, 8, 40000, F32)
    x[0, 123], x[1, 39999] = 40.0, 100.0
    x[2] *= 1e4
    x[3] *= 1e-6
    x[4] += 1e5
    x[5] -= 3e38
    check(x, torch.zeros((2, 4)), 8)


def test_first_step_where_only_one_beam_counts():
    g = rng(10)
    x = logits_of(g, 3, 12345, F16).repeat_interleave(4, 0)
    scores = torch.full((3, 4), -math.inf)
    scores[:, 0] = 0.0
    _, _, parents = check(x, scores, 8)
    assert (parents == 0).all()


def test_no_sequences_workspace_another_stream_and_a_replayed_graph():
    out = qmm.beam_select(torch.empty((0, 100), device="cuda"), torch.empty((0, 4), device="cuda"))
    assert all(t.shape == (0, 4) for t in out)
    g = rng(11)
    x, scores = logits_of(g, 12, 70001, BF16).cuda(), torch.zeros((3, 4), device="cuda")
    want = qmm.beam_select(x, scores, 6)
    workspace = torch.full((qmm.beam_select_workspace_bytes(3, 4, 70001, 6),), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = qmm.beam_select(x, scores, 6, workspace=workspace)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = qmm.beam_select(x, scores, 6)
    for _ in range(3):
        x.copy_(logits_of(g, 12, 70001, BF16))
        scores.copy_(torch.from_numpy(-g.random((3, 4)).astype(np.float32)))
        graph.replay()
        want = qmm.beam_select(x, scores, 6)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
def test_more_equal_candidates_than_are_joined_at_once(dtype):
    """Of 64 beams of equal logits, and with one that is better by less than an fp32 value tells: 64 each of 3 to 5 blocks
    a beam, all of the same fp32 key."""
    x = torch.zeros((64, 40001), dtype=dtype, device="cuda")
    scores = torch.full((1, 64), -3.0, device="cuda")
    best, tokens, parents = qmm.beam_select(x, scores, 64)
    assert tokens[0].tolist() == list(range(64)) and (parents == 0).all() and (best == best[0, 0]).all()
    x[37, 100] = 2.0 ** -20                                  # 2^-20 (1 - 1 / 40001) above, below a step of 13.6 in fp32
    best, tokens, parents = qmm.beam_select(x, scores, 64)
    assert (int(parents[0, 0]), int(tokens[0, 0])) == (37, 100)
    assert tokens[0, 1:].tolist() == list(range(63)) and (parents[0, 1:] == 0).all()
