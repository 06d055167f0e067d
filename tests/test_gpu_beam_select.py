"""Beam selection against the definition in 64 bits: vocabularies around every vector and block size, rows
at every alignment, rows of -inf, NaN and infinities, ties, finished beams, captured and repeated calls."""

import numpy as np
import pytest

from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def outputs(G, B):
    return [torch.full((G, B), 77, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32, torch.int32)]


def bound(V, score):
    """Largest error of a score.  A term e^d, d <= 0, is off by 2^-22 (the base-2 exponential), 2^-24 |d| (the difference) and
    2 log2(e) |d| 2^-24 (the constant and the product), relative to itself; the |d| weigh with their terms, whose mean is at
    most ln V.  A thread adds at most V / 256 + 8 terms, then 13 joins follow: 2^-24 each.  The sum's relative error is the
    log's absolute one; the score is rounded once."""
    rel = 2.0 ** -22 + 4 * np.log(V + 1) * 2.0 ** -24 + (V / 256 + 21) * 2.0 ** -24
    return rel + 2.0 ** -24 * np.abs(score)


def check(logits, scores, done=None, eos=-1, sel=None):
    G, B, V = logits.shape
    out = outputs(G, B)
    sel = sel or K.BeamSelect(G, B, V)
    sel.select(logits, scores, out[0], out[1], out[2], done=done, done_out=out[3], eos=eos)
    torch.cuda.synchronize()
    got = [t.cpu().numpy() for t in out]
    x = logits.double().cpu().numpy()
    s = scores.double().cpu().numpy()
    d = None if done is None else done.cpu().numpy()
    want = S.beam_select(x, s, d, eos)
    finite = np.isfinite(want[0])
    assert np.array_equal(finite, np.isfinite(got[0]))
    assert np.all(got[0][~finite] == want[0][~finite])
    lim = bound(V, np.where(finite, want[0], 0))
    assert np.all(np.abs(np.where(finite, got[0] - want[0], 0)) <= lim)
    # beams' scores nearer than the errors may change places across beams; nothing else may
    for g in range(G):
        for i in range(B):
            if got[1][g, i] == want[1][g, i] and got[2][g, i] == want[2][g, i]:
                continue
            near = [j for j in range(B) if (got[2][g, i], got[1][g, i]) == (want[2][g, j], want[1][g, j])]
            assert near and want[2][g, near[0]] != want[2][g, i], (g, i)
            assert abs(want[0][g, near[0]] - want[0][g, i]) <= 2 * lim[g, i]
    assert np.array_equal(got[3], np.asarray([[int(t == eos or (d is not None and d[g, p])) for t, p in zip(got[1][g], got[2][g])]
                                              for g in range(G)]))
    return got


def random(G, B, V, dtype, seed=0, spread=2.5, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    x = (spread * torch.randn((G, B, V), generator=g)).to(TYPES[dtype])
    return x.to(device), (-10 - 3 * torch.rand((G, B), generator=g)).to(device)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B", [1, 2, 5, 8, 31, 32])
@pytest.mark.parametrize("V", [32, 33, 1023, 2049, 5003])
def test_sizes(dtype, B, V):
    check(*random(3, B, V, dtype, seed=V + B))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 15, 17, 31, 255, 257])
def test_small_vocabularies(dtype, V):
    for B in (1, 4, 32):
        check(*random(2, B, V, dtype, seed=V))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [8191, 32000, 50257])
def test_long_rows(dtype, V):
    check(*random(1, 3, V, dtype, seed=V))


def test_many_groups():
    check(*random(700, 2, 300, "bf16", seed=1))
    check(*random(1, 1, 300000, "fp32", seed=2))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", range(0, 9))
def test_rows_at_any_alignment(dtype, shift):
    G, B, V = 2, 3, 2100 + shift
    x, s = random(G, B, V, dtype, seed=shift)
    room = torch.full((G, B, V + 40), float("nan"), dtype=x.dtype, device="cuda")
    view = room[:, :, shift:shift + V]
    view.copy_(x)
    check(view, s)
    wide = torch.empty((B, G, V), dtype=x.dtype, device="cuda").transpose(0, 1)
    wide.copy_(x)
    check(wide, s)


@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_not_numbers(dtype):
    G, B, V = 6, 4, 3001
    x, s = random(G, B, V, dtype, seed=3)
    lowest = torch.finfo(x.dtype).min
    x[0, 1] = -float("inf")                # a beam that has nothing to go on with
    x[1] = -float("inf")                   # a whole group
    x[2, 0, ::3] = float("nan")
    x[2, 1, 5] = float("inf")
    x[2, 2, :] = float("nan")
    x[3, :, 100:] = lowest                 # masked by the type's lowest value
    x[3, 2, :] = lowest
    x[4, :, 3:] = -float("inf")            # fewer candidates than beams: 4 x 3 here, then fewer
    x[5, :, 1:] = -float("inf")
    x[5, 2:, :] = -float("inf")
    s[5, 1] = -float("inf")
    s[0, 2] = float("nan")
    check(x, s)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_go_to_the_lowest_place(dtype):
    x = torch.zeros((3, 4, 4099), dtype=TYPES[dtype], device="cuda")
    s = torch.zeros((3, 4), device="cuda")
    s[1, 1:] = -float("inf")  # a new search: one live beam
    x[2] = torch.randint(0, 3, (1, 4099), device="cuda").to(x.dtype)  # the same row for every beam
    got = check(x, s)
    assert got[1][0].tolist() == [0, 1, 2, 3] and got[2][0].tolist() == [0, 0, 0, 0]
    assert got[1][1].tolist() == [0, 1, 2, 3] and got[2][1].tolist() == [0, 0, 0, 0]
    first = torch.nonzero(x[2, 0] == 2)[:4, 0].tolist()
    assert got[1][2].tolist() == first and got[2][2].tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("dtype", TYPES)
def test_zeros_of_both_signs(dtype):
    x = torch.full((1, 3, 900), -1.0, device="cuda")
    x[0, :, 100:140:2], x[0, :, 101:140:2] = 0.0, -0.0
    s = torch.tensor([[0.0, -0.0, 0.0]], device="cuda")
    got = check(x.to(TYPES[dtype]), s)
    assert got[1].tolist() == [[100, 101, 102]] and got[2].tolist() == [[0, 0, 0]]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B", [4, 32])
def test_many_infinities_and_few_tokens_left(dtype, B):
    """Every lane holds a value past the finite ones; and rows of which hardly anything may follow."""
    x, s = random(3, B, 9000, dtype, seed=B)
    x[0, 0, ::5] = float("inf")
    x[1, :, 7:] = -float("inf")
    x[2, :, :] = -float("inf")
    x[2, B // 2, 8999] = 3.0
    check(x, s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("order", ["rising", "falling", "equal"])
def test_rows_in_order(dtype, order):
    """Rising rows pass every bound; falling ones are done with the first turn; in equal ones places decide."""
    for B in (8, 32):
        x = torch.arange(20000, device="cuda").float() / 2000 - 5
        x = x.flip(0) if order == "falling" else x * 0 if order == "equal" else x
        x = x.to(TYPES[dtype]).expand(2, B, 20000).contiguous()
        check(x, torch.linspace(-3, -1, 2 * B, device="cuda").view(2, B))


@pytest.mark.parametrize("dtype", TYPES)
def test_finished_beams(dtype):
    G, B, V = 4, 5, 2500
    x, s = random(G, B, V, dtype, seed=4)
    done = torch.zeros((G, B), dtype=torch.int32, device="cuda")
    done[0, 2] = 1
    done[1] = torch.tensor([1, 0, 7, -1, 0])
    done[2] = 1
    s[0, 2] += 4  # the finished ones are among the best
    s[1] += torch.tensor([4.0, 0, 4, 4, 0], device="cuda")
    x[3, 0, 17] = 40  # the end token is chosen now
    x[0, 2] = float("nan")  # what a finished beam's logits hold does not matter
    got = check(x, s, done, eos=17)
    assert got[3][2].tolist() == [1] * 5 and got[1][2].tolist() == [17] * 5 and got[3][3, 0] == 1
    # in place
    sel = K.BeamSelect(G, B, V)
    s2, d2, tok, par = s.clone(), done.clone(), *outputs(G, B)[1:3]
    sel.select(x, s2, s2, tok, par, done=d2, done_out=d2, eos=17)
    torch.cuda.synchronize()
    assert np.array_equal(s2.cpu(), got[0]) and np.array_equal(d2.cpu(), got[3]) and np.array_equal(tok.cpu(), got[1])


def test_calls_in_turn_and_captured():
    G, B, V = 3, 4, 9001
    sel = K.BeamSelect(G, B, V)
    for seed in range(3):  # the workspace serves every call
        check(*random(G, B, V, "fp16", seed=seed), sel=sel)
    x, s = random(G, B, V, "fp16", seed=9)
    out = outputs(G, B)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sel.select(x, s, *out[:3])
    for seed in range(10, 13):
        y, t = random(G, B, V, "fp16", seed=seed)
        x.copy_(y), s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        want = check(y, t)
        assert all(np.array_equal(a.cpu(), b) for a, b in zip(out[:3], want))
    side = torch.cuda.Stream()
    other = K.BeamSelect(G, B, V, stream=side)
    side.wait_stream(torch.cuda.current_stream())
    more = outputs(G, B)
    torch.cuda.synchronize()
    for _ in range(20):  # two at once, a workspace each
        sel.select(x, s, *out[:3])
        other.select(x, s, *more[:3], stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out[:3], more[:3]))


def test_the_same_call_gives_the_same_bits():
    x, s = random(2, 8, 40001, "bf16", seed=5)
    sel, first = K.BeamSelect(2, 8, 40001), None
    for _ in range(5):
        out = outputs(2, 8)
        sel.select(x, s, *out[:3])
        torch.cuda.synchronize()
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(out, first))


@pytest.mark.parametrize("beams,vocab", [(32, 500), (32, 40000), (20, 9000), (17, 300)])
@pytest.mark.parametrize("value", [0.0, -float("inf"), 1.5])
def test_more_equal_candidates_than_are_ranked_at_once(beams, vocab, value):
    """Beams without a difference: every candidate at the bound, the lowest tokens of the first beam."""
    logits = torch.full((3, beams, vocab), value, device="cuda").to(torch.bfloat16)
    scores = torch.zeros((3, beams), device="cuda")
    logits[1, 0, vocab - 1] = 2.0  # one above the others
    scores[2, 1] = 0.25
    sel = K.BeamSelect(3, beams, vocab)
    for _ in range(2):
        got = check(logits, scores, sel=sel)
    if value == 0:
        assert got[1][0].tolist() == list(range(beams)) and not got[2][0].any()


@pytest.mark.parametrize("near", [1e-3, 1.0, 30.0])
def test_beams_apart_and_together(near):
    """Of 32 beams' 1024 candidates those that come through the bound: all from one beam, some of each, nearly all."""
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn((4, 32, 2000), generator=g, device="cuda")
    scores = -near * torch.rand((4, 32), generator=g, device="cuda")
    scores[1] *= 100
    done = torch.zeros((4, 32), dtype=torch.int32, device="cuda")
    done[2, ::3] = 1
    done[3] = 1
    check(logits, scores, done, 7)
