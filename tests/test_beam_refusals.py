"""Arguments that beam selection and the reordering of pages refuse on the host (CPU: the pointers below are never
read), and the selection's definition on closed cases."""

import ctypes
import math

import numpy as np
import pytest

from oracle import serving_oracle as S

K = pytest.importorskip("bit_kv_cache_04_gb300.kvq")
from tests.test_serving_refusals import PAGED, A, _cache, _cfg, _refused  # noqa: E402


def _select(logits=A, dtype=0, gs=4000, bs=1000, groups=2, beams=4, vocab=1000, scores=A, done=None, eos=-1, so=A, tok=A, par=A,
            do=None, ws=A, nbytes=1 << 40):
    return K.LIB.kvq_beam_select(logits, dtype, gs, bs, groups, beams, vocab, scores, done, eos, so, tok, par, do, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), 1), (dict(scores=None), 1), (dict(so=None), 1), (dict(tok=None), 1), (dict(par=None), 1),
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(gs=-1), 1), (dict(bs=-1), 1), (dict(groups=0), 1), (dict(beams=0), 1),
    (dict(vocab=0), 1), (dict(beams=33), 2), (dict(vocab=1 << 26), 2), (dict(groups=1 << 23), 2), (dict(eos=1000), 1),
    (dict(eos=-2), 1), (dict(done=A), 1), (dict(logits=A + 1), 1), (dict(logits=A + 2, dtype=2), 1), (dict(scores=A + 2), 1),
    (dict(tok=A + 1), 1), (dict(done=A + 2, eos=3), 1), (dict(do=A + 2), 1), (dict(ws=None), 5), (dict(ws=A + 16), 5),
    (dict(nbytes=16), 5),
])
def test_select_refusals(kw, status):
    assert _select(**kw) == status


def test_outputs_that_overlap():
    """Every output apart from the others and from the inputs, but for scores and finished beams in place."""
    at = {n: (i + 1) << 24 for i, n in enumerate(("logits", "scores", "done", "so", "tok", "par", "do"))}
    for out in ("so", "tok", "par", "do"):
        for other in at:
            if other == out or (out, other) in (("so", "scores"), ("do", "done")):
                continue
            for shift in (0, 28, -28):  # lists of 32 bytes
                if (other, shift) == ("logits", -28):
                    shift = 15000  # logits reach 2 * (4000 + 3000 + 1000) bytes
                assert _select(**{**at, out: at[other] + shift}, eos=1) == 1, (out, other)
                assert b"overlaps" in K.LIB.kvq_last_error()
    for out, other in (("so", "scores"), ("do", "done")):
        assert _select(**{**at, out: at[other] + 4}, eos=1) == 1


def test_workspace_sizes():
    out = ctypes.c_size_t()
    assert K.LIB.kvq_beam_workspace_bytes(2, 4, 1000, None) == 1
    assert K.LIB.kvq_beam_workspace_bytes(2, 33, 1000, ctypes.byref(out)) == 2
    n = K.kvq_beam_workspace_bytes(2, 4, 1000)
    _refused(K.LIB.kvq_beam_workspace_init, (2, 4, 1000, A, n - 1, None), 5)
    _refused(K.LIB.kvq_beam_workspace_init, (2, 4, 1000, None, n, None), 5)
    assert _select(nbytes=n - 1) == 5


def test_select_wrapper_refuses_other_tensors():
    torch = pytest.importorskip("torch")
    sel = K.BeamSelect.__new__(K.BeamSelect)  # the checks come before any device work
    sel.sizes, sel.index = (2, 3, 50), -1
    x, s, t = torch.zeros(2, 3, 50), torch.zeros(2, 3), torch.zeros(2, 3, dtype=torch.int32)
    for kw in (dict(logits=x.double()), dict(logits=x[:, :2]), dict(logits=x[..., :49]), dict(logits=torch.zeros(2, 3, 100)[..., ::2]),
               dict(scores=s.double()), dict(scores=s[:1]), dict(scores=torch.zeros(3, 2).t()), dict(scores_out=s.half()),
               dict(tokens=t.long()), dict(parents=t[:, :2]), dict(done=t.bool()), dict(done_out=t.long())):
        args = dict(logits=x, scores=s, scores_out=s.clone(), tokens=t, parents=t.clone(), done=None, done_out=None)
        args.update(kw)
        with pytest.raises(ValueError):
            sel.select(**args)
    with pytest.raises(ValueError, match="must be on a GPU"):
        sel.select(x, s, s.clone(), t, t.clone())


def test_reorder_refusals():
    cfg, big = _cfg(**PAGED, residual_window=8), 1 << 30
    c = ctypes.byref(K._to_c(cfg))
    call = K.LIB.kvq_pages_reorder
    n = K.kvq_pages_workspace_bytes(cfg)
    good = [c, _cache(cfg), A, A, A, A, 3, A, big, None]
    for at, value, status in ((0, ctypes.byref(K._to_c(_cfg())), 1), (1, None, 1), (1, _cache(cfg, k_main=None), 1),
                              (1, _cache(cfg, v_resid=None), 1), (2, None, 1), (3, None, 1), (4, None, 1), (5, None, 1),
                              (4, A + 2, 1), (5, A + 1, 1), (6, 0, 1), (6, -1, 1), (6, 2, 1), (6, 6, 1), (7, None, 5),
                              (7, A + 16, 5), (8, n - 1, 5)):
        args = list(good)
        args[at] = value
        _refused(call, tuple(args), status)
    many = _cfg(**{**PAGED, "batch": 66})
    _refused(call, (ctypes.byref(K._to_c(many)), _cache(many), A, A, A, A, 33, A, big, None), 2, "group")
    torch = pytest.importorskip("torch")
    pool = K.PagePool.__new__(K.PagePool)
    pool.cache, pool.index = K.KVCache.__new__(K.KVCache), -1
    pool.cache.cfg = cfg
    lens = torch.zeros(3, dtype=torch.int32)
    for parents in (lens.long(), lens[:2], torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            pool.reorder(parents, 3, lens)


def test_the_definition_on_closed_cases():
    # one beam, two tokens with odds 3 to 1
    s, t, p, d = S.beam_select(np.array([[[math.log(3.0), 0.0]]]), np.array([[-1.0]]))
    assert abs(s[0, 0] - (-1 + math.log(0.75))) < 1e-15 and t[0, 0] == 0 and p[0, 0] == 0 and d[0, 0] == 0
    # the candidates of all beams are a distribution under their scores: all of them together sum up to that of the scores
    rng = np.random.default_rng(0)
    x, sc = rng.standard_normal((1, 6, 1)), rng.standard_normal((1, 6))
    s, t, p, _ = S.beam_select(x, sc)
    assert np.allclose(np.sort(s[0]), np.sort(sc[0])) and (t == 0).all() and sorted(p[0].tolist()) == list(range(6))
    # a finished beam stays as it is
    s, t, p, d = S.beam_select(np.zeros((1, 2, 4)), np.array([[-1.0, -2.0]]), np.array([[1, 0]]), eos=3)
    assert s[0, 0] == -1 and (t[0, 0], p[0, 0], d[0, 0]) == (3, 0, 1)
    assert abs(s[0, 1] - (-2 - math.log(4))) < 1e-15 and (t[0, 1], p[0, 1], d[0, 1]) == (0, 1, 0)
    # nothing to follow
    s, t, p, _ = S.beam_select(np.full((1, 2, 3), -np.inf), np.zeros((1, 2)))
    assert (s == -np.inf).all() and t[0].tolist() == [0, 1] and p[0].tolist() == [0, 0]


def test_reorder_of_the_model():
    m = S.Pages([[0, 1], [0, 2], [3, -1], [4, -1]], 6, 16, 32)
    m.lens[:] = [20, 21, 5, 6]
    m.reorder([1, 1, 1, 0], 2)
    assert m.table.tolist() == [[0, 2], [0, 2], [4, -1], [3, -1]] and m.lens.tolist() == [21, 21, 6, 5]
    assert m.refs.tolist() == [2, 0, 2, 1, 1, 0]
    # two tokens of 16 are quantized: the page behind them is the heir's
    m = S.Pages([[0, 1], [2, 3], [4, 5]], 6, 16, 32, residual_window=10)
    m.lens[:] = 12
    m.reorder([1, 1, 1], 3)
    assert m.table.tolist() == [[2, -1], [2, 3], [2, -1]] and m.refs.tolist() == [0, 0, 3, 1, 0, 0]
    m.lens[:] = 12
    m.reorder([2, 0, 0], 3)
    assert m.table.tolist() == [[2, -1]] * 3 and m.refs.tolist() == [0, 0, 3, 0, 0, 0]
