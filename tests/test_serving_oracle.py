"""The serving operators' oracle against closed forms and against the
decode oracle (CPU)."""

import math

import numpy as np
import pytest

from bit_kv_cache_04_gb300 import workloads as W
from oracle import kvq_oracle as O
from oracle import serving_oracle as S
from tests.helpers import oracle_cfg, raw16


def _filled(name, **shape):
    w = W.make(name).scaled(**shape)
    oc = oracle_cfg(w.cfg)
    bufs = O.new_buffers(oc)
    table = W.page_table(w)
    table = None if table is None else table.numpy()
    ks, vs, cu = W.layer_batch(w, 0, [0] * oc.batch, w.lengths)
    O.append(oc, bufs, 0, raw16(ks), raw16(vs), w.lengths, [0] * oc.batch, block_table=table)
    return w, oc, bufs, table


@pytest.mark.parametrize("name", ["llama2_7b_kivi4", "gqa8b_hadamard4_paged", "mistral7b_hotcold"])
def test_one_token_over_everything_is_decode(name):
    w, oc, bufs, table = _filled(name, L=1, lengths=[200, 45], extra=0)
    q = raw16(W.queries(w, 1))
    want = O.decode_attention(oc, bufs, 0, 1, q, w.lengths, block_table=table)[0]
    got = S.chunk_attention(oc, bufs, 0, q[0], [0, 1, 2], w.lengths, block_table=table)
    assert np.max(np.abs(got - want)) < 1e-12
    wide = S.chunk_attention(oc, bufs, 0, q[0], [0, 1, 2], w.lengths, window=200, sinks=3, block_table=table)
    assert np.max(np.abs(wide - want)) < 1e-12


def test_window_of_one_returns_the_tokens_own_value():
    w, oc, bufs, _ = _filled("llama2_7b_kivi4", L=1, lengths=[70], extra=0)
    rng = np.random.default_rng(0)
    q = rng.standard_normal((5, oc.H_q, oc.D)).astype(np.float16).view(np.uint16)
    got = S.chunk_attention(oc, bufs, 0, q, [0, 5], [70], window=1)
    _, V = O.dequantize(oc, bufs, 0, 0, 70)
    assert np.max(np.abs(got - np.repeat(V[65:70], oc.H_q // oc.H_kv, 1))) < 1e-12


def test_visible_tokens():
    assert S.visible(5, 8, 0, 0).tolist() == [True] * 6 + [False] * 2
    assert S.visible(5, 8, 2, 0).tolist() == [False] * 4 + [True] * 2 + [False] * 2
    assert S.visible(5, 8, 2, 1).tolist() == [True] + [False] * 3 + [True] * 2 + [False] * 2
    assert S.visible(1, 8, 2, 5).tolist() == [True] * 2 + [False] * 6  # a sink ahead of the query stays hidden


def test_turn_keeps_relative_positions_and_norms():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 128)), rng.standard_normal((1, 1, 128))
    for inter in (False, True):
        f, m = S.rope_frequencies(96, 1e4)
        dots = [np.sum(S.turn(q, [a], f, m, inter) * S.turn(k, [a - 7], f, m, inter)) for a in (7, 1000, 123456)]
        assert np.ptp(dots) < 1e-9
        y = S.turn(q, [99], f, m, inter)
        assert abs(np.linalg.norm(y) - np.linalg.norm(q)) < 1e-12
        assert np.array_equal(y[..., 96:], q[..., 96:])


def test_frequency_scalings():
    f0, m0 = S.rope_frequencies(64, 1e4)
    assert m0 == 1.0 and f0[0] == 1.0
    assert np.allclose(S.rope_frequencies(64, 1e4, S.ROPE_LINEAR, 4.0)[0], f0 / 4)
    fn = S.rope_frequencies(64, 1e4, S.ROPE_NTK, 4.0)[0]
    assert fn[0] == 1.0 and abs(fn[-1] * 4 / f0[-1] - 1) < 1e-12  # the slowest pair is slowed by the factor
    fy, my = S.rope_frequencies(64, 1e4, S.ROPE_YARN, 4.0, 1.0, 32.0, 4096)
    assert fy[0] == f0[0] and np.isclose(fy[-1], f0[-1] / 4) and abs(my - (1 + 0.1 * math.log(4))) < 1e-15
    fb = S.rope_frequencies(64, 1e4, S.ROPE_BANDS, 8.0, 1.0, 4.0, 8192)[0]
    turns = 8192 * f0 / (2 * math.pi)
    assert np.allclose(fb[turns >= 4], f0[turns >= 4]) and np.allclose(fb[turns <= 1], f0[turns <= 1] / 8)
    assert np.all(np.diff(fb) <= 0)


def test_rms_norm():
    x = np.full((2, 128), 3.0)
    assert np.allclose(S.rms_norm(x, np.arange(128.0), 0.0), np.arange(128.0))


def test_pages_share_copy_and_compact():
    pool = np.arange(8)[None, :, None] * np.ones((2, 8, 3))
    m = S.Pages([[5, 2, -1], [-1, -1, -1], [-1, -1, -1]], 8, 16, 48, pools=[pool])
    m.lens[0] = 20
    m.fork([0, 0], [1, 2])
    assert m.refs.tolist() == [0, 0, 3, 0, 0, 3, 0, 0]
    m.reserve([0, 1, 2], [1, 13, 1])  # page 2 is half full: two copies, the last reader keeps it
    assert m.table.tolist() == [[5, 0, -1], [5, 1, 3], [5, 2, -1]]
    assert pool[0, :4, 0].tolist() == [2, 2, 2, 3] and m.refs.tolist() == [1, 1, 1, 1, 0, 3, 0, 0]
    m.release([1, 1])
    assert m.refs.tolist() == [1, 0, 1, 0, 0, 2, 0, 0]
    m.compact()
    assert m.table.tolist() == [[1, 0, -1], [-1, -1, -1], [1, 2, -1]] and pool[1, 1, 0] == 5
    assert m.refs.tolist() == [1, 2, 1, 0, 0, 0, 0, 0]
