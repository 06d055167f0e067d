"""Arguments that the attention over shared prefixes refuses on the host (CPU: the pointers below are never read)."""

import ctypes

import pytest

K = pytest.importorskip("bit_kv_cache_04_gb300.kvq")
from tests.test_serving_refusals import PAGED, A, _cache, _cfg, _refused  # noqa: E402

BIG = 1 << 40


def _plan(cfg=None, table=A, groups=A, n=2, cu=A, total=4, most=2, most_group=3, lens=A, ws=A, nbytes=BIG):
    cfg = _cfg(**PAGED) if cfg is None else cfg
    return K.LIB.kvq_prefix_plan(ctypes.byref(K._to_c(cfg)), table, groups, n, cu, total, most, most_group, lens, ws, nbytes, None)


def _attend(cfg=None, cache=None, layer0=0, layers=1, n=2, q=A, total=4, most=2, most_group=3, out=1 << 30, ws=A, nbytes=BIG):
    cfg = _cfg(**PAGED) if cfg is None else cfg
    return K.LIB.kvq_prefix_attention(ctypes.byref(K._to_c(cfg)), cache or _cache(cfg), layer0, layers, n, q, total, most, most_group,
                                      out, ws, nbytes, None)


SIZES = [(dict(n=0), 1), (dict(n=4), 1), (dict(total=-1), 1), (dict(most=-1), 1), (dict(most=4), 1), (dict(most_group=5), 1),
         (dict(most=65, most_group=65, total=100), 4), (dict(ws=None), 5), (dict(ws=A + 16), 5), (dict(nbytes=1000), 5)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(cfg=_cfg()), 1), (dict(cfg=_cfg(D=64)), 2), (dict(table=None), 1), (dict(groups=None), 1), (dict(cu=None), 1),
    (dict(lens=None), 1), (dict(table=A + 2), 1), (dict(groups=A + 1), 1), (dict(cu=A + 2), 1), (dict(lens=A + 3), 1),
])
def test_plan_refusals(kw, status):
    assert _plan(**kw) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(cfg=_cfg()), 1), (dict(layer0=-1), 1), (dict(layer0=2), 1), (dict(layers=3), 1), (dict(layers=0), 1), (dict(q=None), 1),
    (dict(out=None), 1), (dict(q=A + 8), 1), (dict(out=(1 << 30) + 2), 1), (dict(out=A), 1), (dict(out=A + 256), 1),
])
def test_attention_refusals(kw, status):
    assert _attend(**kw) == status


def test_what_the_cache_lacks():
    cfg = _cfg(**PAGED, residual_window=8)
    for bad in (dict(k_main=None), dict(v_main=A + 8), dict(k_resid=None), dict(block_table=None)):
        assert _attend(cfg=cfg, cache=_cache(cfg, **bad)) == 1


def test_no_rows_are_nothing_to_do():
    assert _attend(total=0, most=0, most_group=0, q=None, out=None) == 0
    assert _attend(total=4, most=0, most_group=0) == 0


def test_workspace():
    cfg = _cfg(**PAGED)
    c, out = ctypes.byref(K._to_c(cfg)), ctypes.c_size_t()
    assert K.LIB.kvq_prefix_workspace_bytes(c, 2, 4, None) == 1
    assert K.LIB.kvq_prefix_workspace_bytes(c, 0, 4, ctypes.byref(out)) == 1
    assert K.LIB.kvq_prefix_workspace_bytes(c, 2, -1, ctypes.byref(out)) == 1
    assert K.LIB.kvq_prefix_workspace_bytes(ctypes.byref(K._to_c(_cfg())), 2, 4, ctypes.byref(out)) == 1
    huge = _cfg(page_tokens=16, n_pages=20, max_pages_per_seq=1 << 22, max_T=1 << 26, batch=4096)
    assert K.LIB.kvq_prefix_workspace_bytes(ctypes.byref(K._to_c(huge)), 2, 4, ctypes.byref(out)) == 2
    n = K.kvq_prefix_workspace_bytes(cfg, 2, 4)
    assert n > K.kvq_chunk_workspace_bytes(cfg) and n < K.kvq_prefix_workspace_bytes(cfg, 2, 4000)
    _refused(K.LIB.kvq_prefix_workspace_init, (c, 2, 4, A, n - 1, None), 5)
    _refused(K.LIB.kvq_prefix_workspace_init, (c, 2, 4, None, n, None), 5)
    assert _plan(nbytes=n - 1) == 5 and _attend(nbytes=n - 1) == 5


def test_wrapper_refuses_other_tensors():
    torch = pytest.importorskip("torch")
    cfg = _cfg(**PAGED)
    c = K.KVCache.__new__(K.KVCache)  # the checks come before any device work
    c.cfg, c.index, c.block_table = cfg, -1, torch.zeros((3, 4), dtype=torch.int32)
    p = K.PrefixAttention.__new__(K.PrefixAttention)
    p.cache, p.index, p.groups, p.planned = c, -1, 2, None
    g, cu, lens = (torch.zeros(n, dtype=torch.int32) for n in (3, 4, 3))
    for bad in (dict(g=g[:2]), dict(g=g.long()), dict(cu=cu[:3]), dict(cu=cu.long()), dict(lens=lens[:2]), dict(lens=lens.float()),
                dict(cu=torch.zeros(8, dtype=torch.int32)[::2])):
        a = dict(g=g, cu=cu, lens=lens) | bad
        with pytest.raises(ValueError):
            p.plan(a["g"], a["cu"], 4, 2, 3, a["lens"])
    with pytest.raises(ValueError, match="must be on a GPU"):
        p.plan(g, cu, 4, 2, 3, lens)
    q = torch.zeros((1, 4, 4, 128), dtype=torch.float16)
    with pytest.raises(RuntimeError, match="plan comes before"):
        p.attention(0, 1, q, q.clone())
    p.planned = (4, 2, 3)
    for x, o in ((q.float(), q), (q, q.float()), (q[:, :3], q), (q, q[..., :64]), (q.transpose(1, 2), q)):
        with pytest.raises(ValueError):
            p.attention(0, 1, x, o)
