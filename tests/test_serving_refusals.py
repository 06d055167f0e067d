"""Arguments that the serving entries refuse on the host, with nothing
launched (CPU: the pointers below are never read), and the rotary plan's
host arithmetic."""

import ctypes

import numpy as np
import pytest

from oracle import serving_oracle as S

K = pytest.importorskip("bit_kv_cache_04_gb300.kvq")

A = 1 << 20  # an aligned address that nothing reads


def _cfg(**kw):
    base = dict(L=2, H_kv=2, H_q=4, D=128, batch=3, max_T=64, k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128))
    base.update(kw)
    return K.Config(**base)


PAGED = dict(page_tokens=16, n_pages=20, max_pages_per_seq=4)


def _refused(fn, args, status, words=""):
    st = fn(*args)
    assert st == status, (st, K.LIB.kvq_last_error())
    assert words in K.LIB.kvq_last_error().decode()


# ---- rotary plan ---------------------------------------------------------------


@pytest.mark.parametrize("scaling,kw", [
    (K.ROPE_NONE, {}), (K.ROPE_LINEAR, dict(factor=4.0)), (K.ROPE_NTK, dict(factor=4.0)),
    (K.ROPE_YARN, dict(factor=8.0, low=1.0, high=32.0, original_len=4096)),
    (K.ROPE_YARN, dict(factor=2.0, low=1.0, high=32.0, original_len=64, attn_factor=1.5)),
    (K.ROPE_BANDS, dict(factor=8.0, low=1.0, high=4.0, original_len=8192)),
])
@pytest.mark.parametrize("D,rot", [(128, 128), (256, 64), (128, 2), (256, 250)])
def test_plan_matches_the_definition(scaling, kw, D, rot):
    plan = K.rope_plan(D, rot, False, 10000.0, scaling, **kw)
    f, m = S.rope_frequencies(rot, 10000.0, scaling, **kw)
    got = np.array([t / 2.0 ** 64 for t in plan.turns[: rot // 2]]) * 2 * np.pi
    # pow and the products in between are off by a few units of 2^-53; the fraction is cut at 2^-64 turns
    assert np.all(np.abs(got - f) <= 1e-13 * f + 2.0 ** -60)
    assert plan.scale == np.float32(m)
    assert list(plan.turns[rot // 2:]) == [0] * (128 - rot // 2)


@pytest.mark.parametrize("kw", [
    dict(D=64), dict(rot_dim=0), dict(rot_dim=130), dict(rot_dim=33), dict(theta=1.0), dict(theta=float("nan")),
    dict(theta=float("inf")), dict(scaling=5), dict(scaling=-1), dict(scaling=K.ROPE_LINEAR, factor=0.5),
    dict(scaling=K.ROPE_NTK, factor=float("nan")), dict(scaling=K.ROPE_YARN, factor=2.0),
    dict(scaling=K.ROPE_BANDS, factor=2.0, original_len=64, low=4.0, high=4.0),
    dict(scaling=K.ROPE_BANDS, factor=2.0, original_len=64, low=0.0), dict(attn_factor=-1.0),
    dict(attn_factor=float("nan")), dict(interleaved=2),
])
def test_plan_refusals(kw):
    args = dict(D=128)
    args.update(kw)
    with pytest.raises(K.KvqError):
        K.rope_plan(**args)


# ---- norm and turn -----------------------------------------------------------------


def _nr(cfg=None, plan="own", q=A, qs=(512, 128), k=A, ks=(256, 128), qw=None, kw=None, eps=1e-6, pos=A, n=3, qo=2 * A,
        ko=2 * A):
    cfg = _cfg() if cfg is None else cfg
    if isinstance(plan, str):
        plan = K.rope_plan(cfg.D if cfg.D in (128, 256) else 128)
    return K.LIB.kvq_qk_norm_rope(ctypes.byref(K._to_c(cfg)), None if plan is None else ctypes.byref(plan), q, *qs, k,
                                  *ks, qw, kw, eps, pos, n, qo, ko, None)


@pytest.mark.parametrize("kw,status", [
    (dict(cfg=_cfg(D=64)), 2), (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(ko=None), 1),
    (dict(q=None, qo=None, k=None, ko=None), 1), (dict(q=None, qo=None, qw=A), 1), (dict(n=-1), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(pos=None), 1),
    (dict(pos=A + 2), 1), (dict(q=A + 1), 1), (dict(ko=2 * A + 1), 1), (dict(qw=A + 1), 1), (dict(qs=(-1, 128)), 1),
    (dict(ks=(256, -128)), 1), (dict(q=A, qo=A, qs=(1024, 128)), 1), (dict(k=A, ko=A, ks=(256, 64)), 1),
    (dict(plan=K.rope_plan(256)), 1),
])
def test_norm_rope_refusals(kw, status):
    assert _nr(**kw) == status


def test_norm_rope_of_no_tokens_is_nothing():
    assert _nr(n=0) == 0
    assert _nr(n=0, plan=None, pos=None) == 0


def test_norm_rope_wrapper_refuses_other_layouts():
    torch = pytest.importorskip("torch")
    x, pos = torch.zeros((2, 4, 128), dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    for q, o in ((x[:, :, ::2], x), (x, x[:1]), (x.transpose(0, 1), x.transpose(0, 1)), (x[0], x[0]),
                 (x.float(), x), (x, x.float())):
        with pytest.raises(ValueError):
            K.qk_norm_rope(_cfg(), q, None, pos, o, None)
    with pytest.raises(ValueError):
        K.qk_norm_rope(_cfg(), x[:, :3], None, pos, x[:, :3].contiguous(), None)
    with pytest.raises(ValueError):
        K.qk_norm_rope(_cfg(), x, None, pos[:1], x.clone(), None, plan=K.rope_plan(128))
    with pytest.raises(ValueError):
        K.qk_norm_rope(_cfg(), x, None, pos.long(), x.clone(), None, plan=K.rope_plan(128))


# ---- pages ---------------------------------------------------------------------------


def _cache(cfg, **kw):
    f = dict(k_main=A, v_main=A, k_cold=None, v_cold=None, k_resid=A, v_resid=A, block_table=A)
    f.update(kw)
    return ctypes.byref(K._Cache(*[f[n] for n in (*K.BUFFER_NAMES, "block_table")]))


def test_pages_refusals():
    cfg, big = _cfg(**PAGED), 1 << 30
    c = ctypes.byref(K._to_c(cfg))
    L = K.LIB
    n = K.kvq_pages_workspace_bytes(cfg)
    plain = ctypes.byref(K._to_c(_cfg()))
    out = ctypes.c_size_t()
    assert L.kvq_pages_workspace_bytes(plain, ctypes.byref(out)) == 1
    assert L.kvq_pages_workspace_bytes(c, None) == 1
    assert L.kvq_pages_workspace_bytes(ctypes.byref(K._to_c(_cfg(**PAGED, batch=40000))), ctypes.byref(out)) == 2
    _refused(L.kvq_pages_init, (plain, A, A, A, big, None), 1, "not paged")
    for t, r, w, b, st in ((None, A, A, big, 1), (A, None, A, big, 1), (A + 2, A, A, big, 1), (A, A, None, big, 5),
                           (A, A, A, n - 1, 5), (A, A, A + 16, big, 5)):
        _refused(L.kvq_pages_init, (c, t, r, w, b, None), st)
        _refused(L.kvq_pages_release, (c, t, r, A, A, 1, w, b, None), st)
        _refused(L.kvq_pages_fork, (c, _cache(cfg), t, r, A, A, A, 1, w, b, None), st)
        _refused(L.kvq_pages_reserve, (c, _cache(cfg), t, r, A, A, A, 1, w, b, None), st)
        _refused(L.kvq_pages_compact, (c, _cache(cfg), t, r, A, A, w, b, None), st)
    for lens, l1, l2, k in ((None, A, A, 1), (A, None, A, 1), (A, A, None, 1), (A, A, A, -1), (A, A, A, 4),
                            (A + 1, A, A, 1), (A, A + 2, A, 1)):
        if l2 is not None:
            _refused(L.kvq_pages_release, (c, A, A, lens, l1, k, A, big, None), 1)
        _refused(L.kvq_pages_fork, (c, _cache(cfg), A, A, lens, l1, l2, k, A, big, None), 1)
        _refused(L.kvq_pages_reserve, (c, _cache(cfg), A, A, lens, l1, l2, k, A, big, None), 1)
    for bad in (dict(k_main=None), dict(v_main=A + 8)):
        _refused(L.kvq_pages_fork, (c, _cache(cfg, **bad), A, A, A, A, A, 1, A, big, None), 1)
        _refused(L.kvq_pages_compact, (c, _cache(cfg, **bad), A, A, A, A, A, big, None), 1)
    _refused(L.kvq_pages_fork, (c, None, A, A, A, A, A, 1, A, big, None), 1)
    ring = ctypes.byref(K._to_c(_cfg(**PAGED, residual_window=8)))
    _refused(L.kvq_pages_fork, (ring, _cache(cfg, k_resid=None), A, A, A, A, A, 1, A, big, None), 1)
    for t, r in ((None, A), (A, None), (A + 1, A)):
        _refused(L.kvq_pages_compact, (c, _cache(cfg), A, A, t, r, A, big, None), 1)
    # empty lists are nothing to do
    assert L.kvq_pages_release(c, A, A, A, None, 0, A, big, None) == 0
    assert L.kvq_pages_fork(c, _cache(cfg), A, A, A, None, None, 0, A, big, None) == 0
    assert L.kvq_pages_reserve(c, _cache(cfg), A, A, A, None, None, 0, A, big, None) == 0


# ---- chunk attention -------------------------------------------------------------------


def _ca(cfg=None, cache=None, layer0=0, n_layers=1, q=A, cu=A, total=4, most=2, lens=A, window=0, sinks=0, out=2 * A, ws=A,
        nbytes=1 << 40):
    cfg = _cfg() if cfg is None else cfg
    return K.LIB.kvq_chunk_attention(ctypes.byref(K._to_c(cfg)), cache or _cache(cfg), layer0, n_layers, q, cu, total, most,
                                     lens, window, sinks, out, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(cfg=_cfg(D=64)), 2), (dict(layer0=-1), 1), (dict(n_layers=3), 1), (dict(layer0=2), 1), (dict(n_layers=0), 1),
    (dict(layer0=1, n_layers=2 ** 31 - 1), 1), (dict(q=None), 1), (dict(cu=None), 1), (dict(lens=None), 1),
    (dict(out=None), 1), (dict(total=-1), 1), (dict(most=5), 1), (dict(most=-1), 1), (dict(total=100, most=65), 4),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(q=A + 8), 1), (dict(out=2 * A + 2), 1), (dict(ws=None), 5),
    (dict(ws=A + 16), 5), (dict(nbytes=16), 5), (dict(cu=A + 2), 1), (dict(lens=A + 1), 1), (dict(out=A), 1), (dict(out=A + 256), 1),
])
def test_chunk_attention_refusals(kw, status):
    assert _ca(**kw) == status


def test_chunk_attention_of_no_rows_is_nothing():
    assert _ca(total=0, most=0, q=None, out=None) == 0
    assert _ca(total=4, most=0) == 0


def test_chunk_attention_needs_its_cache():
    cfg = _cfg()
    assert _ca(cache=_cache(cfg, k_main=None)) == 1
    assert _ca(cfg=_cfg(residual_window=4), cache=_cache(cfg, v_resid=None)) == 1
    assert _ca(cfg=_cfg(**PAGED), cache=_cache(cfg, block_table=None)) == 1
    out = ctypes.c_size_t()
    assert K.LIB.kvq_chunk_workspace_bytes(ctypes.byref(K._to_c(cfg)), None) == 1
    assert K.LIB.kvq_chunk_workspace_bytes(ctypes.byref(K._to_c(cfg)), ctypes.byref(out)) == 0
    assert K.LIB.kvq_chunk_workspace_init(ctypes.byref(K._to_c(cfg)), None, out.value, None) == 5
    assert K.LIB.kvq_chunk_workspace_init(ctypes.byref(K._to_c(cfg)), A, out.value - 1, None) == 5


def test_chunk_attention_wrapper_refuses_other_tensors():
    torch = pytest.importorskip("torch")
    cfg = _cfg()
    c = K.KVCache.__new__(K.KVCache)  # the checks come before any device work
    c.cfg, c.device = cfg, torch.device("cpu")
    q, lens = torch.zeros((1, 4, 4, 128), dtype=torch.float16), torch.ones(3, dtype=torch.int32)
    cu = torch.zeros(4, dtype=torch.int32)
    for kw in (dict(q=q.float()), dict(out=q.float()), dict(q=q[:, :3]), dict(q=q[..., :64]), dict(cu_q=cu[:3]),
               dict(cu_q=cu.long()), dict(seq_lens=lens[:2]), dict(seq_lens=lens.long()), dict(q=q.transpose(1, 2)),
               dict(n_layers=2)):
        args = dict(n_layers=1, q=q, cu_q=cu, seq_lens=lens, out=q.clone())
        args.update(kw)
        with pytest.raises(ValueError):
            c.chunk_attention(0, args["n_layers"], args["q"], args["cu_q"], 4, 2, args["seq_lens"], args["out"])


def test_tensors_of_another_device(monkeypatch):
    torch = pytest.importorskip("torch")

    class There(torch.Tensor):  # a host tensor that says it is on device 1
        def get_device(self):
            return 1

    def there(t):
        return t.as_subclass(There)

    cfg = _cfg(**PAGED)
    c = K.KVCache.__new__(K.KVCache)
    c.cfg, c.index, c.chunk_workspace = cfg, -1, torch.empty(1)
    q, n = torch.empty(1, 3, 4, 128, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    cu = torch.zeros(4, dtype=torch.int32)
    for args in ((there(q), cu, 3, 1, n, q), (q, there(cu), 3, 1, n, q), (q, cu, 3, 1, there(n), q), (q, cu, 3, 1, n, there(q))):
        with pytest.raises(ValueError, match="not on device"):
            c.chunk_attention(0, 1, *args)
    with pytest.raises(ValueError, match="not on device"):
        K.qk_norm_rope(cfg, q[0], None, None, there(q[0]), None)
    pool = K.PagePool.__new__(K.PagePool)
    pool.cache, pool.index = c, -1
    with pytest.raises(ValueError, match="not on device"):
        pool.release(there(n), n)
    # all on one device, but not the current one
    monkeypatch.setattr(K, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="not the current"):
        K.qk_norm_rope(cfg, there(q[0]), None, None, there(q[0]), None)


def test_buffers_of_the_caller():
    torch = pytest.importorskip("torch")
    cfg = _cfg(**PAGED)
    sizes = dict(zip(K.BUFFER_NAMES, K.kvq_buffer_sizes(cfg)))
    full = {k: torch.empty(v, dtype=torch.uint8) for k, v in sizes.items() if v}
    for table in (None, torch.zeros(cfg.batch, cfg.max_pages_per_seq - 1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="block table"):
            K.KVCache.from_buffers(cfg, full, table)
    with pytest.raises(ValueError, match="needed"):
        K.KVCache.from_buffers(cfg, {**full, "k_main": full["k_main"][1:]}, torch.zeros(12, dtype=torch.int32))
    with pytest.raises(ValueError, match="one device"):
        K.KVCache.from_buffers(cfg, {**full, "v_main": full["v_main"].to("meta")}, torch.zeros(12, dtype=torch.int32))
