"""Calls at the edge of what the serving entries take, on the CPU: nothing is launched here."""

import ctypes

import pytest

torch = pytest.importorskip("torch")
K = pytest.importorskip("bit_kv_cache_04_gb300.kvq")

A = 1 << 20  # an aligned address that nothing reads


def _cfg(**kw):
    base = dict(L=2, H_kv=2, H_q=4, D=128, batch=3, max_T=64, k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128))
    base.update(kw)
    return K.Config(**base)


@pytest.mark.parametrize("with_k", [False, True])
@pytest.mark.parametrize("plan", [None, 128])
def test_norm_rope_of_no_tokens_is_nothing_in_python(with_k, plan):
    """Empty tensors have no address, which the C entry takes for a missing tensor."""
    q, k = torch.zeros((0, 4, 128), dtype=torch.float16), torch.zeros((0, 2, 128), dtype=torch.float16)
    w, pos = torch.ones(128, dtype=torch.float16), torch.zeros(0, dtype=torch.int32)
    K.qk_norm_rope(_cfg(), q, k if with_k else None, pos, q.clone(), k.clone() if with_k else None,
                   plan=plan and K.rope_plan(plan), q_weight=w, k_weight=w if with_k else None, stream=0)
    with pytest.raises(ValueError):  # the checks stay
        K.qk_norm_rope(_cfg(), q, None, pos, q.float(), None, stream=0)


def test_host_tensors_are_refused():
    """Their addresses would go to a kernel."""
    q, n = torch.zeros((3, 4, 128), dtype=torch.float16), torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        K.qk_norm_rope(_cfg(), q, None, None, q.clone(), None, stream=0)
    c = K.KVCache.__new__(K.KVCache)
    c.cfg, c.index, c.chunk_workspace = _cfg(), -1, None
    with pytest.raises(ValueError, match="GPU"):
        c.chunk_attention(0, 1, q[None], torch.zeros(4, dtype=torch.int32), 3, 1, n, q[None].clone(), stream=0)
    pool = K.PagePool.__new__(K.PagePool)
    pool.cache, pool.index = c, -1
    with pytest.raises(ValueError, match="GPU"):
        pool.release(n, n)


def test_a_paged_cache_needs_its_whole_block_table(monkeypatch):
    """The page calls write the table of every sequence, and chunk attention reads it."""
    monkeypatch.setattr(K, "_here", lambda *_: None)
    cfg = _cfg(page_tokens=16, n_pages=20, max_pages_per_seq=4)
    c = K.KVCache.__new__(K.KVCache)
    c.cfg, c.c_cfg, c.index, c.device = cfg, K._to_c(cfg), -1, torch.device("cpu")
    for table in (None, torch.zeros((3, 3), dtype=torch.int32)):
        c.block_table = table
        with pytest.raises(ValueError, match="block table"):
            K.PagePool(c, stream=None)
    c.chunk_workspace, c.index = None, -1
    q, n = torch.zeros((1, 3, 4, 128), dtype=torch.float16), torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="block table"):
        c.chunk_attention(0, 1, q, torch.zeros(4, dtype=torch.int32), 3, 1, n, q.clone(), stream=0)


PAGED = dict(page_tokens=16, n_pages=20, max_pages_per_seq=4)


def _cache():
    return ctypes.byref(K._Cache(A, A, None, None, A, A, A))


def test_page_calls_count_pages_in_32_bits():
    """One reservation may ask for every page of the table: more than 2^31 - 1 wrapped, and passed for enough."""
    out = ctypes.c_size_t()
    for batch, pages, good in ((32768, 65534, True), (32768, 65535, False), (30000, 2 ** 30, False), (1, 2 ** 31 - 2, True)):
        cfg = _cfg(L=1, batch=batch, page_tokens=1, n_pages=20, max_pages_per_seq=pages)
        c = ctypes.byref(K._to_c(cfg))
        assert K.LIB.kvq_pages_workspace_bytes(c, ctypes.byref(out)) == (0 if good else 2), (batch, pages)
        if not good:
            assert K.LIB.kvq_pages_init(c, A, A, A, 1 << 40, None) == 2
            assert K.LIB.kvq_pages_release(c, A, A, A, A, 1, A, 1 << 40, None) == 2
            assert K.LIB.kvq_pages_fork(c, _cache(), A, A, A, A, A, 1, A, 1 << 40, None) == 2
            assert K.LIB.kvq_pages_reserve(c, _cache(), A, A, A, A, A, 1, A, 1 << 40, None) == 2
            assert K.LIB.kvq_pages_compact(c, _cache(), A, A, A, A, A, 1 << 40, None) == 2


def test_fork_refuses_before_it_launches():
    """The table's part was launched before the windows' grid was looked at."""
    cfg = _cfg(L=65536, H_kv=1, H_q=1, residual_window=8, **PAGED)
    n = K.kvq_pages_workspace_bytes(cfg)
    assert K.LIB.kvq_pages_fork(ctypes.byref(K._to_c(cfg)), _cache(), A, A, A, A, A, 1, A, n, None) == 2
