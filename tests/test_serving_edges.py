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
