"""The serving operators as one program uses them: a prompt's projection goes
through norm and turn, into reserved pages by kvq_append, and its chunk attends; the
prompt is forked into samples that decode on their own; the pool is compacted between steps.
Every sample must read what it would read from a cache of its own."""

import pytest

from oracle import kvq_oracle as O
from oracle import serving_oracle as S
from tests.helpers import oracle_cfg, raw16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import numpy as np  # noqa: E402

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402


@pytest.mark.parametrize("R,pt,window,sinks", [(0, 16, 0, 0), (20, 16, 48, 4), (0, 8, 30, 1)])
def test_prompt_then_samples(R, pt, window, sinks):
    L, H, g, D, B, max_T = 2, 2, 4, 128, 5, 160
    pages = 60
    cfg = K.Config(L=L, H_kv=H, H_q=H * g, D=D, batch=B, max_T=max_T, k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128),
                   flags=K.ROTATE_K | K.ROTATE_V, sign_seed=7, residual_window=R, page_tokens=pt, n_pages=pages,
                   max_pages_per_seq=-(-max_T // pt))
    table = torch.full((B, cfg.max_pages_per_seq), -1, dtype=torch.int32, device="cuda")
    cache = K.KVCache(cfg, "cuda", block_table=table)
    pool, plan = K.PagePool(cache), K.rope_plan(D, theta=10000.0)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = torch.ones(D, dtype=torch.float16, device="cuda")
    own = [[[] for _ in range(B)] for _ in range(L)]  # per layer and sequence: the k, v it has appended
    oc = oracle_cfg(cfg)
    oc = O.Config(**{**oc.__dict__, "page_tokens": 0, "n_pages": 0, "max_pages_per_seq": 0})

    def step(n_new):
        """n_new[b] tokens of every sequence: project, norm and turn, reserve, append, attend, check."""
        live = [b for b in range(B) if n_new[b]]
        total = sum(n_new)
        cu = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
        cu_d = torch.as_tensor(cu, device="cuda")
        start = lens.tolist()
        pos = torch.cat([torch.arange(start[b], start[b] + n_new[b]) for b in live]).to(torch.int32).cuda()
        pool.reserve(torch.tensor(live, dtype=torch.int32, device="cuda"),
                     torch.tensor([n_new[b] for b in live], dtype=torch.int32, device="cuda"), lens)
        q = torch.empty((L, total, H * g, D), dtype=torch.float16, device="cuda")
        k, v = (torch.empty((L, total, H, D), dtype=torch.float16, device="cuda") for _ in range(2))
        for l in range(L):
            qkv = torch.randn((total, (H * g + 2 * H) * D), generator=gen, device="cuda").half()
            K.qk_norm_rope(cfg, qkv[:, :H * g * D].unflatten(1, (H * g, D)), qkv[:, H * g * D:(H * g + H) * D].unflatten(1, (H, D)),
                           pos, q[l], k[l], plan=plan, q_weight=w, k_weight=w)
            v[l].copy_(qkv[:, (H * g + H) * D:].unflatten(1, (H, D)))
        cache.append(0, L, k, v, cu_d, lens, total, max(n_new))
        cache.commit_lengths(cu_d, lens)
        out = torch.empty_like(q)
        cache.chunk_attention(0, L, q, cu_d, total, max(n_new), lens, out, window, sinks)
        torch.cuda.synchronize()
        assert cache.device_status() == 0 and pool.device_status() == 0
        assert cache.chunk_workspace[:4].view(torch.int32).item() == 0
        for l in range(L):
            for b in live:
                own[l][b].append((raw16(k[l, cu[b]:cu[b + 1]]), raw16(v[l, cu[b]:cu[b + 1]])))
            bufs = O.new_buffers(oc)  # contiguous: every sequence its own tokens
            ks = [np.concatenate([x[0] for x in own[l][b]]) if own[l][b] else np.zeros((0, H, D), np.uint16) for b in range(B)]
            vs = [np.concatenate([x[1] for x in own[l][b]]) if own[l][b] else np.zeros((0, H, D), np.uint16) for b in range(B)]
            n = [len(x) for x in ks]
            O.append(oc, bufs, 0, np.concatenate(ks), np.concatenate(vs), n, [0] * B)
            want, bound = S.chunk_attention(oc, bufs, 0, raw16(q[l]), cu, n, window, sinks, None, True)
            err = np.abs(O.input_to_f32(raw16(out[l]), 0) - want)
            # the rotated append may differ from the oracle by one code in 1e-4 values: one step of a block's scale there
            assert np.mean(err <= bound) >= 0.999 and np.max(err) <= np.max(bound) + 0.1

    step([50, 0, 0, 0, 0])
    pool.fork(*(torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 0, 0], [1, 2, 4])), lens)
    for l in range(L):
        for b in (1, 2, 4):
            own[l][b] = list(own[l][0])
    for _ in range(3):
        step([1, 1, 1, 0, 1])
    pool.compact()
    step([3, 1, 2, 37, 1])
    pool.release(torch.tensor([1, 2], dtype=torch.int32, device="cuda"), lens)
    for l in range(L):
        own[l][1], own[l][2] = [], []
    pool.compact()
    pool.fork(torch.tensor([4], dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda"), lens)
    for l in range(L):
        own[l][2] = list(own[l][4])
    step([1, 12, 1, 1, 1])
    refs = torch.bincount(table[table >= 0].long(), minlength=pages)
    assert torch.equal(refs.int(), pool.refs)
