"""Calls at the edge of what the serving entries take."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402


@pytest.mark.parametrize("n,heads,kv", [(1, 4, 2), (1, 1, 1), (5, 1, 1), (1, 8, 1)])
def test_norm_rope_in_place_of_contiguous_views(n, heads, kv):
    """A view is contiguous whatever the strides of its dimensions of one element."""
    cfg = K.Config(L=1, H_kv=kv, H_q=heads, D=128, batch=1, max_T=64, k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128))
    gen = torch.Generator(device="cuda").manual_seed(1)
    plan, pos = K.rope_plan(128), torch.arange(7, 7 + n, dtype=torch.int32, device="cuda")
    w = torch.randn(128, generator=gen, device="cuda").half()

    def view(h):
        if n == 1:  # one token of a fused projection
            return torch.randn((1, 3 * h + 1, 128), generator=gen, device="cuda").half()[:, :h]
        x = torch.randn((n, h, 128), generator=gen, device="cuda").half()  # one head: its stride is anything
        return x.as_strided(x.shape, (h * 128, 999, 1))

    q, k = view(heads), view(kv)
    assert q.is_contiguous() and k.is_contiguous()
    qo, ko = torch.empty((n, heads, 128), dtype=q.dtype, device="cuda"), torch.empty((n, kv, 128), dtype=q.dtype, device="cuda")
    K.qk_norm_rope(cfg, q.clone(), k.clone(), pos, qo, ko, plan=plan, q_weight=w, k_weight=w)
    K.qk_norm_rope(cfg, q, k, pos, q, k, plan=plan, q_weight=w, k_weight=w)
    assert torch.equal(q, qo) and torch.equal(k, ko)


FORMS = [("few", 4, 128, 5), ("lanes", 4, 128, 20), ("paired", 4, 128, 150), ("wide", 6, 256, 40), ("wide_one", 6, 256, 1)]


@pytest.mark.parametrize("form,g,D,n", FORMS, ids=[f[0] for f in FORMS])
@pytest.mark.parametrize("T", [200, 700])
@pytest.mark.parametrize("flags", [0, K.ROTATE_K | K.ROTATE_V], ids=["plain", "rotated"])
def test_every_row_gets_the_values_that_are_not_finite_among_its_tokens(form, g, D, n, T, flags):
    """Infinities and NaN strewn over a 16-bit window of 300 tokens: what a row sees of
    them decides its channels, and all others are as if those values were zeros."""
    R, H = 300, 2
    for dt, torch_dt in ((K.DT_F16, torch.float16), (K.DT_BF16, torch.bfloat16)):
        cfg = K.Config(L=1, H_kv=H, H_q=H * g, D=D, batch=1, max_T=T, k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128), flags=flags,
                       sign_seed=3, residual_window=R, in_dtype=dt)
        cache = K.KVCache(cfg, "cuda")
        gen = torch.Generator(device="cuda").manual_seed(T + n)
        k, v = (torch.randn((1, T, H, D), generator=gen, device="cuda").to(torch_dt) for _ in range(2))
        lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        all_, cu = (torch.tensor([0, x], dtype=torch.int32, device="cuda") for x in (T, n))
        cache.append(0, 1, k, v, all_, lens, T, T)
        cache.commit_lengths(all_, lens)
        q = torch.randn((1, n, H * g, D), generator=gen, device="cuda").to(torch_dt)
        ring = cache.buffers["v_resid"].view(torch_dt).view(H, R + 1, D)
        keep = ring.clone()
        rng = torch.Generator().manual_seed(n)
        qe, m = max(0, T - R), 60
        tok, ch = torch.randint(qe, T, (m,), generator=rng), torch.randint(0, D, (m,), generator=rng)
        ch[m // 2:] = ch[: m - m // 2]  # several in one channel
        kinds = torch.tensor([float("inf"), float("-inf"), float("nan")])[torch.randint(0, 3, (m,), generator=rng)]
        seen = {}
        for t, c, x in zip(tok.tolist(), ch.tolist(), kinds.tolist()):
            seen[(t, c)] = x
        for window, sinks in ((0, 0), (20, 0), (33, 110), (150, qe + 7), (1, 1)):
            ring.copy_(keep)
            for t, c in seen:
                ring[1, t % (R + 1), c] = 0
            ref, got = torch.empty_like(q), torch.empty_like(q)
            cache.chunk_attention(0, 1, q, cu, n, n, lens, ref, window, sinks)
            for (t, c), x in seen.items():
                ring[1, t % (R + 1), c] = x
            cache.chunk_attention(0, 1, q, cu, n, n, lens, got, window, sinks)
            add = torch.zeros((n, D), dtype=torch.float64)
            for (t, c), x in seen.items():
                p = torch.arange(T - n, T)
                see = (t <= p) & ((t > p - window) | (t < sinks) if window else torch.ones(n, dtype=torch.bool))
                add[see, c] += x
            assert torch.isfinite(ref).all() and torch.equal(got[0, :, :g], ref[0, :, :g])  # the other kv head
            want = (ref[0, :, g:].double().cpu() + add[:, None]).to(torch_dt)
            assert torch.equal(got[0, :, g:].cpu().nan_to_num(nan=12345.0), want.nan_to_num(nan=12345.0)), (dt, window, sinks)


@pytest.mark.parametrize("g,D,n,limit", [(1, 256, 128, 40), (4, 128, 64, 40), (1, 128, 8, 4)])
def test_one_value_that_is_not_finite_does_not_hold_a_call_up(g, D, n, limit):
    """Every row went through the whole window for it, token by token: 585, 300 and 8 ms, while the
    other roles wait with a bound.  Once a warp, 8 or 16 tokens at a time, it is some milliseconds at most."""
    T = 16384
    cfg = K.Config(L=1, H_kv=1, H_q=g, D=D, batch=1, max_T=T, k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128), residual_window=T)
    cache = K.KVCache(cfg, "cuda")
    gen = torch.Generator(device="cuda").manual_seed(0)
    for b in ("k_resid", "v_resid"):
        x = cache.buffers[b].view(torch.float16)
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
    cache.buffers["v_resid"].view(torch.float16)[3] = float("nan")
    lens, cu = torch.tensor([T], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q = torch.randn((1, n, g, D), generator=gen, device="cuda").half()
    out = torch.empty_like(q)
    ms = []
    for _ in range(4):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        cache.chunk_attention(0, 1, q, cu, n, n, lens, out)
        b.record()
        torch.cuda.synchronize()
        ms.append(a.elapsed_time(b))
    assert torch.isnan(out).sum() == n * g and torch.isnan(out[..., 3]).all()
    assert min(ms) < limit, ms
