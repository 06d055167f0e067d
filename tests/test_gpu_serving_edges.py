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
