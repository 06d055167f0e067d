"""Failure detection of the attention over shared prefixes, as tests/test_gpu_chunk_stall.py does it for the chunk attention: in the
library's test mode one role of every second CTA gives up waiting; the call returns with KVQ_DEV_STALL set, and the
next call on the workspace, of the same plan, is whole."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402
from tests.test_gpu_prefix_attention import FORMATS, build  # noqa: E402

# few rows, rows as lanes, rows in pairs of tiles; 256 channels; pages whose bytes are loaded directly
CASES = {
    "few": ("rot4", dict(), 1),
    "few_window": ("rot4_bf16_window", dict(), 1),
    "lanes": ("q4_0", dict(g=8), 2),
    "paired": ("rot4", dict(g=8), 20),
    "wide": ("rot4_d256", dict(), 3),
    "direct": ("p5_direct", dict(), 1),
}


@pytest.mark.parametrize("name", CASES)
def test_a_stalled_call_returns_and_the_next_is_whole(name):
    fmt, kw, new = CASES[name]
    c = build([3000, 1700], [[50 + new, 90, 130 + new], [20 + new, 200]], [[new] * 3, [new] * 2], **{**FORMATS[fmt], **kw})
    cache, lens, cu_g, n = c[0], c[2], c[3], c[4]
    cu = torch.tensor([sum(n[:i]) for i in range(6)], dtype=torch.int32, device="cuda")
    dt = torch.float16 if cache.cfg.in_dtype == K.DT_F16 else torch.bfloat16
    qs = torch.randn((2, 1, sum(n), cache.cfg.H_q, cache.cfg.D), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").to(dt)
    pa = K.PrefixAttention(cache, 2, sum(n))
    pa.plan(cu_g, cu, sum(n), new, 3 * new, lens)

    def call(which):
        out = torch.full_like(qs[0], float("nan"))
        pa.attention(0, 1, qs[which], out)
        torch.cuda.synchronize()
        return out, pa.device_status()

    refs = [call(i) for i in range(2)]
    assert all(s == 0 for _, s in refs)
    for _ in range(3):
        K.kvq_test_force_stall(256)
        try:
            assert call(0)[1] == K.DEV_STALL
        finally:
            K.kvq_test_force_stall(0)
        pa.clear_status()
        for i in (1, 0, 1):
            out, status = call(i)
            assert status == 0 and torch.equal(out, refs[i][0])
