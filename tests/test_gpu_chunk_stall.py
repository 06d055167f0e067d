"""Failure detection of the chunk attention without a GPU fault: the roles of
a CTA wait for one another with a bound.  In the library's test mode
(kvq_test_force_stall) one role of every second CTA, each role in turn, waits
on a shared-memory barrier that nothing completes and gives up.  The call must
return with KVQ_DEV_STALL set, whatever the form that its rows choose."""

from dataclasses import replace

import pytest

from tests.gpu_cases import appended_cache

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402
from bit_kv_cache_04_gb300 import workloads as W  # noqa: E402

# (workload, heads, new tokens of the two sequences): few rows, rows as lanes, rows in pairs of tiles; 256 channels;
# pages whose bytes are loaded directly
CASES = {
    "few": ("gqa8b_hadamard4_paged", dict(H_kv=2, H_q=8), [4, 2]),
    "few_kivi": ("llama2_7b_kivi4", dict(H_kv=2, H_q=8), [1, 1]),
    "lanes": ("llama2_7b_kivi4", dict(H_kv=2, H_q=8), [20, 20]),
    "paired": ("gqa8b_hadamard4_paged", dict(H_kv=2, H_q=8), [150, 90]),
    "wide": ("ctx262k_hadamard4", dict(H_kv=1, H_q=6), [40]),
    "direct": ("q4_0_mha_1k", dict(H_kv=2, H_q=4, page_tokens=5), [9, 9]),
}


def started(name):
    base, kw, new = CASES[name]
    w = W.make(base)
    lengths = [3000, 1700][: len(new)]
    w = W.Workload(w.name, replace(w.cfg, **kw), w.lengths, w.values, w.extra_tokens).scaled(L=1, lengths=lengths, extra=0)
    cache, lens, _, _ = appended_cache(w, with_oracle=False)
    cfg = w.cfg
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(5)
    dt = torch.float16 if cfg.in_dtype == K.DT_F16 else torch.bfloat16
    qs = torch.randn((2, 1, sum(new), cfg.H_q, cfg.D), generator=gen, device="cuda").to(dt)

    def call(ws, which=0):
        out = torch.full_like(qs[0], float("nan"))
        cache.chunk_attention(0, 1, qs[which], cu, sum(new), max(new), lens, out, 0, 0, workspace=ws)
        torch.cuda.synchronize()
        return out, ws[:4].view(torch.int32).item()

    return cache, call


@pytest.mark.parametrize("name", CASES)
def test_a_wait_that_runs_out_sets_stall_and_returns(name):
    cache, call = started(name)
    ref, status = call(cache.make_chunk_workspace())
    assert status == 0
    K.kvq_test_force_stall(256)
    try:
        _, status = call(cache.make_chunk_workspace())
        assert status == K.DEV_STALL
    finally:
        K.kvq_test_force_stall(0)
    out, status = call(cache.make_chunk_workspace())
    assert status == 0 and torch.equal(out, ref)


@pytest.mark.parametrize("name", CASES)
def test_the_next_call_on_the_same_workspace_is_whole(name):
    """Sequences cut among CTAs are joined by a count of their parts: parts that a
    stalled call counted must not be counted again."""
    cache, call = started(name)
    ws = cache.make_chunk_workspace()
    refs = [call(ws, i)[0] for i in range(2)]
    for _ in range(3):
        K.kvq_test_force_stall(256)
        try:
            call(ws)
        finally:
            K.kvq_test_force_stall(0)
        K._check(K.LIB.kvq_clear_device_status(ws.data_ptr(), None))
        for i in (1, 0, 1):
            out, status = call(ws, i)
            assert status == 0 and torch.equal(out, refs[i])
