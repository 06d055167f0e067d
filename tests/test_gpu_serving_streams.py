"""The serving entries on several streams: workspaces that the cache makes by
itself, and memory that another stream still writes."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402
from tests.test_gpu_serving_threads import started  # noqa: E402

LONG = 50_000_000  # clock cycles: some 25 ms


def dirty_block(nbytes):
    """A block of the allocator that holds ones, free again, with a write of the current stream still to come."""
    torch.cuda.empty_cache()
    x = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    x.fill_(255)


def test_a_workspace_made_for_another_stream_is_not_overwritten():
    cache, call, refs = started()
    side, out = torch.cuda.Stream(), torch.empty_like(refs[0])
    dirty_block(cache.chunk_ws_bytes)
    ws = cache.make_chunk_workspace(stream=side)
    torch.cuda.synchronize()
    assert not ws[:1024].any()  # prepared, and nothing has written to it since
    call(out, workspace=ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, refs[0])


def test_the_cache_s_own_workspace_on_several_streams():
    cache, call, refs = started()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = torch.full_like(refs, float("nan"))
    dirty_block(cache.chunk_ws_bytes)
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        torch.cuda._sleep(LONG)  # the first call waits here, with the preparation of its workspace
    for i, s in enumerate(streams):
        call(outs[i], i, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs, refs)
    for _ in range(50):
        outs.fill_(float("nan"))
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            call(outs[i], i, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(outs, refs)


def test_a_page_pool_made_on_another_stream_is_not_overwritten():
    cache, _, _ = started()
    ref = K.PagePool(cache).refs.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for nbytes in (K.kvq_pages_workspace_bytes(cache.cfg), 4 * cache.cfg.n_pages):
        dirty_block(nbytes)
        pool = K.PagePool(cache, stream=side)
        torch.cuda.synchronize()
        assert pool.refs.tolist() == ref.tolist() and pool.device_status() == 0


def test_a_captured_call_takes_a_prepared_workspace():
    cache, call, refs = started()
    out, g = torch.empty_like(refs[0]), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(RuntimeError, match="before the capture"):
            call(out)
    call(out, 1)
    own = cache.chunk_workspace
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        call(out)  # the eager call's workspace
    assert cache.chunk_workspace is own
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, refs[0])
    with torch.cuda.stream(side):
        call(out, 2)  # now the stream has one
    torch.cuda.synchronize()
    assert cache.chunk_workspace is not own and torch.equal(out, refs[2])


def test_the_status_of_every_workspace():
    """A bad length shows in the workspace of the call that met it, and in the cache's own taken together."""
    cache, call, refs = started()
    out, side, ws = torch.empty_like(refs[0]), torch.cuda.Stream(), cache.make_chunk_workspace()
    q = torch.zeros_like(out)
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    bad = torch.tensor([3, 1700], dtype=torch.int32, device="cuda")  # fewer tokens than rows
    assert cache.chunk_status() == 0
    call(out)
    torch.cuda.synchronize()
    cache.chunk_attention(0, 1, q, cu, 8, 4, bad, out, workspace=ws)
    assert cache.chunk_status() == 0 and cache.chunk_status(ws) == K.DEV_LENGTH
    cache.clear_chunk_status(ws)
    assert cache.chunk_status(ws) == 0
    torch.cuda.synchronize()
    cache.chunk_attention(0, 1, q, cu, 8, 4, bad, out, stream=side)
    assert cache.chunk_status() == K.DEV_LENGTH
    cache.clear_chunk_status()
    assert cache.chunk_status() == 0 and cache.device_status() == 0


def test_one_workspace_for_caches_in_turn():
    """Other formats, heads and forms of one head size, one call after the other."""
    kinds = [started(), started("llama2_7b_kivi4", H_kv=2, H_q=8), started("q8_0_mha_1k", H_kv=2, H_q=4, new=(60, 200), lengths=(700, 300))]
    ws = kinds[0][0].make_chunk_workspace()
    for _ in range(3):
        for cache, call, refs in kinds:
            assert cache.chunk_ws_bytes == ws.numel()
            out = torch.full_like(refs[0], float("nan"))
            call(out, 2, workspace=ws)
            assert torch.equal(out, refs[2])
    assert kinds[0][0].chunk_status(ws) == 0
