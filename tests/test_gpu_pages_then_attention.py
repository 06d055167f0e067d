"""Page calls straight between two attentions, no other launch of the stream around them: the second attention sees the new table and
the new lengths, whatever of the old ones the first has left in the caches."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(D, lengths, flags, L=4, H=4, g=2, pt=16):
    """A cache of three sequences: two hold tokens, the third is empty."""
    max_T = max(lengths) + 64
    mp = -(-max_T // pt)
    cfg = K.Config(L=L, H_kv=H, H_q=H * g, D=D, batch=3, max_T=max_T, k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128), flags=flags,
                   page_tokens=pt, n_pages=3 * mp, max_pages_per_seq=mp)
    cache = K.KVCache(cfg, "cuda", block_table=torch.full((3, mp), -1, dtype=torch.int32, device="cuda"))
    pool, lens = K.PagePool(cache), torch.zeros(3, dtype=torch.int32, device="cuda")
    pool.reserve(_i([0, 1]), _i(list(lengths)), lens)
    gen = torch.Generator(device="cuda").manual_seed(D)
    k, v = (torch.randn((L, sum(lengths), H, D), generator=gen, device="cuda").half() for _ in range(2))
    cu = _i([0, lengths[0], sum(lengths), sum(lengths)])
    cache.append(0, L, k, v, cu, lens, sum(lengths), max(lengths))
    cache.commit_lengths(cu, lens)
    return cache, pool, lens, gen


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("flags", [0, K.ROTATE_K | K.ROTATE_V])
@pytest.mark.parametrize("n", [1, 40])
def test_release_and_fork_between_attentions(D, flags, n):
    cache, pool, lens, gen = filled(D, (3000, 1111), flags)
    cfg = cache.cfg
    q = torch.randn((cfg.L, 3 * n, cfg.H_q, cfg.D), generator=gen, device="cuda").half()
    cu, third = _i([0, n, 2 * n, 3 * n]), _i([2])
    sources = [_i([0]), _i([1])]
    one, out = torch.empty_like(q[:1]), torch.empty_like(q)

    def step(which, finish=lambda: None):
        cache.chunk_attention(0, 1, q[:1], cu, 3 * n, n, lens, one)  # few tiles: most SMs are free for what comes next
        finish()
        pool.release(third, lens)
        finish()
        pool.fork(sources[which], third, lens)
        finish()
        cache.chunk_attention(0, cfg.L, q, cu, 3 * n, n, lens, out)
        finish()

    pool.fork(sources[1], third, lens)
    want = []
    for which in (0, 1):
        step(which, torch.cuda.synchronize)
        want.append(out.clone())
    assert not torch.equal(want[0][:, 2 * n:], want[1][:, 2 * n:])
    for i in range(60):
        torch.cuda._sleep(200_000)  # the host is ahead, so that the launches follow one another at once
        step(i & 1)
        assert torch.equal(out, want[i & 1]), i
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
        first = out.clone()
        step(1)
    for _ in range(30):
        graph.replay()
        assert torch.equal(first, want[0]) and torch.equal(out, want[1])
    assert cache.chunk_status() == 0 and pool.device_status() == 0


@pytest.mark.parametrize("D", [128, 256])
def test_reservation_and_compaction_between_attentions(D):
    """A page of its own for the copied tail, then pages moved together: what the table says changes, the outputs do not."""
    n = 3
    cache, pool, lens, gen = filled(D, (2001, 777), K.ROTATE_K | K.ROTATE_V)
    cfg = cache.cfg
    q = torch.randn((cfg.L, 3 * n, cfg.H_q, cfg.D), generator=gen, device="cuda").half()
    cu, third, zero, one_new = _i([0, n, 2 * n, 3 * n]), _i([2]), _i([0]), _i([1])
    out, want = torch.empty_like(q), torch.empty_like(q)
    pool.fork(zero, third, lens)
    cache.chunk_attention(0, cfg.L, q, cu, 3 * n, n, lens, want)
    torch.cuda.synchronize()
    for i in range(40):
        torch.cuda._sleep(200_000)
        cache.chunk_attention(0, cfg.L, q, cu, 3 * n, n, lens, out)
        pool.reserve(third, one_new, lens)
        cache.chunk_attention(0, cfg.L, q, cu, 3 * n, n, lens, out)
        assert torch.equal(out, want), i
        pool.release(third, lens)
        pool.fork(zero, third, lens)
        cache.chunk_attention(0, cfg.L, q, cu, 3 * n, n, lens, out)
        pool.compact()
        cache.chunk_attention(0, cfg.L, q, cu, 3 * n, n, lens, out)
        assert torch.equal(out, want), i
    assert cache.chunk_status() == 0 and pool.device_status() == 0
