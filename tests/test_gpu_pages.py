"""The page calls against the sequential model, byte for byte: random
histories of forks, reserves, releases and compactions, each way a call can be passed over
or refused on the device, and captured calls."""

import numpy as np
import pytest

from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(L=2, H=2, D=128, batch=6, max_T=100, pages=40, pt=16, R=0, fmt=K.Fmt(4, 128), vfmt=None, seed=0, table=None):
    mp = -(-max_T // pt)
    cfg = K.Config(L=L, H_kv=H, H_q=H, D=D, batch=batch, max_T=max_T, k_fmt=fmt, v_fmt=vfmt or fmt, residual_window=R,
                   page_tokens=pt, n_pages=pages, max_pages_per_seq=mp)
    t = torch.full((batch, mp), -1, dtype=torch.int32, device="cuda") if table is None else _i(table)
    cache = K.KVCache(cfg, "cuda", block_table=t)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for n in ("k_main", "v_main", "k_resid", "v_resid"):
        b = cache.buffers[n]
        if b is not None:
            b.copy_(torch.randint(0, 256, b.shape, generator=g, device="cuda", dtype=torch.uint8))
    pool = K.PagePool(cache)
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    pools = [cache.buffers[n].cpu().numpy().reshape(L, pages, -1) for n in ("k_main", "v_main")]
    wins = [cache.buffers[n].cpu().numpy().reshape(L, batch, -1) for n in ("k_resid", "v_resid")
            if cache.buffers[n] is not None]
    model = S.Pages(t.cpu().numpy(), pages, pt, max_T, R, pools, wins)
    return cache, pool, lens, model


def same(cache, pool, lens, model):
    torch.cuda.synchronize()
    L, B, P = cache.cfg.L, cache.cfg.batch, cache.cfg.n_pages
    assert np.array_equal(cache.block_table.cpu().numpy(), model.table)
    assert np.array_equal(pool.refs.cpu().numpy(), model.refs)
    assert np.array_equal(lens.cpu().numpy(), model.lens)
    for n, want in zip(("k_main", "v_main"), model.pools):
        assert np.array_equal(cache.buffers[n].cpu().numpy().reshape(L, P, -1), want), n
    for n, want in zip(("k_resid", "v_resid"), model.windows):
        assert np.array_equal(cache.buffers[n].cpu().numpy().reshape(L, B, -1), want), n


@pytest.mark.parametrize("shape", [
    dict(), dict(R=20), dict(pt=1, pages=300, max_T=40), dict(pt=7, R=5, D=256, pages=60), dict(fmt=K.Fmt(8, 32), L=1),
    dict(fmt=K.Fmt(3, 128), vfmt=K.Fmt(4, 32), pt=5, H=1, L=1, pages=80), dict(batch=40, pages=3000, max_T=300, L=1, H=1),
])
def test_random_histories(shape):
    cache, pool, lens, model = make(**shape)
    B, max_T = cache.cfg.batch, cache.cfg.max_T
    rng = np.random.default_rng(7)
    for step in range(40):
        live = [s for s in range(B) if model.lens[s] > 0]
        empty = [s for s in range(B) if model.lens[s] == 0 and (model.table[s] < 0).all()]
        kind = rng.choice(["grow", "grow", "fork", "release", "compact"])
        if kind == "grow":
            seqs = rng.permutation(B)[: rng.integers(1, B + 1)].tolist()
            n_new = [int(min(rng.integers(0, 20), max_T - model.lens[s])) for s in seqs]
            if (model.refs == 0).sum() < sum(n_new) + len(seqs):
                continue
            pool.reserve(_i(seqs), _i(n_new), lens)
            model.reserve(seqs, n_new)
            for s, n in zip(seqs, n_new):  # the append
                model.lens[s] += n
                lens[s] += n
        elif kind == "fork" and live and empty:
            dst = rng.permutation(empty)[: rng.integers(1, len(empty) + 1)].tolist()
            src = rng.choice(live, len(dst)).tolist()
            pool.fork(_i(src), _i(dst), lens)
            model.fork(src, dst)
        elif kind == "release" and live:
            seqs = rng.choice(live, rng.integers(1, min(len(live), 3) + 1)).tolist()  # may list one twice
            pool.release(_i(seqs), lens)
            model.release(seqs)
        elif kind == "compact":
            pool.compact()
            model.compact()
        same(cache, pool, lens, model)
    assert pool.device_status() == 0


def test_init_counts_a_given_table():
    table = [[0, 3, 3, -1], [3, -1, 99, -7]]
    cache, pool, lens, _ = make(batch=2, max_T=64, pages=8, table=[[0, 3, 3, -1], [3, -1, -1, -1]])
    assert pool.refs.tolist() == [1, 0, 0, 3, 0, 0, 0, 0] and pool.device_status() == 0
    cache.block_table.copy_(_i(table))
    pool2 = K.PagePool(cache)
    assert pool2.refs.tolist() == [1, 0, 0, 3, 0, 0, 0, 0] and pool2.device_status() == K.DEV_PAGE


def test_last_reader_keeps_the_page():
    cache, pool, lens, model = make()
    pool.reserve(_i([0]), _i([20]), lens)
    model.reserve([0], [20])
    lens[0] = model.lens[0] = 20
    pool.fork(_i([0, 0, 0]), _i([3, 1, 5]), lens)
    model.fork([0, 0, 0], [3, 1, 5])
    for seqs in ([5, 0], [1, 3]):  # of four readers the last one left keeps the half-full page
        pool.reserve(_i(seqs), _i([1, 1]), lens)
        model.reserve(seqs, [1, 1])
        same(cache, pool, lens, model)
    assert pool.device_status() == 0


def _started():
    cache, pool, lens, model = make(R=4)
    pool.reserve(_i([0, 1]), _i([30, 50]), lens)
    model.reserve([0, 1], [30, 50])
    lens[0] = model.lens[0] = 30
    lens[1] = model.lens[1] = 50
    return cache, pool, lens, model


@pytest.mark.parametrize("seqs,n_new,bit", [
    ([0, 2, 0], [1, 1, 1], K.DEV_SEQ), ([0, 6], [1, 1], K.DEV_SEQ), ([-1, 0], [1, 1], K.DEV_SEQ),
    ([0, 1], [1, -1], K.DEV_LENGTH), ([0, 1], [71, 1], K.DEV_CAPACITY), ([0, 1], [2 ** 31 - 1, 1], K.DEV_CAPACITY),
    ([2, 3, 4, 5], [100, 100, 100, 100 - 0], 0), ([2, 3, 4, 5, 0, 1], [100, 100, 100, 100, 70, 50], K.DEV_CAPACITY),
])
def test_reserve_is_all_or_nothing(seqs, n_new, bit):
    cache, pool, lens, model = _started()
    pool.reserve(_i(seqs), _i(n_new), lens)
    if not bit:
        model.reserve(seqs, n_new)
    same(cache, pool, lens, model)
    assert pool.device_status() == bit
    pool.clear_status()
    pool.reserve(_i([1, 0]), _i([3, 3]), lens)  # and the next call works
    model.reserve([1, 0], [3, 3])
    same(cache, pool, lens, model)
    assert pool.device_status() == 0


def test_reserve_refuses_broken_tables_and_lengths():
    cache, pool, lens, model = _started()
    for at, val, bit in (((0, 1), 77, K.DEV_PAGE), ((0, 1), -1, K.DEV_PAGE), ((0, 2), -9, K.DEV_PAGE)):
        old = cache.block_table[at].item()
        cache.block_table[at] = val
        before = (cache.block_table.clone(), pool.refs.clone())
        pool.reserve(_i([0]), _i([10]), lens)
        assert pool.device_status() == bit
        assert torch.equal(cache.block_table, before[0]) and torch.equal(pool.refs, before[1])
        cache.block_table[at] = old
        pool.clear_status()
    for T in (-1, 101):
        lens[0] = T
        pool.reserve(_i([0]), _i([1]), lens)
        assert pool.device_status() == K.DEV_LENGTH
        pool.clear_status()
    lens[0] = 30
    same(cache, pool, lens, model)


@pytest.mark.parametrize("src,dst,good,bit", [
    ([0, 0, 1], [2, 2, 3], [0, 2], K.DEV_SEQ),      # a target twice: the first pair
    ([0, 2, 1], [2, 3, 4], [2], K.DEV_SEQ),         # a sequence that is target and source: both pairs
    ([0, 1], [1, 4], [], K.DEV_SEQ),                # a target that is not empty and is a source: neither
    ([0, 1], [0, 4], [1], K.DEV_SEQ),               # itself
    ([0, 9, 1, -1], [2, 3, 6, 4], [0], K.DEV_SEQ),  # out of range
    ([4], [5], [0], 0),                             # an empty parent
])
def test_fork_passes_bad_pairs_over(src, dst, good, bit):
    cache, pool, lens, model = _started()
    pool.fork(_i(src), _i(dst), lens)
    model.fork([src[i] for i in good], [dst[i] for i in good])
    same(cache, pool, lens, model)
    assert pool.device_status() == bit


def test_fork_passes_broken_sources_over():
    cache, pool, lens, model = _started()
    cache.block_table[0, 1] = 40
    pool.fork(_i([0]), _i([2]), lens)
    assert pool.device_status() == K.DEV_PAGE
    pool.clear_status()
    lens[1] = 101
    pool.fork(_i([1]), _i([2]), lens)
    assert pool.device_status() == K.DEV_LENGTH
    assert (cache.block_table[2] == -1).all() and lens[2] == 0


def test_release_of_bad_indexes_and_entries():
    cache, pool, lens, model = _started()
    pool.release(_i([0, 6, -1, 0, 3]), lens)
    model.release([0])
    same(cache, pool, lens, model)
    assert pool.device_status() == K.DEV_SEQ
    pool.clear_status()
    cache.block_table[1, 6] = 40  # outside the pool
    free = int((pool.refs == 0).nonzero()[0])
    cache.block_table[1, 5] = free  # nobody's page
    pool.release(_i([1]), lens)
    model.release([1])
    same(cache, pool, lens, model)
    assert pool.device_status() == K.DEV_PAGE


@pytest.mark.parametrize("pages", [1, 3, 33, 1024, 1025, 5000])
def test_compact_out_of_place(pages):
    batch, mp = 7, -(-pages // 7) + 1
    rng = np.random.default_rng(pages)
    for used in sorted({0, 1, pages // 2, pages - 1, pages}):
        perm = rng.permutation(pages)[:used]
        table = np.full(batch * mp, -1)
        table[rng.permutation(batch * mp)[:used]] = perm
        cache, pool, lens, model = make(L=3, H=1, batch=batch, max_T=mp * 16, pages=pages, table=table.reshape(batch, mp).tolist())
        t0, r0 = cache.block_table.clone(), pool.refs.clone()
        t1, r1 = torch.empty_like(t0), torch.empty_like(r0)
        pool.compact(refs_out=r1, table_out=t1)
        model.compact()
        assert torch.equal(cache.block_table, t0) and torch.equal(pool.refs, r0)
        cache.block_table.copy_(t1)
        pool.refs.copy_(r1)
        same(cache, pool, lens, model)
        assert pool.device_status() == 0


def test_compact_flags_entries_of_no_page():
    cache, pool, lens, _ = make(batch=2, max_T=64, pages=8, table=[[7, 6, -1, -1], [5, -1, -1, -1]])
    cache.block_table[1, 1], cache.block_table[1, 2], cache.block_table[1, 3] = 8, -3, 2
    pool.compact()
    assert cache.block_table.tolist() == [[2, 1, -1, -1], [0, -1, -1, -1]]
    assert pool.device_status() == K.DEV_PAGE


def test_a_captured_beam_step():
    cache, pool, lens, model = make(batch=8, R=4)
    pool.reserve(_i([0, 1]), _i([30, 45]), lens)
    model.reserve([0, 1], [30, 45])
    lens[0] = model.lens[0] = 30
    lens[1] = model.lens[1] = 45
    kids, src, ones = _i([2, 3, 4, 5]), _i([0, 1, 0, 1]), _i([1, 1, 1, 1])

    def step():
        pool.release(kids, lens)
        pool.fork(src, kids, lens)
        pool.reserve(kids, ones, lens)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for parents in ([0, 1, 0, 1], [1, 1, 1, 0], [0, 0, 0, 0]):
        src.copy_(_i(parents))
        g.replay()
        model.release([2, 3, 4, 5])
        model.fork(parents, [2, 3, 4, 5])
        model.reserve([2, 3, 4, 5], [1] * 4)
        same(cache, pool, lens, model)
    assert pool.device_status() == 0
