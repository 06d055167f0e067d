"""Reordering of beams' sequences against the sequential model: tables, counts, lengths and windows, byte for byte."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402
from tests.test_gpu_pages import _i, make, same  # noqa: E402


def grow(pool, lens, model, n_new):
    seqs = list(range(len(n_new)))
    pool.reserve(_i(seqs), _i(n_new), lens)
    model.reserve(seqs, n_new)
    for s, n in enumerate(n_new):
        model.lens[s] += n
    lens.copy_(_i(model.lens.tolist()))


def started(group, groups, R=0, **kw):
    """Every group's first slot has a prompt that the others share; then each grows by itself."""
    batch = group * groups
    cache, pool, lens, model = make(batch=batch, pages=batch * 12 + 20, R=R, **kw)
    grow(pool, lens, model, [0 if b % group else 33 + b % 7 for b in range(batch)])
    src = [b // group * group for b in range(batch) if b % group]
    dst = [b for b in range(batch) if b % group]
    if dst:
        pool.fork(_i(src), _i(dst), lens)
        model.fork(src, dst)
    grow(pool, lens, model, [1 + b % 3 for b in range(batch)])
    same(cache, pool, lens, model)
    return cache, pool, lens, model


@pytest.mark.parametrize("group,groups", [(1, 3), (2, 3), (3, 2), (4, 5), (8, 2), (9, 1), (16, 2), (17, 1), (32, 2)])
@pytest.mark.parametrize("R,kw", [(0, {}), (5, {}), (20, dict(D=256, L=3, H=1))])
def test_steps_of_a_search(group, groups, R, kw):
    cache, pool, lens, model = started(group, groups, R, **kw)
    rng = np.random.default_rng(group + R)
    for step in range(6):
        kind = step % 3
        parents = (rng.integers(0, group, (groups, group)) if kind == 0 else  # some die, some branch
                   np.stack([rng.permutation(group) for _ in range(groups)]) if kind == 1 else  # all live, in another order
                   np.repeat(rng.integers(0, group, (groups, 1)), group, 1))  # one is left
        pool.reorder(_i(parents.ravel().tolist()), group, lens)
        model.reorder(parents.ravel().tolist(), group)
        same(cache, pool, lens, model)
        grow(pool, lens, model, [1] * (group * groups))
        same(cache, pool, lens, model)
    assert pool.device_status() == 0


def test_nothing_moves_when_all_stay():
    cache, pool, lens, model = started(4, 3, 20)
    pool.reorder(_i(list(range(4)) * 3), 4, lens)
    same(cache, pool, lens, model)


@pytest.mark.parametrize("bad", [-1, 4, 2 ** 31 - 1, -2 ** 31])
def test_a_bad_parent_leaves_its_group_as_it_was(bad):
    cache, pool, lens, model = started(4, 3, 20)
    parents = [1, 0, 3, 3, 0, 0, bad, 1, 2, 2, 2, 2]
    pool.reorder(_i(parents), 4, lens)
    model.reorder([1, 0, 3, 3, 0, 1, 2, 3, 2, 2, 2, 2], 4)
    same(cache, pool, lens, model)
    assert pool.device_status() == K.DEV_SEQ


@pytest.mark.parametrize("T", [-1, 101, 2 ** 31 - 1])
def test_a_bad_length_leaves_its_group_as_it_was(T):
    cache, pool, lens, model = started(4, 3, 20)
    lens[5] = T
    pool.reorder(_i([1, 0, 3, 3, 0, 0, 1, 1, 2, 2, 2, 2]), 4, lens)
    model.reorder([1, 0, 3, 3, 0, 1, 2, 3, 2, 2, 2, 2], 4)
    model.lens[5] = T
    same(cache, pool, lens, model)
    assert pool.device_status() == K.DEV_LENGTH


def test_entries_outside_the_pool():
    cache, pool, lens, _ = make(batch=4, max_T=64, pages=8, table=[[0, 3, -1, -1], [1, 4, -1, -1], [2, 5, -1, -1], [6, 7, -1, -1]])
    cache.block_table.copy_(_i([[0, 3, -1, -1], [1, 99, -1, -1], [2, 5, -5, -1], [6, 7, -1, -1]]))
    lens.fill_(32)
    pool.reorder(_i([1, 0, 0, 0]), 2, lens)  # the second group's first slot becomes both
    torch.cuda.synchronize()
    assert cache.block_table.tolist() == [[1, 99, -1, -1], [0, 3, -1, -1], [2, 5, -5, -1], [2, 5, -1, -1]]
    assert pool.refs.tolist() == [1, 1, 2, 1, 1, 2, 0, 0] and pool.device_status() == K.DEV_PAGE


def test_long_rows_and_many_slots():
    """More table columns than a block, pages shared by some of a group's slots in some columns."""
    batch, mp = 64, 300
    rng = np.random.default_rng(1)
    table = rng.integers(0, 500, (batch // 16, 1, mp)).repeat(16, 1)
    table = np.where(rng.random((batch // 16, 16, mp)) < 0.3, rng.integers(0, 500, (batch // 16, 16, mp)), table).reshape(batch, mp)
    table[:, 280:] = -1
    cache, pool, lens, model = make(batch=batch, L=1, H=1, max_T=mp * 16, pages=500, table=table.tolist())
    model.lens[:] = rng.integers(0, 281 * 16, batch).clip(max=280 * 16)  # and pages behind the tokens
    lens.copy_(_i(model.lens.tolist()))
    for _ in range(3):
        parents = rng.integers(0, 16, batch).tolist()
        pool.reorder(_i(parents), 16, lens)
        model.reorder(parents, 16)
        same(cache, pool, lens, model)
    assert pool.device_status() == 0


def test_captured():
    cache, pool, lens, model = started(4, 2, 5)
    parents = _i([0] * 8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.reorder(parents, 4, lens)
    for p in ([1, 2, 3, 0, 3, 3, 0, 1], [2, 2, 0, 1, 0, 1, 2, 3]):
        parents.copy_(_i(p))
        graph.replay()
        model.reorder(p, 4)
        same(cache, pool, lens, model)
