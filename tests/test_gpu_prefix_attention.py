"""Attention over shared prefixes against fp64 attention over each sequence's own dequantized cache, with the rounding bound of
oracle.serving_oracle.chunk_attention: groups of every size, prefixes around tile and page borders, every paged
format, empty slots, bad rows and pages, window values that are not finite, captured calls."""

import numpy as np
import pytest

from oracle import kvq_oracle as O
from oracle import serving_oracle as S
from tests.gpu_cases import gpu_buffers_as_oracle
from tests.helpers import oracle_cfg, raw16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402

DT = {0: torch.float16, 1: torch.bfloat16}
ROT4 = dict(k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128), flags=K.ROTATE_K | K.ROTATE_V, sign_seed=7)
FORMATS = {
    "rot4": ROT4,
    "rot4_bf16_window": dict(ROT4, in_dtype=K.DT_BF16, residual_window=37),
    "rot4_d256": dict(ROT4, D=256, H_kv=1, g=6, in_dtype=K.DT_BF16),
    "rot3_d256_fp16": dict(ROT4, k_fmt=K.Fmt(3, 128), D=256, H_kv=1, g=3, residual_window=5),
    "tbq4": dict(ROT4, flags=K.ROTATE_K | K.ROTATE_V | K.TBQ4_K | K.TBQ4_V, in_dtype=K.DT_BF16),
    "q4_0": dict(),
    "q8_0_bf16": dict(k_fmt=K.Fmt(8, 32), v_fmt=K.Fmt(8, 32), in_dtype=K.DT_BF16, g=8),
    "q4_zp": dict(flags=K.ZP_K | K.ZP_V),
    "two_bit_p8": dict(k_fmt=K.Fmt(2, 32), v_fmt=K.Fmt(2, 32), page_tokens=8, residual_window=9),
    "pre_rope": dict(flags=K.K_PRE_ROPE, residual_window=20),
    "p5_direct": dict(page_tokens=5),
    "p64": dict(ROT4, page_tokens=64),
    "mixed": dict(k_fmt=K.Fmt(8, 128), v_fmt=K.Fmt(2, 128), flags=K.ROTATE_V),
}


def build(groups, own, new, L=1, H_kv=2, g=4, D=128, seed=0, page_tokens=16, values=None, empty=(), **kw):
    """A paged cache of len(groups) prompts of groups[i] tokens, each forked into len(own[i]) sequences that go on by own[i][j]
    tokens of their own, the last new[i][j] of them new.  empty: slots (of the batch) that are released again."""
    B = sum(len(x) for x in own)
    flat_own, flat_new = [t for x in own for t in x], [n for x in new for n in x]
    first = np.cumsum([0] + [len(x) for x in own])
    group_of = [i for i, x in enumerate(own) for _ in x]
    lens_np = [groups[group_of[b]] + flat_own[b] for b in range(B)]
    max_T = max(lens_np)
    mp = -(-max_T // page_tokens)
    kw.setdefault("k_fmt", K.Fmt(4, 32))
    kw.setdefault("v_fmt", K.Fmt(4, 32))
    cfg = K.Config(L=L, H_kv=H_kv, H_q=H_kv * g, D=D, batch=B, max_T=max_T, page_tokens=page_tokens,
                   n_pages=sum(-(-t // page_tokens) + 1 for t in lens_np) + 3, max_pages_per_seq=mp, **kw)
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    cache = K.KVCache(cfg, "cuda", block_table=table)
    pool = K.PagePool(cache)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def append(n_new):
        seqs = [b for b in range(B) if n_new[b]]
        if not seqs:
            return
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        pool.reserve(i(seqs), i([n_new[b] for b in seqs]), lens)
        total, cu = sum(n_new), i(np.concatenate([[0], np.cumsum(n_new)]).tolist())
        k, v = (torch.randn((L, total, H_kv, D), generator=gen, device="cuda").to(DT[cfg.in_dtype]) for _ in range(2))
        if values is not None:
            values(k, v, n_new)
        cache.append(0, L, k, v, cu, lens, total, max(n_new))
        cache.commit_lengths(cu, lens)

    append([groups[group_of[b]] if b == first[group_of[b]] else 0 for b in range(B)])
    kids = [b for b in range(B) if b != first[group_of[b]] and groups[group_of[b]]]
    if kids:
        pool.fork(torch.tensor([int(first[group_of[b]]) for b in kids], dtype=torch.int32, device="cuda"),
                  torch.tensor(kids, dtype=torch.int32, device="cuda"), lens)
    append(flat_own)
    if empty:
        pool.release(torch.tensor(list(empty), dtype=torch.int32, device="cuda"), lens)
        for b in empty:
            lens_np[b] = flat_new[b] = 0
    torch.cuda.synchronize()
    assert cache.device_status() == 0 and pool.device_status() == 0
    assert lens.tolist() == lens_np
    cu_g = torch.tensor(first.tolist(), dtype=torch.int32, device="cuda")
    most = max(sum(flat_new[first[i]:first[i + 1]]) for i in range(len(own)))
    return cache, pool, lens, cu_g, flat_new, most


def shared_of(pa):
    """The prefix that every group shares, from the units of the plan in the workspace."""
    cfg = pa.cache.cfg
    B, (total_q, _, _) = cfg.batch, pa.planned

    def up(x):
        return (x + 255) // 256 * 256

    at = up(K.kvq_chunk_workspace_bytes(cfg)) + 256 + up(4 * pa.groups) + up(4 * B) + up(8 * total_q)
    n = total_q * (cfg.H_q // cfg.H_kv) // 128 + B
    units = pa.workspace[at:at + 32 * n].view(torch.int32).view(n, 8).cpu().numpy()  # first row, row, rows, sequence, prefix, own ..
    own = pa.workspace[at + up(32 * n):].view(torch.int32)
    cu, got = pa.cu_groups.tolist(), []
    for i in range(pa.groups):
        mine = [u for u in units if u[2] and cu[i] <= u[3] < cu[i + 1]]
        seqs = {own[4 * (u[5] + k)].item() for u in mine for k in range(u[6])}
        got.append(int(mine[0][4]) if len(seqs) > len({u[3] for u in mine}) else 0)  # several sequences behind one prefix
    return got


def attend(cache, lens, cu_g, n_new, most, q=None, pad=2, seed=1, pa=None):
    cfg = cache.cfg
    cu = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
    total = int(cu[-1]) + pad
    if q is None:
        g = torch.Generator(device="cuda").manual_seed(seed)
        q = torch.randn((cfg.L, total, cfg.H_q, cfg.D), generator=g, device="cuda").to(DT[cfg.in_dtype])
    out = torch.full_like(q, -7.0)
    pa = pa or K.PrefixAttention(cache, cu_g.numel() - 1, total)
    pa.cu_groups = cu_g
    pa.plan(cu_g, torch.as_tensor(cu, device="cuda"), total, max(n_new), most, lens)
    pa.attention(0, cfg.L, q, out)
    torch.cuda.synchronize()
    assert torch.all(out[:, cu[-1]:] == -7.0)
    return q, out, cu, pa


def check(cache, lens, cu_g, n_new, most, want_shared=None, **kw):
    cfg = cache.cfg
    q, out, cu, pa = attend(cache, lens, cu_g, n_new, most, **kw)
    assert pa.device_status() == 0
    if want_shared is not None:
        assert shared_of(pa) == want_shared
    oc = oracle_cfg(cfg)
    bufs = gpu_buffers_as_oracle(cache, oc)
    table = cache.block_table.cpu().numpy()
    u = 2.0 ** -11 if cfg.in_dtype == 0 else 2.0 ** -8
    for l in range(cfg.L):
        want, bound = S.chunk_attention(oc, bufs, l, raw16(q[l]), cu, lens.tolist(), 0, 0, table, True,
                                        4.0 if cfg.flags & (K.ZP_K | K.ZP_V) else 2.0)
        rows = slice(0, int(cu[-1]))
        got = O.input_to_f32(raw16(out[l]), cfg.in_dtype).astype(np.float64)[rows]
        err = np.abs(got - want[rows])
        # the join: two weights and a sum in fp32 of parts no larger than the values
        lim = bound[rows] + 2.0 ** -20 * np.abs(want[rows]).max()
        assert np.all(err <= lim), (float(np.max(err / lim)), np.unravel_index(np.argmax(err / lim), err.shape))
        assert np.linalg.norm(got - want[rows]) <= 4 * u * np.linalg.norm(want[rows])
    return out


@pytest.mark.parametrize("key", FORMATS)
@pytest.mark.parametrize("new", ["one", "few", "many"])
def test_formats(key, new):
    n = {"one": [[1, 1, 1], [1], [1, 1]], "few": [[3, 1, 5], [2], [9, 4]], "many": [[60, 1, 33], [70], [5, 40]]}[new]
    own = [[70, 1, 40], [90], [20, 77]] if new != "many" else [[70, 1, 140], [90], [20, 77]]
    c = build([300, 100, 190], own, n, **FORMATS[key])
    check(c[0], c[2], c[3], c[4], c[5])


@pytest.mark.parametrize("prefix", [1, 15, 16, 63, 64, 127, 128, 129, 143, 144, 145, 255, 256, 271, 300, 513])
@pytest.mark.parametrize("R", [0, 20])
def test_prefix_lengths(prefix, R):
    for D in (128, 256):
        c = build([prefix], [[1, 30, 130]], [[1, 2, 1]], D=D, H_kv=1, g=2, residual_window=R)
        tile = 128 if D == 128 else 64
        # whole pages that are full in all of them, quantized and before the new tokens: own tokens 1 with 1 new, 30 with 2
        pages = min(prefix // 16, max(0, prefix + 1 - max(R, 1)) // 16)
        check(c[0], c[2], c[3], c[4], c[5], want_shared=[pages * 16 // tile * tile])


@pytest.mark.parametrize("g,H", [(1, 1), (2, 3), (3, 2), (5, 1), (7, 1), (8, 2)])
@pytest.mark.parametrize("beams", [2, 3, 8, 33])
def test_heads_and_beams(g, H, beams):
    """Every form of the kernel: up to 32, 128 and more rows a group."""
    c = build([260], [[5 + (7 * i) % 90 for i in range(beams)]], [[1 + i % 3 for i in range(beams)]], H_kv=H, g=g, **ROT4)
    check(c[0], c[2], c[3], c[4], c[5], want_shared=[256])


def test_many_groups_and_layers():
    own = [[1 + (i * j) % 50 for j in range(1 + i % 4)] for i in range(11)]
    c = build([130 * (i % 4) + i for i in range(11)], own, [[1] * len(x) for x in own], L=3, **ROT4)
    check(c[0], c[2], c[3], c[4], c[5])


def test_empty_slots_and_sequences_without_new_tokens():
    c = build([400, 400], [[30, 40, 50, 60], [10, 20, 30, 40]], [[1, 0, 2, 1], [1, 1, 0, 0]], empty=(2, 5))
    out = check(c[0], c[2], c[3], c[4], c[5], want_shared=[384, 0])  # one of the second group's is left with a new token
    assert torch.isfinite(out[:, :sum(c[4])]).all()


def test_groups_as_one_and_as_singles():
    """The result does not depend on how the batch is grouped."""
    c = build([300], [[30, 40, 50, 60]], [[3, 1, 2, 1]])
    cache, lens, n = c[0], c[2], c[4]
    a = check(cache, lens, c[3], n, 7, want_shared=[288 // 128 * 128])
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    check(cache, lens, i([0, 1, 2, 3, 4]), n, 3, want_shared=[0] * 4)
    check(cache, lens, i([0, 0, 2, 2, 4]), n, 7, want_shared=[0, 256, 0, 256])
    cu = i(np.concatenate([[0], np.cumsum(n)]).tolist())
    out, q = torch.full_like(a, -7), attend(cache, lens, c[3], n, 7)[0]
    cache.chunk_attention(0, 1, q, cu, q.shape[1], 3, lens, out)
    torch.cuda.synchronize()
    assert (out.float() - a.float()).norm() <= 2.0 ** -9 * out.float().norm()


def _bits(cache, lens, cu_g, n, most, cu=None, pad=0):
    cfg = cache.cfg
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32) if cu is None else np.asarray(cu, np.int32)
    total = sum(n) + pad
    q = torch.randn((cfg.L, total, cfg.H_q, cfg.D), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").half()
    out = torch.full_like(q, -7.0)
    pa = K.PrefixAttention(cache, cu_g.numel() - 1, total)
    pa.cu_groups = cu_g
    pa.plan(cu_g, torch.as_tensor(cu, device="cuda"), total, max(n), most, lens)
    pa.attention(0, cfg.L, q, out)
    torch.cuda.synchronize()
    return q, out, pa


def test_what_is_out_of_order():
    c = build([300, 300], [[30, 40, 50], [10, 20, 30]], [[1, 2, 1], [1, 1, 1]])
    cache, lens, cu_g, n = c[0], c[2], c[3], c[4]
    q, good, pa = _bits(cache, lens, cu_g, n, 4)
    assert pa.device_status() == 0 and shared_of(pa) == [256, 256]
    # a bad length: that sequence's rows stay, its group goes without the prefix, the others get theirs
    for bad in (-1, 1, cache.cfg.max_T + 1):
        l2 = lens.clone()
        l2[1] = bad
        _, out, pa = _bits(cache, l2, cu_g, n, 4)
        assert pa.device_status() == K.DEV_LENGTH and shared_of(pa) == [0, 256]
        assert torch.all(out[:, 1:3] == -7.0)
        keep = [0, 3, 4, 5, 6]
        assert (out[:, keep].float() - good[:, keep].float()).norm() <= 2.0 ** -9 * good[:, keep].float().norm()
    # more new tokens in a group than the bound
    _, out, pa = _bits(cache, lens, cu_g, n, 3)
    assert pa.device_status() == K.DEV_LENGTH and shared_of(pa) == [0, 256]
    assert (out.float() - good.float()).norm() <= 2.0 ** -9 * good.float().norm()
    # rows that do not ascend, or begin late
    for cu in ([0, 1, 0, 4, 5, 6, 7], [1, 1, 3, 4, 5, 6, 7], [0, 1, 3, 4, 5, 6, 99]):
        _, _, pa = _bits(cache, lens, cu_g, n, 4, cu)
        assert pa.device_status() == K.DEV_LENGTH
    # groups that do not cover the batch in order: nothing is written
    for g in ([0, 2, 5], [1, 3, 6], [0, 7, 6], [0, -1, 6], [0, 2 ** 31 - 1, 6]):
        _, out, pa = _bits(cache, lens, torch.tensor(g, dtype=torch.int32, device="cuda"), n, 4)
        assert pa.device_status() == K.DEV_SEQ and torch.all(out == -7.0)


def test_pages_out_of_range():
    c = build([300], [[30, 40, 50]], [[1, 1, 1]])
    cache, lens, cu_g, n = c[0], c[2], c[3], c[4]
    cache.block_table[:, 9] = cache.cfg.n_pages  # the same in all: the prefix ends before it
    _, out, pa = _bits(cache, lens, cu_g, n, 3)
    assert pa.device_status() == K.DEV_PAGE and shared_of(pa) == [128]
    assert torch.isfinite(out).all()


def test_tables_that_part_early():
    c = build([500], [[30, 40, 50]], [[1, 1, 1]])
    cache, lens, cu_g, n = c[0], c[2], c[3], c[4]
    want = check(cache, lens, cu_g, n, 3, want_shared=[384])
    page = cache.block_table[1, 12].item()
    free = cache.cfg.n_pages - 1
    for b in ("k_main", "v_main"):
        x = cache.buffers[b].view(cache.cfg.L, cache.cfg.n_pages, -1)
        x[:, free] = x[:, page]
    cache.block_table[1, 12] = free  # the same tokens in a page of its own
    out = check(cache, lens, cu_g, n, 3, want_shared=[128])
    assert (out.float() - want.float()).norm() <= 2.0 ** -9 * want.float().norm()


@pytest.mark.parametrize("key", ["rot4_bf16_window", "pre_rope"])
@pytest.mark.parametrize("new", [1, 40])
def test_window_values_that_are_not_finite(key, new):
    """They reach the rows that see them, and no others."""
    kw = FORMATS[key]
    R = kw["residual_window"]

    def spoil(k, v, n_new):
        if len(n_new) == 3 and n_new[1]:  # the sequences' own tokens: the second one's last but three, and a row that all its rows see
            end = n_new[0] + n_new[1]
            v[:, end - 4, 0, 5] = float("nan")
            v[:, end - min(R, 20), 1, 7] = float("inf")

    c = build([300], [[45, 60, 50]], [[new, new, new]], values=spoil, **kw)
    cache, lens, cu_g, n = c[0], c[2], c[3], c[4]
    q, out, cu, pa = attend(cache, lens, cu_g, n, c[5])
    assert pa.device_status() == 0 and shared_of(pa) == [256]
    ref = torch.full_like(q, -7.0)
    cache.chunk_attention(0, 1, q, torch.as_tensor(cu, device="cuda"), q.shape[1], max(n), lens, ref)
    torch.cuda.synchronize()
    for kind in (torch.isnan, lambda x: x == float("inf"), lambda x: x == -float("inf")):
        assert torch.equal(kind(out), kind(ref))
    assert torch.isnan(out[:, new:2 * new]).any() and (out[:, new:2 * new] == float("inf")).any()
    a, b = out.float()[torch.isfinite(ref)], ref.float()[torch.isfinite(ref)]
    assert (a - b).norm() <= 2.0 ** -6 * b.norm()


def test_captured_and_on_two_streams():
    c = build([300, 200], [[30, 40, 50], [20, 10]], [[1, 2, 1], [1, 1]], **ROT4)
    cache, lens, cu_g, n = c[0], c[2], c[3], c[4]
    q, want, cu, pa = attend(cache, lens, cu_g, n, c[5], pad=0)
    cu_d = torch.as_tensor(cu, device="cuda")
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.plan(cu_g, cu_d, int(cu[-1]), max(n), c[5], lens)
        pa.attention(0, 1, q, out)
    q2 = torch.randn_like(q)
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    again = attend(cache, lens, cu_g, n, c[5], q=q2, pad=0)[1]
    assert torch.equal(out, again) and not torch.equal(out, want)
    side = torch.cuda.Stream()
    pb = K.PrefixAttention(cache, 2, int(cu[-1]), stream=side)
    o1, o2 = torch.zeros_like(q), torch.zeros_like(q)
    torch.cuda.synchronize()
    for _ in range(20):
        pa.attention(0, 1, q, o1)
        pb.plan(cu_g, cu_d, int(cu[-1]), max(n), c[5], lens, stream=side)
        pb.attention(0, 1, q, o2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o1, again) and torch.equal(o2, again)


@pytest.mark.parametrize("beams,g", [(2, 4), (2, 17), (40, 8)])
@pytest.mark.parametrize("fmt", [{}, ROT4])
def test_a_call_without_its_plan_writes_nothing(beams, g, fmt):
    """None yet, and one for other sizes: said in the status word."""
    new = g if g > 8 else 1
    c = build([300], [[30 + new + i for i in range(beams)]], [[new] * beams], g=min(g, 8), H_kv=1, **fmt)
    cache, lens, cu_g, n = c[0], c[2], c[3], c[4]
    total = sum(n)
    pa = K.PrefixAttention(cache, 1, total)
    q = torch.randn((1, total, cache.cfg.H_q, 128), device="cuda").half()
    out = torch.full_like(q, -7.0)
    pa.planned = (total, new, total)
    pa.attention(0, 1, q, out)
    torch.cuda.synchronize()
    assert torch.all(out == -7.0) and pa.device_status() == K.DEV_SEQ
    pa.clear_status()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
    pa.plan(cu_g, cu, total, new, total, lens)
    assert pa.device_status() == 0
    for planned in ((total, new, total - 1), (total - 1, new, total - 1), (total, max(1, new - 1), total)):
        if planned == (total, new, total) or planned[2] < planned[1]:
            continue
        pa.planned = planned
        pa.attention(0, 1, q[:, :planned[0]].contiguous(), out[:, :planned[0]].contiguous())
        torch.cuda.synchronize()
        assert pa.device_status() == K.DEV_SEQ
        pa.clear_status()
    assert torch.all(out == -7.0)
    pa.planned = (total, new, total)
    pa.attention(0, 1, q, out)
    torch.cuda.synchronize()
    assert pa.device_status() == 0 and torch.isfinite(out).all() and not (out == -7.0).any()


def test_one_workspace_for_plans_of_several_sizes():
    c = build([300, 150], [[30, 40, 50], [20, 10]], [[3, 2, 1], [1, 4]], **ROT4)
    cache, lens, cu_g, n = c[0], c[2], c[3], c[4]
    pa = K.PrefixAttention(cache, 2, 40)
    for pad in (0, 29, 5, 0):
        check(cache, lens, cu_g, n, 6, pa=pa, pad=pad)
    check(cache, lens, cu_g, [1] * 5, 3, pa=pa, pad=1)


def test_rows_of_many_sequences_in_several_row_tiles():
    """Row tiles that cut sequences, and sequences of more than a row tile, in one group."""
    for D, g, H in ((128, 8, 1), (256, 4, 1), (128, 5, 1)):
        own = [[9 + (13 * i) % 200 for i in range(12)]]
        new = [[1 + (5 * i) % 9 if i != 4 else 61 for i in range(12)]]
        c = build([700], own, new, D=D, H_kv=H, g=g, L=2)
        check(c[0], c[2], c[3], c[4], c[5])


def test_large_batches():
    """More sequences than the plan keeps in shared memory."""
    G, beams = 260, 4
    own = [[1 + (7 * i + 3 * j) % 40 for j in range(beams)] for i in range(G)]
    c = build([(140, 17, 0, 260)[i % 4] for i in range(G)], own, [[1] * beams for _ in range(G)], H_kv=1, g=2)
    check(c[0], c[2], c[3], c[4], c[5])


def test_long_tables():
    """Tables of more columns than a block of the plan looks at: whole, and apart in a later block's share."""
    c = build([5000, 2500], [[30, 40, 50], [20, 300]], [[1, 1, 1], [2, 1]], page_tokens=8, H_kv=1)
    cache, lens, cu_g, n = c[0], c[2], c[3], c[4]
    want = check(cache, lens, cu_g, n, 3, want_shared=[4992, 2432])
    page, free = cache.block_table[1, 300].item(), cache.cfg.n_pages - 1
    for b in ("k_main", "v_main"):
        x = cache.buffers[b].view(cache.cfg.L, cache.cfg.n_pages, -1)
        x[:, free] = x[:, page]
    cache.block_table[1, 300] = free
    out = check(cache, lens, cu_g, n, 3, want_shared=[2304, 2432])
    assert (out.float() - want.float()).norm() <= 2.0 ** -9 * want.float().norm()


def test_some_layers():
    c = build([300], [[30, 40, 50]], [[1, 2, 1]], L=4, **ROT4)
    cache, lens, cu_g, n = c[0], c[2], c[3], c[4]
    q, want, cu, pa = attend(cache, lens, cu_g, n, c[5])
    for layer0, layers in ((0, 1), (1, 2), (3, 1)):
        out = torch.full_like(q[:layers], -7.0)
        pa.attention(layer0, layers, q[layer0:layer0 + layers].contiguous(), out)
        torch.cuda.synchronize()
        ref = want[layer0:layer0 + layers]
        assert pa.device_status() == 0 and torch.equal(out[:, cu[-1]:], ref[:, cu[-1]:])
        assert (out.float() - ref.float()).norm() <= 2.0 ** -9 * ref.float().norm()


@pytest.mark.parametrize("key", ["q4_0", "rot4_d256", "rot4_bf16_window"])
def test_reordered_and_attended_in_turn(key):
    """Reordering, plan and attention over and over with nothing between: every attention sees the tables as they are then."""
    c = build([300, 150], [[40, 90, 170], [20, 60, 130]], [[1] * 3, [1] * 3], **FORMATS[key])
    cache, pool, lens, cu_g, n = c[0], c[1], c[2], c[3], c[4]
    table, refs, lens0 = cache.block_table.clone(), pool.refs.clone(), lens.clone()
    buffers = {k: v.clone() for k, v in cache.buffers.items() if v is not None}
    cu = torch.arange(7, dtype=torch.int32, device="cuda")
    turns = torch.tensor([[1, 2, 0, 2, 0, 1], [1, 0, 2, 0, 2, 1], [0, 1, 2, 2, 1, 0]] * 8, dtype=torch.int32, device="cuda")
    q = torch.randn((1, 6, cache.cfg.H_q, cache.cfg.D), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(DT[cache.cfg.in_dtype])
    pa, outs = K.PrefixAttention(cache, 2, 6), []
    for wait in (False, True):
        cache.block_table.copy_(table)
        pool.refs.copy_(refs)
        lens.copy_(lens0)
        for k, v in buffers.items():
            cache.buffers[k].copy_(v)
        out = torch.zeros((len(turns), *q.shape), dtype=q.dtype, device="cuda")
        torch.cuda.synchronize()
        for i, parents in enumerate(turns):
            pool.reorder(parents, 3, lens)
            pa.plan(cu_g, cu, 6, 1, 3, lens)
            pa.attention(0, 1, q, out[i])
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert pa.device_status() == 0 and pool.device_status() == 0
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and not torch.equal(outs[0][0], outs[0][1])
