"""Chunk attention where a test of its plain cases does not come: batches
above one pass of the tile count, whole sequences against 64 bits at sizes
in earnest, bytes behind the lengths, and errors as large as the roundings
make them, no larger."""

import numpy as np
import pytest

from oracle import kvq_oracle as O
from oracle import serving_oracle as S
from tests.gpu_cases import appended_cache, gpu_buffers_as_oracle
from tests.helpers import oracle_cfg, raw16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402
from tests.test_gpu_chunk_attention import DT, check, queries, workload  # noqa: E402


@pytest.mark.parametrize("name,heads,B,rows", [
    # few rows a sequence: a thread counts a sequence's tiles, and a pass takes 608 (480) of them
    ("gqa8b_hadamard4_paged", (1, 2), 609, 3), ("ctx262k_hadamard4", (1, 1), 500, 2),
    # more than four row tiles: a warp a sequence, and a pass takes 19 (15)
    ("gqa8b_hadamard4_paged", (1, 8), 24, 140), ("ctx262k_hadamard4", (1, 8), 17, 70),
])
def test_batches_of_more_than_one_pass(name, heads, B, rows):
    lengths = [(37 * i) % 90 + rows + 1 for i in range(B)]
    n = [(i * 7) % (rows + 1) for i in range(B)]
    n[B - 1] = n[B // 2] = rows
    check(workload(name, lengths, heads=heads), n, 30, 5)


def expected_square(oc, k, v, r):
    """Expected squared error, over its channels, of one output row whose query r sees the keys k
    and values v (rotated formats: all three in the rotated domain; the turn back keeps
    the sum of squares), from the roundings that the entry states.  A value x rounded to the type is off by at most u |x|,
    and evenly distributed below that at worst: variance (u x)^2 / 3.  To first order
      d o = sum_j p_j (d s_j) (v_j - o) + sum_j p_j (e_j + f_j) v_j + g o,
    d s_j = (sum_c r_c k_jc (a_jc + b_c)) / sqrt(D): a the keys' roundings, b the turned query's (one for
    all keys; rotated formats only), both to fp16, e those of P, f the values', g the output's; all independent."""
    u, uk, D = 2.0 ** -11 if oc.in_dtype == 0 else 2.0 ** -8, 2.0 ** -11, oc.D
    s = k @ r / np.sqrt(D)
    p = np.exp(s - s.max())
    p /= p.sum()
    o = p @ v
    ds = np.sum((k * r) ** 2, -1) / D
    keys = (p ** 2 * ds) @ ((v - o) ** 2)
    if oc.flags & O.ROTATE_K:
        keys = keys + np.sum(((k * r).T @ (p[:, None] * (v - o))) ** 2, 0) / D
    return (uk * uk * keys + u * u * (2 * (p ** 2) @ v ** 2 + o ** 2)).sum() / 3


def expected_error(oc, bufs, rows, lens, window, sinks, table):
    """Root of the sum of the expected squares over rows [(sequence, position, query [H_q, D] in fp64), ..]."""
    g = oc.H_q // oc.H_kv
    d1, d2 = O.hadamard_signs(oc.sign_seed)

    def stored(x, rot):
        return O.rotate_f64(x, d1, d2) if rot else x

    kv = {b: O.dequantize(oc, bufs, 0, b, lens[b], block_table=table) for b in {b for b, _, _ in rows}}
    kv = {b: (stored(k, oc.flags & O.ROTATE_K), stored(v, oc.flags & O.ROTATE_V)) for b, (k, v) in kv.items()}
    total = 0.0
    for b, p, q in rows:
        see = S.visible(p, lens[b], window, sinks)
        r = stored(q, oc.flags & O.ROTATE_K)
        for h in range(oc.H_kv):
            k, v = kv[b][0][see, h], kv[b][1][see, h]
            total += sum(expected_square(oc, k, v, r[h * g + e]) for e in range(g))
    return np.sqrt(total)


@pytest.mark.parametrize("name,heads,T,n,window,sinks", [
    ("gqa8b_hadamard4_paged", (1, 4), 32768, 2048, 4096, 4), ("gqa8b_hadamard4_paged", (2, 4), 20011, 1000, 0, 0),
    ("ctx262k_hadamard4", (1, 6), 20011, 1000, 0, 0), ("gqa8b_hadamard4_paged", (2, 4), 32768, 1, 0, 0),
    ("gqa8b_hadamard4_paged", (2, 4), 32000, 8, 4096, 4)])
def test_long_sequences(name, heads, T, n, window, sinks):
    """Rows picked from a whole call.  (A row sees what the last token of a shorter sequence
    would: these formats keep no 16-bit window, so the cache of the shorter one is a part of this.)"""
    w = workload(name, [T], heads=heads)
    cfg, oc = w.cfg, oracle_cfg(w.cfg)
    cache, lens, _, table = appended_cache(w, with_oracle=False)
    q = queries(cfg, 1, n)
    out = torch.empty_like(q)
    cache.chunk_attention(0, 1, q, torch.tensor([0, n], dtype=torch.int32, device="cuda"), n, n, lens, out, window, sinks)
    torch.cuda.synchronize()
    assert cache.chunk_status() == 0
    bufs = gpu_buffers_as_oracle(cache, oc)
    rows, square = [], 0.0
    for i in sorted({0, 1, 31, 127, 128, n // 2, n - 2, n - 1} & set(range(n))):
        want, bound = S.chunk_attention(oc, bufs, 0, raw16(q[0, i:i + 1]), np.array([0, 1]), [T - n + i + 1], window, sinks, table, True)
        got = O.input_to_f32(raw16(out[0, i:i + 1]), cfg.in_dtype).astype(np.float64)
        assert np.all(np.abs(got - want) <= bound), i
        rows.append((0, T - n + i, O.input_to_f32(raw16(q[0, i]), cfg.in_dtype).astype(np.float64)))
        square += np.sum((got - want) ** 2)
    # (four half steps of the norm, as for benign keys, do not hold a row whose few heavy keys have outlier channels: their
    # roundings move its scores together)
    allowed = expected_error(oc, bufs, rows, [T], window, sinks, table)
    print(f"error {np.sqrt(square):.3e}, expected {allowed:.3e}, ratio {np.sqrt(square) / allowed:.3f}")
    assert np.sqrt(square) <= 1.25 * allowed


@pytest.mark.parametrize("n", [5, 20, 150])
@pytest.mark.parametrize("name,heads", [("gqa8b_hadamard4_paged", (2, 4)), ("llama2_7b_kivi4", (2, 4)), ("ctx262k_hadamard4", (1, 6))])
def test_bytes_behind_the_length_change_nothing(name, heads, n):
    """The buffers' rows, pages' rows and window slots that hold no token, overwritten with ones: the same bits."""
    lengths = [301, 170]
    w = workload(name, lengths, heads=heads, extra=64)
    cfg, oc = w.cfg, oracle_cfg(w.cfg)
    cache, lens, _, table = appended_cache(w, with_oracle=False)
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    q = queries(cfg, 1, 2 * n)
    kinds = ((0, 0), (64, 1), (90, 33), (1, 0))

    def run():
        outs = []
        for window, sinks in kinds:
            outs.append(torch.empty_like(q))
            cache.chunk_attention(0, 1, q, cu, 2 * n, n, lens, outs[-1], window, sinks)
        torch.cuda.synchronize()
        assert cache.chunk_status() == 0
        return outs

    clean = run()
    spoiled = 0
    shapes = O.buffer_shapes(oc)
    for buf in ("k_main", "v_main", "k_resid", "v_resid"):
        t = cache.buffers[buf]
        if t is None:
            continue
        shape, dt = shapes[buf]
        x = t.view(torch.int16 if dt == np.uint16 else torch.uint8).view(shape)
        # per-channel rows hold 32 tokens
        per = 32 if (cfg.k_fmt if buf[0] == "k" else cfg.v_fmt).axis == K.AXIS_CHANNEL and buf.endswith("main") else 1
        for b, T in enumerate(lengths):
            qe = O.q_end(oc, T)
            if buf.endswith("resid"):
                held = {t % x.shape[3] for t in range(qe, T)}
                rows = [(b, r) for r in range(x.shape[3]) if r not in held]
            elif cfg.page_tokens:
                rows = [(int(table[b, t // cfg.page_tokens]), t % cfg.page_tokens) for t in range(qe, cfg.max_T)
                        if table[b, t // cfg.page_tokens] >= 0]
            else:
                rows = [(b, r) for r in range(-(-qe // per), x.shape[3])]
            for i, r in rows:
                x[0, i, :, r] = -1 if dt == np.uint16 else 255
                spoiled += 1
    assert spoiled > 0
    for a, b, kind in zip(clean, run(), kinds):
        assert torch.equal(a, b), kind


@pytest.mark.parametrize("n", [4, 20, 150])
@pytest.mark.parametrize("name,heads,dt", [
    ("llama2_7b_kivi4", (2, 4), K.DT_F16), ("llama2_7b_kivi4", (2, 4), K.DT_BF16), ("gqa8b_hadamard4_paged", (2, 4), K.DT_F16),
    ("gqa8b_hadamard4_paged", (2, 4), K.DT_BF16), ("ctx262k_hadamard4", (1, 6), K.DT_BF16), ("ctx262k_hadamard4", (1, 6), K.DT_F16),
    ("q8_0_mha_1k", (2, 2), K.DT_F16)])
def test_errors_are_those_of_the_stated_roundings(name, heads, dt, n):
    """A quarter above the root of the expected squares, which itself takes every rounding at its worst
    spread: a rounding more, or one bit less anywhere, is above."""
    w = workload(name, [400, 170], heads=heads, in_dtype=dt)
    cfg, oc = w.cfg, oracle_cfg(w.cfg)
    cache, lens, _, table = appended_cache(w, with_oracle=False)
    new = [n, n // 2]
    cu = np.array([0, n, n + n // 2], np.int32)
    q = queries(cfg, 1, int(cu[-1]))
    out = torch.empty_like(q)
    cache.chunk_attention(0, 1, q, torch.as_tensor(cu, device="cuda"), int(cu[-1]), n, lens, out)
    bufs = gpu_buffers_as_oracle(cache, oc)
    want = S.chunk_attention(oc, bufs, 0, raw16(q[0]), cu, w.lengths, 0, 0, table)
    got = O.input_to_f32(raw16(out[0]), dt).astype(np.float64)
    qf = O.input_to_f32(raw16(q[0]), dt).astype(np.float64)
    rows = [(b, w.lengths[b] - new[b] + i, qf[cu[b] + i]) for b in range(2) for i in range(new[b])]
    err, allowed = np.linalg.norm(got - want), expected_error(oc, bufs, rows, w.lengths, 0, 0, table)
    print(f"error {err:.3e}, expected {allowed:.3e}, ratio {err / allowed:.3f}")
    assert err <= 1.25 * allowed


@pytest.mark.parametrize("n", [3, 20, 150])
@pytest.mark.parametrize("name,kw", [
    ("llama2_7b_kivi4", dict()), ("llama2_7b_kivi4_zp", dict()), ("gqa8b_hadamard4_paged", dict(residual_window=37)),
    ("q8_0_mha_1k", dict(residual_window=20)), ("mistral7b_hotcold", dict(hot_window=96, residual_window=40)),
    ("q4_0_mha_1k", dict(flags=K.K_PRE_ROPE))])
@pytest.mark.parametrize("size", [3e4, 1e-3])
def test_bf16_keys_out_of_fp16_s_range(name, kw, n, size):
    """Keys of some 10^5 (queries as much smaller) and of 10^-3, quantized and in the window, against the per-value bound of bf16 keys."""
    w = workload(name, [300], heads=(2, 4), in_dtype=K.DT_BF16, **kw)
    cfg, oc = w.cfg, oracle_cfg(w.cfg)
    T = 300
    table = None
    if cfg.page_tokens:
        table = torch.arange(cfg.max_pages_per_seq, dtype=torch.int32).view(1, -1)
    cache = K.KVCache(cfg, "cuda", block_table=table)
    gen = torch.Generator(device="cuda").manual_seed(11)
    k, v, q = (torch.randn((1, m, h, cfg.D), generator=gen, device="cuda") for m, h in ((T, cfg.H_kv), (T, cfg.H_kv), (n, cfg.H_q)))
    k, v, q = (k * size).bfloat16(), v.bfloat16(), (q / size).bfloat16()
    assert size < 1 or k.abs().max() > 65504
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu_T, cu = (torch.tensor([0, x], dtype=torch.int32, device="cuda") for x in (T, n))
    cache.append(0, 1, k, v, cu_T, lens, T, T)
    cache.commit_lengths(cu_T, lens)
    out = torch.empty_like(q)
    cache.chunk_attention(0, 1, q, cu, n, n, lens, out)
    torch.cuda.synchronize()
    assert cache.chunk_status() == 0
    bufs = gpu_buffers_as_oracle(cache, oc)
    want, bound = S.chunk_attention(oc, bufs, 0, raw16(q[0]), np.array([0, n]), [T], 0, 0, None if table is None else table.numpy(), True,
                                    4.0 if cfg.flags & (K.ZP_K | K.ZP_V) else 2.0)
    err = np.abs(O.input_to_f32(raw16(out[0]), 1).astype(np.float64) - want)
    assert np.all(err <= bound), float(np.max(err / bound))


@pytest.mark.parametrize("n", [3, 20, 150])
@pytest.mark.parametrize("name,dt", [("gqa8b_hadamard4_paged", K.DT_F16), ("gqa8b_hadamard4_paged", K.DT_BF16),
                                     ("ctx262k_hadamard4", K.DT_F16), ("ctx262k_tbq4", K.DT_BF16)])
def test_turned_queries_past_fp16_s_range(name, dt, n):
    """A query along a row of the transform gathers in one channel: 8000 becomes 90500."""
    w = workload(name, [300], heads=(1, 4), in_dtype=dt)
    cfg, oc = w.cfg, oracle_cfg(w.cfg)
    T = 300
    table = torch.arange(cfg.max_pages_per_seq, dtype=torch.int32).view(1, -1) if cfg.page_tokens else None
    cache = K.KVCache(cfg, "cuda", block_table=table)
    gen = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn((1, T, 1, cfg.D), generator=gen, device="cuda") for _ in range(2))
    k, v = (k * 1e-3).to(DT[dt]), v.to(DT[dt])
    q = torch.randn((1, n, 4, cfg.D), generator=gen, device="cuda") * 8
    rows = O.rotation_matrix_f64(*O.hadamard_signs(oc.sign_seed))  # entries of +-1 / sqrt(128)
    q[..., :128] = torch.as_tensor(np.sign(rows[np.arange(4 * n) % 128]).reshape(1, n, 4, 128) * 8000.0, device="cuda")
    q = q.to(DT[dt])
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu_T, cu = (torch.tensor([0, x], dtype=torch.int32, device="cuda") for x in (T, n))
    cache.append(0, 1, k, v, cu_T, lens, T, T)
    cache.commit_lengths(cu_T, lens)
    out = torch.empty_like(q)
    cache.chunk_attention(0, 1, q, cu, n, n, lens, out)
    torch.cuda.synchronize()
    bufs = gpu_buffers_as_oracle(cache, oc)
    want, bound = S.chunk_attention(oc, bufs, 0, raw16(q[0]), np.array([0, n]), [T], 0, 0, None if table is None else table.numpy(), True)
    err = np.abs(O.input_to_f32(raw16(out[0]), dt).astype(np.float64) - want)
    assert np.all(err <= bound), float(np.max(err / bound))


CH = K.AXIS_CHANNEL


@pytest.mark.parametrize("dt", [K.DT_F16, K.DT_BF16])
@pytest.mark.parametrize("kw", [
    dict(flags=0), dict(flags=0, k_fmt=K.Fmt(8, 32, CH), k_cold=K.Fmt(4, 32, CH)), dict(flags=0, k_fmt=K.Fmt(3, 32, CH), k_cold=K.Fmt(8, 32, CH)),
    dict(flags=K.ZP_K | K.ZP_V), dict(flags=K.ZP_K, v_fmt=K.Fmt(8, 32), v_cold=K.Fmt(3, 32)),
    dict(flags=K.K_PRE_ROPE, k_fmt=K.Fmt(8, 32, CH), k_cold=K.Fmt(2, 32, CH)),
    dict(flags=0, k_fmt=K.Fmt(4, 32), k_cold=K.Fmt(8, 32), v_fmt=K.Fmt(4, 32, CH), v_cold=K.Fmt(2, 32, CH))])
def test_two_tiers_of_every_width(dt, kw):
    """Hot and cold keys share one factor, whichever of them is the wider."""
    w = workload("mistral7b_hotcold", [391, 200], L=1, heads=(2, 4), hot_window=96, residual_window=40, in_dtype=dt, **kw)
    for n in ([3, 1], [20, 9], [150, 33]):
        check(w, n)
        check(w, n, window=150, sinks=40)
