"""kvq_chunk_attention against fp64 attention over the dequantized cache.  The
tolerance of every output value is the rounding bound of
oracle.serving_oracle.chunk_attention, worked out from the inputs."""

from dataclasses import replace

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
from bit_kv_cache_04_gb300 import workloads as W  # noqa: E402

DT = {0: torch.float16, 1: torch.bfloat16}


def workload(name, lengths, L=1, heads=None, extra=0, **kw):
    w = W.make(name)
    if heads:
        kw.update(H_kv=heads[0], H_q=heads[0] * heads[1])
    w = W.Workload(w.name, replace(w.cfg, **kw), w.lengths, w.values, w.extra_tokens)
    return w.scaled(L=L, lengths=lengths, extra=extra)


def queries(cfg, L, total, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((L, total, cfg.H_q, cfg.D), generator=g, device="cuda").to(DT[cfg.in_dtype])


def check(w, n_new, window=0, sinks=0, chunks=None, layer0=0, n_layers=None, pad=3):
    """Appends w's tokens, attends with the last n_new[b] of each sequence."""
    cfg = w.cfg
    oc = oracle_cfg(cfg)
    n_layers = n_layers or cfg.L - layer0
    cache, lens, _, table = appended_cache(w, chunks=chunks, with_oracle=False)
    cu = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
    total = int(cu[-1]) + pad
    q = queries(cfg, n_layers, total)
    out = torch.full_like(q, -7.0)
    cache.chunk_attention(layer0, n_layers, q, torch.as_tensor(cu, device="cuda"), total, max(n_new), lens, out, window, sinks)
    torch.cuda.synchronize()
    ws = cache.chunk_workspace[:4].view(torch.int32).item()
    assert ws == 0, ws
    assert torch.all(out[:, cu[-1]:] == -7.0)  # rows of no sequence stay as they were
    bufs = gpu_buffers_as_oracle(cache, oc)
    worst = 0.0
    # roundings of a key on its way to the products: to the dtype, and of a turned
    # query to the dtype; asymmetric bf16 blocks round scale and zero parts on the way
    roundings = 2.0 if not (cfg.flags & (K.ZP_K | K.ZP_V)) else 4.0
    for l in range(n_layers):
        want, bound = S.chunk_attention(oc, bufs, layer0 + l, raw16(q[l]), cu, w.lengths, window, sinks, table, True, roundings)
        rows = slice(0, int(cu[-1]))
        got = O.input_to_f32(raw16(out[l]), cfg.in_dtype).astype(np.float64)[rows]
        err = np.abs(got - want[rows])
        assert np.all(err <= bound[rows]), (float(np.max(err / bound[rows])), np.unravel_index(np.argmax(err / bound[rows]), err.shape))
        worst = max(worst, float(np.linalg.norm(got - want[rows]) / np.linalg.norm(want[rows])))
    # the 2-norm of random roundings: output (u / sqrt 3), values and probabilities (u / sqrt 3 each, averaged over many
    # keys), scores; four half steps of the dtype hold them all
    assert worst <= 4 * (2.0 ** -11 if cfg.in_dtype == 0 else 2.0 ** -8), worst
    return cache, lens, q, out


FORMATS = {
    "kivi4": ("llama2_7b_kivi4", dict(heads=(2, 4))),
    "kivi4_bf16": ("llama2_7b_kivi4", dict(heads=(2, 4), in_dtype=K.DT_BF16)),
    "kivi4_zp": ("llama2_7b_kivi4_zp", dict(heads=(2, 4))),
    "kivi2_zp_bf16": ("llama2_7b_kivi2_zp", dict(heads=(2, 3), in_dtype=K.DT_BF16)),
    "rot4_paged": ("gqa8b_hadamard4_paged", dict(heads=(2, 4))),
    "rot4_paged_bf16_window": ("gqa8b_hadamard4_paged", dict(heads=(2, 4), in_dtype=K.DT_BF16, residual_window=37)),
    "rot4_d256": ("ctx262k_hadamard4", dict(heads=(1, 6))),
    "rot4_d256_fp16": ("ctx262k_hadamard4", dict(heads=(2, 3), in_dtype=K.DT_F16)),
    "rot3_d256": ("ctx262k_hadamard3", dict(heads=(1, 6))),
    "tbq4_d256": ("ctx262k_tbq4", dict(heads=(1, 6))),
    "tbq4_fp16_d128": ("ctx262k_tbq4", dict(heads=(2, 2), in_dtype=K.DT_F16, D=128)),
    "q8_0": ("q8_0_mha_1k", dict(heads=(2, 1))),
    "q8_0_bf16_d256": ("q8_0_mha_1k", dict(heads=(2, 8), in_dtype=K.DT_BF16, D=256)),
    "q4_0_paged_p8": ("q4_0_mha_1k", dict(heads=(2, 2), page_tokens=8, residual_window=9)),
    "q4_0_paged_p1": ("q4_0_mha_1k", dict(heads=(2, 2), page_tokens=1)),
    "q8_0_paged_p5_zp4": ("q4_0_mha_1k", dict(heads=(2, 2), page_tokens=5, flags=K.ZP_K | K.ZP_V)),
    "hotcold": ("mistral7b_hotcold", dict(heads=(2, 4), hot_window=96, residual_window=40)),
    "hotcold_bf16_d256": ("mistral7b_hotcold", dict(heads=(1, 4), hot_window=64, residual_window=0, in_dtype=K.DT_BF16, D=256)),
    "token_pre_rope": ("q8_0_mha_1k", dict(heads=(2, 4), flags=K.K_PRE_ROPE, residual_window=20)),
    "token4_pre_rope_paged": ("q4_0_mha_1k", dict(heads=(2, 4), flags=K.K_PRE_ROPE, page_tokens=16)),
    "v_per_channel": ("llama2_7b_kivi4", dict(heads=(2, 4), v_fmt=K.Fmt(4, 32, K.AXIS_CHANNEL), k_fmt=K.Fmt(4, 32))),
    "both_per_channel": ("llama2_7b_kivi4", dict(heads=(1, 4), v_fmt=K.Fmt(2, 32, K.AXIS_CHANNEL),
                                                 k_fmt=K.Fmt(8, 32, K.AXIS_CHANNEL), residual_window=0)),
    "mixed_group": ("q4_0_mha_1k", dict(heads=(2, 2), k_fmt=K.Fmt(3, 32), v_fmt=K.Fmt(8, 128))),
    "rotate_v_only": ("q4_0_mha_1k", dict(heads=(2, 2), flags=K.ROTATE_V, v_fmt=K.Fmt(2, 128), residual_window=11)),
    "two_bit": ("q4_0_mha_1k", dict(heads=(2, 2), k_fmt=K.Fmt(2, 32), v_fmt=K.Fmt(2, 32))),
}


@pytest.mark.parametrize("key", FORMATS)
@pytest.mark.parametrize("new", ["one", "few", "many"])
def test_formats(key, new):
    name, kw = FORMATS[key]
    w = workload(name, [391, 64, 1, 160], L=1, **kw)
    if w.cfg.batch and key.startswith("hotcold"):
        w = workload(name, [391, 200, 1, 160], L=1, **kw)
    n = {"one": [1, 1, 1, 1], "few": [7, 3, 1, 0], "many": [150, 64, 0, 33]}[new]
    check(w, n)
    check(w, n, window=45, sinks=3)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 5), (31, 0), (32, 4), (128, 128), (129, 1), (300, 33), (10 ** 9, 7),
                                          (0, 9), (64, 10 ** 9), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows_and_sinks(window, sinks):
    check(workload("llama2_7b_kivi4", [700, 129], heads=(2, 4)), [9, 2], window, sinks)
    check(workload("gqa8b_hadamard4_paged", [700, 129], heads=(2, 4)), [200, 129], window, sinks)
    check(workload("ctx262k_hadamard4", [333], heads=(1, 6)), [70], window, sinks)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 385])
def test_lengths(T):
    for name, heads in (("llama2_7b_kivi4", (2, 4)), ("gqa8b_hadamard4_paged", (1, 8)), ("ctx262k_hadamard4", (1, 1))):
        for n in sorted({1, min(T, 5), T}):
            check(workload(name, [T], heads=heads), [n])


@pytest.mark.parametrize("g", [1, 2, 3, 5, 7, 8])
def test_group_sizes_and_row_tiles(g):
    for n in (1, 4, 8, 16, 17, 33, 43, 65, 129):
        check(workload("gqa8b_hadamard4_paged", [300, 140], heads=(2, g)), [n, max(1, n // 3)], 70, 2)


def test_layers_and_multi_layer_calls():
    w = workload("gqa8b_hadamard4_paged", [200, 90], L=4, heads=(2, 4))
    check(w, [5, 2])
    check(w, [5, 2], layer0=1, n_layers=2)
    check(workload("ctx262k_hadamard4", [200], L=3, heads=(2, 3)), [50], layer0=2, n_layers=1)


def test_many_sequences_and_empty_ones():
    lengths = [(37 * i) % 211 + 1 for i in range(70)]
    n = [min(t, i % 4) for i, t in enumerate(lengths)]
    check(workload("gqa8b_hadamard4_paged", lengths, heads=(1, 4)), n)
    check(workload("llama2_7b_kivi4", lengths, heads=(1, 2)), n, 50, 4)


def test_appended_token_by_token():
    check(workload("mistral7b_hotcold", [300, 150], heads=(1, 4), hot_window=64, residual_window=40), [6, 3], chunks=[100, 1, 33, 7, 1, 1, 64])


def test_long_context():
    """A long split: many tiles per sequence, joined from many blocks."""
    check(workload("gqa8b_hadamard4_paged", [6000], heads=(1, 4)), [3])
    check(workload("llama2_7b_kivi4", [5003, 40], heads=(1, 4)), [40, 40], 2500, 4)


def test_same_bits_again_and_on_a_side_stream():
    w = workload("gqa8b_hadamard4_paged", [3000, 500], heads=(2, 4))
    cache, lens, q, out = check(w, [4, 4], pad=0)
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    again = torch.empty_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        cache.chunk_attention(0, 1, q, cu, 8, 4, lens, again, stream=s)
    s.synchronize()
    assert torch.equal(again, out)
    # two workspaces: calls side by side
    ws = [cache.make_chunk_workspace() for _ in range(2)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in ws], [torch.empty_like(out) for _ in ws]
    for _ in range(5):
        for st, o, x in zip(streams, outs, ws):
            cache.chunk_attention(0, 1, q, cu, 8, 4, lens, o, stream=st, workspace=x)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)


def test_captured_and_replayed_with_new_lengths():
    w = workload("gqa8b_hadamard4_paged", [300, 200], heads=(2, 4), extra=0)
    cache, lens, q, _ = check(w, [2, 2], pad=0)
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.chunk_attention(0, 1, q, cu, 4, 2, lens, out, 100, 2)
    for a, b, c in ((300, 200, [0, 2, 4]), (17, 111, [0, 1, 3]), (1, 2, [0, 0, 2])):
        lens.copy_(torch.tensor([a, b], dtype=torch.int32))
        cu.copy_(torch.tensor(c, dtype=torch.int32))
        out.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        oc = oracle_cfg(w.cfg)
        want, bound = S.chunk_attention(oc, gpu_buffers_as_oracle(cache, oc), 0, raw16(q[0]), c, [a, b], 100, 2,
                                        cache.block_table.cpu().numpy(), True)
        got = O.input_to_f32(raw16(out[0]), 0).astype(np.float64)
        assert np.all(np.abs(got - want)[: c[2]] <= bound[: c[2]])
        assert np.all(got[c[2]:] == -7)


def test_not_finite_window_values_reach_only_rows_that_see_them():
    """The newest tokens sit in the 16-bit window.  A NaN or infinity in one of them must not reach
    earlier queries of the chunk, nor queries whose window has passed it."""
    for dt in (0, 1):
        w = workload("llama2_7b_kivi4", [200], heads=(2, 4), in_dtype=dt)
        cache, lens, q, out = check(w, [60], pad=0)
        cu = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
        ring = 160
        for window, sinks in ((0, 0), (20, 0)):
            clean = torch.empty_like(out)
            cache.chunk_attention(0, 1, q, cu, 60, 60, lens, clean, window, sinks)
            for name in ("k_resid", "v_resid"):
                for bad in (float("nan"), float("inf"), float("-inf")):
                    buf = cache.buffers[name].view(DT[dt]).view(1, 1, 2, ring, 128)
                    keep = buf[0, 0, 1, 165 % ring, 9].clone()
                    buf[0, 0, 1, 165 % ring, 9] = bad
                    got = torch.empty_like(out)
                    cache.chunk_attention(0, 1, q, cu, 60, 60, lens, got, window, sinks)
                    buf[0, 0, 1, 165 % ring, 9] = keep
                    see = [165 <= 140 + i and (not window or 165 > 140 + i - window) for i in range(60)]
                    for i in range(60):
                        assert torch.equal(got[0, i, :4], clean[0, i, :4])  # the other kv head
                        if not see[i]:
                            assert torch.equal(got[0, i], clean[0, i]), (name, bad, i)
                        elif name == "v_resid":
                            hit = got[0, i, 4:, 9]
                            assert torch.all(torch.isnan(hit)) if bad != bad else torch.all(hit == bad)
                            assert torch.equal(got[0, i, 4:, :9], clean[0, i, 4:, :9])
                        elif bad != bad:
                            assert torch.all(torch.isnan(got[0, i, 4:]))


def test_not_finite_window_values_among_few_rows():
    """The same with 28 rows a head, which share their exponentials' warps."""
    for dt in (0, 1):
        w = workload("llama2_7b_kivi4", [200], heads=(2, 4), in_dtype=dt)
        cache, lens, q, out = check(w, [7], pad=0)
        cu = torch.tensor([0, 7], dtype=torch.int32, device="cuda")
        for window in (0, 3):
            clean = torch.empty_like(out)
            cache.chunk_attention(0, 1, q, cu, 7, 7, lens, clean, window, 0)
            see = [196 <= 193 + i and (not window or 196 > 193 + i - window) for i in range(7)]
            for name in ("k_resid", "v_resid"):
                for bad in (float("nan"), float("inf"), float("-inf")):
                    buf = cache.buffers[name].view(DT[dt]).view(2, 160, 128)
                    keep = buf[1, 196 % 160, 9].clone()
                    buf[1, 196 % 160, 9] = bad
                    got = torch.empty_like(out)
                    cache.chunk_attention(0, 1, q, cu, 7, 7, lens, got, window, 0)
                    buf[1, 196 % 160, 9] = keep
                    assert torch.equal(got[0, :, :4], clean[0, :, :4])  # the other kv head
                    for i in range(7):
                        mine, ref = got[0, i, 4:], clean[0, i, 4:]
                        if name == "v_resid" and see[i]:
                            assert torch.all(torch.isnan(mine[:, 9])) if bad != bad else torch.all(mine[:, 9] == bad)
                            assert torch.equal(mine[:, :9], ref[:, :9]) and torch.equal(mine[:, 10:], ref[:, 10:])
                        elif see[i] and bad != bad:
                            assert torch.all(torch.isnan(mine))
                        elif not see[i]:
                            # an infinite score of another row moves the group's references: same values, P's
                            # smallest roundings apart; otherwise the same bits
                            assert torch.equal(mine, ref) if name == "v_resid" or bad != bad else torch.isfinite(mine).all()


@pytest.mark.parametrize("n", [1, 5, 20, 40])
def test_a_score_of_minus_infinity_counts_nothing(n):
    """The last token is alone in its tile, and its key makes scores of -inf and +inf: the first leave it out, the second are NaN."""
    for dt in (0, 1):
        w = workload("llama2_7b_kivi4", [257], heads=(2, 4), in_dtype=dt)
        cache, lens, q, _ = check(w, [n], pad=0)
        cache.buffers["k_resid"].view(DT[dt]).view(2, 160, 128)[1, 256 % 160, 9] = float("-inf")
        got = torch.empty_like(q)
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        cache.chunk_attention(0, 1, q, cu, n, n, lens, got)
        last = raw16(q[0, n - 1:])
        oc = oracle_cfg(w.cfg)
        bufs = gpu_buffers_as_oracle(cache, oc)
        want, bound = S.chunk_attention(oc, bufs, 0, last, np.array([0, 1]), [256], with_bound=True)  # without the token
        x = O.input_to_f32(raw16(got[0, n - 1:]), dt).astype(np.float64)
        for h in range(4, 8):
            if float(q[0, n - 1, h, 9]) > 0:
                assert np.all(np.abs(x[0, h] - want[0, h]) <= bound[0, h]), h
            else:
                assert np.all(np.isnan(x[0, h])), h


def test_stale_bytes_past_the_length_do_not_matter():
    w = workload("gqa8b_hadamard4_paged", [300, 40], heads=(2, 4), extra=64)
    cache, lens, q, out = check(w, [5, 5], pad=0)
    cu = torch.tensor([0, 5, 10], dtype=torch.int32, device="cuda")
    cfg = w.cfg
    for name in ("k_main", "v_main"):  # NaN scales in every row past the lengths
        pool = cache.buffers[name].view(1, cfg.n_pages, 2, 16, 66)
        for b, T in enumerate(w.lengths):
            for t in range(T, cfg.max_T):
                page = int(cache.block_table[b, t // 16])
                if page >= 0:
                    pool[0, page, :, t % 16] = 255
    got = torch.empty_like(out)
    for window in (0, 64):
        ref = torch.empty_like(out)
        cache.chunk_attention(0, 1, q, cu, 10, 5, lens, got, window, 1)
        assert torch.isfinite(got).all()
        if not window:
            assert torch.equal(got, out)


def test_bad_device_values_are_flagged_and_passed_over():
    w = workload("gqa8b_hadamard4_paged", [300, 100, 50], heads=(2, 4))
    cache, lens, q, _ = check(w, [2, 2, 2], pad=0)
    good = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda")
    ref = torch.empty_like(q)
    cache.chunk_attention(0, 1, q, good, 6, 2, lens, ref)
    # a sequence that is passed over takes part like one without new tokens: the others' sums are cut alike
    less = torch.empty_like(q[:, :4])
    cache.chunk_attention(0, 1, q[:, [0, 1, 4, 5]].contiguous(), torch.tensor([0, 2, 2, 4], dtype=torch.int32, device="cuda"), 4, 2,
                          lens, less)

    def run(lens=lens, cu=good, bit=K.DEV_LENGTH, max_q=2):
        out = torch.full_like(q, -7)
        cache.chunk_attention(0, 1, q, cu, 6, max_q, lens, out)
        torch.cuda.synchronize()
        status = cache.chunk_workspace[:4].view(torch.int32)
        assert status.item() == bit
        status.zero_()
        return out

    for T in (-1, w.cfg.max_T + 1, 1, 2 ** 31 - 1, -2 ** 31):
        l = lens.clone()
        l[1] = T
        out = run(l)
        assert torch.equal(out[0, :2], less[0, :2]) and torch.equal(out[0, 4:], less[0, 2:]) and torch.all(out[0, 2:4] == -7)
    out = run(cu=torch.tensor([0, 2, 5, 6], dtype=torch.int32, device="cuda"))  # more rows than max_q
    assert torch.equal(out[0, :2], less[0, :2]) and torch.all(out[0, 2:5] == -7)
    out = run(cu=torch.tensor([0, 4, 2, 4], dtype=torch.int32, device="cuda"), max_q=4)  # not ascending
    assert torch.all(out[0, 4:] == -7)
    run(cu=torch.tensor([0, 2, 4, 900], dtype=torch.int32, device="cuda"), max_q=4)  # past total_q
    run(cu=torch.tensor([-2, 2, 4, 6], dtype=torch.int32, device="cuda"), max_q=4)
    cache.block_table[0, 3] = w.cfg.n_pages
    out = run(bit=K.DEV_PAGE)
    assert torch.equal(out[0, 2:], ref[0, 2:]) and torch.isfinite(out).all()
