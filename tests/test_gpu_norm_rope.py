"""kvq_qk_norm_rope against the 64-bit definition.

Tolerance of one output value, derived before the first run: with u the
dtype's half step, the result is rounded once (u |y|); before that everything
is fp32.  The norm factor carries the sum's error (at most 8 + 5 additions of
positive terms and a multiply: 14 x 2^-24, halved by the root), the root, the divide and two products (4 x 2^-24);
the angle is a 64-bit fraction cut to 32 bits and rounded to fp32 (2^-25 half turns, pi 2^-25 radians), cos and sin are
off by 2^-23, times the factor m; a turn adds two products and a sum.  Together below 2e-6 (|a| + |b|) m for a pair (a, b)
of normed values; u covers bf16 / fp16.  fp16 results below 2^-14 round to a multiple of 2^-24: half of
that is added."""

import numpy as np
import pytest

from oracle import kvq_oracle as O
from oracle import serving_oracle as S
from tests.helpers import raw16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402

DT = {0: torch.float16, 1: torch.bfloat16}
SCALE = {K.ROPE_NONE: {}, K.ROPE_LINEAR: dict(factor=4.0), K.ROPE_NTK: dict(factor=8.0),
         K.ROPE_YARN: dict(factor=8.0, low=1.0, high=32.0, original_len=8192),
         K.ROPE_BANDS: dict(factor=8.0, low=1.0, high=4.0, original_len=8192)}


def _cfg(hq, hk, D, dt):
    return K.Config(L=1, H_kv=hk, H_q=hq, D=D, batch=1, max_T=1, in_dtype=dt)


def _pair_of(rot, inter, D):
    i = np.arange(D)
    p = i.copy()
    if inter:
        p[:rot] = i[:rot] ^ 1
    else:
        p[:rot] = (i[:rot] + rot // 2) % rot
    return p


def _check(x, w, pos, got, dt, plan_kw, eps):
    """x, got: tensors [n, h, D]."""
    D = x.shape[-1]
    u = 2.0 ** -11 if dt == 0 else 2.0 ** -8
    y = O.input_to_f32(raw16(x), dt).astype(np.float64)
    if w is not None:
        y = S.rms_norm(y, O.input_to_f32(raw16(w), dt).astype(np.float64), eps)
    m, pair = 1.0, np.arange(D)
    want = y
    if plan_kw is not None:
        rot = plan_kw.get("rot_dim", D)
        kw = {k: v for k, v in plan_kw.items() if k not in ("rot_dim", "interleaved")}
        f, m = S.rope_frequencies(rot, kw.pop("theta", 10000.0), kw.pop("scaling", K.ROPE_NONE), **kw)
        want = S.turn(y, pos.cpu().numpy(), f, m, bool(plan_kw.get("interleaved")))
        pair = _pair_of(rot, plan_kw.get("interleaved"), D)
    tol = u * np.abs(want) + 2e-6 * max(1.0, m) * (np.abs(y) + np.abs(y[..., pair])) + (2.0 ** -25 if dt == 0 else 0)
    g = O.input_to_f32(raw16(got), dt).astype(np.float64)
    assert np.all(np.abs(g - want) <= tol), np.max(np.abs(g - want) - tol)


def _x(shape, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda") * 3
    x[..., 5] *= 20
    return x.to(DT[dt])


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("rot", ["all", 64, 34, 2, 126])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_forms(dt, D, rot, inter, norm):
    rot = D if rot == "all" else rot
    n, hq, hk = 37, 6, 2
    scaling = list(SCALE)[(rot + D + norm) % 5]
    kw = dict(rot_dim=rot, interleaved=inter, theta=500000.0, scaling=scaling, **SCALE[scaling])
    q, k = _x((n, hq, D), dt, 1), _x((n, hk, D), dt, 2)
    qw, kw_ = (_x((D,), dt, 3), _x((D,), dt, 4)) if norm else (None, None)
    pos = torch.randint(0, 1 << 20, (n,), dtype=torch.int32, device="cuda")
    pos[0], pos[1], pos[2], pos[3] = 0, (1 << 31) - 1, -5, 1
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    K.qk_norm_rope(_cfg(hq, hk, D, dt), q, k, pos, qo, ko, plan=K.rope_plan(D, **kw), q_weight=qw, k_weight=kw_, eps=1e-5)
    _check(q, qw, pos, qo, dt, kw, 1e-5)
    _check(k, kw_, pos, ko, dt, kw, 1e-5)


@pytest.mark.parametrize("n,hq,hk", [(1, 1, 1), (1, 32, 8), (2, 24, 4), (1000, 5, 5), (4001, 8, 1), (3, 200, 25)])
def test_sizes(n, hq, hk):
    for D, dt in ((128, 0), (256, 1)):
        q, k = _x((n, hq, D), dt, n), _x((n, hk, D), dt, n + 1)
        w = _x((D,), dt, 5)
        pos = torch.arange(n, dtype=torch.int32, device="cuda") * 7
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        K.qk_norm_rope(_cfg(hq, hk, D, dt), q, k, pos, qo, ko, plan=K.rope_plan(D), q_weight=w)
        _check(q, w, pos, qo, dt, {}, 1e-6)
        _check(k, None, pos, ko, dt, {}, 1e-6)


def test_strides_alignment_in_place_and_halves():
    n, hq, hk, D, dt = 19, 4, 2, 128, 1
    cfg, plan = _cfg(hq, hk, D, dt), K.rope_plan(D, 64)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") + 100
    for pad in (0, 1, 3, 8):  # a fused projection whose rows are padded: odd strides and addresses
        flat = _x((n, (hq + 2 * hk) * D + pad), dt, pad)
        flat = flat.flatten()[: n * flat.shape[1] - 0].view(n, -1)
        q = flat[:, pad:pad + hq * D].unflatten(1, (hq, D))
        k = flat[:, pad + hq * D:pad + (hq + hk) * D].unflatten(1, (hk, D))
        w = _x((D + 1,), dt, 9)[1:]  # a weight at an odd address
        qo, ko = torch.empty((n, hq, D), dtype=DT[dt], device="cuda"), torch.empty((n, hk, D), dtype=DT[dt], device="cuda")
        K.qk_norm_rope(cfg, q, k, pos, qo, ko, plan=plan, q_weight=w, k_weight=w)
        _check(q, w, pos, qo, dt, dict(rot_dim=64), 1e-6)
        _check(k, w, pos, ko, dt, dict(rot_dim=64), 1e-6)
    heads_first = _x((hq, n, D), dt, 3).transpose(0, 1)
    K.qk_norm_rope(cfg, heads_first, None, pos, qo, None, plan=plan)
    _check(heads_first, None, pos, qo, dt, dict(rot_dim=64), 1e-6)
    k = _x((n, hk, D), dt, 4)
    k0 = k.clone()
    K.qk_norm_rope(cfg, None, k, pos, None, k, plan=plan, k_weight=w)  # in place, keys alone
    _check(k0, w, pos, k, dt, dict(rot_dim=64), 1e-6)
    q = _x((n, hq, D), dt, 5)
    K.qk_norm_rope(cfg, q, None, None, qo, None, q_weight=w)  # norm alone
    _check(q, w, pos, qo, dt, None, 1e-6)


def test_zero_rows_and_values_that_are_not_finite():
    n, D = 4, 128
    cfg, plan = _cfg(2, 1, D, 0), K.rope_plan(D)
    q = torch.zeros((n, 2, D), dtype=torch.float16, device="cuda")
    q[1, 0, 3], q[2, 1, 7] = float("inf"), float("nan")
    pos = torch.full((n,), 9, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    K.qk_norm_rope(cfg, q, None, pos, out, None, plan=plan)
    hit = torch.zeros((n, 2, D), dtype=torch.bool, device="cuda")
    hit[1, 0, 3] = hit[1, 0, 67] = hit[2, 1, 7] = hit[2, 1, 71] = True  # the pair, no other value
    assert torch.equal(~torch.isfinite(out), hit)
    assert torch.all(out[~hit] == 0)
    w = torch.ones(D, dtype=torch.float16, device="cuda")
    K.qk_norm_rope(cfg, q, None, pos, out, None, plan=plan, q_weight=w, eps=1e-6)
    assert torch.all(out[0] == 0) and torch.all(torch.isnan(out[2, 1]))


def test_side_stream_and_graph():
    n, hq, hk, D, dt = 64, 8, 2, 128, 0
    cfg, plan = _cfg(hq, hk, D, dt), K.rope_plan(D)
    q, k = _x((n, hq, D), dt, 1), _x((n, hk, D), dt, 2)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    K.qk_norm_rope(cfg, q, k, pos, qo, ko, plan=plan, stream=s)
    s.synchronize()
    _check(q, None, pos, qo, dt, {}, 1e-6)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.qk_norm_rope(cfg, q, k, pos, qo, ko, plan=plan)
    q.copy_(_x((n, hq, D), dt, 3))
    pos += 11
    g.replay()
    torch.cuda.synchronize()
    _check(q, None, pos, qo, dt, {}, 1e-6)
    _check(k, None, pos, ko, dt, {}, 1e-6)
