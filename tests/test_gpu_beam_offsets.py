"""Beam selection of rows that lie far from zero: the log-sum must not depend on where a row's values lie."""

import numpy as np
import pytest

from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def bound(V):
    """Largest error of a log-sum.  A term e^d, d <= 0, goes through its exponential and at most V / 4096 + 5 changes of
    the reference (a thread's turns, then lane, warp, block and group): 2^-22 each for the base-2 exponential; their arguments, all of
    one sign, add up to log2(e) |d| and are rounded by the constant, the product and the difference, 2^-24 |d| log2(e) for each
    of the three and once more for the changes: 8 |d| 2^-24; the |d| weigh with their terms, whose mean is at most
    ln V.  A reference's own rounding is at most 1/16 and taken off again, 2^-24 of it aside.  A thread adds V / 256 + 8 terms, 13 joins
    follow: 2^-24 each.  The sum's relative error is the log's absolute one."""
    return (V / 4096 + 6) * 2.0 ** -22 + (8 * np.log(V + 1) + 1) * 2.0 ** -24 + (V / 256 + 21) * 2.0 ** -24


def check(x, scores):
    G, B, V = x.shape
    out = [torch.full((G, B), 77, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    K.BeamSelect(G, B, V).select(x, scores, *out)
    torch.cuda.synchronize()
    score, token, parent = (t.cpu().numpy() for t in out)
    want, want_token, want_parent, _ = S.beam_select(x.double().cpu().numpy(), scores.double().cpu().numpy())
    lim = bound(V) + 2.0 ** -24 * np.abs(want)
    assert np.all(np.abs(score - want) <= lim), np.abs(score - want).max()
    # beams' scores nearer than the errors may change places across beams; nothing else may
    for g, i in zip(*np.nonzero((token != want_token) | (parent != want_parent))):
        near = [j for j in range(B) if (parent[g, i], token[g, i]) == (want_parent[g, j], want_token[g, j])]
        same = near and want_parent[g, near[0]] != want_parent[g, i] and abs(want[g, near[0]] - want[g, i]) <= 2 * lim[g, i]
        assert same or (not near and abs(score[g, i] - want[g, -1]) <= 2 * lim[g, i] and parent[g, i] != want_parent[g, -1]), (g, i)


def random(G, B, V, dtype, seed, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = (2.5 * torch.randn((G, B, V), generator=g) + offset).to(TYPES[dtype])
    return x.cuda(), (-10 - 3 * torch.rand((G, B), generator=g)).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset", [100, 1e3, 1e4, 6e4, 1e5, 3e5])
@pytest.mark.parametrize("sign", [1, -1])
def test_rows_far_from_zero(dtype, offset, sign):
    """What all logits of a row have in common changes nothing, whatever the parts that the row is summed in."""
    if dtype == "fp16" and offset > 6e4:
        pytest.skip("no such number")
    for B, V in ((2, 5003), (3, 40000)):
        check(*random(2, B, V, dtype, V, sign * offset))
    x, s = random(1, 3, 90001, dtype, 7, sign * offset)
    x[0, 0, :50000] -= min(offset, 500.0)
    x[0, 1, 30000:] += min(offset, 500.0) if dtype != "fp16" else 0
    check(x, s)
