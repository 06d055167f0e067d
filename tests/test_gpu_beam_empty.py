"""Beam selection with empty beams (a score of -inf, or NaN) where there are fewer live candidates than beams: the rest are -inf, the
lowest beams and tokens first, whatever the empty beams' logits are."""

import pytest

from tests.test_gpu_beam_select import check, random

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
@pytest.mark.parametrize("B,V", [(1, 7), (2, 9000), (4, 3), (5, 20011), (8, 2), (32, 6), (32, 31), (32, 5000), (20, 40000)])
@pytest.mark.parametrize("empty", [-float("inf"), float("nan")])
def test_more_beams_than_candidates(dtype, B, V, empty):
    x, s = random(4, B, V, dtype, seed=B)
    s[0] = empty                # nothing at all
    s[1, 1:] = empty            # a new search
    s[2, :B - 1] = empty        # only the last beam
    s[3, ::2] = empty
    x[1:, :, 2:] = -float("inf")  # two tokens may follow, of each beam
    got = check(x, s)
    assert got[1][0].tolist() == ([*range(B)] if V >= B else [i % V for i in range(B)])
    assert got[2][0].tolist() == [i // V for i in range(B)]


@pytest.mark.parametrize("B", [3, 32])
def test_beside_finished_beams(B):
    x, s = random(3, B, 5000, "bf16", seed=B)
    done = torch.zeros((3, B), dtype=torch.int32, device="cuda")
    done[:, 1] = 1
    s[0] = -float("inf")  # the finished one too
    s[1, 0] = s[1, 2:] = -float("inf")
    s[2, 1:] = -float("inf")
    x[2, 0, 1:] = -float("inf")
    check(x, s, done, eos=2)
