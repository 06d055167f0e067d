"""Beam selection of rows masked by large finite numbers and of rows whose logits are all large: the
log-sum must not depend on where a row's values lie."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from tests.test_gpu_beam_offsets import TYPES, check, random  # noqa: E402


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [-6e4, -1e6, -1e9, -1e10, -3e10, -1e12, -1e20, -1e30, -1e35, -3.3e38])
def test_masks_of_any_size(dtype, value):
    """Masked at the front (a thread's first turns see nothing else), at the end, here and there; and whole beams."""
    if dtype == "fp16" and value < -65504:
        pytest.skip("no such number")
    for V in (1000, 20011):
        x, s = random(4, 3, V, dtype, seed=V)
        front = V * 9 // 10
        x[0, :, :front] = value
        x[1, :, V - front:] = value
        hide = torch.rand((3, V), generator=torch.Generator().manual_seed(1)) < 0.9
        x[2][hide.cuda()] = value
        x[3, 1] = value  # a beam masked as a whole, among others
        check(x, s)
        check(x[3:, 1:2].contiguous(), s[3:, 1:2].contiguous())  # and by itself: -ln V


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [1e5, 1e6, 1e7, 1e9, 1e10, 1e11, 1e20, 3e38])
@pytest.mark.parametrize("sign", [1, -1])
def test_equal_logits_of_any_size(dtype, value, sign):
    for V in (1000, 20011):
        x, s = random(2, 4, V, dtype, seed=V)
        x[0] = sign * value
        x[1, 2] = sign * value
        x[1, 3, ::2] = sign * value
        check(x, s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [999990.0, 1e6, 1e6 + 10, 2.0 ** 20, 1e7, 1e9])
@pytest.mark.parametrize("sign", [1, -1])
def test_rows_far_from_zero(dtype, offset, sign):
    """Also where parts of a row lie on both sides of the size at which the sums' reference changes."""
    for B, V in ((2, 5003), (3, 40000)):
        check(*random(2, B, V, dtype, V, sign * offset))
    x, s = random(1, 3, 90001, dtype, 7, sign * offset)
    x[0, 0, :50000] -= 500
    x[0, 1, 30000:] += 500
    x[0, 2, :60000] = -1e10
    check(x, s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masks_below_values_far_from_zero(dtype):
    x, s = random(3, 2, 20011, dtype, 1, -1e6)
    x[0, :, 3::7] = -1e9
    x[1, 0] = -1e10
    x[1, 0, 19000:] = -1e9
    x[2] = -1e10
    x[2, :, 20010] = 1e10
    check(x, s)
