"""Beam selection with scores and finished beams in place, over and over: blocks of finished beams have nothing to read and
are at their group's ticket at once, while others of their threads may not have begun."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402


@pytest.mark.parametrize("G,B,V", [(1, 1, 9), (300, 2, 9), (500, 8, 40), (40, 32, 700), (3, 5, 40000)])
@pytest.mark.parametrize("share", [0.5, 0.9, 1.0])
def test_finished_beams_change_places(G, B, V, share):
    """Every step's scores and finished beams are those of the step with buffers of its own."""
    g = torch.Generator(device="cuda").manual_seed(B + V)
    x = torch.randn((G, B, V), generator=g, device="cuda")
    scores = -torch.rand((G, B), generator=g, device="cuda")
    done = (torch.rand((G, B), generator=g, device="cuda") < share).to(torch.int32)
    apart, together = K.BeamSelect(G, B, V), K.BeamSelect(G, B, V)
    tokens, parents = torch.empty_like(done), torch.empty_like(done)
    for step in range(40):
        want = [torch.empty_like(t) for t in (scores, tokens, parents, done)]
        apart.select(x, scores, *want[:3], done=done, done_out=want[3], eos=7)
        together.select(x, scores, scores, tokens, parents, done=done, done_out=done, eos=7)
        for a, b in zip((scores, tokens, parents, done), want):
            assert torch.equal(a, b), step
        # other beams finished: both values are written over the other one
        scores.copy_(-torch.rand((G, B), generator=g, device="cuda"))
        done.copy_((torch.rand((G, B), generator=g, device="cuda") < share).to(torch.int32))
