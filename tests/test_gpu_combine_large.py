"""The combine of more tokens than one dimension of a grid takes workgroups."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d", [((1 << 24) + 3, 8), ((1 << 23) + 5, 1028), ((1 << 22) - 1, 1028)])
def test_tokens_past_a_line_of_workgroups(T, d):
    """One route each, in order: out[t] = w[t] y[t] exactly."""
    import torch

    import routed_expert_prefill_amd as rep

    g = torch.Generator("cuda").manual_seed(T)
    y = torch.randn(T, d, generator=g, device="cuda")
    w = torch.rand(T, 1, generator=g, device="cuda")
    rows = torch.arange(T, dtype=torch.int32, device="cuda")
    out = torch.full((T + 2, d), 7.0, device="cuda")
    rep.combine(y, rows, w, None, out=out[:T])
    torch.cuda.synchronize()
    assert (out[T:] == 7).all()
    step = 1 << 20
    for a in range(0, T, step):
        b = min(a + step, T)
        assert torch.equal(out[a:b], y[a:b] * w[a:b]), a
