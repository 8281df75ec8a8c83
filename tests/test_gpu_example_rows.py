"""The example's shared expert on fewer rows than it was made for."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_shared_expert_of_fewer_rows():
    """The result has the rows of x alone, each the one that the full batch gives
    it up to the order of the f32 sums; nothing of the call before shows."""
    from examples import shared_and_finetuned_experts as ex
    g = torch.Generator()
    g.manual_seed(7)
    H, F, rows = 512, 256, 200
    r = lambda *n: (torch.randn(*n, generator=g) * 0.05).bfloat16().cuda()  # noqa: E731
    shared = ex.SharedExpert(r(2 * F, H), r(H, F), rows)
    x = torch.randn(rows, H, generator=g).bfloat16().cuda()
    full = shared(x).clone()
    assert full.shape == (rows, H)
    for n in (1, 7, 40, 199, 0, rows):
        print(f"[case] {n} of {rows} rows", flush=True)
        for t in (shared.xq, shared.aq):   # NaN codes where nothing of this call is
            t.view(torch.uint8).fill_(0x7F)
        y = shared(x[:n])
        assert y.shape == (n, H)
        # one bf16 step of h may turn a code of the hidden layer by a step of e4m3 (2^-3 of it):
        # the rows agree to a small part of their norm, and differ from other rows' by the whole of it
        if n:
            assert bool(((y.float() - full[:n].float()).norm(dim=1) < 0.05 * full[:n].float().norm(dim=1)).all())
    with pytest.raises(ValueError):
        shared(torch.zeros(rows + 1, H, dtype=torch.bfloat16, device="cuda"))
