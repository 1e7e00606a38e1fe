"""Verification of drafted tokens where a refused draft leaves nothing of the target above it, so that the target's
own row is drawn from (p need not be normalised), beside test_gpu_verify.py."""
import pytest
import torch

from gpu_util import announce, device
from test_gpu_verify import BF, F32, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("size", [(3, 2, 700), (5, 3, 40960), (5, 3, 41000), (2, 2, 262147), (600, 1, 5003), (1, 1, 1 << 20)],
                         ids=lambda s: "S%d-D%d-V%d" % s)
def test_nothing_is_left(size, dt):
    """p a half of q everywhere: every draft whose u is over a half is refused and leaves nothing.  In some
    sequences one entry is left after all, or one piece of the row has no weight at all."""
    dev = device()
    S, D, V = size
    c = make(S, D, V, dt, False, 31, noise=0.0)
    c["p"] = (c["p"].float() / 2).to(dt)
    c["u"] = 0.5 + c["u"] / 2
    c["draft_len"] = None
    _, kept = check(c, dev, ("nothing is left", size, dt))
    assert (kept < D).all()
    c["p"][0, 0, V - 5] = 2 * c["q"][0, 0, V - 5] + 1e-3   # all that is left
    if S > 1:
        c["p"][1, 0, V // 3:V // 2] = 0.0                 # pieces of nothing
        c["q"][1, 0, V // 3:V // 2] = 0.0
        c["draft"][1, 0] = V - 1
    check(c, dev, ("one entry is left", size, dt))


@pytest.mark.parametrize("V", [9000, 300000])
@pytest.mark.parametrize("dt", [F32, BF])
def test_borders_of_what_is_drawn_instead(dt, V):
    """Greedy drafts whose token has all of the target's weight but for entries that are no weights, refused: the
    token itself is drawn.  And quarters in places that lie in different pieces, r at their borders."""
    dev = device()
    at = torch.tensor([0, 2047, 2048, V - 1])
    S = 9
    p = torch.zeros(S, 2, V)
    p[:, :, at] = 0.25
    q = torch.zeros(S, 1, V)
    q[:, :, at] = 0.25
    r = torch.tensor([0.0, 0.25 - 2.0 ** -26, 0.25, 0.5 - 2.0 ** -25, 0.5, 0.75 - 2.0 ** -24, 0.75, 1.0 - 2.0 ** -24, 1.0])
    c = {"p": p.to(dt), "q": q.to(dt), "draft": torch.full((S, 1), 5), "u": torch.full((S, 1), 0.5), "r": r, "draft_len": None}
    want, kept = check(c, dev, ("borders of p itself", dt, V))
    assert not kept.any() and want[:, 0].tolist() == [at[k].item() for k in (0, 0, 1, 1, 2, 2, 3, 3, 3)]
    p = torch.zeros(3, 2, V)
    p[:, :, 3000] = 0.5
    p[1, 0, 4000], p[2, 0, 8000] = -1.0, float("inf")
    c = {"p": p.to(dt), "q": None, "draft": torch.full((3, 1), 3000), "u": torch.full((3, 1), 0.75), "r": torch.rand(3), "draft_len": None}
    want, kept = check(c, dev, ("the refused token", dt, V))
    assert not kept.any() and (want[:, 0] == 3000).all()


@pytest.mark.parametrize("size", [(255, 2, 1001), (256, 2, 1001), (257, 2, 1001), (400, 1, 9001), (512, 1, 700), (513, 1, 700)],
                         ids=lambda s: "S%d-D%d-V%d" % s)
def test_numbers_of_sequences(size):
    """Around where a workgroup a sequence becomes many."""
    dev = device()
    for dt, greedy in ((F32, False), (BF, True)):
        check(make(*size, dt, greedy, 33), dev, (size, dt, greedy))
