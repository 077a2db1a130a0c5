"""beam_sample's log-probabilities of tokens far below the largest, against the logits themselves.

logprob is (z - top) / t less the log of the kept weights' sum, which is a sum of weights in steps of 2^-44 of the largest: in FP64,
off by no more than V 2^-44 and the weights' 2^-29, and rounded to FP32 once, 2^-24 relative."""
import numpy as np
import pytest
import torch

from oracle import tree as OT
from test_gpu_paged import ints, status
from test_gpu_sample import DEV, draw, floats, logits

pytestmark = pytest.mark.gpu


def near(lp, want, V):
    assert abs(lp - want) <= 2.0 ** -28 + V * 2.0 ** -44 + 2.0 ** -24 * abs(want), (lp, want)


@pytest.mark.parametrize("V", [40, 5000, 201088])
@pytest.mark.parametrize("t", [1.0, 0.7, 3.0])
def test_tokens_far_below_the_largest(V, t):
    """Token 0, which u = 0 draws, from 1 to 30.4 nats below: its weight is down to one step of 2^-44. (At 30.5 nats it is none.)"""
    depths = [1.0, 5.0, 9.0, 15.0, 18.5, 22.0, 25.0, 27.0, 28.4, 29.3, 30.0, 30.4]
    T = len(depths)
    z = logits(V + 1, T, V, 1.0)
    z[:, V // 2] = 12.0
    z[:, 0] = 12.0 - t * floats(depths)
    zz = z.cpu().double().numpy() / np.float64(np.float32(t))
    for m in (None, floats([1e-14] * T)):      # a min-p that keeps all
        token, lp = draw(z, floats([0.0] * T), floats([t] * T), m=m)
        assert status() == 0 and not token.any()
        for r in range(T):
            w = np.exp(zz[r] - zz[r].max())
            near(float(lp[r]), zz[r, 0] - zz[r].max() - np.log(w.sum()), V)


def test_the_same_from_a_short_list():
    """top-k, whose kept tokens are drawn from a list, ties among them."""
    V, depths = 3000, [3.0, 12.0, 20.0, 24.0, 29.0, 30.3]
    T = len(depths)
    z = torch.full((T, V), -60.0, device=DEV)
    z[:, 7], z[:, 9], z[:, 2000] = 5.0, 5.0, 4.0
    z[:, 3] = 5.0 - floats(depths)
    token, lp = draw(z, floats([0.0] * T), k=ints([4] * T))
    assert status() == 0 and token.tolist() == [3] * T
    for r, d in enumerate(depths):
        zr = np.array([5.0, 5.0, 4.0, float(z[r, 3])])
        near(float(lp[r]), zr[3] - 5 - np.log(np.exp(zr - 5).sum()), V)


def test_logprobs_of_all_tokens_add_up():
    """Each token drawn at its own u, logits in ascending order: the logprobs are those of a softmax in 64 bits."""
    z = torch.linspace(-28.0, 2.0, 61, device=DEV)
    w = np.exp(z.cpu().double().numpy())
    u = floats((np.cumsum(w) - w / 2) / w.sum())
    token, got = draw(z.repeat(61, 1), u)
    want = [OT.sample(z.cpu().numpy(), float(x))[0] for x in u]      # by weights in whole steps: the first few may be passed over
    assert token.tolist() == want and len(set(want)) > 55 and status() == 0
    for i, lp in zip(want, got.tolist()):
        if lp > -0.6:      # more than half: by what is missing from 1
            assert abs(lp - np.log(w[i] / w.sum())) <= 2.0 ** -28 + 2.0 ** -24 * abs(lp)
        else:
            near(lp, np.log(w[i] / w.sum()), 61)


def test_differences_past_the_range_of_fp32():
    z = torch.full((2, 100), 3e38, device=DEV)
    z[:, ::2] = -3e38
    for t in (1.0, 1e30, 3e38):
        for u in (0.0, 0.5, 1.0):
            token, lp = draw(z, floats([u] * 2), floats([t] * 2), p=floats([1.0, 0.9]))
            assert status() == 0 and int(token[0]) % 2 == int(token[1]) % 2 == 1 and abs(float(lp[0]) + np.log(50)) < 1e-5
