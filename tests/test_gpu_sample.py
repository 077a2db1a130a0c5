"""GPU parity of beam_sample against float64 NumPy (oracle/tree.py).

Tokens have to be equal. A border (u times the sum, top_p of the sum, a logit next to min_p's) that lies within
the two sides' rounding of a token's own sum could be met by its neighbour; the weights' error is 2^-29 and the tests
draw a few thousand borders over at most 200,000 tokens, so that is not expected to happen, and the inputs
are fixed by seed. logprob: the share's error 2^-28 and its rounding to FP32, 2^-24 relative."""
import numpy as np
import pytest
import torch

from oracle import tree as OT
from hybrid_attention_moe_gb300 import beam as B
from test_gpu_paged import gen, ints, status

pytestmark = pytest.mark.gpu
DEV = "cuda"


def floats(x):
    return torch.tensor(x, dtype=torch.float32, device=DEV)


def draw(z, u, t=None, k=None, p=None, m=None, stream=None):
    T = z.shape[0]
    token, logprob = torch.full((T,), -7, dtype=torch.int32, device=DEV), torch.full((T,), 7.0, device=DEV)
    B.beam_sample(z, u, token, logprob, t, k, p, m, stream)
    return token, logprob


def check(z, u, t=None, k=None, p=None, m=None):
    token, logprob = draw(z, u, t, k, p, m)
    st = status()
    zz = z.cpu().numpy()
    val = [x.cpu().double().numpy() if x is not None else [d] * len(zz) for x, d in ((u, 0), (t, 1.0), (k, 0), (p, 1.0), (m, 0.0))]
    for r in range(len(zz)):
        want, lp = OT.sample(zz[r], *(float(v[r]) if i != 2 else int(v[r]) for i, v in enumerate(val)))
        assert int(token[r]) == want, (r, int(token[r]), want, [float(v[r]) for v in val])
        got = float(logprob[r])
        if want < 0:
            assert np.isnan(got) and st == B.DEV_BAD_LOGITS
        else:
            assert abs(got - lp) <= 2.0 ** -27 + 2.0 ** -23 * abs(lp), (r, got, lp)
    return token, logprob, st


def logits(seed, T, V, scale=2.0, rounded=False):
    z = scale * torch.randn((T, V), generator=gen(seed), device=DEV)
    return z.to(torch.bfloat16).float() if rounded else z


def uniform(seed, T, lo=0.0, hi=1.0):
    return lo + (hi - lo) * torch.rand(T, generator=gen(seed), device=DEV)


@pytest.mark.parametrize("V", [1, 2, 3, 31, 33, 127, 1000, 4097, 32003, 100001])
@pytest.mark.parametrize("rounded", [False, True])
def test_rules_match_the_oracle(V, rounded):
    """Each rule alone and together, over vocabularies of odd sizes, with and without ties."""
    T = 24 if V < 50000 else 8
    z = logits(V, T, V, 2.5, rounded)
    u, t = uniform(V + 1, T), uniform(V + 2, T, 0.5, 1.5)
    k = torch.randint(1, 60, (T,), generator=gen(V + 3), device=DEV).int()
    p, m = uniform(V + 4, T, 0.3, 0.999), uniform(V + 5, T, 0.001, 0.5)
    for kw in ({}, dict(t=t), dict(t=t, k=k), dict(t=t, p=p), dict(t=t, m=m), dict(k=k, p=p), dict(t=t, k=k, p=p, m=m)):
        assert check(z, u, **kw)[2] == 0


def test_flat_and_peaked_rows():
    """All logits equal, two values, one that outweighs all, the type's lowest value and -inf as masks."""
    V = 30000
    z = torch.zeros((8, V), device=DEV)
    z[1, ::2] = 1.0
    z[2, 17] = 40.0
    z[3] = -3.4028234663852886e38
    z[3, 29999] = 1.0
    z[4] = -float("inf")
    z[4, [5, 100, 20000]] = floats([1.0, 2.0, 2.0])
    z[5] = -3.4028234663852886e38                     # nothing but the lowest value: all the same
    z[6] = torch.linspace(-30, 30, V)
    z[7, 1::2] = -0.0                                 # equal to 0
    for kw in ({}, dict(k=ints([700] * 8)), dict(p=floats([0.7] * 8)), dict(m=floats([0.9] * 8)), dict(k=ints([20000] * 8), p=floats([0.5] * 8)),
               dict(t=floats([1e-3] * 8)), dict(t=floats([1e4] * 8), p=floats([0.33] * 8))):
        for x in (0.0, 0.31, 0.9999999):
            assert check(z, floats([x] * 8), **kw)[2] == 0


def test_cuts_among_many():
    """Cuts that lie among more logits than a list holds: flat rows, logits on a coarse grid, masks of the lowest value and of
    -1e9, two far clusters; top-k around a list's size and beyond it, alone and in front of the other rules."""
    V = 20000
    z = torch.stack([logits(31, 1, V, 0.05)[0], logits(32, 1, V, 0.7)[0], logits(33, 1, V, 0.3, True)[0], logits(34, 1, V, 3.0)[0],
                     logits(35, 1, V, 1.0)[0], logits(36, 1, V, 0.2)[0]])
    z[3, 1::2] = -3.4028234663852886e38
    z[4, ::3] = -1e9
    z[5, 5000:] -= 25.0
    z[5, 19000:] = -float("inf")
    T = len(z)
    for n, p in enumerate((0.05, 0.6, 0.97, 0.9999)):
        assert check(z, uniform(40 + n, T), p=floats([p] * T))[2] == 0
        assert check(z, uniform(50 + n, T), t=floats([0.3, 30.0, 1e30, 0.1, 2.0, 0.01]), p=floats([p] * T))[2] == 0
    for n, k in enumerate((511, 512, 513, 700, 6000, V - 1)):
        assert check(z, uniform(60 + n, T), k=ints([k] * T))[2] == 0
        assert check(z, uniform(70 + n, T), k=ints([k] * T), p=floats([0.8] * T))[2] == 0
        assert check(z, uniform(80 + n, T), t=floats([0.5] * T), k=ints([k] * T), p=floats([0.99] * T), m=floats([0.02] * T))[2] == 0


def test_edges_of_the_arguments():
    z, T = logits(9, 12, 500, 3.0), 12
    z[3, 7] = z[3, 9] = 50.0
    top = z.argmax(1).int()
    top[3] = 7
    one = floats([0.5] * T)
    for t in (0.0, -1.0, 1e-31):                       # greedy
        tok, lp = draw(z, one, floats([t] * T))
        assert torch.equal(tok, top) and not lp.any()
    tok, lp = draw(z, one, k=ints([1] * T))
    assert torch.equal(tok, top) and not lp.any()
    assert torch.equal(draw(z, one, p=floats([0.0] * T))[0], top) and torch.equal(draw(z, one, p=floats([-1.0] * T))[0], top)
    ref = draw(z, one)
    for kw in (dict(k=ints([0] * T)), dict(k=ints([-5] * T)), dict(k=ints([500] * T)), dict(k=ints([2 ** 31 - 1] * T)),
               dict(p=floats([1.0] * T)), dict(p=floats([3.0] * T)), dict(m=floats([0.0] * T)), dict(m=floats([-1.0] * T)),
               dict(t=floats([1.0] * T))):
        got = draw(z, one, **kw)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]), kw
    check(z, one, m=floats([1.0] * T))
    check(z, one, m=floats([5.0] * T))                 # the largest stay
    # u at and past its ends: the first and the last kept token that weigh anything (row 3's third weighs nothing)
    lo, hi = draw(z, floats([-1.0] * T), k=ints([3] * T))[0], draw(z, floats([1.0] * T), k=ints([3] * T))[0]
    for r in range(T):
        row = z[r].cpu().numpy()
        assert (int(lo[r]), int(hi[r])) == tuple(OT.sample(row, x, 1.0, 3)[0] for x in (-1.0, 1.0))
    assert status() == 0


def test_rows_without_a_distribution():
    z = logits(11, 6, 1000)
    z[1, 999], z[2, 0], z[3] = float("nan"), float("inf"), -float("inf")
    z[4, 5] = -float("nan")
    tok, lp, st = check(z, floats([0.4] * 6), t=floats([0.0, 0.0, 1.0, 0.0, 1.0, 1.0]), k=ints([0, 1, 3, 2, 0, 5]))
    assert st == B.DEV_BAD_LOGITS and [int(x) < 0 for x in tok] == [False, True, True, True, True, False]
    assert status() == 0


@pytest.mark.parametrize("T,V", [(1, 201088), (3, 851968), (130, 50000), (1, 425985)])
def test_large_vocabularies(T, V):
    z = logits(V, T, V, 3.0)
    check(z, uniform(1, T), uniform(2, T, 0.6, 1.2), None, uniform(3, T, 0.8, 0.99), None)
    check(z, uniform(4, T), None, ints([50] * T), None, None)
    check(z, uniform(5, T))


def test_strided_rows_and_refusals():
    wide = logits(13, 5, 4000)
    u = uniform(14, 5)
    for a, b in ((0, 3001), (1, 3002), (2, 999), (3, 1004)):
        got = draw(wide[:, a:b], u, p=floats([0.8] * 5))
        ref = draw(wide[:, a:b].contiguous(), u, p=floats([0.8] * 5))
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    tok = ints([0] * 5)
    B.beam_sample(wide, u, tok)                        # no logprob wanted
    assert torch.equal(tok, draw(wide, u)[0])
    for f in (lambda: draw(wide.half(), u), lambda: draw(wide.t(), u), lambda: draw(wide[0], u), lambda: draw(wide, u.double()),
              lambda: draw(wide, u[:4]), lambda: draw(wide, u, t=u[:1]), lambda: draw(wide, u, k=u), lambda: draw(wide, u, p=u.cpu()),
              lambda: B.beam_sample(wide, u, tok.long()), lambda: B.beam_sample(wide, u, tok[:4]), lambda: B.beam_sample(wide[:, :0], u, tok),
              lambda: B.beam_sample(wide, u, tok, u.double())):
        with pytest.raises(B.BeamError):
            f()
    B.beam_sample(wide[:0], u[:0], tok[:0])
    assert status() == 0


def test_tokens_do_not_hang_on_the_batch_and_replay():
    """A row alone, in a batch, on a side stream and in a replayed graph gives the same token and logprob."""
    T, V = 40, 60000
    z, u, t = logits(15, T, V, 2.0), uniform(16, T), uniform(17, T, 0.7, 1.2)
    p, k, m = uniform(18, T, 0.5, 0.99), ints([(i % 4) * 300 for i in range(T)]), uniform(19, T, 0, 0.01)
    ref = draw(z, u, t, k, p, m)
    for r in (0, 7, 39):
        one = draw(z[r:r + 1], u[r:r + 1], t[r:r + 1], k[r:r + 1], p[r:r + 1], m[r:r + 1])
        assert torch.equal(one[0], ref[0][r:r + 1]) and torch.equal(one[1], ref[1][r:r + 1])
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = draw(z, u, t, k, p, m, st)
    torch.cuda.synchronize()
    token, logprob = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    st.synchronize()
    again = (token, logprob)
    B.beam_sample(z, u, token, logprob, t, k, p, m)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.beam_sample(z, u, token, logprob, t, k, p, m)
    for x in (got, again):
        assert torch.equal(x[0], ref[0]) and torch.equal(x[1], ref[1])
    z.copy_(logits(20, T, V, 1.0))
    graph.replay()
    ref = draw(z, u, t, k, p, m)
    assert torch.equal(token, ref[0]) and torch.equal(logprob, ref[1]) and status() == 0


def test_two_calls_at_once():
    """Calls on two streams, of one row and of many, side by side."""
    z, u, t = logits(23, 64, 90000, 2.0), uniform(24, 64), uniform(25, 64, 0.6, 1.3)
    p, k = uniform(26, 64, 0.5, 0.99), ints([(i % 3) * 400 for i in range(64)])
    refs = [draw(z[:1], u[:1], t[:1], None, p[:1]), draw(z, u, t, k, p)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[torch.full_like(x, 9) for x in r] for r in refs for _ in range(4)]
    torch.cuda.synchronize()
    for n in range(4):
        B.beam_sample(z[:1], u[:1], *outs[n], t[:1], None, p[:1], None, streams[0])
        B.beam_sample(z, u, *outs[4 + n], t, k, p, None, streams[1])
    torch.cuda.synchronize()
    for n, o in enumerate(outs):
        assert torch.equal(o[0], refs[n // 4][0]) and torch.equal(o[1], refs[n // 4][1])
    assert status() == 0


def test_shares_of_many_draws():
    """One row, evenly spaced u: each token is drawn as often as its weight says, to one draw at either end."""
    V, T = 50, 20000
    z = logits(21, 1, V, 1.5)
    u = (torch.arange(T, device=DEV).float() + 0.5) / T
    tok = draw(z.repeat(T, 1), u)[0]
    w = np.exp(z[0].cpu().double().numpy())
    assert np.all(np.abs(np.bincount(tok.cpu().numpy(), minlength=V) - T * w / w.sum()) <= 1.01)
