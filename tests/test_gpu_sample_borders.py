"""Sampled next tokens where a weight, a temperature or a border lies at the end of its range,
against the definition in 64 bits (tests/_serving.py); `out` holds a poison before every call, so
a token that is not written shows."""
import math

import pytest
import torch

from tests import _serving as S

pytestmark = pytest.mark.gpu

R = pytest.importorskip("recurrent_depth_moe_b200")
NONE = -7
TINY = 2.0 ** -126            # the smallest normal fp32 number
LOWEST = -3.4028234663852886e38


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    R.load_library()


def _sample(x, u, T, **kw):
    """Tokens and log-probabilities (CPU), with the tokens poisoned before the call."""
    dev = lambda a: a.cuda() if isinstance(a, torch.Tensor) else a
    out = torch.full((x.shape[0],), NONE, dtype=torch.int32, device="cuda")
    tok, lp = R.sample_tokens(x.cuda(), u.cuda(), dev(T), out=out, return_logprob=True, **kw)
    return tok.cpu(), lp.cpu()


@pytest.mark.parametrize("V", [2, 33, 1001, 5000, 60000, 201088, 500000])
@pytest.mark.parametrize("kw", [dict(), dict(top_k=-1), dict(min_p=1e-14), dict(top_p=1 - 2.0 ** -24)])
def test_background_at_the_smallest_weight(V, kw):
    """One token in the last place above V - 1 equal ones whose weight is near 2^-45, below which
    it is nothing: gaps of 31.0 to 31.19 (45 ln 2 is 31.1916) leave the background a weight, so u
    = 0 draws token 0, gaps above it leave the last token alone, whatever u."""
    kw = dict(kw, top_k=V - 1) if "top_k" in kw else kw
    us = (0.0, 1e-9, 1e-8, 0.5)
    for gap in (31.0, 31.15, 31.19, 31.2, 31.25, 31.5, 31.9, 32.0, 32.06, 32.1, 33.0):
        x = torch.zeros(len(us), V)
        x[:, V - 1] = gap
        tok, lp = _sample(x, torch.tensor(us), 1.0, **kw)
        back = gap < 45 * math.log(2) and "top_p" not in kw       # (1 - 2^-24 of the weight is the last token's)
        for i, u in enumerate(us):
            # (a weight of the background is off by up to a half of 2^-44, so twice its share)
            share = 2 * (V - 1) * math.exp(-gap) if back else 0.0
            if back and u == 0.0:
                want = [0 if kw.get("top_k", V) > 1 else V - 1]
            elif u < share:
                want = range(V)
            else:
                want = [V - 1]
            assert int(tok[i]) in want, (gap, u, int(tok[i]))
            if int(tok[i]) == V - 1:
                assert abs(float(lp[i])) <= 2.0 ** -20, (gap, u)


@pytest.mark.parametrize("V", [500, 9001, 201088])
def test_infinite_and_huge_temperatures_with_masked_logits(V):
    """An infinite temperature is uniform over the tokens above -inf (NaN and -inf take no part),
    and so is a finite one far above the logits, with every other parameter beside it."""
    g = torch.Generator().manual_seed(V)
    us = torch.tensor([0.0, 0.2, 0.55, 0.999, 1 - 2.0 ** -24])
    x = torch.randn(len(us), V, generator=g) * 3
    x[torch.rand(x.shape, generator=g) < 0.3] = -math.inf
    x[:, 1::97] = math.nan
    x[:, 7] = 0.5
    for T in (math.inf, 3.4e38, 1e38, 1.1e37):
        for kw in (dict(), dict(top_k=V - 2), dict(top_k=37), dict(min_p=0.5), dict(top_p=0.5), dict(top_k=V * 2, top_p=1.0)) + \
                ((dict(min_p=1.0),) if T == math.inf else ()):
            tok, lp = _sample(x, us, torch.full((len(us),), T), **kw)
            for i in range(len(us)):
                live = torch.nonzero(x[i] > -math.inf).flatten()
                n = min(len(live), kw.get("top_k", V), math.ceil(kw.get("top_p", 1.0) * len(live)))
                order = torch.sort(x[i, live], descending=True, stable=True).indices[:n]
                live = live[order].sort().values                  # what is kept, in the vocabulary's order
                pos = int(torch.searchsorted(live, int(tok[i])))
                assert pos < n and int(live[pos]) == int(tok[i]), (T, kw, i, int(tok[i]))
                # n equal weights: u n lies in the drawn token's unit, or within fp32's share of its ends
                assert pos - n * 2.0 ** -21 <= float(us[i]) * n <= pos + 1 + n * 2.0 ** -21, (T, kw, i, pos)
                assert abs(float(lp[i]) + math.log(n)) <= 2.0 ** -20 * math.log(n), (T, kw, i)


def test_rows_of_the_lowest_value_and_minus_infinity():
    """A row whose unmasked logits are all the type's lowest value, beside -inf."""
    V = 3000
    us = torch.tensor([0.0, 0.4, 0.9, 1 - 2.0 ** -24])
    x = torch.full((4, V), -math.inf)
    x[:, ::3] = LOWEST
    n = 1000
    for T in (1.0, 1e-3, 1e30):
        for kw in (dict(), dict(top_k=2999), dict(min_p=0.9), dict(top_k=500), dict(top_p=0.5)):
            tok, lp = _sample(x, us, T, **kw)
            m = kw.get("top_k", n) if kw.get("top_k", n) < n else 500 if "top_p" in kw else n
            for i in range(4):
                assert int(tok[i]) == 3 * int(float(us[i]) * m), (T, kw, i)
                assert abs(float(lp[i]) + math.log(m)) <= 2.0 ** -19, (T, kw, i)
    y = torch.full((4, 200), LOWEST)                              # masked by the lowest value under a huge temperature
    y[:, 100:] = torch.linspace(-1, 1, 100)
    for T in (1e37, 1e38):
        tok, lp = _sample(y, us, T)
        t32 = float(torch.tensor(T))
        for i in range(4):
            want, logp, margin = S.sample_row(y[i], float(us[i]), t32)
            assert int(tok[i]) == want or margin < 4e-7, (T, i)
            assert margin < 4e-7 or abs(float(lp[i]) - logp) <= 2.0 ** -19, (T, i)


def test_tiny_temperatures_beside_neighbouring_logits():
    """Logits one step below the maximum under temperatures far below the step: the maximum alone."""
    V = 2000
    us = torch.tensor([0.0, 0.3, 0.8, 1 - 2.0 ** -24])
    for top in (100.0, -100.0, 1.0, 3e30, 65537.0):
        t = torch.tensor(top)
        x = torch.full((4, V), float(torch.nextafter(t, torch.tensor(-math.inf))))
        x[:, ::2] = float(torch.nextafter(torch.nextafter(t, torch.tensor(-math.inf)), torch.tensor(-math.inf)))
        x[:, V - 3] = top
        step = abs(top) * 2.0 ** -24
        for T in (step / 40, step / 100, step * 1e-4, step * 1e-8, 1e-30 if top < 1e20 else 1.0, TINY):
            if T < TINY:
                continue
            for kw in (dict(), dict(top_k=V - 1), dict(top_k=50), dict(top_p=0.9), dict(min_p=1e-12)):
                tok, lp = _sample(x, us, T, **kw)
                assert tok.tolist() == [V - 3] * 4, (top, T, kw)
                assert float(lp.abs().max()) <= 2.0 ** -20, (top, T, kw)


@pytest.mark.parametrize("V", [64, 5000, 201088])
@pytest.mark.parametrize("k", [0, 20, 40])
def test_top_p_among_logits_near_the_smallest_normal_number(V, k):
    """Temperatures where sixteen bins per power of two pass fp32's range: the exponent's
    histogram is then too coarse to bracket top-p's border, and the whole order decides."""
    g = torch.Generator().manual_seed(7 + V)
    us = torch.tensor([0.0, 0.3, 0.66, 0.7, 0.8, 0.9, 0.99])
    place = torch.randperm(V, generator=g)[:60]
    live = place.sort().values                                    # (the rest is -inf and weighs nothing)
    for T in (1.3e-38, 2e-38, 6e-38):
        T = float(torch.tensor(T, dtype=torch.float32))
        x = torch.full((len(us), V), -math.inf)
        x[:, place] = -(torch.arange(60, dtype=torch.float64) * math.log(1.7) * T).float()
        for p in (0.6, 0.9, 0.99):
            p32 = float(torch.tensor(p))
            tok, lp = _sample(x, us, T, top_k=k, top_p=p)
            for i in range(len(us)):
                want, logp, margin = S.sample_row(x[i, live], float(us[i]), T, k, p32)
                if margin <= 4e-7:
                    continue
                assert int(tok[i]) == int(live[want]), (T, p, i)
                assert abs(float(lp[i]) - logp) <= 2.0 ** -19, (T, p, i)


def test_temperatures_around_the_smallest_normal_number():
    """Below 2^-127 greedy, as 0 is: log2(e) / T is past fp32's range there.  From there on by the
    definition, among logits that are themselves below the smallest normal number."""
    V = 700
    g = torch.Generator().manual_seed(3)
    us = torch.tensor([0.0, 0.31, 0.5, 0.77, 1 - 2.0 ** -24])
    f32 = lambda a: float(torch.tensor(a, dtype=torch.float32))
    for scale in (1e-39, 1e-38, 1e-36, 1.0):
        x = torch.randn(len(us), V, generator=g) * scale
        for kw in (dict(), dict(top_k=5), dict(top_p=0.9), dict(min_p=0.1)):
            for T in (5.8e-39, 4.2e-39, 1e-39, 1e-42, 1.4e-45):
                tok, lp = _sample(x, us, T, **kw)
                assert torch.equal(tok.long(), x.argmax(-1)), (scale, T, kw)
                assert (lp == 0).all()
            for T in (5.9e-39, 8e-39, 1.1e-38, 1.2e-38, 3e-38):
                tok, lp = _sample(x, us, T, **kw)
                for i in range(len(us)):
                    want, logp, margin = S.sample_row(x[i], float(us[i]), f32(T), kw.get("top_k", 0), f32(kw.get("top_p", 1.0)),
                                                      f32(kw.get("min_p", 0.0)))
                    assert margin <= 4e-7 or int(tok[i]) == want, (scale, T, kw, i)


def test_top_k_of_any_integer():
    """A top_k beyond 32 bits is beyond every vocabulary: off; a negative one is refused."""
    x = torch.randn(5, 300, generator=torch.Generator().manual_seed(1)).cuda()
    u = torch.rand(5, generator=torch.Generator().manual_seed(2)).cuda()
    want = R.sample_tokens(x, u)
    for k in (300, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 1, 2 ** 63 - 1):
        assert torch.equal(R.sample_tokens(x, u, top_k=k), want), k
    for k in (-1, -2 ** 32, -2 ** 40):
        with pytest.raises(R.RdtError):
            R.sample_tokens(x, u, top_k=k)
