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
