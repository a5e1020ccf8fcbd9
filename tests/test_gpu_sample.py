"""Sampled next tokens on the GPU against the definition in 64 bits (CPU).

A weight computed in fp32 words is off by at most 2^-22 relatively, so a border moves by at most
2^-21 of the total: rows whose 64-bit margin (distance of u, or of top-p's border, to a running
sum) is above 4e-7 must give the same token, and the inputs are checked to have few others."""
import math

import pytest
import torch

from tests import _serving as S

pytestmark = pytest.mark.gpu

R = pytest.importorskip("recurrent_depth_moe_b200")
MARGIN = 4e-7
ALL = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    R.load_library()


def _check(x, u, T, k, p, m, got, lp, max_near=0):
    near = 0
    for i in range(x.shape[0]):
        at = lambda a: float(a[i]) if isinstance(a, torch.Tensor) else a
        tok, logp, margin = S.sample_row(x[i], float(u[i]), at(T), int(at(k)), at(p), at(m))
        if margin <= MARGIN:
            near += 1
            if max_near == ALL:                       # the drawn token's share holds u, up to two borders' movement
                lo, hi = S.sample_interval(x[i], int(got[i]), at(T), int(at(k)), at(p), at(m))
                assert lo - 2 * MARGIN <= float(u[i]) <= hi + 2 * MARGIN, i
            continue
        assert int(got[i]) == tok, f"row {i}: token {int(got[i])}, the definition's is {tok} (margin {margin:.2e})"
        # a logarithm of a ratio of sums off by 2^-22, rounded to fp32
        assert abs(float(lp[i]) - logp) <= 2.0 ** -21 + 2.0 ** -23 * abs(logp), i
    assert near <= max_near, f"{near} rows too near a border to compare"


def _rows(n, V, seed, spread=2.5, masked=0.02):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, V, generator=g) * spread
    x[torch.rand(n, V, generator=g) < masked] = -math.inf
    x[:, V // 2] = 1.0
    return x, torch.rand(n, generator=g), g


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 1000, 1001, 4096, 50257])
@pytest.mark.parametrize("mode", ["plain", "topk", "topp", "minp", "all"])
def test_sample_matches_the_definition(V, mode):
    n = 24 if V < 10000 else 6
    x, u, g = _rows(n, V, V + len(mode))
    f = lambda lo, hi: lo + (hi - lo) * torch.rand(n, generator=g)
    T = f(0.4, 1.6)
    k = torch.randint(1, max(2, min(V, 300)) + 1, (n,), generator=g, dtype=torch.int32) if mode in ("topk", "all") else 0
    p = f(0.05, 0.99) if mode in ("topp", "all") else 1.0
    m = f(0.0, 0.5) if mode in ("minp", "all") else 0.0
    dev = lambda a: a.cuda() if isinstance(a, torch.Tensor) else a
    tok, lp = R.sample_tokens(x.cuda(), u.cuda(), dev(T), dev(k), dev(p), dev(m), return_logprob=True)
    _check(x, u, T, k, p, m, tok.cpu(), lp.cpu(), max_near=1 if V > 10000 else 0)
    again, lp2 = R.sample_tokens(x.cuda(), u.cuda(), dev(T), dev(k), dev(p), dev(m), return_logprob=True)
    assert torch.equal(tok, again) and torch.equal(lp, lp2)


def test_scalars_equal_rows_of_the_same_value():
    x, u, _ = _rows(16, 777, 3)
    xc, uc = x.cuda(), u.cuda()
    full = lambda v, dt=torch.float32: torch.full((16,), v, dtype=dt, device="cuda")
    a = R.sample_tokens(xc, uc, 0.7, 50, 0.9, 0.01)
    b = R.sample_tokens(xc, uc, full(0.7), full(50, torch.int32), full(0.9), full(0.01))
    assert torch.equal(a, b)
    _check(x, u, float(torch.tensor(0.7)), 50, float(torch.tensor(0.9)), float(torch.tensor(0.01)), a.cpu(),
           R.sample_tokens(xc, uc, 0.7, 50, 0.9, 0.01, return_logprob=True)[1].cpu())


def test_temperature_zero_and_top_one_are_greedy():
    x, u, _ = _rows(9, 5000, 5)
    x[3, 17] = x[3, 4000] = 50.0                                     # a tie: the lower index
    x[4] = -math.inf
    x[5] = math.nan
    x[6, 9] = math.nan
    x[7] = -math.inf
    x[7, :5] = math.nan                                              # the first -inf comes after NaN
    xc, uc = x.cuda(), u.cuda()
    want = R.greedy_tokens(xc)
    assert want.tolist()[3:6] == [17, 0, 0] and int(want[7]) == 5
    tok, lp = R.sample_tokens(xc, uc, 0.0, return_logprob=True)
    assert torch.equal(tok, want) and (lp == 0).all()
    for kw in (dict(top_k=1), dict(top_p=1e-6), dict(min_p=1.0, top_k=1)):
        assert torch.equal(R.sample_tokens(xc, uc, 0.8, **kw), want), kw


def test_ties_at_the_borders_go_to_the_lowest_index():
    """Equal logits: top-k keeps the first k by index, top-p the first tokens whose sum reaches
    it, min-p all; a whole row of equal logits is uniform over what is kept."""
    V = 3000
    x = torch.zeros(8, V)
    x[:, ::7] = -0.0                                                 # the same logit as 0
    u = torch.tensor([0.0, 0.1, 0.25, 0.5, 0.75, 0.9, 0.999, 1 - 2.0 ** -24])
    tok = R.sample_tokens(x.cuda(), u.cuda(), 1.3, top_k=10)
    assert tok.tolist() == [int(float(v) * 10) for v in u]
    tok = R.sample_tokens(x.cuda(), u.cuda(), 1.3, top_p=0.5)
    assert tok.tolist() == [int(float(v) * 1500) for v in u]
    tok = R.sample_tokens(x.cuda(), u.cuda(), 1.3, min_p=1.0)
    assert tok.tolist() == [int(float(v) * V) for v in u]
    x[:, 100:200] = 2.0                                              # 100 tied above 2900 tied
    x[:, 1500:1600] = 2.0
    tok = R.sample_tokens(x.cuda(), u.cuda(), 1.0, top_k=150)
    kept = list(range(100, 200)) + list(range(1500, 1550))
    assert tok.tolist() == [kept[int(float(v) * 150)] for v in u]
    tok, lp = R.sample_tokens(x.cuda(), u.cuda(), 1.0, top_k=201, return_logprob=True)
    _check(x, u, 1.0, 201, 1.0, 0.0, tok.cpu(), lp.cpu())


def test_wide_and_narrow_rows():
    """Spreads from nearly flat to one token far above, infinities above and below, tiny and
    large temperatures, and a uniform number of exactly 0 or just under 1."""
    V = 2048
    g = torch.Generator().manual_seed(6)
    base = torch.randn(V, generator=g)
    rows = [base * 1e-3, base, base * 10, base * 100, base * 1e30, base.clone(), base.clone(), base - 1e4, base * 1e-30,
            torch.full((V,), -3.4028234663852886e38)]
    rows[5][77] = math.inf
    rows[6][700:] = -math.inf
    rows[9][5] = 0.0
    x = torch.stack(rows)
    for uu in (0.0, 0.3, 1 - 2.0 ** -24):
        u = torch.full((len(rows),), uu)
        for T in (1.0, 1e-3, 50.0):
            for kw in (dict(), dict(top_p=0.9), dict(top_k=40), dict(top_k=300, top_p=0.99, min_p=1e-3)):
                tok, lp = R.sample_tokens(x.cuda(), u.cuda(), T, return_logprob=True, **kw)
                p = float(torch.tensor(kw.get("top_p", 1.0))); m = float(torch.tensor(kw.get("min_p", 0.0)))
                _check(x, u, float(torch.tensor(T)), kw.get("top_k", 0), p, m, tok.cpu(), lp.cpu(), max_near=2)


def test_per_row_parameters_out_of_range_are_what_the_header_says():
    x, _, g = _rows(12, 500, 8, masked=0.0)
    u = torch.tensor([0.3] * 8 + [-1.0, 2.0, math.nan, 0.5])
    inf, nan = math.inf, math.nan
    T = torch.tensor([1.0, nan, -1.0, 1.0, 1.0, 1.0, 1.0, inf, 1.0, 1.0, 1.0, 1e-45])
    k = torch.tensor([-5, 3, 3, 10 ** 9, 0, 0, 0, 0, 0, 0, 0, 0], dtype=torch.int32)
    p = torch.tensor([nan, 1.0, 1.0, 2.0, -1.0, 0.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0])
    m = torch.tensor([nan, 0.0, 0.0, -1.0, 0.0, 0.0, 7.0, 0.0, 0.0, 0.0, 0.0, 0.0])
    tok, lp = R.sample_tokens(x.cuda(), u.cuda(), T.cuda(), k.cuda(), p.cuda(), m.cuda(), return_logprob=True)
    top = x.argmax(-1)
    for i in (1, 2, 4, 5, 6, 11):
        assert int(tok[i]) == int(top[i]), i
    plain = lambda i, uu, TT=1.0: S.sample_row(x[i], uu, TT)[0]
    assert int(tok[0]) == plain(0, float(u[0])) and int(tok[3]) == plain(3, float(u[3]))
    assert int(tok[7]) == int(float(u[7]) * 500)                     # an infinite temperature: uniform
    assert int(tok[8]) == plain(8, 0.0) and int(tok[10]) == plain(10, 0.0)
    assert int(tok[9]) == plain(9, 1 - 2.0 ** -24)


def test_strides_streams_and_replay():
    """Logits rows and tokens spaced apart, a side stream, and a graph whose inputs change."""
    n, V = 7, 1003
    x, u, _ = _rows(n, V, 9)
    wide = torch.full((n, V + 13), 100.0)
    wide[:, 5:5 + V] = x
    wc, uc = wide.cuda(), u.cuda()
    view = wc[:, 5:5 + V]
    want = R.sample_tokens(x.cuda(), uc, 0.9, 50, 0.95)
    buf = torch.full((n, 3), -7, dtype=torch.int32, device="cuda")
    R.sample_tokens(view, uc, 0.9, 50, 0.95, out=buf[:, 1])
    assert torch.equal(buf[:, 1], want) and (buf[:, 0] == -7).all() and (buf[:, 2] == -7).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        t = R.sample_tokens(view, uc, 0.9, 50, 0.95)
    side.synchronize()
    assert torch.equal(t, want)
    xin, uin, out = torch.zeros(n, V, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, capture_error_mode="thread_local"):
        R.sample_tokens(xin, uin, 0.9, 50, 0.95, out=out)
    for s in (1, 2):
        y, uu, _ = _rows(n, V, 30 + s)
        xin.copy_(y), uin.copy_(uu)
        gr.replay()
        assert torch.equal(out, R.sample_tokens(y.cuda(), uu.cuda(), 0.9, 50, 0.95))


def test_frequencies():
    """20,000 draws of one row follow its kept distribution (chi-square over 8 kept tokens, 7
    degrees of freedom: 35 has probability 1e-5)."""
    x = torch.linspace(0, 3, 16).repeat(20000, 1)
    u = torch.rand(20000, generator=torch.Generator().manual_seed(10))
    tok = R.sample_tokens(x.cuda(), u.cuda(), 1.0, top_k=8).cpu()
    p = torch.softmax(x[0, 8:].double(), 0)
    cnt = torch.bincount(tok.long() - 8, minlength=8).double()
    assert int(tok.min()) >= 8
    assert float(((cnt - 20000 * p) ** 2 / (20000 * p)).sum()) < 35


@pytest.mark.parametrize("V,n", [(201088, 3), (262147, 2), ((1 << 20) - 1, 1)])
def test_large_vocabularies(V, n):
    """Large vocabularies (vectorised 64-bit form on the GPU in place of the row loop)."""
    x, u, _ = _rows(n, V, 11, spread=1.5, masked=0.01)
    xd = x.double().cuda()
    for T, k, p, m in ((1.0, 0, 1.0, 0.0), (0.8, 0, 0.9, 0.0), (1.1, 5000, 0.97, 1e-4), (1.0, 64, 1.0, 0.05)):
        tok, lp = R.sample_tokens(x.cuda(), u.cuda(), T, k, p, m, return_logprob=True)
        f32 = lambda a: float(torch.tensor(a, dtype=torch.float32))
        for i in range(n):
            val, idx = torch.sort(xd[i], descending=True, stable=True)
            w = torch.exp((val - val[0]) / f32(T))
            keep = torch.arange(V, device="cuda") < (k or V)
            w = torch.where(keep, w, 0.0)
            c = torch.cumsum(w, 0)
            border = f32(p) * c[-1]
            if p < 1:
                keep &= (c - w < border)
            if m > 0:
                keep &= (val - val[0]) / f32(T) >= math.log(f32(m))
            w = torch.where(keep, w, 0.0)
            by = torch.zeros_like(w).scatter_(0, idx, w)
            cum = torch.cumsum(by, 0)
            target = float(u[i]) * float(cum[-1])
            t = int(tok[i])
            lo = float(cum[t] - by[t]) / float(cum[-1])
            hi = float(cum[t]) / float(cum[-1])
            eps = 2e-6                                               # the drawn token's interval holds u up to the sums' rounding
            assert float(by[t]) > 0 and lo - eps <= float(u[i]) < hi + eps, (i, lo, hi, float(u[i]))
            assert abs(float(lp[i]) - math.log(float(by[t]) / float(cum[-1]))) < 1e-5


@pytest.mark.parametrize("kw", [dict(top_k=40), dict(top_k=20000), dict(top_k=59000), dict(top_p=0.9), dict(top_p=0.3), dict(top_p=0.9999),
                                dict(top_k=40, top_p=0.8), dict(top_k=20000, top_p=0.7), dict(top_k=300, top_p=0.9, min_p=0.02)])
def test_logits_of_few_distinct_values(kw):
    """Logits rounded to bf16 (hundreds of tokens share a value, so a border falls among equal
    logits and the lowest indices stay), with kept sets from tens of tokens to nearly all.  Far
    out a token holds less of the weight than MARGIN (normal logits of deviation 2 have their
    weight spread around 4 with that deviation, top_p 0.9999 ends 3.7 deviations below, at -3.4,
    where a token holds exp(-3.4 - 2) / 60000 = 8e-8 of the total), so every row is near some
    border there and is held to its token's share instead."""
    V, n = 60000, 3
    g = torch.Generator().manual_seed(51)
    x = (torch.randn(n, V, generator=g) * 2.0).bfloat16().float()
    u = torch.rand(n, generator=g)
    tok, lp = R.sample_tokens(x.cuda(), u.cuda(), 1.0, return_logprob=True, **kw)
    f32 = lambda a: float(torch.tensor(a, dtype=torch.float32))
    _check(x, u, 1.0, kw.get("top_k", 0), f32(kw.get("top_p", 1.0)), f32(kw.get("min_p", 0.0)), tok.cpu(), lp.cpu(), max_near=ALL)


@pytest.mark.parametrize("V", [4000, 60000, 201088, 500000])
def test_rows_of_one_value(V):
    """Every logit the same: top-k and top-p keep the first indices, and the draw is uniform over
    them; also with one token above the rest, and with all weight in few equal tokens."""
    u = torch.tensor([0.0, 0.3, 0.77, 1 - 2.0 ** -24])
    x = torch.full((4, V), -1.5)
    k = V // 3
    tok = R.sample_tokens(x.cuda(), u.cuda(), 0.9, top_k=k)
    assert tok.tolist() == [int(float(a) * k) for a in u]
    tok = R.sample_tokens(x.cuda(), u.cuda(), 0.9, top_p=0.5)        # the first whose sum reaches half: ceil(V / 2) of them
    assert tok.tolist() == [int(float(a) * ((V + 1) // 2)) for a in u]
    x[:, V - 1] = 40.0
    for kw in (dict(), dict(top_p=0.9), dict(top_k=5), dict(top_k=k, top_p=0.9)):
        assert R.sample_tokens(x.cuda(), u.cuda(), 1.0, **kw).tolist()[1:] == [V - 1] * 3, kw
    x[:, V // 2:V // 2 + 1500] = 40.0                                # 1501 equal tokens above all others
    pos = list(range(V // 2, V // 2 + 1500)) + [V - 1]
    assert R.sample_tokens(x.cuda(), u.cuda(), 1.0, top_k=1200).tolist() == [pos[int(float(a) * 1200)] for a in u]
    kept = math.ceil(float(torch.tensor(0.5)) * 1501)
    assert R.sample_tokens(x.cuda(), u.cuda(), 1.0, top_p=0.5, min_p=0.5).tolist() == [pos[int(float(a) * kept)] for a in u]


def test_two_streams_at_once():
    """Two calls in flight together, each as alone (no state is shared between calls)."""
    x, u, g = _rows(40, 50257, 61)
    y, v, _ = _rows(40, 50257, 62)
    xc, uc, yc, vc = x.cuda(), u.cuda(), y.cuda(), v.cuda()
    a, b = R.sample_tokens(xc, uc, 0.8, top_p=0.9), R.sample_tokens(yc, vc, 1.2, 64)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a2 = R.sample_tokens(xc, uc, 0.8, top_p=0.9)
        with torch.cuda.stream(s2):
            b2 = R.sample_tokens(yc, vc, 1.2, 64)
        torch.cuda.synchronize()
        assert torch.equal(a, a2) and torch.equal(b, b2)
