"""One-token attention over pages whose value rows differ by many powers of two from the ones that
carry the softmax's weight, and over infinite keys and values, against the definition in 64 bits.

The bound holds each channel to its own sum.  With u = 2^-24, p_j the exact weights and ds the
error of a score (tests/_serving.py:attention): a computed weight is off by 2 ds + 2^-21
relatively, its share of the sum of weights by as much again, and the sums by (n + 16) u; a weight
that enters the second product as two 16-bit words is off by 2^-16 of itself in bf16, by 2^-22 in
fp16, so
  rel = 2 (2 ds + 2^-21) + 2 (n + 16) u + 2^-16 (bf16 cache) or 2^-21 (e4m3 cache),
and rel sum_j p_j |v_jd| bounds what these make of channel d.  An fp16 word ends at 2^-24: each of
n weights is off by up to 2^-25 more, where the largest weight times its row's scale so far stands
at 2^7 or more (2^15, less up to 2^8 for rows within that of the largest scale).  A row's largest
value is above 224 of its scale and a channel at most 448 of it, so this adds n 2^-31 max_j p_j
max_d |v_jd| at most.  A weight below the smallest normal number may be nothing: 2^-126 sum_j |v_jd|
(it shows where every other value of a channel is an exact 0).  The output's own rounding adds half
a step."""
import math

import pytest
import torch

from tests import _serving as S

pytestmark = pytest.mark.gpu

R = pytest.importorskip("recurrent_depth_moe_b200")
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    R.load_library()


def _cache(K, V, page, dtype, quant, seed=0):
    """One sequence's keys and values [Hkv, n, hd] in a cache of scattered pages."""
    Hkv, n, hd = K.shape
    per = -(-n // page)
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(per + 2, generator=g)[:per].to(torch.int32).reshape(1, per)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    parts = []
    for x in (K, V):
        pages = torch.zeros(per + 2, Hkv, page, hd, dtype=dt)
        for t in range(per):
            rows = x[:, t * page:(t + 1) * page]
            pages[table[0, t], :, :rows.shape[1]] = rows.to(dt)
        parts.append(S.fast_quantise(pages) if quant else (pages, None))
    (k, ke), (v, ve) = [(a[None].cuda(), None if b is None else b[None].cuda()) for a, b in parts]
    return R.PagedKVCache(k, v, table.cuda(), ke, ve, dtype=dtype)


def _check(cache, q, n, out, without=()):
    """Largest error over its bound (module docstring), and the exact output, of positions 0 .. n - 1
    but those of `without`."""
    H, hd = q.shape
    keep = [j for j in range(n) if j not in without]
    K, V = (x[:, keep] for x in S.cached(cache, 0, n))
    Hkv, u, scale = K.shape[0], 2.0 ** -24, 1.0 / math.sqrt(hd)
    qd = q.cpu().double().reshape(Hkv, H // Hkv, hd)
    s = torch.einsum("ghd,gjd->ghj", qd, K) * scale
    sa = torch.einsum("ghd,gjd->ghj", qd.abs(), K.abs()).amax(-1) * scale
    p = torch.softmax(s, -1)
    o = torch.einsum("ghj,gjd->ghd", p, V)
    ds = ((hd + 4) * u * sa + s.abs().amax(-1) * 2 * u)[..., None]
    words = 0.0 if cache.dtype == "fp32" else 2.0 ** -21 if cache.quantised else 2.0 ** -16
    rel = 2 * (2 * ds + 2.0 ** -21) + 2 * (n + 16) * u + words
    tol = rel * torch.einsum("ghj,gjd->ghd", p, V.abs())
    if cache.quantised and cache.dtype == "bf16":
        tol = tol + n * 2.0 ** -31 * (p * V.abs().amax(-1)[:, None]).amax(-1)[..., None]
    tol = tol + 2.0 ** -126 * V.abs().sum(1)[:, None]
    tol = tol + 1.01 * S.HALF_STEP[out.dtype] * o.abs()
    got = out.cpu().double().reshape(o.shape)
    assert torch.isfinite(got).all()
    ratio = float(((got - o).abs() / tol.clamp_min(1e-300)).max())
    return ratio, o


def _steer(K, q, rows, sign, hd, by=60.0):
    """Moves the scores of `rows` by +-by (natural units, per query head's sign), through channel 0."""
    K[:, :, 0] = 0.0
    K[:, rows, 0] = 4.0
    q[:, 0] = sign * by * math.sqrt(hd) / 4.0


CASES = [("bf16", 128, 16), ("bf16", 64, 16), ("bf16", 256, 32), ("bf16", 128, 8), ("bf16", 96, 16), ("bf16", 40, 16),
         ("fp32", 128, 16)]


@pytest.mark.parametrize("share", [0.5, 1e-2, 1e-3, 1e-6, 1e-9])
@pytest.mark.parametrize("dtype,hd,page", CASES)
@pytest.mark.parametrize("quant", [True, False])
def test_attention_sink_without_a_value(quant, dtype, hd, page, share):
    """A first key that takes all but `share` of the weight and has next to no value (or none)."""
    n, Hkv, G = 4700, 2, 4
    g = torch.Generator().manual_seed(hd + page)
    K = torch.randn(Hkv, n, hd, generator=g)
    V = torch.randn(Hkv, n, hd, generator=g)
    q = torch.randn(Hkv * G, hd, generator=g)
    V[0, 0] = 0.0
    V[1, 0] *= 1e-6
    # the rest weighs about n e^(1/2) of a score 0
    _steer(K, q, [0], 1.0, hd, math.log(n * math.exp(0.5) / share))
    cache = _cache(K, V, page, dtype, quant)
    q = q.to(cache.torch_dtype)
    out = R.paged_attention(q[None].cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), cache)[0]
    ratio, _ = _check(cache, q, n, out)
    assert ratio <= 1.0, ratio


@pytest.mark.parametrize("up", [12, 20, 30, 45, 70])
@pytest.mark.parametrize("rows", ["first", "tile", "last", "spread", "half"])
@pytest.mark.parametrize("dtype,hd,page", CASES)
def test_large_value_rows_that_nobody_attends(dtype, hd, page, rows, up):
    """Value rows 2^up above the others: three query heads of a group give them next to no
    weight, the fourth all of it."""
    n, Hkv, G = 1300, 2, 4
    g = torch.Generator().manual_seed(up + hd)
    K = torch.randn(Hkv, n, hd, generator=g)
    V = torch.randn(Hkv, n, hd, generator=g)
    q = torch.randn(Hkv * G, hd, generator=g)
    at = dict(first=[0], tile=list(range(640, 680)), last=[n - 1], spread=list(range(5, n, 37)),
              half=list(range(n // 2)))[rows]
    V[:, at] *= 2.0 ** up
    sign = torch.tensor([-1.0, -1.0, 1.0, -1.0]).repeat(Hkv)
    _steer(K, q, at, sign, hd, 30.0 + up * math.log(2))
    cache = _cache(K, V, page, dtype, True)
    q = q.to(cache.torch_dtype)
    out = R.paged_attention(q[None].cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), cache)[0]
    ratio, o = _check(cache, q, n, out)
    assert ratio <= 1.0, ratio
    heads = o.abs().amax(-1)
    assert float(heads[:, 2].min()) > 2.0 ** (up - 6) and float(heads[:, 0].max()) < 8.0


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 65, 700, 5000])
@pytest.mark.parametrize("shape", ["rising", "falling", "any"])
@pytest.mark.parametrize("dtype,hd,page", CASES[:4] + CASES[6:])
def test_value_rows_of_every_size(dtype, hd, page, shape, n):
    """Value rows of 2^-40 to 2^40, rising or falling along the cache or in any order, under scores
    that favour the small ones for some heads and the large ones for others."""
    Hkv, G = 2, 8
    g = torch.Generator().manual_seed(n + len(shape))
    e = torch.linspace(-40, 40, n) if n > 1 else torch.tensor([17.0])
    e = e.flip(0) if shape == "falling" else e[torch.randperm(n, generator=g)] if shape == "any" else e
    K = torch.randn(Hkv, n, hd, generator=g)
    V = torch.randn(Hkv, n, hd, generator=g) * torch.exp2(e)[:, None]
    q = torch.randn(Hkv * G, hd, generator=g)
    # a head's slope: natural units of score per power of two of the value row
    slope = torch.tensor([-2.0, -1.0, -0.7, -0.69, -0.3, 0.0, 0.5, 2.0]).repeat(Hkv)
    K[:, :, 0] = e / 8
    q[:, 0] = slope * math.sqrt(hd) * 8
    cache = _cache(K, V, page, dtype, True)
    q = q.to(cache.torch_dtype)
    out = R.paged_attention(q[None].cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), cache)[0]
    ratio, _ = _check(cache, q, n, out)
    assert ratio <= 1.0, ratio


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("bf16", 40), ("bf16", 33), ("fp32", 64)])
@pytest.mark.parametrize("n", [1, 20, 2500])
def test_infinite_keys_and_values(dtype, hd, n):
    """An infinite value is its channel's output, with its sign, for every head (both signs: NaN; a
    NaN value: NaN); a key of -inf (against a positive channel of the query) takes no part."""
    Hkv, G, page = 2, 3, 16
    g = torch.Generator().manual_seed(n + hd)
    K = torch.randn(Hkv, n, hd, generator=g)
    V = torch.randn(Hkv, n, hd, generator=g)
    q = torch.randn(Hkv * G, hd, generator=g)
    r = torch.randint(0, n, (4,), generator=g)
    inf = math.inf
    V[:, r[0], 3] = inf
    V[:, r[1], 8] = -inf
    V[0, r[2], 17] = math.nan
    if n > 1:
        V[1, 0, 20] = inf
        V[1, n - 1, 20] = -inf
    cache = _cache(K, V, page, dtype, False)
    q = q.to(cache.torch_dtype)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = R.paged_attention(q[None].cuda(), lens, cache)[0].cpu().reshape(Hkv, G, hd)
    odd = torch.zeros(Hkv, G, hd, dtype=torch.bool)
    odd[:, :, [3, 8]] = True
    odd[0, :, 17] = True
    if n > 1:
        odd[1, :, 20] = True
        assert torch.isnan(out[1, :, 20]).all()
    assert (out[:, :, 3] == inf).all() and (out[:, :, 8] == -inf).all() and torch.isnan(out[0, :, 17]).all()
    assert torch.isfinite(out[~odd]).all()
    plain = V.clone()
    plain[~torch.isfinite(plain)] = 0.0
    same = R.paged_attention(q[None].cuda(), lens, _cache(K, plain, page, dtype, False))[0].cpu().reshape(Hkv, G, hd)
    assert torch.equal(out[~odd], same[~odd])                       # the other channels are as without them
    if n > 1:
        q[:, 5] = q[:, 5].abs() + 1
        K[:, r[3], 5] = -inf
        cache = _cache(K, plain, page, dtype, False)
        ratio, _ = _check(cache, q, n, R.paged_attention(q[None].cuda(), lens, cache)[0], without=(int(r[3]),))
        assert ratio <= 1.0, ratio
