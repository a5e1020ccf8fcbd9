"""Plain 64-bit CPU forms of the serving operators, written from their definitions (no code of
the package), and the bounds the tests hold the kernels to."""
import math

import torch

F64 = torch.float64
E4M3 = torch.float8_e4m3fn
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}    # largest relative rounding error


def quantise(x: torch.Tensor):
    """e4m3 values and exponent bytes of rows [..., hd], one row at a time in Python integers:
    the smallest E in -127..127 with amax <= 448 * 2^E over the finite values."""
    x = x.detach().cpu().double()
    fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros((), dtype=F64))
    amax = fin.amax(-1)
    E = torch.full(amax.shape, -127, dtype=torch.int64)
    for i in torch.nonzero(amax > 0).tolist():
        a = float(amax[tuple(i)])
        e = max(math.frexp(a)[1] - 10, -127)
        while e < 127 and a > 448.0 * 2.0 ** e:
            e += 1
        E[tuple(i)] = e
    y = torch.ldexp(x, -E.unsqueeze(-1))
    y = torch.where(torch.isfinite(y), y, torch.full((), float("nan"), dtype=F64))
    return y.float().to(E4M3), (E + 127).to(torch.uint8)


def dequantise(q: torch.Tensor, ex: torch.Tensor) -> torch.Tensor:
    return torch.ldexp(q.cpu().float().double(), ex.cpu().to(torch.int64).unsqueeze(-1) - 127)


def make_cache(R, batch, Hkv, hd, t_max, page, dtype, quant, seed, n_loops=1, fill=True, scatter=True, spare=2):
    """A paged cache with its pages in random order (some unused), filled with normal values."""
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    per = -(-t_max // page)
    n_pages = batch * per + spare
    perm = torch.randperm(n_pages, generator=g)[:batch * per] if scatter else torch.arange(batch * per)
    table = perm.to(torch.int32).reshape(batch, per)
    shape = (n_loops, n_pages, Hkv, page, hd)
    parts = []
    for _ in range(2):
        x = torch.randn(shape, generator=g) if fill else torch.zeros(shape)
        x = x.to(dt)
        if quant:
            parts.append(fast_quantise(x))
        else:
            parts.append((x, None))
    (k, ke), (v, ve) = parts
    dev = lambda t: None if t is None else t.cuda()
    return R.PagedKVCache(dev(k), dev(v), table.cuda(), dev(ke), dev(ve), dtype=dtype)


def fast_quantise(x):
    """quantise() on finite values, vectorised (frexp)."""
    amax = x.double().abs().amax(-1)
    m, e = torch.frexp(amax)
    E = torch.where(amax > 0, (e - 9 + (m > 0.875).int()).clamp(-127, 127), torch.full_like(e, -127)).to(torch.int64)
    return torch.ldexp(x.double(), -E.unsqueeze(-1)).float().to(E4M3), (E + 127).to(torch.uint8)


def cached(cache, b, n, loop=0):
    """K and V [Hkv, n, hd] in 64 bits of positions 0 .. n - 1 of sequence b (CPU)."""
    table = cache.page_table.cpu().long()[b]
    out = []
    for x, ex in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
        rows = []
        for t in range(-(-n // cache.page_size)):
            page = int(table[t])
            if ex is None:
                rows.append(x[loop, page].cpu().double())
            else:
                rows.append(dequantise(x[loop, page], ex[loop, page]))
        out.append(torch.cat(rows, dim=1)[:, :n] if rows else torch.zeros(cache.n_kv_heads, 0, cache.head_dim, dtype=F64))
    return out


def attention(q, K, V, scale):
    """q [H, hd], K, V [Hkv, n, hd] in 64 bits -> (o [H, hd], bound on |o - computed| before the
    output's rounding).

    The bound, with u = 2^-24: a score is a sum of hd products of exact inputs, in any order,
    off by at most (hd + 4) u scale sum |q_d k_d| =: ds (the 4: the factor scale * log2 e, its
    product and the subtraction of the maximum); a weight 2^x is then off by 2 ds + 2^-21
    relatively (two ulp of exp2, |x| u from rounding x; |x| < 32 matters, below that the weight
    is under 2^-32); the sums of n weights and of n weighted values by (n + 16) u each, and the
    weights enter the second sum rounded to 11 bits or more, 2^-12 with the values below the
    half type's range off by 2^-25 of the largest, n of them at most."""
    H, Hkv, n = q.shape[0], K.shape[0], K.shape[1]
    if n == 0:
        return torch.zeros_like(q, dtype=F64), torch.zeros(H, 1, dtype=F64)
    u = 2.0 ** -24
    qd = q.double().reshape(Hkv, H // Hkv, -1)
    s = torch.einsum("ghd,gjd->ghj", qd, K) * scale
    sa = torch.einsum("ghd,gjd->ghj", qd.abs(), K.abs()).amax(-1) * abs(scale)
    p = torch.softmax(s, -1)
    o = torch.einsum("ghj,gjd->ghd", p, V)
    ds = (q.shape[-1] + 4) * u * sa + s.abs().amax(-1) * 2 * u
    vmax = V.abs().amax(dim=(1, 2))[:, None]
    rel = 2 * (2 * ds + 2.0 ** -21) + 2 * (n + 16) * u
    return o.reshape(H, -1), (rel * vmax).reshape(H, 1), (vmax * torch.ones_like(sa)).reshape(H, 1)


def check_attention(cache, q, lens, out, scale=None, loop=0, half_weights=None):
    """Every sequence against attention(); returns the largest error / bound."""
    scale = 1.0 / math.sqrt(cache.head_dim) if scale is None else scale
    worst = 0.0
    half = cache.quantised and cache.dtype == "bf16" if half_weights is None else half_weights
    for b in range(q.shape[0]):
        n = max(0, min(int(lens[b]), cache.t_max))
        got = out[b].cpu().double()
        if n == 0:
            assert torch.equal(got, torch.zeros_like(got)), b
            continue
        K, V = cached(cache, b, n, loop)
        o, tol, vmax = attention(q[b].cpu(), K, V, scale)
        tol = tol + HALF_STEP[out.dtype] * o.abs() * 1.01
        if out.dtype == torch.bfloat16:
            # weights of 16 bits (two bf16 words); with an e4m3 cache of 11 (fp16), relative to
            # the largest weight times its value
            tol = tol + (2.0 ** -11 + n * 2.0 ** -25 if half else 2.0 ** -16) * vmax
        err = (got - o).abs()
        assert torch.isfinite(got).all(), b
        ratio = float((err / tol.clamp_min(1e-30)).max())
        assert ratio <= 1.0, f"sequence {b} (length {n}): error {float(err.max()):.3e} is {ratio:.2f} of its bound"
        worst = max(worst, ratio)
    return worst


def sample_interval(x, tok, T=1.0, k=0, p=1.0, m=0.0):
    """The share of the kept weight before token tok and up to it, over the tokens that
    sample_row's definition keeps (tok itself joins them if it is not one)."""
    x = x.detach().cpu().double()
    val, idx = torch.sort(x, descending=True, stable=True)
    w = torch.exp((val - val[0]) / T)
    keep = torch.arange(len(x)) < (k or len(x))
    w = torch.where(keep, w, torch.zeros((), dtype=F64))
    if p < 1:
        keep &= torch.cumsum(w, 0) - w < p * w.sum()
    if m > 0:
        keep &= (val - val[0]) / T >= math.log(m)
    full = torch.zeros_like(w).scatter_(0, idx, torch.where(keep, w, torch.zeros((), dtype=F64)))
    full[tok] = math.exp((float(x[tok]) - float(val[0])) / T)
    c = torch.cumsum(full, 0) / full.sum()
    return float(c[tok] - full[tok] / full.sum()), float(c[tok])


def sample_row(x, u, T=1.0, k=0, p=1.0, m=0.0):
    """The sampled token of one row, from the definition in 64 bits: (token, logprob, margin),
    margin the smallest relative distance of u and of top-p's border to the running sums that
    decide the token (a computation in fewer bits may differ only where it is tiny)."""
    x = x.detach().cpu().double()
    live = ~torch.isnan(x)
    xs = torch.where(live, x, torch.full((), -math.inf, dtype=F64))
    mx = float(xs.max()) if live.any() else -math.inf
    if not T > 0 or mx == -math.inf:
        hit = torch.nonzero(live & (xs == mx))
        return (int(hit[0]) if hit.numel() else 0), 0.0, 1.0
    order = sorted(range(len(xs)), key=lambda v: (-float(xs[v]), v))
    order = [v for v in order if bool(live[v])]
    w = {v: (1.0 if float(xs[v]) == mx else round(math.exp((float(xs[v]) - mx) / T) * 2.0 ** 44) * 2.0 ** -44) for v in order}
    margin = 1.0
    if k > 0:
        order = order[:k]
    if p < 1:
        total, before, kept = math.fsum(w[v] for v in order), 0.0, []
        border = max(p, 0.0) * total
        for i, v in enumerate(order):
            if i and not before < border:
                break
            kept.append(v)
            before += w[v]
        c = 0.0
        for v in order:
            margin = min(margin, abs(c - border) / total) if c > 0 and p > 0 else margin
            c += w[v]
        order = kept
    if m > 0:
        lim = math.log(min(m, 1.0)) * T
        first = order[0]
        order = [v for v in order if v == first or float(xs[v]) - mx >= lim or float(xs[v]) == mx]
    total = math.fsum(w[v] for v in order)
    target = min(max(u, 0.0), 1.0) * total if u == u else 0.0
    c, tok = 0.0, None
    for v in sorted(order):
        c += w[v]
        if tok is None and w[v] > 0 and c > target:
            tok = v
        margin = min(margin, abs(c - target) / total) if w[v] > 1e-9 and c < total * (1 - 1e-12) else margin
    if tok is None:
        tok = max(v for v in order if w[v] > 0)
    return tok, (0.0 if float(xs[tok]) == mx else (float(xs[tok]) - mx) / T) - math.log(total), margin
