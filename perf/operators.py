"""The serving operators of the decode path, as cases to measure: the paged key / value cache
(written, read back, attended by one new token) and the sampled next token.

Each case is a dict of plain values; prepare() makes what a serving program holds before the
call, run() makes the one call.  With own = False run() computes the operator from its formula
with elementary torch operations; with own = True it calls the library's entry point.

  write   K/V rows of new tokens into the pages of their sequences, in the model dtype or as
          e4m3 with one power-of-two scale (a biased exponent byte) per token and kv head
  read    the cached positions of every sequence as contiguous K/V in the model dtype
  attn    one query token per sequence over its cached keys, GQA
  sample  one token per row of logits: temperature, top-k, top-p, min-p and one uniform number
"""
import math

import torch

own = False

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"fp32": 4, "bf16": 2}


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def _write(name, batch, seq, kv_heads, hd, page, dtype, kv, **kw):
    return {"name": name, "op": "write", "batch": batch, "seq": seq, "kv_heads": kv_heads, "hd": hd, "page": page,
            "dtype": dtype, "kv": kv, "len_lo": kw.get("len_lo", 0), "len_hi": kw.get("len_hi", 0)}


def _read(name, batch, kv_heads, hd, len_lo, len_hi, page, dtype, kv):
    return {"name": name, "op": "read", "batch": batch, "kv_heads": kv_heads, "hd": hd, "len_lo": len_lo,
            "len_hi": len_hi, "page": page, "dtype": dtype, "kv": kv}


def _attn(name, batch, heads, kv_heads, hd, len_lo, len_hi, page, dtype, kv):
    return {"name": name, "op": "attn", "batch": batch, "heads": heads, "kv_heads": kv_heads, "hd": hd,
            "len_lo": len_lo, "len_hi": len_hi, "page": page, "dtype": dtype, "kv": kv}


def _sample(name, rows, vocab, spread, mix):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "spread": spread, "mix": mix}


def listed():
    return [
        # a decode step of 64 sequences (8 kv heads of 128) appends one quantised token each
        _write("write_step_e4m3", 64, 1, 8, 128, 16, "bf16", "e4m3", len_lo=100, len_hi=4200),
        # the prompts of two long sequences (the 10B-shaped prefill) are quantised into their pages
        _write("write_prompt_e4m3", 2, 8192, 8, 128, 16, "bf16", "e4m3"),
        # the earlier part of one prompt is read back for the next chunk, fp32 parity mode, odd length
        _read("read_chunk_fp32", 1, 2, 32, 777, 777, 16, "fp32", "e4m3"),
        # 64 ragged quantised sequences are read back for a chunked prefill
        _read("read_batch_e4m3", 64, 8, 128, 37, 4224, 16, "bf16", "e4m3"),
        # the smallest decode: two short sequences of the usage script's model in fp32
        _attn("attn_tiny_fp32", 2, 8, 2, 32, 17, 24, 16, "fp32", "model"),
        # one user with a long context: the cache's length is all there is to split
        _attn("attn_one_long", 1, 32, 8, 128, 131071, 131071, 64, "bf16", "model"),
        # 64 ragged sequences of the 3B-shaped decode (24 query heads on 8 kv heads)
        _attn("attn_batch_bf16", 64, 24, 8, 128, 1, 4224, 16, "bf16", "model"),
        # the same decode at full lengths on the quantised cache: the largest call
        _attn("attn_batch_e4m3", 128, 24, 8, 128, 4097, 8191, 16, "bf16", "e4m3"),
        # one row of a 201,088-token vocabulary: latency of a single user's sample
        _sample("sample_one", 1, 201088, 2.5, "nucleus"),
        # 64 rows of that vocabulary, every request with its own temperature, top-k, top-p and min-p
        _sample("sample_batch_mixed", 64, 201088, 2.5, "mixed"),
        # 256 rows with flat logits: wide nuclei, the largest sample
        _sample("sample_wide", 256, 201088, 1.0, "nucleus"),
        # a small odd vocabulary with top-k alone
        _sample("sample_odd_topk", 33, 1001, 3.0, "topk"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "sample", "sample"])
    if op == "sample":
        vocab = rng.choice([201088, _log_int(rng, 2, 262144), _log_int(rng, 20000, 200000)])
        rows = _log_int(rng, 1, max(1, min(512, 256 * 201088 // vocab)))
        c = _sample("", rows, vocab, rng.uniform(0.5, 4.0), rng.choice(["mixed", "nucleus", "topk", "minp", "plain"]))
    else:
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        hd = rng.choice([64, 128, 128, 128, 32, 96, 80])
        kv_heads = rng.choice([1, 2, 4, 8])
        page = rng.choice([16, 16, 32, 64, 128, 8])
        kv = rng.choice(["model", "e4m3"])
        batch = _log_int(rng, 1, 256)
        # keys (or rows) of one call: at most half a million positions of one kv head of 128
        most = (1 << 20) * 128 // (hd * kv_heads)
        if dtype == "fp32":
            most //= 4
        hi = _log_int(rng, 1, max(2, min(131072, most // batch)))
        lo = rng.choice([hi, 0, 1, rng.randint(0, hi)])
        lo = min(lo, hi)
        if op == "attn":
            c = _attn("", batch, kv_heads * rng.choice([1, 2, 3, 4, 7, 8]), kv_heads, hd, lo, hi, page, dtype, kv)
        elif op == "read":
            c = _read("", batch, kv_heads, hd, lo, hi, page, dtype, kv)
        elif rng.random() < 0.5:
            c = _write("", batch, 1, kv_heads, hd, page, dtype, kv, len_lo=lo, len_hi=min(hi, 16384))
            c["len_lo"] = min(c["len_lo"], c["len_hi"])
        else:
            batch = min(batch, 16)
            c = _write("", batch, max(1, min(hi, 16384 // batch)), kv_heads, hd, page, dtype, kv)
    del c["name"]
    return c


def _lens(case):
    """Lengths of the sequences: spread evenly over len_lo .. len_hi, out of order."""
    B, lo, hi = case["batch"], case["len_lo"], case["len_hi"]
    step = 37 if B % 37 else 41
    return [lo + ((b * step + 11) % B) * (hi - lo) // max(B - 1, 1) for b in range(B)]


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": 4 * n + case["rows"] * 32, "flops": 8 * n}
    es, hd, Hkv = _SIZE[case["dtype"]], case["hd"], case["kv_heads"]
    stored = es * hd if case["kv"] == "model" else hd + 1          # one head of one position, K or V
    if case["op"] == "write":
        rows = case["batch"] * case["seq"]
        return {"bytes": rows * (2 * Hkv * (es * hd + stored) + 8), "flops": 4 * rows * Hkv * hd}
    keys = sum(_lens(case))
    table = 4 * sum(-(-n // case["page"]) for n in _lens(case))
    if case["op"] == "read":
        return {"bytes": 2 * keys * Hkv * (stored + es * hd) + table, "flops": 2 * keys * Hkv * hd}
    H = case["heads"]
    return {"bytes": 2 * keys * Hkv * stored + table + 2 * case["batch"] * H * hd * es, "flops": 4 * keys * H * hd}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    return g


def _rows(g, n, heads, hd, dtype):
    """K or V rows: normal values, each head of each row with a size of its own, some channels
    larger than the others (as trained keys have them)."""
    x = torch.randn(n, heads, hd, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(n, heads, 1, generator=g, device="cuda"))
    x[..., ::16] *= 3.0
    return x.to(dtype)


def _split(x):
    """e4m3 values and biased exponents of rows [..., hd]: x = q * 2^(exp - 127), the exponent the
    smallest that brings the row's largest magnitude to at most 448."""
    amax = x.float().abs().amax(-1)
    m, e = torch.frexp(amax)                                        # amax = m 2^e, 0.5 <= m < 1
    ex = torch.where(amax > 0, (e - 9 + (m > 0.875).int()).clamp(-127, 127), torch.full_like(e, -127))
    q = (x.double() * torch.exp2(-ex.double()).unsqueeze(-1)).float().to(torch.float8_e4m3fn)
    return q, (ex + 127).to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "sample":
        return _prepare_sample(case, g)
    dt, hd, Hkv, B, ps = _DT[case["dtype"]], case["hd"], case["kv_heads"], case["batch"], case["page"]
    s = {"case": case, "dt": dt}
    if case["op"] == "write" and case["seq"] > 1:
        lens = [case["seq"]] * B
    elif case["op"] == "write":
        lens = [n + 1 for n in _lens(case)]                         # the new token's position is len - 1
    else:
        lens = _lens(case)
    per_seq = max(1, -(-max(lens) // ps))
    n_pages = B * per_seq
    # pages handed out in random order; the pool has one page more than the cache uses
    s["table"] = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).reshape(B, per_seq)
    quant = case["kv"] == "e4m3"
    pool_dt = torch.float8_e4m3fn if quant else dt
    for name in ("k", "v"):
        pool = torch.zeros(1, n_pages + 1, Hkv, ps, hd, dtype=pool_dt, device="cuda")
        exps = torch.zeros(1, n_pages + 1, Hkv, ps, dtype=torch.uint8, device="cuda") if quant else None
        if case["op"] != "write":
            for p0 in range(0, n_pages, 4096):                      # filled in pieces: little extra memory
                n = min(4096, n_pages - p0)
                x = _rows(g, n * Hkv * ps, 1, hd, dt).reshape(n, Hkv, ps, hd)
                if quant:
                    pool.view(torch.uint8)[0, p0:p0 + n], exps[0, p0:p0 + n] = (lambda q, e: (q.view(torch.uint8), e))(*_split(x))
                else:
                    pool[0, p0:p0 + n] = x
        s[name + "_pool"], s[name + "_exps"] = pool, exps
        s[name], s[name + "_exp"] = pool[:, :n_pages], exps[:, :n_pages] if quant else None
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["op"] == "write":
        T = case["seq"]
        s["new_k"], s["new_v"] = _rows(g, B * T, Hkv, hd, dt), _rows(g, B * T, Hkv, hd, dt)
        pos = (s["lens"][:, None] - T + torch.arange(T, device="cuda", dtype=torch.int32)[None]).contiguous()
        if T > 1:                                                   # sequence b is padded by its last 3 b rows
            fill = (torch.arange(B, device="cuda")[:, None] * 3 + torch.arange(T, device="cuda")[None]) >= T
            pos[fill] = -1
        s["pos"] = pos.reshape(-1)
    elif case["op"] == "read":
        s["out"] = tuple(torch.zeros(B, Hkv, max(lens), hd, dtype=dt, device="cuda") for _ in range(2)) if max(lens) else ()
    else:
        s["q"] = torch.randn(B, case["heads"], hd, generator=g, device="cuda").to(dt)
        s["out"] = torch.zeros(B, case["heads"], hd, dtype=dt, device="cuda")
    if own:
        import recurrent_depth_moe_b200 as R
        s["cache"] = R.PagedKVCache(s["k"], s["v"], s["table"], s["k_exp"], s["v_exp"], dtype=case["dtype"])
        if case["op"] == "attn":
            s["ws"] = R.paged_attention_workspace(s["cache"], case["heads"])
    return s


def _prepare_sample(case, g):
    n, V = case["rows"], case["vocab"]
    x = torch.randn(n, V, generator=g, device="cuda") * case["spread"]
    # a few likely tokens above the rest, and some masked ones
    top = torch.randint(0, V, (n, 24), generator=g, device="cuda")
    x.scatter_add_(1, top, 4.0 * case["spread"] * torch.rand(n, 24, generator=g, device="cuda"))
    masked = torch.rand(n, V, generator=g, device="cuda") < 0.01
    masked[:, 0] = False
    x.masked_fill_(masked, float("-inf"))
    u = torch.rand(n, generator=g, device="cuda")
    f = lambda lo, hi: lo + (hi - lo) * torch.rand(n, generator=g, device="cuda")
    t, k, p, m = f(0.6, 1.2), torch.zeros(n, device="cuda"), torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    mix = case["mix"]
    if mix in ("mixed", "topk"):
        k = torch.randint(1, 257, (n,), generator=g, device="cuda").float()
    if mix in ("mixed", "nucleus"):
        p = f(0.7, 0.98)
    if mix in ("mixed", "minp"):
        m = f(0.0, 0.2)
    if mix == "mixed":                                              # every request asks for something else
        ask = torch.randint(0, 8, (n,), generator=g, device="cuda")
        k, p, m = torch.where((ask & 1) > 0, k, 0), torch.where((ask & 2) > 0, p, 1), torch.where((ask & 4) > 0, m, 0)
        t[::9] = 0.0                                                # and some the most likely token
    return {"case": case, "logits": x, "u": u, "temperature": t, "top_k": k.to(torch.int32), "top_p": p, "min_p": m}


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import recurrent_depth_moe_b200 as R
    op = s["case"]["op"]
    if op == "write":
        R.paged_kv_write(s["new_k"], s["new_v"], s["pos"], s["cache"], seq=s["case"]["seq"])
        return _pools(s)
    if op == "read":
        if not s["out"]:
            return {"n": 0}
        R.paged_kv_read(s["lens"], s["cache"], out=s["out"])
        return {"k": s["out"][0], "v": s["out"][1]}
    if op == "attn":
        return {"o": R.paged_attention(s["q"], s["lens"], s["cache"], out=s["out"], workspace=s["ws"])}
    tok, lp = R.sample_tokens(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                              return_logprob=True)
    return {"token": tok, "logprob": lp}


def _pools(s):
    r = {"k": s["k"], "v": s["v"]}
    if s["k_exp"] is not None:
        r["k_exp"], r["v_exp"] = s["k_exp"], s["v_exp"]
    return r


def _values(s, name, pages):
    """fp32 values of the pages `pages` [B, P]: [B, Hkv, P * page, hd]."""
    if s[name + "_exp"] is not None:
        x = s[name].view(torch.uint8)[0][pages].view(torch.float8_e4m3fn).float()
        x = x * torch.exp2(s[name + "_exp"][0][pages].float() - 127.0).unsqueeze(-1)
    else:
        x = s[name][0][pages].float()
    B, P, Hkv, ps, hd = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, P * ps, hd)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "sample":
        return _plain_sample(s)
    if case["op"] == "write":
        pos, ps = s["pos"].long(), case["page"]
        b = torch.arange(pos.numel(), device="cuda") // case["seq"]
        page = s["table"].long()[b, pos.clamp_min(0) // ps]
        page = torch.where(pos >= 0, page, s["k_pool"].shape[1] - 1)  # padding rows go to the unused page
        slot = pos.clamp_min(0) % ps
        for name in ("k", "v"):
            x = s["new_" + name]
            if s[name + "_exps"] is not None:
                q, e = _split(x)
                s[name + "_pool"].view(torch.uint8)[0, page, :, slot] = q.view(torch.uint8)
                s[name + "_exps"][0, page, :, slot] = e
            else:
                s[name + "_pool"][0, page, :, slot] = x
        return _pools(s)
    pages = s["table"].long()
    if case["op"] == "read":
        if not s["out"]:
            return {"n": 0}
        for name, out in (("k", s["out"][0]), ("v", s["out"][1])):
            t = out.shape[2]
            live = (torch.arange(t, device="cuda")[None] < s["lens"][:, None])[:, None, :, None]
            out.copy_(torch.where(live, _values(s, name, pages)[:, :, :t], out.float()))
        return {"k": s["out"][0], "v": s["out"][1]}
    B, H, hd = s["q"].shape
    Hkv = case["kv_heads"]
    q = s["q"].float().reshape(B, Hkv, H // Hkv, hd)
    z = torch.matmul(q, _values(s, "k", pages).transpose(-1, -2)) * (1.0 / math.sqrt(hd))
    live = (torch.arange(z.shape[-1], device="cuda")[None] < s["lens"][:, None])[:, None, None, :]
    z = torch.where(live, z, -torch.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.where(live, torch.exp(z - m), 0.0)
    o = torch.matmul(p, _values(s, "v", pages)) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    return {"o": o.reshape(B, H, hd).to(s["dt"])}


def _plain_sample(s):
    """In 64 bits: the token hangs on which side of a border a sum falls."""
    n, V = s["logits"].shape
    x = s["logits"].double()
    x = torch.where(torch.isnan(x), -torch.inf, x)
    xs, order = torch.sort(x, dim=-1, descending=True, stable=True)  # ties: the lower index first
    t = s["temperature"].double()[:, None]
    d = torch.where(xs == xs[:, :1], 0.0, xs - xs[:, :1])
    z = d / t.clamp_min(1e-300)
    rank = torch.arange(V, device="cuda")[None]
    k = s["top_k"].long()[:, None]
    greedy = t <= 0
    keep = (rank < torch.where(k > 0, k, V)) & torch.where(greedy, rank < 1, True)
    w = torch.where(keep, torch.exp(z), 0.0)
    before = torch.cumsum(w, -1) - w
    p = s["top_p"].double()[:, None]
    keep &= (before < p * w.sum(-1, keepdim=True)) | (p >= 1) | (rank < 1)
    keep &= (z >= torch.log(s["min_p"].double()[:, None])) | (rank < 1)
    w = torch.where(keep, w, 0.0)
    wi = torch.zeros_like(w).scatter_(1, order, w)                  # back in the vocabulary's order
    cum = torch.cumsum(wi, -1)
    total = cum[:, -1:]
    tok = ((cum <= s["u"].double()[:, None] * total) | (wi == 0)).to(torch.int8).argmin(-1)
    lp = torch.log(wi.gather(1, tok[:, None]) / total)[:, 0]
    return {"token": tok.to(torch.int32), "logprob": lp.float()}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"] == "write":
        return None                                                 # bytes: nothing to compute in 64 bits
    B, ps, lens, table = case["batch"], case["page"], s["lens"].tolist(), s["table"].long()

    def seq(name, b):
        """[Hkv, len, hd] in 64 bits: the sequence's pages one after another."""
        pages = table[b, :max(1, -(-lens[b] // ps))]
        if s[name + "_exp"] is not None:
            x = s[name].view(torch.uint8)[0, pages].view(torch.float8_e4m3fn).double()
            x = torch.ldexp(x, s[name + "_exp"][0, pages].to(torch.int32).unsqueeze(-1) - 127)
        else:
            x = s[name][0, pages].double()
        return torch.cat(list(x), dim=1)[:, :lens[b]]

    if case["op"] == "read":
        if not s["out"]:
            return None
        out = {}
        for name, buf in (("k", s["out"][0]), ("v", s["out"][1])):
            o = buf.double()
            for b in range(B):
                o[b, :, :lens[b]] = seq(name, b)
            out[name] = o
        return out
    H, hd = case["heads"], case["hd"]
    o = torch.zeros(B, H, hd, dtype=torch.float64, device="cuda")
    for b in range(B):
        if lens[b]:
            K, Vv = seq("k", b), seq("v", b)
            a = torch.einsum("hgd,hjd->hgj", s["q"][b].double().view(K.shape[0], -1, hd), K) / math.sqrt(hd)
            o[b] = torch.einsum("hgj,hjd->hgd", torch.softmax(a, -1), Vv).reshape(H, hd)
    return {"o": o}


def _exact_sample(s):
    n, V = s["logits"].shape
    toks, lps = [], []
    par = torch.stack([s["u"].double(), s["temperature"].double(), s["top_k"].double(), s["top_p"].double(),
                       s["min_p"].double()], 1).tolist()
    for i, (u, t, k, p, m) in enumerate(par):
        x = s["logits"][i].double()
        if t <= 0:
            toks.append(int(torch.nonzero(x == x.max())[0]))
            lps.append(0.0)
            continue
        val, idx = torch.sort(x, descending=True, stable=True)
        if k > 0:
            val, idx = val[:int(k)], idx[:int(k)]
        pr = torch.softmax(val / t, 0)
        if p < 1:
            c = torch.cumsum(pr, 0)
            cut = max(1, int((c - pr < p).sum()))
            pr, idx = pr[:cut], idx[:cut]
        if m > 0:
            live = pr >= m * pr[0]
            pr, idx = pr[live], idx[live]
        by_index = torch.argsort(idx)
        idx, pr = idx[by_index], pr[by_index] / pr.sum()
        c = torch.cumsum(pr, 0)
        j = min(int(torch.searchsorted(c, torch.tensor(u * float(c[-1]), dtype=torch.float64, device="cuda"), right=True)), len(idx) - 1)
        toks.append(int(idx[j]))
        lps.append(float(torch.log(pr[j])))
    return {"token": torch.tensor(toks, dtype=torch.int32), "logprob": torch.tensor(lps, dtype=torch.float64)}
