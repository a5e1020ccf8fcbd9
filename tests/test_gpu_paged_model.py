"""The serving operators as the model uses them: blocks, the looped recurrent block, the decode
graph and the generator over paged caches, and sampled generation.  Compared with the same calls
over contiguous caches (which the oracle pins) at the framework's parity bounds: fp32 max
relative error 1e-4, bf16 relative L2 2e-2."""
import pytest
import torch

import rdt_inputs as RI
from tests._helpers import BF16_TOL, FP32_TOL, max_rel, rel_l2, to_dev

pytestmark = pytest.mark.gpu

R = pytest.importorskip("recurrent_depth_moe_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    R.load_library()


def _cfg(dtype):
    return RI.RDTConfig(dim=512, n_heads=4, n_kv_heads=2, max_seq_len=64, max_loop_iters=4, n_experts=8,
                        n_shared_experts=1, n_experts_per_tok=2, expert_dim=128, lora_rank=8, dtype=dtype)


def _close(a, b, dtype):
    err = max_rel(a, b) if dtype == "fp32" else rel_l2(a, b)
    assert err <= (FP32_TOL if dtype == "fp32" else BF16_TOL), err


def _scattered(cfg, n_loops, batch, t_max, page, quantised, seed=0):
    """A paged cache whose sequences' pages lie in random order, with some pages unused."""
    per = -(-t_max // page)
    perm = torch.randperm(batch * per + 3, generator=torch.Generator().manual_seed(seed))[:batch * per]
    table = perm.to(torch.int32).reshape(batch, per).cuda()
    return R.PagedKVCache.alloc(cfg, n_loops, batch, t_max, page, quantised, n_pages=batch * per + 3, page_table=table)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("page,quantised", [(16, False), (5, False), (16, True)])
def test_block_prefill_chunk_and_decode(dtype, page, quantised):
    """Prefill, a second chunk behind it, then a decode step over pages: the rows of one longer
    prefill (which sees unquantised keys, so a quantised cache is held to e4m3's half step
    through one attention: 2^-4 of each key and value, on a sub-block whose output joins a
    residual of unit size), and the same rows whether a token comes as a decode step or as a
    chunk of one."""
    cfg = _cfg(dtype)
    W = to_dev(RI.dense_block_weights(cfg, 5))
    B, T1, T2 = 3, 21, 9
    T = T1 + T2 + 1
    x = torch.randn(B, T, cfg.dim, generator=torch.Generator().manual_seed(6)).cuda()
    blk = R.Block(cfg, W)
    full = blk.forward(x.reshape(B * T, -1).contiguous(), B, T).reshape(B, T, -1)
    cache = _scattered(cfg, 1, B, T + 4, page, quantised)
    part = lambda a, b: x[:, a:b].reshape(B * (b - a), -1).contiguous()
    one = blk.forward(part(0, T1), B, T1, 0, cache=cache).reshape(B, T1, -1)
    _close(one, full[:, :T1], dtype)                                  # its own rows as projected
    two = blk.forward(part(T1, T1 + T2), B, T2, T1, cache=cache).reshape(B, T2, -1)
    clen = torch.full((B,), T1 + T2, dtype=torch.int32, device="cuda")
    step = blk.forward(part(T1 + T2, T), B, 1, 0, cache=cache, cache_len=clen)
    if quantised:
        for got, want in ((two, full[:, T1:T1 + T2]), (step, full[:, T - 1])):
            assert rel_l2(got, want) <= 2.0 ** -4
    else:
        _close(two, full[:, T1:T1 + T2], dtype)
        _close(step, full[:, T - 1], dtype)
    chunk = blk.forward(part(T1 + T2, T), B, 1, T1 + T2, cache=cache)
    _close(chunk, step, dtype)
    assert cache.read_status() == 0


@pytest.mark.parametrize("dtype,act,T", [("fp32", 0.0, 18), ("fp32", 0.9, 18), ("bf16", 0.0, 18), ("bf16", 0.9, 24)])
def test_recurrent_block_prefill_and_decode(dtype, act, T):
    """The looped block: prefill and two decode steps over pages (one table, a page set per
    loop) against contiguous caches; ragged lengths in the decode.  (In bf16 with halting and a
    length of whole tiles, halted rows leave the queries and keep writing keys and values.)"""
    cfg = _cfg(dtype)
    W = RI.block_weights(cfg, 11, attn_std=0.08, halt_b=-1.0)
    blk = R.RecurrentBlock(cfg, to_dev(W))
    B, L, t_max = 3, 3, 32
    h0, e = RI.recurrent_inputs(cfg, B, T, 12)
    h0, e = h0.cuda(), e.cuda()
    k = torch.zeros(L, B, cfg.n_kv_heads, t_max, cfg.head_dim, dtype=blk.dtype, device="cuda")
    flat = R.KVCache(k, torch.zeros_like(k))
    paged = _scattered(cfg, L, B, t_max, 16, False, 1)
    a = blk.forward(h0, e, B, T, L, act, cache=flat)
    a = [t.clone() for t in a]
    b = blk.forward(h0, e, B, T, L, act, cache=paged)
    for i in range(2):
        assert torch.equal(a[i], b[i])                               # the same kernels on the same rows
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    for t in range(L):
        for x, y in zip(R.paged_kv_read(lens, paged, t_out=t_max, loop=t), (flat.k[t], flat.v[t])):
            assert torch.equal(x, y)
    start = torch.tensor([T, 4, T - 1], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(13)
    for i in range(2):
        hd = torch.randn(B, cfg.dim, generator=g).cuda()
        ed = torch.randn(B, cfg.dim, generator=g).to(blk.dtype).cuda()
        x = blk.decode_step(hd, ed, start + i, flat, L, act)
        x = [t.clone() for t in x]
        y = blk.decode_step(hd, ed, start + i, paged, L, act)
        assert blk.read_status() == 0
        if torch.equal(x[2], y[2]):                                  # (a near-tie may route elsewhere)
            _close(y[0], x[0], dtype)
        else:
            assert dtype == "bf16"


def test_decode_graph_over_pages():
    """DecodeGraph replays over a paged cache give the eager steps' bits."""
    cfg = _cfg("bf16")
    blk = R.RecurrentBlock(cfg, to_dev(RI.block_weights(cfg, 21, attn_std=0.08)))
    B, L = 4, 2
    g = torch.Generator().manual_seed(22)
    h = torch.randn(5, B, cfg.dim, generator=g).cuda()
    e = torch.randn(5, B, cfg.dim, generator=g).to(torch.bfloat16).cuda()
    outs = []
    for graph in (False, True):
        cache = _scattered(cfg, L, B, 48, 16, True, 2)
        clen = torch.tensor([0, 7, 15, 16], dtype=torch.int32, device="cuda")
        if graph:
            dg = R.DecodeGraph(blk, B, cache, clen, L)
            outs.append([dg.step(h[i], e[i])[0].clone() for i in range(5)])
        else:
            ws = blk.workspace(B, 1, cache.t_max, cache=cache)
            outs.append([blk.decode_step(h[i], e[i], clen + i, cache, L, workspace=ws)[0].clone() for i in range(5)])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def _generator(cfg, MW, cuda_graph=True, **kw):
    return R.Generator(cfg, MW, 2, 16, 8, 4, cuda_graph=cuda_graph, **kw)


def test_generation_over_pages_equals_contiguous():
    wl = RI.get_workload("tiny_gqa_fp32")
    MW = to_dev(RI.model_weights(wl.cfg, wl.seed))
    ids = torch.randint(0, wl.cfg.vocab_size, (2, 16), generator=torch.Generator().manual_seed(31)).int().cuda()
    runs = []
    for kw in (dict(), dict(page_size=8), dict(page_size=8, cuda_graph=False)):
        gen = _generator(wl.cfg, MW, **kw)
        gen.prefill(ids)
        logits = [gen.logits.clone()]
        for s in range(1, 8):
            gen.decode(s)
            logits.append(gen.logits.clone())
        runs.append((gen.tokens.clone(), torch.stack(logits)))
    assert torch.equal(runs[1][0], runs[2][0]) and torch.equal(runs[1][1], runs[2][1])
    for s in range(8):
        _close(runs[1][1][s], runs[0][1][s], "fp32")
        if not torch.equal(runs[1][0][s], runs[0][0][s]):            # a near-tie: the steps after it differ
            top = runs[0][1][s].topk(2, dim=-1).values
            assert ((top[:, 0] - top[:, 1]) < 1e-4).any()
            break


@pytest.mark.parametrize("quantised", [False, True])
def test_sampled_generation(quantised):
    """Each step's token is the sample of that step's logits with that step's uniform numbers,
    eagerly and replayed; temperature 0 is the greedy generation; a quantised cache changes the
    logits by its rounding alone (2^-4 of keys and values, relative L2)."""
    wl = RI.get_workload("tiny_gqa_fp32")
    cfg = wl.cfg
    MW = to_dev(RI.model_weights(cfg, wl.seed))
    ids = torch.randint(0, cfg.vocab_size, (2, 16), generator=torch.Generator().manual_seed(41)).int().cuda()
    u = torch.rand(8, 2, generator=torch.Generator().manual_seed(42)).cuda()
    samp = R.Sampling(temperature=torch.tensor([0.7, 1.3], device="cuda"), top_k=200, top_p=0.95, min_p=0.001)
    kw = dict(page_size=16, quantised=True) if quantised else {}
    tokens = []
    for graph in (False, True):
        gen = _generator(cfg, MW, graph, sampling=samp, **kw)
        gen.u.copy_(u)
        gen.prefill(ids)
        for s in range(8):
            if s:
                gen.decode(s)
            want = R.sample_tokens(gen.logits, u[s].contiguous(), samp.temperature, 200, 0.95, 0.001)
            assert torch.equal(gen.tokens[s], want), s
        tokens.append(gen.tokens.clone())
        again = gen.run(ids, u)
        assert torch.equal(again.t(), tokens[-1])
    assert torch.equal(tokens[0], tokens[1])
    greedy = R.generate(cfg, MW, ids, 8, 4, **kw)
    cold = R.generate(cfg, MW, ids, 8, 4, sampling=R.Sampling(temperature=0.0), u=u, **kw)
    assert torch.equal(greedy, cold)
    if quantised:
        first = _generator(cfg, MW, False)
        first.prefill(ids), first.decode(1)
        gq = _generator(cfg, MW, False, **kw)
        gq.prefill(ids)
        gq.tokens[0].copy_(first.tokens[0])
        gq.decode(1)
        assert rel_l2(gq.logits, first.logits) <= 2.0 ** -4


def test_model_refusals():
    cfg = _cfg("bf16")
    with pytest.raises(ValueError):
        R.Generator(cfg, {}, 1, 4, 4, 1, quantised=True)
    blk = R.RecurrentBlock(cfg, to_dev(RI.block_weights(cfg, 51)))
    cache = _scattered(cfg, 2, 2, 32, 16, False)
    h = torch.zeros(2, cfg.dim, device="cuda")
    e = torch.zeros(2, cfg.dim, dtype=torch.bfloat16, device="cuda")
    clen = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(R.RdtError):
        blk.decode_step(h, e, clen, cache, 3)                        # more loops than the cache has
    with pytest.raises(R.RdtError):
        blk.decode_step(h, e, clen, cache, 2, workspace=torch.empty(1 << 12, dtype=torch.uint8, device="cuda"))
    with pytest.raises(R.RdtError):
        blk.forward(h, e, 1, 2, 2, start_pos=31, cache=cache)        # past the table's positions
    with pytest.raises(ValueError):
        blk.forward(h, e, 1, 2, 2, cache=cache, flags=R.RDT_FLAG_TRANSFORMER_OFF)
    other = _scattered(_cfg("fp32"), 2, 2, 32, 16, False)
    with pytest.raises(R.RdtError):
        blk.decode_step(h, e, clen, other, 2)                        # another model dtype
