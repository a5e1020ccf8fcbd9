"""The model's calls over pages: what they record of bad pages and positions and where, what a
prefill makes of positions that it cannot read, and comparisons with contiguous caches that no
routing or near-tie skips."""
import pytest
import torch

import rdt_inputs as RI
from tests._helpers import BF16_TOL, FP32_TOL, max_rel, rel_l2, to_dev

pytestmark = pytest.mark.gpu

R = pytest.importorskip("recurrent_depth_moe_b200")
BOUNDS = 6                                # RDT_ERR_DEVICE_BOUNDS


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    R.load_library()


def _cfg(dtype, **kw):
    return RI.RDTConfig(**dict(dict(dim=512, n_heads=4, n_kv_heads=2, max_seq_len=64, max_loop_iters=4, n_experts=8,
                                    n_shared_experts=1, n_experts_per_tok=2, expert_dim=128, lora_rank=8, dtype=dtype), **kw))


def _close(a, b, dtype):
    err = max_rel(a, b) if dtype == "fp32" else rel_l2(a, b)
    assert err <= (FP32_TOL if dtype == "fp32" else BF16_TOL), err


def _table(batch, per, seed=0):
    return torch.randperm(batch * per + 3, generator=torch.Generator().manual_seed(seed))[:batch * per].to(
        torch.int32).reshape(batch, per).cuda()


def _paged(cfg, loops, B, t_max, page, quantised=False, seed=0):
    per = -(-t_max // page)
    return R.PagedKVCache.alloc(cfg, loops, B, t_max, page, quantised, n_pages=B * per + 3, page_table=_table(B, per, seed))


@pytest.mark.parametrize("quantised", [False, True])
def test_bad_pages_and_positions_reach_the_caches_status(quantised):
    """Prefill, chunk, decode step, replayed decode step and looped block: a bad table entry, and a
    length out of range, are in the cache's status word (and, as ever, in the call's workspace),
    until it is read."""
    cfg = _cfg("bf16")
    B, T = 2, 20
    blk = R.Block(cfg, to_dev(RI.dense_block_weights(cfg, 5)))
    cache = _paged(cfg, 1, B, 48, 16, quantised)
    x = torch.randn(B * T, cfg.dim, generator=torch.Generator().manual_seed(6)).cuda()
    row = x[:B].contiguous()
    clen = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    ws = blk.workspace(B, T, 48, T, cache)
    good = cache.page_table.clone()
    calls = dict(prefill=lambda: blk.forward(x, B, T, 0, cache=cache, workspace=ws),
                 chunk=lambda: blk.forward(x, B, T, T, cache=cache, workspace=ws),
                 decode=lambda: blk.forward(row, B, 1, 0, cache=cache, cache_len=clen(30, 17)))
    for name, call in calls.items():
        call()
        assert cache.read_status() == 0, name
        for bad in (-1, cache.n_pages, 1 << 30):
            cache.page_table[1, 1] = bad
            call()
            cache.page_table.copy_(good)
            call()                                                    # a good call does not clear the record
            assert cache.read_status() == BOUNDS, (name, bad)
            assert cache.read_status() == 0, (name, bad)
    for bad in (-1, 48, 1 << 30):
        blk.forward(row, B, 1, 0, cache=cache, cache_len=clen(3, bad))
        assert cache.read_status() == BOUNDS, bad
    rec = R.RecurrentBlock(cfg, to_dev(RI.block_weights(cfg, 21, attn_std=0.08)))
    loops = _paged(cfg, 2, B, 48, 16, quantised)
    h, e = row, row.to(torch.bfloat16)
    good = loops.page_table.clone()
    dg = R.DecodeGraph(rec, B, loops, clen(20, 20), 2)
    for i in range(4):                                                # eager, captured, replayed
        dg.step(h, e)
        assert loops.read_status() == 0, i
    loops.page_table[0, 1] = -5
    dg.step(h, e)
    assert rec.read_status() == BOUNDS and loops.read_status() == BOUNDS
    loops.page_table.copy_(good)
    dg.step(h, e)
    assert rec.read_status() == 0 and loops.read_status() == 0


def test_the_generators_status():
    wl = RI.get_workload("tiny_gqa_fp32")
    MW = to_dev(RI.model_weights(wl.cfg, wl.seed))
    ids = torch.randint(0, wl.cfg.vocab_size, (2, 16), generator=torch.Generator().manual_seed(31)).int().cuda()
    for kw in (dict(), dict(page_size=8)):
        gen = R.Generator(wl.cfg, MW, 2, 16, 4, 4, **kw)
        gen.run(ids)
        assert gen.read_status() == 0
    for cache in (gen.pre_cache[0], gen.rec_cache, gen.coda_cache[0]):
        good = cache.page_table.clone()
        cache.page_table[1, 0] = 99
        gen.run(ids)
        cache.page_table.copy_(good)
        assert gen.read_status() == BOUNDS and gen.read_status() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("page", [16, 5])
def test_prefill_behind_unreadable_pages_is_of_this_call_alone(dtype, quantised, page):
    """A chunk behind cached positions whose page is bad: rows of zeros in their place (what the
    same chunk gives over zeroed pages), whatever the workspace held."""
    cfg = _cfg(dtype)
    B, T = 2, 20
    blk = R.Block(cfg, to_dev(RI.dense_block_weights(cfg, 5)))
    x = torch.randn(B * T, cfg.dim, generator=torch.Generator().manual_seed(6)).cuda()
    y = torch.randn(B * T, cfg.dim, generator=torch.Generator().manual_seed(7)).cuda()
    cache = _paged(cfg, 1, B, 45, page, quantised)
    blk.forward(x, B, T, 0, cache=cache)
    ws = blk.workspace(B, T, 45, T, cache)
    page1 = int(cache.page_table[1, 0])
    outs = []
    for fill in (0, 255, 0x42):                                       # 255: NaN in both types
        cache.page_table[1, 0] = -1
        ws.fill_(fill)
        ws[:16] = 0
        outs.append(blk.forward(y, B, T, T, cache=cache, workspace=ws).clone())
        assert cache.read_status() == BOUNDS
        cache.page_table[1, 0] = page1
    assert torch.isfinite(outs[0]).all()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for t in (cache.k, cache.v):
        t[:, page1].zero_()
    want = blk.forward(y, B, T, T, cache=cache, workspace=ws)
    assert cache.read_status() == 0
    assert torch.equal(outs[0], want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("act", [0.0, 0.9])
def test_decode_steps_with_every_expert_in_use(dtype, act):
    """Decode steps over pages against contiguous caches with as many experts per token as there
    are, so that no near-tie of the router can send a token elsewhere: always compared."""
    cfg = _cfg(dtype, n_experts=2)
    W = RI.block_weights(cfg, 11, attn_std=0.08, halt_b=-1.0)
    blk = R.RecurrentBlock(cfg, to_dev(W))
    B, T, L, t_max = 3, 24, 3, 32
    h0, e = (t.cuda() for t in RI.recurrent_inputs(cfg, B, T, 12))
    k = torch.zeros(L, B, cfg.n_kv_heads, t_max, cfg.head_dim, dtype=blk.dtype, device="cuda")
    flat = R.KVCache(k, torch.zeros_like(k))
    paged = _paged(cfg, L, B, t_max, 16, False, 1)
    for cache in (flat, paged):
        blk.forward(h0, e, B, T, L, act, cache=cache)
    start = torch.tensor([T, 4, T - 1], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(13)
    for i in range(3):
        hd = torch.randn(B, cfg.dim, generator=g).cuda()
        ed = torch.randn(B, cfg.dim, generator=g).to(blk.dtype).cuda()
        x = [t.clone() for t in blk.decode_step(hd, ed, start + i, flat, L, act)]
        y = blk.decode_step(hd, ed, start + i, paged, L, act)
        assert torch.equal(x[2].sort(-1).values, y[2].sort(-1).values)
        _close(y[0], x[0], dtype)
        _close(y[1], x[1], dtype)


def test_generation_steps_fed_the_same_tokens():
    """Each step of generation over pages, given the contiguous run's token, has its logits."""
    wl = RI.get_workload("tiny_gqa_fp32")
    MW = to_dev(RI.model_weights(wl.cfg, wl.seed))
    ids = torch.randint(0, wl.cfg.vocab_size, (2, 16), generator=torch.Generator().manual_seed(31)).int().cuda()
    flat = R.Generator(wl.cfg, MW, 2, 16, 8, 4)
    gens = [R.Generator(wl.cfg, MW, 2, 16, 8, 4, page_size=8, cuda_graph=g) for g in (True, False)]
    for s in range(8):
        for gen in [flat] + gens:
            gen.decode(s) if s else gen.prefill(ids)
        for gen in gens:
            _close(gen.logits, flat.logits, "fp32")
            gen.tokens[s].copy_(flat.tokens[s])


def test_sampling_changed_between_generations():
    """A generator whose parameters are changed draws with the new ones, replayed or not; values
    changed inside a parameter's tensor count at once."""
    wl = RI.get_workload("tiny_gqa_fp32")
    MW = to_dev(RI.model_weights(wl.cfg, wl.seed))
    ids = torch.randint(0, wl.cfg.vocab_size, (2, 16), generator=torch.Generator().manual_seed(41)).int().cuda()
    u = torch.rand(8, 2, generator=torch.Generator().manual_seed(42)).cuda()
    rows = torch.tensor([0.5, 2.0], device="cuda")
    plans = [R.Sampling(temperature=1.5), R.Sampling(temperature=1.5, top_k=3), R.Sampling(temperature=rows),
             R.Sampling(temperature=rows.clone() * 3, top_p=0.9), R.Sampling(temperature=0.0)]
    gen = R.Generator(wl.cfg, MW, 2, 16, 8, 4, sampling=plans[0])
    seen = []
    for plan in plans + plans[:1]:
        want = R.generate(wl.cfg, MW, ids, 8, 4, sampling=plan, u=u)[:, 16:]
        gen.sampling = plan
        assert torch.equal(gen.run(ids, u), want)
        assert torch.equal(gen.run(ids, u), want)
        seen.append(want.clone())
    assert any(not torch.equal(a, seen[0]) for a in seen[1:])
    gen.sampling.temperature = 0.7                                    # in place
    assert torch.equal(gen.run(ids, u), R.generate(wl.cfg, MW, ids, 8, 4, sampling=R.Sampling(temperature=0.7), u=u)[:, 16:])
    gen.sampling = plans[2]
    gen.run(ids, u)
    rows.fill_(1.1)
    assert torch.equal(gen.run(ids, u), R.generate(wl.cfg, MW, ids, 8, 4, sampling=R.Sampling(temperature=1.1), u=u)[:, 16:])
    gen.sampling = None
    assert torch.equal(gen.run(ids), R.generate(wl.cfg, MW, ids, 8, 4)[:, 16:])


def test_depth_batch_refuses_pages():
    cfg = _cfg("bf16")
    blk = R.RecurrentBlock(cfg, to_dev(RI.block_weights(cfg, 51)))
    h0 = torch.zeros(2, 3, cfg.dim, device="cuda")
    with pytest.raises(ValueError, match="paged"):
        R.DepthBatch(blk, h0, h0.to(torch.bfloat16), torch.zeros(2, dtype=torch.int32, device="cuda"),
                     _paged(cfg, 2, 2, 32, 16), 2)


def test_greedy_generation_reads_no_uniform_numbers():
    wl = RI.get_workload("tiny_gqa_fp32")
    MW = to_dev(RI.model_weights(wl.cfg, wl.seed))
    ids = torch.randint(0, wl.cfg.vocab_size, (2, 16), generator=torch.Generator().manual_seed(31)).int().cuda()
    want = R.Generator(wl.cfg, MW, 2, 16, 4, 4).run(ids)
    gen = R.Generator(wl.cfg, MW, 2, 16, 4, 4)
    gen.u = gen.u_in = None
    assert torch.equal(gen.run(ids), want)


@pytest.mark.parametrize("quantised", [False, True])
def test_a_length_out_of_range_writes_nothing(quantised):
    """A decode step whose sequence has no valid position, over pages that others read (a common
    prefix): recorded, and the pages hold what they held but for the other sequence's new row,
    whose output is what it is alone."""
    cfg = _cfg("bf16")
    B, cap = 2, 48
    blk = R.Block(cfg, to_dev(RI.dense_block_weights(cfg, 5)))
    rec = R.RecurrentBlock(cfg, to_dev(RI.block_weights(cfg, 21, attn_std=0.08)))
    x = torch.randn(B * 20, cfg.dim, generator=torch.Generator().manual_seed(6)).cuda()
    row = x[:B].contiguous()
    clen = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for loops, prefill, step in (
            (1, lambda c: blk.forward(x, B, 20, 0, cache=c), lambda c, n: blk.forward(row, B, 1, 0, cache=c, cache_len=n)),
            (2, lambda c: rec.forward(x, x.to(torch.bfloat16), B, 20, 2, cache=c),
             lambda c, n: rec.decode_step(row, row.to(torch.bfloat16), n, c, 2)[0].clone())):
        cache = _paged(cfg, loops, B, cap, 16, quantised)
        prefill(cache)
        cache.page_table[1] = cache.page_table[0]
        bits = [t.view(torch.uint8) for t in (cache.k, cache.v)] + ([cache.k_exp, cache.v_exp] if quantised else [])
        held = [t.clone() for t in bits]
        want = step(cache, clen(20, 21))[0].clone()                   # (position 21 is past what sequence 0 sees)
        after = [t.clone() for t in bits]
        page, slot = int(cache.page_table[0, 1]), 4
        assert cache.read_status() == 0
        for bad in (-1, cap, cap + 16, 1 << 30, 2 ** 31 - 1, -2 ** 31):
            for t, h in zip(bits, held):
                t.copy_(h)
            got = step(cache, clen(20, bad))
            assert cache.read_status() == BOUNDS, bad
            assert torch.equal(got[0], want), bad
            for t, h, a in zip(bits, held, after):
                h = h.clone()
                h[:, page, :, slot] = a[:, page, :, slot]
                assert torch.equal(t, h), bad
