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
        cache.page_table[1, 0] = page1
    assert torch.isfinite(outs[0]).all()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for t in (cache.k, cache.v):
        t[:, page1].zero_()
    want = blk.forward(y, B, T, T, cache=cache, workspace=ws)
    assert torch.equal(outs[0], want)
