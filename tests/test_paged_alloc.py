"""What PagedKVCache.alloc refuses before it allocates (CPU)."""
import pytest

import rdt_inputs as RI

R = pytest.importorskip("recurrent_depth_moe_b200")


def test_fewer_pages_than_the_table_names_are_refused():
    cfg = RI.RDTConfig(dim=512, n_heads=4, n_kv_heads=2, max_seq_len=64, max_loop_iters=4, n_experts=8,
                       n_shared_experts=1, n_experts_per_tok=2, expert_dim=128, lora_rank=8, dtype="bf16")
    for n_pages in (0, 1, 11):                                        # 3 sequences of 4 pages of 16
        with pytest.raises(ValueError, match="n_pages"):
            R.PagedKVCache.alloc(cfg, 1, 3, 64, 16, n_pages=n_pages, device="cpu")
