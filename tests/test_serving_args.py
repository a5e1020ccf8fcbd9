"""What the serving entry points refuse, and their host logic (CPU: nothing is launched).  The C
calls get stand-in addresses, which the host never reads."""
import ctypes

import pytest
import torch

import rdt_inputs as RI

P = 0x1000   # a non-null stand-in for a device pointer (256-byte aligned)


@pytest.fixture(scope="module")
def nat():
    from recurrent_depth_moe_b200 import build as B
    B.build()
    from recurrent_depth_moe_b200 import _native as N
    N.load()
    return N


def _cache(N, **kw):
    a = dict(k=P, v=P, k_exp=None, v_exp=None, page_table=P, dtype=1, kv_type=0, n_loops=2, n_pages=8, page_size=16,
             n_kv_heads=2, head_dim=128, batch=4, max_pages=2)
    a.update(kw)
    c = N.rdt_paged_cache()
    for n, v in a.items():
        setattr(c, n, v)
    return c


BAD_CACHES = [dict(k=None), dict(v=None), dict(page_table=None), dict(dtype=2), dict(kv_type=2), dict(kv_type=1),
              dict(kv_type=1, k_exp=P), dict(n_loops=0), dict(n_pages=0), dict(page_size=0), dict(n_kv_heads=0),
              dict(head_dim=0), dict(batch=0), dict(max_pages=0)]
UNSUPPORTED = [dict(head_dim=257), dict(batch=65536), dict(max_pages=1 << 28), dict(n_kv_heads=5000)]


@pytest.mark.parametrize("kw,code", [(k, 1) for k in BAD_CACHES] + [(k, 2) for k in UNSUPPORTED])
def test_bad_caches_are_refused_by_every_call(nat, kw, code):
    lib, c = nat.load(), _cache(nat, **kw)
    r = ctypes.byref(c)
    assert lib.rdt_paged_kv_write(r, 0, P, P, 256, P, 4, 1, None, None) == code
    assert lib.rdt_paged_kv_read(r, 0, P, 2, 16, P, P, None, None) == code
    assert lib.rdt_paged_attention(r, 0, P, 1024, P, 2, 8, 1.0, P + 256, 1024, P, 1 << 30, None, None) == code
    assert lib.rdt_paged_attention_workspace_size(r, 2, 8) == 0


def test_bad_arguments_are_refused(nat):
    lib, c = nat.load(), _cache(nat)
    r = ctypes.byref(c)
    write = lambda loop=0, k=P, v=P, ld=256, pos=P, n=4, seq=1: lib.rdt_paged_kv_write(r, loop, k, v, ld, pos, n, seq, None, None)
    for kw in (dict(loop=-1), dict(loop=2), dict(k=None), dict(v=None), dict(ld=255), dict(pos=None), dict(n=-1),
               dict(seq=0), dict(n=5, seq=2), dict(n=5), dict(n=10, seq=2)):
        assert write(**kw) == 1, kw
    assert write(n=0, k=None) == 0
    read = lambda loop=0, lens=P, b=4, t=16, k=P, v=P: lib.rdt_paged_kv_read(r, loop, lens, b, t, k, v, None, None)
    for kw in (dict(loop=2), dict(lens=None), dict(b=-1), dict(b=5), dict(t=-1), dict(k=None), dict(v=None)):
        assert read(**kw) == 1, kw
    assert read(b=0) == 0 and read(t=0) == 0
    nan, inf = float("nan"), float("inf")

    def attn(loop=0, q=P, qld=1024, lens=P, b=4, H=8, scale=1.0, o=P + 256, old=1024, ws=P, n=1 << 30):
        return lib.rdt_paged_attention(r, loop, q, qld, lens, b, H, scale, o, old, ws, n, None, None)
    for kw in (dict(loop=-1), dict(loop=2), dict(q=None), dict(qld=1023), dict(lens=None), dict(b=-1), dict(b=5),
               dict(H=0), dict(H=7), dict(scale=nan), dict(scale=inf), dict(o=None), dict(o=P), dict(old=1023)):
        assert attn(**kw) == 1, kw
    need = lib.rdt_paged_attention_workspace_size(r, 4, 8)
    assert need > 0 and need % 256 == 0
    assert attn(ws=None) == 3 and attn(ws=P + 16) == 3 and attn(n=need - 1) == 3 and attn(b=0, ws=None) == 0


def test_bad_sampling_arguments_are_refused(nat):
    lib = nat.load()
    nan, inf = float("nan"), float("inf")

    def call(t=1.0, k=0, p=1.0, m=0.0, logits=P, ld=100, n=2, V=100, u=P, tok=P, out_ld=1, null=False, **rows):
        a = nat.rdt_sampling(t, k, p, m)
        for name, v in rows.items():
            setattr(a, name, v)
        return lib.rdt_sample_tokens(logits, ld, n, V, u, None if null else ctypes.byref(a), tok, out_ld, None, None)
    for kw in (dict(t=-0.1), dict(t=nan), dict(t=inf), dict(k=-1), dict(p=0.0), dict(p=1.01), dict(p=nan), dict(m=-0.1),
               dict(m=1.1), dict(m=nan), dict(logits=None), dict(ld=99), dict(n=-1), dict(V=0), dict(u=None),
               dict(tok=None), dict(out_ld=0), dict(null=True)):
        assert call(**kw) == 1, kw
    assert call(V=1 << 20, ld=1 << 20) == 2
    assert call(n=0, logits=None, u=None, tok=None) == 0
    assert call(n=0, t=nan, temperature_rows=P) == 0                 # a row array takes the scalar's place


def test_python_checks():
    """The binding's own refusals (CPU tensors never reach the library)."""
    import recurrent_depth_moe_b200 as R
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    with pytest.raises(ValueError):
        R.PagedKVCache(z(1, 4, 2, 16, 64), z(1, 4, 2, 16, 64), z(2, 2, dt=torch.int32))           # not on a GPU
    with pytest.raises(ValueError):
        R.PagedKVCache(z(4, 2, 16, 64), z(4, 2, 16, 64), z(2, 2, dt=torch.int32))                 # four axes
    with pytest.raises(ValueError):
        R.PagedKVCache(z(1, 4, 2, 16, 64, dt=torch.float8_e4m3fn), z(1, 4, 2, 16, 64, dt=torch.float8_e4m3fn),
                       z(2, 2, dt=torch.int32))                                                    # no model dtype
    with pytest.raises(ValueError):
        R.PagedKVCache(z(1, 4, 2, 16, 64, dt=torch.float16), z(1, 4, 2, 16, 64, dt=torch.float16), z(2, 2, dt=torch.int32))
    with pytest.raises(ValueError):
        R.sample_tokens(z(2, 5, dt=torch.float32), z(2, dt=torch.float32))
    with pytest.raises(ValueError):
        R.PagedKVCache.alloc(RI.get_workload("tiny_mla_fp32").cfg, 1, 2, 32)


def test_paged_model_calls_refuse(nat):
    """The model's paged entry points: host checks (no launch is reached)."""
    from recurrent_depth_moe_b200 import api
    lib = nat.load()
    gqa = api.config_struct(RI.get_workload("tiny_gqa_fp32").cfg)
    mla = api.config_struct(RI.get_workload("tiny_mla_fp32").cfg)
    fits = dict(dtype=0, n_kv_heads=2, head_dim=32)
    size = lambda cs, b=2, s=1, start=0, **kw: lib.rdt_paged_workspace_size(ctypes.byref(cs), b, s, start,
                                                                            ctypes.byref(_cache(nat, **{**fits, **kw})))
    assert size(gqa) > 0 and size(gqa) % 256 == 0
    assert size(gqa, s=16, start=16) > size(gqa, s=16)               # the positions read back
    for kw in (dict(dtype=1), dict(n_kv_heads=4), dict(head_dim=64), dict(batch=1), dict(kv_type=1), dict(max_pages=0)):
        assert size(gqa, **kw) == 0, kw
    assert size(mla) == 0 and size(gqa, b=0) == 0 and size(gqa, s=0) == 0 and size(gqa, start=-1) == 0
    assert size(gqa, s=16, start=17) == 0                            # past the table
    w = nat.rdt_weights()
    r, wr = ctypes.byref(gqa), ctypes.byref(w)
    none = [None, None, P, 1 << 30, None]
    assert lib.rdt_recurrent_decode_step_paged(r, wr, P, P, 2, P, 1, 0.0, None, P, P, P, None, None, P, 1 << 30, None) == 1
    assert lib.rdt_recurrent_forward_paged(r, wr, P, P, 2, 4, 0, 1, 0.0, None, P, P, P, *none) == 1
    assert lib.rdt_block_forward_paged(r, wr, P, P + 256, 2, 4, 0, None, None, P, 1 << 30, None) == 1
