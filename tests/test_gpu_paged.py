"""Paged key / value cache on the GPU: writing (both storage forms), reading back and one-token
attention, against 64-bit CPU forms written from the definitions."""
import math

import pytest
import torch

from tests import _serving as S

pytestmark = pytest.mark.gpu

R = pytest.importorskip("recurrent_depth_moe_b200")
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    R.load_library()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- write ------------------------------------------------------------------------------------
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype,Hkv,hd,page,seq", [
    ("bf16", 8, 128, 16, 1), ("bf16", 2, 128, 64, 37), ("fp32", 2, 32, 16, 5), ("bf16", 1, 64, 8, 19),
    ("fp32", 4, 128, 16, 33), ("bf16", 3, 80, 5, 11), ("fp32", 1, 7, 3, 4), ("bf16", 1, 256, 1, 6), ("bf16", 2, 96, 32, 3)])
def test_write_places_and_quantises_every_row(dtype, Hkv, hd, page, seq, quant):
    """Rows land in their slots with the definition's values and exponents, other slots and
    loops keep theirs, padding rows (position -1) write nothing; the rows are slices of a wider
    projection."""
    B, t_max = 3, 2 * seq + 9
    cache = S.make_cache(R, B, Hkv, hd, t_max, page, dtype, quant, 1, n_loops=2)
    g = torch.Generator().manual_seed(2)
    W = (2 + 2 * Hkv) * hd
    qkv = torch.randn(B * seq, W, generator=g)
    qkv[:, 2 * hd:] *= torch.exp2(torch.randint(-20, 20, (B * seq, 2 * Hkv), generator=g).float()).repeat_interleave(hd, 1)
    qkv[0, 2 * hd:3 * hd] = 0.0                                      # a row of zeros
    qkv = qkv.to(DT[dtype]).cuda()
    k = qkv[:, 2 * hd:(2 + Hkv) * hd].unflatten(1, (Hkv, hd))
    v = qkv[:, (2 + Hkv) * hd:].unflatten(1, (Hkv, hd))
    start = [0, 9, t_max - seq]
    pos = torch.tensor([[s + i for i in range(seq)] for s in start])
    pos[1, 0] = -1
    want = [t.clone() for t in (cache.k, cache.v)]
    wex = [None if t is None else t.clone() for t in (cache.k_exp, cache.v_exp)]
    table = cache.page_table.cpu()
    for x, t, ex in ((k, want[0], wex[0]), (v, want[1], wex[1])):
        rows, ebytes = (S.quantise(x) if quant else (x.cpu(), None))
        for b in range(B):
            for i in range(seq):
                p = int(pos[b, i])
                if p < 0:
                    continue
                page_i, slot = int(table[b, p // page]), p % page
                dst = t.view(torch.uint8) if quant else t
                dst[1, page_i, :, slot] = (rows[b * seq + i].view(torch.uint8) if quant else rows[b * seq + i]).cuda()
                if quant:
                    ex[1, page_i, :, slot] = ebytes[b * seq + i].cuda()
    R.paged_kv_write(k, v, _i32(pos.reshape(-1).tolist()), cache, seq=seq, loop=1)
    assert cache.read_status() == 0
    for got, w in ((cache.k, want[0]), (cache.v, want[1])):
        assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))
    if quant:
        assert torch.equal(cache.k_exp, wex[0]) and torch.equal(cache.v_exp, wex[1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_quantised_edges(dtype):
    """Rows whose largest value sits at a border of the exponent rule, subnormal rows, zeros,
    infinities and NaN: the definition's bytes (an infinity and a NaN are both stored as NaN and
    leave the scale alone), and the read back value within half a step of e4m3 of the input."""
    hd = 64
    top = [448.0, 449.0 if dtype == "fp32" else 452.0, 447.0 if dtype == "fp32" else 446.0, 1.0, 0.875, 0.877, 2.0 ** -126, 2.0 ** -133, 0.0, 3.0e38, 1e-30]
    x = torch.zeros(len(top) + 3, 1, hd)
    g = torch.Generator().manual_seed(4)
    for i, t in enumerate(top):
        x[i, 0] = (torch.rand(hd, generator=g) * 2 - 1) * 0.99 * t
        x[i, 0, 5] = t
    x[-3, 0] = torch.randn(hd, generator=g)
    x[-3, 0, 7], x[-3, 0, 8] = math.inf, -math.inf
    x[-2, 0] = torch.randn(hd, generator=g)
    x[-2, 0, 0] = math.nan
    x[-1, 0] = math.nan
    x = x.to(DT[dtype])
    n = x.shape[0]
    cache = S.make_cache(R, 1, 1, hd, n, 16, dtype, True, 3, fill=False)
    R.paged_kv_write(x.cuda(), x.cuda(), _i32(list(range(n))), cache, seq=n)
    q, ex = S.quantise(x)
    table = cache.page_table.cpu()[0]
    for i in range(n):
        page, slot = int(table[i // 16]), i % 16
        got = cache.k[0, page, 0, slot].cpu().float()
        want = q[i, 0].float()
        assert int(cache.k_exp[0, page, 0, slot]) == int(ex[i, 0]), i
        assert torch.equal(torch.isnan(got), torch.isnan(want)), i
        assert torch.equal(got.nan_to_num(), want.nan_to_num()), i
    k, _ = R.paged_kv_read(_i32([n]), cache, t_out=n)
    back = k[0, 0].cpu().double()
    for i in range(len(top)):
        if top[i] == 3.0e38:
            continue                                                 # its rounding may pass the type's range
        xi = x[i, 0].double()
        step = torch.clamp(2.0 ** -4 * xi.abs(), min=2.0 ** (int(ex[i, 0]) - 127 - 10))   # normal values, and e4m3's subnormal grid of 2^-9
        assert ((back[i] - xi).abs() <= step + 2.0 ** -134).all(), i


def test_write_out_of_range_is_recorded_and_skipped():
    """A position past the table and a table entry past the pages: recorded as bounds errors,
    nothing written for them, the other rows in place."""
    from recurrent_depth_moe_b200 import _native as N
    cache = S.make_cache(R, 2, 2, 64, 32, 16, "bf16", False, 5, fill=False)
    k = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    R.paged_kv_write(k, k, _i32([32, 3]), cache)
    assert cache.read_status() == N.RDT_ERR_DEVICE_BOUNDS and cache.read_status() == 0
    assert float(cache.k.float().sum()) == 128
    cache.page_table[0, 0] = cache.n_pages
    R.paged_kv_write(k, k, _i32([0, 4]), cache)
    assert cache.read_status() == N.RDT_ERR_DEVICE_BOUNDS
    assert float(cache.k.float().sum()) == 256
    cache.page_table[0, 0] = -1
    R.paged_kv_write(k, k, _i32([0, 4]), cache)
    assert cache.read_status() == N.RDT_ERR_DEVICE_BOUNDS
    assert float(cache.k.float().sum()) == 256


# ---- read -------------------------------------------------------------------------------------
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype,Hkv,hd,page,t_max", [
    ("bf16", 8, 128, 16, 130), ("fp32", 2, 32, 16, 50), ("bf16", 1, 80, 8, 33), ("fp32", 1, 7, 3, 10),
    ("bf16", 2, 256, 1, 5), ("bf16", 2, 64, 128, 300), ("fp32", 3, 96, 64, 65)])
def test_read_back(dtype, Hkv, hd, page, t_max, quant):
    """Exact values of every cached position; rows behind a sequence's length keep what the
    output held; a length of zero, of one, of a page's end and past t_out."""
    lens = [0, 1, page, min(page + 1, t_max), t_max - 1, t_max]
    cache = S.make_cache(R, len(lens), Hkv, hd, t_max, page, dtype, quant, 6, n_loops=2)
    for t_out in (t_max, max(1, t_max - 3)):
        out = tuple(torch.full((len(lens), Hkv, t_out, hd), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
        got = R.paged_kv_read(_i32(lens), cache, loop=1, out=out)
        assert cache.read_status() == 0
        for b, n in enumerate(lens):
            n = min(n, t_out)
            for x, y in zip(got, S.cached(cache, b, n, loop=1)):
                assert torch.equal(x[b, :, :n].cpu().double(), y)
                assert (x[b, :, n:] == 7.0).all()


def test_read_without_out_and_bad_pages():
    from recurrent_depth_moe_b200 import _native as N
    cache = S.make_cache(R, 2, 1, 32, 40, 16, "fp32", True, 7)
    k, v = R.paged_kv_read(_i32([3, 40]), cache)
    assert k.shape == (2, 1, 48, 32) and float(k[0, :, 3:].abs().sum()) == 0
    cache.page_table[0, 0] = 1 << 30
    k, v = R.paged_kv_read(_i32([3, 60]), cache)                     # bad page; a length past the table
    assert cache.read_status() == N.RDT_ERR_DEVICE_BOUNDS
    assert float(k[0].abs().sum()) == 0 and torch.equal(k[1].cpu().double(), S.cached(cache, 1, 48)[0])


# ---- attention --------------------------------------------------------------------------------
CASES = [  # dtype, H, Hkv, hd, page, lens
    ("bf16", 24, 8, 128, 16, [1, 2, 15, 16, 17, 63, 64, 65, 700, 0]),
    ("bf16", 32, 8, 128, 64, [4097, 1, 333]),
    ("bf16", 8, 1, 64, 32, [129, 31, 1000]),
    ("bf16", 4, 4, 128, 16, [50, 300]),
    ("bf16", 14, 2, 128, 16, [257, 12]),
    ("bf16", 17, 1, 64, 16, [90]),
    ("bf16", 64, 2, 128, 16, [77, 260]),
    ("bf16", 6, 2, 96, 16, [45, 190]),
    ("bf16", 4, 2, 32, 16, [10, 100]),
    ("bf16", 4, 2, 192, 48, [47, 48, 49, 500]),
    ("bf16", 2, 1, 256, 16, [5, 80]),
    ("bf16", 3, 1, 80, 8, [9, 77]),
    ("bf16", 5, 1, 72, 16, [33, 77]),
    ("bf16", 2, 1, 128, 5, [6, 44]),
    ("fp32", 8, 2, 32, 16, [17, 24]),
    ("fp32", 9, 3, 128, 16, [1, 40, 513]),
    ("fp32", 2, 2, 7, 3, [5, 14]),
    ("fp32", 12, 1, 64, 128, [128, 129, 0, 1500]),
]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype,H,Hkv,hd,page,lens", CASES)
def test_attention(dtype, H, Hkv, hd, page, lens, quant):
    """Ragged batches of every head layout, width and page size; unused slots, unused pages and
    the slots behind a length hold NaN, the query is a slice of a wider row, and the output rows
    are spaced apart (what lies between them is left alone)."""
    B = len(lens)
    cache = S.make_cache(R, B, Hkv, hd, max(lens) + page + 3, page, dtype, quant, 8, n_loops=2)
    _poison(cache, lens, loop=1)
    g = torch.Generator().manual_seed(9)
    wide = torch.randn(B, (H + 2) * hd, generator=g).to(DT[dtype]).cuda()
    q = wide[:, hd:(H + 1) * hd].unflatten(1, (H, hd))
    buf = torch.full((B, (H + 1) * hd), 5.0, dtype=DT[dtype], device="cuda")
    out = buf[:, :H * hd].unflatten(1, (H, hd))
    got = R.paged_attention(q, _i32(lens), cache, loop=1, out=out)
    assert got is out and cache.read_status() == 0
    S.check_attention(cache, q, lens, out, loop=1)
    assert (buf[:, H * hd:] == 5.0).all()
    # one call after another gives the same bits
    assert torch.equal(R.paged_attention(q, _i32(lens), cache, loop=1), out)


def _poison(cache, lens, loop):
    """NaN wherever no key of a sequence lives."""
    live = torch.zeros(cache.n_pages, cache.page_size, dtype=torch.bool)
    table = cache.page_table.cpu()
    for b, n in enumerate(lens):
        for t in range(n):
            live[int(table[b, t // cache.page_size]), t % cache.page_size] = True
    dead = ~live[:, None].expand(-1, cache.n_kv_heads, -1).cuda()
    for x, ex in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
        if ex is None:
            x[loop][dead] = math.nan
        else:
            x.view(torch.uint8)[loop][dead] = 0x7f
            ex[loop][dead] = 255


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_scores_of_every_size(dtype, quant):
    """Scores that grow along the cache (every tile raises the maximum), fall along it, tie, and
    differ by hundreds; value rows whose sizes differ by 2^20."""
    H, Hkv, hd, n, B = 8, 2, 128, 700, 4
    cache = S.make_cache(R, B, Hkv, hd, n, 16, dtype, False, 10)
    g = torch.Generator().manual_seed(11)
    q = torch.randn(B, H, hd, generator=g)
    q = q / q.norm(dim=-1, keepdim=True) + 0.3
    ramp = torch.linspace(0, 8, n)
    sizes = torch.exp2(torch.randint(-10, 11, (n,), generator=g).float())
    rows_k, rows_v = torch.randn(B, n, Hkv, hd, generator=g) * 0.1, torch.randn(B, n, Hkv, hd, generator=g)
    rows_k[0] += ramp[:, None, None]
    rows_k[1] += ramp.flip(0)[:, None, None]
    rows_k[2] = 0.25
    rows_k[3] *= 40
    rows_v[3] *= sizes[:, None, None]
    if quant:
        cache = S.make_cache(R, B, Hkv, hd, n, 16, dtype, True, 10)
    pos = torch.arange(n, dtype=torch.int32).repeat(B).cuda()
    R.paged_kv_write(rows_k.reshape(-1, Hkv, hd).to(DT[dtype]).cuda(), rows_v.reshape(-1, Hkv, hd).to(DT[dtype]).cuda(),
                     pos, cache, seq=n)
    q = q.to(DT[dtype]).cuda()
    for scale in (None, 1.0, 0.01):
        out = R.paged_attention(q, _i32([n] * B), cache, scale=scale)
        S.check_attention(cache, q, [n] * B, out, scale=scale)


@pytest.mark.parametrize("dtype,quant", [("bf16", False), ("bf16", True), ("fp32", False)])
def test_attention_long_and_shared_pages(dtype, quant):
    """One long sequence split over the whole GPU, and sequences that share a prefix's pages."""
    H, Hkv, hd, n = 8, 2, 128, 20011
    cache = S.make_cache(R, 1, Hkv, hd, n, 16, dtype, quant, 12)
    q = torch.randn(1, H, hd, generator=torch.Generator().manual_seed(13)).to(DT[dtype]).cuda()
    out = R.paged_attention(q, _i32([n]), cache)
    S.check_attention(cache, q, [n], out)
    base = S.make_cache(R, 3, Hkv, hd, 200, 16, dtype, quant, 14)
    base.page_table[1:, :6] = base.page_table[0, :6]
    q = torch.randn(3, H, hd, generator=torch.Generator().manual_seed(15)).to(DT[dtype]).cuda()
    out = R.paged_attention(q, _i32([96, 200, 131]), base)
    S.check_attention(base, q, [96, 200, 131], out)


@pytest.mark.parametrize("dtype,hd,page", [("bf16", 128, 16), ("bf16", 80, 8), ("fp32", 64, 16)])
@pytest.mark.parametrize("quant", [False, True])
def test_attention_bad_pages_and_lengths(dtype, hd, page, quant):
    """A bad table entry leaves its positions out (recorded); a length past the table is cut to
    it (recorded); a negative length is an empty row."""
    from recurrent_depth_moe_b200 import _native as N
    H, Hkv = 6, 2
    cache = S.make_cache(R, 3, Hkv, hd, 20 * page, page, dtype, quant, 16)
    q = torch.randn(3, H, hd, generator=torch.Generator().manual_seed(17)).to(DT[dtype]).cuda()
    lens = [20 * page + 5, -3, 7 * page + 2]
    out = R.paged_attention(q, _i32(lens), cache)
    assert cache.read_status() == N.RDT_ERR_DEVICE_BOUNDS
    S.check_attention(cache, q, lens, out)
    good = cache.page_table.clone()
    cache.page_table[2, 1], cache.page_table[2, 6] = -5, cache.n_pages
    out = R.paged_attention(q, _i32([3, 0, 7 * page + 2]), cache)
    assert cache.read_status() == N.RDT_ERR_DEVICE_BOUNDS
    # the same positions without those pages: their entries moved out of the table row
    cache.page_table.copy_(good)
    keep = [i for i in range(20) if i not in (1, 6)]
    cache.page_table[2, :18] = good[2, keep]
    want = R.paged_attention(q, _i32([3, 0, 5 * page + 2]), cache)
    K, V = S.cached(cache, 2, 5 * page + 2)
    o, tol, vmax = S.attention(q[2].cpu(), K, V, 1 / math.sqrt(hd))
    bound = tol + S.HALF_STEP[DT[dtype]] * o.abs() * 1.01 + 2.0 ** -10 * vmax * (dtype == "bf16")
    assert ((out[2].cpu().double() - o).abs() <= bound).all() and ((want[2].cpu().double() - o).abs() <= bound).all()
    cache.page_table[2, :] = -1                                      # nothing left
    out = R.paged_attention(q, _i32([3, 0, 30]), cache)
    assert cache.read_status() == N.RDT_ERR_DEVICE_BOUNDS
    assert (out[2] == 0).all()


def test_offsets_past_32_bits():
    """Pages whose element offsets pass 2^31 and byte offsets pass 2^32: the same results as
    the same rows in a small cache."""
    Hkv, hd, page = 8, 128, 64
    n_pages = (1 << 32) // (Hkv * hd * page) + 70                    # 4 G elements
    k = torch.empty(1, n_pages, Hkv, page, hd, dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.empty_like(k)
    ke = torch.empty(1, n_pages, Hkv, page, dtype=torch.uint8, device="cuda")
    ve = torch.empty_like(ke)
    last = torch.arange(n_pages - 5, n_pages, dtype=torch.int32, device="cuda").reshape(1, 5)
    big = R.PagedKVCache(k, v, last, ke, ve, dtype="bf16")
    small = S.make_cache(R, 1, Hkv, hd, 5 * page, page, "bf16", True, 18, fill=False)
    g = torch.Generator().manual_seed(19)
    n = 5 * page - 3
    rows = torch.randn(2, n, Hkv, hd, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(1, 16, hd, generator=g).to(torch.bfloat16).cuda()
    res = []
    for c in (big, small):
        R.paged_kv_write(rows[0], rows[1], torch.arange(n, dtype=torch.int32, device="cuda"), c, seq=n)
        res.append((R.paged_attention(q, _i32([n]), c), *R.paged_kv_read(_i32([n]), c, t_out=n)))
        assert c.read_status() == 0
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_write_then_attend_as_a_decode_loop_captured_and_on_another_stream():
    """Steps of write -> attention: eagerly, replayed from a graph whose inputs are updated in
    place, and on a side stream, give the same bits; two graphs share one workspace."""
    H, Hkv, hd, B = 8, 2, 128, 5
    g = torch.Generator().manual_seed(20)
    rows = torch.randn(6, 2, B, Hkv, hd, generator=g).to(torch.bfloat16).cuda()
    qs = torch.randn(6, B, H, hd, generator=g).to(torch.bfloat16).cuda()
    start = _i32([0, 15, 16, 40, 63])

    def fresh():
        return S.make_cache(R, B, Hkv, hd, 96, 16, "bf16", True, 21)

    def steps(cache, ws):
        pos, outs = start.clone(), []
        for i in range(6):
            R.paged_kv_write(rows[i, 0], rows[i, 1], pos, cache)
            pos += 1
            outs.append(R.paged_attention(qs[i], pos, cache, workspace=ws))
        return outs

    a = fresh()
    ws = R.paged_attention_workspace(a, H)
    eager = steps(a, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c = fresh()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = steps(c, R.paged_attention_workspace(c, H))
    side.synchronize()
    b = fresh()
    k_in, v_in, q_in = rows[0, 0].clone(), rows[0, 1].clone(), qs[0].clone()
    pos, out = start.clone(), torch.empty_like(qs[0])
    graphs = []
    for _ in range(2):                                               # two graphs of the same step, one workspace
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, capture_error_mode="thread_local"):
            R.paged_kv_write(k_in, v_in, pos, b)
            pos.add_(1)
            R.paged_attention(q_in, pos, b, out=out, workspace=ws)
        graphs.append(gr)
    for i in range(6):
        k_in.copy_(rows[i, 0]), v_in.copy_(rows[i, 1]), q_in.copy_(qs[i])
        graphs[i % 2].replay()
        assert torch.equal(out, eager[i]) and torch.equal(other[i], eager[i]), i
    assert b.read_status() == 0
    S.check_attention(a, qs[5], (start + 6).tolist(), eager[5])


def test_empty_calls():
    """No rows, no sequences, nothing to read: nothing happens."""
    cache = S.make_cache(R, 2, 1, 32, 16, 16, "fp32", False, 22)
    z = torch.zeros(0, 1, 32, device="cuda")
    before = cache.k.clone()
    R.paged_kv_write(z, z, _i32([]), cache)
    assert torch.equal(cache.k, before)
    assert R.paged_attention(z, _i32([]), cache).shape == (0, 1, 32)
    k, _ = R.paged_kv_read(_i32([]), cache, t_out=4)
    assert k.shape == (0, 1, 4, 32)
    assert R.paged_kv_read(_i32([1, 1]), cache, t_out=0)[0].shape == (2, 1, 0, 32)


MORE = [  # dtype, H, Hkv, hd, page, lens: every head count of the plain kernel, its widths, groups of more than 8
    ("fp32", 4, 2, 256, 16, [70, 33]), ("fp32", 10, 2, 6, 4, [9, 40]), ("fp32", 3, 1, 128, 16, [200, 1]), ("fp32", 1, 1, 64, 64, [300]),
    ("bf16", 4, 2, 100, 16, [50, 129]), ("bf16", 9, 1, 36, 16, [64, 31]), ("bf16", 20, 2, 128, 32, [100, 65]), ("bf16", 2, 2, 16, 8, [33, 5]),
    ("bf16", 16, 2, 64, 16, [2000, 31, 32, 33]), ("bf16", 5, 1, 256, 24, [900, 4])]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype,H,Hkv,hd,page,lens", MORE)
def test_attention_other_shapes(dtype, H, Hkv, hd, page, lens, quant):
    cache = S.make_cache(R, len(lens), Hkv, hd, max(lens) + 1, page, dtype, quant, 30)
    _poison(cache, lens, loop=0)
    q = torch.randn(len(lens), H, hd, generator=torch.Generator().manual_seed(31)).to(DT[dtype]).cuda()
    S.check_attention(cache, q, lens, R.paged_attention(q, _i32(lens), cache))
    assert cache.read_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("quant", [False, True])
def test_attention_many_short_sequences(dtype, quant):
    """More sequences than lengths fit on chip, empty ones and single tokens among them."""
    B, H, Hkv, hd = 700, 6, 2, 64
    lens = [(b * 37) % 41 for b in range(B)]
    cache = S.make_cache(R, B, Hkv, hd, 48, 16, dtype, quant, 32)
    q = torch.randn(B, H, hd, generator=torch.Generator().manual_seed(33)).to(DT[dtype]).cuda()
    out = R.paged_attention(q, _i32(lens), cache)
    S.check_attention(cache, q, lens, out)
    fewer = R.paged_attention(q[:5].contiguous(), _i32(lens[:5]), cache, workspace=R.paged_attention_workspace(cache, H))
    S.check_attention(cache, q[:5], lens[:5], fewer)


@pytest.mark.parametrize("quant", [False, True])
def test_bases_off_16_bytes(quant):
    """Pools, rows and outputs whose addresses 16 does not divide take the value-wise paths."""
    Hkv, hd, page, n = 2, 64, 16, 40
    good = S.make_cache(R, 1, Hkv, hd, n, page, "bf16", quant, 34, fill=False)

    def moved(t):
        flat = torch.zeros(t.numel() + 8, dtype=torch.uint8 if quant else t.dtype, device="cuda")
        view = flat[1:1 + t.numel()]
        return (view.view(t.dtype) if quant else view).view(t.shape)
    exps = [torch.zeros_like(good.k_exp) if quant else None for _ in range(2)]
    odd = R.PagedKVCache(moved(good.k), moved(good.v), good.page_table, *exps, dtype="bf16")
    g = torch.Generator().manual_seed(35)
    rows = torch.randn(2, n, Hkv, hd, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(1, 6, hd, generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    for c in (good, odd):
        R.paged_kv_write(rows[0], rows[1], pos, c, seq=n)
    for a, b in zip(R.paged_kv_read(_i32([n]), good, t_out=n), R.paged_kv_read(_i32([n]), odd, t_out=n)):
        assert torch.equal(a, b)
    S.check_attention(good, q, [n], R.paged_attention(q, _i32([n]), good))
    S.check_attention(good, q, [n], R.paged_attention(q, _i32([n]), odd))
    buf = torch.zeros(6 * hd + 1, dtype=torch.bfloat16, device="cuda")[1:].view(1, 6, hd)
    R.paged_attention(q, _i32([n]), good, out=buf)
    S.check_attention(good, q, [n], buf)


def test_two_workspaces_on_two_streams():
    """Two calls in flight together, each with its own workspace, give what each gives alone."""
    cache = S.make_cache(R, 6, 2, 128, 700, 16, "bf16", False, 36)
    g = torch.Generator().manual_seed(37)
    qs = [torch.randn(6, 8, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    lens = [_i32([700, 3, 0, 333, 64, 512]), _i32([1, 699, 200, 17, 0, 90])]
    alone = [R.paged_attention(q, n, cache) for q, n in zip(qs, lens)]
    ws = [R.paged_attention_workspace(cache, 8) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        outs = []
        for q, n, w, s in zip(qs, lens, ws, streams):
            with torch.cuda.stream(s):
                outs.append(R.paged_attention(q, n, cache, workspace=w))
        torch.cuda.synchronize()
        for a, b in zip(outs, alone):
            assert torch.equal(a, b)
