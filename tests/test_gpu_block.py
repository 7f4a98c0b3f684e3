"""RMS norm, the paged KV cache and attention over it against plain 64-bit
references, at the sizes and masks where they can go wrong."""
import math

import pytest

torch = pytest.importorskip("torch")

from mixture_experts_layer_19_amd import binding as B
from mixture_experts_layer_19_amd import block

import _block as R

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ----------------------------------------------------------------------------- norm


def check_norm(x, residual, weight, res, eps, quant, fp8_scale=None):
    s, y = R.norm_ref(x.cpu(), None if residual is None else residual.cpu(), weight.cpu(), eps)
    half, n = R.half_step(x.dtype), x.shape[1]
    # fp32: one rounding of the sum, n of the mean of squares (half of which
    # reach the root), a few of the root, the quotient and the products
    rel = (n / 2 + 8) * R.F32_HALF
    if residual is not None:
        assert ((res.residual.cpu().double() - s).abs() <= (half + R.F32_HALF) * s.abs()).all()
    # the sum's rounding is relative to the operands' sum, which the sum itself bounds
    if res.y is not None:
        assert ((res.y.cpu().double() - y).abs() <= (half + rel) * y.abs() + 1e-38).all()
    if quant == "mxfp8":
        q, sb = res.q.cpu(), res.scale.cpu()
        top = y.unflatten(-1, (-1, 32)).abs().amax(-1)
        exp = (torch.frexp(top)[1] - 9).clamp(min=-127)
        exp[top == 0] = -127
        # the exponent may differ only where the maximum is within rel of a power of two
        near = (torch.frexp(top * (1 + rel))[1] != torch.frexp(top * (1 - rel))[1])
        assert ((sb.int() - 127 == exp) | near).all()
        unit = R.e8m0(sb).repeat_interleave(32, -1)
        want = (y / unit).clamp(-448, 448)
        got = q.view(torch.float8_e4m3fn).double()
        assert ((got - want).abs() <= R.MX_HALF * want.abs() + 2.0 ** -10 + 2 * rel * want.abs()).all()
    elif quant == "fp8":
        want = (y / fp8_scale).clamp(-448, 448)
        got = res.q.cpu().view(torch.float8_e4m3fn).double()
        assert ((got - want).abs() <= R.MX_HALF * want.abs() + 2.0 ** -10 + 2 * rel * want.abs()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,hidden", [(1, 32), (5, 96), (7, 512), (3, 544), (66, 1024), (2, 2048), (9, 4096),
                                         (4, 5152), (3, 8192), (2, 8224), (1, 20000)])
@pytest.mark.parametrize("quant", ["none", "mxfp8", "fp8"])
def test_norm(dtype, rows, hidden, quant):
    g = gen(rows * 7 + hidden)
    x = torch.randn(rows, hidden, generator=g).to(dtype).cuda()
    r = (4 * torch.randn(rows, hidden, generator=g)).to(dtype).cuda()
    w = (1 + 0.1 * torch.randn(hidden, generator=g)).to(dtype).cuda()
    norm = block.RMSNorm(w, eps=1e-5, quant=quant, fp8_scale=2.0 ** -5)
    check_norm(x, r, w, norm(x, r), 1e-5, quant, 2.0 ** -5)
    res = norm(x)
    assert res.residual is None
    check_norm(x, None, w, res, 1e-5, quant, 2.0 ** -5)
    if quant != "none":
        lean = norm(x, r, want_y=False)
        assert lean.y is None and torch.equal(lean.q, norm(x, r).q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,hidden", [(1, 1), (3, 7), (5, 100), (4, 1023), (2, 4097)])
@pytest.mark.parametrize("quant", ["none", "fp8"])
def test_norm_odd_lengths(dtype, rows, hidden, quant):
    g = gen(hidden)
    x = torch.randn(rows, hidden, generator=g).to(dtype).cuda()
    r = torch.randn(rows, hidden, generator=g).to(dtype).cuda()
    w = torch.randn(hidden, generator=g).to(dtype).cuda()
    norm = block.RMSNorm(w, eps=1e-6, quant=quant, fp8_scale=0.01)
    check_norm(x, r, w, norm(x, r), 1e-6, quant, 0.01)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_strided_and_unaligned_rows(dtype):
    g = gen(3)
    wide = torch.randn(9, 3 * 512 + 5, generator=g).to(dtype).cuda()
    w = torch.randn(512, generator=g).to(dtype).cuda()
    for start in (0, 1, 8, 512):
        x = wide[:, start:start + 512]
        norm = block.RMSNorm(w, quant="mxfp8")
        check_norm(x, x, w, norm(x, x), 1e-5, "mxfp8")


def test_norm_zero_rows_and_special_values():
    w = torch.ones(64, device="cuda")
    norm = block.RMSNorm(w, eps=1e-5, quant="mxfp8")
    res = norm(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, device="cuda"))
    assert res.y.shape == (0, 64) and res.scale.shape == (0, 2)
    x = torch.zeros(4, 64, device="cuda")
    x[1, 3] = math.nan
    x[2, 40] = math.inf
    x[3] = 1e-30
    res = norm(x)
    y, q, sb = res.y.cpu(), res.q.cpu(), res.scale.cpu()
    assert (y[0] == 0).all() and (q[0] == 0).all() and (sb[0] == 0).all()
    assert y[1].isnan().all() and ((q[1] & 0x7F) == 0x7F).all()
    assert y[2].isnan().sum() == 1 and (y[2][:40] == 0).all()       # inf / inf, and zeros over inf
    assert torch.isfinite(y[3]).all()


# ----------------------------------------------------------------------------- cache


CACHES = ["bf16", "mxfp8", "f32"]
BATCHES = [
    # new, past, page, kv_heads, head_dim
    ([1], [0], 8, 1, 64),
    ([1, 1, 1], [0, 7, 8], 8, 2, 128),
    ([0, 5, 1, 0, 17], [3, 12, 0, 0, 31], 16, 4, 64),
    ([33, 1, 70], [0, 63, 1], 64, 8, 128),
    ([9], [250], 1, 1, 256),
    ([130, 2], [5, 300], 256, 2, 256),
]


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("new,past,page,kvh,hd", BATCHES)
def test_write_then_read(orc, dtype, new, past, page, kvh, hd):
    g = gen(11 * page + hd)
    p = R.Paged(g, new, past, page, kvh, hd, dtype, lead_rows=2, pad_rows=3)
    cache, batch = p.device()
    fused = torch.randn(p.rows, 2 * kvh + 1, hd, generator=g)
    fused *= torch.exp(6 * torch.rand(p.rows, 1, 1, generator=g) - 3)
    fused = fused.to(p.act)
    k, v = fused.cuda()[:, :kvh], fused.cuda()[:, kvh + 1:]
    before = [t.clone() for t in (cache.k, cache.v)]
    cache.write(batch, k, v)
    rk, rv = cache.read(batch)
    first = int(p.offsets[0])
    for which, (src, got, pool, scale) in enumerate(((fused[:, :kvh], rk, cache.k, cache.k_scale),
                                                     (fused[:, kvh + 1:], rv, cache.v, cache.v_scale))):
        want_pool = before[which].cpu()
        if dtype == "mxfp8":
            codes, sb = orc.mxq(src.float().numpy().reshape(-1, hd))
            codes = torch.from_numpy(codes).view(p.rows, kvh, hd)
            sb = torch.from_numpy(sb).view(p.rows, kvh, hd // 32)
            want_rows = R.mx_values(codes, sb)
            want_scale = p.pools[which][1].clone()
        else:
            codes, want_rows = src, src.double()
        r = first
        for s, n in enumerate(new):
            for i in range(n):
                pos = p.total[s] - n + i
                page_id = p.table[s, pos // page]
                want_pool[page_id, :, pos % page] = codes[r]
                if dtype == "mxfp8":
                    want_scale[page_id, :, pos % page] = sb[r]
                r += 1
        view = torch.uint8 if dtype == "mxfp8" else torch.int32 if dtype == "f32" else torch.int16
        assert torch.equal(pool.cpu().view(view), want_pool.view(view))
        if dtype == "mxfp8":
            assert torch.equal(scale.cpu(), want_scale)
        inside = torch.zeros(p.rows, dtype=torch.bool)
        inside[first:r] = True
        got = got.cpu().double()
        # an E4M3 value times a power of two is exact in bf16
        assert torch.equal(got[inside], want_rows[inside])
        assert (got[~inside] == 0).all()


def test_quantised_write_of_extremes(orc):
    p = R.Paged(gen(1), [6], [0], 8, 1, 64, "mxfp8")
    cache, batch = p.device()
    k = torch.zeros(6, 1, 64, dtype=torch.bfloat16)
    k[1, 0, :32] = 2.0 ** -126
    k[1, 0, 3] = 3.0 * 2.0 ** -128            # below the smallest normal of fp32
    k[2, 0, 5], k[2, 0, 6] = 3.38e38, -3.38e38
    k[3, 0, 0], k[3, 0, 1] = -0.0, 448.0
    k[4] = torch.arange(64).view(1, 64) / 7.0
    k[5, 0, 0], k[5, 0, 1], k[5, 0, 2] = math.nan, 1.0, -2.0
    cache.write(batch, k.cuda(), k.cuda())
    kk, vv = cache.read(batch)
    assert torch.equal(kk.view(torch.int16), vv.view(torch.int16))
    codes, sb = orc.mxq(k[:5].float().numpy().reshape(-1, 64))
    got = torch.stack([cache.k.cpu()[p.table[0, 0], :, i] for i in range(6)])
    scales = torch.stack([cache.k_scale.cpu()[p.table[0, 0], :, i] for i in range(6)])
    assert torch.equal(got[:5].reshape(-1, 64), torch.from_numpy(codes))
    assert torch.equal(scales[:5].reshape(-1, 2), torch.from_numpy(sb))
    assert torch.equal(kk[:5].cpu().double().view(-1, 64), R.mx_values(torch.from_numpy(codes), torch.from_numpy(sb)))
    row = kk[5].cpu().double()[0]
    assert row[0].isnan() and row[1] == 1.0 and row[2] == -2.0 and (row[3:] == 0).all()


def test_read_covers_every_code():
    """Every E4M3 code under the scales 2^-127 .. 2^119 (finite products)."""
    for byte in (0, 1, 60, 127, 200, 246):
        p = R.Paged(gen(2), [4], [0], 4, 1, 64, "mxfp8")
        cache, batch = p.device()
        codes = torch.arange(256, dtype=torch.uint8).view(4, 1, 64)
        for i in range(4):
            cache.k[p.table[0, 0], :, i] = codes[i].cuda()
        cache.k_scale.fill_(byte)
        got = cache.read(batch)[0].cpu().double()
        want = R.mx_values(codes, torch.full((4, 1, 2), byte, dtype=torch.uint8))
        want = want.to(torch.bfloat16).double()       # one rounding: subnormals of bf16 under 2^-127
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


def test_pages_that_do_not_exist():
    p = R.Paged(gen(5), [20], [0], 8, 2, 64, "bf16")
    p.table[0, 1] = -1
    p.table[0, 2] = p.num_pages
    cache, batch = p.device()
    before = cache.k.clone()
    x = torch.randn(20, 2, 64).to(torch.bfloat16).cuda()
    cache.write(batch, x, x)
    k, _ = cache.read(batch)
    assert torch.equal(k[:8], x[:8]) and (k[8:] == 0).all()
    keep = torch.ones(p.num_pages, dtype=torch.bool)
    keep[p.table[0, 0]] = False
    assert torch.equal(cache.k.view(torch.int16)[keep.cuda()], before.view(torch.int16)[keep.cuda()])


# ----------------------------------------------------------------------------- attention


def check_attention(p, heads, window=0, sinks=0, scale=None, seed=0, q=None, strided=False):
    g = gen(seed)
    scale = p.hd ** -0.5 if scale is None else scale
    if q is None:
        q = torch.randn(p.rows, heads + 2 * strided, p.hd, generator=g).to(p.act)
    qd = q.cuda()[:, strided:strided + heads]
    cache, batch = p.device()
    got = cache.attention(batch, qd, scale=scale, window=window, sinks=sinks)
    again = cache.attention(batch, qd, scale=scale, window=window, sinks=sinks)
    assert got.dtype == p.act and torch.equal(got, again)
    want, bound = R.attention_ref(p, q[:, strided:strided + heads], scale, window, sinks)
    far = (got.cpu().double() - want).abs()
    bad = ~(far <= bound)
    assert not bad.any(), "%d of %d off, worst %.3g times the bound at %s" % (
        int(bad.sum()), bad.numel(), float((far / bound.clamp(min=1e-300)).nan_to_num(1e9).max()),
        bad.nonzero()[0].tolist())


ATT = [
    # new, past, page, kv_heads, group, head_dim
    ([1], [0], 8, 1, 1, 64),
    ([1], [936], 16, 8, 8, 128),
    ([1, 1, 1, 1], [0, 15, 16, 700], 16, 2, 7, 128),
    ([1, 1], [1500, 129], 64, 1, 16, 256),
    ([4, 4, 4], [100, 0, 61], 32, 2, 4, 64),
    ([4, 2], [5, 250], 8, 2, 8, 128),
    ([2, 1], [40, 300], 16, 1, 8, 256),
    ([0, 3, 0, 1], [9, 0, 0, 77], 8, 4, 2, 64),
    ([37, 1, 90], [0, 200, 31], 16, 2, 4, 128),
    ([129], [0], 64, 1, 1, 64),
    ([65, 3], [70, 1], 8, 2, 2, 256),
    ([40], [600], 256, 1, 7, 128),
    ([200, 17], [3, 64], 128, 2, 8, 64),
]


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("new,past,page,kvh,group,hd", ATT)
def test_attention(dtype, new, past, page, kvh, group, hd):
    p = R.Paged(gen(hd + page + len(new)), new, past, page, kvh, hd, dtype, lead_rows=len(new) % 2, pad_rows=2)
    check_attention(p, kvh * group, strided=len(new) == 1)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 2), (64, 4), (100, 300), (130, 0), (4096, 16)])
@pytest.mark.parametrize("new,past,hd", [([1, 1], [700, 3], 128), ([150, 3], [100, 500], 64), ([33], [300], 256)])
def test_attention_window(dtype, window, sinks, new, past, hd):
    p = R.Paged(gen(window + hd), new, past, 32, 2, hd, dtype)
    check_attention(p, 8, window, sinks)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("new", [[1, 2], [80, 40]])
def test_attention_window_over_freed_pages(dtype, hd, new):
    """Pages that the window has left may be gone from the table."""
    p = R.Paged(gen(4), new, [400, 333], 16, 1, hd, dtype)
    window, sinks = 50, 20
    for s in range(2):
        low = p.total[s] - new[s] - window + 1
        for a in range(2, p.table.shape[1]):
            if a * 16 >= 32 and (a + 1) * 16 <= low:
                p.table[s, a] = -1 if a % 2 else p.num_pages + 5
    check_attention(p, 4, window, sinks)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("new", [[3, 2], [70, 30]])
def test_attention_rows_that_see_nothing(dtype, new):
    """Rows before the start of their sequence, and sequences whose pages are all gone."""
    p = R.Paged(gen(9), new + [2], [-2, -30, 10], 8, 2, 64, dtype)
    p.table[2] = -1
    check_attention(p, 4)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("new", [[1, 2], [80, 40]])
def test_attention_over_holes_in_the_table(dtype, hd, new):
    """Entries that are no page in the middle of what a row sees hide their keys;
    page 0, which stands in for them, is full of NaN."""
    p = R.Paged(gen(8), new, [1500, 700], 16, 1, hd, dtype)
    unused = int(p.unused.all(-1).nonzero()[0])
    swap = p.table == 0
    p.table[swap] = unused
    for data, scales in p.pools:
        data[[0, unused]] = data[[unused, 0]]
        if scales is not None:
            scales[[0, unused]] = scales[[unused, 0]]
    for a in (0, 3, 4, 17, 18, 19, 20, 21, 22, 23, 24, 25, 26, 27, 40):
        p.table[a % 2, a] = -1
    p.table[0, 30:47] = p.num_pages + 1
    check_attention(p, 4)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_attention_scales(dtype, scale):
    p = R.Paged(gen(21), [2, 45], [60, 20], 16, 1, 64, dtype)
    check_attention(p, 8, scale=scale)


def test_attention_scores_beyond_the_softmax_range():
    """One key far above the others, and scores far below zero for all keys."""
    for dtype in CACHES:
        p = R.Paged(gen(22), [1, 40], [150, 100], 16, 1, 64, dtype)
        q = torch.randn(p.rows, 2, 64, generator=gen(23)).to(p.act) * 16
        check_attention(p, 2, scale=1.0, q=q)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("kind", ["nan", "inf"])
@pytest.mark.parametrize("new,window", [([3, 4], 0), ([90, 70], 0), ([90, 70], 20), ([200], 33)])
def test_later_tokens_do_not_reach_earlier_rows(dtype, kind, new, window):
    """A token whose key and value are not finite: rows before it (and rows
    whose window has left it) come out as if it were not there."""
    p = R.Paged(gen(31), new, [40] * len(new), 16, 2, 64, dtype)
    bad = []
    for s, n in enumerate(new):
        at = p.total[s] - n + n * 2 // 3
        bad.append(at)
        page, slot = p.table[s, at // 16], at % 16
        for data, _ in p.pools:
            if dtype == "mxfp8":
                data[page, :, slot, 5] = 0x7F
            else:
                data[page, :, slot, 5] = math.nan if kind == "nan" else math.inf
    q = torch.randn(p.rows, 4, 64, generator=gen(1)).to(p.act)
    cache, batch = p.device()
    got = cache.attention(batch, q.cuda(), window=window).cpu().double()
    want, bound = R.attention_ref(p, q, 64 ** -0.5, window, 0)
    first = 0
    for s, n in enumerate(new):
        pos = torch.arange(p.total[s] - n, p.total[s])
        sees = (pos >= bad[s]) & ((pos - bad[s] < window) | (window == 0))
        rows = torch.arange(first, first + n)
        clean = rows[~sees]
        assert ((got[clean] - want[clean]).abs() <= bound[clean]).all()
        assert not torch.isfinite(got[rows[sees]][..., 5]).any()
        first += n


def test_attention_long_context_is_split():
    """One sequence over many workgroups: 70000 keys, of which the reference takes
    all; two heads of one token."""
    p = R.Paged(gen(40), [1, 1], [70000, 40], 64, 1, 64, "bf16", spare=1)
    check_attention(p, 2)
    p = R.Paged(gen(41), [2], [30000], 256, 1, 128, "mxfp8", spare=1)
    check_attention(p, 8, window=20000, sinks=1000)


def test_attention_many_sequences():
    n = 150
    p = R.Paged(gen(42), [1 + (s == 77) for s in range(n)], [(s * 37) % 211 for s in range(n)], 16, 1, 64, "bf16")
    check_attention(p, 4)
    p = R.Paged(gen(43), [1 + (s % 9) * 4 for s in range(n)], [(s * 37) % 97 for s in range(n)], 16, 1, 64, "mxfp8")
    check_attention(p, 4)


def test_operators_follow_other_streams_and_out():
    p = R.Paged(gen(50), [1, 1], [300, 20], 16, 2, 64, "bf16")
    cache, batch = p.device()
    q = torch.randn(2, 4, 64, generator=gen(51)).to(torch.bfloat16).cuda()
    want = cache.attention(batch, q)
    out = torch.full_like(want, 7.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cache.attention(batch, q, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got is out and torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_step_in_a_graph_follows_the_lengths(dtype):
    """norm, write and attention captured once; lengths, tokens and pages
    change between the replays; every replay equals the eager step."""
    g = gen(60)
    p = R.Paged(g, [1, 1, 1], [60, 300, 5], 16, 2, 64, dtype, spare=12)
    cache, batch = p.device()
    free = torch.arange(p.num_pages)[p.unused.all(-1)].to(torch.int32)[:3].cuda()
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    norm = block.RMSNorm(w, quant="mxfp8")
    x, r = (torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda") for _ in "xr")

    def step():
        res = norm(x, r)
        q = res.y.view(3, 4, 64)
        cache.write(batch, q[:, :2], q[:, 2:])
        return res, cache.attention(batch, q, window=128, sinks=4)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gres, gout = step()
    for it in range(5):
        x.copy_(torch.randn(3, 256, generator=g))
        r.copy_(torch.randn(3, 256, generator=g))
        batch.kv_len += 1
        batch.page_table[:, batch.page_table.shape[1] - 1] = free       # a page for each
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        a = [t.clone() for t in (gres.residual, gres.y, gres.q, gres.scale, gout)]
        res, out = step()
        torch.cuda.synchronize()
        for t, u in zip(a, (res.residual, res.y, res.q, res.scale, out)):
            assert torch.equal(t, u), it


def test_bound_tensors_are_not_replaced():
    """Assigning another tensor would leave the old address in the C structs."""
    p = R.Paged(gen(70), [1], [20], 16, 2, 64, "mxfp8")
    cache, batch = p.device()
    norm = block.RMSNorm(torch.ones(64, device="cuda"))
    for obj, names in ((batch, ("page_table", "row_offsets", "kv_len")), (cache, ("k", "v", "k_scale", "v_scale")),
                       (norm, ("weight",))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(obj, name, getattr(obj, name).clone())


@pytest.mark.parametrize("dtype,hd,new,group", [("bf16", 64, 1, 2), ("mxfp8", 64, 1, 4), ("mxfp8", 128, 1, 8), ("f32", 128, 1, 1),
                                                ("mxfp8", 128, 3, 8), ("bf16", 256, 1, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (600, 5)])
def test_attention_cut_of_uneven_sequences(dtype, hd, new, group, window, sinks):
    """More sequences than a wave has lanes and more tiles than runs; most are
    short, some are empty or long, so that runs begin and end anywhere in a unit."""
    n = 130
    past = [(s * 37) % 211 if s % 9 else 900 + (s * 131) % 1500 for s in range(n)]
    p = R.Paged(gen(80 + hd), [new * (s % 13 != 5) for s in range(n)], past, 16, 2, hd, dtype)
    check_attention(p, 2 * group, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("past", [769, 1023, 1024, 1025, 1535])
def test_attention_of_one_token_just_past_the_cut(dtype, past):
    """Few units: about as many runs as positions, some without tiles."""
    p = R.Paged(gen(90), [1], [past], 64, 1, 64, dtype)
    check_attention(p, 3)


def test_norm_codes_of_maxima_next_to_a_power_of_two():
    """Rows whose largest y lies as close below or above 2^k as the inputs allow: the
    scale is that of the 64-bit value, the codes are its nearest."""
    g = gen(91)
    x = torch.randn(512, 256, generator=g)
    x[:, ::32] = x[:, ::32].abs() + 6.0                        # the largest of each block
    s = x.to(torch.float32)
    rms = (s.double().square().mean(1, keepdim=True) + 1e-5).sqrt()
    w = torch.ones(256)
    w[::32] = (4.0 / (s[0, ::32].double() / rms[0])).float()     # row 0: within a step of 4
    near = s[0].clone()
    rows = torch.stack([near * f for f in torch.linspace(0.999999, 1.000001, 512)])
    res = block.RMSNorm(w.cuda(), quant="mxfp8")(rows.cuda())
    rows64 = rows.double()
    y = rows64 / (rows64.square().mean(1, keepdim=True) + float(torch.tensor(1e-5, dtype=torch.float32))).sqrt() * w.double()
    top = y.unflatten(-1, (-1, 32)).abs().amax(-1)
    # what the order of a 64-bit sum of 256 squares may move
    sure = (top * (1 - 2.0 ** -44)).frexp()[1] == (top * (1 + 2.0 ** -44)).frexp()[1]
    got = res.scale.cpu().int() - 127
    assert ((got == top.frexp()[1] - 9) | ~sure).all() and sure.float().mean() > 0.9
