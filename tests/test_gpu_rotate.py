"""Norms of queries and keys with their rotation, by themselves and into the paged
cache, against plain 64-bit forms."""
import math

import pytest

torch = pytest.importorskip("torch")

from mixture_experts_layer_19_amd import binding as B
from mixture_experts_layer_19_amd import block

import _answer as R
import _block as P

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def weights(g, d, dtype):
    return [(1 + 0.2 * torch.randn(d, generator=g)).to(dtype) for _ in "qk"]


def near(got, want, bound, dtype):
    off = (got.cpu().double() - want).abs()
    lim = R.half_step(dtype) * (want.abs() + bound) + bound + 1e-38
    assert (off <= lim).all(), float((off / lim).max())


SHAPES = [
    # rows, heads, kv_heads, head_dim, rotary
    (1, 1, 1, 64, 64), (3, 5, 1, 128, 128), (7, 8, 2, 256, 256), (2, 64, 8, 128, 128), (33, 7, 7, 64, 32),
    (5, 3, 3, 256, 64), (9, 16, 2, 128, 48), (4, 28, 4, 256, 160), (70, 9, 1, 128, 16),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,h,kvh,d,rot", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("after", [False, True])
def test_turn(dtype, rows, h, kvh, d, rot, inter, after):
    g = gen(rows * 7 + h + d + rot)
    wq, wk = weights(g, d, dtype)
    fused = (3 * torch.randn(rows, h + kvh + 1, d, generator=g)).to(dtype)
    q, k = fused[:, :h], fused[:, h + 1:]
    pos = torch.randint(0, 1 << 20, (rows,), generator=g, dtype=torch.int32)
    dev = fused.cuda()
    rope = block.HeadNormRope(wq.cuda(), wk.cuda(), base=500000.0, rotary_dim=rot, eps=1e-6, interleaved=inter,
                              norm_after=after)
    gq, gk = rope(dev[:, :h], dev[:, h + 1:], pos.cuda())
    for got, x, w in ((gq, q, wq), (gk, k, wk)):
        assert got.shape == x.shape and got.dtype == dtype and got.is_contiguous()
        near(got, *R.turned(x, w, pos, rope.inv_freq.cpu(), 1e-6, inter, after), dtype)


def test_far_and_negative_positions_and_own_frequencies():
    g = gen(1)
    wq, wk = weights(g, 128, F32)
    q, k = torch.randn(6, 2, 128, generator=g), torch.randn(6, 2, 128, generator=g)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32)
    for inv in (torch.rand(64, generator=g), torch.rand(24, generator=g, dtype=torch.float64) * 3):
        rope = block.HeadNormRope(wq.cuda(), wk.cuda(), inv_freq=inv.cuda())
        assert rope.rotary_dim == 2 * inv.numel()
        gq, gk = rope(q.cuda(), k.cuda(), pos.cuda())
        near(gq, *R.turned(q, wq, pos, inv, 1e-5, False, False), F32)
        near(gk, *R.turned(k, wk, pos, inv, 1e-5, False, False), F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_extremes(dtype):
    """Heads of the largest and smallest values, of zeros, with an infinity or NaN."""
    g = gen(2)
    wq, wk = weights(g, 64, dtype)
    q = torch.randn(4, 3, 64, generator=g)
    q[0] *= 1e37
    q[1] *= 1e-37
    q[2] = 0
    q = q.to(dtype)
    pos = torch.arange(4, dtype=torch.int32)
    rope = block.HeadNormRope(wq.cuda(), wk.cuda(), eps=0.0)
    gq, _ = rope(q.cuda(), q.cuda(), pos.cuda())
    keep = torch.tensor([0, 1, 3])
    near(gq[keep.cuda()], *R.turned(q[keep], wq, pos[keep], rope.inv_freq.cpu(), 0.0, False, False), dtype)
    assert gq[2].isnan().all()                                  # 0 / 0
    rope = block.HeadNormRope(wq.cuda(), wk.cuda(), rotary_dim=32)
    gq, _ = rope(q.cuda(), q.cuda(), pos.cuda())
    assert (gq[2] == 0).all()
    q[3, 0, 40], q[3, 1, 40] = math.inf, math.nan
    gq, _ = rope(q.cuda(), q.cuda(), pos.cuda())
    head = gq[3, 0].cpu()
    assert head[40].isnan() and (head[:40] == 0).all() and (head[41:] == 0).all()
    assert gq[3, 1].isnan().all() and gq[3, 2].isfinite().all()


def test_no_rows():
    w = torch.ones(128, device="cuda")
    rope = block.HeadNormRope(w, w)
    e = torch.empty(0, 4, 128, device="cuda")
    q, k = rope(e, e[:, :2], torch.empty(0, dtype=torch.int32, device="cuda"))
    assert q.shape == (0, 4, 128) and k.shape == (0, 2, 128)


# ----------------------------------------------------------------------------- into the cache

BATCHES = [
    # new, past, page, heads, kv_heads, head_dim, rotary
    ([1], [0], 8, 1, 1, 64, 64),
    ([1, 1, 1], [0, 7, 8], 8, 6, 2, 128, 128),
    ([0, 5, 1, 0, 17], [3, 12, 0, 0, 31], 16, 28, 4, 64, 32),
    ([33, 1, 70], [0, 63, 1], 64, 64, 8, 128, 128),
    ([9], [250], 1, 3, 1, 256, 256),
    ([6, 4], [-3, 20], 4, 4, 2, 128, 64),                       # rows before the start
]


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8", "f32"])
@pytest.mark.parametrize("new,past,page,h,kvh,d,rot", BATCHES)
@pytest.mark.parametrize("inter", [False, True])
def test_write(dtype, new, past, page, h, kvh, d, rot, inter):
    g = gen(page + d + h)
    p = P.Paged(g, new, past, page, kvh, d, dtype, lead_rows=2, pad_rows=3)
    cache, batch = p.device()
    wq, wk = weights(g, d, p.act)
    fused = (2 * torch.randn(p.rows, h + 2 * kvh, d, generator=g)).to(p.act)
    dev = fused.cuda()
    q, k, v = dev[:, :h], dev[:, h:h + kvh], dev[:, h + kvh:]
    before = [t.cpu().clone() for t in (cache.k, cache.v)]
    rope = block.HeadNormRope(wq.cuda(), wk.cuda(), rotary_dim=rot, interleaved=inter)
    out = rope.write(cache, batch, q, k, v)
    # where each row goes
    pos, page_at, slot = (torch.full((p.rows,), -1) for _ in range(3))
    first = 2
    for s, n in enumerate(new):
        for i in range(n):
            at = p.total[s] - n + i
            if at >= 0:
                pos[first + i], page_at[first + i], slot[first + i] = at, int(p.table[s, at // page]), at % page
        first += n
    own = pos >= 0
    inv = rope.inv_freq.cpu()
    assert (out.cpu()[~own] == 0).all()
    near(out.cpu()[own], *R.turned(fused[own][:, :h], wq, pos[own], inv, 1e-5, inter, False), p.act)
    want_k, bound = R.turned(fused[own][:, h:h + kvh], wk, pos[own], inv, 1e-5, inter, False)
    where = (page_at[own], slot[own])
    if dtype != "mxfp8":
        near(cache.k.cpu().transpose(1, 2)[where], want_k, bound, p.act)
        assert torch.equal(cache.v.cpu().transpose(1, 2)[where], fused[own][:, h + kvh:])
    else:
        sb = cache.k_scale.cpu().transpose(1, 2)[where]
        top = want_k.unflatten(-1, (-1, 32)).abs().amax(-1)
        slack = bound.unflatten(-1, (-1, 32)).amax(-1)
        exp = (torch.frexp(top)[1] - 9).clamp(min=-127)
        close = torch.frexp(top + slack)[1] != torch.frexp(top - slack)[1]
        assert ((sb.int() - 127 == exp) | close).all()
        unit = P.e8m0(sb).repeat_interleave(32, -1)
        want = (want_k / unit).clamp(-448, 448)
        got = cache.k.cpu().transpose(1, 2)[where].view(torch.float8_e4m3fn).double()
        assert ((got - want).abs() <= P.MX_HALF * want.abs() + 2.0 ** -10 + 2 * bound / unit).all()
        # values: exactly what the cache's own write makes of them
        plain, _ = p.device()
        plain.write(batch, k, v)
        for a, b in ((cache.v, plain.v), (cache.v_scale, plain.v_scale)):
            assert torch.equal(a.cpu().transpose(1, 2)[where], b.cpu().transpose(1, 2)[where])
    # every other slot is as it was
    kept = torch.ones(p.num_pages, page, dtype=torch.bool)
    kept[where] = False
    for t, old in zip((cache.k, cache.v), before):
        a, b = t.cpu().transpose(1, 2)[kept], old.transpose(1, 2)[kept]
        bits = torch.uint8 if dtype == "mxfp8" else torch.int16 if dtype == "bf16" else torch.int32
        assert torch.equal(a.contiguous().view(bits), b.contiguous().view(bits))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_is_turn_then_write(dtype):
    """Into a cache of the activations' type: the same bits as in two steps."""
    g = gen(9)
    p = P.Paged(g, [40, 1, 0, 13], [5, 100, 7, 0], 16, 4, 128, dtype)
    (one, batch), (two, _) = p.device(), p.device()
    wq, wk = (w.cuda() for w in weights(g, 128, p.act))
    q, k, v = (torch.randn(p.rows, n, 128, generator=g).to(p.act).cuda() for n in (12, 4, 4))
    rope = block.HeadNormRope(wq, wk)
    pos = torch.cat([torch.arange(t - n, t) for n, t in zip(p.new, p.total)]).to(torch.int32).cuda()
    a = rope.write(one, batch, q, k, v)
    b, kk = rope(q, k, pos)
    two.write(batch, kk, v)
    assert torch.equal(a, b)
    for x, y in ((one.k, two.k), (one.v, two.v)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_write_without_a_page():
    """Rows whose table entry is no page drop their keys and values; their queries are
    computed all the same."""
    g = gen(4)
    p = P.Paged(g, [20], [0], 8, 2, 64, "bf16")
    p.table[0, 1] = -1
    cache, batch = p.device()
    before = cache.k.clone()
    wq, wk = (w.cuda() for w in weights(g, 64, BF16))
    q, k, v = (torch.randn(20, n, 64, generator=g).to(BF16).cuda() for n in (4, 2, 2))
    rope = block.HeadNormRope(wq, wk)
    out = rope.write(cache, batch, q, k, v)
    want, _ = rope(q, k, torch.arange(20, dtype=torch.int32).cuda())
    assert torch.equal(out, want)
    used = [int(t) for t in p.table[0] if t >= 0]
    rest = [i for i in range(p.num_pages) if i not in used]
    assert torch.equal(cache.k[rest].view(torch.int16), before[rest].view(torch.int16))


def test_captured():
    g = gen(8)
    p = P.Paged(g, [1, 1, 1], [5, 30, 0], 16, 2, 128, "mxfp8")
    cache, batch = p.device()
    wq, wk = (w.cuda() for w in weights(g, 128, BF16))
    rope = block.HeadNormRope(wq, wk)
    q, k, v = (torch.randn(3, n, 128, generator=g).to(BF16).cuda() for n in (4, 2, 2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = rope.write(cache, batch, q, k, v)
    for step in range(3):
        batch.kv_len.copy_(torch.tensor(p.total, dtype=torch.int32) - step % 2)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, rope.write(cache, batch, q, k, v))


def test_refuses():
    w = torch.ones(128, device="cuda", dtype=BF16)
    for bad in (dict(q_weight=w, k_weight=w[:64]), dict(q_weight=w, k_weight=w.float()), dict(q_weight=w[:96], k_weight=w[:96]),
                dict(q_weight=w.half(), k_weight=w.half()), dict(q_weight=w, k_weight=w, rotary_dim=0),
                dict(q_weight=w, k_weight=w, rotary_dim=24), dict(q_weight=w, k_weight=w, rotary_dim=144),
                dict(q_weight=w, k_weight=w, rotary_dim=3, interleaved=True), dict(q_weight=w, k_weight=w, eps=-1.0),
                dict(q_weight=w, k_weight=w, base=0.0), dict(q_weight=w, k_weight=w, inv_freq=torch.ones(64)),
                dict(q_weight=w, k_weight=w, inv_freq=torch.ones(65, device="cuda")),
                dict(q_weight=w, k_weight=w, rotary_dim=64, inv_freq=torch.ones(64, device="cuda")),
                dict(q_weight=w.cpu(), k_weight=w.cpu())):
        with pytest.raises(ValueError):
            block.HeadNormRope(**bad)
    rope = block.HeadNormRope(w, w)
    q = torch.randn(4, 3, 128, device="cuda").to(BF16)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for a in ((q.float(), q, pos), (q, q[:3], pos), (q[..., :64], q, pos), (q[:, :0], q, pos), (q, q, pos.long()),
              (q, q, pos[:3]), (q, q, pos.cpu()), (q.transpose(1, 2), q, pos)):
        with pytest.raises(ValueError):
            rope(*a)
    wide = torch.zeros(4, 3 * 128 + 4, device="cuda", dtype=BF16)
    with pytest.raises(B.MoeError):                            # strides of no whole 16 bytes
        rope(wide[:, :384].unflatten(1, (3, 128)), q, pos)
    cache = block.PagedKVCache(2, 64, 4, 16)
    batch = block.KVBatch(torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                          torch.tensor([0, 4], dtype=torch.int32, device="cuda"),
                          torch.tensor([4], dtype=torch.int32, device="cuda"), rows=4)
    with pytest.raises(ValueError):                            # another head_dim
        rope.write(cache, batch, q, q[:, :2], q[:, :2])
    cache = block.PagedKVCache(2, 128, 4, 16, dtype="f32")
    with pytest.raises(ValueError):                            # another type
        rope.write(cache, batch, q, q[:, :2], q[:, :2])
    cache = block.PagedKVCache(2, 128, 4, 16)
    with pytest.raises(ValueError):
        rope.write(cache, batch, q[:3], q[:, :2], q[:, :2])
