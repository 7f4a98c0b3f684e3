"""The layer on codes that the norm made, and the decoder block of
examples/decoder_block.py: norm, cache, attention, norm with codes, experts."""
import dataclasses
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

from mixture_experts_layer_19_amd import binding as B
from mixture_experts_layer_19_amd import inputs as I
from mixture_experts_layer_19_amd.layer import DeviceLayer

import _block as R

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")
_spec = importlib.util.spec_from_file_location("decoder_block", _path)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


def work(dtype):
    return dataclasses.replace(I.workload("tiny"), H=512, I=256, Is=256, dtype=dtype)


@pytest.fixture(scope="module")
def layers():
    made = {}

    def get(dtype):
        if dtype not in made:
            made[dtype] = DeviceLayer(work(dtype))
        return made[dtype]

    yield get
    for lay in made.values():
        lay.close()


def codes_of(lay, x):
    """What the layer itself makes of x."""
    q = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    if lay.w.dtype == "fp8":
        B.moe_fp8_quantize(x, B.MOE_BF16, x.numel(), lay.w.fp8_x_scale, q)
        return q, None
    scale = torch.empty((x.shape[0], x.shape[1] // 32), dtype=torch.uint8, device="cuda")
    B.moe_mx_quantize(x, B.MOE_BF16, x.shape[0], x.shape[1], q, scale)
    return q, scale


@pytest.mark.parametrize("dtype", ["mxfp8", "w4a8", "fp8"])
@pytest.mark.parametrize("rows", [1, 5, 64, 300])
def test_layer_on_codes_is_the_layer(layers, dtype, rows):
    """Its own codes give its own result, bit for bit; other codes another."""
    lay = layers(dtype)
    x = torch.randn(rows, lay.w.H, generator=torch.Generator().manual_seed(rows)).to(torch.bfloat16).cuda()
    want = lay.forward(x).clone()
    q, scale = codes_of(lay, x)
    assert torch.equal(lay.forward(x, codes=(q, scale)), want)
    assert not torch.equal(lay.forward(x, codes=(q ^ 0x80, scale)), want)


def test_layer_refuses_codes_of_another_shape(layers):
    lay = layers("mxfp8")
    x = torch.randn(4, lay.w.H, device="cuda").to(torch.bfloat16)
    q, scale = codes_of(lay, x)
    for bad in ((q[:3], scale), (q, scale[:, :4]), (q.view(torch.int8), scale), (q, scale.T)):
        with pytest.raises(ValueError):
            lay.forward(x, codes=bad)
    with pytest.raises(B.MoeError):
        lay.forward(x, codes=(q, None))


def reference(blk, batch, new, total, x, residual):
    """(residual after the attention half in 64 bits, how far it may be off), from
    the block's own q and the cache's content."""
    n = blk.norm1(x, residual)
    qkv = torch.matmul(n.y, blk.wqkv).unflatten(1, (-1, blk.head_dim))
    q = qkv[:, :blk.heads].double().cpu()
    whole = example.batch_of(batch.page_table, total, total)
    ks, vs = (t.double().cpu().split(total) for t in blk.cache.read(whole))
    group, outs, bounds = blk.heads // blk.kv_heads, [], []
    for qs, k, v, nn, t in zip(q.split(new), ks, vs, new, total):
        k, v = (a.repeat_interleave(group, 1).transpose(0, 1) for a in (k, v))
        qh = qs.transpose(0, 1)
        sc = qh @ k.transpose(1, 2) * blk.head_dim ** -0.5
        mag = qh.abs() @ k.abs().transpose(1, 2) * blk.head_dim ** -0.5
        j, pos = torch.arange(t)[None], (t - nn + torch.arange(nn))[:, None]
        see = j <= pos
        if blk.window:
            see &= (j > pos - blk.window) | (j < blk.sinks)
        w = sc.masked_fill(~see, -torch.inf).softmax(-1)
        o, a = w @ v, w @ v.abs()
        # as in _block.attention_ref
        ds = (blk.head_dim + 2) * R.F32_HALF * mag.masked_fill(~see, 0).amax(-1, keepdim=True)
        rel = 2 * ds + 2.0 ** -21 + (t + 64) * R.F32_HALF
        if blk.cache.dtype != "f32":
            rel = rel + R.BF16_HALF
        outs.append(o.transpose(0, 1).flatten(1))
        bounds.append((R.half_step(blk.cache.act_dtype) * o.abs() + rel * a).transpose(0, 1).flatten(1))
    o, b, wo = torch.cat(outs), torch.cat(bounds), blk.wo.double().cpu()
    p, res = o @ wo, n.residual.double().cpu()
    half = R.half_step(blk.cache.act_dtype)
    bp = b @ wo.abs() + wo.shape[0] * R.F32_HALF * (o.abs() @ wo.abs())
    bp = bp + half * (p.abs() + bp)                            # the product's rounding
    s = p + res
    return s, bp + (half + R.F32_HALF) * (s.abs() + bp)


@pytest.mark.parametrize("dtype,cache,window,sinks", [("f32", "f32", 0, 0), ("bf16", "bf16", 0, 0),
                                                      ("mxfp8", "mxfp8", 0, 0), ("w4a8", "mxfp8", 40, 3),
                                                      ("fp8", "bf16", 100, 0)])
def test_decoder_block(layers, dtype, cache, window, sinks):
    """A prefill and single tokens after it: the attention half against 64 bits,
    the experts' half as the layer gives it on the second norm's output."""
    lay = layers(dtype)
    blk = example.DecoderBlock(lay.w, heads=8, kv_heads=2, head_dim=64, cache=cache, num_pages=64, page_size=16,
                               window=window, sinks=sinks, layer=lay)
    act = blk.cache.act_dtype
    total = [70, 1, 33, 130]
    table = example.page_table([t + 3 for t in total], 16, 64)
    g = torch.Generator().manual_seed(5)
    new = list(total)
    for _ in range(4):
        x, r = (torch.randn(sum(new), lay.w.H, generator=g).to(act).cuda() for _ in "xr")
        batch = example.batch_of(table, new, total)
        got, residual = blk(batch, x, r)
        want, bound = reference(blk, batch, new, total, x, r)
        assert ((residual.double().cpu() - want).abs() <= bound).all()
        n = blk.norm1(x, r)
        q = torch.matmul(n.y, blk.wqkv).unflatten(1, (-1, 64))[:, :8]
        a = blk.cache.attention(batch, q, window=window, sinks=sinks)
        n = blk.norm2(torch.matmul(a.flatten(1), blk.wo), n.residual)
        assert torch.equal(n.residual, residual)
        assert torch.equal(got, lay.forward(n.y, codes=None if n.q is None else (n.q, n.scale)))
        new, total = [1] * len(total), [t + 1 for t in total]
    with pytest.raises(ValueError):
        example.page_table([1000, 1000], 16, 64)
