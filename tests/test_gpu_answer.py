"""The decoder block of examples/decoder_block.py with block-scaled projections and turned
heads, and the answer behind it: each step against its own inputs in 64 bits, over a
prefill and single tokens, and as a captured graph."""
import dataclasses
import importlib.util
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from mixture_experts_layer_19_amd import inputs as I
from mixture_experts_layer_19_amd.layer import DeviceLayer

import _answer as A
import _block as R

pytestmark = pytest.mark.gpu

_root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_path = os.path.join(_root, "examples", "decoder_block.py")
_spec = importlib.util.spec_from_file_location("decoder_block_answer", _path)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


@pytest.fixture(scope="module")
def layer():
    lay = DeviceLayer(dataclasses.replace(I.workload("tiny"), H=512, I=256, Is=256, dtype="mxfp8"))
    yield lay
    lay.close()


def near(got, want, bound):
    off = (got.cpu().double() - want).abs()
    assert (off <= bound + 1e-38).all(), float((off / (bound + 1e-38)).max())


def check_product(lin, x, y):
    codes = A.unpack(lin.q.cpu(), lin.out_features, lin.in_features)[:lin.out_features, :lin.in_features]
    xq, xs = A.quantize_rows(x.cpu())
    near(y, *A.linear_ref(xq, xs, codes.view(torch.float8_e4m3fn).double(), lin.scale.cpu(), y.dtype))


def check_attention(blk, batch, q, out, new, total):
    whole = example.batch_of(batch.page_table, total, total)
    ks, vs = (t.double().cpu().split(total) for t in blk.cache.read(whole))
    group, at = blk.heads // blk.kv_heads, 0
    for k, v, n, t in zip(ks, vs, new, total):
        qh = q[at:at + n].double().cpu().transpose(0, 1)
        k, v = (a.repeat_interleave(group, 1).transpose(0, 1) for a in (k, v))
        see = torch.arange(t)[None] <= (t - n + torch.arange(n))[:, None]
        scale = blk.head_dim ** -0.5
        w = (qh @ k.transpose(1, 2) * scale).masked_fill(~see, -torch.inf).softmax(-1)
        mag = (qh.abs() @ k.abs().transpose(1, 2) * scale).masked_fill(~see, 0).amax(-1, keepdim=True)
        o, a = w @ v, w @ v.abs()
        # as in _block.attention_ref
        rel = 2 * (blk.head_dim + 2) * R.F32_HALF * mag + 2.0 ** -21 + (t + 64) * R.F32_HALF + R.BF16_HALF
        near(out[at:at + n].transpose(0, 1), o, R.half_step(out.dtype) * o.abs() + rel * a)
        at += n


@pytest.mark.parametrize("cache", ["bf16", "mxfp8"])
def test_block_and_answer(layer, cache):
    blk = example.DecoderBlock(layer.w, heads=8, kv_heads=2, head_dim=64, cache=cache, num_pages=64, page_size=16,
                               layer=layer, projections="fp8", base=10000.0)
    answer = example.Answer(layer.w.H, 1003)
    act = blk.cache.act_dtype
    total = [70, 1, 33, 130]
    table = example.page_table([t + 3 for t in total], 16, 64)
    g = torch.Generator().manual_seed(5)
    new = list(total)
    for _ in range(3):
        x, r = (torch.randn(sum(new), layer.w.H, generator=g).to(act).cuda() for _ in "xr")
        batch = example.batch_of(table, new, total)
        got, residual = blk(batch, x, r)
        # the same by its steps
        n = blk.norm1(x, r)
        qkv = blk.project_qkv(n.y)
        check_product(blk.project_qkv, n.y, qkv)
        q, k, v = qkv.unflatten(1, (-1, 64)).split((8, 2, 2), 1)
        turned = blk.rope.write(blk.cache, batch, q, k, v)
        pos = torch.cat([torch.arange(t - m, t) for m, t in zip(new, total)])
        inv, ones = blk.rope.inv_freq.cpu(), torch.ones(64)
        want, bound = A.turned(q.cpu(), ones, pos, inv, 1e-5, False, False)
        near(turned, want, A.half_step(act) * (want.abs() + bound) + bound)
        if cache == "bf16":
            kept, values = blk.cache.read(batch)
            want, bound = A.turned(k.cpu(), ones, pos, inv, 1e-5, False, False)
            near(kept, want, A.half_step(act) * (want.abs() + bound) + bound)
            assert torch.equal(values, v)
        a = blk.cache.attention(batch, turned)
        check_attention(blk, batch, turned, a, new, total)
        o = blk.project_o(a.flatten(1))
        check_product(blk.project_o, a.flatten(1), o)
        n2 = blk.norm2(o, n.residual)
        assert torch.equal(n2.residual, residual)
        assert torch.equal(got, layer.forward(n2.y, codes=(n2.q, n2.scale)))
        # the answer
        tokens = torch.randint(0, 1003, (sum(new),), generator=g)
        said = answer(got, residual, tokens.cuda(), top=5)
        y = answer.norm(got, residual).y
        logits = answer.head(y)
        check_product(answer.head, y, logits)
        lp, h, values, ids, b_lp, b_h, b_top = A.logprobs_ref(logits.cpu(), tokens, 5)
        near(said.logprob, lp, b_lp)
        near(said.entropy, h, b_h)
        near(said.top_logprob, values, b_top)
        assert torch.equal(said.top_token.cpu().long(), ids)
        new, total = [1] * len(total), [t + 1 for t in total]


def test_captured_step(layer):
    """A step of single tokens through block and answer as a graph, whose lengths are
    counted up between replays."""
    blk = example.DecoderBlock(layer.w, heads=8, kv_heads=2, head_dim=64, cache="mxfp8", num_pages=64, page_size=16,
                               layer=layer, projections="fp8", base=10000.0)
    answer = example.Answer(layer.w.H, 1003)
    g = torch.Generator().manual_seed(6)
    total = [20, 3, 47]
    table = example.page_table([t + 4 for t in total], 16, 64)
    x = torch.randn(sum(total), layer.w.H, generator=g).to(torch.bfloat16).cuda()
    blk(example.batch_of(table, total, total), x, torch.zeros_like(x))
    step = example.batch_of(table, [1] * 3, [t + 1 for t in total])
    x, r = (torch.randn(3, layer.w.H, generator=g).to(torch.bfloat16).cuda() for _ in "xr")
    tokens = torch.tensor([1, 500, 1002]).cuda()

    def run():
        y, res = blk(step, x, r)
        return (y, res) + tuple(answer(y, res, tokens, top=2))

    run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = run()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, run()):
            assert torch.equal(a, b)
        step.kv_len.add_(1)


def test_example_runs():
    """One whole run of the example, as its command line starts it."""
    p = subprocess.run([sys.executable, _path, "--steps", "3"], cwd=_root, capture_output=True, text=True, timeout=100)
    assert p.returncode == 0, p.stderr[-2000:]
    assert "log probabilities of tokens" in p.stdout
