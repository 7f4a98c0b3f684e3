"""Refusals of the head norms with rotation, the block-scaled product and the token
log probabilities: everything here is decided on the host, no GPU needed."""
import os

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_19_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from mixture_experts_layer_19_amd import build
        build.build()
    binding.lib()
    return binding


P = 1 << 20          # a pointer that is aligned and never read


def refused(B, status, f, *args):
    with pytest.raises(B.MoeError) as ei:
        f(*args)
    assert ei.value.status == status



# ----------------------------------------------------------------------------- head norms


def head_norm(B, kw):
    a = dict(q_weight=P, k_weight=P, inv_freq=P, head_dim=128, rotary_dim=128, interleaved=0, norm_after=0,
             dtype=B.MOE_BF16, eps=1e-5)
    a.update({k: kw.pop(k) for k in list(kw) if k in a})
    return B.MoeHeadNorm(**a)


def turn(B, **kw):
    n = head_norm(B, kw)
    a = dict(q=P, q_row=1024, q_head=128, heads=8, k=P, k_row=256, k_head=128, kv_heads=2, positions=P, rows=4,
             q_out=P, k_out=P)
    a.update(kw)
    B.moe_head_norm_rope(n, *a.values())


def write(B, cache=None, batch=None, **kw):
    c = dict(k=P, v=P, k_scale=P, v_scale=P, num_pages=10, page_size=16, kv_heads=2, head_dim=128, dtype=B.MOE_MXFP8)
    c.update(cache or {})
    b = dict(page_table=P, row_offsets=P, kv_len=P, seqs=3, max_pages=5, rows=6, max_rows=2)
    b.update(batch or {})
    n = head_norm(B, kw)
    a = dict(q=P, q_row=1024, q_head=128, heads=8, k=P, k_row=256, k_head=128, v=P, v_row=256, v_head=128, q_out=P)
    a.update(kw)
    B.moe_head_norm_rope_write(n, B.MoeKvCache(**c), B.MoeKvBatch(**b), *a.values())


SHARED = [dict(q_weight=None), dict(k_weight=P + 8), dict(inv_freq=None), dict(inv_freq=P + 4), dict(rotary_dim=0),
          dict(rotary_dim=130), dict(rotary_dim=24), dict(rotary_dim=3, interleaved=1), dict(dtype=2), dict(eps=-1.0),
          dict(eps=float("nan")), dict(heads=0), dict(q=None), dict(q=P + 8), dict(k=None), dict(q_out=P + 8),
          dict(q_row=1020), dict(q_head=4), dict(k_row=252), dict(k_head=1)]


@pytest.mark.parametrize("kw", SHARED)
def test_head_norms_refuse(B, kw):
    refused(B, B.MOE_ERR_INVALID_ARG, lambda: turn(B, **kw))
    refused(B, B.MOE_ERR_INVALID_ARG, lambda: write(B, **kw))


@pytest.mark.parametrize("kw", [dict(positions=None), dict(positions=P + 2), dict(k_out=None), dict(rows=-1),
                                dict(kv_heads=0)])
def test_turn_refuses(B, kw):
    refused(B, B.MOE_ERR_INVALID_ARG, lambda: turn(B, **kw))


def test_head_norms_unsupported(B):
    refused(B, B.MOE_ERR_UNSUPPORTED, lambda: turn(B, head_dim=96, rotary_dim=96))
    refused(B, B.MOE_ERR_UNSUPPORTED, lambda: turn(B, heads=70000))
    refused(B, B.MOE_ERR_UNSUPPORTED, lambda: turn(B, kv_heads=2000))
    turn(B, rows=0, q=None, k=None, positions=None, q_out=None, k_out=None)


def test_write_refuses(B):
    bad = B.MOE_ERR_INVALID_ARG
    for kw in (dict(v=None), dict(v=P + 4), dict(v_row=2), dict(v_head=12), dict(head_dim=64, rotary_dim=64),
               dict(dtype=B.MOE_F32)):
        refused(B, bad, lambda: write(B, **kw))
    refused(B, bad, lambda: write(B, cache=dict(dtype=B.MOE_F32)))
    refused(B, bad, lambda: write(B, cache=dict(k=None)))
    refused(B, bad, lambda: write(B, batch=dict(row_offsets=None)))
    refused(B, bad, lambda: write(B, batch=dict(max_rows=0)))
    refused(B, B.MOE_ERR_UNSUPPORTED, lambda: write(B, cache=dict(page_size=48)))
    write(B, batch=dict(rows=0), q=None, k=None, v=None, q_out=None)


# ----------------------------------------------------------------------------- product


def test_sizes(B):
    assert B.moe_block_packed_bytes(1, 1) == 2048
    assert B.moe_block_packed_bytes(17, 129) == 2 * 2 * 2048
    assert B.moe_block_packed_bytes(0, 5) == 0 and B.moe_block_packed_bytes(5, -1) == 0
    assert B.moe_block_packed_bytes((1 << 30) + 1, 5) == 0
    assert B.moe_block_packed_bytes(1 << 20, 1 << 20) == 1 << 40
    assert B.moe_block_linear_workspace_bytes(0, 5, 5) == 0
    assert B.moe_block_linear_workspace_bytes(17, 5, 3000) >= 2 * 24 * 2048 + 24 * 32 * 4
    assert B.moe_block_linear_workspace_bytes(17, 5, 3000, codes=True) == 0
    assert B.moe_block_linear_workspace_bytes(17, 5, 129) == 0                      # codes in the LDS
    assert B.moe_block_linear_workspace_bytes(70, 100, 8192, codes=True) > 0       # split blocks


@pytest.mark.parametrize("kw", [dict(dt=2), dict(rows=-1), dict(cols=0), dict(x=None), dict(x=P + 1), dict(q=None),
                                dict(q=P + 8), dict(s=None), dict(s=P + 4)])
def test_quantize_refuses(B, kw):
    a = dict(x=P, dt=B.MOE_BF16, stride=256, rows=4, cols=256, q=P, s=P)
    a.update(kw)
    refused(B, B.MOE_ERR_INVALID_ARG, B.moe_block_quantize, *a.values())


def test_quantize_limits(B):
    refused(B, B.MOE_ERR_UNSUPPORTED, B.moe_block_quantize, P, B.MOE_BF16, 1, (1 << 30) + 1, 1, P, P)
    B.moe_block_quantize(None, B.MOE_F32, 1, 0, 1, None, None)


@pytest.mark.parametrize("kw", [dict(dt=2), dict(n=0), dict(k=-1), dict(w=None), dict(w=P + 1), dict(q=None),
                                dict(q=P + 8), dict(s=None), dict(s=P + 2)])
def test_pack_refuses(B, kw):
    a = dict(w=P, dt=B.MOE_BF16, stride=256, n=4, k=256, q=P, s=P)
    a.update(kw)
    refused(B, B.MOE_ERR_INVALID_ARG, B.moe_block_pack, *a.values())


def test_pack_limits(B):
    refused(B, B.MOE_ERR_UNSUPPORTED, B.moe_block_pack, P, B.MOE_FP8, 1, 1 << 30, 1 << 30, P, None)


LINEAR = dict(w=P, ws_=P, n=256, k=512, x=P, xdt=1, xs=512, xq=None, xqs=None, rows=100, out=P, odt=1, ws=P,
              size=1 << 30)


@pytest.mark.parametrize("kw", [dict(w=None), dict(w=P + 8), dict(ws_=None), dict(ws_=P + 2), dict(n=0), dict(k=0),
                                dict(x=None), dict(x=P + 1), dict(xdt=2), dict(xq=P), dict(xqs=P), dict(rows=-1),
                                dict(out=None), dict(out=P + 8), dict(odt=2), dict(ws=P + 8),
                                dict(xq=P + 8, xqs=P), dict(xq=P, xqs=P + 8)])
def test_linear_refuses(B, kw):
    refused(B, B.MOE_ERR_INVALID_ARG, B.moe_block_linear, *{**LINEAR, **kw}.values())


def test_linear_workspace_and_limits(B):
    need = B.moe_block_linear_workspace_bytes(100, 256, 512)
    refused(B, B.MOE_ERR_WORKSPACE, B.moe_block_linear, *{**LINEAR, "size": need - 1}.values())
    refused(B, B.MOE_ERR_WORKSPACE, B.moe_block_linear, *{**LINEAR, "ws": None}.values())
    split = {**LINEAR, "rows": 70, "n": 100, "k": 8192, "x": None, "xs": 0, "xq": P, "xqs": P}
    need = B.moe_block_linear_workspace_bytes(70, 100, 8192, codes=True)
    refused(B, B.MOE_ERR_WORKSPACE, B.moe_block_linear, *{**split, "size": need - 1}.values())
    refused(B, B.MOE_ERR_UNSUPPORTED, B.moe_block_linear, *{**LINEAR, "k": (1 << 30) + 1}.values())
    refused(B, B.MOE_ERR_UNSUPPORTED, B.moe_block_linear, *{**LINEAR, "rows": 1 << 30, "n": 1 << 30}.values())
    B.moe_block_linear(*{**LINEAR, "rows": 0, "x": None, "out": None, "ws": None}.values())


# ----------------------------------------------------------------------------- log probabilities


LOGPROBS = dict(x=P, dt=1, stride=1000, t=P, tb=4, rows=4, vocab=1000, top=5, lp=P, h=P, tl=P, tt=P)


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=P + 1), dict(dt=2), dict(t=None), dict(t=P + 2), dict(tb=2),
                                dict(tb=8, t=P + 4), dict(rows=-1), dict(vocab=0), dict(top=-1), dict(top=65),
                                dict(vocab=4), dict(lp=None), dict(h=P + 1), dict(tl=None), dict(tt=None)])
def test_logprobs_refuse(B, kw):
    refused(B, B.MOE_ERR_INVALID_ARG, B.moe_token_logprobs, *{**LOGPROBS, **kw}.values())


def test_logprobs_of_no_rows(B):
    B.moe_token_logprobs(*{**LOGPROBS, "rows": 0, "x": None, "t": None}.values())


def test_python_refuses_what_is_not_on_a_gpu():
    from mixture_experts_layer_19_amd import block
    w = torch.ones(128)
    with pytest.raises(ValueError):
        block.HeadNormRope(w, w)
    with pytest.raises(ValueError):
        block.BlockLinear(torch.ones(4, 128))
    with pytest.raises(ValueError):
        block.token_logprobs(torch.ones(4, 128), torch.zeros(4, dtype=torch.int32))
