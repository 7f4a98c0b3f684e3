"""Refusals of the norm, cache and attention entry points: everything here is
decided on the host, no GPU needed."""
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


def norm_args(B, **kw):
    a = dict(x=P, xs=64, r=P, rs=64, w=P, dt=B.MOE_BF16, rows=4, hidden=64, eps=1e-5, ro=P, y=P, qd=B.MOE_MXFP8,
             fs=1.0, q=P, s=P)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(hidden=0), dict(eps=-1.0), dict(eps=float("nan")), dict(dt=2),
                                dict(qd=7), dict(hidden=48), dict(x=None), dict(w=None), dict(ro=None), dict(r=None),
                                dict(q=None), dict(s=None), dict(q=P + 8), dict(x=P + 1), dict(y=P + 1)])
def test_norm_refuses(B, kw):
    refused(B, B.MOE_ERR_INVALID_ARG, B.moe_rms_norm, *norm_args(B, **kw))


def test_norm_refuses_by_output(B):
    refused(B, B.MOE_ERR_INVALID_ARG, B.moe_rms_norm, *norm_args(B, qd=B.MOE_NO_QUANT, y=None))
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        refused(B, B.MOE_ERR_INVALID_ARG, B.moe_rms_norm, *norm_args(B, qd=B.MOE_FP8, fs=bad))
    B.moe_rms_norm(*norm_args(B, rows=0, x=None))


def cache(B, **kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, num_pages=10, page_size=16, kv_heads=2, head_dim=128, dtype=B.MOE_MXFP8)
    a.update(kw)
    return B.MoeKvCache(**a)


def batch(B, **kw):
    a = dict(page_table=P, row_offsets=P, kv_len=P, seqs=3, max_pages=5, rows=6, max_rows=2)
    a.update(kw)
    return B.MoeKvBatch(**a)


INVALID = [(dict(num_pages=0), {}), (dict(page_size=0), {}), (dict(kv_heads=0), {}), (dict(head_dim=0), {}),
           (dict(dtype=9), {}), (dict(k=None), {}), (dict(v=P + 8), {}), (dict(k_scale=None), {}),
           ({}, dict(seqs=-1)), ({}, dict(seqs=0)), ({}, dict(rows=-1)), ({}, dict(max_rows=0)),
           ({}, dict(max_pages=0)), ({}, dict(page_table=None)), ({}, dict(row_offsets=None)),
           ({}, dict(kv_len=P + 2))]
UNSUPPORTED = [(dict(page_size=24), {}), (dict(page_size=1 << 17), {}), (dict(head_dim=96), {}),
               (dict(dtype=3), {}), (dict(dtype=4), {}), ({}, dict(max_pages=1 << 27)),
               ({}, dict(max_pages=(1 << 27) - 1, rows=20))]


@pytest.mark.parametrize("which,c,b", [("INVALID_ARG", c, b) for c, b in INVALID]
                         + [("UNSUPPORTED", c, b) for c, b in UNSUPPORTED])
def test_cache_calls_refuse(B, which, c, b):
    st = getattr(B, "MOE_ERR_" + which)
    c, b = cache(B, **c), batch(B, **b)
    refused(B, st, B.moe_kv_write, c, b, P, 256, 128, P, 256, 128)
    refused(B, st, B.moe_kv_read, c, b, P, P)
    refused(B, st, B.moe_attention, c, b, P, 512, 128, 4, 0.1, 0, 0, P, P, 1 << 30)
    assert B.moe_attention_workspace_bytes(c, b, 4, 0, 0) == 0


def test_operand_refusals(B):
    c, b, inv = cache(B), batch(B), B.MOE_ERR_INVALID_ARG
    for a in ((None, 256, 128, P, 256, 128), (P + 8, 256, 128, P, 256, 128), (P, 257, 128, P, 256, 128),
              (P, 256, 128, P, 256, 4)):
        refused(B, inv, B.moe_kv_write, c, b, *a)
    refused(B, inv, B.moe_kv_read, c, b, P, None)
    ok = dict(q=P, row=512, head=128, heads=4, scale=0.1, window=0, sinks=0, out=P, ws=P, n=1 << 30)
    for kw in (dict(q=None), dict(out=None), dict(out=P + 4), dict(ws=P + 4), dict(row=511), dict(head=129),
               dict(heads=3), dict(heads=0), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        refused(B, inv, B.moe_attention, c, b, *dict(ok, **kw).values())
    assert B.moe_attention_workspace_bytes(c, b, 4, 0, 0) == 0         # a short context needs none
    b = batch(B, max_pages=200)
    n = B.moe_attention_workspace_bytes(c, b, 4, 0, 0)
    assert n > 0
    refused(B, B.MOE_ERR_WORKSPACE, B.moe_attention, c, b, *dict(ok, n=n - 1).values())
    refused(B, B.MOE_ERR_WORKSPACE, B.moe_attention, c, b, *dict(ok, ws=None).values())


def test_calls_without_rows_do_nothing(B):
    c, b = cache(B), batch(B, rows=0, max_rows=0, seqs=0, page_table=None, row_offsets=None, kv_len=None)
    B.moe_kv_write(c, b, None, 0, 0, None, 0, 0)
    B.moe_kv_read(c, b, None, None)
    B.moe_attention(c, b, None, 0, 0, 4, 0.1, 0, 0, None, None, 0)


def test_python_entry_points_refuse(B):
    from mixture_experts_layer_19_amd import block
    with pytest.raises(ValueError):
        block.RMSNorm(torch.ones(64))                                  # not on a GPU
    with pytest.raises(ValueError):
        block.RMSNorm(torch.ones(48), quant="mxfp8")
    with pytest.raises(ValueError):
        block.RMSNorm(torch.ones(64), quant="int8")
    with pytest.raises(ValueError):
        block.RMSNorm(torch.ones(64), quant="fp8")
    with pytest.raises(ValueError):
        block.RMSNorm(torch.ones(64, dtype=torch.float16))
    for kw in (dict(dtype="fp16"), dict(page_size=24), dict(head_dim=80), dict(kv_heads=0)):
        a = dict(kv_heads=2, head_dim=64, num_pages=4, page_size=16, dtype="bf16", device="cpu")
        a.update(kw)
        with pytest.raises(ValueError):
            block.PagedKVCache(**a)
    with pytest.raises(ValueError):
        block.PagedKVCache(2, 64, 4, 16, device="cpu")
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        block.KVBatch(torch.zeros(2, 3, **i32), torch.zeros(2, **i32), torch.zeros(2, **i32), 2, 1)
    with pytest.raises(ValueError):
        block.KVBatch(torch.zeros(2, 3, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32), 2, 1)   # on the CPU


def test_layer_on_codes_refuses(B):
    def desc(expert):
        return B.MoeDesc(hidden=256, num_experts=4, top_k=2, inter=256, shared_inter=256, router_scaling_factor=1.0,
                         route_norm=1, act_dtype=B.MOE_BF16, expert_dtype=expert, out_dtype=B.MOE_BF16,
                         fp8_x_scale=1.0, fp8_h_scale=1.0, fp8_sh_h_scale=1.0)

    def call(expert, q, scale, status, T=4, ctx=None):
        refused(B, status, B.moe_layer_forward_quantized, ctx, desc(expert), B.MoeWeights(), P, q, scale, T, P, P, 1 << 30)

    call(B.MOE_BF16, P, P, B.MOE_ERR_UNSUPPORTED)
    for expert in (B.MOE_MXFP8, B.MOE_MXFP4):
        call(expert, None, P, B.MOE_ERR_INVALID_ARG)
        call(expert, P, None, B.MOE_ERR_INVALID_ARG)
        call(expert, P + 8, P, B.MOE_ERR_INVALID_ARG)
        call(expert, P, P + 8, B.MOE_ERR_INVALID_ARG)
    call(B.MOE_FP8, P, P, B.MOE_ERR_INVALID_ARG)
    call(B.MOE_MXFP8, P, P, B.MOE_ERR_INVALID_ARG)          # no context


def test_decoder_block_example_knows_every_format():
    import importlib.util
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    from mixture_experts_layer_19_amd import block, layer
    assert set(example.QUANT) == set(layer._DT)
    assert set(example.QUANT.values()) <= set(block._QUANT)
