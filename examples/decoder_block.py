"""A decoder block around the MoE layer: prompts of different lengths go in at
once, then one token of each sequence a step.

    python examples/decoder_block.py [--cache bf16|mxfp8] [--experts bf16|mxfp8|w4a8|fp8]
                                     [--projections fp8|torch] [--base B]
                                     [--window W --sinks S] [--steps N]

    residual += x;  n = norm(residual);  q, k, v = n Wqkv
    q, k = norms of their heads, turned by position;  cache <- k, v
    a = attention(q, cache) Wo
    residual += a;  n, codes = norm(residual);  x = moe(n, codes)

and behind the block

    residual += x;  logits = norm(residual) Whead;  log p of a token, entropy, the best ones

Projections and logits are products in E4M3 with a scale per block of 128 (or
torch's); base 0 leaves the norms and the turn of heads out.  The second norm writes the activations' 8-bit codes beside the rows, and the
experts read those.  Weights and inputs are random.
"""
import argparse
import dataclasses
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from mixture_experts_layer_19_amd import block, inputs
from mixture_experts_layer_19_amd.layer import DeviceLayer

# 8-bit activations of the experts' formats
QUANT = {"f32": "none", "bf16": "none", "mxfp8": "mxfp8", "w4a8": "mxfp8", "fp8": "fp8"}


class DecoderBlock:
    """Weights, cache and layer of one block of `workload`'s hidden size.

    projections: "torch", or "fp8" for block-scaled ones; base: of the rotation by
    position, with which queries and keys are normed for each head (None: neither)."""

    def __init__(self, workload, heads=64, kv_heads=8, head_dim=128, cache="mxfp8", num_pages=1024, page_size=64,
                 window=0, sinks=0, layer=None, projections="torch", base=None):
        dev = torch.device("cuda")
        act = torch.float32 if workload.dtype == "f32" else torch.bfloat16
        if (cache == "f32") != (act == torch.float32):
            raise ValueError("an fp32 layer goes with an f32 cache, the others with bf16 or mxfp8")
        g = torch.Generator(device=dev).manual_seed(7)
        H = workload.H

        def weight(rows, cols):
            return torch.randn((rows, cols), generator=g, device=dev).mul_(cols ** -0.5).to(act)

        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.window, self.sinks = window, sinks
        self.wqkv = weight((heads + 2 * kv_heads) * head_dim, H).T
        self.wo = weight(H, heads * head_dim).T
        self.project_qkv, self.project_o = (
            (lambda x, w=w: torch.matmul(x, w)) if projections == "torch" else block.BlockLinear(w.T, dtype=act)
            for w in (self.wqkv, self.wo))
        ones = torch.ones(H, dtype=act, device=dev)
        self.rope = None if base is None else block.HeadNormRope(ones[:head_dim].clone(), ones[:head_dim].clone(), base)
        self.norm1 = block.RMSNorm(ones)
        self.norm2 = block.RMSNorm(ones.clone(), quant=QUANT[workload.dtype], fp8_scale=workload.fp8_x_scale)
        self.cache = block.PagedKVCache(kv_heads, head_dim, num_pages, page_size, dtype=cache)
        self.moe = layer or DeviceLayer(workload)

    def __call__(self, batch, x, residual):
        """x, residual [rows, H] of the batch's new tokens -> the same after the block."""
        n = self.norm1(x, residual)
        qkv = self.project_qkv(n.y).unflatten(1, (-1, self.head_dim))
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)      # strided views
        if self.rope is None:
            self.cache.write(batch, k, v)
        else:
            q = self.rope.write(self.cache, batch, q, k, v)
        a = self.cache.attention(batch, q, window=self.window, sinks=self.sinks)
        n = self.norm2(self.project_o(a.flatten(1)), n.residual)
        return self.moe.forward(n.y, codes=None if n.q is None else (n.q, n.scale)), n.residual


class Answer:
    """From the last block's rows to tokens: a norm, the logits over `vocab` tokens, and what
    they say of given ones."""

    def __init__(self, hidden, vocab, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(11)
        self.norm = block.RMSNorm(torch.ones(hidden, dtype=dtype, device="cuda"))
        weight = torch.randn((vocab, hidden), generator=g, device="cuda").mul_(2 * hidden ** -0.5)
        self.head = block.BlockLinear(weight, dtype=dtype, out_dtype=torch.float32)

    def __call__(self, x, residual, tokens, top=0):
        return block.token_logprobs(self.head(self.norm(x, residual).y), tokens, top)


def page_table(lengths, page_size, num_pages):
    """[seqs, width] int32: consecutive pages for sequences of up to `lengths` tokens."""
    need = [-(-n // page_size) for n in lengths]
    if sum(need) > num_pages:
        raise ValueError("%d pages do not hold the sequences, which need %d" % (num_pages, sum(need)))
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.arange(at, at + n)
        at += n
    return table.cuda()


def batch_of(table, new, total):
    """KVBatch of `new` new tokens a sequence, `total` with them."""
    offsets = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    kv_len = torch.tensor(total, dtype=torch.int32).cuda()
    return block.KVBatch(table, offsets, kv_len, rows=sum(new), max_rows=max(new))


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--cache", default="mxfp8", choices=("bf16", "mxfp8"))
    ap.add_argument("--experts", default="mxfp8", choices=("bf16", "mxfp8", "w4a8", "fp8"))
    ap.add_argument("--projections", default="fp8", choices=("fp8", "torch"))
    ap.add_argument("--base", type=float, default=10000.0, help="of the rotation (0: no norms of heads, no rotation)")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    work = dataclasses.replace(inputs.workload("tiny"), H=1024, I=256, Is=256, dtype=a.experts)
    prompts = [611, 7, 64, 255, 1030, 1, 129, 400]
    blk = DecoderBlock(work, heads=16, kv_heads=2, head_dim=64, cache=a.cache, window=a.window, sinks=a.sinks,
                       projections=a.projections, base=a.base or None)
    table = page_table([n + a.steps for n in prompts], blk.cache.page_size, blk.cache.num_pages)
    g = torch.Generator(device="cuda").manual_seed(1)

    def rows(n):
        return torch.randn((n, work.H), generator=g, device="cuda").to(torch.bfloat16)

    x = rows(sum(prompts))
    x, _ = blk(batch_of(table, prompts, prompts), x, torch.zeros_like(x))
    print("prompts of %s tokens: output %s, rms %.3f" % (prompts, list(x.shape), x.float().square().mean().sqrt()))
    # one batch for all steps: its lengths are counted up on the device
    step = batch_of(table, [1] * len(prompts), [n + 1 for n in prompts])
    x = rows(len(prompts))
    residual = torch.zeros_like(x)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in "be")
    for i in range(a.steps):
        if i == min(2, a.steps - 1):
            begin.record()
        y, r = blk(step, x, residual)
        step.kv_len.add_(1)
    end.record()
    answer = Answer(work.H, 1000)
    said = answer(y, r, torch.arange(len(prompts), device="cuda"), top=3)
    torch.cuda.synchronize()
    timed = a.steps - min(2, a.steps - 1)
    print("%d steps of %d sequences: %.3f ms a step, rms %.3f"
          % (a.steps, len(prompts), begin.elapsed_time(end) / timed, y.float().square().mean().sqrt()))
    print("log probabilities of tokens 0 .. %d: %s\nbest alternatives: %s, entropies %s"
          % (len(prompts) - 1, ["%.2f" % v for v in said.logprob.tolist()], said.top_token.tolist(),
             ["%.2f" % v for v in said.entropy.tolist()]))


if __name__ == "__main__":
    main()
