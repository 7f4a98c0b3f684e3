"""Plain 64-bit references and inputs for the tests of the norm, the paged
cache and attention (not collected by pytest)."""
import math

import torch

MX_HALF = 2.0 ** -4            # E4M3: half a step, relative
BF16_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def e8m0(b):
    return torch.ldexp(torch.ones(b.shape, dtype=torch.float64), b.to(torch.int32) - 127)


def mx_values(codes, scales):
    """f64 values of E4M3 codes (uint8 [..., n]) under E8M0 bytes [..., n / 32]."""
    v = codes.view(torch.float8_e4m3fn).to(torch.float64)
    return (v.unflatten(-1, (-1, 32)) * e8m0(scales).unsqueeze(-1)).flatten(-2)


class Paged:
    """A cache and a batch on the host: random pages in random order, the rest
    of the pool (and the unused slots) full of NaN."""

    def __init__(self, g, new, past, page, kv_heads, head_dim, dtype, spare=3, pad_rows=0, lead_rows=0):
        self.new, self.page, self.kvh, self.hd, self.dtype = new, page, kv_heads, head_dim, dtype
        self.total = [max(0, n + p) for n, p in zip(new, past)]     # past may be negative: rows before the start
        act = torch.float32 if dtype == "f32" else torch.bfloat16
        self.act = act
        need = [-(-t // page) for t in self.total]
        self.num_pages = sum(need) + spare
        order = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        width = max(need + [1]) + 1
        table, at = [], 0
        for p in need:
            table.append(torch.nn.functional.pad(order[at:at + p], (0, width - p), value=-1))
            at += p
        self.table = torch.stack(table)
        off = [lead_rows]
        for n in new:
            off.append(off[-1] + n)
        self.offsets = torch.tensor(off, dtype=torch.int32)
        self.kv_len = torch.tensor(self.total, dtype=torch.int32)
        self.rows = off[-1] + pad_rows
        shape = (self.num_pages, kv_heads, page, head_dim)
        self.pools = []
        for _ in "kv":
            if dtype == "mxfp8":
                codes = (torch.randn(shape, generator=g) * 120).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                scales = torch.randint(117, 124, shape[:-1] + (head_dim // 32,), generator=g, dtype=torch.uint8)
                self.pools.append([codes, scales])
            else:
                self.pools.append([torch.randn(shape, generator=g).to(act), None])
        used = torch.zeros(self.num_pages, page, dtype=torch.bool)
        for s, t in enumerate(self.total):
            for j in range(t):
                used[self.table[s, j // page], j % page] = True
        self.unused = ~used
        for data, scales in self.pools:
            bad = 0x7F if dtype == "mxfp8" else math.nan
            data.masked_fill_(self.unused[:, None, :, None], bad)

    def values(self, which):
        data, scales = self.pools[which]
        return data.to(torch.float64) if scales is None else mx_values(data, scales)

    def context(self, s, which):
        """f64 [kv_heads, total, head_dim] of sequence s (NaN where there is no page)."""
        pool, t = self.values(which), self.total[s]
        out = torch.full((self.kvh, t, self.hd), math.nan, dtype=torch.float64)
        for j in range(t):
            p = int(self.table[s, j // self.page])
            if 0 <= p < self.num_pages:
                out[:, j] = pool[p, :, j % self.page]
        return out

    def device(self):
        from mixture_experts_layer_19_amd import block
        (k, ks), (v, vs) = [[None if x is None else x.cuda() for x in p] for p in self.pools]
        cache = block.PagedKVCache(self.kvh, self.hd, self.num_pages, self.page, dtype=self.dtype,
                                   storage=(k, v, ks, vs))
        batch = block.KVBatch(self.table.cuda(), self.offsets.cuda(), self.kv_len.cuda(), rows=self.rows,
                              max_rows=max(self.new + [1]) if self.rows else 0)
        return cache, batch


def attention_ref(p: Paged, q, scale, window, sinks):
    """(out, bound): f64 attention row by row, and how far a result in the
    cache's arithmetic may be off, element by element:
      half a step of the output's type, relative to the output; and relative to
      sum_j w_j |v_j|: half a step of bf16 where the weights are rounded to it,
      twice the error of a score (head_dim + 2 roundings of fp32, relative to
      scale * sum |q k|), and a rounding of fp32 or the exponential (2^-21) for
      each of n additions and rescalings (n + 64) * 2^-24."""
    heads = q.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64)
    bound = torch.zeros(q.shape, dtype=torch.float64)
    group = heads // p.kvh
    first = int(p.offsets[0])
    for s, n in enumerate(p.new):
        k, v = p.context(s, 0), p.context(s, 1)
        for i in range(n):
            pos = p.total[s] - n + i
            j = torch.arange(max(pos + 1, 0))
            if window:
                j = j[(j > pos - window) | (j < sinks)]
            j = j[[0 <= int(p.table[s, a // p.page]) < p.num_pages for a in j.tolist()]] if len(j) else j
            if not len(j):
                continue
            qq = q[first + i].to(torch.float64).view(p.kvh, group, -1)
            sc = torch.matmul(qq, k[:, j].transpose(1, 2)) * scale
            mag = torch.matmul(qq.abs(), k[:, j].abs().transpose(1, 2)) * abs(scale)
            w = torch.softmax(sc, -1)
            o = torch.matmul(w, v[:, j])
            a = torch.matmul(w, v[:, j].abs())
            ds = (p.hd + 2) * F32_HALF * mag.amax(-1, keepdim=True)
            rel = 2 * ds + 2.0 ** -21 + (len(j) + 64) * F32_HALF
            if p.dtype != "f32":
                rel = rel + BF16_HALF
            out[first + i] = o.reshape(heads, -1)
            bound[first + i] = (half_step(p.act) * o.abs() + rel * a).reshape(heads, -1)
        first += n
    return out, bound


def norm_ref(x, residual, weight, eps):
    s = x.to(torch.float64) + (0 if residual is None else residual.to(torch.float64))
    return s, s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps) * weight.to(torch.float64)
