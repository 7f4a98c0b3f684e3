"""Cases of the operators from the norm to the cache and from the last norm to an
answer: the matrix product in 8 bits with a scale for each block of 128, the norms of
queries and keys for each head with the rotation by position (and, in the same pass,
the write into the paged KV cache), and the log probabilities of given tokens with
the entropy and the best alternatives.

``run`` computes a case in plain torch (``own`` false) or through the package
(``own`` true).  Lengths follow from the case alone; values, the order of the pages
and, where rows are free, positions follow from the seed.

Layouts: activations [rows, heads, head_dim]; weights [out, in] as E4M3 codes with
one f32 scale per 128 x 128; the pool of pages [num_pages, kv_heads, page_size,
head_dim] (bf16, f32, or E4M3 codes with one E8M0 scale byte per 32 elements);
page_table [seqs, max_pages] int32, -1 past a sequence's pages; row_offsets
[seqs + 1] int32; kv_len [seqs] int32, the tokens of each sequence with its new ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
E4M3_MAX = 448.0
THETA = 11158840.0
BLOCK = 128


# ----------------------------------------------------------------------------- cases


def listed():
    return [
        # one sequence's token through the output projection of 64 heads of 128: latency
        _linear("linear_one", 1, 4096, 8192),
        # a decode step of 64 sequences through the projection to 64 + 2 x 8 heads of 128
        _linear("linear_decode", 64, 10240, 4096),
        # the logits of those 64 over a vocabulary, left in f32
        _linear("linear_vocabulary", 64, 120832, 4096, out="f32"),
        # a chunk of one prompt, of no round length, back to the hidden size
        _linear("linear_chunk", 1409, 4096, 8192),
        # a prefill batch of the layer through the projection to queries, keys and values
        _linear("linear_prefill", 8192, 10240, 4096),
        # one new token of each of 64 sequences: norms, rotation, into the quantised cache
        _into("rotate_decode", "mxfp8", seqs=64, new=(1, 1), past=(1, 511), page=64),
        # the new tokens of a prefill batch of ragged prompts
        _into("rotate_prefill", "mxfp8", seqs=5, new=(1111, 2171), past=(0, 77), page=64),
        # the same without a cache, f32, part of each head rotated, neighbouring pairs, far positions
        _rotate("rotate_far", "f32", rows=2311, far=1 << 20, heads=32, kv_heads=4, head_dim=128, rotary=64,
                interleaved=True, after=True),
        # one sequence's next token: the chosen one and a few others
        _logprobs("logprobs_one", 1, 120832, "f32", top=5),
        # a decode step of 64 sequences, most of the vocabulary masked by a grammar
        _logprobs("logprobs_decode", 64, 120832, "f32", top=20, masked=0.9),
        # the tokens of prompts, scored
        _logprobs("logprobs_prompt", 4096, 120832, "bf16", top=1),
        # a small vocabulary of odd size: rows of no whole vectors
        _logprobs("logprobs_odd", 2048, 32003, "bf16", top=8),
    ]


def _named(name, c):
    return {"name": name, **c} if name else c


def _linear(name, rows, n, k, act="bf16", out="bf16"):
    return _named(name, {"op": "linear", "rows": rows, "out_features": n, "in_features": k, "act": act, "out": out})


def _heads(heads, kv_heads, head_dim, rotary, interleaved, after):
    return {"heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "rotary": rotary or head_dim,
            "interleaved": interleaved, "after": after}


def _into(name, cache, seqs, new, past, page, heads=64, kv_heads=8, head_dim=128, rotary=0, interleaved=False,
          after=False):
    return _named(name, {"op": "into", "cache": cache, "seqs": seqs, "new_lo": new[0], "new_hi": new[1],
                         "past_lo": past[0], "past_hi": past[1], "page": page,
                         **_heads(heads, kv_heads, head_dim, rotary, interleaved, after)})


def _rotate(name, act, rows, far, heads=64, kv_heads=8, head_dim=128, rotary=0, interleaved=False, after=False):
    return _named(name, {"op": "rotate", "act": act, "rows": rows, "far": far,
                         **_heads(heads, kv_heads, head_dim, rotary, interleaved, after)})


def _logprobs(name, rows, vocab, act, top, masked=0.0):
    return _named(name, {"op": "logprobs", "rows": rows, "vocab": vocab, "act": act, "top": top, "masked": masked})


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "into", "rotate", "logprobs"])
    if op == "linear":
        act = rng.choice(["bf16", "bf16", "bf16", "f32"])
        k = _log(rng, 1, 128) * 128 if rng.random() < 0.6 else _log(rng, 1, 16384)
        n = _log(rng, 1, 32768)
        rows = _log(rng, 1, min(8192, 8192 * 10240 * 4096 // (n * k)))
        return _linear("", rows, n, k, act, rng.choice([act, "f32"]))
    if op == "logprobs":
        vocab = _log(rng, 16, 262144)
        rows = _log(rng, 1, min(8192, 4096 * 120832 // vocab))
        return _logprobs("", rows, vocab, rng.choice(["bf16", "f32"]), min(vocab, rng.choice([0, 1, 5, 20, 64])),
                         rng.choice([0.0, 0.0, 0.5, 0.99]) if vocab >= 4096 else 0.0)
    head_dim, kv_heads = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
    shape = dict(head_dim=head_dim, kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 4, 7, 8]),
                 rotary=rng.choice([head_dim, head_dim, head_dim // 2, 48]), interleaved=rng.random() < 0.3,
                 after=rng.random() < 0.3)
    most = 8192 * 80 * 128 // ((shape["heads"] + 2 * kv_heads) * head_dim)
    if op == "rotate":
        return _rotate("", rng.choice(["bf16", "f32"]), _log(rng, 1, min(16384, most // 2)),
                       rng.choice([1, 5000, 1 << 20]), **shape)
    cache = rng.choice(["bf16", "mxfp8", "mxfp8", "f32"])
    seqs = _log(rng, 1, 64)
    hi = _log(rng, 1, max(1, min(16384, most // 2) // seqs))
    return _into("", cache, seqs, (max(1, hi // rng.choice([1, 2, 7])), hi), (0, rng.choice([0, 50, 333])),
                 rng.choice([1, 8, 16, 64, 256]), **shape)


def _spread(lo, hi, count):
    """count lengths of lo..hi, the longest first and the others spread."""
    return [hi if i == 0 else lo + int((hi - lo) * (i * 0.6180339887 % 1.0)) for i in range(count)]


def _lengths(c):
    """New tokens and whole length of each sequence."""
    new = _spread(c["new_lo"], c["new_hi"], c["seqs"])
    past = _spread(c["past_lo"], c["past_hi"], c["seqs"])
    return new, [n + p for n, p in zip(new, past[1:] + past[:1])]


def _blocks(n):
    return -(-n // BLOCK)


# ----------------------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    {"linear": _prepare_linear, "into": _prepare_into, "rotate": _prepare_rotate,
     "logprobs": _prepare_logprobs}[case["op"]](case, g, s)
    return s


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _prepare_linear(case, g, s):
    rows, n, k = case["rows"], case["out_features"], case["in_features"]
    # channels of different size, as activations have
    s["x"] = _normal(g, rows, k).mul_(_normal(g, k).mul_(0.5).exp_()).to(DTYPES[case["act"]])
    codes = _normal(g, n, k).mul_(120.0).clamp_(-E4M3_MAX, E4M3_MAX)
    s["weight"] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    s["scale"] = (0.5 + torch.rand((_blocks(n), _blocks(k)), generator=g, device="cuda")) * (k ** -0.5 / 120.0)
    if own:
        from mixture_experts_layer_19_amd import block
        s["linear"] = block.BlockLinear(s["weight"], s["scale"], dtype=DTYPES[case["act"]],
                                        out_dtype=DTYPES[case["out"]])


def _prepare_norms(case, g, s, act):
    d = case["head_dim"]
    s["q_weight"], s["k_weight"] = ((1.0 + 0.1 * _normal(g, d)).to(act) for _ in "qk")
    r = case["rotary"]
    s["inv_freq"] = THETA ** (torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / -r)
    if own:
        from mixture_experts_layer_19_amd import block
        s["rope"] = block.HeadNormRope(s["q_weight"], s["k_weight"], inv_freq=s["inv_freq"], eps=EPS,
                                       interleaved=case["interleaved"], norm_after=case["after"])


def _prepare_qkv(case, g, s, act):
    """Slices of one fused projection: the rows are strided."""
    h, kvh = case["heads"], case["kv_heads"]
    fused = _normal(g, s["rows"], h + 2 * kvh, case["head_dim"]).to(act)
    s["q"], s["k"], s["v"] = fused[:, :h], fused[:, h:h + kvh], fused[:, h + kvh:]


def _prepare_rotate(case, g, s):
    act, s["rows"] = DTYPES[case["act"]], case["rows"]
    _prepare_norms(case, g, s, act)
    _prepare_qkv(case, g, s, act)
    s["positions"] = torch.randint(0, case["far"], (s["rows"],), generator=g, device="cuda", dtype=torch.int32)


def _prepare_into(case, g, s):
    new, total = _lengths(case)
    act = DTYPES["f32" if case["cache"] == "f32" else "bf16"]
    pages = [-(-t // case["page"]) for t in total]
    num_pages = sum(pages) + 1
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    width = max(pages) + 1
    at, table, offsets = 0, [], [0]
    for p, n in zip(pages, new):
        table.append(torch.nn.functional.pad(order[at:at + p], (0, width - p), value=-1))
        at += p
        offsets.append(offsets[-1] + n)
    s["table"], s["rows"] = torch.stack(table), offsets[-1]
    s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    _prepare_norms(case, g, s, act)
    _prepare_qkv(case, g, s, act)
    shape = (num_pages, case["kv_heads"], case["page"], case["head_dim"])
    s["pool"] = [_pool(case, shape, act, g) for _ in "kv"]
    if own:
        from mixture_experts_layer_19_amd import block
        (k, ks), (v, vs) = s["pool"]
        s["kv"] = block.PagedKVCache(case["kv_heads"], case["head_dim"], num_pages, case["page"],
                                     dtype=case["cache"], storage=(k, v, ks, vs))
        s["batch"] = block.KVBatch(s["table"], s["offsets"], s["kv_len"], rows=s["rows"], max_rows=max(new))


def _pool(case, shape, act, g):
    """A pool of pages full of earlier tokens: (values or codes, scale bytes or None)."""
    if case["cache"] != "mxfp8":
        return torch.empty(shape, dtype=act, device="cuda").normal_(generator=g), None
    codes = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(0.0, 120.0, generator=g)
    codes = codes.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, torch.randint(119, 122, shape[:-1] + (shape[-1] // 32,), generator=g, device="cuda",
                                dtype=torch.uint8)


def _prepare_logprobs(case, g, s):
    rows, vocab = case["rows"], case["vocab"]
    # rows of different sharpness, from nearly even to one token far ahead
    x = torch.empty((rows, vocab), device="cuda").normal_(generator=g)
    x.mul_(0.5 + 3.5 * torch.rand((rows, 1), generator=g, device="cuda"))
    s["tokens"] = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    ahead = 12.0 * torch.rand((rows, 1), generator=g, device="cuda")
    x.scatter_add_(1, s["tokens"].long().unsqueeze(1), ahead)
    if case["masked"]:
        hide = torch.empty((rows, vocab), device="cuda").uniform_(generator=g) < case["masked"]
        hide.scatter_(1, s["tokens"].long().unsqueeze(1), False)       # the chosen token is an allowed one
        x.masked_fill_(hide, -math.inf)
    s["logits"] = x.to(DTYPES[case["act"]])


# ----------------------------------------------------------------------------- one pass


def run(state):
    op = state["case"]["op"]
    if op == "linear":
        return state["linear"](state["x"]) if own else _plain_linear(state)
    if op == "logprobs":
        if own:
            from mixture_experts_layer_19_amd import block
            r = block.token_logprobs(state["logits"], state["tokens"], top=state["case"]["top"])
            return _logprobs_result(*r)
        return _plain_logprobs(state)
    if op == "rotate":
        if own:
            q, k = state["rope"](state["q"], state["k"], state["positions"])
        else:
            q, k = _plain_rotate(state, state["positions"])
            q, k = q.to(state["q"].dtype), k.to(state["k"].dtype)
        return {"q": q, "k": k}
    q = state["rope"].write(state["kv"], state["batch"], state["q"], state["k"], state["v"]) if own else \
        _plain_into(state)
    return {"q": q, **_pool_values(state)}


def _logprobs_result(logprob, entropy, top_logprob, top_token):
    r = {"logprob": logprob, "entropy": entropy}
    if top_token is not None and top_token.shape[1]:
        r["top_logprob"], r["top_token"] = top_logprob, top_token
    return r


def _pool_values(state):
    """The whole pool after a write, 8-bit codes and scales as the numbers they stand for."""
    (k, ks), (v, vs) = state["pool"]
    if ks is None:
        return {"k": k, "v": v}
    return {"k": k.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn),
            "k_scale": ks.view(torch.float8_e8m0fnu), "v_scale": vs.view(torch.float8_e8m0fnu)}


# ----------------------------------------------------------------------------- plain forms


def _plain_linear(state):
    case, x, w = state["case"], state["x"].float(), state["weight"]
    rows, n, k = case["rows"], case["out_features"], case["in_features"]
    pad = _blocks(k) * BLOCK - k
    b = torch.nn.functional.pad(x, (0, pad)).unflatten(1, (-1, BLOCK))
    scale = b.abs().amax(-1, keepdim=True).div_(E4M3_MAX)
    # the quotient in 64 bits, to whole steps of the code it falls on: a value next to
    # the border of two codes falls on the right side of it
    q = b.double().div_(torch.where(scale > 0, scale, 1.0).double())
    step = torch.ldexp(torch.ones_like(q), torch.frexp(q)[1].clamp_(min=-5) - 4)
    q = q.div_(step).round_().mul_(step).clamp_(-E4M3_MAX, E4M3_MAX).float()
    xd = q.mul_(scale).flatten(1)[:, :k]
    grow = state["scale"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    wd = w.view(torch.float8_e4m3fn).float().mul_(grow)
    return torch.matmul(xd, wd.T).to(DTYPES[case["out"]])


def _plain_rotate(state, positions):
    """f32 q and k with their norms and rotations."""
    case = state["case"]
    r, inter = case["rotary"], case["interleaved"]
    angle = positions.double().unsqueeze(1) * state["inv_freq"]           # far positions: 64 bits
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    out = []
    for x, weight in ((state["q"], state["q_weight"]), (state["k"], state["k_weight"])):
        x, weight = x.float(), weight.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        if not case["after"]:
            x = x * weight
        if inter:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = x[..., :r // 2], x[..., r // 2:r]
            turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        x = torch.cat((turned, x[..., r:]), -1)
        out.append(x * weight if case["after"] else x)
    return out


def _mx_codes(x):
    """E4M3 codes (uint8) and E8M0 bytes of blocks of 32 along the last axis of
    an f32 tensor: X = floor(log2 max) - 8, codes of x / 2^X, saturating."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    exp = torch.frexp(top)[1] - 9
    exp = torch.where(top > 0, exp, -127).clamp_(-127, 127)
    codes = torch.ldexp(b, -exp.unsqueeze(-1)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.flatten(-2).view(torch.uint8), (exp + 127).to(torch.uint8)


def _plain_into(state):
    off, size = state["offsets"].long(), state["case"]["page"]
    row = torch.arange(state["rows"], device="cuda")
    seq = torch.searchsorted(off, row, right=True) - 1
    pos = state["kv_len"].long()[seq] - off[seq + 1] + row
    page, slot = state["table"][seq, pos // size].long(), pos % size
    q, k = _plain_rotate(state, pos)
    for x, (data, scales) in zip((k, state["v"]), state["pool"]):
        if scales is None:
            data[page, :, slot] = x.to(data.dtype)
        else:
            data[page, :, slot], scales[page, :, slot] = _mx_codes(x.float())
    return q.to(state["q"].dtype)


def _plain_logprobs(state):
    x, top = state["logits"].float(), state["case"]["top"]
    chosen = x.gather(1, state["tokens"].long().unsqueeze(1))
    most = x.amax(1, keepdim=True)
    away = x - most
    e = away.exp()
    total = e.sum(1, keepdim=True)
    log_total = total.log()
    entropy = log_total - e.mul_(away.clamp_(min=-1e30)).sum(1, keepdim=True) / total
    del away, e
    values = tokens = None
    if top:
        # one whole number for each value and index: higher values first, then lower indices
        bits = (x + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long().mul_(1 << 32)
        key.add_(torch.arange(x.shape[1] - 1, -1, -1, device="cuda"))
        tokens = x.shape[1] - 1 - (key.topk(top, 1).values & 0xFFFFFFFF)
        values = x.gather(1, tokens) - most - log_total
        tokens = tokens.to(torch.int32)
    return _logprobs_result((chosen - most - log_total).squeeze(1), entropy.squeeze(1), values, tokens)


# ----------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "into": _exact_into, "rotate": _exact_rotate,
            "logprobs": _exact_logprobs}[case["op"]](case, s)


def _exact_e4m3(v):
    """The E4M3 value nearest to each f64 value, ties to even, at most 448."""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    return torch.copysign((torch.round(a / step) * step).clamp(max=E4M3_MAX), v)


def _exact_linear(case, s):
    """Block by block of K: codes of the block, their product, scaled and added."""
    n, x, w = case["out_features"], s["x"], s["weight"].view(torch.float8_e4m3fn)
    y = torch.zeros((case["rows"], n), dtype=torch.float64, device="cuda")
    owner = torch.arange(n, device="cuda") // BLOCK
    for b in range(_blocks(case["in_features"])):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        xb = x[:, at].double()
        most = xb.abs().max(1, keepdim=True).values
        unit = (most.float() / E4M3_MAX).double()          # the scale is an f32
        unit[most == 0] = 1.0
        codes = _exact_e4m3(xb / unit) * unit
        y += codes @ (w[:, at].double() * s["scale"].double()[owner, b:b + 1]).T
    return y


def _exact_turned(case, s, x, weight, positions):
    y = x.double()
    w = weight.double()
    y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["head_dim"] + EPS)
    if not case["after"]:
        y = y * w
    half = case["rotary"] // 2
    i = torch.arange(half, device="cuda")
    lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    angle = torch.outer(positions.double(), s["inv_freq"])[:, None]
    z = torch.polar(torch.ones_like(angle), angle) * torch.complex(y[..., lo], y[..., hi])
    y[..., lo], y[..., hi] = z.real, z.imag
    return y * w if case["after"] else y


def _exact_rotate(case, s):
    return {n: _exact_turned(case, s, s[n], s[n + "_weight"], s["positions"]) for n in "qk"}


def _exact_mx(v):
    """E4M3 values and the power of two of each block of 32 of an f64 tensor."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    top = b.abs().max(-1).values
    power = torch.frexp(top)[1].double() - 9.0
    power[top == 0] = -127.0
    scale = torch.exp2(power.clamp(-127.0, 127.0))
    return _exact_e4m3(b / scale[..., None]).reshape(v.shape), scale


def _exact_into(case, s):
    new, total = _lengths(case)
    pos = torch.cat([torch.arange(t - n, t, device="cuda") for n, t in zip(new, total)])
    out = {"q": _exact_turned(case, s, s["q"], s["q_weight"], pos)}
    sides = {"k": _exact_turned(case, s, s["k"], s["k_weight"], pos), "v": s["v"].double()}
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device="cuda"), torch.tensor(new, device="cuda"))
    place = s["table"].long()[seq, pos // case["page"]] * case["page"] + pos % case["page"]
    for (name, x), (data, scales) in zip(sides.items(), s["pool"]):
        value = (data if scales is None else data.view(torch.float8_e4m3fn)).double()
        flat = value.transpose(1, 2).reshape(-1, case["kv_heads"], case["head_dim"])
        like = value.transpose(1, 2).shape
        if scales is None:
            flat[place] = x
        else:
            power = torch.exp2(scales.double() - 127.0).transpose(1, 2)
            rows = power.reshape(-1, case["kv_heads"], case["head_dim"] // 32)
            flat[place], rows[place] = _exact_mx(x)
            out[name + "_scale"] = rows.reshape(power.shape).transpose(1, 2).contiguous()
        out[name] = flat.reshape(like).transpose(1, 2).contiguous()
    return out


def _exact_logprobs(case, s):
    parts = []
    for x, token in zip(s["logits"].split(256), s["tokens"].split(256)):
        x = x.double()
        lp = x - torch.logsumexp(x, 1, keepdim=True)
        p = lp.exp()
        part = {"logprob": lp[torch.arange(len(x), device="cuda"), token.long()],
                "entropy": -torch.where(p > 0, p * lp, 0.0).sum(1)}
        if case["top"]:
            part["top_token"] = x.sort(dim=1, descending=True, stable=True).indices[:, :case["top"]].to(torch.int32)
            part["top_logprob"] = lp.gather(1, part["top_token"].long())
        parts.append(part)
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}


# ----------------------------------------------------------------------------- work


def work(case):
    if case["op"] == "linear":
        rows, n, k = case["rows"], case["out_features"], case["in_features"]
        size = {"bf16": 2, "f32": 4}
        return {"bytes": rows * k * size[case["act"]] + n * k + 4 * _blocks(n) * _blocks(k)
                + rows * n * size[case["out"]], "flops": 2 * rows * n * k}
    if case["op"] == "logprobs":
        size = 2 if case["act"] == "bf16" else 4
        return {"bytes": case["rows"] * (case["vocab"] * size + 4 + 8 + 8 * case["top"]), "flops": 0}
    d, kvh = case["head_dim"], case["kv_heads"]
    if case["op"] == "rotate":
        size = 2 if case["act"] == "bf16" else 4
        return {"bytes": case["rows"] * (2 * (case["heads"] + kvh) * d * size + 4), "flops": 0}
    size = 4 if case["cache"] == "f32" else 2
    kept = d + d // 32 if case["cache"] == "mxfp8" else d * size
    return {"bytes": sum(_lengths(case)[0]) * ((2 * case["heads"] + 2 * kvh) * d * size + 2 * kvh * kept), "flops": 0}
