"""The operators around the QKV projection of a 4-bit layer, as calls to be timed and compared.

Four operators serve attention over a paged cache whose keys and values are held
in the 4-bit formats of the linear layer (NVFP4: E2M1 codes, an E4M3 scale per
16 values; FP4 g32: a scale per 32; INT4: codes in [-7, 7], an fp16 scale per 64):

  plan       cu_q, positions, slots, total lengths and new block-table entries of
             a batch, from its request lengths and a list of free pages;
  norm_rope  RMS norm of each query and key head and the position rotation, in
             one pass over the QKV projection's output rows;
  append     quantize keys and values into their cache slots, and read the same
             slots back as the values that the codes stand for;
  attention  softmax(scale q k^T) v over the cache, with lse.

`run` computes them in elementary torch operations (own = False) or through the
package's entry points (own = True), on the same inputs.
"""
import math
import random

import torch

own = False

GROUP = {"nvfp4": 16, "fp4g32": 32, "int4": 64}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases ---
def listed():
    heads = {"heads": 32, "kv_heads": 8, "dim": 128}
    return [
        # one decode step of a small serving batch: a single launch's latency
        {"name": "plan_decode_64", "op": "plan", "batch": 64, "q": 1, "kv": 4000, "page": 64, "pad": 0},
        # a large batch of ragged prompts, padded to a captured graph's row count
        {"name": "plan_mixed_1000", "op": "plan", "batch": 1000, "q": 61, "kv": 2047, "page": 16, "pad": 517},
        # one decode step of 16 requests
        {"name": "norm_rope_decode_16", "op": "norm_rope", "rows": 16, **heads, "rot": 128, "interleaved": False,
         "positions": 131072},
        # a long prompt with a rotation over half of each head
        {"name": "norm_rope_prefill_16383", "op": "norm_rope", "rows": 16383, **heads, "rot": 64,
         "interleaved": False, "positions": 32768},
        # the image and text tokens of the attention layer that the QKV projection feeds, interleaved pairs
        {"name": "norm_rope_image_4608", "op": "norm_rope", "rows": 4608, "heads": 24, "kv_heads": 24, "dim": 128,
         "rot": 128, "interleaved": True, "positions": 4608},
        # one decode step's keys and values of 64 requests
        {"name": "append_decode_64", "op": "append", "rows": 64, "fmt": "nvfp4", "kv_heads": 8, "dim": 128, "page": 64,
         "pages": 512},
        # a prompt's keys and values
        {"name": "append_prefill_8191", "op": "append", "rows": 8191, "fmt": "int4", "kv_heads": 8, "dim": 128,
         "page": 16, "pages": 1024},
        # one request, one new token, a short cache: the latency of a decode step
        {"name": "decode_1x1000", "op": "attention", "fmt": "nvfp4", "batch": 1, "q": 1, "kv": 1000, "ragged": False,
         **heads, "page": 16, "causal": True, "window": 0},
        # a serving batch of ragged lengths, one new token each
        {"name": "decode_64x8192", "op": "attention", "fmt": "nvfp4", "batch": 64, "q": 1, "kv": 8192, "ragged": True,
         **heads, "page": 64, "causal": True, "window": 0},
        # a few requests over very long caches: work split along the cache
        {"name": "decode_3x131000", "op": "attention", "fmt": "int4", "batch": 3, "q": 1, "kv": 131000,
         "ragged": False, **heads, "page": 128, "causal": True, "window": 0},
        # chunks of prompts over what is already cached
        {"name": "prefill_3x1500_on_6000", "op": "attention", "fmt": "fp4g32", "batch": 3, "q": 1500, "kv": 6000,
         "ragged": True, **heads, "page": 64, "causal": True, "window": 0},
        # every token of an image and its text attends to every token
        {"name": "image_4608", "op": "attention", "fmt": "nvfp4", "batch": 1, "q": 4608, "kv": 4608, "ragged": False,
         "heads": 24, "kv_heads": 24, "dim": 128, "page": 128, "causal": False, "window": 0},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["plan", "norm_rope", "append", "attention", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["nvfp4", "fp4g32", "int4"])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
    if op == "plan":
        return {"op": op, "batch": _log(rng, 1, 1000), "q": _log(rng, 1, 60), "kv": _log(rng, 1, 4000), "page": page,
                "pad": rng.choice([0, rng.randrange(300)])}
    if op == "norm_rope":
        return {"op": op, "rows": _log(rng, 1, 16000), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2]), "interleaved": rng.random() < 0.5,
                "positions": _log(rng, 16, 131072)}
    if op == "append":
        rows = _log(rng, 1, 8000)
        return {"op": op, "rows": rows, "fmt": fmt, "kv_heads": kv_heads, "dim": dim, "page": page,
                "pages": rows // page + 1 + rng.randrange(200)}
    case = {"op": op, "fmt": fmt, "batch": 1, "q": 1, "kv": 1, "ragged": rng.random() < 0.7, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "causal": rng.random() < 0.7, "window": 0}
    if rng.random() < 0.5:    # decode: one to four new tokens
        case["q"] = rng.choice([1, 1, 2, 4])
        case["batch"] = _log(rng, 1, 64)
        case["kv"] = _log(rng, 4, min(100000, 400000 // case["batch"]))
    else:                     # prompts and chunks of prompts
        case["batch"] = _log(rng, 1, 6)
        case["q"] = _log(rng, 5, 3000 // case["batch"])
        case["kv"] = case["q"] + _log(rng, 1, 4000)
    if case["causal"] and rng.random() < 0.3:
        case["window"] = _log(rng, 4, 4000)
    return case


def _lengths(case):
    """(new tokens, all tokens) of each request: a property of the case, not of the seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    got = []
    for _ in range(case["batch"]):
        q, kv = case["q"], case["kv"]
        if case["op"] == "plan":
            got.append((rng.randint(0 if q > 1 else 1, q), rng.randint(0, kv)))
            continue
        if case["ragged"]:
            q = rng.randint((q + 1) // 2, q)
            kv = rng.randint(max(q, kv // 4), max(q, kv))
        got.append((q, max(q, kv)))
    return got


def _token_bytes(fmt, dim):
    """Cache bytes of one head's key (or value) of one token: codes and scales."""
    return dim // 2 + dim // GROUP[fmt] * (2 if fmt == "int4" else 1)


def _pairs(case):
    """Query-key pairs of one head that the masks leave, over all requests."""
    total = 0
    for q, kv in _lengths(case):
        for i in range(q):
            last = kv - q + i + 1 if case["causal"] else kv
            total += min(last, case["window"]) if case["window"] else last
    return total


def work(case):
    if case["op"] == "plan":
        lens, page = _lengths(case), case["page"]
        rows = sum(q for q, _ in lens) + case["pad"]
        new = sum(-(-(q + kv) // page) - -(-kv // page) for q, kv in lens)
        # lengths in and out, cu_q, positions and slots, each new page read and entered
        return {"bytes": 16 * case["batch"] + 12 * rows + 8 * new, "flops": 0}
    if case["op"] == "norm_rope":
        n = case["rows"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        table = min(case["rows"], case["positions"]) * case["rot"] * 4
        return {"bytes": 4 * n + table + 4 * case["rows"], "flops": 8 * n}
    if case["op"] == "append":
        n = case["rows"] * case["kv_heads"] * 2
        out = 4 if case["fmt"] == "int4" else 2
        return {"bytes": n * ((2 + out) * case["dim"] + 2 * _token_bytes(case["fmt"], case["dim"])) + 8 * case["rows"],
                "flops": 6 * n * case["dim"]}
    rows = sum(q for q, _ in _lengths(case))
    keys = sum(min(kv, q + case["window"] - 1) if case["window"] else kv for q, kv in _lengths(case))
    cache = keys * case["kv_heads"] * 2 * _token_bytes(case["fmt"], case["dim"])
    return {"bytes": cache + rows * case["heads"] * (4 * case["dim"] + 4) + 4 * keys // case["page"],
            "flops": 4 * case["dim"] * case["heads"] * _pairs(case)}


# ------------------------------------------------------------ plain helpers ---
def _quantize(x, fmt):
    """(codes 0..15 as uint8, scales) of bf16 x along its last axis: the linear layer's
    quantizer, scale = rounded amax / q_max, code = rounded x * RN(1 / scale) in fp32."""
    g = GROUP[fmt]
    v = x.float().unflatten(-1, (-1, g))
    amax = v.abs().amax(-1)
    if fmt == "int4":
        scale = (amax / 7.0).clamp(max=65504.0).to(torch.float16)
    else:
        scale = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()
    r = v * torch.where(s > 0, 1.0 / s, torch.zeros_like(s)).unsqueeze(-1)
    if fmt == "int4":
        code = r.round_().clamp_(-7, 7).to(torch.int8).view(torch.uint8) & 15
    else:
        a = r.abs()
        # midpoints of the E2M1 grid, ties to the even code
        code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
                + (a > 5.0))
        code |= ((r < 0) & (code > 0)).to(torch.uint8) << 3
    return code.flatten(-2), scale


def _pack(code):
    """Two codes a byte, element 2i in the low nibble."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _parts(case):
    """Byte ranges of a (page, head) block of the pool: key codes, key scales, value codes, value scales."""
    page, dim = case["page"], case["dim"]
    c, s = page * dim // 2, page * (_token_bytes(case["fmt"], dim) - dim // 2)
    return (0, c, c + s, 2 * c + s, 2 * c + 2 * s)


def _store(pool, case, which, slots, code, scale):
    """Write packed codes and scales [rows, heads, ...] at the slots of keys (0) or values (1)."""
    at, page = _parts(case), case["page"]
    p, o = slots // page, slots % page
    heads = pool.shape[1]
    pool[:, :, at[2 * which]:at[2 * which + 1]].unflatten(-1, (page, -1))[p, :, o] = _pack(code)
    pool[:, :, at[2 * which + 1]:at[2 * which + 2]].unflatten(-1, (page, -1))[p, :, o] = \
        scale.contiguous().view(torch.uint8).reshape(scale.shape[0], heads, -1)


def _load(pool, case, which, slots):
    """The values at the slots (any shape), as fp32 [*slots.shape, heads, dim]."""
    at, page, fmt = _parts(case), case["page"], case["fmt"]
    p, o = slots // page, slots % page
    code = pool[:, :, at[2 * which]:at[2 * which + 1]].unflatten(-1, (page, -1)).transpose(1, 2)[p, o]
    scale = pool[:, :, at[2 * which + 1]:at[2 * which + 2]].unflatten(-1, (page, -1)).transpose(1, 2)[p, o]
    if fmt == "int4":
        table = torch.tensor([i if i < 8 else i - 16 for i in range(16)], device=pool.device, dtype=torch.float32)
        s = scale.contiguous().view(torch.float16).float()
    else:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=pool.device, dtype=torch.float32)
        s = scale.contiguous().view(torch.float8_e4m3fn).float()
    v = torch.stack((table[(code & 15).int()], table[(code >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, GROUP[fmt])) * s.unsqueeze(-1)).flatten(-2)


def _outliers(x, g):
    """Scale one channel in 32 up, as keys and values of trained models have them."""
    dim = x.shape[-1]
    x[..., torch.randperm(dim, generator=g, device=x.device)[:dim // 32]] *= 8.0
    return x


def _rotation(positions, rot):
    """cos and sin of position * 10000^(-2i / rot), angles in 64 bits: [positions, rot] fp32."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / rot)
    return torch.cat((angle.cos(), angle.sin()), -1).float()


# ----------------------------------------------------------------- prepare ---
def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dev = torch.device("cuda", torch.cuda.current_device())
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    bf16 = dict(dtype=torch.bfloat16, device=dev)
    s = {"case": dict(case)}
    if case["op"] == "plan":
        lens, page = _lengths(case), case["page"]
        held = [-(-kv // page) for _, kv in lens]
        need = [-(-(q + kv) // page) for q, kv in lens]
        pages = torch.randperm(sum(need) + 7, generator=g, device=dev).to(torch.int32)
        width = max(need) + 3
        column = torch.arange(width, device=dev)
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device=dev)
        table[column[None, :] < ints(held)[:, None]] = pages[:sum(held)]
        s.update(rows=sum(q for q, _ in lens) + case["pad"], q_lens=ints([q for q, _ in lens]),
                 kv_lens=ints([kv for _, kv in lens]), table=table, free=pages[sum(held):].clone(),
                 pages=sum(need) + 7)
        return s
    if case["op"] == "norm_rope":
        hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
        qkv = torch.randn(case["rows"], (hq + 2 * hk) * d, generator=g, **bf16)
        s["q"] = qkv[:, :hq * d].unflatten(-1, (hq, d))     # rows of the projection's output, as it leaves them
        s["k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
        s["q_weight"] = 1 + 0.2 * torch.randn(d, generator=g, **bf16)
        s["k_weight"] = 1 + 0.2 * torch.randn(d, generator=g, **bf16)
        s["table"] = _rotation(case["positions"], case["rot"])
        s["positions"] = torch.randint(0, case["positions"], (case["rows"],), generator=g, device=dev,
                                       dtype=torch.int32)
        return s
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    block = _parts(case)[-1]
    if case["op"] == "append":
        rows = case["rows"]
        s["pool"] = torch.randint(0, 256, (case["pages"], hk, block), generator=g, device=dev, dtype=torch.uint8)
        s["k"] = _outliers(torch.randn(rows, hk, d, generator=g, **bf16), g)
        s["v"] = torch.randn(rows, 3 * hk, d, generator=g, **bf16)[:, 2 * hk:]
        s["slots"] = torch.randperm(case["pages"] * page, generator=g, device=dev)[:rows].clone()
        return s
    lens = _lengths(case)
    need = [-(-kv // page) for _, kv in lens]
    pages = torch.randperm(sum(need) + 5, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device=dev)
    table[torch.arange(max(need) + 1, device=dev)[None, :] < ints(need)[:, None]] = pages[:sum(need)]
    # what other requests left in the pages stays there: any bytes
    pool = torch.randint(0, 256, (sum(need) + 5, hk, block), generator=g, device=dev, dtype=torch.uint8)
    for b, (_, kv) in enumerate(lens):
        t = torch.arange(kv, device=dev)
        slots = table[b, t // page].long() * page + t % page
        for which in (0, 1):
            x = torch.randn(kv, hk, d, generator=g, **bf16)
            _store(pool, case, which, slots, *_quantize(_outliers(x, g) if which == 0 else x, case["fmt"]))
    q = torch.randn(sum(q for q, _ in lens), case["heads"], d, generator=g, **bf16)
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    s.update(pool=pool, table=table, q=q, cu_q=ints(cu), kv_lens=ints([kv for _, kv in lens]),
             max_q=max(n for n, _ in lens), max_kv=max(kv for _, kv in lens), scale=d ** -0.5)
    return s


# --------------------------------------------------------------- plain forms ---
def _plan(s):
    page, rows, dev = s["case"]["page"], s["rows"], s["table"].device
    q, kv, table = s["q_lens"].long(), s["kv_lens"].long(), s["table"]
    total = q + kv
    cu = torch.cat((q.new_zeros(1), q.cumsum(0)))
    held, need = (kv + page - 1) // page, (total + page - 1) // page
    first = torch.cumsum(need - held, 0) - (need - held)      # the request's first page of the free list
    column = torch.arange(table.shape[1], device=dev)[None, :]
    new = (column >= held[:, None]) & (column < need[:, None])
    index = (first[:, None] + column - held[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(new, s["free"][index], table))
    t = torch.arange(rows, device=dev)
    request = torch.searchsorted(cu[1:], t, right=True).clamp(max=q.numel() - 1)
    live = t < cu[-1]
    position = torch.where(live, kv[request] + t - cu[request], torch.full_like(t, -1))
    at = position.clamp(min=0)
    slot = torch.where(live, table[request, at // page].long() * page + at % page, torch.full_like(t, -1))
    return {"cu_q": cu.int(), "kv_lens": total.int(), "positions": position.int(), "slots": slot,
            "used": (need - held).sum().int().reshape(1), "table": table}


def _norm_rope(x, weight, rotation, interleaved):
    v = x.float()
    v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    half = rotation.shape[-1] // 2
    cos, sin = rotation[:, None, :half], rotation[:, None, half:]
    if interleaved:
        a, b = v[..., 0:2 * half:2], v[..., 1:2 * half:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = v[..., :half], v[..., half:2 * half]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, v[..., 2 * half:]), -1).to(x.dtype)


def _attention(s):
    case, pool, dev = s["case"], s["pool"], s["pool"].device
    page, hk, rep = case["page"], case["kv_heads"], case["heads"] // case["kv_heads"]
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    n = cu[1:] - cu[:-1]
    t, i = torch.arange(s["max_kv"], device=dev), torch.arange(s["max_q"], device=dev)
    live = t[None, :] < kv[:, None]
    slots = torch.where(live, s["table"][:, t // page].long() * page + t % page, torch.zeros_like(live, dtype=torch.long))
    alive = live[:, :, None, None]
    k = torch.where(alive, _load(pool, case, 0, slots), torch.zeros((), device=dev))     # [batch, keys, heads, dim]
    v = torch.where(alive, _load(pool, case, 1, slots), torch.zeros((), device=dev))
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().unflatten(2, (hk, rep))           # [batch, queries, kv heads, rep, dim]
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                # [batch, kv heads, rep * queries, dim]
    score = (q @ k.permute(0, 2, 3, 1)).unflatten(2, (rep, -1)) * s["scale"]
    at = kv[:, None] - n[:, None] + i                         # each query's position
    seen = live[:, None, :].expand(-1, i.numel(), -1)
    if case["causal"]:
        seen = seen & (t <= at[:, :, None])
    if case["window"]:
        seen = seen & (t > at[:, :, None] - case["window"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = score.sum(-1, keepdim=True)
    out = score.flatten(2, 3) @ v.transpose(1, 2)
    out = out.unflatten(2, (rep, -1)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)
    used = i[None, :] < n[:, None]
    return {"out": out[used].to(s["q"].dtype), "lse": lse[used]}


def run(state):
    s, case = state, state["case"]
    if case["op"] == "plan":
        if own:
            import w4a4_gemm_b200 as svdq
            cu_q, kv_lens, positions, slots, used = svdq.svdq_kv_plan(
                s["q_lens"], s["kv_lens"], s["table"], s["free"], s["rows"], case["page"])
            return {"cu_q": cu_q, "kv_lens": kv_lens, "positions": positions, "slots": slots, "used": used,
                    "table": s["table"]}
        return _plan(s)
    if case["op"] == "norm_rope":
        if own:
            import w4a4_gemm_b200 as svdq
            q, k = svdq.svdq_qk_norm_rope(s["q"], s["k"], s["table"], s["positions"], s["q_weight"], s["k_weight"],
                                          eps=1e-6, interleaved=case["interleaved"])
            return {"q": q, "k": k}
        rotation = s["table"][s["positions"].long()]
        return {"q": _norm_rope(s["q"], s["q_weight"], rotation, case["interleaved"]),
                "k": _norm_rope(s["k"], s["k_weight"], rotation, case["interleaved"])}
    if own:
        import w4a4_gemm_b200 as svdq
        cache = svdq.KVCache(case["fmt"], case["kv_heads"], case["dim"], case["page"], s["pool"])
    if case["op"] == "append":
        kind = torch.float32 if case["fmt"] == "int4" else torch.bfloat16      # the values are exact in it
        if own:
            svdq.svdq_kv_append(cache, s["k"], s["v"], s["slots"])
            k, v = svdq.svdq_kv_read(cache, s["slots"], kind)
            return {"k": k, "v": v}
        _store(s["pool"], case, 0, s["slots"], *_quantize(s["k"], case["fmt"]))
        _store(s["pool"], case, 1, s["slots"], *_quantize(s["v"], case["fmt"]))
        return {"k": _load(s["pool"], case, 0, s["slots"]).to(kind), "v": _load(s["pool"], case, 1, s["slots"]).to(kind)}
    if own:
        out, lse = svdq.svdq_kv_attention(cache, s["q"], s["cu_q"], s["kv_lens"], s["table"], scale=s["scale"],
                                          causal=case["causal"], window=case["window"], return_lse=True)
        return {"out": out, "lse": lse}
    return _attention(s)


# ------------------------------------------------------------------- exact ---
def _exact_values(x, fmt):
    """What the codes of x stand for, in 64 bits, by the quantizer's definition: two roundings
    to fp32 are part of it (1 / scale and the product), the others are to the grid itself."""
    g = {"nvfp4": 16, "fp4g32": 32, "int4": 64}[fmt]
    v = x.double().reshape(*x.shape[:-1], x.shape[-1] // g, g)
    top = v.abs().max(-1).values
    if fmt == "int4":
        scale = (top / 7).float().clamp(max=65504).half().double()
    else:
        raw = (top / 6).float().double()
        step = torch.exp2(torch.floor(torch.log2(raw.clamp(min=2.0 ** -6))) - 3)   # E4M3: 3 bits, subnormal below 2^-6
        scale = (torch.round(raw / step) * step).clamp(max=448)
    inverse = torch.where(scale > 0, 1 / scale, 0.0).float().double()
    r = (v * inverse[..., None]).float().double()
    if fmt == "int4":
        value = torch.round(r).clamp(-7, 7)
    else:
        a = r.abs().clamp(max=6)
        step = torch.where(a >= 4, 2.0, torch.where(a >= 2, 1.0, 0.5)).double()    # E2M1: 1 bit below the leading one
        value = torch.round(a / step) * step * torch.sign(r)
    return (value * scale[..., None]).reshape(x.shape)


def _exact_read(pool, case, which, slots):
    """Values of a list of slots from the pool's bytes, in 64 bits: [slots, heads, dim]."""
    page, dim, fmt = case["page"], case["dim"], case["fmt"]
    g = {"nvfp4": 16, "fp4g32": 32, "int4": 64}[fmt]
    width = dim // g * (2 if fmt == "int4" else 1)
    half = page * (dim // 2 + width)
    start = which * half
    flat = pool.reshape(-1)
    heads, block = pool.shape[1], pool.shape[2]
    base = ((slots // page)[:, None] * heads + torch.arange(heads, device=pool.device)) * block + start
    off = (slots % page)[:, None]
    byte = flat[(base + off * (dim // 2))[..., None] + torch.arange(dim // 2, device=pool.device)].int()
    nib = torch.stack((byte % 16, byte // 16), -1).reshape(*byte.shape[:-1], dim)
    raw = flat[(base + page * (dim // 2) + off * width)[..., None] + torch.arange(width, device=pool.device)].int()
    if fmt == "int4":
        value = torch.where(nib < 8, nib, nib - 16).double()
        bits = raw[..., 0::2] + 256 * raw[..., 1::2]
        e, m = bits // 1024, (bits % 1024).double()
        scale = torch.where(e > 0, (1 + m / 1024) * torch.exp2((e - 15).double()), m * 2.0 ** -24)
    else:
        e, m = nib % 8 // 2, (nib % 2).double()
        value = torch.where(e > 0, (1 + m / 2) * torch.exp2((e - 1).double()), m / 2)
        value = torch.where(nib >= 8, -value, value)
        e, m = raw // 8, (raw % 8).double()
        scale = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m * 2.0 ** -9)
    return (value.reshape(*value.shape[:-1], dim // g, g) * scale[..., None]).reshape(value.shape)


def exact(case, seed):
    if case["op"] == "plan":
        return None                                    # whole numbers: the plain form's own
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        got = {}
        angle = torch.zeros(case["rows"], case["dim"] // 2, 2, dtype=torch.float64, device=s["q"].device)
        half = case["rot"] // 2
        row = s["table"][s["positions"].long()].double()
        angle[..., 0] = 1.0                            # pairs behind the rotated ones turn by nothing
        angle[:, :half, 0], angle[:, :half, 1] = row[:, :half], row[:, half:]
        turn = torch.view_as_complex(angle)[:, None]
        order = torch.arange(case["dim"], device=s["q"].device)
        if not case["interleaved"]:                    # bring each pair together, turn it, and put it back
            order = torch.cat((torch.stack((order[:half], order[half:2 * half]), -1).reshape(-1), order[2 * half:]))
        for name in ("q", "k"):
            x = s[name].double()
            x = x / (x.pow(2).sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt() * s[name + "_weight"].double()
            z = torch.view_as_complex(x[..., order].reshape(*x.shape[:2], -1, 2).contiguous()) * turn
            got[name] = torch.empty_like(x)
            got[name][..., order] = torch.view_as_real(z).flatten(-2)
        return got
    if case["op"] == "append":
        return {"k": _exact_values(s["k"], case["fmt"]), "v": _exact_values(s["v"], case["fmt"])}
    if 4 * case["dim"] * case["heads"] * _pairs(case) > 6e12:
        return None
    outs, lses, first, rep = [], [], 0, case["heads"] // case["kv_heads"]
    for b, (n, kv) in enumerate(_lengths(case)):
        t = torch.arange(kv, device=s["q"].device)
        slots = s["table"][b, t // case["page"]].long() * case["page"] + t % case["page"]
        k, v = (_exact_read(s["pool"], case, w, slots) for w in (0, 1))
        at = (kv - n + torch.arange(n, device=t.device))[:, None]
        hidden = torch.zeros(n, kv, dtype=torch.bool, device=t.device)
        if case["causal"]:
            hidden |= t > at
        if case["window"]:
            hidden |= t <= at - case["window"]
        out = torch.zeros(n, case["heads"], case["dim"], dtype=torch.float64, device=t.device)
        lse = torch.zeros(n, case["heads"], dtype=torch.float64, device=t.device)
        for h in range(case["heads"]):
            w = s["q"][first:first + n, h].double() @ k[:, h // rep].T * s["scale"]
            w = w.masked_fill(hidden, -math.inf)
            lse[:, h] = torch.logsumexp(w, -1)
            out[:, h] = torch.softmax(w, -1) @ v[:, h // rep]
        outs.append(out)
        lses.append(lse)
        first += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
