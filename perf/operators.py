"""The workloads on which the balance loss, the 4-bit matrix-vector products and the block-quantized
paged cache are timed: their inputs, a plain torch form, the library's calls and a float64 form.

With `own` false, run() computes an operator in elementary torch operations in 32 bits; with `own` true
it makes the calls a program that uses the library makes.  Both take what prepare() returns.
"""

import math

import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16, "mxfp8": 32}


# ------------------------------------------------------------------------------------------------
# Cases.


def listed():
    return [
        # training: the router of a 4-expert layer on 16 tokens; launches and the autograd engine are what counts
        dict(name="balance_tiny", op="balance", T=16, E=4, k=2, masked=False),
        # training: one step's tokens over 128 experts, top-8
        dict(name="balance_step", op="balance", T=8192, E=128, k=8, masked=False),
        # training: a long padded batch (odd token count) over 384 experts
        dict(name="balance_padded", op="balance", T=65533, E=384, k=8, masked=True),
        # serving one token through a small projection: latency
        dict(name="matvec_small", op="matvec", fmt="mxfp4", M=1, N=256, K=256, bias=True),
        # serving one token through a large projection with 16-element groups: weight bandwidth
        dict(name="matvec_token", op="matvec", fmt="nvfp4", M=1, N=7168, K=7168, bias=False),
        # a small batch of tokens through a projection that widens
        dict(name="matvec_batch", op="matvec", fmt="mxfp4", M=16, N=7168, K=2048, bias=False),
        # sizes that fill no tile: odd outputs, a half-filled last group of columns, more rows than one tile
        dict(name="matvec_odd", op="matvec", fmt="nvfp4", M=21, N=4099, K=2032, bias=True),
        # one token's eight experts, first product with its SwiGLU
        dict(name="expert_token", op="expert", fmt="mxfp4", T=1, E=128, k=8, N=1536, K=2048, swiglu=True, bias=False),
        # a decode batch: nearly every expert is touched; second product, one input row per pair
        dict(name="expert_batch", op="expert", fmt="nvfp4", T=64, E=128, k=8, N=2048, K=768, swiglu=False, bias=True),
        # one short conversation, one new token: latency
        dict(name="cache_token", op="cache", fmt="mxfp4", B=1, new=1, context=77, heads=2, k_dim=64, v_dim=64, page=16),
        # a decode step of a batch with ragged contexts: one new token each, the contexts read back for attention
        dict(name="cache_decode", op="cache", fmt="mxfp8", B=32, new=1, context=3900, heads=8, k_dim=128, v_dim=128, page=64),
        # a prefill: every token of the batch is written, then read back; pages end inside it
        dict(name="cache_prefill", op="cache", fmt="nvfp4", B=5, new=5000, context=0, heads=8, k_dim=192, v_dim=128, page=24),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "matvec", "expert", "cache"])
    fmt = rng.choice(["mxfp4", "nvfp4"])
    b = BLOCK[fmt]
    if op == "balance":
        E = _log_int(rng, 2, 1024)
        T = _log_int(rng, 1, min(65536, (65536 * 384) // E))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), masked=rng.random() < 0.5)
    if op == "matvec":
        K = b * _log_int(rng, 2, 16384 // b)
        N = _log_int(rng, 16, min(16384, (7168 * 7168) // K))
        return dict(op=op, fmt=fmt, M=_log_int(rng, 1, 32), N=N, K=K, bias=rng.random() < 0.5)
    if op == "expert":
        E = _log_int(rng, 2, 128)
        K = b * _log_int(rng, 2, 4096 // b)
        N = 2 * _log_int(rng, 8, min(2048, (128 * 1536 * 2048) // (2 * E * K)))
        T = _log_int(rng, 1, 64)
        return dict(op=op, fmt=fmt, T=T, E=E, k=rng.randint(1, min(8, E)), N=N, K=K, swiglu=rng.random() < 0.5,
                    bias=rng.random() < 0.5)
    fmt = rng.choice(["mxfp4", "nvfp4", "mxfp8"])
    b = BLOCK[fmt]
    heads = _log_int(rng, 1, 16)
    k_dim, v_dim = b * rng.randint(1, 256 // b), b * rng.randint(1, 256 // b)
    rows = min(65536, 100_000_000 // (heads * (k_dim + v_dim)))  # tokens in the cache, about
    B = _log_int(rng, 1, 64)
    context = _log_int(rng, 1, max(1, rows // B))
    new = rng.choice([1, rng.randint(1, context)])
    return dict(op=op, fmt=fmt, B=B, new=new, context=context - new if context > new else 0, heads=heads, k_dim=k_dim,
                v_dim=v_dim, page=rng.choice([1, 16, 24, 32, 64, 128]))


def _lengths(case):
    """(tokens in the cache before, new tokens) of each sequence: ragged, the same for every seed."""
    have = [case["context"] - (7919 * i) % (case["context"] // 2 + 1) for i in range(case["B"])]
    new = [case["new"] - (104729 * i) % (case["new"] // 2 + 1) for i in range(case["B"])]
    return have, new


def work(case):
    op = case["op"]
    if op == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        # the logits are needed whole on both sides of the loss; the gradient is written once
        return {"bytes": 3 * T * E * 4 + T * k * 4 + E * 4 + (2 * T if case["masked"] else 0), "flops": 14 * T * E}
    if op == "cache":
        have, new = _lengths(case)
        width = case["heads"] * (case["k_dim"] + case["v_dim"])
        held = width * (1.0 if case["fmt"] == "mxfp8" else 0.5) + width // BLOCK[case["fmt"]]
        total = sum(have) + sum(new)
        return {"bytes": sum(new) * (2 * width + held) + total * (held + 2 * width), "flops": 2 * width * (total + sum(new))}
    N, K = case["N"], case["K"]
    per_matrix = N * K / 2 + N * K / BLOCK[case["fmt"]] + (2 * N if case["bias"] else 0)
    if op == "matvec":
        M = case["M"]
        return {"bytes": per_matrix + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    touched = E * (1 - (1 - k / E) ** T)  # expected over the routings
    rows, out = (T, N // 2) if case["swiglu"] else (T * k, N)
    return {"bytes": touched * per_matrix + 2 * rows * K + 2 * T * k * out + 4 * T * k + 4 * E, "flops": 2 * T * k * N * K}


# ------------------------------------------------------------------------------------------------
# The block formats in 32 bits.


def _e2m1_code(v):
    """Codes of the magnitudes v: the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    c = (v > 0.25).to(torch.uint8)
    for edge, closed in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (v >= edge) if closed else (v > edge)
    return c


def _power(e):
    """2^e as float32, -126 <= e <= 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _encode(x, fmt, gs=1.0):
    """x float32 [..., D] holding bf16 values -> (codes uint8, two to a byte in the 4-bit formats; scale bytes)."""
    b = BLOCK[fmt]
    v = x.reshape(*x.shape[:-1], -1, b)
    mag = v.abs()
    top = mag.amax(-1, keepdim=True)
    if fmt == "nvfp4":
        r6 = torch.tensor(1.0 / 6.0, dtype=torch.float32, device=x.device)
        s8 = (gs * (top * r6)).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = s8.float()
        ratio = torch.where(s > 0, gs / s, torch.zeros_like(s))
        code = _e2m1_code(mag * ratio)
        scale = s8.view(torch.uint8)
    else:
        biased = (top.contiguous().view(torch.int32) + (1 << 21)) >> 23
        e = (biased - (8 if fmt == "mxfp8" else 2)).clamp(0, 254)
        e = torch.where(top > 0, e, torch.zeros_like(e))
        scaled = v * _power(127 - e)
        scale = e.to(torch.uint8)
        if fmt == "mxfp8":
            return scaled.to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape), scale.squeeze(-1)
        code = _e2m1_code(scaled.abs())
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.squeeze(-1)


def _decode(q, s, fmt):
    """Values in float32, without the global scale."""
    b = BLOCK[fmt]
    if fmt == "mxfp8":
        v = q.view(torch.float8_e4m3fn).float()
    else:
        code = torch.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1)
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
        v = table[(code & 7).int()] * (1.0 - 2.0 * (code >> 3))
    f = s.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else _power(s.int() - 127)
    return (v.reshape(*s.shape, b) * f[..., None]).reshape(v.shape)


# ------------------------------------------------------------------------------------------------
# Inputs.


def _weights(shape, fmt, g, sigma):
    """Quantized N(0, sigma) weights [..., N, K], a slice of at most 2^26 values at a time."""
    lead = math.prod(shape[:-2])
    N, K = shape[-2:]
    per = max(1, (1 << 26) // (N * K))
    gs = 448.0 * 6.0 / (6.0 * sigma)  # maps six standard deviations to the formats' largest value
    q = torch.empty(lead, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(lead, N, K // BLOCK[fmt], dtype=torch.uint8, device="cuda")
    for i in range(0, lead, per):
        n = min(per, lead - i)
        w = (torch.randn(n, N, K, device="cuda", generator=g) * sigma).bfloat16().float()
        q[i:i + n], s[i:i + n] = _encode(w, fmt, gs)
    return q.reshape(*shape[:-1], -1), s.reshape(*shape[:-1], -1), gs if fmt == "nvfp4" else None


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    op, st = case["op"], dict(case)
    if op == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        logits = randn(T, E) + 1.5 * randn(1, E)  # uneven expert loads
        st["ids"] = logits.topk(k, dim=1).indices.int()
        # the rows that a padded batch masks hold whatever the padding left there
        st["mask"] = torch.rand(T, device="cuda", generator=g) < 0.8 if case["masked"] else None
        st["logits"] = logits.requires_grad_()
        st["weight"] = torch.rand((), device="cuda", generator=g) * 0.01 + 0.005
    elif op == "matvec":
        M, N, K = case["M"], case["N"], case["K"]
        st["x"] = randn(M, K).bfloat16()
        st["wq"], st["ws"], st["gs"] = _weights((N, K), case["fmt"], g, 0.02)
        st["b"] = (randn(N) * 0.01).bfloat16() if case["bias"] else None
    elif op == "expert":
        T, E, k, N, K = case["T"], case["E"], case["k"], case["N"], case["K"]
        st["ids"] = randn(T, E).topk(k, dim=1).indices.int()
        flat = st["ids"].reshape(-1).long()
        st["pairs"] = torch.argsort(flat, stable=True).int()
        st["offsets"] = torch.cat((flat.new_zeros(1), torch.bincount(flat, minlength=E).cumsum(0))).int()
        st["x"] = randn(T if case["swiglu"] else T * k, K).bfloat16()
        st["wq"], st["ws"], gs = _weights((E, N, K), case["fmt"], g, 0.02)
        st["gs"] = None if gs is None else torch.full((E,), gs, device="cuda")
        st["b"] = (randn(E, N) * 0.01).bfloat16() if case["bias"] else None
    else:
        have, new = _lengths(case)
        total = [h + n for h, n in zip(have, new)]
        P, heads, fmt = case["page"], case["heads"], case["fmt"]
        pages = [-(-n // P) for n in total]
        order = torch.randperm(sum(pages), device="cuda", generator=g).int()
        table = torch.full((case["B"], max(pages)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(pages):
            table[i, :n] = order[at:at + n]
            at += n
        cu = lambda n: torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
        st.update(table=table, cu_new=cu(new), cu_all=cu(total), start=torch.tensor(have, dtype=torch.int32, device="cuda"),
                  total=sum(total), gs=448.0 * 6.0 / 8.0)
        for name in ("k", "v"):
            dim = case[name + "_dim"]
            st[name] = randn(sum(new), heads, dim).bfloat16()
            q, s = _encode(randn(sum(pages) * P, heads, dim).bfloat16().float(), fmt, st["gs"])
            st[name + "_q"], st[name + "_s"] = (t.reshape(sum(pages), P, heads, -1) for t in (q, s))
        if own:  # the handle that a serving program keeps over its cache's memory
            import mixed_precision_moe_amd as mx
            st["cache"] = mx.PagedCache(sum(pages), P, heads, case["k_dim"], case["v_dim"], _formats(mx)[fmt],
                                        k_global_scale=st["gs"], v_global_scale=st["gs"],
                                        storage=(st["k_q"], st["k_s"], st["v_q"], st["v_s"]))
    return st


# ------------------------------------------------------------------------------------------------
# One pass.


def _formats(mx):
    return {"mxfp4": mx.FMT_MXFP4, "nvfp4": mx.FMT_NVFP4, "mxfp8": mx.FMT_MXFP8}


def _run_own(st):
    import mixed_precision_moe_amd as mx
    if st["op"] == "balance":
        loss, counts = mx.balance_loss(st["logits"], st["ids"], st["mask"])
        grad, = torch.autograd.grad(loss, st["logits"], st["weight"])
        return {"loss": loss.detach(), "counts": counts, "grad": grad}
    fmt = _formats(mx)[st["fmt"]]
    if st["op"] == "matvec":
        return mx.fp4_matvec(st["x"], st["wq"], st["ws"], st["b"], fmt=fmt, global_scale=st["gs"])
    if st["op"] == "expert":
        return mx.fp4_expert_matvec(st["x"], st["wq"], st["ws"], st["offsets"], st["pairs"], st["b"], fmt=fmt,
                                    global_scales=st["gs"], top_k=st["k"] if st["swiglu"] else 1, swiglu=st["swiglu"])
    st["cache"].write(st["k"], st["v"], st["table"], st["cu_new"], st["start"])
    k, v = st["cache"].read(st["table"], st["cu_all"], rows=st["total"])
    return {"k": k, "v": v}


def _plain_balance(st):
    logits, ids, mask = st["logits"].detach(), st["ids"], st["mask"]
    T, E = logits.shape
    k = ids.shape[1]
    live = torch.ones(T, dtype=torch.bool, device=logits.device) if mask is None else mask
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    p = torch.where(live[:, None], p, torch.zeros_like(p))
    counts = torch.zeros(E, dtype=torch.int64, device=logits.device)
    counts.index_add_(0, ids.reshape(-1).long(), live[:, None].expand(T, k).reshape(-1).long())
    tokens = live.sum()
    # 64 bits for the long sums and for counts next to their mean
    each = torch.where(tokens > 0, E / (k * tokens.double().square()), torch.zeros((), dtype=torch.float64, device=p.device))
    loss = (each * (counts * p.sum(0, dtype=torch.float64)).sum()).float()
    d = (each * (counts - counts.double().mean())).float()
    d = d - (p * d).sum(1, keepdim=True)
    # the mean taken off twice: what its rounding left counts where one expert holds nearly all of a row
    grad = st["weight"] * p * (d - (p * d).sum(1, keepdim=True))
    return {"loss": loss, "counts": counts.int(), "grad": grad}


def _plain_expert(st):
    E, N = st["wq"].shape[:2]
    flat = st["ids"].reshape(-1).long()
    rows = torch.arange(flat.numel(), device=flat.device) // (st["k"] if st["swiglu"] else 1)
    x = st["x"].float()
    if flat.numel() <= E:  # each pair's expert
        y = torch.bmm(_decode(st["wq"][flat], st["ws"][flat], st["fmt"]), x[rows][:, :, None])[:, :, 0]
    else:  # all experts on all rows
        w = _decode(st["wq"], st["ws"], st["fmt"])
        y = (w.reshape(E * N, -1) @ x.t()).reshape(E, N, -1)[flat, :, rows]
    if st["gs"] is not None:
        y = y / st["gs"][flat][:, None]
    if st["b"] is not None:
        y = y + st["b"].float()[flat]
    if st["swiglu"]:
        gate, up = y[:, :N // 2], y[:, N // 2:]
        y = gate / (1 + torch.exp(-gate)) * up
    return y.bfloat16()


def _slots(table, cu, start, rows, page):
    """The cache slot of each of `rows` ragged rows."""
    t = torch.arange(rows, device=table.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    at = t - cu[b] + (0 if start is None else start[b])
    return table[b, at // page].long() * page + at % page


def _plain_cache(st):
    out = {}
    page, fmt = st["page"], st["fmt"]
    new = _slots(st["table"], st["cu_new"], st["start"], st["k"].shape[0], page)
    every = _slots(st["table"], st["cu_all"], None, st["total"], page)
    for name in ("k", "v"):
        q, s = (st[name + part].flatten(0, 1) for part in ("_q", "_s"))
        q[new], s[new] = _encode(st[name].float(), fmt, st["gs"])
        v = _decode(q[every], s[every], fmt)
        out[name] = (v / st["gs"] if fmt == "nvfp4" else v).bfloat16()
    return out


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "balance":
        return _plain_balance(st)
    if st["op"] == "matvec":
        y = st["x"].float() @ _decode(st["wq"], st["ws"], st["fmt"]).t()
        if st["gs"] is not None:
            y = y / st["gs"]
        if st["b"] is not None:
            y = y + st["b"].float()
        return y.bfloat16()
    return _plain_expert(st) if st["op"] == "expert" else _plain_cache(st)


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits.


def _values64(q, s, fmt):
    """Each code from its bits: sign, exponent and mantissa fields, times its block's scale."""
    def minifloat(c, mant, bias):
        c = c.long()
        expo, frac = (c >> mant), (c & ((1 << mant) - 1)).double() / (1 << mant)
        lead = (expo > 0).double()
        return (lead + frac) * torch.exp2((torch.clamp(expo, min=1) - bias).double())
    b = BLOCK[fmt]
    if fmt == "mxfp8":
        v = minifloat(q & 127, 3, 7) * torch.where(q >= 128, -1.0, 1.0).double()
    else:
        c = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.uint8, device=q.device)
        c[..., 0::2], c[..., 1::2] = q % 16, q // 16
        v = minifloat(c % 8, 1, 1) * torch.where(c >= 8, -1.0, 1.0).double()
    f = minifloat(s, 3, 7) if fmt == "nvfp4" else torch.exp2(s.double() - 127)
    return v * f.repeat_interleave(b, -1)


def _nearest64(v, mant, bias, top):
    """|v| rounded to a format of `mant` fraction bits, ties to even, no larger than `top`."""
    a = v.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a))))
    e = e + (torch.exp2(e + 1) <= a).double() - (torch.exp2(e) > a).double()
    step = torch.exp2(torch.clamp(e, min=1 - bias) - mant)
    return torch.clamp(torch.round(a / step) * step, max=top) * torch.where(v < 0, -1.0, 1.0).double()


def _held64(x, fmt, gs):
    """What a row of x is once it is held in the format."""
    v = x.double().unflatten(-1, (-1, BLOCK[fmt]))
    top = v.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        s = _nearest64(gs * top / 6.0, 3, 7, 448.0)
        code = _nearest64(torch.where(s > 0, v * gs / s, torch.zeros_like(v)), 1, 1, 6.0)
        return (code * s / gs).flatten(-2)
    # the largest magnitude's exponent, one more from a significand of 1.75 on
    m, e = torch.frexp(torch.where(top > 0, top, torch.ones_like(top)))
    e = (e - 1 + (m >= 0.875).int()).double() - (8.0 if fmt == "mxfp8" else 2.0)
    scale = torch.exp2(e)
    code = _nearest64(v / scale, 3, 7, 448.0) if fmt == "mxfp8" else _nearest64(v / scale, 1, 1, 6.0)
    return (code * scale).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "balance":
        l, ids, mask = st["logits"].detach().double(), st["ids"].long(), st["mask"]
        T, E = l.shape
        k = ids.shape[1]
        keep = torch.arange(T, device=l.device) if mask is None else mask.nonzero()[:, 0]
        grad = torch.zeros_like(l)
        n = torch.bincount(ids[keep].reshape(-1), minlength=E)
        if keep.numel() == 0:
            return {"loss": l.new_zeros(()), "counts": n, "grad": grad}
        p = torch.softmax(l[keep], 1)
        loss = (E * n.double() / (k * keep.numel()) * p.mean(0)).sum()
        f = (E * n - n.sum()).double() / (k * keep.numel())  # less its mean, which the gradient does not see
        grad[keep] = st["weight"].double() / keep.numel() * p * (f - p @ f[:, None])
        return {"loss": loss, "counts": n, "grad": grad}
    if op == "matvec":
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        for i in range(0, case["N"], 1024):
            y[:, i:i + 1024] = st["x"].double() @ _values64(st["wq"][i:i + 1024], st["ws"][i:i + 1024], case["fmt"]).t()
        y = y / (st["gs"] or 1.0)
        return y + st["b"].double() if case["bias"] else y
    if op == "expert":
        N, flat = case["N"], st["ids"].reshape(-1)
        y = torch.zeros(flat.numel(), N, dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            pairs = (flat == e).nonzero()[:, 0]
            if pairs.numel():
                x = st["x"][pairs // case["k"] if case["swiglu"] else pairs].double()
                y[pairs] = x @ _values64(st["wq"][e], st["ws"][e], case["fmt"]).t()
                if st["gs"] is not None:
                    y[pairs] /= st["gs"][e].double()
                if case["bias"]:
                    y[pairs] += st["b"][e].double()
        return torch.nn.functional.silu(y[:, :N // 2]) * y[:, N // 2:] if case["swiglu"] else y
    have, new = _lengths(case)
    out = {}
    for name in ("k", "v"):
        parts, at = [], 0
        for i in range(case["B"]):
            pos = torch.arange(have[i], device="cuda")
            page, slot = st["table"][i].long()[pos // case["page"]], pos % case["page"]
            old = _values64(st[name + "_q"][page, slot], st[name + "_s"][page, slot], case["fmt"])
            parts += [old / st["gs"] if case["fmt"] == "nvfp4" else old, _held64(st[name][at:at + new[i]], case["fmt"], st["gs"])]
            at += new[i]
        out[name] = torch.cat(parts)
    return out
