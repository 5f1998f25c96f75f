"""The workloads on which rotary positions, attention of drafted tokens over the block-quantized paged cache, the
compaction of accepted drafts and the page pool are timed: their inputs, a plain torch form, the library's calls and a
64-bit form.

With `own` false, run() computes an operator in elementary torch operations in 32 bits (angles in 64); with `own` true
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
        # serving one token: queries and keys of a small layer; launch latency
        dict(name="rotary_token", op="rotary", T=1, q_heads=4, k_heads=2, dim=64, rot=64, offset=0, pairs="half",
             scaling="none", dtype="bf16", train=False),
        # a prompt's queries and keys, views of one packed projection, far positions of a scaled context
        dict(name="rotary_prompt", op="rotary", T=8192, q_heads=32, k_heads=8, dim=128, rot=128, offset=0, pairs="half",
             scaling="ramp", dtype="bf16", train=False),
        # training: both directions, an odd token count, the last third of each head turned, neighbouring pairs
        dict(name="rotary_train", op="rotary", T=4099, q_heads=16, k_heads=16, dim=192, rot=64, offset=128,
             pairs="interleaved", scaling="linear", dtype="fp32", train=True),
        # one new token of one short conversation: latency
        dict(name="attend_token", op="attend", fmt="mxfp4", B=1, new=1, context=77, heads=2, group=2, k_dim=64, v_dim=64,
             page=16, tree=False),
        # a decode step of a batch with ragged contexts, one new token each: the cache's bytes count
        dict(name="attend_decode", op="attend", fmt="mxfp8", B=32, new=1, context=3900, heads=8, group=4, k_dim=128,
             v_dim=128, page=64, tree=False),
        # trees of drafted tokens, many query heads to a key head, keys wider than values, pages that end inside a tile
        dict(name="attend_tree", op="attend", fmt="nvfp4", B=12, new=33, context=5000, heads=4, group=8, k_dim=192,
             v_dim=128, page=24, tree=True),
        # one very long context with a few drafts: the work has to be split over it
        dict(name="attend_long", op="attend", fmt="mxfp4", B=1, new=7, context=130000, heads=8, group=5, k_dim=128,
             v_dim=128, page=128, tree=True),
        # a chunk of a prompt against what is cached: arithmetic counts
        dict(name="attend_chunk", op="attend", fmt="mxfp8", B=2, new=1024, context=4096, heads=8, group=4, k_dim=128,
             v_dim=128, page=64, tree=False),
        # after a decode step: the accepted branch of each small tree is moved together
        dict(name="compact_step", op="compact", fmt="mxfp8", B=16, new=8, context=300, heads=8, k_dim=128, v_dim=128,
             page=64),
        # a large batch of large trees, long accepted branches, an odd page size
        dict(name="compact_batch", op="compact", fmt="nvfp4", B=250, new=64, context=130, heads=8, k_dim=192, v_dim=128,
             page=24),
        # between two decode steps: pages of rejected drafts go back, pages for the next drafts are taken
        dict(name="pool_step", op="pool", kind="step", fmt="mxfp8", B=64, samples=0, new=33, context=2000, heads=2,
             k_dim=64, v_dim=64, page=16),
        # several samples of each prompt: whole pages are shared, the last one is copied
        dict(name="pool_fork", op="pool", kind="fork", fmt="mxfp8", B=48, samples=7, new=1, context=1500, heads=8,
             k_dim=128, v_dim=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "attend", "attend", "compact", "pool"])
    if op == "rotary":
        k_heads = _log_int(rng, 1, 16)
        q_heads = k_heads * _log_int(rng, 1, 8)
        dim = 16 * rng.randint(2, 16)
        rot = min(dim, rng.choice([dim, 16 * rng.randint(1, 16), 2 * rng.randint(1, 128)]))
        train = rng.random() < 0.4
        T = _log_int(rng, 1, 40_000_000 // ((q_heads + k_heads) * dim * (2 if train else 1)))
        return dict(op=op, T=T, q_heads=q_heads, k_heads=k_heads, dim=dim, rot=rot,
                    offset=rng.choice([0, dim - rot]), pairs=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ramp"]), dtype=rng.choice(["bf16", "fp32"]), train=train)
    fmt = rng.choice(["mxfp4", "nvfp4", "mxfp8"])
    b = BLOCK[fmt]
    heads = _log_int(rng, 1, 16)
    k_dim, v_dim = b * rng.randint(1, 256 // b), b * rng.randint(1, 256 // b)
    page = rng.choice([1, 16, 24, 32, 64, 128])
    B = _log_int(rng, 1, 64)
    rows = 60_000_000 // (heads * (k_dim + v_dim))  # tokens in the cache, about
    if op == "compact":
        new = _log_int(rng, 2, 64)
        context = _log_int(rng, 1, max(1, min(2000, rows // B - new)))
        return dict(op=op, fmt=fmt, B=B, new=new, context=context, heads=heads, k_dim=k_dim, v_dim=v_dim, page=page)
    if op == "pool":
        kind = rng.choice(["step", "fork"])
        samples = _log_int(rng, 1, 8) if kind == "fork" else 0
        context = _log_int(rng, 1, max(1, min(20000, rows // (2 * B))))
        return dict(op=op, kind=kind, fmt=fmt, B=B, samples=samples, new=_log_int(rng, 1, 64), context=context, heads=heads,
                    k_dim=k_dim, v_dim=v_dim, page=max(page, 16))
    group = _log_int(rng, 1, 16)
    context = _log_int(rng, 1, max(1, rows // B))
    most = 40_000_000_000 // (B * heads * group * (context + 64) * (k_dim + v_dim))  # scores and sums of all rows
    new = rng.choice([1, _log_int(rng, 1, 64)])
    return dict(op=op, fmt=fmt, B=B, new=max(1, min(new, most)), context=context, heads=heads, group=group, k_dim=k_dim,
                v_dim=v_dim, page=page, tree=rng.random() < 0.7)


def _lengths(case):
    """(tokens in the cache before, new tokens) of each sequence: ragged, the same for every seed."""
    have = [case["context"] - (7919 * i) % (case["context"] // 2 + 1) for i in range(case["B"])]
    new = [case["new"] - (104729 * i) % (case["new"] // 2 + 1) for i in range(case["B"])]
    return have, new


def _path_lengths(case):
    """Accepted drafts of each sequence, and how many of them stay where they are."""
    new = _lengths(case)[1]
    count = [min(n, 1 + (31 * i + n // 2) % (n // 2 + 1)) for i, n in enumerate(new)]
    return count, [min(c, 1 + i % 3) for i, c in enumerate(count)]


def _row_bytes(case):
    width = case["heads"] * (case["k_dim"] + case["v_dim"])
    return width // (1 if case["fmt"] == "mxfp8" else 2) + width // BLOCK[case["fmt"]]


def work(case):
    op = case["op"]
    if op == "rotary":
        n = case["T"] * (case["q_heads"] + case["k_heads"])
        both = 2 if case["train"] else 1
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": both * (2 * n * case["dim"] * size + 4 * case["T"]), "flops": both * 3 * n * case["rot"]}
    have, new = _lengths(case)
    if op == "attend":
        total = sum(h + n for h, n in zip(have, new))
        per_row = case["heads"] * case["group"] * (case["k_dim"] + case["v_dim"])
        # what the rows see: all before the drafts, and of those about half where a mask or the order leaves half
        seen = sum(n * (h + (n + 1) / 2) for h, n in zip(have, new))
        return {"bytes": total * _row_bytes(case) + sum(new) * (2 * per_row + (max(new) if case["tree"] else 0)),
                "flops": 2 * per_row * seen}
    if op == "compact":
        count, stay = _path_lengths(case)
        return {"bytes": 2 * _row_bytes(case) * (sum(count) - sum(stay)) + 4 * case["B"] * (case["new"] + 2), "flops": 0}
    rows, pages, width, kept, later = _pool_sizes(case)
    if case["kind"] == "step":
        changed = sum(-(-n // case["page"]) - k // case["page"] for k, n in zip(kept, later))
        return {"bytes": 4 * (rows * width + pages + 2 * 2 * changed + 2 * rows), "flops": 0}
    copied = sum(k % case["page"] for k in kept) * case["samples"]
    shared = sum(k // case["page"] for k in kept) * case["samples"]
    return {"bytes": 2 * _row_bytes(case) * copied + 4 * (rows * width + pages + 2 * shared), "flops": 0}


def _pool_sizes(case):
    """(rows of the table, pages of the cache, columns, tokens that each sequence keeps, tokens it then has room for)."""
    have, new = _lengths(case)
    rows = case["B"] * (1 + case["samples"])
    later = [h + n for h, n in zip(have, new)]
    width = max(-(-n // case["page"]) for n in later) + 1
    return rows, sum(-(-n // case["page"]) for n in later) + rows * 2 + 16, width, have, later


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


def _encode(v, fmt, gs):
    """v float32 [..., D], drawn from a normal distribution -> (codes uint8, two to a byte in the 4-bit formats; scale bytes)."""
    v = v.unflatten(-1, (-1, BLOCK[fmt]))
    top = v.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        scale = (gs * top / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
        code = _e2m1_code(v.abs() * (gs / scale.float()))
        scale = scale.view(torch.uint8)
    else:
        e = ((top.contiguous().view(torch.int32) + (1 << 21)) >> 23) - (8 if fmt == "mxfp8" else 2)
        scale = e.to(torch.uint8)
        if fmt == "mxfp8":
            return (v * _power(127 - e)).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2), scale.squeeze(-1)
        code = _e2m1_code(v.abs() * _power(127 - e))
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.squeeze(-1)


def _decode(q, s, fmt):
    """Values in float32, without the global scale."""
    if fmt == "mxfp8":
        v = q.view(torch.float8_e4m3fn).float()
    else:
        code = torch.stack((q & 15, q >> 4), -1).flatten(-2)
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
        v = table[(code & 7).int()] * (1.0 - 2.0 * (code >> 3))
    f = s.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else _power(s.int() - 127)
    return (v.unflatten(-1, (-1, BLOCK[fmt])) * f[..., None]).flatten(-2)


# ------------------------------------------------------------------------------------------------
# Inputs.

# what a scaled layer's configuration says: positions divided by 4; or frequencies that turn fewer than `slow` times
# over the original length divided by 16, those that turn more than `fast` times kept, a ramp between, and the lengths
# of the turned vectors scaled along
SCALING = {"none": None, "linear": dict(kind="linear", factor=4.0),
           "ramp": dict(kind="ramp", factor=16.0, length=8192, fast=32.0, slow=1.0, magnitude=1.0 + 0.1 * math.log(16.0))}


def _frequencies(rot, scaling):
    """(radians per position of each pair in 64 bits, the factor of the turned vectors)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    s = SCALING[scaling]
    if s is None:
        return f, 1.0
    if s["kind"] == "linear":
        return f / s["factor"], 1.0
    # the index of a pair that turns n times over the original length
    pair = lambda n: rot * math.log(s["length"] / (2 * math.pi * n)) / (2 * math.log(10000.0))  # noqa: E731
    low, high = max(0, math.floor(pair(s["fast"]))), min(rot - 1, math.ceil(pair(s["slow"])))
    ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
    return f * (1 - ramp) + f / s["factor"] * ramp, s["magnitude"]


def _cu(n):
    return torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")


def _i32(n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def _trees(new, g):
    """Which drafts each draft sees: itself and its ancestors in a random tree of its sequence's drafts."""
    B, W = len(new), max(new)
    parent = (torch.rand(B, W, device="cuda", generator=g) * torch.arange(W, device="cuda")).long()
    sees = torch.zeros(B, W, W, device="cuda").scatter_(2, parent[:, :, None], 1.0)
    sees = ((sees + torch.eye(W, device="cuda")) > 0).float()  # itself and its parent
    for _ in range(max(1, W).bit_length()):
        sees = ((sees @ sees) > 0).float()
    # the first draft's parent is itself: a root
    return torch.cat([sees[i, :n] for i, n in enumerate(new)]).bool()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    op, st = case["op"], dict(case)
    if own:
        import mixed_precision_moe_amd as mx
    if op == "rotary":
        T, Hq, Hk, D = case["T"], case["q_heads"], case["k_heads"], case["dim"]
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # queries, keys and values as one projection gives them
        packed = randn(T, Hq + 2 * Hk, D).to(dtype)
        st["q"], st["k"] = packed[:, :Hq], packed[:, Hq:Hq + Hk]
        top = 131072 if case["scaling"] == "ramp" else 32768
        st["positions"] = (torch.arange(T, device="cuda") + torch.randint(0, top - T + 1, (), device="cuda", generator=g)).int()
        freqs, st["magnitude"] = _frequencies(case["rot"], case["scaling"])
        st["freqs"] = freqs.cuda()
        if case["train"]:
            st["gq"], st["gk"] = randn(T, Hq, D).to(dtype), randn(T, Hk, D).to(dtype)
            st["q"], st["k"] = st["q"].detach().requires_grad_(), st["k"].detach().requires_grad_()
        if own:  # the layer's handle
            st["rotary"] = mx.Rotary(case["rot"], interleaved=case["pairs"] == "interleaved", offset=case["offset"],
                                     scaling=SCALING[case["scaling"]])
        return st
    P, heads, fmt, B = case["page"], case["heads"], case["fmt"], case["B"]
    have, new = _lengths(case)
    total = [h + n for h, n in zip(have, new)]
    if op == "pool":
        rows, pages, width, kept, later = _pool_sizes(case)
        held = [-(-n // P) for n in later]  # the last step's drafts had pages too
    else:
        held = [-(-n // P) for n in total]
        rows, pages, width = B, sum(held), max(held)
    order = torch.randperm(pages, device="cuda", generator=g).int()
    st["table"] = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(held):
        st["table"][i, :n] = order[at:at + n]
        at += n
    st["gs"] = 448.0 * 6.0 / 8.0
    for name in ("k", "v"):
        dim = case[name + "_dim"]
        if op == "attend":
            q, s = _encode(randn(pages * P, heads, dim), fmt, st["gs"])
        else:  # moved as they are: any bytes
            q, s = (torch.randint(0, 256, (pages * P, heads, n), dtype=torch.uint8, device="cuda", generator=g)
                    for n in (dim // (1 if fmt == "mxfp8" else 2), dim // BLOCK[fmt]))
        st[name + "_q"], st[name + "_s"] = (t.reshape(pages, P, heads, -1) for t in (q, s))
    if own:  # the handle that a serving program keeps over its cache's memory
        formats = {"mxfp4": mx.FMT_MXFP4, "nvfp4": mx.FMT_NVFP4, "mxfp8": mx.FMT_MXFP8}
        st["cache"] = mx.PagedCache(pages, P, heads, case["k_dim"], case["v_dim"], formats[fmt], st["gs"], st["gs"],
                                    storage=(st["k_q"], st["k_s"], st["v_q"], st["v_s"]))
    if op == "attend":
        st.update(q=randn(sum(new), heads * case["group"], case["k_dim"]).bfloat16(), cu=_cu(new), start=_i32(have),
                  mask=_trees(new, g) if case["tree"] else None, longest=max(total), most=max(new))
    elif op == "compact":
        # a drafter numbers its best chain first: the accepted branch follows it for a few tokens, then leaves it for
        # alternatives that are numbered behind all places that the branch moves to
        count, stay = _path_lengths(case)
        path = torch.full((B, case["new"]), -1, dtype=torch.int32, device="cuda")
        for i, (c, keep, n) in enumerate(zip(count, stay, new)):
            later = c + torch.randperm(n - c, device="cuda", generator=g)[:c - keep].sort().values
            keep = c - later.numel()
            path[i, :keep] = torch.arange(keep, device="cuda").int()
            path[i, keep:c] = later.int()
        st.update(path=path, start=_i32(have))
    else:
        st["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
        st["refs"][order[:at].long()] = 1
        if case["kind"] == "step":
            st.update(kept=_i32(kept), later=_i32(later))
        else:
            st.update(src=torch.arange(B, device="cuda").repeat_interleave(case["samples"]).int(),
                      dst=torch.arange(B, rows, device="cuda").int(),
                      lengths=_i32(kept).repeat_interleave(case["samples"]))
        if own:
            st["pool"] = mx.PagePool(st["cache"], refs=st["refs"])
    return st


# ------------------------------------------------------------------------------------------------
# One pass.


def _run_own(st):
    op = st["op"]
    if op == "rotary":
        q, k = st["rotary"](st["q"], st["k"], st["positions"])
        if not st["train"]:
            return {"q": q, "k": k}
        gq, gk = torch.autograd.grad((q, k), (st["q"], st["k"]), (st["gq"], st["gk"]))
        return {"q": q.detach(), "k": k.detach(), "gq": gq, "gk": gk}
    if op == "attend":
        return st["cache"].attend(st["q"], st["table"], st["cu"], st["start"], tree_mask=st["mask"])
    if op == "compact":
        lengths = st["cache"].compact(st["table"], st["start"], st["path"])
        return {"lengths": lengths, "k_q": st["k_q"], "k_s": st["k_s"], "v_q": st["v_q"], "v_s": st["v_s"]}
    if st["kind"] == "step":
        st["pool"].resize(st["table"], st["kept"])
        missing = st["pool"].resize(st["table"], st["later"])
        return {"table": st["table"], "refs": st["refs"], "missing": missing}
    missing = st["pool"].fork(st["table"], st["src"], st["dst"], st["lengths"])
    return {"table": st["table"], "refs": st["refs"], "missing": missing, "k_q": st["k_q"], "k_s": st["k_s"],
            "v_q": st["v_q"], "v_s": st["v_s"]}


def _turn(x, cos, sin, st):
    """The pairs of x turned in 32 bits, the rest as it is, rounded once."""
    rot, at = st["rot"], st["offset"]
    part = x[..., at:at + rot].float()
    a, b = (part[..., 0::2], part[..., 1::2]) if st["pairs"] == "interleaved" else (part[..., :rot // 2], part[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    part = torch.stack((a, b), -1).flatten(-2) if st["pairs"] == "interleaved" else torch.cat((a, b), -1)
    return torch.cat((x[..., :at], part.to(x.dtype), x[..., at + rot:]), -1)


def _plain_rotary(st):
    angle = st["positions"].double()[:, None, None] * st["freqs"]
    cos, sin = (st["magnitude"] * angle.cos()).float(), (st["magnitude"] * angle.sin()).float()
    out = {"q": _turn(st["q"].detach(), cos, sin, st), "k": _turn(st["k"].detach(), cos, sin, st)}
    if st["train"]:
        out.update(gq=_turn(st["gq"], cos, -sin, st), gk=_turn(st["gk"], cos, -sin, st))
    return out


def _plain_attend(st):
    heads, group, page, fmt = st["heads"], st["group"], st["page"], st["fmt"]
    cu, start, device = st["cu"].long(), st["start"].long(), st["q"].device
    n = cu[1:] - cu[:-1]
    at = torch.arange(st["longest"], device=device)
    slot = st["table"][:, at // page].clamp(min=0).long() * page + at % page
    k, v = (_decode(*(st[name + part].flatten(0, 1)[slot] for part in ("_q", "_s")), fmt).transpose(1, 2).contiguous()
            for name in ("k", "v"))  # [B, heads, longest, dim]
    draft = torch.arange(st["most"], device=device)
    row = (cu[:-1, None] + draft).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[row].unflatten(2, (heads, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = q @ k.transpose(2, 3) * (st["k_dim"] ** -0.5 / (st["gs"] if fmt == "nvfp4" else 1.0))
    place = at - start[:, None]  # as a draft of its sequence
    inside = (place < n[:, None])[:, None]
    if st["mask"] is None:
        sees = inside & (place[:, None] <= draft[:, None])
    else:
        drafts = st["mask"][row].gather(2, place[:, None].clamp(0, st["mask"].shape[1] - 1).expand(-1, st["most"], -1))
        sees = inside & ((place < 0)[:, None] | drafts)
    s = s.unflatten(2, (st["most"], group)).masked_fill_(~sees[:, None, :, None], -math.inf)
    s = torch.exp_(s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30))).flatten(2, 3)
    o = s @ v / (s.sum(-1, keepdim=True).clamp(min=1e-30) * (st["gs"] if fmt == "nvfp4" else 1.0))
    o = o.unflatten(2, (st["most"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, most, heads * group, v_dim]
    t = torch.arange(st["q"].shape[0], device=device)
    b = torch.searchsorted(cu[1:], t, right=True)
    return o[b, t - cu[b]].bfloat16()


def _planes(st):
    return [st[name].flatten(0, 1) for name in ("k_q", "k_s", "v_q", "v_s")]


def _plain_compact(st):
    page, path, start = st["page"], st["path"].long(), st["start"].long()
    i = torch.arange(path.shape[1], device=path.device)
    before = torch.cat((path.new_full((path.shape[0], 1), -1), path[:, :-1]), 1)
    good = (path > before).long().cumprod(1).bool()

    def slot(at):
        return st["table"].gather(1, (at // page).clamp(max=st["table"].shape[1] - 1)).long() * page + at % page

    # what does not move is written onto itself
    to = slot(start[:, None] + i)
    source = torch.where(good, slot(start[:, None] + torch.where(good, path, 0)), to)
    there = good.flatten().nonzero()[:, 0]
    for plane in _planes(st):
        plane[to.flatten()[there]] = plane[source.flatten()[there]]
    return {"lengths": (start + good.sum(1)).int(), "k_q": st["k_q"], "k_s": st["k_s"], "v_q": st["v_q"], "v_s": st["v_s"]}


def _plain_take(st, table, add, shared):
    """Pages for the marked entries of the table, row by row, the lowest free page first; an entry in `shared` is
    replaced.  Returns (the entries' new pages, which got one, how many did not)."""
    refs = st["refs"]
    free = torch.argsort((refs > 0).to(torch.uint8), stable=True)
    rank = add.flatten().long().cumsum(0).sub_(1).view_as(add)
    got = add & (rank < (refs <= 0).sum())
    page = free[rank.clamp(0, refs.numel() - 1)]
    refs.index_add_(0, page.flatten(), got.flatten().int())
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -(got & shared).flatten().int())
    return page.int(), got, (add & ~got).sum().int()


def _plain_copy(st, source, to, rows):
    """The first `rows` rows of page source[i] to page to[i]."""
    r = torch.arange(st["page"], device=source.device)
    i, r = (r < rows[:, None]).nonzero().unbind(1)
    for plane in _planes(st):
        plane[to[i].long() * st["page"] + r] = plane[source[i].long() * st["page"] + r]


def _plain_resize(st, lengths):
    table, refs, page = st["table"], st["refs"], st["page"]
    i = torch.arange(table.shape[1], device=table.device)
    want = ((lengths.long() + page - 1) // page)[:, None]
    held = (table >= 0).long().cumprod(1).sum(1, keepdim=True)
    drop = (i >= want) & (i < held)
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -drop.flatten().int())
    table.masked_fill_(i >= want, -1)
    ends = (i == want - 1) & (held >= want) & (lengths % page != 0)[:, None]
    shared = ends & (refs[table.clamp(min=0).long()] > 1)
    new, got, missing = _plain_take(st, table, (i >= held) & (i < want) | shared, shared)
    copied = (got & shared).any(1)
    last = (want - 1).clamp(min=0)
    _plain_copy(st, table.gather(1, last)[:, 0], new.gather(1, last)[:, 0], (lengths % page) * copied)
    table.copy_(torch.where(got, new, table))
    return missing


def _plain_fork(st):
    table, refs, page = st["table"], st["refs"], st["page"]
    src, dst, lengths = st["src"].long(), st["dst"].long(), st["lengths"].long()
    i = torch.arange(table.shape[1], device=table.device)
    old, from_row = table[dst], table[src]
    held = (old >= 0).long().cumprod(1).bool()
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -held.flatten().int())
    whole = (lengths // page)[:, None]
    share = (i < whole) & (from_row >= 0)
    refs.index_add_(0, from_row.clamp(min=0).flatten().long(), share.flatten().int())
    part = (i == whole) & (lengths % page != 0)[:, None] & (from_row >= 0)
    new, got, missing = _plain_take(st, from_row, part, torch.zeros_like(part))
    at = whole.clamp(max=table.shape[1] - 1)
    _plain_copy(st, from_row.gather(1, at)[:, 0], new.gather(1, at)[:, 0], (lengths % page) * got.any(1))
    table[dst] = torch.where(share, from_row, torch.where(got, new, torch.full_like(new, -1)))
    return missing


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "rotary":
        return _plain_rotary(st)
    if st["op"] == "attend":
        return _plain_attend(st)
    if st["op"] == "compact":
        return _plain_compact(st)
    if st["kind"] == "step":
        _plain_resize(st, st["kept"])
        missing = _plain_resize(st, st["later"])
        return {"table": st["table"], "refs": st["refs"], "missing": missing}
    missing = _plain_fork(st)
    return {"table": st["table"], "refs": st["refs"], "missing": missing, "k_q": st["k_q"], "k_s": st["k_s"],
            "v_q": st["v_q"], "v_s": st["v_s"]}


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits.


def _values64(q, s, fmt):
    """Each code from its bits: sign, exponent and mantissa fields, times its block's scale."""
    def minifloat(c, mant, bias):
        c = c.long()
        expo, frac = (c >> mant), (c & ((1 << mant) - 1)).double() / (1 << mant)
        lead = (expo > 0).double()
        return (lead + frac) * torch.exp2((torch.clamp(expo, min=1) - bias).double())
    if fmt == "mxfp8":
        v = minifloat(q & 127, 3, 7) * torch.where(q >= 128, -1.0, 1.0).double()
    else:
        c = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.uint8, device=q.device)
        c[..., 0::2], c[..., 1::2] = q % 16, q // 16
        v = minifloat(c % 8, 1, 1) * torch.where(c >= 8, -1.0, 1.0).double()
    f = minifloat(s, 3, 7) if fmt == "nvfp4" else torch.exp2(s.double() - 127)
    return v * f.repeat_interleave(BLOCK[fmt], -1)


def exact(case, seed):
    op = case["op"]
    if op in ("compact", "pool"):
        return None  # bytes and whole numbers, moved or counted
    st = prepare(case, seed)
    if op == "rotary":
        rot, at = case["rot"], case["offset"]
        turn = torch.polar(torch.full((case["T"], 1, rot // 2), st["magnitude"], dtype=torch.float64, device="cuda"),
                           (st["positions"].double()[:, None] * st["freqs"])[:, None])

        def turned(x, by):
            x = x.detach().double()
            y, part = x.clone(), x[..., at:at + rot]
            if case["pairs"] == "interleaved":
                z = torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * by
                y[..., at:at + rot:2], y[..., at + 1:at + rot:2] = z.real, z.imag
            else:
                z = torch.complex(part[..., :rot // 2].contiguous(), part[..., rot // 2:].contiguous()) * by
                y[..., at:at + rot // 2], y[..., at + rot // 2:at + rot] = z.real, z.imag
            return y
        out = {"q": turned(st["q"], turn), "k": turned(st["k"], turn)}
        if case["train"]:
            out.update(gq=turned(st["gq"], turn.conj()), gk=turned(st["gk"], turn.conj()))
        return out
    have, new = _lengths(case)
    heads, group, page = case["heads"], case["group"], case["page"]
    div = st["gs"] if case["fmt"] == "nvfp4" else 1.0
    out = torch.zeros(sum(new), heads * group, case["v_dim"], dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["B"]):
        pos = torch.arange(have[b] + new[b], device="cuda")
        where = st["table"][b].long()[pos // page], pos % page
        sees = torch.ones(new[b], pos.numel(), dtype=torch.bool, device="cuda")
        drafts = torch.ones(new[b], new[b], dtype=torch.bool, device="cuda").tril()
        sees[:, have[b]:] = drafts if st["mask"] is None else st["mask"][at:at + new[b], :new[b]]
        for h in range(heads):
            k, v = (_values64(*(st[name + part][:, :, h][where] for part in ("_q", "_s")), case["fmt"]) / div for name in ("k", "v"))
            q = st["q"][at:at + new[b], h * group:(h + 1) * group].double()
            s = torch.where(sees[:, None], q @ k.t() / math.sqrt(case["k_dim"]), -math.inf)
            out[at:at + new[b], h * group:(h + 1) * group] = torch.softmax(s, -1) @ v
        at += new[b]
    return out
