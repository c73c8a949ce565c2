"""The gated delta rule and a key-value cache held in 8 bits with a scale for each block of tokens and
head, measured: the delta rule over prompts and for single tokens, quantising a cache as it is written,
reading it back, and attention of one token over it.

Each case is one call of one operator; a written cache is read back whole, for the values that its codes
stand for. `run` computes it in elementary torch operations, or with the library's kernels where `own` is
true. Lengths of a ragged batch follow from the case itself.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8, "fp8": torch.float8_e4m3fn}
MOST = {"int8": 127.0, "fp8": 448.0}  # largest magnitude of a code
LEAST = 2.0 ** -126                   # and the least scale
CHUNK = 64                            # tokens per block of the plain chunked form


def listed():
    return [
        # Short ragged prompts of several requests that go on from earlier states.
        dict(name="delta 9x300 ragged", op="delta", batch=9, length=300, heads=16, qk=16, dk=128, dv=128,
             type="fp16", decay="token", initial=True, salt=1),
        # One long prompt, two value heads to a key head.
        dict(name="delta 1x20000", op="delta", batch=1, length=20000, heads=32, qk=16, dk=128, dv=128,
             type="bf16", decay="token", initial=False, salt=2),
        # Single-stream decode of a delta-rule layer: latency.
        dict(name="step 1", op="step", batch=1, heads=32, qk=16, dk=128, dv=128, type="bf16", decay="token",
             salt=3),
        # Batched decode: every state is read and written once.
        dict(name="step 250", op="step", batch=250, heads=32, qk=32, dk=128, dv=128, type="bf16",
             decay="token", salt=4),
        # A decode step's 16 tokens, most of them into blocks that hold others.
        dict(name="store decode 16", op="store", batch=16, ctx=4000, new=1, heads=8, dim=128, page=16, block=16,
             type="bf16", cache="int8", layout="hnd", salt=5),
        # Prompts beside decoding requests, e4m3 codes, two blocks to a page.
        dict(name="store prompts 40", op="store", batch=40, ctx=3000, new=900, heads=8, dim=128, page=64, block=32,
             type="bf16", cache="fp8", layout="nhd", salt=6),
        # A short history read back, for the rest of its prompt.
        dict(name="load 500", op="load", tokens=500, heads=4, dim=128, page=16, block=16, type="fp16", cache="int8",
             layout="hnd", salt=7),
        # A long one.
        dict(name="load 60000", op="load", tokens=60000, heads=8, dim=128, page=64, block=64, type="bf16", cache="fp8",
             layout="nhd", salt=8),
        # Single-stream decode at an ordinary length: latency.
        dict(name="attend 1x1100", op="attend", batch=1, length=1100, heads=32, kv=8, dim=128, page=16, block=16,
             type="bf16", cache="int8", layout="hnd", window=0, lse=False, salt=9),
        # Single-stream decode over a long cache: work must be split over the length.
        dict(name="attend 1x131000", op="attend", batch=1, length=131000, heads=32, kv=8, dim=128, page=16, block=16,
             type="bf16", cache="int8", layout="nhd", window=0, lse=True, salt=10),
        # Batched serving, ragged lengths, the largest cache read here.
        dict(name="attend 64x8192 ragged", op="attend", batch=64, length=8192, heads=64, kv=8, dim=128, page=32,
             block=32, type="bf16", cache="int8", layout="hnd", window=0, lse=False, salt=11),
        # An odd head ratio, e4m3 codes, float16 activations.
        dict(name="attend 48x5000 e4m3", op="attend", batch=48, length=5000, heads=28, kv=4, dim=128, page=64, block=16,
             type="fp16", cache="fp8", layout="nhd", window=0, lse=False, salt=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "step", "store", "load", "attend", "attend"])
    salt = rng.randrange(1 << 20)
    kind, cache, layout = rng.choice(["bf16", "fp16"]), rng.choice(["int8", "fp8"]), rng.choice(["hnd", "nhd"])
    page, block = rng.choice([(16, 16), (32, 16), (32, 32), (48, 48), (64, 16), (64, 64), (128, 64), (128, 32)])
    if op in ("delta", "step"):
        heads, dk, dv = rng.choice([4, 8, 16, 32]), rng.choice([64, 128]), rng.choice([64, 128])
        c = dict(op=op, heads=heads, qk=heads // rng.choice([1, 1, 2]), dk=dk, dv=dv, type=kind,
                 decay=rng.choice(["token", "head"]), salt=salt)
        if op == "step":
            return dict(c, batch=_log(rng, 1, 300))
        batch = _log(rng, 1, 40)
        return dict(c, batch=batch, length=_log(rng, 1, max(1, 12000 // batch)), initial=rng.choice([True, False]))
    c = dict(op=op, page=page, block=block, type=kind, cache=cache, layout=layout, salt=salt)
    if op == "store":
        batch = _log(rng, 1, 300)
        return dict(c, batch=batch, ctx=_log(rng, 1, 8000), new=_log(rng, 1, max(1, 12000 // batch)),
                    heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]))
    if op == "load":
        return dict(c, tokens=_log(rng, 1, 40000), heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 96, 128, 256]))
    kv, dim, batch = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 192, 256]), _log(rng, 1, 200)
    most = max(1, min(131000, (1 << 28) // (batch * kv * dim)))
    return dict(c, batch=batch, length=_log(rng, 1, most), heads=kv * rng.choice([1, 2, 4, 5, 7, 8, 16]), kv=kv, dim=dim,
                window=rng.choice([0, 0, 0, 500]), lse=rng.choice([True, False]))


# ---- sizes that follow from a case ---------------------------------------------------------------

def _ragged(count, most, salt):
    """Lengths from 1 to `most`, spread over their logarithm's upper part, the first one `most`."""
    r = np.random.RandomState(salt)
    n = np.exp(r.uniform(math.log(max(1.0, most / 8)), math.log(most + 0.5), count)).astype(np.int64)
    n[0] = most
    return np.clip(n, 1, most)


def _lengths(case):
    n = _ragged(case["batch"], case["length"], case["salt"])
    if case["batch"] > 6:
        n[3] = 0  # a slot of the batch that holds no request
    return n


def _requests(case):
    """(cached tokens, new tokens) of each request; every fourth one of a ragged batch decodes."""
    r = np.random.RandomState(case["salt"])
    c = r.randint(0, case["ctx"] + 1, case["batch"])
    n = _ragged(case["batch"], case["new"], case["salt"] + 1)
    n[1::4] = 1
    if case["batch"] > 6:
        n[5] = 0
        c[2] = 0
    return c, n


def _pages(tokens, page):
    return -(-tokens // page)


def _stored(case):
    """Pages of a written cache (those that the call reaches, and two that it does not)."""
    c, n = _requests(case)
    return int((_pages(c + n, case["page"]) - c // case["page"])[n > 0].sum()) + 2


def work(case):
    op = case["op"]
    if op in ("delta", "step"):
        step = op == "step"
        t = case["batch"] if step else int(_lengths(case).sum())
        state = case["heads"] * case["dk"] * case["dv"]
        token = 2 * (2 * case["qk"] * case["dk"] + 2 * case["heads"] * case["dv"]) + 4 * case["heads"] * (
            2 if case["decay"] == "token" else 1)
        return {"bytes": t * token + 4 * state * case["batch"] * (2 if step or case["initial"] else 1), "flops": 7 * t * state}
    row = case.get("kv", case["heads"]) * case["dim"] * 2
    scale = 8 * case.get("kv", case["heads"])  # of a block of tokens
    if op == "store":  # new tokens in and into the cache, and the cache read back
        t, pages = int(_requests(case)[1].sum()), _stored(case)
        return {"bytes": t * row * 3 + pages * (3 * case["page"] * row + 2 * case["page"] // case["block"] * scale),
                "flops": 0}
    if op == "load":
        return {"bytes": case["tokens"] * row * 3 + _pages(case["tokens"], case["block"]) * scale, "flops": 0}
    n = _lengths(case)
    seen = int((np.minimum(n, case["window"]) if case["window"] else n).sum())
    return {"bytes": seen * row + seen // case["block"] * scale
            + case["batch"] * case["heads"] * (case["dim"] * 4 + (4 if case["lse"] else 0)),
            "flops": 4 * seen * case["heads"] * case["dim"]}


# ---- inputs --------------------------------------------------------------------------------------

def _cache(case, pages, heads, gen):
    """A cache [pages, page, heads, dim] of codes in either order in memory, and the scales of its blocks."""
    page, dim = case["page"], case["dim"]
    shape = (pages, heads, page, dim) if case["layout"] == "hnd" else (pages, page, heads, dim)
    if case["cache"] == "int8":
        x = torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)
    else:
        x = (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16) * 128).clamp(-448, 448).to(TYPES["fp8"])
    rows = torch.rand((pages, page // case["block"], heads), generator=gen, device="cuda") * 2 + 1
    return x.permute(0, 2, 1, 3) if case["layout"] == "hnd" else x, rows / MOST[case["cache"]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + case["salt"])
    s = dict(case)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(TYPES[case["type"]])

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", torch.int32)

    op = case["op"]
    if op in ("delta", "step"):
        step = op == "step"
        n = np.ones(case["batch"], np.int64) if step else _lengths(case)
        t, heads, qk, dk, dv = int(n.sum()), case["heads"], case["qk"], case["dk"], case["dv"]

        def unit(*shape):
            return torch.nn.functional.normalize(torch.randn(shape, generator=gen, device="cuda"),
                                                 dim=-1).to(TYPES[case["type"]])

        s.update(q=unit(t, qk, dk), k=unit(t, qk, dk), v=normal(t, heads, dv), scale=1.0, lens=n)
        s["beta"] = torch.sigmoid(torch.randn((t, heads), generator=gen, device="cuda"))
        if case["decay"] == "token":  # a gate's logits, most heads slow and some fast
            rate = torch.rand(heads, generator=gen, device="cuda") * 0.2
            s["log_decay"] = -torch.nn.functional.softplus(torch.randn((t, heads), generator=gen, device="cuda")) * rate
        else:  # a horizon of 32 to 8192 tokens for each head
            s["log_decay"] = torch.log1p(-torch.exp2(-torch.linspace(5, 13, heads, device="cuda")))
            s["log_decay"] = s["log_decay"] * (0.9 + 0.2 * torch.rand(heads, generator=gen, device="cuda"))
        s["state"] = None
        if step or case["initial"]:
            s["state"] = torch.randn((case["batch"], heads, dk, dv), generator=gen, device="cuda")
        # the state after the step goes to a buffer of its own, as where a step may be taken back
        s["state_out"] = torch.empty((case["batch"], heads, dk, dv), device="cuda")
        if not step:
            cu = np.concatenate([[0], np.cumsum(n)])
            s["cu"] = ints(cu)
            # where token i of sequence b lies in the packed inputs, and where it comes from
            most = _pages(int(n.max()), CHUNK) * CHUNK
            at = np.arange(most)[None]
            s["gather"] = torch.from_numpy(np.where(at < n[:, None], cu[:-1, None] + at, t)).to("cuda")
            row = np.repeat(np.arange(case["batch"]), n)
            s["back"] = torch.from_numpy(row * most + np.arange(t) - cu[row]).to("cuda")
        if own:
            import weight_only_int4_w4a16_amd as w
            s["out"] = torch.empty_like(s["v"])
            if not step:
                s["workspace"] = w.delta_rule_workspace(s["q"], s["v"], case["batch"])
        return s
    heads, page = case.get("kv", case["heads"]), case["page"]
    if op == "store":
        c, n = _requests(case)
        t, pages = int(n.sum()), _stored(case)
        order = np.random.RandomState(case["salt"] + 2).permutation(pages)
        slots, used = [], 0
        for b in range(case["batch"]):
            pos = np.arange(c[b], c[b] + n[b])
            if n[b]:
                slots.append(order[used + pos // page - c[b] // page] * page + pos % page)
                used += int(_pages(c[b] + n[b], page) - c[b] // page)
        slots.append(np.full(5, -1))  # a step padded to a size of its own
        s.update(k=normal(t + 5, heads, case["dim"]), v=normal(t + 5, heads, case["dim"]),
                 slots=ints(np.concatenate(slots)), all=torch.arange(pages * page, device="cuda", dtype=torch.int32))
    elif op == "load":
        pages = _pages(case["tokens"], page) + 3
        pos = torch.arange(case["tokens"], device="cuda")
        s["slots"] = (torch.randperm(pages, generator=gen, device="cuda")[pos // page] * page + pos % page).to(torch.int32)
    else:
        n = _lengths(case)
        each = _pages(n, page)
        pages, blocks = int(each.sum()) + 3, max(1, int(each.max()))
        table = torch.full((case["batch"], blocks), -1, dtype=torch.int32, device="cuda")
        held = torch.arange(blocks, device="cuda")[None] < ints(each)[:, None]
        table[held] = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)[:int(each.sum())]
        s.update(q=normal(case["batch"], case["heads"], case["dim"]), table=table, lens=ints(n), scale=case["dim"] ** -0.5)
    for name in ("k", "v"):
        s[name + "_cache"], s[name + "_scale"] = _cache(case, pages, heads, gen)
    if own:
        import weight_only_int4_w4a16_amd as w
        if op == "attend":
            s["workspace"] = w.quantized_attention_workspace(s["q"], s["k_cache"])
            s["out"] = torch.empty_like(s["q"])
            s["sums"] = torch.empty(s["q"].shape[:2], device="cuda") if case["lse"] else None
        else:
            rows = s["all"] if op == "store" else s["slots"]
            s["out"] = tuple(torch.empty((rows.numel(), heads, case["dim"]), dtype=TYPES[case["type"]], device="cuda")
                             for _ in range(2))
    return s


# ---- one pass ------------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _plain_delta(s):
    batch, heads, dk, dv = s["batch"], s["heads"], s["dk"], s["dv"]
    at = s["gather"]
    share = heads // s["qk"]
    blocks = at.shape[1] // CHUNK

    def padded(x):  # [blocks, batch, heads, CHUNK, dim], zeros past a sequence's end
        x = torch.cat([x, torch.zeros_like(x[:1])])[at]
        return x.reshape(batch, blocks, CHUNK, x.shape[2], -1).permute(1, 0, 3, 2, 4).contiguous()

    q = padded(s["q"].float()).repeat_interleave(share, 2) * s["scale"]
    k = padded(s["k"].float()).repeat_interleave(share, 2)
    v = padded(s["v"].float())
    beta = padded(s["beta"])
    inner = padded(s["log_decay"].expand(s["v"].shape[0], heads).double()).cumsum(3)   # from a block's start
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    weight = torch.where(low, inner - inner.transpose(-1, -2), -math.inf).exp().float()
    kt = k.transpose(-1, -2).contiguous()
    score = torch.matmul(q, kt) * weight
    # the block's triangular system, (1 + lower) u = beta (v - decay k S): its inverse, row by row
    lower = torch.where(low.tril(-1), torch.matmul(k, kt) * weight * beta, 0.0)
    inverse = torch.eye(CHUNK, device=q.device).expand(lower.shape).clone()
    for i in range(1, CHUNK):
        inverse[..., i, :i] = -torch.matmul(lower[..., i:i + 1, :i], inverse[..., :i, :i].contiguous())[..., 0, :]
    inverse = inverse * beta.transpose(-1, -2)
    from_start = inner.exp().float()
    kt = kt * (inner[..., -1:, :] - inner).exp().float().transpose(-1, -2)
    state = torch.zeros(batch, heads, dk, dv, device=q.device) if s["state"] is None else s["state"]
    out = torch.empty_like(v)
    for i in range(blocks):
        u = torch.matmul(inverse[i], v[i] - from_start[i] * torch.matmul(k[i], state))
        out[i] = from_start[i] * torch.matmul(q[i], state) + torch.matmul(score[i], u)
        state = from_start[i][..., -1:, :] * state + torch.matmul(kt[i], u)
    o = out.permute(1, 0, 3, 2, 4).reshape(-1, heads, dv)[s["back"]]
    return {"out": o.to(s["v"].dtype), "state": state}


def _own_delta(s):
    import weight_only_int4_w4a16_amd as w
    o, state = w.delta_rule(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], cu_seqlens=s["cu"], state=s["state"],
                            state_out=s["state_out"], scale=s["scale"], out=s["out"], workspace=s["workspace"])
    return {"out": o, "state": state}


def _plain_step(s):
    share = s["heads"] // s["qk"]
    q = s["q"].float().repeat_interleave(share, 1) * s["scale"]
    k = s["k"].float().repeat_interleave(share, 1)
    state = s["state"] * s["log_decay"].expand(s["batch"], s["heads"]).exp()[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (k[..., :, None] * state).sum(-2))
    state = state + k[..., :, None] * u[..., None, :]
    o = (q[..., :, None] * state).sum(-2)
    return {"out": o.to(s["v"].dtype), "state": state}


def _own_step(s):
    import weight_only_int4_w4a16_amd as w
    o = w.delta_rule_step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["state"], state_out=s["state_out"],
                          scale=s["scale"], out=s["out"])
    return {"out": o, "state": s["state_out"]}


def _codes(x, kind):
    """The nearest codes to float64 values in units of the scale. Many lie next to a border, as their scale comes
    from one of them, so they are not rounded to float32 on the way."""
    x = x.clamp(-MOST[kind], MOST[kind])
    if kind == "int8":
        return x.round().to(torch.int8)
    last = torch.exp2((torch.frexp(x)[1].clamp(min=-5) - 4).double())  # of four bits; subnormal codes share one
    return ((x / last).round() * last).to(TYPES["fp8"])


def _values(codes):
    return codes.float() if codes.dtype == torch.int8 else codes.view(torch.uint8).view(TYPES["fp8"]).float()


def _plain_store(s):
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    slot = s["slots"][live].long()
    page, block, kind = s["page"], s["block"], s["cache"]
    got = {}
    for name in ("k", "v"):
        x, cache, scale = s[name][live].float(), s[name + "_cache"], s[name + "_scale"]
        heads = x.shape[1]
        at = slot // block                                      # blocks one after the other
        old = scale.reshape(-1, heads)
        most = torch.zeros_like(old).index_reduce(0, at, x.abs().amax(-1), "amax")
        some = torch.zeros(old.shape[0], dtype=torch.bool, device=x.device)
        fresh = some.index_fill(0, at[slot % block == 0], True)[:, None]
        some = some.index_fill(0, at, True)[:, None]
        new = (most.double() / MOST[kind]).float().clamp(min=LEAST)  # values next to a border go by its last bit
        new = torch.where(some, torch.where(fresh, new, torch.maximum(new, old)), old)
        # what a block held goes over to its new scale
        held = _values(cache).reshape(-1, block, heads, s["dim"])
        factor = torch.where(fresh | (new == old), 1.0, old.double() / new.double())[:, None, :, None]
        codes = _codes(held.double() * factor, kind).reshape(cache.shape)
        raw = torch.uint8
        codes.view(raw)[slot // page, slot % page] = _codes(x.double() / new[at].double()[..., None], kind).view(raw)
        cache.view(raw).copy_(codes.view(raw))
        scale.copy_(new.reshape(scale.shape))
        value = _values(codes).reshape(-1, block, heads, s["dim"]) * new[:, None, :, None]
        got[name] = value.reshape(-1, heads, s["dim"]).to(TYPES[s["type"]])
        got[name + "_scale"] = scale
    return got


def _own_store(s):
    import weight_only_int4_w4a16_amd as w
    w.quantized_kv_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"])
    k, v = w.quantized_kv_read(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["all"], out=s["out"])
    return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_load(s):
    slot = s["slots"].long()
    got = {}
    for name in ("k", "v"):
        codes = s[name + "_cache"].view(torch.uint8)[slot // s["page"], slot % s["page"]].view(TYPES[s["cache"]])
        scale = s[name + "_scale"][slot // s["page"], slot % s["page"] // s["block"]]
        got[name] = (_values(codes) * scale[..., None]).to(TYPES[s["type"]])
    return got


def _own_load(s):
    import weight_only_int4_w4a16_amd as w
    k, v = w.quantized_kv_read(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"], out=s["out"])
    return {"k": k, "v": v}


def _plain_attend(s):
    batch, heads, dim = s["q"].shape
    kv, page = s["kv"], s["page"]
    at = s["table"].long().clamp(min=0)
    rows = []
    for name in ("k", "v"):
        codes = s[name + "_cache"].view(torch.uint8)[at].view(TYPES[s["cache"]])
        scale = s[name + "_scale"][at].repeat_interleave(s["block"], 2)
        rows.append((_values(codes) * scale[..., None]).reshape(batch, -1, kv, dim))
    k, v = rows
    q = s["q"].float().reshape(batch, kv, heads // kv, dim)
    x = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * s["scale"]
    pos, n = torch.arange(k.shape[1], device=q.device)[None], s["lens"][:, None]
    seen = pos < n
    if s["window"]:
        seen = seen & (pos >= n - s["window"])
    x = torch.where(seen[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, :, None, None], v, 0.0)
    o = torch.matmul(p, v.permute(0, 2, 1, 3).contiguous()) / total.clamp(min=1e-30)
    o = o.reshape(batch, heads, dim).to(s["q"].dtype)
    return {"out": o, "lse": (top + total.log()).reshape(batch, heads)} if s["lse"] else {"out": o}


def _own_attend(s):
    import weight_only_int4_w4a16_amd as w
    o = w.quantized_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                              scale=s["scale"], window=s["window"], out=s["out"], lse=s["sums"], workspace=s["workspace"])
    return {"out": o, "lse": s["sums"]} if s["lse"] else {"out": o}


_plain = {"delta": _plain_delta, "step": _plain_step, "store": _plain_store, "load": _plain_load, "attend": _plain_attend}
_own = {"delta": _own_delta, "step": _own_step, "store": _own_store, "load": _own_load, "attend": _own_attend}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _nearest(x, kind):
    """Values in units of the scale to the nearest that a code has, ties to the even one."""
    x = x.clamp(-MOST[kind], MOST[kind])
    if kind == "int8":
        return x.round()
    unit = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)  # 3 bits behind the first
    unit = torch.where(x.abs() >= unit * 16, unit * 2, torch.where(x.abs() < unit * 8, (unit / 2).clamp(min=2.0 ** -9), unit))
    return (x / unit).round() * unit


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "store":
        got = {}
        slots = s["slots"].tolist()
        for name in ("k", "v"):
            x, scale = s[name].double(), s[name + "_scale"].double()
            flat = _values(s[name + "_cache"]).double().reshape(-1, case["heads"], case["dim"])
            steps = scale.reshape(-1, case["heads"])
            first = 0
            while first < len(slots):  # runs of tokens that follow each other in a block
                end = first + 1
                if slots[first] < 0:
                    first = end
                    continue
                at = slots[first] // case["block"]
                while end < len(slots) and slots[end] == slots[end - 1] + 1 and slots[end] // case["block"] == at:
                    end += 1
                new = (x[first:end].abs().amax((0, 2)) / MOST[case["cache"]]).clamp(min=LEAST).float().double()
                rows = flat[at * case["block"]:(at + 1) * case["block"]]
                if slots[first] % case["block"]:
                    new = torch.maximum(new, steps[at])
                    rows[:] = torch.where((new > steps[at])[:, None],
                                          _nearest(rows * (steps[at] / new)[:, None], case["cache"]), rows)
                steps[at] = new
                flat[slots[first]:slots[end - 1] + 1] = _nearest(x[first:end] / new[:, None], case["cache"])
                first = end
            got[name] = flat * steps.repeat_interleave(case["block"], 0)[..., None]
            got[name + "_scale"] = steps.reshape(scale.shape)
        return got
    if op == "load":
        got = {}
        for name in ("k", "v"):
            values = _values(s[name + "_cache"]).double() * s[name + "_scale"].double().repeat_interleave(
                case["block"], 1)[..., None]
            got[name] = values.reshape(-1, case["heads"], case["dim"])[s["slots"].long()]
        return got
    if op == "attend":
        out, lse = [], []
        group = case["heads"] // case["kv"]
        for b, n in enumerate(_lengths(case).tolist()):
            lo = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                out.append(torch.zeros(case["heads"], case["dim"], dtype=torch.float64, device="cuda"))
                lse.append(torch.full((case["heads"],), -math.inf, dtype=torch.float64, device="cuda"))
                continue
            pos = torch.arange(lo, n, device="cuda")
            where, off = s["table"][b, pos // case["page"]].long(), pos % case["page"]
            rows = []
            for name in ("k", "v"):
                x = _values(s[name + "_cache"].view(torch.uint8)[where, off].view(TYPES[case["cache"]])).double()
                rows.append(x * s[name + "_scale"][where, off // case["block"]].double()[..., None])
            heads, sums = [], []
            for h in range(case["kv"]):
                x = s["q"][b, h * group:(h + 1) * group].double() @ rows[0][:, h].T.contiguous() * s["scale"]
                sums.append(torch.logsumexp(x, -1))
                heads.append(torch.softmax(x, -1) @ rows[1][:, h].contiguous())
            out.append(torch.cat(heads))
            lse.append(torch.cat(sums))
        return {"out": torch.stack(out), "lse": torch.stack(lse)} if case["lse"] else {"out": torch.stack(out)}
    # the recurrence, one token after the other, all sequences side by side
    n = torch.from_numpy(s["lens"]).to("cuda")
    share = case["heads"] // case["qk"]
    start = torch.cumsum(n, 0) - n
    state = torch.zeros((case["batch"], case["heads"], case["dk"], case["dv"]), dtype=torch.float64, device="cuda")
    if s["state"] is not None:
        state += s["state"].double()
    t = s["v"].shape[0]
    out = torch.zeros((t + 1, case["heads"], case["dv"]), dtype=torch.float64, device="cuda")
    q, k, v, beta = (torch.cat([s[x], s[x][:1]]).double() for x in ("q", "k", "v", "beta"))
    g = s["log_decay"].double().expand(t, case["heads"])
    g = torch.cat([g, g[:1]]).exp()
    for i in range(int(n.max())):
        live = i < n
        at = torch.where(live, start + i, t)
        ki = k[at].repeat_interleave(share, 1)
        state = state * torch.where(live[:, None], g[at], 1.0)[..., None, None]
        u = torch.where(live[:, None], beta[at], 0.0)[..., None] * (v[at] - torch.matmul(ki[..., None, :], state)[..., 0, :])
        state = state + ki[..., :, None] * u[..., None, :]
        qi = q[at].repeat_interleave(share, 1) * s["scale"]
        out[at] = torch.matmul(qi[..., None, :], state)[..., 0, :]
    return {"out": out[:t], "state": state}
