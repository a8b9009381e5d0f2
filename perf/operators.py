"""Timed cases of the operators of a single-token serving step.

Three operators that one step of a server calls one after another:

  blocks    fdllm_plan_blocks / fdllm_release_blocks: block tables, positions and slot maps from
            the requests' lengths, pages taken from and given back to a free list, on the GPU
  attend    fdllm_decode_attention: one new token per sequence over the paged cache: RoPE of its
            q and k, its k and v into their slot, attention over the visible slots
  linear    fdllm_linear: y = residual + act(x W + b), or residual + act(x Wg + bg) * (x W + b)

`run` computes a case in its plain form (elementary torch operations in 32 bits, RoPE in 64) or,
with `own` true, through this framework's calls. `exact` is the operators' definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _blocks(name, kind, batch, page, past, new, cap_extra=0):
    """past / new: the largest context and the largest number of new tokens of a request;
    new = 1 is a decode step (every request gets one token)."""
    return {"name": name, "op": "blocks", "kind": kind, "batch": batch, "page": page,
            "past": past, "new": new, "cap_extra": cap_extra}


def _attend(name, dtype, batch, kv_heads, group, dim, page, lo, hi, starts=False):
    """lo, hi: range of the visible lengths, the new token included."""
    return {"name": name, "op": "attend", "dtype": dtype, "batch": batch, "kv_heads": kv_heads,
            "group": group, "dim": dim, "page": page, "lo": lo, "hi": hi, "starts": starts}


def _linear(name, rows, n_in, n_out, act="none", bias="", gate=False, residual=False, pad=0):
    """bias: "", "bf16" or "f32"; pad: extra columns between the rows of x."""
    return {"name": name, "op": "linear", "rows": rows, "n_in": n_in, "n_out": n_out, "act": act,
            "bias": bias, "gate": gate, "residual": residual, "pad": pad}


def listed():
    return [
        # one token for each of 32 running requests: what every decode step begins with (latency)
        _blocks("blocks_step_b32", "plan", 32, 64, 1024, 1),
        # a scheduler's largest mixed step: ragged prompts of up to 4095 tokens, many requests
        _blocks("blocks_prompts_b509", "plan", 509, 64, 4096, 4095, cap_extra=77),
        # rejected drafts and finished requests of a large server give their pages back; small pages
        _blocks("blocks_release_b1000", "release", 1000, 6, 2048, 2048),
        # one user: the LLaDA-8B layer's heads over its 768-slot cache (latency)
        _attend("attend_b1_768", "bf16", 1, 32, 1, 128, 64, 768, 768),
        # the divergent batch of 32: lengths of 256 to 1024
        _attend("attend_b32_divergent", "bf16", 32, 32, 1, 128, 64, 256, 1024),
        # two very long documents, 8 key-value heads under 32 query heads (split over the length)
        _attend("attend_b2_long", "bf16", 2, 8, 4, 128, 64, 120001, 131071),
        # fp32 cache, 6-slot pages, three query heads a key head, and slots dropped at the front
        _attend("attend_f32_b61_odd", "f32", 61, 4, 3, 96, 6, 1, 2999, starts=True),
        # one token through a square projection, onto the residual stream (latency)
        _linear("linear_b1", 1, 4096, 4096, residual=True),
        # the feed-forward's two input projections for 32 running requests: the weights' bytes
        _linear("gated_b32", 32, 4096, 12288, act="silu", gate=True),
        # odd sizes, a strided x, an fp32 bias and a residual
        _linear("linear_odd", 1001, 1304, 2696, act="relu", bias="f32", residual=True, pad=24),
        # the same two projections for the 1536 rows of the divergent batch
        _linear("gated_1536", 1536, 4096, 12288, act="silu", gate=True),
        # a prompt of 8192 tokens: the tensor cores' rate
        _linear("linear_8192", 8192, 4096, 12288, act="gelu", bias="bf16"),
    ]


_MOST_FLOPS = 2.0 * 8192 * 4096 * 12288
_MOST_SLOTS = 2 * 131071 * 8 * 128 * 2        # bytes of K of the largest listed attention


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("blocks", "attend", "attend", "linear", "linear"))
    if op == "blocks":
        kind = rng.choice(("plan", "plan", "release"))
        batch = _log(rng, 1, 1000)
        past = _log(rng, 1, 4096)
        new = rng.choice((1, past)) if kind == "plan" else past
        new = max(1, min(new, 1000000 // batch))
        c = _blocks("", kind, batch, rng.choice((1, 6, 16, 64, 100)), past, new, rng.randrange(0, 300))
    elif op == "attend":
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        batch = _log(rng, 1, 96)
        kv = rng.choice((1, 2, 4, 8, 32))
        group = rng.choice((1, 2, 3, 4, 7, 8, 12))
        dim = rng.choice((32, 64, 96, 128, 128))
        size = 2 if dtype == "bf16" else 4
        # (at least three quarters of the largest listed case's bytes are never passed)
        top = min(131071, _MOST_SLOTS // (batch * kv * dim * size * 2))
        hi = max(1, _log(rng, 16, max(17, top)))
        c = _attend("", dtype, batch, kv, group, dim, rng.choice((6, 16, 64, 64, 128)),
                    rng.choice((1, max(1, hi // 2), hi)), hi, rng.random() < 0.3)
    else:
        gate = rng.random() < 0.4
        n_in, n_out = 8 * _log(rng, 16, 1536), 8 * _log(rng, 16, 1536)
        rows = _log(rng, 1, 8192)
        rows = max(1, min(rows, int(_MOST_FLOPS / (2 * n_in * n_out * (2 if gate else 1)))))
        c = _linear("", rows, n_in, n_out, rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")),
                    rng.choice(("", "bf16", "f32")), gate, rng.random() < 0.5,
                    rng.choice((0, 0, 8, 40)))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _lens(rs, lo, hi, n):
    """n lengths spread evenly over lo .. hi (one alone: hi), in an order of the seed's."""
    return rs.permutation(np.linspace(hi if n == 1 else lo, hi, n).round()).astype(np.int32)


def prepare(case, seed):
    return {"blocks": _prepare_blocks, "attend": _prepare_attend, "linear": _prepare_linear}[
        case["op"]](case, seed)


def _prepare_blocks(c, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    B, ps = c["batch"], c["page"]
    lens = _lens(rs, 0, c["past"], B)
    if c["kind"] == "plan":
        new = np.ones(B, np.int32) if c["new"] == 1 else _lens(rs, 0, c["new"], B)
        top = c["past"] + c["new"]
    else:
        new = (lens * rs.rand(B)).astype(np.int32)                              # tokens kept
        new[rs.rand(B) < 0.3] = 0                                               # finished requests
        top = c["past"]
    width = -(-top // ps) + 1
    held = -(-lens // ps)
    need = (-(-(lens + new) // ps) - held) if c["kind"] == "plan" else np.zeros(B, np.int64)
    # one page in sixteen too few for prompts: the last requests are refused
    spare = int(need.sum()) if c["new"] == 1 else max(1, int(need.sum() * 15 // 16))
    pages = rs.permutation(B * width).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    own_pages = np.arange(width)[None, :] < held[:, None]
    table[own_pages] = pages[:int(held.sum())]
    free = np.full(pages.size, -1, np.int32)
    free[:spare] = pages[int(held.sum()):int(held.sum()) + spare]
    cap = (int(new.sum()) if c["kind"] == "plan" else 0) + c["cap_extra"]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    i32 = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"op": "blocks", "kind": c["kind"], "page": ps, "seq_lens": dev(lens), "new": dev(new),
            "table": dev(table), "free": dev(free),
            "n_free": torch.tensor([spare], dtype=torch.int32, device="cuda"),
            "out": {"cu_rows": i32(B + 1), "positions": i32(cap), "slots": i32(cap),
                    "row_seq": i32(cap),
                    "slot_map": torch.full((cap,), -7, dtype=torch.int64, device="cuda"),
                    "seq_lens": i32(B), "granted": i32(B), "n_free": i32(1)}}


def _prepare_attend(c, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    g = _gen(seed)
    B, hk, D, ps = c["batch"], c["kv_heads"], c["dim"], c["page"]
    hq, dt = hk * c["group"], DT[c["dtype"]]
    lens = _lens(rs, c["lo"], c["hi"], B)
    width = -(-c["hi"] // ps)
    held = -(-lens // ps)
    n_pages = B * width
    pages = rs.permutation(n_pages).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    table[np.arange(width)[None, :] < held[:, None]] = pages[:int(held.sum())]
    shape = (1, n_pages, hk, ps, D)
    # keys of the scale that a projection of normalised activations gives
    k_pool = torch.randn(shape, generator=g, device="cuda", dtype=dt).mul_(1.28)
    v_pool = torch.randn(shape, generator=g, device="cuda", dtype=dt).mul_(1.28)
    qkv = torch.randn(B, (hq + 2 * hk) * D, generator=g, device="cuda", dtype=dt).mul_(1.28)
    angle = (torch.arange(c["hi"], dtype=torch.float64, device="cuda")[:, None]
             * 10000.0 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device="cuda") / D))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    starts = None
    if c["starts"]:
        first = np.where(rs.rand(B) < 0.5, 0, (lens * rs.rand(B)).astype(np.int32))
        first[rs.rand(B) < 0.05] = c["hi"]                                # nothing visible
        starts = dev(first.astype(np.int32))
    return {"op": "attend", "q": qkv[:, :hq * D], "k": qkv[:, hq * D:(hq + hk) * D],
            "v": qkv[:, (hq + hk) * D:], "k_pool": k_pool, "v_pool": v_pool, "table": dev(table),
            "seq_lens": dev(lens), "positions": dev(lens - 1), "cos": torch.cos(angle),
            "sin": torch.sin(angle), "starts": starts}


def _prepare_linear(c, seed):
    g = _gen(seed)
    n, i, o = c["rows"], c["n_in"], c["n_out"]
    bf = torch.bfloat16
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=bf)  # noqa: E731
    x = rnd(n, i + c["pad"])[:, :i]
    s = {"op": "linear", "x": x, "w": rnd(i, o).mul_(i ** -0.5), "act": c["act"], "b": None,
         "wg": None, "bg": None, "r": None}
    if c["gate"]:
        s["wg"] = rnd(i, o).mul_(i ** -0.5)
    if c["bias"]:
        s["b"] = rnd(o).mul_(0.5).to(DT[c["bias"]])
        if c["gate"]:
            s["bg"] = rnd(o).mul_(0.5).to(DT[c["bias"]])
    if c["residual"]:
        s["r"] = rnd(n, o)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"blocks": _plain_blocks, "attend": _plain_attend, "linear": _plain_linear}[state["op"]](state)


def _run_own(s):
    import kv_cache_attention_flash_b200 as fd
    if s["op"] == "linear":
        return fd.fdllm_linear(s["x"], s["w"], bias=s["b"], act=s["act"], w_gate=s["wg"],
                               bias_gate=s["bg"], residual=s["r"])
    if s["op"] == "attend":
        out, lse = fd.fdllm_decode_attention(
            s["q"], s["k_pool"], s["v_pool"], 0, s["table"], s["seq_lens"], k=s["k"], v=s["v"],
            positions=s["positions"], rope_cos=s["cos"], rope_sin=s["sin"], starts=s["starts"],
            out_dtype=s["q"].dtype, with_lse=True)
        return out, lse, s["k_pool"], s["v_pool"]
    if s["kind"] == "plan":
        p = fd.fdllm_plan_blocks(s["seq_lens"], s["new"], s["table"], s["page"], s["free"],
                                 s["n_free"], out=s["out"])
        return (p["cu_rows"], p["positions"], p["slots"], p["row_seq"], p["slot_map"],
                p["seq_lens"], p["granted"], p["n_free"], s["table"])
    p = fd.fdllm_release_blocks(s["seq_lens"], s["new"], s["table"], s["page"], s["free"],
                                s["n_free"], out=s["out"])
    return p["seq_lens"], p["n_free"], s["free"]


def _plain_blocks(s):
    ps, lens, table, free = s["page"], s["seq_lens"].long(), s["table"], s["free"]
    n_free = s["n_free"].long()
    held = (lens + ps - 1) // ps
    if s["kind"] == "release":
        keep = torch.minimum(s["new"].long(), lens)
        kept = (keep + ps - 1) // ps
        given = held - kept
        before = torch.cumsum(given, 0) - given
        page = torch.arange(table.shape[1], device=table.device)
        gone = (page >= kept[:, None]) & (page < held[:, None])
        at = n_free + before[:, None] + page - kept[:, None]
        at = torch.where(gone, at, free.numel())
        longer = torch.cat([free, free.new_zeros(1)])          # the last place takes what is not given
        longer[at] = table
        free.copy_(longer[:-1])
        return keep.int(), (n_free + given.sum()).int(), free
    new = s["new"].long()
    after = lens + new
    need = (after + ps - 1) // ps - held
    upto = torch.cumsum(need, 0)
    granted = (need == 0) | (upto <= n_free)
    # (a request that needs no page is granted after refused ones, whose pages `upto` counts)
    taken = torch.where(granted & (need > 0), upto, 0).amax(0, keepdim=True)
    page = torch.arange(table.shape[1], device=table.device)
    fresh = (page >= held[:, None]) & (page < (held + need)[:, None]) & granted[:, None]
    at = n_free - 1 - ((upto - need)[:, None] + page - held[:, None])
    table.copy_(torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table))
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    row = torch.arange(s["out"]["positions"].numel(), device=table.device)
    b = torch.searchsorted(cu[1:], row, right=True)
    there = b < lens.numel()
    b = b.clamp(max=lens.numel() - 1)
    pos = lens[b] + row - cu[b]
    ok = granted[b]
    at = table[b, (pos // ps).clamp(0, table.shape[1] - 1)].long() * ps + pos % ps
    put = lambda name, v: torch.where(there, v, s["out"][name]).to(s["out"][name].dtype)  # noqa: E731
    return (cu.int(), put("positions", pos), put("slots", torch.where(ok, pos, -1)),
            put("row_seq", b), put("slot_map", torch.where(ok, at, -1)),
            torch.where(granted, after, lens).int(), granted.int(), (n_free - taken).int(), table)


def _rotated(x, cos, sin):
    """Rotate-half RoPE in 64 bits: x [B, heads, D], cos / sin [B, 1, D / 2]."""
    a, b = x.double().chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_attend(s):
    kp, vp, table = s["k_pool"], s["v_pool"], s["table"].long()
    B, (hk, ps, D) = table.shape[0], kp.shape[2:]
    pos = s["positions"].long()
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    q = _rotated(s["q"].reshape(B, -1, D), cos, sin).float().reshape(B, hk, -1, D)
    k = _rotated(s["k"].reshape(B, hk, D), cos, sin).to(kp.dtype)
    page = table.gather(1, (pos // ps)[:, None])[:, 0]
    kp[0, page, :, pos % ps] = k
    vp[0, page, :, pos % ps] = s["v"].reshape(B, hk, D)
    width = table.shape[1]
    keys = kp[0][table.clamp(min=0)].float().transpose(1, 2).reshape(B, hk, width * ps, D)
    values = vp[0][table.clamp(min=0)].float().transpose(1, 2).reshape(B, hk, width * ps, D)
    slot = torch.arange(width * ps, device=kp.device)
    seen = slot < s["seq_lens"][:, None]
    if s["starts"] is not None:
        seen = seen & (slot >= s["starts"][:, None])
    seen = seen[:, None, None]
    score = (q @ keys.transpose(2, 3)) * D ** -0.5
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    o = (e @ values) / torch.where(total == 0, 1.0, total)
    lse = (torch.log(total) + top).reshape(B, -1)
    return o.reshape(B, -1).to(s["q"].dtype), lse, kp, vp


def _activated(x, act):
    if act == "relu":
        return torch.where(x > 0, x, 0.0)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh((2 / math.pi) ** 0.5 * (x + 0.044715 * x * x * x)))
    return x


def _plain_linear(s):
    x = s["x"].float()
    y = x @ s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    if s["wg"] is not None:
        a = x @ s["wg"].float()
        if s["bg"] is not None:
            a = a + s["bg"].float()
        y = _activated(a, s["act"]) * y
    else:
        y = _activated(y, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ what it cannot do without
def work(case):
    c = case
    if c["op"] == "blocks":
        # lengths in and out, the table's new or given-back entries, and 20 bytes for each row
        rs_rows = 0 if c["kind"] == "release" else c["batch"] * (1 if c["new"] == 1 else c["new"] / 2)
        moved = c["batch"] * (c["past"] / 2 if c["kind"] == "release" else
                              (1 if c["new"] == 1 else c["new"] / 2)) / c["page"]
        return {"bytes": 24 * c["batch"] + 8 * moved + 20 * rs_rows, "flops": 0}
    if c["op"] == "attend":
        size = 2 if c["dtype"] == "bf16" else 4
        hq = c["kv_heads"] * c["group"]
        slots = c["batch"] * (c["lo"] + c["hi"]) / 2 * (0.75 if c["starts"] else 1.0)
        io = c["batch"] * c["dim"] * (2 * hq + 4 * c["kv_heads"]) * size
        return {"bytes": slots * c["kv_heads"] * c["dim"] * 2 * size + io,
                "flops": 4.0 * slots * hq * c["dim"]}
    n, i, o, two = c["rows"], c["n_in"], c["n_out"], 2 if c["gate"] else 1
    bias = {"": 0, "bf16": 2, "f32": 4}[c["bias"]]
    return {"bytes": 2 * (n * i + two * i * o + n * o * (2 if c["residual"] else 1)) + two * bias * o,
            "flops": 2.0 * n * i * o * two}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"blocks": _exact_blocks, "attend": _exact_attend, "linear": _exact_linear}[s["op"]](s)


def _exact_blocks(s):
    """Request by request on the host."""
    ps = s["page"]
    lens, new, table, free = (s[n].cpu().numpy().copy() for n in ("seq_lens", "new", "table", "free"))
    left = int(s["n_free"].item())
    if s["kind"] == "release":
        for b in range(len(lens)):
            for p in range(-(-int(new[b]) // ps), -(-int(lens[b]) // ps)):
                free[left] = table[b, p]
                left += 1
        return new, np.array([left], np.int32), free
    o = {k: v.cpu().numpy().copy() for k, v in s["out"].items()}
    wanted, at, budget = 0, 0, left
    o["cu_rows"][0] = 0
    for b in range(len(lens)):
        first, last = -(-int(lens[b]) // ps), -(-int(lens[b] + new[b]) // ps)
        ok = last == first or wanted + last - first <= budget
        if ok:
            for p in range(first, last):
                table[b, p] = free[budget - 1 - wanted - (p - first)]
            if last > first:
                left = budget - wanted - (last - first)
        wanted += last - first
        pos = np.arange(lens[b], lens[b] + new[b])
        rows = slice(at, at + len(pos))
        o["positions"][rows], o["row_seq"][rows] = pos, b
        o["slots"][rows] = pos if ok else -1
        o["slot_map"][rows] = table[b, pos // ps].astype(np.int64) * ps + pos % ps if ok else -1
        at += len(pos)
        o["cu_rows"][b + 1], o["granted"][b] = at, ok
        o["seq_lens"][b] = lens[b] + (new[b] if ok else 0)
    return (o["cu_rows"], o["positions"], o["slots"], o["row_seq"], o["slot_map"], o["seq_lens"],
            o["granted"], np.array([left], np.int32), table)


def _exact_attend(s):
    """Sequence by sequence, RoPE as a product of complex numbers; the new key and value enter as
    the cache's type holds them."""
    kp, vp = s["k_pool"], s["v_pool"]
    B, (hk, ps, D) = s["table"].shape[0], kp.shape[2:]
    out, lse = [], []
    turn = torch.complex(s["cos"], s["sin"])
    for b in range(B):
        n, p = int(s["seq_lens"][b]), int(s["positions"][b])
        def turned(x):
            x = x.double().reshape(-1, 2, D // 2)
            z = torch.complex(x[:, 0], x[:, 1]) * turn[p]
            return torch.cat([z.real, z.imag], 1)
        page = int(s["table"][b, p // ps])
        kp[0, page, :, p % ps] = turned(s["k"][b]).to(kp.dtype)
        vp[0, page, :, p % ps] = s["v"][b].reshape(hk, D)
        first = min(n, int(s["starts"][b])) if s["starts"] is not None else 0
        at = torch.arange(first, n, device=kp.device)
        pages = s["table"][b][at // ps].long()
        q = turned(s["q"][b]).reshape(hk, -1, D)
        for h in range(hk):
            sc = (kp[0, pages, h, at % ps].double() @ q[h].T) / D ** 0.5      # [keys, group]
            lse.append(torch.logsumexp(sc, 0))
            out.append(torch.softmax(sc, 0).T @ vp[0, pages, h, at % ps].double())
    return torch.stack(out).reshape(B, -1), torch.stack(lse).reshape(B, -1), kp, vp


def _exact_linear(s):
    act = {"none": lambda a: a, "relu": torch.relu, "silu": torch.nn.functional.silu,
           "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda a: torch.nn.functional.gelu(a, approximate="tanh")}[s["act"]]
    x = s["x"].double()
    up = x @ s["w"].double() + (0 if s["b"] is None else s["b"].double())
    if s["wg"] is None:
        y = act(up)
    else:
        y = act(x @ s["wg"].double() + (0 if s["bg"] is None else s["bg"].double())) * up
    return y if s["r"] is None else y + s["r"].double()
