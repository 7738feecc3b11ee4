"""Timed cases for the serving operators around the attention: rotary positions (forward and backward), the paged
key-value cache (writing, also with 8-bit quantisation, and reading back) and the attention of one new token over it.

Each operator is here in two forms: its plain form in elementary torch operations, and (with ``own`` set) the calls of
this library.  ``exact`` gives the same results from the definitions in 64 bits.

Definitions.
  rope        theta = position[axis(i), t] * base^(-2i/r) for pair i < r/2;  y1 = x1 cos - x2 sin, y2 = x2 cos + x1 sin;
              the pair is (x[i], x[i + r/2]), or (x[2i], x[2i+1]) when interleaved; elements from r on are copied.
              The backward pass rotates by -theta.
  write       row of (sequence b, new token i, head g) goes to position start[b] + i: page table[b, pos / size], slot
              pos % size.  8 bits: a = max(max |x|, 2^-110), scale = a / 448, y = e4m3(x * (448 / a)).
  read        the reverse: bf16(y * scale), or the bf16 row.
  attention   softmax over the first len[b] positions of scale * q . k, times v; the log-sum-exp in log2 units.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of 16 sequences: latency
        dict(name="rope_decode", op="rope", total=16, h_q=32, h_kv=2, d=128, rot=128, axes=1, inter=False, back=False,
             f32=False, far=131072),
        # a 32K prefill with time, height and width positions
        dict(name="rope_prefill_3axes", op="rope", total=32768, h_q=32, h_kv=2, d=128, rot=128, axes=3, inter=False,
             back=False, f32=False, far=32768),
        # the gradients that the attention's backward pass leaves in fp32, odd number of tokens, part of d rotated
        dict(name="rope_backward", op="rope", total=9973, h_q=32, h_kv=2, d=128, rot=96, axes=2, inter=True, back=True,
             f32=True, far=32768),
        # one new token a sequence into an 8-bit cache
        dict(name="write_decode_e4m3", op="write", batch=16, total=16, h_kv=2, d=128, page=64, e4m3=True, start=8192,
             single=True),
        # the keys and values of a 128K packed prefill, quantised as they are written
        dict(name="write_prefill_e4m3", op="write", batch=9, total=131072, h_kv=2, d=128, page=64, e4m3=True, start=0,
             single=False),
        # chunks of an odd number of tokens behind cached prefixes, small pages, many short rows
        dict(name="write_chunk_bf16", op="write", batch=33, total=8209, h_kv=8, d=64, page=16, e4m3=False, start=1500,
             single=False),
        # an 8-bit cached prefix brought back for the sparse prefill
        dict(name="read_prefix_e4m3", op="read", batch=3, total=65521, h_kv=2, d=128, page=64, e4m3=True),
        # short cached prefixes of many sequences
        dict(name="read_ragged_bf16", op="read", batch=64, total=12007, h_kv=2, d=128, page=16, e4m3=False),
        # one short sequence: latency
        dict(name="attn_1x1000", op="attn", batch=1, longest=1000, spread=False, h_q=32, h_kv=2, d=128, page=64,
             e4m3=False),
        # a batch on the dense side of the switch, ragged lengths up to the threshold
        dict(name="attn_64x8k_bf16", op="attn", batch=64, longest=8192, spread=True, h_q=32, h_kv=2, d=128, page=64,
             e4m3=False),
        # many short sequences, small pages, small heads, 8 bits
        dict(name="attn_200x2k_e4m3", op="attn", batch=200, longest=2048, spread=True, h_q=16, h_kv=4, d=64, page=16,
             e4m3=True),
        # the long-context batch, 8 bits
        dict(name="attn_16x128k_e4m3", op="attn", batch=16, longest=131072, spread=False, h_q=32, h_kv=2, d=128,
             page=64, e4m3=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn"])
    d = rng.choice([64, 128])
    h_kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    e4m3 = rng.random() < 0.5
    if op == "rope":
        f32 = rng.random() < 0.4
        return dict(op=op, total=_log(rng, 1, 12000), h_q=h_kv * rng.choice([1, 2, 4]), h_kv=h_kv, d=d,
                    rot=rng.choice([d // 2, d // 2 + 16, d]), axes=rng.choice([1, 2, 3]), inter=rng.random() < 0.4,
                    back=rng.random() < 0.4, f32=f32, far=_log(rng, 1000, 1 << 20))
    if op == "write":
        batch = _log(rng, 1, 256)
        single = rng.random() < 0.4
        return dict(op=op, batch=batch, total=batch if single else _log(rng, batch, 65536), h_kv=h_kv, d=d, page=page,
                    e4m3=e4m3, start=_log(rng, 1, 4000), single=single)
    if op == "read":
        batch = _log(rng, 1, 128)
        return dict(op=op, batch=batch, total=_log(rng, batch, 65536), h_kv=h_kv, d=d, page=page, e4m3=e4m3)
    batch = _log(rng, 1, 256)
    longest = _log(rng, 1, min(131072, (1 << 20) // (batch * h_kv) * (2 if e4m3 else 1) * (128 // d)))
    return dict(op=op, batch=batch, longest=longest, spread=rng.random() < 0.7, h_q=h_kv * rng.choice([1, 2, 4, 8, 16]),
                h_kv=h_kv, d=d, page=page, e4m3=e4m3)


# ------------------------------------------------------------------ inputs
def _sections(rot, axes):
    """Pairs of each axis: a quarter of them for time and the rest shared by height and width, or halves."""
    n = rot // 2
    return {1: [n], 2: [n // 2, n - n // 2], 3: [n // 4, (n - n // 4) // 2, n - n // 4 - (n - n // 4) // 2]}[axes]


def _lengths(total, batch, gen):
    """Random positive lengths of `batch` sequences that sum to `total`."""
    cut = torch.randperm(total - 1, generator=gen)[:batch - 1].add_(1).sort().values
    ends = torch.cat([torch.zeros(1, dtype=torch.int64), cut, torch.tensor([total])])
    return ends


def _quantise(x):
    """Rows of 8-bit values and their scales.  (Tensor by tensor: with a plain number torch multiplies by a rounded
    reciprocal instead of dividing.)"""
    x = x.float()
    a = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -110)
    top = torch.full_like(a, 448.0)
    return (x * (top / a)).to(F8), (a / top).squeeze(-1)


def _pool(case, lens, gen, cpu, poison, most=0):
    """Pages of random keys and values (for `most` tokens at least, spare ones among them), and a table that gives
    every sequence its own pages in random order.  What no sequence has written holds NaN where `poison` is set."""
    page, h_kv, d, batch = case["page"], case["h_kv"], case["d"], len(lens)
    need = [(n + page - 1) // page for n in lens]
    width = max(1, max(need))
    pages = max(sum(need), most // page + batch) + 3
    order = torch.randperm(pages, generator=cpu)
    table = torch.zeros(batch, width, dtype=torch.int64)
    row = torch.repeat_interleave(torch.arange(batch), torch.tensor(need))
    first = torch.cat([torch.zeros(1, dtype=torch.int64), torch.tensor(need).cumsum(0)])
    col = torch.arange(sum(need)) - first[row]
    table[row, col] = order[:sum(need)]
    table = table.to(DEV)
    s = {"table": table.to(torch.int32)}
    written = torch.zeros(pages, page, dtype=torch.bool, device=DEV)
    if sum(need):
        row, col = row.to(DEV), col.to(DEV)
        pos = col[:, None] * page + torch.arange(page, device=DEV)
        written[table[row, col]] = pos < torch.tensor(lens, device=DEV)[row][:, None]
    for name in ("k", "v"):
        x = torch.randn(pages, h_kv, page, d, device=DEV, generator=gen)
        if name == "k":
            x += 0.5 * torch.randn(pages, h_kv, 1, d, device=DEV, generator=gen)
        if case["e4m3"]:
            q, sc = _quantise(x.bfloat16())
            if poison:
                q.view(torch.uint8).masked_fill_(~written[:, None, :, None], 0x7F)
                sc.masked_fill_(~written[:, None, :], math.nan)
            s[name + "_pages"], s[name + "_scale"] = q, sc.contiguous()
        else:
            x = x.bfloat16()
            if poison:
                x.masked_fill_(~written[:, None, :, None], math.nan)
            s[name + "_pages"], s[name + "_scale"] = x, None
    return s


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    s = dict(case=case, op=case["op"])
    if case["op"] == "rope":
        dt = torch.float32 if case["f32"] else torch.bfloat16
        n, d = case["total"], case["d"]
        s["q"] = torch.randn(n, case["h_q"], d, device=DEV, generator=gen).to(dt)
        s["k"] = torch.randn(n, case["h_kv"], d, device=DEV, generator=gen).to(dt)
        s["pos"] = torch.randint(0, case["far"], (case["axes"], n), device=DEV, generator=gen, dtype=torch.int32)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["sections"] = _sections(case["rot"], case["axes"])
    elif case["op"] == "write":
        ends = _lengths(case["total"], case["batch"], cpu)
        start = torch.randint(0, case["start"] + 1, (case["batch"],), generator=cpu)
        most = case["total"] + case["batch"] * case["start"]
        s.update(_pool(case, (start + ends.diff()).tolist(), gen, cpu, False, most))
        s["cu"] = None if case["single"] else ends.to(DEV, torch.int32)
        s["start"] = start.to(DEV, torch.int32)
        for name in ("K", "V"):
            s[name] = torch.randn(case["total"], case["h_kv"], case["d"], device=DEV, generator=gen).bfloat16()
    elif case["op"] == "read":
        ends = _lengths(case["total"], case["batch"], cpu)
        s.update(_pool(case, ends.diff().tolist(), gen, cpu, True))
        s["cu"] = ends.to(DEV, torch.int32)
        for name in ("K", "V"):
            s[name] = torch.empty(case["total"], case["h_kv"], case["d"], device=DEV, dtype=torch.bfloat16)
    else:
        lens = torch.full((case["batch"],), case["longest"])
        if case["spread"]:
            lens = torch.randint(0, case["longest"] + 1, (case["batch"],), generator=cpu)
            lens[0] = case["longest"]
        s.update(_pool(case, lens.tolist(), gen, cpu, True))
        s["len"] = lens.to(DEV, torch.int32)
        s["q"] = torch.randn(case["batch"], case["h_q"], case["d"], device=DEV, generator=gen).bfloat16()
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["batch"], case["h_q"], device=DEV)
    if own:  # the handles and the workspace that a serving program keeps beside its buffers
        import trainable_block_sparse_pool_b200 as T
        s["T"] = T
        if case["op"] == "rope":
            s["rope"] = T.make_rope(case["rot"], sections=s["sections"], interleaved=case["inter"])
        else:
            s["cache"] = T.make_paged_cache(s["k_pages"], s["v_pages"], s["table"], s["k_scale"], s["v_scale"])
        if case["op"] == "attn":
            s["ws"] = torch.empty(T.infllm2_paged_workspace_bytes(s["cache"], case["h_q"]), dtype=torch.uint8,
                                  device=DEV)
    return s


# ------------------------------------------------------------------ the operators
def _rope(s):
    c = s["case"]
    half, n = c["rot"] // 2, c["total"]
    freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=DEV), torch.tensor(s["sections"], device=DEV),
                                   output_size=half)
    theta = s["pos"][axis].t().double() * freq                       # far positions: angles in 64 bits
    cos, sin = theta.cos().float()[:, None], theta.sin().float()[:, None]
    if c["back"]:
        sin = -sin

    def turn(x):
        r = x[..., :c["rot"]].float()
        x1, x2 = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :half], r[..., half:])
        y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
        y = torch.stack([y1, y2], -1).flatten(-2) if c["inter"] else torch.cat([y1, y2], -1)
        return torch.cat([y.to(x.dtype), x[..., c["rot"]:]], -1)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _slots(s):
    """Page and slot of every packed row."""
    n, page = s["K"].shape[0], s["case"]["page"]
    r = torch.arange(n, device=DEV)
    if s["cu"] is None:
        b, i = r, torch.zeros_like(r)
    else:
        b = (torch.searchsorted(s["cu"], r.int(), right=True) - 1)
        i = r - s["cu"][b]
    pos = i + s["start"][b] if "start" in s else i
    return s["table"][b, pos // page].long(), pos % page


def _write(s):
    at, slot = _slots(s)
    for name in ("k", "v"):
        x, pages = s[name.upper()], s[name + "_pages"]
        if s["k_scale"] is None:
            pages[at, :, slot] = x
        else:
            y, sc = _quantise(x)
            pages.view(torch.uint8)[at, :, slot] = y.view(torch.uint8)
            s[name + "_scale"][at, :, slot] = sc
    return _pages(s)


def _pages(s):
    return {n: s[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale") if s[n] is not None}


def _values(s, name):
    """All pages' values in 32 bits."""
    return s[name + "_pages"].float() if s["k_scale"] is None else s[name + "_pages"].float() * s[name + "_scale"][..., None]


def _read(s):
    at, slot = _slots(s)
    out = {}
    for name in ("k", "v"):
        pages = s[name + "_pages"]
        if s["k_scale"] is None:
            out[name] = pages[at, :, slot]
        else:
            y = pages.view(torch.uint8)[at, :, slot].view(F8).float()
            out[name] = (y * s[name + "_scale"][at, :, slot][..., None]).bfloat16()
    return out


def _attn(s):
    c, table = s["case"], s["table"].long()
    batch, h_kv, d = c["batch"], c["h_kv"], c["d"]
    inside = torch.arange(table.shape[1] * c["page"], device=DEV) < s["len"][:, None]       # [batch, positions]

    def rows(name):
        pages = s[name + "_pages"]
        if s["k_scale"] is None:
            x = pages[table].float()
        else:
            x = pages.view(torch.uint8)[table].view(F8).float() * s[name + "_scale"][table][..., None]
        x = x.transpose(1, 2).reshape(batch, h_kv, -1, d)
        return x.masked_fill_(~inside[:, None, :, None], 0.0)

    q = s["q"].float().view(batch, h_kv, -1, d)
    z = (q @ rows("k").transpose(2, 3)) * (1.0 / math.sqrt(d))
    z = z.masked_fill_(~inside[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (z - top).exp()
    tot = p.sum(-1, keepdim=True)
    out = (p @ rows("v")) / tot.clamp(min=1e-30)
    lse = (top + tot.log()) * math.log2(math.e)
    return {"out": out.reshape(batch, -1, d).bfloat16(), "lse": lse.reshape(batch, -1)}


def run(s):
    if not own:
        return {"rope": _rope, "write": _write, "read": _read, "attn": _attn}[s["op"]](s)
    T, op = s["T"], s["op"]
    if op == "rope":
        call = T.infllm2_rope_backward if s["case"]["back"] else T.infllm2_rope
        call(s["q"], s["k"], s["pos"], s["rope"], s["q_out"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "write":
        T.infllm2_paged_write(s["cache"], s["K"], s["V"], s["start"], s["cu"])
        return _pages(s)
    if op == "read":
        T.infllm2_paged_read(s["cache"], s["K"], s["V"], s["cu"])
        return {"k": s["K"], "v": s["V"]}
    T.infllm2_paged_decode_attn(s["cache"], s["q"], s["len"], s["out"], s["ws"], s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def work(case):
    c = case
    es = 1 if c.get("e4m3") else 2
    if c["op"] == "rope":
        n = c["total"] * (c["h_q"] + c["h_kv"]) * c["d"]
        return {"bytes": 2 * n * (4 if c["f32"] else 2) + 4 * c["axes"] * c["total"], "flops": 3 * n}
    row = c["d"] * es + (4 if c["e4m3"] else 0)
    if c["op"] != "attn":
        rows = 2 * c["total"] * c["h_kv"]
        return {"bytes": rows * (2 * c["d"] + row) + 4 * c["total"] // c["page"], "flops": rows * c["d"] * (2 if c["e4m3"] else 0)}
    tokens = c["batch"] * c["longest"]
    if c["spread"]:
        tokens = c["longest"] + (c["batch"] - 1) * c["longest"] // 2
    return {"bytes": 2 * tokens * c["h_kv"] * row + 4 * c["batch"] * c["h_q"] * (c["d"] + 1),
            "flops": 4 * tokens * c["h_q"] * c["d"]}


# ------------------------------------------------------------------ 64 bits
def _e4m3_64(x):
    """The nearest e4m3 value, ties to even: steps of 2^(e-3), e >= -6, at most 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        half = c["rot"] // 2
        theta = torch.empty(c["total"], half, dtype=torch.float64, device=DEV)
        i = 0
        for a, n in enumerate(s["sections"]):
            for _ in range(n):
                theta[:, i] = s["pos"][a].double() / 10000.0 ** (2 * i / c["rot"])
                i += 1
        z = torch.polar(torch.ones_like(theta), -theta if c["back"] else theta)
        out = {}
        for name in ("q", "k"):
            y = s[name].double()
            x = y[..., :c["rot"]]
            x = x.unflatten(-1, (half, 2)) if c["inter"] else x.unflatten(-1, (2, half)).transpose(-1, -2)
            t = torch.view_as_real(torch.view_as_complex(x.contiguous()) * z[:, None])
            y[..., :c["rot"]] = (t if c["inter"] else t.transpose(-1, -2)).flatten(-2)
            out[name] = y
        return out
    page = c["page"]
    if c["op"] == "attn":
        out, lse = [], []
        for b in range(c["batch"]):
            n, g = int(s["len"][b]), c["h_q"] // c["h_kv"]
            if n == 0:
                out.append(torch.zeros(c["h_q"], c["d"], dtype=torch.float64, device=DEV))
                lse.append(torch.full((c["h_q"],), -math.inf, dtype=torch.float64, device=DEV))
                continue
            at = s["table"][b, :(n + page - 1) // page].long()
            kv = []
            for name in ("k", "v"):
                x = s[name + "_pages"].view(torch.uint8)[at].view(s[name + "_pages"].dtype).double()
                if c["e4m3"]:
                    x *= s[name + "_scale"][at].double()[..., None]
                kv.append(x.transpose(0, 1).reshape(c["h_kv"], -1, c["d"])[:, :n].repeat_interleave(g, 0))
            w = torch.einsum("hd,hnd->hn", s["q"][b].double(), kv[0]) / math.sqrt(c["d"])
            m = torch.logsumexp(w, 1)
            out.append(torch.einsum("hn,hnd->hd", torch.exp(w - m[:, None]), kv[1]))
            lse.append(m / math.log(2.0))
        return {"out": torch.stack(out), "lse": torch.stack(lse)}
    ends = list(range(c["total"] + 1)) if s["cu"] is None else s["cu"].tolist()
    start = s["start"].tolist() if "start" in s else [0] * c["batch"]
    result = _pages({n: None if s[n] is None else s[n].double() for n in ("k_pages", "v_pages", "k_scale", "v_scale")})
    if c["op"] == "read":
        result = {"k": torch.empty_like(s["K"], dtype=torch.float64), "v": torch.empty_like(s["V"], dtype=torch.float64)}
    for b in range(c["batch"]):
        lo, hi = ends[b], ends[b + 1]
        pos = torch.arange(start[b], start[b] + hi - lo, device=DEV)
        at, slot = s["table"][b].long()[torch.div(pos, page, rounding_mode="floor")], torch.remainder(pos, page)
        for name in ("k", "v"):
            if c["op"] == "read":
                x = s[name + "_pages"].view(torch.uint8)[at, :, slot].view(s[name + "_pages"].dtype).double()
                if c["e4m3"]:
                    x = x * s[name + "_scale"][at, :, slot].double()[..., None]
                result[name][lo:hi] = x
            else:
                x = s[name.upper()][lo:hi].double()
                if c["e4m3"]:
                    scale = x.abs().amax(-1).clamp(min=2.0 ** -110) / 448
                    result[name + "_scale"][at, :, slot] = scale
                    x = _e4m3_64(x / scale[..., None])
                result[name + "_pages"][at, :, slot] = x
    return result
