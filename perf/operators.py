"""Measured cases of the chunk operators: several-axis RoPE, the chunk's RoPE + store into paged K/V (and the read
back), and the attention of chunks of new tokens over paged caches and, with a sliding window and sinks, over arenas.

A case names an operator and its sizes; the lengths of a ragged batch follow from the case alone, so that its work is
known without its inputs.  Where `own` is false, run() computes the plain form in torch; where it is true it makes the
calls of this package.
"""
import math
import random

import torch

own = False

THETA = 1e6
BLOCKS = (16, 32, 64, 128, 256)
GEOMETRIES = {  # heads, kv heads, head size: the two geometries of this package's workloads and neighbours of them
    "14/2/64": (14, 2, 64),
    "16/8/128": (16, 8, 128),
    "8/1/64": (8, 1, 64),
    "12/4/128": (12, 4, 128),
}


def listed():
    return [
        # a captioning prompt's patch rows, rotated in place of their time, height and width
        dict(name="axes image rows", op="axes", geom="16/8/128", n_seq=1, chunk=16384, past=0, axes=3, style=0, ragged=0),
        # one decode token's query heads
        dict(name="axes one token", op="axes", geom="14/2/64", n_seq=1, chunk=1, past=0, axes=3, style=1, ragged=0),
        # a decode step's store, one sequence: latency
        dict(name="store one token f16", op="store", geom="14/2/64", kind="f16", n_seq=1, chunk=1, past=127, axes=1,
             style=0, block=64, ragged=0),
        # ragged prompts with images appended to binary16 pages
        dict(name="store images f16", op="store", geom="16/8/128", kind="f16", n_seq=7, chunk=2500, past=900, axes=3,
             style=0, block=64, ragged=11),
        # ragged text chunks quantised into Q8_0 pages
        dict(name="store chunks q8", op="store", geom="16/8/128", kind="q8", n_seq=16, chunk=1000, past=4000, axes=1,
             style=0, block=32, ragged=12),
        # one decode token over a short paged cache: latency
        dict(name="chunk one token f16", op="chunk", geom="14/2/64", kind="f16", n_seq=1, chunk=1, past=127, block=64,
             window=0, sinks=0, ragged=0),
        # the prefill workload's 512 tokens, into fp32 pages
        dict(name="chunk prompt f32", op="chunk", geom="14/2/64", kind="f32", n_seq=1, chunk=512, past=0, block=64,
             window=0, sinks=0, ragged=0),
        # ragged chunks that continue long binary16 caches
        dict(name="chunk ragged long f16", op="chunk", geom="16/8/128", kind="f16", n_seq=6, chunk=2048, past=12000,
             block=128, window=0, sinks=0, ragged=13),
        # a batch that mixes single tokens with a few chunks, over Q8_0 pages
        dict(name="chunk mixed q8", op="chunk", geom="16/8/128", kind="q8", n_seq=34, chunk=391, past=8192, block=16,
             window=0, sinks=0, ragged=-3),
        # batched decode of 64 sequences of up to 8192 rows, a window of 4096 and four sinks
        dict(name="window decode f16", op="window", geom="16/8/128", kind="f16", n_seq=64, chunk=1, past=8192,
             window=4096, sinks=4, ragged=14),
        # batched decode over Q8_0 rows, a window that ends inside tiles
        dict(name="window decode q8", op="window", geom="14/2/64", kind="q8", n_seq=64, chunk=1, past=8192, window=1000,
             sinks=5, ragged=15),
        # a long prompt under a window
        dict(name="window prompt f16", op="window", geom="16/8/128", kind="f16", n_seq=1, chunk=6000, past=100,
             window=1024, sinks=4, ragged=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["axes", "store", "chunk", "chunk", "window", "window"])
    geom = rng.choice(sorted(GEOMETRIES))
    case = dict(op=op, geom=geom)
    if op == "axes":
        case.update(n_seq=1, chunk=_log_int(rng, 1, 16384), past=0, axes=rng.randint(1, 4), style=rng.randint(0, 1),
                    ragged=0)
        return case
    case["kind"] = rng.choice(["f32", "f16", "q8"])
    ragged = rng.choice([0, rng.randint(1, 1 << 20)])
    if op == "store":
        n_seq = _log_int(rng, 1, 32)
        case.update(n_seq=n_seq, chunk=_log_int(rng, 1, 16000 // n_seq), past=rng.randint(0, 6000),
                    axes=rng.randint(1, 4), style=rng.randint(0, 1), block=rng.choice(BLOCKS), ragged=ragged)
        return case
    decode = rng.random() < 0.4
    if decode:
        case.update(n_seq=_log_int(rng, 1, 64), chunk=rng.choice([1, 1, 2, 3]), past=_log_int(rng, 1, 8192))
    else:
        n_seq = _log_int(rng, 1, 8)
        case.update(n_seq=n_seq, chunk=_log_int(rng, 2, 5000 // n_seq), past=rng.choice([0, _log_int(rng, 1, 8000)]))
    if op == "chunk":
        case["block"] = rng.choice(BLOCKS)
        case["window"], case["sinks"] = rng.choice([(0, 0), (0, 0), (_log_int(rng, 16, 4096), rng.randint(0, 8))])
    else:
        case["window"], case["sinks"] = _log_int(rng, 1, 4096), rng.randint(0, 8)
    case["ragged"] = ragged
    return case


def _lengths(case):
    """(new tokens, cached rows before them) of every sequence; ragged 0: all the same, -n: n chunks among single
    tokens, otherwise lengths spread below the given ones."""
    n, c, p, r = case["n_seq"], case["chunk"], case["past"], case["ragged"]
    if r == 0:
        return [c] * n, [p] * n
    rng = random.Random(abs(r) * 7919 + n)
    past = [rng.randint(p // 8, p) for _ in range(n)]
    if r < 0:
        new = [1] * n
        for i in rng.sample(range(n), min(n, -r)):
            new[i] = rng.randint(max(1, c // 2), c)
        return new, past
    return [rng.randint(max(1, c // 4), c) for _ in range(n)], past


def _pair_axis(case, hd):
    """Axis of each rotated pair: the first quarter goes by time, the others share the rest."""
    half, axes = hd // 2, case["axes"]
    if axes == 1:
        return [0] * half
    first = half // 4
    return [0] * first + [1 + (i * (axes - 1)) // (half - first) for i in range(half - first)]


def _axis_positions(case, new, past, device, gen):
    """int32 [axes, tokens]: text positions on the first axis; on the others, places in an image's grid."""
    first = torch.cat([torch.arange(p, p + c, device=device) for c, p in zip(new, past)])
    rows = [first]
    for _ in range(case["axes"] - 1):
        rows.append(first + torch.randint(0, 64, (first.numel(),), generator=gen, device=device))
    return torch.stack(rows).to(torch.int32).contiguous()


def _q8_row_bytes(w):
    return w + ((w // 32) * 2 + 15) // 16 * 16


def _quantize(x):
    """Q8_0 rows: per 32 values d = max|x| / 127, q = round(x * (1 / d)), halves away from zero; the int8 quants, then
    the binary16 scales, then zeros to a multiple of 16 bytes."""
    n, w = x.shape
    b = x.view(n, w // 32, 32)
    d = b.abs().amax(-1, keepdim=True) / 127
    y = b * torch.where(d > 0, 1 / d, torch.zeros_like(d))
    q = torch.trunc(y + torch.where(y < 0, -0.5, 0.5)).to(torch.int8).view(n, w)
    rows = torch.zeros(n, _q8_row_bytes(w), dtype=torch.uint8, device=x.device)
    rows[:, :w] = q.view(torch.uint8)
    rows[:, w:w + w // 16] = d.view(n, w // 32).half().view(torch.uint8)
    return rows


def _to_kind(x, kind):
    return x if kind == "f32" else x.half() if kind == "f16" else _quantize(x)


def _to_f32(rows, kind, w):
    """The values that rows [..., row] of a pool stand for, in 32 bits."""
    if kind == "f32":
        return rows
    if kind == "f16":
        return rows.float()
    q = rows[..., :w].contiguous().view(torch.int8).float()
    d = rows[..., w:w + w // 16].contiguous().view(torch.float16).float()
    return (q.view(*q.shape[:-1], w // 32, 32) * d[..., None]).view(q.shape)


def _fill(rows, w, kind, gen):
    """rows of N(0, 1) values held as `kind`, made in pieces."""
    out = torch.empty(rows, _q8_row_bytes(w) if kind == "q8" else w, device="cuda",
                      dtype={"f32": torch.float32, "f16": torch.float16, "q8": torch.uint8}[kind])
    step = max(1, (1 << 26) // w)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        out[a:b] = _to_kind(torch.randn(b - a, w, generator=gen, device="cuda"), kind)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    nh, nk, hd = GEOMETRIES[case["geom"]]
    new, past = _lengths(case)
    nt, n, w = sum(new), case["n_seq"], nk * hd
    s = dict(case=case, nh=nh, nk=nk, hd=hd, w=w, nt=nt, n=n, max_chunk=max(new),
             max_len=max(a + b for a, b in zip(new, past)), scale=hd ** -0.5,
             q=torch.randn(nt, nh * hd, generator=gen, device="cuda"),
             err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] in ("axes", "store"):
        s["pos"] = _axis_positions(case, new, past, "cuda", gen)
        s["pair_axis"] = _pair_axis(case, hd)
        s["q_out"] = torch.empty_like(s["q"])
    if case["op"] == "axes":
        return s
    starts = [0]
    for c in new:
        starts.append(starts[-1] + c)
    s["chunk_off"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["n_past"] = torch.tensor(past, dtype=torch.int32, device="cuda")
    if case["op"] == "window":  # an arena: each sequence's rows, with room to grow
        caps = [a + b + 8 for a, b in zip(new, past)]
        offs = [0]
        for c in caps:
            offs.append(offs[-1] + c)
        s["row_off"] = torch.tensor(offs[:-1], dtype=torch.int64, device="cuda")
        s["cap"] = torch.tensor(caps, dtype=torch.int32, device="cuda")
        s["max_cap"], rows = max(caps), offs[-1]
    else:  # a pool: each sequence's blocks, scattered
        block = case["block"]
        need = [-(-(a + b) // block) for a, b in zip(new, past)]
        total = sum(need) + 5
        ids = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((n, max(need) + 1), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, c in enumerate(need):
            table[i, :c] = ids[at:at + c]
            at += c
        s["table"], rows = table, total * block
    s["k_pool"], s["v_pool"] = _fill(rows, w, case["kind"], gen), _fill(rows, w, case["kind"], gen)
    if case["op"] == "store":
        s["k"] = torch.randn(nt, w, generator=gen, device="cuda")
        s["v"] = torch.randn(nt, w, generator=gen, device="cuda")
        s["k_out"] = torch.empty_like(s["k"])
        s["k_back"], s["v_back"] = torch.empty_like(s["k"]).half(), torch.empty_like(s["v"]).half()
    else:
        s["out"] = torch.empty(nt, nh * hd, device="cuda")
    return s


# ----------------------------------------------------------------------------- the plain forms
def _plain_rope(x, pos, pair_axis, heads, hd, style):
    half = hd // 2
    i = torch.arange(half, device=x.device, dtype=torch.float64)
    axis = torch.tensor(pair_axis, device=x.device)
    angle = pos[axis].double().t() * THETA ** (-2 * i / hd)  # far positions: 64 bits, [tokens, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.view(-1, heads, hd)
    a, b = (x[..., :half], x[..., half:]) if style == 0 else (x[..., 0::2], x[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.cat([a, b], -1) if style == 0 else torch.stack([a, b], -1)
    return y.reshape(x.shape[0], heads * hd)


def _token_rows(s):
    """The pool row of every new token."""
    block = s["case"]["block"]
    new = (s["chunk_off"][1:] - s["chunk_off"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(s["n"], device="cuda"), new, output_size=s["nt"])
    p = s["n_past"][seq].long() + torch.arange(s["nt"], device="cuda") - s["chunk_off"][seq].long()
    return s["table"][seq, p // block].long() * block + p % block


def _plain_store(s):
    c = s["case"]
    q = _plain_rope(s["q"], s["pos"], s["pair_axis"], s["nh"], s["hd"], c["style"])
    k = _plain_rope(s["k"], s["pos"], s["pair_axis"], s["nk"], s["hd"], c["style"])
    rows = _token_rows(s)
    s["k_pool"][rows] = _to_kind(k, c["kind"])
    s["v_pool"][rows] = _to_kind(s["v"], c["kind"])
    return dict(q=q, k=k, k_back=_to_f32(s["k_pool"][rows], c["kind"], s["w"]).half(),
                v_back=_to_f32(s["v_pool"][rows], c["kind"], s["w"]).half())


def _plain_attention(s):
    """Attention of padded chunks over the rows that any token of a sequence can see."""
    c, n, nk, hd, w = s["case"], s["n"], s["nk"], s["hd"], s["w"]
    g, most, window, sinks = s["nh"] // s["nk"], s["max_chunk"], c["window"], c["sinks"]
    past, off = s["n_past"].long()[:, None], s["chunk_off"].long()
    if window and sinks + window + most < s["max_len"]:
        first = (past - window + 1).clamp(min=sinks)
        j = torch.cat([torch.arange(sinks, device="cuda").expand(n, -1),
                       first + torch.arange(window + most - 1, device="cuda")], 1)
    else:
        j = torch.arange(s["max_len"], device="cuda").expand(n, -1)
    if c["op"] == "window":
        rows = (s["row_off"][:, None] + j).clamp(max=s["k_pool"].shape[0] - 1)
    else:
        at = (j // c["block"]).clamp(max=s["table"].shape[1] - 1)
        rows = s["table"].long().gather(1, at).clamp(min=0) * c["block"] + j % c["block"]
    keys = _to_f32(s["k_pool"][rows], c["kind"], w).view(n, -1, nk, hd).permute(0, 2, 3, 1)
    values = _to_f32(s["v_pool"][rows], c["kind"], w).view(n, -1, nk, hd).permute(0, 2, 1, 3)
    i = torch.arange(most, device="cuda")
    live = i < (off[1:] - off[:-1])[:, None]
    token = (off[:-1, None] + i).clamp(max=s["nt"] - 1)
    q = s["q"][token].view(n, most, nk, g, hd).permute(0, 2, 3, 1, 4).reshape(n, nk, g * most, hd)
    p = past + i
    see = j[:, None] <= p[:, :, None]
    if window:
        see &= (j[:, None] > p[:, :, None] - window) | (j[:, None] < sinks)
    x = (q @ keys).mul_(s["scale"]).view(n, nk, g, most, -1)
    x = x.masked_fill_(~see[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    x = x.div_(x.sum(-1, keepdim=True)).view(n, nk, g * most, -1)
    o = (x @ values).view(n, nk, g, most, hd).permute(0, 3, 1, 2, 4).reshape(n, most, s["nh"] * hd)
    return o[live]


def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "axes":
            return _plain_rope(state["q"], state["pos"], state["pair_axis"], state["nh"], state["hd"], c["style"])
        return _plain_store(state) if c["op"] == "store" else _plain_attention(state)
    import gqa_attention_kv_rope_gb300 as m

    s, end = state, {"f32": "", "f16": "_f16", "q8": "_q8"}[c.get("kind", "f32")]
    if c["op"] == "axes":
        m.minf_rope_axes(s["q_out"], s["q"], s["pos"], s["pair_axis"], s["nh"], s["hd"], THETA, 1.0, c["style"],
                         s["err"])
        return s["q_out"]
    if c["op"] == "store":
        getattr(m, "minf_rope_kv_append_chunk_paged" + end)(
            s["q_out"], s["k_out"], s["q"], s["k"], s["v"], s["pos"], s["pair_axis"], s["chunk_off"], s["n_past"],
            s["nh"], s["nk"], s["hd"], s["hd"], THETA, 1.0, c["style"], s["k_pool"], s["v_pool"], s["table"],
            c["block"], s["err"])
        getattr(m, "minf_kv_read_chunk_paged" + end)(
            s["k_back"], s["v_back"], s["k_pool"], s["v_pool"], s["table"], c["block"], s["chunk_off"], s["n_past"],
            s["err"])
        return dict(q=s["q_out"], k=s["k_out"], k_back=s["k_back"], v_back=s["v_back"])
    if "ws" not in s:
        s["ws"] = m.kv.chunk_workspace(s["nt"], s["n"], s["nh"], s["nk"], s["hd"], s["max_chunk"])
    if c["op"] == "chunk":
        getattr(m, "minf_gqa_attn_chunk_paged" + end)(
            s["out"], s["q"], s["k_pool"], s["v_pool"], s["table"], c["block"], s["chunk_off"], s["n_past"],
            s["max_chunk"], s["nh"], s["nk"], s["hd"], s["hd"], s["scale"], c["window"], c["sinks"], s["ws"], s["err"])
    else:
        getattr(m, "minf_gqa_attn_window" + end)(
            s["out"], s["q"], s["k_pool"], s["v_pool"], s["row_off"], s["cap"], s["max_cap"], s["chunk_off"],
            s["n_past"], s["max_chunk"], s["nh"], s["nk"], s["hd"], s["hd"], s["scale"], c["window"], c["sinks"],
            s["ws"], s["err"])
    return s["out"]


# ----------------------------------------------------------------------------- what a pass cannot do without
def _row_bytes(case, w):
    kind = case["kind"]
    return 4 * w if kind == "f32" else 2 * w if kind == "f16" else _q8_row_bytes(w)


def work(case):
    nh, nk, hd = GEOMETRIES[case["geom"]]
    new, past = _lengths(case)
    nt, w = sum(new), nk * hd
    if case["op"] == "axes":
        return {"bytes": nt * (8 * nh * hd + 4 * case["axes"]), "flops": 3 * nt * nh * hd}
    if case["op"] == "store":  # q and k in and out, v in, the rows written, read back and returned in 16 bits
        row = _row_bytes(case, w)
        return {"bytes": nt * (8 * nh * hd + 8 * w + 4 * w + 4 * row + 4 * w + 4 * case["axes"]),
                "flops": 3 * nt * (nh * hd + w)}
    window, sinks, rows, pairs = case["window"], case["sinks"], 0, 0
    for c, p in zip(new, past):
        seen = c + p
        rows += seen if not window else min(seen, window + c - 1 + min(sinks, max(0, p - window + 1)))
        for i in range(c):
            at = p + i + 1
            pairs += at if not window else min(at, window + min(sinks, max(0, at - window)))
    return {"bytes": 8 * nt * nh * hd + 2 * rows * _row_bytes(case, w), "flops": 4 * hd * nh * pairs}


# ----------------------------------------------------------------------------- the definition in 64 bits
def _exact_rope(x, pos, pair_axis, heads, hd, style):
    x = x.double().view(x.shape[0], heads, hd)
    y = torch.empty_like(x)
    for i in range(hd // 2):
        a, b = (i, i + hd // 2) if style == 0 else (2 * i, 2 * i + 1)
        th = (pos[pair_axis[i]].double() * math.pow(THETA, -2.0 * i / hd))[:, None]
        y[:, :, a] = x[:, :, a] * torch.cos(th) - x[:, :, b] * torch.sin(th)
        y[:, :, b] = x[:, :, a] * torch.sin(th) + x[:, :, b] * torch.cos(th)
    return y.view(x.shape[0], -1)


def _exact_held(x, kind):
    """The values that a stored row stands for, before the last rounding to 16 bits."""
    if kind != "q8":
        return x
    b = x.view(x.shape[0], -1, 32)
    d = b.abs().max(-1, keepdim=True).values / 127
    r = (b / d).nan_to_num(0.0)
    q = torch.sign(r) * torch.floor(r.abs() + 0.5)
    return (q * d.half().double()).view(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    nh, nk, hd, w = s["nh"], s["nk"], s["hd"], s["w"]
    if case["op"] == "axes":
        return _exact_rope(s["q"], s["pos"], s["pair_axis"], nh, hd, case["style"])
    if case["op"] == "store":
        q = _exact_rope(s["q"], s["pos"], s["pair_axis"], nh, hd, case["style"])
        k = _exact_rope(s["k"], s["pos"], s["pair_axis"], nk, hd, case["style"])
        return dict(q=q, k=k, k_back=_exact_held(k, case["kind"]), v_back=_exact_held(s["v"].double(), case["kind"]))
    new, past = _lengths(case)
    out = torch.empty(s["nt"], nh, hd, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["n_seq"]):
        length = new[b] + past[b]
        j = torch.arange(length, device="cuda")
        if case["op"] == "window":
            rows = int(s["row_off"][b]) + j
        else:
            rows = s["table"][b].long()[j // case["block"]] * case["block"] + j % case["block"]
        k = _to_f32(s["k_pool"][rows], case["kind"], w).double().view(length, nk, hd)
        v = _to_f32(s["v_pool"][rows], case["kind"], w).double().view(length, nk, hd)
        for first in range(0, new[b], 512):
            count = min(512, new[b] - first)
            p = past[b] + first + torch.arange(count, device="cuda")[:, None]
            hidden = j > p
            if case["window"]:
                hidden |= (j <= p - case["window"]) & (j >= case["sinks"])
            q = s["q"][at + first:at + first + count].double().view(count, nh, hd)
            for h in range(nh):
                x = q[:, h] @ k[:, h // (nh // nk)].t() / math.sqrt(hd)
                x = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
                out[at + first:at + first + count, h] = x @ v[:, h // (nh // nk)]
        at += new[b]
    return out.view(s["nt"], nh * hd)
