"""Measured cases of the 4-bit cache and of the block tables: RoPE + store of ragged chunks into paged Q4 rows (and the
read back), the attention of chunks of new tokens over paged Q4 caches and, with a sliding window and sinks, over Q4
arenas, and the tables, offsets, positions and rows of a step built on the device from the sequences' lengths.

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
        # a decode step's store, one sequence: latency
        dict(name="store one token", op="store", geom="14/2/64", n_seq=1, chunk=1, past=127, style=0, block=64, ragged=0),
        # ragged text prompts appended to paged rows
        dict(name="store prompts", op="store", geom="16/8/128", n_seq=16, chunk=1000, past=4000, style=0, block=32,
             ragged=21),
        # one decode token over a short paged cache: latency
        dict(name="chunk one token", op="chunk", geom="14/2/64", n_seq=1, chunk=1, past=127, block=64, window=0, sinks=0,
             ragged=0),
        # batched decode of 64 sequences of up to 8192 rows
        dict(name="chunk decode", op="chunk", geom="16/8/128", n_seq=64, chunk=1, past=8192, block=64, window=0, sinks=0,
             ragged=22),
        # drafted tokens checked, a few of each sequence
        dict(name="chunk drafts", op="chunk", geom="16/8/128", n_seq=32, chunk=5, past=6000, block=16, window=0, sinks=0,
             ragged=23),
        # ragged chunks that continue long caches
        dict(name="chunk ragged long", op="chunk", geom="16/8/128", n_seq=6, chunk=2048, past=12000, block=128, window=0,
             sinks=0, ragged=13),
        # a batch that mixes single tokens with a few chunks
        dict(name="chunk mixed", op="chunk", geom="16/8/128", n_seq=34, chunk=391, past=8192, block=16, window=0, sinks=0,
             ragged=-3),
        # batched decode of 64 sequences under a window that ends inside tiles
        dict(name="window decode", op="window", geom="14/2/64", n_seq=64, chunk=1, past=8192, window=4000, sinks=4,
             ragged=24),
        # a long prompt under a window
        dict(name="window prompt", op="window", geom="16/8/128", n_seq=1, chunk=6000, past=100, window=1024, sinks=4,
             ragged=0),
        # the tables of a decode step: latency
        dict(name="tables decode step", op="tables", n_seq=64, chunk=1, past=8192, block=16, pad=0, ragged=25),
        # the tables of a large prefill batch, its rows padded to a captured size
        dict(name="tables prompts", op="tables", n_seq=1024, chunk=190, past=4000, block=16, pad=1000, ragged=26),
        # a step's blocks taken and, its sequences preempted, given back
        dict(name="tables taken back", op="turnover", n_seq=300, chunk=700, past=2000, block=32, pad=100, ragged=27),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "chunk", "chunk", "window", "window", "tables", "turnover"])
    ragged = rng.choice([0, rng.randint(1, 1 << 20)])
    if op in ("tables", "turnover"):
        n_seq = _log_int(rng, 1, 1500)
        return dict(op=op, n_seq=n_seq, chunk=_log_int(rng, 1, max(1, 200000 // n_seq)), past=rng.randint(0, 8192),
                    block=rng.choice(BLOCKS), pad=rng.choice([0, _log_int(rng, 1, 2000)]), ragged=ragged)
    case = dict(op=op, geom=rng.choice(sorted(GEOMETRIES)))
    if op == "store":
        n_seq = _log_int(rng, 1, 32)
        case.update(n_seq=n_seq, chunk=_log_int(rng, 1, 16000 // n_seq), past=rng.randint(0, 6000),
                    style=rng.randint(0, 1), block=rng.choice(BLOCKS), ragged=ragged)
        return case
    kind = rng.choice(["decode", "drafts", "chunks", "mixed"])
    if kind == "chunks":
        n_seq = _log_int(rng, 1, 8)
        case.update(n_seq=n_seq, chunk=_log_int(rng, 2, 5000 // n_seq), past=rng.choice([0, _log_int(rng, 1, 8000)]))
    elif kind == "mixed":
        case.update(n_seq=_log_int(rng, 4, 40), chunk=_log_int(rng, 16, 400), past=_log_int(rng, 100, 8192))
        ragged = -rng.randint(1, 3)
    else:
        case.update(n_seq=_log_int(rng, 1, 64), chunk=1 if kind == "decode" else rng.randint(2, 8),
                    past=_log_int(rng, 1, 8192))
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


def _row_bytes(w):
    """Bytes of a Q4 row: the codes, the scales, zeros to a multiple of 16."""
    return w // 2 + ((w // 32) * 2 + 15) // 16 * 16


# The places of 8 values' codes in their 4 bytes, low half of each byte first.
_ORDER = [0, 2, 4, 6, 1, 3, 5, 7]
_BACK = [_ORDER.index(i) for i in range(8)]


def _quantize(x):
    """Q4 rows: per 32 values m is the value of largest magnitude (the positive of two), the scale d = m / -8 in
    bfloat16's 8 bits as binary16, q = round(x * (1 / d)) within -8 .. 7, halves away from zero; q + 8 in 4 bits."""
    n, w = x.shape
    b = x.view(n, w // 32, 32)
    top, low = b.amax(-1, keepdim=True), b.amin(-1, keepdim=True)
    d = (torch.where(top >= -low, top, low) / -8).bfloat16().half()
    r = d.float()
    y = b * torch.where(r != 0, 1 / r, torch.zeros_like(r))
    q = torch.trunc(y + torch.where(y < 0, -0.5, 0.5)).clamp(-8, 7)
    u = (q + 8).to(torch.uint8).view(n, w // 8, 8)[..., _ORDER]
    rows = torch.zeros(n, _row_bytes(w), dtype=torch.uint8, device=x.device)
    rows[:, :w // 2] = (u[..., 0::2] | (u[..., 1::2] << 4)).view(n, w // 2)
    rows[:, w // 2:w // 2 + w // 16] = d.view(n, w // 32).view(torch.uint8)
    return rows


def _values(rows, w):
    """The values that Q4 rows [..., row] stand for, in 32 bits."""
    lead = rows.shape[:-1]
    c = rows[..., :w // 2].reshape(*lead, w // 8, 4)
    u = torch.stack([c & 15, c >> 4], -1).view(*lead, w // 8, 8)[..., _BACK]
    d = rows[..., w // 2:w // 2 + w // 16].contiguous().view(torch.float16).float()
    return ((u.view(*lead, w // 32, 32).float() - 8) * d[..., None]).view(*lead, w)


def _bell(shape, gen):
    """Values of unit variance without far ones, as the rows of normalised keys are."""
    x = torch.rand(2, *shape, generator=gen, device="cuda")
    return (x[0] + x[1] - 1) * math.sqrt(6)


def _fill(rows, w, gen):
    """Q4 rows of N(0, 1) values, made in pieces."""
    out = torch.empty(rows, _row_bytes(w), device="cuda", dtype=torch.uint8)
    step = max(1, (1 << 26) // w)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        out[a:b] = _quantize(torch.randn(b - a, w, generator=gen, device="cuda"))
    return out


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_tables(case, gen):
    """The tables as a step finds them: each sequence's blocks of its cached rows, the rest of the pool on the list."""
    new, past = _lengths(case)
    n, block = case["n_seq"], case["block"]
    held = [-(-p // block) for p in past]
    need = [-(-(p + c) // block) for p, c in zip(past, new)]
    blocks = sum(need) + 37
    ids = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((n, max(need) + 2), -1, dtype=torch.int32, device="cuda")
    columns = torch.arange(table.shape[1], device="cuda")
    own_blocks = columns < _i32(held)[:, None]
    table[own_blocks] = ids[:sum(held)]
    free = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
    free[:blocks - sum(held)] = ids[sum(held):]
    nt = sum(new) + case["pad"]
    s = dict(case=case, n=n, nt=nt, block=block, table=table, pool_rows=blocks * block, free=free,
             n_past=_i32(past), n_new=_i32(new), n_free=_i32([blocks - sum(held)]))
    for name, size in (("chunk_off", n + 1), ("pos", nt), ("slot", nt), ("n_free_out", 1), ("n_free_end", 1), ("err", 1)):
        s[name] = torch.zeros(size, dtype=torch.int32, device="cuda")
    # what is given back where the step is taken back: every block behind the cached rows
    s["row_lo"] = _i32([h * block for h in held])
    s["row_hi"] = _i32([h * block for h in need])
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] in ("tables", "turnover"):
        return _prepare_tables(case, gen)
    nh, nk, hd = GEOMETRIES[case["geom"]]
    new, past = _lengths(case)
    nt, n, w = sum(new), case["n_seq"], nk * hd
    s = dict(case=case, nh=nh, nk=nk, hd=hd, w=w, nt=nt, n=n, max_chunk=max(new),
             max_len=max(a + b for a, b in zip(new, past)), scale=hd ** -0.5,
             q=torch.randn(nt, nh * hd, generator=gen, device="cuda"),
             err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    starts = [0]
    for c in new:
        starts.append(starts[-1] + c)
    s["chunk_off"], s["n_past"] = _i32(starts), _i32(past)
    if case["op"] == "window":  # an arena: each sequence's rows, with room to grow
        caps = [a + b + 8 for a, b in zip(new, past)]
        offs = [0]
        for c in caps:
            offs.append(offs[-1] + c)
        s["row_off"] = torch.tensor(offs[:-1], dtype=torch.int64, device="cuda")
        s["cap"] = _i32(caps)
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
    s["k_pool"], s["v_pool"] = _fill(rows, w, gen), _fill(rows, w, gen)
    if case["op"] == "store":
        s["k"], s["v"] = _bell((nt, w), gen), torch.randn(nt, w, generator=gen, device="cuda")
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["k_back"], s["v_back"] = torch.empty_like(s["k"]).half(), torch.empty_like(s["v"]).half()
    else:
        s["out"] = torch.empty(nt, nh * hd, device="cuda")
    return s


# ----------------------------------------------------------------------------- the plain forms
def _token_places(s):
    """The sequence and the cache position of every new token."""
    new = (s["chunk_off"][1:] - s["chunk_off"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(s["n"], device="cuda"), new, output_size=s["nt"])
    return seq, s["n_past"][seq].long() + torch.arange(s["nt"], device="cuda") - s["chunk_off"][seq].long()


def _plain_rope(x, pos, heads, hd, style):
    half = hd // 2
    i = torch.arange(half, device=x.device, dtype=torch.float64)
    angle = pos.double()[:, None] * THETA ** (-2 * i / hd)  # far positions: 64 bits, [tokens, pairs]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    x = x.view(-1, heads, hd).double()  # (values next to a border of the quantisation: 64 bits)
    a, b = (x[..., :half], x[..., half:]) if style == 0 else (x[..., 0::2], x[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.cat([a, b], -1) if style == 0 else torch.stack([a, b], -1)
    return y.reshape(x.shape[0], heads * hd).float()


def _plain_store(s):
    c, block = s["case"], s["case"]["block"]
    seq, pos = _token_places(s)
    q = _plain_rope(s["q"], pos, s["nh"], s["hd"], c["style"])
    k = _plain_rope(s["k"], pos, s["nk"], s["hd"], c["style"])
    rows = s["table"][seq, pos // block].long() * block + pos % block
    s["k_pool"][rows] = _quantize(k)
    s["v_pool"][rows] = _quantize(s["v"])
    return dict(q=q, k=k, k_back=_values(s["k_pool"][rows], s["w"]).half(),
                v_back=_values(s["v_pool"][rows], s["w"]).half())


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
    keys = _values(s["k_pool"][rows], w).view(n, -1, nk, hd).permute(0, 2, 3, 1)
    values = _values(s["v_pool"][rows], w).view(n, -1, nk, hd).permute(0, 2, 1, 3)
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


def _plain_grow(s):
    n, block, past, new = s["n"], s["block"], s["n_past"].long(), s["n_new"].long()
    held = (past + block - 1).div(block, rounding_mode="floor")
    take = (past + new + block - 1).div(block, rounding_mode="floor") - held
    upto = take.cumsum(0)
    b = torch.arange(s["table"].shape[1], device="cuda") - held[:, None]
    nth = (upto - take)[:, None] + b
    taken = (b >= 0) & (b < take[:, None])
    ids = s["free"][(s["n_free"].long() - 1 - nth).clamp(min=0, max=s["free"].shape[0] - 1)]
    s["table"].copy_(torch.where(taken, ids, s["table"]))
    off = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    t = torch.arange(s["nt"], device="cuda")
    seq = (torch.searchsorted(off, t, right=True) - 1).clamp(max=n - 1)
    pos = past[seq] + t - off[seq]
    there = t < off[-1]
    slot = s["table"][seq, (pos // block).clamp(max=s["table"].shape[1] - 1)].long() * block + pos % block
    return dict(chunk_off=off.int(), pos=torch.where(there, pos, -1).int(), slot=torch.where(there, slot, -1).int(),
                n_free=s["n_free"] - upto[-1:].int())


def _plain_release(s, n_free):
    """Every block in the given rows back on the list, the last one first; a list with one more place, cut off again."""
    b = torch.arange(s["table"].shape[1], device="cuda") * s["block"]
    out = (b >= s["row_lo"][:, None]) & (b + s["block"] <= s["row_hi"][:, None]) & (s["table"] >= 0)
    nth = out.view(-1).cumsum(0)
    place = torch.where(out.view(-1), n_free.long() + nth[-1] - nth, s["free"].shape[0])
    s["free"].copy_(torch.cat([s["free"], s["free"][:1]]).scatter(0, place, s["table"].view(-1))[:-1])
    s["table"].masked_fill_(out, -1)
    return n_free + nth[-1:].int()


def _plain_tables(s):
    out = _plain_grow(s)
    if s["case"]["op"] == "turnover":
        out["n_free_end"] = _plain_release(s, out["n_free"])
        out["free"] = s["free"]
    out["table"] = s["table"]
    return out


def _own_tables(m, s):
    m.minf_block_table_grow(s["table"], s["block"], s["pool_rows"], s["n_past"], s["n_new"], s["free"], s["n_free"],
                            s["n_free_out"], s["chunk_off"], s["pos"], s["slot"], s["err"])
    out = dict(chunk_off=s["chunk_off"], pos=s["pos"], slot=s["slot"], n_free=s["n_free_out"])
    if s["case"]["op"] == "turnover":
        m.minf_block_table_release(s["table"], s["block"], s["pool_rows"], s["row_lo"], s["row_hi"], s["free"],
                                   s["n_free_out"], s["n_free_end"], s["err"])
        out["n_free_end"] = s["n_free_end"]
        out["free"] = s["free"]
    out["table"] = s["table"]
    return out


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] in ("tables", "turnover"):
            return _plain_tables(s)
        return _plain_store(s) if c["op"] == "store" else _plain_attention(s)
    import gqa_attention_kv_rope_gb300 as m

    if c["op"] in ("tables", "turnover"):
        return _own_tables(m, s)
    if c["op"] == "store":
        m.minf_rope_kv_append_chunk_paged_q4(
            s["q_out"], s["k_out"], s["q"], s["k"], s["v"], None, None, s["chunk_off"], s["n_past"], s["nh"], s["nk"],
            s["hd"], s["hd"], THETA, 1.0, c["style"], s["k_pool"], s["v_pool"], s["table"], c["block"], s["err"])
        m.minf_kv_read_chunk_paged_q4(s["k_back"], s["v_back"], s["k_pool"], s["v_pool"], s["table"], c["block"],
                                      s["chunk_off"], s["n_past"], s["err"])
        return dict(q=s["q_out"], k=s["k_out"], k_back=s["k_back"], v_back=s["v_back"])
    if "ws" not in s:
        s["ws"] = m.kv.chunk_workspace(s["nt"], s["n"], s["nh"], s["nk"], s["hd"], s["max_chunk"])
    if c["op"] == "chunk":
        m.minf_gqa_attn_chunk_paged_q4(
            s["out"], s["q"], s["k_pool"], s["v_pool"], s["table"], c["block"], s["chunk_off"], s["n_past"],
            s["max_chunk"], s["nh"], s["nk"], s["hd"], s["hd"], s["scale"], c["window"], c["sinks"], s["ws"], s["err"])
    else:
        m.minf_gqa_attn_window_q4(
            s["out"], s["q"], s["k_pool"], s["v_pool"], s["row_off"], s["cap"], s["max_cap"], s["chunk_off"],
            s["n_past"], s["max_chunk"], s["nh"], s["nk"], s["hd"], s["hd"], s["scale"], c["window"], c["sinks"],
            s["ws"], s["err"])
    return s["out"]


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    new, past = _lengths(case)
    nt, n = sum(new), case["n_seq"]
    if case["op"] in ("tables", "turnover"):
        # the lengths, the offsets, positions and rows, ids from the list to the table, the partly filled blocks' ids
        block = case["block"]
        taken = sum(-(-(p + c) // block) - -(-p // block) for p, c in zip(past, new))
        moved = 8 * n + 4 * (n + 1) + 8 * (nt + case["pad"]) + 8 * taken + 4 * sum(p % block > 0 for p in past) + 8
        if case["op"] == "turnover":  # the rows' bounds, the ids back to the list, the entries cleared
            moved += 8 * n + 12 * taken + 8
        return {"bytes": moved, "flops": 2 * nt}
    nh, nk, hd = GEOMETRIES[case["geom"]]
    w = nk * hd
    row = _row_bytes(w)
    if case["op"] == "store":  # q and k in and out, v in, the rows written, read back and returned in 16 bits
        return {"bytes": nt * (8 * nh * hd + 8 * w + 4 * w + 4 * row + 4 * w), "flops": 3 * nt * (nh * hd + w)}
    window, sinks, rows, pairs = case["window"], case["sinks"], 0, 0
    for c, p in zip(new, past):
        seen = c + p
        rows += seen if not window else min(seen, window + c - 1 + min(sinks, max(0, p - window + 1)))
        for i in range(c):
            at = p + i + 1
            pairs += at if not window else min(at, window + min(sinks, max(0, at - window)))
    return {"bytes": 8 * nt * nh * hd + 2 * rows * row, "flops": 4 * hd * nh * pairs}


# ----------------------------------------------------------------------------- the definition in 64 bits
def _exact_rope(x, pos, heads, hd, style):
    x = x.double().view(x.shape[0], heads, hd)
    y = torch.empty_like(x)
    for i in range(hd // 2):
        a, b = (i, i + hd // 2) if style == 0 else (2 * i, 2 * i + 1)
        th = (pos.double() * math.pow(THETA, -2.0 * i / hd))[:, None]
        y[:, :, a] = x[:, :, a] * torch.cos(th) - x[:, :, b] * torch.sin(th)
        y[:, :, b] = x[:, :, a] * torch.sin(th) + x[:, :, b] * torch.cos(th)
    return y.view(x.shape[0], -1)


def _exact_held(x):
    """The values that a stored row stands for."""
    b = x.view(x.shape[0], -1, 32)
    at = b.abs().max(-1, keepdim=True).indices
    d = (-b.gather(-1, at) / 8).to(torch.bfloat16).to(torch.float16).double()
    r = (b / d).nan_to_num(0.0)
    q = (torch.sign(r) * torch.floor(r.abs() + 0.5)).clamp(-8, 7)
    return (q * d).view(x.shape)


def _exact_rows(rows, w):
    """The values of Q4 rows [n, row], code by code."""
    n = rows.shape[0]
    out = torch.empty(n, w // 8, 8, dtype=torch.float64, device=rows.device)
    words = rows[:, :w // 2].contiguous().view(torch.int32).long()
    for i in range(4):
        out[..., 2 * i] = ((words >> (4 * i)) & 15).double() - 8
        out[..., 2 * i + 1] = ((words >> (16 + 4 * i)) & 15).double() - 8
    d = rows[:, w // 2:w // 2 + w // 16].contiguous().view(torch.float16).double()
    return out.view(n, w) * d.repeat_interleave(32, 1)


def exact(case, seed):
    if case["op"] in ("tables", "turnover"):
        return None
    s = prepare(case, seed)
    nh, nk, hd, w = s["nh"], s["nk"], s["hd"], s["w"]
    new, past = _lengths(case)
    if case["op"] == "store":
        pos = torch.cat([torch.arange(p, p + c, device="cuda") for c, p in zip(new, past)])
        q = _exact_rope(s["q"], pos, nh, hd, case["style"])
        k = _exact_rope(s["k"], pos, nk, hd, case["style"])
        return dict(q=q, k=k, k_back=_exact_held(k), v_back=_exact_held(s["v"].double()))
    out = torch.empty(s["nt"], nh, hd, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["n_seq"]):
        length = new[b] + past[b]
        j = torch.arange(length, device="cuda")
        if case["op"] == "window":
            rows = int(s["row_off"][b]) + j
        else:
            rows = s["table"][b].long()[j // case["block"]] * case["block"] + j % case["block"]
        k = _exact_rows(s["k_pool"][rows], w).view(length, nk, hd)
        v = _exact_rows(s["v_pool"][rows], w).view(length, nk, hd)
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
