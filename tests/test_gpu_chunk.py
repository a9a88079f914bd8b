"""GPU parity of the chunk operators: several-axis RoPE, RoPE + store of ragged chunks into paged
regions (fp32, binary16, Q8_0) and the read back, and the attention of ragged chunks over paged
regions and arenas with a sliding window and sinks -- against a plain evaluation in 64 bits.

Tolerances.  Attention: the scores' operands carry 22 bits or more and sums are fp32, so a score
of unit-variance inputs is off by a few 2^-24 * sum|q k| * scale (sum|q k| * scale < 10 at hd 128)
and an output by that times its spread of values: the fp32 tolerance of the other attention tests,
|d| <= 1e-5 + 1e-4 |ref|, leaves a factor of about five.  Rotation: the angle in half turns is
rounded once (2^-25 of at most pi), sine and cosine are good to 2 ulp (2^-23), each of the two
products and their sum round once (2^-24 each): |d| <= (|a| + |b|) * (pi 2^-25 + 2^-23 + 2 * 2^-24)
< 3.5e-7 (|a| + |b|).  A binary16 store adds half a step (2^-11 of the value, 2^-25 below the
normal range); a Q8_0 store is compared bit for bit with the quantization of the rotated rows."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ATOL, RTOL = 1e-5, 1e-4
KINDS = ["f32", "f16", "q8"]
END = {"f32": "", "f16": "_f16", "q8": "_q8"}
THETA = 1e6
GEOMS = [(14, 2, 64, 64), (16, 8, 128, 128), (8, 1, 64, 64), (3, 3, 128, 128), (4, 2, 128, 64), (6, 2, 256, 128)]


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gqa_attention_kv_rope_gb300 as pkg
    from gqa_attention_kv_rope_gb300 import build

    build.build()
    pkg.binding.lib()
    return pkg


def rng(*key):
    return np.random.default_rng([int(k) for k in key])


def dev(x, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(x))
    return (t.to(dtype) if dtype is not None else t).cuda()


def i32(x):
    return dev(np.asarray(x, np.int32))


def close(got, ref, what=""):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    d = np.abs(got - ref)
    bad = d > ATOL + RTOL * np.abs(ref)
    assert not bad.any(), f"{what}: {int(bad.sum())} elements off, max abs {np.nanmax(d):.3g}"


# ----------------------------------------------------------------------------- Q8_0 rows on the host
def q8_row_bytes(w):
    return w + ((w // 32) * 2 + 15) // 16 * 16


def quantize(x):
    """float32 [n, W] -> uint8 rows, every step rounded to fp32 as the store's."""
    n, w = x.shape
    b = np.asarray(x, np.float32).reshape(n, w // 32, 32)
    d = (np.abs(b).max(-1) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore"):
        r = np.where(d > 0, np.float32(1) / d, np.float32(0)).astype(np.float32)
    y = (b * r[..., None]).astype(np.float32).astype(np.float64)
    q = (np.sign(y) * np.floor(np.abs(y) + 0.5)).astype(np.int8).reshape(n, w)
    rows = np.zeros((n, q8_row_bytes(w)), np.uint8)
    rows[:, :w] = q.view(np.uint8)
    rows[:, w:w + w // 16] = d.astype(np.float16).view(np.uint8)
    return rows


def hold(x, kind):
    """The bytes a pool of `kind` holds for the fp32 rows x."""
    return x.astype(np.float32) if kind == "f32" else x.astype(np.float16) if kind == "f16" else quantize(x)


def value(rows, kind, w):
    if kind != "q8":
        return rows.astype(np.float64)
    q = rows[:, :w].view(np.int8).astype(np.float64)
    d = np.ascontiguousarray(rows[:, w:w + w // 16]).view(np.float16).astype(np.float64)
    return (q.reshape(len(rows), w // 32, 32) * d[..., None]).reshape(len(rows), w)


# ----------------------------------------------------------------------------- attention: 64-bit reference
def ref_attention(q, k, v, p0, cap, nh, nk, hd_kv, scale, window, sinks):
    """q [c, nh, hd] at positions p0 + i over rows k, v [cap, nk, hd_kv] of one sequence."""
    out = np.zeros((len(q), nh, hd_kv))
    for i in range(len(q)):
        p = p0 + i
        last = min(p, cap - 1)
        if last < 0:
            continue
        j = np.arange(last + 1)
        if window:
            j = j[(j > p - window) | (j < sinks)]
        if not len(j):
            continue
        for h in range(nh):
            s = k[j, h // (nh // nk)] @ q[i, h, :hd_kv].astype(np.float64) * scale
            w = np.exp(s - s.max())
            out[i, h] = (w / w.sum()) @ v[j, h // (nh // nk)]
    return out.reshape(len(q), nh * hd_kv)


class Batch:
    """Sequences with cached rows and new tokens, paged or in an arena, on the host and the device."""

    def __init__(self, geom, kind, new, past, paged, block=16, seed=0, pad=(0, 0), room=5, poison=None, window=0,
                 sinks=0):
        self.geom, self.kind, self.new, self.past, self.paged, self.block = geom, kind, new, past, paged, block
        self.window, self.sinks = window, sinks
        nh, nk, hd, hd_kv = geom
        r = rng(seed, nh, hd, len(new), sum(new))
        w = self.w = nk * hd_kv
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + pad[0]
        self.nt = int(self.starts[-1]) + pad[1]
        self.q = r.standard_normal((self.nt, nh, hd)).astype(np.float32)
        self.caps = [max(1, c + p + room) if not paged else 0 for c, p in zip(new, past)]
        n = len(new)
        if paged:
            need = [max(0, -(-(c + p) // block)) for c, p in zip(new, past)]
            self.max_blocks = max(1, max(need)) + 1
            ids = r.permutation(sum(need) + 3)
            self.table = np.full((n, self.max_blocks), -1, np.int32)
            at = 0
            for s, c in enumerate(need):
                self.table[s, :c] = ids[at:at + c]
                at += c
            self.pool_rows = (sum(need) + 3) * block
            self.caps = [self.max_blocks * block] * n
        else:
            self.row_off = np.concatenate([[0], np.cumsum(self.caps)[:-1]]).astype(np.int64) + 7
            self.pool_rows = int(sum(self.caps)) + 11
        xk = r.standard_normal((self.pool_rows, w)).astype(np.float32)
        xv = r.standard_normal((self.pool_rows, w)).astype(np.float32)
        if poison is not None:  # rows that no token sees hold what must not reach a result
            seen = np.zeros(self.pool_rows, bool)
            for s in range(n):
                for i in range(new[s]):
                    p = past[s] + i
                    for j in range(max(0, min(p, self.caps[s] - 1) + 1)):
                        if not window or j > p - window or j < sinks:
                            seen[self.row(s, j)] = True
            xk[~seen], xv[~seen] = poison, poison
        with np.errstate(over="ignore", invalid="ignore"):
            self.k, self.v = hold(xk, kind), hold(xv, kind)
        if poison is not None and kind == "q8":
            for rows in (self.k, self.v):
                rows[~seen, w:w + w // 16] = np.full(w // 32, poison, np.float16).view(np.uint8)

    def row(self, s, j):
        if not self.paged:
            return int(self.row_off[s]) + j
        return int(self.table[s, j // self.block]) * self.block + j % self.block

    def run(self, m, max_chunk=None, out=None, ws=None, scale=None, stream=None):
        nh, nk, hd, hd_kv = self.geom
        n = len(self.new)
        max_chunk = max_chunk or max(1, max(self.new))
        self.scale = hd ** -0.5 if scale is None else scale
        out = torch.full((self.nt, nh * hd_kv), 7.0, device="cuda") if out is None else out
        ws = m.kv.chunk_workspace(self.nt, n, nh, nk, hd_kv, max_chunk) if ws is None else ws
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        tail = (i32(self.starts), i32(self.past), max_chunk, nh, nk, hd, hd_kv, self.scale, self.window, self.sinks, ws,
                err)
        q, k, v = dev(self.q), dev(self.k), dev(self.v)
        if self.paged:
            getattr(m, "minf_gqa_attn_chunk_paged" + END[self.kind])(out, q, k, v, i32(self.table), self.block, *tail,
                                                                     stream=stream)
        else:
            getattr(m, "minf_gqa_attn_window" + END[self.kind])(out, q, k, v, dev(self.row_off), i32(self.caps),
                                                                max(self.caps), *tail, stream=stream)
        torch.cuda.synchronize()
        return out.cpu().numpy(), int(err.item())

    def ref(self):
        nh, nk, hd, hd_kv = self.geom
        out = np.full((self.nt, nh * hd_kv), 7.0)
        for s, (c, p) in enumerate(zip(self.new, self.past)):
            rows = [self.row(s, j) for j in range(min(max(0, p + c), self.caps[s]))]
            k = value(self.k[rows], self.kind, self.w).reshape(-1, nk, hd_kv)
            v = value(self.v[rows], self.kind, self.w).reshape(-1, nk, hd_kv)
            a = int(self.starts[s])
            out[a:a + c] = ref_attention(self.q[a:a + c], k, v, p, self.caps[s], nh, nk, hd_kv, self.scale, self.window,
                                         self.sinks)
        return out


def check(m, b, err=0, **kw):
    got, e = b.run(m, **kw)
    close(got, b.ref(), f"{b.geom} {b.kind} new {b.new} past {b.past} window {b.window}/{b.sinks}")
    assert e == err
    return got


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_single_tokens(m, geom, kind):
    # one token a sequence: no past, a tile's end, beyond it, several tiles
    check(m, Batch(geom, kind, [1] * 7, [0, 1, 62, 63, 64, 127, 391], paged=True, block=32, seed=1))
    check(m, Batch(geom, kind, [1] * 3, [0, 64, 300], paged=False, seed=2))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_chunks(m, geom, kind):
    # a sequence without tokens, one token, odd chunks, chunks with and without a past
    check(m, Batch(geom, kind, [5, 0, 1, 130, 33], [0, 40, 200, 65, 0], paged=True, block=16, seed=3))
    check(m, Batch(geom, kind, [67, 2], [130, 17], paged=False, seed=4))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_few_tokens(m, geom, kind):
    # drafted tokens: up to 8, 16 and 32 query rows a kv head, with and without a window
    g = geom[0] // geom[1]
    for rows, past in ((8, [0, 63, 200]), (16, [130, 5, 64]), (32, [700, 0, 31])):
        n = max(1, rows // g)
        check(m, Batch(geom, kind, [n, max(1, n - 1), 1], past, paged=True, block=32, seed=28))
        check(m, Batch(geom, kind, [1, n], past[:2], paged=False, seed=29, window=70, sinks=2))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (40, 4), (63, 70), (64, 1), (1000, 4)])
def test_window_and_sinks(m, kind, window, sinks):
    check(m, Batch((14, 2, 64, 64), kind, [1, 150, 9], [333, 20, 0], paged=False, seed=5, window=window, sinks=sinks))
    check(m, Batch((16, 8, 128, 128), kind, [1, 1, 1, 2], [0, 500, 129, 250], paged=True, block=16, seed=6,
                   window=window, sinks=sinks))


@pytest.mark.parametrize("block", [16, 64, 256, 4096])
def test_block_sizes(m, block):
    check(m, Batch((16, 8, 128, 128), "f16", [70, 1], [250, 511], paged=True, block=block, seed=7))
    check(m, Batch((14, 2, 64, 64), "q8", [1, 3], [250, 511], paged=True, block=block, seed=8))


@pytest.mark.parametrize("kind", KINDS)
def test_long_rows_split_and_joined(m, kind):
    # few rows over many keys: the keys are split and the parts joined
    check(m, Batch((14, 2, 64, 64), kind, [1], [5000], paged=True, block=64, seed=9))
    check(m, Batch((3, 3, 128, 128), kind, [40], [3000], paged=False, seed=10))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("poison", [np.inf, np.nan, -np.inf, 1e30])
@pytest.mark.parametrize("paged", [True, False])
def test_hidden_rows_do_not_matter(m, kind, poison, paged):
    if kind == "f32" and poison == 1e30:
        poison = 3e38  # the type's largest magnitudes
    for new, window, sinks in (([1, 1], 0, 0), ([1, 1], 50, 3), ([70, 5], 0, 0), ([70, 5], 50, 3)):
        check(m, Batch((16, 8, 128, 128), kind, new, [200, 90], paged=paged, block=32, seed=11, poison=poison,
                       window=window, sinks=sinks))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [np.nan, np.inf, 6e4])
def test_a_row_reaches_only_the_tokens_that_see_it(m, kind, bad):
    # the chunk's own row 200 + 9 is seen by later tokens only, and only within their window
    for new in ([40], [12]):
        b = Batch((14, 2, 64, 64), kind, new, [200], paged=True, block=16, seed=12, window=20, sinks=2)
        row = b.row(0, 209)
        if kind == "q8":
            b.v[row, b.w:b.w + 2] = np.array([bad], np.float16).view(np.uint8)
        else:
            b.v[row, 3] = bad
        got, err = b.run(m)
        clean = Batch((14, 2, 64, 64), kind, new, [200], paged=True, block=16, seed=12, window=20, sinks=2)
        clean.scale = b.scale
        want = clean.ref()
        blind = [i for i in range(new[0]) if i < 9 or i >= 29]
        close(got[blind], want[blind], "tokens that do not see the row")
        assert err == 0
        sees = got[9:min(29, new[0])].reshape(-1, 14, 64)[:, 0]
        hit = sees if kind == "q8" else sees[:, 3:4]
        if not np.isfinite(bad):
            assert not np.isfinite(hit[:, :1]).any()


@pytest.mark.parametrize("kind", KINDS)
def test_ranges_of_values(m, kind):
    # rows of very different magnitude side by side, large and small queries
    for scale_k, scale_v in ((1e-3, 1e-4), (30.0, 100.0)):
        b = Batch((16, 8, 128, 128), kind, [20, 1], [100, 77], paged=True, block=16, seed=13)
        x = rng(13, 7).standard_normal((b.pool_rows, b.w)).astype(np.float32)
        mag = np.exp2(rng(13, 8).integers(-6, 7, (b.pool_rows, 1))).astype(np.float32)
        b.k, b.v = hold(x * np.float32(scale_k), kind), hold(x * mag * np.float32(scale_v), kind)
        b.q = (b.q / np.float32(scale_k)).astype(np.float32)
        got, err = b.run(m)
        ref = b.ref()
        # relative to the largest value a row can take
        big = scale_v * 2.0 ** 6 * 5
        assert np.abs(got - ref).max() <= 1e-5 * big and err == 0


def test_rows_outside_every_chunk_stay(m):
    b = Batch((14, 2, 64, 64), "f16", [3, 0, 40], [5, 9, 100], paged=True, seed=14, pad=(2, 6))
    got = check(m, b)
    assert (got[:2] == 7).all() and (got[-6:] == 7).all()
    b = Batch((14, 2, 64, 64), "q8", [1, 2], [5, 100], paged=True, seed=14, pad=(1, 3))
    got = check(m, b)
    assert (got[:1] == 7).all() and (got[-3:] == 7).all()


@pytest.mark.parametrize("new", [[1, 1], [40, 3]])
def test_positions_outside_are_reported(m, new):
    # a negative past: the tokens before position 0 see nothing
    b = Batch((16, 8, 128, 128), "f32", new, [-2, 30], paged=False, seed=15)
    got = check(m, b, err=0x4)
    assert (got[0] == 0).all()
    # positions past the capacity: the window is clamped
    b = Batch((16, 8, 128, 128), "f16", new, [90, 10], paged=False, seed=16)
    b.caps = [80, b.caps[1]]
    check(m, b, err=0x4)


@pytest.mark.parametrize("new", [[1, 1], [40, 3]])
def test_missing_blocks(m, new):
    # a block that is needed: reported, read as zeros, the other sequence is not touched
    b = Batch((16, 8, 128, 128), "f16", new, [100, 60], paged=True, block=16, seed=17)
    b.table[0, 2] = -1
    got, err = b.run(m)
    assert err == 0x10
    a = int(b.starts[1])
    want = Batch((16, 8, 128, 128), "f16", new, [100, 60], paged=True, block=16, seed=17)
    want.scale = b.scale
    close(got[a:], want.ref()[a:])
    b.table[0, 2] = b.pool_rows // b.block
    assert b.run(m)[1] == 0x10
    # blocks that left the window are not needed
    b = Batch((16, 8, 128, 128), "f16", new, [100, 60], paged=True, block=16, seed=18, window=20, sinks=3)
    ref_b = Batch((16, 8, 128, 128), "f16", new, [100, 60], paged=True, block=16, seed=18, window=20, sinks=3)
    b.table[0, 1:5] = [-1, 9999, -5, -1]
    got, err = b.run(m)
    ref_b.scale = b.scale
    close(got, ref_b.ref())
    assert err == 0


@pytest.mark.parametrize("starts", [[0, 5, 3, 8], [-1, 2, 4, 8], [0, 3, 5, 9]])
def test_chunk_offsets_out_of_order_are_reported(m, starts):
    b = Batch((14, 2, 64, 64), "f16", [3, 2, 3], [5, 9, 100], paged=True, seed=19)
    b.starts = np.array(starts, np.int32)
    for max_chunk in (1, 64):
        got, err = b.run(m, max_chunk=max_chunk)
        assert err & 0x40 and (got == 7).all()


@pytest.mark.parametrize("kind", KINDS)
def test_max_chunk_is_only_a_hint(m, kind):
    b = Batch((14, 2, 64, 64), kind, [50, 1, 3], [70, 200, 0], paged=True, seed=20)
    a = check(m, b, max_chunk=1)
    c = check(m, b, max_chunk=4096)
    close(a, c)


def test_scale_is_the_callers(m):
    for scale in (0.0, -0.3, 1.7):
        check(m, Batch((14, 2, 64, 64), "f16", [20], [70], paged=True, seed=21), scale=scale)
        check(m, Batch((14, 2, 64, 64), "q8", [1], [70], paged=True, seed=21), scale=scale)


def test_repeatable_and_on_another_stream(m):
    # joined splits in a fixed order: the same bits every time, on any stream
    for new in ([1, 1, 1], [100, 30, 1]):
        b = Batch((16, 8, 128, 128), "f16", new, [900, 1500, 3], paged=True, block=64, seed=22)
        first, _ = b.run(m)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        for k in range(3):
            again, _ = b.run(m, stream=stream if k else None)
            assert np.array_equal(first, again)


def test_two_calls_at_once(m):
    # on two streams, each with a workspace of its own: the bits of the calls made alone
    calls = []
    for kind, new in (("f16", [200, 3, 90]), ("q8", [60, 1, 1]), ("f32", [1, 1, 1])):
        b = Batch((16, 8, 128, 128), kind, new, [900, 1500, 40], paged=True, block=64, seed=35)
        alone, err = b.run(m)
        assert err == 0
        nh, nk, hd, hd_kv = b.geom
        args = (dev(b.q), dev(b.k), dev(b.v), i32(b.table), b.block, i32(b.starts), i32(b.past), max(new), nh, nk, hd, hd_kv,
                b.scale, 0, 0)
        calls.append((getattr(m, "minf_gqa_attn_chunk_paged" + END[kind]), args, alone,
                      m.kv.chunk_workspace(b.nt, 3, nh, nk, hd_kv, max(new)), torch.cuda.Stream(),
                      [torch.full((b.nt, nh * hd_kv), 7.0, device="cuda") for _ in range(6)], i32([0])))
    torch.cuda.synchronize()
    for k in range(6):
        for f, args, _, ws, stream, outs, err in calls:
            f(outs[k], *args, ws, err, stream=stream)
    torch.cuda.synchronize()
    for _, _, alone, _, _, outs, err in calls:
        assert err.item() == 0
        for out in outs:
            assert np.array_equal(out.cpu().numpy(), alone)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("max_chunk", [1, 64])
def test_graph_replays_with_other_lengths(m, kind, max_chunk):
    nh, nk, hd, hd_kv = geom = (16, 8, 128, 128)
    plans = [([3, 1, 2], [100, 7, 300]), ([1, 4, 1], [513, 0, 40]), ([0, 5, 1], [9, 500, 700])]
    base = Batch(geom, kind, [0, 0, 0], [800, 800, 800], paged=True, block=32, seed=23)
    q, k, v, table = dev(base_q(6, nh, hd)), dev(base.k), dev(base.v), i32(base.table)
    off, past = i32([0, 3, 4, 6]), i32([100, 7, 300])
    out, err = torch.zeros(6, nh * hd_kv, device="cuda"), i32([0])
    ws = m.kv.chunk_workspace(6, 3, nh, nk, hd_kv, max_chunk)
    ws.fill_(0xA5)  # needs no preparation

    def call():
        getattr(m, "minf_gqa_attn_chunk_paged" + END[kind])(out, q, k, v, table, 32, off, past, max_chunk, nh, nk, hd,
                                                            hd_kv, hd ** -0.5, 0, 0, ws, err)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for new, pst in plans:
        base.new, base.past, base.starts = new, pst, np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        base.nt, base.q, base.scale = 6, q.cpu().numpy(), hd ** -0.5
        off.copy_(i32(base.starts))
        past.copy_(i32(pst))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        ref = base.ref()
        ref[int(base.starts[-1]):] = 0
        close(out.cpu().numpy(), ref, f"replay {new}")
    assert err.item() == 0


def base_q(nt, nh, hd):
    return rng(31).standard_normal((nt, nh, hd)).astype(np.float32)


def test_two_calls_share_a_workspace_in_turn(m):
    a = Batch((16, 8, 128, 128), "f16", [90, 30], [900, 0], paged=True, block=64, seed=24)
    b = Batch((14, 2, 64, 64), "q8", [1, 1], [4000, 3], paged=False, seed=25)
    need = max(m.minf_attn_chunk_workspace_bytes(120, 2, 16, 8, 128, 90), m.minf_attn_chunk_workspace_bytes(2, 2, 14, 2, 64, 1))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        check(m, a, ws=ws)
        check(m, b, ws=ws)


def test_offsets_past_32_bits(m):
    # the sequence's rows start 4.4 GB into a binary16 arena
    nh, nk, hd, w = 16, 8, 128, 1024
    rows = 2_200_000
    k, v = (torch.empty(rows, w, dtype=torch.float16, device="cuda") for _ in range(2))
    r0, past = rows - 300, 250
    b = Batch((nh, nk, hd, hd), "f16", [1, 40], [past, 100], paged=False, seed=26)
    for s, at in ((0, r0), (1, 2_150_000)):
        idx = [b.row(s, j) for j in range(b.caps[s])]
        k[at:at + b.caps[s]] = dev(b.k[idx])
        v[at:at + b.caps[s]] = dev(b.v[idx])
    off, cap = dev(np.array([r0, 2_150_000], np.int64)), i32(b.caps)
    for max_chunk in (1, 40):
        out, err = torch.empty(41, nh * hd, device="cuda"), i32([0])
        ws = m.kv.chunk_workspace(41, 2, nh, nk, hd, max_chunk)
        m.minf_gqa_attn_window_f16(out, dev(b.q), k, v, off, cap, max(b.caps), i32(b.starts), i32(b.past), max_chunk, nh,
                                   nk, hd, hd, hd ** -0.5, 0, 0, ws, err)
        b.scale = hd ** -0.5
        close(out.cpu().numpy(), b.ref())
        assert err.item() == 0


def test_regions_of_one_sequence(m):
    # seq_row_off and chunk_off left out: plain regions, one token
    b = Batch((14, 2, 64, 64), "f32", [1], [333], paged=False, seed=27, window=100, sinks=4)
    nh, nk, hd, hd_kv = b.geom
    k, v = dev(b.k[7:7 + b.caps[0]]), dev(b.v[7:7 + b.caps[0]])
    out, err = torch.empty(1, nh * hd_kv, device="cuda"), i32([0])
    ws = m.kv.chunk_workspace(1, 1, nh, nk, hd_kv, 1)
    m.minf_gqa_attn_window(out, dev(b.q), k, v, None, None, b.caps[0], None, i32([333]), 1, nh, nk, hd, hd_kv,
                           hd ** -0.5, 100, 4, ws, err)
    b.scale = hd ** -0.5
    close(out.cpu().numpy(), b.ref())
    assert err.item() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("long", [0, 25])
def test_many_sequences(m, kind, long):
    # more sequences than the plan has threads, and than it holds in shared memory; some without tokens
    r = rng(30, long)
    new = r.integers(0, 3, 1300)
    new[[3, 600, 1299]] = max(2, long)
    check(m, Batch((8, 1, 64, 64), kind, new.tolist(), r.integers(0, 150, 1300).tolist(), paged=True, block=16, seed=30))


def test_many_token_tiles(m):
    # more token tiles than the plan holds in shared memory
    check(m, Batch((8, 1, 64, 64), "f16", [18000], [5], paged=False, seed=31, window=24, sinks=2))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [[20, 1], [3]])
def test_rows_of_one_tile_far_apart(m, kind, new):
    # rows whose magnitudes differ by up to 2^24 in one tile of keys, and blocks that differ in one row;
    # an output is off by no more than 1e-5 of the largest value that it could have been
    b = Batch((16, 8, 128, 128), kind, new, [300, 77][:len(new)], paged=True, block=16, seed=32)
    mag_k, mag_v = (np.exp2(rng(32, k).integers(-12, 13, (b.pool_rows, 1))).astype(np.float32) for k in (1, 2))
    x, y = (rng(32, k).standard_normal((b.pool_rows, b.w)).astype(np.float32) for k in (3, 4))
    y[:, ::64] *= np.float32(2.0 ** -8)
    b.k, b.v = hold(x * mag_k, kind), hold(y * mag_v, kind)
    b.q = b.q * np.float32(2.0 ** -12)
    got, err = b.run(m)
    assert np.abs(got - b.ref()).max() <= 1e-5 * 5 * 2.0 ** 12 and err == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [[1], [32]])
@pytest.mark.parametrize("gap", [13, 17, 20])
def test_many_small_weights_beside_a_large_one(m, kind, new, gap):
    # row 0 weighs 2^gap times any other row.  60032 weights that are each off by 2^-37 of the largest, in the
    # numerator and (not rounded) the sum: 4.4e-7; a stretch of at most 4 tiles adds 4 * 16 products' sums
    # a row, each off by 2^-23 of it: 7.6e-6.  Together below 1e-5.
    nk, hd, past = 1, 64, 60000
    b = Batch((4, nk, hd, hd), kind, new, [past], paged=False, seed=33)
    k, v = np.zeros((b.pool_rows, b.w), np.float32), np.ones((b.pool_rows, b.w), np.float32)
    row = b.row(0, 0)
    k[row, 0], v[row] = gap * np.log(2.0), -1.0
    b.k, b.v = hold(k, kind), hold(v, kind)
    b.q[:] = 0.0
    b.q[:, :, 0] = 1.0
    got, err = b.run(m, scale=1.0)
    assert np.abs(got - b.ref()).max() <= 1e-5 and err == 0


def test_scale_that_is_not_a_number(m):
    for new in ([20], [1]):
        b = Batch((14, 2, 64, 64), "f16", new, [70], paged=True, seed=34)
        got, err = b.run(m, scale=float("nan"))
        assert np.isnan(got).all() and err == 0


def test_rows_that_take_long_do_not_run_out_of_time(m):
    # an infinity that every token sees: all rows are computed again key by key, far beyond a wait's limit
    nh, hd, new, past = 8, 64, 4864, 80000
    cap = new + past
    k, v = (torch.randn(cap, hd, device="cuda", generator=torch.Generator("cuda").manual_seed(s)).half() for s in (1, 2))
    v[0, 0] = float("inf")
    q = torch.randn(new, nh, hd, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    out, err = torch.empty(new, nh * hd, device="cuda"), i32([0])
    ws = m.kv.chunk_workspace(new, 1, nh, 1, hd, new)
    m.minf_gqa_attn_window_f16(out, q, k, v, None, None, cap, i32([0, new]), i32([past]), new, nh, 1, hd, hd, hd ** -0.5, 0,
                               0, ws, err)
    assert err.item() == 0
    out = out.view(new, nh, hd)
    assert torch.isinf(out[:, :, 0]).all() and torch.isfinite(out[:, :, 1:]).all()
    for t in (0, 777, new - 1):
        s = (q[t].double() @ k[:past + t + 1].double().T) * hd ** -0.5
        ref = torch.softmax(s, -1) @ v[:past + t + 1, 1:].double()
        close(out[t, :, 1:].cpu().numpy(), ref.cpu().numpy())


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("n_seq,new,past", [(152, 1, 65536), (152, 3, 50000), (40, 64, 30000)])
def test_sums_over_many_keys(m, kind, n_seq, new, past):
    # one CTA goes over all of a sequence's keys.  Sums of 16 or 128 keys are cut off below 2^-23, once; adding
    # up to 512 of them rounds by 2^-25 each, independently: 7e-7; a weight is off by its score's rounding and
    # the exponential's, below 2e-6 together: 4e-6 of the result in the 2-norm.
    # (The sequences share their rows.)
    nh, hd, cap = 8, 64, past + new
    gen = torch.Generator("cuda").manual_seed(past)
    k, v = (torch.randn(cap, hd, device="cuda", generator=gen).to(torch.float16 if kind == "f16" else torch.float32)
            for _ in range(2))
    v = v + 1
    nt = n_seq * new
    q = torch.randn(nt, nh, hd, device="cuda", generator=gen)
    out, err = torch.empty(nt, nh * hd, device="cuda"), i32([0])
    ws = m.kv.chunk_workspace(nt, n_seq, nh, 1, hd, new)
    getattr(m, "minf_gqa_attn_window" + END[kind])(
        out, q, k, v, torch.zeros(n_seq, dtype=torch.int64, device="cuda"), None, cap, i32(np.arange(n_seq + 1) * new),
        i32([past] * n_seq), new, nh, 1, hd, hd, hd ** -0.5, 0, 0, ws, err)
    assert err.item() == 0
    for t in (0, nt // 2, nt - 1):
        p = past + t % new
        ref = torch.softmax(q[t].double() @ k[:p + 1].double().T * hd ** -0.5, -1) @ v[:p + 1].double()
        assert (out[t].view(nh, hd) - ref).norm() <= 4e-6 * ref.norm()


# ----------------------------------------------------------------------------- rotation
def ref_rope(x, pos, axis, hd, style):
    """x [nt, heads, hd], pos [n_axis, nt]: (rotated, |a| + |b| of each value's pair), in 64 bits."""
    y, size = np.array(x, np.float64), np.zeros(x.shape)
    for i in range(hd // 2):
        a, b = (i, i + hd // 2) if style == 0 else (2 * i, 2 * i + 1)
        th = pos[axis[i]].astype(np.float64)[:, None] * THETA ** (-2.0 * i / hd)
        ok = (pos[sorted(set(axis))] >= 0).all(0)[:, None]
        th = np.where(ok, th, 0.0)
        xa, xb = x[:, :, a].astype(np.float64), x[:, :, b].astype(np.float64)
        y[:, :, a], y[:, :, b] = xa * np.cos(th) - xb * np.sin(th), xa * np.sin(th) + xb * np.cos(th)
        size[:, :, a] = size[:, :, b] = np.abs(xa) + np.abs(xb)
    return y, size


def sections(hd, counts):
    out = []
    for a, c in enumerate(counts):
        out += [a] * c
    assert len(out) == hd // 2
    return out


AXES = {2: [0], 6: [0, 1, 2], 30: [1] * 5 + [0] * 10, 64: sections(64, [8, 12, 12]), 100: [0, 1] * 25,
        128: sections(128, [16, 24, 24]), 256: [i % 4 for i in range(128)]}


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("hd", sorted(AXES))
@pytest.mark.parametrize("nt", [1, 3, 700])
def test_rope_axes(m, hd, style, nt):
    r = rng(41, hd, nt)
    axis = AXES[hd]
    n_axis, heads = max(axis) + 1, 3
    x = r.standard_normal((nt, heads, hd)).astype(np.float32)
    pos = r.integers(0, 1 << r.integers(1, 18), (n_axis, nt)).astype(np.int32)
    pos[:, 0] = [5_000_001, 0, 40961, 5][:n_axis]  # (2^-53 of such an angle is still below 1e-8)
    y, err = torch.full((nt, heads, hd), 9.0, device="cuda"), i32([0])
    xd = dev(x)
    m.minf_rope_axes(y, xd, i32(pos), axis, heads, hd, THETA, 1.0, style, err)
    want, size = ref_rope(x, pos, axis, hd, style)
    assert (np.abs(y.cpu().numpy() - want) <= 3.5e-7 * size).all() and err.item() == 0
    assert np.array_equal(xd.cpu().numpy(), x)
    m.minf_rope_axes(xd, xd, i32(pos), axis, heads, hd, THETA, 1.0, style, err)  # in place: the same bits
    assert torch.equal(xd, y)


def test_rope_axes_is_plain_rope_with_one_axis(m):
    # against minf_rope at positions where its fp32 angle loses little (2^-24 of at most 500)
    x, pos = rng(42).standard_normal((50, 4, 128)).astype(np.float32), rng(43).integers(0, 500, 50).astype(np.int32)
    a, b, err = dev(x), dev(x), i32([0])
    m.minf_rope(a, i32(pos), 4, 128, THETA, 1.0, 0, err)
    m.minf_rope_axes(b, b, i32(pos), None, 4, 128, THETA, 1.0, 0, err)
    assert (a - b).abs().max().item() <= 500 * 2 ** -24 * 10 and err.item() == 0


def test_rope_axes_negative_position(m):
    x = rng(44).standard_normal((4, 2, 64)).astype(np.float32)
    pos = np.array([[1, 2, -3, 4], [5, 6, 7, 8]], np.int32)
    y, err = torch.empty(4, 2, 64, device="cuda"), i32([0])
    m.minf_rope_axes(y, dev(x), i32(pos), [0] * 16 + [1] * 16, 2, 64, THETA, 1.0, 0, err)
    got = y.cpu().numpy()
    assert err.item() == 0x2 and np.array_equal(got[2], x[2]) and not np.array_equal(got[1], x[1])


# ----------------------------------------------------------------------------- store and read back
def store_case(m, geom, kind, new, past, axis, style, block=16, seed=0, pad=(0, 0), k_back=True, rope_pos=True):
    nh, nk, hd, hd_kv = geom
    b = Batch(geom, kind, new, past, paged=True, block=block, seed=seed, pad=pad)
    r = rng(51, seed)
    n_axis = max(axis) + 1
    k = r.standard_normal((b.nt, nk, hd_kv)).astype(np.float32)
    v = r.standard_normal((b.nt, b.w)).astype(np.float32)
    k[:, 0, :2] *= 100
    v[-1, :32] = 0  # a block of zeros
    pos = r.integers(0, 30000, (n_axis, b.nt)).astype(np.int32)
    kp, vp, q, err = dev(b.k), dev(b.v), dev(b.q), i32([0])
    q_out, k_out = torch.full_like(q, 3.0), torch.full((b.nt, nk, hd_kv), 3.0, device="cuda")
    getattr(m, "minf_rope_kv_append_chunk_paged" + END[kind])(
        q_out, k_out if k_back else None, q, dev(k), dev(v), i32(pos) if rope_pos else None,
        axis if n_axis > 1 else None, i32(b.starts), i32(past), nh, nk, hd, hd_kv, THETA, 1.0, style, kp, vp,
        i32(b.table), block, err)
    torch.cuda.synchronize()
    return b, k, v, pos, q_out.cpu().numpy(), k_out.cpu().numpy(), kp, vp, int(err.item())


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_store_and_read_back(m, geom, kind, style):
    nh, nk, hd, hd_kv = geom
    axis = [min(2, i // 12) for i in range(hd // 2)]
    for new, past in (([1], [31]), ([5, 0, 30, 1], [0, 4, 14, 100]), ([700, 900, 300, 600], [0, 31, 5, 8])):
        b, k, v, pos, q_out, k_out, kp, vp, err = store_case(m, geom, kind, new, past, axis, style, seed=len(new))
        assert err == 0
        want, size = ref_rope(b.q, pos, axis, hd, style)
        assert (np.abs(q_out - want) <= 3.5e-7 * size).all()
        want, size = ref_rope(k, pos, axis[:hd_kv // 2], hd_kv, style)
        assert (np.abs(k_out - want) <= 3.5e-7 * size).all()
        # the pools: the tokens' rows hold k_out and v exactly as the kind holds them, all others are as they were
        want_k, want_v = b.k.copy(), b.v.copy()
        rows = [b.row(s, past[s] + i) for s in range(len(new)) for i in range(new[s])]
        want_k[rows], want_v[rows] = hold(k_out.reshape(b.nt, b.w), kind), hold(v, kind)
        assert np.array_equal(kp.cpu().numpy().view(np.uint8), want_k.view(np.uint8))
        assert np.array_equal(vp.cpu().numpy().view(np.uint8), want_v.view(np.uint8))
        for dt in (torch.float32, torch.float16):
            kr, vr = (torch.full((b.nt, b.w), 5.0, dtype=dt, device="cuda") for _ in range(2))
            e = i32([0])
            getattr(m, "minf_kv_read_chunk_paged" + END[kind])(kr, vr, kp, vp, i32(b.table), 16, i32(b.starts),
                                                               i32(past), e)
            for got, held in ((kr, want_k), (vr, want_v)):
                x = value(held[rows], kind, b.w).astype(np.float32)
                assert np.array_equal(got.cpu().numpy(), x if dt == torch.float32 else x.astype(np.float16))
            assert e.item() == 0


def test_store_without_rope_positions_and_without_k_out(m):
    geom = (14, 2, 64, 64)
    b, k, v, _, q_out, k_out, kp, vp, err = store_case(m, geom, "f32", [4, 3], [10, 0], [0] * 32, 0, rope_pos=False,
                                                       k_back=False)
    pos = np.concatenate([10 + np.arange(4), np.arange(3)]).astype(np.int32)[None]
    want, size = ref_rope(k, pos, [0] * 32, 64, 0)
    rows = [b.row(0, 10 + i) for i in range(4)] + [b.row(1, i) for i in range(3)]
    got = kp.cpu().numpy()[rows].reshape(7, 2, 64)
    assert (np.abs(got - want) <= 3.5e-7 * size).all() and err == 0 and (k_out == 3).all()


@pytest.mark.parametrize("kind", KINDS)
def test_store_leaves_padding_and_refused_rows(m, kind):
    geom, axis = (16, 8, 128, 128), [0] * 64
    b, k, v, pos, q_out, k_out, kp, vp, err = store_case(m, geom, kind, [3, 2], [0, 7], axis, 0, pad=(2, 4))
    assert err == 0
    assert (q_out[:2] == 3).all() and (q_out[-4:] == 3).all() and (k_out[:2] == 3).all() and (k_out[-4:] == 3).all()
    assert (q_out[2:-4] != 3).any()
    # positions below 0 and past the capacity, and a missing block: reported, nothing else written
    nh, nk, hd, hd_kv = geom
    before = dev(b.k), dev(b.v)
    for past, table, bit in (([-1, 7], b.table, 0x1 | 0x2), ([b.max_blocks * 16 - 1, 7], None, 0x1 | 0x10),
                             ([0, 7], np.full_like(b.table, -1), 0x10)):
        kp, vp, e = before[0].clone(), before[1].clone(), i32([0])
        table = b.table if table is None else table
        q, kk = dev(b.q), dev(k)
        getattr(m, "minf_rope_kv_append_chunk_paged" + END[kind])(
            q, kk, q, kk, dev(v), None, None, i32(b.starts), i32(past), nh, nk, hd, hd_kv, THETA, 1.0, 0, kp, vp,
            i32(table), 16, e)
        assert e.item() == bit
        touched = [b.row(s, past[s] + i) for s in range(2) for i in range((3, 2)[s])
                   if 0 <= past[s] + i < b.max_blocks * 16 and table[s, (past[s] + i) // 16] >= 0]
        same = np.ones(b.pool_rows, bool)
        same[touched] = False
        keep = torch.from_numpy(same).cuda()
        assert torch.equal(kp[keep].view(torch.uint8), before[0][keep].view(torch.uint8))
        assert torch.equal(vp[keep].view(torch.uint8), before[1][keep].view(torch.uint8))


def test_read_back_of_rows_that_are_not_there(m):
    b = Batch((14, 2, 64, 64), "f16", [2, 2], [15, 3], paged=True, seed=60, pad=(0, 2))
    b.table[0, 1] = -1
    kr, vr, e = torch.full((6, b.w), 5.0, device="cuda"), torch.full((6, b.w), 5.0, device="cuda"), i32([0])
    m.minf_kv_read_chunk_paged_f16(kr, vr, dev(b.k), dev(b.v), i32(b.table), 16, i32(b.starts), i32(b.past), e)
    got = kr.cpu().numpy()
    assert e.item() == 0x10 and (got[1] == 0).all() and (got[4:] == 5).all()
    assert np.array_equal(got[0], b.k[b.row(0, 15)].astype(np.float32))
    assert np.array_equal(vr.cpu().numpy()[2], b.v[b.row(1, 3)].astype(np.float32))


# ----------------------------------------------------------------------------- together
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_layer_steps_prompt_then_decode(m, kind, window, sinks):
    """Two prompts in two chunks each, then three decode steps, through the layer step; the separate
    calls give the same bits, and the last token's output is the 64-bit attention over what the
    pools hold."""
    nh, nk, hd, hd_kv = geom = (14, 2, 64, 64)
    n_embd, block, w = 224, 16, nk * hd_kv
    r = rng(71)
    table = r.permutation(20)[:18].reshape(2, 9).astype(np.int32)
    axis = sections(64, [8, 12, 12])
    pools = [torch.zeros(20 * block, q8_row_bytes(w) if kind == "q8" else w, device="cuda",
                         dtype={"f32": torch.float32, "f16": torch.float16, "q8": torch.uint8}[kind]) for _ in range(4)]
    past = np.array([0, 0], np.int32)
    gain = dev(r.uniform(0.5, 1.5, n_embd).astype(np.float32))
    for new in ([40, 33], [25, 1], [1, 1], [1, 1], [1, 1]):
        nt, off = sum(new), i32(np.concatenate([[0], np.cumsum(new)]))
        h = dev(r.standard_normal((nt, n_embd)).astype(np.float32))
        q, k, v = (dev(r.standard_normal((nt, c)).astype(np.float32)) for c in (nh * hd, w, w))
        q2, k2 = q.clone(), k.clone()
        pos = i32(r.integers(0, 500, (3, nt)))
        xn, xn2, out, out2 = torch.empty_like(h), torch.empty_like(h), *(torch.empty(nt, nh * hd_kv, device="cuda")
                                                                        for _ in range(2))
        err, np_dev = i32([0]), i32(past)
        ws = m.kv.chunk_workspace(nt, 2, nh, nk, hd_kv, max(new))
        getattr(m, "minf_layer_attn_step_chunk_paged" + END[kind])(
            xn, h, gain, 1e-6, q, k, v, pos, axis, off, np_dev, max(new), pools[0], pools[1], i32(table), block, nh, nk,
            hd, hd_kv, THETA, 1.0, 0, window, sinks, out, ws, err)
        m.minf_rms_norm(xn2, h, gain, 1e-6)
        getattr(m, "minf_rope_kv_append_chunk_paged" + END[kind])(
            q2, k2, q2, k2, v, pos, axis, off, np_dev, nh, nk, hd, hd_kv, THETA, 1.0, 0, pools[2], pools[3], i32(table),
            block, err)
        getattr(m, "minf_gqa_attn_chunk_paged" + END[kind])(
            out2, q2, pools[2], pools[3], i32(table), block, off, np_dev, max(new), nh, nk, hd, hd_kv, hd ** -0.5,
            window, sinks, ws, err)
        for a, b in ((xn, xn2), (q, q2), (k, k2), (out, out2), (pools[0], pools[2]), (pools[1], pools[3])):
            assert torch.equal(a, b)
        assert err.item() == 0
        at = 0
        for s in range(2):
            rows = [int(table[s, j // block]) * block + j % block for j in range(past[s] + new[s])]
            kk = value(pools[0].cpu().numpy()[rows], kind, w).reshape(-1, nk, hd_kv)
            vv = value(pools[1].cpu().numpy()[rows], kind, w).reshape(-1, nk, hd_kv)
            want = ref_attention(q.cpu().numpy()[at:at + new[s]].reshape(-1, nh, hd), kk, vv, int(past[s]), 9 * block,
                                 nh, nk, hd_kv, hd ** -0.5, window, sinks)
            close(out.cpu().numpy()[at:at + new[s]], want, f"layer step, sequence {s}, {new}")
            at += new[s]
        past = past + np.array(new, np.int32)


def test_decode_agrees_with_the_paged_decode(m):
    # the same rows through minf_gqa_attn_decode_paged_f16
    nh, nk, hd, hd_kv = geom = (16, 8, 128, 128)
    b = Batch(geom, "f16", [1, 1, 1], [5, 300, 1000], paged=True, block=64, seed=80)
    got, _ = b.run(m)
    out, err = torch.empty(3, nh * hd_kv, device="cuda"), i32([0])
    ws = m.kv.decode_workspace(3, nh, nk, hd_kv, b.max_blocks * 64)
    table = b.table.copy()
    table[table < 0] = 0
    m.minf_gqa_attn_decode_paged_f16(out, dev(b.q), dev(b.k), dev(b.v), i32(table), 64, i32(b.past), nh, nk, hd, hd_kv,
                                     hd ** -0.5, ws, err)
    close(got, out.cpu().numpy())


def test_the_binding_checks_sizes(m):
    nh, nk, hd, hd_kv = 14, 2, 64, 64
    q, pool = torch.zeros(4, nh * hd, device="cuda"), torch.zeros(64, nk * hd_kv, device="cuda")
    out, err, table = torch.zeros(4, nh * hd_kv, device="cuda"), i32([0]), i32([[0, 1], [2, 3]])
    ws = m.kv.chunk_workspace(4, 2, nh, nk, hd_kv, 2)

    def call(q=q, pool=pool, table=table, off=i32([0, 2, 4]), past=i32([0, 0]), ws=ws, window=0, end="", hd=hd, mc=2):
        getattr(m, "minf_gqa_attn_chunk_paged" + end)(out, q, pool, pool, table, 16, off, past, mc, nh, nk, hd, hd_kv,
                                                      0.1, window, 0, ws, err)

    call()
    for kw in (dict(q=q[:3]), dict(pool=pool[:, :64]), dict(table=table[:1]), dict(off=i32([0, 4])), dict(off=None)):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(TypeError):
        call(end="_f16")
    with pytest.raises(TypeError):
        call(off=torch.tensor([0, 2, 4], device="cuda"))
    for kw, status in ((dict(window=-1), 1), (dict(ws=ws[:0]), 5), (dict(mc=0), 1)):
        with pytest.raises(m.MinfError) as e:
            call(**kw)
        assert e.value.status == status
    with pytest.raises(ValueError):
        m.minf_rope_axes(q, q, i32([0, 1, 2, 3]), [0] * 5, nh, hd, THETA, 1.0, 0, err)
