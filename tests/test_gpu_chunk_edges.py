"""The chunk operators at their edges, against the definition in 64 bits.

Tolerances are those of test_gpu_chunk.py.  Where values of very different magnitude are summed, an output is held
to 1e-5 of sum_j p_j |V_j|, the weighted sum of magnitudes: a score is off by less than 2e-6 (a few
2^-24 sum|q k| scale, below 10 here) and so a weight by 4e-6 of itself in numerator and sum together, the exponential
and the 22 bits of a value add less than 1e-6."""
import numpy as np
import pytest
import torch

from test_gpu_chunk import END, KINDS, Batch, check, close, dev, i32, m, q8_row_bytes, rng  # noqa: F401

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------- values of far apart magnitudes
def magnitude_sums(b):
    """sum_j p_j |V_j| of every output."""
    v, b.v = b.v, np.abs(b.v)
    sums = b.ref()
    b.v = v
    return sums


@pytest.mark.parametrize("new", [[40, 2], [3]])
@pytest.mark.parametrize("past", [10, 400, 3000])
def test_values_near_the_largest(m, new, past):
    # fp32 rows up to 1.5e38 beside rows of zeros: the weighted sum is finite, the sum of many such values is not
    for by_tile in (False, True):
        b = Batch((14, 2, 64, 64), "f32", new, [past, 5][:len(new)], paged=False, seed=100)
        zero = rng(100, past).random(b.pool_rows) < 0.5
        if by_tile:
            zero = (np.arange(b.pool_rows) // 128) % 2 == 0
        b.v[zero] = 0
        b.v *= np.float32(3e37)
        got, err = b.run(m)
        d = np.abs(got - b.ref())
        assert np.isfinite(got).all() and (d <= 1e-5 * magnitude_sums(b)).all() and err == 0


@pytest.mark.parametrize("new", [[40, 2], [3]])
@pytest.mark.parametrize("past", [10, 60, 400, 3000])
@pytest.mark.parametrize("sizes", [(0.0, 1.0, 1e30), (0.0, 1e-20, 1.0, 1e30), (1e-20, 1e20)])
def test_values_of_all_magnitudes_keep_their_weights(m, new, past, sizes):
    # fp32 rows, side by side in one tile and tile by tile
    for by_tile in (False, True):
        b = Batch((14, 2, 64, 64), "f32", new, [past, 5][:len(new)], paged=False, seed=101)
        pick = rng(101, past).integers(0, len(sizes), b.pool_rows)
        if by_tile:
            pick = (np.arange(b.pool_rows) // 128) % len(sizes)
        b.v = (b.v * np.array(sizes)[pick][:, None]).astype(np.float32)
        got, err = b.run(m)
        d = np.abs(got - b.ref())
        assert np.isfinite(got).all() and (d <= 1e-5 * magnitude_sums(b) + 1e-25).all() and err == 0


def test_a_row_of_zeros_beside_a_large_one_is_a_third(m):
    # equal scores, V rows 0, 1 and 1e30: a third of 1e30, for tokens that see the three
    b = Batch((14, 2, 64, 64), "f32", [40], [0], paged=False, seed=102)
    b.q[:] = 0
    b.v[:] = 0
    b.v[b.row(0, 1)], b.v[b.row(0, 2)] = 1.0, 1e30
    got, err = b.run(m)
    want = np.array([0.0, 0.5] + [1e30 / (i + 1) for i in range(2, 40)])[:, None]
    assert (np.abs(got - want) <= 1e-6 * want).all() and err == 0


# ----------------------------------------------------------------------------- scores that are minus infinity
def minus_infinity(b, rows):
    """Keys of score minus infinity (b.q's first values are positive)."""
    b.q[:, :, :32] = np.abs(b.q[:, :, :32]) + np.float32(0.1)
    for r in rows:
        if b.kind == "q8":  # a block's scale: its quants are ones
            for h in range(b.geom[1]):
                b.k[r, h * b.geom[3]:h * b.geom[3] + 32] = 1
                at = b.w + h * (b.geom[3] // 32) * 2
                b.k[r, at:at + 2] = np.array([-np.inf], np.float16).view(np.uint8)
        else:
            b.k[r, ::b.geom[3]] = -np.inf


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [[1, 1], [3, 1], [40, 2]])
@pytest.mark.parametrize("geom", [(14, 2, 64, 64), (16, 8, 128, 128)], ids=str)
def test_rows_whose_every_visible_score_is_minus_infinity(m, kind, new, geom):
    # without a past: the first token sees one key.  The softmax of nothing but minus infinities is not a number.
    b = Batch(geom, kind, new, [0, 30], paged=True, block=16, seed=103)
    minus_infinity(b, [b.row(0, 0)])
    got = check(m, b)
    assert np.isnan(got[0]).all() and np.isfinite(got[1:]).all()
    # a window that holds such keys alone, and sinks that are such keys
    for window, sinks in ((6, 0), (6, 2)):
        b = Batch(geom, kind, new, [150, 30], paged=False, seed=104, window=window, sinks=sinks)
        minus_infinity(b, [b.row(0, j) for j in list(range(sinks)) + list(range(140, 155))])
        got = check(m, b)
        assert np.isnan(got[0]).all() and np.isfinite(got[new[0]:]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_minus_infinity_over_many_parts(m, kind):
    # all of a long row's keys: the parts that are joined are all empty
    b = Batch((14, 2, 64, 64), kind, [1], [3000], paged=True, block=64, seed=105)
    minus_infinity(b, range(b.pool_rows))
    assert np.isnan(check(m, b)).all()
    b = Batch((14, 2, 64, 64), kind, [20], [3000], paged=False, seed=106)
    minus_infinity(b, range(b.pool_rows))
    assert np.isnan(check(m, b)).all()


@pytest.mark.parametrize("new", [[1, 1], [40, 2]])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_scores_past_the_range_of_fp32(m, new, sign):
    # finite rows whose products are not: about 1e40, 1e38 and more apart, so that one key has all of the weight
    b = Batch((14, 2, 64, 64), "f32", new, [70, 0], paged=True, block=16, seed=107)
    b.q = (np.abs(b.q) + 0.1).astype(np.float32) * np.float32(1e19)
    b.k = (sign * (np.abs(b.k) + 0.1) * 1e20).astype(np.float32)
    check(m, b, scale=1.0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [[1], [40]])
def test_a_scale_of_zero_times_an_infinite_score(m, kind, new):
    b = Batch((14, 2, 64, 64), kind, new, [70], paged=True, block=16, seed=108)
    minus_infinity(b, [b.row(0, 70)])
    with np.errstate(invalid="ignore"):
        got = check(m, b, scale=0.0)
    assert np.isnan(got).all()


# ----------------------------------------------------------------------------- nothing to do
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_seq", [0, 2])
def test_calls_without_tokens(m, kind, n_seq):
    # a step in which no sequence has a new token: tensors of no elements have no address
    nh, nk, hd, hd_kv = 14, 2, 64, 64
    w, end = nk * hd_kv, END[kind]
    dt = {"f32": torch.float32, "f16": torch.float16, "q8": torch.uint8}[kind]
    kp, vp = (torch.zeros(64, q8_row_bytes(w) if kind == "q8" else w, dtype=dt, device="cuda") for _ in range(2))
    q, k, v, out, h, xn = (torch.empty(0, c, device="cuda") for c in (nh * hd, w, w, nh * hd_kv, 896, 896))
    table, off = torch.zeros(n_seq, 2, dtype=torch.int32, device="cuda"), torch.zeros(n_seq + 1, dtype=torch.int32, device="cuda")
    past, err = torch.zeros(n_seq, dtype=torch.int32, device="cuda"), i32([0])
    ws, pos = m.kv.chunk_workspace(0, n_seq, nh, nk, hd_kv, 1), torch.empty(3, 0, dtype=torch.int32, device="cuda")
    axis = [0] * 10 + [1] * 10 + [2] * 12
    m.minf_rope_axes(q, q, pos, axis, nh, hd, 1e6, 1.0, 0, err)
    for p, a in ((None, None), (pos, axis)):
        getattr(m, "minf_rope_kv_append_chunk_paged" + end)(q, k, q, k, v, p, a, off, past, nh, nk, hd, hd_kv, 1e6, 1.0, 0, kp,
                                                            vp, table, 16, err)
    getattr(m, "minf_kv_read_chunk_paged" + end)(k, v, kp, vp, table, 16, off, past, err)
    getattr(m, "minf_gqa_attn_chunk_paged" + end)(out, q, kp, vp, table, 16, off, past, 1, nh, nk, hd, hd_kv, 0.1, 0, 0, ws, err)
    getattr(m, "minf_gqa_attn_window" + end)(out, q, kp, vp, torch.zeros(n_seq, dtype=torch.int64, device="cuda"), None, 32, off,
                                             past, 1, nh, nk, hd, hd_kv, 0.1, 4, 1, ws, err)
    getattr(m, "minf_layer_attn_step_chunk_paged" + end)(xn, h, None, 1e-6, q, k, v, None, None, off, past, 1, kp, vp, table, 16,
                                                         nh, nk, hd, hd_kv, 1e6, 1.0, 0, 0, 0, out, ws, err)
    torch.cuda.synchronize()
    assert err.item() == 0 and not kp.any() and not vp.any()


# ----------------------------------------------------------------------------- many sequences without tokens
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("new,count", [(1, 200), (500, 2), (1, 5)])
def test_sequences_without_tokens_between_others(m, kind, paged, new, count):
    # 30000 sequences, most of them without tokens: a stretch of work goes from the first ones to the last
    r, n = rng(110), 30000
    lens, past = np.zeros(n, int), np.zeros(n, int)
    lens[:count] = lens[-count:] = new
    lens[[4000, 12345, 20000]] = 1, new, 2 if new > 1 else 1
    past[lens > 0] = r.integers(0, 300, (lens > 0).sum())
    check(m, Batch((14, 2, 64, 64), kind, lens.tolist(), past.tolist(), paged=paged, block=16, seed=110))


# ----------------------------------------------------------------------------- missing blocks
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [[1, 1], [3, 1], [40, 3]])
@pytest.mark.parametrize("block", [16, 128])
@pytest.mark.parametrize("missing", [-1, 1 << 20])
def test_missing_blocks_are_read_as_zeros(m, kind, new, block, missing):
    # their keys score 0 and count in the sum
    def batch():
        return Batch((16, 8, 128, 128), kind, new, [300, 200], paged=True, block=block, seed=109)

    b, clean = batch(), batch()
    rows = [clean.row(0, block + i) for i in range(block)]
    clean.k[rows], clean.v[rows] = 0, 0
    b.table[0, 1] = missing
    got, err = b.run(m)
    clean.scale = b.scale
    close(got, clean.ref())
    assert err == 0x10


# ----------------------------------------------------------------------------- rotation and store
@pytest.mark.parametrize("theta,freq_scale", [(1e4, 0.25), (1e4, 3.0), (5e5, 1 / 3)])
@pytest.mark.parametrize("style", [0, 1])
def test_other_angular_speeds(m, theta, freq_scale, style):
    nt, heads, hd = 50, 3, 128
    r, axis = rng(111), [0] * 16 + [1] * 24 + [2] * 24
    x = r.standard_normal((nt, heads, hd)).astype(np.float32)
    pos = r.integers(0, 1 << 17, (3, nt)).astype(np.int32)
    want, size = np.array(x, np.float64), np.zeros(x.shape)
    for i in range(hd // 2):
        a, b = (i, i + hd // 2) if style == 0 else (2 * i, 2 * i + 1)
        th = pos[axis[i]][:, None] * (float(np.float32(freq_scale)) * float(np.float32(theta)) ** (-2.0 * i / hd))
        xa, xb = x[:, :, a].astype(np.float64), x[:, :, b].astype(np.float64)
        want[:, :, a], want[:, :, b] = xa * np.cos(th) - xb * np.sin(th), xa * np.sin(th) + xb * np.cos(th)
        size[:, :, a] = size[:, :, b] = np.abs(xa) + np.abs(xb)
    y, err = torch.empty(nt, heads, hd, device="cuda"), i32([0])
    m.minf_rope_axes(y, dev(x), i32(pos), axis, heads, hd, theta, freq_scale, style, err)
    assert (np.abs(y.cpu().numpy() - want) <= 3.5e-7 * size).all()
    # the store turns q and k alike
    table, pool = i32([[0, 1, 2, 3]]), [torch.zeros(64, heads * hd, device="cuda") for _ in range(2)]
    q_out, k_out = torch.empty_like(y), torch.empty_like(y)
    m.minf_rope_kv_append_chunk_paged(q_out, k_out, dev(x), dev(x), dev(x), i32(pos), axis, i32([0, nt]), i32([7]), heads,
                                      heads, hd, hd, theta, freq_scale, style, *pool, table, 16, err)
    assert torch.equal(q_out, y) and torch.equal(k_out, y) and err.item() == 0
    assert torch.equal(pool[0][7:57].view(nt, heads, hd), y)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("starts", [[0, 5, 3, 8], [-1, 2, 4, 8], [0, 3, 5, 9]])
def test_store_and_read_back_report_offsets_out_of_order(m, kind, starts):
    geom = (14, 2, 64, 64)
    nh, nk, hd, hd_kv = geom
    b = Batch(geom, kind, [3, 2, 3], [5, 9, 100], paged=True, seed=112)
    q, k, v = (torch.randn(8, c, device="cuda") for c in (nh * hd, b.w, b.w))
    kp, vp, off, err = dev(b.k), dev(b.v), i32(starts), i32([0])
    getattr(m, "minf_rope_kv_append_chunk_paged" + END[kind])(q, k, q, k, v, None, None, off, i32(b.past), nh, nk, hd, hd_kv,
                                                              1e6, 1.0, 0, kp, vp, i32(b.table), 16, err)
    assert err.item() & 0x40
    err.zero_()
    getattr(m, "minf_kv_read_chunk_paged" + END[kind])(torch.empty_like(k), torch.empty_like(v), kp, vp, i32(b.table), 16, off,
                                                       i32(b.past), err)
    assert err.item() & 0x40
