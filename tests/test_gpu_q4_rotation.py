"""K of the Q4 store: rotated as exactly as it is quantized.

Tolerances.  The store's cosines and sines are within 2^-36; angles of positions below 2^13 are within 2^-39 of a radian in
the store and in the evaluation in 64 bits alike; products and their sum lose 2^-46 of themselves; and the result is
rounded to fp32 once, by 2^-24 of itself at most: |d| <= 2^-24 |y| + 2^-35 (|a| + |b|).  A value so near rounds another way
than the exact one in about 2^-11 of the cases, and has another code than that in 2^-20 of these: one of 2^31 values."""
import numpy as np
import pytest
import torch

import test_gpu_q4 as q4
from test_gpu_q4 import err_word, i32, m, normal  # noqa: F401

pytestmark = pytest.mark.gpu

THETA = 1e6


def rotated(x, pos, nk, hd, style, theta=THETA):
    """x [nt, nk * hd], pos [nt] or [hd / 2, nt], in 64 bits; and |a| + |b| of each value's pair."""
    i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    pos = pos.double().expand(hd // 2, -1).t()
    angle = (pos * theta ** (-2 * i / hd))[:, None]
    x = x.double().view(-1, nk, hd)
    a, b = (x[..., :hd // 2], x[..., hd // 2:]) if style == 0 else (x[..., 0::2], x[..., 1::2])
    y = a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()
    size = a.abs() + b.abs()
    join = (lambda p: torch.cat(p, -1)) if style == 0 else (lambda p: torch.stack(p, -1))
    return join(y).reshape(x.shape[0], nk * hd), join((size, size)).reshape(x.shape[0], nk * hd)


def store(m, k, v, geom, past, style, rope_pos=None, axes=None, want_k=True, theta=THETA):
    nh, nk, hd, hd_kv = geom
    nt, w = k.shape
    table = torch.arange((past + nt + 63) // 64, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    pool = torch.zeros(table.numel() * 64, q4.row_bytes(w), dtype=torch.uint8, device="cuda")
    kp, vp, err = pool, pool.clone(), err_word()
    q = normal(nt, nh * hd, seed=9)
    k_out = torch.empty_like(k) if want_k else None
    m.minf_rope_kv_append_chunk_paged_q4(torch.empty_like(q), k_out, q, k, v, rope_pos, axes, i32([0, nt]), i32([past]), nh, nk, hd,
                                         hd_kv, theta, 1.0, style, kp, vp, table, 64, err)
    assert int(err) == 0
    p = past + torch.arange(nt, device="cuda")
    rows = table[0, p // 64].long() * 64 + p % 64
    return k_out, kp[rows]


@pytest.mark.parametrize("geom", [(14, 2, 64, 64), (16, 8, 128, 128), (4, 2, 128, 64), (6, 2, 256, 128)])
@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("past,nt", [(0, 1), (0, 700), (7000, 1100)])
def test_k_is_the_exact_rotation_rounded_once(m, geom, style, past, nt):
    nh, nk, hd, hd_kv = geom
    w = nk * hd_kv
    k = normal(nt, w, seed=nt) * 2.0 ** torch.randint(-20, 20, (nt, 1), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    got, rows = store(m, k, normal(nt, w, seed=2), geom, past, style)
    want, size = rotated(k, past + torch.arange(nt, device="cuda"), nk, hd_kv, style)
    assert bool(((got.double() - want).abs() <= 2.0 ** -24 * want.abs() + 2.0 ** -35 * size).all())
    assert torch.equal(rows.cpu(), q4.quantize(got))


@pytest.mark.parametrize("style", [0, 1])
def test_positions_of_several_axes_all_around(m, style):
    """Every 256th of a turn and its borders: with theta 1 and a freq_scale of 1 each pair turns by its position in radians."""
    nh, nk, hd, nt = 2, 1, 64, 4096
    k = normal(nt, nk * hd, seed=3)
    pos = torch.stack([torch.arange(nt), torch.arange(nt) * 2 + 1, torch.full((nt,), 355)]).to(torch.int32).cuda()
    axes = [i % 3 for i in range(32)]
    got, rows = store(m, k, k, (nh, nk, hd, hd), 0, style, rope_pos=pos, axes=axes, theta=1.0)
    want, size = rotated(k, pos[torch.tensor(axes)], nk, hd, style, theta=1.0)
    assert bool(((got.double() - want).abs() <= 2.0 ** -24 * want.abs() + 2.0 ** -35 * size).all())
    assert torch.equal(rows.cpu(), q4.quantize(got))


def test_infinities_and_nan_stay(m):
    nk, hd = 2, 64
    k = normal(6, nk * hd, seed=4)
    k[1, 5], k[2, 40], k[3, 64], k[4, 100] = torch.inf, -torch.inf, torch.nan, 3e38
    got, rows = store(m, k, k, (2, nk, hd, hd), 3, 0)
    want = rotated(k, torch.arange(3, 9, device="cuda"), nk, hd, 0)[0].float()
    same = (got == want) | (got.isnan() & want.isnan())
    near = (got - want).abs() <= 2.0 ** -23 * want.abs()
    assert bool((same | near).all())
    assert torch.equal(rows[[0, 5]].cpu(), q4.quantize(got)[[0, 5]])


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("seed", [1, 2])
def test_codes_are_those_of_the_exact_rotation(m, seed, style):
    """Eight million values, as a rotation in 64 bits rounded to fp32 gives their codes; with and without k wanted."""
    nh, nk, hd, nt = 16, 8, 128, 8192 - 100
    k = normal(nt, nk * hd, seed=100 + seed)
    want = rotated(k, 100 + torch.arange(nt, device="cuda"), nk, hd, style)[0].float()
    codes = q4.quantize(want)
    for want_k in (True, False):
        _, rows = store(m, k, k, (nh, nk, hd, hd), 100, style, want_k=want_k)
        assert int((rows.cpu() != codes).sum()) == 0
