"""The chunk operators' refusals, before anything is launched (no GPU needed)."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE = P(0x1000)  # never dereferenced: validation rejects before any launch
ODD = P(0x1004)


@pytest.fixture(scope="module")
def lib():
    from gqa_attention_kv_rope_gb300 import binding, build

    build.build()
    return binding.lib()


def attn_args(**kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, pool_rows=256, table=FAKE, max_blocks=4, block_rows=16, off=FAKE,
             past=FAKE, nt=8, n_seq=2, max_chunk=4, nh=14, nk=2, hd=64, hd_kv=64, scale=0.125, window=0, n_sink=0,
             ws=FAKE, ws_bytes=1 << 40, err=FAKE, stream=None)
    a.update(kw)
    return list(a.values())


def window_args(**kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, row_off=FAKE, cap=None, max_cap=100, arena_rows=500, off=FAKE, past=FAKE,
             nt=8, n_seq=2, max_chunk=4, nh=14, nk=2, hd=64, hd_kv=64, scale=0.125, window=0, n_sink=0, ws=FAKE,
             ws_bytes=1 << 40, err=FAKE, stream=None)
    a.update(kw)
    return list(a.values())


SHARED = [(dict(out=None), 1), (dict(q=None), 1), (dict(q=ODD), 1), (dict(k=ODD), 1), (dict(v=None), 1),
          (dict(past=None), 1), (dict(err=None), 1), (dict(off=None), 1), (dict(nt=-1), 1), (dict(n_seq=-1), 1),
          (dict(max_chunk=0), 1), (dict(window=-1), 1), (dict(n_sink=-1), 1), (dict(nh=15), 2), (dict(hd_kv=128), 2),
          (dict(hd=96, hd_kv=96), 3), (dict(nh=18), 3), (dict(nh=0), 1), (dict(hd=260), 3), (dict(ws=None), 5),
          (dict(ws=ODD), 5), (dict(ws_bytes=0), 5)]


@pytest.mark.parametrize("end", ["", "_f16", "_q8"])
@pytest.mark.parametrize("bad,status", SHARED + [
    (dict(table=None), 1), (dict(pool_rows=0), 1), (dict(max_blocks=0), 1), (dict(block_rows=8), 3),
    (dict(block_rows=48), 3), (dict(block_rows=8192), 3), (dict(pool_rows=250), 3),
    (dict(max_blocks=1 << 30), 3), (dict(pool_rows=1 << 32), 3)])
def test_chunk_attention_refuses(lib, end, bad, status):
    assert getattr(lib, "minf_gqa_attn_chunk_paged" + end)(*attn_args(**bad)) == status


@pytest.mark.parametrize("end", ["", "_f16", "_q8"])
@pytest.mark.parametrize("bad,status", SHARED + [(dict(row_off=None), 1), (dict(max_cap=0), 1), (dict(arena_rows=0), 1),
                                                 (dict(arena_rows=1 << 31), 3), (dict(max_cap=(1 << 31) - 1), 3)])
def test_window_attention_refuses(lib, end, bad, status):
    assert getattr(lib, "minf_gqa_attn_window" + end)(*window_args(**bad)) == status


@pytest.mark.parametrize("end", ["", "_f16", "_q8"])
def test_empty_calls_launch_nothing(lib, end):
    assert getattr(lib, "minf_gqa_attn_chunk_paged" + end)(*attn_args(nt=0)) == 0
    assert getattr(lib, "minf_gqa_attn_chunk_paged" + end)(*attn_args(n_seq=0)) == 0
    assert getattr(lib, "minf_gqa_attn_window" + end)(*window_args(nt=0, ws=None, ws_bytes=0)) == 0


def axes(*values):
    return (ctypes.c_uint8 * len(values))(*values)


@pytest.mark.parametrize("bad,status", [
    (dict(y=None), 1), (dict(x=None), 1), (dict(pos=None), 1), (dict(err=None), 1), (dict(nt=-1), 1), (dict(n_axis=0), 1),
    (dict(n_axis=256), 1), (dict(pair_axis=None), 1), (dict(pair_axis=axes(0, 1, 2, 0)), 1), (dict(nh=0), 1),
    (dict(hd=7), 1), (dict(hd=258, pair_axis=axes(*[0] * 129)), 1), (dict(style=2), 1), (dict(nh=1 << 20), 3)])
def test_rope_axes_refuses(lib, bad, status):
    a = dict(y=FAKE, x=FAKE, pos=FAKE, nt=4, n_axis=2, pair_axis=axes(0, 1, 1, 0), nh=2, hd=8, theta=1e4, fs=1.0, style=0,
             err=FAKE, stream=None)
    a.update(bad)
    assert lib.minf_rope_axes(*a.values()) == status


@pytest.mark.parametrize("end", ["", "_f16", "_q8"])
@pytest.mark.parametrize("bad,status", [
    (dict(q_out=None), 1), (dict(k_out=ODD), 1), (dict(q=ODD), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(off=None), 1), (dict(past=None), 1), (dict(n_axis=2), 1), (dict(style=3), 1), (dict(nh=15), 2),
    (dict(hd=68), 3), (dict(hd_kv=32), 3), (dict(kp=ODD), 1), (dict(table=None), 1), (dict(block_rows=24), 3),
    (dict(err=None), 1)])
def test_store_refuses(lib, end, bad, status):
    a = dict(q_out=FAKE, k_out=None, q=FAKE, k=FAKE, v=FAKE, pos=None, n_axis=1, pair_axis=None, off=FAKE, past=FAKE,
             nt=4, n_seq=2, nh=14, nk=2, hd=64, hd_kv=64, theta=1e4, fs=1.0, style=0, kp=FAKE, vp=FAKE, rows=256,
             table=FAKE, max_blocks=4, block_rows=16, err=FAKE, stream=None)
    a.update(bad)
    assert getattr(lib, "minf_rope_kv_append_chunk_paged" + end)(*a.values()) == status


@pytest.mark.parametrize("end", ["", "_f16", "_q8"])
@pytest.mark.parametrize("bad,status", [
    (dict(k_rows=None), 1), (dict(v_rows=ODD), 1), (dict(w=0), 1), (dict(w=2), 1), (dict(f16=1, w=36), 1),
    (dict(table=None), 1), (dict(rows=100), 3), (dict(off=None), 1), (dict(err=None), 1)])
def test_read_refuses(lib, end, bad, status):
    a = dict(k_rows=FAKE, v_rows=FAKE, f16=0, kp=FAKE, vp=FAKE, rows=256, w=128, table=FAKE, max_blocks=4, block_rows=16,
             off=FAKE, past=FAKE, nt=4, n_seq=2, err=FAKE, stream=None)
    a.update(bad)
    assert getattr(lib, "minf_kv_read_chunk_paged" + end)(*a.values()) == status


@pytest.mark.parametrize("end", ["", "_f16", "_q8"])
@pytest.mark.parametrize("bad,status", [
    (dict(xn=None), 1), (dict(h=None), 1), (dict(n_embd=0), 1), (dict(q=ODD), 1), (dict(n_axis=3), 1), (dict(off=None), 1),
    (dict(max_chunk=0), 1), (dict(hd=68), 3), (dict(hd_kv=128), 2), (dict(window=-2), 1), (dict(out=None), 1),
    (dict(ws=None), 5), (dict(ws_bytes=8), 5)])
def test_layer_step_refuses_before_its_first_launch(lib, end, bad, status):
    a = dict(xn=FAKE, h=FAKE, gain=None, eps=1e-6, n_embd=896, q=FAKE, k=FAKE, v=FAKE, pos=None, n_axis=1, pair_axis=None,
             off=FAKE, past=FAKE, nt=4, n_seq=2, max_chunk=4, kp=FAKE, vp=FAKE, rows=256, table=FAKE, max_blocks=4,
             block_rows=16, nh=14, nk=2, hd=64, hd_kv=64, theta=1e4, fs=1.0, style=0, window=0, n_sink=0, out=FAKE,
             ws=FAKE, ws_bytes=1 << 40, err=FAKE, stream=None)
    a.update(bad)
    assert getattr(lib, "minf_layer_attn_step_chunk_paged" + end)(*a.values()) == status


def test_workspace_sizes(lib):
    f = lib.minf_attn_chunk_workspace_bytes
    assert f(0, 1, 14, 2, 64, 1) == 0 and f(4, 1, 15, 2, 64, 1) == 0 and f(4, 1, 14, 2, 96, 1) == 0
    assert f(1, 1, 14, 2, 64, 1) >= 256 and f(5000, 64, 16, 8, 128, 4096) >= 256


@pytest.mark.parametrize("end", ["", "_f16", "_q8"])
@pytest.mark.parametrize("at", [0, 16, 8 * 14 * 64 * 4 - 16, -8 * 14 * 64 * 4 + 16])
def test_out_may_not_overlap_q(lib, end, at):
    q = 1 << 20
    for f, args in (("minf_gqa_attn_chunk_paged", attn_args), ("minf_gqa_attn_window", window_args)):
        assert getattr(lib, f + end)(*args(q=P(q), out=P(q + at))) == 1


@pytest.mark.parametrize("nh,nk", [(9, 1), (16, 1), (32, 1), (129, 1), (1 << 20, 1), (64, 4)])
def test_workspace_of_geometries_that_no_call_takes(lib, nh, nk):
    for max_chunk in (1, 4, 1000):
        assert lib.minf_attn_chunk_workspace_bytes(4, 2, nh, nk, 64, max_chunk) == 0
    assert lib.minf_gqa_attn_chunk_paged(*attn_args(nh=nh, nk=nk)) == 3


@pytest.mark.parametrize("end", ["", "_f16", "_q8"])
def test_calls_without_tokens_take_null_arrays(lib, end):
    # tensors of no elements have no address
    none = dict(out=None, q=None, nt=0)
    for f, args in (("minf_gqa_attn_chunk_paged", attn_args), ("minf_gqa_attn_window", window_args)):
        assert getattr(lib, f + end)(*args(**none)) == 0
        assert getattr(lib, f + end)(*args(**none, n_seq=0, past=None)) == 0
        assert getattr(lib, f + end)(*args(**none, n_seq=0, past=None, off=None)) == 0
        assert getattr(lib, f + end)(*args(**none, err=None)) == 1
        assert getattr(lib, f + end)(*args(**none, past=None)) == 1
        assert getattr(lib, f + end)(*args(**none, k=None)) == 1
    assert getattr(lib, "minf_gqa_attn_chunk_paged" + end)(*attn_args(**none, n_seq=0, past=None, table=None)) == 0
    assert getattr(lib, "minf_gqa_attn_chunk_paged" + end)(*attn_args(**none, table=None)) == 1
    a = dict(q_out=None, k_out=None, q=None, k=None, v=None, pos=None, n_axis=1, pair_axis=None, off=FAKE, past=FAKE, nt=0,
             n_seq=2, nh=14, nk=2, hd=64, hd_kv=64, theta=1e4, fs=1.0, style=0, kp=FAKE, vp=FAKE, rows=256, table=FAKE,
             max_blocks=4, block_rows=16, err=FAKE, stream=None)
    assert getattr(lib, "minf_rope_kv_append_chunk_paged" + end)(*a.values()) == 0
    a.update(style=2)
    assert getattr(lib, "minf_rope_kv_append_chunk_paged" + end)(*a.values()) == 1
    a = dict(k_rows=None, v_rows=None, f16=0, kp=FAKE, vp=FAKE, rows=256, w=128, table=FAKE, max_blocks=4, block_rows=16,
             off=FAKE, past=FAKE, nt=0, n_seq=2, err=FAKE, stream=None)
    assert getattr(lib, "minf_kv_read_chunk_paged" + end)(*a.values()) == 0
    a = dict(xn=None, h=None, gain=None, eps=1e-6, n_embd=896, q=None, k=None, v=None, pos=None, n_axis=1, pair_axis=None,
             off=FAKE, past=FAKE, nt=0, n_seq=2, max_chunk=4, kp=FAKE, vp=FAKE, rows=256, table=FAKE, max_blocks=4,
             block_rows=16, nh=14, nk=2, hd=64, hd_kv=64, theta=1e4, fs=1.0, style=0, window=0, n_sink=0, out=None,
             ws=None, ws_bytes=0, err=FAKE, stream=None)
    assert getattr(lib, "minf_layer_attn_step_chunk_paged" + end)(*a.values()) == 0
    assert lib.minf_rope_axes(None, None, None, 0, 1, None, 2, 8, 1e4, 1.0, 0, FAKE, None) == 0


Q, K, V = 1 << 20, 1 << 21, 1 << 22  # 4 rows: of 14336 bytes (14 heads of 64), of 2048 (two)


@pytest.mark.parametrize("end", ["", "_f16", "_q8"])
@pytest.mark.parametrize("bad", [dict(q_out=Q + 16), dict(q_out=Q - 14320), dict(q_out=K), dict(q_out=V + 2032),
                                 dict(q_out=Q, k_out=Q + 14320), dict(k_out=K + 16), dict(k_out=K - 2032), dict(k_out=V),
                                 dict(k_out=Q), dict(q_out=1 << 23, k_out=(1 << 23) + 32)])
def test_store_refuses_outputs_that_overlap(lib, end, bad):
    a = dict(q_out=Q, k_out=None, q=Q, k=K, v=V, pos=None, n_axis=1, pair_axis=None, off=FAKE, past=FAKE, nt=4, n_seq=2,
             nh=14, nk=2, hd=64, hd_kv=64, theta=1e4, fs=1.0, style=0, kp=FAKE, vp=FAKE, rows=256, table=FAKE, max_blocks=4,
             block_rows=16, err=FAKE, stream=None)
    a.update(bad)
    assert getattr(lib, "minf_rope_kv_append_chunk_paged" + end)(*[P(x) if isinstance(x, int) and x >= Q - 14336 else x
                                                                   for x in a.values()]) == 1


@pytest.mark.parametrize("end", ["", "_f16", "_q8"])
@pytest.mark.parametrize("f16,at", [(0, 0), (0, 2032), (0, -16), (1, 1008), (1, -1008)])
def test_read_refuses_outputs_that_overlap(lib, end, f16, at):
    a = dict(k_rows=P(K), v_rows=P(K + at), f16=f16, kp=FAKE, vp=FAKE, rows=256, w=128, table=FAKE, max_blocks=4,
             block_rows=16, off=FAKE, past=FAKE, nt=4, n_seq=2, err=FAKE, stream=None)
    assert getattr(lib, "minf_kv_read_chunk_paged" + end)(*a.values()) == 1


@pytest.mark.parametrize("at", [4, -4, 4 * 2 * 8 * 4 - 4])
def test_rope_axes_refuses_partly_in_place(lib, at):
    assert lib.minf_rope_axes(P(Q + at), P(Q), FAKE, 4, 1, None, 2, 8, 1e4, 1.0, 0, FAKE, None) == 1


@pytest.mark.parametrize("end", ["", "_f16", "_q8"])
@pytest.mark.parametrize("bad", [dict(k=P(Q + 16)), dict(v=P(Q)), dict(v=P(K)), dict(v=P(K + 2032))])
def test_layer_step_refuses_rows_that_overlap(lib, end, bad):
    a = dict(xn=FAKE, h=FAKE, gain=None, eps=1e-6, n_embd=896, q=P(Q), k=P(K), v=P(V), pos=None, n_axis=1, pair_axis=None,
             off=FAKE, past=FAKE, nt=4, n_seq=2, max_chunk=4, kp=FAKE, vp=FAKE, rows=256, table=FAKE, max_blocks=4,
             block_rows=16, nh=14, nk=2, hd=64, hd_kv=64, theta=1e4, fs=1.0, style=0, window=0, n_sink=0, out=P(1 << 24),
             ws=FAKE, ws_bytes=1 << 40, err=FAKE, stream=None)
    a.update(bad)
    assert getattr(lib, "minf_layer_attn_step_chunk_paged" + end)(*a.values()) == 1
