"""Q4 arenas filled a sequence at a time: positions are held to the sequence's own capacity."""
import pytest
import torch

import test_gpu_q4 as q4
from test_gpu_q4 import err_word, i32, m, normal  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_sequence_cannot_reach_its_neighbours(m):
    w, caps = 128, [5, 3, 7]
    arena = m.kv.KvArena(2, w, caps, dtype="q4")
    arena.k.fill_(0x33)
    arena.v.fill_(0x44)
    want_k, want_v = arena.k.clone().cpu(), arena.v.clone().cpu()
    for s, (pos, bit) in enumerate([([0, 4, 2], 0), ([2, 3, -1, 0], m.ERRBIT_STORE_POS), ([6, 7, 1 << 30], m.ERRBIT_STORE_POS)]):
        k, v, err = normal(len(pos), w, seed=s), normal(len(pos), w, seed=10 + s), err_word()
        m.minf_kv_append_q4(*arena.seq_view(1, s), k, v, i32(pos), err)
        assert int(err) == bit
        at = sum(caps[:s])
        for t, p in enumerate(pos):
            if 0 <= p < caps[s]:
                want_k[1, at + p], want_v[1, at + p] = q4.quantize(k)[t], q4.quantize(v)[t]
    assert torch.equal(arena.k.cpu(), want_k) and torch.equal(arena.v.cpu(), want_v)


def test_attention_over_an_arena_filled_so(m):
    nh, nk, hd, caps, have = 4, 2, 64, [40, 9, 130], [40, 9, 77]
    w = nk * hd
    arena = m.kv.KvArena(1, w, caps, dtype="q4")
    arena.k.fill_(0xff)  # rows that nobody wrote: scales that are not numbers
    arena.v.fill_(0xff)
    err, rows = err_word(), []
    for s, n in enumerate(have):
        k, v = normal(n, w, seed=s), normal(n, w, seed=20 + s)
        m.minf_kv_append_q4(*arena.seq_view(0, s), k, v, torch.arange(n, dtype=torch.int32, device="cuda"), err)
        rows.append([q4.value(q4.quantize(x), w).cuda().view(n, nk, hd) for x in (k, v)])
    q, out = normal(3, nh * hd, seed=5), torch.empty(3, nh * hd, device="cuda")
    ws = m.kv.chunk_workspace(3, 3, nh, nk, hd, 1)
    m.minf_gqa_attn_window_q4(out, q, *arena.view(0), arena.row_off, arena.cap, arena.max_cap, None, i32([n - 1 for n in have]), 1, nh, nk,
                              hd, hd, hd ** -0.5, 0, 0, ws, err)
    assert int(err) == 0
    for s, n in enumerate(have):
        ref = q4.ref_attention(q[s:s + 1].view(1, nh, hd), *rows[s], n - 1, caps[s], (nh, nk, hd, hd), hd ** -0.5, 0, 0)
        q4.close(out[s:s + 1], ref)
