"""Q4 regions handed to the Q8_0 calls: both are bytes, so their size tells them apart (no GPU needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import gqa_attention_kv_rope_gb300 as pkg
    from gqa_attention_kv_rope_gb300 import build

    build.build()
    return pkg


def calls(m, k, v):
    """Every Q8_0 call that takes regions, an arena or pools of 64 rows of 128 values, with tensors of the host."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    x, q, h = torch.zeros(1, 128), torch.zeros(1, 256), torch.zeros(1, 512)
    ws, err, table, off = torch.zeros(256, dtype=torch.uint8), i32(0), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    g = (4, 2, 64, 64)
    rope = (1e4, 1.0, 0)
    step = (h, h, None, 1e-6, q, x, x, i32(0))
    return [lambda: m.minf_kv_append_q8(k, v, x, x, i32(0), err),
            lambda: m.minf_rope_kv_append_q8(q, x, x, i32(0), *g, *rope, k, v, err),
            lambda: m.minf_gqa_attn_decode_q8(q, q, k, v, None, None, 64, i32(0), *g, 0.1, ws, err),
            lambda: m.minf_gqa_attn_prefill_q8(q, q, k, v, i32(0), *g, 0.1, ws, err),
            lambda: m.minf_layer_attn_step_q8(*step, k, v, *g, *rope, q, ws, err),
            lambda: m.minf_layer_attn_step_chained_q8(*step, k, v, *g, *rope, q, ws, err),
            lambda: m.minf_layer_attn_step_batched_q8(*step, k, v, off, i32(64), 64, *g, *rope, q, ws, err),
            lambda: m.minf_kv_append_paged_q8(k, v, table, 16, x, x, i32(0), err),
            lambda: m.minf_gqa_attn_decode_paged_q8(q, q, k, v, table, 16, i32(0), *g, 0.1, ws, err),
            lambda: m.minf_layer_attn_step_paged_q8(*step, k, v, table, 16, *g, *rope, q, ws, err)]


@pytest.mark.parametrize("which", [0, 1, 2])
def test_q4_regions_are_refused(m, which):
    q4, q8 = (m.kv.KvRegions(1, 128, 64, device="cpu", dtype=d).k[0] for d in ("q4", torch.uint8))
    for call in calls(m, q4 if which != 1 else q8, q4 if which != 0 else q8):
        with pytest.raises(ValueError, match="Q8_0"):
            call()


def test_q8_regions_are_not(m):
    """(what comes next refuses tensors of the host)"""
    q8 = m.kv.KvRegions(1, 128, 64, device="cpu", dtype=torch.uint8).k[0]
    more = torch.zeros(70, 144, dtype=torch.uint8)
    for call in calls(m, q8, q8) + calls(m, q8, more):
        with pytest.raises(TypeError, match="CUDA"):
            call()
