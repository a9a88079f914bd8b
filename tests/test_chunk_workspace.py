"""Workspaces of the chunk attention: what Q4 rows take is not asked of the other types (no GPU needed)."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE, ROWS = P(0x1000), P(0x100000)


@pytest.fixture(scope="module")
def lib():
    from gqa_attention_kv_rope_gb300 import binding, build

    build.build()
    return binding.lib()


# Two parts a stretch (at most 160 of them), each rows x (128 outputs, a maximum and a sum) in fp32, and the plan.  Rows of
# a part: those of a token's heads of one kv head, up to 8, 16 or 32.
def parts(rows):
    return 2 * 160 * rows * 130 * 4 + (1 << 17)


@pytest.mark.parametrize("nt,n_seq,max_chunk,rows", [(64, 64, 1, 8), (160, 32, 5, 16), (128, 8, 16, 32)])
@pytest.mark.parametrize("end,refused", [("", False), ("_f16", False), ("_q8", False), ("_q4", True)])
def test_workspaces_of_the_other_types_are_as_before_q4(lib, nt, n_seq, max_chunk, rows, end, refused):
    need = parts(rows) if max_chunk < 16 else lib.minf_attn_chunk_workspace_bytes(nt, n_seq, 16, 8, 128, max_chunk)
    # out is q: what comes after the workspace in the checks refuses the call, so that nothing is launched
    args = [ROWS, ROWS, FAKE, FAKE, 256, FAKE, 4, 16, FAKE, FAKE, nt, n_seq, max_chunk, 16, 8, 128, 128, 0.1, 0, 0, FAKE]
    f = getattr(lib, "minf_gqa_attn_chunk_paged" + end)
    assert f(*args, need, FAKE, None) == (5 if refused and max_chunk < 16 else 1)
    args = [ROWS, ROWS, FAKE, FAKE, FAKE, None, 100, 500, FAKE, FAKE, nt, n_seq, max_chunk, 16, 8, 128, 128, 0.1, 0, 0, FAKE]
    f = getattr(lib, "minf_gqa_attn_window" + end)
    assert f(*args, need, FAKE, None) == (5 if refused and max_chunk < 16 else 1)
    args = [FAKE, FAKE, None, 1e-6, 896, ROWS, FAKE, FAKE, None, 1, None, FAKE, FAKE, nt, n_seq, max_chunk, FAKE, FAKE, 256, FAKE,
            4, 16, 16, 8, 128, 128, 1e4, 1.0, 0, 0, 0, ROWS, FAKE]
    f = getattr(lib, "minf_layer_attn_step_chunk_paged" + end)
    assert f(*args, need, FAKE, None) == (5 if refused and max_chunk < 16 else 1)


def test_the_size_covers_every_type(lib):
    need = lib.minf_attn_chunk_workspace_bytes(64, 64, 16, 8, 128, 1)
    assert need > parts(8)
    args = [ROWS, ROWS, FAKE, FAKE, 256, FAKE, 4, 16, FAKE, FAKE, 64, 64, 1, 16, 8, 128, 128, 0.1, 0, 0, FAKE]
    for end in ("", "_f16", "_q8", "_q4"):
        assert getattr(lib, "minf_gqa_attn_chunk_paged" + end)(*args, need, FAKE, None) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "f16", "q8"])
@pytest.mark.parametrize("paged", [False, True])
def test_calls_stay_inside_less_than_q4_takes(kind, paged):
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gqa_attention_kv_rope_gb300 as m
    import test_gpu_chunk as chunk

    for new, rows in (([1] * 64, 8), ([5] * 32, 16)):
        b = chunk.Batch((16, 8, 128, 128), kind, new, [30 * i for i in range(len(new))], paged=paged, seed=5)
        room = torch.full((parts(rows) + (1 << 20),), 0xAB, dtype=torch.uint8, device="cuda")
        chunk.check(m, b, ws=room[:parts(rows)])
        assert bool((room[parts(rows):] == 0xAB).all())
