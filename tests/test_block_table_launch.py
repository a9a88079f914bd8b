"""The launches of the block-table calls against a stand-in for the CUDA runtime (no GPU needed): shared memory that a
kernel is allowed, and calls of several host threads."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
P = ctypes.c_void_p
OWN = 1024  # bytes of the kernels' own arrays: no less than they are (640 and 784 when this was written)


def at(i):
    return P(0x10000000 * (i + 1))  # never dereferenced: no kernel runs


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from gqa_attention_kv_rope_gb300 import build

    build.build()
    obj = os.path.join(build.BUILD, "minf_block_tables.o")
    if not os.path.exists(obj):
        obj = build._compile("minf_block_tables.cu", False)
    so = tmp_path_factory.mktemp("fake") / "tables.so"
    # (-Bsymbolic: its own stand-ins, not the runtime that torch has loaded)
    subprocess.run([build.nvcc(), "-shared", "-cudart", "none", "-Xcompiler", "-fPIC", "-Xlinker", "-Bsymbolic", "-o", str(so),
                    os.path.join(HERE, "fake_cuda_runtime.cpp"), obj], check=True, capture_output=True)
    lib = ctypes.CDLL(str(so))
    i, i64 = ctypes.c_int, ctypes.c_int64
    lib.minf_block_table_grow.argtypes = [P, i, i, i64, P, P, i, P, i, P, P, P, P, P, i, P, P]
    lib.minf_block_table_release.argtypes = [P, i, i, i64, P, P, i, P, i, P, P, P, P]
    return lib


def grow(lib, n_seq, nt=0, max_blocks=4):
    return lib.minf_block_table_grow(at(0), max_blocks, 16, 1 << 20, at(1), at(2), n_seq, at(3), 1 << 16, at(4), at(5), at(6),
                                     at(7), at(8), nt, at(9), None)


def release(lib, n_seq, max_blocks=4):
    return lib.minf_block_table_release(at(0), max_blocks, 16, 1 << 20, at(1), at(2), n_seq, at(3), 1 << 16, at(4), at(5),
                                        at(9), None)


@pytest.mark.parametrize("call", [grow, release])
@pytest.mark.parametrize("mine,other", [(16384, 5000), (16384, 12000), (9000, 6500)])
def test_no_call_lowers_what_another_is_allowed(lib, call, mine, other):
    """A smaller call of another thread lands between a call's own setting and its launch."""
    lib.fake_reset(OWN)
    theirs = []
    hook = ctypes.CFUNCTYPE(ctypes.c_int32)(lambda: theirs.append(call(lib, other)) or 0)
    lib.fake_meanwhile(hook)
    assert call(lib, mine) == 0 and theirs == [0]
    assert lib.fake_launches() == 2 and lib.fake_last_error() == 0


@pytest.mark.parametrize("call,bytes_a_seq", [(grow, 12), (release, 8)])
def test_a_kernels_own_arrays_count(lib, call, bytes_a_seq):
    """Sums that fit 48 KB by themselves, but not with the kernel's own arrays, as the first call and after larger ones."""
    near = 48 * 1024 // bytes_a_seq - 1
    for first in (None, 16384):
        for n in [*range(near - 200, near + 3, 7), near - 1, near, near + 1]:
            lib.fake_reset(OWN)
            assert first is None or call(lib, first) == 0
            assert call(lib, n) == 0 and lib.fake_last_error() == 0, n
            assert lib.fake_dynamic() == bytes_a_seq * (n + 1)


@pytest.mark.parametrize("clusters", [0, -1, None])
def test_without_large_clusters(lib, clusters):
    """Where no cluster of 16 can be had -- the query says none, or fails, or the attribute is refused -- the largest calls
    run in eight CTAs, and nothing is left behind that the next operator would take for its own error."""
    for call in (lambda: grow(lib, 1024, nt=121000), lambda: release(lib, 3000, max_blocks=40)):
        lib.fake_reset(OWN)
        assert call() == 0 and lib.fake_cluster() == 16
        lib.fake_reset(OWN)
        if clusters is None:
            lib.fake_refuse_large_clusters()
        else:
            lib.fake_clusters_of_16(clusters)
        assert call() == 0 and lib.fake_cluster() == 8
        assert lib.fake_last_error() == 0
