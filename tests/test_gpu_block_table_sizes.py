"""Block tables of numbers of sequences whose sums take shared memory near and above 48 KB."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# In a process of its own: what a kernel may take is state of the whole context, which a larger call raises.
FRESH = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import gqa_attention_kv_rope_gb300 as m
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
err, n_free = i32([0]), i32([0])
for op, sizes in (("release", (6045, 6046, 6143, 6144, 16384)), ("grow", (4041, 4042, 4095, 4096, 16384))):
    for n in sizes:
        table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
        free, zero, one = i32([-1] * n), i32([0] * n), i32([1] * n)
        off, slot = i32([0] * (n + 1)), i32([0] * n)
        if op == "release":
            m.minf_block_table_release(table, 16, 16 * n, zero, zero + 16, free, n_free, n_free, err)
            assert bool((table == -1).all()) and bool((free.sort().values.cpu() == torch.arange(n)).all()) and int(n_free) == n
            n_free.zero_()
        else:
            m.minf_block_table_grow(table, 16, 16 * n, one, one, free, n_free, n_free, off, None, slot, err)
            assert bool((off.cpu() == torch.arange(n + 1)).all()) and bool((slot.cpu() == 16 * torch.arange(n) + 1).all())
        # (an operator that goes by the runtime's last error)
        y = torch.ones(2, 64, device="cuda")
        m.minf_rope_axes(y, y.clone(), i32([0, 0]), None, 1, 64, 1e4, 1.0, 0, err)
        assert int(err) == 0
print("done")
"""


def test_any_number_of_sequences_in_a_fresh_process():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_attention_kv_rope_gb300 import build

    build.build()
    r = subprocess.run([sys.executable, "-c", FRESH.format(root=ROOT, tests=os.path.join(ROOT, "tests"))],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr


def test_host_threads_at_once():
    """Threads that grow tables of different sizes, over lists of their own, on streams of their own."""
    import threading

    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gqa_attention_kv_rope_gb300 as m
    from gqa_attention_kv_rope_gb300 import build

    build.build()
    m.binding.lib()
    failed = []

    def work(n, turns):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
                one = torch.ones(n, dtype=torch.int32, device="cuda")
                free, n_free, err = one.clone(), torch.zeros_like(one[:1]), torch.zeros_like(one[:1])
                off = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
                for _ in range(turns):
                    m.minf_block_table_grow(table, 16, 16 * n, one, one, free, n_free, n_free, off, None, None, err)
                torch.cuda.current_stream().synchronize()
                assert int(err) == 0 and int(off[n]) == n
        except Exception as e:  # noqa: BLE001
            failed.append(f"{n}: {e!r}")

    torch.zeros(1, device="cuda")
    threads = [threading.Thread(target=work, args=(n, 2000)) for n in (16384, 4500, 9000, 5000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
