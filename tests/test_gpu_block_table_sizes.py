"""Block tables of numbers of sequences whose sums take shared memory near and above 48 KB."""
import pytest

pytestmark = pytest.mark.gpu


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
