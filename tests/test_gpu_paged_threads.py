"""GPU: gqa_paged_attn_t on cudaStreamPerThread, one handle for a stream of each host thread,
with the library's workspace."""
import ctypes
import threading

import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa
from test_gpu_paged_attn import DEV, make

pytestmark = pytest.mark.gpu
PER_THREAD = ctypes.c_void_p(2)  # cudaStreamPerThread


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


def attend(x, out):
    d = [gqa._desc(t, "t") for t in (*x, out)]
    return gqa.lib().gqa_paged_attn_t(*map(ctypes.byref, d), None, 1.0, 1.0, 1.0, 0, 0.0, None, 0, PER_THREAD)


def in_threads(work, n):
    threads = [threading.Thread(target=work, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()


def test_threads_on_their_own_default_streams():
    """Batches of other sizes and lengths from four threads at once: none reads another's pieces."""
    data = [make(lens, hq=16, hkv=1, page=64, poison=False, seed=i) for i, lens in enumerate(([4000, 3, 900, 50], [10, 3500], [1, 2, 4096], [2222]))]
    want = [gqa.gqa_paged_attn(*x) for x in data]
    outs = [[torch.empty_like(w) for _ in range(50)] for w in want]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(4)

    def work(i):
        start.wait(60)
        bad.extend(st for st in (attend(data[i], o) for o in outs[i]) if st)
    in_threads(work, 4)
    torch.cuda.synchronize()
    assert not bad
    for o, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in o)


def test_threads_that_come_and_go_leave_nothing_behind():
    x = make([3000], hq=16, hkv=1, page=64, poison=False, seed=9)
    want, out = gqa.gqa_paged_attn(*x), torch.empty(1, 16, 128, dtype=torch.float16, device=DEV)
    torch.cuda.synchronize()

    def work(_):
        assert attend(x, out) == 0
    in_threads(work, 1)
    free = torch.cuda.mem_get_info(0)[0]
    for _ in range(50):
        in_threads(work, 1)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert free - torch.cuda.mem_get_info(0)[0] < 100 << 20  # (50 workspaces are 250 MB)
