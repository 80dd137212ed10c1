"""How the paged calls behave beside one another: host threads, routes through the
kernels, workspaces, and calls with nothing to do."""
import math
import threading

import pytest
import torch

import exact_io_aware_54_b200 as fa
from exact_io_aware_54_b200 import synth
from tests._harness import f64
from tests.test_gpu_paged import INVALID, Cache, _check, _close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 40])
def test_two_host_threads_on_one_stream(new):
    """Both threads' calls go to the default stream and its workspace, and units are cut between
    CTAs, so that every call hands partial states from one launch to the next."""
    c = Cache(400, [3000, 700], 2, 128, 16, True)
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
    qs = [synth._normal((2 * new, 8, 128), 401 + i).cuda() for i in range(2)]
    call = lambda q: fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, new, 3000, True, **c.kw)
    want = [call(q) for q in qs]
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2), [0, 0]

    def work(i):
        start.wait()
        for _ in range(40):
            out = [call(qs[i]) for _ in range(10)]
            wrong[i] += sum(not (torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])) for o, lse in out)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]
    _check()


def test_first_calls_of_two_threads():
    """A stream's workspace is made once, whichever thread comes first."""
    stream, start, got = torch.cuda.Stream(), threading.Barrier(4), []

    def work():
        with torch.cuda.stream(stream):
            start.wait()
            got.append(fa.paged_workspace().data_ptr())

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(set(got)) == 1
