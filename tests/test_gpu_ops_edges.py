"""GPU tests of the FP8 products whose inputs are shorter than one block, and
of calls that overlap on the GPU, each with a workspace of its own."""
import threading

import pytest
import torch

from routed_moe_decode_router_gb300 import ops
from tests import ops_ref as R
from tests import test_gpu_ops as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_status() == 0


@pytest.mark.parametrize("m", [16, 17, 100, 300])
@pytest.mark.parametrize("n,k", [(64, 16), (257, 48), (128, 112), (1000, 16), (513, 96)])
def test_matmul_of_less_than_one_block(m, n, k):
    a, sa, b, sb = T.operands(m, n, k)
    for t in (torch.float32, torch.bfloat16):
        T.check_product(a, sa, b, sb, ops.matmul_fp8(a, sa, b, sb, out_dtype=t))


def jobs():
    """Expert calls of three sizes: few pairs, one tile to an expert, many."""
    lay = T.layer(16, 512, 256)
    out = []
    for t in (4, 150, 2000):
        q, s = R.rows_fp8(T.randn(t, 512, seed=t))
        ids, wts = T.choice(t, 4, 16, seed=t)
        out.append((t, lambda ws, q=q, s=s, ids=ids, wts=wts: ops.experts_fp8(
            q, s, ids, wts, *lay, ws=ws)))
    return out


def test_calls_on_two_streams():
    work = jobs()
    want = [f(None) for _, f in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [ops.ExpertsWorkspace(2000, 4, 512, 256, 16) for _ in streams]
    torch.cuda.synchronize()
    got = []
    for r in range(20):
        for i, (s, ws) in enumerate(zip(streams, spaces)):
            j = (r + i) % len(work)
            with torch.cuda.stream(s):
                got.append((j, work[j][1](ws)))
    torch.cuda.synchronize()
    for j, y in got:
        assert torch.equal(y, want[j])


def test_calls_of_two_threads():
    work = jobs()
    want = [f(None) for _, f in work]
    torch.cuda.synchronize()
    bad = []

    def run(first):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            ws = ops.ExpertsWorkspace(2000, 4, 512, 256, 16)
            torch.cuda.current_stream().synchronize()
            with torch.cuda.stream(stream):
                for r in range(30):
                    j = (first + r) % len(work)
                    y = work[j][1](ws)
                    stream.synchronize()
                    if not torch.equal(y, want[j]):
                        bad.append(j)
                with pytest.raises(ValueError):
                    ops.route_topk(torch.zeros(2, 8), 2)
        except Exception as e:
            bad.append(repr(e))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
