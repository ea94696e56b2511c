"""What a kernel reports is not lost with the workspace of a call that was given none."""
import pytest
import torch

import dynamic_block_sparse_shape_b200 as P
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def status(stream=None):
    try:
        P.check_device_status(stream=stream)
    except P.PrismError as e:
        return e.name
    return "PRISM_OK"


def pool_args(bad):
    """Pooling over two zones; a zone shape outside the candidates is caught in the kernel and reported."""
    geo = P.Geometry((8, 8, 16), (8, 8, 8), ((4, 4, 4),))
    q = torch.ones((8 * 8 * 16, 1, 64), dtype=torch.bfloat16, device="cuda")
    return geo, torch.tensor([0, 5 if bad else 0], dtype=torch.int32, device="cuda"), q, q


@pytest.mark.parametrize("side", [False, True])
def test_a_report_outlives_its_call(side):
    require_gpu()
    stream = torch.cuda.Stream() if side else None
    status()
    good, bad = pool_args(False), pool_args(True)
    torch.cuda.synchronize()
    P.block_pool(*good, stream=stream)
    assert status(stream) == "PRISM_OK"
    P.block_pool(*bad, stream=stream)
    P.block_pool(*good, stream=stream)  # later calls leave the report
    assert status(stream) == "PRISM_ERR_DEVICE"
    assert status(stream) == "PRISM_OK"  # read once
    ws = P.Workspace("cuda")
    P.block_pool(*bad, ws=ws, stream=stream)  # a kept workspace's report is its own
    assert status(stream) == "PRISM_OK"
    with pytest.raises(P.PrismError):
        P.check_device_status(ws, stream=stream)


def test_a_timeout_is_told_from_a_bad_index():
    """The status word as a wait that ran out leaves it."""
    require_gpu()
    status()
    for bits, name in ((1, "PRISM_ERR_TIMEOUT"), (3, "PRISM_ERR_TIMEOUT"), (2, "PRISM_ERR_DEVICE"), (0, "PRISM_OK")):
        word = torch.zeros(64, dtype=torch.int32, device="cuda")
        word[0] = bits
        s = torch.cuda.current_stream().cuda_stream
        assert P.lib().prism_keep_device_status(word.data_ptr(), s) == 0
        assert status() == name


def test_in_a_captured_graph():
    require_gpu()
    status()
    geo, zs, q, k = pool_args(False)
    P.block_pool(geo, zs, q, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.block_pool(geo, zs, q, k)
    graph.replay()
    assert status() == "PRISM_OK"
    zs[1] = 7
    graph.replay()
    assert status() == "PRISM_ERR_DEVICE"
    zs[1] = 0
    graph.replay()
    assert status() == "PRISM_OK"
