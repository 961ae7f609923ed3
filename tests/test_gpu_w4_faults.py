"""4-bit expert products when something goes wrong: bad offsets, waits that run out, calls cut short.

No GPU is faulted: bad offsets are checked in the kernel, and every wait has a time limit.
"""
import ctypes
import time

import pytest
import torch

import sparse_mixture_experts_08_b200 as moe
from gpu_helpers import require_gpu
from test_gpu_w4 import _segments, make_experts

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


# rows of 3 segments, d, f: tiles of 16, 32, 64, 128, 192 rows, and of 224 in the first, the second and both products
HEIGHTS = [(12, 64, 96), (45, 352, 544), (90, 352, 1120), (300, 352, 544), (600, 352, 544), (600, 4096, 96),
           (600, 96, 4128), (600, 4128, 4096)]


def _grouped(rows, d, f, m=3, act=moe.SWIGLU):
    """A configuration, weights, input rows and good offsets of m segments that share `rows` rows."""
    gen = torch.Generator().manual_seed(rows + d + f)
    wq, _ = make_experts(gen, m, d, f, 32, act)
    x = torch.randn(rows, d, generator=gen).to(torch.bfloat16).cuda()
    lengths = [rows // m] * (m - 1)
    return moe.make_config(rows, d, f, m, 1, act=act), wq, x, _segments(lengths + [rows - sum(lengths)])


@pytest.mark.parametrize("rows,d,f", HEIGHTS)
def test_bad_offsets_leave_everything_unwritten_in_every_tile_height(rows, d, f):
    """All blocks of a launch come to the same verdict: no row is written, and none of them waits for another that
    dropped its work (the wait limit is 2 s)."""
    c, wq, x, good = _grouped(rows, d, f)
    ws = moe.w4_workspace(c)
    want = torch.empty(rows, d, device="cuda")
    moe.moe_grouped_ffn_w4(c, x, good, wq, None, None, want, ws)
    assert moe.moe_read_device_status(ws) == moe.OK
    a, b = good.tolist()[1:3]
    for offsets in ([0, a, b, rows + 1], [0, a, a - 1, rows], [-1, a, b, rows], [0, a, b, -5], [0, rows + 7, b, rows]):
        bad = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        y = torch.full((rows, d), -7.0, device="cuda")
        torch.cuda.synchronize()
        start = time.perf_counter()
        moe.moe_grouped_ffn_w4(c, x, bad, wq, None, None, y, ws)
        assert moe.moe_read_device_status(ws) == moe.ERR_DEVICE_INDEX
        assert time.perf_counter() - start < 1.0
        assert (y == -7.0).all()
    y = torch.empty_like(want)
    moe.moe_grouped_ffn_w4(c, x, good, wq, None, None, y, ws)
    assert moe.moe_read_device_status(ws) == moe.OK and torch.equal(y, want)


@pytest.mark.parametrize("rows", [100, 2200])
def test_one_bad_offset_among_many_groups(rows):
    c, wq, x, good = _grouped(rows, 96, 64, m=70)
    ws = moe.w4_workspace(c)
    for at, value in ((70, rows + 1), (64, 0), (1, rows)):
        bad = good.clone()
        bad[at] = value
        y = torch.full((rows, 96), -7.0, device="cuda")
        moe.moe_grouped_ffn_w4(c, x, bad, wq, None, None, y, ws)
        assert moe.moe_read_device_status(ws) == moe.ERR_DEVICE_INDEX and (y == -7.0).all()


class _Cudart:
    """The runtime calls that take a node out of a graph."""

    def __init__(self):
        self.lib = ctypes.CDLL("libcudart.so.12")

    def call(self, name, *args):
        assert getattr(self.lib, name)(*args) == 0, name

    def nodes(self, graph):
        n = ctypes.c_size_t(0)
        self.call("cudaGraphGetNodes", graph, None, ctypes.byref(n))
        nodes = (ctypes.c_void_p * n.value)()
        self.call("cudaGraphGetNodes", graph, nodes, ctypes.byref(n))
        return [ctypes.c_void_p(v) for v in nodes]

    def last_node(self, graph):
        """The node that no other depends on."""
        def dependents(node):
            n = ctypes.c_size_t(0)
            self.call("cudaGraphNodeGetDependentNodes", node, None, ctypes.byref(n))
            return n.value
        last = [node for node in self.nodes(graph) if dependents(node) == 0]
        assert len(last) == 1
        return last[0]


@pytest.mark.parametrize("rows,d,f", [(300, 352, 4128), (600, 352, 4128), (600, 4128, 4096)])
def test_a_call_cut_short_after_its_first_product_leaves_no_counters(rows, d, f):
    """The first product is launched, the second is not (what a call leaves that returns an error between them): the
    next calls on the workspace find their counters of cut tiles at zero."""
    c, wq, x, good = _grouped(rows, d, f)
    ws, y = moe.w4_workspace(c), torch.empty(rows, d, device="cuda")
    inputs = [torch.roll(x, i, 1) for i in range(4)]  # other rows each time: what the workspace holds of h is stale
    want = []
    for xi in inputs:
        want.append(torch.empty(rows, d, device="cuda"))
        moe.moe_grouped_ffn_w4(c, xi, good, wq, None, None, want[-1], moe.w4_workspace(c))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        moe.moe_grouped_ffn_w4(c, x, good, wq, None, None, y, ws)
    rt, handle = _Cudart(), ctypes.c_void_p(graph.raw_cuda_graph())
    assert len(rt.nodes(handle)) == 2  # a launch for each product
    rt.call("cudaGraphDestroyNode", rt.last_node(handle))
    graph.instantiate()
    for cut_short in (1, 2, 3):
        for _ in range(cut_short):
            graph.replay()
        y.fill_(float("nan"))
        moe.moe_grouped_ffn_w4(c, inputs[cut_short], good, wq, None, None, y, ws)
        assert moe.moe_read_device_status(ws) == moe.OK and torch.equal(y, want[cut_short])


# rows of 3 segments, d, f: several tiles a block in every tile height (16, 32, 64, 128, 192, 224), a few chunks each
STALLED = [(12, 288, 30752), (45, 288, 30752), (90, 288, 30752), (300, 288, 10240), (700, 288, 10240),
           (700, 4128, 2080)]


@pytest.mark.parametrize("stall", [1, 2, 3])
@pytest.mark.parametrize("rows,d,f", STALLED)
def test_stalled_products_time_out_and_the_next_calls_are_right(rows, d, f, stall):
    """The hook keeps a barrier from ever completing (1), or stops the input rows of a block, of either block of a
    pair, whose copies the other block's barrier counts (2, 3): the call can only end at its time limit, 1 ms, with
    every copy settled, and the workspace works again."""
    c, wq, x, good = _grouped(rows, d, f, act=moe.RELU)
    ws = moe.w4_workspace(c)
    want, y = torch.empty(rows, d, device="cuda"), torch.empty(rows, d, device="cuda")
    moe.moe_grouped_ffn_w4(c, x, good, wq, None, None, want, ws)
    assert moe.moe_read_device_status(ws) == moe.OK
    start = time.perf_counter()
    try:
        moe.moe_debug_set_wait_limit_ns(1_000_000)
        moe.moe_debug_set_barrier_extra(stall)
        for _ in range(2):
            moe.moe_grouped_ffn_w4(c, x, good, wq, None, None, y, ws)
            status = moe.moe_read_device_status(ws)
            # (blocks without a pair have no second block to stop)
            assert status == (moe.OK if stall == 3 and rows < 90 else moe.ERR_TIMEOUT)
    finally:
        moe.moe_debug_set_barrier_extra(0)
        moe.moe_debug_set_wait_limit_ns(0)
    # every copy is settled: a barrier that lacks one is waited for 200 ms in each of the two calls
    assert time.perf_counter() - start < 0.4
    for _ in range(3):
        y.fill_(float("nan"))
        moe.moe_grouped_ffn_w4(c, x, good, wq, None, None, y, ws)
        assert moe.moe_read_device_status(ws) == moe.OK and torch.equal(y, want)


def test_one_buffer_for_atomic_and_4_bit_calls():
    """What an atomic-expert call writes into a workspace leaves the 4-bit products' counters alone."""
    ac = moe.make_atomic_config(8, 256, 64, 64, 16, moe.ATOMIC_SILU)
    gen = torch.Generator().manual_seed(2)
    ax, wr, wc, wi, wo = ((torch.randn(n, 256, generator=gen) / 16).to(torch.bfloat16).cuda()
                          for n in (8, 64, 64, 4096, 4096))
    out, first = torch.empty_like(ax), torch.empty_like(ax)
    for rows, d, f in HEIGHTS[:6]:
        c, wq, x, good = _grouped(rows, d, f)
        want, y = torch.empty(rows, d, device="cuda"), torch.full((rows, d), float("nan"), device="cuda")
        moe.moe_grouped_ffn_w4(c, x, good, wq, None, None, want, moe.w4_workspace(c))
        size = max(moe.moe_w4_workspace_size(c), moe.moe_atomic_workspace_size(ac))
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        moe.moe_atomic_forward(ac, ax, wr, wc, wi, wo, first, ws)
        moe.moe_grouped_ffn_w4(c, x, good, wq, None, None, y, ws)
        moe.moe_atomic_forward(ac, ax, wr, wc, wi, wo, out, ws)
        assert moe.moe_read_device_status(ws) == moe.OK
        assert torch.equal(y, want) and torch.equal(out, first)
