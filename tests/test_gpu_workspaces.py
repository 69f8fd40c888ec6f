"""One workspace for calls of several operators and sizes, in turn: each has the
results that it has with a workspace of its own, and leaves the tickets, its first
16 KB, zeroed."""
import pytest
import torch

from weight_streaming_gemv_bf16_gb300 import binding as wb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert wb.device_error(reset=True) == 0
    yield
    torch.cuda.synchronize()
    assert wb.device_error() == 0


def _gemv(M, K, B):
    g = torch.Generator().manual_seed(M + B)
    W = (torch.randn(M, K, generator=g) * 0.02).bfloat16().cuda()
    x = torch.randn(B, K, generator=g).bfloat16().cuda()

    def call(ws):
        y = torch.full((B, M), 7.0, device="cuda")
        wb.gemv_bf16(W, x, y, workspace=ws)
        return [y]
    return wb.workspace_bytes(wb.OP_GEMV, M, K, B), call


def _lmhead(V, K, B):
    g = torch.Generator().manual_seed(V + B)
    W = (torch.randn(V, K, generator=g) * 0.02).bfloat16().cuda()
    h = torch.randn(B, K, generator=g).bfloat16().cuda()
    gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")

    def call(ws):
        idx = torch.full((B,), -7, dtype=torch.int32, device="cuda")
        wb.lmhead_argmax(h, gamma, W, idx, 1e-6, ws)
        return [idx]
    return wb.workspace_bytes(wb.OP_LMHEAD_ARGMAX, V, K, B), call


def _argmax(rows, cols):
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(rows)).cuda()

    def call(ws):
        idx = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
        wb.argmax_rows(x, idx, ws)
        return [idx]
    return wb.workspace_bytes(wb.OP_ARGMAX_ROWS, rows, cols, 1), call


GEMV = [(256, 1536, 3), (128, 4096, 16), (512, 8960, 1), (2048, 1536, 2), (96, 8960, 4), (1536, 8960, 16),
        (20000, 8960, 16)]  # more row groups than the first 16 KB have tickets
LMHEAD = [(20000, 512, 16), (20000, 512, 1), (5000, 1024, 4)]
ARGMAX = [(16, 151936), (1, 1000), (300, 5000), (64, 40), (9000, 700)]


def _calls(which):
    of = {"gemv": (_gemv, GEMV), "lmhead": (_lmhead, LMHEAD), "argmax": (_argmax, ARGMAX)}
    return [of[name][0](*c) for name in which for c in of[name][1]]


@pytest.mark.parametrize("which", [["gemv"], ["lmhead"], ["argmax"], ["gemv", "lmhead", "argmax"]],
                         ids=", ".join)
def test_one_workspace_in_turn(which):
    calls = _calls(which)
    ws = torch.zeros(max(n for n, _ in calls), dtype=torch.uint8, device="cuda")
    own = [call(torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")) for n, call in calls]
    order = list(range(len(calls)))
    for i in order + order[::-1] + order[::2] + order[1::2]:
        got = calls[i][1](ws)
        for x, y in zip(got, own[i]):
            assert torch.equal(x, y), i
        assert int(ws[:16384].count_nonzero()) == 0, i


def test_the_sizes_that_this_is_about():
    """Products split along K, of few and of more than 4096 row groups."""
    for M, K, B in GEMV:
        plan = wb.gemv_plan(M, K, B)
        assert M == 2048 or plan["S"] > 1, (M, K, B)
        assert (plan["RG"] > 4096) == (M == 20000), (M, K, B)


def test_replayed_in_turn_from_a_graph():
    """Calls of several operators and sizes on one workspace in one graph, the memset ahead of the
    large ones among them."""
    calls = _calls(["argmax", "gemv", "lmhead"])
    ws = torch.zeros(max(n for n, _ in calls), dtype=torch.uint8, device="cuda")
    own = [call(ws) for _, call in calls]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = [call(ws) for _, call in calls + calls[::-1]]
        for _ in range(3):
            for x in got:
                x[0].fill_(-7)
            graph.replay()
            side.synchronize()
            for x, y in zip(got, own + own[::-1]):
                assert torch.equal(x[0], y[0])
