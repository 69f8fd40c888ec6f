"""Serving from a paged cache where the calls meet one another or the ends of
their types: one workspace for caches of several sizes."""
import pytest
import torch

from oracle import paged as op
from test_gpu_kv_pages import Cache, _ints
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


# --------------------------------------------------------------------------- the pages' upkeep

def _resize(c, want, ws):
    wb.kv_pages_resize(*c.d, _ints(want), c.ps, ws)
    c.check(op.resize(c.table, c.refs, c.tokens, want, c.ps))


def _fork(c, src, dst, ws):
    wb.kv_pages_fork(*c.d, _ints(src), _ints(dst), c.dk, c.dv, ws)
    c.check(op.fork(c.table, c.refs, c.tokens, src, dst, c.kp, c.vp, c.ps))


def _compact(c, ws):
    wb.kv_pages_compact(*c.d[:2], c.dk, c.dv, ws)
    op.compact(c.table, c.refs, c.kp, c.vp)
    c.check(set())


@pytest.mark.parametrize("last", ["resize", "fork", "compact"])
def test_one_workspace_for_caches_of_few_and_of_many_rows(last):
    """Whatever a call for the one cache leaves there, the other's fork is right."""
    few = Cache(4, 120, 500, 16, layers=1, nkv=1, seed=1).fill([16 * 100, 33, 0, 0])
    many = Cache(300, 3, 700, 16, layers=1, nkv=1, seed=2).fill([40, 17, 32] + [0] * 297)
    ws = torch.zeros(max(wb.kv_pages_workspace_bytes(4, 500), wb.kv_pages_workspace_bytes(300, 700)),
                     dtype=torch.uint8, device="cuda")
    dst = list(range(3, 300))
    for _ in range(2):
        _resize(few, [16 * 20, 16 * 119, -1, -1], ws)
        if last != "resize":
            _fork(few, [1, 1], [3, 2], ws)
        if last == "compact":
            _compact(few, ws)
        _fork(many, [i % 3 for i in dst], dst, ws)
        _resize(many, [-1] * 3 + [0] * 297, ws)
        _compact(many, ws)
        _resize(few, [16 * 100, 33, 0, 0], ws)
