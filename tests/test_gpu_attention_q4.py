"""GPU parity of the decode attention over the 4-bit cache against the double
oracle on the same bytes.

Tolerance (fp32 output).  A score is sum_g s_g (sum q (code - 8)) + z_g (sum
q): q enters as a bf16 pair (2^-17 of each element) in both, so it is off by at
most 2^-17 of `top` = sum |q| (|s (code - 8)| + |z|) / sqrt(128), and by the
fp32 sums of 128 and 4 terms, 132 2^-24 of it: together under 2^-16 top.  That
moves a probability by 2^-16 top relative, twice (numerator and sum).  The
values enter as s (code - 8) and z apart, each times a probability: the pair adds
2^-17 of either part, exp2, the sums and the merges a few 2^-22: |error| <= mag
(2^-15 top + 2^-15), mag = sum p (|s (code - 8)| + |z|).  The bf16 output is the
fp32 one rounded."""
import numpy as np
import pytest
import torch

from oracle import serving as sv
from weight_streaming_gemv_bf16_gb300 import binding as wb

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert wb.device_error(reset=True) == 0
    yield
    torch.cuda.synchronize()
    assert wb.device_error() == 0


def _inputs(B, nh, nkv, S, pos, seed, q_std=1.0):
    """Caches filled up to pos; what lies from pos on is 0xff bytes (NaN scales)."""
    r = np.random.default_rng(seed)
    q = (r.standard_normal((B, nh * D)) * q_std).astype(np.float32)
    kn = r.standard_normal((B, nkv * D)).astype(np.float32)
    vn = r.standard_normal((B, nkv * D)).astype(np.float32)
    kc = np.full((B, nkv, S, 80), 255, np.uint8)
    vc = np.full((B, nkv, S, 80), 255, np.uint8)
    off = r.standard_normal(D).astype(np.float32)
    for b, p in enumerate(pos):
        p = min(max(p, 0), S)
        kc[b, :, :p] = sv.quantize_rows(r.standard_normal((nkv, p, D)).astype(np.float32) + off, True)
        vc[b, :, :p] = sv.quantize_rows(r.standard_normal((nkv, p, D)).astype(np.float32), False)
    return q, kn, vn, kc, vc


def _dev(*arrays):
    return [torch.from_numpy(np.array(a)).cuda() for a in arrays]


def _ws(B, nh, nkv, S):
    return torch.zeros(wb.attention_q4_workspace_bytes(B, nh, nkv, S), dtype=torch.uint8,
                       device="cuda")


def _compare(q, kn, vn, kc, vc, pos, o32, o16, dk, dv):
    out, mag, top, rk, rv = sv.decode_attention_q4(q, kn, vn, kc, vc, pos)
    assert np.array_equal(dk.cpu().numpy(), rk), "key cache"
    assert np.array_equal(dv.cpu().numpy(), rv), "value cache"
    got = o32.cpu().numpy().astype(np.float64)
    live = ~np.isnan(out)
    assert (got[~live] == 7.0).all(), "a row without a sequence changed"
    tol = mag * 2.0 ** -15 * (np.repeat(top, D, axis=1) + 1)
    err = np.abs(got - out)
    assert (err[live] <= tol[live]).all(), f"worst {(err / tol)[live].max():.2f} of the tolerance"
    if o16 is not None:
        assert torch.equal(o16, o32.to(torch.bfloat16))


def _run(B, nh, nkv, S, pos, seed, q_std=1.0, ws=None, both=True):
    host = _inputs(B, nh, nkv, S, pos, seed, q_std)
    q, kn, vn, kc, vc = _dev(*host)
    o32 = torch.full((B, nh * D), 7.0, device="cuda")
    o16 = torch.full((B, nh * D), 7.0, dtype=torch.bfloat16, device="cuda") if both else None
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    wb.decode_attention_q4(q, kn, vn, kc, vc, p, _ws(B, nh, nkv, S) if ws is None else ws,
                           out_f32=o32, out_bf16=o16)
    torch.cuda.synchronize()
    _compare(*host, pos, o32, o16, kc, vc)


@pytest.mark.parametrize("n", [1, 2, 3, 8, 9, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 200, 1000])
def test_lengths(n):
    _run(2, 12, 2, 1000, [n - 1, (n - 1) // 2], n)


@pytest.mark.parametrize("nh,nkv", [(1, 1), (2, 1), (3, 1), (4, 1), (5, 1), (6, 2), (7, 1), (8, 1),
                                    (8, 8), (16, 2), (32, 8)])
def test_group_sizes(nh, nkv):
    _run(3, nh, nkv, 300, [299, 130, 4], nh * 10 + nkv)


@pytest.mark.parametrize("S", [1, 5, 16, 77, 257])
def test_odd_caches_filled_to_the_last_slot(S):
    _run(2, 4, 2, S, [S - 1, 0], S)


@pytest.mark.parametrize("B", [1, 16, 33])
def test_ragged_batches(B):
    r = np.random.default_rng(B)
    pos = r.integers(0, 640, B).tolist()
    pos[0] = 639
    _run(B, 12, 2, 640, pos, B)


# 96 rows and 8 heads: more (row, head)s than CTAs are resident on the device,
# so one CTA works through several short ones, some of its warps on none of them
@pytest.mark.parametrize("nh", [8, 40])
@pytest.mark.parametrize("top", [1, 33, 65, 130])
def test_many_short_sequences(nh, top):
    r = np.random.default_rng(nh + top)
    pos = r.integers(-1, top, 96).tolist()
    pos[:3] = [top - 1, 0, -1]
    _run(96, nh, 8, top, pos, nh + top)


def test_many_short_sequences_and_a_long_one():
    r = np.random.default_rng(11)
    pos = r.integers(0, 160, 70).tolist()
    pos[35] = 4999
    _run(70, 12, 4, 5000, pos, 11)


def test_long_cache_in_many_splits():
    _run(1, 12, 2, 40000, [39999], 3)
    _run(2, 8, 8, 9001, [9000, 17], 4)


@pytest.mark.parametrize("q_std", [0.0, 8.0, 100.0])
def test_flat_and_sharp_softmax(q_std):
    _run(2, 12, 2, 1024, [1023, 700], 5, q_std)


def test_rows_without_a_sequence_and_positions_outside():
    _run(4, 4, 2, 100, [-1, 50, -7, 99], 6)
    host = _inputs(2, 4, 2, 100, [100, 40], 7)
    q, kn, vn, kc, vc = _dev(*host)
    o32 = torch.full((2, 512), 7.0, device="cuda")
    p = torch.tensor([100, 40], dtype=torch.int32, device="cuda")
    wb.decode_attention_q4(q, kn, vn, kc, vc, p, _ws(2, 4, 2, 100), out_f32=o32)
    torch.cuda.synchronize()
    assert wb.device_error(reset=True) == 2
    _compare(*host, [100, 40], o32, None, kc, vc)


def test_nan_rows_in_the_cache():
    """A cached key or value that stands for NaN gives NaN to the heads that
    read it, a value in its group's dimensions alone, and to no other."""
    host = list(_inputs(2, 4, 2, 300, [200, 200], 8))
    host[3][0, 0, 77, 64:68] = 255     # key row 77 of head 0: group 0 NaN
    host[4][0, 1, 150, 68:72] = 255    # value row 150 of head 1: group 1 NaN
    q, kn, vn, kc, vc = _dev(*host)
    o = torch.zeros((2, 512), device="cuda")
    p = torch.tensor([200, 200], dtype=torch.int32, device="cuda")
    wb.decode_attention_q4(q, kn, vn, kc, vc, p, _ws(2, 4, 2, 300), out_f32=o)
    nan = torch.isnan(o).cpu().view(2, 4, 4, 32)
    assert nan[0, :2].all() and not nan[1].any()
    assert nan[0, 2:, 1].all() and not nan[0, 2:, 0].any() and not nan[0, 2:, 2:].any()


@pytest.mark.parametrize("S", [64, 5000])
def test_one_workspace_for_many_calls_and_graph_replay(S):
    """One workspace serves calls of falling and rising lengths, eager and
    replayed; each step's appended row is read by the next."""
    B, nh, nkv = 3, 12, 2
    pos = np.array([S // 2, 3, 0], np.int32)
    host = list(_inputs(B, nh, nkv, S, pos, 9))
    q, kn, vn, kc, vc = _dev(*host)
    ws = _ws(B, nh, nkv, S)
    o32 = torch.full((B, nh * D), 7.0, device="cuda")
    p = torch.tensor(pos, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        wb.decode_attention_q4(q, kn, vn, kc, vc, p, ws, out_f32=o32, stream=s)
    torch.cuda.synchronize()
    _compare(*host, pos, o32, None, kc, vc)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        wb.decode_attention_q4(q, kn, vn, kc, vc, p, ws, out_f32=o32)
    host[3], host[4] = kc.cpu().numpy(), vc.cpu().numpy()
    for step in range(4):
        pos = pos + 1 if step != 2 else np.array([1, S - 1, S - 1], np.int32) - [0, 1, 2]
        if step == 2:  # fill what the jump skips
            fill = _inputs(B, nh, nkv, S, pos, 90)
            host[3], host[4] = fill[3], fill[4]
            kc.copy_(torch.from_numpy(host[3])), vc.copy_(torch.from_numpy(host[4]))
        new = _inputs(B, nh, nkv, 1, [0] * B, 100 + step)[:3]
        host[:3] = new
        for d, h in zip((q, kn, vn), new):
            d.copy_(torch.from_numpy(h))
        p.copy_(torch.from_numpy(pos.astype(np.int32)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _compare(*host, pos, o32, None, kc, vc)
        host[3], host[4] = kc.cpu().numpy(), vc.cpu().numpy()


def test_runs_are_bit_identical():
    host = _inputs(4, 32, 8, 3000, [2999, 1500, 64, 0], 12)
    q, kn, vn, kc, vc = _dev(*host)
    p = torch.tensor([2999, 1500, 64, 0], dtype=torch.int32, device="cuda")
    ws = _ws(4, 32, 8, 3000)
    outs = []
    for _ in range(4):
        o = torch.zeros((4, 32 * D), device="cuda")
        wb.decode_attention_q4(q, kn, vn, kc, vc, p, ws, out_f32=o)
        outs.append(o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


def test_two_calls_at_once_on_two_streams():
    """Each with a workspace of its own, long enough to overlap; replayed from
    two graphs too."""
    hosts = [_inputs(2, 12, 2, 6000, [5999, 3000], 31), _inputs(3, 8, 8, 2500, [2499, 1200, 7], 32)]
    pos = [[5999, 3000], [2499, 1200, 7]]
    dev = [_dev(*h) for h in hosts]
    ps = [torch.tensor(p, dtype=torch.int32, device="cuda") for p in pos]
    wss = [_ws(2, 12, 2, 6000), _ws(3, 8, 8, 2500)]
    outs = [torch.full((d[0].shape[0], d[0].shape[1]), 7.0, device="cuda") for d in dev]
    streams = [torch.cuda.Stream() for _ in dev]
    torch.cuda.synchronize()
    def call(i, stream=None):
        wb.decode_attention_q4(*dev[i], ps[i], wss[i], out_f32=outs[i], stream=stream)
    for _ in range(5):
        for i in range(2):
            call(i, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        _compare(*hosts[i], pos[i], outs[i], None, dev[i][3], dev[i][4])
        outs[i].fill_(7.0)
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            call(i)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        _compare(*hosts[i], pos[i], outs[i], None, dev[i][3], dev[i][4])


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e6, 1e18])
def test_values_of_every_size(size):
    """Values far from one, down to steps near the smallest normals of bf16."""
    host = list(_inputs(2, 6, 2, 200, [199, 30], 15))
    r = np.random.default_rng(15)
    for b, p in enumerate([199, 30]):
        host[4][b, :, :p] = sv.quantize_rows((r.standard_normal((2, p, D)) * size).astype(np.float32), False)
    host[2] = (host[2] * size).astype(np.float32)
    q, kn, vn, kc, vc = _dev(*host)
    o = torch.full((2, 6 * D), 7.0, device="cuda")
    p = torch.tensor([199, 30], dtype=torch.int32, device="cuda")
    wb.decode_attention_q4(q, kn, vn, kc, vc, p, _ws(2, 6, 2, 200), out_f32=o)
    torch.cuda.synchronize()
    _compare(*host, [199, 30], o, None, kc, vc)


@pytest.mark.parametrize("nh", [2, 6])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_queries_that_are_not_finite(nh, bad):
    """One head's query: NaN for that head alone."""
    host = list(_inputs(1, nh, 1, 100, [80], 16))
    host[0][0, D + 5] = bad
    q, kn, vn, kc, vc = _dev(*host)
    o = torch.zeros((1, nh * D), device="cuda")
    p = torch.tensor([80], dtype=torch.int32, device="cuda")
    wb.decode_attention_q4(q, kn, vn, kc, vc, p, _ws(1, nh, 1, 100), out_f32=o)
    nan = torch.isnan(o).cpu().view(nh, D)
    assert nan[1].all() and not nan[0].any() and not nan[2:].any()


def test_appends_the_bytes_that_the_store_writes():
    host = _inputs(3, 4, 2, 20, [0, 7, 19], 13)
    q, kn, vn, kc, vc = _dev(*host)
    p = torch.tensor([0, 7, 19], dtype=torch.int32, device="cuda")
    k2, v2 = kc.clone(), vc.clone()
    wb.decode_attention_q4(q, kn, vn, kc, vc, p, _ws(3, 4, 2, 20),
                           out_f32=torch.zeros((3, 512), device="cuda"))
    wb.kv_store_q4(kn.view(3, 2, D), vn.view(3, 2, D), k2, v2, p)
    torch.cuda.synchronize()
    assert torch.equal(kc, k2) and torch.equal(vc, v2)


def test_offsets_past_four_gigabytes():
    """The second row's last head of a 4.4 GB cache."""
    S, n = 6_900_000, 50
    kc = torch.full((2, 4, S, 80), 255, dtype=torch.uint8, device="cuda")
    vc = torch.full((2, 4, S, 80), 255, dtype=torch.uint8, device="cuda")
    host = _inputs(2, 4, 4, n, [n - 1] * 2, 14)
    q, kn, vn, k, v = _dev(*host)
    kc[:, :, :n], vc[:, :, :n] = k, v
    o = torch.full((2, 512), 7.0, device="cuda")
    p = torch.tensor([n - 1] * 2, dtype=torch.int32, device="cuda")
    wb.decode_attention_q4(q, kn, vn, kc, vc, p, _ws(2, 4, 4, S), out_f32=o)
    torch.cuda.synchronize()
    _compare(*host, [n - 1] * 2, o, None, kc[:, :, :n], vc[:, :, :n])


@pytest.mark.parametrize("nh", [4, 6])
@pytest.mark.parametrize("n,best", [(1, 0), (40, 0), (40, 39), (200, 70), (9000, 5000), (9000, 8999)])
def test_scores_far_below_zero(n, best, nh):
    """Finite scores of -6e34 and less: one slot's is the largest by far, so its
    probability is 1, the others' 0, and the output the value that its row stands
    for, to the bit (the part of the codes is exact, the zero joins in one
    rounding, as in the load)."""
    host = list(_inputs(1, nh, 1, n, [n - 1], n + best))
    host[0][:] = 2.0 ** 56
    k = np.full((1, n, D), -(2.0 ** 58), np.float32)
    k[0, best] = -(2.0 ** 56)
    host[3][0, :, :n - 1] = sv.quantize_rows(k[:, :n - 1], True)
    host[1][:] = k[0, n - 1]
    q, kn, vn, kc, vc = _dev(*host)
    o = torch.full((1, nh * D), 7.0, device="cuda")
    p = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    wb.decode_attention_q4(q, kn, vn, kc, vc, p, _ws(1, nh, 1, n), out_f32=o)
    torch.cuda.synchronize()
    ref = sv.dequantize_rows(vc[0, 0, best].cpu().numpy(), False)
    assert np.array_equal(o.cpu().numpy().reshape(nh, D), np.broadcast_to(ref, (nh, D)))
