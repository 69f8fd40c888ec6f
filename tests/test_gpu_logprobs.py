"""GPU parity of the token log-probabilities against the double oracle.

Tolerance.  x - m is off by 2^-24 of its size; log Z is off by the relative
error of a sum of V terms of one sign, each exp good to 2^-21 and added in
chains of at most V / 256 + 40 fp32 additions: c = (V / 256 + 40) 2^-24 + 2^-21.
A log-probability of size L is off by at most c + 2^-22 (L + 1).  The entropy is
log Z minus a ratio of such sums, whose terms have one sign too: the ratio R is
at most log V in the mean, so c + 2 c R + 2^-22 (R + 1)."""
import numpy as np
import pytest
import torch

from oracle import serving as sv
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


def _call(x, k, targets, ws=None, stream=None):
    rows, V = x.shape
    d = "cuda"
    o = {"logprob": torch.full((rows,), 9.0, device=d), "entropy": torch.full((rows,), 9.0, device=d)}
    if k:
        o["top_idx"] = torch.full((rows, k), -9, dtype=torch.int32, device=d)
        o["top_logprob"] = torch.full((rows, k), 9.0, device=d)
    if ws is None:
        ws = torch.zeros(wb.logprobs_workspace_bytes(rows, V, k), dtype=torch.uint8, device=d)
    t = torch.tensor(targets, dtype=torch.int32, device=d)
    wb.token_logprobs(x, ws, targets=t, stream=stream, **o)
    torch.cuda.synchronize()
    return {n: v.cpu().numpy() for n, v in o.items()}


def _close(got, ref, tol):
    assert np.array_equal(np.isnan(got), np.isnan(ref)), "NaN in other places"
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf])
    f = np.isfinite(ref)
    if f.any():
        e = np.abs(got[f] - ref[f]) / (tol[f] if np.ndim(tol) else tol)
        assert e.max() <= 1, f"worst {e.max():.2f} of the tolerance"


def _check(x, k, targets, got):
    """x: the rows as the kernel read them, on the CPU."""
    rows, V = x.shape
    lp, ent, top = sv.token_logprobs(x.double().numpy(), k)
    c = (V / 256 + 40) * 2.0 ** -24 + 2.0 ** -21
    t = np.asarray(targets)
    ref = np.where(t < 0, 0.0, np.where(t >= V, np.nan, lp[np.arange(rows), np.clip(t, 0, V - 1)]))
    _close(got["logprob"], ref, c + 2.0 ** -22 * (np.abs(ref) + 1))
    R = np.log(max(V, 3)) + 1
    _close(got["entropy"], ent, c + 2 * c * R + 2.0 ** -22 * (R + 1))
    if k:
        assert np.array_equal(got["top_idx"], top), "alternatives"
        r = np.where(top < 0, np.nan, np.take_along_axis(lp, np.maximum(top, 0), -1))
        _close(got["top_logprob"], r, c + 2.0 ** -22 * (np.abs(r) + 1))


def _logits(rows, V, dtype, seed, std=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, V, generator=g) * std).to(dtype)


def _targets(rows, V, seed):
    return np.random.default_rng(seed).integers(0, V, rows).tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 257, 1000, 4096, 4097, 32001, 151936])
def test_vocabulary_sizes(V, dtype):
    rows = 3
    x = _logits(rows, V, dtype, V)
    k = min(V, 20)
    t = _targets(rows, V, V)
    _check(x, k, t, _call(x.cuda(), k, t))


@pytest.mark.parametrize("k", [0, 1, 2, 5, 16, 31, 32])
@pytest.mark.parametrize("rows", [1, 7, 200])
def test_alternatives_and_rows(rows, k):
    x = _logits(rows, 5003, torch.float32, rows + k)
    t = _targets(rows, 5003, k)
    _check(x, k, t, _call(x.cuda(), k, t))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("pad,skip", [(1, 0), (64, 0), (7, 1), (3, 3)])
def test_padded_and_unaligned_rows(pad, skip, dtype):
    """Rows of an odd length inside a wider matrix whose other columns hold NaN."""
    V = 3001
    x = _logits(5, V, dtype, pad)
    wide = torch.full((5, skip + V + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, skip:skip + V] = x.cuda()
    t = _targets(5, V, 1)
    _check(x, 9, t, _call(wide[:, skip:skip + V], 9, t))


@pytest.mark.parametrize("V", [32, 5000, 70000])
def test_equal_values_go_to_the_lower_index(V):
    k = 32
    x = torch.zeros(4, V)
    x[1, V // 2:] = 1.0
    x[2] = torch.arange(V) % 3
    x[3, 1::2] = -0.0   # -0 and +0 are equal
    t = [0, V - 1, V // 3, 1]
    _check(x, k, t, _call(x.cuda(), k, t))


@pytest.mark.parametrize("V", [40, 20000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rising_and_falling_rows(V, dtype):
    """Orders in which every value is a new largest one, or none is."""
    up = torch.linspace(-20, 20, V)
    x = torch.stack([up, -up, up.abs(), -up.abs()]).to(dtype)
    _check(x, 32, [0] * 4, _call(x.cuda(), 32, [0] * 4))


def test_ruled_out_tokens_and_bad_values():
    V, k = 3000, 20
    x = _logits(8, V, torch.float32, 4)
    x[0, ::2] = float("-inf")
    x[1] = float("-inf")
    x[1, 77] = -5.0                      # one token left: log-probability 0, entropy 0
    x[2] = float("-inf")                 # nothing left
    x[3, 100] = float("nan")
    x[4, 100] = float("inf")
    x[5] = float("nan")
    x[6, 5:] = float("nan")              # fewer numbers than alternatives
    x[7] = torch.finfo(torch.float32).min
    t = [0, 77, 3, 4, 100, 0, 2, 9]
    _check(x, k, t, _call(x.cuda(), k, t))


def test_targets_without_a_token_and_outside():
    x = _logits(4, 100, torch.float32, 1)
    t = [-1, 99, -2**31, 5]
    _check(x, 0, t, _call(x.cuda(), 0, t))
    t = [100, 3, 2**31 - 1, 0]
    _check(x, 3, t, _call(x.cuda(), 3, t))
    assert wb.device_error(reset=True) == 4


@pytest.mark.parametrize("std", [0.0, 1e-3, 30.0, 1e4])
def test_flat_and_sharp_rows(std):
    x = _logits(3, 50257, torch.float32, 9, std)
    t = _targets(3, 50257, 3)
    _check(x, 10, t, _call(x.cuda(), 10, t))


def test_outputs_may_be_left_out():
    x = _logits(3, 1000, torch.float32, 2).cuda()
    t = [1, 2, 3]
    whole = _call(x, 4, t)
    ws = torch.zeros(wb.logprobs_workspace_bytes(3, 1000, 4), dtype=torch.uint8, device="cuda")
    lp, ent = torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda")
    ti = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    tl = torch.zeros((3, 4), device="cuda")
    wb.token_logprobs(x, ws, targets=torch.tensor(t, dtype=torch.int32, device="cuda"), logprob=lp)
    wb.token_logprobs(x, ws, entropy=ent)
    wb.token_logprobs(x, ws, top_idx=ti)
    wb.token_logprobs(x, ws, top_logprob=tl)
    torch.cuda.synchronize()
    for a, n in ((lp, "logprob"), (ent, "entropy"), (ti, "top_idx"), (tl, "top_logprob")):
        assert np.array_equal(a.cpu().numpy(), whole[n]), n


def test_rows_past_four_gigabytes():
    """The last of 8200 padded fp32 rows lies past 4 GB."""
    x = torch.zeros((8200, 140000), device="cuda")
    x[8199, 139990] = 11.0
    got = _call(x, 2, [139990] * 8200)
    _check(x[8199:].cpu(), 2, [139990], {n: v[8199:] for n, v in got.items()})
    _check(x[:1].cpu(), 2, [139990], {n: v[:1] for n, v in got.items()})


def test_one_workspace_graph_replay_and_repeated_bits():
    rows, V, k = 5, 33000, 7
    ws = torch.zeros(wb.logprobs_workspace_bytes(rows, V, k), dtype=torch.uint8, device="cuda")
    x = torch.zeros((rows, V), device="cuda")
    t = torch.zeros(rows, dtype=torch.int32, device="cuda")
    o = {"logprob": torch.zeros(rows, device="cuda"), "entropy": torch.zeros(rows, device="cuda"),
         "top_idx": torch.zeros((rows, k), dtype=torch.int32, device="cuda"),
         "top_logprob": torch.zeros((rows, k), device="cuda")}
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    wb.token_logprobs(x, ws, targets=t, stream=s, **o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        wb.token_logprobs(x, ws, targets=t, **o)
    for seed in range(3):
        h = _logits(rows, V, torch.float32, seed)
        tt = _targets(rows, V, seed)
        x.copy_(h)
        t.copy_(torch.tensor(tt, dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        a = {n: v.cpu().numpy() for n, v in o.items()}
        _check(h, k, tt, a)
        g.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(a[n], o[n].cpu().numpy()) for n in a)
        wide = _call(x[:2], k, tt[:2], ws=ws)   # another shape on the same workspace
        _check(h[:2], k, tt[:2], wide)


def test_two_calls_at_once_on_two_streams():
    xs = [_logits(6, 90000, torch.float32, 1), _logits(40, 20000, torch.bfloat16, 2)]
    ts = [_targets(6, 90000, 1), _targets(40, 20000, 2)]
    ks = [20, 5]
    dev = [x.cuda() for x in xs]
    td = [torch.tensor(t, dtype=torch.int32, device="cuda") for t in ts]
    wss = [torch.zeros(wb.logprobs_workspace_bytes(*x.shape, k), dtype=torch.uint8, device="cuda")
           for x, k in zip(xs, ks)]
    outs = [{"logprob": torch.zeros(x.shape[0], device="cuda"),
             "entropy": torch.zeros(x.shape[0], device="cuda"),
             "top_idx": torch.zeros((x.shape[0], k), dtype=torch.int32, device="cuda"),
             "top_logprob": torch.zeros((x.shape[0], k), device="cuda")} for x, k in zip(xs, ks)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            wb.token_logprobs(dev[i], wss[i], targets=td[i], stream=streams[i], **outs[i])
    torch.cuda.synchronize()
    for i in range(2):
        _check(xs[i], ks[i], ts[i], {n: v.cpu().numpy() for n, v in outs[i].items()})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_candidates_than_there_is_room_for(dtype):
    """Rows whose every step beats all before it, in runs of equal values and in
    falling runs inside a rising row, on one CTA a row and on several."""
    V = 40000
    step = torch.arange(V) // 4096
    a = step.float() * 8 + (torch.arange(V) % 4096).float() / 1024
    b = step.float() * 8 - (torch.arange(V) % 4096).float() / 1024
    c = step.float()
    x = torch.stack([a, b, c]).to(dtype)
    for rows in (x, x.repeat(210, 1)):
        t = [7] * rows.shape[0]
        got = _call(rows.cuda(), 32, t)
        _check(rows[:3], 32, t[:3], {n: v[:3] for n, v in got.items()})
        _check(rows[-3:], 32, t[-3:], {n: v[-3:] for n, v in got.items()})


@pytest.mark.parametrize("k", [0, 5, 32])
def test_row_counts_around_the_cuts_on_one_workspace(k):
    """Rows of three steps over three, two and one CTA each, one call after the
    other on the same workspace."""
    V, counts = 9001, [405, 406, 608, 609, 1216, 1217]
    ws = torch.zeros(max(wb.logprobs_workspace_bytes(n, V, k) for n in counts), dtype=torch.uint8,
                     device="cuda")
    for n in counts + counts[:1]:
        x = _logits(n, V, torch.bfloat16, n)
        t = _targets(n, V, n)
        _check(x, k, t, _call(x.cuda(), k, t, ws=ws))


@pytest.mark.parametrize("rows,V,cta,copy", [(2, 151936, 1, 0), (2, 151936, 0, 0), (3, 300000, 50, 1),
                                             (1300, 9001, 7, 0), (1300, 9001, 7, 1), (1300, 9001, 7, 2)])
@pytest.mark.parametrize("k", [0, 5, 20])
def test_a_copy_that_does_not_come(rows, V, cta, copy, k):
    """The wait for it runs out: error 1, that row NaN, the others as ever, back
    after one limit; and the workspace serves the next calls."""
    from _util import tuning
    dtype = torch.bfloat16 if rows > 100 else torch.float32
    limit_ms = 100
    ws = torch.zeros(wb.logprobs_workspace_bytes(rows, V, k), dtype=torch.uint8, device="cuda")
    x, t = _logits(rows, V, dtype, 1), _targets(rows, V, 1)
    whole = _call(x.cuda(), k, t, ws=ws)
    y = _logits(rows, V, dtype, 2)
    other = _call(y.cuda(), k, t, ws=ws)
    dev = x.cuda()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with tuning(timeout_ns=limit_ms * 1_000_000):
        wb.test_withhold(cta, copy)
        try:
            a.record()
            got = _call(dev, k, t, ws=ws)
            b.record()
            torch.cuda.synchronize()
        finally:
            wb.test_withhold(-1)
    assert wb.device_error(reset=True) == 1
    assert limit_ms - 1 <= a.elapsed_time(b) < 1.8 * limit_ms
    bad = 0 if V == 151936 else 1 if V == 300000 else cta
    rest = np.arange(rows) != bad
    for n in whole:
        assert np.array_equal(got[n][rest], whole[n][rest]), n
        if n != "top_idx":
            assert np.isnan(got[n][bad]).all(), n
    for _ in range(2):
        again = _call(y.cuda(), k, t, ws=ws)
        assert all(np.array_equal(again[n], other[n]) for n in other)
        again = _call(dev, k, t, ws=ws)
        assert all(np.array_equal(again[n], whole[n]) for n in whole)
