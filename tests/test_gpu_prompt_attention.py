"""GPU parity of the packed prompt attention against the double oracle.

Tolerance.  u = half a step of the type (bf16 2^-8, fp16 2^-11, relative).  The
probabilities are rounded to the type before the second product (u of each,
so u of sum p |v| = `mag`), the result once more (u of its size); for fp16 a
probability below its smallest normal is off by at most 2^-25 of the row's
reference maximum, n of them by n 2^-25 of the largest |v|.  The scores are
fp32 sums of 128 exact products: off by at most 128 2^-24 of sum |q k| /
sqrt(128), which moves a probability by that much relative, twice (numerator
and sum).  exp2, the sums and the division add a few 2^-22."""
import numpy as np
import pytest
import torch

from oracle import serving as sv
from weight_streaming_gemv_bf16_gb300 import binding as wb

pytestmark = pytest.mark.gpu
D = 128
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert wb.device_error(reset=True) == 0
    yield
    torch.cuda.synchronize()
    assert wb.device_error() == 0


def _inputs(T, nh, nkv, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(T, nh, D, generator=g) * scale).to(dtype)
    k = (torch.randn(T, nkv, D, generator=g) + 0.3).to(dtype)
    v = torch.randn(T, nkv, D, generator=g).to(dtype)
    return q, k, v


def _call(q, k, v, bounds, lse=True, fill=7.0, stream=None):
    """Device run on views of one fused matrix, behind a few columns of another use."""
    T, nh, nkv = q.shape[0], q.shape[1], k.shape[1]
    fused = torch.full((T, (nh + 2 * nkv) * D + 64), float("nan"), dtype=q.dtype, device="cuda")
    w = fused[:, 64:].view(T, nh + 2 * nkv, D)
    w[:, :nh], w[:, nh:nh + nkv], w[:, nh + nkv:] = q.cuda(), k.cuda(), v.cuda()
    out = torch.full((T, nh * D), fill, dtype=q.dtype, device="cuda")
    ls = torch.full((T, nh), fill, device="cuda") if lse else None
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    wb.prompt_attention(w[:, :nh], w[:, nh:nh + nkv], w[:, nh + nkv:], cu, out, lse=ls,
                        stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), None if ls is None else ls.cpu().numpy()


def _check(q, k, v, bounds, out, lse, fill=7.0):
    T, nh = q.shape[:2]
    dq, dk, dv = (x.double().numpy() for x in (q, k, v))
    ref, mag, rl = sv.prompt_attention(dq, dk, dv, bounds)
    got = out.double().numpy().reshape(T, nh, D)
    inside = np.zeros(T, bool)
    for a, b in zip(bounds[:-1], bounds[1:]):
        inside[a:b] = True
    assert (got[~inside] == fill).all(), "rows outside the sequences changed"
    if lse is not None:
        assert (lse[~inside] == fill).all()
    got, ref, mag, rl = got[inside], ref[inside], mag[inside], rl[inside]
    assert np.array_equal(np.isnan(got), np.isnan(ref)), "NaN in other places"
    f = np.isfinite(ref)
    assert np.array_equal(got[~f & ~np.isnan(ref)], ref[~f & ~np.isnan(ref)])
    if not f.any():
        return
    u = U[q.dtype]
    fin = [np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0) for x in (dq, dk, dv)]
    grp = nh // k.shape[1]
    most = max(np.abs(fin[0][:, h]).max(0) @ np.abs(fin[1][:, h // grp]).max(0)
               for h in range(nh)) / np.sqrt(D)
    n = max(b - a for a, b in zip(bounds[:-1], bounds[1:]))
    ds = 128 * 2.0 ** -24 * most
    tol = mag * (u + 2 * ds + 2.0 ** -20) + u * np.abs(ref) + 2.0 ** -24
    if q.dtype == torch.float16:
        tol = tol + n * 2.0 ** -25 * np.abs(fin[2]).max() + 2.0 ** -25
    with np.errstate(invalid="ignore"):
        bad = f & (np.abs(got - ref) > tol)
    assert not bad.any(), (f"{bad.sum()} of {f.sum()} off, worst "
                           f"{(np.abs(got - ref) / tol)[f].max():.2f} of the tolerance at "
                           f"{np.argwhere(bad)[:3].tolist()}")
    if lse is not None:
        r = rl[np.isfinite(rl)]
        assert np.abs(lse[inside][np.isfinite(rl)] - r).max() <= ds + 2.0 ** -21 * (
            np.abs(r).max() + 1)


LENS = [[1], [2], [37], [64], [127], [128], [129], [255], [256], [257], [300, 1, 0, 64, 128, 130],
        [0, 5, 0, 0, 33, 0], [600], [1] * 40, [385, 127, 512]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x))[:24])
def test_lengths(lens, dtype):
    q, k, v = _inputs(sum(lens), 4, 2, dtype, sum(lens) + len(lens))
    bounds = np.concatenate([[0], np.cumsum(lens)]).tolist()
    _check(q, k, v, bounds, *_call(q, k, v, bounds))


@pytest.mark.parametrize("nh,nkv", [(1, 1), (2, 1), (3, 1), (5, 1), (7, 1), (8, 1), (16, 1), (6, 6),
                                    (12, 2), (12, 4), (14, 2), (16, 16), (32, 8)])
@pytest.mark.parametrize("lens", [[200, 77], [390]], ids=["200-77", "390"])
def test_head_layouts(nh, nkv, lens):
    q, k, v = _inputs(sum(lens), nh, nkv, torch.bfloat16, nh * 31 + nkv)
    bounds = np.concatenate([[0], np.cumsum(lens)]).tolist()
    _check(q, k, v, bounds, *_call(q, k, v, bounds))


@pytest.mark.parametrize("nh,nkv", [(4, 2), (3, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_outside_the_sequences(nh, nkv, dtype):
    """Tokens before the first and behind the last sequence hold NaN and
    infinities: they reach nothing, and their rows of out and lse stay."""
    q, k, v = _inputs(500, nh, nkv, dtype, 5)
    for x in (q, k, v):
        x[:9] = float("inf")
        x[333:] = float("nan")
    bounds = [9, 150, 150, 333]
    _check(q, k, v, bounds, *_call(q, k, v, bounds))
    _check(q, k, v, bounds, *_call(q, k, v, bounds, lse=False))


@pytest.mark.parametrize("nh,nkv", [(4, 2), (3, 1), (1, 1)])
@pytest.mark.parametrize("where", [0, 5, 127, 128, 140, 255, 256, 299])
def test_values_that_are_not_finite_reach_only_later_tokens(where, nh, nkv):
    """A NaN or an infinity in one token's value: earlier tokens of its tile,
    and the next sequence, are as without it."""
    q, k, v = _inputs(420, nh, nkv, torch.bfloat16, where + nh)
    v[where, 0, 7] = float("nan")
    v[where, nkv - 1, 30] = float("inf")
    if where > 3:
        v[where - 3, 0, 99] = float("-inf")
    bounds = [0, 300, 420]
    _check(q, k, v, bounds, *_call(q, k, v, bounds))


@pytest.mark.parametrize("where", [3, 130, 299])
def test_keys_that_are_not_finite(where):
    q, k, v = _inputs(420, 4, 2, torch.bfloat16, where)
    k[where, 0, 64] = float("nan")
    bounds = [0, 300, 420]
    _check(q, k, v, bounds, *_call(q, k, v, bounds))
    # a key of the lowest values: scores of -infinity or +infinity by the query's sign
    q, k, v = _inputs(420, 4, 2, torch.bfloat16, where)
    q[:, :2] = q[:, :2].abs() + 0.01
    k[where, 0] = float("-inf")
    _check(q, k, v, bounds, *_call(q, k, v, bounds))


def test_every_score_minus_infinity():
    """The first token's only score is -infinity: its row is 0 / 0; later
    tokens, whose other scores are finite, are not touched by it."""
    q, k, v = _inputs(200, 2, 1, torch.bfloat16, 8)
    q = q.abs() + 0.01
    k[0] = float("-inf")
    _check(q, k, v, [0, 200], *_call(q, k, v, [0, 200]))


@pytest.mark.parametrize("scale", [0.0, 8.0, 60.0])
def test_flat_and_sharp_softmax(scale):
    """Scores from all equal to spread over hundreds, so that the running
    maximum moves by more than any single step allows for."""
    q, k, v = _inputs(700, 4, 2, torch.bfloat16, 17, scale)
    _check(q, k, v, [0, 700], *_call(q, k, v, [0, 700]))


@pytest.mark.parametrize("grow", [1.0, -1.0])
def test_scores_that_grow_along_the_sequence(grow):
    q, k, v = _inputs(900, 2, 1, torch.bfloat16, 23)
    ramp = torch.linspace(0.0, 1.0, 900)[:, None, None] * grow
    k = (k.float() * 0.2 + 3.0 * ramp).to(torch.bfloat16)
    q = (q.float() * 0.2 + 1.0).to(torch.bfloat16)
    _check(q, k, v, [0, 900], *_call(q, k, v, [0, 900]))


def test_bounds_out_of_range_are_skipped_and_flagged():
    q, k, v = _inputs(100, 2, 1, torch.bfloat16, 3)
    for bounds, ok in (([0, 40, 101], [0, 40]), ([-1, 40, 100], [40, 100]),
                       ([0, 60, 50, 100], [0, 60])):
        out, lse = _call(q, k, v, bounds)
        assert wb.device_error(reset=True) == 3
        if bounds == [0, 60, 50, 100]:  # the pair out of order is skipped, the others stand
            _check(q[:50], k[:50], v[:50], [0, 50], out[:50], lse[:50])
        else:
            _check(q, k, v, ok, out, lse)


@pytest.mark.parametrize("at", [0, 31, 32, 50, 69])
def test_one_bad_bound_among_many_sequences(at):
    """70 sequences of 3 tokens, one of them with an end past the tokens (and so
    a start past them for the next): both are skipped and flagged."""
    q, k, v = _inputs(210, 2, 1, torch.bfloat16, at)
    bounds = list(range(0, 211, 3))
    bounds[at + 1] = 100000
    out, lse = _call(q, k, v, bounds)
    assert wb.device_error(reset=True) == 3
    good = [(3 * i, 3 * i + 3) for i in range(70) if i not in (at, at + 1)]
    ref, mag, _ = sv.prompt_attention(*(x.double().numpy() for x in (q, k, v)),
                                      list(range(0, 211, 3)))
    got = out.double().numpy().reshape(210, 2, D)
    rows = np.zeros(210, bool)
    for a, b in good:
        rows[a:b] = True
    assert (got[~rows] == 7.0).all()
    assert (np.abs(got - ref)[rows] <= (U[torch.bfloat16] * (mag + np.abs(ref)) * 1.01 + 1e-6)[rows]).all()


def test_long_sequence_against_the_gpu_in_64_bits():
    """2100 tokens: many tiles of keys per row."""
    q, k, v = _inputs(2100, 4, 2, torch.bfloat16, 99)
    _check(q, k, v, [0, 2100], *_call(q, k, v, [0, 2100]))


def test_runs_are_bit_identical_and_graphs_replay():
    """Captured once, replayed with other inputs and other bounds; the same
    inputs give the same bits every time."""
    T, nh, nkv = 400, 6, 2
    q, k, v = (x.cuda() for x in _inputs(T, nh, nkv, torch.bfloat16, 1))
    cu = torch.tensor([0, 150, 400], dtype=torch.int32, device="cuda")
    out = torch.zeros((T, nh * D), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((T, nh), device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        wb.prompt_attention(q, k, v, cu, out, lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        wb.prompt_attention(q, k, v, cu, out, lse)
    for seed, bounds in ((2, [0, 150, 400]), (3, [0, 390, 400]), (4, [10, 10, 300])):
        hq, hk, hv = _inputs(T, nh, nkv, torch.bfloat16, seed)
        q.copy_(hq), k.copy_(hk), v.copy_(hv)
        cu.copy_(torch.tensor(bounds, dtype=torch.int32))
        out.fill_(7.0), lse.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        first = out.clone(), lse.clone()
        _check(hq, hk, hv, bounds, out.cpu(), lse.cpu().numpy())
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_two_calls_at_once_on_two_streams():
    a = _inputs(700, 4, 2, torch.bfloat16, 51)
    b = _inputs(300, 3, 1, torch.float16, 52)
    dev = [[x.cuda() for x in i] for i in (a, b)]
    cus = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (700, 300)]
    outs = [torch.zeros((d[0].shape[0], d[0].shape[1] * D), dtype=d[0].dtype, device="cuda")
            for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    for _ in range(3):
        for d, c, o, s in zip(dev, cus, outs, streams):
            wb.prompt_attention(*d, c, o, stream=s)
    torch.cuda.synchronize()
    _check(*a, [0, 700], outs[0].cpu(), None)
    _check(*b, [0, 300], outs[1].cpu(), None)


def _withheld(q, k, v, bounds, copy, limit_ms=100):
    """The call with one copy of CTA 0 left out: (out, milliseconds)."""
    from _util import tuning
    dev = [x.cuda() for x in (q, k, v)]
    out = torch.full((q.shape[0], q.shape[1] * D), 7.0, dtype=q.dtype, device="cuda")
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with tuning(timeout_ns=limit_ms * 1_000_000):
        wb.test_withhold(0, copy)
        try:
            a.record()
            wb.prompt_attention(*dev, cu, out)
            b.record()
            torch.cuda.synchronize()
        finally:
            wb.test_withhold(-1)
    return out, a.elapsed_time(b)


# CTA 0 is the longest tile: of one block; of six; of the last two runs of 600
# tokens of one head (blocks 4 and 5 of which tile 1 alone has the last)
@pytest.mark.parametrize("nh,nkv,n,copies", [(2, 1, 100, [0, 1, 2, 3]), (1, 1, 100, [0, 2, 3]),
                                             (2, 1, 700, [0, 1, 2, 3, 4, 5, 6, 9, 10, 11, 12, 13]),
                                             (1, 1, 700, [0, 1, 2, 3, 6, 7, 10, 11, 12, 13])])
def test_a_copy_that_does_not_come(nh, nkv, n, copies):
    """The wait for it runs out: error 1, the other CTAs' rows as ever, and the
    call back after that one limit: what is waited for then are copies and
    products under way, never the one that was not started (that would take a
    second limit).  The next call is right."""
    q, k, v = _inputs(n + 30, nh, nkv, torch.bfloat16, n + nh)
    bounds = [0, n, n + 30]
    whole, _ = _call(q, k, v, bounds)
    _check(q, k, v, bounds, whole, None)
    rows = 128 if nh == 2 else 256
    rest = torch.ones(n + 30, dtype=torch.bool)
    rest[(n - 1) // rows * rows:n] = False  # the longest tile's rows
    for copy in copies:
        out, ms = _withheld(q, k, v, bounds, copy)
        assert wb.device_error(reset=True) == 1, copy
        assert 99 <= ms < 180, (copy, ms)
        assert torch.equal(out.cpu()[rest], whole[rest]), copy
        assert torch.equal(_call(q, k, v, bounds)[0], whole), copy


@pytest.mark.parametrize("nh,nkv", [(2, 1), (1, 1)])
@pytest.mark.parametrize("first", [0, 70, 200])
def test_scores_far_below_zero(first, nh, nkv):
    """Finite scores of -6e34 and less: one key's is the largest by far, so its
    probability is 1, the others' 0, and the output that key's value to the bit;
    a token before it, and the only token of a sequence, take theirs likewise.
    Every score is a power of two's multiple, exact in fp32; the log-sum-exp is
    the score, off by four roundings."""
    T = 300
    _, _, v = _inputs(T + 1, nh, nkv, torch.bfloat16, first)
    q = torch.full((T + 1, nh, D), 2.0 ** 56, dtype=torch.bfloat16)
    k = torch.full((T + 1, nkv, D), -(2.0 ** 58), dtype=torch.bfloat16)
    k[:first] = -(2.0 ** 60) * (1 + torch.arange(first) % 128 / 128)[:, None, None].bfloat16()
    k[first] = -(2.0 ** 56)
    bounds = [0, T, T + 1]
    out, lse = _call(q, k, v, bounds)
    out = out.view(T + 1, nh, D)
    for h in range(nh):
        assert torch.equal(out[first:T, h], v[first, 0].expand(T - first, D))
        assert torch.equal(out[T, h], v[T, 0]) and torch.equal(out[0, h], v[0, 0])
    ref = -128 * 2.0 ** 112 / np.sqrt(D)
    assert np.abs(lse[first:T] / ref - 1).max() <= 2.0 ** -22
    assert np.abs(lse[T] / (4 * ref) - 1).max() <= 2.0 ** -22


@pytest.mark.parametrize("nh,nkv", [(4, 2), (3, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_many_sequences_of_several_tiles(nh, nkv, dtype):
    """More than 32 sequences, some of several tiles, before and behind the 32nd."""
    r = np.random.default_rng(45)
    lens = r.choice([0, 1, 64, 128, 129, 300], 45).tolist()
    lens[3], lens[31], lens[32], lens[33], lens[44] = 513, 257, 640, 0, 385
    bounds = np.concatenate([[0], np.cumsum(lens)]).tolist()
    q, k, v = _inputs(bounds[-1] + 9, nh, nkv, dtype, nh)
    _check(q, k, v, bounds, *_call(q, k, v, bounds))
