"""Serving from a paged cache where the calls meet one another or the ends of
their types and sizes: one workspace for caches of several sizes, queries and keys
at the ends of their types, copies that do not come, offsets beyond 32 bits.
Tolerances are test_gpu_paged's where none is given."""
import numpy as np
import pytest
import torch

from _util import tuning
from oracle import paged as op
from test_gpu_kv_pages import Cache, _ints
from test_gpu_paged import DT, Case, D, _ws
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


# --------------------------------------------------------------------------- attention

def _one_hot_keys(c, dims, sizes):
    """Slot j's key: sizes[j] in dimension dims[j] (one power of two times a short fraction), zeros
    elsewhere; the last slot is the new row.  Products with it are exact, and so are their sums."""
    c.kp[c.kp == c.kp] = 0.0
    n = c.pos[0] + 1
    for j in range(n):
        if j < n - 1:
            c.kp[c.table[0][j // c.ps], :, j % c.ps, dims[j]] = sizes[j]
    c.kn[:] = 0.0
    c.kn.view(-1, c.nkv, D)[:, :, dims[n - 1]] = sizes[n - 1]
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", [2.0 ** 60, 2.0 ** 110, 2.0 ** 118, 2.0 ** 126, 1.5 * 2.0 ** 127])
def test_fp32_queries_of_any_size(dtype, size):
    """Finite scores, the largest 2^-6 of itself and more above the others: its slot's value to the
    bit, and the log-sum-exp that score, off by the queries' 2^-22 and four roundings (2^-22)."""
    n = 40
    c = Case([n - 1], 2, 1, 16, dtype, seed=31)
    c.q[:] = size
    c.q[:, 1::2] *= -1.0
    _one_hot_keys(c, [2 * j for j in range(n)], [2.0 ** -14 * (1 + j / 64) for j in range(n)])
    c.device()
    c.call(_ws(2, 1))
    best = c.vn[0].to(c.dt).float()
    ref = size * 2.0 ** -14 * (1 + (n - 1) / 64) / D ** 0.5
    for h in range(2):
        assert torch.equal(c.o32[0, h * D:(h + 1) * D].cpu(), best)
    assert (c.lse.cpu().double() / ref - 1).abs().max() <= 2.0 ** -21


@pytest.mark.parametrize("dtype,q", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinite_key_counts_as_its_scores_do(sign, dtype, q):
    """Head 0's score of slot 19 is -infinity: weight 0, what the other slots give (or NaN, where an
    fp32 query's terms differ in sign or one of them is 0); head 1's is +infinity: NaN.  The
    tolerance is that of finite keys."""
    c = Case([40], 2, 1, 16, dtype, q, seed=32)
    c.kp[c.table[0][1], 0, 3, 5] = sign * float("inf")
    c.q[0, 5], c.q[0, D + 5] = -sign, sign
    c.device()
    c.call(_ws(2, 1))
    pages = torch.tensor(c.table[0])
    K, V = (x[pages, 0].reshape(-1, D)[:41].double().numpy() for x in (c.kp, c.vp))
    K[40], V[40] = (x[0].to(c.dt).double().numpy() for x in (c.kn, c.vn))
    rest = np.arange(41) != 19
    s = K[rest] @ c.q[0, :D].double().numpy() / np.sqrt(D)
    top = (np.abs(K[rest]) @ np.abs(c.q[0, :D].double().numpy())).max() / np.sqrt(D)
    e = np.exp(s - s.max())
    out, mag = e / e.sum() @ V[rest], e / e.sum() @ np.abs(V[rest])
    got, lse = c.o32.cpu().double().numpy()[0], c.lse.cpu().double().numpy()[0]
    assert np.isnan(got[D:]).all() and np.isnan(lse[1])
    if q == "f32" and np.isnan(lse[0]):
        assert np.isnan(got[:D]).all()
        return
    assert (np.abs(got[:D] - out) <= mag * 2.0 ** -15 * (top + 1)).all()
    assert abs(lse[0] - s.max() - np.log(e.sum())) <= 2.0 ** -16 * top + 2.0 ** -18 + 2.0 ** -21 * abs(lse[0])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 2, 40])
def test_fp32_queries_enter_with_all_their_terms(n, dtype):
    """Keys with one element each, so that no sum is rounded: what is left is the queries' terms.  A
    query of 1 + 2^-9 + 2^-17 - 2^-23 takes three bf16 terms (exactly) or two fp16 ones (to 2^-22).
    Scores then carry the scale's rounding, the product's, its difference from the maximum's and
    the change of base: 4 x 2^-24 of the largest (2^-22), in fp16 twice that; the log-sum-exp two
    more of its own, and exp2, the sum and the logarithm a few 2^-22 (2^-19).  So 2^-20 top +
    2^-19; with one term fewer the scores are off by 2^-17 of themselves, which is 4 times as much
    as that and more (checked here in 64 bits)."""
    c = Case([n - 1], 2, 1, 16, dtype, seed=33)
    r = np.random.default_rng(n)
    x = 1 + 2.0 ** -9 + 2.0 ** -17 - 2.0 ** -23
    c.q[:] = torch.from_numpy(x * r.choice([-1.0, 1.0], c.q.shape)).float()
    sizes = r.choice([256.0, 512.0, 1024.0, 2048.0], n)
    sizes[r.integers(n)] = 4096.0
    _one_hot_keys(c, r.permutation(D)[:n].tolist(), sizes.tolist())
    c.device()
    c.call(_ws(2, 1))
    (out, mag, lse, top), _, _ = c.oracle()
    got, glse = c.o32.cpu().double().numpy().reshape(out.shape), c.lse.cpu().double().numpy()
    tol = 2.0 ** -20 * top + 2.0 ** -19
    assert (np.abs(glse - lse) <= tol).all()
    # a probability moves by twice a score's error; the pairs' 2^-17, exp2 and the sums: 2^-16
    assert (np.abs(got - out) <= mag * (2 * tol + 2.0 ** -16)[..., None]).all()
    if dtype == "bf16":
        hi = c.q.bfloat16().float()
        c.q = hi + (c.q - hi).bfloat16().float()
        (_, _, two, _), _, _ = c.oracle()
        assert (np.abs(two - lse) >= 4 * tol)[np.abs(lse) > 0.7 * top].all()


# units of 16 slots that CTA 0 has: one of each warp; two a warp; three or four a warp, more than the
# ring's stages; the only units of several rows, each of which it begins
@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("pos,own,units", [([200, 100], [0], [0, 1, 3]), ([40000, 333], [0], [0, 5, 7]),
                                           ([60000], [0], [0, 5, 8, 11]), ([15] * 1024, [0, 1, 2, 3], [0])])
def test_a_copy_that_does_not_come(pos, own, units, q):
    """The wait for it runs out: error 1, the rows of other CTAs as ever, and the call back within a
    limit for each copy under way and one; the workspace serves the next call."""
    limit_ms = 50
    c = Case(pos, 2, 1, 64, "bf16", q, seed=34).device()
    ws = _ws(2, 1, len(pos))
    c.call(ws)
    torch.cuda.synchronize()
    whole = [x.clone() for x in (c.o32, c.o16, c.lse)]
    rest = torch.tensor([b not in own for b in range(len(pos))])
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for unit in units:
        for x in (c.o32, c.o16, c.lse):
            x.fill_(7.0)
        with tuning(timeout_ns=limit_ms * 1_000_000):
            wb.test_withhold(0, unit)
            try:
                begin.record()
                c.call(ws)
                end.record()
                torch.cuda.synchronize()
            finally:
                wb.test_withhold(-1)
        assert wb.device_error(reset=True) == 1, unit
        assert limit_ms - 1 <= begin.elapsed_time(end) < 4.5 * limit_ms
        for x, y in zip((c.o32, c.o16, c.lse), whole):
            assert torch.equal(x[rest], y[rest]), unit
        c.call(ws)
        torch.cuda.synchronize()
        for x, y in zip((c.o32, c.o16, c.lse), whole):
            assert torch.equal(x, y), unit


def test_one_table_row_read_by_several_batch_rows():
    """Without new rows a sequence may be read any number of times, to other lengths too."""
    c = Case([40, 200], 4, 2, 32, seed=35, rows=[0, 1], new=False)
    c.pos, c.rows = [200, 64, 200, 13], [1, 1, 1, 0]
    c.q = torch.cat([c.q, -c.q])
    c.device()
    c.call(_ws(4, 2, 4))
    c.check()


def test_pages_beyond_32_bits():
    """A cache of more than 2^31 elements, its last pages in use: stored into, read, brought down."""
    nkv, ps = 2, 64
    n_pages = (1 << 24) // (nkv * ps) + 700
    c = Case([150, 63], 4, nkv, ps, seed=36)
    low = {p for row in c.table for p in row if p >= 0}
    up = {p: n_pages - 1 - 3 * i for i, p in enumerate(sorted(low))}
    kp, vp = (wb.new_kv_pages(n_pages, nkv, ps) for _ in range(2))
    table, refs, tokens = wb.new_page_table(2, len(c.table[0]), n_pages)
    table.copy_(_ints([[up.get(p, -1) for p in row] for row in c.table]))
    for p, at in up.items():
        refs[at] = 1
    # the rows' tokens but the last through the store, the last by the attention
    for b, n in enumerate(c.pos):
        pages = torch.tensor(c.table[b][:n // ps + 1])
        k, v = (x[pages].transpose(1, 2).reshape(-1, nkv, D)[:n].contiguous().cuda() for x in (c.kp, c.vp))
        wb.kv_store_paged(k, v, kp, vp, table, _ints([0]), cu_seqlens=_ints([0, n]), rows=_ints([b]))
    c.device()
    c.d[3:] = [kp, vp]
    c.dtable = table

    def check():
        (out, mag, lse, top), hk, hv = c.oracle()
        got = c.o32.cpu().double().numpy().reshape(out.shape)
        assert (np.abs(got - out) <= mag * 2.0 ** -15 * (top[..., None] + 1)).all()
        for b, n in enumerate(c.pos):
            for j, page in enumerate(table[b].tolist()[:n // ps + 1]):
                held = min(ps, n + 1 - j * ps)
                for dev, host in ((kp, hk), (vp, hv)):
                    assert np.array_equal(dev[page, :, :held].cpu().double().numpy(), host[c.table[b][j], :, :held])

    c.call(_ws(4, nkv))
    check()
    ws = torch.zeros(wb.kv_pages_workspace_bytes(2, n_pages), dtype=torch.uint8, device="cuda")
    wb.kv_pages_compact(table, refs, kp, vp, ws)
    n = len(up)
    assert refs[:n].tolist() == [1] * n and int(refs.sum()) == n
    assert sorted(p for p in table.flatten().tolist() if p >= 0) == list(range(n))
    c.o32.fill_(7.0)
    c.call(_ws(4, nkv))
    check()


# --------------------------------------------------------------------------- the store

@pytest.mark.parametrize("src,dst", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("nkv", [1, 2, 3, 4, 5, 7])
def test_store_of_several_tokens_a_warp(nkv, src, dst):
    """More than 16384 (token, head) pairs of fewer than 8 heads; sequences that end inside a warp's
    tokens, without a slot, and tokens behind the last; rows padded."""
    g = torch.Generator().manual_seed(nkv)
    lens = [1, 0, 7, 16400 // nkv, 3, 500, 64]
    start = [5, 3, 0, 2, -1, 40, 0]
    rows = [6, 5, 4, 3, 2, 1, 0]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    T, ps = cu[-1] + 5, 48
    max_pages = max(lens) // ps + 2
    n_pages = 7 * max_pages
    table = torch.randperm(n_pages, generator=g).view(7, max_pages).int()
    wide = torch.randn(T, nkv + 1, D, generator=g).to(DT[src]).cuda()
    k = wide[:, :nkv]
    v = (wide * 2)[:, 1:]
    kp = torch.full((n_pages, nkv, ps, D), 7.0, dtype=DT[dst], device="cuda")
    vp = kp.clone()
    rk, rv = kp.clone(), vp.clone()
    wb.kv_store_paged(k, v, kp, vp, table.cuda(), _ints(start), cu_seqlens=_ints(cu), rows=_ints(rows))
    for i, n in enumerate(lens):
        if start[i] < 0 or n == 0:
            continue
        slot = torch.arange(start[i], start[i] + n)
        page = table[rows[i]].long()[slot // ps].cuda()
        at = (slot % ps).cuda()
        rk[page, :, at] = k[cu[i]:cu[i + 1]].to(DT[dst])
        rv[page, :, at] = v[cu[i]:cu[i + 1]].to(DT[dst])
    assert torch.equal(kp, rk) and torch.equal(vp, rv)
