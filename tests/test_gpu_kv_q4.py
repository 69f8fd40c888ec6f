"""GPU parity of the 4-bit key-value rows: the store bit for bit against the
oracle's quantiser (its decisions in fp32 on both sides), the load bit for bit
against the values that the rows stand for, placement by sequence bounds, rows
and starts, and what is skipped or flagged."""
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


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _kv(T, nkv, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(T, nkv, D, generator=g) * torch.rand(D, generator=g) * 4 + 0.5
    v = torch.randn(T, nkv, D, generator=g)
    return k.to(dtype), v.to(dtype)


def _place(T, bounds, rows, start, n_rows, S):
    """(token, row, slot) of every token that has a place."""
    got = []
    for i in range(len(start)):
        a, b = (i, i + 1) if bounds is None else (bounds[i], bounds[i + 1])
        r = i if rows is None else rows[i]
        for t in range(a, b):
            slot = start[i] + t - a
            if start[i] >= 0 and 0 <= r < n_rows and slot < S and t < T:
                got.append((t, r, slot))
    return got


def _roundtrip(k, v, bounds, rows, start, n_rows, S, flag=0):
    T, nkv = k.shape[:2]
    kc = torch.full((n_rows, nkv, S, 80), 171, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    cu = None if bounds is None else _i32(bounds)
    rw = None if rows is None else _i32(rows)
    wb.kv_store_q4(k.cuda(), v.cuda(), kc, vc, _i32(start), cu_seqlens=cu, rows=rw)
    assert wb.device_error(reset=True) == flag
    place = _place(T, bounds, rows, start, n_rows, S)
    for c, x, keys in ((kc, k, True), (vc, v, False)):
        ref = np.full(c.shape, 171, np.uint8)
        q = sv.quantize_rows(x.float().numpy(), keys)
        for t, r, s in place:
            ref[r, :, s] = q[t]
        assert np.array_equal(c.cpu().numpy(), ref), "cached bytes"
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        kb = torch.full((T, nkv, D), 3.0, dtype=dt, device="cuda")
        vb = kb.clone()
        wb.kv_load_q4(kc, vc, _i32(start), kb, vb, cu_seqlens=cu, rows=rw)
        assert wb.device_error(reset=True) == flag
        for got, x, keys in ((kb, k, True), (vb, v, False)):
            ref = torch.full((T, nkv, D), 3.0, dtype=dt)
            val = torch.from_numpy(sv.dequantize_rows(sv.quantize_rows(x.float().numpy(), keys), keys))
            for t, r, s in place:
                ref[t] = val[t].to(dt)
            assert torch.equal(got.cpu(), ref), f"values in {dt}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,nkv,S", [(1, 1, 1), (1, 2, 7), (5, 3, 64), (16, 8, 33)])
def test_one_token_a_row(B, nkv, S, dtype):
    k, v = _kv(B, nkv, dtype, B + S)
    _roundtrip(k, v, None, None, [(7 * b) % S for b in range(B)], B, S)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,first", [([1], 0), ([33], 0), ([7, 0, 1, 64, 9], 0), ([5, 6], 3),
                                        ([0, 0, 130, 0], 0)])
def test_packed_prompts(lens, first, dtype):
    """Sequences to rows of their own in another order, behind what the rows
    hold; tokens before the first and behind the last are skipped."""
    n = len(lens)
    bounds = (first + np.concatenate([[0], np.cumsum(lens)])).tolist()
    k, v = _kv(bounds[-1] + 4, 2, dtype, sum(lens))
    rows = [(3 * i + 1) % (n + 2) if (n + 2) % 3 else n + 1 - i for i in range(n)]
    assert len(set(rows)) == n
    _roundtrip(k, v, bounds, rows, [(11 * i) % 20 for i in range(n)], n + 2, 200)


def test_skipped_and_flagged_places():
    k, v = _kv(30, 2, torch.float32, 1)
    b = [0, 10, 20, 30]
    _roundtrip(k, v, b, None, [-1, 0, -5], 3, 40)                  # rows without a sequence
    _roundtrip(k, v, b, None, [35, 0, 40], 3, 40, flag=2)          # past the last slot
    _roundtrip(k, v, b, [0, 3, -1], [0, 0, 0], 3, 40, flag=2)      # rows outside the cache
    _roundtrip(k, v, None, None, [2**31 - 1] + [0] * 29, 30, 4, flag=2)
    _roundtrip(k[:10], v[:10], [0, 10, 25], None, [0, 0], 3, 40)   # bounds past T


def test_special_values():
    k, v = _kv(12, 1, torch.float32, 2)
    k[0] = 0.0
    k[1] = 3.25
    k[2, 0, :32] = torch.tensor([1e-40, 0.0] * 16)     # steps below the smallest normal
    k[3, 0, 5] = float("nan")
    k[4, 0, 40] = float("inf")
    k[5, 0, 70] = float("-inf")
    k[6, 0, :64] = torch.tensor([3e38, -3e38] * 32)    # a range beyond fp32
    k[7, 0, ::2] = -0.0
    k[8] = 2.0 ** -120 * torch.arange(128)
    v[:9] = k[:9]
    _, sz = None, sv.quantize_rows(k.numpy(), True)
    kc = torch.zeros((12, 1, 1, 80), dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    st = _i32([0] * 12)
    wb.kv_store_q4(k.cuda(), v.cuda(), kc, vc, st)
    assert np.array_equal(kc.cpu().numpy()[:, :, 0], sz)
    assert np.array_equal(vc.cpu().numpy()[:, :, 0], sv.quantize_rows(v.numpy(), False))
    kb = torch.zeros((12, 1, D), device="cuda")
    vb = kb.clone()
    wb.kv_load_q4(kc, vc, st, kb, vb)
    assert np.array_equal(kb.cpu().numpy(), sv.dequantize_rows(sz, True), equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_codes_next_to_ties_and_of_every_size(dtype):
    """Groups whose values lie on, next to and between the ties of their own
    steps, at sizes from the subnormals up: the codes are those of the division."""
    r = np.random.default_rng(11)
    T = 3000
    top = 2.0 ** r.integers(*((-13, 15) if dtype == torch.float16 else (-133, 124)), (T, 1, 1))
    x = r.standard_normal((T, 4, 32)) * top
    n = r.integers(0, 30, (T, 4, 32)) / 2.0
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    on = lo + n * ((hi - lo) / 15)                    # a multiple of half a step from the least
    x = np.where(r.random(x.shape) < 0.7, on, x)
    s = torch.from_numpy(((hi - lo) / 15).astype(np.float32)).bfloat16().float().numpy()
    z = torch.from_numpy((lo + 8 * s).astype(np.float32)).bfloat16().float().numpy()
    tie = (z + (n - 8.5) * s).astype(np.float32)      # on the ties of the step as it is stored
    x = np.where(r.random(x.shape) < 0.4, tie, x)
    k = torch.from_numpy(x.reshape(T, 1, D)).float().to(dtype)
    kc = torch.zeros((T, 1, 1, 80), dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    wb.kv_store_q4(k.cuda(), k.cuda(), kc, vc, _i32([0] * T))
    torch.cuda.synchronize()
    for c, keys in ((kc, True), (vc, False)):
        ref = sv.quantize_rows(k.float().numpy(), keys)
        bad = (c.cpu().numpy()[:, :, 0] != ref).any(-1)
        assert not bad.any(), f"{bad.sum()} rows differ, first {np.argwhere(bad)[0]}"


def test_strided_rows_of_a_fused_projection():
    T, nkv = 19, 2
    k, v = _kv(T, nkv, torch.bfloat16, 4)
    fused = torch.full((T, 5 * D + 2 * nkv * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    w = fused.view(T, 5 + 2 * nkv, D)
    w[:, 5:5 + nkv], w[:, 5 + nkv:] = k.cuda(), v.cuda()
    kc = wb.new_kv_cache_q4(1, nkv, 32)
    vc = wb.new_kv_cache_q4(1, nkv, 32)
    wb.kv_store_q4(w[:, 5:5 + nkv], w[:, 5 + nkv:], kc, vc, _i32([0]), cu_seqlens=_i32([0, T]))
    torch.cuda.synchronize()
    ref = sv.quantize_rows(k.float().numpy(), True)
    assert np.array_equal(kc.cpu().numpy()[0].transpose(1, 0, 2)[:T], ref)
    ref = sv.quantize_rows(v.float().numpy(), False)
    assert np.array_equal(vc.cpu().numpy()[0].transpose(1, 0, 2)[:T], ref)


def test_places_past_four_gigabytes():
    """The last row of a cache of 4.4 GB: its offsets pass 32 bits."""
    S = 6_900_000
    kc = torch.zeros((2, 4, S, 80), dtype=torch.uint8, device="cuda")
    k, v = _kv(2, 4, torch.bfloat16, 5)
    wb.kv_store_q4(k.cuda(), v.cuda(), kc, torch.zeros_like(kc), _i32([S - 1, S - 1]))
    torch.cuda.synchronize()
    assert np.array_equal(kc[:, :, S - 1].cpu().numpy(), sv.quantize_rows(k.float().numpy(), True))
    assert int(kc[:, :, :S - 1].any())  == 0


def test_graph_replay_and_another_stream():
    """Starts and bounds are read when the graph runs."""
    k, v = _kv(6, 2, torch.float32, 6)
    dk, dv = k.cuda(), v.cuda()
    kc, vc = wb.new_kv_cache_q4(6, 2, 16), wb.new_kv_cache_q4(6, 2, 16)
    st = _i32([0] * 6)
    kb, vb = torch.zeros((6, 2, D), device="cuda"), torch.zeros((6, 2, D), device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    wb.kv_store_q4(dk, dv, kc, vc, st, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        wb.kv_store_q4(dk, dv, kc, vc, st)
        wb.kv_load_q4(kc, vc, st, kb, vb)
    for step in range(3):
        k, v = _kv(6, 2, torch.float32, 60 + step)
        dk.copy_(k), dv.copy_(v)
        st.fill_(step + 1)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(kc[:, :, step + 1].cpu().numpy(), sv.quantize_rows(k.numpy(), True))
        assert np.array_equal(
            vb.cpu().numpy(), sv.dequantize_rows(sv.quantize_rows(v.numpy(), False), False))


@pytest.mark.parametrize("low", [-2147483643, -2147483648])
def test_bounds_far_below_the_tokens(low):
    """The tokens' slots would lie far past the last one (their count passes 32
    bits): skipped and flagged."""
    k, v = _kv(10, 2, torch.bfloat16, 7)
    kc = torch.full((1, 2, 64, 80), 171, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    kb = torch.full((10, 2, D), 3.0, dtype=torch.bfloat16, device="cuda")
    vb = kb.clone()
    wb.kv_store_q4(k.cuda(), v.cuda(), kc, vc, _i32([0]), cu_seqlens=_i32([low, 10]))
    assert wb.device_error(reset=True) == 2
    wb.kv_load_q4(kc, vc, _i32([0]), kb, vb, cu_seqlens=_i32([low, 10]))
    assert wb.device_error(reset=True) == 2
    for c in (kc, vc):
        assert bool((c == 171).all())
    for x in (kb, vb):
        assert bool((x == 3.0).all())


def test_a_first_bound_before_the_tokens():
    """Sequence -2 .. 10: its token 0 is the third one, in slot start + 2."""
    k, v = _kv(10, 2, torch.bfloat16, 7)
    kc = torch.full((1, 2, 64, 80), 171, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    wb.kv_store_q4(k.cuda(), v.cuda(), kc, vc, _i32([4]), cu_seqlens=_i32([-2, 10]))
    assert wb.device_error(reset=True) == 0
    ref = np.full((1, 2, 64, 80), 171, np.uint8)
    ref[0, :, 6:16] = sv.quantize_rows(k.float().numpy(), True).transpose(1, 0, 2)
    assert np.array_equal(kc.cpu().numpy(), ref)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,first,behind", [
    ([700, 0, 1001, 3, 129, 1290, 1, 64, 900, 7], 5, 400),    # 4500 tokens of 4 heads
    ([4500], 0, 0), ([1] * 60 + [4000, 0, 0, 333], 107, 0),
])
def test_many_tokens_a_warp(lens, first, behind, dtype):
    """Above 16384 tokens and heads a warp takes 16 tokens, eight apart, and keeps a
    sequence's place between them: ends at every offset, sequences without a row,
    rows past the last slot, tokens of no sequence."""
    n, T = len(lens), first + sum(lens) + behind
    bounds = (first + np.concatenate([[0], np.cumsum(lens)])).tolist()
    k, v = _kv(T, 4, dtype, T)
    start = [(11 * i) % 20 for i in range(n)]
    rows = list(range(n))[::-1]
    _roundtrip(k, v, bounds, rows, start, n, 5000)
    if n > 4:
        start[0], start[4] = -1, 4950   # no sequence; 79 of 129 tokens past the end
        rows[8 if n == 10 else 2] = n   # a row outside the cache
        _roundtrip(k, v, bounds, rows, start, n, 5000, flag=2)


@pytest.mark.parametrize("T,nkv", [(16384, 1), (16385, 1), (4096, 4), (4097, 4), (2341, 7)])
def test_token_counts_around_the_change_of_form(T, nkv):
    k, v = _kv(T, nkv, torch.bfloat16, T)
    _roundtrip(k, v, [0, T // 3, T], None, [0, 9], 2, T)
    if T < 5000:
        _roundtrip(k, v, None, None, [t % 2 for t in range(T)], T, 2)
