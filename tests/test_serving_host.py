"""The serving entry points without a GPU: their refusals (validated before
anything is launched), workspace sizes, the binding's checks of tensors, and
the oracle of the 4-bit row against its own definition."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import serving as sv
from weight_streaming_gemv_bf16_gb300 import binding as wb

A = 0x7F0000000000  # fake device addresses: nothing touches them
MIS = A + 8


@pytest.fixture(scope="module")
def lib():
    from weight_streaming_gemv_bf16_gb300 import _build
    _build.build()
    return wb.load()


PROMPT = dict(q=A, k=A, v=A, dtype=1, cu=A, out=A, lse=None, T=64, n=1, nh=4, nkv=2, d=128,
              qs=512, ks=256, vs=256)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(cu=None), -1),
    (dict(out=None), -1), (dict(dtype=0), -1), (dict(dtype=3), -1),
    (dict(T=0), -3), (dict(n=0), -3), (dict(nh=0), -3), (dict(nkv=0), -3), (dict(nh=3), -3),
    (dict(d=64), -3), (dict(qs=508), -3), (dict(qs=504), -3), (dict(ks=248), -3),
    (dict(vs=260), -3), (dict(qs=0), -3),
    (dict(q=MIS), -2), (dict(k=MIS), -2), (dict(v=MIS), -2), (dict(out=MIS), -2),
])
def test_prompt_attention_refusals(lib, change, status):
    a = {**PROMPT, **change}
    assert lib.ws_prompt_attention(a["q"], a["k"], a["v"], a["dtype"], a["cu"], a["out"],
                                   a["lse"], a["T"], a["n"], a["nh"], a["nkv"], a["d"], a["qs"],
                                   a["ks"], a["vs"], None) == status
    assert lib.ws_last_error()


STORE = dict(k=A, v=A, dtype=1, cu=A, rows=None, start=A, kc=A, vc=A, T=64, n=2, n_rows=2, nkv=2,
             d=128, S=100, ks=256, vs=256)


@pytest.mark.parametrize("change,status", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(start=None), -1), (dict(kc=None), -1),
    (dict(vc=None), -1), (dict(dtype=7), -1), (dict(T=0), -3), (dict(n=0), -3),
    (dict(n_rows=0), -3), (dict(nkv=0), -3), (dict(nkv=65536), -3), (dict(S=0), -3),
    (dict(d=64), -3), (dict(cu=None), -3), (dict(T=(1 << 30) + 1), -3), (dict(kc=MIS), -2), (dict(vc=MIS), -2),
    (dict(k=MIS), -2), (dict(v=MIS), -2),
])
def test_kv_store_and_load_refusals(lib, change, status):
    a = {**STORE, **change}
    assert lib.ws_kv_store_q4(a["k"], a["v"], a["dtype"], a["cu"], a["rows"], a["start"], a["kc"],
                              a["vc"], a["T"], a["n"], a["n_rows"], a["nkv"], a["d"], a["S"],
                              a["ks"], a["vs"], None) == status
    assert lib.ws_kv_load_q4(a["kc"], a["vc"], a["cu"], a["rows"], a["start"], a["k"], a["v"],
                             a["dtype"], a["T"], a["n"], a["n_rows"], a["nkv"], a["d"], a["S"],
                             None) == status


@pytest.mark.parametrize("ks,vs", [(248, 256), (256, 248), (260, 256), (256, 0)])
def test_kv_store_stride_refusals(lib, ks, vs):
    a = STORE
    assert lib.ws_kv_store_q4(A, A, 1, A, None, A, A, A, 64, 2, 2, 2, 128, 100, ks, vs, None) == -3


def test_kv_row_bytes(lib):
    assert wb.kv_q4_row_bytes(128) == sv.ROW == 80
    assert wb.kv_q4_row_bytes(64) == 0


DECODE = dict(q=A, kn=A, vn=A, kc=A, vc=A, pos=A, o32=A, o16=None, B=2, nh=4, nkv=2, d=128, S=77,
              ws=A, wsb=1 << 30)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), -1), (dict(kn=None), -1), (dict(vn=None), -1), (dict(kc=None), -1),
    (dict(vc=None), -1), (dict(pos=None), -1), (dict(o32=None), -1), (dict(ws=None), -1),
    (dict(wsb=16), -1), (dict(B=0), -3), (dict(B=1025), -3), (dict(nh=3), -3), (dict(nh=0), -3),
    (dict(nkv=0), -3), (dict(nh=18), -3), (dict(d=64), -3), (dict(S=0), -3),
    (dict(q=MIS), -2), (dict(kn=MIS), -2), (dict(vn=MIS), -2), (dict(kc=MIS), -2),
    (dict(vc=MIS), -2), (dict(o32=MIS), -2), (dict(o16=MIS), -2), (dict(ws=MIS), -2),
])
def test_decode_attention_q4_refusals(lib, change, status):
    a = {**DECODE, **change}
    assert lib.ws_decode_attention_q4(a["q"], a["kn"], a["vn"], a["kc"], a["vc"], a["pos"],
                                      a["o32"], a["o16"], a["B"], a["nh"], a["nkv"], a["d"],
                                      a["S"], a["ws"], a["wsb"], None) == status


def test_decode_attention_q4_workspace(lib):
    assert wb.attention_q4_workspace_bytes(1, 12, 2, 1) > 0
    assert wb.attention_q4_workspace_bytes(16, 32, 8, 16384) > 0
    for bad in ((0, 12, 2, 64), (1, 12, 5, 64), (1, 18, 2, 64), (1, 12, 2, 0), (1025, 2, 2, 8)):
        assert wb.attention_q4_workspace_bytes(*bad) == 0


LOGP = dict(x=A, dtype=0, ld=100, tgt=A, lp=A, ent=A, ti=A, tl=A, rows=2, V=100, k=5, ws=A,
            wsb=1 << 30)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), -1), (dict(ws=None), -1), (dict(tgt=None), -1), (dict(lp=None), -1),
    (dict(ti=None, tl=None), -1), (dict(tgt=None, lp=None, ent=None, k=0), -1),
    (dict(dtype=9), -1), (dict(wsb=16), -1), (dict(rows=0), -3), (dict(V=0), -3),
    (dict(ld=99), -3), (dict(V=(1 << 28) + 1, ld=1 << 30), -3), (dict(k=-1), -3), (dict(k=33), -3), (dict(V=4, k=5), -3),
    (dict(x=A + 2), -2), (dict(dtype=1, x=A + 1), -2), (dict(ws=MIS), -2),
])
def test_token_logprobs_refusals(lib, change, status):
    a = {**LOGP, **change}
    assert lib.ws_token_logprobs(a["x"], a["dtype"], a["ld"], a["tgt"], a["lp"], a["ent"],
                                 a["ti"], a["tl"], a["rows"], a["V"], a["k"], a["ws"], a["wsb"],
                                 None) == status


def test_logprobs_workspace(lib):
    assert wb.logprobs_workspace_bytes(1, 1, 0) > 0
    assert wb.logprobs_workspace_bytes(2048, 151936, 32) > 0
    for bad in ((0, 5, 0), (1, 0, 0), (1, 5, 6), (1, 50, 33), (1, 50, -1)):
        assert wb.logprobs_workspace_bytes(*bad) == 0


def test_binding_refuses_tensors_off_the_current_device_or_misshapen(lib, monkeypatch):
    """The binding looks at shapes, types, strides and devices before the call
    crosses the ABI.  Tensors on the CPU report device -1: taken as the current
    one, they reach the checks behind that of the device."""
    bf = torch.bfloat16
    q, kv = torch.zeros(8, 4, 128, dtype=bf), torch.zeros(8, 2, 128, dtype=bf)
    cu, out = torch.zeros(2, dtype=torch.int32), torch.zeros(8, 512, dtype=bf)
    kc = torch.zeros(2, 2, 10, 80, dtype=torch.uint8)
    st = torch.zeros(2, dtype=torch.int32)
    f, n = torch.zeros(2, 512), torch.zeros(2, 256)
    monkeypatch.setattr(wb, "_here", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        wb.prompt_attention(q, kv, kv, cu, out)
    with pytest.raises(ValueError, match="current device"):
        wb.kv_store_q4(kv, kv, kc, kc, st, cu_seqlens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="current device"):
        wb.kv_load_q4(kc, kc, st, kv, kv)
    with pytest.raises(ValueError, match="current device"):
        wb.decode_attention_q4(f, n, n, kc, kc, st, kc, out_f32=f)
    with pytest.raises(ValueError, match="current device"):
        wb.token_logprobs(f, kc, entropy=torch.zeros(2))
    monkeypatch.setattr(wb, "_here", lambda: -1)
    with pytest.raises(ValueError, match="heads must be contiguous"):
        wb.prompt_attention(q.transpose(0, 1), kv, kv, cu, out)
    with pytest.raises(ValueError, match="expected .tokens, heads"):
        wb.prompt_attention(out, kv, kv, cu, out)
    with pytest.raises(ValueError, match="disagree in shape"):
        wb.prompt_attention(q, kv[:7], kv, cu, out)
    with pytest.raises(ValueError, match="disagree in type"):
        wb.prompt_attention(q, kv.half(), kv, cu, out)
    with pytest.raises(ValueError, match="out"):
        wb.prompt_attention(q, kv, kv, cu, out[:, :256])
    with pytest.raises(ValueError, match="cu_seqlens"):
        wb.prompt_attention(q, kv, kv, cu.long(), out)
    with pytest.raises(ValueError, match="lse"):
        wb.prompt_attention(q, kv, kv, cu, out, lse=torch.zeros(4, 8))
    with pytest.raises(ValueError, match="cu_seqlens"):
        wb.kv_store_q4(kv, kv, kc, kc, st, cu_seqlens=cu)
    with pytest.raises(ValueError, match="v_cache"):
        wb.kv_store_q4(kv, kv, kc, kc[:1], st)
    with pytest.raises(ValueError, match="disagree"):
        wb.kv_store_q4(kv, kv.half(), kc, kc, st)
    with pytest.raises(ValueError, match="k_cache"):
        wb.kv_store_q4(q, q, kc, kc, st)
    with pytest.raises(ValueError, match="contiguous"):
        wb.kv_load_q4(kc, kc, st, kv[::2], kv[::2])
    with pytest.raises(ValueError, match="pos"):
        wb.decode_attention_q4(f, n, n, kc, kc, st.long(), kc, out_f32=f)
    with pytest.raises(ValueError, match="k_new"):
        wb.decode_attention_q4(f, f, n, kc, kc, st, kc, out_f32=f)
    with pytest.raises(ValueError, match="out_bf16"):
        wb.decode_attention_q4(f, n, n, kc, kc, st, kc, out_bf16=f)
    with pytest.raises(ValueError, match="contiguous"):
        wb.token_logprobs(f.t(), kc)
    with pytest.raises(ValueError, match="top_logprob"):
        wb.token_logprobs(f, kc, top_idx=torch.zeros(2, 4, dtype=torch.int32),
                          top_logprob=torch.zeros(2, 5))


def test_binding_refuses_a_workspace_in_pieces(monkeypatch):
    """The size that crosses the ABI is that of one piece: a view whose bytes do
    not lie behind one another (or are one byte many times) is refused."""
    monkeypatch.setattr(wb, "_here", lambda: -1)
    f, st = torch.zeros(2, 512), torch.zeros(2, dtype=torch.int32)
    n, kc = torch.zeros(2, 256), torch.zeros(2, 2, 10, 80, dtype=torch.uint8)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 12)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            wb.decode_attention_q4(f, n, n, kc, kc, st, ws, out_f32=f)
        with pytest.raises(ValueError, match="workspace"):
            wb.token_logprobs(f, ws, entropy=torch.zeros(2))


@pytest.mark.parametrize("keys", [True, False])
def test_oracle_rows_are_within_half_a_step(keys):
    """Each value is off by at most half a step, the rounding of the zero (a
    half unit of bf16, eps / 2 = 2^-8 of it) and what the range loses at its
    ends through both roundings: 7.5 steps are at most 2^-8 of a step short
    each, and the zero's own error."""
    rng = np.random.default_rng(3)
    x = (rng.normal(size=(200, 128)) * rng.uniform(0.01, 30, (200, 1)) + 2).astype(np.float32)
    rows = sv.quantize_rows(x, keys)
    assert rows.shape == (200, 80) and rows.dtype == np.uint8
    c, s, z = sv.row_values(rows, keys)
    assert c.min() >= -8 and c.max() <= 7
    err = np.abs(sv.dequantize_rows(rows, keys) - x)
    assert (err <= s * (0.5 + 8 * 2.0 ** -8) + 2.0 ** -8 * np.abs(z) + 1e-6 * np.abs(x)).all()


def test_oracle_rows_of_special_groups():
    x = np.ones((3, 128), np.float32)
    x[0, :32] = 2.5            # a constant group: s = 0
    x[1, 40] = np.nan
    x[2, 100] = -np.inf
    v = sv.dequantize_rows(sv.quantize_rows(x, True), True)
    assert (v[0] == x[0]).all()
    assert np.isnan(v[1, 32:64]).all() and (v[1, :32] == 1).all() and (v[1, 64:] == 1).all()
    assert np.isnan(v[2, 96:]).all() and (v[2, :96] == 1).all()


def test_oracle_logprobs_by_hand():
    x = np.array([[0.0, np.log(3.0), -np.inf, np.log(3.0)], [np.nan, 1, 2, 3]])
    lp, ent, top = sv.token_logprobs(x, 3)
    assert np.allclose(np.exp(lp[0]), [1 / 7, 3 / 7, 0, 3 / 7])
    assert np.isclose(ent[0], -(np.log(1 / 7) / 7 + 6 / 7 * np.log(3 / 7)))
    assert top.tolist() == [[1, 3, 0], [3, 2, 1]]
    assert np.isnan(ent[1]) and np.isnan(lp[1]).all()


def _places_by_definition(cu, rows, start, T, n_rows, S):
    """Each token's row * S + slot, -1 skipped, -2 flagged, in Python's integers."""
    got = [-1] * T
    for i, s0 in enumerate(start):
        lo, hi = (i, i + 1) if cu is None else (cu[i], cu[i + 1])
        r = i if rows is None else rows[i]
        for t in range(max(lo, 0), min(hi, T)):
            if s0 >= 0:
                ok = 0 <= r < n_rows and s0 + t - lo < S
                got[t] = r * S + s0 + t - lo if ok else -2
    return got


@pytest.mark.parametrize("cu,rows,start,S", [
    ([0, 3, 3, 9], None, [0, 5, 4], 16),
    ([2, 9], [1], [0], 5),                              # the last two have no slot
    ([0, 4, 10], [7, -1], [0, 0], 16),                  # rows outside the cache
    ([0, 4, 10], None, [-1, 2**31 - 1], 16),
    (None, None, [0] * 5 + [15, 16, -1, -2**31, 2**31 - 1], 16),
    ([-2147483643, 10], None, [0], 64),                 # hi - lo passes 32 bits
    ([-2147483648, 10], None, [0], 64),
    ([-2147483648, 2147483647], None, [0], 64),
    ([-2147483648, 2147483647], [1], [2147483647], 2147483647),
    ([-5, 2147483647], [1], [3], 64),
    ([-3, 6, 2147483647], [1, 0], [2147483640, 0], 2147483647),
])
def test_kv_places_whatever_the_bounds(lib, cu, rows, start, S):
    """The kernels' placement on the CPU: no token gets a slot outside its row,
    however far the bounds lie outside the tokens."""
    T, n_rows = 10, 10
    got = wb.debug_kv_places(cu, rows, start, T, n_rows, S)
    assert got == _places_by_definition(cu, rows, start, T, n_rows, S)


def test_kv_places_of_random_bounds_that_rise(lib):
    rng = np.random.default_rng(5)
    edges = [-2**31, -2**31 + 7, -2**30, -100, -1, 0, 1, 5, 17, 40, 41, 2**30, 2**31 - 1]
    for _ in range(400):
        n = int(rng.integers(1, 6))
        cu = sorted(int(x) for x in rng.choice(edges, n + 1))
        rows = [int(x) for x in rng.integers(-1, 4, n)] if rng.random() < 0.7 else None
        start = [int(x) for x in rng.choice([-1, 0, 3, 30, 2**31 - 1], n)]
        S = int(rng.choice([1, 8, 33, 2**31 - 1]))
        got = wb.debug_kv_places(cu, rows, start, 40, 3, S)
        assert got == _places_by_definition(cu, rows, start, 40, 3, S), (cu, rows, start, S)


def test_kv_places_of_bounds_in_any_order_stay_in_the_cache(lib):
    """Bounds that fall: tokens may go with another sequence, never past a row."""
    rng = np.random.default_rng(6)
    for _ in range(400):
        n, S = int(rng.integers(1, 6)), int(rng.choice([1, 8, 33]))
        cu = [int(x) for x in rng.choice([-2**31, -9, 0, 3, 12, 40, 90, 2**31 - 1], n + 1)]
        start = [int(x) for x in rng.choice([-1, 0, 3, 30], n)]
        got = wb.debug_kv_places(cu, None, start, 40, 3, S)
        assert all(-2 <= p < 3 * S for p in got), (cu, start, S)
