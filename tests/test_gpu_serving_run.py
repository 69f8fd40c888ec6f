"""The serving operators as one program would run them: packed prompts through
the causal attention, their keys and values into the 4-bit cache, decode steps
that append and attend, and the answers' log-probabilities; each stage against
the oracle on the GPU's own previous stage."""
import numpy as np
import pytest
import torch

from oracle import serving as sv
from weight_streaming_gemv_bf16_gb300 import binding as wb

pytestmark = pytest.mark.gpu
D = 128


def test_prompts_cache_decode_and_answers():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    wb.device_error(reset=True)
    nh, nkv, S, V, lens = 12, 2, 160, 1000, [70, 129, 1]
    rows = [2, 0, 3]                     # cache rows that the prompts take; row 1 has no sequence
    T = sum(lens)
    g = torch.Generator().manual_seed(0)
    qkv = torch.randn(T, nh + 2 * nkv, D, generator=g).bfloat16().cuda()
    q, k, v = qkv[:, :nh], qkv[:, nh:nh + nkv], qkv[:, nh + nkv:]
    bounds = np.concatenate([[0], np.cumsum(lens)]).tolist()
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    out = torch.zeros((T, nh * D), dtype=torch.bfloat16, device="cuda")
    kc, vc = wb.new_kv_cache_q4(4, nkv, S), wb.new_kv_cache_q4(4, nkv, S)
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    rw = torch.tensor(rows, dtype=torch.int32, device="cuda")
    wb.prompt_attention(q, k, v, cu, out)
    wb.kv_store_q4(k, v, kc, vc, zero, cu_seqlens=cu, rows=rw)
    hq, hk, hv = (x.double().cpu().numpy() for x in (q, k, v))
    ref, mag, _ = sv.prompt_attention(hq, hk, hv, bounds)
    err = np.abs(out.double().cpu().numpy().reshape(T, nh, D) - ref)
    assert (err <= 2.0 ** -8 * (mag + np.abs(ref)) * 1.01 + 1e-6).all()
    for i, (a, b) in enumerate(zip(bounds, bounds[1:])):
        for c, x, keys in ((kc, k, True), (vc, v, False)):
            want = sv.quantize_rows(x[a:b].float().cpu().numpy(), keys)
            assert np.array_equal(c[rows[i], :, :b - a].cpu().numpy().transpose(1, 0, 2), want)

    pos = np.full(4, -1, np.int32)
    pos[rows] = lens
    dpos = torch.tensor(pos, device="cuda")
    ws = torch.zeros(wb.attention_q4_workspace_bytes(4, nh, nkv, S), dtype=torch.uint8, device="cuda")
    lws = torch.zeros(wb.logprobs_workspace_bytes(4, V, 3), dtype=torch.uint8, device="cuda")
    head = (torch.randn(V, nh * D, generator=g) * 0.02).cuda()
    o32 = torch.zeros((4, nh * D), device="cuda")
    lp, ent = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    top = torch.zeros((4, 3), dtype=torch.int32, device="cuda")
    tlp = torch.zeros((4, 3), device="cuda")
    for step in range(3):
        dq = torch.randn(4, nh * D, generator=g).cuda()
        kn, vn = (torch.randn(4, nkv * D, generator=g).cuda() for _ in range(2))
        before = kc.cpu().numpy(), vc.cpu().numpy()
        wb.decode_attention_q4(dq, kn, vn, kc, vc, dpos, ws, out_f32=o32)
        ref, mag, big, rk, rv = sv.decode_attention_q4(
            dq.cpu().numpy(), kn.cpu().numpy(), vn.cpu().numpy(), *before, pos)
        live = ~np.isnan(ref)
        err = np.abs(o32.cpu().numpy() - ref)
        assert (err[live] <= (mag * 2.0 ** -15 * (np.repeat(big, D, 1) + 1))[live]).all()
        assert np.array_equal(kc.cpu().numpy(), rk) and np.array_equal(vc.cpu().numpy(), rv)
        logits = o32 @ head.t()
        idx = torch.zeros(4, dtype=torch.int32, device="cuda")
        aws = wb.new_workspace(wb.OP_ARGMAX_ROWS, 4, V, 1)
        wb.argmax_rows(logits, idx, aws)
        target = torch.where(dpos >= 0, idx, torch.full_like(idx, -1))
        wb.token_logprobs(logits, lws, targets=target, logprob=lp, entropy=ent, top_idx=top,
                          top_logprob=tlp)
        torch.cuda.synchronize()
        assert torch.equal(top[:, 0], idx)  # the first alternative is the argmax
        on = dpos >= 0
        assert torch.equal(lp[on], tlp[on, 0]) and lp[~on].abs().max() == 0
        rlp, rent, rtop = sv.token_logprobs(logits.cpu().numpy(), 3)
        assert np.array_equal(top.cpu().numpy(), rtop)
        assert np.abs(ent.cpu().numpy() - rent).max() <= 1e-4
        dpos += (dpos >= 0).int()
        pos = dpos.cpu().numpy()
    assert wb.device_error(reset=True) == 0


def test_calls_that_feed_one_another():
    """Each call reads what the one before it wrote, with nothing in between but
    the stream's order; the same calls with a synchronisation after each give
    the same bits."""
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    g = torch.Generator().manual_seed(3)
    T, nh, nkv, S, V = 300, 4, 2, 400, 5000
    q0 = torch.randn(T, nh, D, generator=g).bfloat16().cuda()
    kv = torch.randn(T, 2 * nkv, D, generator=g).bfloat16().cuda()
    cu = torch.tensor([0, 170, 300], dtype=torch.int32, device="cuda")
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    dec = torch.randn(2, nh * D, generator=g).cuda()
    new = torch.randn(2, nkv * D, generator=g).cuda()
    head = torch.randn(V, nh * D, generator=g).cuda()
    lws = torch.zeros(wb.logprobs_workspace_bytes(2, V, 4), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(wb.attention_q4_workspace_bytes(2, nh, nkv, S), dtype=torch.uint8, device="cuda")

    def program(sync):
        done = torch.cuda.synchronize if sync else (lambda: None)
        a, b = torch.zeros_like(q0).view(T, nh * D), torch.zeros_like(q0).view(T, nh * D)
        kc, vc = wb.new_kv_cache_q4(2, nkv, S), wb.new_kv_cache_q4(2, nkv, S)
        kb, vb = torch.zeros(T, nkv, D, device="cuda").bfloat16(), torch.zeros(T, nkv, D, device="cuda").bfloat16()
        q, k, v = q0, kv[:, :nkv], kv[:, nkv:]
        o, prev = torch.zeros_like(dec), dec
        ent = torch.zeros(2, device="cuda")
        top = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
        pos = torch.tensor([170, 130], dtype=torch.int32, device="cuda")
        seen = []
        for i in range(6):
            out = a if i % 2 == 0 else b
            wb.prompt_attention(q, k, v, cu, out); done()
            wb.kv_store_q4(k, out.view(T, nh, D)[:, :nkv], kc, vc, start, cu_seqlens=cu); done()
            wb.kv_load_q4(kc, vc, start, kb, vb, cu_seqlens=cu); done()
            q, k, v = out.view(T, nh, D), kb, vb
            wb.decode_attention_q4(prev, new, new, kc, vc, pos, ws, out_f32=o); done()
            logits = o @ head.t(); done()
            wb.token_logprobs(logits, lws, entropy=ent, top_idx=top); done()
            prev = o.clone() * ent[:, None].clamp(0.5, 2.0); done()
            seen += [out.clone(), kb.clone(), o.clone(), ent.clone(), top.clone()]
            done()
        torch.cuda.synchronize()
        return seen

    once = program(True)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(once, program(False)))
    assert wb.device_error(reset=True) == 0
