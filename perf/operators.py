"""The serving operators next to the decode chain, as measurable cases: causal
attention over packed prompts, the 4-bit key-value cache (rows stored, rows
read back, decode attention over it) and the log-probabilities of given tokens.

``own`` False: each operator in elementary torch operations, fp32 inside (the
plain form).  ``own`` True: the library's calls.  Both take what ``prepare``
gives.  Head dimension 128; groups of 32 dimensions carry a bf16 scale and
zero; a cached row is 80 bytes.
"""
import math

import torch

own = False

D = 128        # head dimension
GROUP = 32     # dimensions that share a scale and a zero
NG = D // GROUP
ROW = D // 2 + 4 * NG  # bytes of a cached row

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a chat's first short question: 12 query heads over 2 key-value heads, latency only
        {"name": "prompt_short", "op": "prompt", "lens": "37", "tail": 0, "nh": 12, "nkv": 2,
         "dtype": "bf16", "lse": False},
        # a serving step's waiting prompts, packed, one of them empty, padded to a bucket's length
        {"name": "prompt_packed", "op": "prompt", "lens": "700,1,0,129,1025,64,333", "tail": 51,
         "nh": 12, "nkv": 2, "dtype": "bf16", "lse": False},
        # one key-value head per query head, fp16, with the log-sum-exp kept
        {"name": "prompt_heads_f16", "op": "prompt", "lens": "1500,517", "tail": 0, "nh": 16,
         "nkv": 16, "dtype": "f16", "lse": True},
        # a long document
        {"name": "prompt_long", "op": "prompt", "lens": "8192", "tail": 0, "nh": 32, "nkv": 8,
         "dtype": "bf16", "lse": False},
        # one new token for each of 16 running sequences
        {"name": "store_step", "op": "store", "lens": "", "rows": 16, "nkv": 2, "s_max": 1024,
         "dtype": "f32"},
        # packed prompts of many users written behind what their cache rows hold
        {"name": "store_prompts", "op": "store", "lens": "16000,8191,20003,1,3000,9000", "rows": 8,
         "nkv": 8, "s_max": 24576, "dtype": "bf16"},
        # one user's decode step
        {"name": "decode_one", "op": "decode", "B": 1, "nh": 12, "nkv": 2, "s_max": 1024,
         "longest": 1000},
        # a ragged batch at medium lengths, a key-value head for each query head
        {"name": "decode_ragged", "op": "decode", "B": 13, "nh": 8, "nkv": 8, "s_max": 4099,
         "longest": 4099},
        # a full batch of long contexts
        {"name": "decode_long", "op": "decode", "B": 16, "nh": 32, "nkv": 8, "s_max": 16384,
         "longest": 16384},
        # one answer token's log-probability with 20 alternatives, odd vocabulary
        {"name": "logprobs_one", "op": "logprobs", "rows": 1, "V": 50257, "ld": 50257, "k": 20,
         "dtype": "f32", "banned": 0.0},
        # a decode step's answers over the LM head's fp32 logits, some tokens ruled out
        {"name": "logprobs_step", "op": "logprobs", "rows": 16, "V": 151936, "ld": 151936, "k": 5,
         "dtype": "f32", "banned": 0.01},
        # scoring a long prompt: bf16 logits in rows padded to a wider matrix
        {"name": "logprobs_prompt", "op": "logprobs", "rows": 2048, "V": 151665, "ld": 151936,
         "k": 20, "dtype": "bf16", "banned": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "store", "decode", "logprobs"])
    if op == "prompt":
        nkv = rng.choice([1, 2, 4, 8])
        nh = nkv * rng.choice([1, 2, 3, 4, 6, 7, 8])
        n = _log_int(rng, 1, 24)
        # scores of all heads and sequences: no more than the long document's
        longest = int(min(8192, math.sqrt(32 * 8192 * 8192 / (n * nh))))
        lens = [rng.choice([0, 1, longest])] if rng.random() < 0.1 and n > 1 else []
        lens += [_log_int(rng, 1, longest) for _ in range(n - len(lens))]
        return {"op": op, "lens": ",".join(map(str, lens)), "tail": rng.choice([0, 0, 1, 100]),
                "nh": nh, "nkv": nkv, "dtype": rng.choice(["bf16", "f16"]),
                "lse": rng.random() < 0.5}
    if op == "store":
        nkv = rng.choice([1, 2, 4, 8])
        s_max = _log_int(rng, 64, 24576)
        n = _log_int(rng, 1, 16)
        rows = n + rng.randrange(3)
        if rng.random() < 0.3:
            return {"op": op, "lens": "", "rows": rows, "nkv": nkv, "s_max": s_max,
                    "dtype": rng.choice(["f32", "bf16", "f16"])}
        top = min(s_max, 56000 // n)
        lens = [_log_int(rng, 1, max(1, top)) for _ in range(n)]
        return {"op": op, "lens": ",".join(map(str, lens)), "rows": rows, "nkv": nkv,
                "s_max": s_max, "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op == "decode":
        nkv = rng.choice([1, 2, 4, 8])
        nh = nkv * rng.randint(1, 8)
        B = _log_int(rng, 1, 16)
        s_max = _log_int(rng, 1, min(32768, 16 * 8 * 16384 // (B * nkv)))
        return {"op": op, "B": B, "nh": nh, "nkv": nkv, "s_max": s_max,
                "longest": rng.choice([s_max, rng.randint(1, s_max)])}
    V = _log_int(rng, 32, 200000)
    pad = rng.choice([0, 0, 1, 64])
    dtype = rng.choice(["f32", "bf16", "f16"])
    most = 2048 * 151936 // (2 if dtype == "f32" else 1)
    return {"op": op, "rows": _log_int(rng, 1, max(1, min(4096, most // (V + pad)))), "V": V,
            "ld": V + pad, "k": rng.choice([0, 1, 5, 20, 32]), "dtype": dtype,
            "banned": rng.choice([0.0, 0.0, 0.05])}


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if case["lens"] else []


def _positions(case):
    """Slot of each row's new token, spread from the longest down to the shortest."""
    B, n = case["B"], case["longest"]
    return [max(0, n - 1 - (b * n) // (2 * B)) for b in range(B)]


def _starts(case, lens):
    """Slots that the rows hold already, at most what leaves room for the new ones."""
    return [((i * 37) % 101) % (case["s_max"] - n + 1) for i, n in enumerate(lens)]


# --------------------------------------------------------------------------- the 4-bit rows

def _quantize(x):
    """fp32 [..., 128] -> codes [..., 4, 32] (0..15), bf16 scale and zero [..., 4]."""
    g = x.float().unflatten(-1, (NG, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((hi - lo) / torch.full_like(hi, 15.0)).bfloat16()  # a true division
    s = torch.where(s.float() < 2.0 ** -126, torch.zeros_like(s), s)
    z = (lo + 8.0 * s.float()).bfloat16()
    sf, zf = s.float()[..., None], z.float()[..., None]
    q = torch.round((g - zf) / torch.where(sf == 0, torch.ones_like(sf), sf)) + 8.0
    q = torch.where(sf == 0, torch.full_like(q, 8.0), q.clamp(0.0, 15.0))
    return q.to(torch.uint8), s, z


def _pack(x, keys):
    """fp32 [..., 128] -> cached rows uint8 [..., 80].  Keys: 32-bit word 4t + g
    holds dimensions 32g + 8t .. + 7; values: 16-bit unit 4r + g holds
    dimensions 32g + 4r .. + 3; nibbles in order, then (scale, zero) per group."""
    q, s, z = _quantize(x)
    per = 8 if keys else 4
    n = q.unflatten(-1, (GROUP // per, per)).transpose(-3, -2).flatten(-3)
    n = n.unflatten(-1, (D // 2, 2))
    codes = n[..., 0] | (n[..., 1] << 4)
    sz = torch.stack([s, z], -1).contiguous().view(torch.uint8).flatten(-2)
    return torch.cat([codes, sz], -1)


def _unpack(rows, keys):
    """Cached rows uint8 [..., 80] -> the fp32 values they stand for [..., 128]."""
    per = 8 if keys else 4
    c = rows[..., :D // 2]
    n = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    n = n.unflatten(-1, (GROUP // per, NG, per)).transpose(-3, -2).flatten(-2)  # [..., 4, 32]
    sz = rows[..., D // 2:].contiguous().view(torch.bfloat16).float().unflatten(-1, (NG, 2))
    return (sz[..., :1] * (n.float() - 8.0) + sz[..., 1:]).flatten(-2)


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)


def _keys_values(shape, gen, dtype=torch.float32):
    """Keys with a few strong channels and an offset, as a projection gives them; values normal."""
    k = torch.randn(shape, generator=gen, device="cuda")
    chan = torch.randn(D, generator=gen, device="cuda")
    k = k * (1.0 + 3.0 * (chan > 1.6)) * 0.7 + 0.5 * chan
    v = torch.randn(shape, generator=gen, device="cuda")
    return k.to(dtype), v.to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "prompt":
        lens = _lens(case)
        T = sum(lens) + case["tail"]
        nh, nkv, dt = case["nh"], case["nkv"], DTYPES[case["dtype"]]
        # the rows of one fused projection; those behind the last sequence hold anything
        qkv = torch.empty((T, nh + 2 * nkv, D), dtype=dt, device="cuda")
        qkv[:, :nh] = torch.randn((T, nh, D), generator=g, device="cuda").to(dt)
        k, v = _keys_values((T, nkv, D), g, dt)
        qkv[:, nh:nh + nkv] = k
        qkv[:, nh + nkv:] = v
        qkv[sum(lens):] = float("nan")
        st["q"], st["k"], st["v"] = qkv[:, :nh], qkv[:, nh:nh + nkv], qkv[:, nh + nkv:]
        st["ends"] = [sum(lens[:i]) for i in range(len(lens) + 1)]
        st["cu"] = _ints(st["ends"])
        st["out"] = torch.zeros((T, nh * D), dtype=dt, device="cuda")
        st["lse_out"] = torch.zeros((T, nh), device="cuda") if case["lse"] else None
    elif case["op"] == "store":
        lens = _lens(case)
        nkv, rows, dt = case["nkv"], case["rows"], DTYPES[case["dtype"]]
        one = not lens
        n = rows if one else len(lens)
        T = n if one else sum(lens)
        st["k"], st["v"] = _keys_values((T, nkv, D), g, dt)
        starts = _starts(case, [1] * n if one else lens)
        st["start"] = _ints(starts)
        st["cu"] = None if one else _ints([sum(lens[:i]) for i in range(n + 1)])
        # the sequences take the cache's rows from the last one down
        st["cache_rows"] = None if one else _ints([rows - 1 - i for i in range(n)])
        shape = (rows, nkv, case["s_max"], ROW)
        st["k_cache"] = torch.full(shape, 255, dtype=torch.uint8, device="cuda")
        st["v_cache"] = torch.full(shape, 255, dtype=torch.uint8, device="cuda")
        back = torch.float32 if dt == torch.float32 else dt
        st["k_back"] = torch.zeros((T, nkv, D), dtype=back, device="cuda")
        st["v_back"] = torch.zeros((T, nkv, D), dtype=back, device="cuda")
    elif case["op"] == "decode":
        B, nh, nkv, S = case["B"], case["nh"], case["nkv"], case["s_max"]
        pos = _positions(case)
        st["pos"] = _ints(pos)
        st["q"] = torch.randn((B, nh * D), generator=g, device="cuda")
        kn, vn = _keys_values((B, nkv, D), g)
        st["k_new"], st["v_new"] = kn.reshape(B, nkv * D), vn.reshape(B, nkv * D)
        kc = torch.full((B, nkv, S, ROW), 255, dtype=torch.uint8, device="cuda")
        vc = torch.full((B, nkv, S, ROW), 255, dtype=torch.uint8, device="cuda")
        for b in range(B):  # the slots before the new token; those after it hold anything
            k, v = _keys_values((nkv, pos[b], D), g)
            kc[b, :, :pos[b]] = _pack(k, True)
            vc[b, :, :pos[b]] = _pack(v, False)
        st["k_cache"], st["v_cache"] = kc, vc
        st["out"] = torch.zeros((B, nh * D), dtype=torch.bfloat16, device="cuda")
        st["k_back"] = torch.zeros((B, nkv, D), device="cuda")
        st["v_back"] = torch.zeros((B, nkv, D), device="cuda")
        st["ws"] = None
    else:
        rows, V, k = case["rows"], case["V"], case["k"]
        x = torch.randn((rows, case["ld"]), generator=g, device="cuda").mul_(2.5)
        x += 4.0 * torch.randn(case["ld"], generator=g, device="cuda").clamp_(min=1.5)
        if case["banned"]:
            x.masked_fill_(torch.rand(case["ld"], generator=g, device="cuda") < case["banned"],
                           float("-inf"))
        x = x.to(DTYPES[case["dtype"]])
        x[:, V:] = float("nan")  # columns behind the vocabulary hold anything
        st["logits"] = x[:, :V]
        st["targets"] = torch.randint(V, (rows,), generator=g, device="cuda", dtype=torch.int32)
        st["logprob"] = torch.zeros(rows, device="cuda")
        st["entropy"] = torch.zeros(rows, device="cuda")
        st["top_idx"] = torch.zeros((rows, k), dtype=torch.int32, device="cuda") if k else None
        st["top_logprob"] = torch.zeros((rows, k), device="cuda") if k else None
        st["ws"] = None
    return st


# --------------------------------------------------------------------------- plain forms

def _prompt_plain(st):
    nh, nkv = st["nh"], st["nkv"]
    G = nh // nkv
    for a, b in zip(st["ends"], st["ends"][1:]):
        if a == b:
            continue
        L = b - a
        q = st["q"][a:b].float().unflatten(1, (nkv, G)).permute(1, 2, 0, 3).reshape(nkv, G * L, D)
        k = st["k"][a:b].float().permute(1, 2, 0)
        v = st["v"][a:b].float().permute(1, 0, 2)
        s = torch.bmm(q, k).mul_(1.0 / math.sqrt(D)).view(nkv, G, L, L)
        i = torch.arange(L, device="cuda")
        s.masked_fill_(i[None, :] > i[:, None], float("-inf"))
        m = s.amax(-1, keepdim=True)
        p = s.sub_(m).exp_()
        tot = p.sum(-1, keepdim=True)
        o = torch.bmm(p.view(nkv, G * L, L), v).view(nkv, G, L, D) / tot
        st["out"][a:b] = o.permute(2, 0, 1, 3).reshape(L, nh * D).to(st["out"].dtype)
        if st["lse_out"] is not None:
            st["lse_out"][a:b] = (m + tot.log()).view(nh, L).t()
    return {"out": st["out"], "lse": st["lse_out"]} if st["lse"] else {"out": st["out"]}


def _store_plain(st):
    T = st["k"].shape[0]
    t = torch.arange(T, device="cuda")
    if st["cu"] is None:
        seq, slot = t, st["start"].long()
    else:
        cu = st["cu"].long()
        seq = (t[:, None] >= cu[None, 1:]).sum(1)
        slot = st["start"].long()[seq] + t - cu[seq]
    row = seq if st["cache_rows"] is None else st["cache_rows"].long()[seq]
    st["k_cache"][row, :, slot] = _pack(st["k"], True)
    st["v_cache"][row, :, slot] = _pack(st["v"], False)
    st["k_back"].copy_(_unpack(st["k_cache"][row, :, slot], True))
    st["v_back"].copy_(_unpack(st["v_cache"][row, :, slot], False))
    return {"k": st["k_back"], "v": st["v_back"]}


def _decode_plain(st):
    B, nh, nkv, S = st["B"], st["nh"], st["nkv"], st["s_max"]
    pos = st["pos"].long()
    b = torch.arange(B, device="cuda")
    st["k_cache"][b, :, pos] = _pack(st["k_new"].view(B, nkv, D), True)
    st["v_cache"][b, :, pos] = _pack(st["v_new"].view(B, nkv, D), False)
    st["k_back"].copy_(_unpack(st["k_cache"][b, :, pos], True))
    st["v_back"].copy_(_unpack(st["v_cache"][b, :, pos], False))
    gone = (torch.arange(S, device="cuda")[None, :] > pos[:, None])[:, None, :, None]
    k = _unpack(st["k_cache"], True).masked_fill_(gone, 0.0)
    v = _unpack(st["v_cache"], False).masked_fill_(gone, 0.0)
    q = st["q"].view(B, nkv, nh // nkv, D)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D))
    s.masked_fill_(gone.transpose(-1, -2), float("-inf"))
    p = (s - s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    st["out"].copy_(o.reshape(B, nh * D))
    return {"out": st["out"], "k": st["k_back"], "v": st["v_back"]}


def _logprobs_plain(st):
    x = st["logits"].float()
    m = x.amax(-1, keepdim=True)
    y = x - m
    e = y.exp()
    tot = e.sum(-1)
    log_tot = tot.log()
    tgt = st["targets"].long()[:, None]
    st["logprob"].copy_(y.gather(1, tgt)[:, 0] - log_tot)
    st["entropy"].copy_(log_tot - torch.where(e == 0, torch.zeros_like(e), e * y).sum(-1) / tot)
    r = {"logprob": st["logprob"], "entropy": st["entropy"]}
    if st["k"]:
        # one key orders by value, then by the lower index
        bits = (x + 0.0).view(torch.int32).long()
        bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
        key = bits * (1 << 32) + (0x7FFFFFFF - torch.arange(x.shape[1], device="cuda"))
        top = 0x7FFFFFFF - (key.topk(st["k"], dim=-1).values & 0xFFFFFFFF)
        st["top_idx"].copy_(top)
        st["top_logprob"].copy_(y.gather(1, top) - log_tot[:, None])
        r["top_idx"], r["top_logprob"] = st["top_idx"], st["top_logprob"]
    return r


# --------------------------------------------------------------------------- the library's calls

def _run_own(st):
    from weight_streaming_gemv_bf16_gb300 import binding as wb
    if st["op"] == "prompt":
        wb.prompt_attention(st["q"], st["k"], st["v"], st["cu"], st["out"], lse=st["lse_out"])
        return {"out": st["out"], "lse": st["lse_out"]} if st["lse"] else {"out": st["out"]}
    if st["op"] == "store":
        wb.kv_store_q4(st["k"], st["v"], st["k_cache"], st["v_cache"], st["start"],
                       cu_seqlens=st["cu"], rows=st["cache_rows"])
        wb.kv_load_q4(st["k_cache"], st["v_cache"], st["start"], st["k_back"], st["v_back"],
                      cu_seqlens=st["cu"], rows=st["cache_rows"])
        return {"k": st["k_back"], "v": st["v_back"]}
    if st["op"] == "decode":
        if st["ws"] is None:  # kept by the program for all its steps
            n = wb.attention_q4_workspace_bytes(st["B"], st["nh"], st["nkv"], st["s_max"])
            st["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        wb.decode_attention_q4(st["q"], st["k_new"], st["v_new"], st["k_cache"], st["v_cache"],
                               st["pos"], st["ws"], out_bf16=st["out"])
        # the rows that the step added, as the cache holds them
        wb.kv_load_q4(st["k_cache"], st["v_cache"], st["pos"], st["k_back"], st["v_back"])
        return {"out": st["out"], "k": st["k_back"], "v": st["v_back"]}
    if st["ws"] is None:
        n = wb.logprobs_workspace_bytes(st["rows"], st["V"], st["k"])
        st["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    wb.token_logprobs(st["logits"], st["ws"], targets=st["targets"], logprob=st["logprob"],
                      entropy=st["entropy"], top_idx=st["top_idx"],
                      top_logprob=st["top_logprob"])
    r = {"logprob": st["logprob"], "entropy": st["entropy"]}
    if st["k"]:
        r["top_idx"], r["top_logprob"] = st["top_idx"], st["top_logprob"]
    return r


_PLAIN = {"prompt": _prompt_plain, "store": _store_plain, "decode": _decode_plain,
          "logprobs": _logprobs_plain}


def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


# --------------------------------------------------------------------------- work

def work(case):
    """Each input read once, each output written once; the multiply-adds of the unmasked pairs."""
    if case["op"] == "prompt":
        lens = _lens(case)
        nh, nkv = case["nh"], case["nkv"]
        n = sum(lens)
        b = n * (2 * nh + 2 * nkv) * D * 2 + (n * nh * 4 if case["lse"] else 0)
        return {"bytes": b, "flops": sum(4 * D * nh * L * (L + 1) // 2 for L in lens)}
    if case["op"] == "store":
        T = sum(_lens(case)) or case["rows"]
        e = 4 if case["dtype"] == "f32" else 2
        # k and v in, rows out; rows in, k and v out
        return {"bytes": T * case["nkv"] * 2 * (2 * D * e + 2 * ROW),
                "flops": T * case["nkv"] * 2 * D * 8}
    if case["op"] == "decode":
        slots = sum(p + 1 for p in _positions(case))
        B, nh, nkv = case["B"], case["nh"], case["nkv"]
        b = slots * nkv * 2 * ROW + B * nh * D * (4 + 2) + B * nkv * 2 * D * (4 + 4)
        return {"bytes": b, "flops": slots * nh * 4 * D}
    e = 4 if case["dtype"] == "f32" else 2
    rows, V = case["rows"], case["V"]
    return {"bytes": rows * (V * e + 12 + 8 * case["k"]), "flops": rows * V * 6}


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(case, st)
    if case["op"] == "store":
        k, v = _exact_rows(st["k"]), _exact_rows(st["v"])
        return {"k": k, "v": v}
    if case["op"] == "decode":
        return _exact_decode(case, st)
    return _exact_logprobs(case, st)


def _exact_prompt(case, st):
    T, nh, nkv = st["q"].shape[0], case["nh"], case["nkv"]
    out = torch.zeros((T, nh, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, nh), dtype=torch.float64, device="cuda")
    begin = 0
    for n in _lens(case):
        rows = slice(begin, begin + n)
        begin += n
        if n == 0:
            continue
        later = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
        for h in range(nh):
            key = st["k"][rows, h * nkv // nh].double()
            val = st["v"][rows, h * nkv // nh].double()
            score = st["q"][rows, h].double() @ key.T / D ** 0.5
            score[later] = -math.inf
            total = torch.logsumexp(score, dim=1)
            out[rows, h] = torch.exp(score - total[:, None]) @ val
            lse[rows, h] = total
    out = out.reshape(T, nh * D)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_rows(x):
    """What a stored row stands for: scale and zero as stored (bf16), the nearest of the 16 steps."""
    y = x.double().reshape(*x.shape[:-1], NG, GROUP)
    least = y.min(-1, keepdim=True).values
    step = ((y.max(-1, keepdim=True).values - least) / 15).float().bfloat16().double()
    mid = (least + 8 * step).float().bfloat16().double()
    n = torch.nan_to_num((y - mid) / step).round().clamp(-8, 7)
    return (mid + step * n).reshape(x.shape)


def _exact_value(rows, width):
    """Cached rows -> the values they stand for, by the format's own words: nibble n of the codes
    is dimension 32 g + width * t + i where n = (4 t + g) * width + i."""
    dim = torch.arange(D, device="cuda")
    g, t, i = dim // GROUP, dim % GROUP // width, dim % width
    nib = (4 * t + g) * width + i
    code = (rows[..., nib // 2].long() >> (4 * (nib % 2))) & 15
    word = rows[..., 64:].long()
    pair = ((word[..., 0::2] | (word[..., 1::2] << 8)) << 16).to(torch.int32)
    sz = pair.view(torch.float32).double()
    return sz[..., 2 * g] * (code - 8) + sz[..., 2 * g + 1]


def _exact_decode(case, st):
    B, nh, nkv = case["B"], case["nh"], case["nkv"]
    kn = _exact_rows(st["k_new"].view(B, nkv, D))
    vn = _exact_rows(st["v_new"].view(B, nkv, D))
    out = torch.zeros((B, nh, D), dtype=torch.float64, device="cuda")
    for b, p in enumerate(_positions(case)):
        for j in range(nkv):
            key = torch.cat([_exact_value(st["k_cache"][b, j, :p], 8), kn[b, j:j + 1]])
            val = torch.cat([_exact_value(st["v_cache"][b, j, :p], 4), vn[b, j:j + 1]])
            heads = slice(j * nh // nkv, (j + 1) * nh // nkv)
            score = st["q"].view(B, nh, D)[b, heads].double() @ key.T / D ** 0.5
            out[b, heads] = torch.softmax(score, dim=-1) @ val
    return {"out": out.reshape(B, nh * D), "k": kn, "v": vn}


def _exact_logprobs(case, st):
    rows, k = case["rows"], case["k"]
    r = {"logprob": torch.empty(rows, dtype=torch.float64, device="cuda"),
         "entropy": torch.empty(rows, dtype=torch.float64, device="cuda")}
    if k:
        r["top_idx"] = torch.empty((rows, k), dtype=torch.int32, device="cuda")
        r["top_logprob"] = torch.empty((rows, k), dtype=torch.float64, device="cuda")
    for a in range(0, rows, 256):
        x = st["logits"][a:a + 256].double()
        lp = torch.log_softmax(x, dim=-1)
        b = a + x.shape[0]
        r["logprob"][a:b] = lp.gather(1, st["targets"][a:b, None].long())[:, 0]
        p = lp.exp()
        r["entropy"][a:b] = -(p * lp.masked_fill(p == 0, 0.0)).sum(-1)
        if k:
            order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :k]
            r["top_idx"][a:b] = order
            r["top_logprob"][a:b] = lp.gather(1, order)
    return r
