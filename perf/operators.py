"""Cases and plain forms of the language-model operators: rotary positions,
attention (forward and backward) and the softmax cross entropy of the tied head.

With `own` false, run() computes each operator from elementary torch operations
in 32 bits (64 for the rotary angles), rounded once at the end; with `own` true
it makes the calls a user of the library makes.  exact() gives the same outputs
from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases

def _rope(name, **kw):
    c = {"name": name, "op": "rope", "tokens": 64, "heads": 12, "head_dim": 64, "rotary": 64,
         "interleaved": False, "dtype": "bf16", "far": 0, "scaling": "none", "factor": 1.0,
         "inverse": False, "seq": 1024}
    c.update(kw)
    return c


def _attn(name, **kw):
    c = {"name": name, "op": "attn", "train": True, "heads": 8, "kv_heads": 4, "head_dim": 80,
         "batch": 16, "q_len": 1024, "k_len": 1024, "causal": True, "window": 0, "ragged": False}
    c.update(kw)
    return c


def _ce(name, **kw):
    c = {"name": name, "op": "ce", "train": True, "tokens": 65536, "vocab": 8192, "d": 512,
         "ignored": 0.0}
    c.update(kw)
    return c


def listed():
    return [
        # queries and keys of one training step of the 512-wide model, 64 sequences of 1,024
        _rope("rope_step", tokens=65536),
        # 16 of 64 dimensions rotated, adjacent pairs, positions far beyond the trained length
        _rope("rope_partial_far", tokens=16383, rotary=16, interleaved=True, dtype="fp32",
              far=2000000, scaling="yarn", factor=16.0),
        # the gradient's inverse rotation on a short remainder batch of the 640-wide core
        _rope("rope_back_small", tokens=77, head_dim=80, rotary=80, inverse=True),
        # the 640-wide recurrent core: 16 sequences of 1,024 tokens, 8 query and 4 KV heads of 80
        _attn("attn_train_core"),
        # the same core's forward alone (validation)
        _attn("attn_fwd_core", train=False),
        # sliding evaluation: the last 64 tokens of each 1,024-token window are scored
        _attn("attn_eval_tail", train=False, head_dim=64, batch=256, q_len=64),
        # documents of many lengths packed into one batch, long ones among them
        _attn("attn_train_packed", heads=8, kv_heads=2, head_dim=128, batch=7, q_len=8192,
              k_len=8192, ragged=True),
        # a few short documents with a sliding window: the smallest training call
        _attn("attn_train_short", head_dim=64, batch=3, q_len=129, k_len=129, window=50,
              ragged=True),
        # the tied 8,192-word head of the throughput workload at 65,536 tokens
        _ce("ce_train_head"),
        # validation loss of the 1,024-word model
        _ce("ce_eval", train=False, tokens=16384, vocab=1024),
        # a large odd vocabulary, padded rows that count for nothing
        _ce("ce_train_large_vocab", tokens=4099, vocab=50257, d=640, ignored=0.1),
        # one short batch: the smallest training call
        _ce("ce_train_short", tokens=130, vocab=1024, ignored=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attn", "ce"])
    if op == "rope":
        hd = 8 * rng.randint(2, 16)
        rot = hd if rng.random() < 0.5 else 2 * rng.randint(1, hd // 2)
        c = _rope("", tokens=_log(rng, 1, 65536), heads=rng.randint(1, 16), head_dim=hd, rotary=rot,
                  interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp32"]),
                  far=rng.choice([0, 0, 100000, 2000000]),
                  scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                  factor=float(rng.choice([2, 4, 16])), inverse=rng.random() < 0.5,
                  seq=rng.choice([512, 1000, 2048]))
        if c["dtype"] == "fp32":
            c["tokens"] = max(1, c["tokens"] // 2)
    elif op == "attn":
        group = rng.choice([1, 2, 4])
        kvh = rng.randint(1, 4)
        hd = 8 * rng.randint(2, 16)
        k_len = _log(rng, 1, 4096)
        q_len = k_len if rng.random() < 0.6 else _log(rng, 1, 4096)
        causal = rng.random() < 0.75
        pairs = max(1, q_len) * max(1, k_len) * group * kvh
        batch = max(1, min(32, int(rng.uniform(0.2, 1.0) * 2.4e8 / pairs)))
        c = _attn("", train=rng.random() < 0.6, heads=group * kvh, kv_heads=kvh, head_dim=hd,
                  batch=batch, q_len=q_len, k_len=k_len, causal=causal,
                  window=_log(rng, 1, k_len) if causal and rng.random() < 0.3 else 0,
                  ragged=rng.random() < 0.5)
    else:
        vocab = _log(rng, 500, 65536)
        d = 8 * rng.randint(8, 128)
        tokens = _log(rng, 1, max(2, min(65536, int(2.5e11 / (vocab * d)))))
        c = _ce("", train=rng.random() < 0.6, tokens=tokens, vocab=vocab, d=d,
                ignored=rng.choice([0.0, 0.1]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _spread(n, top):
    """Lengths of n packed sequences: short ones most often, one of length `top`."""
    v = [int(top * ((i + 0.5) / n) ** 2) for i in range(n)]
    v[-1] = top
    return v


def _lengths(case, g, top):
    n = case["batch"]
    if not case["ragged"]:
        return torch.full((n,), top, dtype=torch.int64, device=DEV)
    lens = torch.tensor(_spread(n, top), device=DEV)
    return lens[torch.randperm(n, generator=g, device=DEV)]


def prepare(case, seed):
    g = _gen(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    if case["op"] == "rope":
        T, width = case["tokens"], case["heads"] * case["head_dim"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # queries and keys are a column range of the projection's output
        full = rand(T, width + 4 * case["head_dim"]).to(dt)
        first = torch.randint(0, case["far"] + 1, (1,), generator=g, device=DEV)
        pos = torch.arange(T, device=DEV) % case["seq"] + first
        return {"case": case, "x": full[:, :width], "pos": pos, **_plan(case)}
    if case["op"] == "attn":
        lk = _lengths(case, g, case["k_len"])
        same = case["q_len"] == case["k_len"]
        lq = lk if same else _lengths(case, g, case["q_len"])
        cu = lambda v: torch.cat([v.new_zeros(1), v.cumsum(0)]).to(torch.int32)
        cu_q, cu_k = cu(lq), cu(lk)
        tq, tk = int(cu_q[-1]), int(cu_k[-1])
        wq, wk = case["heads"] * case["head_dim"], case["kv_heads"] * case["head_dim"]
        if same:  # one projection's output
            qkv = rand(tq, wq + 2 * wk).bfloat16()
            q, k, v = qkv[:, :wq], qkv[:, wq:wq + wk], qkv[:, wq + wk:]
        else:
            q, kv = rand(tq, wq).bfloat16(), rand(tk, 2 * wk).bfloat16()
            k, v = kv[:, :wk], kv[:, wk:]
        return {"case": case, "q": q, "k": k, "v": v, "cu_q": cu_q, "cu_k": cu_k,
                "dO": (rand(tq, wq) * 1e-2).bfloat16()}
    T, V, d = case["tokens"], case["vocab"], case["d"]
    w = rand(V, d) * 0.02
    s = w.abs().amax(dim=1, keepdim=True).clamp(min=1e-12) / 127
    operand = ((w / s).round().clamp(-127, 127) * s).bfloat16()  # the head's int8 operand
    targets = torch.randint(0, V, (T,), generator=g, device=DEV)
    # a model that has learnt something: the state leans to the next word's row
    lean = w[targets] * (8.0 * torch.rand(T, 1, generator=g, device=DEV) / (0.02 * math.sqrt(d)))
    z = (rand(T, d) + lean).bfloat16()
    if case["ignored"] > 0:
        drop = torch.rand(T, generator=g, device=DEV) < case["ignored"]
        targets = torch.where(drop, torch.full_like(targets, -100), targets)
    return {"case": case, "z": z, "operand": operand, "targets": targets}


def _plan(case):
    """Turns per position of each rotated pair (64 bits) and the factor of cos and sin."""
    rot, base, trained = case["rotary"], 10000.0, case["seq"]
    f = case["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    m = 1.0
    if case["scaling"] == "ntk" and rot > 2:
        base = base * f ** (rot / (rot - 2))
    freq = base ** (-2.0 * i / rot) / (2 * math.pi)
    if case["scaling"] == "linear":
        freq = freq / f
    if case["scaling"] == "yarn":
        low = rot * math.log(trained / (32.0 * 2 * math.pi)) / (2 * math.log(base))
        high = rot * math.log(trained / (1.0 * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        freq = freq * (1 - ramp) + freq / f * ramp
        m = 0.1 * math.log(f) + 1.0
    return {"freqs": freq, "mscale": m}


# -------------------------------------------------------------- plain forms

def _plain_rope(st):
    c, x = st["case"], st["x"]
    H, hd, rot = c["heads"], c["head_dim"], c["rotary"]
    turns = st["pos"].double()[:, None] * st["freqs"][None]
    ang = (turns - turns.round()) * (2 * math.pi)
    cos, sin = (ang.cos() * st["mscale"]).float()[:, None], (ang.sin() * st["mscale"]).float()[:, None]
    if c["inverse"]:
        sin = -sin
    xf = x.float().reshape(-1, H, hd)
    r = xf[..., :rot]
    if c["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([y, xf[..., rot:]], dim=-1).reshape(x.shape).to(x.dtype)


def _padded(cu, top):
    """Row of each place of the padded [batch, top] layout, and whether it holds one."""
    at = cu[:-1, None].long() + torch.arange(top, device=cu.device)[None]
    ok = at < cu[1:, None].long()
    return torch.where(ok, at, torch.zeros_like(at)), ok


def _plain_attn(st):
    c = st["case"]
    H, KH, hd = c["heads"], c["kv_heads"], c["head_dim"]
    G, B, Lq, Lk = H // KH, c["batch"], c["q_len"], c["k_len"]
    tq, tk = st["q"].shape[0], st["k"].shape[0]
    iq, okq = _padded(st["cu_q"], Lq)
    ik, okk = _padded(st["cu_k"], Lk)
    if tk == 0:  # no keys at all
        ik, okk, st = ik * 0, okk & False, {**st, "k": st["k"].new_zeros(1, KH * hd),
                                            "v": st["v"].new_zeros(1, KH * hd)}
    if tq == 0:
        iq, okq, st = iq * 0, okq & False, {**st, "q": st["q"].new_zeros(1, H * hd),
                                            "dO": st["dO"].new_zeros(1, H * hd)}
    # [B, KH, G, L, hd] queries and [B, KH, 1, L, hd] keys and values
    q = st["q"].float()[iq].view(B, Lq, KH, G, hd).permute(0, 2, 3, 1, 4)
    k = st["k"].float()[ik].view(B, Lk, KH, 1, hd).permute(0, 2, 3, 1, 4)
    v = st["v"].float()[ik].view(B, Lk, KH, 1, hd).permute(0, 2, 3, 1, 4)
    nq, nk = (st["cu_q"][1:] - st["cu_q"][:-1]).long(), (st["cu_k"][1:] - st["cu_k"][:-1]).long()
    mask = okk[:, None, :] & okq[:, :, None]
    if c["causal"]:  # the last query is aligned with the last key
        p = torch.arange(Lq, device=DEV)[None, :, None] + (nk - nq)[:, None, None]
        j = torch.arange(Lk, device=DEV)[None, None, :]
        mask = mask & (j <= p)
        if c["window"]:
            mask = mask & (j > p - c["window"])
    mask = mask[:, None, None]
    scale = 1.0 / math.sqrt(hd)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~mask, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = (s - top).exp_()
    del s
    z = e.sum(-1, keepdim=True)
    lse = (top + z.log()).squeeze(-1)
    p = e.div_(torch.where(z == 0, torch.ones_like(z), z))
    o = torch.matmul(p, v)

    def rows(x, n, width, at, ok):  # padded [B, KH, G, L, hd] -> packed rows
        out = torch.zeros(n + 1, width, device=DEV)
        out[torch.where(ok, at, torch.full_like(at, n))] = x.permute(0, 3, 1, 2, 4).reshape(B, -1, width)
        return out[:n].bfloat16()

    lse_rows = torch.zeros(tq + 1, H, device=DEV)
    lse_rows[torch.where(okq, iq, torch.full_like(iq, tq))] = lse.permute(0, 3, 1, 2).reshape(B, Lq, H)
    out = {"o": rows(o, tq, H * hd, iq, okq), "lse": lse_rows[:tq].t().contiguous()}
    if not c["train"]:
        return out
    do = st["dO"].float()[iq].view(B, Lq, KH, G, hd).permute(0, 2, 3, 1, 4) * okq[:, None, None, :, None]
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
    dp = torch.matmul(do, v.transpose(-1, -2))
    ds = (dp - (p * dp).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    del dp, p
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2, keepdim=True)
    out["dq"] = rows(dq, tq, H * hd, iq, okq)
    out["dk"] = rows(dk, tk, KH * hd, ik, okk)
    out["dv"] = rows(dv, tk, KH * hd, ik, okk)
    return out


def _plain_ce(st):
    c, tgt = st["case"], st["targets"]
    z, w = st["z"].float(), st["operand"].float()
    logits = z @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = (top + (logits - top).exp().sum(1, keepdim=True).log())
    ok = tgt >= 0
    at = torch.where(ok, tgt, torch.zeros_like(tgt))[:, None]
    loss = torch.where(ok, (lse - logits.gather(1, at)).squeeze(1), torch.zeros_like(lse[:, 0]))
    inv = 1.0 / ok.sum().clamp(min=1).float()
    mean = loss.double().sum().float() * inv
    out = {"loss": loss, "lse": lse.squeeze(1), "mean": mean}
    if c["train"]:
        g = logits.sub_(lse).exp_()
        g.scatter_add_(1, at, -torch.ones_like(at, dtype=torch.float32))
        g.mul_((ok.float() * inv)[:, None])
        out["dZ"] = (g @ w).bfloat16()
        out["dW"] = g.t() @ z
    return out


# ---------------------------------------------------------- the library's calls

def _own_rope(st):
    from quantization_aware_tiny_b200 import qat
    c, x = st["case"], st["x"]
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    qat.qat_rope(x, y, c["heads"], c["head_dim"], st["freqs"], positions=st["pos"],
                 interleaved=c["interleaved"], scale=st["mscale"], inverse=c["inverse"])
    return y


def _own_attn(st):
    from quantization_aware_tiny_b200 import qat
    c, q, k, v = st["case"], st["q"], st["k"], st["v"]
    H, KH, hd = c["heads"], c["kv_heads"], c["head_dim"]
    kw = {"causal": c["causal"], "window": c["window"], "cu_q": st["cu_q"], "cu_k": st["cu_k"],
          "max_q": c["q_len"], "max_k": c["k_len"]}
    tq, tk = q.shape[0], k.shape[0]
    o = torch.empty(tq, H * hd, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(H, tq, device=DEV)
    qat.qat_attn_fwd(q, k, v, o, lse, H, KH, hd, **kw)
    out = {"o": o, "lse": lse}
    if c["train"]:
        # one buffer, as the projection's backward takes it, where queries and keys share rows
        if tq == tk:
            dqkv = torch.empty(tq, (H + 2 * KH) * hd, dtype=torch.bfloat16, device=DEV)
            dq, dk, dv = dqkv[:, :H * hd], dqkv[:, H * hd:(H + KH) * hd], dqkv[:, (H + KH) * hd:]
        else:
            dq = torch.empty(tq, H * hd, dtype=torch.bfloat16, device=DEV)
            dk = torch.empty(tk, KH * hd, dtype=torch.bfloat16, device=DEV)
            dv = torch.empty(tk, KH * hd, dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(qat.workspace_size(qat.QAT_OP_ATTN_BWD, H, hd, tq, False),
                         dtype=torch.uint8, device=DEV)
        qat.qat_attn_bwd(st["dO"], q, k, v, o, lse, dq, dk, dv, H, KH, hd, workspace=ws, **kw)
        out.update(dq=dq, dk=dk, dv=dv)
    return out


def _own_ce(st):
    from quantization_aware_tiny_b200 import qat
    c, z, tgt = st["case"], st["z"], st["targets"]
    T, V, d = c["tokens"], c["vocab"], c["d"]
    qw = qat.QWeight(st["operand"], None, None, 8)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    mean = torch.empty(2, device=DEV)  # mean loss, 1 / counted tokens
    op = qat.QAT_OP_CE_BWD if c["train"] else qat.QAT_OP_CE_FWD
    ws = torch.empty(qat.workspace_size(op, V, d, T, False), dtype=torch.uint8, device=DEV)
    qat.qat_ce_fwd(z, tgt, loss, lse, 8, qw=qw, mean=mean, workspace=ws)
    out = {"loss": loss, "lse": lse, "mean": mean[0]}
    if c["train"]:
        dZ = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
        dW = torch.empty(V, d, device=DEV)
        qat.qat_ce_bwd(z, tgt, lse, 8, qw=qw, gscale=mean[1:], dZ=dZ, dW=dW, workspace=ws)
        out.update(dZ=dZ, dW=dW)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "attn": _own_attn, "ce": _own_ce}[op](state)
    return {"rope": _plain_rope, "attn": _plain_attn, "ce": _plain_ce}[op](state)


# ---------------------------------------------------------------------- work

def work(case):
    if case["op"] == "rope":
        b = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * case["heads"] * case["head_dim"]
        return {"bytes": 2 * n * b + 8 * case["tokens"], "flops": 3 * n}
    if case["op"] == "attn":
        lens = _work_lengths(case)
        H, KH, hd = case["heads"], case["kv_heads"], case["head_dim"]
        pairs = sum(_pairs(case, a, b) for a, b in lens)
        tq, tk = sum(a for a, _ in lens), sum(b for _, b in lens)
        qo, kv = 2 * tq * H * hd, 2 * 2 * tk * KH * hd
        # forward: q, k, v in, o and lse out; backward: dO in, dq, dk, dv out
        by = 2 * qo + kv + 4 * H * tq
        fl = 4 * hd * H * pairs
        if case["train"]:
            by += 2 * qo + kv
            fl += 10 * hd * H * pairs
        return {"bytes": by, "flops": fl}
    T, V, d = case["tokens"], case["vocab"], case["d"]
    by = 2 * T * d + 2 * V * d + 8 * T + 8 * T
    fl = 2 * T * V * d
    if case["train"]:
        by += 2 * T * d + 4 * V * d
        fl *= 3
    return {"bytes": by, "flops": fl}


def _work_lengths(case):
    n, same = case["batch"], case["q_len"] == case["k_len"]
    some = lambda top: _spread(n, top) if case["ragged"] else [top] * n
    k = some(case["k_len"])
    return list(zip(k if same else some(case["q_len"]), k))


def _pairs(case, nq, nk):
    """Query-key pairs that the mask keeps in one sequence."""
    if not case["causal"]:
        return nq * nk
    n = 0
    for i in range(nq):
        last = i + nk - nq
        first = max(0, last - case["window"] + 1) if case["window"] else 0
        n += max(0, last - first + 1)
    return n


# --------------------------------------------------------- definitions, 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, st)
    if case["op"] == "attn":
        return _exact_attn(case, st)
    return _exact_ce(case, st)


def _exact_rope(case, st):
    """Each pair as a complex number times m * exp(+-2 pi i turns)."""
    T, H, hd, rot = case["tokens"], case["heads"], case["head_dim"], case["rotary"]
    x = st["x"].double().reshape(T, H, hd).clone()
    turns = torch.remainder(st["pos"].double().unsqueeze(1) * st["freqs"], 1.0)
    ang = turns * (-2 * math.pi if case["inverse"] else 2 * math.pi)
    unit = torch.polar(torch.full_like(ang, st["mscale"]), ang).unsqueeze(1)
    i = torch.arange(rot // 2, device=DEV)
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
    w = torch.complex(x[..., first], x[..., second]) * unit
    x[..., first], x[..., second] = w.real, w.imag
    return x.reshape(T, H * hd)


def _exact_attn(case, st):
    """Sequence by sequence and head by head."""
    H, KH, hd = case["heads"], case["kv_heads"], case["head_dim"]
    q, k, v, do = (st[n].double() for n in ("q", "k", "v", "dO"))
    cq, ck = st["cu_q"].tolist(), st["cu_k"].tolist()
    o, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.full((H, q.shape[0]), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(case["batch"]):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        if nq == 0 or nk == 0:
            continue
        rq, rk = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        keep = torch.ones(nq, nk, dtype=torch.bool, device=DEV)
        if case["causal"]:
            keep = keep.tril(nk - nq)
            if case["window"]:
                keep = keep.triu(nk - nq - case["window"] + 1)
        none = ~keep.any(1)
        for h in range(H):
            cols = slice(h * hd, (h + 1) * hd)
            kcols = slice(h // (H // KH) * hd, (h // (H // KH) + 1) * hd)
            a, kk, vv = q[rq, cols] / math.sqrt(hd), k[rk, kcols], v[rk, kcols]
            s = torch.where(keep, a @ kk.T, -math.inf)
            lse[h, rq] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1).masked_fill(none[:, None], 0.0)
            o[rq, cols] = p @ vv
            if case["train"]:
                dd = do[rq, cols]
                dv[rk, kcols] += p.T @ dd
                ds = p * (dd @ vv.T - (dd * o[rq, cols]).sum(1, keepdim=True))
                dq[rq, cols] = ds @ kk / math.sqrt(hd)
                dk[rk, kcols] += ds.T @ a
    out = {"o": o, "lse": lse}
    if case["train"]:
        out.update(dq=dq, dk=dk, dv=dv)
    return out


def _exact_ce(case, st):
    """Log probabilities row block by row block."""
    z, w, tgt = st["z"].double(), st["operand"].double(), st["targets"]
    T = z.shape[0]
    ok = tgt >= 0
    count = max(1, int(ok.sum()))
    loss = torch.zeros(T, dtype=torch.float64, device=DEV)
    lse, dz, dw = torch.zeros_like(loss), torch.zeros_like(z), torch.zeros_like(w)
    for t in range(0, T, 8192):
        r = slice(t, min(T, t + 8192))
        logits = z[r] @ w.T
        lse[r] = torch.logsumexp(logits, 1)
        live = ok[r].nonzero().squeeze(1)
        loss[r][live] = lse[r][live] - logits[live, tgt[r][live]]
        if case["train"]:
            g = torch.zeros_like(logits)
            g[live] = torch.softmax(logits[live], 1)
            g[live, tgt[r][live]] -= 1
            g /= count
            dz[r] = g @ w
            dw += g.T @ z[r]
    out = {"loss": loss, "lse": lse, "mean": loss.sum() / count}
    if case["train"]:
        out.update(dZ=dz, dW=dw)
    return out
