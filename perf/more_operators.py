"""Cases for the operators of one rollout step beside the frozen NVFP4 linears:

  append  new keys and values, bf16, quantised into a 4-bit cache (E2M1 codes, one E4M3 scale per 16 values, a fixed
          scale per cache), and the values that the cache then holds for them;
  attn    attention over such caches: every sequence's queries over the prompt that its group shares and over its own
          tokens, one softmax over both;
  sample  the next token of every row of logits from a given uniform number: temperature, top-k, top-p, min-p, and the
          token's log-probability in the whole and in the cut distribution.

``own`` False: plain torch operations in 32 bits (64 where tokens lie next to a border); True: the calls of
nvfp4_weight_only_quantize_gb300.  ``exact``: the definitions in 64 bits, written apart.
"""
import math

import torch

own = False
DEV = "cuda"

# Head layouts (query heads, key/value heads) of the decoder layers this repository works on: hidden 2048, 3584, 5120.
HEADS = ((16, 2), (28, 4), (40, 8))
K_SCALE, V_SCALE = 1.0, 0.5  # the fixed scales of the caches


# ------------------------------------------------------------------ cases
def listed():
    sm = dict(op="sample", dtype="bf16", temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, per_row=False)
    at = dict(op="attn", Lq=1, D=128, ragged=True)
    return [
        # the new token of 64 sequences: latency
        dict(op="append", name="append_step_of_64", B=64, L=1, Hkv=8, D=128, T=4096),
        # eight prompts of up to 4001 tokens
        dict(op="append", name="append_prompts", B=8, L=4001, Hkv=8, D=128, T=4096),
        # one sequence's token after a short prompt: latency
        dict(at, name="attn4_first_token", B=1, G=1, Hq=28, Hkv=4, P=512, S=1, ragged=False),
        # a rollout batch of eight prompts with eight long answers each: the answers dominate
        dict(at, name="attn4_8_prompts_x_8", B=64, G=8, Hq=40, Hkv=8, P=512, S=4096),
        # two sequences with nothing shared and a long past
        dict(at, name="attn4_two_long", B=2, G=1, Hq=28, Hkv=4, P=0, S=131072),
        # 64 samples of one long prompt: the prompt dominates
        dict(at, name="attn4_64_on_long_prompt", B=64, G=64, Hq=28, Hkv=4, P=16384, S=999),
        # a turn's new tokens (a tool's answer) for each sample of a group, causal among themselves
        dict(at, name="attn4_turn_of_129", B=8, G=8, Hq=16, Hkv=2, Lq=129, P=4001, S=257),
        # one sequence's token with the usual cuts: latency
        dict(sm, name="sample_one", T=1, V=131072, top_k=50, top_p=0.95),
        # a rollout batch as it is trained on: no cut
        dict(sm, name="sample_64_uncut", T=64, V=131072),
        # a large batch, nucleus alone
        dict(sm, name="sample_1024_nucleus", T=1024, V=131072, top_p=0.95),
        # FP32 logits of an odd vocabulary (rows start at every alignment), every cut, each row its own
        dict(sm, name="sample_odd_vocab_f32", T=257, V=100003, dtype="f32", temperature=0.8, top_k=50, top_p=0.9, min_p=0.05, per_row=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    top = {}
    for c in listed():
        w, t = work(c), top.setdefault(c["op"], [0.0, 0.0])
        t[0], t[1] = max(t[0], w["bytes"]), max(t[1], w["flops"])
    op = rng.choice(("attn", "attn", "sample", "sample", "append"))
    while True:
        if op == "attn":
            Hq, Hkv = rng.choice(HEADS)
            G = _log_int(rng, 1, 64)
            n = _log_int(rng, 1, max(1, 64 // G))
            Lq = 1 if rng.random() < 0.7 else _log_int(rng, 2, 160)
            long = rng.random() < 0.2
            c = dict(op=op, B=n * G, G=G, Hq=Hq, Hkv=Hkv, D=rng.choice((64, 128, 128)), Lq=Lq, P=0 if long else _log_int(rng, 1, 16384),
                     S=max(Lq, _log_int(rng, 1, 131072 if long else 4096)), ragged=rng.random() < 0.8)
        elif op == "sample":
            cut = rng.random() < 0.75
            c = dict(op=op, T=_log_int(rng, 1, 1024), V=_log_int(rng, 500, 152000), dtype=rng.choice(("bf16", "bf16", "f32")),
                     temperature=rng.choice((1.0, 0.8, 0.6)), top_k=rng.choice((0, 1, 20, 50, 1000)) if cut else 0,
                     top_p=rng.choice((1.0, 0.95, 0.8)) if cut else 1.0, min_p=rng.choice((0.0, 0.0, 0.05)) if cut else 0.0,
                     per_row=rng.random() < 0.3)
        else:
            L = _log_int(rng, 1, 4096)
            c = dict(op=op, B=_log_int(rng, 1, 64), L=L, Hkv=rng.choice(HEADS)[1], D=rng.choice((64, 128, 128)),
                     T=L + _log_int(rng, 1, 4096))
        w = work(c)
        if w["bytes"] <= top[op][0] and w["flops"] <= top[op][1] and (op != "append" or c["B"] * c["T"] <= 1 << 18):
            return c


def _spread(n, lo, hi):
    """n lengths over [lo, hi], a fixed set for the case."""
    return [lo + ((k + 1) * 2654435761 + 97) % 4294967296 * (hi - lo + 1) // 4294967296 for k in range(n)]


def _attn_lens(case):
    """(prefix length of each group, length of each sequence's own tokens, its new ones among them)."""
    n = case["B"] // case["G"]
    if not case["ragged"]:
        return [case["P"]] * n, [case["S"]] * case["B"]
    return [case["P"]] + _spread(n - 1, (case["P"] + 1) // 2, case["P"]), [case["S"]] + _spread(case["B"] - 1, case["Lq"], case["S"])


def _cell(D):
    """Bytes of one key or value of one head."""
    return D // 2 + D // 16


def work(case):
    if case["op"] == "append":
        n = case["B"] * case["L"] * case["Hkv"] * 2
        return {"bytes": n * (4 * case["D"] + _cell(case["D"])), "flops": 4 * n * case["D"]}
    if case["op"] == "attn":
        pl, sl = _attn_lens(case)
        G, Lq, Hq, Hkv, D = (case[k] for k in ("G", "Lq", "Hq", "Hkv", "D"))
        seen = sum(pl[b // G] * Lq + Lq * n - Lq * (Lq - 1) // 2 for b, n in enumerate(sl))
        rows = case["B"] * Lq * Hq
        return {"bytes": 2 * rows * D * 2 + rows * 4 + (sum(pl) + sum(sl)) * Hkv * _cell(D) * 2, "flops": 4 * seen * Hq * D}
    return {"bytes": case["T"] * (case["V"] * (2 if case["dtype"] == "bf16" else 4) + 20), "flops": 4 * case["T"] * case["V"]}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def prepare(case, seed):
    return {"append": _prepare_append, "attn": _prepare_attn, "sample": _prepare_sample}[case["op"]](case, seed)


def _keys(g, B, L, Hkv, D):
    """Keys or values: some channels are larger than others in every token."""
    x = torch.randn(B, L, Hkv, D, generator=g, device=DEV, dtype=torch.bfloat16)
    return x * torch.exp(0.5 * torch.randn(Hkv, D, generator=g, device=DEV)).to(torch.bfloat16)


def _prepare_append(case, seed):
    g = _gen(seed)
    B, L, Hkv, D, T = (case[k] for k in ("B", "L", "Hkv", "D", "T"))
    lens = torch.tensor(_spread(B, L, T), dtype=torch.int32, device=DEV)
    s = dict(case=case, k=_keys(g, B, L, Hkv, D), v=_keys(g, B, L, Hkv, D), lens=lens)
    if own:
        import nvfp4_weight_only_quantize_gb300 as q
        s["cache"] = q.Kv4Cache(B, T, Hkv, D, k_scale=K_SCALE, v_scale=V_SCALE)
        s["out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    else:
        s["cache"] = [(torch.zeros(B, T, Hkv, D // 2, dtype=torch.uint8, device=DEV), torch.zeros(B, T, Hkv, D // 16, dtype=torch.uint8, device=DEV))
                      for _ in range(2)]
    return s


def _prepare_attn(case, seed):
    g = _gen(seed)
    B, n, Lq, Hq, Hkv, D, P, S = case["B"], case["B"] // case["G"], *(case[k] for k in ("Lq", "Hq", "Hkv", "D", "P", "S"))
    pl, sl = _attn_lens(case)
    order = torch.randperm(B, generator=g, device=DEV)
    s = dict(case=case, q=torch.randn(B, Lq, Hq, D, generator=g, device=DEV, dtype=torch.bfloat16) * 1.5,
             pl=torch.tensor(pl, dtype=torch.int32, device=DEV), sl=torch.tensor(sl, dtype=torch.int32, device=DEV)[order].contiguous())
    held = [(_keys(g, n, P, Hkv, D), _keys(g, n, P, Hkv, D)) if P else None, (_keys(g, B, S, Hkv, D), _keys(g, B, S, Hkv, D))]
    if own:
        import nvfp4_weight_only_quantize_gb300 as q
        caches = []
        for kv in held:
            caches.append(None)
            if kv is not None:
                T = kv[0].shape[1]
                caches[-1] = q.Kv4Cache(kv[0].shape[0], T, Hkv, D, k_scale=K_SCALE, v_scale=V_SCALE)
                caches[-1].append(*kv, torch.full((kv[0].shape[0],), T, dtype=torch.int32, device=DEV))
        s["plan"] = q.Kv4Attention(caches[1], q_heads=Hq, q_len=Lq, prefix=caches[0])
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, Lq, Hq, device=DEV)
    else:
        s["prefix"], s["suffix"] = (None if kv is None else [_quantised(x, f) for x, f in zip(kv, (K_SCALE, V_SCALE))] for kv in held)
    return s


def _prepare_sample(case, seed):
    g = _gen(seed)
    T, V = case["T"], case["V"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    logits = torch.randn(T, V, generator=g, device=DEV, dtype=dt).mul_(2.5)
    # a few tokens stand out, in some rows by far and in others hardly
    at = torch.arange(40, device=DEV) * (V // 40) + torch.randint(V // 40, (T, 40), generator=g, device=DEV)
    height = torch.rand(T, 1, generator=g, device=DEV) * 14 + 4
    logits.scatter_(1, at, (height + 3 * torch.randn(T, 40, generator=g, device=DEV)).to(dt))
    s = dict(case=case, logits=logits, u=torch.rand(T, generator=g, device=DEV), temperature=case["temperature"], top_k=case["top_k"],
             top_p=case["top_p"], min_p=case["min_p"])
    if case["per_row"]:  # every request of the batch has its own settings, some of them no cut
        f = lambda x: torch.full((T,), float(x), device=DEV)  # noqa: E731
        some = lambda: torch.rand(T, generator=g, device=DEV)  # noqa: E731
        s["temperature"] = f(case["temperature"]) * (0.5 + some())
        s["top_k"] = torch.where(some() < 0.3, 0, torch.full((T,), case["top_k"], device=DEV)).int()
        s["top_p"], s["min_p"] = torch.where(some() < 0.3, 1.0, f(case["top_p"])), torch.where(some() < 0.5, 0.0, f(case["min_p"]))
    if own:
        import nvfp4_weight_only_quantize_gb300 as q
        s["q"] = q
        s["ids"], s["logp"], s["logq"] = torch.empty(T, dtype=torch.int64, device=DEV), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    return s


# ------------------------------------------------------------------ the 4-bit format
STEPS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantised(x, fixed):
    """(codes [..., D / 2], the even element in the low half; scales [..., D / 16]) of x [..., D]: the block's scale is the
    smallest E4M3 number that is at least amax / (6 fixed), each code the nearest value, ties to the even code."""
    w = x.float().unflatten(-1, (-1, 16))
    t = (w.abs().amax(-1) / torch.tensor(6.0 * fixed, device=DEV)).clamp(max=448.0)
    near = t.to(torch.float8_e4m3fn)
    byte = near.view(torch.uint8)
    byte = byte + (near.float() < t).to(torch.uint8)
    scale = byte.view(torch.float8_e4m3fn).float() * fixed
    q = w / torch.where(scale > 0, scale, 1.0)[..., None]
    a = q.abs()
    code = (a > 0.25).byte()
    for at, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += ((a >= at) if up else (a > at)).byte()
    code += 8 * ((q < 0) & (code > 0)).byte()
    code = (code * (scale > 0)[..., None].byte()).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, byte


def _values(held, fixed):
    """The values of (codes, scales), FP32."""
    codes, scales = held
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    v = torch.tensor(STEPS + tuple(-x for x in STEPS), device=DEV)[code]
    return (v.unflatten(-1, (-1, 16)) * (scales.view(torch.float8_e4m3fn).float() * fixed)[..., None]).flatten(-2)


# ------------------------------------------------------------------ one pass
def run(state):
    return {"append": _run_append, "attn": _run_attn, "sample": _run_sample}[state["case"]["op"]](state)


def _run_append(s):
    if own:
        s["cache"].append(s["k"], s["v"], s["lens"])
        s["cache"].read(s["lens"], s["case"]["L"], *s["out"])
        return {"k": s["out"][0], "v": s["out"][1]}
    B, L = s["case"]["B"], s["case"]["L"]
    at = (s["lens"].view(B, 1) - L + torch.arange(L, device=DEV)).long()
    row = torch.arange(B, device=DEV).view(B, 1).expand(B, L)
    out = []
    for x, held, fixed in zip((s["k"], s["v"]), s["cache"], (K_SCALE, V_SCALE)):
        for to, new in zip(held, _quantised(x, fixed)):
            to[row, at] = new
        out.append(_values([t[row, at] for t in held], fixed).to(torch.bfloat16))
    return {"k": out[0], "v": out[1]}


def _run_attn(s):
    if own:
        s["plan"].run(s["q"], s["sl"], prefix_lens=s["pl"] if s["case"]["P"] else None, out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    c = s["case"]
    B, G, Lq, Hq, Hkv, D = (c[k] for k in ("B", "G", "Lq", "Hq", "Hkv", "D"))
    n, gs, P, S = B // G, Hq // Hkv, c["P"], c["S"]
    q = s["q"].float().mul(1.0 / math.sqrt(D)).view(B, Lq, Hkv, gs, D).permute(0, 2, 1, 3, 4)  # [B, Hkv, Lq, gs, D]
    ks, vs = (_values(h, f) for h, f in zip(s["suffix"], (K_SCALE, V_SCALE)))
    ss = q.reshape(B, Hkv, Lq * gs, D) @ ks.permute(0, 2, 3, 1)  # [B, Hkv, Lq gs, S]
    sees = s["sl"].view(B, 1) - Lq + 1 + torch.arange(Lq, device=DEV)  # own tokens that token l of sequence b sees
    ss.masked_fill_(torch.arange(S, device=DEV) >= sees.repeat_interleave(gs, 1).view(B, 1, Lq * gs, 1), -math.inf)
    mx = ss.amax(-1, keepdim=True)
    back = lambda t: t.reshape(n, Hkv, G, Lq * gs, -1).transpose(1, 2).reshape(B, Hkv, Lq * gs, -1)  # noqa: E731
    if P:
        kp, vp = (_values(h, f) for h, f in zip(s["prefix"], (K_SCALE, V_SCALE)))
        qg = q.reshape(n, G, Hkv, Lq * gs, D).transpose(1, 2).reshape(n, Hkv, G * Lq * gs, D)
        sp = qg @ kp.permute(0, 2, 3, 1)  # [n, Hkv, G Lq gs, P]
        sp.masked_fill_(torch.arange(P, device=DEV) >= s["pl"].view(n, 1, 1, 1), -math.inf)
        mx = torch.maximum(mx, back(sp.amax(-1, keepdim=True)))
    es = torch.exp(ss - mx)
    z, o = es.sum(-1, keepdim=True), es @ vs.transpose(1, 2)
    if P:
        ep = torch.exp(sp - mx.reshape(n, G, Hkv, Lq * gs, 1).transpose(1, 2).reshape(n, Hkv, -1, 1))
        z, o = z + back(ep.sum(-1, keepdim=True)), o + back(ep @ vp.transpose(1, 2))
    order = lambda t: t.reshape(B, Hkv, Lq, gs, -1).permute(0, 2, 1, 3, 4)  # noqa: E731
    return {"out": order(o / z).reshape(B, Lq, Hq, D).to(torch.bfloat16), "lse": order(mx + torch.log(z)).reshape(B, Lq, Hq)}


def _run_sample(s):
    if own:
        s["q"].qerl_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                           ids=s["ids"], logp=s["logp"], logq=s["logq"])
        return {"ids": s["ids"], "logp": s["logp"], "logq": s["logq"]}
    T, V = s["case"]["T"], s["case"]["V"]
    setting = lambda k, dt: s[k].view(T, 1) if torch.is_tensor(s[k]) else torch.full((T, 1), s[k], dtype=dt, device=DEV)  # noqa: E731
    tau, top_k, top_p, min_p = setting("temperature", torch.float32), setting("top_k", torch.int32), setting("top_p", torch.float32), setting("min_p", torch.float32)
    ids, logp, logq = torch.empty(T, dtype=torch.int64, device=DEV), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    for a in range(0, T, 128):
        r = slice(a, min(a + 128, T))
        x = s["logits"][r].double() / tau[r].double()
        x -= x.amax(-1, keepdim=True)
        y, at = torch.sort(x, dim=-1, descending=True, stable=True)
        p = torch.exp(y)
        whole = p.sum(-1)
        rank = torch.arange(V, device=DEV)
        p = torch.where((rank < top_k[r]) | (top_k[r] <= 0), p, 0.0)
        upto = p.cumsum(-1)
        p = torch.where((upto - p < top_p[r].double() * upto[:, -1:]) | (top_p[r] >= 1) | (rank == 0), p, 0.0)
        p = torch.where(p >= min_p[r].double(), p, 0.0)
        upto = torch.zeros_like(p).scatter_(1, at, p).cumsum(-1)
        target = s["u"][r].double()[:, None] * upto[:, -1:]
        ids[r] = torch.searchsorted(upto, target, right=True)[:, 0]
        mine = x.gather(1, ids[r][:, None])[:, 0]
        logp[r] = (mine - torch.log(whole)).float()
        logq[r] = (mine - torch.log(upto[:, -1])).float()
    return {"ids": ids, "logp": logp, "logq": logq}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attn": _exact_attn, "sample": _exact_sample}[case["op"]](case, s)


def _e4m3_table():
    """The non-negative finite E4M3 numbers, by their byte."""
    return torch.tensor([(m * 2.0 ** -9) if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127], dtype=torch.float64, device=DEV)


def _nearest(x, fixed):
    """x [..., 16 n] in 64 bits on the grid of its blocks' values."""
    table, half = _e4m3_table(), torch.tensor(STEPS, dtype=torch.float64, device=DEV)
    blocks = x.double().reshape(-1, 16)
    want = blocks.abs().max(dim=1).values / (6.0 * fixed)
    unit = table[torch.searchsorted(table, want).clamp(max=126)] * fixed
    q = torch.where(unit[:, None] > 0, blocks.abs() / unit[:, None], 0.0).clamp(max=6.0)
    hi = torch.searchsorted(half, q).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    below, above = q - half[lo], half[hi] - q
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return (half[pick] * unit[:, None] * torch.sign(blocks)).reshape(x.shape)


def _exact_append(c, s):
    cut = lambda x, f: torch.stack([_nearest(b, f) for b in x])  # noqa: E731
    return {"k": cut(s["k"], K_SCALE), "v": cut(s["v"], V_SCALE)}


def _exact_held(held, fixed, i, n, h):
    """Keys or values of one head of one sequence, 64 bits, [n, D]."""
    codes, scales = held[0][i, :n, h].long(), held[1][i, :n, h].long()
    half = torch.tensor(STEPS, dtype=torch.float64, device=DEV)
    e = torch.empty(n, 2 * codes.shape[1], dtype=torch.int64, device=DEV)
    e[:, 0::2], e[:, 1::2] = codes % 16, codes // 16
    return half[e % 8] * (1 - 2 * (e // 8)) * _e4m3_table()[scales].repeat_interleave(16, 1) * fixed


def _exact_attn(c, s):
    B, G, Lq, Hq, Hkv, D = (c[k] for k in ("B", "G", "Lq", "Hq", "Hkv", "D"))
    out = torch.empty(B, Lq, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, Lq, Hq, dtype=torch.float64, device=DEV)
    pl, sl = s["pl"].tolist(), s["sl"].tolist()
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            both = [[_exact_held(s["suffix"][t], f, b, sl[b], h)] for t, f in enumerate((K_SCALE, V_SCALE))]
            if c["P"]:
                both = [[_exact_held(s["prefix"][t], f, b // G, pl[b // G], h)] + both[t] for t, f in enumerate((K_SCALE, V_SCALE))]
            k, v = torch.cat(both[0]), torch.cat(both[1])
            a = torch.einsum("lhd,kd->lhk", s["q"][b, :, heads].double(), k) / D ** 0.5
            last = len(k) - Lq + torch.arange(Lq, device=DEV)
            a = a.masked_fill(torch.arange(len(k), device=DEV) > last[:, None, None], -math.inf)
            lse[b, :, heads] = torch.logsumexp(a, -1)
            out[b, :, heads] = torch.einsum("lhk,kd->lhd", torch.exp(a - lse[b, :, heads, None]), v)
    return {"out": out, "lse": lse}


def _exact_sample(c, s):
    """Row by row: the tokens in order of probability, cut, put back in order of index, and the first that carries the
    sum beyond u."""
    T, V = c["T"], c["V"]
    of = lambda k, t: float(s[k][t]) if torch.is_tensor(s[k]) else float(torch.tensor(s[k], dtype=torch.float32))  # noqa: E731
    ids = torch.empty(T, dtype=torch.int64, device=DEV)
    logp, logq = (torch.empty(T, dtype=torch.float64, device=DEV) for _ in range(2))
    for t in range(T):
        lp = torch.log_softmax(s["logits"][t].double() / of("temperature", t), 0)
        order = torch.argsort(-lp, stable=True)
        top_k, top_p, min_p = int(of("top_k", t)), of("top_p", t), of("min_p", t)
        kept = order[:top_k] if top_k > 0 else order
        if top_p < 1:
            share = torch.softmax(lp[kept], 0)
            kept = kept[:int((share.cumsum(0) < top_p).sum()) + 1]
        if min_p > 0:
            kept = kept[lp[kept] - lp[order[0]] >= math.log(min_p)]
        kept = kept.sort().values
        share = torch.softmax(lp[kept], 0)
        i = kept[min(int((share.cumsum(0) <= float(s["u"][t])).sum()), len(kept) - 1)]
        ids[t], logp[t], logq[t] = i, lp[i], lp[i] - torch.logsumexp(lp[kept], 0)
    return {"ids": ids, "logp": logp, "logq": logq}
