"""Cases for the operators of one reinforcement-learning step around the frozen NVFP4 linears:

  attn    attention of a rollout batch whose sequences share a long prefix (the prompt of a group of samples): every
          sequence's queries over the shared prefix and over its own suffix, joined into one softmax;
  loss    the clipped policy loss with a KL term, from the logits: token log-probabilities, entropy, the loss and the
          gradient of the logits; or the log-probabilities and entropy alone (old and reference policy);
  adamw   one AdamW step over all LoRA adapters, states in 32 bits or in 8 (blocks of 256, stochastic rounding), with
          the clip by the global gradient norm.

``own`` False: plain torch operations in 32 bits; True: the calls of nvfp4_weight_only_quantize_gb300.  ``exact``: the
definitions in 64 bits, written apart.
"""
import functools
import math

import torch

own = False
DEV = "cuda"

# Head layouts (query heads, key/value heads) of the decoder layers this repository works on: hidden 2048, 3584, 5120.
HEADS = ((16, 2), (28, 4), (40, 8))
BLOCK = 256  # elements that share one scale in the 8-bit states
QM, QV = 1.9375, 1.96875  # the largest magnitude of the 8-bit codes of m and of sqrt(v)
BETA1, BETA2, EPS, STEP, LR = 0.9, 0.999, 1e-8, 7, 2e-5


# ------------------------------------------------------------------ cases
def listed():
    a = dict(op="attn", Lq=1, D=128, ragged=True)
    lo = dict(op="loss", beta=0.04, temperature=1.0, grad=True, dtype="bf16", masked=0.1)
    ad = dict(op="adamw", layers=1)
    return [
        # the first sampled token after a short prompt, one sequence: latency
        dict(a, name="attn_first_token", B=1, G=1, Hq=28, Hkv=4, P=512, S=1, ragged=False),
        # one prompt, a group of eight samples half way through their answers
        dict(a, name="attn_group_of_8", B=8, G=8, Hq=28, Hkv=4, P=512, S=1024),
        # a rollout batch of eight prompts with eight long answers each: the suffixes dominate
        dict(a, name="attn_8_prompts_x_8", B=64, G=8, Hq=40, Hkv=8, P=512, S=4096),
        # 64 samples of one long prompt: the prefix dominates
        dict(a, name="attn_64_on_long_prompt", B=64, G=64, Hq=28, Hkv=4, P=16384, S=999),
        # a turn's new tokens (a tool's answer) for each sample of a group, causal among themselves
        dict(a, name="attn_turn_of_129", B=8, G=8, Hq=16, Hkv=2, Lq=129, P=4001, S=257),
        # a few tokens of a small vocabulary shard: latency
        dict(lo, name="loss_16_tokens", T=16, V=16000),
        # a training micro-batch: loss and gradient over a full vocabulary
        dict(lo, name="loss_4096_tokens", T=4096, V=131072),
        # FP32 logits of an odd vocabulary (rows start at every alignment), sampled at a temperature
        dict(lo, name="loss_odd_vocab_f32", T=1001, V=100003, dtype="f32", temperature=0.8, masked=0.3),
        # log-probabilities of the old or reference policy: no gradient
        dict(lo, name="logp_2048_tokens", T=2048, V=131072, grad=False, masked=0.0),
        # the adapter of one 2048 x 2048 linear: latency
        dict(ad, name="adamw_one_linear", hidden=2048, kv=0, inter=0, r=16, state=32, param="f32", grad="f32", clip=0.0),
        # every adapter of 28 layers, FP32 states, bf16 weights beside FP32 masters, clipped
        dict(ad, name="adamw_28_layers_32bit", layers=28, hidden=3584, kv=512, inter=18944, r=32, state=32, param="bf16",
             grad="f32", clip=1.0),
        # the same with 8-bit states
        dict(ad, name="adamw_28_layers_8bit", layers=28, hidden=3584, kv=512, inter=18944, r=32, state=8, param="bf16",
             grad="f32", clip=1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    top = {}
    for c in listed():
        w, t = work(c), top.setdefault(c["op"], [0.0, 0.0])
        t[0], t[1] = max(t[0], w["bytes"]), max(t[1], w["flops"])
    op = rng.choice(("attn", "attn", "loss", "adamw"))
    while True:
        if op == "attn":
            Hq, Hkv = rng.choice(HEADS)
            G = _log_int(rng, 1, 64)
            n = _log_int(rng, 1, max(1, 64 // G))
            Lq = 1 if rng.random() < 0.7 else _log_int(rng, 2, 160)
            c = dict(op=op, B=n * G, G=G, Hq=Hq, Hkv=Hkv, D=rng.choice((64, 128, 128)), Lq=Lq, P=_log_int(rng, 1, 16384),
                     S=max(Lq, _log_int(rng, 1, 4096)), ragged=rng.random() < 0.8)
        elif op == "loss":
            c = dict(op=op, T=_log_int(rng, 1, 4096), V=_log_int(rng, 500, 152000), dtype=rng.choice(("bf16", "bf16", "f32")),
                     grad=rng.random() < 0.75, beta=rng.choice((0.0, 0.04)), temperature=rng.choice((1.0, 0.8)),
                     masked=rng.choice((0.0, 0.1, 0.4)))
        else:
            c = dict(op=op, layers=_log_int(rng, 1, 28), hidden=_log_int(rng, 100, 5120), kv=_log_int(rng, 64, 1024),
                     inter=_log_int(rng, 100, 27648), r=rng.choice((4, 7, 8, 16, 32, 33, 64)), state=rng.choice((8, 8, 32)),
                     param=rng.choice(("bf16", "f32")), grad=rng.choice(("f32", "bf16")), clip=rng.choice((0.0, 1.0)))
        w = work(c)
        if w["bytes"] <= top[op][0] and w["flops"] <= max(top[op][1], 1.0):
            return c


def _spread(n, lo, hi):
    """n lengths over [lo, hi], a fixed set for the case."""
    return [lo + (k * 2654435761 + 97) % 4294967296 * (hi - lo + 1) // 4294967296 for k in range(n)]


def _attn_lens(case):
    """(prefix length of each group, suffix length of each sequence, its new tokens among them)."""
    n = case["B"] // case["G"]
    if not case["ragged"]:
        return [case["P"]] * n, [case["S"]] * case["B"]
    return [case["P"]] + _spread(n - 1, (case["P"] + 1) // 2, case["P"]), [case["S"]] + _spread(case["B"] - 1, case["Lq"], case["S"])


def _adapter_sizes(case):
    """Element counts of A [r, K] and B [N, r] of every linear, layer by layer."""
    h, kv, it, r = case["hidden"], case["kv"], case["inter"], case["r"]
    lin = [(h, h)] + ([(kv, h), (kv, h), (h, h)] if kv else []) + ([(it, h), (it, h), (h, it)] if it else [])
    return [s for _ in range(case["layers"]) for N, K in lin for s in (r * K, N * r)]


def work(case):
    if case["op"] == "attn":
        pl, sl = _attn_lens(case)
        G, Lq, Hq, Hkv, D = (case[k] for k in ("G", "Lq", "Hq", "Hkv", "D"))
        seen = sum(pl[b // G] * Lq + Lq * n - Lq * (Lq - 1) // 2 for b, n in enumerate(sl))
        rows = case["B"] * Lq * Hq
        return {"bytes": 2 * rows * D * 2 + rows * 4 + (sum(pl) + sum(sl)) * Hkv * D * 2 * 2, "flops": 4 * seen * Hq * D}
    if case["op"] == "loss":
        e = 2 if case["dtype"] == "bf16" else 4
        active = case["T"] - int(case["T"] * case["masked"])
        return {"bytes": e * case["V"] * (active + (case["T"] if case["grad"] else 0)) + case["T"] * 40,
                "flops": (8 if case["grad"] else 4) * active * case["V"]}
    n = sum(_adapter_sizes(case))
    g = 2 if case["grad"] == "bf16" else 4
    st = 16 if case["state"] == 32 else 2 + 2 + 4 + 16 / BLOCK  # codes read and written, the values handed out in bf16
    return {"bytes": n * (g + 8 + (2 if case["param"] == "bf16" else 0) + st), "flops": 14 * n}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def prepare(case, seed):
    return {"attn": _prepare_attn, "loss": _prepare_loss, "adamw": _prepare_adamw}[case["op"]](case, seed)


def _prepare_attn(case, seed):
    g = _gen(seed)
    B, n, Lq, Hq, Hkv, D, P, S = case["B"], case["B"] // case["G"], *(case[k] for k in ("Lq", "Hq", "Hkv", "D", "P", "S"))
    pl, sl = _attn_lens(case)
    order = torch.randperm(B, generator=g, device=DEV)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    s = dict(case=case, q=rnd(B, Lq, Hq, D) * 1.5, kp=rnd(n, P, Hkv, D), vp=rnd(n, P, Hkv, D), ks=rnd(B, S, Hkv, D), vs=rnd(B, S, Hkv, D),
             pl=torch.tensor(pl, dtype=torch.int32, device=DEV), sl=torch.tensor(sl, dtype=torch.int32, device=DEV)[order].contiguous())
    s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, Lq, Hq, device=DEV)
    if own:
        import nvfp4_weight_only_quantize_gb300 as q
        s["plan"] = q.PrefixAttention(s["kp"], s["vp"], s["ks"], s["vs"], q_heads=Hq, q_len=Lq)
    return s


def _prepare_loss(case, seed):
    g = _gen(seed)
    T, V, tau = case["T"], case["V"], case["temperature"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    logits = torch.randn(T, V, generator=g, device=DEV, dtype=dt).mul_(2.5)
    ids = torch.randint(V, (T,), generator=g, device=DEV)
    vec = lambda: torch.randn(T, generator=g, device=DEV)  # noqa: E731
    # a sampled token is a likely one: from far down the tail to nearly certain
    at = torch.arange(T, device=DEV)
    logits[at, ids] = (14.0 + 4.0 * vec()).to(dt)
    logp = torch.cat([torch.log_softmax(logits[i:i + 256].float() / tau, -1).gather(1, ids[i:i + 256, None])[:, 0] for i in range(0, T, 256)])
    weight = torch.full((T,), 1.0 / T, device=DEV)
    weight[torch.randperm(T, generator=g, device=DEV)[:int(T * case["masked"])]] = 0.0
    s = dict(case=case, logits=logits, ids=ids, old=logp + 0.15 * vec(), ref=logp + 0.3 * vec() if case["beta"] else None, adv=vec(),
             weight=weight, dlogits=torch.empty_like(logits) if case["grad"] else None, logp=torch.empty(T, device=DEV),
             entropy=torch.empty(T, device=DEV), sums=torch.empty(4, device=DEV))
    if own:
        import nvfp4_weight_only_quantize_gb300 as q
        s["q"] = q
        s["ws"] = q.workspace(q.OP_POLICY_LOSS, T, V, 0, 0)
    return s


def _blocks(sizes):
    return [-(-n // BLOCK) for n in sizes]


def _prepare_adamw(case, seed):
    """Every adapter starts on a multiple of 256 elements of flat buffers, as an arena of adapters lays them out; what
    lies between them is zero."""
    g = _gen(seed)
    sizes = _adapter_sizes(case)
    nb = _blocks(sizes)
    N = sum(nb) * BLOCK
    sz = torch.tensor(sizes, device=DEV)
    nbt = torch.tensor(nb, device=DEV)
    first = (nbt.cumsum(0) - nbt) * BLOCK
    which = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), nbt * BLOCK)
    inside = torch.arange(N, device=DEV) - first[which] < sz[which]
    del which
    rnd = lambda std: torch.randn(N, generator=g, device=DEV).mul_(std).masked_fill_(~inside, 0.0)  # noqa: E731
    # gradients differ in size from row to row; some elements have had none yet
    grad = rnd(1e-3) * torch.exp(torch.randn(N // 64, generator=g, device=DEV)).repeat_interleave(64)
    gdt = torch.float32 if case["grad"] == "f32" else torch.bfloat16
    s = dict(case=case, sizes=sizes, sizes_t=sz, blocks_t=nbt, seed=1234 + seed, grad=grad.to(gdt), master=rnd(0.02),
             lr_scale=torch.tensor([1.0, 4.0], device=DEV).repeat(len(sizes) // 2), norm=torch.zeros(1, device=DEV))
    s["param"] = s["master"].to(torch.bfloat16) if case["param"] == "bf16" else None
    if case["state"] == 32:
        s["m"], s["v"] = rnd(3e-4), rnd(5e-4).square_()
    else:
        code = lambda lo, hi: torch.randint(lo, hi, (N,), generator=g, device=DEV, dtype=torch.int16).masked_fill_(~inside, 0).to(torch.uint8)  # noqa: E731
        s["m"], s["v"] = code(0, 256), code(1, 256)
        s["m"].masked_fill_(s["m"] == 128, 0)  # zero has one code
        s["ms"], s["vs"] = (torch.rand(N // BLOCK, generator=g, device=DEV) * k + k / 4 for k in (1e-3, 1e-3))
        s["m_out"], s["v_out"] = (torch.zeros(N, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    if own:
        import nvfp4_weight_only_quantize_gb300 as q
        starts = first.tolist()
        cut = lambda t: None if t is None else [t[a:a + n] for a, n in zip(starts, sizes)]  # noqa: E731
        cutb = lambda t: None if t is None else [t[a // BLOCK:a // BLOCK + b] for a, b in zip(starts, nb)]  # noqa: E731
        p32 = s["param"] is None
        s["opt"] = q.AdamW(cut(s["master"] if p32 else s["param"]), cut(s["grad"]), masters=None if p32 else cut(s["master"]),
                           m=cut(s["m"]), v=cut(s["v"]), m_scale=cutb(s.get("ms")), v_scale=cutb(s.get("vs")), betas=(BETA1, BETA2), eps=EPS,
                           weight_decay=0.01, lr_scale=[1.0, 4.0] * (len(sizes) // 2))
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return {"attn": _run_attn, "loss": _run_loss, "adamw": _run_adamw}[state["case"]["op"]](state)


def _run_attn(s):
    if own:
        s["plan"].run(s["q"], s["sl"], prefix_lens=s["pl"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    c = s["case"]
    B, G, Lq, Hq, Hkv, D = (c[k] for k in ("B", "G", "Lq", "Hq", "Hkv", "D"))
    n, gs, P, S = B // G, Hq // Hkv, c["P"], c["S"]
    q = s["q"].float().mul(1.0 / math.sqrt(D)).view(B, Lq, Hkv, gs, D).permute(0, 2, 1, 3, 4)  # [B, Hkv, Lq, gs, D]
    qg = q.reshape(n, G, Hkv, Lq * gs, D).transpose(1, 2).reshape(n, Hkv, G * Lq * gs, D)
    sp = qg @ s["kp"].float().permute(0, 2, 3, 1)  # [n, Hkv, G Lq gs, P]
    sp.masked_fill_(torch.arange(P, device=DEV) >= s["pl"].view(n, 1, 1, 1), -math.inf)
    ss = q.reshape(B, Hkv, Lq * gs, D) @ s["ks"].float().permute(0, 2, 3, 1)  # [B, Hkv, Lq gs, S]
    sees = s["sl"].view(B, 1) - Lq + 1 + torch.arange(Lq, device=DEV)  # suffix keys that token l of sequence b sees
    ss.masked_fill_(torch.arange(S, device=DEV) >= sees.repeat_interleave(gs, 1).view(B, 1, Lq * gs, 1), -math.inf)
    back = lambda t: t.reshape(n, Hkv, G, Lq * gs, -1).transpose(1, 2).reshape(B, Hkv, Lq * gs, -1)  # noqa: E731
    mx = torch.maximum(back(sp.amax(-1, keepdim=True)), ss.amax(-1, keepdim=True))
    es = torch.exp(ss - mx)
    ep = torch.exp(sp - mx.reshape(n, G, Hkv, Lq * gs, 1).transpose(1, 2).reshape(n, Hkv, -1, 1))
    z = es.sum(-1, keepdim=True) + back(ep.sum(-1, keepdim=True))
    o = (es @ s["vs"].float().transpose(1, 2) + back(ep @ s["vp"].float().transpose(1, 2))) / z
    order = lambda t: t.reshape(B, Hkv, Lq, gs, -1).permute(0, 2, 1, 3, 4)  # noqa: E731
    return {"out": order(o).reshape(B, Lq, Hq, D).to(torch.bfloat16), "lse": order(mx + torch.log(z)).reshape(B, Lq, Hq)}


CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def _run_loss(s):
    c = s["case"]
    if own:
        q = s["q"]
        if not c["grad"]:
            q.qerl_token_logp(s["logits"], s["ids"], weights=s["weight"], temperature=c["temperature"], logp=s["logp"], entropy=s["entropy"])
            return {"logp": s["logp"], "entropy": s["entropy"]}
        q.qerl_policy_loss(s["logits"], s["ids"], s["old"], s["adv"], s["weight"], ref_logp=s["ref"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                           beta=c["beta"], temperature=c["temperature"], dlogits=s["dlogits"], logp=s["logp"], entropy=s["entropy"],
                           sums=s["sums"], ws=s["ws"])
        return {"sums": s["sums"], "logp": s["logp"], "entropy": s["entropy"], "dlogits": s["dlogits"]}
    w = s["weight"]
    takes = w != 0
    x = s["logits"].float() / torch.tensor(c["temperature"], device=DEV)
    x = x.sub_(x.amax(-1, keepdim=True))
    e = torch.exp(x)
    z = e.sum(-1)
    logp = torch.where(takes, x.gather(1, s["ids"][:, None])[:, 0] - torch.log(z), 0.0)
    entropy = torch.where(takes, torch.log(z) - (e * x).sum(-1) / z, 0.0)
    if not c["grad"]:
        return {"logp": logp, "entropy": entropy}
    a = s["adv"]
    ratio = torch.exp(logp - s["old"])
    keeps = torch.where(a >= 0, ratio <= 1 + CLIP_HIGH, ratio >= 1 - CLIP_LOW)
    policy = -torch.minimum(ratio * a, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * a)
    d = (s["ref"] if s["ref"] is not None else logp) - logp
    kl = torch.expm1(d) - d
    add = lambda t: torch.where(takes, w * t, 0.0).double().sum().float()  # noqa: E731
    sums = torch.stack([add(policy + c["beta"] * kl), add(policy), add(kl), add((~keeps).float())])
    dlogp = torch.where(takes, w * (c["beta"] * -torch.expm1(d) - torch.where(keeps, ratio * a, 0.0)), 0.0) / c["temperature"]
    dx = e.mul_((-dlogp / z)[:, None])
    dx[torch.arange(c["T"], device=DEV), s["ids"]] += dlogp
    return {"sums": sums, "logp": logp, "entropy": entropy, "dlogits": dx.to(s["logits"].dtype)}


M32 = 0xFFFFFFFF


def _philox_round(x, r, seed):
    """One round of Philox4x32 (Salmon et al., 2011) on int64 tensors that hold 32-bit words."""
    k0, k1 = ((seed & M32) + r * 0x9E3779B9) & M32, ((seed >> 32) + r * 0xBB67AE85) & M32
    p, q = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
    return (q >> 32 & M32) ^ x[1] ^ k0, q & M32, (p >> 32 & M32) ^ x[3] ^ k1, p & M32


def _coef(s):
    """The factor of the clip by the global norm, from a sum in 64 bits."""
    norm = s["grad"].double().square().sum().sqrt()
    clip = s["case"]["clip"]
    s["norm"].copy_(norm.float())
    return torch.where(norm > clip, clip / norm, 1.0).float()


def _store8(x, rnd, bits, top):
    """Block-scaled codes of x >= 0 [blocks, 256]: 3 exponent bits, `bits` of mantissa, rounded by `rnd` (16 bits)."""
    amax = x.amax(1, keepdim=True)
    holds = amax >= 2.0 ** -100
    q = torch.full_like(amax, top)
    y = x * torch.where(holds, q / amax, 0.0)
    drop = 23 - bits
    u = (y * 2.0 ** -120).view(torch.int32) + (rnd << (drop - 16)) + (1 << (drop - 17))
    return (u >> drop).clamp_(max=(8 << bits) - 1), torch.where(holds, amax / q, 0.0), holds


def _load8(code, bits, scale):
    return (code << (23 - bits)).view(torch.float32) * 2.0 ** 120 * scale


def _run_adamw(s):
    c = s["case"]
    if own:
        if c["clip"]:
            s["opt"].step(LR, STEP, seed=s["seed"], max_grad_norm=c["clip"], grad_norm=s["norm"])
        else:
            s["opt"].step(LR, STEP, seed=s["seed"])
        m, v = s["m"], s["v"]
        if c["state"] == 8:
            s["opt"].read_state(s["m_out"], s["v_out"])
            m, v = s["m_out"], s["v_out"]
        return {"param": s["param"], "master": s["master"], "m": m, "v": v, "norm": s["norm"]}
    per_tensor = lambda t: torch.repeat_interleave(t, s["blocks_t"])[:, None]  # noqa: E731
    grid = lambda t: t.view(-1, BLOCK)  # noqa: E731
    lr = LR * s["lr_scale"].double()
    step_size, decay = per_tensor((lr / (1 - BETA1 ** STEP)).float()), per_tensor((1 - lr * 0.01).float())
    g = grid(s["grad"].float())
    if c["clip"]:
        g = g * _coef(s)
    if c["state"] == 32:
        m, v = grid(s["m"]), grid(s["v"])
    else:
        ms, vs = s["ms"][:, None], s["vs"][:, None]
        cm = grid(s["m"]).int()
        m = _load8(cm & 127, 4, ms) * torch.where(cm >= 128, -1.0, 1.0)
        v = _load8(grid(s["v"]).int(), 5, vs)
        v = v * v
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    root = v.sqrt()
    p = grid(s["master"])
    p = p * decay - step_size * (m / (root * (1 / math.sqrt(1 - BETA2 ** STEP)) + EPS))
    s["master"].view(-1, BLOCK).copy_(p)
    if s["param"] is not None:
        s["param"].copy_(s["master"])
    if c["state"] == 32:
        grid(s["m"]).copy_(m)
        grid(s["v"]).copy_(v)
        return {"param": s["param"], "master": s["master"], "m": s["m"], "v": s["v"], "norm": s["norm"]}
    # the random words: counter (group of four elements of the tensor, its high word, tensor, step), key seed
    first = s["blocks_t"].cumsum(0) - s["blocks_t"]
    tensor = torch.repeat_interleave(torch.arange(len(s["sizes"]), device=DEV), s["blocks_t"])[:, None]
    group = (torch.arange(len(tensor), device=DEV)[:, None] - first[tensor]) * (BLOCK // 4) + torch.arange(BLOCK // 4, device=DEV)
    start = (group & M32, group >> 32, tensor.expand_as(group), torch.full_like(group, STEP))
    word = torch.stack(functools.reduce(lambda x, r: _philox_round(x, r, s["seed"]), range(10), start), -1).view(-1, BLOCK).to(torch.int64)
    cm, sm, _ = _store8(m.abs(), (word & 0xFFFF).int(), 4, QM)
    cv, sv, kept = _store8(root, (word >> 16).int(), 5, QV)
    cv = torch.where(kept & (root > 0), cv.clamp(min=1), cv)
    grid(s["m"]).copy_(cm + torch.where((m < 0) & (cm > 0), 128, 0))
    grid(s["v"]).copy_(cv)
    s["ms"].copy_(sm[:, 0])
    s["vs"].copy_(sv[:, 0])
    mv = _load8(cm, 4, sm) * torch.where(m < 0, -1.0, 1.0)
    vv = _load8(cv, 5, sv)
    s["m_out"].copy_(mv.flatten())
    s["v_out"].copy_((vv * vv).flatten())
    return {"param": s["param"], "master": s["master"], "m": s["m_out"], "v": s["v_out"], "norm": s["norm"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "loss": _exact_loss, "adamw": _exact_adamw}[case["op"]](case, s)


def _exact_attn(c, s):
    B, G, Lq, Hq, Hkv, D = (c[k] for k in ("B", "G", "Lq", "Hq", "Hkv", "D"))
    out = torch.empty(B, Lq, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, Lq, Hq, dtype=torch.float64, device=DEV)
    pl, sl = s["pl"].tolist(), s["sl"].tolist()
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            k = torch.cat([s["kp"][b // G, :pl[b // G], h], s["ks"][b, :sl[b], h]]).double()
            v = torch.cat([s["vp"][b // G, :pl[b // G], h], s["vs"][b, :sl[b], h]]).double()
            a = torch.einsum("lhd,kd->lhk", s["q"][b, :, heads].double(), k) / D ** 0.5
            last = len(k) - Lq + torch.arange(Lq, device=DEV)
            a = a.masked_fill(torch.arange(len(k), device=DEV) > last[:, None, None], -math.inf)
            lse[b, :, heads] = torch.logsumexp(a, -1)
            out[b, :, heads] = torch.einsum("lhk,kd->lhd", torch.exp(a - lse[b, :, heads, None]), v)
    return {"out": out, "lse": lse}


def _exact_loss(c, s):
    T = c["T"]
    at = {k: torch.zeros(T, dtype=torch.float64, device=DEV) for k in ("logp", "entropy", "policy", "kl", "cut")}
    dl = torch.zeros(T, c["V"], dtype=torch.float64, device=DEV) if c["grad"] else None
    w = s["weight"].double()
    for t0 in range(0, T, 512):
        i = torch.arange(t0, min(t0 + 512, T), device=DEV)
        i = i[w[i] != 0]
        lp = torch.log_softmax(s["logits"][i].double() / c["temperature"], -1)
        p = lp.exp()
        tok = lp.gather(1, s["ids"][i, None])[:, 0]
        at["logp"][i], at["entropy"][i] = tok, -(p * lp).sum(-1)
        if not c["grad"]:
            continue
        a, rho = s["adv"][i].double(), torch.exp(tok - s["old"][i].double())
        up, down = a * rho, a * rho.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
        free = (up <= down)
        at["policy"][i] = -torch.where(free, up, down)
        dlp = -torch.where(free, up, 0.0)
        at["cut"][i] = (~free).double()
        if s["ref"] is not None:
            u = s["ref"][i].double() - tok
            at["kl"][i] = u.exp() - u - 1
            dlp = dlp + c["beta"] * (1 - u.exp())
        one = torch.zeros_like(p)
        one[torch.arange(len(i), device=DEV), s["ids"][i]] = 1.0
        dl[i] = (w[i] * dlp / c["temperature"])[:, None] * (one - p)
    if not c["grad"]:
        return {"logp": at["logp"], "entropy": at["entropy"]}
    sums = torch.stack([(w * (at["policy"] + c["beta"] * at["kl"])).sum(), (w * at["policy"]).sum(), (w * at["kl"]).sum(), (w * at["cut"]).sum()])
    return {"sums": sums, "logp": at["logp"], "entropy": at["entropy"], "dlogits": dl}


def _value8(code, bits):
    """The value of a code with 3 exponent bits and `bits` of mantissa, in [0, 2)."""
    e, f = code >> bits, (code & (1 << bits) - 1).double() / (1 << bits)
    return torch.where(e > 0, (1 + f) * 2.0 ** (e.double() - 7), f * 2.0 ** -6)


def _round8(x, rnd, bits, top):
    """Blocks [n, 256] of magnitudes on the grid of their block's codes, rounded up or down by `rnd` (16 bits)."""
    amax = x.amax(1, keepdim=True)
    y = x * (top / amax.clamp(min=2.0 ** -100))
    grid = 2.0 ** (torch.floor(torch.log2(y.clamp(min=2.0 ** -20))).clamp(-6, 0) - bits)
    got = (torch.floor(y / grid + (rnd.double() + 0.5) / 65536) * grid).clamp(max=top) * (amax / top)
    return torch.where(amax < 2.0 ** -100, 0.0, got)


def _words(n, tensor, seed):
    """Philox4x32-10 of elements 0..n of a tensor."""
    c = torch.arange(-(-n // 4), device=DEV)
    a, b, d, e = c & M32, c >> 32, torch.full_like(c, tensor), torch.full_like(c, STEP)
    for r in range(10):
        ka, kb = (seed + r * 0x9E3779B9) & M32, ((seed >> 32) + r * 0xBB67AE85) & M32
        ha, hd = a * 0xD2511F53, d * 0xCD9E8D57
        a, b, d, e = ((hd >> 32) & M32) ^ b ^ ka, hd & M32, ((ha >> 32) & M32) ^ e ^ kb, ha & M32
    return torch.stack([a, b, d, e], 1).flatten()[:n]


def _exact_adamw(c, s):
    N = s["master"].numel()
    got = {k: torch.zeros(N, dtype=torch.float64, device=DEV) for k in ("master", "m", "v")}
    g_all = s["grad"].double()
    norm = torch.linalg.vector_norm(g_all) if c["clip"] else torch.zeros((), dtype=torch.float64, device=DEV)
    coef = min(1.0, c["clip"] / float(norm)) if c["clip"] else 1.0
    a = 0
    for t, n in enumerate(s["sizes"]):
        b = a + -(-n // BLOCK) * BLOCK
        g = g_all[a:b] * coef
        if c["state"] == 8:
            scale = lambda k: s[k][a // BLOCK:b // BLOCK].double().repeat_interleave(BLOCK)  # noqa: E731,B023
            code = s["m"][a:b].int()
            m = _value8(code & 127, 4) * scale("ms") * torch.where(code > 127, -1.0, 1.0)
            v = (_value8(s["v"][a:b].int(), 5) * scale("vs")).square()
        else:
            m, v = s["m"][a:b].double(), s["v"][a:b].double()
        m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
        lr = LR * float(s["lr_scale"][t])
        step = m / (1 - BETA1 ** STEP) / ((v / (1 - BETA2 ** STEP)).sqrt() + EPS)
        got["master"][a:b] = s["master"][a:b].double() * (1 - lr * 0.01) - lr * step
        if c["state"] == 8:
            w, root = _words(b - a, t, s["seed"]).view(-1, BLOCK), v.sqrt().view(-1, BLOCK)
            m = _round8(m.abs().view(-1, BLOCK), w & 0xFFFF, 4, QM).flatten() * torch.sign(m)
            r8, low = _round8(root, w >> 16, 5, QV), root.amax(1, keepdim=True) / QV * 2.0 ** -11
            v = torch.where((root > 0) & (r8.amax(1, keepdim=True) > 0), torch.maximum(r8, low), r8).square().flatten()
        got["m"][a:b], got["v"][a:b] = m, v
        a = b
    return {"param": got["master"] if s["param"] is not None else None, "master": got["master"], "m": got["m"], "v": got["v"], "norm": norm.view(1)}
