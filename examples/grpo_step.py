"""GRPO on a toy model with the library's calls from end to end: a group of answers per prompt sampled over a shared prefix
cache, the policy loss with its gradient, the adapter's backward and its AdamW step with 8-bit states.

The model: an embedding, one attention block (NVFP4 + LoRA linears, noisy norms, no positions) and an NVFP4 + LoRA head.
Only the head's adapter learns.  The reward is the share of even tokens in an answer, so it starts near one half.

    python examples/grpo_step.py [steps]
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import nvfp4_weight_only_quantize_gb300 as q  # noqa: E402
from nvfp4_weight_only_quantize_gb300 import synth  # noqa: E402

HIDDEN, HEADS, KV_HEADS, HEAD_DIM, VOCAB, RANK = 512, 8, 2, 64, 256, 16
PROMPTS, GROUP, PROMPT_LEN, ANSWER_LEN = 4, 32, 96, 12
LORA_SCALE, EPS, CLIP_LOW, CLIP_HIGH, BETA, TEMPERATURE = 2.0, 1e-6, 0.2, 0.28, 0.01, 1.0
SIGMA_START, SIGMA_END, STAGES = 1e-2, 5e-4, 4


class Model:
    def __init__(self, seed):
        kv = KV_HEADS * HEAD_DIM
        self.embed = synth.activations(VOCAB, HIDDEN, seed, "cuda")
        self.gamma = [synth.norm_gamma(HIDDEN, seed + k, "cuda") for k in (1, 2)]
        self.linear = {}
        for k, (name, n) in enumerate([("q", HIDDEN), ("k", kv), ("v", kv), ("o", HIDDEN), ("head", VOCAB)]):
            codes, scales, ts = q.qerl_nvfp4_quantize(synth.weight(n, HIDDEN, seed + 10 + k, "cuda"))
            A = synth.lora_A(RANK, HIDDEN, seed + 20 + k, "cuda")
            B = torch.zeros(n, RANK, dtype=torch.bfloat16, device="cuda")  # LoRA starts as the base model
            self.linear[name] = (codes, scales, ts, A, B)

    def norm(self, h, which, sigma, step):
        return q.qerl_aqn_rmsnorm(h, self.gamma[which], EPS, sigma, 1, step, which)

    def qkv(self, h, sigma, step):
        return q.qerl_nvfp4_lora_linear_fwd_grouped(self.norm(h, 0, sigma, step), [self.linear[n] for n in "qkv"], LORA_SCALE)

    def after_attention(self, h, attn, sigma, step):
        """(the head's input, logits) of the tokens whose attention output is given."""
        h = q.qerl_residual_add(h, q.qerl_nvfp4_lora_linear_fwd(attn, *self.linear["o"], LORA_SCALE))
        x = self.norm(h, 1, sigma, step)
        return x, q.qerl_nvfp4_lora_linear_fwd(x, *self.linear["head"], LORA_SCALE)


def rollout(model, prompts, sigma, step, gen):
    """GROUP answers for every prompt: (tokens [B, T], the head's inputs [B, T, H], log-probabilities [B, T])."""
    B = PROMPTS * GROUP
    cache = lambda n, t: torch.empty(n, t, KV_HEADS, HEAD_DIM, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    kp, vp, ks, vs = cache(PROMPTS, PROMPT_LEN), cache(PROMPTS, PROMPT_LEN), cache(B, ANSWER_LEN), cache(B, ANSWER_LEN)
    # the prompts' keys and values once, for all answers
    _, k, v = model.qkv(model.embed[prompts.flatten()], sigma, step)
    kp.copy_(k.view(kp.shape))
    vp.copy_(v.view(vp.shape))
    attention = q.PrefixAttention(kp, vp, ks, vs, q_heads=HEADS)
    tok = prompts[:, -1].repeat_interleave(GROUP)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    tokens, inputs, logps = [], [], []
    for t in range(ANSWER_LEN):
        h = model.embed[tok]
        qh, k, v = model.qkv(h, sigma, step)
        ks[:, t] = k.view(B, KV_HEADS, HEAD_DIM)
        vs[:, t] = v.view(B, KV_HEADS, HEAD_DIM)
        lens += 1
        attn = attention.run(qh.view(B, 1, HEADS, HEAD_DIM), lens)
        x, logits = model.after_attention(h, attn.view(B, HIDDEN), sigma, step)
        tok = torch.multinomial(torch.softmax(logits.float() / TEMPERATURE, -1), 1, generator=gen)[:, 0]
        logp, _ = q.qerl_token_logp(logits, tok, temperature=TEMPERATURE)
        tokens.append(tok)
        inputs.append(x)
        logps.append(logp)
    return torch.stack(tokens, 1), torch.stack(inputs, 1), torch.stack(logps, 1)


def train(steps=12, seed=0, epochs=2, log=print):
    """Rewards of the steps' rollouts."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = Model(seed)
    codes, scales, ts, A, Bm = model.linear["head"]
    grads = [torch.zeros(t.shape, device="cuda") for t in (A, Bm)]
    opt = q.AdamW([A, Bm], grads, masters=[A.float(), Bm.float()], state_bits=8, weight_decay=0.0, lr_scale=[1.0, 4.0])
    norm = torch.zeros(1, device="cuda")
    prompts = torch.randint(VOCAB, (PROMPTS, PROMPT_LEN), generator=gen, device="cuda")
    rewards, updates = [], 0
    ref_B = torch.zeros_like(Bm)  # the reference policy: the adapter as it was
    for step in range(steps):
        sigma = q.qerl_aqn_sigma(step, steps, SIGMA_START, SIGMA_END, STAGES)
        tokens, x, old = rollout(model, prompts, sigma, step, gen)
        reward = (tokens % 2 == 0).float().mean(1)
        grouped = reward.view(PROMPTS, GROUP)
        adv = ((grouped - grouped.mean(1, keepdim=True)) / (grouped.std(1, keepdim=True) + 1e-4)).view(-1, 1)
        T = tokens.numel()
        x, ids, old = x.view(T, HIDDEN), tokens.view(T), old.reshape(T)
        adv = adv.expand(-1, ANSWER_LEN).reshape(T).contiguous()
        weight = torch.full((T,), 1.0 / T, device="cuda")
        ref, _ = q.qerl_token_logp(q.qerl_nvfp4_lora_linear_fwd(x, codes, scales, ts, A, ref_B, LORA_SCALE), ids, temperature=TEMPERATURE)
        for _ in range(epochs):
            logits = q.qerl_nvfp4_lora_linear_fwd(x, codes, scales, ts, A, Bm, LORA_SCALE)
            sums, _, entropy, dlogits = q.qerl_policy_loss(logits, ids, old, adv, weight, ref_logp=ref, clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                                                           beta=BETA, temperature=TEMPERATURE, dlogits=logits)  # in place
            q.qerl_nvfp4_lora_linear_bwd(dlogits, x, codes, scales, ts, A, Bm, LORA_SCALE, dA=grads[0], dB=grads[1], want=())
            updates += 1
            opt.step(5e-3, updates, seed=seed, max_grad_norm=1.0, grad_norm=norm)
        rewards.append(float(reward.mean()))
        loss, _, kl, clipped = sums.tolist()
        log(f"step {step:2d}  reward {rewards[-1]:.3f}  loss {loss:+.4f}  kl {kl:.4f}  clipped {clipped:.3f}  "
            f"entropy {float(entropy.mean()):.3f}  |grad| {float(norm):.3f}  sigma {sigma:.4f}")
    assert q.get_error() == 0
    return rewards


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 12)
