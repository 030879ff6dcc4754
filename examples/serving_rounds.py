"""Draft -> schedule -> verify rounds around a paged key/value cache, on a small random model.

The target is one attention layer: x = E[token] + P[position], q, k, v = x Wq, x Wk, x Wv, hidden =
E[token] + attention Wo, logits = hidden LM. The drafter is its Markov part: W1 = E and W2 = LM over base logits of
zero, so that drafts are often, not always, what the target takes. All requests share a prefix (a system
prompt), whose keys and values are in the cache once.

  prefill  page_plan -> kv_append for the shared prefix, then page_plan -> kv_append -> prefix_attention -> lm_head for
           every request's prompt, and sample for its first token
  round    draft_sequential, schedule; then for the anchor and the scheduled drafts of all requests page_plan ->
           kv_append -> prefix_attention -> lm_head -> truncate, and verify on the truncated rows. Accepted
           tokens stay in the cache, the pages behind the last one go back to the free list.

Run it with a GPU:  python examples/serving_rounds.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_draft_seq_gb300 import dspark  # noqa: E402

BF16, I32, I64, F32, F64 = torch.bfloat16, torch.int32, torch.int64, torch.float32, torch.float64


class Model:
    """Random weights; small enough that a test can follow every token on the host."""

    def __init__(self, V=1000, d=64, Hq=8, Hkv=2, D=64, positions=4096, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def w(*shape, sd):
            return (torch.randn(*shape, generator=g) * sd).to(BF16).to(device)

        self.V, self.d, self.Hq, self.Hkv, self.D, self.device = V, d, Hq, Hkv, D, device
        self.E, self.P = w(V, d, sd=0.7), w(positions, d, sd=0.1)
        self.Wq, self.Wk, self.Wv = w(d, Hq * D, sd=0.1), w(d, Hkv * D, sd=0.1), w(d, Hkv * D, sd=0.3)
        self.Wo, self.LM = w(Hq * D, d, sd=0.05), w(d, V, sd=0.5)

    def qkv(self, tokens, positions):
        x = self.E[tokens] + self.P[positions]
        return ((x @ self.Wq).view(-1, self.Hq, self.D), (x @ self.Wk).view(-1, self.Hkv, self.D),
                (x @ self.Wv).view(-1, self.Hkv, self.D))

    def hidden(self, tokens, attention):
        return self.E[tokens] + attention.view(len(tokens), -1) @ self.Wo


class Server:
    """Requests of one model over one paged cache. `rule`: (temperature, top_k, top_p, min_p) of all requests."""

    def __init__(self, model, prefix, prompts, rule=(1.0, 20, 0.95, 0.02), gamma=4, page=16, new_tokens=64, seed=1):
        m, dev = model, model.device
        self.m, self.gamma, self.page, self.R, self.seed, self.rounds = m, gamma, page, len(prompts), seed, 0
        self.max_pages = -(-(max(map(len, prompts)) + new_tokens + 2 * gamma + 2) // page)
        n_pages = -(-len(prefix) // page) + self.R * self.max_pages
        self.k_cache = torch.zeros((n_pages, page, m.Hkv, m.D), dtype=BF16, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        # pages in an order of their own: nothing needs them to be neighbours
        self.free = list(np.random.default_rng(seed).permutation(n_pages))
        self.table = torch.full((self.R, self.max_pages), -1, dtype=I32, device=dev)
        self.cached = torch.zeros(self.R, dtype=I32, device=dev)
        self.prefix_len = len(prefix)
        self.prefix_pages = torch.full((1, -(-len(prefix) // page)), -1, dtype=I32, device=dev)

        most = max(self.R * (gamma + 1), sum(map(len, prompts)))
        self.ws = dspark.new_workspace(self.R, gamma, m.V, m.d, dspark.BF16, self.R * (gamma + 1), dev)
        self.attn_ws = dspark.new_attention_workspace(self.R, most, m.Hq, m.Hkv, m.D, dev)
        self.out = dspark.RoundOutputs(self.R, gamma, dev)
        self.base = torch.zeros((self.R, gamma, m.V), dtype=BF16, device=dev)
        self.conf = torch.full((self.R, gamma), 0.8, dtype=F32, device=dev)
        B = torch.arange(1, self.R * (gamma + 1) + 1, dtype=F32)
        self.sps = (1.0 / (1.0 + B / (4.0 * self.R))).to(dev)  # steps a second at B verified tokens

        # the shared prefix: planned like a request, its pages kept as the prefix's
        if prefix:
            plan, _ = self.plan(self.prefix_pages, torch.zeros(1, dtype=I32, device=dev), [len(prefix)])
            _, k, v = m.qkv(torch.tensor(prefix, dtype=I64, device=dev), plan["positions"].long())
            dspark.kv_append(k, v, plan["slots"], self.k_cache, self.v_cache, self.ws)

        tokens = torch.tensor([t for p in prompts for t in p], dtype=I64, device=dev)
        logits, plan = self.target(tokens, [len(p) for p in prompts])
        last = logits[plan["q_start"][1:].long() - 1].contiguous()
        self.anchor = torch.empty(self.R, dtype=I32, device=dev)
        u = torch.from_numpy(np.random.default_rng(seed + 1).random(self.R)).to(dev)
        dspark.sample(last, *self.rule_rows(rule, self.R), u, self.anchor, self.ws)
        self.cached += torch.tensor([len(p) for p in prompts], dtype=I32, device=dev)
        self.rule = rule
        self.emitted = [[int(t)] for t in self.anchor.cpu()]
        self.check()

    def rule_rows(self, rule, n):
        dev = self.m.device
        return tuple(torch.full((n,), x, dtype=t, device=dev) for x, t in zip(rule, (F32, I32, F32, F32)))

    def check(self):
        for ws in (self.ws, self.attn_ws):
            status = dspark.device_status(ws)
            if status != dspark.OK:
                raise RuntimeError(dspark.status_string(status))

    def plan(self, table, cached, new):
        """Pages and slots of `new` tokens a request (a device tensor, or a list of known lengths)."""
        dev, R = self.m.device, table.shape[0]
        known = not torch.is_tensor(new)
        capacity = sum(new) if known else self.R * (self.gamma + 1)
        new = torch.tensor(new, dtype=I32, device=dev) if known else new
        free = torch.tensor(self.free, dtype=I32, device=dev)
        p = {"q_start": torch.empty(R + 1, dtype=I32, device=dev), "kv_len": torch.empty(R, dtype=I32, device=dev),
             "positions": torch.empty(capacity, dtype=I32, device=dev),
             "slots": torch.empty(capacity, dtype=I64, device=dev)}
        used = torch.empty(1, dtype=I32, device=dev)
        dspark.page_plan(cached, new, free, self.page, table, p["q_start"], p["kv_len"], p["positions"], p["slots"], used,
                         self.ws)
        self.free = self.free[int(used):]
        return p, new

    def target(self, tokens, new):
        """Logits of the new tokens (packed), their keys and values into the cache. `tokens` may be a function of
        the plan."""
        m = self.m
        plan, new = self.plan(self.table, self.cached, new)
        tokens = tokens(plan) if callable(tokens) else tokens
        positions = plan["positions"].long().clamp_min(0) + self.prefix_len
        q, k, v = m.qkv(tokens, positions)
        dspark.kv_append(k, v, plan["slots"], self.k_cache, self.v_cache, self.ws)
        out = torch.zeros_like(q)  # tokens past the plan's have no row of their own
        dspark.prefix_attention(q, self.k_cache, self.v_cache, self.prefix_pages[0], self.prefix_len, self.table,
                                plan["q_start"], plan["kv_len"], m.D ** -0.5, out, self.attn_ws)
        logits = torch.empty((len(tokens), m.V), dtype=BF16, device=m.device)
        dspark.lm_head(m.hidden(tokens, out), m.LM, logits, self.ws)
        return logits, plan

    def round(self):
        m, R, n, o, dev = self.m, self.R, self.gamma + 1, self.out, self.m.device
        T = self.rule[0]
        seed = self.seed + (self.rounds << 32)
        dspark.draft_sequential(self.base, self.anchor, m.E, m.LM, T, seed, o.tokens, o.q_tok, o.q_stats, self.ws)
        dspark.schedule(self.conf, None, self.sps, 0, o.sched_len, o.K, o.tau_theta, self.ws)

        block = torch.cat([self.anchor[:, None], o.tokens], dim=1).long()  # [R, gamma + 1]
        place = {}

        def packed(plan):  # token i of request r stands at q_start[r] + i; the rows past the last one repeat it
            t = torch.arange(R * n, device=dev)
            r = torch.searchsorted(plan["q_start"][1:].long(), t, right=True).clamp_max(R - 1)
            i = (t - plan["q_start"][r].long()).clamp_max(self.gamma)
            place["row"] = torch.where(plan["positions"] >= 0, r * n + i, R * n)
            return block[r, i]

        before = self.cached
        logits, plan = self.target(packed, o.sched_len + 1)
        dspark.truncate(logits, *self.rule_rows(self.rule, R * n), logits, self.ws)
        rows = torch.zeros((R * n + 1, m.V), dtype=BF16, device=dev)  # [R, gamma + 1] and one for the rows past T
        rows[place["row"]] = logits
        dspark.verify(rows[:R * n].view(R, n, m.V), self.base, self.anchor, m.E, m.LM, o.tokens, o.q_tok, o.q_stats,
                      o.sched_len, T, seed, o.out_tokens, o.accepted_len, o.p_tok, self.ws)

        # accepted drafts and the anchor stay; the corrected or bonus token is the next anchor
        a = o.accepted_len.long()
        self.anchor = o.out_tokens.gather(1, a[:, None])[:, 0].contiguous()
        self.cached = before + o.accepted_len + 1
        self.rounds += 1
        self.check()
        keep, held = (-(-x.cpu().numpy() // self.page) for x in (self.cached, plan["kv_len"]))
        table, out, acc = self.table.cpu().numpy(), o.out_tokens.cpu().numpy(), a.cpu().numpy()
        for r in range(R):
            self.free.extend(int(x) for x in table[r, keep[r]:held[r]])
            self.emitted[r].extend(int(x) for x in out[r, :acc[r] + 1])
        return acc


def main():
    model = Model()
    rng = np.random.default_rng(5)
    prefix = [int(t) for t in rng.integers(0, model.V, 200)]
    prompts = [[int(t) for t in rng.integers(0, model.V, 3 + 5 * r)] for r in range(8)]
    server = Server(model, prefix, prompts)
    accepted = [server.round() for _ in range(10)]
    print(f"{len(prompts)} requests, {len(accepted)} rounds: {np.mean(accepted):.2f} of {server.gamma} drafts accepted "
          f"a round, {sum(map(len, server.emitted))} tokens, {len(server.free)} pages free")
    for r, tokens in enumerate(server.emitted[:3]):
        print(f"request {r}: {tokens}")


if __name__ == "__main__":
    main()
