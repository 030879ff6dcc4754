"""Rounds with a drafter that has no distribution: tokens looked up in what a request has produced, several samples of each
prompt over shared pages, every length, page and token on the device; and a Markov drafter taught by the target's rows.

The target is the one of serving_rounds.py. The prompts enter the cache once; page_fork gives each its samples, which share
the prompt's full pages and copy the one that they write next.

  round    lookup -> page_collect (the free list) -> page_plan -> kv_append -> prefix_attention -> lm_head -> truncate ->
           probabilities -> verify_probs. Rejected tokens leave by the lengths alone: the next page_collect finds their pages.
  compact  page_compact -> page_copy: what is held moves to the front of the cache
  teach    the drafter's logits W[previous token] LM against the target's largest ones: distill gives the divergence and
           its gradient, and W a step down it

Run it with a GPU:  python examples/lookup_rounds.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from serving_rounds import Model  # noqa: E402
from speculative_decoding_draft_seq_gb300 import dspark  # noqa: E402

BF16, I32, I64, F32, F64 = torch.bfloat16, torch.int32, torch.int64, torch.float32, torch.float64


class Samples:
    """`samples` continuations of each prompt. `rule`: (temperature, top_k, top_p, min_p) of all rows, or one of each a row."""

    def __init__(self, model, prefix, prompts, samples=3, rule=(0.0, 0, 1.0, 0.0), gamma=4, page=16, new_tokens=64, seed=1):
        m, dev = model, model.device
        self.m, self.gamma, self.page, self.R = m, gamma, page, len(prompts) * samples
        R = self.R
        longest = max(map(len, prompts)) + new_tokens + 2 * gamma + 2
        width = -(-longest // page)
        self.n_pages = -(-len(prefix) // page) + (R + len(prompts)) * width
        self.prefix_len = len(prefix)
        self.uniforms = np.random.default_rng(seed)
        i32 = lambda *shape: torch.empty(shape, dtype=I32, device=dev)  # noqa: E731
        self.k, self.v = (torch.zeros((self.n_pages, page, m.Hkv, m.D), dtype=BF16, device=dev) for _ in range(2))
        most = max(R * (gamma + 1), sum(map(len, prompts)), len(prefix))
        self.ws = dspark.new_page_workspace(self.n_pages, dev)
        self.attn_ws = dspark.new_attention_workspace(R, most, m.Hq, m.Hkv, m.D, dev)
        self.refs, self.free, self.n_free = i32(self.n_pages), i32(self.n_pages), i32(1)
        self.pinned = i32(0)
        rows = [torch.as_tensor(x).expand(R) if np.ndim(x) == 0 else torch.tensor(x) for x in rule]
        self.rule = tuple(x.to(t).contiguous().to(dev) for x, t in zip(rows, (F32, I32, F32, F32)))

        # the shared prefix, then the prompts, each planned like rows of their own
        if prefix:
            table = torch.full((1, -(-len(prefix) // page)), -1, dtype=I32, device=dev)
            plan, _ = self.plan(table, torch.zeros(1, dtype=I32, device=dev), torch.tensor([len(prefix)], dtype=I32, device=dev),
                                len(prefix))
            _, k, v = m.qkv(torch.tensor(prefix, dtype=I64, device=dev), plan["positions"].long())
            dspark.kv_append(k, v, plan["slots"], self.k, self.v, self.ws)
            self.pinned = table[0].contiguous()
        P = len(prompts)
        table = torch.full((P, width), -1, dtype=I32, device=dev)
        length = torch.tensor([len(p) for p in prompts], dtype=I32, device=dev)
        tokens = torch.tensor([t for p in prompts for t in p], dtype=I64, device=dev)
        logits, plan = self.target(table, torch.zeros(P, dtype=I32, device=dev), length, len(tokens), lambda plan: tokens)

        # samples of each prompt
        parent = torch.arange(P, device=dev, dtype=I32).repeat_interleave(samples)
        self.collect(table, length)
        self.table, self.cached = i32(R, width), i32(R)
        src, dst, count, used = i32(R), i32(R), i32(R), i32(1)
        dspark.page_fork(table, length, parent, None, page, self.n_pages, self.free, self.table, self.cached, src, dst, count, used,
                         self.ws, pinned=self.pinned)
        dspark.page_copy(src, dst, self.k, self.v, self.ws, tokens=count)
        last = logits[plan["q_start"][1:].long() - 1][parent.long()].contiguous()
        self.anchor = i32(R)
        dspark.sample(last, *self.rule, self.random(R), self.anchor, self.ws)
        # what each row has produced so far: prompt, tokens, -1
        self.history = torch.full((R, longest), -1, dtype=I64, device=dev)
        for r in range(R):
            p = prompts[r // samples]
            self.history[r, :len(p)] = torch.tensor(p, dtype=I64, device=dev)
        self.length = self.cached.long()
        self.history.scatter_(1, self.length[:, None], self.anchor.long()[:, None])
        self.first = self.cached.clone()
        self.check()

    def random(self, *shape):
        return torch.from_numpy(self.uniforms.random(shape)).to(self.m.device)

    def check(self):
        for ws in (self.ws, self.attn_ws):
            status = dspark.device_status(ws)
            if status != dspark.OK:
                raise RuntimeError(dspark.status_string(status))

    def collect(self, table, length):
        dspark.page_collect(table, length, self.page, self.refs, self.free, self.n_free, self.ws, pinned=self.pinned)

    def plan(self, table, cached, new, capacity):
        """Pages and slots of `new` tokens a row, the free list formed from what the rows hold now."""
        dev, R = self.m.device, table.shape[0]
        self.collect(table, cached)
        p = {"q_start": torch.empty(R + 1, dtype=I32, device=dev), "kv_len": torch.empty(R, dtype=I32, device=dev),
             "positions": torch.empty(capacity, dtype=I32, device=dev), "slots": torch.empty(capacity, dtype=I64, device=dev)}
        dspark.page_plan(cached, new, self.free, self.page, table, p["q_start"], p["kv_len"], p["positions"], p["slots"],
                         torch.empty(1, dtype=I32, device=dev), self.ws)
        return p, new

    def target(self, table, cached, new, capacity, tokens):
        """Logits of the new tokens, packed, their keys and values into the cache; tokens(plan) gives them."""
        m = self.m
        plan, new = self.plan(table, cached, new, capacity)
        tokens = tokens(plan)
        q, k, v = m.qkv(tokens, plan["positions"].long().clamp_min(0) + self.prefix_len)
        dspark.kv_append(k, v, plan["slots"], self.k, self.v, self.ws)
        out = torch.zeros_like(q)
        dspark.prefix_attention(q, self.k, self.v, self.pinned, self.prefix_len, table, plan["q_start"], plan["kv_len"],
                                m.D ** -0.5, out, self.attn_ws)
        logits = torch.empty((len(tokens), m.V), dtype=BF16, device=m.device)
        dspark.lm_head(m.hidden(tokens, out), m.LM, logits, self.ws)
        return logits, plan

    def lookup(self):
        """(drafts [R, gamma], their number): what followed the anchor's last earlier occurrence in the row."""
        at = torch.arange(self.history.shape[1], device=self.m.device)
        seen = (self.history == self.anchor.long()[:, None]) & (at < self.length[:, None])
        found = torch.where(seen, at, -1).amax(-1)
        index = found[:, None] + 1 + torch.arange(self.gamma, device=self.m.device)
        drafts = self.history.gather(1, index.clamp_max(self.history.shape[1] - 1))
        n = torch.where(found >= 0, (self.length + 1 - found - 1).clamp_max(self.gamma), torch.zeros_like(found))
        return drafts.clamp_min(0).int(), n.int()

    def round(self):
        m, R, g, dev = self.m, self.R, self.gamma, self.m.device
        drafts, n = self.lookup()
        block = torch.cat([self.anchor[:, None], drafts], 1).long()
        place = {}

        def packed(plan):  # token i of row r stands at q_start[r] + i
            t = torch.arange(R * (g + 1), device=dev)
            r = torch.searchsorted(plan["q_start"][1:].long(), t, right=True).clamp_max(R - 1)
            place["row"] = r
            return block[r, (t - plan["q_start"][r].long()).clamp_max(g)]

        logits, plan = self.target(self.table, self.cached, n + 1, R * (g + 1), packed)
        rule = [x[place["row"]].contiguous() for x in self.rule]
        dspark.truncate(logits, *rule, logits, self.ws)
        probs = torch.empty(logits.shape, dtype=F32, device=dev)
        dspark.probabilities(logits, rule[0], probs, self.ws)
        out = torch.empty((R, g + 1), dtype=I32, device=dev)
        accepted = torch.empty(R, dtype=I32, device=dev)
        p_tok = torch.empty((R, g), dtype=F32, device=dev)
        dspark.verify_probs(probs, plan["q_start"], None, drafts, self.random(R, g + 1), out, accepted, p_tok, self.ws)
        # the anchor and the accepted tokens stay in the cache; the new token is the next anchor
        i = torch.arange(g + 1, device=dev)
        keep = i <= accepted[:, None]
        at = (self.length[:, None] + 1 + i).clamp_max(self.history.shape[1] - 1)
        self.history.scatter_(1, at, torch.where(keep, out.long(), self.history.gather(1, at)))
        self.length = self.length + 1 + accepted.long()
        self.anchor = out.gather(1, accepted.long()[:, None])[:, 0].contiguous()
        self.cached = self.cached + accepted + 1
        return accepted

    def compact(self):
        dev, half = self.m.device, self.n_pages // 2
        src, dst = (torch.empty(half, dtype=I32, device=dev) for _ in range(2))
        n_live = torch.empty(1, dtype=I32, device=dev)
        dspark.page_compact(self.table, self.cached, self.page, self.n_pages, self.table, src, dst, n_live, self.ws, pinned=self.pinned,
                            new_pinned=self.pinned)
        dspark.page_copy(src, dst, self.k, self.v, self.ws)
        return n_live

    def emitted(self):
        first, end, history = self.first.tolist(), (self.length + 1).tolist(), self.history.cpu()
        return [history[r, first[r]:end[r]].tolist() for r in range(self.R)]


def teach(W, LM, previous, target_logits, temperature=1.0, top=32, lr=0.0):
    """Divergence of the Markov drafter W [V, d] (logits W[previous] LM) from the target's `top` largest logits of each
    row, with their whole sum, and its gradient for W; a step of size lr down it."""
    logits = W[previous] @ LM
    teacher, ids = torch.topk(target_logits.float(), top)
    lse = torch.logsumexp(target_logits.float() / temperature, -1)
    N = len(previous)
    loss, grad = torch.empty(N, dtype=F32, device=W.device), torch.empty_like(logits)
    weight = torch.full((N,), 1.0 / N, dtype=F32, device=W.device)
    ws = dspark.new_workspace(1, 1, 1, 1, dspark.FP32, 1, W.device)
    dspark.distill(logits, ids.int(), teacher, temperature, loss, ws, grad=grad, weight=weight, teacher_lse=lse)
    if dspark.device_status(ws) != dspark.OK:
        raise RuntimeError(dspark.status_string(dspark.device_status(ws)))
    dW = torch.zeros(W.shape, dtype=F32, device=W.device).index_add_(0, previous, (grad @ LM.t()).float())
    if lr:
        W -= (lr * dW).to(W.dtype)
    return loss.mean(), dW


def main():
    m = Model()
    rng = np.random.default_rng(5)
    prefix = [int(t) for t in rng.integers(0, m.V, 100)]
    prompts = [[int(t) for t in rng.integers(0, 40, 20 + 7 * r)] for r in range(4)]
    s = Samples(m, prefix, prompts, samples=3, rule=(0.8, 20, 0.95, 0.0))
    accepted = torch.stack([s.round() for _ in range(12)])
    live = s.compact()
    accepted2 = torch.stack([s.round() for _ in range(4)])
    s.check()
    print(f"{s.R} samples of {len(prompts)} prompts, {len(accepted) + len(accepted2)} rounds: {accepted.float().mean():.2f} looked-up "
          f"tokens accepted a round; {int(live)} of {s.n_pages} pages held when the cache was compacted")
    for r in range(3):
        print(f"sample {r}: {s.emitted()[r]}")
    W = m.E.float()
    previous = torch.from_numpy(rng.integers(0, m.V, 256)).to(m.device)
    target = (m.hidden(previous, torch.zeros(256, m.Hq * m.D, dtype=BF16, device=m.device)) @ m.LM).float()
    losses = [float(teach(W, m.LM.float(), previous, target * 1.2, lr=20.0)[0]) for _ in range(5)]
    print("divergence of the Markov drafter from the target's rows: " + " ".join(f"{x:.4f}" for x in losses))


if __name__ == "__main__":
    main()
