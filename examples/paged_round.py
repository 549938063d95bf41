"""Speculative decoding rounds with a paged cache, every part of a round on the GPU.

A toy target model (one attention layer, random weights) stands where a user's model would:
each round drafts a block, schedules its prefix, plans the rows the target has to run,
stores their keys and values, attends over the paged cache, applies the requests'
penalties and token mask to the target rows and verifies.  What is accepted advances
the requests' lengths; the pages of rejected rows are reused.  Nothing is read back
between rounds.  With `rotary` the model turns its queries and keys by their positions, with
`four_bits` the cache holds them in 4 bits; one call then rotates and stores.

    python examples/paged_round.py            # greedy, against decoding token by token
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import serving_draft_verify_gb300 as dsv  # noqa: E402


class Model:
    """Random weights: embedding, one attention layer with Hkv key heads, output head, and the drafter's."""

    def __init__(self, V=512, dim=64, Hq=8, Hkv=2, D=16, r=16, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def w(*shape, scale=1.0):
            return (torch.randn(shape, generator=g) * scale).to(device)

        self.V, self.dim, self.Hq, self.Hkv, self.D, self.r = V, dim, Hq, Hkv, D, r
        self.emb = w(V, dim)
        self.qkv = w(dim, (Hq + 2 * Hkv) * D, scale=dim ** -0.5)
        self.out = w(Hq * D, dim, scale=(Hq * D) ** -0.5)
        self.head = w(dim, V, scale=2 * dim ** -0.5)
        self.W1, self.W2 = w(V, r, scale=0.05), w(V, r, scale=0.05)
        self.conf = w(dim + r, scale=0.05)


class Rounds:
    """The serving state of B requests and the calls of one round, in order."""

    def __init__(self, model, prompts, gamma=4, page=8, blocks=256, room=None, repetition=1.3, presence=0.4,
                 banned=(), max_new=64, rotary=False, four_bits=False):
        self.m, self.B, self.gamma, self.page = model, len(prompts), gamma, page
        dev, B = model.emb.device, self.B
        self.room = room or B * (gamma + 1)
        i32 = dict(dtype=torch.int32, device=dev)
        width = max(len(p) for p in prompts) + max_new + gamma + 2
        self.history = torch.zeros((B, width), **i32)
        for b, p in enumerate(prompts):
            self.history[b, :len(p)] = torch.tensor(p, **i32)
        self.prompt_len = torch.tensor([len(p) for p in prompts], **i32)
        self.history_len = self.prompt_len.clone()
        self.length = torch.zeros(B, **i32)              # rows in the cache
        self.held = torch.zeros(B, **i32)
        self.advance = torch.zeros(B, **i32)             # rows of the last step that stay
        self.free_state = torch.tensor([0, blocks], **i32)
        self.free_ring = torch.arange(blocks, **i32)
        self.table = torch.zeros((B, -(-width // page)), **i32)
        self.freq = dsv.dspark_rotary_frequencies(model.D, device=dev)[0] if rotary else None
        self.scales = {}
        if four_bits:
            self.k_cache, self.v_cache = (dsv.kv4_cache(blocks, model.Hkv, page, model.D, dev) for _ in range(2))
            # a head's scale: its values' largest, here a few, over what a code and a block's scale reach
            self.scales = {k: torch.full((model.Hkv,), 0.002, device=dev) for k in ("k_scale", "v_scale")}
        else:
            shape = (blocks, model.Hkv, page, model.D)
            self.k_cache, self.v_cache = torch.zeros(shape, device=dev), torch.zeros(shape, device=dev)
        self.repetition = torch.full((B,), repetition, device=dev)
        self.presence = torch.full((B,), presence, device=dev)
        allowed = torch.ones(-(-model.V // 32) * 32, dtype=torch.bool)
        allowed[list(banned)] = False
        bits = (allowed.view(-1, 32).long() << torch.arange(32)).sum(1)
        self.mask = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32)[None].to(dev)
        self.mask_row = torch.zeros((B, gamma + 1), **i32)
        self.sps = (torch.arange(B * (gamma + 1) + 1, dtype=torch.float64) / 20).to(dev)
        self.positions = torch.arange(gamma + 1, device=dev)

    # -- the target over planned rows: hidden rows [rows, dim] of `tokens` [rows]
    def target(self, plan, tokens, most):
        m = self.m
        x = m.emb[tokens.clamp(min=0).long()]
        qkv = (x @ m.qkv).view(-1, m.Hq + 2 * m.Hkv, m.D)
        q, k, v = qkv[:, :m.Hq], qkv[:, m.Hq:m.Hq + m.Hkv], qkv[:, m.Hq + m.Hkv:]
        if self.freq is not None:
            q = dsv.dspark_rotate_write_kv(q, k, v, plan["position"], self.freq, plan["slot"], self.k_cache, self.v_cache,
                                           out=q, **self.scales)
        else:
            dsv.dspark_write_kv(k, v, plan["slot"], self.k_cache, self.v_cache, **self.scales)
        o = torch.zeros((x.shape[0], m.Hq, m.D), device=x.device)
        dsv.dspark_paged_attention(q, plan["row_offset"], plan["length"], self.table, self.k_cache, self.v_cache, most,
                                   out=dict(out=o), **self.scales)
        return x + o.reshape(x.shape[0], -1) @ m.out

    def plan(self, rows, room):
        p = dsv.dspark_plan_rows(self.length, rows, self.held, self.free_state, self.free_ring, self.table, self.page,
                                 room, advance=self.advance)
        self.length, self.held, self.free_state = p["length"], p["held"], p["free_state"]
        return p

    def prefill(self):
        """The prompts' tokens but the last, which is the first round's anchor."""
        rows = self.prompt_len - 1
        room = int(rows.sum())                           # known to whoever admits the requests
        p = self.plan(rows.contiguous(), room)
        at = p["position"].clamp(min=0).long()
        tokens = self.history[p["row_request"].clamp(min=0).long(), at]
        self.target(p, tokens, max(1, int(rows.max())))
        self.advance = rows.contiguous()
        self.anchor = self.history.gather(1, (self.prompt_len - 1).long()[:, None])[:, 0].contiguous()

    def round(self, seed=0, temperature=0.0):
        """One round; returns tokens [B, gamma + 1] (accepted, then the emitted one) and how many count."""
        m, B, G = self.m, self.B, self.gamma
        # a stand-in for the drafter's backbone: the output head on the anchor's embedding
        x0 = m.emb[self.anchor.long()]
        U = (x0 @ m.head)[:, None].expand(B, G, m.V).contiguous()
        h = x0[:, None].expand(B, G, m.dim).contiguous()
        d = dsv.dspark_draft_block(U, h, m.W1, m.W2, m.conf, 2.0, self.anchor, temperature, seed)
        ell = dsv.dspark_schedule_prefix(d["a"], self.sps)["ell"]
        p = self.plan(ell + 1, self.room)
        # row i of a request: the anchor, then its draft
        block = torch.cat([self.anchor[:, None], d["x"]], 1)
        req = p["row_request"].clamp(min=0).long()
        place = (p["position"] - p["length"][req]).clamp(min=0, max=G).long()
        hidden = self.target(p, block[req, place], G + 1)
        logits = torch.zeros((B, G + 1, m.V), device=U.device)
        live = (p["row_request"] >= 0)[:, None]
        logits[req, place] = torch.where(live, hidden @ m.head, logits[req, place])
        t = dsv.dspark_adjust_logits(logits, self.history, self.prompt_len, self.history_len, draft=d["x"], ell=ell,
                                     repetition=self.repetition, presence=self.presence, mask_row=self.mask_row,
                                     mask=self.mask, out=logits)
        v = dsv.dspark_verify(t, U, m.W1, m.W2, self.anchor, d["x"], d["lse_d"], d["logp_d"], ell, temperature, seed)
        n = v["n_accept"]
        took = self.positions[None] < n[:, None]
        tokens = torch.where(took, torch.cat([d["x"], d["x"][:, :1]], 1), v["next_token"][:, None])
        count = n + 1
        where = self.history_len[:, None] + self.positions[None]
        keep = self.positions[None] <= n[:, None]
        where = torch.where(keep, where, torch.full_like(where, self.history.shape[1] - 1)).long()
        self.history.scatter_(1, where, torch.where(keep, tokens, torch.zeros_like(tokens)))
        self.history_len = self.history_len + count
        self.advance, self.anchor = count, v["next_token"]
        return tokens, count


def turned(x, freq):
    """Row n of x [rows, heads, D] turned by n freq, in float64."""
    a = torch.arange(x.shape[0], device=x.device)[:, None, None] * freq.double()
    x1, x2 = x.chunk(2, -1)
    return torch.cat([x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()], -1)


def token_by_token(model, prompts, steps, repetition=1.3, presence=0.4, banned=(), freq=None, stored=None):
    """The same greedy decoding without drafts, pages or the library, one request at a time; `stored` makes
    of rows of keys or values what a cache holds of them."""
    got = []
    for p in prompts:
        said, new = list(p), []
        for _ in range(steps):
            x = model.emb[torch.tensor(said, device=model.emb.device)].double()
            qkv = (x @ model.qkv.double()).view(len(said), -1, model.D)
            G = model.Hq // model.Hkv
            if freq is not None:
                qkv[:, :model.Hq + model.Hkv] = turned(qkv[:, :model.Hq + model.Hkv], freq)
            kv = (qkv[:, model.Hq:model.Hq + model.Hkv], qkv[:, model.Hq + model.Hkv:])
            k, v = ((stored(y) if stored else y).repeat_interleave(G, 1) for y in kv)
            s = torch.einsum("hd,khd->hk", qkv[-1, :model.Hq], k) * model.D ** -0.5
            o = torch.einsum("hk,khd->hd", s.softmax(-1), v).reshape(-1)
            y = (x[-1] + o @ model.out.double()) @ model.head.double()
            seen = torch.tensor(sorted(set(said)), device=y.device)
            y[seen] = torch.where(y[seen] > 0, y[seen] / repetition, y[seen] * repetition)
            if new:
                y[torch.tensor(sorted(set(new)), device=y.device)] -= presence
            if banned:
                y[torch.tensor(sorted(banned), device=y.device)] = float("-inf")
            t = int(y.argmax())
            said.append(t)
            new.append(t)
        got.append(new)
    return got


def main(rounds=12):
    model = Model()
    prompts = [[5, 17, 400, 3], [9], [100, 101, 102, 103, 104, 105, 106, 107, 108, 109], [7, 7, 7], [511, 0]]
    banned = (1, 2, 3, 77, 300)
    s = Rounds(model, prompts, banned=banned)
    s.prefill()
    total = 0
    for i in range(rounds):
        total = total + s.round(seed=i)[1]
    start, end = s.prompt_len.tolist(), s.history_len.tolist()
    got = [s.history[b, start[b]:end[b]].tolist() for b in range(len(prompts))]
    want = token_by_token(model, prompts, max(len(g) for g in got), banned=banned)
    for b, (g, w) in enumerate(zip(got, want)):
        assert g == w[:len(g)], (b, g, w)
    print(f"{rounds} rounds, {sum(map(len, got))} tokens of {len(prompts)} requests as decoded token by token; "
          f"{int(s.free_state[1])} pages free")
    return got


if __name__ == "__main__":
    main()
