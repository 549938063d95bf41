"""Cases of the target model's side of a decoding round, measured one operator at a time.

Between the draft and the verification of a round the target model runs over the
scheduled rows of every request.  Four operators of that step are measured here:

  plan    dspark_plan_rows: pages, positions and cache slots of the rows a step adds
  write   dspark_write_kv: the rows' keys and values into the paged cache
  attend  dspark_paged_attention: the rows' attention over the paged cache
  adjust  dspark_adjust_logits: penalties, biases and grammar masks on the target rows

With `own` false, run() computes an operator from elementary torch operations in
32 bits (the plain form); with `own` true it calls the library.
"""
import random

import torch

own = False

VOCAB = 151936          # the vocabulary of this repository's serving configurations
_BF16, _F32 = torch.bfloat16, torch.float32
_TYPES = {"bf16": _BF16, "f32": _F32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------- cases ---
def listed():
    return [
        # sixteen interactive requests, one verification step each: the call is all latency
        dict(name="plan 16 requests", op="plan", B=16, page=16, ctx=4096, rows=8, finish=0.0),
        # a loaded server: a thousand requests, a few finishing, some still reading their prompts
        dict(name="plan 1024 requests", op="plan", B=1024, page=16, ctx=8192, rows=256, finish=0.02),
        # one row for each of sixteen requests
        dict(name="write 16 rows", op="write", N=16, Hkv=8, D=128, page=16, dtype="bf16", cache="bf16", fused=True),
        # prompts being read in, stored in 8 bits; the keys are slices of the fused projection
        dict(name="write 16384 rows e4m3", op="write", N=16384, Hkv=8, D=128, page=16, dtype="bf16", cache="e4m3",
             fused=True),
        # one interactive request, one new token
        dict(name="attend 1 request", op="attend", B=1, rows=1, ctx=1900, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", cache="bf16", window=0),
        # plain decoding of a full batch
        dict(name="attend 64 requests", op="attend", B=64, rows=1, ctx=16384, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", cache="bf16", window=0),
        # verification of up to sixteen drafted tokens and the bonus row
        dict(name="attend verify 17 rows", op="attend", B=128, rows=17, ctx=6000, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", cache="bf16", window=0),
        # verification of a block of seven in few, very long conversations on an 8-bit cache
        dict(name="attend long e4m3", op="attend", B=3, rows=8, ctx=131001, Hq=32, Hkv=8, D=128, page=32,
             dtype="bf16", cache="e4m3", window=0),
        # the checking type, an uncommon group of heads and a sliding window
        dict(name="attend f32 window", op="attend", B=9, rows=3, ctx=2500, Hq=28, Hkv=4, D=64, page=24,
             dtype="f32", cache="f32", window=1024),
        # one chat request with penalties and a grammar
        dict(name="adjust 1 row", op="adjust", B=1, R=1, V=VOCAB, dtype="bf16", history=900, bias=4, masks=1),
        # a verification step of 64 requests with everything on
        dict(name="adjust 64 requests f32", op="adjust", B=64, R=8, V=VOCAB, dtype="f32", history=8192, bias=32,
             masks=16),
        # a verification step of a loaded server
        dict(name="adjust 256 requests", op="adjust", B=256, R=17, V=VOCAB, dtype="bf16", history=4096, bias=8,
             masks=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["plan", "write", "attend", "attend", "attend", "adjust"])
    if op == "plan":
        return dict(op=op, B=_log_int(rng, 1, 2048), page=rng.choice([8, 16, 24, 32, 64]), ctx=_log_int(rng, 16, 8192),
                    rows=_log_int(rng, 1, 256), finish=rng.choice([0.0, 0.02, 0.2]))
    if op == "write":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, N=_log_int(rng, 1, 16384), Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 96, 128, 256]),
                    page=rng.choice([8, 16, 24, 32, 64]), dtype=dtype, cache=rng.choice([dtype, "e4m3"]),
                    fused=rng.random() < 0.5)
    if op == "adjust":
        R = _log_int(rng, 1, 17)
        V = rng.choice([VOCAB, 32000, 50264, 128256])
        return dict(op=op, B=_log_int(rng, 1, max(1, min(256, 256 * 17 // R))), R=R, V=V,
                    dtype=rng.choice(["bf16", "bf16", "f32"]) if R < 9 else "bf16", history=_log_int(rng, 1, 8192),
                    bias=rng.choice([0, 1, 8, 32]), masks=rng.choice([0, 1, 16]))
    cache = rng.choice(["bf16", "bf16", "bf16", "e4m3", "f32"])
    Hq, Hkv = rng.choice([(32, 8), (32, 8), (32, 4), (28, 4), (16, 16), (64, 8), (12, 1)])
    D = rng.choice([64, 128, 128, 96, 256])
    rows = rng.choice([1, 1, 2, 4, 5, 8, 17])
    B = _log_int(rng, 1, 256)
    # the padded cache stays below half of the largest listed one
    most = min(65536, (1 << 29) // (B * Hkv * D))
    if cache == "f32":
        most = min(most, (1 << 26) // (B * Hkv * D))
    ctx = _log_int(rng, 32, max(64, most))
    return dict(op=op, B=B, rows=rows, ctx=ctx, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 16, 24, 32, 64]),
                dtype="f32" if cache == "f32" else "bf16", cache=cache, window=rng.choice([0, 0, 0, 512]))


# ------------------------------------------------------------------ shapes ---
def _shape_rng(case):
    """Lengths belong to the case, so that its work is known; values belong to the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _plan_lengths(case):
    """Per request: rows held before the step's advance, advance, rows to add, pages held."""
    r, out = _shape_rng(case), []
    page = case["page"]
    for b in range(case["B"]):
        last = r.randint(1, 17)                       # rows of the last step, some rejected
        n = r.randint(0, max(0, case["ctx"] - last))
        adv = r.randint(1, last)
        held = -(-(n + last) // page)
        if r.random() < case["finish"]:
            n, adv, rows = 0, 0, 0                    # finished: every page goes back
        elif r.random() < 0.1:
            rows = r.randint(1, case["rows"])
        else:
            rows = r.randint(1, min(17, case["rows"]))
        out.append((n, adv, rows, held))
    return out


def _attend_lengths(case):
    """Per request: (keys before the step, rows of the step)."""
    r = _shape_rng(case)
    got = []
    for b in range(case["B"]):
        rows = r.randint(1, case["rows"]) if b else case["rows"]
        total = max(rows, r.randint(case["ctx"] // 8, case["ctx"]) if b else case["ctx"])
        got.append((total - rows, rows))
    return got


def _adjust_lengths(case):
    """Per request: (prompt tokens, history tokens, scheduled draft tokens)."""
    r = _shape_rng(case)
    got = []
    for b in range(case["B"]):
        h = r.randint(max(1, case["history"] // 4), case["history"]) if b else case["history"]
        got.append((r.randint(0, h), h, r.randint(0, case["R"] - 1) if b else case["R"] - 1))
    return got


def work(case):
    if case["op"] == "plan":
        new = sum(max(0, -(-(n + a + q) // case["page"]) - h) for n, a, q, h in _plan_lengths(case))
        back = sum(max(0, h - -(-(n + a + q) // case["page"])) for n, a, q, h in _plan_lengths(case))
        N = sum(q for _, _, q, _ in _plan_lengths(case))
        # per request: four numbers in, three out; per row: three out; per page that moves: one in, one out;
        # per row, the page it lies on comes from the table or the ring (rows of a page share it)
        return {"bytes": case["B"] * 28 + N * 16 + (new + back) * 8 + N * 4 // case["page"], "flops": 0}
    if case["op"] == "write":
        n = 2 * case["N"] * case["Hkv"] * case["D"]
        size = {"bf16": 2, "f32": 4, "e4m3": 1}
        return {"bytes": n * (size[case["dtype"]] + size[case["cache"]]) + 8 * case["N"], "flops": n}
    if case["op"] == "attend":
        size = {"bf16": 2, "f32": 4, "e4m3": 1}
        keys = pairs = rows = 0
        for n, q in _attend_lengths(case):
            seen = n + q
            if case["window"]:
                seen = min(seen, case["window"] + q - 1)
            keys += seen
            rows += q
            for i in range(q):
                pairs += min(n + i + 1, case["window"] or n + i + 1)
        D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
        return {"bytes": 2 * keys * Hkv * D * size[case["cache"]] + 2 * rows * Hq * D * size[case["dtype"]]
                + rows * Hq * 4 + keys // case["page"] * 4, "flops": 4 * pairs * Hq * D}
    rows = sum(e + 1 for _, _, e in _adjust_lengths(case))
    hist = sum(h for _, h, _ in _adjust_lengths(case))
    size = 2 if case["dtype"] == "bf16" else 4
    masked = rows // 2 if case["masks"] else 0
    return {"bytes": rows * case["V"] * 2 * size + hist * 4 + masked * (case["V"] // 8) + case["B"] * case["bias"] * 8,
            "flops": rows * case["V"]}


# ----------------------------------------------------------------- prepare ---
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _tables(case, g, pages):
    """Block tables over a shuffled pool: request b holds pages[b] pages."""
    total = sum(pages)
    cap = total + 64 + total // 8
    perm = torch.randperm(cap, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(pages))
    col = torch.arange(width, device="cuda")
    held = _ints(pages, torch.int64)
    first = held.cumsum(0) - held
    table = perm[(first[:, None] + col[None]).clamp(max=cap - 1)]
    return torch.where(col[None] < held[:, None], table, torch.zeros_like(table)).contiguous(), perm, total, cap


def _workspace(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def _prepare_plan(case, g):
    lens = _plan_lengths(case)
    B, page = case["B"], case["page"]
    held = [h for *_, h in lens]
    need = [-(-(n + a + q) // page) for n, a, q, _ in lens]
    _, perm, total, _ = _tables(case, g, held)
    taken = sum(max(0, n - h) for n, h in zip(need, held))
    cap = total + taken + 37
    perm = torch.randperm(cap, generator=g, device="cuda").to(torch.int32)
    width = max(max(held), max(need), 1) + 3
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    flat = perm[:total]
    rows = torch.repeat_interleave(torch.arange(B, device="cuda"), _ints(held, torch.int64))
    h64 = _ints(held, torch.int64)
    cols = torch.arange(total, device="cuda") - (h64.cumsum(0) - h64)[rows]
    table[rows, cols] = flat
    # the ring of free pages: its live part starts somewhere inside and wraps around
    at = int(torch.randint(0, cap, (1,), generator=g, device="cuda"))
    ring = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    free = cap - total
    ring[(torch.arange(free, device="cuda") + at) % cap] = perm[total:]
    N = sum(q for _, _, q, _ in lens)
    room = N + 5                                      # a little room, as for a captured step
    s = dict(B=B, page=page, room=room, table=table, ring=ring, length=_ints([n for n, *_ in lens]),
             advance=_ints([a for _, a, *_ in lens]), rows=_ints([q for _, _, q, _ in lens]), held=_ints(held),
             free=_ints([at, free]), ws=_workspace(1 << 16))
    s["out"] = dict(length=torch.empty(B, dtype=torch.int32, device="cuda"),
                    held=torch.empty(B, dtype=torch.int32, device="cuda"),
                    free_state=torch.empty(2, dtype=torch.int32, device="cuda"),
                    row_offset=torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                    row_request=torch.empty(room, dtype=torch.int32, device="cuda"),
                    position=torch.empty(room, dtype=torch.int32, device="cuda"),
                    slot=torch.empty(room, dtype=torch.int64, device="cuda"))
    return s


def _cache(case, g, blocks):
    shape = (blocks, case["Hkv"], case["page"], case["D"])
    t = _TYPES[case["cache"]]
    make = _F32 if t == _F32 else _BF16
    k = torch.randn(shape, generator=g, device="cuda", dtype=make)
    v = torch.randn(shape, generator=g, device="cuda", dtype=make)
    if case["cache"] != "e4m3":
        return k, v, None, None
    # stored values fill the range of the 8-bit type; the heads' scales bring them back
    ks = (torch.rand(case["Hkv"], generator=g, device="cuda") + 0.5) * 0.0125
    vs = (torch.rand(case["Hkv"], generator=g, device="cuda") + 0.5) * 0.0125
    return k.mul_(80).clamp_(-448, 448).to(t), v.mul_(80).clamp_(-448, 448).to(t), ks, vs


def _prepare_write(case, g):
    N, Hkv, D, page = case["N"], case["Hkv"], case["D"], case["page"]
    blocks = -(-N // page) + 8
    kc, vc, ks, vs = _cache(case, g, blocks)
    t = _TYPES[case["dtype"]]
    if case["fused"]:
        qkv = torch.randn((N, 6 * Hkv, D), generator=g, device="cuda", dtype=t)     # 4 query heads to a key head
        k, v = qkv[:, 4 * Hkv:5 * Hkv], qkv[:, 5 * Hkv:]
    else:
        k = torch.randn((N, Hkv, D), generator=g, device="cuda", dtype=t)
        v = torch.randn((N, Hkv, D), generator=g, device="cuda", dtype=t)
    # runs of rows on shuffled pages, the last rows of the padded step without a slot
    perm = torch.randperm(blocks, generator=g, device="cuda")
    i = torch.arange(N, device="cuda")
    slot = perm[i // page] * page + i % page
    if N > 8:
        slot[N - N // 16 - 1:] = -1
    return dict(k=k, v=v, slot=slot, kc=kc, vc=vc, ks=ks, vs=vs, ws=_workspace(4096))


def _prepare_attend(case, g):
    lens = _attend_lengths(case)
    page = case["page"]
    table, _, _, cap = _tables(case, g, [-(-(n + q) // page) for n, q in lens])
    kc, vc, ks, vs = _cache(case, g, cap)
    N = sum(q for _, q in lens)
    t = _TYPES[case["dtype"]]
    q = torch.randn((N, case["Hq"], case["D"]), generator=g, device="cuda", dtype=t) * 2
    offs = [0]
    for _, n in lens:
        offs.append(offs[-1] + n)
    return dict(q=q, offset=_ints(offs), length=_ints([n for n, _ in lens]), table=table, kc=kc, vc=vc, ks=ks, vs=vs,
                rows=case["rows"], most=max(n + q for n, q in lens), window=case["window"],
                ws=_workspace(192 << 20),
                out=dict(out=torch.empty_like(q), lse=torch.empty((N, case["Hq"]), dtype=_F32, device="cuda")))


def _prepare_adjust(case, g):
    B, R, V = case["B"], case["R"], case["V"]
    lens = _adjust_lengths(case)
    t = _TYPES[case["dtype"]]
    logits = torch.randn((B, R, V), generator=g, device="cuda", dtype=t) * 2
    width = case["history"]
    # text repeats itself: most tokens come from a small part of the vocabulary
    u = torch.rand((B, width), generator=g, device="cuda")
    history = (u.pow(4) * (V - 1)).to(torch.int32)
    draft = (torch.rand((B, max(1, R - 1)), generator=g, device="cuda").pow(4) * (V - 1)).to(torch.int32)
    s = dict(logits=logits, history=history, draft=draft[:, :R - 1].contiguous() if R > 1 else None,
             prompt=_ints([p for p, _, _ in lens]), length=_ints([h for _, h, _ in lens]),
             ell=_ints([e for *_, e in lens]),
             rep=1 + torch.rand(B, generator=g, device="cuda") * 0.5,
             freq=torch.rand(B, generator=g, device="cuda"), pres=torch.rand(B, generator=g, device="cuda"),
             bias_token=None, bias_value=None, mask_row=None, mask=None, ws=_workspace(4096),
             out=torch.zeros((B, R, V), dtype=t, device="cuda"))
    if case["bias"]:
        first = torch.randint(0, V // case["bias"], (B, 1), generator=g, device="cuda")
        s["bias_token"] = (first + torch.arange(case["bias"], device="cuda") * (V // case["bias"])).to(torch.int32)
        s["bias_value"] = torch.randn((B, case["bias"]), generator=g, device="cuda") * 5
    if case["masks"]:
        words = -(-V // 32)
        s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (case["masks"], words), generator=g, device="cuda",
                                  dtype=torch.int64).to(torch.int32)
        which = torch.randint(0, case["masks"], (B, R), generator=g, device="cuda", dtype=torch.int64)
        every = torch.arange(B * R, device="cuda").view(B, R)
        s["mask_row"] = torch.where(every % 2 == 0, which, torch.full_like(which, -1)).to(torch.int32)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    make = {"plan": _prepare_plan, "write": _prepare_write, "attend": _prepare_attend, "adjust": _prepare_adjust}
    return dict(make[case["op"]](case, g), op=case["op"])


# ------------------------------------------------------------- plain forms ---
def _plain_plan(s):
    page, room, table, ring = s["page"], s["room"], s["table"], s["ring"]
    dev = table.device
    cap = ring.numel()
    base = (s["length"] + s["advance"]).long()
    rows, held = s["rows"].long(), s["held"].long()
    need = (base + rows + page - 1) // page
    take = (need - held).clamp(min=0)
    give = (held - need).clamp(min=0)
    head, count = s["free"][0].long(), s["free"][1].long()
    offset = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), rows.cumsum(0)])
    take_at, give_at = take.cumsum(0) - take, give.cumsum(0) - give
    N = offset[-1]
    i = torch.arange(room, device=dev)
    live = i < N
    i = torch.minimum(i, (N - 1).clamp(min=0))
    b = torch.searchsorted(offset[1:].contiguous(), i, right=True).clamp(max=s["B"] - 1)
    pos = base[b] + i - offset[b]
    block = pos // page
    fresh = ring[(head + take_at[b] + block - held[b]) % cap]
    where = b * table.shape[1] + block
    got = torch.where(block >= held[b], fresh, table.view(-1)[where])
    # pages that go back follow the live part of the ring, request by request
    j = torch.arange(table.shape[1], device=dev)[None]
    back = (j >= need[:, None]) & (j < held[:, None])
    to = torch.where(back, (head + count + give_at[:, None] + j - need[:, None]) % cap, torch.full_like(j, cap))
    longer = torch.cat([ring, ring[:1]])
    longer[to.view(-1)] = table.view(-1)
    ring.copy_(longer[:cap])
    table.view(-1)[where] = got
    none = torch.full_like(i, -1)
    taken = take.sum()
    return dict(length=base.int(), held=need.int(),
                free_state=torch.stack([(head + taken) % cap, count - taken + give.sum()]).int(),
                row_offset=offset.int(), row_request=torch.where(live, b, none).int(),
                position=torch.where(live, pos, none).int(),
                slot=torch.where(live, got.long() * page + pos % page, none), block_table=table, free_ring=ring)


def _plain_write(s):
    kc, vc = s["kc"], s["vc"]
    page = kc.shape[2]
    live = s["slot"] >= 0
    # rows without a slot repeat row 0, which always has one
    i = torch.where(live, torch.arange(live.numel(), device=live.device), torch.zeros_like(s["slot"]))
    at = s["slot"][i]
    block, off = at // page, at % page
    for x, cache, scale in ((s["k"], kc, s["ks"]), (s["v"], vc, s["vs"])):
        x = x[i].float()
        if scale is not None:
            x = (x / scale[None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[block, :, off] = x.view(torch.uint8)
        else:
            cache[block, :, off] = x.to(cache.dtype)
    return dict(k_cache=kc, v_cache=vc)


def _plain_attend(s):
    q, kc, vc, table = s["q"], s["kc"], s["vc"], s["table"]
    N, Hq, D = q.shape
    Hkv, page = kc.shape[1], kc.shape[2]
    B, R, G = table.shape[0], s["rows"], Hq // Hkv
    dev = q.device
    offset = s["offset"].long()
    n = offset[1:] - offset[:-1]
    total = s["length"].long() + n
    L = table.shape[1] * page

    def gather(cache, scale):
        x = cache[table.long()].float()                                   # B, blocks, Hkv, page, D
        x = x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)
        return x if scale is None else x * scale[None, :, None, None]

    i = torch.arange(R, device=dev)[None]
    at = (offset[:-1, None] + i).clamp(max=N - 1)                          # B, R
    qq = q[at].float().view(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    sc = torch.matmul(qq, gather(kc, s["ks"]).transpose(2, 3)) * (D ** -0.5)
    pos = (s["length"].long()[:, None] + i)[:, :, None]                    # B, R, 1
    key = torch.arange(L, device=dev)[None, None]
    seen = (key <= pos) & (key < total[:, None, None])
    if s["window"]:
        seen = seen & (key > pos - s["window"])
    sc = sc.view(B, Hkv, R, G, L).masked_fill_(~seen[:, None, :, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, R * G, L), gather(vc, s["vs"])).view(B, Hkv, R, G, D)
    o = o / torch.where(z == 0, torch.ones_like(z), z)
    lse = (m + z.log())[..., 0]
    b = torch.searchsorted(offset[1:].contiguous(), torch.arange(N, device=dev), right=True)
    r = torch.arange(N, device=dev) - offset[b]
    return dict(out=o.permute(0, 2, 1, 3, 4)[b, r].reshape(N, Hq, D).to(q.dtype),
                lse=lse.permute(0, 2, 1, 3)[b, r].reshape(N, Hq))


def _plain_adjust(s):
    x = s["logits"]
    B, R, V = x.shape
    dev = x.device
    j = torch.arange(s["history"].shape[1], device=dev)[None]
    hist = s["history"].long()
    is_prompt = (j < s["prompt"][:, None]).float()
    is_out = ((j >= s["prompt"][:, None]) & (j < s["length"][:, None])).float()
    prompt = torch.zeros((B, V), device=dev).scatter_add_(1, hist, is_prompt)
    count = torch.zeros((B, R, V), device=dev)
    count[:, 0].scatter_add_(1, hist, is_out)
    if R > 1:
        # row k follows the draft's first k - 1 tokens
        d = s["draft"].long()
        count[:, 1:].scatter_(2, d[..., None], 1.0)
        count = count.cumsum_(1)
    y = x.float()
    again = (count > 0) | (prompt > 0)[:, None]
    rep = s["rep"][:, None, None]
    y = torch.where(again, torch.where(y > 0, y / rep, y * rep), y)
    y = y - s["freq"][:, None, None] * count
    y = torch.where(count > 0, y - s["pres"][:, None, None], y)
    if s["bias_token"] is not None:
        bias = torch.zeros((B, V), device=dev).scatter_add_(1, s["bias_token"].long(), s["bias_value"])
        y = y + bias[:, None]
    if s["mask"] is not None:
        v = torch.arange(V, device=dev)
        allowed = ((s["mask"][:, v // 32] >> (v % 32)) & 1).bool()
        which = s["mask_row"].long()
        y = y.masked_fill((which >= 0)[..., None] & ~allowed[which.clamp(min=0)], float("-inf"))
    wanted = (torch.arange(R, device=dev)[None] <= s["ell"][:, None])[..., None]
    s["out"].copy_(torch.where(wanted, y.to(x.dtype), s["out"]))
    return s["out"]


# --------------------------------------------------------------------- run ---
def run(s):
    op = s["op"]
    if not own:
        return {"plan": _plain_plan, "write": _plain_write, "attend": _plain_attend, "adjust": _plain_adjust}[op](s)
    import serving_draft_verify_gb300 as dsv
    if op == "plan":
        out = dsv.dspark_plan_rows(s["length"], s["rows"], s["held"], s["free"], s["ring"], s["table"], s["page"],
                                   s["room"], advance=s["advance"], out=s["out"], workspace=s["ws"])
        return dict(out, block_table=s["table"], free_ring=s["ring"])
    if op == "write":
        dsv.dspark_write_kv(s["k"], s["v"], s["slot"], s["kc"], s["vc"], k_scale=s["ks"], v_scale=s["vs"],
                            workspace=s["ws"])
        return dict(k_cache=s["kc"], v_cache=s["vc"])
    if op == "attend":
        return dsv.dspark_paged_attention(s["q"], s["offset"], s["length"], s["table"], s["kc"], s["vc"], s["rows"],
                                          window=s["window"], k_scale=s["ks"], v_scale=s["vs"], out=s["out"],
                                          workspace=s["ws"])
    return dsv.dspark_adjust_logits(s["logits"], s["history"], s["prompt"], s["length"], draft=s["draft"],
                                    ell=s["ell"], repetition=s["rep"], frequency=s["freq"], presence=s["pres"],
                                    bias_token=s["bias_token"], bias_value=s["bias_value"], mask_row=s["mask_row"],
                                    mask=s["mask"], out=s["out"], workspace=s["ws"])


# ------------------------------------------------------------------- exact ---
def _exact_write(s):
    """The caches after the rows were stored; 8-bit ones as the numbers that are rounded to them."""
    out = {}
    page = s["kc"].shape[2]
    at = s["slot"].tolist()
    rows = torch.tensor([i for i, a in enumerate(at) if a >= 0], device="cuda")
    flat = torch.tensor([a for a in at if a >= 0], device="cuda")
    for name, x, cache, scale in (("k_cache", s["k"], s["kc"], s["ks"]), ("v_cache", s["v"], s["vc"], s["vs"])):
        new = x.index_select(0, rows).double()
        if scale is not None:
            new = torch.clamp(new / scale.double().view(1, -1, 1), min=-448, max=448)
        whole = cache.double().transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])
        whole.index_copy_(0, flat, new)
        out[name] = whole.view(-1, page, cache.shape[1], cache.shape[3]).transpose(1, 2).contiguous()
    return out


def _exact_attend(s):
    q = s["q"].double()
    N, Hq, D = q.shape
    Hkv = s["kc"].shape[1]
    out = torch.zeros((N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((N, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    offset, length = s["offset"].tolist(), s["length"].tolist()
    for b in range(len(length)):
        lo, hi = offset[b], offset[b + 1]
        total = length[b] + hi - lo
        if hi == lo or total == 0:
            continue
        ids = s["table"][b].long()

        def keys(cache, scale, h):
            x = cache[ids, h].reshape(-1, D)[:total].double()
            return x if scale is None else x * scale[h].double()

        at = torch.arange(length[b], total, device="cuda")[:, None]
        col = torch.arange(total, device="cuda")[None]
        hide = col > at
        if s["window"]:
            hide |= col <= at - s["window"]
        for h in range(Hkv):
            K, V = keys(s["kc"], s["ks"], h), keys(s["vc"], s["vs"], h)
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = torch.einsum("rgd,ld->grl", q[lo:hi, heads], K) / D ** 0.5
            x = x.masked_fill(hide, float("-inf"))
            lse[lo:hi, heads] = torch.logsumexp(x, -1).T
            out[lo:hi, heads] = torch.einsum("grl,ld->rgd", torch.softmax(x, -1), V)
    return dict(out=out, lse=lse)


def _exact_adjust(s):
    x = s["logits"]
    B, R, V = x.shape
    out = s["out"].double()
    for b in range(B):
        p, h = int(s["prompt"][b]), int(s["length"][b])
        hist = s["history"][b].long()
        seen = torch.bincount(hist[:h], minlength=V) > 0
        count = torch.bincount(hist[p:h], minlength=V).double()
        rep, freq, pres = (float(s[k][b].double()) for k in ("rep", "freq", "pres"))
        for k in range(int(s["ell"][b]) + 1):
            if k:
                count[int(s["draft"][b, k - 1])] += 1
                seen[int(s["draft"][b, k - 1])] = True
            y = x[b, k].double()
            y[seen] = torch.where(y[seen] > 0, y[seen] / rep, y[seen] * rep)
            y -= freq * count + pres * (count > 0)
            if s["bias_token"] is not None:
                y.index_add_(0, s["bias_token"][b].long(), s["bias_value"][b].double())
            if s["mask"] is not None and int(s["mask_row"][b, k]) >= 0:
                word = s["mask"][int(s["mask_row"][b, k])].long()
                bit = (word[:, None] >> torch.arange(32, device="cuda")[None]) & 1
                y[bit.view(-1)[:V] == 0] = float("-inf")
            out[b, k] = y
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None                                   # whole numbers only
    return {"write": _exact_write, "attend": _exact_attend, "adjust": _exact_adjust}[case["op"]](prepare(case, seed))
