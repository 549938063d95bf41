"""Cases of the target step's rotation and of the cache in 4 bits, measured one operator at a time.

Beside the calls of operators.py, a step of the target model rotates its queries and
keys by their positions, stores them, and attends over what is stored.  Measured here:

  rotate  dspark_rotate: rotary positions of rows of heads, and their gradient
  store   dspark_rotate_write_kv, then dspark_read_kv: a step's queries rotated, its keys and
          values stored in the paged cache, and read back as the values that the cache holds
  read    dspark_read_kv: rows of a cache by their slots
  attend  dspark_paged_attention over a cache in 4 bits

A cache in 4 bits holds, for each page and head, `page` rows of D / 2 bytes (two e2m1 values a
byte, the even element in the low half) and behind them `page` rows of one e4m3 scale for each 16
elements (their bytes rounded up to 4), together rounded up to 16 bytes; a value is e2m1 times
its block's scale times its head's.

With `own` false, run() computes an operator from elementary torch operations in 32 bits (angles
in 64), the plain form; with `own` true it calls the library.
"""
import functools
import random

import torch

own = False

_BF16, _F32 = torch.bfloat16, torch.float32
_TYPES = {"bf16": _BF16, "f32": _F32, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


# ------------------------------------------------------------------- cases ---
def listed():
    return [
        # one row each of sixteen requests: the call is all latency
        dict(name="rotate 16 rows", op="rotate", N=16, heads=40, D=128, rot=128, inter=False, back=False, dtype="bf16",
             far=4096),
        # a batch of prompts, queries and keys of the fused projection in one call
        dict(name="rotate 16384 rows", op="rotate", N=16384, heads=40, D=128, rot=128, inter=False, back=False,
             dtype="bf16", far=131072),
        # the gradient of an interleaved rotation of half the head, in the checking type, far positions
        dict(name="rotate back f32", op="rotate", N=6001, heads=12, D=128, rot=64, inter=True, back=True, dtype="f32",
             far=1000000),
        # one row each of sixteen requests, in 4 bits
        dict(name="store 16 rows", op="store", N=16, Hq=32, Hkv=8, D=128, rot=128, inter=False, page=16, dtype="bf16",
             cache="e2m1", far=4096),
        # prompts being read in
        dict(name="store 16384 rows", op="store", N=16384, Hq=32, Hkv=8, D=128, rot=128, inter=False, page=16,
             dtype="bf16", cache="e2m1", far=32768),
        # the rows of one short prompt that another request shares
        dict(name="read 500 rows", op="read", N=500, Hkv=8, D=128, page=16, dtype="bf16", cache="e2m1"),
        # the rows of a long conversation that continues
        dict(name="read 131001 rows", op="read", N=131001, Hkv=8, D=128, page=16, dtype="bf16", cache="e2m1"),
        # one interactive request, one new token
        dict(name="attend 1 request", op="attend", B=1, rows=1, ctx=1900, Hq=32, Hkv=8, D=128, page=16, dtype="bf16",
             window=0),
        # plain decoding of a full batch
        dict(name="attend 64 requests", op="attend", B=64, rows=1, ctx=16384, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", window=0),
        # verification of a block of seven drafted tokens and the bonus row in long conversations
        dict(name="attend 8 rows", op="attend", B=16, rows=8, ctx=32768, Hq=32, Hkv=8, D=128, page=16, dtype="bf16",
             window=0),
        # verification of up to sixteen drafted tokens and the bonus row
        dict(name="attend verify 17 rows", op="attend", B=128, rows=17, ctx=6000, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", window=0),
        # the checking type, an uncommon group of heads, odd pages and a sliding window
        dict(name="attend f32 window", op="attend", B=9, rows=3, ctx=2500, Hq=28, Hkv=4, D=64, page=24, dtype="f32",
             window=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rotate", "store", "read", "attend", "attend", "attend"])
    D = rng.choice([64, 128, 128, 96, 256])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rot = rng.choice([D, D, D // 64 * 32 or 32])
    if op == "rotate":
        heads = rng.choice([1, 8, 12, 40])
        return dict(op=op, N=_log_int(rng, 1, min(16384, 16384 * 40 * 128 // (heads * D * _BYTES[dtype]))), heads=heads,
                    D=D, rot=rot, inter=rng.random() < 0.5, back=rng.random() < 0.5, dtype=dtype,
                    far=rng.choice([500, 32768, 1000000]))
    cache = rng.choice(["e2m1", "e2m1", "e2m1", "e4m3", dtype])
    page = rng.choice([8, 16, 16, 24, 32, 64, 5])
    if op == "store":
        Hq, Hkv = rng.choice([(32, 8), (28, 4), (16, 16), (12, 1)])
        return dict(op=op, N=_log_int(rng, 1, 16384 * 48 * 128 * 2 // ((Hq + 2 * Hkv) * D * _BYTES[dtype] * 2)), Hq=Hq,
                    Hkv=Hkv, D=D, rot=rot, inter=rng.random() < 0.3, page=page, dtype=dtype, cache=cache,
                    far=rng.choice([500, 32768, 1000000]))
    if op == "read":
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, N=_log_int(rng, 1, 131001 * 8 * 128 // (8 * D * _BYTES[dtype])), Hkv=Hkv, D=D, page=page,
                    dtype=dtype, cache=cache)
    Hq, Hkv = rng.choice([(32, 8), (32, 8), (32, 4), (28, 4), (16, 16), (64, 8), (12, 1)])
    rows = rng.choice([1, 1, 2, 4, 5, 8, 17])
    B = _log_int(rng, 1, 256)
    # the padded cache stays below half of the largest listed one
    most = min(65536, (1 << (29 if dtype == "bf16" else 26)) // (B * Hkv * D))
    return dict(op=op, B=B, rows=rows, ctx=_log_int(rng, 32, max(64, most)), Hq=Hq, Hkv=Hkv, D=D, page=page,
                dtype=dtype, window=rng.choice([0, 0, 0, 512]))


# ------------------------------------------------------------------ shapes ---
def _attend_lengths(case):
    """Per request: (keys before the step, rows of the step).  Lengths belong to the case, so that
    its work is known; values belong to the seed."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    got = []
    for b in range(case["B"]):
        rows = r.randint(1, case["rows"]) if b else case["rows"]
        total = max(rows, r.randint(case["ctx"] // 8, case["ctx"]) if b else case["ctx"])
        got.append((total - rows, rows))
    return got


def _row_bytes(case):
    """What one head's row takes in the cache."""
    D = case["D"]
    return D // 2 + D // 16 if case["cache"] == "e2m1" else D * _BYTES[case["cache"]]


def work(case):
    if case["op"] == "rotate":
        n = case["N"] * case["heads"] * case["D"]
        return {"bytes": 2 * n * _BYTES[case["dtype"]] + 4 * case["N"],
                "flops": 3 * case["N"] * case["heads"] * case["rot"]}
    size = _BYTES[case["dtype"]]
    if case["op"] == "store":
        rows, new = case["N"] * case["D"] * size, 2 * case["N"] * case["Hkv"] * _row_bytes(case)
        # q in and out, k and v in, stored, and out again (what was just stored need not come from memory)
        return {"bytes": (2 * case["Hq"] + 4 * case["Hkv"]) * rows + new + 12 * case["N"],
                "flops": 3 * case["N"] * (case["Hq"] + 2 * case["Hkv"]) * case["D"]}
    if case["op"] == "read":
        n = 2 * case["N"] * case["Hkv"]
        return {"bytes": n * (_row_bytes(case) + case["D"] * size) + 8 * case["N"], "flops": n * case["D"]}
    keys = pairs = rows = 0
    for n, q in _attend_lengths(case):
        keys += min(n + q, case["window"] + q - 1) if case["window"] else n + q
        rows += q
        for i in range(q):
            pairs += min(n + i + 1, case["window"] or n + i + 1)
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    return {"bytes": 2 * keys * Hkv * (D // 2 + D // 16) + 2 * rows * Hq * D * size + rows * Hq * 4
            + keys // case["page"] * 4, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------ 4-bit caches ---
def _sizes(page, D):
    """Bytes of a page's codes, of one row's scales and of the whole page of one head."""
    codes, row = page * D // 2, -(-(D // 16) // 4) * 4
    return codes, row, -(-(codes + page * row) // 16) * 16


@functools.lru_cache(maxsize=None)
def _constant(*values):
    return torch.tensor(values, device="cuda")


def _nearest_code(a):
    """The e2m1 code (without sign) nearest to a >= 0, ties to the even code, past the largest the largest."""
    edge = _constant(0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
    # a tie goes up where the code above is the even one
    up = _constant(False, True, False, True, False, True, False)
    return ((a[..., None] > edge) | ((a[..., None] == edge) & up)).sum(-1)


def _quantised(x, head_scale):
    """Codes [..., D] (with sign) and scales [..., D / 16] e4m3 of x [..., heads, D] in 32 bits."""
    blocks = x.unflatten(-1, (-1, 16))
    g = head_scale[:, None]
    s = (blocks.abs().amax(-1) * (1.0 / (6.0 * g))).clamp(max=448.0).to(torch.float8_e4m3fn)
    inv = 1.0 / (s.float() * g)
    y = blocks * torch.where(inv.isinf(), torch.zeros_like(inv), inv)[..., None]
    return (_nearest_code(y.abs()) + 8 * torch.signbit(y)).flatten(-2).to(torch.uint8), s


def _packed(codes, scales, page, D):
    """A cache [blocks, heads, bytes] from codes [blocks, heads, page, D] and their scales."""
    n, row, whole = _sizes(page, D)
    cache = torch.zeros(codes.shape[:2] + (whole,), dtype=torch.uint8, device=codes.device)
    cache[..., :n] = (codes[..., 0::2] | (codes[..., 1::2] << 4)).flatten(-2)
    cache[..., n:n + page * row].unflatten(-1, (page, row))[..., :D // 16] = scales.view(torch.uint8)
    return cache


def _values(cache, page, D, head_scale):
    """The values [..., page, D] float32 of pages [..., heads, bytes] of a 4-bit cache."""
    n, row, _ = _sizes(page, D)
    levels = _constant(0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
    code = cache[..., :n].unflatten(-1, (page, D // 2))
    x = torch.stack([levels[(code & 15).int()], levels[(code >> 4).int()]], -1).flatten(-2)
    s = cache[..., n:n + page * row].unflatten(-1, (page, row))[..., :D // 16].contiguous()
    s = s.view(torch.float8_e4m3fn).float() * head_scale[:, None, None]
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


# ----------------------------------------------------------------- prepare ---
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _workspace(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def _randn(g, *shape, dtype=_F32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _frequencies(rot):
    return (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def _positions(case, g):
    """Runs of positions of a batch's requests, the last rows of the padded step without one."""
    N = case["N"]
    start = torch.randint(0, max(1, case["far"] - N // 8), (8,), generator=g, device="cuda")
    i = torch.arange(N, device="cuda")
    position = (start[i * 8 // max(1, N)] + i % max(1, -(-N // 8))).int()
    if N > 32:
        position[N - N // 32:] = -1
    return position


def _head_scales(g, heads, kind):
    """One float32 a head: a value of a few standard deviations fills the type's range."""
    return (torch.rand(heads, generator=g, device="cuda") + 0.5) * (0.0125 if kind == "e4m3" else 0.002)


def _cache(case, g, blocks):
    """Two caches of values around 1 and the heads' scales."""
    Hkv, page, D, kind = case["Hkv"], case["page"], case["D"], case["cache"]
    got, scales = [], []
    for _ in range(2):
        scale = _head_scales(g, Hkv, kind) if kind in ("e4m3", "e2m1") else None
        if kind == "e2m1":
            made = torch.empty((blocks, Hkv, _sizes(page, D)[2]), dtype=torch.uint8, device="cuda")
            for part in made.split(max(1, (1 << 25) // (Hkv * page * D))):
                x = _randn(g, part.shape[0], page, Hkv, D, dtype=_BF16).float()
                codes, s = _quantised(x, scale)
                part.copy_(_packed(codes.transpose(1, 2), s.transpose(1, 2).contiguous(), page, D))
        else:
            made = _randn(g, blocks, Hkv, page, D, dtype=_F32 if kind == "f32" else _BF16)
            made = made.mul_(80).clamp_(-448, 448).to(_TYPES[kind]) if kind == "e4m3" else made
        got.append(made)
        scales.append(scale)
    return got[0], got[1], scales[0], scales[1]


def _prepare_rotate(case, g):
    x = _randn(g, case["N"], case["heads"] + 8, case["D"], dtype=_TYPES[case["dtype"]])
    return dict(x=x[:, :case["heads"]], position=_positions(case, g), freq=_frequencies(case["rot"]),
                inter=case["inter"], back=case["back"], ws=_workspace(4096),
                out=torch.zeros((case["N"], case["heads"], case["D"]), dtype=_TYPES[case["dtype"]], device="cuda"))


def _slots(g, N, page, blocks):
    """Runs of rows on shuffled pages."""
    perm = torch.randperm(blocks, generator=g, device="cuda")
    i = torch.arange(N, device="cuda")
    return perm[i // page] * page + i % page


def _prepare_store(case, g):
    N, Hq, Hkv, D, page = case["N"], case["Hq"], case["Hkv"], case["D"], case["page"]
    t = _TYPES[case["dtype"]]
    blocks = -(-N // page) + 8
    kind = case["cache"]
    shape = (blocks, Hkv, _sizes(page, D)[2]) if kind == "e2m1" else (blocks, Hkv, page, D)
    kc, vc = (torch.zeros(shape, dtype=_TYPES.get(kind, torch.uint8), device="cuda") for _ in range(2))
    ks, vs = (_head_scales(g, Hkv, kind) if kind in ("e4m3", "e2m1") else None for _ in range(2))
    qkv = _randn(g, N, Hq + 2 * Hkv, D, dtype=t)
    position = _positions(case, g)
    slot = torch.where(position >= 0, _slots(g, N, page, blocks), torch.full_like(position, -1, dtype=torch.int64))
    new = lambda heads: torch.zeros((N, heads, D), dtype=t, device="cuda")  # noqa: E731
    return dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], position=position, slot=slot,
                freq=_frequencies(case["rot"]), inter=case["inter"], kind=kind, page=page, kc=kc, vc=vc, ks=ks, vs=vs,
                out=new(Hq), back=dict(k=new(Hkv), v=new(Hkv)), ws=_workspace(4096))


def _prepare_read(case, g):
    N, Hkv, D, page = case["N"], case["Hkv"], case["D"], case["page"]
    blocks = -(-N // page) + 8
    kc, vc, ks, vs = _cache(case, g, blocks)
    new = lambda: torch.zeros((N, Hkv, D), dtype=_TYPES[case["dtype"]], device="cuda")  # noqa: E731
    return dict(slot=_slots(g, N, page, blocks), kind=case["cache"], page=page, kc=kc, vc=vc, ks=ks, vs=vs,
                back=dict(k=new(), v=new()), ws=_workspace(4096))


def _prepare_attend(case, g):
    lens = _attend_lengths(case)
    page = case["page"]
    pages = [-(-(n + q) // page) for n, q in lens]
    total, width = sum(pages), max(pages)
    cap = total + 16 + total // 8
    perm = torch.randperm(cap, generator=g, device="cuda").to(torch.int32)
    held, col = _ints(pages, torch.int64), torch.arange(width, device="cuda")
    first = held.cumsum(0) - held
    table = perm[(first[:, None] + col[None]).clamp(max=cap - 1)]
    table = torch.where(col[None] < held[:, None], table, torch.zeros_like(table)).contiguous()
    kc, vc, ks, vs = _cache(dict(case, cache="e2m1"), g, cap)
    N = sum(q for _, q in lens)
    q = _randn(g, N, case["Hq"], case["D"], dtype=_TYPES[case["dtype"]]) * 2
    offs = [0]
    for _, n in lens:
        offs.append(offs[-1] + n)
    return dict(q=q, offset=_ints(offs), length=_ints([n for n, _ in lens]), table=table, kc=kc, vc=vc, ks=ks, vs=vs,
                page=page, rows=case["rows"], window=case["window"], ws=_workspace(192 << 20),
                out=dict(out=torch.empty_like(q), lse=torch.empty((N, case["Hq"]), dtype=_F32, device="cuda")))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    make = {"rotate": _prepare_rotate, "store": _prepare_store, "read": _prepare_read, "attend": _prepare_attend}
    return dict(make[case["op"]](case, g), op=case["op"])


# ------------------------------------------------------------- plain forms ---
def _rotated(x, position, freq, inter, back):
    """x [N, heads, D] rotated, in 32 bits; the angles in 64."""
    rot = 2 * freq.numel()
    angle = position.clamp(min=0).double()[:, None] * freq.double()
    if back:
        angle = -angle
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    y = x.float().clone()
    if inter:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rotate(s):
    y = _rotated(s["x"], s["position"], s["freq"], s["inter"], s["back"]).to(s["x"].dtype)
    return torch.where((s["position"] >= 0)[:, None, None], y, s["out"])


def _plain_put(x, slot, cache, scale, kind, page):
    """Rows x [N, heads, D] in 32 bits into the cache at their slots; rows without a slot repeat row 0."""
    i = torch.where(slot >= 0, torch.arange(slot.numel(), device=slot.device), torch.zeros_like(slot))
    block, off = slot[i] // page, slot[i] % page
    x = x[i]
    if kind == "e2m1":
        D = x.shape[-1]
        n, row, _ = _sizes(page, D)
        codes, s = _quantised(x, scale)
        head = torch.arange(x.shape[1], device=x.device)[:, None]
        at = (off * (D // 2))[:, None, None] + torch.arange(D // 2, device=x.device)
        cache[block[:, None, None], head, at] = codes[..., 0::2] | (codes[..., 1::2] << 4)
        at = (n + off * row)[:, None, None] + torch.arange(D // 16, device=x.device)
        cache[block[:, None, None], head, at] = s.view(torch.uint8)
    elif kind == "e4m3":
        x = (x / scale[:, None]).clamp(-448.0, 448.0).to(cache.dtype)
        cache.view(torch.uint8)[block, :, off] = x.view(torch.uint8)
    else:
        cache[block, :, off] = x.to(cache.dtype)


def _plain_get(slot, cache, scale, kind, page, like):
    """Rows [N, heads, D] of the cache at their slots; `like` in the rows without one."""
    at = slot.clamp(min=0)
    block, off = at // page, at % page
    if kind == "e2m1":
        D = like.shape[-1]
        n, row, _ = _sizes(page, D)
        head = torch.arange(like.shape[1], device=slot.device)[:, None]
        code = cache[block[:, None, None], head, (off * (D // 2))[:, None, None] + torch.arange(D // 2, device=slot.device)]
        s = cache[block[:, None, None], head, (n + off * row)[:, None, None] + torch.arange(row, device=slot.device)]
        x = _values(torch.cat([code, s], -1), 1, D, scale)[..., 0, :]
    else:
        x = (cache.view(torch.uint8)[block, :, off].view(cache.dtype) if kind == "e4m3" else cache[block, :, off]).float()
        x = x if scale is None else x * scale[:, None]
    return torch.where((slot >= 0)[:, None, None], x.to(like.dtype), like)


def _plain_store(s):
    live = (s["position"] >= 0)[:, None, None]
    q = _rotated(s["q"], s["position"], s["freq"], s["inter"], False).to(s["q"].dtype)
    k = _rotated(s["k"], s["position"], s["freq"], s["inter"], False)
    _plain_put(k, s["slot"], s["kc"], s["ks"], s["kind"], s["page"])
    _plain_put(s["v"].float(), s["slot"], s["vc"], s["vs"], s["kind"], s["page"])
    return dict(_plain_read(s), q=torch.where(live, q, s["out"]))


def _plain_read(s):
    return dict(k=_plain_get(s["slot"], s["kc"], s["ks"], s["kind"], s["page"], s["back"]["k"]),
                v=_plain_get(s["slot"], s["vc"], s["vs"], s["kind"], s["page"], s["back"]["v"]))


def _plain_attend(s):
    q, table, page = s["q"], s["table"], s["page"]
    N, Hq, D = q.shape
    Hkv = s["kc"].shape[1]
    B, R, G = table.shape[0], s["rows"], Hq // Hkv
    dev = q.device
    offset = s["offset"].long()
    n = offset[1:] - offset[:-1]
    total = s["length"].long() + n
    L = table.shape[1] * page

    def gather(cache, scale):
        x = _values(cache[table.long()], page, D, scale)                      # B, blocks, Hkv, page, D
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)

    i = torch.arange(R, device=dev)[None]
    at = (offset[:-1, None] + i).clamp(max=N - 1)                             # B, R
    qq = q[at].float().view(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    sc = torch.matmul(qq, gather(s["kc"], s["ks"]).transpose(2, 3)) * (D ** -0.5)
    pos = (s["length"].long()[:, None] + i)[:, :, None]                       # B, R, 1
    key = torch.arange(L, device=dev)[None, None]
    seen = (key <= pos) & (key < total[:, None, None])
    if s["window"]:
        seen = seen & (key > pos - s["window"])
    sc = sc.view(B, Hkv, R, G, L).masked_fill_(~seen[:, None, :, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, R * G, L), gather(s["vc"], s["vs"])).view(B, Hkv, R, G, D)
    o = o / torch.where(z == 0, torch.ones_like(z), z)
    lse = (m + z.log())[..., 0]
    b = torch.searchsorted(offset[1:].contiguous(), torch.arange(N, device=dev), right=True)
    r = torch.arange(N, device=dev) - offset[b]
    return dict(out=o.permute(0, 2, 1, 3, 4)[b, r].reshape(N, Hq, D).to(q.dtype),
                lse=lse.permute(0, 2, 1, 3)[b, r].reshape(N, Hq))


# --------------------------------------------------------------------- run ---
def run(s):
    op = s["op"]
    if not own:
        return {"rotate": _plain_rotate, "store": _plain_store, "read": _plain_read, "attend": _plain_attend}[op](s)
    import serving_draft_verify_gb300 as dsv
    if op == "rotate":
        return dsv.dspark_rotate(s["x"], s["position"], s["freq"], interleaved=s["inter"], transposed=s["back"],
                                 out=s["out"], workspace=s["ws"])
    if op == "store":
        q = dsv.dspark_rotate_write_kv(s["q"], s["k"], s["v"], s["position"], s["freq"], s["slot"], s["kc"], s["vc"],
                                       k_scale=s["ks"], v_scale=s["vs"], interleaved=s["inter"], out=s["out"],
                                       workspace=s["ws"])
        back = dsv.dspark_read_kv(s["slot"], s["kc"], s["vc"], k_scale=s["ks"], v_scale=s["vs"], out=s["back"],
                                  workspace=s["ws"])
        return dict(back, q=q)
    if op == "read":
        return dict(dsv.dspark_read_kv(s["slot"], s["kc"], s["vc"], k_scale=s["ks"], v_scale=s["vs"], out=s["back"],
                                       workspace=s["ws"]))
    return dsv.dspark_paged_attention(s["q"], s["offset"], s["length"], s["table"], s["kc"], s["vc"], s["rows"],
                                      window=s["window"], k_scale=s["ks"], v_scale=s["vs"], out=s["out"],
                                      workspace=s["ws"])


# ------------------------------------------------------------------- exact ---
def _exact_turn(x, position, freq, inter, sign):
    """The rotation as a product of complex numbers, in 64 bits."""
    half = freq.numel()
    head, rest = x.double()[..., :2 * half], x.double()[..., 2 * half:]
    pairs = head.unflatten(-1, (half, 2)) if inter else head.unflatten(-1, (2, half)).transpose(-1, -2)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       sign * position.double().unsqueeze(1) * freq.double().unsqueeze(0))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn.unsqueeze(1))
    z = z.flatten(-2) if inter else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, rest], -1)


def _exact_stored(x, scale, kind, dtype):
    """What a cache of this kind holds of x [N, heads, D], in 64 bits."""
    if kind in ("bf16", "f32"):
        return x if kind == "f32" else x.to(_BF16).double()
    g = scale.double().view(1, -1, 1)

    def grid(y, bits, low, top):
        # nearest value with `bits` bits behind the leading one, exponents from `low`, even on ties
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** low))).clamp(min=low) - bits)
        return torch.clamp(torch.round(y / step) * step, -top, top)

    if kind == "e4m3":
        return grid(x / g, 3, -6, 448.0) * g
    blocks = x.reshape(*x.shape[:-1], -1, 16)
    s = grid(blocks.abs().amax(-1) / (6 * g), 3, -6, 448.0)
    unit = (s * g).unsqueeze(-1)
    coded = grid(blocks / torch.where(unit == 0, torch.ones_like(unit), unit), 1, 0, 6.0)
    return (coded * unit).reshape(x.shape)


def _exact_rows(s):
    """The cache's rows in 64 bits, one page at a time by a reshaping of the whole cache."""
    got = {}
    N, heads, D = s["back"]["k"].shape
    for name, cache, scale in (("k", s["kc"], s["ks"]), ("v", s["vc"], s["vs"])):
        if s["kind"] == "e2m1":
            flat = _exact_flat(cache, s["page"], D, scale)
        else:
            flat = cache.double().permute(0, 2, 1, 3).reshape(-1, heads, D)
            flat = flat if scale is None else flat * scale.double().view(1, -1, 1)
        got[name] = flat[s["slot"]]
    return got


def _exact_flat(cache, page, D, scale):
    """All rows [blocks * page, heads, D] of a 4-bit cache in 64 bits, from the bits of its codes."""
    blocks, heads, _ = cache.shape
    row = (D // 16 + 3) // 4 * 4
    code = cache[:, :, :page * D // 2].reshape(blocks, heads, page, D // 2, 1).int()
    code = torch.cat([code % 16, code // 16], -1).reshape(blocks, heads, page, D)
    e, m = code % 8 // 2, (code % 2).double()
    x = torch.where(e == 0, m / 2, torch.exp2(e.double() - 1) * (1 + m / 2))
    x = torch.where(code >= 8, -x, x)
    b = cache[:, :, page * D // 2:page * (D // 2 + row)].reshape(blocks, heads, page, row)[..., :D // 16].int()
    e, m = b % 128 // 8, (b % 8).double()
    s = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e.double() - 7) * (1 + m / 8))
    x = x * s.repeat_interleave(16, -1) * scale.double().view(1, -1, 1, 1)
    return x.permute(0, 2, 1, 3).reshape(blocks * page, heads, D)


def _exact_attend(s):
    q = s["q"].double()
    N, Hq, D = q.shape
    Hkv, page = s["kc"].shape[1], s["page"]
    out = torch.zeros((N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((N, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    offset, length = s["offset"].tolist(), s["length"].tolist()
    for b in range(len(length)):
        lo, hi = offset[b], offset[b + 1]
        total = length[b] + hi - lo
        ids = s["table"][b].long()
        K, V = (_exact_flat(c[ids], page, D, g)[:total] for c, g in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        at = torch.arange(length[b], total, device="cuda")[:, None]
        col = torch.arange(total, device="cuda")[None]
        hide = col > at
        if s["window"]:
            hide |= col <= at - s["window"]
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = torch.einsum("rgd,ld->grl", q[lo:hi, heads], K[:, h]) / D ** 0.5
            x = x.masked_fill(hide, float("-inf"))
            lse[lo:hi, heads] = torch.logsumexp(x, -1).T
            out[lo:hi, heads] = torch.einsum("grl,ld->rgd", torch.softmax(x, -1), V[:, h])
    return dict(out=out, lse=lse)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        y = _exact_turn(s["x"], s["position"], s["freq"], s["inter"], -1.0 if s["back"] else 1.0)
        y[s["position"] < 0] = 0
        return y
    if case["op"] == "store":
        gone = s["position"] < 0
        q, k = (_exact_turn(s[x], s["position"], s["freq"], s["inter"], 1.0) for x in ("q", "k"))
        k = _exact_stored(k, s["ks"], s["kind"], case["dtype"])
        v = _exact_stored(s["v"].double(), s["vs"], s["kind"], case["dtype"])
        for x in (q, k, v):
            x[gone] = 0
        return dict(k=k, v=v, q=q)
    if case["op"] == "read":
        return _exact_rows(s)
    return _exact_attend(s)
