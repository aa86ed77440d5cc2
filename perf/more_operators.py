"""The operators that fill, share and read a paged key-value cache, as measured cases.

Between a block's projections and its attention a server normalizes the heads
of the queries and keys, rotates them by their positions and puts keys and
values into their pages, in bf16 or in 4 bits; the attention of the next
tokens reads 4-bit pages; and completions that share a prompt share its pages
until one of them writes, which takes forks, copies and, when the pool has
holes, compaction.

4-bit values are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), two to a byte,
the even column in the low half, with an e4m3 scale per row of 16 columns:
scale = max |y| / 6 rounded, at least 2^-9, with y already divided by its
head's factor.

``run`` computes each case in plain torch operations in 32 bits (the angles in
64: positions are far), or, with ``own`` set, by the package's calls.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
GROUP = 16  # columns per 4-bit scale
LEAST = 2.0 ** -9  # smallest scale


def listed():
    return [
        # One user's next token: its keys and values into a bf16 cache; pure latency.
        dict(name="rope_1", op="rope", T=1, Hq=32, Hkv=8, D=128, rot=128, axes=1, pairs="halves", norm=True,
             cache="bf16", page=16),
        # A server's batch of next tokens into a 4-bit cache, a few rows of it padding.
        dict(name="rope_batch", op="rope", T=96, Hq=64, Hkv=8, D=128, rot=128, axes=1, pairs="halves", norm=True,
             cache="fp4", page=24),
        # An image or video prompt, positions of time, height and width, neighbouring columns as pairs.
        dict(name="rope_axes", op="rope", T=4099, Hq=12, Hkv=12, D=64, rot=64, axes=3, pairs="neighbours", norm=True,
             cache="none", page=1),
        # A long prompt at once: bandwidth.
        dict(name="rope_prompt", op="rope", T=16384, Hq=32, Hkv=8, D=128, rot=128, axes=1, pairs="halves", norm=True,
             cache="bf16", page=64),
        # One user in a chat.
        dict(name="attn4_1", op="attn4", B=1, Hq=32, Hkv=8, D=128, page=16, longest=8191, lens="all", factors=False),
        # Heads without sharing, short caches, small pages.
        dict(name="attn4_heads", op="attn4", B=16, Hq=12, Hkv=12, D=64, page=8, longest=1000, lens="mixed",
             factors=True),
        # A server's batch, lengths from none to long, pages that end inside whatever tile is used.
        dict(name="attn4_batch", op="attn4", B=64, Hq=64, Hkv=8, D=128, page=24, longest=16384, lens="mixed",
             factors=True),
        # A few very long documents.
        dict(name="attn4_long", op="attn4", B=4, Hq=32, Hkv=8, D=128, page=64, longest=131071, lens="all",
             factors=False),
        # A second completion of one prompt: latency.
        dict(name="pages_branch_1", op="branch", prompts=1, each=1, longest=1000, new=1, layers=2, Hkv=8, D=128, page=16,
             kind="bf16"),
        # Seven completions of each of 32 prompts, every one with a page of its own to copy, in every layer.
        dict(name="pages_branch", op="branch", prompts=32, each=7, longest=2000, new=3, layers=8, Hkv=8, D=128, page=16,
             kind="bf16"),
        # Pages of a 4-bit cache copied to places that the caller names.
        dict(name="pages_copy", op="copy", n=300, pages=1024, layers=6, Hkv=8, D=128, page=64, kind="fp4"),
        # Half of a pool's pages in use, scattered: its upper half is to be given back.
        dict(name="pages_compact", op="compact", pages=4096, used=0.5, rows=300, layers=1, Hkv=8, D=128, page=64,
             kind="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "attn4", "attn4", "branch", "copy", "compact"])
    if op == "rope":
        cache = rng.choice(["none", "bf16", "fp4"])
        D, Hkv = rng.choice([(64, 1), (64, 4), (64, 12), (128, 1), (128, 2), (128, 8), (256, 1), (256, 4)])
        if cache == "none" and rng.random() < 0.3:
            D = rng.choice([32, 80, 96, 112, 192])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        axes = rng.choice([1, 1, 2, 3])
        rot = rng.choice([D, D, D // 32 * 16])
        # up to the work of the longest prompt; 4-bit keys up to half a million values, so that a last bit of a
        # 32-bit sum that puts one of them across the middle of two steps stays a rare thing
        most = 100_000_000 // ((Hq + 2 * Hkv) * D)
        T = _log_uniform(rng, 1, min(16384, most, (1 << 19) // (Hkv * D) if cache == "fp4" else most))
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, axes=axes, pairs=rng.choice(["halves", "neighbours"]),
                    norm=rng.random() < 0.75, cache=cache, page=rng.choice([1, 8, 16, 24, 64, 100]))
    if op == "attn4":
        D, Hkv = rng.choice([(64, 1), (64, 4), (64, 12), (128, 1), (128, 2), (128, 8), (128, 32), (256, 1), (256, 4)])
        G = rng.choice([1, 2, 4, 5, 8, 16, 24])
        longest = _log_uniform(rng, 1, 131072)
        # the plain form holds the caches padded to the longest: at most 4 GiB in 32 bits each
        most = max(1, (1 << 30) // (longest * Hkv * D))
        B = _log_uniform(rng, 1, min(256, most))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([1, 8, 16, 24, 32, 64, 100, 128]),
                    longest=longest, lens=rng.choice(["all", "mixed"]), factors=rng.random() < 0.5)
    Hkv, D = rng.choice([(1, 64), (4, 64), (2, 128), (8, 128), (4, 256)])
    page = rng.choice([8, 16, 24, 64])
    kind = rng.choice(["bf16", "fp4"])
    layers = rng.randint(1, 8)
    if op == "branch":
        each = _log_uniform(rng, 1, 8)
        return dict(op=op, prompts=_log_uniform(rng, 1, 32), each=each, longest=_log_uniform(rng, 1, 2000),
                    new=rng.randint(1, 40), layers=layers, Hkv=Hkv, D=D, page=page, kind=kind)
    size = page * Hkv * D * (2 if kind == "bf16" else 1) * 2 * layers  # bytes of a page in all layers, 4 bits rounded up
    pages = _log_uniform(rng, 4, max(8, min(20000, (1 << 30) // size)))
    if op == "copy":
        return dict(op=op, n=_log_uniform(rng, 1, pages // 2), pages=pages, layers=layers, Hkv=Hkv, D=D, page=page, kind=kind)
    return dict(op=op, pages=pages, used=round(rng.uniform(0.1, 0.95), 2), rows=_log_uniform(rng, 1, 300), layers=layers,
                Hkv=Hkv, D=D, page=page, kind=kind)


# ------------------------------------------------------------------ shapes --

def _mixed(count, longest):
    """Lengths spread over the logarithm with the longest, one token and none among them."""
    lens = [int((longest + 1) ** ((b + 0.5) / count)) for b in range(count)]
    lens[-1] = longest
    if count > 2:
        lens[0], lens[1] = 0, 1
    order = [(b * 7919 + 3) % count for b in range(count)] if math.gcd(7919, count) == 1 else range(count)
    return [lens[b] for b in order]


def _lens(case):
    return [case["longest"]] * case["B"] if case["lens"] == "all" else _mixed(case["B"], case["longest"])


def _prompt_lens(case):
    return [max(1, n) for n in _mixed(case["prompts"], case["longest"])]


def _page_bytes(case):
    """Bytes of one page of keys and values in all layers."""
    values = case["page"] * case["Hkv"] * case["D"] * 2 * case["layers"]
    return 2 * values if case["kind"] == "bf16" else values // 2 + values // GROUP


def _tail(case, n):
    """Tokens in the last page of n, if it is not full."""
    return n % case["page"]


def work(case):
    op = case["op"]
    if op == "rope":
        T, Hq, Hkv, D = (case[n] for n in ("T", "Hq", "Hkv", "D"))
        v = case["cache"] != "none"
        cost = T * 2 * D * (Hq + Hkv + (Hkv if v else 0)) + T * 2 * D * (Hq + Hkv) + 4 * T * case["axes"]
        if case["cache"] == "bf16":
            cost += T * (2 * D * Hkv + 8)
        elif case["cache"] == "fp4":  # beside the stored bytes the values that they stand for
            cost += T * (2 * D * Hkv + 2 * Hkv * (D // 2 + D // GROUP) + 8)
        return {"bytes": cost, "flops": T * (Hq + Hkv) * (7 * D if case["norm"] else 3 * D)}
    if op == "attn4":
        tokens, D, Hq = sum(_lens(case)), case["D"], case["Hq"]
        pages = sum(-(-n // case["page"]) for n in _lens(case))
        cost = 2 * tokens * case["Hkv"] * (D // 2 + D // GROUP) + 4 * pages + case["B"] * (4 * Hq * D + 4 * Hq + 4)
        return {"bytes": cost, "flops": 4 * tokens * Hq * D}
    size = _page_bytes(case)
    if op == "branch":
        cost = 0
        for n in _prompt_lens(case):
            row = 8 * -(-n // case["page"])  # the entries of the parent's row, once read and once written
            copied = 2 * size if _tail(case, n) else 0
            cost += case["each"] * (row + copied + 8 * case["new"] + 16)
        return {"bytes": cost, "flops": 0}
    if op == "copy":
        return {"bytes": case["n"] * (2 * size + 8), "flops": 0}
    used = max(1, int(case["pages"] * case["used"]))
    moved = used * (1 - used / case["pages"])  # pages in use above that many, on average
    return {"bytes": 2 * size * moved + 8 * case["pages"] + 8 * used, "flops": 0}


# ------------------------------------------------------------------ inputs --

def _fp4_bytes(gen, *shape):
    """Bytes of two e2m1 values each, distributed as those of normal values scaled by the largest of 16."""
    # of 16 normal values the largest is 1.77 on average; the steps' middles divide the rest of the bell
    edges = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    phi = [math.erf(e * 1.77 / 6 / math.sqrt(2)) for e in edges]
    share = [b - a for a, b in zip([0.0] + phi, phi + [1.0])]
    codes = [c for c, s in enumerate(share) for _ in range(round(s * 128))]
    codes = (codes + [3] * 128)[:128]
    nibble = torch.tensor([c | sign for sign in (0, 8) for c in codes], dtype=torch.uint8, device="cuda")  # 256 alike
    raw = torch.randint(0, 65536, shape, generator=gen, device="cuda", dtype=torch.int32)
    return nibble[raw & 255] | (nibble[raw >> 8] << 4)


def _fp4_cache(gen, pages, page, Hkv, D):
    """Keys or values of a layer in 4 bits and their scales, a head's rows of a page side by side."""
    q = torch.empty((pages, Hkv, page, D // 2), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (page * Hkv * D // 2))
    for p in range(0, pages, step):
        q[p:p + step] = _fp4_bytes(gen, *q[p:p + step].shape)
    s = torch.randn((pages, Hkv, page, D // GROUP), generator=gen, device="cuda")
    s = (0.3 * torch.exp(0.3 * s)).to(torch.float8_e4m3fn)
    return q.transpose(1, 2), s.transpose(1, 2)


def _pools(gen, case):
    """Every layer's caches, filled: one tensor per kind, and the list that a program passes."""
    n, page, Hkv, D, layers = (case[k] for k in ("pages", "page", "Hkv", "D", "layers"))
    if case["kind"] == "bf16":
        kv = torch.empty((layers, 2, n, page, Hkv, D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        return [kv], [kv[i, j] for i in range(layers) for j in range(2)]
    q = torch.randint(0, 256, (layers, 2, n, Hkv, page, D // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s = torch.randint(0, 120, (layers, 2, n, Hkv, page, D // GROUP), generator=gen, device="cuda", dtype=torch.uint8)
    return [q, s], [t[i, j].transpose(1, 2) for t in (q, s) for i in range(layers) for j in range(2)]


def _prepare_rope(case, gen, randn, s):
    T, Hq, Hkv, D, rot, axes = (case[n] for n in ("T", "Hq", "Hkv", "D", "rot", "axes"))
    # what the projection gives: queries, keys and values of a token in a row
    qkv = torch.empty((T, (Hq + 2 * Hkv) * D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    qkv *= (1 + 8 * (randn((Hq + 2 * Hkv) * D) > 2.5)).bfloat16()
    s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    s["q_weight"] = (1 + 0.1 * randn(D)).bfloat16() if case["norm"] else None
    s["k_weight"] = (1 + 0.1 * randn(D)).bfloat16() if case["norm"] else None
    s["inv_freq"] = torch.tensor([THETA ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float32, device="cuda")
    # a prompt's positions follow one another, those of a batch's next tokens are far apart
    if T >= 1024:
        where = torch.arange(T, device="cuda")
    else:
        where = torch.randint(0, 131072, (T,), generator=gen, device="cuda")
    pos = torch.stack([where if a == 0 else (where // 37 ** (axes - 1 - a)) % 37 for a in range(axes)])
    s["positions"] = (pos if axes > 1 else pos[0]).to(torch.int32)
    s["pair_axis"] = [min(axes - 1, i * axes // (rot // 2)) for i in range(rot // 2)] if axes > 1 else None
    if case["cache"] == "none":
        return
    page = case["page"]
    pages = -(-(T + T // 7 + 3) // page)
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:T]
    if 8 <= T < 1024:
        slots[torch.arange(5, T, 32, device="cuda")] = -1  # padding of the batch
    s["slots"] = slots
    if case["cache"] == "bf16":
        kv = torch.empty((pages, 2, page, Hkv, D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        s["cache"] = kv
        s["k_cache"], s["v_cache"] = kv[:, 0], kv[:, 1]
        return
    (s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"]) = (_fp4_cache(gen, pages, page, Hkv, D) for _ in range(2))
    s["k_factor"], s["v_factor"] = (torch.exp(0.2 * randn(Hkv)) for _ in range(2))


def _prepare_attn4(case, gen, randn, s):
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    lens = _lens(case)
    need = [-(-n // page) for n in lens]
    most = max(max(need), 1)
    pages = max(sum(need), 1) + 3
    (s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"]) = (_fp4_cache(gen, pages, page, Hkv, D) for _ in range(2))
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((B, most), dtype=torch.int32, device="cuda")
    used = torch.tensor(need, device="cuda")
    table[torch.arange(most, device="cuda")[None, :] < used[:, None]] = order[:sum(need)]
    s.update(table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=D ** -0.5,
             q=(1.5 * randn(B, case["Hq"], D)).bfloat16(), k_factor=None, v_factor=None)
    if case["factors"]:
        s["k_factor"], s["v_factor"] = (torch.exp(0.2 * randn(Hkv)) for _ in range(2))


def _prepare_branch(case, gen, s):
    page, each, new = case["page"], case["each"], case["new"]
    lens = _prompt_lens(case)
    need = [-(-n // page) for n in lens]
    n = len(lens)
    own_pages = each * sum(1 + -(-new // page) for _ in lens)
    pages = sum(need) + own_pages + 5
    wide = max(need) + -(-new // page) + 1
    rows = n * (1 + each)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((rows, wide), -1, dtype=torch.int32, device="cuda")
    used = torch.zeros(rows, dtype=torch.int64, device="cuda")
    used[:n] = torch.tensor(need, device="cuda")
    table[torch.arange(wide, device="cuda")[None, :] < used[:, None]] = order[:sum(need)]
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:sum(need)].long()] = 1
    seq_lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    seq_lens[:n] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    child = torch.arange(n, rows, device="cuda", dtype=torch.int32)
    s["stack"], s["caches"] = _pools(gen, dict(case, pages=pages))
    s.update(table=table, refs=refs, lens=seq_lens, child=child, parent=(child - n) // each,
             count=torch.full_like(child, new))


def _prepare_compact(case, gen, s):
    pages, rows = case["pages"], case["rows"]
    used = max(1, int(pages * case["used"]))
    rows = min(rows, used)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    per = torch.full((rows,), used // rows, device="cuda", dtype=torch.int64)
    per[:used - int(used // rows) * rows] += 1
    wide = used // rows + 3
    table = torch.randint(-9, 9 + pages, (rows, wide), generator=gen, device="cuda", dtype=torch.int32)  # no pages behind the last
    table[torch.arange(wide, device="cuda")[None, :] < per[:, None]] = order[:used]
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:used].long()] = 1
    # a prompt's first pages stand in every fourth row beside its own
    if rows > 4:
        table[4::4, 0] = table[0, 0]
        refs.zero_()
        held = table[torch.arange(wide, device="cuda")[None, :] < per[:, None]].long()
        refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    short = torch.randint(0, case["page"], (rows,), generator=gen, device="cuda")
    s["stack"], s["caches"] = _pools(gen, case)
    s.update(table=table, refs=refs, lens=(per * case["page"] - short).to(torch.int32))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    state = {"case": case}
    if case["op"] == "rope":
        _prepare_rope(case, gen, randn, state)
    elif case["op"] == "attn4":
        _prepare_attn4(case, gen, randn, state)
    elif case["op"] == "branch":
        _prepare_branch(case, gen, state)
    elif case["op"] == "compact":
        _prepare_compact(case, gen, state)
    else:
        state["stack"], state["caches"] = _pools(gen, case)
        order = torch.randperm(case["pages"], generator=gen, device="cuda").to(torch.int32)
        state["src"], state["dst"] = order[:case["n"]].clone(), order[case["n"]:2 * case["n"]].clone()
    return state


# -------------------------------------------------------------- plain form --

def _plain_quantize(y):
    """The e2m1 codes of y[..,D], and the scale of each 16 columns."""
    g = y.unflatten(-1, (-1, GROUP))
    scale = (g.abs().amax(-1) / 6).clamp(max=448.0).to(torch.float8_e4m3fn).float().clamp(min=LEAST)
    x = g / scale[..., None]
    m = x.abs()
    # ties go to the even code
    code = ((m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    return (code + 8 * (torch.signbit(x)).byte()).flatten(-2), scale.to(torch.float8_e4m3fn)


def _plain_values(codes, scale):
    steps = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    steps = torch.cat([steps, -steps])
    return (steps[codes.int()].unflatten(-1, (-1, GROUP)) * scale.float()[..., None]).flatten(-2)


def _plain_head(x, weight, cos, sin, rot, pairs):
    """Norm and rotation of x[T,h,D] in 32 bits; cos and sin [T,rot/2]."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    cos, sin = cos[:, None], sin[:, None]
    if pairs == "halves":
        a, b, rest = x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b, rest = x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _plain_rope(s):
    case = s["case"]
    pos = s["positions"] if case["axes"] > 1 else s["positions"][None]
    each = torch.tensor(s["pair_axis"], device=pos.device) if s["pair_axis"] else torch.zeros_like(s["inv_freq"], dtype=torch.int64)
    angle = pos[each].double().T * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _plain_head(s["q"], s["q_weight"], cos, sin, case["rot"], case["pairs"]).bfloat16()
    k = _plain_head(s["k"], s["k_weight"], cos, sin, case["rot"], case["pairs"])
    if case["cache"] == "none":
        return {"q": q, "k": k.bfloat16()}
    live = s["slots"] >= 0
    at = s["slots"][live]
    page, token = at // case["page"], at % case["page"]
    if case["cache"] == "bf16":
        s["k_cache"][page, token] = k[live].bfloat16()
        s["v_cache"][page, token] = s["v"][live]
        return {"q": q, "cache": s["cache"]}
    got = {"q": q}
    for name, y in (("k", k), ("v", s["v"].float())):
        factor = s[name + "_factor"][:, None]
        codes, scale = _plain_quantize(y / factor)
        s[name + "_cache"][page, token] = (codes[..., 0::2] | codes[..., 1::2] << 4)[live]
        s[name + "_scales"].view(torch.uint8)[page, token] = scale.view(torch.uint8)[live]
        got[name] = (_plain_values(codes, scale) * factor).bfloat16()
        got[name + "_scales"] = s[name + "_scales"]
    return got


def _plain_attn4(s):
    q, lens, page = s["q"], s["lens"].long(), s["case"]["page"]
    B, Hq, D = q.shape
    Hkv, longest = s["k_cache"].shape[2], s["case"]["longest"]
    key = torch.arange(longest, device=q.device)
    where = s["table"][:, key // page].long()
    steps = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=q.device)
    steps = torch.cat([steps, -steps])
    both = torch.stack([steps.repeat(16), steps.repeat_interleave(16)], 1)  # the two values of a byte

    def values(cache, scales, factor):  # [B, longest, Hkv, D]
        x = both[cache[where, key % page].int()].flatten(-2).unflatten(-1, (-1, GROUP))
        x *= scales.view(torch.uint8)[where, key % page].view(torch.float8_e4m3fn).float()[..., None]
        if factor is not None:
            x *= factor[:, None, None]
        return x.flatten(-2)

    valid = (key[None, :] < lens[:, None])[:, None, None, :]
    scores = torch.einsum("bhgd,blhd->bhgl", q.float().view(B, Hkv, Hq // Hkv, D),
                          values(s["k_cache"], s["k_scales"], s["k_factor"])) * s["scale"]
    scores = scores.masked_fill(~valid, -math.inf)
    top = scores.amax(dim=3, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(dim=3, keepdim=True)
    v = values(s["v_cache"], s["v_scales"], s["v_factor"])
    out = torch.einsum("bhgl,blhd->bhgd", p, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = torch.where(total == 0, torch.full_like(total, -math.inf), top + torch.log(total))
    return {"out": out.reshape(B, Hq, D).bfloat16(), "lse": lse.reshape(B, Hq)}


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for t in s["stack"]:
        t[:, :, dst] = t[:, :, src]
    return {"caches": s["stack"]}


def _plain_branch(s):
    """The children give their pages back and take their parents', then each gets room for its new tokens: a page
    that is not full and still another's is copied first; new pages are the lowest free ones."""
    page, new = s["case"]["page"], s["case"]["new"]
    table, refs, lens, stack = s["table"], s["refs"], s["lens"], s["stack"]
    child, parent = s["child"].long(), s["parent"].long()
    col = torch.arange(table.shape[1], device=table.device)
    held = lambda rows: col < (lens[rows].long()[:, None] + page - 1) // page  # noqa: E731
    count = lambda entries, by: refs.index_add_(0, entries.long(), torch.full_like(entries, by, dtype=torch.int32))  # noqa: E731
    before, theirs = table[child], table[parent]
    count(before[held(child)], -1)
    count(theirs[held(parent)], 1)
    table[child] = torch.where(held(parent), theirs, before)
    lens[child] = lens[parent]

    n0 = lens[child].long()
    n1 = n0 + s["count"].long()
    have, want = (n0 + page - 1) // page, (n1 + page - 1) // page
    last = table[child, (have - 1).clamp(min=0)].long()
    rank = ((last[None, :] == last[:, None]) & (n0 % page != 0)[None, :]).tril(-1).sum(1)  # earlier ones with that page
    shared = (n0 % page != 0) & (refs[last].long() - rank > 1)
    fresh = want - have + shared
    first = torch.cumsum(fresh, 0) - fresh
    free = torch.nonzero(refs == 0)[:, 0].to(torch.int32)
    src, dst = last[shared], free[first[shared]]
    for t in stack:
        t[:, :, dst.long()] = t[:, :, src]
    count(src, -1)
    table[child[shared], have[shared] - 1] = dst
    where = (col >= have[:, None]) & (col < want[:, None])
    at = (first + shared - have)[:, None] + col
    table[child] = torch.where(where, free[at.clamp(0, len(free) - 1)], table[child])
    refs[free[:int(fresh.sum())].long()] = 1
    lens[child] = n1.to(torch.int32)
    token = n0[:, None] + torch.arange(new, device=table.device)
    slots = torch.gather(table[child].long(), 1, token // page) * page + token % page
    return {"table": table, "refs": refs, "lens": lens, "slots": slots, "caches": stack}


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    used = refs > 0
    n = used.sum()
    index = torch.arange(len(refs), device=refs.device)
    src, dst = torch.nonzero(used & (index >= n))[:, 0], torch.nonzero(~used & (index < n))[:, 0]
    to = index.to(torch.int32)
    to[src] = dst.to(torch.int32)
    held = torch.arange(table.shape[1], device=table.device) < ((s["lens"].long() + s["case"]["page"] - 1) // s["case"]["page"])[:, None]
    new_table = torch.where(held, to[torch.where(held, table, torch.zeros_like(table)).long()], table)
    new_refs = refs.clone()
    new_refs[dst] = refs[src]
    new_refs[src] = 0
    for t in s["stack"]:
        t[:, :, dst] = t[:, :, src]
    return {"table": new_table, "refs": new_refs, "caches": s["stack"]}


# --------------------------------------------------------------------- run --

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"rope": _plain_rope, "attn4": _plain_attn4, "branch": _plain_branch, "copy": _plain_copy,
                "compact": _plain_compact}[op](s)
    import moe_token_dispatch_persistent_gb300 as mk

    if op == "rope":
        common = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=case["pairs"] == "neighbours",
                      pair_axis=s["pair_axis"], check=False)
        if case["cache"] == "none":
            return mk.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], **common)
        common.update(v=s["v"], slots=s["slots"], k_cache=s["k_cache"], v_cache=s["v_cache"])
        if case["cache"] == "bf16":
            o = mk.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], **common)
            return {"q": o["q"], "cache": s["cache"]}
        o = mk.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                            k_factor=s["k_factor"], v_factor=s["v_factor"], keep=True, **common)
        return {"q": o["q"], "k": o["k"], "v": o["v"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    if op == "attn4":
        return mk.paged_attention_fp4(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"],
                                      s["lens"], scale=s["scale"], k_factor=s["k_factor"], v_factor=s["v_factor"],
                                      check=False)
    if op == "copy":
        mk.copy_pages(s["caches"], s["src"], s["dst"], check=False)
        return {"caches": s["stack"]}
    if op == "branch":
        mk.fork_sequences(s["table"], s["lens"], s["refs"], s["parent"], s["child"], case["page"], check=False)
        slots = mk.extend_sequences(s["table"], s["lens"], s["refs"], s["child"], s["count"], case["new"], s["caches"],
                                    case["page"], check=False)
        return {"table": s["table"], "refs": s["refs"], "lens": s["lens"], "slots": slots, "caches": s["stack"]}
    o = mk.compact_pages(s["table"], s["lens"], s["refs"], s["caches"], case["page"], check=False)
    return {"table": o["block_table"], "refs": o["refs"], "caches": s["stack"]}


# ----------------------------------------------------- 64 bits, from the definitions --

_STEPS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_rope(s):
    case = s["case"]
    T, rot, D = case["T"], case["rot"], case["D"]
    if T * (case["Hq"] + 2 * case["Hkv"]) * D > 120_000_000:
        return None
    pos = s["positions"].double().view(case["axes"], T)
    turn = torch.empty((T, rot // 2), dtype=torch.float64, device="cuda")
    for i in range(rot // 2):
        turn[:, i] = pos[s["pair_axis"][i] if s["pair_axis"] else 0] * float(s["inv_freq"][i])
    unit = torch.polar(torch.ones_like(turn), turn)[:, None, :]

    def head(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt((x * x).sum(2, keepdim=True) / D + EPS) * weight.double()
        x = x.clone()
        first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if case["pairs"] == "halves" else (slice(0, rot, 2), slice(1, rot, 2))
        z = torch.complex(x[..., first], x[..., second]) * unit
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k = head(s["q"], s["q_weight"]), head(s["k"], s["k_weight"])
    if case["cache"] == "none":
        return {"q": q, "k": k}
    slots = s["slots"]
    rows = torch.nonzero(slots >= 0)[:, 0]
    at = torch.div(slots[rows], case["page"], rounding_mode="floor"), slots[rows] % case["page"]
    if case["cache"] == "bf16":
        cache = s["cache"].double()
        cache[at[0], 0, at[1]] = k[rows]
        cache[at[0], 1, at[1]] = s["v"].double()[rows]
        return {"q": q, "cache": cache}
    got = {"q": q}
    steps = torch.tensor(_STEPS, dtype=torch.float64, device="cuda")
    for name, y in (("k", k), ("v", s["v"].double())):
        y = y / s[name + "_factor"].double()[:, None]
        g = y.reshape(T, case["Hkv"], -1, GROUP)
        scale = (g.abs().max(3).values / 6).clamp(max=448).float().to(torch.float8_e4m3fn).double().clamp(min=LEAST)
        m = (g / scale[..., None]).abs()
        # the nearest step; of two alike the one with the even code
        near = (m[..., None] - steps).abs() + 1e-15 * torch.tensor([0, 1] * 4, dtype=torch.float64, device="cuda")
        value = steps[near.argmin(-1)] * torch.sign(g) * scale[..., None]
        got[name] = value.reshape(T, case["Hkv"], D) * s[name + "_factor"].double()[:, None]
        scales = s[name + "_scales"].double()
        scales[at[0], at[1]] = scale[rows]
        got[name + "_scales"] = scales
    return got


def _exact_attn4(s):
    B, Hq, D = s["q"].shape
    Hkv, page = s["k_cache"].shape[2], s["case"]["page"]
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    steps = torch.tensor(_STEPS + [-v for v in _STEPS], dtype=torch.float64, device="cuda")

    def head(name, pages, h, n):
        b = s[name + "_cache"][pages, :, h].reshape(-1, D // 2)[:n].long()
        x = torch.empty((n, D), dtype=torch.float64, device="cuda")
        x[:, 0::2], x[:, 1::2] = steps[b % 16], steps[b // 16]
        x *= s[name + "_scales"].view(torch.uint8)[pages, :, h].view(torch.float8_e4m3fn).reshape(-1, D // GROUP)[:n].double().repeat_interleave(GROUP, 1)
        return x if s[name + "_factor"] is None else x * s[name + "_factor"][h].double()

    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        for h in range(Hkv):
            mine = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            scores = (s["q"][b, mine].double() @ head("k", pages, h, n).T) * s["scale"]
            lse[b, mine] = torch.logsumexp(scores, dim=1)
            out[b, mine] = torch.softmax(scores, dim=1) @ head("v", pages, h, n)
    return {"out": out, "lse": lse}


def _copied(s, moves):
    """The caches with page a's content in page b for each (a, b)."""
    src, dst = (torch.tensor([m[i] for m in moves], dtype=torch.int64, device="cuda") for i in range(2))
    stack = [t.clone() for t in s["stack"]]
    for t, old in zip(stack, s["stack"]):
        t.index_copy_(2, dst, old.index_select(2, src))
    return stack


def _exact_branch(s):
    page = s["case"]["page"]
    table, refs, lens = s["table"].tolist(), s["refs"].tolist(), s["lens"].tolist()
    child, parent, count = s["child"].tolist(), s["parent"].tolist(), s["count"].tolist()
    old = [list(r) for r in table]
    was = list(lens)
    for c, p in zip(child, parent):
        for j in range(-(-was[c] // page)):
            refs[old[c][j]] -= 1
        for j in range(-(-was[p] // page)):
            refs[old[p][j]] += 1
            table[c][j] = old[p][j]
        lens[c] = was[p]
    free = [i for i, r in enumerate(refs) if r == 0]
    moves, slots = [], []
    for c, more in zip(child, count):
        have = -(-lens[c] // page)
        if lens[c] % page and refs[table[c][have - 1]] > 1:
            to = free.pop(0)
            moves.append((table[c][have - 1], to))
            refs[table[c][have - 1]] -= 1
            refs[to] = 1
            table[c][have - 1] = to
        for j in range(have, -(-(lens[c] + more) // page)):
            table[c][j] = free.pop(0)
            refs[table[c][j]] = 1
        slots.append([table[c][n // page] * page + n % page for n in range(lens[c], lens[c] + more)])
        lens[c] += more
    whole = lambda v, dtype: torch.tensor(v, dtype=dtype, device="cuda")  # noqa: E731
    return {"table": whole(table, torch.int32), "refs": whole(refs, torch.int32), "lens": whole(lens, torch.int32),
            "slots": whole(slots, torch.int64), "caches": _copied(s, moves)}


def _exact_compact(s):
    page = s["case"]["page"]
    table, refs, lens = s["table"].tolist(), s["refs"].tolist(), s["lens"].tolist()
    top = sum(r > 0 for r in refs)
    holes = [i for i in range(top) if refs[i] == 0]
    moves = list(zip([i for i in range(top, len(refs)) if refs[i] > 0], holes))
    to = dict(moves)
    for row, n in zip(table, lens):
        for j in range(-(-n // page)):
            row[j] = to.get(row[j], row[j])
    for a, b in moves:
        refs[b], refs[a] = refs[a], 0
    return {"table": torch.tensor(table, dtype=torch.int32, device="cuda"),
            "refs": torch.tensor(refs, dtype=torch.int32, device="cuda"), "caches": _copied(s, moves)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "copy":
        return {"caches": _copied(s, list(zip(s["src"].tolist(), s["dst"].tolist())))}
    return {"rope": _exact_rope, "attn4": _exact_attn4, "branch": _exact_branch, "compact": _exact_compact}[case["op"]](s)
