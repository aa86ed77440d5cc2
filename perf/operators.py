"""The three operators of a decode step around the expert layer, as measured cases.

A step of a mixture-of-experts decoder for a batch of sequences that each add
one token runs, per block: attention of the new token over a paged key-value
cache; the residual's addition with a root-mean-square norm, whose result
goes on in bf16 (router) and, for 8-bit experts, in e4m3 with one scale per
128 columns; and the whole expert layer for those few tokens.  The norm also
runs on the long prompts that fill the cache.

``run`` computes each case in plain torch operations in 32 bits, or, with
``own`` set, by the package's calls.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
GROUP = 128  # columns per 8-bit scale, and rows and columns per weight scale

# Layer shapes (H, F, E, k) that this repository runs.
LAYERS = {
    "tiny": (512, 1024, 8, 2),
    "wide": (4096, 14336, 8, 2),
    "fine": (7168, 2048, 256, 8),
    "medium": (4096, 1536, 128, 8),
}


def listed():
    return [
        # The norm of one sequence's new token before 8-bit experts: pure latency.
        dict(name="norm_1", op="norm", T=1, H=7168, residual=True, out=True, q8=True),
        # No residual yet, and a width that fills neither vectors nor groups: a first layer of an odd model.
        dict(name="norm_odd", op="norm", T=333, H=1001, residual=False, out=True, q8=False),
        # A long prompt's tokens at once: bandwidth.
        dict(name="norm_prompt", op="norm", T=16384, H=4096, residual=True, out=True, q8=True),
        # One user in a chat: few heads of work, a cache that has to be split to fill the GPU.
        dict(name="attn_1", op="attn", B=1, Hq=32, Hkv=8, D=128, page=16, longest=8191, lens="all"),
        # Heads without sharing, short caches, small pages.
        dict(name="attn_heads", op="attn", B=16, Hq=12, Hkv=12, D=64, page=8, longest=1000, lens="mixed"),
        # A server's batch, lengths from none to long, pages that end inside whatever tile is used.
        dict(name="attn_batch", op="attn", B=64, Hq=64, Hkv=8, D=128, page=24, longest=16384, lens="mixed"),
        # A few very long documents.
        dict(name="attn_long", op="attn", B=4, Hq=32, Hkv=8, D=128, page=64, longest=131071, lens="all"),
        # Two tokens through a tiny layer: latency.
        dict(name="moe_tiny", op="moe", T=2, layer="tiny", bits=16, dead=0),
        # One token, two experts of a few wide ones: 0.7 GB of weights.
        dict(name="moe_1", op="moe", T=1, layer="wide", bits=16, dead=0),
        # A batch that uses nearly every expert of a medium layer, a part of them switched off.
        dict(name="moe_batch", op="moe", T=48, layer="medium", bits=16, dead=16),
        # A few tokens over many small experts with 8-bit weights and activations.
        dict(name="moe8_few", op="moe", T=4, layer="fine", bits=8, dead=0),
        # A full decode batch of the same: nearly all 11 GB of weights.
        dict(name="moe8_batch", op="moe", T=128, layer="fine", bits=8, dead=0),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = _draw(rng)
        if 3072 not in case.values():  # a size that nothing here runs
            return case


def _draw(rng):
    op = rng.choice(["norm", "attn", "moe"])
    if op == "norm":
        H = rng.choice([_log_uniform(rng, 64, 8192), 8 * _log_uniform(rng, 8, 1024), 128 * rng.randint(1, 64)])
        T = _log_uniform(rng, 1, 16384 * 4096 // max(H, 4096))
        out, q8 = rng.choice([(True, False), (True, True), (False, True)])
        return dict(op=op, T=T, H=H, residual=rng.random() < 0.75, out=out, q8=q8)
    if op == "attn":
        D, Hkv = rng.choice([(64, 1), (64, 4), (64, 12), (128, 1), (128, 2), (128, 8), (128, 32), (256, 1), (256, 4)])
        G = rng.choice([1, 2, 4, 5, 8, 16, 24])
        longest = _log_uniform(rng, 1, 131072)
        # the plain form holds the caches padded to the longest: at most 4 GiB in 32 bits each
        most = max(1, (1 << 30) // (longest * Hkv * D))
        B = _log_uniform(rng, 1, min(256, most))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([1, 8, 16, 24, 32, 64, 100, 128]),
                    longest=longest, lens=rng.choice(["all", "mixed"]))
    layer = rng.choice(sorted(LAYERS) + ["drawn"])
    bits = rng.choice([8, 16])
    if layer == "drawn":
        unit = 128 if bits == 8 else 64
        E = rng.choice([4, 7, 16, 60, 64])
        return dict(op=op, T=_log_uniform(rng, 1, 128), H=unit * rng.randint(1, 4096 // unit),
                    F=unit * rng.randint(1, 4096 // unit), E=E, k=rng.randint(1, min(E, 8)), bits=bits, dead=0)
    if layer == "fine":
        bits = 8  # in 16 bits the layer alone would take 22 GB
    return dict(op=op, T=_log_uniform(rng, 1, 127), layer=layer, bits=bits,
                dead=rng.choice([0, 0, LAYERS[layer][2] // 8]))


# ------------------------------------------------------------------ shapes --

def _layer(case):
    return LAYERS[case["layer"]] if "layer" in case else tuple(case[n] for n in ("H", "F", "E", "k"))


def _lens(case):
    """Cache lengths: all the longest, or spread over the logarithm with the longest, one token and none among them."""
    B, longest = case["B"], case["longest"]
    if case["lens"] == "all":
        return [longest] * B
    lens = [int((longest + 1) ** ((b + 0.5) / B)) for b in range(B)]
    lens[-1] = longest
    if B > 2:
        lens[0], lens[1] = 0, 1
    order = [(b * 7919 + 3) % B for b in range(B)] if math.gcd(7919, B) == 1 else range(B)
    return [lens[b] for b in order]


def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["H"]
        groups = case["T"] * -(-case["H"] // GROUP)
        cost = 2 * n + 2 * case["H"] + (4 * n if case["residual"] else 0)
        cost += (2 * n if case["out"] else 0) + (n + 4 * groups if case["q8"] else 0)
        return {"bytes": cost, "flops": 6 * n}
    if case["op"] == "attn":
        tokens, D, Hq = sum(_lens(case)), case["D"], case["Hq"]
        pages = sum(-(-n // case["page"]) for n in _lens(case))
        cost = 4 * tokens * case["Hkv"] * D + 4 * pages + case["B"] * (4 * Hq * D + 4 * Hq + 4)
        return {"bytes": cost, "flops": 4 * tokens * Hq * D}
    H, F, E, k = _layer(case)
    T, size = case["T"], case["bits"] // 8
    live = E - case["dead"]
    used = live * (1 - (1 - min(k, live) / live) ** T)  # experts that some token chooses, on average
    cost = used * 3 * H * F * size + T * (H * size + 2 * H + 4 * E)
    if size == 1:
        cost += used * 3 * 4 * (H // GROUP) * (F // GROUP) + 4 * T * (H // GROUP)
    return {"bytes": cost, "flops": 6 * T * k * H * F}


# ------------------------------------------------------------------ inputs --

def _quantized_weights(gen, E, rows, cols):
    """Normal weights of variance 1/rows in e4m3 with a scale per 128 x 128 block, some experts at a time."""
    w8 = torch.empty((E, rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((E, rows // GROUP, cols // GROUP), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 28) // (rows * cols))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.randn((n, rows // GROUP, GROUP, cols // GROUP, GROUP), generator=gen, device="cuda")
        w *= rows ** -0.5
        s = w.abs().amax(dim=(2, 4)) / E4M3_MAX
        scale[e:e + n] = s
        w8[e:e + n] = (w / s[:, :, None, :, None]).view(n, rows, cols).to(torch.float8_e4m3fn)
    return w8, scale


def _quantized_rows(x):
    """e4m3 values and a scale per row and 128 columns (H a multiple of 128)."""
    g = x.view(x.shape[0], -1, GROUP)
    s = g.abs().amax(dim=2) / E4M3_MAX
    return (g / s[:, :, None]).view_as(x).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    state = {"case": case}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        state["x"] = randn(T, H).bfloat16()
        # a residual stream: a few columns are far larger than the rest
        state["residual"] = (randn(T, H) * (1 + 30 * (randn(H) > 2.5))).bfloat16() if case["residual"] else None
        state["weight"] = (1 + 0.1 * randn(H)).bfloat16()
    elif case["op"] == "attn":
        B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
        lens = _lens(case)
        need = [-(-n // page) for n in lens]
        most = max(max(need), 1)
        pages = max(sum(need), 1) + 3
        # keys and values of a page side by side, pages given out in random order
        kv = torch.empty((pages, 2, page, Hkv, D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros((B, most), dtype=torch.int32, device="cuda")
        used = torch.tensor(need, device="cuda")
        at = torch.arange(most, device="cuda")[None, :] < used[:, None]
        table[at] = order[:sum(need)]
        state.update(k=kv[:, 0], v=kv[:, 1], table=table, scale=D ** -0.5,
                     lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                     q=(1.5 * randn(B, case["Hq"], D)).bfloat16())
    else:
        H, F, E, k = _layer(case)
        T = case["T"]
        x, logits = randn(T, H), randn(T, E)
        if case["dead"]:
            logits[:, torch.randperm(E, generator=gen, device="cuda")[:case["dead"]]] = -math.inf
        state.update(logits=logits, k=k)
        if case["bits"] == 8:
            state["x"], state["x_scale"] = _quantized_rows(x)
            for name, rows, cols in (("W1", H, F), ("W3", H, F), ("W2", F, H)):
                state[name], state[name + "_scale"] = _quantized_weights(gen, E, rows, cols)
        else:
            state["x"] = x.bfloat16()
            for name, rows, cols in (("W1", H, F), ("W3", H, F), ("W2", F, H)):
                w = torch.empty((E, rows, cols), dtype=torch.bfloat16, device="cuda")
                state[name] = w.normal_(std=rows ** -0.5, generator=gen)
    return state


# -------------------------------------------------------------- plain form --

def _quantize(y):
    """e4m3 values of each row and the scale per 128 columns: the largest magnitude maps to 448."""
    T, H = y.shape
    padded = torch.nn.functional.pad(y, (0, -H % GROUP)).view(T, -1, GROUP)
    amax = padded.abs().amax(dim=2)
    scale = torch.where(amax < 2.0 ** -100, torch.ones_like(amax), amax / E4M3_MAX)
    return (padded / scale[:, :, None]).view(T, -1)[:, :H].to(torch.float8_e4m3fn), scale


def _plain_norm(s):
    x = s["x"].float()
    got = {}
    if s["residual"] is not None:
        x = x + s["residual"].float()
        got["residual"] = x.bfloat16()
    y = x * torch.rsqrt(x.square().mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    if s["case"]["out"]:
        got["out"] = y.bfloat16()
    if s["case"]["q8"]:
        got["out8"], got["scale"] = _quantize(y)
    return got


def _plain_attn(s):
    q, lens, page = s["q"], s["lens"].long(), s["case"]["page"]
    B, Hq, D = q.shape
    Hkv, longest = s["k"].shape[2], s["case"]["longest"]
    key = torch.arange(longest, device=q.device)
    where = s["table"][:, key // page].long()
    k = s["k"][where, key % page].float()  # [B, longest, Hkv, D]
    v = s["v"][where, key % page].float()
    valid = (key[None, :] < lens[:, None])[:, None, None, :]
    scores = torch.einsum("bhgd,blhd->bhgl", q.float().view(B, Hkv, Hq // Hkv, D), k) * s["scale"]
    scores = scores.masked_fill(~valid, -math.inf)
    top = scores.amax(dim=3, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(dim=3, keepdim=True)
    v = v.masked_fill(~valid[:, 0, 0, :, None, None], 0.0)
    out = torch.einsum("bhgl,blhd->bhgd", p, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = torch.where(total == 0, torch.full_like(total, -math.inf), top + torch.log(total))
    return {"out": out.reshape(B, Hq, D).bfloat16(), "lse": lse.reshape(B, Hq)}


def _rows_of(s, name, experts):
    """The experts' matrices in 32 bits, one for each entry of `experts`."""
    w = s[name]
    if w.dtype == torch.bfloat16:
        return w[experts].float()
    n, rows, cols = len(experts), w.shape[1], w.shape[2]
    f = w.view(torch.uint8)[experts].view(torch.float8_e4m3fn).float()
    f = f.view(n, rows // GROUP, GROUP, cols // GROUP, GROUP)
    f *= s[name + "_scale"][experts][:, :, None, :, None]
    return f.view(n, rows, cols)


def _plain_moe(s):
    T, H = s["x"].shape
    k, F = s["k"], s["W1"].shape[2]
    value, chosen = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    value, chosen = value[:, :k], chosen[:, :k].reshape(-1)
    top = value[:, :1]
    gate = torch.exp(value - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = gate.sum(dim=1, keepdim=True)
    gate = gate / torch.where(total == 0, torch.ones_like(total), total)
    x = s["x"].float()
    if "x_scale" in s:
        x = (x.view(T, -1, GROUP) * s["x_scale"][:, :, None]).view(T, H)
    x = x.repeat_interleave(k, dim=0)[:, None, :]
    y = torch.empty((T * k, H), dtype=torch.float32, device=x.device)
    step = max(1, (1 << 29) // (H * F))  # (token, expert) pairs whose matrices are gathered together
    for r in range(0, T * k, step):
        e = chosen[r:r + step]
        a = torch.bmm(x[r:r + step], _rows_of(s, "W1", e))
        h = a / (1 + torch.exp(-a)) * torch.bmm(x[r:r + step], _rows_of(s, "W3", e))
        if "x_scale" in s:
            h8, hs = _quantize(h[:, 0])
            h = (h8.float().view(len(e), -1, GROUP) * hs[:, :, None]).view(len(e), 1, F)
        y[r:r + step] = torch.bmm(h, _rows_of(s, "W2", e))[:, 0]
    return {"out": (y.view(T, k, H) * gate[:, :, None]).sum(dim=1).bfloat16()}


# --------------------------------------------------------------------- run --

def run(state):
    case = state["case"]
    if not own:
        return {"norm": _plain_norm, "attn": _plain_attn, "moe": _plain_moe}[case["op"]](state)
    import moe_token_dispatch_persistent_gb300 as mk

    if case["op"] == "norm":
        return mk.add_rmsnorm(state["x"], state["weight"], residual=state["residual"], eps=EPS, bf16=case["out"],
                              e4m3=case["q8"], check=False)
    if case["op"] == "attn":
        return mk.paged_attention(state["q"], state["k"], state["v"], state["table"], state["lens"],
                                  scale=state["scale"], check=False)
    scales = {n: state[n] for n in ("x_scale", "W1_scale", "W3_scale", "W2_scale") if n in state}
    return mk.moe_ffn_decode(state["x"], state["logits"], state["W1"], state["W3"], state["W2"], state["k"],
                             check=False, **scales)


# ----------------------------------------------------- 64 bits, from the definitions --

def _e4m3_groups(y):
    """Round each row's groups of 128 to e4m3 after scaling its largest magnitude to 448; values, scales."""
    q, scales = torch.empty_like(y), []
    for c in range(0, y.shape[1], GROUP):
        part = y[:, c:c + GROUP]
        s = part.abs().max(dim=1, keepdim=True).values / E4M3_MAX
        s = torch.where(s == 0, torch.ones_like(s), s)
        q[:, c:c + GROUP] = (part / s).to(torch.float8_e4m3fn).double()
        scales.append(s)
    return q, torch.cat(scales, dim=1)


def _exact_norm(s):
    z = s["x"].double()
    if s["residual"] is not None:
        z = z + s["residual"].double()
    y = z / (z.pow(2).sum(dim=1, keepdim=True) / z.shape[1] + EPS).sqrt() * s["weight"].double()
    got = {"out": y if s["case"]["out"] else None}
    if s["residual"] is not None:
        got["residual"] = z
    if s["case"]["q8"]:
        got["out8"], got["scale"] = _e4m3_groups(y)
    return got


def _exact_attn(s):
    B, Hq, D = s["q"].shape
    Hkv, page = s["k"].shape[2], s["case"]["page"]
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        for h in range(Hkv):
            keys = s["k"][pages, :, h].reshape(-1, D)[:n].double()
            values = s["v"][pages, :, h].reshape(-1, D)[:n].double()
            mine = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            scores = (s["q"][b, mine].double() @ keys.T) * s["scale"]
            lse[b, mine] = torch.logsumexp(scores, dim=1)
            out[b, mine] = torch.softmax(scores, dim=1) @ values
    return {"out": out, "lse": lse}


def _exact_moe(s):
    def matrix(name, e):
        w = s[name][e].double()
        if name + "_scale" in s:
            w = w * s[name + "_scale"][e].double().repeat_interleave(GROUP, 0).repeat_interleave(GROUP, 1)
        return w

    x, k = s["x"].double(), s["k"]
    if "x_scale" in s:
        x = x * s["x_scale"].double().repeat_interleave(GROUP, 1)
    out = torch.zeros_like(x)
    chosen, gates = [], []
    for row in s["logits"].double().cpu().tolist():
        best = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        weight = [math.exp(row[e] - row[best[0]]) if row[e] > -math.inf else 0.0 for e in best]
        chosen.append(best)
        gates.append([w / sum(weight) if sum(weight) else 0.0 for w in weight])
    for e in range(s["W1"].shape[0]):
        at = [(t, j) for t, best in enumerate(chosen) for j, c in enumerate(best) if c == e]
        if not at:
            continue
        rows = torch.tensor([t for t, _ in at], device="cuda")
        gate = torch.tensor([gates[t][j] for t, j in at], dtype=torch.float64, device="cuda")
        a = x[rows] @ matrix("W1", e)
        h = a * torch.sigmoid(a) * (x[rows] @ matrix("W3", e))
        if "x_scale" in s:
            q, scale = _e4m3_groups(h)
            h = q * scale.repeat_interleave(GROUP, 1)
        out.index_add_(0, rows, gate[:, None] * (h @ matrix("W2", e)))
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "attn": _exact_attn, "moe": _exact_moe}[case["op"]](s)
