"""The operators of one decoding step, each with its plain form and its cases.

A model whose linears hold 4-bit weights and whose keys and values are kept in
a paged cache answers one token at a time with four operators:

  quantize  weights to 4-bit codes with one step per group of inputs (once)
  gemv      a few tokens times those weights
  append    new keys and values into the paged cache, rotated on the way
  attend    one new token of every sequence against its cached keys and values

`run` computes them with elementary torch operations, or, where `own` is set,
with the calls of `w4a4_post_quantized_b200.w4a4`.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
FRAME = 1374  # tokens of one frame: 37 x 37 patches and 5 special tokens


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a 1024-wide layer's projection prepared for decoding, groups of 128 inputs
        {"name": "quantize 1024x1024", "op": "quantize", "dtype": "bf16", "N": 1024, "K": 1024, "group": 128},
        # the fc1 of an 8192-wide model, small groups
        {"name": "quantize 20000x8192", "op": "quantize", "dtype": "fp16", "N": 20000, "K": 8192, "group": 32},
        # one token through a 1024-wide layer's projection: latency
        {"name": "gemv m1 1024x1024", "op": "gemv", "dtype": "bf16", "M": 1, "N": 1024, "K": 1024, "group": 128,
         "bias": True},
        # five tokens (a small batch) through fc2, odd output width
        {"name": "gemv m5 1021x4096", "op": "gemv", "dtype": "fp16", "M": 5, "N": 1021, "K": 4096, "group": 32,
         "bias": False},
        # a batch of eight through a large output layer: weight traffic
        {"name": "gemv m8 32768x8192", "op": "gemv", "dtype": "bf16", "M": 8, "N": 32768, "K": 8192, "group": 128,
         "bias": True},
        # a decoding step of 16 sequences, 16 heads of 64
        {"name": "append t16", "op": "append", "dtype": "bf16", "T": 16, "S": 16, "Hq": 16, "Hkv": 16, "D": 64,
         "rot": 64, "pairs": False, "page": 16, "layout": "nhd"},
        # 8 frames of a scene enter the cache, queries rotated with them
        {"name": "append 8 frames", "op": "append", "dtype": "bf16", "T": 8 * FRAME, "S": 8, "Hq": 16, "Hkv": 16,
         "D": 64, "rot": 64, "pairs": False, "page": 64, "layout": "hnd"},
        # a ragged batch of prompts, shared heads, part of each head rotated, in pairs
        {"name": "append ragged prompts", "op": "append", "dtype": "fp16", "T": 5003, "S": 23, "Hq": 32, "Hkv": 8,
         "D": 128, "rot": 64, "pairs": True, "page": 24, "layout": "nhd"},
        # one sequence over one frame: latency
        {"name": "attend b1 1 frame", "op": "attend", "dtype": "bf16", "B": 1, "L": FRAME, "spread": 1.0, "Hq": 16,
         "Hkv": 16, "D": 64, "page": 16, "window": 0, "layout": "nhd"},
        # one sequence over 64 frames: the cache is split to fill the GPU
        {"name": "attend b1 64 frames", "op": "attend", "dtype": "bf16", "B": 1, "L": 64 * FRAME, "spread": 1.0,
         "Hq": 16, "Hkv": 16, "D": 64, "page": 64, "window": 0, "layout": "hnd"},
        # a ragged batch with shared heads, one sequence empty, pages that end inside a tile
        {"name": "attend b23 ragged", "op": "attend", "dtype": "fp16", "B": 23, "L": 4001, "spread": 0.02, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 24, "window": 0, "layout": "nhd"},
        # a full serving batch over long caches
        {"name": "attend b64 8k", "op": "attend", "dtype": "bf16", "B": 64, "L": 8192, "spread": 0.5, "Hq": 32,
         "Hkv": 4, "D": 128, "page": 64, "window": 0, "layout": "hnd"},
    ]


def log_int(rng, low, high):
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    op = rng.choice(["quantize", "gemv", "gemv", "append", "append", "attend", "attend", "attend"])
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16"])}
    if op in ("quantize", "gemv"):
        group = rng.choice([32, 64, 128])
        case.update(N=log_int(rng, 257, 16384), K=group * max(1, log_int(rng, 512, 8192) // group), group=group)
        if op == "gemv":
            case.update(M=log_int(rng, 1, 16), bias=rng.random() < 0.5)
        return case
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    G = rng.choice([1, 1, 2, 4, 5, 8, 12])
    case.update(Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([1, 7, 16, 24, 32, 64, 128]),
                layout=rng.choice(["nhd", "hnd"]))
    if op == "append":
        T = log_int(rng, 1, 6000)
        case.update(T=T, S=min(T, log_int(rng, 1, 64)), rot=rng.choice([D, D // 2]), pairs=rng.random() < 0.5)
    else:
        B = log_int(rng, 1, 64)
        L = log_int(rng, 1, max(1, min(60000, 250_000_000 // (B * Hkv * D))))
        case.update(B=B, L=L, spread=rng.choice([1.0, 0.5, 0.02]), window=rng.choice([0, 0, 1 + L // 3]))
    return case


# --------------------------------------------- sizes that follow from a case
def lengths(case):
    """Cached tokens of every sequence: from L down to spread * L, and where
    the batch is ragged one sequence that has none yet."""
    B, L, spread = case["B"], case["L"], case["spread"]
    out = [max(1, int(L * (1.0 - (1.0 - spread) * ((i * 7919) % B) / B))) for i in range(B)]
    if spread < 0.1 and B > 2:
        out[B // 2] = 0
    return out


def seen(case):
    """Tokens that every sequence's new token attends to."""
    w = case["window"]
    return [min(n, w) if w else n for n in lengths(case)]


def token_counts(case):
    """New tokens of every sequence in an append: T split unevenly over S."""
    T, S = case["T"], case["S"]
    cuts = [T * i // S for i in range(S + 1)]
    for i in range(1, S):
        room = cuts[i + 1] - cuts[i]
        cuts[i] += (room * ((i * 37) % 11)) // 23
    return [cuts[i + 1] - cuts[i] for i in range(S)]


def start_of(i):
    """Tokens that sequence i of an append holds already."""
    return (i * 131) % 200


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["N"] * case["K"]
        return {"bytes": 4 * n, "flops": 4 * n}
    if op == "gemv":
        M, N, K = case["M"], case["N"], case["K"]
        nbytes = N * K // 2 + 2 * N * (K // case["group"]) + 2 * M * (K + N) + (2 * N if case["bias"] else 0)
        return {"bytes": nbytes, "flops": 2 * M * N * K}
    if op == "append":
        T, D = case["T"], case["D"]
        per_token = 2 * 2 * D * (case["Hq"] + 2 * case["Hkv"]) + 4 * case["rot"] + 8
        return {"bytes": T * per_token, "flops": 3 * T * case["rot"] * (case["Hq"] + case["Hkv"])}
    tokens, D = sum(seen(case)), case["D"]
    nbytes = 2 * 2 * tokens * case["Hkv"] * D + 2 * 2 * case["B"] * case["Hq"] * D
    return {"bytes": nbytes, "flops": 4 * tokens * case["Hq"] * D}


# ------------------------------------------------------------------ inputs
def randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def page_table(gen, counts, page):
    """Pages of every sequence in a shuffled pool, and the pool's size; unused
    entries of the table are -1."""
    need = [-(-n // page) for n in counts]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(counts), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, total


def pool(gen, pages, case, dtype):
    """A cache of keys or values as [pages, page, heads, D], in either memory order."""
    H, D, page = case["Hkv"], case["D"], case["page"]
    if case["layout"] == "hnd":
        return randn(gen, pages, H, page, D, dtype=dtype).transpose(1, 2)
    return randn(gen, pages, page, H, D, dtype=dtype)


def rotation_table(n, rot, base=10000.0):
    """cos in the first half of each row, sin in the second; angles in 64 bits."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    op = case["op"]
    if op == "quantize":
        state = {"W": randn(gen, case["N"], case["K"], dtype=dtype, scale=0.02), "group": case["group"]}
        if own:
            from w4a4_post_quantized_b200 import w4a4
            state["out"] = w4a4.GroupWeights(case["N"], case["K"], case["group"], dtype)
    elif op == "gemv":
        M, N, K, group = case["M"], case["N"], case["K"], case["group"]
        codes = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        scales = (torch.rand(N, K // group, generator=gen, device="cuda") * 0.004 + 0.004).to(dtype)
        x = torch.randn(M, K, generator=gen, device="cuda")
        x[:, torch.randint(0, K, (8,), generator=gen, device="cuda")] *= 15.0  # outlier channels
        state = {"X": x.to(dtype), "bias": randn(gen, N, dtype=dtype, scale=0.01) if case["bias"] else None}
        if own:
            from w4a4_post_quantized_b200 import w4a4
            state["w"] = w4a4.w4a4_group_pack(codes, scales)
        else:
            state.update(codes=codes, scales=scales, group=group)
    elif op == "append":
        T, D, Hq, Hkv = case["T"], case["D"], case["Hq"], case["Hkv"]
        counts = token_counts(case)
        ends = [start_of(i) + n for i, n in enumerate(counts)]
        pages, total = page_table(gen, ends, case["page"])
        seq = torch.tensor([i for i, n in enumerate(counts) for _ in range(n)], dtype=torch.int32)
        pos = torch.tensor([start_of(i) + j for i, n in enumerate(counts) for j in range(n)], dtype=torch.int32)
        # q, k and v as the views of one linear's output
        qkv = randn(gen, T, Hq + 2 * Hkv, D, dtype=dtype)
        state = {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv], "v": qkv[:, Hq + Hkv:],
                 "K": pool(gen, total, case, dtype), "V": pool(gen, total, case, dtype),
                 "pages": pages, "seq": seq.cuda(), "pos": pos.cuda(), "pairs": case["pairs"],
                 "table": rotation_table(max(ends), case["rot"])}
        if own:
            from w4a4_post_quantized_b200 import w4a4
            state["cache"] = w4a4.KVCache(state["K"], state["V"])
    else:
        lens = lengths(case)
        pages, total = page_table(gen, lens, case["page"])
        state = {"q": randn(gen, case["B"], case["Hq"], case["D"], dtype=dtype, scale=1.5),
                 "K": pool(gen, total, case, dtype), "V": pool(gen, total, case, dtype), "pages": pages,
                 "lens": torch.tensor(lens, dtype=torch.int32).cuda(), "window": case["window"]}
        if own:
            from w4a4_post_quantized_b200 import w4a4
            state["cache"] = w4a4.KVCache(state["K"], state["V"])
            state["workspace"] = torch.empty(
                w4a4.w4a4_kv_attend_workspace_bytes(case["B"], case["Hq"], case["Hkv"], case["D"]),
                dtype=torch.uint8, device="cuda")
    state["op"] = op
    return state


# --------------------------------------------------------------- plain forms
def plain_quantize(s):
    W, g = s["W"], s["group"]
    N, K = W.shape
    w = W.float().view(N, K // g, g)
    step = (w.abs().amax(2, keepdim=True) / 7.0).to(W.dtype).float()
    code = torch.where(step > 0, torch.round(w / torch.where(step > 0, step, 1.0)), 0.0).clamp(-8, 7)
    return (code * step).to(W.dtype).view(N, K)


def unpacked(codes):
    """[N, K/2] bytes to [N, K] signed codes: element 2i in the low nibble."""
    c = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1)
    return (c ^ 8).to(torch.int16) - 8


def plain_gemv(s):
    X, group = s["X"], s["group"]
    w = unpacked(s["codes"]).float().view(s["codes"].shape[0], -1, group) * s["scales"].float()[:, :, None]
    y = X.float() @ w.view(w.shape[0], -1).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(X.dtype)


def rotated(x, cos, sin, pairs):
    """The first 2 * cos.shape[1] elements of every head turned by the token's
    angles: element i with element i + half, or neighbours (2i, 2i + 1)."""
    half = cos.shape[1]
    c, s = cos[:, None, :], sin[:, None, :]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (head[..., 0::2], head[..., 1::2]) if pairs else (head[..., :half], head[..., half:])
    ra, rb = a * c - b * s, b * c + a * s
    head = torch.stack([ra, rb], -1).flatten(-2) if pairs else torch.cat([ra, rb], -1)
    return torch.cat([head, rest], -1)


def plain_append(s):
    pos, page = s["pos"].long(), s["K"].shape[1]
    at = s["pages"][s["seq"].long(), pos // page].long(), pos % page
    half = s["table"].shape[1] // 2
    cos, sin = s["table"][pos, :half], s["table"][pos, half:]
    dtype = s["k"].dtype
    s["K"][at] = rotated(s["k"].float(), cos, sin, s["pairs"]).to(dtype)
    s["V"][at] = s["v"]
    return {"q": rotated(s["q"].float(), cos, sin, s["pairs"]).to(dtype), "K": s["K"], "V": s["V"]}


def plain_attend(s):
    q, lens, page = s["q"], s["lens"], s["K"].shape[1]
    B, Hq, D = q.shape
    Hkv = s["K"].shape[2]
    table = s["pages"].clamp(min=0).long()
    L = table.shape[1] * page
    at = torch.arange(L, device=q.device)
    live = at < lens[:, None]
    if s["window"]:
        live = live & (at >= lens[:, None] - s["window"])
    k = s["K"][table].reshape(B, L, Hkv, D).permute(0, 2, 3, 1).float()
    v = s["V"][table].reshape(B, L, Hkv, D).permute(0, 2, 1, 3).float()
    v = torch.where(live[:, None, :, None], v, 0.0)
    scores = (q.float().view(B, Hkv, Hq // Hkv, D) @ k) / math.sqrt(D)
    scores = torch.where(live[:, None, None, :], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0.0, 1.0, total)
    return out.view(B, Hq, D).to(q.dtype)


def run(state):
    op = state["op"]
    if own:
        from w4a4_post_quantized_b200 import w4a4
        if op == "quantize":
            return w4a4.w4a4_group_dequantize(w4a4.w4a4_group_quantize(state["W"], state["group"], out=state["out"]))
        if op == "gemv":
            return w4a4.w4a4_group_gemv(state["X"], state["w"], state["bias"])
        if op == "append":
            flags = w4a4.W4A4_FLAG_ROPE_PAIRS if state["pairs"] else 0
            q = w4a4.w4a4_kv_append(state["cache"], state["k"], state["v"], state["pages"], state["pos"],
                                    q=state["q"], table=state["table"], seq=state["seq"], flags=flags)
            return {"q": q, "K": state["K"], "V": state["V"]}
        return w4a4.w4a4_kv_attend(state["q"], state["cache"], state["pages"], state["lens"],
                                   window=state["window"], workspace=state["workspace"])
    return {"quantize": plain_quantize, "gemv": plain_gemv, "append": plain_append, "attend": plain_attend}[op](state)


# ------------------------------------------------- the definitions in 64 bits
def exact_quantize(s):
    out = []
    for rows in s["W"].split(4096):
        w = rows.double().unflatten(1, (-1, s["group"]))
        step = (w.abs().max(2).values / 7).to(rows.dtype).double().unsqueeze(2)
        live = step != 0
        code = torch.round(w / torch.where(live, step, torch.ones_like(step)))
        code = torch.minimum(torch.maximum(code, torch.full_like(code, -8)), torch.full_like(code, 7))
        out.append(torch.where(live, code * step, torch.zeros_like(w)).flatten(1))
    return torch.cat(out)


def exact_gemv(s):
    X = s["X"].double()
    parts = []
    for codes, scales in zip(s["codes"].split(2048), s["scales"].split(2048)):
        w = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
        w[:, 0::2] = (codes % 16).double()
        w[:, 1::2] = (codes // 16).double()
        w = torch.where(w > 7, w - 16, w) * scales.double().repeat_interleave(s["group"], 1)
        parts.append(X @ w.T)
    y = torch.cat(parts, 1)
    return y if s["bias"] is None else y + s["bias"].double()


def exact_append(s):
    n, rot = s["table"].shape
    turn = torch.complex(s["table"][:, :rot // 2].double(), s["table"][:, rot // 2:].double())[s["pos"].long()][:, None]

    def turned(x):
        x = x.double()
        r = x[..., :rot]
        z = r.unflatten(-1, (-1, 2)) if s["pairs"] else r.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        r = z.flatten(-2) if s["pairs"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([r, x[..., rot:]], -1)

    K, V = s["K"].double(), s["V"].double()
    page = K.shape[1]
    pos = s["pos"].long()
    row = s["pages"].long()[s["seq"].long(), torch.div(pos, page, rounding_mode="floor")]
    K.index_put_((row, pos % page), turned(s["k"]))
    V.index_put_((row, pos % page), s["v"].double())
    return {"q": turned(s["q"]), "K": K, "V": V}


def exact_attend(s):
    q, page = s["q"].double(), s["K"].shape[1]
    B, Hq, D = q.shape
    out = torch.zeros_like(q)
    for b, n in enumerate(s["lens"].tolist()):
        first = max(0, n - s["window"]) if s["window"] else 0
        if n == first:
            continue
        at = torch.arange(first, n, device=q.device)
        rows = s["pages"][b].long()[at // page], at % page
        k, v = s["K"][rows], s["V"][rows]
        group = Hq // k.shape[1]
        for h in range(k.shape[1]):
            heads = slice(h * group, (h + 1) * group)
            weight = torch.softmax(q[b, heads] @ k[:, h].double().T * D ** -0.5, -1)
            out[b, heads] = weight @ v[:, h].double()
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = was
    return {"quantize": exact_quantize, "gemv": exact_gemv, "append": exact_append, "attend": exact_attend}[
        case["op"]](state)
