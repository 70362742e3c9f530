"""Measured cases of the paged 2-bit cache and the operators around it.

Five passes stand for how a serving program uses them:

  rope     rotary positions applied to a step's queries and keys (or undone: the gradient)
  attend   attention of each sequence's new tokens over its pages, its residual and the new tokens themselves
  extend   a branch of each sequence takes a chunk of tokens, is read back dequantized and is freed
  branch   every sequence is forked, each fork takes one token and attends, and the forks are freed (a search step)
  compact  sequences are copied to new pages, the old ones freed, the pool compacted and the copies read back

The 2-bit code of the cache: groups of 32 (keys: 32 tokens of one channel; values: 32 channels of one token), scale =
fp16((max - min) / 3), zero = fp16(min), code = clamp(rint((x - zero) / scale), 0, 3) in fp32, value = zero + scale * code.
The newest tokens (1 to R of them) stay as they are.
"""
import math

import torch

own = False

G = 32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---- cases ----------------------------------------------------------------------
def listed():
    return [
        # One decode step of a batch of 64: rotate 64 tokens' heads (latency).
        dict(name="rope step", op="rope", tokens=64, H_q=32, H_kv=8, D=128, rot=128, layout="half", scaling="none",
             inverse=False, start=4095, dtype="bf16"),
        # A long prompt, interleaved pairs on half of the head, frequencies stretched for long contexts.
        dict(name="rope prompt partial", op="rope", tokens=16384, H_q=32, H_kv=32, D=128, rot=64, layout="interleaved",
             scaling="yarn", inverse=False, start=100000, dtype="fp16"),
        # The gradient of a rotation (odd token count, head_dim 64).
        dict(name="rope gradient", op="rope", tokens=8191, H_q=40, H_kv=8, D=64, rot=64, layout="half",
             scaling="linear", inverse=True, start=0, dtype="bf16"),
        # One new token for each of a few short sequences (latency).
        dict(name="attend small", op="attend", B=2, H_q=2, H_kv=2, D=64, R=128, T=256, n=1, ragged=False, dtype="fp16",
             outliers=2, outlier_scale=50.0),
        # One new token, one query head per kv head, batch 8 at 4K tokens.
        dict(name="attend token mha", op="attend", B=8, H_q=32, H_kv=32, D=128, R=128, T=4096, n=1, ragged=False,
             dtype="bf16", outliers=4, outlier_scale=100.0),
        # One new token, four query heads per kv head, 32 sequences between 16K and 8K tokens.
        dict(name="attend token gqa", op="attend", B=32, H_q=32, H_kv=8, D=128, R=128, T=16384, n=1, ragged=True,
             dtype="bf16", outliers=2, outlier_scale=200.0),
        # Verification of five drafted tokens per sequence, ragged.
        dict(name="attend draft", op="attend", B=16, H_q=32, H_kv=8, D=128, R=64, T=8001, n=5, ragged=True,
             dtype="fp16", outliers=2, outlier_scale=20.0),
        # Chunked prefill: 500-token chunks of four requests of different lengths.
        dict(name="attend chunk", op="attend", B=4, H_q=32, H_kv=8, D=128, R=128, T=6000, n=500, ragged=True,
             dtype="bf16", outliers=2, outlier_scale=20.0),
        # The next 2K-token chunk of one long context.
        dict(name="attend long chunk", op="attend", B=1, H_q=32, H_kv=8, D=128, R=128, T=30001, n=2048, ragged=False,
             dtype="bf16", outliers=2, outlier_scale=20.0),
        # Chunks written for a batch of requests (quantize what leaves the residual, then read back).
        dict(name="extend chunk", op="extend", B=8, H_kv=8, D=128, R=128, T=1000, n=2048, ragged=True, dtype="bf16",
             outliers=2, outlier_scale=200.0),
        # A search step: eight sequences, four branches each.
        dict(name="branch step", op="branch", B=8, branches=4, H_q=32, H_kv=8, D=128, R=128, T=4224, n=1, ragged=True,
             dtype="bf16", outliers=2, outlier_scale=20.0),
        # Defragmentation: sequences moved to the front of the pool.
        dict(name="compact", op="compact", B=6, H_kv=8, D=128, R=64, T=5000, n=0, ragged=True, dtype="fp16", outliers=2,
             outlier_scale=20.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "attend", "extend", "branch", "compact"])
    dtype = rng.choice(["bf16", "fp16"])
    D = rng.choice([64, 128, 128])
    if op == "rope":
        H_kv = rng.choice([1, 2, 5, 8, 32])
        return dict(op=op, tokens=_log(rng, 1, 16000), H_q=H_kv * rng.choice([1, 2, 4]) if H_kv < 32 else 32, H_kv=H_kv,
                    D=D, rot=rng.choice([D, D, D // 2, D // 4]), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "yarn"]), inverse=rng.random() < 0.3,
                    start=_log(rng, 1, 400000), dtype=dtype)
    H_kv = rng.choice([1, 2, 3, 8, 8, 16])
    c = dict(op=op, B=_log(rng, 1, 16), H_q=H_kv * rng.choice([1, 2, 3, 4, 4, 8]), H_kv=H_kv, D=D,
             R=rng.choice([32, 64, 128, 128]), T=_log(rng, 1, 16000), n=1, ragged=rng.random() < 0.7, dtype=dtype,
             outliers=2, outlier_scale=rng.choice([1.0, 20.0, 100.0]))
    if op == "attend":
        c["n"] = _log(rng, 1, 2048)
    elif op == "extend":
        c.pop("H_q")
        c.update(n=_log(rng, 1, 2048), T=_log(rng, 1, 2000))
    elif op == "branch":
        c.update(branches=rng.choice([1, 2, 3, 4]), T=_log(rng, 1, 5000))
    else:
        c.pop("H_q")
        c.update(n=0, T=_log(rng, 1, 6000))
    top = {x["op"]: x for x in listed()}["compact" if op == "compact" else op]
    if op == "attend":   # below the long chunk's products and a quarter of the large batch's cache
        top = [x for x in listed() if x["name"] == "attend long chunk"][0]
        while c["B"] > 1 and (c["B"] * c["H_q"] * c["n"] * (c["T"] + c["n"]) > top["H_q"] * top["n"] * top["T"] // 2
                              or c["B"] * c["H_kv"] * c["T"] > 1 << 20):
            c["B"] = (c["B"] + 1) // 2
        while c["H_q"] * c["n"] * (c["T"] + c["n"]) > top["H_q"] * top["n"] * top["T"] // 2:
            c["n"] = (c["n"] + 1) // 2
    else:
        while c["B"] > 1 and (c["B"] * c["H_kv"] * (c["T"] + c["n"]) * c["D"] * c.get("branches", 1)
                              > top["B"] * top["H_kv"] * (top["T"] + top["n"]) * top["D"] * top.get("branches", 1)):
            c["B"] = (c["B"] + 1) // 2
    return c


def _lengths(c):
    """Cached and new tokens of each sequence; ragged: from the full length down to about half of it."""
    B = c["B"]
    cut = [b / (2 * B) if c["ragged"] else 0.0 for b in range(B)]
    return ([max(1, int(c["T"] * (1 - x))) for x in cut], [max(min(1, c["n"]), int(c["n"] * (1 - x))) for x in cut])


def _split(T, R):
    n_q = R * ((T - 1) // R) if T > 0 else 0
    return n_q, T - n_q


# ---- inputs ----------------------------------------------------------------------
def _frequencies(c):
    """Inverse frequencies (fp64, to be rounded to fp32) and the factor on cosine and sine."""
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64)
    f = 10000.0 ** (-i / c["rot"])
    if c["scaling"] == "linear":
        return f / 4.0, 1.0
    if c["scaling"] == "yarn":   # by parts: turns over 4096 positions, blended between 1 and 32 of them; factor 16
        turns = 4096.0 * f / (2 * math.pi)
        keep = ((turns.log() - math.log(1.0)) / (math.log(32.0) - math.log(1.0))).clamp(0, 1)
        return f * keep + f / 16.0 * (1 - keep), 0.1 * math.log(16.0) + 1.0
    return f, 1.0


def _rope_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    N, H = c["tokens"], c["H_q"] + 2 * c["H_kv"]
    qkv = torch.randn((N, H, c["D"]), generator=g, device="cuda").to(dt)      # one projection's output
    f, m = _frequencies(c)
    return dict(q=qkv[:, :c["H_q"]], k=qkv[:, c["H_q"]:c["H_q"] + c["H_kv"]],
                positions=(torch.arange(N, device="cuda") + c["start"] + seed % 7).to(torch.int32),
                inv_freq=f.to(torch.float32).to("cuda"), m=m)


def _kv_inputs(c, seed):
    """Per sequence history K, V [T_b, H_kv, D], and the new tokens' q, k, v, rows of one sequence after another."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    H, D = c["H_kv"], c["D"]
    T, n = _lengths(c)
    scale = torch.ones((H, D), device="cuda")
    for h in range(H):
        scale[h, torch.randperm(D, generator=g, device="cuda")[:c["outliers"]]] = c["outlier_scale"]
    N = sum(n) * c.get("branches", 1)
    K = (torch.randn((sum(T), H, D), generator=g, device="cuda") * scale).to(dt)
    V = torch.randn((sum(T), H, D), generator=g, device="cuda").to(dt)
    k = (torch.randn((N, H, D), generator=g, device="cuda") * scale).to(dt)
    v = torch.randn((N, H, D), generator=g, device="cuda").to(dt)
    q = torch.randn((N, c.get("H_q", H), D), generator=g, device="cuda").to(dt)
    return K, V, q, k, v


# ---- plain forms -------------------------------------------------------------------
def _quantize(x, dim):
    """Codes (uint8), scale and zero (fp16) of groups of G along `dim`, which comes back as (groups, G)."""
    x = x.float().unflatten(dim, (-1, G))
    lo, hi = x.amin(dim + 1, keepdim=True), x.amax(dim + 1, keepdim=True)
    s, z = ((hi - lo) / 3.0).half(), lo.half()
    code = torch.where(s.float() > 0, torch.round((x - z.float()) / s.float()), 0.0).clamp(0, 3)
    return code.to(torch.uint8), s, z


def _dequantize(code, s, z, dim):
    return (z.float() + s.float() * code.float()).flatten(dim, dim + 1)


def _paged(c, K, V, T):
    """The history as a paged store: codes, scales and zeros [pages, H, ...] of R-token pages, a page table [B, pages]
    and the residual tokens [B, H, R, D]."""
    R, H, D, B = c["R"], c["H_kv"], c["D"], c["B"]
    at = [sum(T[:b]) for b in range(B)]
    full = [_split(t, R)[0] // R for t in T]
    table = torch.zeros((B, max(1, max(full))), dtype=torch.int64)
    rows, res = [], torch.zeros((2, B, H, R, D), dtype=K.dtype, device=K.device)
    for b in range(B):
        table[b, :full[b]] = torch.arange(full[b]) + sum(full[:b])
        rows.append(torch.arange(at[b], at[b] + full[b] * R))
        r = T[b] - full[b] * R
        res[0, b, :, :r] = K[at[b] + full[b] * R:at[b] + T[b]].transpose(0, 1)
        res[1, b, :, :r] = V[at[b] + full[b] * R:at[b] + T[b]].transpose(0, 1)
    rows = torch.cat(rows).to(K.device)
    pk = K[rows].view(-1, R, H, D).transpose(1, 2)      # [pages, H, R, D]
    pv = V[rows].view(-1, R, H, D).transpose(1, 2)
    if not len(rows):
        pk = pv = torch.zeros((1, H, R, D), dtype=K.dtype, device=K.device)
    return dict(k=_quantize(pk, 2), v=_quantize(pv, 3), table=table.to(K.device), full=full, res=res)


def _dense(store, R):
    """Dequantized keys and values [B, H, pages * R, D] through the page table."""
    pages = store["table"]
    k = _dequantize(*[x[pages] for x in store["k"]], 3)      # [B, pages, H, R, D]
    v = _dequantize(*[x[pages] for x in store["v"]], 4)
    return k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)


def _softmax_attention(q, k, v, visible):
    """q [B, H, g, n, D], k and v [B, H, T, D] in fp32, visible [B, 1, 1, n, T]."""
    score = (q.flatten(2, 3) @ k.transpose(2, 3)).view(*q.shape[:4], k.shape[2]) / math.sqrt(q.shape[-1])
    score = score.masked_fill(~visible, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    out = (p.flatten(2, 3) @ v).view(q.shape)
    return out / p.sum(-1, keepdim=True)


def _plan(T, n, R, device):
    """Where each new token sits in [B, most new tokens], and which keys each may see."""
    most = max(n)
    full = [_split(t, R)[0] for t in T]
    b = torch.cat([torch.full((x,), i) for i, x in enumerate(n)]).to(device)
    i = torch.cat([torch.arange(x) for x in n]).to(device)
    paged = torch.arange(max(R, max(full)), device=device)[None, :] < torch.tensor(full, device=device)[:, None]
    kept = (torch.arange(R, device=device)[None, :]
            < torch.tensor([t - f for t, f in zip(T, full)], device=device)[:, None])
    new = torch.arange(most, device=device)
    causal = (new[None, :] <= new[:, None])[None].expand(len(T), -1, -1)
    old = torch.cat([paged, kept], 1)[:, None, :].expand(-1, most, -1)
    return b, i, torch.cat([old, causal], 2)[:, None, None]


def _attend(c, store, plan, q, k, v):
    b, i, visible = plan
    H, D, most = c["H_kv"], c["D"], visible.shape[3]
    n_seq = visible.shape[0]
    kd, vd = _dense(store, c["R"])
    new = torch.zeros((3, n_seq, most, c["H_q"], D), dtype=torch.float32, device=q.device)
    new[0, b, i] = q.float()
    new[1, b, i, :H] = k.float()
    new[2, b, i, :H] = v.float()
    kd = torch.cat([kd, store["res"][0].float(), new[1, :, :, :H].transpose(1, 2)], 2)
    vd = torch.cat([vd, store["res"][1].float(), new[2, :, :, :H].transpose(1, 2)], 2)
    qd = new[0].view(n_seq, most, H, -1, D).permute(0, 2, 3, 1, 4)
    out = _softmax_attention(qd, kd, vd, visible)
    return out.permute(0, 3, 1, 2, 4).reshape(n_seq, most, c["H_q"], D)[b, i].to(q.dtype)


def _rope_one(x, c, cos, sin):
    rot = c["rot"]
    a = x[..., :rot].float()
    if c["layout"] == "half":
        u, w = a[..., :rot // 2], a[..., rot // 2:]
    else:
        u, w = a[..., 0::2], a[..., 1::2]
    y = (u * cos - w * sin, w * cos + u * sin)
    y = torch.cat(y, -1) if c["layout"] == "half" else torch.stack(y, -1).flatten(-2)
    return torch.cat([y.to(x.dtype), x[..., rot:]], -1)


def _plain_rope(c, s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos = (torch.cos(angle) * s["m"]).float()[:, None]
    sin = (torch.sin(angle) * (-s["m"] if c["inverse"] else s["m"])).float()[:, None]
    return _rope_one(s["q"], c, cos, sin), _rope_one(s["k"], c, cos, sin)


def _plain_extend(c, s):
    """The chunk after the history: tokens that are no longer among the newest become codes; all read back densely."""
    kd, vd = _dense(s["store"], c["R"])
    old = torch.cat([kd, s["store"]["res"][0].float()], 2), torch.cat([vd, s["store"]["res"][1].float()], 2)
    b, at, src, page_rows = s["rows"]
    out = []
    for x, new, dim in ((old[0], s["k"], 2), (old[1], s["v"], 3)):
        raw = torch.cat([x.transpose(1, 2)[b, at], new.float()])[src]            # [tokens, H, D]
        pages = raw[page_rows].view(-1, c["R"], c["H_kv"], c["D"]).transpose(1, 2)
        coded = _dequantize(*_quantize(pages, dim), dim).transpose(1, 2).flatten(0, 1)
        out.append(raw.index_copy(0, page_rows, coded).to(new.dtype))
    return out


def _plain_branch(c, s):
    F = c["branches"]
    t = s["store"]
    twig = dict(k=t["k"], v=t["v"], table=t["table"].repeat_interleave(F, 0), res=t["res"].repeat_interleave(F, 1))
    return _attend(c, twig, s["plan"], s["q"], s["k"], s["v"])


def _plain_compact(c, s):
    t = s["store"]
    pages = t["table"][s["b"], s["at"]]              # the live pages, in the order of the sequences
    moved = {x: [y[pages] for y in t[x]] for x in ("k", "v")}
    back = torch.zeros_like(t["table"])
    back[s["b"], s["at"]] = torch.arange(len(pages), device=pages.device)
    kd, vd = _dense(dict(moved, table=back), c["R"]) if len(pages) else _dense(t, c["R"])
    res = t["res"].clone()
    kd, vd = torch.cat([kd, res[0].float()], 2), torch.cat([vd, res[1].float()], 2)
    return [x.transpose(1, 2)[s["rows"]].to(res.dtype) for x in (kd, vd)]


# ---- the tools' entry points -------------------------------------------------------
def prepare(case, seed):
    c = case
    if c["op"] == "rope":
        return dict(_rope_inputs(c, seed), case=c)
    K, V, q, k, v = _kv_inputs(c, seed)
    T, n = _lengths(c)
    R, B, F = c["R"], c["B"], c.get("branches", 1)
    s = dict(case=c, q=q, k=k, v=v, T=T, n=n)
    if own:
        import bit_asymmetric_kv_prefill_b200 as kivi
        need = sum(-(-(t + x) // R) for t, x in zip(T, n))
        pool = kivi.KiviPool(pages=2 * need + B * F, sequences=B * (F + 1), H_kv=c["H_kv"], D=c["D"], G=G, R=R,
                             dtype=DTYPES[c["dtype"]], T_max=max(T) + max(n))
        s["pool"], s["seqs"] = pool, pool.open(B)
        pool.extend(s["seqs"], K, V, T)
        return s
    s["store"] = _paged(c, K, V, T)
    full = s["store"]["full"]
    dev = K.device
    if c["op"] == "attend":
        s["plan"] = _plan(T, n, R, dev)
    elif c["op"] == "branch":
        s["plan"] = _plan([t for t in T for _ in range(F)], [1] * (B * F), R, dev)
    elif c["op"] == "extend":
        # Rows of the dense history (its padded positions) and of the chunk, in the order of the sequences' tokens,
        # and which of them sit in newly written pages.
        wide = max(1, max(full)) * R
        b, at, src, page_rows, hist, base = [], [], [], [], 0, 0
        for i in range(B):
            r = T[i] - full[i] * R
            b.append(torch.full((T[i],), i))
            at.append(torch.cat([torch.arange(full[i] * R), torch.arange(wide, wide + r)]))
            src.append(torch.cat([torch.arange(hist, hist + T[i]), sum(T) + torch.arange(sum(n[:i]), sum(n[:i + 1]))]))
            page_rows.append(torch.arange(base + full[i] * R, base + _split(T[i] + n[i], R)[0]))
            hist += T[i]
            base += T[i] + n[i]
        s["rows"] = [torch.cat(x).to(dev) for x in (b, at, src, page_rows)]
    else:
        s["b"] = torch.cat([torch.full((f,), i) for i, f in enumerate(full)]).to(dev)
        s["at"] = torch.cat([torch.arange(f) for f in full]).to(dev)
        wide = max(1, max(full)) * R
        s["rows"] = (torch.cat([torch.full((t,), i) for i, t in enumerate(T)]).to(dev),
                     torch.cat([torch.cat([torch.arange(f * R), torch.arange(wide, wide + t - f * R)])
                                for f, t in zip(full, T)]).to(dev))
    return s


def _own_run(c, s):
    import bit_asymmetric_kv_prefill_b200 as kivi
    if c["op"] == "rope":
        return kivi.rope(s["q"], s["k"], s["positions"], s["inv_freq"], rotary_dim=c["rot"],
                         interleaved=c["layout"] == "interleaved", scale=s["m"], inverse=c["inverse"])
    pool, seqs = s["pool"], s["seqs"]
    if c["op"] == "attend":
        return pool.attend(seqs, s["q"], s["k"], s["v"], s["n"])
    if c["op"] == "extend":
        twigs = pool.fork(seqs)
        pool.extend(twigs, s["k"], s["v"], s["n"])
        out = pool.gather(twigs)
        pool.free(twigs)
        return out
    if c["op"] == "branch":
        F = c["branches"]
        twigs = pool.fork([x for x in seqs for _ in range(F)])
        out = pool.attend(twigs, s["q"], s["k"], s["v"], [1] * len(twigs))
        pool.extend(twigs, s["k"], s["v"], [1] * len(twigs))
        pool.free(twigs)
        return out
    moved = pool.copy(seqs)
    pool.free(seqs)
    pool.compact()
    s["seqs"] = moved
    return pool.gather(moved)


def run(state):
    c = state["case"]
    if own:
        return _own_run(c, state)
    if c["op"] == "rope":
        return _plain_rope(c, state)
    if c["op"] == "attend":
        return _attend(c, state["store"], state["plan"], state["q"], state["k"], state["v"])
    return {"extend": _plain_extend, "branch": _plain_branch, "compact": _plain_compact}[c["op"]](c, state)


def work(case):
    c = case
    if c["op"] == "rope":
        el = c["tokens"] * (c["H_q"] + c["H_kv"]) * c["D"]
        return {"bytes": 4 * el + 4 * c["tokens"], "flops": 3 * el * c["rot"] / c["D"]}
    T, n = _lengths(c)
    H, D, R, F = c["H_kv"], c["D"], c["R"], c.get("branches", 1)
    coded = sum(_split(t, R)[0] for t in T)                # tokens held in codes: 0.75 D bytes a head, K and V
    kept = sum(T) - coded
    store = H * D * (0.75 * coded + 4.0 * kept)
    if c["op"] in ("attend", "branch"):
        pairs = sum(x * (t + (x + 1) / 2) * F for t, x in zip(T, n))
        new = sum(n) * F * (2 * H + 2 * c["H_q"]) * D * 2
        return {"bytes": store + new, "flops": 4 * pairs * c["H_q"] * D}
    if c["op"] == "extend":
        total = sum(T) + sum(n)
        after = sum(_split(t + x, R)[0] for t, x in zip(T, n))
        return {"bytes": store + H * D * (4.0 * sum(n) + 0.75 * (after - coded) + 4.0 * total), "flops": 12 * H * D * total}
    return {"bytes": H * D * 4.0 * sum(T) + 2 * store, "flops": 4 * H * D * sum(T)}


# ---- the definition in 64 bits -----------------------------------------------------
def _exact_codes(x, dim):
    """x [tokens, H, D] quantized in groups of G along dim and decoded, by the definition: fp32 roundings where it has
    them, everything else in 64 bits."""
    x = x.double()
    g = x.reshape(-1, G, *x.shape[1:]) if dim == 0 else x.reshape(*x.shape[:-1], -1, G)
    a = 1 if dim == 0 else -1
    lo, hi = g.min(a, keepdim=True).values, g.max(a, keepdim=True).values
    s = ((hi - lo).float().double() / 3).float().half().double()
    z = lo.float().half().double()
    quotient = ((g - z).float().double() / torch.where(s == 0, 1.0, s)).float()
    code = torch.where(s == 0, 0.0, quotient.round().clamp(0, 3).double())
    return (z + s * code).reshape(x.shape)


def _exact_cache(K, V, R):
    n_q = _split(K.shape[0], R)[0]
    return (torch.cat([_exact_codes(K[:n_q], 0) if n_q else K[:0].double(), K[n_q:].double()]),
            torch.cat([_exact_codes(V[:n_q], -1) if n_q else V[:0].double(), V[n_q:].double()]))


def _exact_rows(q, K, V, k, v):
    """One sequence: row i of the new tokens sees the cached K, V and the new k, v up to its own."""
    n, H_q, D = q.shape
    out = torch.empty((n, H_q, D), dtype=torch.float64, device=q.device)
    keys, values = torch.cat([K, k.double()]), torch.cat([V, v.double()])
    late = torch.arange(len(keys), device=q.device)[None] > torch.arange(n, device=q.device)[:, None] + len(K)
    for h in range(H_q):
        u = h // (H_q // K.shape[1])
        w = q[:, h].double() @ keys[:, u].T / math.sqrt(D)
        out[:, h] = torch.softmax(w.masked_fill(late, -math.inf), 1) @ values[:, u]
    return out


def exact(case, seed):
    c = case
    if c["op"] == "rope":
        s = _rope_inputs(c, seed)
        turn = torch.polar(torch.full_like(s["inv_freq"], s["m"], dtype=torch.float64).expand(c["tokens"], -1),
                           s["positions"].double().outer(s["inv_freq"].double()) * (-1 if c["inverse"] else 1))
        out = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            a = y[..., :c["rot"]]
            z = torch.complex(*(a.chunk(2, -1) if c["layout"] == "half" else (a[..., ::2], a[..., 1::2]))) * turn[:, None]
            y[..., :c["rot"]] = torch.cat([z.real, z.imag], -1) if c["layout"] == "half" else torch.view_as_real(z).flatten(-2)
            out.append(y)
        return tuple(out)
    K, V, q, k, v = _kv_inputs(c, seed)
    T, n = _lengths(c)
    F, rows, kept, made = c.get("branches", 1), [], [[], []], 0
    for b, (t, x) in enumerate(zip(T, n)):
        h = slice(sum(T[:b]), sum(T[:b + 1]))
        if c["op"] in ("attend", "branch"):
            old = _exact_cache(K[h], V[h], c["R"])
            for _ in range(F):
                w = slice(made, made + x)
                rows.append(_exact_rows(q[w], *old, k[w], v[w]))
                made += x
        else:
            w = slice(sum(n[:b]), sum(n[:b + 1]))
            for side, y in zip(kept, _exact_cache(torch.cat([K[h], k[w]]), torch.cat([V[h], v[w]]), c["R"])):
                side.append(y)
    return torch.cat(rows) if rows else [torch.cat(x) for x in kept]
