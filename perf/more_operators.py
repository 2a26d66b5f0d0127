"""A KV cache in 4 bits with the attention that reads it, and sampling: what is measured, in plain form and
through the library.

* ``write``: keys and values of some tokens quantised into the pages of a cache, then read back.
* ``read``: rows of such a cache as keys (turned to new positions) and values.
* ``attention``: new queries over the cache, a few tokens of every sequence of a batch.
* ``sample``: tokens drawn from logits with temperature, top-k, top-p and min-p, from given random numbers.

The 4-bit form.  A group is 32 consecutive channels of one token's key or value of one head.  With lo, hi its
smallest and largest number, d = hi - lo (one fp32 subtraction) and a = max(|lo|, |hi|):
    scale = the smallest bf16 number >= max(d / 14.75, a / 64, 2^-120)
    zero  = floor(4 lo / scale) / 4                      (a multiple of 1/4 of at most 64: exact in bf16)
    code  = min(max(nearest(x / scale - zero), 0), 15)   (ties to even)
    value = scale (code + zero)                          (exact in fp32)
A group whose d or a is not finite has scale and zero NaN and codes 0.

A cache is [n_pages, heads, page_tokens / 16, 20 head_dim] bytes: blocks of 16 tokens of one head.  In a
block of D channels, NG = D / 32 groups, the bytes of token r are
    key codes    r D/2 + (8c' NG/2 + 4g) + i/2 for the channels 32g + 8c' + i, i even in the low nibble,
    value codes  8D + 512 (j / 4) + 64n + 16 ((r % 8) / 2) + 4 (j % 4) + 2 (r % 2) + r / 8 for the channels
                 16j + n (low nibble) and 16j + n + 8, n below 8,
    key scales and zeros    16D + 4 NG r: NG bf16 scales, then NG zeros,
    value scales and zeros  64 NG bytes further.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 32
BLOCK = 16
LEVELS = 14.75


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the whole Yi-34B-shaped prompt of 8320 tokens enters the cache of one layer
        {"name": "write_prompt_8320x8x128", "kind": "write", "n": 1, "t": 8320, "ctx": 8320, "order": "prompt", "hkv": 8, "dh": 128, "page": 64, "x": "bf16"},
        # one new token of each of 16 sequences (the smallest call: its latency counts)
        {"name": "write_decode_16x8x128", "kind": "write", "n": 16, "t": 1, "ctx": 4096, "order": "decode", "hkv": 8, "dh": 128, "page": 64, "x": "bf16"},
        # recomputed tokens of three small fp32 prompts, scattered over them
        {"name": "write_sparse_3x77x4x64_f32", "kind": "write", "n": 3, "t": 77, "ctx": 515, "order": "sparse", "hkv": 4, "dh": 64, "page": 16, "x": "f32"},
        # a cached context of 4096 tokens with 32 heads (Llama-7B-shaped) back in bf16, its keys moved on by 64 positions
        {"name": "read_4096x32x128", "kind": "read", "n": 1, "t": 4096, "ctx": 4096, "order": "prompt", "hkv": 32, "dh": 128, "page": 64, "x": "bf16", "delta": 64},
        # a few rows at far positions, in fp32
        {"name": "read_sparse_2x33x4x64_f32", "kind": "read", "n": 2, "t": 33, "ctx": 1000, "order": "sparse", "hkv": 4, "dh": 64, "page": 48, "x": "f32", "delta": 100000},
        # one decoded token after a Mistral-7B-shaped prompt of 3200 tokens
        {"name": "attention_1x1_3200x8x128", "kind": "attention", "n": 1, "t": 1, "lo": 3200, "hi": 3200, "hkv": 8, "g": 4, "dh": 128, "page": 64, "x": "bf16"},
        # a ragged batch of 32 Yi-34B-shaped sequences (7 query heads a KV head)
        {"name": "attention_32x1_8320x8x128", "kind": "attention", "n": 32, "t": 1, "lo": 100, "hi": 8320, "hkv": 8, "g": 7, "dh": 128, "page": 64, "x": "bf16"},
        # four drafted tokens of each of 16 Llama-70B-shaped sequences, checked at once
        {"name": "attention_16x4_8200x8x128", "kind": "attention", "n": 16, "t": 4, "lo": 2000, "hi": 8200, "hkv": 8, "g": 8, "dh": 128, "page": 64, "x": "bf16"},
        # a Llama-7B-shaped batch of 4 with a KV head for every query head, in fp32
        {"name": "attention_4x1_4128x32x128_f32", "kind": "attention", "n": 4, "t": 1, "lo": 4000, "hi": 4128, "hkv": 32, "g": 1, "dh": 128, "page": 16, "x": "f32"},
        # one answer's next token, every filter on
        {"name": "sample_1x32000", "kind": "sample", "rows": 1, "vocab": 32000, "x": "f32", "top_k": True, "top_p": True, "min_p": True},
        # a batch with nucleus sampling alone
        {"name": "sample_64x64000_top_p", "kind": "sample", "rows": 64, "vocab": 64000, "x": "f32", "top_k": False, "top_p": True, "min_p": False},
        # a large batch of bf16 logits (many of them equal) with every filter
        {"name": "sample_512x64000_bf16", "kind": "sample", "rows": 512, "vocab": 64000, "x": "bf16", "top_k": True, "top_p": True, "min_p": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["write", "read", "attention", "attention", "sample", "sample"])
    if kind == "sample":
        vocab = _log(rng, 1000, 64000)
        on = [rng.random() < 0.6 for _ in range(3)]
        return {"kind": kind, "rows": _log(rng, 1, 512), "vocab": vocab, "x": rng.choice(["f32", "bf16"]),
                "top_k": on[0], "top_p": on[1], "min_p": on[2]}
    hkv, dh, page, x = rng.choice([1, 2, 4, 8, 32]), rng.choice([64, 128]), rng.choice([16, 48, 64, 256]), rng.choice(["f32", "bf16"])
    if kind == "attention":
        n, t = _log(rng, 1, 32), rng.choice([1, 1, 1, 2, 3, 5, 8, 16])
        hi = _log(rng, max(64, t), max(128, min(65536, 32 * 8320 * 8 // (n * hkv * t))))
        return {"kind": kind, "n": n, "t": t, "lo": max(t, _log(rng, 1, hi)), "hi": hi, "hkv": hkv,
                "g": rng.choice([1, 2, 4, 7, 8] if hkv < 32 else [1, 2]), "dh": dh, "page": page, "x": x}
    order = rng.choice(["prompt", "decode", "sparse"])
    if order == "decode":
        n, t = _log(rng, 1, 256), 1
    else:
        n = rng.choice([1, 2, 3])
        t = _log(rng, 1, 8320 * 8 // (hkv * n) if x == "bf16" else 4160 * 8 // (hkv * n))
    case = {"kind": kind, "n": n, "t": t, "ctx": _log(rng, t, max(t, 8320)), "order": order, "hkv": hkv, "dh": dh, "page": page, "x": x}
    if kind == "read":
        case["delta"] = rng.choice([0, _log(rng, 1, 100000)])
    return case


def _lengths(case):
    """The sequences' lengths, spread evenly over lo..hi in an order that is not ascending."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    step = next(s for s in (7, 5, 3, 1) if math.gcd(s, n) == 1)
    return [hi - (hi - lo) * ((i * step) % n) // max(1, n - 1) for i in range(n)]


# ------------------------------------------------------------------------------------- the 4-bit form
def _encode(x):
    """(scale, zero [..., D / 32], codes [..., D]) of x, in 64 bits."""
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    spread = (hi.float() - lo.float()).double()
    top = torch.maximum(lo.abs(), hi.abs()).double()
    s = torch.maximum(spread / torch.full_like(spread, LEVELS), top / 64).clamp(min=2.0 ** -120)
    scale = s.to(torch.bfloat16)
    scale = torch.where(scale.double() < s, (scale.view(torch.int16) + 1).view(torch.bfloat16), scale).double()
    zero = torch.floor(4 * lo.double() / scale) / 4
    bad = ~torch.isfinite(spread + top)
    codes = torch.round(g.double() / scale[..., None] - zero[..., None]).clamp(0, 15)
    codes = torch.where(bad[..., None], 0.0, codes)
    return scale.masked_fill(bad, math.nan), zero.masked_fill(bad, math.nan), codes.flatten(-2).to(torch.uint8)


def _offsets(dh, device):
    """[16, 1.25 D] offsets in a block of the bytes of each of its tokens: key codes (channels 2m and 2m + 1),
    value codes (16j + n and 16j + n + 8), key scales and zeros, value scales and zeros."""
    ng = dh // GROUP
    r = torch.arange(BLOCK, device=device)[:, None]
    c = 2 * torch.arange(dh // 2, device=device)
    k = r * (dh // 2) + (c % 32 // 8 * ng + c // 32) * 4 + c % 8 // 2
    p = torch.arange(dh // 2, device=device)
    j, n = p // 8, p % 8
    v = 8 * dh + 512 * (j // 4) + 64 * n + 16 * (r % 8 // 2) + 4 * (j % 4) + 2 * (r % 2) + r // 8
    q = torch.arange(4 * ng, device=device)
    return torch.cat([k, v, 16 * dh + 4 * ng * r + q, 16 * dh + 64 * ng + 4 * ng * r + q], dim=1)


def _bytes_of(scale, zero):
    return torch.cat([scale, zero], -1).to(torch.bfloat16).contiguous().view(torch.uint8)


def _pack(k, v):
    """The bytes, in the order of _offsets, of keys and values [..., D]."""
    (ks, kz, kc), (vs, vz, vc) = _encode(k), _encode(v)
    kc = kc.unflatten(-1, (-1, 2))
    vc = vc.unflatten(-1, (-1, 2, 8))
    return torch.cat([kc[..., 0] | kc[..., 1] << 4, (vc[..., 0, :] | vc[..., 1, :] << 4).flatten(-2), _bytes_of(ks, kz), _bytes_of(vs, vz)], -1)


def _unpack(b, dh, dtype=torch.float32):
    """Keys and values [..., D] of such bytes."""
    ng = dh // GROUP
    kc, vc, kp, vp = b.split([dh // 2, dh // 2, 4 * ng, 4 * ng], dim=-1)
    kc = torch.stack([kc & 15, kc >> 4], -1).flatten(-2)
    vc = vc.unflatten(-1, (-1, 8))
    vc = torch.stack([vc & 15, vc >> 4], -2).flatten(-3)
    out = []
    for codes, p in ((kc, kp), (vc, vp)):
        p = p.contiguous().view(torch.bfloat16).to(dtype)
        scale, zero = p[..., :ng, None], p[..., ng:, None]
        out.append((scale * (codes.unflatten(-1, (ng, GROUP)).to(dtype) + zero)).flatten(-2))
    return out


def _where(pool, table, seq, pos):
    """Byte indices [rows, heads, 1.25 D] in the pool of the tokens at positions pos of the sequences seq."""
    n_pages, heads, blocks, size = pool.shape
    dh, tokens = size // 20, blocks * BLOCK
    page = table[seq.long(), (pos // tokens).long()].long()
    block = (page[:, None] * heads + torch.arange(heads, device=pool.device)) * blocks + (pos % tokens // BLOCK).long()[:, None]
    return (block * size)[..., None] + _offsets(dh, pool.device)[(pos % BLOCK).long()][:, None, :]


# ------------------------------------------------------------------------------------------ inputs
def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _keys(gen, *shape):
    """Keys as models have them: a few channels of every head far larger than the others."""
    k = _rand(gen, *shape)
    loud = torch.randint(0, shape[-1], (max(1, shape[-1] // 32),), generator=gen, device="cuda")
    k[..., loud] *= 6.0
    return k


def _pages(gen, n, tokens, page):
    """A page table of n sequences of the given lengths, the pages in no order, and the number of pages."""
    per = [-(-t // page) for t in tokens]
    order = torch.randperm(sum(per), generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(n, max(per), dtype=torch.int32, device="cuda")
    at = 0
    for i, p in enumerate(per):
        table[i, :p] = order[at:at + p]
        at += p
    return table, sum(per)


def _filled(gen, n_pages, case):
    """A pool of keys and values."""
    hkv, blocks, dh = case["hkv"], case["page"] // BLOCK, case["dh"]
    pool = torch.zeros(n_pages, hkv, blocks, 20 * dh, dtype=torch.uint8, device="cuda")
    flat, off = pool.view(-1, 20 * dh), _offsets(dh, "cuda").flatten()
    step = max(1, (1 << 25) // (BLOCK * dh))
    for i in range(0, flat.shape[0], step):
        m = min(step, flat.shape[0] - i)
        flat[i:i + m, off] = _pack(_keys(gen, m, BLOCK, dh), _rand(gen, m, BLOCK, dh)).flatten(1)
    return pool


def _positions(gen, case):
    """Positions of the t rows of each sequence, [n, t]."""
    n, t, ctx = case["n"], case["t"], case["ctx"]
    if case["order"] == "prompt":
        return torch.arange(t, device="cuda").expand(n, t)
    if case["order"] == "decode":
        return torch.randint(0, ctx, (n, 1), generator=gen, device="cuda")
    return torch.stack([torch.randperm(ctx, generator=gen, device="cuda")[:t].sort().values for _ in range(n)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["kind"]
    s = {"kind": kind}
    if kind == "sample":
        rows, vocab = case["rows"], case["vocab"]
        x = 2.0 * _rand(gen, rows, vocab)
        # the few tokens that a model finds likely
        for _ in range(24):
            at = torch.randint(0, vocab, (rows, 1), generator=gen, device="cuda")
            x.scatter_(1, at, 4.0 + 5.0 * torch.rand(rows, 1, generator=gen, device="cuda"))
        rand = lambda: torch.rand(rows, generator=gen, device="cuda")  # noqa: E731
        s.update(logits=x.to(DT[case["x"]]), uniform=rand(), temperature=0.5 + 0.8 * rand(), top_k=None, top_p=None,
                 min_p=None, out=torch.empty(rows, dtype=torch.int32, device="cuda"))
        if case["top_k"]:
            s["top_k"] = torch.randint(1, 1 + min(vocab, 200), (rows,), generator=gen, device="cuda").to(torch.int32)
        if case["top_p"]:
            s["top_p"] = 0.5 + 0.49 * rand()
        if case["min_p"]:
            s["min_p"] = 0.1 * rand()
        return s
    n, hkv, dh, dtype = case["n"], case["hkv"], case["dh"], DT[case["x"]]
    if kind == "attention":
        t, lens = case["t"], _lengths(case)
        s["table"], pages = _pages(gen, n, lens, case["page"])
        s["pool"] = _filled(gen, pages, case)
        s["q"] = _rand(gen, n, t, hkv * case["g"], dh).to(dtype)
        s["q_pos"] = (torch.tensor(lens, device="cuda")[:, None] - t + torch.arange(t, device="cuda")).to(torch.int32)
        s["out"] = torch.empty_like(s["q"])
        if own:
            import rag_non_prefix_gb300 as cb

            s["scratch"] = cb.kvq_scratch()
        return s
    s["table"], pages = _pages(gen, n, [case["ctx"]] * n, case["page"])
    s["seq"] = torch.arange(n, device="cuda").repeat_interleave(case["t"]).to(torch.int32)
    s["pos"] = _positions(gen, case).flatten().to(torch.int32)
    rows = n * case["t"]
    if kind == "write":
        s["pool"] = torch.zeros(pages, hkv, case["page"] // BLOCK, 20 * dh, dtype=torch.uint8, device="cuda")
        s["k"], s["v"] = _keys(gen, rows, hkv, dh).to(dtype), _rand(gen, rows, hkv, dh).to(dtype)
        s.update(delta=0, dtype=torch.float32)
    else:
        s["pool"] = _filled(gen, pages, case)
        s.update(delta=case["delta"], dtype=dtype)
    s["k_out"], s["v_out"] = (torch.empty(rows, hkv, dh, dtype=s["dtype"], device="cuda") for _ in range(2))
    return s


THETA = 10000.0


# ------------------------------------------------------------------------------------------ passes
def _turn(k, delta):
    """Keys moved on by delta positions: channels i and i + D / 2 are a pair."""
    if delta == 0:
        return k
    half = k.shape[-1] // 2
    a = delta * torch.pow(torch.tensor(THETA, dtype=torch.float64, device=k.device), torch.arange(half, dtype=torch.float64, device=k.device) / -half)
    c, s = torch.cos(a).float(), torch.sin(a).float()
    x, y = k[..., :half], k[..., half:]
    return torch.cat([x * c - y * s, x * s + y * c], -1)


def _attend(s):
    q = s["q"].float()
    n, t, h, dh = q.shape
    hkv = s["pool"].shape[1]
    out = torch.zeros_like(q)
    lens = (s["q_pos"].amax(1) + 1).tolist()
    for i, keys in enumerate(lens):
        pos = torch.arange(keys, device=q.device)
        k, v = _unpack(s["pool"].view(-1)[_where(s["pool"], s["table"], torch.full_like(pos, i), pos)], dh)
        qi = q[i].view(t, hkv, h // hkv, dh).permute(1, 2, 0, 3).reshape(hkv, -1, dh)
        score = (qi @ k.permute(1, 2, 0)).view(hkv, -1, t, keys) / math.sqrt(dh)
        score = score.masked_fill(pos > s["q_pos"][i][:, None], -math.inf)
        p = torch.exp(score - score.amax(-1, keepdim=True))
        p = (p / p.sum(-1, keepdim=True)).view(hkv, -1, keys)
        out[i] = (p @ v.permute(1, 0, 2)).view(hkv, -1, t, dh).permute(2, 0, 1, 3).reshape(t, h, dh)
    return out.to(s["q"].dtype)


def _sample(s):
    x = s["logits"].double()
    rows, vocab = x.shape
    w = torch.exp((x - x.amax(1, keepdim=True)) / s["temperature"].double()[:, None])
    order = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices
    w_sorted = w.gather(1, order)
    rank = torch.arange(vocab, device=x.device)
    if s["top_k"] is not None:
        w_sorted = torch.where(rank < s["top_k"][:, None], w_sorted, 0.0)
    before = w_sorted.cumsum(1) - w_sorted
    keep = w_sorted > 0
    if s["top_p"] is not None:
        keep &= (before < s["top_p"].double()[:, None] * w_sorted.sum(1, keepdim=True)) | (rank == 0)
    if s["min_p"] is not None:
        keep &= w_sorted >= s["min_p"].double()[:, None]
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w_sorted, 0.0))
    total = kept.cumsum(1)
    hit = (total > s["uniform"].double()[:, None] * total[:, -1:]) & (kept > 0)
    last = vocab - 1 - (kept.flip(1) > 0).to(torch.uint8).argmax(1)
    return torch.where(hit.any(1), hit.to(torch.uint8).argmax(1), last).to(torch.int32)


def run(s):
    kind = s["kind"]
    if own:
        import rag_non_prefix_gb300 as cb

        if kind == "sample":
            return cb.cb_sample(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], out=s["out"], by_id=True)
        if kind == "attention":
            return cb.cb_kvq_attention(s["q"], s["q_pos"], s["pool"], s["table"], out=s["out"], scratch=s.get("scratch"))
        if kind == "write":
            cb.cb_kvq_write(s["pool"], s["table"], s["k"], s["v"], s["pos"], s["seq"])
        return cb.cb_kvq_read(s["pool"], s["table"], s["pos"], s["seq"], delta_pos=s["delta"], theta=THETA, k_out=s["k_out"], v_out=s["v_out"])

    if kind == "sample":
        return _sample(s)
    if kind == "attention":
        return _attend(s)
    at = _where(s["pool"], s["table"], s["seq"], s["pos"])
    if kind == "write":
        s["pool"].view(-1)[at] = _pack(s["k"].float(), s["v"].float())
    k, v = _unpack(s["pool"].view(-1)[at], s["pool"].shape[3] // 20)
    return _turn(k, s["delta"]).to(s["dtype"]), v.to(s["dtype"])


# -------------------------------------------------------------------------------- 64-bit definition
def _rounded(x):
    """What the 4-bit form holds of x [..., D], group by group, in 64 bits."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c in range(0, x.shape[-1], GROUP):
        g = x[..., c:c + GROUP]
        lo, hi = g.min(dim=-1, keepdim=True).values, g.max(dim=-1, keepdim=True).values
        spread = (hi.float() - lo.float()).double()
        least = torch.maximum(spread * 4 / torch.full_like(spread, 59.0), torch.maximum(-lo, hi).double() / 64).clamp(min=2.0 ** -120)
        # 8 significant bits, upwards: a power of two below, then whole steps of its 128th
        unit = (least.view(torch.int64) >> 52 << 52).view(torch.float64) / 128
        scale = torch.ceil(least / unit) * unit
        zero = torch.floor(lo.double() / scale * 4) * 0.25
        out[..., c:c + GROUP] = scale * (torch.clamp(torch.round(g.double() / scale - zero), 0, 15) + zero)
    return out


def _values_at(pool, table, seq, pos):
    """Keys and values [positions, heads, D] of one sequence in 64 bits, page by page through the layout."""
    n_pages, heads, blocks, size = pool.shape
    dh = size // 20
    ng = dh // GROUP
    tokens = blocks * BLOCK
    out = []
    for p in range(int(pos.max()) // tokens + 1):
        b = pool[int(table[seq, p])].cpu().numpy().reshape(heads * blocks, size)
        half = b[:, :8 * dh].reshape(-1, BLOCK, 4, ng, 4)
        k = np.stack([half & 15, half >> 4], -1).reshape(-1, BLOCK, 4, ng, 8).transpose(0, 1, 3, 2, 4).reshape(-1, BLOCK, dh)
        half = b[:, 8 * dh:16 * dh].reshape(-1, dh // 64, 8, 4, 4, 2, 2)  # j / 4, n, (r % 8) / 2, j % 4, r % 2, r / 8
        v = np.stack([half & 15, half >> 4], 5)                            # ..., j % 4, which half of 16j, r % 2, r / 8
        v = v.transpose(0, 7, 3, 6, 1, 4, 5, 2).reshape(-1, BLOCK, dh)
        both = []
        for codes, start in ((k, 16 * dh), (v, 16 * dh + 64 * ng)):
            f = (np.ascontiguousarray(b[:, start:start + 64 * ng]).view(np.uint16).astype(np.uint32) << 16).view(np.float32)
            f = f.reshape(-1, BLOCK, 2, ng, 1).astype(np.float64)
            x = (f[:, :, 0] * (codes.reshape(-1, BLOCK, ng, GROUP) + f[:, :, 1])).reshape(heads, tokens, dh)
            both.append(x.transpose(1, 0, 2))
        out.append(both)
    return [torch.from_numpy(np.concatenate([o[i] for o in out])).to(pool.device)[pos.long()] for i in (0, 1)]


def _sample_exact(s):
    """Row by row: the kept tokens by falling logit, then the walk over them by rising index."""
    x = s["logits"].double().cpu().numpy()
    row = {k: None if s[k] is None else s[k].double().cpu().numpy() for k in ("uniform", "temperature", "top_k", "top_p", "min_p")}
    out = []
    for i in range(x.shape[0]):
        w = np.exp((x[i] - x[i].max()) / row["temperature"][i])
        order = np.argsort(-x[i], kind="stable")
        if row["top_k"] is not None:
            order = order[:int(row["top_k"][i])]
        ws = w[order]
        n = ws.size
        if row["top_p"] is not None:
            n = min(n, 1 + int(np.searchsorted(np.cumsum(ws), row["top_p"][i] * ws.sum(), side="left")))
        if row["min_p"] is not None:
            n = min(n, int(np.count_nonzero(ws >= row["min_p"][i])))
        kept = np.sort(order[:max(n, 1)])
        mass = np.cumsum(w[kept])
        at = int(np.searchsorted(mass, row["uniform"][i] * mass[-1], side="right"))
        out.append(int(kept[min(at, kept.size - 1)]))
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "sample":
        return _sample_exact(s)
    if kind == "attention":
        q = s["q"].double()
        n, t, h, dh = q.shape
        hkv = s["pool"].shape[1]
        if sum(_lengths(case)) * hkv * dh > 1 << 28:
            return None  # (the way through the host takes too long)
        out = torch.zeros_like(q)
        for i in range(n):
            pos = torch.arange(int(s["q_pos"][i].max()) + 1, device="cuda")
            k, v = _values_at(s["pool"], s["table"], i, pos)
            for head in range(h):
                kv = head // (h // hkv)
                score = (q[i, :, head] @ k[:, kv].t()) * dh ** -0.5
                score[pos[None, :] > s["q_pos"][i][:, None]] = -math.inf
                out[i, :, head] = torch.softmax(score, dim=1) @ v[:, kv]
        return out
    if kind == "write":
        return _rounded(s["k"].double()), _rounded(s["v"].double())
    parts = [_values_at(s["pool"], s["table"], i, s["pos"].view(case["n"], -1)[i]) for i in range(case["n"])]
    k, v = (torch.cat([p[j] for p in parts]) for j in (0, 1))
    half = k.shape[-1] // 2
    angle = case["delta"] * torch.tensor([THETA ** (-i / half) for i in range(half)], dtype=torch.float64, device="cuda")
    z = torch.complex(k[..., :half], k[..., half:]) * torch.polar(torch.ones_like(angle), angle)
    return torch.cat([z.real, z.imag], -1), v


# -------------------------------------------------------------------------------------------- work
def work(case):
    size = {"bf16": 2, "f32": 4}[case["x"]]
    if case["kind"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        return {"bytes": rows * (vocab * size + 8 + 4 * (1 + case["top_k"] + case["top_p"] + case["min_p"])), "flops": 10 * rows * vocab}
    hkv, dh = case["hkv"], case["dh"]
    held = 5 * dh // 4  # bytes of one token's key and value of one head
    if case["kind"] == "attention":
        keys, rows, h = sum(_lengths(case)), case["n"] * case["t"], hkv * case["g"]
        return {"bytes": keys * hkv * held + 2 * rows * h * dh * size + 4 * rows, "flops": 4 * keys * case["t"] * h * dh}
    rows = case["n"] * case["t"]
    if case["kind"] == "write":  # the numbers in, the form out and in again, and its values in fp32 out
        return {"bytes": rows * (hkv * (2 * dh * size + 2 * held + 8 * dh) + 8), "flops": 20 * rows * hkv * dh}
    return {"bytes": rows * (hkv * (held + 2 * dh * size) + 8), "flops": 12 * rows * hkv * dh}
