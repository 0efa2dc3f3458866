"""Measured cases of the cache-eviction and rotary-insert operators.

Five operators of a serving loop over the packed key/value cache:

* ``rope``    rotary positions of one to three axes applied to query (or key) heads,
* ``insert``  new keys (rotated the same way) and values quantised into the cache's blocks,
* ``attend``  one query token per sequence against the packed cache, the attention weight
              that every cached token got added to its accumulator,
* ``select``  the tokens of each (sequence, KV head) that stay: the first, the last, and
              those with the largest accumulated weight,
* ``compact`` the kept tokens' blocks and accumulators moved together inside the cache.

Packed blocks hold 128 values: an fp16 norm, then codes of 2, 3 or 4 bits (lowest element in
the lowest bits; 3-bit codes as a 2-bit plane and a 1-bit plane).  The vector that a block
stands for is norm * D H c[code] / sqrt(128), H the Sylvester-Hadamard matrix, D random signs,
c the Lloyd-Max levels of a coordinate of the rotated unit vector.

``own`` False runs every operator in its plain form (elementary torch operations); True runs
the library's calls.
"""

import functools
import math

import numpy as np
import torch

own = False

D = 128
SIGN_SEED = 1
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 16 sequences: the query heads of one layer, three-axis positions
        dict(name="rope-step", op="rope", tokens=16, heads=32, dtype="bf16", style="half", rot=128,
             sections="16,24,24", interleaved=False, start=700, base=1000000.0),
        # a prompt with images at far positions, interleaved axes, an odd number of tokens
        dict(name="rope-prompt", op="rope", tokens=16411, heads=32, dtype="bf16", style="half", rot=128,
             sections="24,20,20", interleaved=True, start=1000000, base=5000000.0),
        # a decode step of 16 sequences: one new key and value per KV head
        dict(name="insert-step", op="insert", tokens=16, hkv=8, kb=4, vb=2, dtype="bf16", style="half", rot=128,
             sections="16,24,24", interleaved=False, start=700, base=1000000.0, page=0, padded=0),
        # a chunk of prompts in pages of 16 tokens, every 7th token padding, one position axis
        dict(name="insert-pages", op="insert", tokens=5001, hkv=4, kb=3, vb=3, dtype="f16", style="half", rot=128,
             sections="64", interleaved=False, start=0, base=10000.0, page=16, padded=7),
        # the prompts of 16 sequences of 8192 tokens
        dict(name="insert-prompt", op="insert", tokens=131072, hkv=8, kb=4, vb=2, dtype="bf16", style="half", rot=128,
             sections="16,24,24", interleaved=False, start=0, base=1000000.0, page=0, padded=0),
        # one short conversation
        dict(name="attend-one", op="attend", batch=1, hq=32, hkv=8, T=1001, kb=4, vb=2, dtype="bf16", page=0,
             ragged=False, decay=1.0),
        # 16 conversations of different lengths in pages of 64 tokens, older weights fading
        dict(name="attend-pages", op="attend", batch=16, hq=32, hkv=8, T=8192, kb=4, vb=2, dtype="bf16", page=64,
             ragged=True, decay=0.98),
        # a full serving batch at 32k tokens, seven query heads for each KV head
        dict(name="attend-batch", op="attend", batch=64, hq=28, hkv=4, T=32769, kb=3, vb=3, dtype="bf16", page=0,
             ragged=False, decay=1.0),
        # one conversation over its budget
        dict(name="select-one", op="select", batch=1, hkv=8, T=4096, keep=1024, first=4, last=256, ragged=False),
        # a full serving batch halved
        dict(name="select-batch", op="select", batch=64, hkv=4, T=32769, keep=16384, first=4, last=1000,
             ragged=True),
        # one conversation's cache after the selection
        dict(name="compact-one", op="compact", batch=1, hkv=8, T=4096, keep=1024, first=4, last=256, kb=4, vb=2,
             page=0, ragged=False),
        # 16 caches of 8192 tokens halved
        dict(name="compact-batch", op="compact", batch=16, hkv=8, T=8192, keep=4095, first=4, last=256, kb=4, vb=2,
             page=0, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _rope_params(rng):
    rot = rng.choice([128, 128, 64, 96, 32])
    style = rng.choice(["half", "half", "adjacent"])
    pairs = rot // 2
    if rng.random() < 0.5:
        h = rng.randint(1, pairs // 3)
        w = rng.randint(1, pairs // 3)
        sections, inter = "%d,%d,%d" % (pairs - h - w, h, w), rng.random() < 0.5
    else:
        sections, inter = "%d" % pairs, False
    return dict(style=style, rot=rot, sections=sections, interleaved=inter,
                start=rng.choice([0, rng.randint(1, 1000000)]),
                base=rng.choice([10000.0, 500000.0, 1000000.0]))


def draw(rng):
    op = rng.choice(["rope", "insert", "attend", "select", "compact"])
    if op == "rope":
        heads, dtype = rng.randint(1, 64), rng.choice(["bf16", "f16", "f32"])
        return dict(op=op, tokens=_log(rng, 1, 16411 * 64 // (heads * SIZES[dtype])), heads=heads, dtype=dtype,
                    **_rope_params(rng))
    if op == "insert":
        hkv, dtype = rng.choice([1, 2, 4, 5, 8]), rng.choice(["bf16", "f16", "f32"])
        return dict(op=op, tokens=_log(rng, 1, 131072 * 2 // SIZES[dtype]), hkv=hkv, kb=rng.choice([2, 3, 4]),
                    vb=rng.choice([2, 3, 4]), dtype=dtype, page=rng.choice([0, 8, 16, 64]), padded=rng.choice([0, 5]),
                    **_rope_params(rng))
    batch, hkv = _log(rng, 1, 64), rng.choice([1, 2, 4, 8])
    T = _log(rng, 1, min(131072, 64 * 4 * 32769 // (batch * hkv)))
    if op == "attend":
        return dict(op=op, batch=batch, hkv=hkv, hq=hkv * rng.randint(1, 8), T=T, kb=rng.choice([2, 3, 4]),
                    vb=rng.choice([2, 3, 4]), dtype=rng.choice(["bf16", "f16"]), page=rng.choice([0, 0, 32, 64, 128]),
                    ragged=rng.random() < 0.5, decay=rng.choice([1.0, 0.95, 0.0]))
    T = max(T, 16)
    if op == "compact":
        T = min(T, 16 * 8 * 8192 // (batch * hkv))
    keep = int(T * rng.uniform(0.2, 0.95))
    first = rng.randint(0, min(8, keep // 4))
    case = dict(op=op, batch=batch, hkv=hkv, T=T, keep=keep, first=first,
                last=rng.randint(0, max(0, (keep - first) // 2)), ragged=rng.random() < 0.5)
    if op == "compact":
        case.update(kb=rng.choice([2, 3, 4]), vb=rng.choice([2, 3, 4]), page=rng.choice([0, 8, 16, 64]))
    return case


def _lengths(case):
    """Tokens of each sequence: T, or (ragged) a fixed pattern from T down to none."""
    B, T = case["batch"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [T if b == 0 else (T * ((b * 7) % 16 + 1)) // 16 - 1 - 3 * b % 11 if b % 5 else b % 2 - 1 for b in range(B)]


def _lens_clamped(case):
    return [min(max(n, 0), case["T"]) for n in _lengths(case)]


def _bytes(bits):
    return 2 + 16 * bits


def _cap(case):
    """Token slots per sequence of the cache."""
    unit = case["page"] or 8
    return -(-case["T"] // unit) * unit


def work(case):
    op = case["op"]
    if op == "rope":
        n, h = case["tokens"], case["heads"]
        axes = len(case["sections"].split(","))
        return {"bytes": 2 * n * h * D * SIZES[case["dtype"]] + 8 * n * axes, "flops": n * h * 3 * case["rot"]}
    if op == "insert":
        n, h = case["tokens"], case["hkv"]
        axes = len(case["sections"].split(","))
        slots = _insert_slots(case) * h
        live = n - (n // case["padded"] if case["padded"] else 0)
        return {"bytes": live * h * (2 * D * SIZES[case["dtype"]] + _bytes(case["kb"]) + _bytes(case["vb"])) +
                8 * n * (axes + 1) + slots * 4 * D, "flops": live * h * 2 * (D * 7 + 6 * D)}
    B, h, T = case["batch"], case["hkv"], case["T"]
    lens = _lens_clamped(case)
    if op == "attend":
        live, hq = sum(lens) * h, case["hq"]
        return {"bytes": live * (_bytes(case["kb"]) + _bytes(case["vb"]) + (4 if case["decay"] == 0.0 else 8)) +
                B * hq * D * 2 * SIZES[case["dtype"]], "flops": 4 * sum(lens) * hq * D}
    kept = sum(min(n, case["keep"]) for n in lens) * h
    if op == "select":
        return {"bytes": sum(n for n in lens if n > case["keep"]) * h * 4 + B * h * case["keep"] * 4,
                "flops": sum(lens) * h}
    moved = sum(min(n, case["keep"]) for n in lens if n > case["keep"]) * h
    unit = _bytes(case["kb"]) + _bytes(case["vb"])
    return {"bytes": moved * (2 * unit + 8) + kept * 4 + (B * T - sum(min(n, case["keep"]) for n in lens)) * h * 4,
            "flops": moved}


# ---------------------------------------------------------------- the format (plain)

@functools.lru_cache(None)
def _levels(bits):
    """Lloyd-Max levels and boundaries (float32) of y = 2u - 1, u ~ Beta(64, 64): each level the
    mean of its cell, each boundary the midpoint of two levels."""
    n = 1 << bits
    x, w = np.polynomial.legendre.leggauss(96)

    def mean(lo, hi):
        y = 0.5 * (hi - lo)[:, None] * x + 0.5 * (hi + lo)[:, None]
        m = np.exp(63.0 * np.log1p(-y * y)) * w
        return (m * y).sum(1) / m.sum(1)

    c = (np.arange(n) + 0.5 - n / 2) * (4.0 / n) / math.sqrt(D)
    for _ in range(20000):
        b = 0.5 * (c[1:] + c[:-1])
        new = mean(np.concatenate([[-0.75], b]), np.concatenate([b, [0.75]]))
        new = 0.5 * (new - new[::-1])
        done = np.abs(new - c).max() < 1e-16
        c = new
        if done:
            break
    return c.astype(np.float32), (0.5 * (c[1:] + c[:-1])).astype(np.float32)


@functools.lru_cache(None)
def _signs():
    """+-1 diagonal D: output j of splitmix64 from the seed, top bit set means -1."""
    out, state, m = [], SIGN_SEED, (1 << 64) - 1
    for _ in range(D):
        state = (state + 0x9E3779B97F4A7C15) & m
        z = ((state ^ (state >> 30)) * 0xBF58476D1CE4E5B9) & m
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return np.array(out)


@functools.lru_cache(None)
def _rotation(dtype):
    """R = H D / sqrt(128) on the GPU, rows the outputs."""
    h = np.array([[1.0]])
    for _ in range(7):
        h = np.block([[h, h], [h, -h]])
    return torch.from_numpy(h * _signs()[None, :] / math.sqrt(D)).to("cuda", dtype)


@functools.lru_cache(None)
def _table(bits, dtype):
    return torch.from_numpy(_levels(bits)[0]).to("cuda", dtype)


@functools.lru_cache(None)
def _bounds(bits):
    return torch.from_numpy(_levels(bits)[1]).cuda()


def _pack(codes, norms, bits):
    """Codes (uint8 [..., 128]) and fp16 norms [...] -> blocks [..., 2 + 16 * bits]."""
    def plane(c, width):
        per = 8 // width
        c = c.reshape(*c.shape[:-1], -1, per)
        out = c[..., 0]
        for i in range(1, per):
            out = out | (c[..., i] << (width * i))
        return out

    parts = [norms.to(torch.float16).unsqueeze(-1).contiguous().view(torch.uint8)]
    parts += [plane(codes & 3, 2), plane(codes >> 2, 1)] if bits == 3 else [plane(codes, bits)]
    return torch.cat(parts, -1)


def _unpack(blocks, bits):
    """Blocks -> codes (int32 [..., 128]) and fp16 norms [...]."""
    norms = blocks[..., :2].contiguous().view(torch.float16).squeeze(-1)

    def plane(p, width):
        s = torch.arange(0, 8, width, device=p.device, dtype=torch.uint8)
        return ((p.unsqueeze(-1) >> s) & ((1 << width) - 1)).flatten(-2)

    if bits == 3:
        codes = plane(blocks[..., 2:34], 2) | (plane(blocks[..., 34:], 1) << 2)
    else:
        codes = plane(blocks[..., 2:], bits)
    return codes.int(), norms


def _rotated(blocks, bits, dtype):
    """Values of the blocks in the rotated domain: norm * c[code]."""
    codes, norms = _unpack(blocks, bits)
    return _table(bits, dtype)[codes] * norms.to(dtype).unsqueeze(-1)


# ---------------------------------------------------------------- rotary positions (plain)

def _pairs(case):
    """Axis and frequency (radians per position) of each rotated pair."""
    rot, sec = case["rot"], [int(s) for s in case["sections"].split(",")]
    n = rot // 2
    if case["interleaved"]:
        axis = [i % len(sec) if i < len(sec) * sec[i % len(sec)] else 0 for i in range(n)]
    else:
        axis = [a for a, s in enumerate(sec) for _ in range(s)]
    return axis, [case["base"] ** (-2.0 * i / rot) for i in range(n)]


def _plain_rope(x, pos, case):
    """x [n, heads, 128] rotated, in 64-bit (the angles of far positions need it)."""
    axis, freq = _pairs(case)
    n = case["rot"] // 2
    angle = pos.double()[torch.tensor(axis, device=pos.device)].T * torch.tensor(freq, device=pos.device,
                                                                                 dtype=torch.float64)
    cos, sin = angle.cos().unsqueeze(1), angle.sin().unsqueeze(1)
    x = x.double()
    a, b = (x[..., :n], x[..., n:2 * n]) if case["style"] == "half" else (x[..., 0:2 * n:2], x[..., 1:2 * n:2])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([ra, rb], -1) if case["style"] == "half" else torch.stack([ra, rb], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _positions(case, n, g):
    """Positions [axes, n]: text, then images (time fixed, height and width counting), text again."""
    axes = len(case["sections"].split(","))
    i = torch.arange(n, device="cuda", dtype=torch.int64)
    jitter = int(torch.randint(0, 64, (1,), generator=g, device="cuda"))
    t = case["start"] + jitter + i
    if axes == 1:
        return t.unsqueeze(0).contiguous()
    side = max(2, int(math.sqrt(max(1, n // 3))))
    image = (i >= n // 3) & (i < 2 * (n // 3))
    r = i - n // 3
    base = case["start"] + jitter + n // 3
    rows = [torch.where(image, base, t), torch.where(image, base + r // side, t), torch.where(image, base + r % side, t)]
    return torch.stack(rows[:axes]).contiguous()


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(shape, dtype, g):
    """N(0, 1) with a few loud channels, as keys and values of language models have them."""
    loud = torch.exp(0.5 * torch.randn(shape[-2:], generator=g, device="cuda"))
    return (torch.randn(shape, generator=g, device="cuda") * loud).to(DTYPES[dtype])


def _random_blocks(shape, bits, g):
    """Blocks as the encode makes them of Gaussian vectors, the norms log-normal."""
    out = torch.empty(*shape, _bytes(bits), dtype=torch.uint8, device="cuda")
    edges = _bounds(bits) * math.sqrt(D)
    flat = out.view(-1, _bytes(bits))
    for i in range(0, flat.shape[0], 1 << 20):
        n = min(1 << 20, flat.shape[0] - i)
        codes = torch.bucketize(torch.randn(n, D, generator=g, device="cuda"), edges, out_int32=True).to(torch.uint8)
        norm = math.sqrt(D) * torch.exp(0.3 * torch.randn(n, generator=g, device="cuda"))
        flat[i:i + n] = _pack(codes, norm, bits)
    return out


def _page_table(B, pages, g):
    """Every page of the pool used once, in a shuffled order."""
    return torch.randperm(B * pages, generator=g, device="cuda").int().view(B, pages)


def _logical(pool, table):
    """Pool [pages, hkv, page, bytes] -> [B, hkv, tokens, bytes]."""
    v = pool[table.long()]                                   # [B, pages, hkv, page, bytes]
    return v.transpose(1, 2).reshape(v.shape[0], v.shape[2], -1, v.shape[4])


def _insert_slots(case):
    return -(-case["tokens"] // case["page"]) * case["page"] if case["page"] else case["tokens"]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "rope":
        n, h = case["tokens"], case["heads"]
        # the query heads' part of one projection's output (queries, then two more heads)
        s["x"] = _activations((n, h + 2, D), case["dtype"], g)[:, :h]
        s["pos"] = _positions(case, n, g)
    elif op == "insert":
        n, h = case["tokens"], case["hkv"]
        kv = _activations((n, 2 * h, D), case["dtype"], g)
        s["k"], s["v"] = kv[:, :h], kv[:, h:]
        s["pos"] = _positions(case, n, g)
        slots = _insert_slots(case)
        token = torch.arange(n, device="cuda", dtype=torch.int64)
        if case["page"]:
            page = case["page"]
            table = torch.randperm(slots // page, generator=g, device="cuda")
            s["dst"], s["head_stride"] = table[token // page] * h * page + token % page, page
            shape = (slots // page, h, page)
        else:
            s["dst"], s["head_stride"] = token, slots
            shape = (1, h, slots)
        if case["padded"]:
            s["dst"] = torch.where((token + 1) % case["padded"] == 0, -1, s["dst"])
        s["k_blocks"] = torch.zeros(*shape, _bytes(case["kb"]), dtype=torch.uint8, device="cuda")
        s["v_blocks"] = torch.zeros(*shape, _bytes(case["vb"]), dtype=torch.uint8, device="cuda")
    else:
        B, h, T, cap = case["batch"], case["hkv"], case["T"], None
        s["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        if op in ("attend", "compact"):
            cap, page = _cap(case), case["page"]
            shape = (B * (cap // page), h, page) if page else (B, h, cap)
            s["table"] = _page_table(B, cap // page, g) if page else None
            s["k_blocks"] = _random_blocks(shape, case["kb"], g)
            s["v_blocks"] = _random_blocks(shape, case["vb"], g)
        # accumulated weights: most of it on few tokens, many equal (and zero) entries
        w = torch.randn(B, h, T, generator=g, device="cuda").mul_(2.0).exp_()
        s["weights"] = torch.where(w < 0.2, torch.zeros_like(w), (w * 64).round() / 64)
        if op == "attend":
            q = torch.randn(B, h, case["hq"] // h, D, generator=g, device="cuda")
            # every query looks at the first token and at one of its own (sinks and heavy tokens)
            at = torch.randint(0, T, (B, h), generator=g, device="cuda")
            for t in (torch.zeros_like(at), at):
                if s["table"] is None:
                    blk = s["k_blocks"][torch.arange(B, device="cuda")[:, None], torch.arange(h, device="cuda"), t]
                else:
                    pg = s["table"].long().gather(1, t // page)
                    blk = s["k_blocks"][pg, torch.arange(h, device="cuda"), t % page]
                y = _rotated(blk, case["kb"], torch.float32)
                y = y / y.norm(dim=-1, keepdim=True)
                q += 5.0 * (y @ _rotation(torch.float32)).unsqueeze(2)
            s["q"] = q.view(B, case["hq"], D).to(DTYPES[case["dtype"]])
        if op == "compact":
            s["kept"], s["new_lens"] = _plain_select(s["weights"], s["lens"], case)
    return s


# ---------------------------------------------------------------- plain forms

def _half(x):
    """float64 -> fp16 in one rounding (torch's own conversion goes through float32 and rounds twice): a float32
    rounded to odd keeps what the second rounding needs to know."""
    f = x.float()
    f = torch.where(f.double().abs() > x.abs(), torch.nextafter(f, torch.zeros_like(f)), f)
    return (f.view(torch.int32) | (f.double() != x).int()).view(torch.float32).half()


def _plain_encode(x, bits):
    """Rows (float64) -> blocks: y = R x / ||x|| in 64 bits, compared in float32."""
    n = x.norm(dim=-1, keepdim=True)
    y = torch.where(n > 0, (x @ _rotation(torch.float64).T) / n.clamp_min(1e-300), 0.0)
    codes = torch.bucketize(y.float(), _bounds(bits), right=True, out_int32=True).to(torch.uint8)
    return _pack(codes, _half(n.squeeze(-1)), bits)


def _plain_decode(blocks, bits):
    return (_rotated(blocks, bits, torch.float32) @ _rotation(torch.float32)).to(torch.bfloat16)


def _plain_insert(s):
    c = s["case"]
    h = c["hkv"]
    live = s["dst"] >= 0
    at = (s["dst"][live].unsqueeze(1) + torch.arange(h, device="cuda") * s["head_stride"]).flatten()
    for x, blocks, bits in ((_plain_rope(s["k"], s["pos"], c), s["k_blocks"], c["kb"]),
                            (s["v"].double(), s["v_blocks"], c["vb"])):
        blocks.view(-1, blocks.shape[-1])[at] = _plain_encode(x[live], bits).flatten(0, 1)
    return {"k": _plain_decode(s["k_blocks"], c["kb"]), "v": _plain_decode(s["v_blocks"], c["vb"])}


def _plain_attend(s):
    c = s["case"]
    B, h, T = c["batch"], c["hkv"], c["T"]
    kb, vb = s["k_blocks"], s["v_blocks"]
    if s["table"] is not None:
        kb, vb = _logical(kb, s["table"]), _logical(vb, s["table"])
    R = _rotation(torch.float32)
    q = (s["q"].float() @ R.T).view(B, h, -1, D)
    score = q @ _rotated(kb[:, :, :T], c["kb"], torch.float32).transpose(-1, -2) / math.sqrt(D)
    live = (torch.arange(T, device="cuda") < s["lens"].clamp(0, T).unsqueeze(1))[:, None, None]
    score = score.masked_fill(~live, -math.inf)
    p = (score - score.amax(-1, keepdim=True).clamp_min(-1e30)).exp()
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    out = (p @ _rotated(vb[:, :, :T], c["vb"], torch.float32)) @ R
    s["weights"] = torch.where(live[:, 0], c["decay"] * s["weights"] + p.sum(2), s["weights"])
    return {"out": out.view(B, -1, D).to(s["q"].dtype), "weights": s["weights"]}


def _plain_select(weights, lens, c):
    """Indices (ascending, -1 past the last) of the tokens that stay, and their number."""
    T, keep = c["T"], c["keep"]
    n = lens.clamp(0, T).long()[:, None, None]
    t = torch.arange(T, device="cuda")
    score = torch.where((t < c["first"]) | (t >= n - c["last"]) | (n <= keep), math.inf, weights)
    score = torch.where(t < n, score, -math.inf)
    kept = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.where(kept < n, kept, T).sort(-1).values
    return torch.where(kept < n, kept, -1).int(), lens.clamp(0, min(T, keep)).int()


def _plain_compact(s):
    c = s["case"]
    B, h, T = c["batch"], c["hkv"], c["T"]
    m = min(c["keep"], T)
    j = torch.arange(m, device="cuda")
    live = (j < s["new_lens"].unsqueeze(1)).unsqueeze(1).expand(B, h, m)
    src = torch.where(live, s["kept"][..., :m].long(), j)
    if s["table"] is None:
        bh = torch.arange(B * h, device="cuda").view(B, h, 1) * s["k_blocks"].shape[2]
        a, b = bh + src, bh + j
    else:
        page = c["page"]
        head = torch.arange(h, device="cuda").view(1, h, 1)

        def slot(t):
            pg = s["table"].long().unsqueeze(1).expand(B, h, -1).gather(2, (t // page).expand(B, h, m))
            return (pg * h + head) * page + t % page

        a, b = slot(src), slot(j)
    for blocks in (s["k_blocks"], s["v_blocks"]):
        flat = blocks.view(-1, blocks.shape[-1])
        flat[b.flatten()] = flat[a.flatten()]
    w = torch.zeros_like(s["weights"])
    w[..., :m] = torch.where(live, s["weights"].gather(2, src), 0.0)
    s["weights"] = w
    return {"k_blocks": s["k_blocks"], "v_blocks": s["v_blocks"], "weights": w}


# ---------------------------------------------------------------- the library's calls

@functools.lru_cache(None)
def _lib():
    from turboquant_bit_kv_gb300 import tq
    return tq, {b: tq.tq_codebook_load(128, b) for b in (2, 3, 4)}, tq.tq_signs_from_seed(SIGN_SEED)


@functools.lru_cache(None)
def _own_rope(rot, base, style, sections, interleaved):
    tq = _lib()[0]
    return tq.tq_rope_load(rot, base, tq.TQ_ROPE_HALF if style == "half" else tq.TQ_ROPE_ADJACENT,
                           [int(x) for x in sections.split(",")], interleaved)


def _own_rope_of(c):
    return _own_rope(c["rot"], c["base"], c["style"], c["sections"], c["interleaved"])


def _own_run(s):
    tq, books, signs = _lib()
    c = s["case"]
    op = c["op"]
    if op == "rope":
        if "out" not in s:
            s["out"] = torch.empty(s["x"].shape, dtype=s["x"].dtype, device="cuda")
        return {"out": tq.tq_rope_apply(s["x"], s["pos"], _own_rope_of(c), s["out"])}
    if op == "insert":
        kb, vb = s["k_blocks"], s["v_blocks"]
        if "k_out" not in s:
            s["k_out"] = torch.empty(*kb.shape[:3], D, dtype=torch.bfloat16, device="cuda")
            s["v_out"] = torch.empty_like(s["k_out"])
        tq.tq_insert_kv(s["k"], s["v"], s["pos"], _own_rope_of(c), books[c["kb"]], books[c["vb"]], signs, kb, vb,
                        s["dst"], s["head_stride"])
        n = kb.shape[0] * kb.shape[1] * kb.shape[2]
        tq.tq_decode_kv(kb, n, books[c["kb"]], signs, s["k_out"])
        tq.tq_decode_kv(vb, n, books[c["vb"]], signs, s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "attend":
        if "ws" not in s:
            n = tq.tq_attn_weights_workspace_bytes(c["batch"], c["hq"], c["hkv"], c["T"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
            s["out"] = torch.empty_like(s["q"])
        tq.tq_attn_decode_weights(s["q"], s["k_blocks"], books[c["kb"]], s["v_blocks"], books[c["vb"]], s["weights"],
                                  s["out"], s["ws"], c["T"], 1 / math.sqrt(D), signs, seq_lens=s["lens"],
                                  block_table=s["table"], decay=c["decay"])
        return {"out": s["out"], "weights": s["weights"]}
    if op == "select":
        if "kept" not in s:
            s["kept"] = torch.empty(c["batch"], c["hkv"], c["keep"], dtype=torch.int32, device="cuda")
            s["new_lens"] = torch.empty_like(s["lens"])
        tq.tq_evict_select(s["weights"], s["kept"], s["new_lens"], c["T"], c["first"], c["last"], seq_lens=s["lens"])
        return {"kept": s["kept"], "new_lens": s["new_lens"]}
    tq.tq_evict_compact(s["k_blocks"], s["v_blocks"], s["kept"], s["new_lens"], c["T"], weights=s["weights"],
                        block_table=s["table"])
    return {"k_blocks": s["k_blocks"], "v_blocks": s["v_blocks"], "weights": s["weights"]}


def run(state):
    if own:
        return _own_run(state)
    c = state["case"]
    op = c["op"]
    if op == "rope":
        return {"out": _plain_rope(state["x"], state["pos"], c).to(state["x"].dtype)}
    if op == "insert":
        return _plain_insert(state)
    if op == "attend":
        return _plain_attend(state)
    if op == "select":
        kept, new_lens = _plain_select(state["weights"], state["lens"], c)
        return {"kept": kept, "new_lens": new_lens}
    return _plain_compact(state)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_butterfly(x):
    """Unnormalised Walsh-Hadamard transform of the last axis (128), Sylvester order."""
    for i in range(7):
        y = x.reshape(*x.shape[:-1], 128 >> (i + 1), 2, 1 << i)
        x = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(x.shape)
    return x


def _exact_vectors(blocks, bits):
    """The 128-element vectors that blocks stand for, one element of the code at a time."""
    raw = blocks.to(torch.int32)
    j = torch.arange(D, device="cuda")
    if bits == 4:
        code = (raw[..., 2 + j // 2] >> (4 * (j % 2))) & 15
    elif bits == 2:
        code = (raw[..., 2 + j // 4] >> (2 * (j % 4))) & 3
    else:
        code = ((raw[..., 2 + j // 4] >> (2 * (j % 4))) & 3) + 4 * ((raw[..., 34 + j // 8] >> (j % 8)) & 1)
    c = torch.from_numpy(_levels(bits)[0]).cuda().double()[code.long()]
    norm = blocks[..., :2].contiguous().view(torch.float16).double()
    sign = torch.from_numpy(_signs()).cuda()
    return _exact_butterfly(c) * sign * norm / math.sqrt(D)


def _exact_turn(x, pos, case):
    """Rotary positions as complex products, one pair after the other's definition."""
    axis, freq = _pairs(case)
    n, x = case["rot"] // 2, x.double().clone()
    half = case["style"] == "half"
    first = torch.arange(n, device="cuda") if half else 2 * torch.arange(n, device="cuda")
    second = first + (n if half else 1)
    z = torch.complex(x[..., first], x[..., second])
    turn = torch.stack([pos[axis[i]].double() * freq[i] for i in range(n)], -1)
    z = z * torch.polar(torch.ones_like(turn), turn).unsqueeze(1)
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_quantised(x, bits):
    """What the encode keeps of each row: nearest level of every coordinate, the norm in fp16."""
    norm = x.square().sum(-1, keepdim=True).sqrt()
    sign = torch.from_numpy(_signs()).cuda()
    y = _exact_butterfly(x * sign) / (math.sqrt(D) * norm)
    y = torch.where(norm > 0, y, 0.0).float()
    code = torch.zeros(y.shape, dtype=torch.int64, device="cuda")
    for b in _levels(bits)[1].tolist():
        code += y >= b
    c = torch.from_numpy(_levels(bits)[0]).cuda().double()[code]
    step = torch.exp2(torch.floor(torch.log2(norm.clamp_min(2.0**-14))) - 10)      # spacing of fp16 at the norm
    return _exact_butterfly(c) * sign * (torch.round(norm / step) * step) / math.sqrt(D)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return {"out": _exact_turn(s["x"], s["pos"], case)}
    if op == "insert":
        n, h = case["tokens"], case["hkv"]
        out = {}
        for name, x, blocks, bits in (("k", s["k"], s["k_blocks"], case["kb"]), ("v", s["v"], s["v_blocks"], case["vb"])):
            full = torch.zeros(blocks.shape[0] * blocks.shape[1] * blocks.shape[2], D, dtype=torch.float64, device="cuda")
            for i in range(0, n, 8192):
                part, dst = x[i:i + 8192], s["dst"][i:i + 8192]
                part = _exact_turn(part, s["pos"][:, i:i + 8192], case) if name == "k" else part.double()
                got = _exact_quantised(part, bits)
                for head in range(h):
                    full[(dst + head * s["head_stride"])[dst >= 0]] = got[dst >= 0, head]
            out[name] = full.view(*blocks.shape[:3], D)
        return out
    if op == "attend":
        B, h, T = case["batch"], case["hkv"], case["T"]
        G = case["hq"] // h
        out = torch.zeros(B, case["hq"], D, dtype=torch.float64, device="cuda")
        weights = s["weights"].double()
        for b, n in enumerate(_lens_clamped(case)):
            if n == 0:
                continue
            for head in range(h):
                vec = []
                for blocks, bits in ((s["k_blocks"], case["kb"]), (s["v_blocks"], case["vb"])):
                    rows = blocks[b, head] if s["table"] is None else blocks[s["table"][b].long(), head].flatten(0, 1)
                    vec.append(_exact_vectors(rows[:n], bits))
                q = s["q"][b, head * G:(head + 1) * G].double()
                p = torch.softmax(vec[0] @ q.T / math.sqrt(D), 0)
                out[b, head * G:(head + 1) * G] = p.T @ vec[1]
                weights[b, head, :n] = case["decay"] * weights[b, head, :n] + p.sum(1)
        return {"out": out, "weights": weights}
    if op == "compact":
        w, kept = s["weights"].cpu().numpy().astype(np.float64), s["kept"].cpu().numpy()
        new = np.zeros_like(w)
        for b, m in enumerate(s["new_lens"].tolist()):
            for head in range(case["hkv"]):
                new[b, head, :m] = w[b, head, kept[b, head, :m]]
        return {"k_blocks": None, "v_blocks": None, "weights": torch.from_numpy(new)}
    return None
