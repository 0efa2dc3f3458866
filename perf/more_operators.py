"""Measured cases of the operators of a paged serving step over the packed key/value cache.

Three operators that a step of a serving loop runs one after the other:

* ``plan``    block tables and slot maps from the requests' lengths: pages for the new tokens
              taken from a list of free ones, each token's slot and position,
* ``norm``    queries and keys normalised head by head (RMS, with weights) and turned by rotary
              positions, in one pass over a projection's output,
* ``shared``  one query token per sequence against a packed cache whose first part, a prefix,
              is the same for the whole batch, and each sequence's own tokens after it.

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
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 64 conversations, a few of them finished
        dict(name="plan-step", op="plan", batch=64, kind="decode", tokens=64, page=64, hkv=8, cached=8192, prefix=0,
             ahead=False, short=False, padded=0),
        # a step that mixes prompt chunks with decodes behind a common prefix, after an eviction (positions ahead of
        # the slots), with too few free pages for all, the token batch padded
        dict(name="plan-mixed", op="plan", batch=257, kind="mixed", tokens=12001, page=16, hkv=4, cached=4096,
             prefix=1024, ahead=True, short=True, padded=97),
        # 512 prompts of up to 1024 tokens at once, in small pages
        dict(name="plan-prompts", op="plan", batch=512, kind="prompt", tokens=262144, page=16, hkv=8, cached=0,
             prefix=0, ahead=False, short=False, padded=0),
        # a decode step of 16 sequences: query and key heads of one layer, three-axis positions
        dict(name="norm-step", op="norm", tokens=16, hq=32, hkv=8, dtype="bf16", style="half", rot=128,
             sections="16,24,24", interleaved=False, start=700, base=1000000.0),
        # a chunk of prompts, seven query heads for each key head, half of each head turned
        dict(name="norm-chunk", op="norm", tokens=2049, hq=28, hkv=4, dtype="f16", style="adjacent", rot=64,
             sections="32", interleaved=False, start=0, base=10000.0),
        # a prompt with images at far positions, interleaved axes, an odd number of tokens
        dict(name="norm-prompt", op="norm", tokens=16411, hq=32, hkv=8, dtype="bf16", style="half", rot=128,
             sections="24,20,20", interleaved=True, start=1000000, base=5000000.0),
        # four samples of one prompt, a little way into their answers
        dict(name="shared-few", op="shared", batch=4, hq=32, hkv=8, P=1001, T=100, kb=4, vb=2, dtype="bf16", page=0,
             ragged=False, slack=0),
        # 32 samples of a prompt of 8192 tokens, answers of up to 1024
        dict(name="shared-samples", op="shared", batch=32, hq=32, hkv=8, P=8192, T=1024, kb=4, vb=2, dtype="bf16",
             page=0, ragged=True, slack=0),
        # 17 conversations behind a system prompt in pages of 16 tokens, some slots of the batch empty, a captured
        # step's bound on the prefix above its length
        dict(name="shared-pages", op="shared", batch=17, hq=40, hkv=8, P=10007, T=2000, kb=4, vb=4, dtype="f16",
             page=16, ragged=True, slack=700),
        # a full serving batch behind a document of 32k tokens, seven query heads for each KV head
        dict(name="shared-batch", op="shared", batch=64, hq=28, hkv=4, P=32769, T=1000, kb=3, vb=3, dtype="bf16",
             page=64, ragged=True, slack=0),
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
    op = rng.choice(["plan", "norm", "shared", "shared"])
    if op == "plan":
        kind = rng.choice(["decode", "mixed", "prompt"])
        batch = _log(rng, 1, 512 if kind == "prompt" else 4096)
        tokens = batch if kind == "decode" else _log(rng, batch, 262144)
        return dict(op=op, batch=batch, kind=kind, tokens=tokens, page=rng.choice([8, 16, 32, 64, 128, 100]),
                    hkv=rng.choice([1, 2, 4, 8]), cached=_log(rng, 1, 8192),
                    prefix=rng.choice([0, 0, _log(rng, 1, 4096)]), ahead=rng.random() < 0.3,
                    short=rng.random() < 0.3, padded=rng.choice([0, rng.randint(1, 300)]))
    if op == "norm":
        hkv, dtype = rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice(["bf16", "f16", "f32"])
        hq = hkv * rng.randint(1, 8)
        return dict(op=op, tokens=_log(rng, 1, 16411 * 80 // ((hq + hkv) * SIZES[dtype])), hq=hq, hkv=hkv, dtype=dtype,
                    **_rope_params(rng))
    batch, hkv = _log(rng, 1, 128), rng.choice([1, 2, 4, 8])
    hq = hkv * rng.randint(1, 8)
    room = 64 * 28 * 33769 // (batch * hq)
    P = _log(rng, 1, min(131072, room * 3 // 4))
    return dict(op=op, batch=batch, hq=hq, hkv=hkv, P=P, T=_log(rng, 1, min(4096, max(1, room // 4))),
                kb=rng.choice([2, 3, 4]), vb=rng.choice([2, 3, 4]), dtype=rng.choice(["bf16", "f16"]),
                page=rng.choice([0, 0, 8, 16, 32, 64, 128, 72]), ragged=rng.random() < 0.6,
                slack=rng.choice([0, 0, rng.randint(1, 1000)]))


def _spread(case):
    """Own tokens of each sequence behind the prefix: T, or (ragged) a fixed pattern from T down to none, -1 for an
    empty slot of the batch."""
    B, T = case["batch"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [T if b == 0 else max(0, (T * ((b * 7) % 16 + 1)) // 16 - 3 * b % 11) if b % 5 else b % 2 - 1
            for b in range(B)]


def _new_tokens(case):
    """New tokens of each request."""
    B, kind = case["batch"], case["kind"]
    if kind == "decode":
        return [0 if i % 7 == 6 else 1 for i in range(B)]
    if kind == "mixed":
        chunk = max(1, case["tokens"] * 8 // B)
        return [max(1, chunk - (i * 37) % (chunk // 2 + 1)) if i % 8 == 3 else 1 for i in range(B)]
    most = max(1, case["tokens"] // B)
    return [max(1, most - (i * 7919) % (most // 2 + 1)) for i in range(B)]


def _max_pages(case):
    """Entries of a request's row of the block table."""
    return -(-(case["prefix"] + case["cached"] + max(_new_tokens(case))) // case["page"]) + 2


def _bytes(bits):
    return 2 + 16 * bits


def work(case):
    op = case["op"]
    if op == "plan":
        B, new = case["batch"], sum(_new_tokens(case))
        # lengths, pages held, first tokens of the requests, the new pages (read and entered), slots and positions
        return {"bytes": 4 * (6 * B + 3) + 8 * (new // case["page"]) + 16 * (new + case["padded"]),
                "flops": 8 * B + 4 * new}
    if op == "norm":
        n, h = case["tokens"], case["hq"] + case["hkv"]
        axes = len(case["sections"].split(","))
        return {"bytes": 2 * n * h * D * SIZES[case["dtype"]] + 8 * n * axes + 4 * D,
                "flops": n * h * (4 * D + 3 * case["rot"])}
    B, h, hq, P = case["batch"], case["hkv"], case["hq"], case["P"]
    lens = _spread(case)
    live = sum(max(n, 0) for n in lens)
    active = sum(n >= 0 for n in lens)
    return {"bytes": (P + live) * h * (_bytes(case["kb"]) + _bytes(case["vb"])) + B * hq * D * 2 * SIZES[case["dtype"]],
            "flops": 4 * hq * D * (active * P + live)}


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


# ---------------------------------------------------------------- rotary positions

def _pairs(case):
    """Axis and frequency (radians per position) of each rotated pair."""
    rot, sec = case["rot"], [int(s) for s in case["sections"].split(",")]
    n = rot // 2
    if case["interleaved"]:
        axis = [i % len(sec) if i < len(sec) * sec[i % len(sec)] else 0 for i in range(n)]
    else:
        axis = [a for a, s in enumerate(sec) for _ in range(s)]
    return axis, [case["base"] ** (-2.0 * i / rot) for i in range(n)]


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


def _prepare_plan(case, g):
    B, page = case["batch"], case["page"]
    most = _max_pages(case)
    order = torch.randperm(B, generator=g, device="cuda")
    new = torch.tensor(_new_tokens(case), dtype=torch.int32, device="cuda")[order]
    cached = case["prefix"] + torch.randint(0, case["cached"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    held = (cached + page - 1) // page
    # the requests' pages: the common prefix's, then pages of their own, shuffled over the pool
    shared = case["prefix"] // page
    pool = torch.randperm(shared + B * most, generator=g, device="cuda").int()
    table = pool[shared:].view(B, most).clone()
    table[:, :shared] = pool[:shared]
    column = torch.arange(most, device="cuda")
    free = table[column >= held.unsqueeze(1)]
    free = free[torch.randperm(free.numel(), generator=g, device="cuda")].contiguous()
    table[column >= held.unsqueeze(1)] = -1
    need = int((((cached + new + page - 1) // page) - held).sum())
    count = need * 2 // 3 if case["short"] else min(free.numel(), need + 1 + B)
    return {"cached": cached, "new": new, "held": held.int(), "table": table, "free": free,
            "count": torch.tensor([count], dtype=torch.int32, device="cuda"),
            "pos_start": cached.long() + 1000 * order if case["ahead"] else None,
            "n_tok": sum(_new_tokens(case)) + case["padded"]}


def _prepare_norm(case, g):
    n, hq, h = case["tokens"], case["hq"], case["hkv"]
    x = _activations((n, hq + 2 * h, D), case["dtype"], g)      # one projection's output: queries, keys, values
    axes = len(case["sections"].split(","))
    i = torch.arange(n, device="cuda", dtype=torch.int64)
    base = case["start"] + int(torch.randint(0, 64, (1,), generator=g, device="cuda"))
    t = base + i
    # text, then images (time fixed, height and width counting), text again
    side = max(2, int(math.sqrt(max(1, n // 3))))
    image, r = (i >= n // 3) & (i < 2 * (n // 3)), i - n // 3
    first = base + n // 3
    pos = torch.stack([torch.where(image, first, t), torch.where(image, first + r // side, t),
                       torch.where(image, first + r % side, t)][:axes] if axes > 1 else [t]).contiguous()
    weights = (1.0 + 0.2 * torch.randn(2, D, generator=g, device="cuda")).to(DTYPES[case["dtype"]])
    return {"q": x[:, :hq], "k": x[:, hq:hq + h], "q_weight": weights[0], "k_weight": weights[1], "pos": pos}


def _prepare_shared(case, g):
    B, h, hq, P, T, page = case["batch"], case["hkv"], case["hq"], case["P"], case["T"], case["page"]
    bound = P + case["slack"]
    s = {"lens": torch.tensor(_spread(case), dtype=torch.int32, device="cuda"), "bound": bound,
         "prefix_len": torch.tensor([P], dtype=torch.int32, device="cuda") if case["slack"] else None}
    if page:
        # one pool; every row of the table starts with the prefix's pages
        np_, no = -(-bound // page), -(-T // page)
        order = torch.randperm(np_ + B * no, generator=g, device="cuda").int()
        s["table"] = torch.cat([order[:np_].expand(B, np_), order[np_:].view(B, no)], 1).contiguous()
        s["prefix_table"], s["own_table"] = s["table"][0, :np_], s["table"][:, np_:]
        shape = (np_ + B * no, h, page)
        s["k"] = s["k_prefix"] = _random_blocks(shape, case["kb"], g)
        s["v"] = s["v_prefix"] = _random_blocks(shape, case["vb"], g)
    else:
        s["prefix_table"] = s["own_table"] = None
        for name, bits in (("k", case["kb"]), ("v", case["vb"])):
            s[name + "_prefix"] = _random_blocks((h, -(-bound // 8) * 8), bits, g)
            s[name] = _random_blocks((B, h, -(-T // 8) * 8), bits, g)
    q = torch.randn(B, h, hq // h, D, generator=g, device="cuda")
    # every query looks at the prefix's first token and at one of its own choice (sinks and heavy tokens)
    kp = _prefix(s, "k", P)
    at = torch.randint(0, P, (B, h), generator=g, device="cuda")
    for t in (torch.zeros_like(at), at):
        y = _rotated(kp[torch.arange(h, device="cuda"), t], case["kb"], torch.float32)
        q += 5.0 * ((y / y.norm(dim=-1, keepdim=True)) @ _rotation(torch.float32)).unsqueeze(2)
    s["q"] = q.view(B, hq, D).to(DTYPES[case["dtype"]])
    return s


def _prefix(s, name, P):
    """The prefix's blocks [hkv, P, bytes]."""
    blocks = s[name + "_prefix"]
    if s["prefix_table"] is None:
        return blocks[:, :P]
    return blocks[s["prefix_table"].long()].transpose(0, 1).flatten(1, 2)[:, :P]


def _owned(s, name, T):
    """The sequences' own blocks [B, hkv, T, bytes]."""
    if s["own_table"] is None:
        return s[name][:, :, :T]
    v = s[name][s["own_table"].long()]                       # [B, pages, hkv, page, bytes]
    return v.transpose(1, 2).flatten(2, 3)[:, :, :T]


def prepare(case, seed):
    make = {"plan": _prepare_plan, "norm": _prepare_norm, "shared": _prepare_shared}[case["op"]]
    return {"case": case, **make(case, _gen(seed))}


# ---------------------------------------------------------------- plain forms

def _plain_plan(s):
    c = s["case"]
    page, most, n_tok = c["page"], s["table"].shape[1], s["n_tok"]
    cached, new, held = s["cached"].long(), s["new"].long(), s["held"].long()
    total = cached + new
    last = new.cumsum(0)                                     # first token of the next request
    fits = (total <= most * page) & (last <= n_tok)
    need = torch.where(fits & (new > 0), (total + page - 1) // page - held, 0).clamp_min(0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= s["count"]))
    need = torch.where(ok, need, 0)
    column = torch.arange(most, device="cuda")
    fresh = column - held.unsqueeze(1)                       # how many pages of the request come before
    take = (fresh >= 0) & (fresh < need.unsqueeze(1))
    at = (s["count"].long() - 1 - (upto - need).unsqueeze(1) - fresh).clamp(0, max(0, s["free"].numel() - 1))
    table = torch.where(take, s["free"][at], s["table"]) if s["free"].numel() else s["table"]
    start = last - new
    n = torch.arange(n_tok, device="cuda")
    b = torch.searchsorted(last, n, right=True).clamp_max(c["batch"] - 1)
    live = n < last[-1]
    slot = cached[b] + n - start[b]
    pg = table[b, (slot // page).clamp(0, most - 1)].long()
    dst = torch.where(live & ok[b], pg * c["hkv"] * page + slot % page, -1)
    first = cached if s["pos_start"] is None else s["pos_start"]
    return {"block_table": table, "held": (held + need).int(), "free_count": (s["count"] - need.sum()).int(),
            "seq_lens": torch.where(ok, total, cached).int(),
            "tok_start": torch.cat([last.new_zeros(1), last]).int(),
            "dst": dst, "pos": torch.where(live, first[b] + n - start[b], 0)}


def _plain_norm(s):
    c = s["case"]
    axis, freq = _pairs(c)
    n, half = c["rot"] // 2, c["style"] == "half"
    angle = s["pos"].double()[torch.tensor(axis, device="cuda")].T * torch.tensor(freq, device="cuda", dtype=torch.float64)
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s[name + "_weight"].float()
        a, b = (x[..., :n], x[..., n:2 * n]) if half else (x[..., 0:2 * n:2], x[..., 1:2 * n:2])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        turned = torch.cat([ra, rb], -1) if half else torch.stack([ra, rb], -1).flatten(-2)
        out[name] = torch.cat([turned, x[..., 2 * n:]], -1).to(s[name].dtype)
    return out


def _plain_shared(s):
    c = s["case"]
    B, h, P, T = c["batch"], c["hkv"], c["P"], c["T"]
    R = _rotation(torch.float32)
    q = (s["q"].float() @ R.T).view(B, h, -1, D)
    G = q.shape[2]
    rows = q.transpose(0, 1).reshape(h, B * G, D)            # every query of a KV head against the prefix
    kp, vp = (_rotated(_prefix(s, n, P), c[n + "b"], torch.float32) for n in "kv")
    ko, vo = (_rotated(_owned(s, n, T), c[n + "b"], torch.float32) for n in "kv")
    before = (rows @ kp.transpose(-1, -2)).view(h, B, G, P).transpose(0, 1)
    score = torch.cat([before, q @ ko.transpose(-1, -2)], -1) / math.sqrt(D)
    n = s["lens"].unsqueeze(1)
    live = torch.cat([(n >= 0).expand(B, P), torch.arange(T, device="cuda") < n], 1)[:, None, None]
    score = score.masked_fill(~live, -math.inf)
    p = (score - score.amax(-1, keepdim=True).clamp_min(-1e30)).exp()
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = (p[..., :P].transpose(0, 1).reshape(h, B * G, P) @ vp).view(h, B, G, D).transpose(0, 1) + p[..., P:] @ vo
    return {"out": (o @ R).reshape(B, -1, D).to(s["q"].dtype)}


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


def _own_run(s):
    tq, books, signs = _lib()
    c = s["case"]
    if c["op"] == "plan":
        if "out" not in s:
            B, n = c["batch"], s["n_tok"]
            i32, i64 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.int64, device="cuda")
            s["out"] = {"block_table": s["table"], "held": torch.empty(B, **i32), "free_count": torch.empty(1, **i32),
                        "seq_lens": torch.empty(B, **i32), "tok_start": torch.empty(B + 1, **i32),
                        "dst": torch.empty(n, **i64), "pos": torch.empty(n, **i64)}
        o = s["out"]
        tq.tq_page_plan(s["cached"], s["new"], s["held"], s["table"], s["free"], s["count"], c["page"], c["hkv"],
                        o["held"], o["free_count"], o["seq_lens"], o["tok_start"], o["dst"], o["pos"],
                        pos_start=s["pos_start"])
        return o
    if c["op"] == "norm":
        if "out" not in s:
            s["out"] = {n: torch.empty(s[n].shape, dtype=s[n].dtype, device="cuda") for n in ("q", "k")}
        rope = _own_rope(c["rot"], c["base"], c["style"], c["sections"], c["interleaved"])
        tq.tq_norm_rope_apply(s["q"], s["k"], s["q_weight"], s["k_weight"], EPS, s["pos"], rope, s["out"]["q"],
                              s["out"]["k"])
        return s["out"]
    if "ws" not in s:
        n = tq.tq_attn_shared_workspace_bytes(c["batch"], c["hq"], c["hkv"], s["bound"], c["T"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty_like(s["q"])
    tq.tq_attn_decode_shared(s["q"], s["k_prefix"], s["v_prefix"], s["k"], books[c["kb"]], s["v"], books[c["vb"]],
                             s["out"], s["ws"], s["bound"], c["T"], 1 / math.sqrt(D), signs,
                             prefix_len=s["prefix_len"], prefix_table=s["prefix_table"], seq_lens=s["lens"],
                             block_table=s["own_table"])
    return {"out": s["out"]}


def run(state):
    if own:
        return _own_run(state)
    return {"plan": _plain_plan, "norm": _plain_norm, "shared": _plain_shared}[state["case"]["op"]](state)


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


def _exact_turned(x, weight, pos, case):
    """RMS-normalised heads, rotary positions as complex products."""
    axis, freq = _pairs(case)
    x = x.double()
    x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
    i = torch.arange(case["rot"] // 2, device="cuda")
    first, second = (i, i + case["rot"] // 2) if case["style"] == "half" else (2 * i, 2 * i + 1)
    turn = torch.stack([pos[a].double() * f for a, f in zip(axis, freq)], -1)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(turn), turn).unsqueeze(1)
    x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None                                          # whole numbers only: the plain form's are the definition's
    if case["op"] == "norm":
        return {n: _exact_turned(s[n], s[n + "_weight"], s["pos"], case) for n in ("q", "k")}
    B, h, P = case["batch"], case["hkv"], case["P"]
    G = case["hq"] // h
    out = torch.zeros(B, case["hq"], D, dtype=torch.float64, device="cuda")
    for head in range(h):
        kp, vp = (_exact_vectors(_prefix(s, n, P)[head], case[n + "b"]) for n in "kv")
        for b, n in enumerate(_spread(case)):
            if n < 0:
                continue
            k, v = (torch.cat([p, _exact_vectors(_owned(s, name, case["T"])[b, head, :n], case[name + "b"])])
                    for name, p in (("k", kp), ("v", vp)))
            q = s["q"][b, head * G:(head + 1) * G].double()
            out[b, head * G:(head + 1) * G] = torch.softmax(q @ k.T / math.sqrt(D), -1) @ v
    return {"out": out}
