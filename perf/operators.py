"""The decode step's attention side, measured: rotary positions, the append of
rotated keys and values to a paged 4-bit cache, and the attention that reads
it.

``own`` false: ``run`` computes each operator in its plain form, elementary
torch operations in 32 bits (angles in 64).  ``own`` true: ``run`` calls the
library's entry points.  Both work on the state ``prepare`` makes; ``exact``
evaluates the definitions in 64 bits, separately from the plain form.

The 4-bit cache holds blocks of 32 consecutive values of a head: 32 codes of
1 sign, 2 exponent and 1 mantissa bits (the magnitudes 0, 0.5, 1, 1.5, 2, 3,
4, 6) and one 8-bit power-of-two scale 2^(s - 127) (the OCP microscaling
format).  For a block with largest magnitude a, the scale's exponent is
floor(log2 a) - 2, one more where a scaled by that exceeds 7, held to
-125..125; values round to the nearest code, ties to the even code, and
saturate at 6.  Pages hold ``page`` consecutive positions of one sequence; a
block table names each sequence's pages.
"""

import math
import random

import numpy as np
import torch

own = False

# --------------------------------------------------------------------- cases

# Head layouts: the 68M-parameter decoder of the workloads has 12 query and 12
# key heads of 64, the 14B-parameter one 40 query and 8 key heads of 128.


def listed():
    return [
        # one token of one session of the small decoder: its query and key
        # heads rotated, where only the latency of the call counts
        dict(name="rotary_one_row", op="rotary", rows=1, heads=24, dim=64, rot=64,
             interleaved=False, scaling="none", base=1e4, stride=2304, top_pos=2048),
        # a full 16-slot step of the large decoder, as its QKV rows stand
        dict(name="rotary_step", op="rotary", rows=16, heads=48, dim=128, rot=128,
             interleaved=False, scaling="none", base=1e6, stride=7168, top_pos=40960),
        # the queries of a long prompt, adjacent pairs, three quarters of the
        # head rotated, frequencies stretched to four times the trained length
        dict(name="rotary_prompt", op="rotary", rows=4099, heads=40, dim=128, rot=96,
             interleaved=True, scaling="yarn", base=1e6, stride=7168, top_pos=131072),
        # one token of one session of the small decoder put into its cache
        dict(name="append_one_row", op="append", rows=1, seqs=1, q_heads=12, kv_heads=12, dim=64,
             rot=64, interleaved=False, scaling="none", base=1e4, page=64, top_pos=2048),
        # a full 16-slot step of the large decoder: 16 sessions at their own positions
        dict(name="append_step", op="append", rows=16, seqs=16, q_heads=40, kv_heads=8, dim=128,
             rot=128, interleaved=False, scaling="none", base=1e6, page=64, top_pos=40960),
        # three prompts of the large decoder's shape put into the cache at once
        dict(name="append_prompt", op="append", rows=4099, seqs=3, q_heads=40, kv_heads=8, dim=128,
             rot=64, interleaved=True, scaling="linear", base=1e6, page=32, top_pos=8192),
        # the small decoder's first tokens: one query row on a short context
        dict(name="attend_one_short", op="attend", seqs=1, tokens=1, q_heads=12, kv_heads=12,
             dim=64, page=64, ctx_lo=77, ctx_hi=77, window=0, empty=False, lens=1),
        # an ordinary serving step: 16 sessions between a few and 8192 tokens
        dict(name="attend_step", op="attend", seqs=16, tokens=1, q_heads=40, kv_heads=8,
             dim=128, page=64, ctx_lo=5, ctx_hi=8192, window=0, empty=False, lens=2),
        # the same step with every session near the model's full context
        dict(name="attend_long", op="attend", seqs=16, tokens=1, q_heads=40, kv_heads=8,
             dim=128, page=64, ctx_lo=24001, ctx_hi=32768, window=0, empty=False, lens=3),
        # speculative decoding: 16 sessions of 3 drafted tokens each, one slot idle
        dict(name="attend_drafts", op="attend", seqs=16, tokens=4, q_heads=40, kv_heads=8,
             dim=128, page=64, ctx_lo=1000, ctx_hi=6001, window=0, empty=True, lens=4),
        # a 64-column piece of one session's prompt over what is cached already
        dict(name="attend_prompt_piece", op="attend", seqs=1, tokens=64, q_heads=40, kv_heads=8,
             dim=128, page=128, ctx_lo=8193, ctx_hi=8193, window=0, empty=False, lens=5),
        # sliding-window layers with another head size and page size
        dict(name="attend_window", op="attend", seqs=7, tokens=1, q_heads=15, kv_heads=5,
             dim=96, page=96, ctx_lo=300, ctx_hi=20000, window=1024, empty=False, lens=6),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotary", "append", "attend", "attend"))
    dim = rng.choice((32, 64, 64, 96, 128, 128, 128, 160, 256))
    kv = rng.choice((1, 2, 3, 4, 5, 8, 12))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8))
    scaling = rng.choice(("none", "linear", "ntk", "bands", "yarn"))
    rot = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
    base = rng.choice((1e4, 5e5, 1e6))
    inter = rng.random() < 0.4
    if op == "rotary":
        heads = kv * group
        rows = _log(rng, 1, max(1, min(8192, 4099 * 40 * 128 // (heads * dim))))
        return dict(op=op, rows=rows, heads=heads, dim=dim, rot=rot, interleaved=inter,
                    scaling=scaling, base=base, stride=heads * dim + rng.choice((0, 4, 37, 256)),
                    top_pos=_log(rng, 64, 262144))
    page = rng.choice((32, 64, 64, 96, 128, 256))
    if op == "append":
        rows = _log(rng, 1, max(1, min(8192, 4099 * 56 * 128 // ((group + 2) * kv * dim))))
        return dict(op=op, rows=rows, seqs=rng.randint(1, min(rows, 16)), q_heads=kv * group,
                    kv_heads=kv, dim=dim, rot=rot, interleaved=inter, scaling=scaling, base=base,
                    page=page, top_pos=max(_log(rng, 64, 65536), rows))
    tokens = rng.choice((1, 1, 1, 1, 2, 4, 5, 8, 17, 64))
    seqs = _log(rng, 1, 64 // tokens if tokens < 64 else 1)
    # no more cached values than the largest listed case, and no more products
    top = 16 * 28000 * 8 * 128 // (seqs * kv * dim)
    top = min(top, 400 * 8193 * 8 * 128 * 5 // (seqs * tokens * kv * group * dim), 120000)
    hi = _log(rng, tokens + 1, max(tokens + 2, top))
    lo = rng.randint(tokens, hi)
    window = rng.choice((0, 0, 0, _log(rng, 1, 4096)))
    return dict(op="attend", seqs=seqs, tokens=tokens, q_heads=kv * group, kv_heads=kv, dim=dim,
                page=page, ctx_lo=lo, ctx_hi=hi, window=window, empty=rng.random() < 0.25,
                lens=rng.randint(1, 1 << 30))


# ------------------------------------------------- shapes that follow a case

def _lengths(case):
    """Cached tokens of each sequence, the step's own tokens among them."""
    r = random.Random(case["lens"])
    out = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["seqs"])]
    out[-1] = case["ctx_hi"]
    return out


def _row_positions(case):
    """Position of each query row (-1: an idle row), sequence by sequence."""
    t = case["tokens"]
    rows = [[n - t + j for j in range(t)] for n in _lengths(case)]
    if case["empty"]:
        if case["seqs"] > 1:
            rows[0] = [-1] * t          # an idle slot
        if t > 1:
            rows[-1][-1] = -1           # a sequence with one draft fewer
    return rows


def _visible(case, p):
    """Positions [lo, hi) that a row at position p attends to."""
    if p < 0:
        return 0, 0
    w = case["window"]
    return (max(0, p + 1 - w) if w else 0), p + 1


def _append_rows(case):
    """(sequence, first position, rows) of each sequence's run of new tokens."""
    n, s = case["rows"], case["seqs"]
    r = random.Random(n * 1000003 + s)
    counts = [n // s + (1 if i < n % s else 0) for i in range(s)]
    return [(i, r.randint(0, max(0, case["top_pos"] - c)), c) for i, c in enumerate(counts)]


def work(case):
    d = case["dim"]
    if case["op"] == "rotary":
        n = case["rows"] * case["heads"] * d
        return {"bytes": 8 * n + 4 * case["rows"] + 4 * case["rot"],
                "flops": 3 * case["rows"] * case["heads"] * case["rot"]}
    kv = case["kv_heads"]
    held = 2 * kv * (d // 2 + d // 32)  # bytes of one position's keys and values
    if case["op"] == "append":
        n, q = case["rows"], case["q_heads"]
        # rows in, rotated queries out, the cache written, and what it then
        # holds for these rows read back as values
        return {"bytes": n * (4 * d * (q + 2 * kv) + 4 * d * q + 8 + 2 * held + 8 * d * kv),
                "flops": n * (3 * case["rot"] * (q + kv) + 4 * d * kv)}
    byts = flops = 0
    for rows in _row_positions(case):
        spans = [_visible(case, p) for p in rows if p >= 0]
        if spans:
            byts += held * (max(b for _, b in spans) - min(a for a, _ in spans))
        flops += sum(4 * case["q_heads"] * d * (b - a) for a, b in spans)
    n = case["seqs"] * case["tokens"]
    return {"bytes": byts + n * (8 * case["q_heads"] * d + 8), "flops": flops}


# -------------------------------------------------------------- frequencies

SCALE_FACTOR = 4.0
TRAINED = 8192


def _frequencies(case):
    """(inverse frequencies in 64 bits, amplitude) of a case's rotary plan."""
    rot, base, kind, f = case["rot"], case["base"], case["scaling"], SCALE_FACTOR
    i = np.arange(rot // 2, dtype=np.float64)
    if kind == "ntk" and rot > 2:
        base = base * f ** (rot / (rot - 2))
    w = base ** (-2.0 * i / rot)
    if kind == "linear":
        return w / f, 1.0
    if kind == "bands":      # long wavelengths divided, short ones kept, a ramp between
        ramp = (TRAINED * w / (2 * math.pi) - 1.0) / (4.0 - 1.0)
        ramp = np.clip(ramp, 0.0, 1.0)
        return (1 - ramp) * w / f + ramp * w, 1.0
    if kind == "yarn":       # the same by turns over the trained length, 1 .. 32
        ramp = np.clip((TRAINED * w / (2 * math.pi) - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return (1 - ramp) * w / f + ramp * w, 0.1 * math.log(f) + 1.0
    return w, 1.0


def _own_plan(case):
    import quantized_weight_streaming_q8_amd as q8
    return q8.rotary_plan(case["rot"], base=case["base"], interleaved=case["interleaved"],
                          scaling=case["scaling"], factor=SCALE_FACTOR, original_context=TRAINED)


# ------------------------------------------------------------------ the cache

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pow2(e):
    """2^e in fp32 for integers e in -126..128 (128: infinity), by its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x):
    """fp32 [..., d] -> (codes uint8 [..., d/2], two a byte, the even value
    low; scale bytes uint8 [..., d/32])."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    a = b.abs().amax(-1, keepdim=True)
    bad = ~(a < math.inf)
    m, e = torch.frexp(a.masked_fill(bad, 1.0))
    e = (e - 3 + (8 * m > 7)).clamp(-125, 125)
    y = (b * _pow2(-e)).abs()                # exact where it decides a code
    c = ((y > .25).to(torch.uint8) + (y >= .75) + (y > 1.25) + (y >= 1.75) + (y > 2.5)
         + (y >= 3.5) + (y > 5)).to(torch.uint8)
    c = torch.where(torch.signbit(b), c + 8, c).masked_fill(bad, 0).to(torch.uint8)
    c = c.reshape(*x.shape[:-1], -1, 2)
    s = (e + 127).masked_fill(bad, 255).to(torch.uint8).squeeze(-1)
    return c[..., 0] | (c[..., 1] << 4), s


def _decode(codes, scales):
    """The fp32 values that codes and scale bytes stand for."""
    lut = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    v = lut[nib].reshape(*scales.shape, 32)
    s = _pow2(scales.int() - 127).masked_fill(scales == 255, math.nan)
    return (v * s.unsqueeze(-1)).flatten(-2)


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 16 + salt)
    return g


def _heads(g, n, kv, d):
    """Keys or values as projections give them: every channel with its own
    spread and offset, a few of them large."""
    spread = torch.exp(0.4 * torch.randn(kv, d, generator=g, device="cuda"))
    spread[:, torch.randint(0, d, (2,), generator=g, device="cuda")] *= 6
    offset = 0.5 * torch.randn(kv, d, generator=g, device="cuda")
    x = torch.randn(n, kv, d, generator=g, device="cuda")
    return x.mul_(spread).add_(offset)


def _tables(case, lengths, g):
    """A block table whose pages lie in the pool in no order (device tensor,
    pages in the pool)."""
    most = max(-(-n // case["page"]) for n in lengths)
    pool = len(lengths) * most + 3
    perm = torch.randperm(pool, generator=g, device="cuda").int()
    return perm[:len(lengths) * most].reshape(len(lengths), most).contiguous(), pool


# ------------------------------------------------------------------- prepare

def prepare(case, seed):
    op = case["op"]
    if op == "rotary":
        return _prepare_rotary(case, seed)
    return _prepare_append(case, seed) if op == "append" else _prepare_attend(case, seed)


def _prepare_rotary(case, seed):
    g = _gen(seed, 1)
    st = dict(case=case)
    st["x"] = torch.randn(case["rows"], case["stride"], generator=g, device="cuda")
    st["pos"] = torch.randint(0, case["top_pos"], (case["rows"],), generator=g, device="cuda").int()
    st["y"] = torch.empty(case["rows"], case["heads"] * case["dim"], device="cuda")
    f, st["amplitude"] = _frequencies(case)
    st["freq"] = torch.from_numpy(f).cuda()
    if own:
        st["plan"] = _own_plan(case)
    return st


def _prepare_append(case, seed):
    g = _gen(seed, 2)
    n, q, kv, d = case["rows"], case["q_heads"], case["kv_heads"], case["dim"]
    st = dict(case=case)
    runs = _append_rows(case)
    st["qkv"] = torch.cat([torch.randn(n, q * d, generator=g, device="cuda"),
                           _heads(g, n, kv, d).flatten(1), _heads(g, n, kv, d).flatten(1)], 1)
    order = torch.randperm(n, generator=g, device="cuda")  # rows come in any order
    seq = torch.tensor([s for s, _, c in runs for _ in range(c)], dtype=torch.int32)
    pos = torch.tensor([p + j for _, p, c in runs for j in range(c)], dtype=torch.int32)
    st["seq"], st["pos"] = seq.cuda()[order], pos.cuda()[order]
    st["table"], st["pool"] = _tables(case, [case["top_pos"]] * case["seqs"], g)
    st["q"] = torch.empty(n, q * d, device="cuda")
    st["k"], st["v"] = (torch.empty(n, kv * d, device="cuda") for _ in range(2))
    f, st["amplitude"] = _frequencies(case)
    st["freq"] = torch.from_numpy(f).cuda()
    if own:
        import quantized_weight_streaming_q8_amd as q8
        st["plan"] = _own_plan(case)
        st["cache"] = q8.KV4Cache(st["pool"], case["page"], kv, d, st["table"])
    else:
        st["pages"] = [(torch.zeros(st["pool"], case["page"], kv, d // 2, dtype=torch.uint8, device="cuda"),
                        torch.zeros(st["pool"], case["page"], kv, d // 32, dtype=torch.uint8, device="cuda"))
                       for _ in range(2)]
    return st


PIECE = 16384  # positions made at a time


def _cached(case, g, length):
    """(keys, values) of one sequence, fp32, piece by piece."""
    for a in range(0, length, PIECE):
        n = min(PIECE, length - a)
        yield (a, n, _heads(g, n, case["kv_heads"], case["dim"]),
               _heads(g, n, case["kv_heads"], case["dim"]))


def _prepare_attend(case, seed):
    g = _gen(seed, 3)
    kv, d, page = case["kv_heads"], case["dim"], case["page"]
    lengths = _lengths(case)
    st = dict(case=case, lengths=lengths, scale=d ** -0.5)
    n = case["seqs"] * case["tokens"]
    st["q"] = torch.randn(n, case["q_heads"] * d, generator=g, device="cuda")
    st["o"] = torch.empty_like(st["q"])
    st["table"], st["pool"] = _tables(case, lengths, g)
    st["seq"] = torch.arange(case["seqs"], device="cuda").int().repeat_interleave(case["tokens"])
    st["pos"] = torch.tensor(_row_positions(case), dtype=torch.int32).flatten().cuda()
    if own:
        import quantized_weight_streaming_q8_amd as q8
        st["cache"] = q8.KV4Cache(st["pool"], page, kv, d, st["table"])
        st["workspace"] = q8.kv4_attend_workspace(st["cache"], case["seqs"], case["tokens"],
                                                  case["q_heads"])
    else:
        st["pages"] = [(torch.zeros(st["pool"], page, kv, d // 2, dtype=torch.uint8, device="cuda"),
                        torch.zeros(st["pool"], page, kv, d // 32, dtype=torch.uint8, device="cuda"))
                       for _ in range(2)]
    for s, length in enumerate(lengths):
        for a, m, k, v in _cached(case, g, length):
            pos = torch.arange(a, a + m, device="cuda").int()
            seq = torch.full_like(pos, s)
            if own:
                rows = torch.cat([k.flatten(1), v.flatten(1)], 1)
                q8.q8_kv4_append(st["cache"], rows, m, 2 * kv * d, seq, pos)
            else:
                _scatter(st, seq, pos, k, v)
    return st


# ----------------------------------------------------------------- plain form

def _rotate(x, pos, freq, amplitude, rot, interleaved):
    """x [rows, heads, dim] fp32, rotated by each row's position; 64 bits
    inside, rounded once."""
    t = pos.double()[:, None, None] * freq
    c, s = torch.cos(t) * amplitude, torch.sin(t) * amplitude
    h = x[..., :rot].double()
    y = x.clone()
    if interleaved:
        a, b = h[..., 0::2], h[..., 1::2]
        y[..., 0:rot:2] = (a * c - b * s).float()
        y[..., 1:rot:2] = (a * s + b * c).float()
    else:
        a, b = h[..., :rot // 2], h[..., rot // 2:]
        y[..., :rot // 2] = (a * c - b * s).float()
        y[..., rot // 2:rot] = (a * s + b * c).float()
    return y


def _place(st, seq, pos):
    page = st["case"]["page"]
    return st["table"][seq.long(), (pos // page).long()].long(), (pos % page).long()


def _scatter(st, seq, pos, k, v):
    where = _place(st, seq, pos)
    for (codes, scales), x in zip(st["pages"], (k, v)):
        c, s = _encode(x)
        codes[where] = c
        scales[where] = s


def _plain_rotary(st):
    c = st["case"]
    x = st["x"][:, :c["heads"] * c["dim"]].reshape(c["rows"], c["heads"], c["dim"])
    return _rotate(x, st["pos"], st["freq"], st["amplitude"], c["rot"], c["interleaved"]).flatten(1)


def _plain_append(st):
    c = st["case"]
    q, kv, d = c["q_heads"], c["kv_heads"], c["dim"]
    x = st["qkv"].reshape(c["rows"], q + 2 * kv, d)
    turned = _rotate(x[:, :q + kv], st["pos"], st["freq"], st["amplitude"], c["rot"], c["interleaved"])
    _scatter(st, st["seq"], st["pos"], turned[:, q:], x[:, q + kv:])
    where = _place(st, st["seq"], st["pos"])
    held = [_decode(codes[where], scales[where]).flatten(1) for codes, scales in st["pages"]]
    return [turned[:, :q].flatten(1), held[0], held[1]]


def _plain_attend(st):
    c = st["case"]
    t, kv, d, page = c["tokens"], c["kv_heads"], c["dim"], c["page"]
    group = c["q_heads"] // kv
    positions = _row_positions(c)
    out = []
    for s, length in enumerate(st["lengths"]):
        live = [p for p in positions[s] if p >= 0]
        q = st["q"][s * t:(s + 1) * t].reshape(t, kv, group, d)
        if not live:
            out.append(torch.zeros_like(q).reshape(t, -1))
            continue
        first = min(_visible(c, p)[0] for p in live) // page * page
        last = max(live) + 1
        pages = st["table"][s, first // page:-(-last // page)].long()
        k, v = (_decode(codes[pages], scales[pages]).reshape(-1, kv, d)[:last - first]
                .transpose(0, 1).contiguous() for codes, scales in st["pages"])
        rows = q.permute(1, 0, 2, 3).reshape(kv, t * group, d)
        scores = torch.matmul(rows, k.transpose(1, 2).contiguous()) * st["scale"]
        at = torch.arange(first, last, device="cuda")
        p = st["pos"][s * t:(s + 1) * t, None]
        seen = (at <= p) & (at > p - c["window"] if c["window"] else at >= 0)
        seen = seen.repeat_interleave(group, 0)
        scores = scores.masked_fill(~seen, -math.inf)
        top = scores.amax(-1, keepdim=True)
        e = torch.exp(scores - top.masked_fill(top == -math.inf, 0.0))
        o = torch.matmul(e, v) / e.sum(-1, keepdim=True)
        o = o.masked_fill(~seen.any(-1, keepdim=True), 0.0)
        out.append(o.reshape(kv, t, group, d).permute(1, 0, 2, 3).reshape(t, -1))
    return torch.cat(out)


# ------------------------------------------------------------------------ run

def run(state):
    c = state["case"]
    if not own:
        return {"rotary": _plain_rotary, "append": _plain_append, "attend": _plain_attend}[c["op"]](state)
    import quantized_weight_streaming_q8_amd as q8
    if c["op"] == "rotary":
        q8.q8_rotary(state["x"], state["y"], c["rows"], c["stride"], state["pos"], c["heads"],
                     c["dim"], state["plan"])
        return state["y"]
    if c["op"] == "append":
        n, width = c["rows"], (c["q_heads"] + 2 * c["kv_heads"]) * c["dim"]
        q8.q8_kv4_append(state["cache"], state["qkv"], n, width, state["seq"], state["pos"],
                         rotary=state["plan"], n_q_heads=c["q_heads"], Q=state["q"])
        q8.q8_kv4_read(state["cache"], state["seq"], state["pos"], n, state["k"], state["v"])
        return [state["q"], state["k"], state["v"]]
    q8.q8_kv4_attend(state["cache"], state["q"], c["seqs"], c["tokens"], c["q_heads"],
                     state["seq"], state["pos"], state["o"], state["workspace"],
                     scale=state["scale"], window=c["window"])
    return state["o"]


# ---------------------------------------------------------------------- exact

def _turn64(x, pos, case):
    """The rotation as products with exp(i theta), 64 bits."""
    f, amp = _frequencies(case)
    rot = case["rot"]
    ang = torch.outer(pos.double(), torch.from_numpy(f).to(pos.device))[:, None, :]
    z = x[..., :rot].double()
    z = (z.unflatten(-1, (rot // 2, 2)) if case["interleaved"]
         else z.unflatten(-1, (2, rot // 2)).transpose(-1, -2)).contiguous()
    z = torch.view_as_complex(z) * torch.polar(torch.full_like(ang, amp), ang)
    z = torch.view_as_real(z)
    z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, x[..., rot:].double()], -1)


def _hold64(x):
    """What a 4-bit block of the fp32 values x holds, in 64 bits: the nearest
    of a block's 8 magnitudes by distance, even index on a tie."""
    b = x.double().unflatten(-1, (-1, 32))
    a = b.abs().amax(-1, keepdim=True)
    # floor(log2 a) is the exponent field of a
    e = ((a.view(torch.int64) >> 52) & 2047) - 1023 - 2
    unit = ((e + 1023) << 52).view(torch.float64)
    e = torch.where(a > 7 * unit, e + 1, e).clamp(-125, 125)
    unit = ((e + 1023) << 52).view(torch.float64)
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    y = (b.abs() / unit).clamp_max(6.0)
    hi = torch.searchsorted(grid, y.contiguous()).clamp(1, 7)
    lo = hi - 1
    up, down = grid[hi] - y, y - grid[lo]
    pick = torch.where(up < down, hi, torch.where(up > down, lo, torch.where(hi % 2 == 0, hi, lo)))
    return (torch.copysign(grid[pick], b) * unit).flatten(-2)


def exact(case, seed):
    op = case["op"]
    if op == "rotary":
        g = _gen(seed, 1)
        x = torch.randn(case["rows"], case["stride"], generator=g, device="cuda")
        pos = torch.randint(0, case["top_pos"], (case["rows"],), generator=g, device="cuda")
        h, d = case["heads"], case["dim"]
        return _turn64(x[:, :h * d].unflatten(1, (h, d)), pos, case).flatten(1)
    if op == "append":
        st = _prepare_inputs_append(case, seed)
        q, kv, d = case["q_heads"], case["kv_heads"], case["dim"]
        x = st["qkv"].unflatten(1, (q + 2 * kv, d))
        turned = _turn64(x[:, :q + kv], st["pos"], case)
        return [turned[:, :q].flatten(1), _hold64(turned[:, q:].float()).flatten(1),
                _hold64(x[:, q + kv:]).flatten(1)]
    g = _gen(seed, 3)
    lengths, rows = _lengths(case), _row_positions(case)
    t, kv, d = case["tokens"], case["kv_heads"], case["dim"]
    group = case["q_heads"] // kv
    q = torch.randn(case["seqs"] * t, case["q_heads"] * d, generator=g, device="cuda")
    _tables(case, lengths, g)
    q = q.double().unflatten(1, (kv, group, d))
    out = torch.zeros_like(q)
    for s, length in enumerate(lengths):
        parts = [(_hold64(k), _hold64(v)) for _, _, k, v in _cached(case, g, length)]
        k = torch.cat([p[0] for p in parts]) if len(parts) > 1 else parts[0][0]
        v = torch.cat([p[1] for p in parts]) if len(parts) > 1 else parts[0][1]
        for j, p in enumerate(rows[s]):
            a, b = _visible(case, p)
            if a == b:
                continue
            for h in range(kv):
                w = torch.softmax(k[a:b, h] @ q[s * t + j, h].T * d ** -0.5, 0)
                out[s * t + j, h] = w.T @ v[a:b, h]
    return out.flatten(1)


def _prepare_inputs_append(case, seed):
    """The rows and positions of an append case."""
    global own
    kept, own = own, False
    try:
        return _prepare_append(case, seed)
    finally:
        own = kept
