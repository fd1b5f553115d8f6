"""The serving operators around the paged 4-bit / 2-bit cache, as cases that can be timed and compared:
rotary tables, per-head norm with rotation, the append of new tokens, the read-back of tokens and the
attention of a chunk of new tokens.

`own = False` computes each operator from elementary torch operations in 32 bits (angles in 64);
`own = True` makes the calls a server makes of this package."""
import math

import torch

own = False

D = 128          # head dimension and tokens per group of the paged format
CAP = 128        # rows of the raw window
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # the table a server fills when it starts, short context
        dict(name="table 4k", op="table", n_pos=4096, rot=128, scaling="plain", base=10000.0),
        # the same for a context of 128k, frequencies scaled by wavelength bands
        dict(name="table 128k bands", op="table", n_pos=131072, rot=128, scaling="bands", base=500000.0),
        # q and k heads of one decode step over 64 sequences, norm and half-layout rotation
        dict(name="norm_rope decode 64", op="norm_rope", tokens=64, heads=32, kv_heads=8, head_dim=128, rot=128, inter=False, norm=True, dtype="bf16", n_pos=32768),
        # q and k heads of a prompt of 8191 tokens; interleaved pairs on half of the head
        dict(name="norm_rope prompt 8191", op="norm_rope", tokens=8191, heads=32, kv_heads=8, head_dim=128, rot=64, inter=True, norm=True, dtype="bf16", n_pos=32768),
        # one new token for each of 64 sequences, an eighth of their windows filling up
        dict(name="append step 64", op="append", seqs=64, kv_heads=8, n=1, ctx=4096, ragged=True, fresh=False, n_sink=1, dtype="bf16", rot=128, inter=False),
        # a batch of prompts of 4k tokens and less, some empty, written from the first token on
        dict(name="append prompts", op="append", seqs=13, kv_heads=8, n=4096, ctx=0, ragged=True, fresh=True, n_sink=1, dtype="bf16", rot=128, inter=False),
        # the last tokens of 8 sequences read back
        dict(name="read tails", op="read", seqs=8, kv_heads=8, n=300, ctx=4096, ragged=True, n_sink=1, dtype="bf16", wht=False),
        # whole prefixes of 8 sequences read back, to be handed on
        dict(name="read prefixes", op="read", seqs=8, kv_heads=8, n=16384, ctx=16384, ragged=True, n_sink=1, dtype="bf16", wht=False),
        # one new token of one young sequence
        dict(name="attention short", op="attention", seqs=1, kv_heads=8, group=4, n=1, ctx=100, ragged=False, n_sink=1, causal=True, dtype="bf16", wht=False),
        # drafts of 4 tokens checked against contexts of 32k and less
        dict(name="attention drafts 32k", op="attention", seqs=8, kv_heads=8, group=4, n=4, ctx=32768, ragged=True, n_sink=1, causal=True, dtype="bf16", wht=False),
        # chunks of prompts of many lengths in one batch, one query head per KV head
        dict(name="attention chunks", op="attention", seqs=13, kv_heads=32, group=1, n=509, ctx=4096, ragged=True, n_sink=0, causal=True, dtype="bf16", wht=False),
        # one chunk of 2048 tokens of a long prompt
        dict(name="attention prompt 16k", op="attention", seqs=1, kv_heads=8, group=4, n=2048, ctx=18432, ragged=False, n_sink=1, causal=True, dtype="bf16", wht=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["table", "norm_rope", "append", "read", "attention", "attention"])
    if op == "table":
        return dict(op=op, n_pos=spread(1, 131072), rot=rng.choice([32, 64, 128]), scaling=rng.choice(["plain", "linear", "bands", "ramp"]), base=rng.choice([10000.0, 500000.0]))
    if op == "norm_rope":
        d = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 8])
        return dict(op=op, tokens=spread(1, 8192 * 128 // d * 8 // (8 + kv)), heads=kv * rng.choice([1, 3, 4]), kv_heads=kv, head_dim=d, rot=rng.choice([32, d // 2, d]), inter=rng.random() < 0.5, norm=rng.random() < 0.7, dtype=rng.choice(["bf16", "fp16", "fp32"]), n_pos=32768)
    n_sink, dtype = rng.choice([0, 1, 4]), rng.choice(["bf16", "fp16"])
    seqs = spread(1, 32)
    if op == "append":
        kv, fresh = rng.choice([2, 8]), rng.random() < 0.5
        return dict(op=op, seqs=seqs, kv_heads=kv, n=spread(1, 32768 // seqs), ctx=0 if fresh else spread(1, 8192), ragged=rng.random() < 0.7, fresh=fresh, n_sink=n_sink, dtype=dtype, rot=rng.choice([64, 128]), inter=rng.random() < 0.5)
    if op == "read":
        ctx = spread(1, 65536 // seqs)
        return dict(op=op, seqs=seqs, kv_heads=rng.choice([2, 8]), n=spread(1, ctx), ctx=ctx, ragged=rng.random() < 0.7, n_sink=n_sink, dtype=dtype, wht=rng.random() < 0.3)
    group = rng.choice([1, 2, 3, 4])
    n = spread(1, 1024)
    ctx = max(n, spread(1, 32768))
    seqs = max(1, min(seqs, (1 << 25) // (n * ctx), (1 << 18) // ctx))
    return dict(op=op, seqs=seqs, kv_heads=rng.choice([2, 8]), group=group, n=n, ctx=ctx, ragged=rng.random() < 0.7, n_sink=n_sink, causal=rng.random() < 0.8, dtype="bf16", wht=rng.random() < 0.3)


# ---------------------------------------------------------------------------------------------
# lengths: from the case alone
# ---------------------------------------------------------------------------------------------
def new_counts(c):
    """New (or read) tokens of each sequence; in a ragged batch from n downwards, one in six empty."""
    if not c["ragged"]:
        return [c["n"]] * c["seqs"]
    got = [max(1, c["n"] - (c["n"] * ((5 * s) % 8)) // 9) for s in range(c["seqs"])]
    return [0 if s % 6 == 5 and c["n"] > 1 else x for s, x in enumerate(got)]


def held_counts(c):
    """Tokens each sequence holds: before an append, at a read, after the chunk at an attention."""
    got = [c["ctx"]] * c["seqs"] if not c["ragged"] else [c["ctx"] - c["ctx"] * (s % 8) // 9 for s in range(c["seqs"])]
    if c["op"] == "append":
        # without a prompt before them, windows in every state of filling, some full but for one row
        return got if c["fresh"] else [c["n_sink"] + (x // CAP) * CAP + (CAP - 1 if s % 8 == 3 else (37 * s + 11) % CAP) for s, x in enumerate(got)]
    return [max(x, m) for x, m in zip(got, new_counts(c))]


def split(n_sink, held):
    """(packed, raw) tokens of a sequence of `held` tokens; raw < 0 while the sink still fills."""
    rest = held - n_sink
    return (0, rest) if rest <= 0 else (rest - rest % CAP, rest % CAP)


def frequencies(c):
    """Rotary frequencies in 64 bits, one for each pair."""
    half = c["rot"] // 2
    w = c.get("base", 10000.0) ** (-torch.arange(half, dtype=torch.float64) / half)
    scaling, factor, original, low, high = c.get("scaling", "plain"), 8.0, 8192.0, 1.0, 4.0
    if scaling == "linear":
        return w / factor
    if scaling == "bands":      # by turns within the original context
        t = ((original * w / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        return (1 - t) * w / factor + t * w
    if scaling == "ramp":       # by index, between those that turn `low` and `high` times
        a, b = (c["rot"] * math.log(original / (x * 2 * math.pi)) / (2 * math.log(c["base"])) for x in (32.0, 1.0))
        a, b = max(math.floor(a), 0), min(math.ceil(b), c["rot"] - 1)
        t = ((torch.arange(half, dtype=torch.float64) - a) / max(b - a, 0.001)).clamp(0, 1)
        return (1 - t) * w + t * w / factor
    return w


def amplitude(c):
    return 0.1 * math.log(8.0) + 1.0 if c.get("scaling") == "ramp" else 1.0


def make_table(c, n_pos, device):
    a = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * frequencies(c).to(device)
    return (amplitude(c) * torch.cat([a.cos(), a.sin()], 1)).float()


# ---------------------------------------------------------------------------------------------
# the packed format in elementary operations
# ---------------------------------------------------------------------------------------------
def fp16_toward(x, up):
    """fp32 -> the nearest fp16 not below (up) or not above x."""
    h = x.half()
    f, bits = h.float(), h.view(torch.int16).to(torch.int32)
    away = torch.where(f == 0, torch.full_like(bits, 1 if up else -32767), bits + torch.where((f > 0) == up, 1, -1))
    return torch.where(f < x if up else f > x, away, bits).to(torch.int16).view(torch.float16)


def parameters(lo, hi, steps):
    """Scale and zero-point in fp16 of values in [lo, hi] coded in 0 .. steps."""
    z = fp16_toward(lo, False)
    s = fp16_toward((hi - z.float()) / torch.full_like(hi, steps), True)
    return torch.where(s == 0, torch.ones_like(s), s), z


def pack_keys(x):
    """[..., 128 tokens, D] fp32 -> codes [..., 128, 64] bytes, scale and zero [..., D]."""
    s, z = parameters(x.amin(-2), x.amax(-2), 15.0)
    q = ((x - z.float()[..., None, :]) / s.float()[..., None, :]).round().clamp(0, 15).to(torch.uint8)
    return q[..., 0::2] | q[..., 1::2] << 4, s, z


def pack_values(x):
    """[..., 128 tokens, D] fp32 -> codes [..., 64 pairs, 64] bytes, scale and zero [..., 128]."""
    s, z = parameters(x.amin(-1), x.amax(-1), 3.0)
    q = ((x - z.float()[..., None]) / s.float()[..., None]).round().clamp(0, 3).to(torch.uint8)
    q = q[..., 0::4] | q[..., 1::4] << 2 | q[..., 2::4] << 4 | q[..., 3::4] << 6     # [..., 128, 32]
    q = q.unflatten(-1, (16, 2)).unflatten(-3, (64, 2)).transpose(-3, -2)            # [..., 64, 16, 2 tokens, 2]
    return q.flatten(-3), s, z


def unpack_keys(codes, s, z):
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return q.float() * s.float()[..., None, :] + z.float()[..., None, :]


def unpack_values(codes, s, z):
    b = codes.unflatten(-1, (16, 2, 2)).transpose(-3, -2)                            # [..., 64, 2 tokens, 16, 2]
    q = torch.stack([b & 3, b >> 2 & 3, b >> 4 & 3, b >> 6], -1).flatten(-3).flatten(-3, -2)
    return q.float() * s.float()[..., None] + z.float()[..., None]


def hadamard(dtype, device):
    i = torch.arange(D, device=device)
    bits = (i[:, None] & i)[..., None] >> torch.arange(7, device=device) & 1
    return (1 - 2 * (bits.sum(-1) & 1)).to(dtype) / math.sqrt(D)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def values(shape, dtype, gen, channels=False):
    """Normal values; keys have a few channels ten times as large."""
    x = torch.randn(shape, device=gen.device, generator=gen)
    if channels:
        x[..., torch.randperm(shape[-1], generator=gen, device=gen.device)[:3]] *= 10
    return x.to(dtype)


def ints(x, device):
    return torch.tensor(x, dtype=torch.int32, device=device)


def starts(counts):
    return [sum(counts[:i]) for i in range(len(counts) + 1)]


def prepare(case, seed):
    c = dict(case)
    device = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device).manual_seed(seed)
    st = {"case": c, "device": device}
    if c["op"] == "table":
        # the first position is the only input; a server may fill a table from any position on
        st["pos0"] = seed % 1000
        return st
    dt = DTYPES[c["dtype"]]
    if c["op"] == "norm_rope":
        hq, hk, d, t = c["heads"], c["kv_heads"], c["head_dim"], c["tokens"]
        qkv = values((t, hq + 2 * hk, d), dt, gen)      # the projection's output: q, k and v heads side by side
        st.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], table=make_table(c, c["n_pos"], device),
                  positions=torch.randint(0, c["n_pos"], (t,), device=device, generator=gen, dtype=torch.int32))
        st["wq"], st["wk"] = ((1 + 0.1 * torch.randn(2, d, device=device, generator=gen)).to(dt).unbind() if c["norm"] else (None, None))
        return st

    seqs, hk, ns = c["seqs"], c["kv_heads"], c["n_sink"]
    counts, held = new_counts(c), held_counts(c)
    tq, tr = (list(x) for x in zip(*(split(ns, h) for h in held)))
    after = [h + n for h, n in zip(held, counts)] if c["op"] == "append" else held
    columns = max(1, max(split(ns, a)[0] for a in after) // D)
    used = [split(ns, a)[0] // D for a in after]
    blocks = max(1, sum(used))
    order = torch.randperm(blocks, device=device, generator=gen).to(torch.int32)     # blocks in shuffled order
    table = torch.full((seqs, columns), -1, dtype=torch.int32, device=device)
    at = ints(starts(used), device)
    col = torch.arange(columns, device=device, dtype=torch.int32)
    mine = col < (at[1:] - at[:-1])[:, None]
    table[mine] = order[(at[:-1, None] + col)[mine].long()]
    if c["op"] == "append":
        kc = torch.zeros(blocks, hk, D, D // 2, dtype=torch.uint8, device=device)
        vc = torch.zeros(blocks, hk, D // 2, D // 2, dtype=torch.uint8, device=device)
        meta = [torch.zeros(blocks, hk, D, dtype=torch.float16, device=device) for _ in range(4)]
        kc, ks, kz, vc, vs, vz = kc, meta[0], meta[1], vc, meta[2], meta[3]
    else:
        x = values((blocks, hk, D, D), dt, gen, channels=True).float()
        kc, ks, kz = pack_keys(x @ hadamard(torch.float32, device) if c["wht"] else x)
        del x
        vc, vs, vz = pack_values(values((blocks, hk, D, D), dt, gen).float())
    st.update(k_codes=kc, k_scale=ks, k_zero=kz, v_codes=vc, v_scale=vs, v_zero=vz,
              sink_k=values((seqs, hk, ns, D), dt, gen, True), sink_v=values((seqs, hk, ns, D), dt, gen),
              res_k=values((seqs, hk, CAP, D), dt, gen, True), res_v=values((seqs, hk, CAP, D), dt, gen),
              table=table, t_quant=ints(tq, device), t_res=ints(tr, device), cu=ints(starts(counts), device),
              total=sum(counts), n=max(1, max(counts)), max_tq=max(tq), max_tr=max(0, max(tr)))
    if c["op"] == "append":
        st.update(new_k=values((st["total"], hk, D), dt, gen, True), new_v=values((st["total"], hk, D), dt, gen),
                  rope_table=make_table(c, max(after) + 1, device), t_quant_out=torch.zeros_like(st["t_quant"]), t_res_out=torch.zeros_like(st["t_res"]))
        # what the append may have changed: the window before it and the new tokens
        back = [max(0, r) + n for r, n in zip(tr, counts)]
        st.update(read_cu=ints(starts(back), device), read_total=sum(back), read_n=max(1, max(back)), read_from=ints([h - max(0, r) for h, r in zip(held, tr)], device))
    elif c["op"] == "read":
        # the last tokens of what each sequence holds
        st.update(read_cu=st["cu"], read_total=st["total"], read_n=st["n"], read_from=ints([h - n for h, n in zip(held, counts)], device))
    else:
        st["q"] = values((st["total"], hk * c["group"], D), dt, gen)
    return st


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def rotate(x, table, pos, inter):
    """x [..., heads, d] with positions [...]: pairs of the first table.shape[1] channels turned."""
    r = table.shape[1]
    row = table[pos.long()][..., None, :]
    cos, sin = row[..., :r // 2], row[..., r // 2:]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1), x[..., r:]], -1)


def normed(x, w):
    return x if w is None else x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.float()


def plain_norm_rope(st):
    dt = st["q"].dtype
    return [rotate(normed(x.float(), w), st["table"], st["positions"], st["case"]["inter"]).to(dt) for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"]))]


def gathered(st, name, unpack):
    """Every sequence's tokens in the columns sink, pages, window: [seqs, heads, columns, D] fp32."""
    page = st["table"].clamp(min=0).long()
    x = unpack(*(st[name + p][page] for p in ("_codes", "_scale", "_zero")))         # [seqs, pages, heads, 128, D]
    x = x.transpose(1, 2).flatten(2, 3)
    if name == "k" and st["case"].get("wht"):
        x = x @ hadamard(torch.float32, x.device)
    return torch.cat([st["sink_" + name].float(), x, st["res_" + name].float()], 2)


def columns(st):
    """Position and validity of those columns: [seqs, columns]."""
    ns, dev = st["case"]["n_sink"], st["device"]
    tq, tr = st["t_quant"][:, None], st["t_res"][:, None]
    sink, page, raw = (torch.arange(n, device=dev) for n in (ns, st["table"].shape[1] * D, CAP))
    pos = torch.cat([sink.expand(len(tq), ns), (ns + page).expand(len(tq), -1), ns + tq + raw], 1)
    return pos, torch.cat([sink < ns + tq + tr, page < tq, raw < tr], 1)


def owner(cu, total):
    """Sequence and place in it of each row of a ragged batch."""
    row = torch.arange(total, device=cu.device)
    s = torch.searchsorted(cu[1:], row, right=True)
    return s, row - cu[s]


def plain_read(st, cu, total, first, t_quant, t_res):
    s, i = owner(cu, total)
    ns, pos = st["case"]["n_sink"], (first[s] + i).long()
    packed = pos - ns                                                                # place after the sink
    raw = packed - t_quant[s]
    at = packed.clamp(min=0)
    page = st["table"][s, (at // D).clamp(max=st["table"].shape[1] - 1)].clamp(min=0).long()
    at = at % D
    byte = st["k_codes"][page, :, at]                                                # [tokens, heads, 64]
    k = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).float() * st["k_scale"][page].float() + st["k_zero"][page].float()
    if st["case"].get("wht"):
        k = k @ hadamard(torch.float32, k.device)
    byte = st["v_codes"][page, :, at // 2].unflatten(-1, (16, 2, 2))
    byte = torch.where((at % 2 == 1)[:, None, None, None], byte[..., 1, :], byte[..., 0, :])
    v = torch.stack([byte & 3, byte >> 2 & 3, byte >> 4 & 3, byte >> 6], -1).flatten(-3).float()
    v = v * st["v_scale"][page, :, at].float()[..., None] + st["v_zero"][page, :, at].float()[..., None]
    outs = []
    for name, x in (("k", k), ("v", v)):
        x = torch.where((raw >= 0)[:, None, None], st["res_" + name][s, :, raw.clamp(0, CAP - 1)].float(), x)
        if ns:
            x = torch.where((packed < 0)[:, None, None], st["sink_" + name][s, :, pos.clamp(max=ns - 1)].float(), x)
        outs.append(x.to(st["res_k"].dtype))
    return outs


def plain_attention(st):
    c, q = st["case"], st["q"]
    hk, g, n = c["kv_heads"], c["group"], st["n"]
    k, v = gathered(st, "k", unpack_keys), gathered(st, "v", unpack_values)
    pos, valid = columns(st)
    cu = st["cu"]
    i = torch.arange(n, device=q.device)
    count = (cu[1:] - cu[:-1])[:, None]
    held = (c["n_sink"] + st["t_quant"] + st["t_res"])[:, None]
    limit = held - count + i if c["causal"] else held.expand(-1, n)
    see = valid[:, None] & (pos[:, None] <= limit[..., None])                        # [seqs, n, columns]
    rows = q[(cu[:-1, None] + i).clamp(max=st["total"] - 1).long()].float()          # [seqs, n, heads, D]
    rows = rows.unflatten(2, (hk, g)).permute(0, 2, 3, 1, 4).flatten(2, 3)           # [seqs, hk, g * n, D]
    score = (rows @ k.transpose(-1, -2) / math.sqrt(D)).unflatten(2, (g, n))
    score = score.masked_fill_(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = score.sub_(top).exp_()
    out = p.flatten(2, 3) @ v / p.sum(-1, keepdim=True).flatten(2, 3).clamp(min=1e-30)
    out = out.unflatten(2, (g, n)).permute(0, 3, 1, 2, 4).flatten(2, 3)              # [seqs, n, heads, D]
    s, at = owner(cu, st["total"])
    return out[s, at].to(q.dtype)


def plain_append(st):
    c, cu, tq, tr, table = st["case"], st["cu"], st["t_quant"], st["t_res"], st["table"]
    ns, dev, dt = c["n_sink"], cu.device, st["res_k"].dtype
    n = (cu[1:] - cu[:-1])[:, None]
    i = torch.arange(st["n"], device=dev)
    row = (cu[:-1, None] + i).clamp(max=st["total"] - 1).long()
    pos = (ns + tq + tr)[:, None] + i
    new_k = rotate(st["new_k"][row].float(), st["rope_table"], pos.clamp(max=st["rope_table"].shape[0] - 1), c["inter"]).to(dt)
    new = {"k": new_k, "v": st["new_v"][row]}                                        # [seqs, n, heads, D]
    seq = torch.arange(len(tq), device=dev)[:, None]
    to_sink = torch.minimum(n, (-tr[:, None]).clamp(min=0))
    raw = tr[:, None].clamp(min=0)
    total = raw + n - to_sink                                                        # rows after the sink
    flushed = torch.where(total >= CAP, total // D, 0)
    rooms = (CAP + st["n"] + D - 1) // D * D
    r = torch.arange(rooms, device=dev)
    group = torch.arange(rooms // D, device=dev)
    there = group < flushed
    dest = table[seq, (tq[:, None] // D + group).clamp(max=table.shape[1] - 1)][there].long()
    first = ns + tr[:, None]
    sink = torch.arange(ns, device=dev)
    left = torch.arange(CAP, device=dev)
    for name, pack in (("k", pack_keys), ("v", pack_values)):
        x, old = new[name], st["res_" + name].transpose(1, 2)                        # [seqs, rows, heads, D]
        both = torch.where((r < raw)[..., None, None], old[:, r.clamp(max=CAP - 1)], x[seq, (r - raw + to_sink).clamp(0, st["n"] - 1)])
        codes, s, z = pack(both.unflatten(1, (-1, D)).transpose(2, 3)[there].float())
        st[name + "_codes"][dest], st[name + "_scale"][dest], st[name + "_zero"][dest] = codes, s, z
        keep = left < total - flushed * D
        kept = torch.where(keep[..., None, None], both[seq, (flushed * D + left).clamp(max=rooms - 1)], old)
        st["res_" + name].copy_(kept.transpose(1, 2))
        fills = (sink >= first) & (sink < first + to_sink)
        held = st["sink_" + name].transpose(1, 2)
        st["sink_" + name].copy_(torch.where(fills[..., None, None], x[seq, (sink - first).clamp(0, st["n"] - 1)], held).transpose(1, 2))
    done = flushed[:, 0] * D
    after_q, after_r = (tq + done).int(), torch.where(done > 0, total[:, 0] - done, tr + n[:, 0]).int()
    back = plain_read(st, st["read_cu"], st["read_total"], st["read_from"], after_q, after_r)
    return [*back, after_q, after_r]


def plain_table(st):
    c = st["case"]
    p = torch.arange(c["n_pos"], dtype=torch.float64, device=st["device"]) + st["pos0"]
    a = p[:, None] * frequencies(c).to(st["device"])
    return (amplitude(c) * torch.cat([a.cos(), a.sin()], 1)).float()


# ---------------------------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------------------------
def own_handles(st):
    """What a server makes once for a cache: the format, the cache over its arrays, a workspace."""
    from quantized_decode_attention_quantize_b200 import kvq
    c = st["case"]
    h = {"kvq": kvq}
    if c["op"] == "table":
        kind = {"plain": kvq.ROPE_PLAIN, "linear": kvq.ROPE_LINEAR, "bands": kvq.ROPE_BANDS, "ramp": kvq.ROPE_RAMP}[c["scaling"]]
        low, high = (1.0, 32.0) if c["scaling"] == "ramp" else (1.0, 4.0)
        h["spec"] = kvq.make_rope_spec(c["rot"], base=c["base"], scaling=kind, factor=8.0, original_len=8192.0, low=low, high=high, amplitude=amplitude(c))
    elif c["op"] == "norm_rope":
        h["rope"] = kvq.Rope(st["table"], interleaved=c["inter"])
    else:
        h["fmt"] = kvq.make_format(dict(
            head_dim=D, group_tokens=D, src_dtype=kvq.KVQ_DTYPE[DTYPES[c["dtype"]]], k_scheme=kvq.ASYM, k_bits=4, k_axis=kvq.CHANNEL, k_outliers=0,
            v_scheme=kvq.ASYM, v_bits=2, v_axis=kvq.TOKEN, v_outliers=0, mixed_hi=0, mixed_mid=0, n_sink=c["n_sink"], residual_cap=CAP, rope=0,
            rope_base=10000.0, k_rotate=int(c.get("wht", False))))
        names = ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero", "sink_k", "sink_v", "res_k", "res_v")
        h["cache"] = kvq.PagedCache(h["fmt"], c["kv_heads"], st["k_codes"].shape[0], c["seqs"], st["table"].shape[1], device=st["device"],
                                    arrays=dict({n: st[n] for n in names}, block_table=st["table"]))
        if c["op"] == "append":
            h["rope"] = kvq.Rope(st["rope_table"], interleaved=c["inter"])
        if c["op"] == "attention":
            need = kvq.attention_paged_workspace_bytes(h["fmt"], c["seqs"], c["kv_heads"] * c["group"], c["kv_heads"], st["total"], st["n"], st["max_tq"], st["max_tr"])
            h["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device=st["device"])
    return h


def own_run(st):
    h = st.get("handles")
    if h is None:
        h = st["handles"] = own_handles(st)
    kvq, c = h["kvq"], st["case"]
    if c["op"] == "table":
        return kvq.rope_table(h["spec"], c["n_pos"], pos0=st["pos0"], device=st["device"])
    if c["op"] == "norm_rope":
        return list(kvq.norm_rope(st["q"], st["k"], st["wq"], st["wk"], eps=1e-6, rope=h["rope"], positions=st["positions"]))
    f, cache = h["fmt"], h["cache"]
    if c["op"] == "append":
        kvq.append_paged(f, cache, st["cu"], st["n"], st["t_quant"], st["t_res"], st["new_k"], st["new_v"], st["t_quant_out"], st["t_res_out"], rope=h["rope"])
        k, v = kvq.read_paged(f, cache, st["read_cu"], st["read_n"], st["read_from"], st["t_quant_out"], st["t_res_out"], st["read_total"])
        return [k, v, st["t_quant_out"], st["t_res_out"]]
    if c["op"] == "read":
        return list(kvq.read_paged(f, cache, st["read_cu"], st["read_n"], st["read_from"], st["t_quant"], st["t_res"], st["read_total"]))
    return kvq.attention_paged(f, cache, st["cu"], st["n"], st["t_quant"], st["t_res"], st["max_tq"], st["max_tr"], st["q"], 1.0 / math.sqrt(D),
                               causal=c["causal"], out_dtype=kvq.KVQ_DTYPE[st["q"].dtype], workspace=h["workspace"])


def run(state):
    if own:
        return own_run(state)
    op = state["case"]["op"]
    if op == "read":
        return plain_read(state, state["read_cu"], state["read_total"], state["read_from"], state["t_quant"], state["t_res"])
    return {"table": plain_table, "norm_rope": plain_norm_rope, "append": plain_append, "attention": plain_attention}[op](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c = dict(case)
    if c["op"] == "table":
        return {"bytes": 4.0 * c["n_pos"] * c["rot"], "flops": 0.0}
    size = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "norm_rope":
        rows = c["tokens"] * (c["heads"] + c["kv_heads"])
        return {"bytes": 2.0 * size * rows * c["head_dim"] + c["tokens"] * (4.0 + 4 * c["rot"]), "flops": 0.0}
    counts, held, hk, ns = new_counts(c), held_counts(c), c["kv_heads"], c["n_sink"]
    raw, packed = 2.0 * size * D * hk, (D / 2 + D / 4 + 4 + 4.0) * hk      # bytes of a token: k and v as rows; codes and their share of metadata
    if c["op"] == "append":
        total = 0.0
        for n, h in zip(counts, held):
            (q0, r0), (q1, r1) = split(ns, h), split(ns, h + n)
            flushed, rows = q1 - q0, n - (q1 - q0) + max(0, r0) if q1 > q0 else n   # rows: new tokens that stay raw
            # the new tokens read, the window read when it is packed, what is written, and all of that read back
            total += n * raw + n * 4.0 * c["rot"] + (max(0, r0) * raw if flushed else 0) + flushed * packed + rows * raw
            back = max(0, r0) + n
            total += back * raw + flushed * packed + (back - flushed) * raw
        return {"bytes": max(total, 1.0), "flops": 0.0}
    if c["op"] == "read":
        in_pages = [max(0, min(h, ns + split(ns, h)[0]) - max(h - n, ns)) for n, h in zip(counts, held)]
        return {"bytes": sum(n * raw + p * packed + (n - p) * raw for n, p in zip(counts, in_pages)), "flops": 0.0}
    g = c["group"]
    seen = [n * h - (n * (n - 1) // 2 if c["causal"] else 0) for n, h in zip(counts, held)]
    cache = [split(ns, h)[0] * packed + (h - split(ns, h)[0]) * raw if n else 0.0 for n, h in zip(counts, held)]
    return {"bytes": sum(cache) + 2.0 * size * D * hk * g * sum(counts), "flops": 4.0 * D * hk * g * sum(seen)}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------------------------
def exact_tokens(st, s, which, t_quant, t_res):
    """Sequence s's tokens in order: [heads, tokens, D] fp64."""
    ns = st["case"]["n_sink"]
    raw_sink, raw_rows = st["sink_" + which][s].double(), st["res_" + which][s].double()
    parts = [raw_sink[:, :ns + min(0, t_res)]]
    for j in range(t_quant // D):
        b = int(st["table"][s, j])
        codes = st[which + "_codes"][b]
        scale, zero = st[which + "_scale"][b].double(), st[which + "_zero"][b].double()
        if which == "k":       # channel c in byte c / 2, the even one low
            q = torch.empty(codes.shape[0], D, D, dtype=torch.float64, device=codes.device)
            q[..., 0::2], q[..., 1::2] = (codes % 16).double(), (codes // 16).double()
            x = q * scale[:, None] + zero[:, None]
            parts.append(x @ hadamard(torch.float64, x.device) if st["case"].get("wht") else x)
        else:                  # four bytes: eight channels of the even token, then of the odd one
            q = torch.empty(codes.shape[0], D, D, dtype=torch.float64, device=codes.device)
            for token in range(2):
                for byte in range(2):
                    for k in range(4):
                        q[:, token::2, byte * 4 + k::8] = (codes[:, :, token * 2 + byte::4] // 4 ** k % 4).double()
            parts.append(q * scale[..., None] + zero[..., None])
    parts.append(raw_rows[:, :max(0, t_res)])
    return torch.cat(parts, 1)


def exact_rotate(x, table, pos, inter):
    """x [heads, tokens, d] fp64 by complex numbers."""
    r = table.shape[1]
    turn = torch.complex(table[pos, :r // 2].double(), table[pos, r // 2:].double())
    z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) if inter else torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous())
    z = z * turn
    y = x.clone()
    if inter:
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    else:
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    return y


def exact_coded(x, axis, levels):
    """x [heads, 128, D] fp64 as the values its codes stand for; scale up and zero down to fp16."""
    lo, hi = x.amin(axis, keepdim=True), x.amax(axis, keepdim=True)
    z = fp16_toward(lo.float(), False).double()
    s = fp16_toward(((hi - z) / levels).float(), True).double()
    s = torch.where(s == 0, torch.ones_like(s), s)
    return ((x - z) / s).round().clamp(0, levels) * s + z


def exact(case, seed):
    st = prepare(case, seed)
    c, op = st["case"], st["case"]["op"]
    if op == "table":
        angle = (torch.arange(c["n_pos"], dtype=torch.float64) + st["pos0"])[:, None] * frequencies(c)[None]
        z = torch.polar(torch.full_like(angle, amplitude(c)), angle)
        return torch.cat([z.real, z.imag], 1)
    if op == "norm_rope":
        out = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            x = x.double().transpose(0, 1)
            if w is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()
            out.append(exact_rotate(x, st["table"], st["positions"].long(), c["inter"]).transpose(0, 1).contiguous())
        return out
    ns, counts, held = c["n_sink"], new_counts(c), held_counts(c)
    tq, tr = st["t_quant"].tolist(), st["t_res"].tolist()
    empty = torch.zeros(0, c["kv_heads"], D, dtype=torch.float64, device=st["device"])
    if op == "read":
        return [torch.cat([empty] + [exact_tokens(st, s, w, tq[s], tr[s])[:, held[s] - n:].transpose(0, 1) for s, n in enumerate(counts)]) for w in "kv"]
    if op == "append":
        outs, dt = [], DTYPES[c["dtype"]]
        for w, axis, levels in (("k", 1, 15.0), ("v", 2, 3.0)):
            rows = [empty]
            for s, n in enumerate(counts):
                new = st["new_" + w][sum(counts[:s]):sum(counts[:s + 1])].double().transpose(0, 1)
                if w == "k" and n:
                    at = torch.arange(held[s], held[s] + n, device=st["device"])
                    new = exact_rotate(new, st["rope_table"], at, c["inter"]).to(dt).double()
                x = torch.cat([st["res_" + w][s, :, :max(0, tr[s])].double(), new], 1)
                skip = min(n, max(0, -tr[s]))                     # tokens of the sink stay as they are
                body = x[:, skip:]
                f = body.shape[1] // D if body.shape[1] >= CAP else 0
                packed = [exact_coded(body[:, j * D:(j + 1) * D], axis, levels) for j in range(f)]
                rows.append(torch.cat([x[:, :skip], *packed, body[:, f * D:]], 1).transpose(0, 1))
            outs.append(torch.cat(rows))
        return [*outs, None, None]
    g, outs = c["group"], [torch.zeros(0, c["kv_heads"] * c["group"], D, dtype=torch.float64, device=st["device"])]
    for s, n in enumerate(counts):
        if n == 0:
            continue
        q = st["q"][sum(counts[:s]):sum(counts[:s + 1])].double()
        k, v = exact_tokens(st, s, "k", tq[s], tr[s]), exact_tokens(st, s, "v", tq[s], tr[s])
        heads = []
        for h in range(q.shape[1]):
            a = q[:, h] @ k[h // g].T / math.sqrt(D)
            if c["causal"]:
                a = a + torch.full_like(a, -math.inf).triu(held[s] - n + 1)
            heads.append(torch.softmax(a, -1) @ v[h // g])
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs)
