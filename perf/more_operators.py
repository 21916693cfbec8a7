"""Operators next to the 8-bit cache, as they are measured: a key/value cache held in 4 bits (writing tokens, reading them
back, attention over it), and the norms of queries and keys for each head with the rotation by their positions.

The 4-bit cache is paged like the 8-bit one. A row of a block (a token of a head) has E2M1 codes, two columns to a byte
(the even one in the low half) and rows of a multiple of 16 bytes, and a scale for every 16 columns: 8 bits, 5 of them an
exponent and 3 a fraction, the bits 14 to 7 of an IEEE half. A number is code * scale. New tokens of a sequence are the last
of its `lens` tokens."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # E2M1, then the same with the sign
EPS = 1e-6


def _case(name, op, seqs, len_min, len_max, new_min, new_max, heads=32, kv_heads=8, dim=128, block=64, dtype="bf16",
          causal=True, window=0, rot=0, interleaved=False, norm=False):
    return dict(name=name, op=op, seqs=seqs, len_min=len_min, len_max=len_max, new_min=new_min, new_max=new_max,
                heads=heads, kv_heads=kv_heads, dim=dim, block=block, dtype=dtype, causal=causal, window=window, rot=rot,
                interleaved=interleaved, norm=norm)


def listed():
    return [
        # one decoding step's queries and keys, 32 sequences in service: the smallest rotation, latency counts
        _case("rotate_step", "rotate", 32, 100, 4000, 1, 1, rot=128, norm=True),
        # five prompts admitted at once, the usual rotation
        _case("rotate_prompts", "rotate", 5, 1500, 5000, 1500, 5000, rot=128, norm=True),
        # chunks far into long documents: float16, neighbouring columns turned, part of an odd head size, no norms
        _case("rotate_far", "rotate", 3, 40000, 131072, 200, 900, heads=12, kv_heads=6, dim=80, dtype="fp16", rot=32,
              interleaved=True),
        # one decoding step's keys and values written, and read back as the numbers that later steps will see
        _case("write_step", "write", 32, 100, 4000, 1, 1),
        # five prompts admitted at once: written, and read back for the prompts' own layers
        _case("write_prompts", "write", 5, 1500, 5000, 1500, 5000),
        # one shared prefix read back, for a form that wants 16-bit keys and values
        _case("read_prefix", "read", 1, 777, 777, 777, 777, block=16, dtype="fp16"),
        # long documents read back before they are moved to another store: the largest read
        _case("read_documents", "read", 3, 20000, 65536, 20000, 65536, block=128),
        # one user's next token, short context: the smallest attention, latency counts
        _case("attend_token", "attend", 1, 1023, 1023, 1, 1),
        # one user's next token over a long document: few rows, a long axis
        _case("attend_token_long", "attend", 1, 131072, 131072, 1, 1),
        # next tokens of a full batch of uneven length: what serving does most
        _case("attend_batch", "attend", 64, 300, 8192, 1, 1, block=32),
        # drafted tokens checked in one step, sliding window, float16, 8 query heads to a head, 96 columns
        _case("attend_drafts", "attend", 16, 200, 6000, 2, 5, heads=16, kv_heads=2, dim=96, block=16, dtype="fp16", window=4096),
        # a whole prompt: the largest amount of arithmetic
        _case("attend_prompt", "attend", 1, 8192, 8192, 8192, 8192),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["rotate", "rotate", "write", "read", "attend", "attend", "attend"])
    dtypes = ["bf16", "fp16"] if op == "attend" else ["bf16", "fp16", "fp32"]
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    dim = rng.choice([32, 64, 80, 96, 112, 128, 128])
    c = dict(heads=kv_heads * group, kv_heads=kv_heads, dim=dim, block=rng.choice([16, 32, 48, 64, 128]), dtype=rng.choice(dtypes),
             causal=True, window=0, rot=0, interleaved=False, norm=False)
    if op == "rotate":
        seqs = log(1, 64)
        hi = log(1, max(2, 16384 // seqs))
        lo = log(1, hi)
        past = rng.choice([0, log(1, 131072)])
        c.update(rot=rng.choice([dim, dim, max(16, dim // 32 * 16)]), interleaved=rng.choice([False, False, True]), norm=rng.choice([True, True, False]))
        return dict(c, op=op, seqs=seqs, len_min=lo + past, len_max=hi + past, new_min=lo, new_max=hi)
    if op in ("write", "read"):
        seqs = log(1, 64)
        most = max(2, 16384 // seqs)
        hi = log(2, most)
        lo = log(1, hi)
        past = rng.choice([0, log(1, 3000)]) if op == "write" else 0
        return dict(c, op=op, seqs=seqs, len_min=lo + past, len_max=hi + past, new_min=lo, new_max=hi)
    kind = rng.choice(["token", "drafts", "chunk", "prompt"])
    if kind in ("token", "drafts"):
        seqs = log(1, 64)
        hi = log(16, 8192 if seqs > 4 else 65536)
        lo = log(8, hi)
        new = 1 if kind == "token" else rng.randint(2, 8)
        c.update(window=rng.choice([0, 0, log(64, 4096)]))
        return dict(c, op=op, seqs=seqs, len_min=lo, len_max=hi, new_min=1, new_max=new)
    seqs = log(1, 4)
    if kind == "chunk":
        hi = log(600, 12000)
        return dict(c, op=op, seqs=seqs, len_min=log(600, hi), len_max=hi, new_min=log(9, 100), new_max=log(100, 600))
    hi = log(64, 6000 // seqs)
    c.update(causal=rng.choice([True, True, False]), window=rng.choice([0, 0, log(64, 2000)]))
    return dict(c, op=op, seqs=seqs, len_min=hi, len_max=hi, new_min=hi, new_max=hi)


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], the first the largest, in an order that looks like none."""
    return [hi if i == 0 else lo + int((hi - lo) * ((0.381966 + i * 0.618034) % 1.0)) for i in range(n)]


def _lengths(case):
    n = case["seqs"]
    lens = _spread(case["len_min"], case["len_max"], n)
    if case["len_min"] - case["new_min"] == case["len_max"] - case["new_max"]:
        past = case["len_min"] - case["new_min"]
        return lens, [v - past for v in lens]
    return lens, [min(a, b) for a, b in zip(lens, _spread(case["new_min"], case["new_max"], n))]


def _pairs(case):
    """Query and key pairs that the masks leave, and keys that some query sees, over the sequences."""
    pairs = keys = 0
    for total, new in zip(*_lengths(case)):
        first, w = total - new, case["window"]
        if case["causal"]:
            pairs += sum(min(p + 1, w) for p in range(first, total)) if w else new * first + new * (new + 1) // 2
        else:
            pairs += sum(total - max(0, p - w + 1) for p in range(first, total)) if w else new * total
        keys += total - (max(0, first - w + 1) if w else 0)
    return pairs, keys


def work(case):
    lens, news = _lengths(case)
    tokens, seqs, b, dim = sum(news), case["seqs"], case["block"], case["dim"]
    elt = 4 if case["dtype"] == "fp32" else 2
    row = case["kv_heads"] * dim
    stored = row // 2 + row // 16  # bytes of a token's codes and scales, of K or of V
    blocks = sum(-(-t // b) - (t - n) // b for t, n in zip(lens, news))
    if case["op"] == "rotate":
        both = tokens * (case["heads"] + case["kv_heads"]) * dim
        # a square and its sum, two multiplications by the norm, a turn of two columns: 8 a column
        return {"bytes": 2 * both * elt + 2 * dim * elt * case["norm"] + 8 * case["rot"] // 2 + 8 * seqs, "flops": 8 * both}
    if case["op"] == "read":
        return {"bytes": 2 * tokens * (row * elt + stored) + 4 * (blocks + 2 * seqs), "flops": 2 * tokens * row}
    if case["op"] == "write":  # written once, and read back once
        return {"bytes": 2 * tokens * (2 * row * elt + 2 * stored) + 4 * (blocks + 2 * seqs), "flops": 2 * 3 * tokens * row}
    pairs, keys = _pairs(case)
    q = tokens * case["heads"] * dim * 2
    return {"bytes": 2 * keys * stored + 2 * q + 4 * tokens * case["heads"] + 4 * (keys // b + 2 * seqs),
            "flops": 4 * pairs * case["heads"] * dim}


def _frequencies(case):
    """Radians a position, of each pair of columns that turns."""
    return [500000.0 ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lens, news = _lengths(case)
    block, hkv, dim = case["block"], case["kv_heads"], case["dim"]
    dtype = DTYPES[case["dtype"]]
    per = [-(-t // block) for t in lens]
    width = max(per)
    n_blocks = sum(per) + 3
    # blocks are handed out in no order, as in a pool that has been in use for a while
    order = torch.randperm(n_blocks, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([0] + per, device=dev).cumsum(0)
    at = first[:-1, None] + torch.arange(width, device=dev)[None]
    inside = torch.arange(width, device=dev)[None] < torch.tensor(per, device=dev)[:, None]
    table = torch.where(inside, order[at.clamp(max=n_blocks - 1)], torch.zeros((), dtype=torch.int32, device=dev))
    st = dict(case=case, table=table.contiguous(), total=sum(news), most=max(news),
              cu=torch.tensor([0] + news, device=dev).cumsum(0).to(torch.int32),
              lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    if case["op"] == "rotate":
        # projections as they come: a few channels larger, some tokens louder than the rest; queries and keys are views of one
        # tensor, as a fused projection leaves them
        heads = case["heads"] + 2 * hkv
        loud = torch.exp2(2.0 * torch.randn(st["total"], 1, 1, generator=g, device=dev).clamp(-2, 2))
        chan = torch.exp2(torch.randn(1, heads, dim, generator=g, device=dev))
        qkv = (torch.randn(st["total"], heads, dim, generator=g, device=dev) * loud * chan).to(dtype)
        st["q"], st["k"] = qkv[:, : case["heads"]], qkv[:, case["heads"]: case["heads"] + hkv]
        st["frequencies"] = torch.tensor(_frequencies(case), dtype=torch.float64, device=dev)
        if case["norm"]:
            st["wq"], st["wk"] = ((1.0 + 0.2 * torch.randn(dim, generator=g, device=dev)).to(dtype) for _ in range(2))
        if own:
            import entropy_coding_gb300 as zc
            st["cache"] = zc.KV4Cache.empty(n_blocks, hkv, dim, block, dev)
            st["batch"] = zc.KVBatch(st["table"], st["cu"], st["lens"], st["total"], st["most"])
            st["rotation"] = zc.KVRotation(_frequencies(case), interleaved=case["interleaved"], device=dev)
        return st

    def pool():
        codes = torch.randint(0, 256, (n_blocks, hkv, block, -(-dim // 32) * 16), generator=g, device=dev, dtype=torch.uint8)
        # scales of 2^-5 to 2^-2, as activations around one have them
        return codes, torch.randint(80, 104, (n_blocks, hkv, block, dim // 16), generator=g, device=dev, dtype=torch.uint8)

    st["k"], st["k_scale"] = pool()
    st["v"], st["v_scale"] = pool()
    if case["op"] == "write":
        # activations: unit normal, a few channels larger, some tokens louder than the rest
        loud = torch.exp2(2.0 * torch.randn(st["total"], 1, 1, generator=g, device=dev).clamp(-2, 2))
        chan = torch.exp2(torch.randn(1, hkv, dim, generator=g, device=dev))
        st["new_k"] = (torch.randn(st["total"], hkv, dim, generator=g, device=dev) * loud * chan).to(dtype)
        st["new_v"] = (torch.randn(st["total"], hkv, dim, generator=g, device=dev) * loud).to(dtype)
    if case["op"] == "attend":
        st["q"] = torch.randn(st["total"], case["heads"], dim, generator=g, device=dev).to(dtype)
    if own:
        import entropy_coding_gb300 as zc
        st["cache"] = zc.KV4Cache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        st["batch"] = zc.KVBatch(st["table"], st["cu"], st["lens"], st["total"], st["most"])
    return st


def run(st):
    case = st["case"]
    dtype = DTYPES[case["dtype"]]
    if own:
        import entropy_coding_gb300 as zc
        if case["op"] == "rotate":
            return zc.kv_rotate(st["cache"], st["batch"], st["rotation"], st["q"], st["k"], st.get("wq"), st.get("wk"), eps=EPS)
        if case["op"] == "write":
            zc.kv_write(st["cache"], st["batch"], st["new_k"], st["new_v"])
            return zc.kv_read(st["cache"], st["batch"], dtype=dtype)
        if case["op"] == "read":
            return zc.kv_read(st["cache"], st["batch"], dtype=dtype)
        return zc.kv_attend(st["cache"], st["batch"], st["q"], causal=case["causal"], window=case["window"])
    if case["op"] == "rotate":
        return _rotate(st, st["q"], st.get("wq")), _rotate(st, st["k"], st.get("wk"))
    if case["op"] == "attend":
        return _attend(st)
    if case["op"] == "write":
        _write(st, st["new_k"], st["k"], st["k_scale"])
        _write(st, st["new_v"], st["v"], st["v_scale"])
    return _read(st, st["k"], st["k_scale"]), _read(st, st["v"], st["v_scale"])


def _places(st):
    """Sequence and position of each token of the batch."""
    cu, lens = st["cu"].long(), st["lens"].long()
    new = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(len(lens), device=cu.device), new, output_size=st["total"])
    return seq, torch.arange(st["total"], device=cu.device) - cu[seq] + (lens - new)[seq]


def _rotate(st, x, weight):
    case = st["case"]
    rot = case["rot"]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()
    _, pos = _places(st)
    angle = pos.double()[:, None] * st["frequencies"]  # (32 bits would lose the angles of far positions)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = y.clone()
    if case["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        out[..., : rot // 2], out[..., rot // 2: rot] = a * cos - b * sin, b * cos + a * sin
    return out.to(x.dtype)


def _numbers(codes, scales):
    """The numbers of rows of codes [..., bytes] and scales [..., dim / 16], in 32 bits."""
    values = torch.tensor(CODES + [-c for c in CODES], device=codes.device)
    x = torch.stack([values[(codes & 15).int()], values[(codes >> 4).int()]], -1).flatten(-2)[..., : scales.shape[-1] * 16]
    s = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _write(st, x, codes, scales):
    block, hkv, dim = st["case"]["block"], st["case"]["kv_heads"], st["case"]["dim"]
    seq, pos = _places(st)
    home = st["table"][seq, pos // block].long()               # each token's block
    at = (home[:, None], torch.arange(hkv, device=x.device)[None], (pos % block)[:, None])
    x = x.double().unflatten(-1, (-1, 16))  # (64 bits: numbers next to the border of two codes)
    # a scale is the nearest of those there are to largest / 6, ties to the even one
    steps = (torch.arange(0xE3, device=x.device, dtype=torch.int16) << 7).view(torch.float16).double()
    need = x.abs().amax(-1) / 6.0
    byte = torch.bucketize(need, (steps[:-1] + steps[1:]) / 2)  # borders below the number
    tie = need == ((steps[:-1] + steps[1:]) / 2)[byte.clamp(max=len(steps) - 2)]
    byte = torch.where(tie & (byte % 2 == 1), byte + 1, byte).clamp(1, 0xE2)
    scales[at] = byte.to(torch.uint8)
    q = x / steps[byte][..., None]
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device, dtype=torch.float64)
    a = q.abs()
    c = torch.bucketize(a, borders)
    tie = a == borders[c.clamp(max=6)]
    c = torch.where(tie & (c % 2 == 1), c + 1, c) + 8 * (torch.signbit(q))
    c = c.flatten(-2).to(torch.uint8)
    c = torch.nn.functional.pad(c, (0, 2 * codes.shape[-1] - dim))
    codes[at] = c[..., 0::2] | c[..., 1::2] << 4


def _read(st, codes, scales):
    block, hkv = st["case"]["block"], st["case"]["kv_heads"]
    seq, pos = _places(st)
    home = st["table"][seq, pos // block].long()
    at = (home[:, None], torch.arange(hkv, device=codes.device)[None], (pos % block)[:, None])
    return _numbers(codes[at], scales[at]).to(DTYPES[st["case"]["dtype"]])


def _attend(st):
    case, table = st["case"], st["table"].long()
    hkv, dim, group = case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    cu, lens, most = st["cu"].long(), st["lens"].long(), st["most"]
    seqs, keys = len(lens), table.shape[1] * case["block"]

    def gather(codes, scales):  # [seqs, kv heads, keys, dim]
        return _numbers(codes[table], scales[table]).transpose(1, 2).reshape(seqs, hkv, keys, dim)

    new = cu[1:] - cu[:-1]
    i = torch.arange(most, device=cu.device)
    q = st["q"][(cu[:-1, None] + i).clamp(max=st["total"] - 1)].float()            # [seqs, most, heads, dim]
    q = q.reshape(seqs, most, hkv, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, group * most, dim)
    s = torch.matmul(q, gather(st["k"], st["k_scale"]).transpose(2, 3)).mul_(dim ** -0.5)
    s = s.view(seqs, hkv, group, most, keys)
    pos = (lens - new)[:, None] + i                                                # of each query
    j = torch.arange(keys, device=cu.device)
    seen = (j[None, None] < lens[:, None, None]).expand(seqs, most, keys)
    if case["causal"]:
        seen = seen & (j <= pos[..., None])
    if case["window"]:
        seen = seen & (j > pos[..., None] - case["window"])
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hkv, group * most, keys), gather(st["v"], st["v_scale"])).view(seqs, hkv, group, most, dim)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log())[..., 0]
    seq, at = _places(st)
    row = at - (lens - new)[seq]
    o = o.permute(0, 3, 1, 2, 4)[seq, row].reshape(st["total"], case["heads"], dim)
    lse = lse.permute(0, 3, 1, 2)[seq, row].reshape(st["total"], case["heads"])
    return o.to(DTYPES[case["dtype"]]), lse


def _value_of_byte(b):
    e, m = b >> 3, b & 7
    return (8 + m) * 2.0 ** (e - 18) if e else m * 2.0 ** -17


def exact(case, seed):
    st = prepare(case, seed)
    lens, news = _lengths(case)
    block, hkv, dim, group = case["block"], case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    starts = [sum(news[:s]) for s in range(len(news))]
    dev = "cuda"
    if case["op"] == "rotate":
        rot, done = case["rot"], []
        turns = [f / (2.0 * math.pi) for f in _frequencies(case)]
        pos = torch.cat([torch.arange(t - n, t, device=dev, dtype=torch.float64) for t, n in zip(lens, news)])
        angle = 2.0 * math.pi * torch.frac(pos[:, None] * torch.tensor(turns, dtype=torch.float64, device=dev))
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        for x, w in ((st["q"], st.get("wq")), (st["k"], st.get("wk"))):
            y = x.double()
            if w is not None:
                y = y / (y.square().sum(-1, keepdim=True) / dim + EPS).sqrt() * w.double()
            y = y.clone()
            pair = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(y[..., pair[0]].contiguous(), y[..., pair[1]].contiguous()) * turn
            y[..., pair[0]], y[..., pair[1]] = z.real, z.imag
            done.append(y)
        return tuple(done)
    if case["op"] == "write":
        if sum(news) * hkv * dim > 1 << 28:
            return None
        sizes = torch.tensor([_value_of_byte(b) for b in range(0xE3)], dtype=torch.float64, device=dev)
        values = torch.tensor(CODES, dtype=torch.float64, device=dev)

        def nearest(a, of):  # index of the nearest (ties: the even index) of rising numbers
            hi = torch.searchsorted(of, a.contiguous()).clamp(1, len(of) - 1)
            up, down = of[hi] - a, a - of[hi - 1]
            return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)

        done = []
        for x in (st["new_k"], st["new_v"]):
            x = x.double().reshape(-1, 16)
            a = x.abs().amax(-1)
            # of a and 6 sizes, which are exact, and not of a quotient
            s = sizes[nearest(a, 6.0 * sizes).clamp(min=1)][:, None]
            y = values[nearest((x.abs() / s).clamp(max=6.0), values)] * s
            done.append(torch.where(x < 0, -y, y).view(-1, hkv, dim))
        return tuple(done)

    def rows_of(codes, scales, s, total):  # [kv heads, tokens, dim]
        at = st["table"][s, : -(-total // block)].long()
        c, z = codes[at].long(), scales[at].long()
        c = torch.stack([c % 16, c // 16], -1).flatten(-2)[..., :dim]
        e, m = c % 8 // 2, c % 2
        x = torch.where(e > 0, (2.0 + m) * torch.exp2(e.double() - 2.0), 0.5 * m)
        x = torch.where(c >= 8, -x, x)
        z = torch.where(z >= 8, (8.0 + z % 8) * torch.exp2((z // 8).double() - 18.0), z * 2.0 ** -17)
        x = x * z.repeat_interleave(16, -1)
        return x.transpose(0, 1).reshape(hkv, -1, dim)[:, :total]

    if case["op"] == "read":
        if sum(lens) * hkv * dim > 1 << 29:
            return None
        return tuple(torch.cat([rows_of(codes, scales, s, t).transpose(0, 1)[t - n:] for s, (t, n) in enumerate(zip(lens, news))])
                     for codes, scales in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])))
    out = torch.empty(st["total"], case["heads"], dim, dtype=torch.float64, device=dev)
    lse = torch.empty(st["total"], case["heads"], dtype=torch.float64, device=dev)
    for s, (total, new) in enumerate(zip(lens, news)):
        k, v = rows_of(st["k"], st["k_scale"], s, total), rows_of(st["v"], st["v_scale"], s, total)
        j = torch.arange(total, device=dev)
        for lo in range(0, new, 1024):
            n = min(1024, new - lo)
            at = slice(starts[s] + lo, starts[s] + lo + n)
            pos = total - new + lo + torch.arange(n, device=dev)
            hidden = torch.zeros(n, total, dtype=torch.bool, device=dev)
            if case["causal"]:
                hidden |= j > pos[:, None]
            if case["window"]:
                hidden |= j <= pos[:, None] - case["window"]
            for h in range(case["heads"]):
                z = st["q"][at, h].double() @ k[h // group].T / dim ** 0.5
                z = z.masked_fill(hidden, float("-inf"))
                lse[at, h] = torch.logsumexp(z, -1)
                out[at, h] = torch.softmax(z, -1) @ v[h // group]
    return out, lse
