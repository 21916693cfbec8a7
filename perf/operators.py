"""The 8-bit key/value cache operators, as they are measured: writing tokens into the cache, reading them back, and
attention over it.

The cache is paged. A pool holds blocks of `block` tokens; for each block and key/value head it has the tokens' codes
(E4M3, 8 bits) and one float32 scale for the keys and one for the values: a number is code * scale. A block table gives
each sequence's blocks. New tokens of a sequence are the last of its `lens` tokens."""
import torch

own = False

F8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LARGEST = 448.0  # of an E4M3 code


def _case(name, op, seqs, len_min, len_max, new_min, new_max, heads=32, kv_heads=8, dim=128, block=64, dtype="bf16",
          causal=True, window=0):
    return dict(name=name, op=op, seqs=seqs, len_min=len_min, len_max=len_max, new_min=new_min, new_max=new_max,
             heads=heads, kv_heads=kv_heads, dim=dim, block=block, dtype=dtype, causal=causal, window=window)


def listed():
    return [
        # one decoding step's keys and values, 32 sequences in service: the smallest write, latency counts
        _case("write_step", "write", 32, 100, 4000, 1, 1),
        # five prompts admitted at once, the usual prompt write
        _case("write_prompts", "write", 5, 1500, 5000, 1500, 5000),
        # chunks appended behind what the cache holds, float32 activations, small blocks and a small odd head size
        _case("write_chunks_fp32", "write", 7, 700, 2111, 33, 517, heads=12, kv_heads=6, dim=80, block=16, dtype="fp32"),
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
        # drafted tokens checked in one step, sliding window, float16, 8 query heads to a head
        _case("attend_drafts", "attend", 16, 200, 6000, 2, 5, heads=16, kv_heads=2, block=16, dtype="fp16", window=4096),
        # a chunk of a prompt over what was written before it, and another user's: few rows, long axis, tensor-core work
        _case("attend_chunk", "attend", 2, 12000, 16384, 400, 512),
        # a whole prompt: the largest amount of arithmetic
        _case("attend_prompt", "attend", 1, 8192, 8192, 8192, 8192),
        # decoding and prompts in one batch, head size 64, no grouping of heads
        _case("attend_mixed", "attend", 24, 40, 2500, 1, 300, heads=8, kv_heads=8, dim=64, block=16, dtype="fp16"),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["write", "read", "attend", "attend"])
    dtypes = ["bf16", "fp16"] if op == "attend" else ["bf16", "fp16", "fp32"]
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    c = dict(heads=kv_heads * group, kv_heads=kv_heads, dim=rng.choice([32, 64, 80, 112, 128, 128]),
             block=rng.choice([16, 32, 64, 128]), dtype=rng.choice(dtypes), causal=True, window=0)
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
    if case["new_min"] == case["len_min"] and case["new_max"] == case["len_max"]:
        return lens, list(lens)
    if case["op"] != "attend" and case["len_min"] - case["new_min"] == case["len_max"] - case["new_max"]:
        return lens, [v - case["len_min"] + case["new_min"] for v in lens]
    return lens, [min(a, b) for a, b in zip(lens, _spread(case["new_min"], case["new_max"], n))]


def _pairs(case):
    """Query and key pairs that the masks leave, and keys that some query sees, over the sequences."""
    pairs = keys = 0
    for total, new in zip(*_lengths(case)):
        first, w = total - new, case["window"]
        for_all = 0
        if case["causal"]:
            for_all = sum(min(p + 1, w) for p in range(first, total)) if w else new * first + new * (new + 1) // 2
        else:
            for_all = sum(total - max(0, p - w + 1) for p in range(first, total)) if w else new * total
        pairs += for_all
        keys += total - (max(0, first - w + 1) if w else 0)
    return pairs, keys


def work(case):
    lens, news = _lengths(case)
    tokens, seqs = sum(news), case["seqs"]
    elt = 4 if case["dtype"] == "fp32" else 2
    row = case["kv_heads"] * case["dim"]
    b = case["block"]
    blocks = sum(-(-t // b) - (t - n) // b for t, n in zip(lens, news))
    if case["op"] in ("write", "read"):
        scales = 2 * 4 * blocks * case["kv_heads"]
        return {"bytes": 2 * tokens * row * (elt + 1) + scales + 4 * (blocks + 2 * seqs), "flops": 2 * 2 * tokens * row}
    pairs, keys = _pairs(case)
    scales = 2 * 4 * (keys // b) * case["kv_heads"]
    q = tokens * case["heads"] * case["dim"] * 2
    return {"bytes": 2 * keys * row + scales + 2 * q + 4 * tokens * case["heads"] + 4 * (keys // b + 2 * seqs),
            "flops": 4 * pairs * case["heads"] * case["dim"]}


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

    def pool():
        # blocks differ in magnitude by a few powers of two
        scale = torch.exp2(torch.randint(-8, -4, (n_blocks, hkv), generator=g, device=dev).float())
        x = torch.randn(n_blocks, hkv, block, dim, generator=g, device=dev) * 64.0
        return x.clamp_(-LARGEST, LARGEST).to(F8), scale

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
        st["cache"] = zc.KVCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        st["batch"] = zc.KVBatch(st["table"], st["cu"], st["lens"], st["total"], st["most"])
    return st


def run(st):
    case = st["case"]
    if own:
        import entropy_coding_gb300 as zc
        if case["op"] == "write":
            zc.kv_write(st["cache"], st["batch"], st["new_k"], st["new_v"])
            return st["k"], st["v"], st["k_scale"], st["v_scale"]
        if case["op"] == "read":
            return zc.kv_read(st["cache"], st["batch"], dtype=DTYPES[case["dtype"]])
        return zc.kv_attend(st["cache"], st["batch"], st["q"], causal=case["causal"], window=case["window"])
    if case["op"] == "write":
        _write(st, st["new_k"], st["k"], st["k_scale"])
        _write(st, st["new_v"], st["v"], st["v_scale"])
        return st["k"], st["v"], st["k_scale"], st["v_scale"]
    if case["op"] == "read":
        return _read(st, st["k"], st["k_scale"]), _read(st, st["v"], st["v_scale"])
    return _attend(st)


def _places(st):
    """Sequence and position of each token of the batch."""
    cu, lens = st["cu"].long(), st["lens"].long()
    new = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(len(lens), device=cu.device), new, output_size=st["total"])
    return seq, torch.arange(st["total"], device=cu.device) - cu[seq] + (lens - new)[seq]


def _write(st, x, codes, scales):
    block, hkv, dim = st["case"]["block"], st["case"]["kv_heads"], st["case"]["dim"]
    seq, pos = _places(st)
    home = st["table"][seq, pos // block].long()               # each token's block
    x = x.float()
    # the largest magnitude of the new rows of each block and head
    amax = torch.zeros_like(scales).index_reduce_(0, home, x.abs().amax(-1), "amax")
    # the least power of two that holds it: frexp gives a = m 2^e with m in [1/2, 1), and 448 = 7/8 2^9
    m, e = torch.frexp(amax)
    need = torch.exp2((e - 9 + (m > 0.875)).float().clamp(min=-126.0))
    need = torch.where(amax > 0, need, torch.full_like(need, 2.0 ** -126))
    new = (st["cu"][1:] - st["cu"][:-1]).long()
    start = st["lens"].long() - new
    kept = torch.zeros(len(codes), dtype=torch.long, device=codes.device)  # rows of a block that were there before
    held = start % block
    # a sequence that begins inside a block keeps that block's first rows
    kept[st["table"][torch.arange(len(start), device=start.device), start // block % st["table"].shape[1]].long()] = held
    mine = torch.zeros(len(codes), dtype=torch.bool, device=codes.device).index_fill_(0, home, True)
    kept = kept * mine
    then = torch.where((kept > 0)[:, None], scales, torch.zeros_like(scales))
    now = torch.where(mine[:, None], torch.maximum(then, need), scales)
    # rows of grown blocks that were there before move to the new scale
    grown = ((now != scales) & (kept > 0)[:, None])[:, :, None] & (torch.arange(block, device=codes.device) < kept[:, None])[:, None]
    first = st["table"][torch.arange(len(start), device=start.device), start // block % st["table"].shape[1]].long()
    old = codes.view(torch.uint8)[first].view(F8).float()
    moved = (old * (scales / now)[first][:, :, None, None]).to(F8)
    bytes_ = codes.view(torch.uint8)
    bytes_[first] = torch.where(grown[first][..., None], moved.view(torch.uint8), bytes_[first])
    scales.copy_(now)
    q = (x / now[home][:, :, None]).clamp(-LARGEST, LARGEST).to(F8)
    bytes_[home[:, None], torch.arange(hkv, device=codes.device)[None], (pos % block)[:, None]] = q.view(torch.uint8)


def _read(st, codes, scales):
    block, hkv = st["case"]["block"], st["case"]["kv_heads"]
    seq, pos = _places(st)
    home = st["table"][seq, pos // block].long()
    head = torch.arange(hkv, device=codes.device)[None]
    rows = codes.view(torch.uint8)[home[:, None], head, (pos % block)[:, None]].view(F8)
    return (rows.float() * scales[home][:, :, None]).to(DTYPES[st["case"]["dtype"]])


def _attend(st):
    case, table = st["case"], st["table"].long()
    hkv, dim, group = case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    cu, lens, most = st["cu"].long(), st["lens"].long(), st["most"]
    seqs, keys = len(lens), table.shape[1] * case["block"]

    def gather(codes, scales):  # [seqs, kv heads, keys, dim]
        x = codes.view(torch.uint8)[table].view(F8).float() * scales[table][..., None, None]
        return x.transpose(1, 2).reshape(seqs, hkv, keys, dim)

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


def _round_e4m3(x):
    """x (float64, |x| <= 448) rounded to the nearest E4M3 value, ties to the even code."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())  # four significant bits; 2^-9 below the normal range
    return torch.round(x / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    lens, news = _lengths(case)
    block, hkv, dim, group = case["block"], case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    table = st["table"].tolist()
    starts = [sum(news[:s]) for s in range(len(news))]
    if case["op"] == "write":
        done = []
        for x, codes, scales in ((st["new_k"], st["k"], st["k_scale"]), (st["new_v"], st["v"], st["v_scale"])):
            values, scales, x = codes.double(), scales.double(), x.double()
            for s, (total, new) in enumerate(zip(lens, news)):
                first = total - new
                for b in range(first // block, -(-total // block)):
                    lo, hi = max(first, b * block), min(total, (b + 1) * block)
                    rows = x[starts[s] + lo - first: starts[s] + hi - first].transpose(0, 1)  # [kv heads, rows, dim]
                    a = rows.abs().amax((1, 2))
                    # log2 is only a guess at the exponent here: the comparison below settles it
                    e = torch.ceil(torch.log2(a / LARGEST).clamp(min=-126.0))
                    e = torch.where(LARGEST * torch.exp2(e - 1) >= a, e - 1, e)
                    e = torch.where(LARGEST * torch.exp2(e) < a, e + 1, e).clamp(min=-126.0)
                    need, at, n0 = torch.exp2(e), table[s][b], lo - b * block
                    if n0:
                        now = torch.maximum(scales[at], need)
                        values[at, :, :n0] = _round_e4m3(values[at, :, :n0] * (scales[at] / now)[:, None, None])
                    else:
                        now = need
                    scales[at] = now
                    y = (rows / now[:, None, None]).clamp(-LARGEST, LARGEST)
                    values[at, :, n0: n0 + hi - lo] = _round_e4m3(y)
            done.append((values, scales))
        return done[0][0], done[1][0], done[0][1], done[1][1]

    def keys_of(codes, scales, s, total):  # [kv heads, tokens, dim]
        at = torch.tensor(table[s][: -(-total // block)], device=codes.device)
        x = codes.view(torch.uint8)[at].view(F8).double() * scales[at].double()[:, :, None, None]
        return x.permute(1, 0, 2, 3).reshape(hkv, -1, dim)[:, :total]

    if case["op"] == "read":
        if sum(lens) * hkv * dim > 1 << 29:
            return None
        both = []
        for codes, scales in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
            both.append(torch.cat([keys_of(codes, scales, s, t).transpose(0, 1)[t - n:] for s, (t, n) in enumerate(zip(lens, news))]))
        return tuple(both)
    out = torch.empty(st["total"], case["heads"], dim, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["total"], case["heads"], dtype=torch.float64, device="cuda")
    for s, (total, new) in enumerate(zip(lens, news)):
        k, v = keys_of(st["k"], st["k_scale"], s, total), keys_of(st["v"], st["v_scale"], s, total)
        j = torch.arange(total, device="cuda")
        for lo in range(0, new, 1024):
            n = min(1024, new - lo)
            at = slice(starts[s] + lo, starts[s] + lo + n)
            pos = total - new + lo + torch.arange(n, device="cuda")
            hidden = torch.zeros(n, total, dtype=torch.bool, device="cuda")
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
