"""Cases, plain forms and exact values of the 4-bit KV cache operators and of the token sampler.

Three kinds of pass, each as a serving program makes it:

* ``store``: rows of K and V quantised into a paged 4-bit pool (``ql_kv4_write``) and the same
  rows read back (``ql_kv4_read``): what a prompt chunk does before it attends to itself. The
  answer is the values read back.
* ``read``: a sequence's whole context read back from the pool.
* ``attn``: the single-token attention of a batch of sequences over the pool
  (``ql_paged_attn_decode_kv4``).
* ``sample``: the next token of each row of logits from one uniform number a row
  (``ql_sample``), and its probability.

The 4-bit format. A row of ``head_dim`` values is cut into blocks of 32; a block keeps
m = f16(min), d = f16((max - min) / 15) and 32 codes c = clamp(rint((x - m) / d), 0, 15) (0 where
d = 0; ties to even); its values are d c + m. The 16 rows of a pool block and one kv head are one
record of 20 head_dim bytes; ``include/ql.h`` has its layout, which `_slots_of` restates.
"""
import math

import torch

own = False

BLOCK = 16          # tokens of a pool block


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one sequence's decode step appends one row per layer: latency only
        dict(name="store one row", op="store", n=1, n_kv=8, hd=128, f16=False, pad=0, strided=False),
        # a prompt chunk, K and V being slices of the f32 q|k|v projection
        dict(name="store a chunk", op="store", n=256, n_kv=8, hd=128, f16=False, pad=0, strided=True),
        # a context taken over from an f16 cache, with padded rows
        dict(name="store a prompt", op="store", n=16000, n_kv=8, hd=64, f16=True, pad=37, strided=False),
        # a short context read back for a prompt chunk
        dict(name="read a short context", op="read", n=333, n_kv=8, hd=128, f16=True),
        # a long context
        dict(name="read a long context", op="read", n=40960, n_kv=8, hd=128, f16=True),
        # batch 1: the latency of a decode step
        dict(name="attn batch 1", op="attn", batch=1, n_heads=32, n_kv=8, hd=128, low=2048, high=2048, empty=False),
        # small heads, one query head per kv head, ragged lengths from one token on, an idle slot
        dict(name="attn small heads", op="attn", batch=9, n_heads=12, n_kv=12, hd=64, low=1, high=1500, empty=True),
        # continuous batching
        dict(name="attn batch 32", op="attn", batch=32, n_heads=32, n_kv=8, hd=128, low=128, high=8192, empty=False),
        # long contexts, eight query heads per kv head
        dict(name="attn long contexts", op="attn", batch=16, n_heads=32, n_kv=4, hd=128, low=20000, high=40960, empty=False),
        # one sequence that answers
        dict(name="sample one row", op="sample", batch=1, vocab=151936, f16=False, top_k=50, top_p=0.95, min_p=0.0,
             greedy=False, pad=0),
        # continuous batching, the filters of a chat server, some rows greedy
        dict(name="sample batch 32", op="sample", batch=32, vocab=151936, f16=False, top_k=0, top_p=0.9, min_p=0.02,
             greedy=True, pad=0),
        # many rows of an odd vocabulary, no filter, rows that are not aligned
        dict(name="sample many rows", op="sample", batch=256, vocab=50021, f16=False, top_k=0, top_p=1.0, min_p=0.0,
             greedy=False, pad=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "read", "attn", "attn", "sample", "sample"])
    if op in ("store", "read"):
        c = dict(op=op, n=_log(rng, 1, 16000), n_kv=rng.choice([1, 2, 4, 8, 5]), hd=rng.choice([64, 128]),
                 f16=rng.random() < 0.5)
        if op == "store":
            c["pad"] = rng.choice([0, rng.randrange(1, 64)])
            c["strided"] = rng.random() < 0.5
        return c
    if op == "attn":
        n_kv = rng.choice([1, 2, 4, 8])
        high = _log(rng, 16, 16384)
        hd = rng.choice([64, 128, 128])
        batch = min(_log(rng, 1, 32), max(1, 16 * 30000 * 4 * 128 // (high * n_kv * hd)))
        return dict(op=op, batch=batch, n_heads=n_kv * rng.choice([1, 2, 3, 4, 6, 8, 16]), n_kv=n_kv, hd=hd,
                    low=max(1, int(high * rng.random())), high=high, empty=batch > 1 and rng.random() < 0.3)
    return dict(op=op, batch=_log(rng, 1, 64), vocab=_log(rng, 500, 151936), f16=rng.random() < 0.3,
                top_k=rng.choice([0, 0, rng.randrange(1, 200)]), top_p=rng.choice([1.0, 0.5 + 0.49 * rng.random()]),
                min_p=rng.choice([0.0, 0.1 * rng.random()]), greedy=rng.random() < 0.3, pad=rng.randrange(0, 5))


# ---------------------------------------------------------------- the record layout
def _slots_of(hd):
    """Where a record keeps its fields, as index tensors: the byte of a key code and of a value code [16, hd] with its
    shift, and the 16-bit word of a key scale, key minimum, value scale and value minimum [16, hd / 32]."""
    nb = hd // 32
    s = torch.arange(BLOCK).reshape(-1, 1)
    i = torch.arange(hd).reshape(1, -1)
    b, e = i // 32, i % 32
    # keys: byte 4 (nb j + b) + t holds elements 4 j + t (low four bits) and 4 j + t + 16 (high)
    j, t, high = (e % 16) // 4, e % 4, e // 16
    kb = s * (hd // 2) + 4 * (nb * j + b) + t
    ks = (4 * high).expand(BLOCK, hd)
    # values: unit u = e % 8 (of 2 nb bytes; at head_dim 128 u ^ 4 where bit 1 of the slot is set), word b: element u + 8 q is nibble q
    u, q = e % 8, e // 8
    if hd == 128:
        u = u ^ (4 * ((s >> 1) & 1))
    vb = 8 * hd + s * (hd // 2) + 2 * nb * u + 2 * b + q // 2
    vs = (4 * (q % 2)).expand(BLOCK, hd)
    b2 = torch.arange(nb).reshape(1, -1)
    kd = 8 * hd + s * nb + b2                       # 16-bit words from here on: byte 16 hd is word 8 hd
    km = kd + hd // 2
    vd = 9 * hd + (s & 3) * (4 * nb) + ((s >> 3) & 1) * (2 * nb) + 2 * b2 + ((s >> 2) & 1)
    vm = vd + hd // 2
    return kb, ks, vb.expand(BLOCK, hd), vs, kd, km, vd, vm


def _values(records, hd, dtype):
    """records u8 [..., 20 hd] -> keys and values [..., 16, hd] in `dtype`."""
    dev = records.device
    kb, ks, vb, vs, kd, km, vd, vm = (x.to(dev) for x in _slots_of(hd))
    words = records.view(torch.float16)

    def side(at, shift, d, m):
        c = ((records[..., at.reshape(-1)].reshape(*records.shape[:-1], BLOCK, hd).to(torch.int16) >> shift) & 15).to(dtype)
        scale, least = (words[..., x.reshape(-1)].reshape(*records.shape[:-1], BLOCK, hd // 32).to(dtype) for x in (d, m))
        return (c.reshape(*c.shape[:-1], hd // 32, 32) * scale.unsqueeze(-1) + least.unsqueeze(-1)).reshape(c.shape)

    return side(kb, ks, kd, km), side(vb, vs, vd, vm)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _random_pool(g, blocks, n_kv, hd):
    """Records as rows of unit variance give them: codes, scales near 0.27, minima near -2."""
    pool = torch.randint(0, 256, (blocks, n_kv, 20 * hd), dtype=torch.uint8, device="cuda", generator=g)
    w = pool.view(torch.float16)
    n = hd // 2
    for k in (0, 2):    # scales, then the minima that centre the codes on zero but for a tenth of the spread
        d = 0.27 * (1 + 0.15 * torch.randn((blocks, n_kv, n), device="cuda", generator=g)).clamp(0.4, 2.0)
        w[..., 8 * hd + k * n:8 * hd + (k + 1) * n] = d.half()
        w[..., 8 * hd + (k + 1) * n:8 * hd + (k + 2) * n] = (
            -7.5 * d + 0.4 * torch.randn((blocks, n_kv, n), device="cuda", generator=g)).half()
    return pool


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    if op in ("store", "read"):
        n, n_kv, hd = case["n"], case["n_kv"], case["hd"]
        dt = torch.float16 if case["f16"] else torch.float32
        blocks = (n + BLOCK - 1) // BLOCK + 3
        table = torch.randperm(blocks, device="cuda", generator=g)
        pos = torch.arange(n, device="cuda")
        slots = table[pos // BLOCK] * BLOCK + pos % BLOCK
        s["k_out"] = torch.zeros((n, n_kv, hd), dtype=dt, device="cuda")
        s["v_out"] = torch.zeros((n, n_kv, hd), dtype=dt, device="cuda")
        s["blocks"] = blocks
        if op == "read":
            s["pool"] = _random_pool(g, blocks, n_kv, hd)
        else:
            if case["pad"]:     # padded rows at the end: written nowhere, read as they were
                slots[max(1, n - case["pad"]):] = -1
            s["pool"] = torch.zeros((blocks, n_kv, 20 * hd), dtype=torch.uint8, device="cuda")
            width = (2 * n_kv + (4 * n_kv if case["strided"] else 0)) * hd
            rows = torch.randn((n, width), device="cuda", generator=g)
            # channels of different size, as rotated keys have them
            rows *= (0.5 + torch.rand((1, width), device="cuda", generator=g) ** 4 * 6)
            rows = rows.to(dt)
            if case["strided"]:
                s["k"] = rows[:, 4 * n_kv * hd:5 * n_kv * hd].unflatten(1, (n_kv, hd))
                s["v"] = rows[:, 5 * n_kv * hd:].unflatten(1, (n_kv, hd))
            else:
                s["k"] = rows[:, :n_kv * hd].reshape(n, n_kv, hd).contiguous()
                s["v"] = rows[:, n_kv * hd:].reshape(n, n_kv, hd).contiguous()
        s["slots"] = slots
        return s
    if op == "attn":
        batch, n_heads, n_kv, hd = case["batch"], case["n_heads"], case["n_kv"], case["hd"]
        lens = torch.randint(case["low"], case["high"] + 1, (batch,), generator=torch.Generator().manual_seed(int(seed) & 0x7FFFFFFF))
        if case["empty"]:
            lens[batch // 2] = 0
        need = (lens + BLOCK - 1) // BLOCK
        maxb = (case["high"] + BLOCK - 1) // BLOCK
        blocks = int(need.sum()) + 5
        ids = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
        table = torch.zeros((batch, maxb), dtype=torch.int32, device="cuda")
        at = 0
        for b in range(batch):
            table[b, :int(need[b])] = ids[at:at + int(need[b])]
            at += int(need[b])
        s |= {"pool": _random_pool(g, blocks, n_kv, hd), "table": table, "maxb": maxb, "blocks": blocks,
              "q": torch.randn((batch, n_heads, hd), device="cuda", generator=g).half(),
              "lens": lens.to("cuda", torch.int32), "host_lens": [int(x) for x in lens],
              "out": torch.zeros((batch, n_heads, hd), dtype=torch.float16, device="cuda")}
        if own:
            import quantized_transformer_decode_ql_gb300 as ql
            nbytes = ql.ql_paged_attn_kv4_workspace_bytes(batch, n_heads, n_kv, hd, maxb)
            s["workspace"] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        return s
    batch, vocab = case["batch"], case["vocab"]
    x = torch.randn((batch, vocab + case["pad"]), device="cuda", generator=g) * 2.5
    # a handful of likely tokens, and words that a grammar forbids
    x.scatter_add_(1, torch.randint(0, vocab, (batch, 8), device="cuda", generator=g),
                   4 * torch.rand((batch, 8), device="cuda", generator=g))
    x[torch.rand(x.shape, device="cuda", generator=g) < 0.02] = -math.inf
    x = x.half() if case["f16"] else x
    s["logits"] = x[:, :vocab]
    s["u"] = torch.rand((batch,), device="cuda", generator=g)
    s["t"] = 0.6 + 0.6 * torch.rand((batch,), device="cuda", generator=g)
    if case["greedy"]:
        s["t"][::5] = 0.0
    s["k"] = torch.full((batch,), case["top_k"], dtype=torch.int32, device="cuda") if case["top_k"] else None
    s["p"] = torch.full((batch,), case["top_p"], device="cuda") if case["top_p"] < 1 else None
    s["m"] = torch.full((batch,), case["min_p"], device="cuda") if case["min_p"] else None
    s["tokens"] = torch.zeros((batch,), dtype=torch.int32, device="cuda")
    s["probs"] = torch.zeros((batch,), device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _f16_of(x):
    """f64 -> the nearest f16 value, ties to even, in f64 (a conversion by way of f32 rounds twice)."""
    e = torch.frexp(x)[1].clamp(min=-13) - 11
    step = ((e.long() + 1023) << 52).view(torch.float64)     # 2^e exactly
    return torch.round(x / step) * step


def _quantised(x):
    """Rows [..., hd] -> the codes and the f16 scales and minima of their blocks, in f64: codes sit next to borders."""
    x = x.double().reshape(*x.shape[:-1], -1, 32)
    least = x.amin(-1)
    m = _f16_of(least) + 0.0
    d = _f16_of((x.amax(-1) - least) / 15)
    c = torch.round((x - m.unsqueeze(-1)) / torch.where(d > 0, d, torch.ones_like(d)).unsqueeze(-1)).clamp(0, 15)
    return torch.where(d.unsqueeze(-1) > 0, c, torch.zeros_like(c)), d, m


def _plain_write(s):
    hd, n_kv = s["case"]["hd"], s["case"]["n_kv"]
    dev = s["pool"].device
    kb, ks, vb, vs, kd, km, vd, vm = (x.to(dev) for x in _slots_of(hd))
    live = s["slots"] >= 0
    slots = s["slots"][live]
    block, at = slots // BLOCK, slots % BLOCK
    heads = torch.arange(n_kv, device=dev).reshape(1, -1, 1)
    for rows, byte, shift, dw, mw in ((s["k"], kb, ks, kd, km), (s["v"], vb, vs, vd, vm)):
        c, d, m = _quantised(rows[live])
        c = (c.reshape(len(slots), n_kv, hd).to(torch.int32) << shift[0]).to(torch.uint8)
        # the two nibbles of a byte belong to one row
        to = s["pool"]
        first = shift[0] == 0
        pair = torch.zeros((len(slots), n_kv, 20 * hd), dtype=torch.uint8, device=dev)
        pair.scatter_(2, byte[at][:, None, first].expand(-1, n_kv, -1), c[..., first])
        low = pair.gather(2, byte[at][:, None, ~first].expand(-1, n_kv, -1))
        to[block[:, None, None], heads, byte[at][:, None, ~first].expand(-1, n_kv, -1)] = low | c[..., ~first]
        words = to.view(torch.float16)
        words[block[:, None, None], heads, dw[at][:, None, :].expand(-1, n_kv, -1)] = d.half()
        words[block[:, None, None], heads, mw[at][:, None, :].expand(-1, n_kv, -1)] = m.half()


def _plain_read(s):
    hd = s["case"]["hd"]
    live = s["slots"] >= 0
    slots = s["slots"][live]
    step = 4096
    for lo in range(0, len(slots), step):
        part = slots[lo:lo + step]
        blocks, back = torch.unique(part // BLOCK, return_inverse=True)
        k, v = _values(s["pool"][blocks], hd, torch.float32)
        n = torch.arange(lo, lo + len(part), device=part.device)
        rows = torch.nonzero(live).reshape(-1)[n]
        s["k_out"][rows] = k[back, :, part % BLOCK].to(s["k_out"].dtype)
        s["v_out"][rows] = v[back, :, part % BLOCK].to(s["v_out"].dtype)
    return s["k_out"], s["v_out"]


def _plain_attn(s):
    c = s["case"]
    group, scale = c["n_heads"] // c["n_kv"], 1.0 / math.sqrt(c["hd"])
    for b, n in enumerate(s["host_lens"]):
        if n == 0:
            continue        # an idle slot: its row stays as it was
        k, v = _values(s["pool"][s["table"][b, :(n + BLOCK - 1) // BLOCK].long()], c["hd"], torch.float32)
        k, v = (x.permute(1, 0, 2, 3).reshape(c["n_kv"], -1, c["hd"])[:, :n] for x in (k, v))
        q = s["q"][b].float().reshape(c["n_kv"], group, c["hd"])
        x = torch.matmul(q, k.transpose(1, 2)) * scale
        p = torch.exp(x - x.amax(-1, keepdim=True))
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        s["out"][b] = o.reshape(c["n_heads"], c["hd"]).half()
    return s["out"]


def _plain_sample(s):
    x = s["logits"].double()        # sums over the vocabulary next to a border
    batch, vocab = x.shape
    t = s["t"].double().unsqueeze(1)
    greedy = t == 0
    top = x.amax(1, keepdim=True)
    w = torch.exp((x - top) / torch.where(greedy, torch.ones_like(t), t))
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    ws = w.gather(1, order)
    if s["k"] is not None:
        ws = torch.where(torch.arange(vocab, device=x.device) < s["k"].long().unsqueeze(1), ws, torch.zeros_like(ws))
    total = ws.sum(1, keepdim=True)
    if s["p"] is not None:
        ws = torch.where(torch.cumsum(ws, 1) - ws < s["p"].double().unsqueeze(1) * total, ws, torch.zeros_like(ws))
    kept = torch.zeros_like(w).scatter_(1, order, ws)
    if s["m"] is not None:
        kept = torch.where(x - top >= t * torch.log(s["m"].double().unsqueeze(1)), kept, torch.zeros_like(kept))
    total = kept.sum(1, keepdim=True)
    token = (torch.cumsum(kept, 1) > s["u"].double().unsqueeze(1) * total).int().argmax(1, keepdim=True)
    best = (x == top).int().argmax(1, keepdim=True)
    token = torch.where(greedy, best, token)
    prob = torch.where(greedy, torch.ones_like(t), kept.gather(1, token) / total)
    return token[:, 0].to(torch.int32), prob[:, 0].float()


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if not own:
        if s["op"] == "store":
            _plain_write(s)
        return {"store": _plain_read, "read": _plain_read, "attn": _plain_attn, "sample": _plain_sample}[s["op"]](s)
    import quantized_transformer_decode_ql_gb300 as ql
    if s["op"] in ("store", "read"):
        if s["op"] == "store":
            ql.ql_kv4_write(s["k"], s["v"], s["slots"], c["n_kv"], c["hd"], s["pool"], s["blocks"])
        ql.ql_kv4_read(s["pool"], s["slots"], c["n_kv"], c["hd"], s["blocks"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if s["op"] == "attn":
        ql.ql_paged_attn_decode_kv4(s["q"], s["pool"], s["table"], s["lens"], c["batch"], c["n_heads"], c["n_kv"], c["hd"],
                                    BLOCK, s["maxb"], s["blocks"], 1.0 / math.sqrt(c["hd"]), s["out"], s["workspace"])
        return s["out"]
    ql.ql_sample(s["logits"], s["u"], s["tokens"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"],
                 probs=s["probs"])
    return s["tokens"], s["probs"]


# ---------------------------------------------------------------- exact values
def _exact_rows(pool, hd, block, row, head):
    """Keys and values of pool rows, element by element, in 64 bits: block, row and head broadcast to [..., 1]."""
    e = torch.arange(hd, device=pool.device)
    nb, b, i = hd // 32, e // 32, e % 32
    word = pool.view(torch.float16)
    kc = pool[block, head, row * (hd // 2) + 4 * (nb * (i % 16 // 4) + b) + i % 4] >> (4 * (i // 16)) & 15
    unit = torch.bitwise_xor(i % 8, 4 * (row >> 1 & 1)) if hd == 128 else i % 8
    vc = pool[block, head, 8 * hd + row * (hd // 2) + 2 * nb * unit + 2 * b + i // 16] >> (4 * (i // 8 % 2)) & 15
    kw = 8 * hd + row * nb + b
    vw = 9 * hd + (row % 4) * 4 * nb + row // 8 * 2 * nb + 2 * b + row // 4 % 2
    return (kc * word[block, head, kw].double() + word[block, head, kw + hd // 2].double(),
            vc * word[block, head, vw].double() + word[block, head, vw + hd // 2].double())


def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits: rows one block at a time, weights by order statistics."""
    import numpy as np
    s = prepare(case, seed)
    if s["op"] == "store":
        hd, n_kv = case["hd"], case["n_kv"]
        live = (s["slots"] >= 0).cpu().numpy()
        out = []
        for name in ("k", "v"):
            x = s[name].cpu().numpy().astype(np.float64).reshape(case["n"] * n_kv * (hd // 32), 32)
            low, high = x.min(1), x.max(1)
            m, d = low.astype(np.float16).astype(np.float64), ((high - low) / 15).astype(np.float16).astype(np.float64)
            with np.errstate(divide="ignore", invalid="ignore"):
                c = np.where(d[:, None] > 0, np.clip(np.rint((x - m[:, None]) / d[:, None]), 0, 15), 0.0)
            y = (c * d[:, None] + m[:, None]).reshape(case["n"], n_kv, hd)
            y[~live] = 0
            out.append(y)
        return tuple(out)
    if s["op"] == "read":
        slots = s["slots"].reshape(-1, 1, 1)
        parts = [_exact_rows(s["pool"], case["hd"], at // BLOCK, at % BLOCK,
                             torch.arange(case["n_kv"], device=at.device).reshape(1, -1, 1)) for at in slots.split(4096)]
        return tuple(torch.cat(x) for x in zip(*parts))
    if s["op"] == "attn":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        group = case["n_heads"] // case["n_kv"]
        for b, n in enumerate(s["host_lens"]):
            at = torch.arange(n, device="cuda").reshape(-1, 1)
            for g in range(case["n_kv"] if n else 0):
                k, v = _exact_rows(s["pool"], case["hd"], s["table"][b].long()[at // BLOCK], at % BLOCK, torch.full_like(at, g))
                q = s["q"][b, g * group:(g + 1) * group].double()
                p = torch.softmax(torch.einsum("hd,td->ht", q, k) / math.sqrt(case["hd"]), 1)
                out[b, g * group:(g + 1) * group] = torch.einsum("ht,td->hd", p, v)
        return out
    probs = np.zeros(case["batch"])
    tokens = np.zeros(case["batch"], dtype=np.int32)
    u, t = s["u"].cpu().numpy().astype(np.float64), s["t"].cpu().numpy().astype(np.float64)
    k, p, m = (None if s[n] is None else s[n].cpu().numpy() for n in ("k", "p", "m"))
    for r in range(case["batch"]):
        x = s["logits"][r].cpu().numpy().astype(np.float64)
        at = np.argsort(-x, kind="stable")
        if t[r] == 0:
            tokens[r], probs[r] = at[0], 1.0
            continue
        w = np.exp((x[at] - x[at[0]]) / t[r])
        count = len(at) if k is None else min(len(at), int(k[r]))
        if p is not None:
            before = np.concatenate([[0.0], np.cumsum(w[:count])])
            count = max(1, int(np.searchsorted(before[:-1], float(p[r]) * before[-1], side="left")))
        if m is not None:
            count = min(count, int(np.count_nonzero(x[at] - x[at[0]] >= t[r] * math.log(float(m[r])))))
        index = np.sort(at[:count])
        w = np.exp((x[index] - x[at[0]]) / t[r])
        total = np.cumsum(w)
        n = min(int(np.searchsorted(total, u[r] * total[-1], side="right")), count - 1)
        tokens[r], probs[r] = index[n], w[n] / total[-1]
    return tokens, probs


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("store", "read"):
        values = case["n"] * case["n_kv"] * case["hd"] * 2
        size = 2 if case["f16"] else 4
        # a store takes the rows in, leaves their records and gives the values back; a read takes the records
        moved = values * 20 // 32 + values * size * (2 if op == "store" else 1) + 8 * case["n"]
        return {"bytes": moved, "flops": values * (8 if op == "store" else 2)}
    if op == "attn":
        # lengths are uniform between low and high
        tokens = case["batch"] * (case["low"] + case["high"]) / 2
        if case["empty"]:
            tokens *= 1 - 1 / case["batch"]
        moved = tokens * case["n_kv"] * case["hd"] * 20 / 16 + tokens / 4 + case["batch"] * case["n_heads"] * case["hd"] * 4
        return {"bytes": moved, "flops": 4 * tokens * case["n_heads"] * case["hd"]}
    values = case["batch"] * case["vocab"]
    return {"bytes": values * (2 if case["f16"] else 4) + 28 * case["batch"], "flops": 6 * values}
