"""Cases, plain forms and exact values of the latent attention operators.

Latent attention keeps one row a token for all heads: a normalised latent vector c of ``rank`` values and one rotated key
part of ``ROPE`` values. Head h has keys [Wk_h c | rotated part] and values Wv_h c, where Wk_h and Wv_h are ``hd`` rows of
``rank`` weights each. Three kinds of pass, each as a serving program makes it:

* ``append``: the projections of n tokens: the latents normalised and their key parts rotated into a paged cache, the
  queries' last ROPE values rotated (``ql_mla_append``). The answer is the queries and the cache.
* ``decode``: one new token of each sequence over the paged cache (``ql_mla_attn_decode``), the form in which the weights
  are multiplied into the query and into the answer, and the cache is read as it is.
* ``chunk``: a chunk of a prompt over the cache that holds it (``ql_mla_attn_chunk``), causal, the form in which keys and
  values are made from the latents.
"""
import math

import torch

own = False

BLOCK = 16              # tokens of a pool block
ROPE = 64               # values of the rotated part
EPS = 1e-6
MAX_POSITION = 40960    # rows of the rotation tables


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one sequence's step appends one row a layer: latency only
        dict(name="append one row", op="append", n=1, heads=32, hd=128, rank=512, f16=False, pad=0, strided=False),
        # a batch's step, its rows slices of the projections, padded to a larger batch
        dict(name="append a batch", op="append", n=61, heads=40, hd=64, rank=256, f16=True, pad=7, strided=True),
        # a long prompt
        dict(name="append a prompt", op="append", n=8000, heads=32, hd=128, rank=512, f16=False, pad=0, strided=False),
        # batch 1: the latency of a step
        dict(name="decode batch 1", op="decode", batch=1, heads=32, hd=128, rank=512, low=2048, high=2048, empty=False),
        # small heads, ragged lengths from one token on, an idle slot
        dict(name="decode small heads", op="decode", batch=9, heads=11, hd=64, rank=256, low=1, high=1500, empty=True),
        # continuous batching
        dict(name="decode batch 32", op="decode", batch=32, heads=32, hd=128, rank=512, low=128, high=8192, empty=False),
        # long contexts
        dict(name="decode long contexts", op="decode", batch=16, heads=64, hd=128, rank=512, low=20000, high=40960, empty=False),
        # more heads than one tile of a tensor core takes
        dict(name="decode many heads", op="decode", batch=8, heads=96, hd=128, rank=512, low=4000, high=16000, empty=False),
        # the first tokens of a conversation, a small model
        dict(name="chunk first tokens", op="chunk", n=17, before=0, heads=4, hd=64, rank=256),
        # a chunk of a prompt whose first part is in the cache
        dict(name="chunk after a context", op="chunk", n=256, before=7936, heads=32, hd=128, rank=512),
        # odd sizes, small heads
        dict(name="chunk of odd size", op="chunk", n=777, before=1234, heads=20, hd=64, rank=256),
        # a whole prompt
        dict(name="chunk a prompt", op="chunk", n=4096, before=0, heads=32, hd=128, rank=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "chunk", "chunk"])
    c = dict(op=op, heads=_log(rng, 1, 64), hd=rng.choice([64, 128, 128]), rank=rng.choice([256, 512, 512]))
    if op == "append":
        c |= dict(n=_log(rng, 1, 8000 * 32 // max(32, c["heads"])), f16=rng.random() < 0.5, strided=rng.random() < 0.5,
                  pad=rng.choice([0, rng.randrange(1, 64)]))
    elif op == "decode":
        high = _log(rng, 16, 40960)
        batch = min(_log(rng, 1, 64), max(1, 16 * 30000 // high))
        c |= dict(batch=batch, low=max(1, int(high * rng.random())), high=high, empty=batch > 1 and rng.random() < 0.3)
    else:
        c["heads"] = min(c["heads"], 32)
        n = _log(rng, 1, 2500)
        c |= dict(n=n, before=rng.choice([0, rng.randrange(1, 2 * n + 2), _log(rng, 1, 8000 - n)]))
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _pool(g, blocks, rank):
    """Normalised latents and rotated key parts, as rows of unit variance give them."""
    return torch.randn((blocks, BLOCK, rank + ROPE), device="cuda", generator=g).half()


def _weights(g, heads, hd, rank):
    """Each head's hd key rows, then its hd value rows."""
    return (torch.randn((heads, 2 * hd, rank), device="cuda", generator=g) / math.sqrt(rank)).half()


def prepare(case, seed):
    g = _gen(seed)
    op, heads, hd, rank = case["op"], case["heads"], case["hd"], case["rank"]
    s = {"op": op, "case": dict(case), "scale": 1.0 / math.sqrt(hd + ROPE)}
    if op == "append":
        n = case["n"]
        dt = torch.float16 if case["f16"] else torch.float32
        blocks = (n + BLOCK - 1) // BLOCK + 3
        table = torch.randperm(blocks, device="cuda", generator=g)
        at = torch.arange(n, device="cuda")
        slots = table[at // BLOCK] * BLOCK + at % BLOCK
        if case["pad"]:     # padded rows at the end: written nowhere
            slots[max(1, n - case["pad"]):] = -1
        first = torch.randint(0, MAX_POSITION - n, (1,), device="cuda", generator=g)
        angle = torch.outer(torch.arange(MAX_POSITION, device="cuda", dtype=torch.float64),
                            1e6 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE))
        extra = 8 * 16 if case["strided"] else 0
        q = torch.randn((n, heads * (hd + ROPE) + extra), device="cuda", generator=g).to(dt)
        kv = torch.randn((n, rank + ROPE + extra), device="cuda", generator=g)
        kv = (kv * (0.3 + 3 * torch.rand((1, kv.shape[1]), device="cuda", generator=g) ** 3)).to(dt)
        s |= {"q": q[:, extra:].unflatten(1, (heads, hd + ROPE)), "kv": kv[:, :rank + ROPE], "slots": slots, "blocks": blocks,
              "norm": 1 + 0.1 * torch.randn((rank,), device="cuda", generator=g), "cos": angle.cos().float(),
              "sin": angle.sin().float(), "positions": (first + at).to(torch.int32), "pool": _pool(g, blocks, rank),
              "q_out": torch.zeros((n, heads, hd + ROPE), dtype=torch.float16, device="cuda")}
        return s
    host = torch.Generator().manual_seed(int(seed) & 0x7FFFFFFF)
    if op == "decode":
        rows = case["batch"]
        lens = torch.randint(case["low"], case["high"] + 1, (rows,), generator=host)
        if case["empty"]:
            lens[rows // 2] = 0
        maxb = (case["high"] + BLOCK - 1) // BLOCK
    else:
        rows = case["n"]
        lens = torch.tensor([case["before"] + rows])
        maxb = (int(lens[0]) + BLOCK - 1) // BLOCK
    need = (lens + BLOCK - 1) // BLOCK
    blocks = int(need.sum()) + 5
    ids = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros((len(lens), maxb), dtype=torch.int32, device="cuda")
    at = 0
    for b in range(len(lens)):
        table[b, :int(need[b])] = ids[at:at + int(need[b])]
        at += int(need[b])
    s |= {"pool": _pool(g, blocks, rank), "w": _weights(g, heads, hd, rank), "table": table, "maxb": maxb, "blocks": blocks,
          "q": (1.5 * torch.randn((rows, heads, hd + ROPE), device="cuda", generator=g)).half(),
          "lens": lens.to("cuda", torch.int32), "host_lens": [int(x) for x in lens],
          "out": torch.zeros((rows, heads, hd), dtype=torch.float16, device="cuda")}
    if op == "chunk":
        s["position"] = torch.tensor([case["before"]], dtype=torch.int32, device="cuda")
    if own:
        import quantized_transformer_decode_ql_gb300 as ql
        size = ql.ql_mla_decode_workspace_bytes if op == "decode" else ql.ql_mla_chunk_workspace_bytes
        s["workspace"] = torch.empty(size(rows, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _rotate(x, cos, sin):
    """Pairs (i, i + ROPE / 2) of the last axis turned by the angles whose cosines and sines are given."""
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    c = s["case"]
    live = s["slots"] >= 0
    at = s["positions"][live].long()
    cos, sin = s["cos"][at], s["sin"][at]
    x = s["kv"][live].float()
    latent = x[:, :c["rank"]]
    latent = latent / torch.sqrt((latent * latent).mean(-1, keepdim=True) + EPS) * s["norm"]
    slots = s["slots"][live]
    s["pool"][slots // BLOCK, slots % BLOCK] = torch.cat([latent, _rotate(x[:, c["rank"]:], cos, sin)], -1).half()
    q = s["q"][live].float()
    q = torch.cat([q[..., :c["hd"]], _rotate(q[..., c["hd"]:], cos[:, None], sin[:, None])], -1)
    s["q_out"][live] = q.half()
    return s["q_out"], s["pool"]


def _rows(s, b, n):
    """The first n rows of sequence b in 32 bits: latents and rotated parts."""
    x = s["pool"][s["table"][b, :(n + BLOCK - 1) // BLOCK].long()].reshape(-1, s["case"]["rank"] + ROPE)[:n].float()
    return x[:, :s["case"]["rank"]], x


def _plain_decode(s):
    hd = s["case"]["hd"]
    wk, wv = s["w"][:, :hd].float(), s["w"][:, hd:].float()
    q = s["q"].float()
    qc = torch.matmul(q[..., :hd].transpose(0, 1), wk).transpose(0, 1)       # [batch, heads, rank]
    q = torch.cat([qc, q[..., hd:]], -1)
    o = torch.zeros_like(qc)
    for b, n in enumerate(s["host_lens"]):
        if n:
            latent, row = _rows(s, b, n)
            x = torch.matmul(q[b], row.t()) * s["scale"]
            p = torch.exp(x - x.amax(-1, keepdim=True))
            o[b] = torch.matmul(p, latent) / p.sum(-1, keepdim=True)
    o = torch.matmul(o.transpose(0, 1), wv.transpose(1, 2)).transpose(0, 1)  # [batch, heads, hd]
    live = (s["lens"] > 0).reshape(-1, 1, 1)
    s["out"].copy_(torch.where(live, o.half(), s["out"]))       # an idle slot: its row stays as it was
    return s["out"]


def _plain_chunk(s):
    c = s["case"]
    hd, n, before = c["hd"], c["n"], c["before"]
    latent, row = _rows(s, 0, before + n)
    turned = row[:, c["rank"]:]
    at = torch.arange(before + n, device=row.device)
    later = at[None, :] > at[before:, None]
    for h in range(c["heads"]):
        w = s["w"][h].float()
        k = torch.cat([torch.matmul(latent, w[:hd].t()), turned], -1)
        x = torch.matmul(s["q"][:, h].float(), k.t()) * s["scale"]
        x.masked_fill_(later, -math.inf)
        p = torch.exp(x - x.amax(-1, keepdim=True))
        s["out"][:, h] = (torch.matmul(p, torch.matmul(latent, w[hd:].t())) / p.sum(-1, keepdim=True)).half()
    return s["out"]


# ---------------------------------------------------------------- one pass
def run(s):
    if not own:
        return {"append": _plain_append, "decode": _plain_decode, "chunk": _plain_chunk}[s["op"]](s)
    import quantized_transformer_decode_ql_gb300 as ql
    c = s["case"]
    if s["op"] == "append":
        ql.ql_mla_append(s["q"], s["kv"], s["norm"], s["cos"], s["sin"], s["positions"], s["slots"], EPS, c["heads"], c["hd"],
                         c["rank"], ROPE, s["q_out"], s["pool"], s["blocks"], MAX_POSITION)
        return s["q_out"], s["pool"]
    if s["op"] == "decode":
        ql.ql_mla_attn_decode(s["q"], s["w"], s["pool"], s["table"], s["lens"], c["batch"], c["heads"], c["hd"], c["rank"], ROPE,
                              BLOCK, s["maxb"], s["blocks"], s["scale"], s["out"], s["workspace"])
    else:
        ql.ql_mla_attn_chunk(s["q"], s["w"], s["pool"], s["table"], s["position"], c["n"], c["heads"], c["hd"], c["rank"], ROPE,
                             BLOCK, s["maxb"], s["blocks"], s["scale"], s["out"], s["workspace"])
    return s["out"]


# ---------------------------------------------------------------- exact values
def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits: tokens one by one or a head's keys and values at a time."""
    s = prepare(case, seed)
    hd, rank, heads = case["hd"], case["rank"], case["heads"]
    if case["op"] == "append":
        q_out, pool = s["q_out"].double(), s["pool"].double()
        i = torch.arange(ROPE // 2, device="cuda")
        for part in torch.nonzero(s["slots"] >= 0).reshape(-1).split(1000):
            slot, at = s["slots"][part], s["positions"][part].long()
            turn = torch.complex(s["cos"][at].double(), s["sin"][at].double())
            x, q = s["kv"][part].double(), s["q"][part].double()
            size = torch.sqrt(x[:, :rank].square().sum(-1) / rank + EPS)
            pool[slot // BLOCK, slot % BLOCK, :rank] = x[:, :rank] * s["norm"].double() / size.unsqueeze(-1)
            z = turn * torch.complex(x[:, rank + i], x[:, rank + ROPE // 2 + i])
            pool[slot // BLOCK, slot % BLOCK, rank:] = torch.cat([z.real, z.imag], -1)
            z = turn.unsqueeze(1) * torch.complex(q[..., hd + i], q[..., hd + ROPE // 2 + i])
            q_out[part] = torch.cat([q[..., :hd], z.real, z.imag], -1)
        return q_out, pool
    if case["op"] == "decode":
        tokens, pairs = sum(s["host_lens"]), sum(s["host_lens"])
    else:
        tokens = case["n"] + case["before"]
        pairs = case["n"] * tokens
    if 2.0 * heads * (2 * hd * rank * tokens + (2 * hd + ROPE) * pairs) > 1.2e13:
        return None         # a minute of 64-bit products
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["host_lens"]):
        if n == 0:
            continue
        t = torch.arange(n, device="cuda")
        row = s["pool"][s["table"][b].long()[t // BLOCK], t % BLOCK].double()
        for h in range(heads):
            # k and v of the head for every token
            kv = torch.einsum("tr,er->te", row[:, :rank], s["w"][h].double())
            q = s["q"][:, h] if case["op"] == "chunk" else s["q"][b:b + 1, h]
            score = (torch.einsum("qe,te->qt", q[:, :hd].double(), kv[:, :hd])
                     + torch.einsum("qe,te->qt", q[:, hd:].double(), row[:, rank:])) / math.sqrt(hd + ROPE)
            if case["op"] == "chunk":
                score = score.tril(case["before"]).where(torch.ones_like(score).tril(case["before"]) > 0,
                                                         torch.full_like(score, -math.inf))
            o = torch.softmax(score, -1) @ kv[:, hd:]
            if case["op"] == "chunk":
                out[:, h] = o
            else:
                out[b, h] = o[0]
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    heads, hd, rank = case["heads"], case["hd"], case["rank"]
    row = heads * (hd + ROPE)
    if case["op"] == "append":
        values = case["n"] * (row + rank + ROPE)
        return {"bytes": values * ((2 if case["f16"] else 4) + 2) + case["n"] * (12 + 4 * ROPE) + 4 * rank, "flops": 4 * values}
    weights = heads * 2 * hd * rank
    if case["op"] == "decode":
        rows = case["batch"]
        tokens = rows * (case["low"] + case["high"]) / 2        # lengths are uniform between low and high
        if case["empty"]:
            tokens *= 1 - 1 / rows
        flops = 2 * rows * weights + 2 * tokens * heads * (2 * rank + ROPE)
    else:
        rows = case["n"]
        tokens = case["before"] + rows
        pairs = rows * case["before"] + rows * (rows + 1) / 2
        # the cheaper of keys and values made once a token, and the weights multiplied into each query and answer
        flops = min(2 * tokens * weights + 2 * pairs * heads * (2 * hd + ROPE),
                    2 * rows * weights + 2 * pairs * heads * (2 * rank + ROPE))
    return {"bytes": 2 * tokens * (rank + ROPE) + tokens / 4 + 2 * weights + 2 * rows * (row + heads * hd), "flops": flops}
