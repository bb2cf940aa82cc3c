"""More measured cases of the vocabulary operators: log-probabilities of given
tokens with entropy and top alternatives, their gradient, and a vocabulary table
held in 4 bits: made from float weights, looked up, and multiplied with hidden
rows for the logits.

`run` takes one pass: with `own` false in plain torch operations, with `own`
true through `lm_head_vocab_gb300.VocabOps`, on the inputs that `prepare` made.
`exact` gives the same outputs from the definitions in 64 bits.

A table [V, D] has groups of `group` columns; a value is
scales[g, v] * (q - zeros[g, v]), q in 0..15 (two to a byte, the lower column in
the low half), zeros 8 where the table has none.
"""
import functools
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_IGNORE = -100


def listed():
    return [
        # a small model's table with a group that ends past the last column, scales in fp32, read back
        dict(name="quantize_ragged", op="quantize", V=32003, D=1001, group=32, w="fp32", scales="fp32", zeros=True),
        # loading a model: its bf16 table becomes a 4-bit one, read back
        dict(name="quantize_whole", op="quantize", V=128256, D=4096, group=128, w="bf16", scales="fp16", zeros=False),
        # the embeddings of one decoding step for a batch of eight sequences
        dict(name="lookup_step", op="lookup", T=8, V=128256, D=4096, group=128, scales="fp16", zeros=False, out="bf16",
             scale=64.0, ignored=0.0),
        # the embeddings of a long packed prompt, some positions without a token
        dict(name="lookup_packed", op="lookup", T=32767, V=151936, D=2048, group=64, scales="bf16", zeros=True,
             out="bf16", scale=1.0, ignored=0.02),
        # the LM head for a single token: what a decoding step waits for
        dict(name="logits_one", op="logits", T=1, V=128256, D=4096, group=128, scales="fp16", zeros=False, x="bf16",
             out="bf16"),
        # beams of a small fp32 model: odd width, odd vocabulary, small groups with zeros
        dict(name="logits_ragged", op="logits", T=40, V=32003, D=1001, group=32, scales="fp32", zeros=True, x="fp32",
             out="fp32"),
        # the logits of a prompt's last part, to be scored
        dict(name="logits_prompt", op="logits", T=512, V=128256, D=4096, group=128, scales="fp16", zeros=False,
             x="bf16", out="bf16"),
        # one sampled token's log-probability with twenty alternatives: latency
        dict(name="logprobs_one", op="logprobs", T=1, V=128256, dtype="bf16", n=1, M=20, temperature=1.0, mask="none"),
        # constrained answers of a small fp32 model: eight choices a row, masks (one row allows nothing)
        dict(name="logprobs_masked", op="logprobs", T=61, V=32003, dtype="fp32", n=8, M=5, temperature=0.7,
             mask="rows"),
        # a prompt's tokens scored, five alternatives each: bandwidth
        dict(name="logprobs_prompt", op="logprobs", T=4096, V=128256, dtype="bf16", n=1, M=5, temperature=1.0,
             mask="none"),
        # distillation on sixteen tokens a row of a small fp32 model
        dict(name="grad_sparse", op="grad", T=100, V=32003, dtype="fp32", n=16, entropy=False, temperature=2.0,
             mask="none"),
        # policy gradient with an entropy bonus over a batch of sampled answers
        dict(name="grad_policy", op="grad", T=4096, V=128256, dtype="bf16", n=1, entropy=True, temperature=1.0,
             mask="none"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["quantize", "lookup", "logits", "logits", "logprobs", "logprobs", "grad"])
    V = _log_int(rng, 1000, 262144)
    if op in ("logprobs", "grad"):
        c = dict(op=op, T=_log_int(rng, 1, 4096), V=V, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                 n=rng.choice([1, 1, 2, 8, 16, 64]), temperature=rng.choice([1.0, 1.0, 0.7, 2.0]),
                 mask=rng.choice(["none", "none", "shared", "rows"]))
        if op == "logprobs":
            return dict(c, M=rng.choice([0, 1, 5, 20, 64]))
        return dict(c, entropy=rng.random() < 0.5)
    # usual widths, and odd ones
    D = rng.choice([64, 128, 192, 256, 384, 512, 640, 768, 1024, 1280, 1536, 2048, 2560, 4096, 5120, 6144, 8192])
    if rng.random() < 0.3:
        D = _log_int(rng, 64, 8192) | 1
    c = dict(op=op, V=V, D=D, group=rng.choice([32, 64, 128]), scales=rng.choice(["fp16", "bf16", "fp32"]),
             zeros=rng.random() < 0.5)
    if op == "quantize":
        return dict(c, w=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "lookup":
        return dict(c, T=_log_int(rng, 1, 65536), out=rng.choice(["bf16", "fp16", "fp32"]),
                    scale=rng.choice([1.0, round(math.sqrt(D), 3)]), ignored=rng.choice([0.0, 0.02, 0.3]))
    x, out = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("bf16", "fp32")])
    return dict(c, T=_log_int(rng, 1, 512), x=x, out=out)


@functools.lru_cache(maxsize=None)
def _most(op):
    """The most that a listed case of this operator handles: bytes, operations, and what its state holds."""
    of = [c for c in listed() if c["op"] == op]
    return max(work(c)["bytes"] for c in of), max(work(c)["flops"] for c in of), max(_held(c) for c in of)


def _held(c):
    """Elements that a plain pass widens at once."""
    if c["op"] in ("logprobs", "grad"):
        return c["T"] * c["V"]
    return c["V"] * c["D"] if c["op"] != "lookup" else max(c["V"] * c["D"] // 2, c["T"] * c["D"])


def draw(rng):
    while True:
        c = _draw_once(rng)
        bytes_, flops, held = _most(c["op"])
        if work(c)["bytes"] <= bytes_ and work(c)["flops"] <= flops and _held(c) <= held:
            return c


# ------------------------------------------------------------------ inputs
def _frequent(shape, V, gen):
    """Token ids as text has them: the n-th most frequent about 1/n as often as the first."""
    u = torch.rand(shape, generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
    return (ids * 48271) % V if math.gcd(48271, V) == 1 else ids     # frequent ids are spread over the table


def _groups(c):
    return (c["D"] + c["group"] - 1) // c["group"]


def _table(c, gen):
    """A 4-bit table as a checkpoint holds it: rows of bytes padded to 16, scales and zeros [G, V padded to 16]."""
    V, D, G = c["V"], c["D"], _groups(c)
    values = torch.empty(V, (D + 31) // 32 * 16, dtype=torch.uint8, device="cuda")
    for r in range(0, V, 16384):        # weights are about normal: the middle of the range is the most frequent
        n = torch.randn(min(V, r + 16384) - r, values.shape[1], 2, generator=gen, device="cuda")
        q = (n * 2.6 + 8).round_().clamp_(0, 15).to(torch.uint8)
        values[r:r + 16384] = q[..., 0] | q[..., 1] << 4
    wide = (V + 15) // 16 * 16
    scales = (0.02 / 2.6 * (0.5 + torch.rand(G, wide, generator=gen, device="cuda"))).to(_TYPES[c["scales"]])[:, :V]
    zeros = None
    if c["zeros"]:
        zeros = torch.randint(6, 11, (G, wide), generator=gen, device="cuda", dtype=torch.uint8)[:, :V]
    return dict(values=values[:, :(D + 1) // 2], scales=scales, zeros=zeros)


def _logits(c, gen):
    T, V = c["T"], c["V"]
    z = torch.empty(T, V, device="cuda").normal_(0.0, 2.0, generator=gen)
    z -= torch.log1p(torch.arange(V, device="cuda"))[None] * 0.5         # frequent tokens first
    peaks = torch.randint(0, V, (T, 12), generator=gen, device="cuda")   # what the context suggests
    z.scatter_add_(1, peaks, torch.rand(T, 12, generator=gen, device="cuda") * 12)
    z = z.to(_TYPES[c["dtype"]])
    mask = None
    if c["mask"] != "none":
        rows, words = (T if c["mask"] == "rows" else 1), (V + 31) // 32
        mask = torch.randint(-2 ** 31, 2 ** 31, (rows, words), generator=gen, device="cuda", dtype=torch.int64).int()
        if c["mask"] == "rows" and T > 1:
            mask[T // 2] = 0                                             # a grammar with no way on
    tokens = _frequent((T, c["n"]), V, gen)
    tokens[:, 0] = peaks[:, 0]
    tokens = torch.where(torch.rand(T, c["n"], generator=gen, device="cuda") < 0.05, _IGNORE, tokens)
    return z, tokens, mask


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case=dict(c))
    if c["op"] == "quantize":
        w = torch.empty(c["V"], c["D"], device="cuda", dtype=_TYPES[c["w"]])
        s["weight"] = w.normal_(0.0, 0.02, generator=gen)
        s["ids"] = torch.arange(c["V"], device="cuda")
    elif c["op"] == "lookup":
        s["table"] = _table(c, gen)
        ids = _frequent((c["T"],), c["V"], gen)
        s["ids"] = torch.where(torch.rand(c["T"], generator=gen, device="cuda") < c["ignored"], _IGNORE, ids)
    elif c["op"] == "logits":
        s["table"] = _table(c, gen)
        s["x"] = torch.empty(c["T"], c["D"], device="cuda").normal_(0.0, 1.0, generator=gen).to(_TYPES[c["x"]])
    else:
        s["logits"], s["tokens"], s["mask"] = _logits(c, gen)
        if c["op"] == "grad":
            T = c["T"]
            s["grad_logp"] = torch.randn(T, c["n"], generator=gen, device="cuda")
            s["grad_entropy"] = torch.randn(T, generator=gen, device="cuda") * 0.1 if c["entropy"] else None
            # what the forward pass left
            lse, ent = [], []
            for r in range(0, T, 512):
                y = s["logits"][r:r + 512].double() / c["temperature"]
                if s["mask"] is not None:
                    y.masked_fill_(~_allowed(s["mask"][r:r + 512] if len(s["mask"]) > 1 else s["mask"], c["V"]), -math.inf)
                a = torch.logsumexp(y, 1)
                lse.append(a)
                ent.append(torch.special.entr(torch.exp(y - torch.where(a > -math.inf, a, 0.0)[:, None])).sum(1))
            s["lse"], s["entropy"] = torch.cat(lse).float(), torch.cat(ent).float()
            s["grad"] = torch.empty_like(s["logits"])
    return s


def _allowed(mask, V):
    bit = torch.arange(32, device="cuda", dtype=torch.int32)
    return ((mask[:, :, None] >> bit) & 1).flatten(1)[:, :V].bool()


# --------------------------------------------------------------- one pass
@functools.lru_cache(maxsize=None)
def _ops():
    from lm_head_vocab_gb300 import VocabOps
    return VocabOps(0, max_tokens=0, max_dim=8192, max_rows=4096)


def _own_table(s, c):
    from lm_head_vocab_gb300 import Table4
    t = s["table"]
    return Table4(t["values"], t["scales"], t["zeros"], c["D"], c["group"])


def run(state):
    c = state["case"]
    return {"quantize": _quantize, "lookup": _lookup, "logits": _product, "logprobs": _logprobs,
            "grad": _grad}[c["op"]](state, c)


def _values(t, c, rows):
    """The given rows of a table, in 32 bits."""
    b = t["values"][rows]
    q = torch.stack([b & 15, b >> 4], -1).flatten(1)[:, :c["D"]].float()
    scales = t["scales"][:, rows].float().t().repeat_interleave(c["group"], 1)[:, :c["D"]]
    zeros = 8.0
    if t["zeros"] is not None:
        zeros = t["zeros"][:, rows].float().t().repeat_interleave(c["group"], 1)[:, :c["D"]]
    return (q - zeros) * scales


def _quantize(s, c):
    """The weights in 4 bits, as the values that they stand for.  Without zeros: s = max |w| / 7,
    q = w / s rounded + 8; with zeros: s = (max - min) / 15 over the weights and 0, z = -min / s
    rounded, q = w / s rounded + z.  s is rounded to the scales' type first."""
    if own:
        ops = _ops()
        t = ops.quantize_table(s["weight"], group_size=c["group"], zeros=c["zeros"], scale_dtype=_TYPES[c["scales"]])
        return ops.table4_lookup(t, s["ids"], out_dtype=torch.float32)
    V, D, g = c["V"], c["D"], c["group"]
    w = torch.nn.functional.pad(s["weight"].float(), (0, _groups(c) * g - D)).view(V, -1, g)
    if c["zeros"]:
        lo, hi = w.amin(2, keepdim=True).clamp(max=0), w.amax(2, keepdim=True).clamp(min=0)
        scale = ((hi - lo) / torch.full_like(hi, 15)).to(_TYPES[c["scales"]])    # (a quotient: by a number it would be a product)
        by = torch.where(scale > 0, scale, 1.0).double()     # next to a border 32 bits would round a quotient
        z = (-lo.double() / by).round().clamp(0, 15)
        q = ((w.double() / by).round_() + z).clamp_(0, 15)
        q -= z
    else:
        most = w.abs().amax(2, keepdim=True)
        scale = (most / torch.full_like(most, 7)).to(_TYPES[c["scales"]])
        q = (w.double() / torch.where(scale > 0, scale, 1.0).double()).round_().clamp_(-8, 7)
    return (q.float() * scale.float()).view(V, -1)[:, :D].contiguous()


def _lookup(s, c):
    """out[t] = scale * the table's row ids[t], zeros where a position has no token"""
    if own:
        return _ops().table4_lookup(_own_table(s, c), s["ids"], scale=c["scale"], out_dtype=_TYPES[c["out"]])
    some = s["ids"] != _IGNORE
    rows = _values(s["table"], c, torch.where(some, s["ids"], 0)) * c["scale"]
    return torch.where(some[:, None], rows, 0.0).to(_TYPES[c["out"]])


def _product(s, c):
    """out[t, v] = x[t] . the table's row v"""
    if own:
        return _ops().table4_logits(_own_table(s, c), s["x"], out_dtype=_TYPES[c["out"]])
    return (s["x"].float() @ _values(s["table"], c, slice(None)).t()).to(_TYPES[c["out"]])


def _logprobs(s, c):
    """Each row's softmax over its allowed columns at a temperature: the given tokens' log-probabilities,
    the logsumexp, the entropy, and the M largest with their tokens, equal ones by token."""
    if own:
        r = _ops().token_logprobs(s["logits"], s["tokens"], num_top=c["M"], temperature=c["temperature"],
                                  token_mask=s["mask"])
        return (r.logp, r.lse, r.entropy) + ((r.top_logp, r.top_tokens) if c["M"] else ())
    z, M, t = s["logits"].float(), c["M"], c["temperature"]
    if s["mask"] is not None:
        z = torch.where(_allowed(s["mask"], c["V"]), z, -math.inf)
    y = z / t
    top = y.amax(1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    y = y - top
    e = torch.exp(y)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    some = s["tokens"] != _IGNORE
    logp = y.gather(1, torch.where(some, s["tokens"], 0)) - torch.where(total > 0, log_total, 0.0)
    logp = torch.where(some, logp, 0.0)
    entropy = log_total - (e * torch.where(e > 0, y, 0.0)).sum(1, keepdim=True) / total
    entropy = torch.where(total > 0, entropy, 0.0)
    out = (logp, (top + log_total)[:, 0], entropy[:, 0])
    if not M:
        return out
    # the M largest, equal values by their place: every value above the M-th largest, and the first of those equal to it
    least = z.topk(M, dim=1)[0][:, -1:]
    above, equal = z > least, z == least
    keep = above | (equal & (equal.cumsum(1) <= M - above.sum(1, keepdim=True)))
    place = keep.nonzero()[:, 1].view(-1, M)
    best, order = z.gather(1, place).sort(dim=1, descending=True, stable=True)
    place = place.gather(1, order)
    some = best > -math.inf
    return out + (torch.where(some, y.gather(1, place) - log_total, -math.inf), torch.where(some, place, _IGNORE))


def _grad(s, c):
    """The logits' gradient from those of the given tokens' log-probabilities and of the entropy."""
    if own:
        return _ops().token_logprobs_backward(s["logits"], s["lse"], s["tokens"], s["grad_logp"],
                                              entropy=s["entropy"] if c["entropy"] else None,
                                              grad_entropy=s["grad_entropy"], temperature=c["temperature"],
                                              token_mask=s["mask"], grad=s["grad"])
    y = s["logits"].float() / c["temperature"]
    may = None if s["mask"] is None else _allowed(s["mask"], c["V"])
    if may is not None:
        y = torch.where(may, y, -math.inf)
    lse = torch.where(s["lse"] > -math.inf, s["lse"], 0.0)[:, None]
    some = s["tokens"] != _IGNORE
    g = torch.where(some & (s["lse"] > -math.inf)[:, None], s["grad_logp"], 0.0)
    p = torch.exp(y - lse)
    by = g.sum(1, keepdim=True)
    if c["entropy"]:
        by = by + s["grad_entropy"][:, None] * (torch.where(p > 0, y - lse, 0.0) + s["entropy"][:, None])
    d = (-p * by).scatter_add_(1, torch.where(some, s["tokens"], 0), g)
    if may is not None:
        d = torch.where(may, d, 0.0)
    return s["grad"].copy_(d / c["temperature"])


# ---------------------------------------------------------------- the work
def work(case):
    c = case
    if c["op"] in ("logprobs", "grad"):
        T, V = c["T"], c["V"]
        mask = {"none": 0, "shared": 1, "rows": T}[c["mask"]] * ((V + 31) // 32) * 4
        z = T * V * _BYTES[c["dtype"]]
        if c["op"] == "logprobs":
            # a difference, an exponential, its sum and the sum of its products for each logit
            return {"bytes": z + mask + T * (c["n"] * 12 + 8 + c["M"] * 12), "flops": 5 * T * V}
        return {"bytes": 2 * z + mask + T * (c["n"] * 12 + 4 + (8 if c["entropy"] else 0)),
                "flops": (6 if c["entropy"] else 3) * T * V}
    V, D = c["V"], c["D"]
    side = _groups(c) * (_BYTES[c["scales"]] + (1 if c["zeros"] else 0))
    row = (D + 1) // 2 + side
    if c["op"] == "quantize":
        return {"bytes": V * (D * _BYTES[c["w"]] + 2 * row + 4 * D), "flops": 4 * V * D}
    if c["op"] == "lookup":
        return {"bytes": c["T"] * 8 + min(V, c["T"]) * row + c["T"] * D * _BYTES[c["out"]], "flops": 2 * c["T"] * D}
    T = c["T"]
    return {"bytes": V * row + T * D * _BYTES[c["x"]] + T * V * _BYTES[c["out"]], "flops": 2 * T * V * D}


# ------------------------------------------------- the definitions, in 64 bits
def _table64(t, c, rows):
    n = t["values"][rows].shape[0]
    out = torch.empty(n, c["D"], dtype=torch.float64, device="cuda")
    out[:, 0::2] = (t["values"][rows] % 16).double()[:, :out[:, 0::2].shape[1]]
    out[:, 1::2] = torch.div(t["values"][rows], 16, rounding_mode="floor").double()[:, :out[:, 1::2].shape[1]]
    for k in range(_groups(c)):
        part = out[:, k * c["group"]:(k + 1) * c["group"]]
        part -= 8.0 if t["zeros"] is None else t["zeros"][k, rows].double()[:, None]
        part *= t["scales"][k, rows].double()[:, None]
    return out


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "quantize":
        out = torch.empty(c["V"], c["D"], dtype=torch.float64, device="cuda")
        for k in range(_groups(c)):
            w = s["weight"][:, k * c["group"]:(k + 1) * c["group"]]
            if c["zeros"]:
                hi = torch.maximum(w.float().max(1)[0], torch.zeros(1, device="cuda"))
                lo = torch.minimum(w.float().min(1)[0], torch.zeros(1, device="cuda"))
                scale = ((hi - lo).double() / 15).float().to(_TYPES[c["scales"]]).double()[:, None]
                by = scale.masked_fill(scale == 0, 1.0)
                z = torch.round(-lo.double()[:, None] / by).clamp(0, 15)
                q = torch.minimum(torch.maximum(torch.round(w.double() / by), -z), 15 - z)
            else:
                scale = (w.double().abs().max(1)[0] / 7).float().to(_TYPES[c["scales"]]).double()[:, None]
                q = torch.round(w.double() / scale.masked_fill(scale == 0, 1.0)).clamp(-8, 7)
            out[:, k * c["group"]:(k + 1) * c["group"]] = q * scale
        return out
    if c["op"] == "lookup":
        ids = s["ids"].cpu().numpy()
        rows = torch.from_numpy(np.where(ids < 0, 0, ids)).cuda()
        gone = torch.from_numpy(ids < 0).cuda()
        return (_table64(s["table"], c, rows) * c["scale"]).masked_fill_(gone[:, None], 0.0)
    if c["op"] == "logits":
        x = s["x"].double()
        out = torch.empty(c["T"], c["V"], dtype=torch.float64, device="cuda")
        for r in range(0, c["V"], 16384):
            rows = slice(r, min(c["V"], r + 16384))
            out[:, rows] = torch.matmul(_table64(s["table"], c, rows), x.t()).t()
        return out
    bits = None
    if s["mask"] is not None:
        words = s["mask"].cpu().numpy().view(np.uint8)
        bits = torch.from_numpy(np.unpackbits(words, axis=1, bitorder="little")[:, :c["V"]].astype(bool)).cuda()
    parts = []
    for r in range(0, c["T"], 256):
        rows = slice(r, r + 256)
        y = s["logits"][rows].double() / c["temperature"]
        if bits is not None:
            y.masked_fill_(~(bits if len(bits) == 1 else bits[rows]), -math.inf)
        tokens = s["tokens"][rows]
        gone = tokens < 0
        empty = ~(y > -math.inf).any(1)
        if c["op"] == "logprobs":
            lse = torch.logsumexp(y, 1)
            lp = torch.where(empty[:, None], -math.inf, torch.log_softmax(y, 1))
            entropy = torch.special.entr(lp.exp()).sum(1)
            part = [lp.gather(1, tokens.masked_fill(gone, 0)).masked_fill_(gone, 0.0), lse, entropy]
            if c["M"]:
                part.append(lp.sort(dim=1, descending=True)[0][:, :c["M"]])
        else:
            p = torch.exp(y - s["lse"][rows].double()[:, None]).masked_fill_(empty[:, None], 0.0)
            g = s["grad_logp"][rows].double().masked_fill(gone | empty[:, None], 0.0)
            d = -p * g.sum(1, keepdim=True)
            if c["entropy"]:
                each = -torch.special.entr(p) + p * s["entropy"][rows].double()[:, None]
                d -= s["grad_entropy"][rows].double()[:, None] * each
            d.scatter_add_(1, tokens.masked_fill(gone, 0), g)
            if bits is not None:
                d.masked_fill_(~(bits if len(bits) == 1 else bits[rows]), 0.0)
            part = [d / c["temperature"]]
        parts.append(part)
    out = [torch.cat(x) for x in zip(*parts)]
    if c["op"] == "grad":
        return out[0]
    return tuple(out) + ((None,) if c["M"] else ())
