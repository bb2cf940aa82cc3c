"""The vocabulary operators' measured cases: embedding lookup and its gradient
at the input end of the vocabulary, the beam step and the reordering of beam
states at its output end.

`run` takes one pass: with `own` false in plain torch operations, with `own`
true through `lm_head_vocab_gb300.VocabOps`, on the inputs that `prepare` made.
`exact` gives the same outputs from the definitions in 64 bits.
"""
import functools
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "int64": torch.int64, "int32": torch.int32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "int64": 8, "int32": 4}
_IGNORE = -100


def listed():
    return [
        # the embeddings of one decoding step for a batch of eight sequences
        dict(name="embed_step", op="embed", T=8, V=128256, D=4096, w="bf16", out="bf16", ids="int64",
             scale=64.0, ignored=0.0),
        # packed training rows: fp32 master weights looked up into bf16 activations, one row short
        # of a round count, some positions without a token
        dict(name="embed_packed", op="embed", T=32767, V=151936, D=2048, w="fp32", out="bf16", ids="int32",
             scale=45.25, ignored=0.02),
        # the gradient in a small fp32 model's step
        dict(name="grad_small", op="grad", T=64, V=1024, D=512, g="fp32", out="fp32", ids="int64",
             scale=1.0, ignored=0.0, accumulate=False),
        # a table tied to the LM head: added to the head's fp32 weight gradient
        dict(name="grad_tied", op="grad", T=16384, V=128256, D=4096, g="bf16", out="fp32", ids="int64",
             scale=64.0, ignored=0.02, accumulate=True),
        # the largest batch and vocabulary: a whole bf16 gradient is written, most of it zeros
        dict(name="grad_whole", op="grad", T=65536, V=262144, D=2048, g="bf16", out="bf16", ids="int64",
             scale=1.0, ignored=0.02, accumulate=False),
        # odd width, odd counts: rows that start at no vector boundary
        dict(name="grad_ragged", op="grad", T=4097, V=32003, D=1001, g="bf16", out="bf16", ids="int32",
             scale=31.6, ignored=0.1, accumulate=False),
        # one sequence, four beams, candidates for beams that may end: latency
        dict(name="beam_one", op="beam", B=1, K=4, M=8, V=128256, dtype="bf16", finished=False, alpha=0.0,
             mask="none"),
        # constrained decoding in fp32 at an odd vocabulary: a mask for every row (one row allows nothing),
        # ended beams, scores normalised by length
        dict(name="beam_masked", op="beam", B=12, K=5, M=5, V=32003, dtype="fp32", finished=True, alpha=0.6,
             mask="rows"),
        # a full batch at the largest vocabulary: bandwidth
        dict(name="beam_batch", op="beam", B=64, K=8, M=16, V=262144, dtype="bf16", finished=False, alpha=0.0,
             mask="none"),
        # token histories of a few beams
        dict(name="reorder_history", op="reorder", B=8, K=4, kind="history", layers=1, heads=1, length=513,
             valid=211, width=1, survivors=3, inplace=False),
        # key/value caches of four layers copied into the other half of a double buffer
        dict(name="reorder_cache", op="reorder", B=8, K=8, kind="cache", layers=4, heads=8, length=2048,
             valid=1531, width=128, survivors=5, inplace=False),
        # the same in place, where the surviving beams keep their slots
        dict(name="reorder_inplace", op="reorder", B=16, K=4, kind="cache", layers=2, heads=4, length=1024,
             valid=777, width=80, survivors=2, inplace=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["embed", "grad", "beam", "reorder"])
    if op in ("embed", "grad"):
        # usual widths, and odd ones
        D = rng.choice([64, 128, 192, 256, 384, 512, 640, 768, 1024, 1280, 1536, 2048, 2560, 4096, 5120, 6144, 8192])
        if rng.random() < 0.4:
            D = _log_int(rng, 64, 8192) | 1
        c = dict(op=op, T=_log_int(rng, 1, 65536), V=_log_int(rng, 1000, 262144), D=D,
                 ids=rng.choice(["int64", "int32"]), scale=rng.choice([1.0, round(math.sqrt(D), 3)]),
                 ignored=rng.choice([0.0, 0.02, 0.3]))
        a, b = rng.choice([("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "fp16")]
                          + ([("fp32", "bf16"), ("bf16", "fp32"), ("fp32", "fp16")] if op == "embed"
                             else [("bf16", "fp32"), ("fp16", "fp32")]))
        if op == "embed":
            return dict(c, w=a, out=b)
        return dict(c, g=a, out=b, accumulate=rng.random() < 0.5)
    if op == "beam":
        K = rng.randint(1, 16)
        return dict(op=op, B=_log_int(rng, 1, 64), K=K, M=rng.choice([K, 2 * K]), V=_log_int(rng, 1000, 262144),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), finished=rng.random() < 0.5,
                    alpha=rng.choice([0.0, 0.0, 0.6, 1.0]), mask=rng.choice(["none", "shared", "rows"]))
    K = rng.randint(2, 16)
    s = rng.randint((K + 1) // 2, K)
    if rng.random() < 0.3:
        n = _log_int(rng, 16, 8192)
        return dict(op=op, B=_log_int(rng, 1, 64), K=K, kind="history", layers=1, heads=1, length=n,
                    valid=rng.randint(1, n), width=1, survivors=s, inplace=rng.random() < 0.5)
    n = _log_int(rng, 64, 4096)
    return dict(op=op, B=_log_int(rng, 1, 32), K=K, kind="cache", layers=rng.randint(1, 4), heads=rng.randint(1, 8),
                length=n, valid=rng.randint(1, n), width=rng.choice([64, 80, 96, 128]),
                survivors=min(s, K - 1), inplace=rng.random() < 0.5)


@functools.lru_cache(maxsize=None)
def _most(op):
    """The most that a listed case of this operator handles: what a pass moves, and what its state holds."""
    of = [c for c in listed() if c["op"] == op]
    return max(work(c)["bytes"] for c in of), max(_held(c) for c in of)


def _held(c):
    if c["op"] in ("embed", "grad"):
        return c["V"] * c["D"] * _BYTES[c["out" if c["op"] == "grad" else "w"]] + c["T"] * c["D"] * 2
    if c["op"] == "beam":
        return c["B"] * c["K"] * c["V"] * 4
    return 2 * c["layers"] * c["B"] * c["K"] * c["heads"] * c["length"] * c["width"] * 2


def draw(rng):
    while True:
        c = _draw_once(rng)
        bytes_, held = _most(c["op"])
        if work(c)["bytes"] <= bytes_ and _held(c) <= held:
            return c


# ------------------------------------------------------------------ inputs
def _tokens(c, gen):
    """Token ids as text has them: the n-th most frequent about 1/n as often as the first, and some
    positions (padding, other modalities) without a token."""
    u = torch.rand(c["T"], generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(c["V"] + 1)) - 1).long().clamp_(0, c["V"] - 1)
    ids = (ids * 48271) % c["V"] if math.gcd(48271, c["V"]) == 1 else ids     # frequent ids are spread over the table
    gone = torch.rand(c["T"], generator=gen, device="cuda") < c["ignored"]
    return torch.where(gone, _IGNORE, ids).to(_TYPES[c["ids"]])


def _distinct(c):
    """Different tokens expected among the T drawn."""
    n = np.arange(1, c["V"] + 1, dtype=np.float64)
    p = np.log1p(1 / n) / math.log(c["V"] + 1)
    return float(-np.expm1(c["T"] * (1 - c["ignored"]) * np.log1p(-p)).sum())


def _parents(c, gen):
    """[B, K] int32: which beam each new beam continues.  `survivors` of the K old beams live on; with
    `inplace` they keep their slots and the other slots take copies of different survivors."""
    B, K, s = c["B"], c["K"], c["survivors"]
    order = torch.rand(B, K, generator=gen, device="cuda").argsort(1)
    live = order[:, :s]
    if c["inplace"]:
        parents = torch.arange(K, device="cuda").repeat(B, 1)
        return parents.scatter_(1, order[:, s:], live[:, :K - s]).int()
    more = torch.randint(0, s, (B, K - s), generator=gen, device="cuda")
    parents = torch.cat([live, live.gather(1, more)], 1)
    return parents.gather(1, torch.rand(B, K, generator=gen, device="cuda").argsort(1)).int()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape, dtype, std=1.0):
        t = torch.empty(shape, device="cuda", dtype=_TYPES[dtype])
        return t.normal_(0.0, std, generator=gen)

    s = dict(case=dict(c))
    if c["op"] == "embed":
        s.update(weight=normal(c["V"], c["D"], dtype=c["w"], std=0.02), ids=_tokens(c, gen))
    elif c["op"] == "grad":
        s.update(grad=normal(c["T"], c["D"], dtype=c["g"], std=1e-2), ids=_tokens(c, gen))
        if c["accumulate"]:
            s["total"] = normal(c["V"], c["D"], dtype=c["out"], std=1e-2)
        else:
            s["total"] = torch.empty(c["V"], c["D"], device="cuda", dtype=_TYPES[c["out"]])
    elif c["op"] == "beam":
        B, K, V, N = c["B"], c["K"], c["V"], c["B"] * c["K"]
        z = normal(N, V, dtype="fp32", std=2.0)
        z -= torch.log1p(torch.arange(V, device="cuda"))[None] * 0.5         # frequent tokens first
        peaks = torch.randint(0, V, (N, 12), generator=gen, device="cuda")   # what the context suggests
        z.scatter_add_(1, peaks, torch.rand(N, 12, generator=gen, device="cuda") * 12)
        s["logits"] = z.to(_TYPES[c["dtype"]])
        del z
        s["scores"] = -20 * torch.rand(B, K, generator=gen, device="cuda").sort(1)[0]
        if K > 1:
            s["scores"][::7, 1:] = -math.inf                                 # sequences at their first step
        s["finished"] = s["lengths"] = s["token_mask"] = None
        if c["finished"]:
            s["finished"] = (torch.rand(B, K, generator=gen, device="cuda") < 0.2).to(torch.uint8)
        if c["alpha"]:
            s["lengths"] = torch.randint(1, 200, (B, K), generator=gen, device="cuda", dtype=torch.int32)
        if c["mask"] != "none":
            rows, words = (N if c["mask"] == "rows" else 1), (V + 31) // 32
            m = torch.randint(-2 ** 31, 2 ** 31, (rows, words), generator=gen, device="cuda", dtype=torch.int64)
            if c["mask"] == "rows":
                m &= torch.randint(-2 ** 31, 2 ** 31, (rows, words), generator=gen, device="cuda", dtype=torch.int64)
                m[N // 2] = 0                                                # a grammar with no way on
            s["token_mask"] = m.int()
    else:
        s["parents"] = _parents(c, gen)
        N = c["B"] * c["K"]
        if c["kind"] == "history":
            # token histories beside a row of running statistics
            states = [torch.randint(0, 32000, (N, c["length"]), generator=gen, device="cuda"),
                      normal(N, 33, dtype="fp32")]
            s["states"] = [states[0][:, :c["valid"]], states[1]]
            s["dim"] = 0
        else:
            # keys and values of all layers, the positions written so far
            kv = normal(2 * c["layers"], N, c["heads"], c["length"], c["width"], dtype="bf16")
            s["states"] = [kv[:, :, :, :c["valid"]]]
            s["dim"] = 1
        s["out"] = s["states"]
        if not c["inplace"]:
            # the other half of the double buffer, of the same layout
            s["out"] = [torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda") for t in s["states"]]
    return s


# --------------------------------------------------------------- one pass
@functools.lru_cache(maxsize=None)
def _ops():
    from lm_head_vocab_gb300 import VocabOps
    return VocabOps(0, max_tokens=65536, max_dim=8192, max_rows=1024)


def run(state):
    c = state["case"]
    return {"embed": _embed, "grad": _grad, "beam": _beam, "reorder": _reorder}[c["op"]](state, c)


def _embed(s, c):
    """out[t] = scale * weight[ids[t]], zeros where a position has no token"""
    if own:
        return _ops().embedding_forward(s["weight"], s["ids"], scale=c["scale"], out_dtype=_TYPES[c["out"]])
    ids = s["ids"].long()
    some = ids != _IGNORE
    rows = s["weight"][torch.where(some, ids, 0)].float() * c["scale"]
    return torch.where(some[:, None], rows, 0.0).to(_TYPES[c["out"]])


def _grad(s, c):
    """total[v] (+)= scale * the sum of grad[t] over the positions t that hold token v"""
    if own:
        return _ops().embedding_backward(s["grad"], s["ids"], s["total"], scale=c["scale"],
                                         accumulate=c["accumulate"])
    ids = s["ids"].long()
    some = ids != _IGNORE
    rows = torch.where(some[:, None], s["grad"].float(), 0.0)
    sums = torch.zeros(c["V"], c["D"], device="cuda").index_add_(0, torch.where(some, ids, 0), rows)
    sums *= c["scale"]
    if c["accumulate"]:
        sums += s["total"].float()
    return s["total"].copy_(sums)


def _beam(s, c):
    """The M best continuations of each sequence's K beams: the beam's score plus the token's
    log-probability, over all tokens of all beams; equal ones by beam, then by token."""
    if own:
        r = _ops().beam_step(s["logits"], s["scores"], num_candidates=c["M"], finished=s["finished"], eos_token=2,
                             lengths=s["lengths"], length_penalty=c["alpha"], token_mask=s["token_mask"])
        return r.scores, r.parents, r.tokens, r.lse, r.finished, r.lengths
    B, K, M, V = c["B"], c["K"], c["M"], c["V"]
    z = s["logits"].double()
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    z -= lse
    z += s["scores"].double().view(-1, 1)
    z = torch.where(torch.isfinite(z), z, -math.inf)
    if s["token_mask"] is not None:
        bit = torch.arange(32, device="cuda", dtype=torch.int32)
        may = ((s["token_mask"][:, :, None] >> bit) & 1).flatten(1)[:, :V]
        z = torch.where(may.bool(), z, -math.inf)
    z = z.view(B, K, V)
    done = torch.zeros(B, K, dtype=torch.bool, device="cuda") if s["finished"] is None else s["finished"].bool()
    if s["finished"] is not None:       # an ended beam goes on as it is, with its end token
        stay = torch.full((B, K, V), -math.inf, device="cuda", dtype=torch.float64)
        stay[:, :, 2] = s["scores"].double()
        z = torch.where(done[:, :, None], stay, z)
    key = z
    if s["lengths"] is not None:
        new = s["lengths"] + (~done).int()
        key = z / new.clamp(min=1).double()[:, :, None] ** c["alpha"]
    key = key.reshape(B, K * V)
    # the M largest, equal values by their place: every value above the M-th largest, and the first of those equal to it
    least = key.topk(M, dim=1)[0][:, -1:]
    above, equal = key > least, key == least
    keep = above | (equal & (equal.cumsum(1) <= M - above.sum(1, keepdim=True)))
    place = keep.nonzero()[:, 1].view(B, M)
    best, order = key.gather(1, place).sort(dim=1, descending=True, stable=True)
    place = place.gather(1, order)
    some = best > -math.inf
    scores = z.reshape(B, K * V).gather(1, place).float()
    parents = torch.where(some, place // V, torch.arange(M, device="cuda") % K)
    tokens = torch.where(some, place % V, _IGNORE)
    ended = done.gather(1, parents)
    lengths = None
    if s["lengths"] is not None:
        lengths = s["lengths"].gather(1, parents) + (some & ~ended).int()
    lse = torch.where(done, 0.0, lse.view(B, K)).float()
    return scores, parents.int(), tokens, lse, (some & (ended | (tokens == 2))).to(torch.uint8), lengths


def _reorder(s, c):
    """new beam k of sequence b continues old beam parents[b, k]: every state's rows follow"""
    if own:
        return _ops().beam_reorder(s["states"], s["parents"], out=s["out"], dim=s["dim"])
    rows = (s["parents"] + torch.arange(c["B"], device="cuda")[:, None] * c["K"]).flatten().long()
    return [o.copy_(t.index_select(s["dim"], rows)) for t, o in zip(s["states"], s["out"])]


# ---------------------------------------------------------------- the work
def work(case):
    c = case
    if c["op"] == "embed":
        return {"bytes": c["T"] * _BYTES[c["ids"]] + _distinct(c) * c["D"] * _BYTES[c["w"]]
                + c["T"] * c["D"] * _BYTES[c["out"]], "flops": c["T"] * c["D"]}
    if c["op"] == "grad":
        n = c["T"] * (1 - c["ignored"]) * c["D"]
        rows = 2 * _distinct(c) if c["accumulate"] else c["V"]
        return {"bytes": c["T"] * _BYTES[c["ids"]] + n * _BYTES[c["g"]] + rows * c["D"] * _BYTES[c["out"]], "flops": n}
    if c["op"] == "beam":
        N = c["B"] * c["K"]
        mask = {"none": 0, "shared": 1, "rows": N}[c["mask"]] * ((c["V"] + 31) // 32) * 4
        # a difference, an exponential and a sum for each logit
        return {"bytes": N * c["V"] * _BYTES[c["dtype"]] + mask + N * 17 + c["B"] * c["M"] * 21, "flops": 3 * N * c["V"]}
    K, s = c["K"], c["survivors"]
    row = c["valid"] * 8 + 33 * 4 if c["kind"] == "history" else 2 * c["layers"] * c["heads"] * c["valid"] * c["width"] * 2
    rows = 2 * (K - s) if c["inplace"] else s + K
    return {"bytes": c["B"] * (rows * row + 4 * K), "flops": 0}


# ------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "embed":
        ids = s["ids"].cpu().tolist()
        table = torch.cat([s["weight"].double() * c["scale"], torch.zeros(1, c["D"], device="cuda").double()])
        return torch.index_select(table, 0, torch.tensor([v if v >= 0 else c["V"] for v in ids], device="cuda"))
    if c["op"] == "grad":
        # positions ordered by token; each token's sum is a difference of running sums
        ids, order = s["ids"].long().sort(stable=True)
        last = torch.ones_like(ids, dtype=torch.bool)
        last[:-1] = ids[1:] != ids[:-1]
        ends = last.nonzero()[:, 0]
        total = s["total"].double() if c["accumulate"] else torch.zeros(c["V"], c["D"], device="cuda").double()
        held = ids[ends]
        for d in range(0, c["D"], 512):
            run_ = s["grad"][:, d:d + 512][order].double().cumsum(0)[ends]
            sums = torch.diff(run_, dim=0, prepend=torch.zeros_like(run_[:1]))
            total[held[held >= 0], d:d + 512] += sums[held >= 0] * c["scale"]
        return total
    if c["op"] == "beam":
        scores = []
        for b in range(c["B"]):
            z = s["logits"].view(c["B"], c["K"], c["V"])[b].double()
            z = torch.log_softmax(z, 1) + s["scores"][b].double()[:, None]
            z[~torch.isfinite(z)] = -math.inf
            if s["token_mask"] is not None:
                words = s["token_mask"].cpu().numpy().view(np.uint8)
                bits = np.unpackbits(words, axis=1, bitorder="little")[:, :c["V"]].astype(bool)
                bits = bits if len(bits) == 1 else bits[b * c["K"]:(b + 1) * c["K"]]
                z.masked_fill_(torch.from_numpy(~bits).cuda(), -math.inf)
            steps = torch.ones(c["K"], dtype=torch.float64, device="cuda")
            if s["finished"] is not None:
                for k in s["finished"][b].nonzero()[:, 0].tolist():
                    z[k] = -math.inf
                    z[k, 2] = s["scores"][b, k].double()
                    steps[k] = 0
            by = z
            if s["lengths"] is not None:
                by = z / (s["lengths"][b].double() + steps)[:, None] ** c["alpha"]
            by, at = by.flatten().sort(descending=True, stable=True)
            scores.append(z.flatten()[at[:c["M"]]])
        lse = torch.logsumexp(s["logits"].double(), 1).view(c["B"], c["K"])
        if s["finished"] is not None:
            lse[s["finished"].bool()] = 0.0
        return torch.stack(scores), None, None, lse, None, None
    # copies: whole values for histories, the values themselves for floating states
    out = []
    for t in s["states"]:
        t = t.movedim(s["dim"], 0)
        p = s["parents"].long()
        n = torch.stack([t.unflatten(0, (c["B"], c["K"]))[b][p[b]] for b in range(c["B"])]).flatten(0, 1)
        out.append(n.movedim(0, s["dim"]) if n.is_floating_point() else None)
    return [None if t is None else t.double() for t in out]
