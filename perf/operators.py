"""Cases of the token operators: embedding lookup and its gradient, next-token cross entropy and its
gradient, and sampling of the next token ID.

``run`` computes them in plain torch operations, or, where ``own`` is true, calls the package's entry
points.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
# ID counts of the vocabularies in workloads/vocabs: 256 bytes + 1,000 / 32,768 / 131,072 merges
V1, V2, V3 = 1256, 33024, 131328


def listed():
    return [
        # one decode step: the last sampled IDs of 16 sequences
        dict(name="embed decode 16", op="embed", tokens=16, vocab=V2, dim=2048, table="bf16", out="bf16",
             scale=45.25, pad=0.0),
        # prefill / training forward of a packed batch
        dict(name="embed batch 16384", op="embed", tokens=16384, vocab=V3, dim=4096, table="bf16", out="bf16",
             scale=1.0, pad=0.0),
        # float32 master table read into bfloat16 activations; odd width, padded sequences
        dict(name="embed odd f32", op="embed", tokens=5001, vocab=V1, dim=1001, table="f32", out="bf16",
             scale=31.625, pad=0.1),
        # gradient of a small model's table: few tokens, small vocabulary
        dict(name="embed grad small", op="embed_grad", tokens=777, vocab=V1, dim=320, grad="f16", out="f32",
             scale=1.0, pad=0.05, accumulate=False),
        # dense gradient of a large table from one packed batch: most rows are zeros
        dict(name="embed grad dense", op="embed_grad", tokens=8192, vocab=V3, dim=2048, grad="bf16", out="bf16",
             scale=1.0, pad=0.0, accumulate=False),
        # gradient accumulation over microbatches into the optimiser's float32 buffer (a tied table)
        dict(name="embed grad accumulate", op="embed_grad", tokens=65536, vocab=V3, dim=4096, grad="bf16",
             out="f32", scale=64.0, pad=0.01, accumulate=True),
        # loss and gradient of a small model's batch
        dict(name="loss small f32", op="loss", rows=256, vocab=V1, pad_cols=0, type="f32", ignore=0.1,
             masked=False, fused=True),
        # one training step's logits: 8,192 positions over the largest vocabulary
        dict(name="loss train 8192", op="loss", rows=8192, vocab=V3, pad_cols=0, type="bf16", ignore=0.02,
             masked=False, fused=True),
        # odd vocabulary in padded rows, reserved IDs masked, loss first and gradient later
        dict(name="loss odd f16 two calls", op="loss", rows=1500, vocab=33001, pad_cols=23, type="f16",
             ignore=0.1, masked=True, fused=False),
        # one chat sequence: temperature, top-k and top-p
        dict(name="sample one", op="sample", rows=1, vocab=V3, pad_cols=0, type="bf16", mode="chat", mask=False),
        # a serving batch whose requests each bring their own settings
        dict(name="sample batch 256", op="sample", rows=256, vocab=V3, pad_cols=0, type="bf16", mode="mixed",
             mask=False),
        # rollouts from the full distribution under a mask of allowed IDs
        dict(name="sample masked f32", op="sample", rows=24, vocab=V2, pad_cols=8, type="f32", mode="free",
             mask=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "loss", "sample"])
    vocab = rng.choice([V1, V2, V3, _log_int(rng, 260, V3)])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "embed":
        return dict(op=op, tokens=_log_int(rng, 1, 16384), vocab=vocab, dim=_log_int(rng, 64, 4096), table=kind,
                    out=rng.choice([kind, "bf16"]), scale=rng.choice([1.0, 22.625]), pad=rng.choice([0.0, 0.1]))
    if op == "embed_grad":
        return dict(op=op, tokens=_log_int(rng, 1, 65536), vocab=vocab, dim=_log_int(rng, 64, 2048), grad=kind,
                    out=rng.choice([kind, "f32"]), scale=rng.choice([1.0, 22.625]), pad=rng.choice([0.0, 0.1]),
                    accumulate=rng.random() < 0.4)
    if op == "loss":
        rows = _log_int(rng, 1, 4096)
        return dict(op=op, rows=rows, vocab=vocab, pad_cols=rng.choice([0, 0, 1, 56]), type=kind,
                    ignore=rng.choice([0.0, 0.2]), masked=rng.random() < 0.3, fused=rng.random() < 0.6)
    return dict(op=op, rows=_log_int(rng, 1, 256), vocab=vocab, pad_cols=rng.choice([0, 0, 3, 64]), type=kind,
                mode=rng.choice(["chat", "mixed", "free", "greedy"]), mask=rng.random() < 0.3)


# ---------------------------------------------------------------------------------------------
# inputs

def _ids(gen, n, vocab, pad):
    """Token IDs with the skew of text (log-uniform over the vocabulary: byte and early merge IDs are the
    frequent ones); a share `pad` of them names no row (-1)."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).floor().clamp_(0, vocab - 1).to(torch.int32)
    if pad:
        ids[torch.rand(n, generator=gen, device="cuda") < pad] = -1
    return ids


def _rows(gen, rows, vocab, pad_cols, kind, make):
    full = torch.empty(rows, vocab + pad_cols, dtype=DTYPES[kind], device="cuda")
    step = max(1, (1 << 27) // max(vocab, 1))
    for r in range(0, rows, step):
        full[r:r + step, :vocab] = make(min(step, rows - r))
    if pad_cols:
        full[:, vocab:] = 100.0    # what lies beyond a row's logits is not the row's
    return full[:, :vocab]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    c = case
    s = dict(case=dict(case))
    if c["op"] == "embed":
        s["table"] = torch.randn(c["vocab"], c["dim"], generator=gen, device=dev).to(DTYPES[c["table"]])
        s["ids"] = _ids(gen, c["tokens"], c["vocab"], c["pad"])
        s["out"] = torch.empty(c["tokens"], c["dim"], dtype=DTYPES[c["out"]], device=dev)
    elif c["op"] == "embed_grad":
        s["grad"] = (torch.randn(c["tokens"], c["dim"], generator=gen, device=dev) * 0.05).to(DTYPES[c["grad"]])
        s["ids"] = _ids(gen, c["tokens"], c["vocab"], c["pad"])
        s["out"] = torch.empty(c["vocab"], c["dim"], dtype=DTYPES[c["out"]], device=dev)
        if c["accumulate"]:
            s["out"].normal_(generator=gen)
    elif c["op"] == "loss":
        rows, vocab = c["rows"], c["vocab"]
        s["logits"] = _rows(gen, rows, vocab, c["pad_cols"], c["type"],
                            lambda k: 2.5 * torch.randn(k, vocab, generator=gen, device=dev))
        s["targets"] = _ids(gen, rows, vocab, c["ignore"])
        at = s["targets"].clamp(min=0).long().unsqueeze(1)
        lift = 9.0 * torch.rand(rows, 1, generator=gen, device=dev)
        s["logits"].scatter_(1, at, (s["logits"].gather(1, at).float() + lift).to(DTYPES[c["type"]]))
        if c["masked"]:
            s["logits"][:, vocab - max(1, vocab // 50):] = -math.inf   # reserved IDs
            s["logits"][::97] = -math.inf                              # rows that the mask leaves empty
        s["grad_loss"] = torch.rand(rows, generator=gen, device=dev) / rows
        s["loss"] = torch.empty(rows, device=dev)
        s["lse"] = torch.empty(rows, device=dev)
        s["grad"] = torch.empty(rows, vocab, dtype=DTYPES[c["type"]], device=dev)
    else:
        rows, vocab = c["rows"], c["vocab"]

        def logits(k):   # a power law over ranks, as next-token distributions have, with noise
            u = torch.rand(k, vocab, generator=gen, device=dev)
            return 12.0 - 1.25 * torch.log1p(u * vocab) + 0.3 * torch.randn(k, vocab, generator=gen, device=dev)

        s["logits"] = _rows(gen, rows, vocab, c["pad_cols"], c["type"], logits)
        s["uniform"] = torch.rand(rows, generator=gen, device=dev)

        def pick(values, dtype):
            v = torch.tensor(values, dtype=dtype, device=dev)
            return v[torch.randint(len(values), (rows,), generator=gen, device=dev)].contiguous()

        f, i = torch.float32, torch.int32
        settings = {
            "chat": ([0.7], [50], [0.95], [0.0]),
            "mixed": ([0.0, 0.3, 0.7, 0.9, 1.0, 1.3], [0, 0, 1, 20, 64, 200, 1000], [0.5, 0.8, 0.9, 0.95, 1.0],
                      [0.0, 0.0, 0.02, 0.1]),
            "free": ([1.0], [0], [1.0], [0.0]),
            "greedy": ([0.0], [0], [1.0], [0.0]),
        }[c["mode"]]
        s["temperature"], s["top_k"] = pick(settings[0], f), pick(settings[1], i)
        s["top_p"], s["min_p"] = pick(settings[2], f), pick(settings[3], f)
        s["mask"] = None
        if c["mask"]:
            words = -(-vocab // 32)
            s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (rows, words), generator=gen, device=dev,
                                      dtype=torch.int64).to(torch.int32)
            s["mask"][::13] &= 1 << 4    # a grammar that leaves few IDs
            s["mask"][5::29] = 0         # and one that leaves none
        s["out_ids"] = torch.empty(rows, dtype=i, device=dev)
        s["out_logprobs"] = torch.empty(rows, dtype=f, device=dev)
    return s


# ---------------------------------------------------------------------------------------------
# one pass

def run(state):
    op = state["case"]["op"]
    return (_run_own if own else _run_plain)[op](state)


def _workspace(state, need):
    """The workspace that a program keeps beside its buffers."""
    if "workspace" not in state:
        state["workspace"] = torch.empty(max(need(), 1), dtype=torch.uint8, device="cuda")
    return state["workspace"]


def _own_embed(s):
    import exact_bpe_tokenization_amd as tt
    tt.toktier_embed(s["table"], s["ids"], s["out"], scale=s["case"]["scale"])
    return s["out"]


def _own_embed_grad(s):
    import exact_bpe_tokenization_amd as tt
    c = s["case"]
    ws = _workspace(s, lambda: tt.toktier_embed_backward_workspace_bytes(c["tokens"], c["vocab"], c["dim"]))
    tt.toktier_embed_backward(s["grad"], s["ids"], s["out"], ws, scale=c["scale"], accumulate=c["accumulate"])
    return s["out"]


def _own_loss(s):
    import exact_bpe_tokenization_amd as tt
    c = s["case"]
    ws = _workspace(s, lambda: tt.toktier_cross_entropy_workspace_bytes(c["rows"], c["vocab"]))
    if c["fused"]:
        tt.toktier_cross_entropy(s["logits"], s["targets"], s["loss"], s["lse"], ws, grad_logits=s["grad"],
                                 grad_loss=s["grad_loss"])
    else:
        tt.toktier_cross_entropy(s["logits"], s["targets"], s["loss"], s["lse"], ws)
        tt.toktier_cross_entropy_backward(s["logits"], s["targets"], s["lse"], s["grad"],
                                          grad_loss=s["grad_loss"])
    return s["loss"], s["lse"], s["grad"]


def _own_sample(s):
    import exact_bpe_tokenization_amd as tt
    c = s["case"]
    ws = _workspace(s, lambda: tt.toktier_sample_workspace_bytes(c["rows"], c["vocab"]))
    tt.toktier_sample(s["logits"], s["uniform"], s["out_ids"], s["out_logprobs"], ws,
                      temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                      mask=s["mask"])
    return s["out_ids"], s["out_logprobs"]


_run_own = {"embed": _own_embed, "embed_grad": _own_embed_grad, "loss": _own_loss, "sample": _own_sample}


def _plain_embed(s):
    ids = s["ids"]
    valid = ids >= 0
    x = s["table"][ids.clamp(min=0).long()].float() * s["case"]["scale"]
    return (x * valid.unsqueeze(1)).to(s["out"].dtype)


def _plain_embed_grad(s):
    c, ids = s["case"], s["ids"]
    g = s["grad"].float() * (c["scale"] * (ids >= 0).float()).unsqueeze(1)
    at = ids.clamp(min=0).long()
    if c["accumulate"] and s["out"].dtype == torch.float32:
        return s["out"].index_add_(0, at, g)
    total = s["out"].float() if c["accumulate"] else torch.zeros(s["out"].shape, device="cuda")
    s["out"].copy_(total.index_add_(0, at, g))
    return s["out"]


def _plain_loss(s):
    y = s["targets"].long().unsqueeze(1)
    valid = y >= 0
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    some = top > -math.inf
    e = torch.exp(x - torch.where(some, top, torch.zeros_like(top)))
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(torch.where(some, total, torch.ones_like(total)))
    target = x.gather(1, y.clamp(min=0))
    loss = torch.where(some, lse - target, torch.full_like(lse, math.inf))
    loss = torch.where(valid, loss, torch.zeros_like(loss))
    e /= torch.where(some, total, torch.ones_like(total))
    hit = e.gather(1, y.clamp(min=0)) - 1.0
    e.scatter_(1, y.clamp(min=0), hit)
    e *= torch.where(valid & some, s["grad_loss"].unsqueeze(1), torch.zeros_like(lse))
    return loss.squeeze(1), lse.squeeze(1), e.to(s["grad"].dtype)


def _plain_sample(s):
    # 64 bits: a running mass next to u * total decides which ID is drawn
    x = s["logits"].double()
    rows, vocab = x.shape
    if s["mask"] is not None:
        j = torch.arange(vocab, device="cuda")
        bits = (s["mask"][:, j // 32] >> (j % 32).to(torch.int32)) & 1
        x = torch.where(bits == 1, x, torch.full_like(x, -math.inf))
    top = x.amax(1, keepdim=True)
    some = (top > -math.inf).squeeze(1)
    t = s["temperature"].double().unsqueeze(1)
    greedy = t <= 0
    y = (x - torch.where(some.unsqueeze(1), top, torch.zeros_like(top))) / torch.where(greedy, torch.ones_like(t), t)
    w = torch.exp(y)
    k = s["top_k"].long().unsqueeze(1)
    k = torch.where(greedy, torch.ones_like(k), torch.where(k == 0, torch.full_like(k, vocab), k))
    _, order = torch.sort(x, dim=1, descending=True, stable=True)
    rank = torch.arange(vocab, device="cuda").unsqueeze(0)
    ws = w.gather(1, order) * (rank < k)
    before = ws.cumsum(1) - ws
    keep = (rank < k) & ((before < s["top_p"].double().unsqueeze(1) * ws.sum(1, keepdim=True)) |
                         (s["top_p"].unsqueeze(1) >= 1))
    keep &= ws >= s["min_p"].double().unsqueeze(1)
    keep |= rank == 0
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, torch.zeros_like(ws)))
    mass = kept.cumsum(1)
    total = mass[:, -1:]
    ids = (mass <= s["uniform"].double().unsqueeze(1) * total).sum(1).clamp(max=vocab - 1)
    logprob = torch.log(kept.gather(1, ids.unsqueeze(1)) / total).squeeze(1)
    ids = torch.where(some, ids, torch.full_like(ids, -1))
    logprob = torch.where(some, logprob, torch.full_like(logprob, -math.inf))
    return ids.to(torch.int32), logprob.float()


_run_plain = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "loss": _plain_loss, "sample": _plain_sample}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without

def _distinct(tokens, vocab):
    """Expected number of different IDs among `tokens` of _ids."""
    edges = np.log(np.arange(1, vocab + 2, dtype=np.float64)) / math.log(vocab + 1.0)
    return float(-np.expm1(tokens * np.log1p(-np.minimum(np.diff(edges), 1 - 1e-12))).sum())


def work(case):
    c = case
    if c["op"] == "embed":
        t, d = c["tokens"], c["dim"]
        rows = _distinct(t * (1 - c["pad"]), c["vocab"])
        return {"bytes": 4 * t + rows * d * SIZES[c["table"]] + t * d * SIZES[c["out"]], "flops": t * d}
    if c["op"] == "embed_grad":
        t, d = c["tokens"], c["dim"]
        rows = _distinct(t * (1 - c["pad"]), c["vocab"])
        out = (2 * rows if c["accumulate"] else c["vocab"]) * d * SIZES[c["out"]]
        return {"bytes": 4 * t + t * (1 - c["pad"]) * d * SIZES[c["grad"]] + out, "flops": 2 * t * d}
    cells = c["rows"] * c["vocab"]
    if c["op"] == "loss":
        reads = 1 if c["fused"] else 2
        return {"bytes": cells * SIZES[c["type"]] * (reads + 1) + 20 * c["rows"], "flops": 6 * cells}
    return {"bytes": cells * SIZES[c["type"]] + (cells / 8 if c["mask"] else 0) + 28 * c["rows"], "flops": 3 * cells}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "embed_grad": _exact_embed_grad, "loss": _exact_loss,
            "sample": _exact_sample}[case["op"]](s)


def _exact_embed(s):
    table = torch.cat([s["table"].double() * s["case"]["scale"],
                       torch.zeros(1, s["case"]["dim"], dtype=torch.float64, device="cuda")])
    return torch.index_select(table, 0, torch.where(s["ids"] < 0, s["case"]["vocab"], s["ids"]).long())


def _exact_embed_grad(s):
    # tokens sorted by ID; a row's sum is the difference of two running sums
    c = s["case"]
    out = s["out"].double() if c["accumulate"] else torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    ids, order = torch.sort(s["ids"].long())
    ends = torch.searchsorted(ids, torch.arange(c["vocab"] + 1, device="cuda"))
    for a in range(0, c["dim"], 512):
        part = s["grad"][:, a:a + 512].double()[order]
        run_ = torch.cat([torch.zeros_like(part[:1]), part.cumsum(0)])
        out[:, a:a + 512] += c["scale"] * (run_[ends[1:]] - run_[ends[:-1]])
    return out


def _exact_loss(s):
    x, y = s["logits"], s["targets"].long()
    rows, vocab = x.shape
    loss, lse, grad = [], [], torch.empty(rows, vocab, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 27) // vocab)
    for r in range(0, rows, step):
        part, t = x[r:r + step].double(), y[r:r + step]
        z = torch.logsumexp(part, 1)
        line = torch.arange(t.numel(), device="cuda")
        at = z - part[line, t.clamp(min=0)]
        at[torch.isneginf(z)] = math.inf
        at[t < 0] = 0.0
        p = torch.exp(part - z.unsqueeze(1))
        p[line, t.clamp(min=0)] -= 1.0
        p *= s["grad_loss"][r:r + step].double().unsqueeze(1)
        p[(t < 0) | torch.isneginf(z)] = 0.0
        grad[r:r + step] = p
        loss.append(at)
        lse.append(z)
    return torch.cat(loss), torch.cat(lse), grad


def _exact_sample(s):
    rows, vocab = s["logits"].shape
    x = s["logits"].float().cpu().numpy().astype(np.float64)
    if s["mask"] is not None:
        packed = np.ascontiguousarray(s["mask"].cpu().numpy()).view(np.uint8)
        x[np.unpackbits(packed, axis=1, bitorder="little")[:, :vocab] == 0] = -np.inf
    host = {n: s[n].cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p", "uniform")}
    logprobs = np.empty(rows)
    for r in range(rows):
        row, t = x[r], float(host["temperature"][r])
        if not np.isfinite(row.max()):
            logprobs[r] = -np.inf
            continue
        if t <= 0:
            logprobs[r] = 0.0
            continue
        order = np.argsort(-row, kind="stable")
        if host["top_k"][r]:
            order = order[:host["top_k"][r]]
        w = np.exp((row[order] - row[order[0]]) / t)
        n = len(w)
        if host["top_p"][r] < 1:
            n = min(n, 1 + int(np.searchsorted(np.cumsum(w), float(host["top_p"][r]) * w.sum())))
        n = max(1, min(n, int((w >= float(host["min_p"][r])).sum())))
        by_index = np.argsort(order[:n])
        mass = np.cumsum(w[:n][by_index])
        j = min(int(np.searchsorted(mass, float(host["uniform"][r]) * mass[-1], side="right")), n - 1)
        logprobs[r] = math.log(w[by_index[j]] / mass[-1])
    return None, torch.from_numpy(logprobs)
