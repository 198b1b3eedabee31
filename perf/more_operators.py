"""Cases of the losses over the vocabulary: cross entropy straight from hidden states and the table, with its
gradients and without kept logits; distillation from a teacher's top logits; and the top logits themselves.

``run`` computes them in plain torch operations, or, where ``own`` is true, calls the package's entry
points.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
# ID counts of the vocabularies in workloads/vocabs: 256 bytes + 1,000 / 32,768 / 131,072 merges
V1, V2, V3 = 1256, 33024, 131328


def listed():
    return [
        # a small model's training step in float32, padded sequences
        dict(name="linear small f32", op="linear", rows=256, vocab=V1, dim=320, pad_cols=0, type="f32", ignore=0.1,
             mode="fused"),
        # scoring of one continuation: the losses of 16 positions, no gradient
        dict(name="linear score 16", op="linear", rows=16, vocab=V3, dim=4096, pad_cols=0, type="bf16", ignore=0.0,
             mode="loss"),
        # training step of a large model's head: 8,192 positions over the largest vocabulary
        dict(name="linear train 8192", op="linear", rows=8192, vocab=V3, dim=4096, pad_cols=0, type="bf16", ignore=0.02,
             mode="fused"),
        # fine-tuning on answers: most positions are prompts, which the loss ignores
        dict(name="linear answers 4096", op="linear", rows=4096, vocab=V2, dim=2048, pad_cols=0, type="bf16", ignore=0.6,
             mode="fused"),
        # odd vocabulary and width in padded rows, loss first and gradients later
        dict(name="linear odd f16 two calls", op="linear", rows=1500, vocab=33001, dim=1001, pad_cols=22, type="f16",
             ignore=0.1, mode="two"),
        # a float32 model of medium size, next to the library's float32 products
        dict(name="linear medium f32", op="linear", rows=2048, vocab=V2, dim=1024, pad_cols=0, type="f32", ignore=0.0,
             mode="fused"),
        # a small student in float32 from lists of eight
        dict(name="distill small f32", op="distill", rows=64, vocab=V1, k=8, pad_cols=0, type="f32", temperature=1.0,
             listed=False, pad=0.0, fused=True),
        # one training step of a student: 8,192 positions, the teacher's 64 largest logits, renormalised over them
        dict(name="distill train 8192", op="distill", rows=8192, vocab=V3, k=64, pad_cols=0, type="bf16",
             temperature=2.0, listed=True, pad=0.0, fused=True),
        # odd vocabulary in padded rows, lists of unequal length, the teacher's own log-sum-exp, gradient later
        dict(name="distill odd f16 two calls", op="distill", rows=1500, vocab=33001, k=100, pad_cols=23, type="f16",
             temperature=1.5, listed=False, pad=0.1, fused=False),
        # top log-probabilities of one chat sequence
        dict(name="top one", op="top", rows=1, vocab=V3, k=20, pad_cols=0, type="bf16", temperature=1.0),
        # a teacher's lists for a batch of a student
        dict(name="top teacher 2048", op="top", rows=2048, vocab=V3, k=64, pad_cols=0, type="bf16", temperature=2.0),
        # long lists in float32 from an odd vocabulary in padded rows
        dict(name="top odd f32", op="top", rows=300, vocab=33001, k=1000, pad_cols=7, type="f32", temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "distill", "top"])
    vocab = rng.choice([V1, V2, V3, _log_int(rng, 260, V3)])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "linear":
        return dict(op=op, rows=_log_int(rng, 1, 8192 if kind != "f32" else 2048), vocab=vocab,
                    dim=rng.choice([320, 1024, 2048, 4096, _log_int(rng, 64, 4096)]),
                    pad_cols=rng.choice([0, 0, 1, 64]), type=kind, ignore=rng.choice([0.0, 0.1, 0.6]),
                    mode=rng.choice(["loss", "fused", "fused", "two"]))
    if op == "distill":
        return dict(op=op, rows=_log_int(rng, 1, 4096), vocab=vocab, k=_log_int(rng, 1, 256),
                    pad_cols=rng.choice([0, 0, 1, 56]), type=kind, temperature=rng.choice([1.0, 1.0, 2.0, 0.75]),
                    listed=rng.random() < 0.5, pad=rng.choice([0.0, 0.1]), fused=rng.random() < 0.6)
    return dict(op=op, rows=_log_int(rng, 1, 1024), vocab=vocab, k=_log_int(rng, 1, min(1024, vocab)),
                pad_cols=rng.choice([0, 0, 3, 64]), type=kind, temperature=rng.choice([1.0, 2.0]))


# ---------------------------------------------------------------------------------------------
# inputs

def _ids(gen, n, vocab, ignored):
    """Token IDs with the skew of text (log-uniform over the vocabulary: byte and early merge IDs are the
    frequent ones); a share of them names none (-1)."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).floor().clamp_(0, vocab - 1).to(torch.int32)
    if ignored:    # the first is kept, so that no batch is ignored whole
        ids[1:][torch.rand(n - 1, generator=gen, device="cuda") < ignored] = -1
    return ids


def _rows(rows, cols, pad_cols, kind, make):
    """A matrix whose rows lie pad_cols further apart than they are long."""
    full = torch.empty(rows, cols + pad_cols, dtype=DTYPES[kind], device="cuda")
    step = max(1, (1 << 27) // cols)
    for r in range(0, rows, step):
        full[r:r + step, :cols] = make(min(step, rows - r))
    if pad_cols:
        full[:, cols:] = 100.0    # what lies beyond a row is not the row's
    return full[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev, c = "cuda", case
    s = dict(case=dict(case))
    rows, vocab, kind = c["rows"], c["vocab"], DTYPES[c["type"]]

    def noise(k, n):
        return torch.randn(k, n, generator=gen, device=dev)

    if c["op"] == "linear":
        dim = c["dim"]
        s["weight"] = _rows(vocab, dim, c["pad_cols"], c["type"], lambda k: noise(k, dim) * (2.5 / math.sqrt(dim)))
        s["targets"] = _ids(gen, rows, vocab, c["ignore"])
        # hidden states that know something of their target: its logit is lifted by up to 9
        lift = 9.0 * torch.rand(rows, 1, generator=gen, device=dev) / 6.25
        toward = s["weight"][s["targets"].clamp(min=0).long()].float() * lift
        s["hidden"] = _rows(rows, dim, c["pad_cols"], c["type"], lambda k: noise(k, dim))
        s["hidden"].copy_((s["hidden"].float() + toward).to(kind))
        # the mean over the batch; float16 with the loss scaled, as such training needs it
        s["grad_loss"] = torch.rand(rows, generator=gen, device=dev) / rows
        s["scale"] = 4096.0 if c["type"] == "f16" else 1.0
        s["loss"], s["lse"] = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        if c["mode"] != "loss":
            s["grad_hidden"] = torch.empty(rows, dim, dtype=kind, device=dev)
            s["grad_weight"] = torch.empty(vocab, dim, dtype=kind, device=dev)
    elif c["op"] == "distill":
        k = c["k"]
        ids, top, lse = [], [], []

        def student(n):
            x = 2.5 * noise(n, vocab)
            t = x + noise(n, vocab)
            values, at = torch.topk(t, k, dim=1)
            ids.append(at.to(torch.int32))
            top.append(values)
            lse.append(torch.logsumexp(t / c["temperature"], 1))
            return x

        s["logits"] = _rows(rows, vocab, c["pad_cols"], c["type"], student)
        s["top_ids"], s["top_logits"] = torch.cat(ids).contiguous(), torch.cat(top).contiguous()
        s["teacher_lse"] = None if c["listed"] else torch.cat(lse)
        if c["pad"]:    # lists that hold fewer, and rows that hold none
            s["top_ids"][torch.rand(rows, k, generator=gen, device=dev) < c["pad"]] = -1
            s["top_ids"][36::37] = -1
        s["grad_loss"] = torch.rand(rows, generator=gen, device=dev) / rows
        s["scale"] = c["temperature"] ** 2 * (4096.0 if c["type"] == "f16" else 1.0)
        s["loss"], s["lse"] = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        s["grad"] = torch.empty(rows, vocab, dtype=kind, device=dev)
    else:
        def logits(n):   # a power law over ranks, as next-token distributions have, with noise
            u = torch.rand(n, vocab, generator=gen, device=dev)
            return 12.0 - 1.25 * torch.log1p(u * vocab) + 0.3 * noise(n, vocab)

        s["logits"] = _rows(rows, vocab, c["pad_cols"], c["type"], logits)
        s["out_ids"] = torch.empty(rows, c["k"], dtype=torch.int32, device=dev)
        s["out_logits"] = torch.empty(rows, c["k"], device=dev)
        s["lse"] = torch.empty(rows, device=dev)
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


def _own_linear(s):
    import exact_bpe_tokenization_amd as tt
    c = s["case"]
    grads = c["mode"] != "loss"
    ws = _workspace(s, lambda: tt.toktier_linear_cross_entropy_workspace_bytes(
        c["rows"], c["vocab"], c["dim"], DTYPES[c["type"]], grads))
    if c["mode"] == "fused":
        tt.toktier_linear_cross_entropy(s["hidden"], s["weight"], s["targets"], s["loss"], s["lse"], ws,
                                        grad_hidden=s["grad_hidden"], grad_weight=s["grad_weight"],
                                        grad_loss=s["grad_loss"], grad_scale=s["scale"])
    else:
        tt.toktier_linear_cross_entropy(s["hidden"], s["weight"], s["targets"], s["loss"], s["lse"], ws)
        if grads:
            tt.toktier_linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], s["lse"], ws,
                                                     grad_hidden=s["grad_hidden"], grad_weight=s["grad_weight"],
                                                     grad_loss=s["grad_loss"], grad_scale=s["scale"])
    return (s["loss"], s["lse"], s["grad_hidden"], s["grad_weight"]) if grads else (s["loss"], s["lse"])


def _own_distill(s):
    import exact_bpe_tokenization_amd as tt
    c = s["case"]
    ws = _workspace(s, lambda: tt.toktier_distill_workspace_bytes(c["rows"], c["vocab"], c["k"]))
    grad = dict(grad_logits=s["grad"], grad_loss=s["grad_loss"], grad_scale=s["scale"])
    teacher = dict(temperature=c["temperature"], teacher_lse=s["teacher_lse"])
    if c["fused"]:
        tt.toktier_distill(s["logits"], s["top_ids"], s["top_logits"], s["loss"], s["lse"], ws, **teacher, **grad)
    else:
        tt.toktier_distill(s["logits"], s["top_ids"], s["top_logits"], s["loss"], s["lse"], ws, **teacher)
        tt.toktier_distill_backward(s["logits"], s["top_ids"], s["top_logits"], s["lse"], **teacher, **grad)
    return s["loss"], s["lse"], s["grad"]


def _own_top(s):
    import exact_bpe_tokenization_amd as tt
    c = s["case"]
    ws = _workspace(s, lambda: tt.toktier_top_logits_workspace_bytes(c["rows"], c["vocab"], c["k"]))
    tt.toktier_top_logits(s["logits"], s["out_ids"], s["out_logits"], ws, lse=s["lse"], temperature=c["temperature"])
    return s["out_ids"], s["out_logits"], s["lse"]


_run_own = {"linear": _own_linear, "distill": _own_distill, "top": _own_top}


def _log_sum_exp(x):
    """(row maxima, exponentials less them, their sums, log-sum-exp), each kept as a column."""
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    return top, e, total, top + torch.log(total)


def _plain_linear(s):
    y = s["targets"].long().unsqueeze(1)
    valid = y >= 0
    h, w = s["hidden"].float(), s["weight"].float()
    x = h @ w.t()
    zero = torch.zeros(x.size(0), 1, device="cuda")
    top, e, total, lse = _log_sum_exp(x)
    loss = torch.where(valid, (top - x.gather(1, y.clamp(min=0))) + torch.log(total), zero)
    out = loss.squeeze(1), torch.where(valid, lse, zero).squeeze(1)
    if s["case"]["mode"] == "loss":
        return out
    del x
    e /= total
    e.scatter_(1, y.clamp(min=0), e.gather(1, y.clamp(min=0)) - 1.0)
    e *= torch.where(valid, s["scale"] * s["grad_loss"].unsqueeze(1), zero)
    return out + ((e @ w).to(s["hidden"].dtype), (e.t() @ h).to(s["weight"].dtype))


def _plain_distill(s):
    c, t = s["case"], s["case"]["temperature"]
    x = s["logits"].float() / t
    top, e, total, lse = _log_sum_exp(x)
    valid = s["top_ids"] >= 0
    at = s["top_ids"].clamp(min=0).long()
    y = torch.where(valid, s["top_logits"] / t, torch.full_like(s["top_logits"], -math.inf))
    any_ = valid.any(1, keepdim=True)
    zero = torch.zeros_like(lse)
    most = torch.where(any_, y.amax(1, keepdim=True), zero)
    if s["teacher_lse"] is None:
        listed_ = torch.where(any_, torch.exp(y - most).sum(1, keepdim=True), zero + 1.0)
        log_q = y - most - torch.log(listed_)
    else:
        log_q = y - s["teacher_lse"].unsqueeze(1)
    q = torch.exp(log_q)
    log_p = (x.gather(1, at) - top) - torch.log(total)
    loss = torch.where(valid, q * (log_q - log_p), torch.zeros_like(q)).sum(1)
    del x
    e *= q.sum(1, keepdim=True) / total
    e.scatter_add_(1, at, -q)
    e *= (s["scale"] / t) * s["grad_loss"].unsqueeze(1)
    return loss, lse.squeeze(1), e.to(s["grad"].dtype)


def _plain_top(s):
    c = s["case"]
    x = s["logits"].float()
    _, _, _, lse = _log_sum_exp(x / c["temperature"])
    values, order = torch.sort(x, dim=1, descending=True, stable=True)
    return order[:, :c["k"]].to(torch.int32), values[:, :c["k"]].contiguous(), lse.squeeze(1)


_run_plain = {"linear": _plain_linear, "distill": _plain_distill, "top": _plain_top}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c = case
    cells, size = c["rows"] * c["vocab"], SIZES[c["type"]]
    if c["op"] == "linear":
        kept = c["rows"] * (1 - c["ignore"])    # ignored positions need no products and no hidden state
        ends = (kept + c["vocab"]) * c["dim"] * size
        outs = (c["rows"] + c["vocab"]) * c["dim"] * size
        if c["mode"] == "loss":
            return {"bytes": ends + 12 * c["rows"], "flops": 2 * kept * c["vocab"] * c["dim"]}
        reads = 1 if c["mode"] == "fused" else 2
        return {"bytes": reads * ends + outs + 16 * c["rows"], "flops": 6 * kept * c["vocab"] * c["dim"]}
    if c["op"] == "distill":
        reads = 1 if c["fused"] else 2
        return {"bytes": cells * size * (reads + 1) + c["rows"] * (8 * c["k"] * reads + 16), "flops": 6 * cells}
    return {"bytes": cells * size + c["rows"] * (8 * c["k"] + 4), "flops": 3 * cells}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "distill": _exact_distill, "top": _exact_top}[case["op"]](s)


def _exact_linear(s):
    c = s["case"]
    grads = c["mode"] != "loss"
    w = s["weight"].double().contiguous()
    y = s["targets"].long()
    loss = torch.zeros(c["rows"], dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(loss)
    kept = torch.nonzero(y >= 0).squeeze(1)
    if grads:
        gh = torch.zeros(c["rows"], c["dim"], dtype=torch.float64, device="cuda")
        gw = torch.zeros(c["vocab"], c["dim"], dtype=torch.float64, device="cuda")
    for part in torch.split(kept, max(1, (1 << 28) // c["vocab"])):
        h = s["hidden"][part].double()
        x = torch.mm(h, w.t())
        z = torch.logsumexp(x, 1)
        line = torch.arange(part.numel(), device="cuda")
        lse[part] = z
        loss[part] = z - x[line, y[part]]
        if grads:
            p = torch.exp(x - z.unsqueeze(1))
            p[line, y[part]] -= 1.0
            p *= (s["scale"] * s["grad_loss"][part].double()).unsqueeze(1)
            gh[part] = torch.mm(p, w)
            gw.addmm_(p.t(), h)
    return (loss, lse, gh, gw) if grads else (loss, lse)


def _exact_distill(s):
    c, t = s["case"], s["case"]["temperature"]
    rows, vocab = s["logits"].shape
    loss, lse, grad = [], [], torch.empty(rows, vocab, dtype=torch.float64, device="cuda")
    for r in range(0, rows, max(1, (1 << 27) // vocab)):
        part = slice(r, r + max(1, (1 << 27) // vocab))
        log_p = torch.log_softmax(s["logits"][part].double() / t, 1)
        ids = s["top_ids"][part].long()
        y = (s["top_logits"][part].double() / t).masked_fill(ids < 0, -math.inf)
        z = torch.logsumexp(y, 1) if s["teacher_lse"] is None else s["teacher_lse"][part].double()
        log_q = (y - z.unsqueeze(1)).masked_fill(ids < 0, -math.inf)
        q = torch.exp(log_q)
        terms = q * (log_q - log_p.gather(1, ids.clamp(min=0)))
        loss.append(terms.masked_fill(ids < 0, 0.0).sum(1))
        lse.append(torch.logsumexp(s["logits"][part].double() / t, 1))
        g = torch.exp(log_p) * q.sum(1, keepdim=True)
        g.scatter_add_(1, ids.clamp(min=0), -q)
        grad[part] = g * (s["scale"] / t * s["grad_loss"][part].double()).unsqueeze(1)
    return torch.cat(loss), torch.cat(lse), grad


def _exact_top(s):
    c = s["case"]
    values, lse = [], []
    for part in torch.split(s["logits"], max(1, (1 << 27) // c["vocab"])):
        x = part.double()
        values.append(torch.topk(x, c["k"], dim=1).values)
        lse.append(torch.logsumexp(x / c["temperature"], 1))
    return None, torch.cat(values), torch.cat(lse)
