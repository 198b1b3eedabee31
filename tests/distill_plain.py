"""Distillation from a teacher's top logits in 64 bits, and bounds on what the kernels may be off by (used by the tests).

u = 2^-24.  With T the temperature and d = (m - x) / T:
  exp(-d)  the difference rounds by u, its factor log2(e) / T is off by 3 u, their product by u, the power by 2 u and by
           2 u more for the rounding of log2(e) in its size: relative (5 d + 4) u
  s        a thread adds eight powers of a vector and rescales by a power when its maximum grows (on the way no more
           than the range); 64 lanes meet in six steps, 16 wavefronts in 15: as for the cross entropy (ops_bounds), 13 u a
           vector and 105 u, with 5 u a unit of growth
  log q    from the list's maximum and sum likewise, or t / T - L with 2 u of t / T and u of the result
  loss     every term's own errors, and a sum of k terms."""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SMALLEST = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}   # powers have no subnormal results
FAR = 128.0


def vectors(vocab, least=256):
    return -(-vocab // 2048) if vocab <= 8192 or least == 256 else -(-vocab // 4096) if vocab <= 32768 else -(-vocab // 8192)


def _parts(z, extra):
    """(maximum, sum, probabilities, relative bound of the sum) of rows; the finite ones' range bounds the maximum's growth."""
    m = z.amax(1, keepdim=True)
    d = (m - z).clamp(max=104)
    e = torch.exp(z - m)
    s = e.sum(1, keepdim=True)
    p = e / s
    finite = torch.where(torch.isinf(z), m, z)
    grown = (m - finite.amin(1, keepdim=True)).clamp(max=104)
    return m, s, p, d, U * ((p * (5 * d + 4)).sum(1, keepdim=True) + 5 * grown + extra)


def distill(x, ids, top, temperature, teacher_lse, c, dtype, from_lse=False):
    """dict of (value, bound) of loss, lse and grad.  x: float64 [n, v], no NaN, no +inf, no row of -inf alone; every list has an entry
    with a finite logit; all in float64 but ids."""
    n, v = x.shape
    t = float(temperature)
    z = x / t
    m, s, p, d, rel = _parts(z, 13 * vectors(v, 1024) + 105)
    log_s = torch.log(s)
    lse = (m + log_s).squeeze(1)
    e_log_s = rel + 4 * U * (log_s + 1)
    e_lse = (e_log_s + 3 * U * m.abs()).squeeze(1) + 2 * U * lse.abs()
    ids = ids.long()
    kept = (ids >= 0) & (ids < v)
    at = torch.where(kept, ids, torch.zeros_like(ids))
    y = torch.where(kept, top / t, torch.full_like(top, -float("inf")))
    if teacher_lse is None:
        mt, st, _, _, relt = _parts(y, 13 * 4 + 105)
        log_q = (y - mt) - torch.log(st)   # mt + log(st) would lose the logarithm from |mt| = 2^53 on, in 64 bits
        e_log_q = 3 * U * torch.where(torch.isinf(y), torch.zeros_like(y), (y - mt).abs()) + relt + 4 * U * (torch.log(st) + 1)
    else:
        log_q = y - teacher_lse.unsqueeze(1)
        e_log_q = 3 * U * torch.where(torch.isinf(y), torch.zeros_like(y), y.abs())
    some = ~torch.isinf(y)
    log_q = torch.where(some, log_q, torch.zeros_like(y))
    e_log_q = e_log_q + U * log_q.abs()
    q = torch.where(some, torch.exp(log_q), torch.zeros_like(y))
    rel_q = e_log_q + U * (2 * log_q.abs().clamp(max=104) + 4)
    log_p = torch.where(some, (z.gather(1, at) - m) - log_s, torch.zeros_like(y))
    e_log_p = 3 * U * torch.where(some, (m - z.gather(1, at)), torch.zeros_like(y)) + e_log_s + U * log_p.abs()
    term = torch.where(q > 0, q * (log_q - log_p), torch.zeros_like(q))
    loss = term.sum(1)
    k = ids.size(1)
    e_loss = (q * (rel_q * (log_q - log_p).abs() + e_log_q + e_log_p + 2 * U * (log_q - log_p).abs()) + k * U * term.abs() + 2.0 ** -120).sum(1)
    mass = q.sum(1, keepdim=True)
    e_mass = (q * rel_q).sum(1, keepdim=True) + k * U * mass
    if from_lse:
        far = rel + U * (5 * d + 8) + U * 13 * vectors(v)
        zl = lse.unsqueeze(1)
        near = e_lse.unsqueeze(1) + U * (2 * zl.abs() + 5 * (zl - z).abs().clamp(max=104) + 6)
        own = torch.where(zl.abs() < FAR, near, torch.where(zl.abs() > FAR + 1, far, torch.maximum(near, far)))
    else:
        own = rel + U * (5 * d + 8)
    factor = (c / t).unsqueeze(1)
    listed, e_listed = torch.zeros_like(x), torch.zeros_like(x)
    listed.scatter_add_(1, at, q)
    e_listed.scatter_add_(1, at, q * (rel_q + k * U))
    grad = factor * (mass * p - listed)
    size = factor.abs()
    err = size * (mass * p * own + e_mass * p + e_listed + 4 * U * (mass * p + listed) + 2.0 ** -120) + 4 * U * grad.abs()
    err = err + HALF_STEP[dtype] * (grad.abs() + err) + SMALLEST[dtype]
    return dict(loss=(loss, e_loss), lse=(lse, e_lse), grad=(grad, err))
