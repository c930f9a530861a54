"""Plain 64-bit forms of layer norm, embedding, gradient norm and clipping, and
bounds on how far the library's fp32 arithmetic may be from them.

U = 2^-24 is half a step of fp32. A sum of fp32 terms in any order has an error
of at most depth * U * (sum of the terms' magnitudes), where depth is the
longest chain of additions a term goes through. Outputs are rounded once more,
by at most half a step of their type: eps / 2 relative, or half the smallest
subnormal."""
import torch

U = 2.0 ** -24
# registers: up to 40 terms a thread, 5 + 5 shuffle steps, the mean's factor 1/n
ROW_DEPTH = 64


def row_depth(n):
    """Longest chain of a row's sum: rows too wide for registers are summed with
    a stride of 1024 threads."""
    return ROW_DEPTH + n // 1024


def half_step(value, dtype):
    info = torch.finfo(dtype)
    return value.abs() * (info.eps / 2) + info.smallest_normal * info.eps / 2


def layer_norm(x, weight, bias, eps):
    """y, mean, rstd in fp64."""
    x = x.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * weight.double()
    if bias is not None:
        y = y + bias.double()
    return y, mean, rstd


def layer_norm_bounds(x, weight, bias, eps, y_dtype):
    """Bounds on the errors of y, mean and rstd.

    The mean's error is delta <= K U mean|x|. It is the same for the whole row,
    so it moves sum (x - mean)^2 by n delta^2 only (sum (x - mean) = 0); the
    squares' sum adds K U and the difference's rounding 2 U relative. rstd takes
    half of that, plus a division and a root."""
    y, mean, rstd = layer_norm(x, weight, bias, eps)
    n = x.shape[1]
    K = row_depth(n) + 2
    d = (x.double() - mean[:, None]).abs()
    delta = K * U * x.double().abs().mean(1)
    rel = 0.5 * ((delta * rstd) ** 2 + (K + 4) * U) + 4 * U
    w = 1.0 if weight is None else weight.double().abs()
    b = 0.0 if bias is None else bias.double().abs()
    xh = d * rstd[:, None]
    e = rstd[:, None] * (delta[:, None] + U * d) + xh * rel[:, None]
    e = e * w + 4 * U * (xh * w + b)
    return e * 1.001 + half_step(y, y_dtype), delta * 1.001 + U * mean.abs(), rstd * rel * 1.001


def layer_norm_backward(dy, x, weight, mean, rstd):
    """dx, dweight, dbias in fp64, from the given statistics."""
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * rstd
    g = dy if weight is None else dy * weight.double()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def layer_norm_backward_bounds(dy, x, weight, mean, rstd, dx_dtype):
    """Bounds on the errors of dx, dweight and dbias: xh carries 2 U, g one U, the
    row sums their depth, and the last expression four more roundings."""
    dx, _, _ = layer_norm_backward(dy, x, weight, mean, rstd)
    tokens, n = x.shape
    K = row_depth(n) + 4
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = ((x - mean) * rstd).abs()
    g = dy.abs() if weight is None else (dy * weight.double()).abs()
    m1 = g.mean(1, keepdim=True)
    m2 = (g * xh).mean(1, keepdim=True)
    e = rstd * ((K + 8) * U * (m1 + xh * m2) + 8 * U * g)
    # the sums over rows: a chain of at most all rows and the join of the blocks
    rows = tokens + 100
    return (e * 1.001 + half_step(dx, dx_dtype), (rows + 4) * U * (dy.abs() * xh).sum(0),
            rows * U * dy.abs().sum(0))


def embedding(table, ids, scale):
    V = table.shape[0]
    ids = ids.long()
    ok = (ids >= 0) & (ids < V)
    y = table.double()[ids.clamp(0, V - 1)] * scale
    return y * ok[:, None]


def embedding_backward(dy, ids, vocab, scale, padding_id=-1, old=None):
    """dtable in fp64, and the same sum over magnitudes with each row's count."""
    ids = ids.long()
    keep = (ids >= 0) & (ids < vocab) & (ids != padding_id)
    out = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device=dy.device)
    mag = torch.zeros_like(out)
    out.index_add_(0, ids[keep], dy.double()[keep])
    mag.index_add_(0, ids[keep], dy.double().abs()[keep])
    count = torch.zeros(vocab, dtype=torch.float64, device=dy.device)
    count.index_add_(0, ids[keep], torch.ones(int(keep.sum()), dtype=torch.float64, device=dy.device))
    out, mag = out * scale, mag * abs(scale)
    if old is not None:
        out, mag = out + old.double(), mag + old.double().abs() * (count[:, None] > 0)
    return out, mag, count


def embedding_backward_bound(out, mag, count, dtype):
    """A row's sum is a chain of at most its count of tokens, then the scale and
    the addition to the old value."""
    return (count[:, None] + 3) * U * mag + half_step(out, dtype)


def grad_norm(tensors):
    total = sum(float((t.double() ** 2).sum()) for t in tensors)
    return total ** 0.5


# A thread adds 32 squares in four fp32 chains (8 + 2 additions, one rounding of
# each square) before fp64 takes over: the sum is off by at most 11 U, its root by
# half of that, and storing it rounds once.
NORM_RTOL = 7 * U
# the factor: the norm's error, the division and its rounding to fp32, one product
CLIP_RTOL = 10 * U
