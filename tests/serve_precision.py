"""The bound of attend_token's results, with the weights that it promises: two
BF16 operands within 2^-14 of each weight, so 2^-14 A where serve_util.py, whose
other terms and names hold here too, has one rounding to BF16 (u A).  The
first operand leaves between 2^-7 and 2^-6 of the weight's power of two, and
the second is that rounded to BF16, by at most 2^-8 of it; with 8 bits the
weight times its value's scale is rounded to 32 bits before, which the term 64 e
A covers."""
import torch

import serve_util as U

WEIGHT = 2.0 ** -14


def attend64(q, k, v, scale):
    """(out, bound) of one row q [d] that sees all of k, v [n, d] (64 bits)."""
    n, d = k.shape
    s = (k @ q) * scale
    p = torch.softmax(s, 0)
    out, a = p @ v, p @ v.abs()
    top = float(((k.abs() @ q.abs()) * scale).max())
    return out, U.U * out.abs() + a * (WEIGHT + 2 * d * U.E * top + 64 * U.E * (1 + top) + 2 * n * U.E)


def token64(q, cache, pages, lens, scale):
    q, pages = q.double().cpu(), pages.cpu()
    k, v, ks, vs = (None if x is None else x.cpu() for x in cache)
    group = q.shape[1] // k.shape[1]
    out, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for s, n in enumerate(lens):
        if n == 0:
            continue
        kd, vd = U.gathered(k, ks, pages[s], n), U.gathered(v, vs, pages[s], n)
        for h in range(q.shape[1]):
            out[s, h], bound[s, h] = attend64(q[s, h], kd[:, h // group], vd[:, h // group], scale)
    return out, bound


def balanced(v):
    """Values whose rows come in pairs of opposite sign, nearly: sums cancel, so
    that a result is small beside what is summed, and its own rounding hides
    little of the weights'."""
    v = v.clone()
    n = v.shape[0] // 2 * 2
    v[1:n:2] = -v[0:n:2]
    return v


def emulated(q, k, v, scale, weights):
    """A row's result from weights in the given form: "two" operands, "once"
    rounded to BF16, or the "first" operand alone."""
    p = torch.exp2((k @ q) * scale * 1.4426950408889634 - 8).float()
    cut = (p.view(torch.int32) >> 16) - 1
    first = (cut << 16).view(torch.float32)
    w = {"first": first.double(), "once": p.to(torch.bfloat16).double(),
         "two": first.double() + (p - first).to(torch.bfloat16).double()}[weights]
    return (w @ v / p.double().sum()).to(torch.bfloat16)
