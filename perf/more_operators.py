"""What is measured of the serving operators that prepare heads and attend over
the paged cache: norms of query and key heads with the position rotation, the
same on the way into the cache, attention of a chunk of new tokens over the
cache, and attention inside a sliding window with a few first tokens that stay
visible (sinks).

A case is one call of real use.  `run` computes it in plain torch operations
in 32 bits (angles in 64), or, where `own` is set, by the package's entry
points.  `exact` computes it from the definition in 64 bits.

Definitions:
  norm       y = x / sqrt(mean(x^2) + eps) * w, for each head
  rotation   pair i of a head, elements (i, i + n) of the first 2 n or, with
             neighbours, (2 i, 2 i + 1): (a, b) -> (a c - b s, b c + a s) with
             c, s = cos, sin(position[axis_i] * base^(-i / n)); the other
             elements stay
  8 bits     for each token and head, a = max |x|, scale = a / 127 and codes
             rint(x * (127 / a)), ties to even; a below 2^-100 counts as 2^-100
  attention  the queries of a sequence are its last ones: query i of n over m
             keys stands at p = m - n + i and sees the keys j <= p, in a window
             of w of them those with j > p - w or j < sinks;
             out[i, h] = sum_j p_j v[j, h'] / sum_j p_j with
             p_j = exp(<q[i, h], k[j, h']> / sqrt(head_dim)), h' = h // (heads / kv_heads)
Cache pages: [page, kv_head, position in the page, head_dim]; scales
[page, kv_head, position]; slot = page * page_size + position."""
import math
import random

import torch

own = False

DEVICE = "cuda"
TINY = 2.0 ** -100
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    llama = {"heads": 32, "kv_heads": 8, "head_dim": 128}
    return [
        # the new tokens of 16 sequences through a layer that norms its heads: latency
        {"name": "rotate 16 tokens", "op": "rotate", "seqs": 16, "longest": 1, "first": 900, "len_seed": 1, "rotary_dim": 128,
         "neighbours": False, "axes": 1, "norms": True, "base": 500000.0, **llama},
        # a prompt of text and images, three axes
        {"name": "rotate an image prompt", "op": "rotate", "seqs": 3, "longest": 8111, "first": 0, "len_seed": 2, "rotary_dim": 128,
         "neighbours": False, "axes": 3, "norms": True, "base": 1000000.0, **llama},
        # one new token of each of 64 sequences goes into the cache, rotated
        {"name": "append 64 tokens", "op": "append", "seqs": 64, "longest": 1, "first": 500, "len_seed": 4, "page_size": 16,
         "store": "bf16", "rotary_dim": 128, "neighbours": False, "axes": 1, "norms": False, "base": 500000.0, **llama},
        # prompts go into the cache, rotated
        {"name": "append prompts", "op": "append", "seqs": 5, "longest": 8191, "first": 0, "len_seed": 6, "page_size": 64,
         "store": "bf16", "rotary_dim": 128, "neighbours": False, "axes": 1, "norms": False, "base": 500000.0, **llama},
        # prompts go into the cache in 8 bits, normed and rotated as neighbours, and come back for what follows
        {"name": "append and read, 8 bits", "op": "append_read", "seqs": 3, "longest": 4001, "first": 0, "len_seed": 8, "page_size": 16,
         "store": "int8", "rotary_dim": 64, "neighbours": True, "axes": 1, "norms": True, "base": 10000.0, **llama},
        # a chat turn of 64 tokens behind what was said before: latency
        {"name": "chunk of 64", "op": "chunk", "seqs": 1, "longest": 64, "prefix": 1937, "len_seed": 0, "page_size": 16,
         "store": "bf16", "window": 0, "sinks": 0, **llama},
        # a step of a server that mixes pieces of prompts with single tokens
        {"name": "chunks and tokens", "op": "chunk", "seqs": 32, "longest": 512, "prefix": 8192, "len_seed": 3, "singles": 28,
         "page_size": 16, "store": "bf16", "window": 0, "sinks": 0, **llama},
        # pieces of prompts over a cache in 8 bits
        {"name": "chunks, 8 bits", "op": "chunk", "seqs": 6, "longest": 701, "prefix": 12000, "len_seed": 5, "page_size": 32,
         "store": "int8", "window": 0, "sinks": 0, **llama},
        # the next piece of a long document
        {"name": "piece of a long document", "op": "chunk", "seqs": 1, "longest": 2048, "prefix": 30001, "len_seed": 0, "page_size": 64,
         "store": "bf16", "window": 0, "sinks": 0, **llama},
        # a long prompt through a layer with a window
        {"name": "prompt of 16384 in a window", "op": "chunk", "seqs": 1, "longest": 16384, "prefix": 0, "len_seed": 0, "page_size": 64,
         "store": "bf16", "window": 4096, "sinks": 4, **llama},
        # one user's next token through a layer with a window
        {"name": "token of one in a window", "op": "token", "seqs": 1, "longest": 20001, "len_seed": 0, "page_size": 16,
         "store": "bf16", "window": 1024, "sinks": 4, **llama},
        # the next token of a full batch through a layer with a window
        {"name": "tokens of 64 in a window", "op": "token", "seqs": 64, "longest": 16384, "len_seed": 7, "page_size": 32,
         "store": "bf16", "window": 4096, "sinks": 16, **llama},
    ]


HEADS = ((32, 8), (32, 32), (24, 24), (16, 2), (12, 4), (8, 1), (20, 1))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotate", "append", "append_read", "chunk", "chunk", "chunk", "token", "token"))
    heads, kv_heads = rng.choice(HEADS)
    d = rng.choice((64, 128, 128))
    case = {"op": op, "len_seed": rng.randrange(1 << 20), "heads": heads, "kv_heads": kv_heads, "head_dim": d}
    if op in ("rotate", "append", "append_read"):
        case["seqs"] = _log(rng, 1, 64)
        case["longest"] = _log(rng, 1, 16384 // case["seqs"])
        case["first"] = rng.choice((0, _log(rng, 1, 200000)))
        case["rotary_dim"] = rng.choice((d, d, d // 2, 16, 48))
        case["neighbours"] = rng.random() < 0.4
        case["axes"] = rng.choice((1, 1, 2, 3, 4))
        case["norms"] = rng.random() < 0.5
        case["base"] = rng.choice((10000.0, 500000.0, 1000000.0))
    if op != "rotate":
        case["page_size"] = rng.choice((16, 32, 64, 128))
        case["store"] = {"append": "bf16", "append_read": "int8"}.get(op) or rng.choice(("bf16", "bf16", "int8"))
    if op in ("chunk", "token"):
        windowed = op == "token" or rng.random() < 0.5
        case["window"] = _log(rng, 1, 8192) if windowed else 0
        case["sinks"] = rng.choice((0, 1, 4, 16, 100)) if windowed else 0
    if op == "chunk":
        case["seqs"] = _log(rng, 1, 24)
        case["longest"] = _log(rng, 1, 4096 // case["seqs"])
        case["prefix"] = _log(rng, 1, 12288 // case["seqs"]) if rng.random() < 0.7 else 0
        case["singles"] = rng.choice((0, 0, case["seqs"] // 2))
    if op == "token":
        case["seqs"] = _log(rng, 1, 128)
        case["longest"] = _log(rng, 1, min(65536, (1 << (18 if kv_heads <= 8 else 16)) // case["seqs"]))
    return case


def _lengths(n, longest, seed, least=1):
    """n lengths from `least` to `longest`: the first is the longest, the second the shortest."""
    r = random.Random(seed)
    got = [longest] + [r.randint(least, max(least, longest)) for _ in range(n - 1)]
    if n > 2:
        got[1] = least
    return got


def _case_lengths(case):
    """(new tokens, all tokens) of each sequence."""
    n = case["seqs"]
    if case["op"] == "token":
        return [1] * n, _lengths(n, case["longest"], case["len_seed"])
    new = _lengths(n, case["longest"], case["len_seed"])
    for i in range(case.get("singles", 0)):
        new[n - 1 - i] = 1
    prefix = case.get("prefix", case.get("first", 0))
    before = _lengths(n, prefix, case["len_seed"] + 1, 0) if prefix else [0] * n
    return new, [a + b for a, b in zip(new, before)]


# ---------------------------------------------------------------- the inputs

def _rows(gen, n, heads, d, outliers=False):
    """n rows of `heads` heads: normal values; keys have a few channels that are larger, as trained models have."""
    x = torch.randn(n, heads, d, device=DEVICE, generator=gen)
    if outliers:
        x *= torch.where(torch.rand(heads, d, device=DEVICE, generator=gen) < 0.03, 4.0, 1.0)
    return x.to(torch.bfloat16)


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=DEVICE)


def _tables(gen, lens, page_size):
    """Page tables whose pages lie in any order, and the number of pages."""
    need = [-(-n // page_size) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, device=DEVICE, generator=gen).to(torch.int32)
    first = [sum(need[:i]) for i in range(len(need))]
    width = max(1, max(need))
    at = torch.tensor(first, device=DEVICE)[:, None] + torch.arange(width, device=DEVICE)
    used = torch.arange(width, device=DEVICE) < torch.tensor(need, device=DEVICE)[:, None]
    return torch.where(used, order[torch.where(used, at, 0)], 0).to(torch.int32).contiguous(), n_pages


def _axes(case):
    """The axis of each pair: runs of neighbouring pairs."""
    pairs, n = case["rotary_dim"] // 2, case["axes"]
    return [i * n // pairs for i in range(pairs)]


def _cache(gen, case, n_pages):
    hk, d, ps = case["kv_heads"], case["head_dim"], case["page_size"]
    k = _rows(gen, n_pages * ps, hk, d, outliers=True).view(n_pages, ps, hk, d).transpose(1, 2).contiguous()
    v = _rows(gen, n_pages * ps, hk, d).view(n_pages, ps, hk, d).transpose(1, 2).contiguous()
    if case["store"] == "bf16":
        return k, v, None, None
    (k, ks), (v, vs) = _quantise(k), _quantise(v)
    return k, v, ks, vs


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    new, whole = _case_lengths(case)
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    n = sum(new)
    s = {"case": case}
    if case["op"] in ("chunk", "token"):
        s["pages"], n_pages = _tables(gen, whole, case["page_size"])
        s["cache"] = _cache(gen, case, n_pages)
        s["q"] = _rows(gen, n, h, d)
        s["q_starts"] = _starts(new)
        s["lens"] = torch.tensor(whole, dtype=torch.int32, device=DEVICE)
        s["out"] = torch.empty_like(s["q"])
        return s
    # one projection gave all three
    fused = _rows(gen, n, h + 2 * hk, d)
    fused[:, h:h + hk] = _rows(gen, n, hk, d, outliers=True)
    s["q"], s["k"], s["v"] = fused[:, :h], fused[:, h:h + hk], fused[:, h + hk:]
    s["q_out"] = torch.empty(n, h, d, dtype=torch.bfloat16, device=DEVICE)
    row = torch.arange(n, device=DEVICE)
    starts = _starts(new)
    seq = torch.searchsorted(starts[1:].contiguous(), row.to(torch.int32), right=True)
    before = torch.tensor([b - a for a, b in zip(new, whole)], device=DEVICE)
    at = row - starts[seq] + before[seq]
    # time goes on, height and width go over rows of 40 patches
    s["positions"] = torch.stack([at, at // 40, at % 40, at // 7][:case["axes"]], 1).to(torch.int32)
    if case["axes"] == 1:
        s["positions"] = s["positions"][:, 0].contiguous()
    if case["norms"]:
        s["q_weight"], s["k_weight"] = (torch.rand(d, device=DEVICE, generator=gen).mul_(0.8).add_(0.6).to(torch.bfloat16) for _ in range(2))
    else:
        s["q_weight"] = s["k_weight"] = None
    pairs = case["rotary_dim"] // 2
    s["freqs"] = case["base"] ** (-torch.arange(pairs, dtype=torch.float64, device=DEVICE) / pairs)
    s["axes"] = torch.tensor(_axes(case), device=DEVICE)
    if own:
        import lossless_bf16_weight_amd as df11
        s["rotation"] = df11.rotation(case["rotary_dim"], base=case["base"], axes=_axes(case), interleaved=case["neighbours"])
    if case["op"] == "rotate":
        s["k_out"] = torch.empty(n, hk, d, dtype=torch.bfloat16, device=DEVICE)
        return s
    ps = case["page_size"]
    s["pages"], n_pages = _tables(gen, whole, ps)
    s["cache"] = _cache(gen, case, n_pages)
    s["slots"] = s["pages"][seq, at // ps].to(torch.int64) * ps + at % ps
    if case["op"] == "append_read":
        s["starts"] = _starts(whole)
        s["k_back"] = torch.empty(sum(whole), hk, d, dtype=torch.bfloat16, device=DEVICE)
        s["v_back"] = torch.empty_like(s["k_back"])
    return s


# ---------------------------------------------------------------- plain forms

def _quantise(x):
    x = x.float()
    a = x.abs().amax(-1).clamp_min(TINY)
    top = torch.full_like(a, 127.0)
    return torch.round(x * (top / a)[..., None]).to(torch.int8), a / 127.0


def _plain_heads(s, x, weight):
    """x normed and rotated, in 32 bits."""
    case, x = s["case"], x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    at = s["positions"] if case["axes"] == 1 else s["positions"][:, s["axes"]]
    angle = (at[:, None] if case["axes"] == 1 else at).double() * s["freqs"]
    c, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    r = case["rotary_dim"]
    turned, rest = x[..., :r], x[..., r:]
    if case["neighbours"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * c - b * sn, b * c + a * sn), -1).flatten(-2)
    else:
        a, b = turned[..., :r // 2], turned[..., r // 2:]
        turned = torch.cat((a * c - b * sn, b * c + a * sn), -1)
    return torch.cat((turned, rest), -1)


def _plain_rotate(s):
    return _plain_heads(s, s["q"], s["q_weight"]).to(torch.bfloat16), _plain_heads(s, s["k"], s["k_weight"]).to(torch.bfloat16)


def _plain_append(s):
    k, v, ks, vs = s["cache"]
    ps = k.shape[2]
    page, at = s["slots"] // ps, s["slots"] % ps
    q, new_k = _plain_heads(s, s["q"], s["q_weight"]).to(torch.bfloat16), _plain_heads(s, s["k"], s["k_weight"])
    if ks is None:
        k[page, :, at], v[page, :, at] = new_k.to(torch.bfloat16), s["v"]
    else:
        (k[page, :, at], ks[page, :, at]), (v[page, :, at], vs[page, :, at]) = _quantise(new_k), _quantise(s["v"])
    return q


def _plain_read(s):
    k, v, ks, vs = s["cache"]
    ps = k.shape[2]
    row = torch.arange(s["k_back"].shape[0], device=k.device)
    seq = torch.searchsorted(s["starts"][1:].contiguous(), row.to(torch.int32), right=True)
    pos = row - s["starts"][seq]
    page, at = s["pages"][seq, pos // ps].long(), pos % ps
    kd, vd = k[page, :, at].float(), v[page, :, at].float()
    if ks is not None:
        kd *= ks[page, :, at][..., None]
        vd *= vs[page, :, at][..., None]
    return kd.to(torch.bfloat16), vd.to(torch.bfloat16)


def _seen(case, n, m, device):
    """[n, m]: whether query i of n sees key j of m."""
    at, key = torch.arange(m - n, m, device=device)[:, None], torch.arange(m, device=device)
    seen = key <= at
    if case["window"]:
        seen &= (key > at - case["window"]) | (key < case["sinks"])
    return seen


def _plain_attend(s):
    case, (k, v, ks, vs) = s["case"], s["cache"]
    new, whole = _case_lengths(case)
    h, hk, d, ps = case["heads"], case["kv_heads"], case["head_dim"], case["page_size"]
    out, first = torch.empty_like(s["q"]), 0
    for i, (n, m) in enumerate(zip(new, whole)):
        pages = s["pages"][i, :-(-m // ps)].long()
        kd, vd = k[pages].float(), v[pages].float()
        if ks is not None:
            kd *= ks[pages][..., None]
            vd *= vs[pages][..., None]
        kd, vd = (x.transpose(0, 1).reshape(hk, -1, d)[:, :m] for x in (kd, vd))
        q = s["q"][first:first + n].float().view(n, hk, h // hk, d).permute(1, 2, 0, 3).reshape(hk, -1, d) * (1.0 / math.sqrt(d))
        z = torch.matmul(q, kd.transpose(1, 2).contiguous()).view(hk, h // hk, n, m)
        z.masked_fill_(~_seen(case, n, m, z.device), -math.inf)
        z.sub_(z.amax(-1, keepdim=True)).exp_()
        o = torch.matmul(z.view(hk, -1, m), vd.contiguous()) / z.sum(-1).view(hk, -1, 1)
        out[first:first + n] = o.view(hk, h // hk, n, d).permute(2, 0, 1, 3).reshape(n, h, d).to(torch.bfloat16)
        first += n
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import lossless_bf16_weight_amd as df11
        if op == "rotate":
            df11.rotate_heads(state["q"], state["k"], state["positions"], state["rotation"], state["q_out"], state["k_out"],
                              q_weight=state["q_weight"], k_weight=state["k_weight"], eps=EPS)
            return state["q_out"], state["k_out"]
        cache = df11.KVCache(*state["cache"])
        if op == "chunk":
            df11.attend_chunk(state["q"], cache, state["pages"], state["q_starts"], state["lens"], state["out"],
                              window=case["window"], sinks=case["sinks"])
            return state["out"]
        if op == "token":
            df11.attend_token(state["q"], cache, state["pages"], state["lens"], state["out"], window=case["window"], sinks=case["sinks"])
            return state["out"]
        df11.kv_append(cache, state["k"], state["v"], state["positions"], state["slots"], state["rotation"], k_weight=state["k_weight"],
                       q=state["q"], q_out=state["q_out"], q_weight=state["q_weight"], eps=EPS)
        if op == "append":
            return state["q_out"], *state["cache"][:2]
        df11.kv_read(cache, state["pages"], state["starts"], state["k_back"], state["v_back"])
        return state["q_out"], state["k_back"], state["v_back"]
    if op == "rotate":
        return _plain_rotate(state)
    if op in ("chunk", "token"):
        return _plain_attend(state)
    q = _plain_append(state)
    return (q, *state["cache"][:2]) if op == "append" else (q, *_plain_read(state))


# ---------------------------------------------------------------- what it needs

def work(case):
    new, whole = _case_lengths(case)
    h, hk, d, n = case["heads"], case["kv_heads"], case["head_dim"], sum(new)
    word = 2 * hk * d                                                # bytes of a token's keys or values in BF16
    stored = word if case.get("store") != "int8" else hk * (d + 4)   # and in the cache
    if case["op"] in ("chunk", "token"):
        pairs = keys = tables = 0
        for a, m in zip(new, whole):
            w, sinks = case["window"] or m, case["sinks"] if case["window"] else 0
            for p in range(m - a, m):
                pairs += min(p + 1, w) + min(sinks, max(p + 1 - w, 0))
            first = max(0, m - a - w + 1)       # of the first query's window
            used = m - first + min(sinks, first)
            keys += used
            tables += 4 * -(-used // case["page_size"])
        return {"bytes": 2 * n * 2 * h * d + 2 * keys * stored + tables, "flops": 4 * pairs * h * d}
    turned = (2 * h * d + word) * 2 * n + 4 * n * case["axes"]       # queries and keys, read and written
    if case["op"] == "rotate":
        return {"bytes": turned, "flops": 0}
    append = n * (2 * 2 * h * d + 2 * word + 2 * stored + 8 + 4 * case["axes"])
    if case["op"] == "append":
        return {"bytes": append, "flops": 0}
    return {"bytes": append + sum(whole) * (2 * stored + 2 * word) + 4 * sum(-(-m // case["page_size"]) for m in whole), "flops": 0}


# ---------------------------------------------------------------- 64 bits

def _heads64(s, x, weight):
    """The definition, element by element: element e of a head with its partner."""
    case, x = s["case"], x.double()
    d, r = case["head_dim"], case["rotary_dim"]
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * weight.double()
    out = x.clone()
    pos = s["positions"].double().view(x.shape[0], -1)
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if case["neighbours"] else (i, i + r // 2)
        t = pos[:, _axes(case)[i]] * case["base"] ** (-2.0 * i / r)
        c, sn = torch.cos(t)[:, None], torch.sin(t)[:, None]
        out[..., a] = x[..., a] * c - x[..., b] * sn
        out[..., b] = x[..., b] * c + x[..., a] * sn
    return out


def _stored64(x):
    """What the cache in 8 bits gives back for rows x."""
    a = x.abs().amax(-1, keepdim=True).clamp_min(TINY)
    return torch.round(x * 127 / a) * (a / 127)


def exact(case, seed):
    s = prepare(case, seed)
    new, whole = _case_lengths(case)
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "rotate":
        return _heads64(s, s["q"], s["q_weight"]), _heads64(s, s["k"], s["k_weight"])
    ps = case["page_size"]
    held = [x.double() if scale is None else x.double() * scale.double()[..., None] for x, scale in zip(s["cache"][:2], s["cache"][2:])]
    if case["op"] in ("append", "append_read"):
        for x, rows in zip(held, (_heads64(s, s["k"], s["k_weight"]), s["v"].double())):
            x[s["slots"] // ps, :, s["slots"] % ps] = rows if case["op"] == "append" else _stored64(rows)
    kd, vd = ([x[s["pages"][i, :-(-m // ps)].long()].transpose(1, 2).flatten(0, 1)[:m] for i, m in enumerate(whole)]
              for x in held) if case["op"] != "append" else held
    if case["op"] in ("append", "append_read"):
        q = _heads64(s, s["q"], s["q_weight"])
        return (q, kd, vd) if case["op"] == "append" else (q, torch.cat(kd), torch.cat(vd))
    out, first = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEVICE), 0
    for i, (n, m) in enumerate(zip(new, whole)):
        key, at = torch.arange(m, device=DEVICE), torch.arange(n, device=DEVICE)[:, None] + (m - n)
        hidden = key > at
        if case["window"]:
            hidden |= (key + case["window"] <= at) & (key >= case["sinks"])
        for x in range(h):
            g = x // (h // hk)
            z = (s["q"][first:first + n, x].double() @ kd[i][:, g].T) / math.sqrt(d)
            out[first:first + n, x] = torch.softmax(z.masked_fill_(hidden, -math.inf), -1) @ vd[i][:, g]
        first += n
    return out
