"""What is measured of the serving operators: attention over packed prompts,
attention of one new token over a paged key-value cache, and the cache's
writing and reading back, as BF16 words or as 8-bit codes.

A case is one call of real use.  `run` computes it in plain torch operations
in 32 bits, or, where `own` is set, by the package's entry points.  `exact`
computes it from the definition in 64 bits.

Definitions (query t of sequence s attends to keys 0 .. n_keys - 1 of s):
  attention  out[t, h] = sum_j p_j v[j, h'] / sum_j p_j with
             p_j = exp(scale * <q[t, h], k[j, h']>) over the keys that t may
             see and h' = h // (heads / kv_heads); a row that sees none is 0.
             Causal: the queries are the last ones of their sequence, so
             query i of n_q sees the keys j <= i + n_keys - n_q.
  8 bits     for each token and head, a = max |x|, scale = a / 127 and
             codes rint(x * (127 / a)), ties to even; a below 2^-100 counts
             as 2^-100.  Read back as code * scale, rounded to BF16.
Cache pages: [page, kv_head, position in the page, head_dim]; scales
[page, kv_head, position]; slot = page * page_size + position."""
import math
import random

import torch

own = False

DEVICE = "cuda"
TINY = 2.0 ** -100


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a chat turn of 64 tokens through one block: latency
        {"name": "prompt of 64", "op": "prompt", "seqs": 1, "longest": 64, "prefix": 0, "len_seed": 0,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "causal": True},
        # requests of unequal lengths packed into one batch, one of a single token
        {"name": "packed prompts", "op": "prompt", "seqs": 11, "longest": 2113, "prefix": 0, "len_seed": 3,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "causal": True},
        # one long document
        {"name": "prompt of 16384", "op": "prompt", "seqs": 1, "longest": 16384, "prefix": 0, "len_seed": 0,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "causal": True},
        # the next piece of prompts whose earlier tokens are in the cache
        {"name": "pieces behind a prefix", "op": "prompt", "seqs": 2, "longest": 130, "prefix": 12000, "len_seed": 1,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "causal": True},
        # one user's next token
        {"name": "token of one", "op": "token", "seqs": 1, "longest": 777, "len_seed": 0, "page_size": 16,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "store": "bf16"},
        # the next token of a full batch
        {"name": "tokens of 64", "op": "token", "seqs": 64, "longest": 4096, "len_seed": 5, "page_size": 16,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "store": "bf16"},
        # the next token of two long documents
        {"name": "tokens of two long", "op": "token", "seqs": 2, "longest": 100001, "len_seed": 2, "page_size": 64,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "store": "bf16"},
        # the next token of a batch over a cache of 8-bit codes
        {"name": "tokens of 48, 8 bits", "op": "token", "seqs": 48, "longest": 16384, "len_seed": 7, "page_size": 32,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "store": "int8"},
        # one new token of each of 64 sequences goes into the cache
        {"name": "write 64 tokens", "op": "write", "seqs": 64, "longest": 1, "prefix": 500, "len_seed": 4, "page_size": 16,
         "kv_heads": 8, "head_dim": 128, "store": "bf16"},
        # prompts go into the cache as words
        {"name": "write prompts", "op": "write", "seqs": 5, "longest": 8191, "prefix": 0, "len_seed": 6, "page_size": 64,
         "kv_heads": 8, "head_dim": 128, "store": "bf16"},
        # prompts go into the cache in 8 bits, and come back for the attention of what follows
        {"name": "write and read, 8 bits", "op": "write_read", "seqs": 3, "longest": 4001, "prefix": 0, "len_seed": 8,
         "page_size": 16, "kv_heads": 8, "head_dim": 128, "store": "int8"},
        # the cached prefixes of a batch are read back from 8 bits
        {"name": "read back, 8 bits", "op": "read", "seqs": 8, "longest": 32768, "len_seed": 9, "page_size": 32,
         "kv_heads": 8, "head_dim": 128, "store": "int8"},
    ]


HEADS = ((32, 8), (32, 32), (24, 24), (16, 2), (12, 4), (8, 1), (20, 1))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prompt", "token", "token", "write", "write_read", "read"))
    heads, kv_heads = rng.choice(HEADS)
    case = {"op": op, "len_seed": rng.randrange(1 << 20), "kv_heads": kv_heads, "head_dim": rng.choice((64, 128, 128))}
    if op in ("prompt", "token"):
        case["heads"] = heads
    if op == "prompt":
        case["causal"] = rng.random() < 0.75
        case["seqs"] = _log(rng, 1, 24)
        case["longest"] = _log(rng, 1, 8192 // case["seqs"])
        case["prefix"] = _log(rng, 1, 16384 // case["seqs"]) if rng.random() < 0.4 else 0
    else:
        case["page_size"] = rng.choice((16, 32, 64, 128))
        case["store"] = rng.choice(("bf16", "int8")) if op != "write" else "bf16"
        case["seqs"] = _log(rng, 1, 128)
        if op == "write_read":
            case["store"] = "int8"
        most = 1 << (18 if kv_heads <= 8 else 16)      # tokens in all
        case["longest"] = _log(rng, 1, min(65536, most // case["seqs"]))
        if op in ("write", "write_read"):
            case["prefix"] = rng.choice((0, _log(rng, 1, max(1, min(4096, most // case["seqs"])))))
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
    new = _lengths(case["seqs"], case["longest"], case["len_seed"])
    prefix = case.get("prefix", 0)
    before = _lengths(case["seqs"], prefix, case["len_seed"] + 1, 0) if prefix else [0] * case["seqs"]
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


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    new, whole = _case_lengths(case)
    hk, d = case["kv_heads"], case["head_dim"]
    s = {"case": case}
    if case["op"] == "prompt":
        h, n_q, n_k = case["heads"], sum(new), sum(whole)
        if n_q == n_k:      # one projection gave all three
            fused = _rows(gen, n_q, h + 2 * hk, d)
            fused[:, h:h + hk] = _rows(gen, n_q, hk, d, outliers=True)
            s["q"], s["k"], s["v"] = fused[:, :h], fused[:, h:h + hk], fused[:, h + hk:]
        else:
            s["q"], s["k"], s["v"] = _rows(gen, n_q, h, d), _rows(gen, n_k, hk, d, outliers=True), _rows(gen, n_k, hk, d)
        s["q_starts"], s["k_starts"] = _starts(new), _starts(whole)
        s["out"] = torch.empty(n_q, h, d, dtype=torch.bfloat16, device=DEVICE)
        return s
    ps = case["page_size"]
    s["pages"], n_pages = _tables(gen, whole, ps)
    shape = (n_pages, hk, ps, d)
    k = _rows(gen, n_pages * ps, hk, d, outliers=True).view(n_pages, ps, hk, d).transpose(1, 2).contiguous()
    v = _rows(gen, n_pages * ps, hk, d).view(n_pages, ps, hk, d).transpose(1, 2).contiguous()
    if case["store"] == "int8":
        (k, ks), (v, vs) = _quantise(k), _quantise(v)
        s["cache"] = (k, v, ks, vs)
    else:
        s["cache"] = (k, v, None, None)
    assert s["cache"][0].shape == shape
    if case["op"] == "token":
        s["q"] = _rows(gen, case["seqs"], case["heads"], d)
        s["lens"] = torch.tensor(whole, dtype=torch.int32, device=DEVICE)
        s["out"] = torch.empty_like(s["q"])
    if case["op"] in ("write", "write_read"):
        n = sum(new)
        s["k"], s["v"] = _rows(gen, n, hk, d, outliers=True), _rows(gen, n, hk, d)
        starts = _starts(new)
        row = torch.arange(n, device=DEVICE)
        seq = torch.searchsorted(starts[1:].contiguous(), row.to(torch.int32), right=True)
        before = torch.tensor([w - m for w, m in zip(whole, new)], device=DEVICE)
        at = row - starts[seq] + before[seq]
        s["slots"] = s["pages"][seq, at // ps].to(torch.int64) * ps + at % ps
    if case["op"] in ("read", "write_read"):
        s["starts"] = _starts(whole)
        s["k_out"] = torch.empty(sum(whole), hk, d, dtype=torch.bfloat16, device=DEVICE)
        s["v_out"] = torch.empty_like(s["k_out"])
    return s


# ---------------------------------------------------------------- plain forms

def _quantise(x):
    x = x.float()
    a = x.abs().amax(-1).clamp_min(TINY)
    top = torch.full_like(a, 127.0)
    return torch.round(x * (top / a)[..., None]).to(torch.int8), a / 127.0


def _softmax_product(s, allowed, v):
    """softmax over the allowed last axis of s, times v; rows without any are 0.  s is overwritten."""
    s.masked_fill_(~allowed, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    s.sub_(m).exp_()
    l = s.sum(-1, keepdim=True)
    return torch.matmul(s, v) / torch.where(l == 0, 1.0, l)


def _plain_prompt(s):
    q, k, v, d = s["q"].float(), s["k"].float(), s["v"].float(), s["case"]["head_dim"]
    (n_q, h, _), (n_k, hk, _) = q.shape, k.shape
    at_q, at_k = torch.arange(n_q, device=q.device), torch.arange(n_k, device=q.device)
    seq_q = torch.searchsorted(s["q_starts"][1:].contiguous(), at_q.to(torch.int32), right=True)
    seq_k = torch.searchsorted(s["k_starts"][1:].contiguous(), at_k.to(torch.int32), right=True)
    allowed = seq_q[:, None] == seq_k[None, :]
    if s["case"]["causal"]:     # both counted from the end of the sequence
        from_end_q = s["q_starts"][seq_q + 1] - at_q
        from_end_k = s["k_starts"][seq_k + 1] - at_k
        allowed &= from_end_k[None, :] >= from_end_q[:, None]
    qh = q.view(n_q, hk, h // hk, d).permute(1, 2, 0, 3).reshape(hk, -1, d) * (1.0 / math.sqrt(d))
    scores = torch.matmul(qh, k.permute(1, 2, 0).contiguous()).view(hk, h // hk, n_q, n_k)
    o = _softmax_product(scores, allowed, v.permute(1, 0, 2).contiguous()[:, None])
    return o.permute(2, 0, 1, 3).reshape(n_q, h, d).to(torch.bfloat16)


def _values(x, scale, pages):
    """The values of the tables' pages, [seq, kv_head, position, head_dim] in 32 bits."""
    x = x[pages].float()
    if scale is not None:
        x *= scale[pages][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_token(s):
    k, v, ks, vs = s["cache"]
    b, h, d = s["q"].shape
    hk = k.shape[1]
    kd, vd = _values(k, ks, s["pages"]), _values(v, vs, s["pages"])
    q = s["q"].float().view(b, hk, h // hk, d) * (1.0 / math.sqrt(d))
    scores = torch.matmul(q, kd.transpose(2, 3))
    allowed = torch.arange(kd.shape[2], device=q.device) < s["lens"][:, None, None, None]
    return _softmax_product(scores, allowed, vd).reshape(b, h, d).to(torch.bfloat16)


def _plain_write(s):
    k, v, ks, vs = s["cache"]
    ps = k.shape[2]
    page, at = s["slots"] // ps, s["slots"] % ps
    if ks is None:
        k[page, :, at], v[page, :, at] = s["k"], s["v"]
    else:
        (k[page, :, at], ks[page, :, at]), (v[page, :, at], vs[page, :, at]) = _quantise(s["k"]), _quantise(s["v"])


def _plain_read(s):
    k, v, ks, vs = s["cache"]
    ps = k.shape[2]
    row = torch.arange(s["k_out"].shape[0], device=k.device)
    seq = torch.searchsorted(s["starts"][1:].contiguous(), row.to(torch.int32), right=True)
    pos = row - s["starts"][seq]
    page, at = s["pages"][seq, pos // ps].long(), pos % ps
    kd, vd = k[page, :, at].float(), v[page, :, at].float()
    if ks is not None:
        kd *= ks[page, :, at][..., None]
        vd *= vs[page, :, at][..., None]
    return kd.to(torch.bfloat16), vd.to(torch.bfloat16)


def run(state):
    op = state["case"]["op"]
    if own:
        import lossless_bf16_weight_amd as df11
        if op == "prompt":
            df11.attend_prompt(state["q"], state["k"], state["v"], state["q_starts"], state["k_starts"], state["out"],
                               causal=state["case"]["causal"])
            return state["out"]
        cache = df11.KVCache(*state["cache"])
        if op == "token":
            df11.attend_token(state["q"], cache, state["pages"], state["lens"], state["out"])
            return state["out"]
        if op in ("write", "write_read"):
            df11.kv_write(cache, state["k"], state["v"], state["slots"])
        if op in ("read", "write_read"):
            df11.kv_read(cache, state["pages"], state["starts"], state["k_out"], state["v_out"])
            return state["k_out"], state["v_out"]
        return state["cache"][:2]
    if op == "prompt":
        return _plain_prompt(state)
    if op == "token":
        return _plain_token(state)
    if op in ("write", "write_read"):
        _plain_write(state)
    return _plain_read(state) if op in ("read", "write_read") else state["cache"][:2]


# ---------------------------------------------------------------- what it needs

def work(case):
    new, whole = _case_lengths(case)
    hk, d = case["kv_heads"], case["head_dim"]
    word = 2 * hk * d                                                # bytes of a token's keys or values in BF16
    stored = word if case.get("store") != "int8" else hk * (d + 4)   # and in the cache
    if case["op"] == "prompt":
        h = case["heads"]
        pairs = sum(n * m for n, m in zip(new, whole))
        if case["causal"]:      # the last of n queries sees all m keys, the one before it one less
            pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(new, whole))
        return {"bytes": 2 * sum(new) * 2 * h * d + 2 * sum(whole) * word, "flops": 4 * pairs * h * d}
    tables = 4 * sum(-(-m // case["page_size"]) for m in whole)
    if case["op"] == "token":
        h = case["heads"]
        return {"bytes": 2 * sum(whole) * stored + 2 * case["seqs"] * 2 * h * d + tables, "flops": 4 * sum(whole) * h * d}
    written = sum(new) * (2 * word + 2 * stored + 8)
    read = sum(whole) * (2 * stored + 2 * word) + tables
    return {"write": {"bytes": written, "flops": 0}, "read": {"bytes": read, "flops": 0},
            "write_read": {"bytes": written + read, "flops": 0}}[case["op"]]


# ---------------------------------------------------------------- 64 bits

def _attend64(q, k, v, first):
    """Rows of one sequence and head in 64 bits; row i sees the keys below first + i (all where first is None)."""
    s = (q @ k.T) / math.sqrt(q.shape[1])
    if first is not None:
        n, m = s.shape
        s.masked_fill_(torch.arange(m, device=s.device) >= first + torch.arange(n, device=s.device)[:, None], -math.inf)
    return torch.softmax(s, -1) @ v


def _stored64(x):
    """What the cache in 8 bits gives back for rows x."""
    x = x.double()
    a = x.abs().amax(-1, keepdim=True).clamp_min(TINY)
    return torch.round(x * 127 / a) * (a / 127)


def exact(case, seed):
    s = prepare(case, seed)
    new, whole = _case_lengths(case)
    if case["op"] == "prompt":
        g = case["heads"] // case["kv_heads"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEVICE)
        a = b = 0
        for n, m in zip(new, whole):
            for h in range(case["heads"]):
                kv = (s[x][b:b + m, h // g].double() for x in ("k", "v"))
                out[a:a + n, h] = _attend64(s["q"][a:a + n, h].double(), *kv, m - n + 1 if case["causal"] else None)
            a, b = a + n, b + m
        return out
    ps = case["page_size"]
    if case["op"] == "write":
        got = [x.double() for x in s["cache"][:2]]
        for x, rows in zip(got, (s["k"], s["v"])):
            x[s["slots"] // ps, :, s["slots"] % ps] = rows.double()
        return got
    held = []
    for x, scale in zip(s["cache"][:2], s["cache"][2:]):
        held.append(x.double() if scale is None else x.double() * scale.double()[..., None])
    if case["op"] == "write_read":
        for x, rows in zip(held, (s["k"], s["v"])):
            x[s["slots"] // ps, :, s["slots"] % ps] = _stored64(rows)
    kd, vd = ([x[s["pages"][i, :-(-m // ps)].long()].transpose(1, 2).flatten(0, 1)[:m] for i, m in enumerate(whole)]
              for x in held)
    if case["op"] == "token":
        g = case["heads"] // case["kv_heads"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEVICE)
        for i in range(case["seqs"]):
            for h in range(case["kv_heads"]):
                out[i, g * h:g * h + g] = _attend64(s["q"][i, g * h:g * h + g].double(), kd[i][:, h], vd[i][:, h], None)
        return out
    return torch.cat(kd), torch.cat(vd)
