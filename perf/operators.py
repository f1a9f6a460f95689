"""Cases for timing the token-mixer operators of a serving step.

Four operators, each in a plain form (elementary torch operations, fp32 sums)
and as the calls a user makes of the library:

  delta_prefill  the gated delta rule over a ragged batch of prompts
  delta_step     the same recurrence for the next token(s) of every request
  kv_cache       quantising keys and values into a paged cache as they arrive,
                 and reading the sequences back
  kv_attend      attention of the newest token(s) over that cache
"""
import math
import random

import torch

own = False

D = 128                       # key and value size of the recurrent heads
CHUNK = 64                    # tokens per block of the plain chunked form
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one served chunk of a long prompt through one recurrent layer of 48 heads
        dict(name="prefill one prompt", op="delta_prefill", dtype="bf16", seqs=1, longest=2048, heads=48, qk_heads=16),
        # a scheduler's mixed batch: prompts of all lengths up to a chunk, some continuing, some new
        dict(name="prefill ragged batch", op="delta_prefill", dtype="bf16", seqs=16, longest=2048, heads=48, qk_heads=16),
        # many short prompts (chat turns), none a multiple of a block, a head of its own for every query
        dict(name="prefill short prompts", op="delta_prefill", dtype="fp16", seqs=37, longest=130, heads=32, qk_heads=32),
        # the next token of the 70 requests that the served configuration holds
        dict(name="step batch", op="delta_step", dtype="bf16", seqs=70, new=1, heads=48, qk_heads=16, rows=False),
        # a single stream: latency
        dict(name="step one request", op="delta_step", dtype="bf16", seqs=1, new=1, heads=48, qk_heads=48, rows=False),
        # a draft of four tokens checked at once, gates per key row
        dict(name="step draft rows", op="delta_step", dtype="fp32", seqs=17, new=4, heads=32, qk_heads=32, rows=True),
        # a prompt chunk written behind a long prefix, the whole read back for dense attention over it
        dict(name="cache chunk", op="kv_cache", dtype="bf16", bits=8, seqs=3, longest=16384, new=2048, kv_heads=8, d=128, page=64),
        # one new token for every request of a batch, small pages
        dict(name="cache tokens", op="kv_cache", dtype="fp16", bits=4, seqs=70, longest=300, new=1, kv_heads=4, d=64, page=16),
        # the decode step of a full batch over ragged contexts
        dict(name="attend batch", op="kv_attend", dtype="bf16", bits=8, seqs=70, longest=8192, new=1, heads=32, kv_heads=8,
             d=128, page=64),
        # one request with a very long context
        dict(name="attend long", op="kv_attend", dtype="bf16", bits=4, seqs=1, longest=131072, new=1, heads=32, kv_heads=8,
             d=128, page=64),
        # a few short chats, three drafted tokens each: latency
        dict(name="attend short drafts", op="kv_attend", dtype="fp16", bits=8, seqs=5, longest=300, new=3, heads=16, kv_heads=4,
             d=64, page=16),
        # wide heads, few of them
        dict(name="attend wide heads", op="kv_attend", dtype="bf16", bits=8, seqs=16, longest=20000, new=1, heads=16, kv_heads=2,
             d=256, page=32),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_prefill", "delta_step", "kv_cache", "kv_attend"])
    if op == "delta_prefill":
        qk, group = rng.choice([(16, 3), (16, 1), (8, 2), (32, 1), (5, 4), (16, 2)])
        longest = _log_int(rng, 1, 2048)
        seqs = _log_int(rng, 1, max(1, min(64, 16 * 2048 * 48 // (longest * qk * group * 2))))
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "bf16"]), seqs=seqs, longest=longest, heads=qk * group, qk_heads=qk)
    if op == "delta_step":
        qk, group = rng.choice([(16, 3), (32, 1), (8, 2), (16, 2), (5, 1)])
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), seqs=_log_int(rng, 1, 64), new=rng.choice([1, 1, 2, 4, 7]),
                    heads=qk * group, qk_heads=qk, rows=rng.random() < 0.3)
    d = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    bits = rng.choice([8, 4])
    dtype = rng.choice(["bf16", "fp16", "bf16", "fp32"])
    page = rng.choice([16, 32, 64, 128])
    if op == "kv_cache":
        longest = _log_int(rng, 4, 16384)
        seqs = _log_int(rng, 1, max(1, min(70, 3 * 16384 * 8 * 128 // (2 * longest * kv_heads * d))))
        return dict(op=op, dtype=dtype, bits=bits, seqs=seqs, longest=longest, new=_log_int(rng, 1, longest), kv_heads=kv_heads,
                    d=d, page=page)
    longest = _log_int(rng, 4, 100000)
    seqs = _log_int(rng, 1, max(1, min(96, 70 * 8192 * 8 * 128 // (4 * longest * kv_heads * d))))
    return dict(op=op, dtype=dtype, bits=bits, seqs=seqs, longest=longest, new=rng.choice([1, 1, 1, 2, 3, 5]),
                heads=kv_heads * rng.choice([1, 2, 4, 7, 8]), kv_heads=kv_heads, d=d, page=page)


def _lengths(case):
    """Length of every sequence: the first has `longest` tokens, the others are spread below it."""
    longest, seqs = case["longest"], case["seqs"]
    rng = random.Random(1000 * seqs + longest)
    return [longest] + [rng.randint(max(1, longest // 8), longest) for _ in range(seqs - 1)]


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"].startswith("delta"):
        n, h, hk = case["seqs"], case["heads"], case["qk_heads"]
        tokens = sum(_lengths(case)) if case["op"] == "delta_prefill" else n * case["new"]
        gates = D if case.get("rows") else 1
        read = tokens * ((2 * hk + h) * D * e + h * (gates + 1) * 4) + n * h * D * D * 4
        wrote = tokens * h * D * e + n * h * D * D * 4
        # S'k, S q and the update: three products of D x D a token and head
        return {"bytes": read + wrote, "flops": tokens * h * 6 * D * D}
    lens, h, d, new = _lengths(case), case["kv_heads"], case["d"], case["new"]
    row = d * case["bits"] // 8 + 4                        # codes and the scale of one key or value row
    if case["op"] == "kv_cache":
        fresh = sum(min(new, x) for x in lens)
        return {"bytes": 2 * h * (fresh * (d * e + row) + sum(lens) * (row + d * e)), "flops": 4 * h * d * (fresh + sum(lens))}
    hq = case["heads"]
    return {"bytes": 2 * h * sum(lens) * row + 2 * len(lens) * new * hq * d * e, "flops": 4 * sum(lens) * new * hq * d}


# ---- inputs ----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _prepare_delta(case, seed):
    g, dt = _gen(seed), TYPES[case["dtype"]]
    n, h, hk = case["seqs"], case["heads"], case["qk_heads"]
    ragged = case["op"] == "delta_prefill"
    lens = _lengths(case) if ragged else [case["new"]] * n
    tokens = sum(lens)
    # one row per token as the fused input projection writes it: q | k | v
    x = torch.empty(tokens, (2 * hk + h) * D, dtype=dt, device="cuda")
    x[:, :hk * D] = _normal(g, tokens, hk * D) * D ** -0.5
    key = _normal(g, tokens, hk, D)
    x[:, hk * D:2 * hk * D] = (key / key.norm(dim=-1, keepdim=True)).reshape(tokens, hk * D)
    x[:, 2 * hk * D:] = _normal(g, tokens, h * D)
    del key
    gates = (tokens, h, D) if case.get("rows") else (tokens, h)
    half = torch.exp(math.log(4.0) + (math.log(20000.0) - math.log(4.0)) * _uniform(g, *gates[1:]))
    alpha = torch.exp(-math.log(2.0) / half * (0.5 + _uniform(g, *gates)))
    beta = _uniform(g, tokens, h)
    slots = torch.randperm(n + 1, generator=g, device="cuda")[:n].to(torch.int32)   # one slot stays idle
    pool = _normal(g, n + 1, 1, h, D, D) * 0.5
    s = dict(case=case, lens=lens, x=x, alpha=alpha, beta=beta, slots=slots, pool=pool,
             q=x[:, :hk * D].view(tokens, hk, D), k=x[:, hk * D:2 * hk * D].view(tokens, hk, D),
             v=x[:, 2 * hk * D:].view(tokens, h, D), o=torch.empty(tokens, h, D, dtype=dt, device="cuda"))
    if ragged:
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["fresh"] = (torch.arange(n, device="cuda") % 3 == 1).to(torch.uint8)       # every third prompt is a new one
    else:
        for name in ("q", "k", "v", "o", "alpha", "beta"):
            s[name] = s[name].unflatten(0, (n, case["new"]))
    if own:
        from quantized_recurrent_state_b200 import stepq
        plan = stepq.Plan.build_uniform(1 if case.get("rows") else 0, 1, h, D, 6)
        s["ctx"] = stepq.Context(plan, n + 1)
    return s


def _quantise(x, bits):
    """Codes and row scales of x [..., d]: r = max|x| / qmax (1 for a row of zeros), the nearest integer to x * fl(1 / r)."""
    qmax = 2 ** (bits - 1) - 1
    x = x.float()
    r = x.abs().amax(-1) / torch.full((), qmax, device=x.device)     # a division, rounded once
    r = torch.where(r < torch.finfo(torch.float32).tiny, torch.ones_like(r), r)
    # ties and near-ties of the product are decided in 64 bits
    z = torch.round(x.double() * (1.0 / r).double().unsqueeze(-1)).clamp(-qmax, qmax)
    return z.to(torch.int8), r


def _prepare_kv(case, seed):
    g, dt = _gen(seed), TYPES[case["dtype"]]
    lens, new, h, d, page = _lengths(case), case["new"], case["kv_heads"], case["d"], case["page"]
    n = len(lens)
    pages = [-(-x // page) for x in lens]
    n_pages, most = sum(pages) + 1, max(pages)
    order = torch.randperm(n_pages, generator=g, device="cuda")
    table = torch.zeros(n, most, dtype=torch.int32, device="cuda")
    at = 0
    for i, c in enumerate(pages):
        table[i, :c] = order[at:at + c].to(torch.int32)
        at += c
    length = torch.tensor(lens, device="cuda", dtype=torch.int32)
    # the flat place of every token, sequence by sequence
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), length.long())
    start = torch.tensor([0] + lens, device="cuda").cumsum(0)
    pos = torch.arange(int(sum(lens)), device="cuda") - start[seq]
    place = table[seq, pos // page].long() * page + pos % page
    k, v = (_normal(g, sum(lens), h, d) for _ in range(2))
    k[..., :2] *= 8.0                                       # a few channels of the keys stand out
    k, v = k.to(dt), v.to(dt)
    fresh = pos >= (length.long()[seq] - new)               # tokens of this call; the others are in the cache already
    append = case["op"] == "kv_cache"
    before = ~fresh if append else torch.ones_like(fresh)
    s = dict(case=case, n=n, table=table, lens=length, place=place, cu=start.to(torch.int32))
    if append:
        s.update(k_new=k[fresh], v_new=v[fresh], place_new=place[fresh].contiguous())
        s.update(k_out=torch.empty_like(k), v_out=torch.empty_like(v))
    else:
        s.update(q=_normal(g, n, new, case["heads"], d).to(dt), scale=d ** -0.5)
        s.update(o=torch.empty_like(s["q"]), lse=torch.empty(n, new, case["heads"], device="cuda"))
    if own:
        from quantized_recurrent_state_b200 import stepq
        kv = stepq.KVCache(case["bits"], h, d, page, n_pages)
        cache = torch.zeros(kv.bytes, dtype=torch.uint8, device="cuda")
        kv.append(cache, k[before], v[before], place[before].contiguous())
        s.update(kv=kv, cache=cache)
        if not append:
            s["workspace"] = torch.empty(kv.attend_workspace_bytes(n, new, case["heads"], most), dtype=torch.uint8, device="cuda")
    else:
        s["codes"] = torch.zeros(2, n_pages * page, h, d, dtype=torch.int8, device="cuda")
        s["scales"] = torch.ones(2, n_pages * page, h, device="cuda")
        for i, x in enumerate((k, v)):
            for part in before.nonzero()[:, 0].split(1 << 16):
                s["codes"][i, place[part]], s["scales"][i, place[part]] = _quantise(x[part], case["bits"])
    return s


def prepare(case, seed):
    return _prepare_delta(case, seed) if case["op"].startswith("delta") else _prepare_kv(case, seed)


# ---- plain forms -----------------------------------------------------------

def _plain_prefill(s):
    """Blocks of CHUNK tokens: U = T (V - gamma K S), O = gamma Q S + A U, S = gamma_C S + K^T diag(gamma_C / gamma) U."""
    n, h, hk, lens = s["case"]["seqs"], s["case"]["heads"], s["case"]["qk_heads"], s["lens"]
    blocks = -(-max(lens) // CHUNK)
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(lens, device="cuda"))
    pos = torch.arange(sum(lens), device="cuda") - s["cu"].long()[seq]

    def padded(x, fill):                                    # [tokens, heads, ...] -> [n, blocks, h, CHUNK, ...] in fp32
        y = torch.full((n, blocks * CHUNK) + x.shape[1:], fill, device="cuda")
        y[seq, pos] = x.float()
        return y.unflatten(1, (blocks, CHUNK)).transpose(2, 3)

    k, q = (padded(s[x], 0.0).repeat_interleave(h // hk, dim=2) for x in ("k", "q"))
    v, beta = padded(s["v"], 0.0), padded(s["beta"], 0.0)
    lg = torch.log(padded(s["alpha"], 1.0).double()).cumsum(-1)
    gamma, last = torch.exp(lg).float(), torch.exp(lg[..., -1:] - lg).float()
    ratio = torch.exp((lg.unsqueeze(-1) - lg.unsqueeze(-2)).clamp(max=0.0)).float()
    lower = (beta.unsqueeze(-1) * ratio * (k @ k.transpose(-1, -2))).tril(-1)
    a = (ratio * (q @ k.transpose(-1, -2))).tril()
    del ratio
    t = torch.diag_embed(beta)                              # T = (I + lower)^-1 diag(beta), row after row
    for i in range(1, CHUNK):
        t[..., i, :] -= (lower[..., i, :i].unsqueeze(-2) @ t[..., :i, :]).squeeze(-2)
    state = s["pool"][s["slots"].long(), 0] * (s["fresh"] == 0).view(n, 1, 1, 1)
    o = torch.empty_like(v)
    for c in range(blocks):
        g = gamma[:, c].unsqueeze(-1)
        u = t[:, c] @ (v[:, c] - g * (k[:, c] @ state))
        o[:, c] = g * (q[:, c] @ state) + a[:, c] @ u
        state = gamma[:, c, :, -1, None, None] * state + k[:, c].transpose(-1, -2) @ (last[:, c].unsqueeze(-1) * u)
    s["pool"][s["slots"].long(), 0] = state
    return [o.transpose(2, 3).flatten(1, 2)[seq, pos].to(s["o"].dtype), s["pool"]]


def _plain_step(s):
    case, rep = s["case"], s["case"]["heads"] // s["case"]["qk_heads"]
    state = s["pool"][s["slots"].long(), 0]
    o = []
    for i in range(case["new"]):
        k, q = (s[x][:, i].float().repeat_interleave(rep, dim=1) for x in ("k", "q"))
        alpha = s["alpha"][:, i]
        state = state * (alpha.unsqueeze(-1) if case["rows"] else alpha[..., None, None])
        u = s["beta"][:, i].unsqueeze(-1) * (s["v"][:, i].float() - (k.unsqueeze(-1) * state).sum(-2))
        state = state + k.unsqueeze(-1) * u.unsqueeze(-2)
        o.append((q.unsqueeze(-1) * state).sum(-2))
    s["pool"][s["slots"].long(), 0] = state
    return [torch.stack(o, 1).to(s["o"].dtype), s["pool"]]


def _plain_cache(s):
    out = []
    for i, x in enumerate((s["k_new"], s["v_new"])):
        s["codes"][i, s["place_new"]], s["scales"][i, s["place_new"]] = _quantise(x, s["case"]["bits"])
        out.append((s["codes"][i, s["place"]].float() * s["scales"][i, s["place"]].unsqueeze(-1)).to(x.dtype))
    return out


def _plain_attend(s):
    case, page = s["case"], s["case"]["page"]
    n, new, h, hq = s["n"], case["new"], case["kv_heads"], case["heads"]
    place = (s["table"].long().unsqueeze(-1) * page + torch.arange(page, device="cuda")).flatten(1)   # [n, most]
    at = torch.arange(place.shape[1], device="cuda")
    q = s["q"].float().view(n, new, h, hq // h, case["d"]).permute(0, 2, 1, 3, 4).flatten(2, 3)       # [n, h, new * group, d]
    score = s["codes"][0, place].float().permute(0, 2, 3, 1)                                          # [n, h, d, most]
    score = (q @ score) * (s["scales"][0, place].permute(0, 2, 1).unsqueeze(2) * s["scale"])
    newest = s["lens"].long().unsqueeze(1) - new + torch.arange(new, device="cuda")                   # [n, new]
    seen = (at <= newest.repeat_interleave(hq // h, dim=1).unsqueeze(-1)).unsqueeze(1)                # [n, 1, new * group, most]
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    del score
    total = p.sum(-1, keepdim=True)
    v = s["codes"][1, place].float().permute(0, 2, 1, 3)
    o = (p * s["scales"][1, place].permute(0, 2, 1).unsqueeze(2)) @ v
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (torch.log(total) + top).squeeze(-1)

    def rows(x):                                            # [n, h, new * group, ...] -> [n, new, hq, ...]
        return x.unflatten(2, (new, hq // h)).transpose(1, 2).flatten(2, 3)

    return [rows(o).to(s["o"].dtype), rows(lse)]


PLAIN = {"delta_prefill": _plain_prefill, "delta_step": _plain_step, "kv_cache": _plain_cache, "kv_attend": _plain_attend}


# ---- the library's calls ----------------------------------------------------

def _own_prefill(s):
    s["ctx"].delta_prefill(s["pool"], s["slots"], s["cu"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["o"], fresh=s["fresh"])
    return [s["o"], s["pool"]]


def _own_step(s):
    s["ctx"].delta_step(s["pool"], s["slots"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["o"])
    return [s["o"], s["pool"]]


def _own_cache(s):
    s["kv"].append(s["cache"], s["k_new"], s["v_new"], s["place_new"])
    s["kv"].read(s["cache"], s["table"], s["lens"], s["cu"], s["k_out"], s["v_out"])
    return [s["k_out"], s["v_out"]]


def _own_attend(s):
    s["kv"].attend(s["cache"], s["q"], s["table"], s["lens"], s["scale"], s["o"], s["workspace"], lse=s["lse"])
    return [s["o"], s["lse"]]


OWN = {"delta_prefill": _own_prefill, "delta_step": _own_step, "kv_cache": _own_cache, "kv_attend": _own_attend}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---- in 64 bits ------------------------------------------------------------

def _exact_delta(s):
    """Token after token: S = alpha S, u = beta (v - S^T k), S = S + k u^T, o = S^T q."""
    case = s["case"]
    n, h, hk = case["seqs"], case["heads"], case["qk_heads"]
    if case["op"] == "delta_prefill":
        first, lens = s["cu"].long()[:-1], torch.tensor(s["lens"], device="cuda")
        state = s["pool"].double()[s["slots"].long(), 0]
        state[s["fresh"].bool()] = 0.0
        q, k, v, alpha, beta = (s[x] for x in ("q", "k", "v", "alpha", "beta"))
    else:
        first, lens = torch.arange(n, device="cuda") * case["new"], torch.full((n,), case["new"], device="cuda")
        state = s["pool"].double()[s["slots"].long(), 0]
        q, k, v, alpha, beta = (s[x].flatten(0, 1) for x in ("q", "k", "v", "alpha", "beta"))
    o = torch.zeros(q.shape[0], h, D, dtype=torch.float64, device="cuda")
    head = torch.arange(h, device="cuda") // (h // hk)
    longest = int(lens.max())
    order = torch.argsort(lens, descending=True)             # the sequences still running stand in front
    state, first, count = state[order], first[order], (lens.unsqueeze(0) > torch.arange(longest, device="cuda").unsqueeze(1)).sum(1).tolist()
    for t in range(longest):
        m = count[t]
        at = first[:m] + t
        kt, qt = k[at][:, head].double(), q[at][:, head].double()
        a = alpha[at].double()
        live = state[:m]
        live *= a.unsqueeze(-1) if case.get("rows") else a[..., None, None]
        u = beta[at].double().unsqueeze(-1) * (v[at].double() - torch.einsum("nhi,nhij->nhj", kt, live))
        live += kt.unsqueeze(-1) * u.unsqueeze(-2)
        o[at] = torch.einsum("nhi,nhij->nhj", qt, live)
    pool = s["pool"].double()
    pool[s["slots"].long()[order], 0] = state
    return [o if case["op"] == "delta_prefill" else o.unflatten(0, (n, case["new"])), pool]


def _exact_rows(codes, scales):
    return codes.double() * scales.double().unsqueeze(-1)


def _exact_cache(s):
    qmax, out = 2 ** (s["case"]["bits"] - 1) - 1, []
    for i, x in enumerate((s["k_new"], s["v_new"])):
        old = _exact_rows(s["codes"][i], s["scales"][i])
        r = (x.double().abs().max(-1, keepdim=True).values / torch.tensor(qmax, device="cuda", dtype=torch.float64)).float()
        r = torch.where(r < 2.0 ** -126, torch.ones((), device="cuda"), r)
        z = (x.double() * (1 / r).double()).round()
        old[s["place_new"]] = z.clamp(-qmax, qmax) * r.double()
        out.append(old[s["place"]])
    return out


def _exact_attend(s):
    case = s["case"]
    new, h, hq, page = case["new"], case["kv_heads"], case["heads"], case["page"]
    o = torch.zeros(s["n"], new, hq, case["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((s["n"], new, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["lens"].tolist()):
        at = torch.arange(length, device="cuda")
        at = s["table"][i].long()[at // page] * page + at % page
        k, v = (_exact_rows(s["codes"][j, at], s["scales"][j, at]) for j in (0, 1))
        for t in range(new):
            m = length - new + t + 1
            if m <= 0:
                continue
            q = s["q"][i, t].double().view(h, hq // h, case["d"])
            score = torch.einsum("hgd,mhd->hgm", q, k[:m]) * s["scale"]
            lse[i, t] = torch.logsumexp(score, -1).flatten()
            o[i, t] = torch.einsum("hgm,mhd->hgd", torch.softmax(score, -1), v[:m]).reshape(hq, -1)
    return [o, lse]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("delta"):
        return _exact_delta(s)
    return (_exact_cache if case["op"] == "kv_cache" else _exact_attend)(s)
