"""Attention with its positions and gradients, and a loss on a teacher's top logits: their cases, plain
forms, and calls.

Four operators of a training step's forward and backward pass:

``rotary``    queries and keys turned by angles from their positions on one to three axes (the backward pass
              makes the same call with the angles reversed)
``attention`` out = softmax(scale q k^T) v for every sequence and head, and the logarithm of each row's sum
``attngrad``  its backward pass: dq, dk and dv, from probabilities computed again
``distill``   the divergence from a teacher's top logits with the cross entropy of the labels, and the
              gradient of the student's logits

Sequences lie one behind the other in a tensor of rows, at equal lengths or at the rows that ``offsets`` name.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------
def listed():
    return [
        # a short prompt of the 124M layout (12 heads of 64): one small launch, latency alone
        dict(name="rotary_few", op="rotary", tokens=64, heads=12, kv_heads=12, dim=64, axes=1, rot=64, own_ladder=False,
             interleaved=False, inverse=False, far=0, dtype="bf16"),
        # frames of a video at the 7B layout's width, grouped keys, positions far along the time axis
        dict(name="rotary_video", op="rotary", tokens=16383, heads=32, kv_heads=8, dim=128, axes=3, rot=128,
             own_ladder=False, interleaved=False, inverse=True, far=1000000, dtype="f16"),
        # a short prompt of the 124M layout
        dict(name="attention_few", op="attention", tokens=77, tokens_k=0, sequences=1, ragged=False, heads=12, kv_heads=12,
             dim=64, causal=True, window=0, dtype="bf16"),
        # a micro-step of the 124M layout: 8 replicas, 4 sequences of 1024 tokens each
        dict(name="attention_gpt2", op="attention", tokens=32768, tokens_k=0, sequences=32, ragged=False, heads=12,
             kv_heads=12, dim=64, causal=True, window=0, dtype="f16"),
        # a packed batch of documents with grouped keys and a sliding window, padded at its end
        dict(name="attention_packed", op="attention", tokens=8191, tokens_k=0, sequences=9, ragged=True, heads=32, kv_heads=8,
             dim=80, causal=True, window=1000, dtype="bf16"),
        # a micro-step of the 7B layout: 4 sequences of 4096 tokens, 32 heads of 128
        dict(name="attention_7b", op="attention", tokens=16384, tokens_k=0, sequences=4, ragged=False, heads=32,
             kv_heads=32, dim=128, causal=True, window=0, dtype="bf16"),
        # the backward pass of the 124M layout's micro-step
        dict(name="attngrad_gpt2", op="attngrad", tokens=32768, tokens_k=0, sequences=32, ragged=False, heads=12,
             kv_heads=12, dim=64, causal=True, window=0, dtype="f16"),
        # of the packed batch
        dict(name="attngrad_packed", op="attngrad", tokens=8191, tokens_k=0, sequences=9, ragged=True, heads=32, kv_heads=8,
             dim=80, causal=True, window=1000, dtype="bf16"),
        # of two sequences of the 7B layout
        dict(name="attngrad_7b", op="attngrad", tokens=8192, tokens_k=0, sequences=2, ragged=False, heads=32, kv_heads=32,
             dim=128, causal=True, window=0, dtype="bf16"),
        # the last, ragged part of a batch over the 50257-token table, labels beside the teacher
        dict(name="distill_few", op="distill", tokens=61, vocab=50257, top=20, tail=False, temperature=2.0, soft=0.9,
             hard=0.1, grad=True, dtype="bf16"),
        # evaluation over the 50257-token table in 32 bits: the loss alone
        dict(name="distill_eval", op="distill", tokens=4096, vocab=50257, top=100, tail=False, temperature=2.0, soft=1.0,
             hard=0.0, grad=False, dtype="f32"),
        # a micro-step of the 7B layout's table with the teacher's remaining probability as one more class
        dict(name="distill_7b", op="distill", tokens=16384, vocab=32000, top=64, tail=True, temperature=1.0, soft=1.0,
             hard=0.0, grad=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm; every other one as it falls, else on a grid of 8."""
    x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and x > 64:
        x = x // 8 * 8
    return max(lo, min(hi, x))


def draw(rng):
    op = rng.choice(["rotary", "attention", "attention", "attngrad", "attngrad", "distill"])
    if op == "rotary":
        dim = rng.choice([32, 64, 80, 96, 128])
        kv = rng.choice([1, 2, 4, 8])
        axes = rng.choice([1, 2, 3])
        return dict(op=op, tokens=_log(rng, 1, 16384), heads=kv * rng.choice([1, 2, 4]), kv_heads=kv, dim=dim, axes=axes,
                    rot=rng.choice([dim, dim // 4 * 2]), own_ladder=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, far=rng.choice([0, 5000, 1000000]), dtype=rng.choice(["bf16", "f16", "f32"]))
    if op in ("attention", "attngrad"):
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4])
        while heads > (16 if op == "attention" else 8):
            heads -= kv
        tokens, keys, ragged = _log(rng, 1, 8000), rng.choice([0, 0, 0, _log(rng, 1, 8000)]), rng.random() < 0.7
        sequences = min(tokens, rng.choice([1, 1, 2, 3, 7, 16]))
        if not ragged:  # of equal lengths
            tokens, keys = tokens // sequences * sequences, -(-keys // sequences) * sequences
        return dict(op=op, tokens=tokens, tokens_k=keys, sequences=sequences, ragged=ragged, heads=heads, kv_heads=kv,
                    dim=rng.choice([32, 64, 64, 80, 96, 128, 128]), causal=rng.random() < 0.7,
                    window=rng.choice([0, 0, 100, 1024]),
                    dtype=rng.choice(["bf16", "f16"]))
    vocab = _log(rng, 1000, 131072)
    return dict(op=op, tokens=_log(rng, 1, min(8192, (1 << 28) // vocab)), vocab=vocab, top=_log(rng, 1, 256),
                tail=rng.random() < 0.5, temperature=rng.choice([1.0, 2.0, 0.7]), soft=rng.choice([1.0, 0.5]),
                hard=rng.choice([0.0, 0.5]), grad=rng.random() < 0.7, dtype=rng.choice(["bf16", "f16", "f32"]))


def _spans(c, keys):
    """The rows [begin, end) of every sequence, among the queries or the keys."""
    T, S = c["tokens_k"] if keys and c["tokens_k"] else c["tokens"], c["sequences"]
    if not c["ragged"]:
        return [(s * (T // S), (s + 1) * (T // S)) for s in range(S)]
    rng = random.Random(1000 * T + S)
    used = T - T // 64  # some rows behind the last sequence
    cuts = sorted(rng.randint(0, used) for _ in range(S - 1))
    if S >= 4:
        cuts[1] = cuts[0]  # one sequence without a token
    return list(zip([0, *cuts], [*cuts, used]))


def _pairs(c):
    """How many pairs of a query and a key the mask leaves, over all sequences."""
    n = 0
    for (a, b), (e, f) in zip(_spans(c, False), _spans(c, True)):
        if b == a or f == e:
            continue
        last = torch.arange(b - a, dtype=torch.int64) + (f - e) - (b - a)
        hi = last.clamp(max=f - e - 1) if c["causal"] else torch.full_like(last, f - e - 1)
        lo = (last - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(last)
        n += int((hi - lo + 1).clamp(min=0).sum())
    return n


def work(case):
    c, op, T = case, case["op"], case["tokens"]
    e = 4 if c["dtype"] == "f32" else 2
    if op == "distill":
        passes = 2 if c["grad"] else 1
        return dict(bytes=passes * T * c["vocab"] * e + T * (c["top"] * (e + 4) + 4), flops=T * c["vocab"] * (8 if c["grad"] else 4))
    H, K, D = c["heads"], c["kv_heads"], c["dim"]
    if op == "rotary":
        return dict(bytes=2 * T * (H + K) * D * e + T * c["axes"] * 8, flops=3 * T * (H + K) * D)
    Tk = c["tokens_k"] or T
    q, kv = T * H * D * e, Tk * K * D * e
    if op == "attention":
        return dict(bytes=2 * q + 2 * kv + 4 * T * H, flops=4 * D * H * _pairs(c))
    return dict(bytes=4 * q + 4 * kv + 4 * T * H, flops=10 * D * H * _pairs(c))


# ---- inputs --------------------------------------------------------------------------------------
def _normal(g, shape, sigma, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _sections(c):
    """How many pairs of elements turn with each axis."""
    pairs, axes = c["rot"] // 2, c["axes"]
    rest = pairs // axes
    return (pairs - rest * (axes - 1),) + (rest,) * (axes - 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, dt, op, T = case, DTYPES[case["dtype"]], case["op"], case["tokens"]
    s = dict(case=case, scale=1024.0 if case["dtype"] == "f16" else 1.0)  # the loss scale that 16 bits of range need
    if op == "distill":
        V, K = c["vocab"], c["top"]
        start = torch.randint(0, V, (T, 1), generator=g, device="cuda")
        step = V // K if V % K else max(1, V // K - 1)
        ids = (start + step * torch.arange(K, device="cuda")) % V  # no token twice in a row
        falls = torch.empty((T, K), device="cuda").exponential_(1.0, generator=g)
        teacher = 12.0 - (falls * (8.0 / K)).cumsum(1)
        # the lists of some rows are shorter
        short = torch.rand((T, 1), generator=g, device="cuda") < 1 / 16
        s["teacher"] = teacher.to(dt)
        s["ids"] = torch.where(short & (torch.arange(K, device="cuda") >= (K + 1) // 2), -1, ids)
        logits = torch.randn((T, V), generator=g, device="cuda") * 2.0
        logits.scatter_add_(1, ids, teacher * 0.6)
        s["logits"] = logits.to(dt)
        del logits
        if c["tail"]:
            held = 0.8 + 0.15 * torch.rand((T,), generator=g, device="cuda")
            lists = torch.where(s["ids"] >= 0, s["teacher"].double() / c["temperature"], -math.inf)
            s["total"] = (torch.logsumexp(lists, 1) - held.double().log()).float()
        if c["hard"]:
            pad = torch.rand((T,), generator=g, device="cuda") < 1 / 16
            s["labels"] = torch.where(pad, -100, ids[:, 0])
        skip = torch.rand((T,), generator=g, device="cuda") < 1 / 16
        s["weight"] = torch.where(skip, 0.0, 1.0 / T)
        s["loss"] = torch.empty((T,), device="cuda")
        if c["grad"]:
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    H, K, D = c["heads"], c["kv_heads"], c["dim"]
    if op == "rotary":
        # the rows of one projection: queries, keys and values side by side
        rows = _normal(g, (T, (H + 2 * K) * D), 1.5, dt)
        s["q"], s["k"] = rows[:, :H * D].view(T, H, D), rows[:, H * D:(H + K) * D].view(T, K, D)
        s["out"] = [torch.empty((T, n, D), dtype=dt, device="cuda") for n in (H, K)]
        t = torch.arange(T, device="cuda")
        where = [t] if c["axes"] == 1 else [t // 391, t % 391] if c["axes"] == 2 else [t // 391, t % 391 // 23, t % 23]
        where[0] = where[0] + int(torch.randint(0, c["far"] + 1, (1,), generator=g, device="cuda"))
        s["positions"] = torch.stack(where, 1)
        return s
    Tk = c["tokens_k"] or T
    if Tk == T:
        rows = _normal(g, (T, (H + 2 * K) * D), 1.2, dt)
        s["q"] = rows[:, :H * D].view(T, H, D)
        s["k"], s["v"] = rows[:, H * D:].view(T, 2, K, D).unbind(1)
    else:
        s["q"] = _normal(g, (T, H, D), 1.2, dt)
        s["k"], s["v"] = _normal(g, (Tk, 2, K, D), 1.2, dt).unbind(1)
    if c["ragged"]:
        for name, keys in (("offsets", False), ("offsets_k", True)):
            spans = _spans(c, keys)
            s[name] = torch.tensor([a for a, _ in spans] + [spans[-1][1]], dtype=torch.int32, device="cuda")
    s["out"] = torch.zeros((T, H, D), dtype=dt, device="cuda")
    s["lse"] = torch.zeros((H, T), device="cuda")
    if op == "attngrad":
        out, lse = _plain_attention(s, c)
        s["out"].copy_(out)
        s["lse"].copy_(lse)
        s["dout"] = _normal(g, (T, H, D), 1e-2, dt)
        s["dq"] = torch.zeros_like(s["out"])
        s["dk"], s["dv"] = (torch.zeros((Tk, K, D), dtype=dt, device="cuda") for _ in range(2))
    return s


# ---- one pass ------------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return (_OWN if own else _PLAIN)[case["op"]](state, case)


def _plain_rotary(s, c):
    sections, rot = _sections(c), c["rot"]
    freq, axis = [], []
    for a, n in enumerate(sections):
        for i in range(n):
            freq.append(10000.0 ** (-i / n) if c["own_ladder"] else 10000.0 ** (-2 * len(freq) / rot))
            axis.append(a)
    freq = torch.tensor(freq, dtype=torch.float64, device="cuda")
    # angles of far positions need 64 bits
    angle = s["positions"][:, axis].double() * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["inverse"]:
        sin = -sin
    out = []
    for x in (s["q"], s["k"]):
        x = x.float()
        y = x.clone()
        lo = slice(0, rot, 2) if c["interleaved"] else slice(0, rot // 2)
        hi = slice(1, rot, 2) if c["interleaved"] else slice(rot // 2, rot)
        y[..., lo] = x[..., lo] * cos - x[..., hi] * sin
        y[..., hi] = x[..., lo] * sin + x[..., hi] * cos
        out.append(y.to(s["q"].dtype))
    return out


def _hidden(c, L, Lk):
    """True where query i of L does not see key j of Lk: the last query sees the last key, each one before it
    one key less, and none a key more than a window back."""
    if not c["causal"] and not c["window"]:
        return None
    back = torch.arange(L, device="cuda")[:, None] + (Lk - L) - torch.arange(Lk, device="cuda")
    hidden = back < 0 if c["causal"] else torch.zeros_like(back, dtype=torch.bool)
    return hidden | (back >= c["window"]) if c["window"] else hidden


def _by_key_head(x, K):
    """Rows [L, H, D] in 32 bits as [K, (H / K) L, D]: the heads that share keys behind each other."""
    L, H, D = x.shape
    return x.float().transpose(0, 1).reshape(K, H // K * L, D)


def _scores(s, c, q, k):
    K = c["kv_heads"]
    L, Lk = q.shape[0], k.shape[0]
    x = torch.matmul(_by_key_head(q, K), k.float().permute(1, 2, 0).contiguous()) / math.sqrt(c["dim"])
    hidden = _hidden(c, L, Lk)
    return x if hidden is None else x.view(c["heads"], L, Lk).masked_fill(hidden, -math.inf).view(K, -1, Lk)


def _plain_attention(s, c):
    out, lse, H = torch.zeros_like(s["out"]), torch.zeros_like(s["lse"]), c["heads"]
    for (a, b), (e, f) in zip(_spans(c, False), _spans(c, True)):
        if a == b:
            continue
        if e == f:
            lse[:, a:b] = -math.inf
            continue
        x = _scores(s, c, s["q"][a:b], s["k"][e:f])
        top = x.amax(-1, keepdim=True)
        x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        total = x.sum(-1, keepdim=True)
        y = torch.matmul(x, s["v"][e:f].float().transpose(0, 1).contiguous()) / torch.where(total == 0, 1.0, total)
        out[a:b] = y.view(H, b - a, -1).transpose(0, 1).to(out.dtype)
        lse[:, a:b] = (top + total.log()).view(H, b - a)
    return [out, lse]


def _plain_attngrad(s, c):
    K, H = c["kv_heads"], c["heads"]
    dq, dk, dv = (torch.zeros_like(s[x]) for x in ("dq", "dk", "dv"))
    for (a, b), (e, f) in zip(_spans(c, False), _spans(c, True)):
        if a == b or e == f:
            continue
        x = _scores(s, c, s["q"][a:b], s["k"][e:f])
        lse = s["lse"][:, a:b].reshape(K, -1, 1)
        p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse))
        do, kk, vv = _by_key_head(s["dout"][a:b], K), s["k"][e:f].float(), s["v"][e:f].float()
        dv[e:f] = torch.matmul(p.transpose(1, 2).contiguous(), do).transpose(0, 1).to(dv.dtype)
        delta = (do * _by_key_head(s["out"][a:b], K)).sum(-1, keepdim=True)
        ds = p * (torch.matmul(do, vv.permute(1, 2, 0).contiguous()) - delta) / math.sqrt(c["dim"])
        dk[e:f] = torch.matmul(ds.transpose(1, 2).contiguous(), _by_key_head(s["q"][a:b], K)).transpose(0, 1).to(dk.dtype)
        y = torch.matmul(ds, kk.transpose(0, 1).contiguous())
        dq[a:b] = y.view(H, b - a, -1).transpose(0, 1).to(dq.dtype)
    return [dq, dk, dv]


def _log_sum(u):
    """The largest value, the exponentials below it, and the logarithm of their sum, of each row."""
    top = u.amax(1, keepdim=True)
    e = torch.exp(u - top)
    return top, e, top + e.sum(1, keepdim=True).log()


def _plain_distill(s, c):
    tau, V = c["temperature"], c["vocab"]
    z = s["logits"].float()
    top, e, lse = _log_sum(z / tau)
    there = (s["ids"] >= 0) & (s["ids"] < V)
    ids = s["ids"].clamp(0, V - 1)
    t = torch.where(there, s["teacher"].float() / tau, -math.inf)
    logp = t - (s["total"][:, None] if c["tail"] else _log_sum(t)[2])
    p = torch.exp(logp)
    logq = (z.gather(1, ids) / tau) - lse
    kl = torch.where(there & (p > 0), p * (logp - logq), 0.0).sum(1)
    mass = p.sum(1, keepdim=True)
    if c["tail"]:
        rest = (1.0 - mass).clamp(min=0.0)
        # counted, not written, so that a padded place never takes a token's away
        listed_ = torch.zeros_like(z).scatter_add_(1, ids, there.float()) > 0
        others = torch.where(listed_, 0.0, e)
        s_rest = others.sum(1, keepdim=True)
        kl = kl + torch.where(rest > 0, rest * (rest.log() - (s_rest.log() + top - lse)), 0.0)[:, 0]
    soft = c["soft"] * tau * tau * kl
    loss, used = soft, s["weight"] != 0
    if c["hard"]:
        _, e1, lse1 = _log_sum(z)
        seen = (s["labels"] >= 0) & (s["labels"] < V)
        at = s["labels"].clamp(0, V - 1)[:, None]
        loss = loss + c["hard"] * torch.where(seen, (lse1 - z.gather(1, at))[:, 0], 0.0)
    loss = torch.where(used, loss, 0.0)
    if not c["grad"]:
        return loss
    q = e * torch.exp(top - lse)
    d = q * (mass + rest) - others * (rest / s_rest) if c["tail"] else q * mass
    d.scatter_add_(1, ids, torch.where(there, -p, 0.0))
    d = d * (c["soft"] * tau)
    if c["hard"]:
        h = torch.exp(z - lse1)
        h.scatter_add_(1, at, torch.full_like(lse1, -1.0))
        d = d + c["hard"] * torch.where(seen[:, None], h, 0.0)
    return [loss, (d * (s["weight"] * s["scale"])[:, None]).to(s["logits"].dtype)]


_PLAIN = dict(rotary=_plain_rotary, attention=_plain_attention, attngrad=_plain_attngrad, distill=_plain_distill)


# ---- the framework's calls -----------------------------------------------------------------------
def _own_rotary(s, c):
    import gradient_reduce_adam_amd as dp
    if "rotary" not in s:
        s["rotary"] = dp.Rotary(_sections(c), base=10000.0, own_ladder=c["own_ladder"], interleaved=c["interleaved"])
    dp.dpa_rotary(s["rotary"], s["positions"], (s["q"], s["k"]), s["out"], inverse=c["inverse"])
    return s["out"]


def _attention(s, c):
    """The mask and the sequences' places, as the forward and the backward pass take them."""
    if "attention" not in s:
        import gradient_reduce_adam_amd as dp
        s["attention"] = dp.Attention(causal=c["causal"], window=c["window"])
    return s["attention"], dict(sequences=c["sequences"], offsets=s.get("offsets"), offsets_k=s.get("offsets_k"))


def _own_attention(s, c):
    import gradient_reduce_adam_amd as dp
    attention, places = _attention(s, c)
    dp.dpa_attention(attention, s["q"], s["k"], s["v"], s["out"], s["lse"], **places)
    return [s["out"], s["lse"]]


def _own_attngrad(s, c):
    import gradient_reduce_adam_amd as dp
    attention, places = _attention(s, c)
    if "workspace" not in s:
        size = dp.dpa_attention_workspace(c["tokens"], c["heads"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    dp.dpa_attention_backward(attention, s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["dq"], s["dk"],
                              s["dv"], s["workspace"], **places)
    return [s["dq"], s["dk"], s["dv"]]


def _own_distill(s, c):
    import gradient_reduce_adam_amd as dp
    if "distill" not in s:
        s["distill"] = dp.Distillation(temperature=c["temperature"], soft=c["soft"], hard=c["hard"])
    dp.dpd_distill(s["distill"], s["logits"], s["teacher"], s["ids"], s["loss"], s.get("dlogits"), total=s.get("total"),
                   labels=s.get("labels"), weight=s["weight"], scale=s["scale"])
    return [s["loss"], s["dlogits"]] if c["grad"] else s["loss"]


_OWN = dict(rotary=_own_rotary, attention=_own_attention, attngrad=_own_attngrad, distill=_own_distill)


# ---- the definitions in 64 bits ------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s, case)
    if case["op"] == "distill":
        return _exact_distill(s, case)
    return _exact_attention(s, case)


def _exact_rotary(s, c):
    """Pairs as complex numbers times e^(i angle)."""
    sections, rot, first = _sections(c), c["rot"], 0
    angle = []
    for a, n in enumerate(sections):
        i = torch.arange(n, device="cuda", dtype=torch.float64)
        power = i / n if c["own_ladder"] else (first + i) * 2 / rot
        angle.append(s["positions"][:, a, None].double() * torch.exp(-power * math.log(10000.0)))
        first += n
    turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), torch.cat(angle, 1))[:, None]
    turn = turn.conj() if c["inverse"] else turn
    out = []
    for x in (s["q"], s["k"]):
        x = x.double()
        part = x[..., :rot]
        if c["interleaved"]:
            y = torch.view_as_real(torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
        else:
            z = torch.complex(part[..., :rot // 2].contiguous(), part[..., rot // 2:].contiguous()) * turn
            y = torch.cat([z.real, z.imag], -1)
        out.append(torch.cat([y, x[..., rot:]], -1))
    return out


def _exact_attention(s, c):
    """Sequence by sequence and head by head."""
    f64 = dict(device="cuda", dtype=torch.float64)
    group, H, T = c["heads"] // c["kv_heads"], c["heads"], c["tokens"]
    out, lse = torch.zeros((T, H, c["dim"]), **f64), torch.zeros((H, T), **f64)
    dq, dk, dv = (torch.zeros(s[x].shape, **f64) for x in ("q", "k", "v"))
    for (a, b), (e, f) in zip(_spans(c, False), _spans(c, True)):
        if a == b:
            continue
        i = torch.arange(a, b, device="cuda")[:, None] - b
        j = torch.arange(e, f, device="cuda")[None, :] - f
        seen = torch.ones((b - a, f - e), dtype=torch.bool, device="cuda")
        if c["causal"]:
            seen &= j <= i
        if c["window"]:
            seen &= j > i - c["window"]
        for h in range(H):
            q, k, v = s["q"][a:b, h].double(), s["k"][e:f, h // group].double(), s["v"][e:f, h // group].double()
            x = torch.where(seen, torch.mm(q, k.t().contiguous()) * c["dim"] ** -0.5, -math.inf)
            if f > e:
                lse[h, a:b] = torch.logsumexp(x, 1)
            else:
                lse[h, a:b] = -math.inf
            p = torch.where(seen, torch.exp(x - lse[h, a:b, None]), 0.0)
            out[a:b, h] = torch.mm(p, v)
            if c["op"] == "attention":
                continue
            do = s["dout"][a:b, h].double()
            dp = torch.mm(do, v.t().contiguous())
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) * c["dim"] ** -0.5
            dq[a:b, h] = torch.mm(ds, k)
            dk[e:f, h // group] += torch.mm(ds.t().contiguous(), q)
            dv[e:f, h // group] += torch.mm(p.t().contiguous(), do)
    return [out, lse] if c["op"] == "attention" else [dq, dk, dv]


def _exact_distill(s, c):
    """The loss by its formula, a block of rows at a time, and the gradient by differentiating it."""
    tau, V, T = c["temperature"], c["vocab"], c["tokens"]
    loss = torch.zeros((T,), dtype=torch.float64, device="cuda")
    grad = torch.zeros((T, V), dtype=torch.float64, device="cuda") if c["grad"] else None
    block = max(1, (1 << 26) // V)
    for a in range(0, T, block):
        b = min(T, a + block)
        z = s["logits"][a:b].double().requires_grad_(c["grad"])
        ids, w = s["ids"][a:b], s["weight"][a:b].double()
        there = (ids >= 0) & (ids < V)
        at = torch.where(there, ids, V)
        t = torch.where(there, s["teacher"][a:b].double() / tau, -math.inf)
        logp = t - (s["total"][a:b, None].double() if c["tail"] else torch.logsumexp(t, 1, keepdim=True))
        p = torch.exp(logp)
        logq = torch.log_softmax(z / tau, 1)
        picked = torch.cat([logq, torch.zeros_like(logq[:, :1])], 1).gather(1, at)
        kl = torch.where(there, p * (torch.where(there, logp, 0.0) - picked), 0.0).sum(1)
        if c["tail"]:
            rest = (1 - p.sum(1)).clamp(min=1e-300)
            mark = torch.zeros((b - a, V + 1), dtype=torch.bool, device="cuda").scatter_(1, at, True)[:, :V]
            kl = kl + rest * (rest.log() - torch.logsumexp(logq.masked_fill(mark, -math.inf), 1))
        total = c["soft"] * tau * tau * kl
        if c["hard"]:
            y = s["labels"][a:b]
            seen = (y >= 0) & (y < V)
            ce = -torch.log_softmax(z, 1).gather(1, y.clamp(0, V - 1)[:, None])[:, 0]
            total = total + c["hard"] * torch.where(seen, ce, 0.0)
        total = torch.where(w != 0, total, 0.0)
        loss[a:b] = total.detach()
        if c["grad"]:
            grad[a:b] = torch.autograd.grad(total, z, w * s["scale"])[0]
    return [loss, grad] if c["grad"] else loss
