"""The attention's definition in 64 bits, head by head, with bounds on what a binary32 evaluation with 16-bit
probabilities may be off by.

Bounds (u: half a step of the type relative to the value, 2^-8 for bf16 and 2^-11 for f16; e = 2^-24):
 - a score is a sum of D exact products, in any order, each partial sum off by at most a whole last place: 2 (D + 2) e
   sum |q k| scale; its multiple of log2(e) and the difference from the maximum or lse add at most 4 e (|score| +
   |lse|), the exponential 4 e: a probability is off by r = the sum of these, relative to it (twice, as the row's
   sum is too).
 - p and ds are rounded to the type: u of the value, and below f16's smallest normal number half a step, 2^-25.
 - binary32 exponentials and matrix instructions give 0 for results below the smallest normal number: a probability, and
   a bf16 value, whose range is the same, may lose up to 2^-126, and ds that times |dp| + |delta|.
 - sums over n keys or queries: 2 (n + 4) e of the sum of magnitudes.
 - the result is rounded to the type: u of it, and 2^-25 for f16."""
import torch

E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
FLUSH = 2.0 ** -126
TINY = {"bf16": FLUSH, "f16": 2.0 ** -25}
INF = float("inf")


def seen(L, M, causal, window, device="cpu"):
    """[L, M]: which keys a query sees."""
    place = torch.arange(L, device=device)[:, None] + M - L
    j = torch.arange(M, device=device)[None, :]
    ok = torch.ones((L, M), dtype=torch.bool, device=device)
    if causal:
        ok &= j <= place
    if window:
        ok &= j > place - window
    return ok


def _head(q, k, v, ok, scale, lse=None):
    """Scores, lse and probabilities of a head in 64 bits, and their relative bound r."""
    s = torch.where(ok, q @ k.t() * scale, -INF)
    if lse is None:
        lse = torch.logsumexp(s, 1) if k.shape[0] else torch.full((q.shape[0],), -INF, dtype=torch.float64, device=q.device)
    p = torch.where(ok, torch.exp(s - lse[:, None]), 0.0)
    D = q.shape[1]
    near = torch.where(lse == -INF, torch.zeros_like(lse), lse.abs())[:, None]
    mag = torch.where(ok, s.abs(), torch.zeros_like(s))
    r = 2 * (D + 2) * E * (q.abs() @ k.abs().t()) * scale + 4 * E * (mag + near) + 4 * E
    # what one of a row's probabilities may be off by; the sum is off by no more
    return s, lse, p, 2 * r.amax(1, keepdim=True) if k.shape[0] else r.sum(1, keepdim=True)


def forward(q, k, v, spans, spans_k, causal, window, scale, dt, device="cpu"):
    """(out, lse, bound of out, bound of lse) of rows [T, H, D], [Tk, K, D]; rows of no sequence are NaN."""
    q, k, v = (x.double().to(device) for x in (q, k, v))
    T, H, D = q.shape
    group = H // k.shape[1]
    out, bound = torch.full((T, H, D), float("nan"), dtype=torch.float64, device=device), torch.zeros((T, H, D), dtype=torch.float64, device=device)
    lse, lbound = torch.full((H, T), float("nan"), dtype=torch.float64, device=device), torch.zeros((H, T), dtype=torch.float64, device=device)
    for (a, b), (e, f) in zip(spans, spans_k):
        ok = seen(b - a, f - e, causal, window, device)
        for h in range(H):
            kk, vv = k[e:f, h // group], v[e:f, h // group]
            _, z, p, r = _head(q[a:b, h], kk, vv, ok, scale)
            o = p @ vv
            out[a:b, h], lse[h, a:b] = o, z
            weight = p @ vv.abs()
            bound[a:b, h] = ((U[dt] + r + 2 * (f - e + 4) * E) * weight + U[dt] * o.abs() +
                             TINY[dt] * (1 + (ok.double() @ vv.abs())))
            near = torch.where(z == -INF, torch.zeros_like(z), z.abs())
            lbound[h, a:b] = r[:, 0] + (f - e + 8) * E + 4 * E * near
    return out.cpu(), lse.cpu(), bound.cpu(), lbound.cpu()


def backward(q, k, v, out, lse, dout, spans, spans_k, causal, window, scale, dt, device="cpu"):
    """((dq, dk, dv), their bounds) with the given out and lse; rows of no sequence are NaN."""
    q, k, v, out, dout, lse = (x.double().to(device) for x in (q, k, v, out, dout, lse))
    T, H, D = q.shape
    Tk, K = k.shape[:2]
    group, u = H // K, U[dt]
    grads = [torch.full(s, float("nan"), dtype=torch.float64, device=device) for s in ((T, H, D), (Tk, K, D), (Tk, K, D))]
    bounds = [torch.zeros_like(g) for g in grads]
    for (a, b), (e, f) in zip(spans, spans_k):
        ok = seen(b - a, f - e, causal, window, device)
        for x in (1, 2):
            grads[x][e:f] = 0
        for h in range(H):
            g = h // group
            qq, kk, vv, do, oo = q[a:b, h], k[e:f, g], v[e:f, g], dout[a:b, h], out[a:b, h]
            _, _, p, r = _head(qq, kk, vv, ok, scale, lse[h, a:b])
            dp, delta = do @ vv.t(), (do * oo).sum(1, keepdim=True)
            ds = p * (dp - delta)
            off = 2 * (D + 4) * E * (do.abs() @ vv.abs().t() + (do.abs() * oo.abs()).sum(1, keepdim=True))
            eds = (u + r + 4 * E) * ds.abs() + (1 + r) * p * off + (TINY[dt] + FLUSH * (dp.abs() + delta.abs())) * ok
            ep = (u + r) * p + (TINY[dt] + FLUSH) * ok
            n, m = 2 * (f - e + 4) * E, 2 * (group * (b - a) + 4) * E
            grads[0][a:b, h] = scale * (ds @ kk)
            bounds[0][a:b, h] = scale * ((eds + n * ds.abs()) @ kk.abs())
            grads[1][e:f, g] += scale * (ds.t() @ qq)
            bounds[1][e:f, g] += scale * ((eds + m * ds.abs()).t() @ qq.abs())
            grads[2][e:f, g] += p.t() @ do
            bounds[2][e:f, g] += (ep + m * p).t() @ do.abs()
    grads, bounds = [x.cpu() for x in grads], [x.cpu() for x in bounds]
    return grads, [bo + (u + 4 * E) * gr.nan_to_num().abs() + TINY[dt] for gr, bo in zip(grads, bounds)]


def compare(name, got, want, bound, before=None):
    """Within the bound where the definition has a value, and as it was before where it has none."""
    got = got.double().cpu()
    none = torch.isnan(want)
    if before is not None:
        old = before.double().cpu()
        assert torch.equal(got[none].nan_to_num(7.0), old[none].nan_to_num(7.0)), f"{name}: rows of no sequence were written"
    g, w, t = got[~none], want[~none], bound[~none]
    inf = torch.isinf(w)
    assert torch.equal(g[inf], w[inf]), f"{name}: infinities differ"
    g, w, t = g[~inf], w[~inf], t[~inf]
    assert torch.isfinite(g).all(), f"{name}: not finite"
    if g.numel():
        worst = ((g - w).abs() / t).max().item()
        assert worst <= 1, f"{name}: off by {worst:.3g} times the bound"


def lengths(spans, T):
    """Offsets [sequences + 1] of spans one behind the other."""
    return torch.tensor([spans[0][0]] + [b for _, b in spans], dtype=torch.int64)
