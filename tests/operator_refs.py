"""64-bit forms of the row, router-gradient and 8-bit operators, and the error
bounds of their kernels, for the tests.

Rounding counts: HALF[t] is half a step of the type relative to the value
(torch.finfo(t).eps / 2)."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F32 = 2.0 ** -24


def routing(T, E, k, seed, drop=0.0, one_expert=None):
    """expert_indices [T, k] (distinct per token; -1 where dropped), expert_offsets and inverse on the CPU."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k].to(torch.int32)
    if one_expert is not None:
        idx[:, 0] = one_expert
    if drop:
        idx[torch.rand(T, k, generator=g) < drop] = -1
    return idx, *csr(idx, E)


def csr(idx, E):
    flat = idx.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(flat, stable=True)
    inverse = torch.empty_like(order)
    inverse[order] = torch.arange(flat.numel())
    inverse = torch.where(flat < E, inverse, -1).to(torch.int32)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    return offsets, inverse


def spread(tok, inverse, w, rows_before):
    """rows[p] = w * tok[t]; rows of no slot as they were."""
    T, k = inverse.shape
    out = rows_before.double().clone()
    for j in range(k):
        t = torch.nonzero(inverse[:, j] >= 0).view(-1)
        out[inverse[t, j].long()] = tok[t].double() * (1.0 if w is None else w[t, j].double()[:, None])
    return out


def gather(rows, inverse, w):
    """out[t] = sum_j w * rows[p], and the sum of its terms' magnitudes."""
    T, k = inverse.shape
    out = torch.zeros(T, rows.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for j in range(k):
        t = torch.nonzero(inverse[:, j] >= 0).view(-1)
        term = rows[inverse[t, j].long()].double() * (1.0 if w is None else w[t, j].double()[:, None])
        out[t] += term
        mag[t] += term.abs()
    return out, mag


def dots(tok, rows, inverse):
    """<tok[t], rows[p]> (0 for a slot of no expert) and the sum of the products' magnitudes."""
    T, k = inverse.shape
    out, mag = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for j in range(k):
        t = torch.nonzero(inverse[:, j] >= 0).view(-1)
        prod = tok[t].double() * rows[inverse[t, j].long()].double()
        out[t, j], mag[t, j] = prod.sum(1), prod.abs().sum(1)
    return out, mag


def tol_spread(ref, dtype):
    # one product in fp32 and one rounding to the row type
    return ref.abs() * (HALF[dtype] + 2 * F32)


def tol_gather(ref, mag, k, dtype):
    # k products and k additions in fp32, one rounding to the row type
    return ref.abs() * (HALF[dtype] + F32) + mag * (k + 1) * F32


def tol_dots(mag, H):
    # a thread adds at most H/32 + 8 products, then 5 + 8 levels join the threads
    return mag * (H / 32 + 24) * F32


def route_grad(logits, idx, d_w, d_sink, E, S, sink, route_scale=1.0, global_scale=1.0):
    """d_logits and d_global_scale in 64 bits, and the bound of the kernel's fp32 error before it is rounded."""
    z_all = logits.double()
    T, k = idx.shape
    d_z = torch.zeros(T, E + S, dtype=torch.float64)
    tol = torch.zeros(T, E + S, dtype=torch.float64)
    d_scale, d_scale_mag = 0.0, 0.0
    for t in range(T):
        cols = [int(c) if 0 <= int(c) < E else None for c in idx[t]] + [E + i for i in range(S)]
        dw = [float(v) for v in d_w[t]] + ([float(v) for v in d_sink[t]] if d_sink is not None else [0.0] * S)
        keep = [(c, v) for c, v in zip(cols, dw) if c is not None]
        if not keep:
            continue
        c_, v_ = torch.tensor([c for c, _ in keep]), torch.tensor([v for _, v in keep], dtype=torch.float64)
        z = z_all[t, c_]
        l = torch.nn.functional.logsigmoid(z) if sink else z
        p = torch.softmax(l, 0)
        scale = route_scale * global_scale if sink else 1.0
        d = v_[:, None] - v_[None, :]
        f = scale * p * (torch.sigmoid(-z) if sink else 1.0)
        # l to half a step of its size and the exponentials to 2 steps, in p_i and p_j
        # both; a sum of n terms; ten more roundings
        steps = 4 * float(l.abs().max()) + len(keep) + 40
        d_z[t].index_add_(0, c_, f * (p[None, :] * d).sum(1))
        tol[t].index_add_(0, c_, f.abs() * (p[None, :] * d.abs()).sum(1) * steps * F32)
        d_scale += route_scale * float((p * v_).sum())
        d_scale_mag += abs(route_scale) * float((p * v_.abs()).sum()) * steps * F32
    return d_z, tol, d_scale, d_scale_mag


def quantize(a):
    """q (as integers) and the fp32 scales of rows a (bf16, finite), in 64 bits."""
    m = a.double().abs().amax(-1, keepdim=True)
    q = torch.where(m > 0, torch.round(a.double() * 127 / torch.where(m > 0, m, 1.0)), 0.0)
    return q, (m.float() / torch.tensor(127.0)).squeeze(-1)


ALPHA, LIMIT = 1.702, 7.0


def linear_int8(q, scales, w_q, w_scales, bias, offsets, part, fmt, act, alpha, limit, before):
    """The product in 64 bits ([R, D] or [R, H]), rows of no expert as before, and the kernel's error bound."""
    out, tol = before.double().clone(), torch.zeros(before.shape, dtype=torch.float64)
    E = w_q.shape[0]
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        prod = (q[lo:hi].double() @ w_q[e].double().T) * scales[lo:hi].double()[:, None] * w_scales[e].double()
        b = torch.zeros(w_q.shape[1], dtype=torch.float64) if bias is None else bias[e].double()
        y, dy = prod + b, (prod.abs() + b.abs()) * 4 * F32   # conversion, two products, one sum
        if part == "gate_up":
            n = y.shape[1] // 2
            cut = (lambda v: (v[:, :n], v[:, n:])) if fmt == "concatenated" else (lambda v: (v[:, 0::2], v[:, 1::2]))
            (g, u), (dg, du) = cut(y), cut(dy)
            if act != "gelu_tanh" and limit > 0:
                g, u = g.clamp(max=limit), u.clamp(-limit, limit)
            if act == "silu":
                arg, up = g, u
            elif act == "swigluoai":
                arg, up = alpha * g, u + 1
            else:
                arg, up = 2 * 0.7978845608028654 * (g + 0.044715 * g ** 3), u
            s = g * torch.sigmoid(arg)
            y = s * up
            # |d(g sigmoid)/dg| <= 1.2, |.| <= |g|; the sigmoid's exponential errs by
            # its argument's rounding (four steps of it) and ten steps more
            dy = 1.2 * up.abs() * dg + g.abs() * du + y.abs() * (4 * arg.abs().clamp(max=100) + 10) * 2 * F32 + 1e-30
        out[lo:hi] = y
        tol[lo:hi] = dy + y.abs() * (HALF[torch.bfloat16] + F32)
    return out, tol


def assert_within(got, ref, tol, what=""):
    got = got.detach().cpu().double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside their bound, worst "
                           f"{float(((got - ref).abs() - tol)[bad].max() if not torch.isnan((got - ref)[bad]).any() else float('nan')):.3e}")
