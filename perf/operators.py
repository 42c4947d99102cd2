"""Cases of the training operators around the MoE layer, in plain torch and through the library.

Operators (formulas; t a token, j its rank, e an expert, s a slot):

- token sort: the T*k routed entries (t, j) ordered by expert, then by entry number t*k + j; the
  entry's place is slot_of[t, j], expert e's slots are [offsets[e], offsets[e+1]), and
  x_sorted[slot_of[t, j]] = x[t]. An entry whose expert id lies outside [0, E) is dropped:
  slot_of = -1 and no row; rows from offsets[E] on stay as they were.
- its gradient: dx[t] = sum_j dx_sorted[slot_of[t, j]].
- token unsort: y[t] = add[t] + sum_j w[t, j] * y_sorted[slot_of[t, j]] over the entries kept.
- its gradient: dy_sorted[slot_of[t, j]] = w[t, j] * dy[t] and
  dw[t, j] = <dy[t], y_sorted[slot_of[t, j]]> (0 for a dropped entry).
- orthogonalised update of a stack of weight matrices: the momentum m <- beta m + g, the update
  u = g + beta m (Nesterov) or m (or g alone), X_0 = u / (|u|_F + eps), then five times
  X <- a X + (b A + c A A) X with A = X X^T (of the shorter side), out = scale * X in bf16.

`own` false: elementary torch operations in 32 bits. `own` true: the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
STEPS, COEFFS, EPS, BETA = 5, (3.4445, -4.7750, 2.0315), 1e-7, 0.95
FILL = 0.75  # what the rows that no entry owns hold before the call


def _rows(name, op, T, H, E, k, dtype, drop=0.0, zipf=0.1, add=False):
    return {"name": name, "op": op, "T": T, "H": H, "E": E, "k": k, "dtype": dtype, "drop": drop, "zipf": zipf,
            "add": add}


def _orth(name, n, rows, cols, dtype, momentum, nesterov, tokens):
    return {"name": name, "op": "orthogonalize", "n": n, "rows": rows, "cols": cols, "dtype": dtype,
            "momentum": momentum, "nesterov": nesterov, "tokens": tokens}


def listed():
    return [
        # one decode step of the Step-3.5 shape: 64 tokens to 288 experts, latency counts
        _rows("sort_decode", "sort", 64, 4096, 288, 8, "bf16"),
        # a prefill batch of the Step-3.5 shape
        _rows("sort_prefill", "sort", 4096, 4096, 288, 8, "bf16"),
        # a padded batch on an odd width: a fifth of the entries belong to padding or other ranks
        _rows("sort_ragged", "sort", 1021, 1290, 60, 6, "fp16", drop=0.2),
        # gradient of the sort at the Step-5 skewed shape, the largest batch
        _rows("sort_backward_skewed", "sort_backward", 16384, 4096, 352, 8, "bf16", zipf=0.5),
        # the same in fp32 on a small model
        _rows("sort_backward_fp32", "sort_backward", 777, 514, 16, 4, "fp32", drop=0.1),
        # one decode step: expert outputs weighted and added to the shared expert's
        _rows("unsort_decode", "unsort", 64, 4096, 288, 8, "bf16", add=True),
        # a prefill batch of the Step-5 shape
        _rows("unsort_prefill", "unsort", 8192, 4096, 352, 8, "bf16", add=True),
        # gradient of the weighted unsort at the Step-3.5 prefill shape
        _rows("unsort_backward", "unsort_backward", 4096, 4096, 288, 8, "bf16"),
        # and on an odd width with dropped entries, fp32
        _rows("unsort_backward_ragged", "unsort_backward", 1500, 1023, 40, 3, "fp32", drop=0.2),
        # every gate and up matrix of the tiny layer, updated together: latency counts
        _orth("orthogonalize_tiny", 32, 128, 256, "fp32", True, True, 64),
        # gate and up matrices of the 11 experts that one of 32 ranks holds of the Step-5 shape
        _orth("orthogonalize_gate_up", 22, 1536, 4096, "bf16", False, False, 700),
        # down matrices of the 36 experts that one of 8 ranks holds of the Step-3.5 shape
        _orth("orthogonalize_down", 36, 4096, 1280, "fp32", True, True, 400),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.3:
        most = work(listed()[-1])["flops"]
        while True:
            n, rows, cols = _log(rng, 1, 48), _log(rng, 24, 4200), _log(rng, 24, 4200)
            momentum = rng.random() < 0.6
            c = _orth("", n, rows, cols, rng.choice(("bf16", "fp32")), momentum, momentum and rng.random() < 0.7,
                      _log(rng, 4, 2000))
            if work(c)["flops"] <= most:
                del c["name"]
                return c
    while True:
        E = _log(rng, 4, 512)
        k = rng.randint(1, min(E, 12))
        T, H = _log(rng, 1, 16384), _log(rng, 48, 8192)
        if rng.random() < 0.7:
            H = (H + 7) // 8 * 8
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        if T * k * H * SIZE[dtype] <= 16384 * 8 * 4096 * 2:
            break
    op = rng.choice(("sort", "sort_backward", "unsort", "unsort_backward"))
    c = _rows("", op, T, H, E, k, dtype, rng.choice((0.0, 0.0, round(rng.uniform(0.02, 0.6), 2))),
              round(rng.uniform(0.0, 0.6), 2), op == "unsort" and rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------- inputs
def _routing(c, gen):
    """topk_idx [T, k] int32 (distinct experts of a log-rank popularity) and its sorted places."""
    T, E, k = c["T"], c["E"], c["k"]
    pop = -c["zipf"] * torch.log1p(torch.randperm(E, generator=gen, device="cuda").float())
    u = torch.rand((T, E), generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)
    idx = torch.topk(pop - torch.log(-torch.log(u)), k, dim=1).indices.to(torch.int32)
    if c["drop"] > 0:  # whole tokens of padding, and single entries that other ranks own
        gone = torch.rand((T, k), generator=gen, device="cuda") < c["drop"] / 2
        gone |= torch.rand((T, 1), generator=gen, device="cuda") < c["drop"] / 2
        idx = torch.where(gone, torch.where(torch.rand((T, k), generator=gen, device="cuda") < 0.5, -1, E), idx)
    return idx.to(torch.int32)


def _places(idx, E):
    """The plain sort: order (entry of each slot), slot_of (int32, -1 for dropped) and offsets."""
    key = torch.where((idx >= 0) & (idx < E), idx, E).flatten()
    order = torch.argsort(key, stable=True)
    slot = torch.empty_like(order).scatter_(0, order, torch.arange(key.numel(), device=key.device))
    slot = torch.where(key < E, slot, -1).to(torch.int32).view(idx.shape)
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=key.device, dtype=key.dtype)).to(torch.int32)
    return order, slot, offsets


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    s = {"case": c}
    if c["op"] == "orthogonalize":
        # a gradient is a sum over an expert's tokens of outer products of very different sizes,
        # a momentum the decaying sum over many batches
        n, rows, cols = c["n"], c["rows"], c["cols"]

        def tokens(count):
            size = torch.exp(torch.randn((n, 1, count), generator=gen, device="cuda"))
            left = torch.randn((n, rows, count), generator=gen, device="cuda").mul_(size)
            return torch.bmm(left, torch.randn((n, count, cols), generator=gen, device="cuda")).mul_(1e-4)

        s["grad"] = tokens(c["tokens"]).to(dt)
        s["momentum"] = tokens(min(4 * c["tokens"], 2048)).mul_(3.0) if c["momentum"] else None
        s["out"] = torch.empty((n, rows, cols), dtype=torch.bfloat16, device="cuda")
        if own:
            from sparse_moe_layer_biased_b200.muon import Orthogonalizer

            s["plan"] = Orthogonalizer(n, rows, cols, grad_dtype=dt, steps=STEPS, coeffs=COEFFS, eps=EPS,
                                       scale=_scale(c), beta=BETA, nesterov=c["nesterov"])
        return s
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    s["idx"] = _routing(c, gen)
    if c["op"] == "sort":
        s["x"] = normal(T, H)
        s["x_sorted"] = torch.full((T * k, H), FILL, dtype=dt, device="cuda")
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["slot_of"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
    else:
        s["slot_of"] = _places(s["idx"], E)[1]
        s["rows"] = normal(T * k, H)
        s["w"] = torch.rand((T, k), generator=gen, device="cuda").mul_(3.0 / k)
    if c["op"] == "sort_backward":
        s["dx"] = torch.empty((T, H), dtype=dt, device="cuda")
    elif c["op"] == "unsort":
        s["add"] = normal(T, H) if c["add"] else None
        s["y"] = torch.empty((T, H), dtype=dt, device="cuda")
    elif c["op"] == "unsort_backward":
        s["dy"] = normal(T, H)
        s["drows"] = torch.full((T * k, H), FILL, dtype=dt, device="cuda")
        s["dw"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    if own:
        from sparse_moe_layer_biased_b200.tokens import TokenSorter

        s["plan"] = TokenSorter(T, H, E, k, dtype=dt)
    return s


def _scale(c):
    """The customary size of an update: as large as the matrix is tall against its width."""
    return math.sqrt(max(1.0, c["rows"] / c["cols"]))


# ------------------------------------------------------------------------- the plain forms
def _sort(s):
    c = s["case"]
    order, slot, offsets = _places(s["idx"], c["E"])
    rows = s["x"][order // c["k"]]
    if c["drop"] > 0:
        kept = torch.arange(order.numel(), device=order.device) < offsets[-1]
        rows = torch.where(kept[:, None], rows, s["x_sorted"])
    return rows, offsets, slot


def _gathered(s):
    """The row of every entry in fp32 [T, k, H], zero where the entry was dropped."""
    c, slot = s["case"], s["slot_of"]
    if c["drop"] > 0:
        return torch.where((slot >= 0)[..., None], s["rows"][slot.clamp(min=0).long()].float(), 0.0)
    return s["rows"][slot.long()].float()


def _unsort(s, w, add):
    g = _gathered(s)
    if w is not None:
        g = g * w[..., None]
    y = g.sum(1)
    if add is not None:
        y = y + add.float()
    return y.to(s["rows"].dtype)


def _unsort_backward(s):
    c, slot, dy = s["case"], s["slot_of"], s["dy"].float()
    dw = (_gathered(s) * dy[:, None, :]).sum(-1)
    d = (s["w"][..., None] * dy[:, None, :]).to(s["rows"].dtype).view(-1, c["H"])
    at = slot.flatten().long()
    if c["drop"] > 0:  # the dropped entries go to a row behind the last
        at = torch.where(at < 0, at.numel(), at)
        rows = torch.cat([s["drows"], s["drows"][:1]])
        return rows.index_copy_(0, at, d)[:-1], dw
    return torch.empty_like(d).index_copy_(0, at, d), dw


def _orthogonalize(s):
    c, g, m = s["case"], s["grad"].float(), s["momentum"]
    if m is not None:
        m.mul_(BETA).add_(g)
        g = g + BETA * m if c["nesterov"] else m
    X = g / (g.square().sum((1, 2), keepdim=True, dtype=torch.float64).sqrt() + EPS).float()
    tall = c["rows"] > c["cols"]
    a, b, k = COEFFS
    for _ in range(STEPS):
        A = torch.bmm(X.mT, X) if tall else torch.bmm(X, X.mT)
        B = b * A + k * torch.bmm(A, A)
        X = a * X + (torch.bmm(X, B) if tall else torch.bmm(B, X))
    out = (X * _scale(c)).to(torch.bfloat16)
    return out if m is None else (out, m)


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "sort":
            return _sort(s)
        if op == "sort_backward":
            return _unsort(s, None, None)
        if op == "unsort":
            return _unsort(s, s["w"], s["add"])
        if op == "unsort_backward":
            return _unsort_backward(s)
        return _orthogonalize(s)
    p = s["plan"]
    if op == "sort":
        return p.sort(s["x"], s["idx"], out=(s["x_sorted"], s["offsets"], s["slot_of"]))
    if op == "sort_backward":
        return p.sort_backward(s["rows"], s["slot_of"], out=s["dx"])
    if op == "unsort":
        return p.unsort(s["rows"], s["slot_of"], s["w"], add=s["add"], out=s["y"])
    if op == "unsort_backward":
        return p.unsort_backward(s["dy"], s["rows"], s["slot_of"], s["w"], out=(s["drows"], s["dw"]))
    out = p.orthogonalize(s["grad"], momentum=s["momentum"], out=s["out"])
    return out if s["momentum"] is None else (out, s["momentum"])


# ------------------------------------------------------------------------------- the work
def work(case):
    c = case
    if c["op"] == "orthogonalize":
        n, p, q = c["n"], min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
        # the two symmetric products need one triangle each
        step = p * (p + 1) * q + p * (p + 1) * p + 2 * p * p * q
        each = n * p * q
        return {"bytes": each * (SIZE[c["dtype"]] + 2 + (8 if c["momentum"] else 0)), "flops": n * STEPS * step}
    T, H, E, k, sz = c["T"], c["H"], c["E"], c["k"], SIZE[c["dtype"]]
    kept = round(T * k * (1 - c["drop"] / 2) ** 2)  # entries that the two drops leave
    row, tab = H * sz, T * k * 4
    if c["op"] == "sort":
        return {"bytes": T * row + kept * row + 2 * tab + (E + 1) * 4, "flops": 0}
    if c["op"] == "sort_backward":
        return {"bytes": kept * row + T * row + tab, "flops": kept * H}
    if c["op"] == "unsort":
        return {"bytes": kept * row + T * row * (2 if c["add"] else 1) + 2 * tab, "flops": 2 * kept * H}
    return {"bytes": 2 * kept * row + T * row + 3 * tab, "flops": 3 * kept * H}


# ---------------------------------------------------------------------- in 64 bits, apart
def _exact_orthogonalize(s):
    """Every X of the iteration is Q X_0 (or X_0 Q) with Q a polynomial of the first Gram matrix:
    the recurrence of Q and the Gram matrices alone, one matrix at a time."""
    c, a, b, k = s["case"], *COEFFS
    outs = []
    for i in range(c["n"]):
        u = s["grad"][i].double()
        if s["momentum"] is not None:
            m = BETA * s["momentum"][i].double() + u
            s["momentum64"][i] = m
            u = u + BETA * m if c["nesterov"] else m
        u = u / (torch.linalg.vector_norm(u) + EPS)
        tall = c["rows"] > c["cols"]
        gram = u.T @ u if tall else u @ u.T
        eye = torch.eye(gram.shape[0], dtype=torch.float64, device=u.device)
        Q = eye
        for _ in range(STEPS):
            P = a * eye + gram @ (b * eye + k * gram)
            Q = P @ Q
            gram = P @ gram @ P
            gram = (gram + gram.T) / 2
        outs.append(_scale(c) * (u @ Q if tall else Q @ u))
    return torch.stack(outs)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "orthogonalize":
        if s["momentum"] is None:
            return _exact_orthogonalize(s)
        s["momentum64"] = torch.empty_like(s["momentum"], dtype=torch.float64)
        return _exact_orthogonalize(s), s["momentum64"]
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    entry = torch.arange(T * k, device="cuda")
    if c["op"] == "sort":
        e = s["idx"].flatten().long()
        kept = (e >= 0) & (e < E)
        ranked = torch.sort(e[kept] * (T * k) + entry[kept]).values  # unique keys, so any sort will do
        owner = ranked % (T * k)
        slot = torch.full((T * k,), -1, device="cuda")
        slot[owner] = entry[:owner.numel()]
        count = torch.stack([(e[kept] < x).sum() for x in range(E + 1)])
        rows = s["x_sorted"].double()
        rows[:owner.numel()] = s["x"][torch.div(owner, k, rounding_mode="floor")].double()
        return rows, count.to(torch.int32), slot.to(torch.int32).view(T, k)
    slot, rows = s["slot_of"].long(), s["rows"]
    if c["op"] == "unsort_backward":
        drows, dw = s["drows"].double(), torch.zeros((T, k), dtype=torch.float64, device="cuda")
        dy = s["dy"].double()
        for j in range(k):
            t = torch.nonzero(slot[:, j] >= 0).flatten()
            drows[slot[t, j]] = s["w"][t, j].double()[:, None] * dy[t]
            dw[t, j] = torch.einsum("th,th->t", dy[t], rows[slot[t, j]].double())
        return drows, dw
    weighted = c["op"] == "unsort"
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    if weighted and s["add"] is not None:
        y += s["add"].double()
    for j in range(k):
        t = torch.nonzero(slot[:, j] >= 0).flatten()
        r = rows[slot[t, j]].double()
        y[t] += s["w"][t, j].double()[:, None] * r if weighted else r
    return y
