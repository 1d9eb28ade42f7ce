"""Timed cases of the layer's microscaled 4-bit operators and of its router's training losses.

Three operators, each in a plain form of elementary torch operations in 32 bits (``own = False``)
and as a caller reaches it through the package (``own = True``):

* ``quantize``: rows of activations to MX4 (OCP MX v1.0 MXFP4: E2M1 codes, one E8M0 scale per 32
  values along the row).  The scale is ``2^e`` with ``e = floor(log2(max|v|)) - 2``, codes round to
  nearest with ties to the even code and saturate at 6.
* ``product``: rows times the MX4 weights of the expert that each row is routed to, with an optional
  activation on the result.  ``x`` is ``mx4`` (the rows are quantised first, the batched form) or
  ``bf16`` / ``f32`` (the rows enter exactly, the form for few tokens).
* ``balance``: the router's load-balancing loss ``E sum_e f_e P_e`` and z loss ``mean(lse^2)`` with
  the per-expert counts; with ``grad`` also the gradient with respect to the logits, of both losses
  and of the renormalised top-k weights.

Sizes are those of the layer shapes in ``moe_inputs`` (d_model 2816 / d_ff 704 / 128 experts top-8;
1024 / 2688 / 512 experts top-22; d_model 6144) and generic ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token entering the experts of a decode step: pure latency
        {"name": "quantize-1x2816-bf16", "op": "quantize", "rows": 1, "d": 2816, "dtype": "bf16"},
        # the hidden activations of a 2048-token prompt, eight experts each
        {"name": "quantize-16384x704-f32", "op": "quantize", "rows": 16384, "d": 704, "dtype": "f32"},
        # gate/up of a 2048-token prompt through 128 experts
        {"name": "product-mx4-gateup-2048", "op": "product", "x": "mx4", "T": 2048, "k": 8, "E": 128, "K": 2816,
         "N": 1408, "act": "swiglu", "out": "bf16", "gather": True, "skew": 0.0},
        # the down projection of the same prompt, its rows already in expert order, some experts hot
        {"name": "product-mx4-down-2048", "op": "product", "x": "mx4", "T": 2048, "k": 8, "E": 128, "K": 704,
         "N": 2816, "act": "none", "out": "f32", "gather": False, "skew": 1.1},
        # a dense projection of a long prompt (a shared expert): compute counts, not bytes
        {"name": "product-mx4-dense-4096", "op": "product", "x": "mx4", "T": 4096, "k": 1, "E": 1, "K": 6144,
         "N": 6144, "act": "none", "out": "bf16", "gather": False, "skew": 0.0},
        # gate/up of one token through its eight experts: the serving step
        {"name": "product-bf16-gateup-1", "op": "product", "x": "bf16", "T": 1, "k": 8, "E": 128, "K": 2816,
         "N": 1408, "act": "swiglu", "out": "bf16", "gather": True, "skew": 0.0},
        # the down projection of eight tokens, hidden activations kept in 32 bits
        {"name": "product-f32-down-8", "op": "product", "x": "f32", "T": 8, "k": 8, "E": 128, "K": 704, "N": 2816,
         "act": "none", "out": "f32", "gather": False, "skew": 0.0},
        # ungated up projection of a small serving batch over many small experts
        {"name": "product-bf16-up-relu2-16", "op": "product", "x": "bf16", "T": 16, "k": 22, "E": 512, "K": 1024,
         "N": 2688, "act": "relu2", "out": "f32", "gather": True, "skew": 0.0},
        # load statistics of a small batch: latency again
        {"name": "balance-8x128", "op": "balance", "T": 8, "E": 128, "k": 8, "dtype": "f32", "pad": 0.0, "grad": False},
        # load statistics of many experts over a prompt
        {"name": "balance-2048x512", "op": "balance", "T": 2048, "E": 512, "k": 22, "dtype": "f32", "pad": 0.0,
         "grad": False},
        # a small training micro-batch, odd sizes, a quarter of it padding
        {"name": "balance-grad-333x40-bf16", "op": "balance", "T": 333, "E": 40, "k": 5, "dtype": "bf16", "pad": 0.25,
         "grad": True},
        # the router of a full training batch
        {"name": "balance-grad-32768x128", "op": "balance", "T": 32768, "E": 128, "k": 8, "dtype": "f32", "pad": 0.1,
         "grad": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "product", "balance", "balance"))
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 16384), "d": 64 * _log(rng, 1, 44), "dtype": rng.choice(("bf16", "f32"))}
    if op == "balance":
        E = _log(rng, 4, 512)
        return {"op": op, "T": _log(rng, 1, 32768 if E <= 128 else 8192), "E": E, "k": min(E, _log(rng, 1, 22)),
                "dtype": rng.choice(("bf16", "f32")), "pad": rng.choice((0.0, 0.2)), "grad": rng.random() < 0.6}
    x = rng.choice(("mx4", "mx4", "bf16", "f32"))
    while True:
        E = _log(rng, 1, 256)
        k = min(E, _log(rng, 1, 16))
        T = _log(rng, 1, 2048 if x == "mx4" else 64)
        act = rng.choice(("swiglu", "relu2", "none"))
        N = _log(rng, 24, 3500)
        K = 64 * _log(rng, 1, 44)
        if E * N * K <= 128 * 1408 * 2816 and T * k * N * K <= 16384 * 1408 * 2816:
            return {"op": op, "x": x, "T": T, "k": k, "E": E, "K": K, "N": N + N % 2 if act == "swiglu" else N,
                    "act": act, "out": rng.choice(("bf16", "f32")), "gather": rng.random() < 0.5,
                    "skew": rng.choice((0.0, 1.1))}


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["d"]
        # v read; 4-bit codes, one scale byte per 32 and the values they stand for written
        return {"bytes": n * (2 * _size(c["dtype"]) + 0.5 + 1 / 32), "flops": 0}
    if c["op"] == "balance":
        n = c["T"] * c["E"]
        grad = n * _size(c["dtype"]) if c["grad"] else 0
        return {"bytes": n * _size(c["dtype"]) + c["T"] * c["k"] * (12 if c["grad"] else 4) + grad, "flops": 0}
    P = c["T"] * c["k"]
    active = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])     # experts that an even routing reaches
    xin = (c["T"] if c["gather"] else P) * c["K"] * (4 if c["x"] == "f32" else 2)
    nout = c["N"] // 2 if c["act"] == "swiglu" else c["N"]
    return {"bytes": xin + active * c["N"] * c["K"] * (0.5 + 1 / 32) + P * nout * _size(c["out"]),
            "flops": 2.0 * P * c["N"] * c["K"]}


def _size(dtype):
    return 2 if dtype == "bf16" else 4


# ---------------------------------------------------------------------------------------------
# inputs

def _gen(seed, stream):
    return torch.Generator(device="cuda").manual_seed(seed * 16 + stream)


def _routing(seed, T, E, k, skew):
    """Top-k ids of random logits (ties to the lower index) and the logits."""
    logits = torch.randn((T, E), generator=_gen(seed, 1), device="cuda") * 2.0
    logits -= skew * torch.log(torch.arange(1, E + 1, device="cuda"))
    idx = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    return idx.to(torch.int32).contiguous(), logits


def prepare(case, seed):
    c = case
    if c["op"] == "quantize":
        v = torch.randn((c["rows"], c["d"]), generator=_gen(seed, 0), device="cuda")
        # activations with a few large channels, as a model's are
        v *= torch.exp(torch.randn((1, c["d"]), generator=_gen(seed, 2), device="cuda"))
        return {"case": c, "v": v.to(DTYPES[c["dtype"]])}
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "balance":
        idx, logits = _routing(seed, T, E, k, 0.5)
        w = torch.softmax(torch.gather(logits, 1, idx.long()), 1)
        mask = None
        if c["pad"]:
            mask = torch.rand(T, generator=_gen(seed, 3), device="cuda") >= c["pad"]
            logits[~mask] = float("nan")            # padding holds whatever was there
        return {"case": c, "logits": logits.to(DTYPES[c["dtype"]]), "idx": idx, "w": w, "mask": mask,
                "dw": torch.randn((T, k), generator=_gen(seed, 4), device="cuda") * 1e-3,
                "dloss": torch.tensor([1e-2, 1e-3], device="cuda")}
    P = T * k
    idx, _ = _routing(seed, T, E, k, c["skew"])
    flat = idx.reshape(-1).long()
    perm = torch.sort(flat, stable=True).indices                      # pairs in (expert, pair) order
    counts = torch.zeros(E, dtype=torch.long, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    x = torch.randn((T if c["gather"] else P, c["K"]), generator=_gen(seed, 0), device="cuda")
    x *= torch.exp(0.5 * torch.randn((1, c["K"]), generator=_gen(seed, 2), device="cuda"))
    w, ws = _weights(seed, E, c["N"], c["K"])
    # the plan of the plain form: each group that holds rows padded to the largest
    active = torch.nonzero(counts).reshape(-1)
    cap = int(counts.max())
    start = offsets[:-1].long()[active]
    at = torch.arange(cap, device="cuda")
    live = at[None, :] < counts[active][:, None]
    pad_rows = torch.where(live, start[:, None] + at[None, :], 0).reshape(-1)
    row_slot = torch.nonzero(live.reshape(-1)).reshape(-1)            # ascending: row r's place
    return {"case": c, "x": x.to(torch.float32 if c["x"] == "f32" else torch.bfloat16), "w": w, "ws": ws,
            "offsets": offsets, "perm": perm.to(torch.int32), "active": active, "cap": cap, "pad_rows": pad_rows,
            "row_slot": row_slot}


def _weights(seed, E, N, K):
    """Gaussian weights of deviation 0.02 in MX4: codes [E, N, K/2], scales [E, N, K/32]."""
    w = torch.randn((E, N, K // 32, 32), generator=_gen(seed, 5), device="cuda") * 0.02
    e = _block_exponent(w)
    codes = _nearest_code(w, e).to(torch.uint8).reshape(E, N, K // 2, 2)
    return codes[..., 0] | (codes[..., 1] << 4), (e + 127).to(torch.uint8).reshape(E, N, K // 32)


def _block_exponent(v):
    amax = v.abs().amax(-1, keepdim=True)
    return torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)


def _nearest_code(v, e):
    a = torch.ldexp(v.abs(), -e)
    m = torch.where(a < 2, torch.round(2 * a), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    return m.clamp(max=7) + 8 * torch.signbit(v)


# ---------------------------------------------------------------------------------------------
# one pass

def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    if c["op"] == "quantize":
        return _mx4_values(state["v"].float()).to(state["v"].dtype)
    return _plain_balance(c, state) if c["op"] == "balance" else _plain_product(c, state)


def _own(c, s):
    import sparse_moe_expert_router_amd as moe
    if c["op"] == "quantize":
        return moe.quantize_rows_mx4(s["v"], want_values=True)[2]
    if c["op"] == "balance":
        loss, counts, mean_prob = moe.balance_loss(s["logits"], s["idx"], mask=s["mask"])
        if not c["grad"]:
            return loss, counts, mean_prob
        d = moe.balance_loss_backward(s["logits"], s["idx"], counts, s["dloss"], topk_w=s["w"], d_topk_w=s["dw"],
                                      mask=s["mask"])
        return loss, counts, mean_prob, d
    x, xs = s["x"], None
    if c["x"] == "mx4":
        x, xs = moe.quantize_rows_mx4(x)
    act = {"swiglu": moe.ACT_SWIGLU, "relu2": moe.ACT_RELU2, "none": moe.ACT_NONE}[c["act"]]
    return moe.matmul_mx4(x, s["w"], s["ws"], x_scales=xs, offsets=s["offsets"],
                          perm=s["perm"] if c["gather"] else None, k=c["k"] if c["gather"] else 1, act=act,
                          out_dtype=DTYPES[c["out"]])


def _mx4_values(v):
    """fp32 rows rounded to MX4, as the values the codes and scales stand for; a block that holds a
    NaN or an infinity stands for NaN."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = _block_exponent(b)
    a = torch.ldexp(b.abs(), -e)
    m = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2)))
    q = torch.copysign(m.clamp(max=6.0), b)
    q = torch.where(torch.isfinite(amax), torch.ldexp(q, e), float("nan"))
    return q.reshape(v.shape)


def _plain_product(c, s):
    x = s["x"].float()
    if c["x"] == "mx4":
        x = _mx4_values(x)
    if c["gather"]:
        x = x[s["perm"].long() // c["k"]]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    table = torch.stack((table.repeat(16), table.repeat_interleave(16)), 1)      # byte -> its two values
    codes, scales = s["w"], s["ws"]
    if s["active"].numel() < c["E"]:
        codes, scales = codes[s["active"]], scales[s["active"]]
    A = codes.shape[0]
    w = table[codes.int()].reshape(A, c["N"], c["K"] // 32, 32)
    w = (w * torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)[..., None])
    xt = x[s["pad_rows"]].reshape(A, s["cap"], c["K"]).transpose(1, 2).contiguous()
    y = torch.bmm(w.reshape(A, c["N"], c["K"]), xt)                              # [A, N, cap]
    if c["act"] == "swiglu":
        F = c["N"] // 2
        y = y[:, :F] * torch.sigmoid(y[:, :F]) * y[:, F:]
    elif c["act"] == "relu2":
        y = y.clamp(min=0).square()
    y = y.transpose(1, 2).reshape(A * s["cap"], -1)[s["row_slot"]]
    return y.to(DTYPES[c["out"]])


def _plain_balance(c, s):
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].float()
    top = l.amax(1, keepdim=True)
    valid = top != float("-inf")                       # a row without any expert is as padding
    if s["mask"] is not None:
        valid = valid & s["mask"][:, None]
    l, top = torch.where(valid, l, 0.0), torch.where(valid, top, 0.0)
    ex = torch.exp(l - top)
    total = ex.sum(1, keepdim=True)
    p = torch.where(valid, ex / total, 0.0)
    lse = torch.where(valid, top + torch.log(total), 0.0)
    n = valid.sum().clamp(min=1).float()
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, s["idx"].reshape(-1).long(), valid.expand(T, k).reshape(-1).int())
    f = counts.float() / (n * k)
    mean_prob = p.sum(0) / n
    loss = torch.stack((E * (f * mean_prob).sum(), lse.square().sum() / n))
    if not c["grad"]:
        return loss, counts, mean_prob
    gb, gz = s["dloss"][0], s["dloss"][1]
    d = p * (gb * E / n * (f - (p * f).sum(1, keepdim=True)) + gz * 2 / n * lse)
    w, dw = s["w"], s["dw"]
    dsel = torch.where(valid, w * (dw - (w * dw).sum(1, keepdim=True)), 0.0)
    d = d.scatter_add(1, s["idx"].long(), dsel)
    return loss, counts, mean_prob, d.to(s["logits"].dtype)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        return _mx4_values64(s["v"])
    return _balance64(c, s) if c["op"] == "balance" else _product64(c, s)


def _mx4_values64(v):
    b = v.double().reshape(-1, 32)
    big = b.abs().max(1, keepdim=True).values
    scale = torch.pow(2.0, torch.floor(torch.log2(big.clamp(min=2.0 ** -125))) - 2)
    a = (b / scale).abs()
    code = torch.zeros_like(a)
    for i in range(7):                                 # the midpoint between code i and i + 1
        mid = (E2M1[i] + E2M1[i + 1]) / 2
        code += (a > mid) if i % 2 == 0 else (a >= mid)   # a tie goes to the even code
    q = torch.tensor(E2M1, dtype=torch.float64, device=v.device)[code.long()] * torch.sign(b) * scale
    q[~torch.isfinite(big).expand_as(q)] = float("nan")
    return q.reshape(v.shape)


def _product64(c, s):
    x = s["x"].double()
    if c["x"] == "mx4":
        x = _mx4_values64(s["x"])
    rows = torch.arange(c["T"] * c["k"], device="cuda")
    if c["gather"]:
        rows = torch.div(s["perm"].long(), c["k"], rounding_mode="floor")
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    out = []
    bounds = s["offsets"].tolist()
    for g in range(c["E"]):
        lo, hi = bounds[g], bounds[g + 1]
        if hi == lo:
            continue
        codes = s["w"][g].long()
        w = torch.empty((c["N"], c["K"]), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = values[codes % 16], values[codes // 16]
        w *= torch.pow(2.0, s["ws"][g].double() - 127).repeat_interleave(32, 1)
        y = x[rows[lo:hi]] @ w.T
        if c["act"] == "swiglu":
            gate, up = y.chunk(2, 1)
            y = gate / (1 + torch.exp(-gate)) * up
        elif c["act"] == "relu2":
            y = torch.relu(y) ** 2
        out.append(y)
    return torch.cat(out)


def _balance64(c, s):
    T, E, k = c["T"], c["E"], c["k"]
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"].clone()
    l = s["logits"].double()
    keep &= ~(l == float("-inf")).all(1)
    rows = torch.nonzero(keep).reshape(-1)
    n = rows.numel()
    d = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    if n == 0:
        zero = torch.zeros(E, dtype=torch.float64, device="cuda")
        got = (torch.zeros(2, dtype=torch.float64, device="cuda"), zero.to(torch.int32), zero)
        return got + (d,) if c["grad"] else got
    idx = s["idx"][rows].long()
    counts = (idx.reshape(-1, 1) == torch.arange(E, device="cuda")).sum(0)
    f = counts.double() / (n * k)
    lse = torch.logsumexp(l[rows], 1)
    p = torch.exp(l[rows] - lse[:, None])
    mean_prob = p.mean(0)
    loss = torch.stack((E * torch.dot(f, mean_prob), torch.mean(lse ** 2)))
    got = (loss, counts.to(torch.int32), mean_prob)
    if not c["grad"]:
        return got
    gb, gz = s["dloss"].double()
    g = gb * E / n * p * (f - (p @ f)[:, None]) + gz * 2 / n * lse[:, None] * p
    w, dw = s["w"][rows].double(), s["dw"][rows].double()
    one = torch.nn.functional.one_hot(idx, E).double()                # [n, k, E]
    g += torch.bmm((w * (dw - (w * dw).sum(1, keepdim=True)))[:, None], one)[:, 0]
    d[rows] = g
    return got + (d,)
