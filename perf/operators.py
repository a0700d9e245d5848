"""Cases and plain forms of the serving and adapter operators beside the MoE layer.

  decode            the whole layer for a few tokens (router, top-K, SwiGLU experts, combine)
  adapter_forward   x W + scale_l (x A_l) B_l, every row with the adapter l of its request
  adapter_backward  the gradients of x, A and B of that product (W is frozen)

`run` computes them in elementary torch operations in 32 bits, or, where `own` is true, by
the package's own calls.
"""
import math

import torch

own = False

# Layers: the package's own workloads (a small one, 8 wide experts of which 2 are taken, 128
# narrow ones of which 8, 32 square ones of which 4 with a skewed router and a capacity).
_TINY = dict(d=256, E=8, K=2, n=512)
_WIDE = dict(d=4096, E=8, K=2, n=14336)
_FINE = dict(d=2048, E=128, K=8, n=768)
_SQUARE = dict(d=2880, E=32, K=4, n=2880)


def _decode(name, T, capacity=0.0, bias=False, renormalize=True, **layer):
    return dict(name=name, op="decode", T=T, capacity=capacity, bias=bias,
                renormalize=renormalize, **layer)


def _adapter(name, op, T, d_in, d_out, adapters, rank, requests):
    return dict(name=name, op=op, T=T, d_in=d_in, d_out=d_out, adapters=adapters, rank=rank,
                requests=requests)


def listed():
    return [
        # one token through a small layer: nothing but latency
        _decode("decode_tiny", 1, **_TINY),
        # one request of a chat: a new token, 8 of 128 narrow experts, 2 of 8 wide ones
        _decode("decode_one_fine", 1, **_FINE),
        _decode("decode_one_wide", 1, **_WIDE),
        # an odd number of requests, a skewed router, tokens over the capacity dropped
        _decode("decode_skewed", 37, capacity=1.25, bias=True, **_SQUARE),
        # a server's ordinary batch of requests, one new token each
        _decode("decode_batch_fine", 64, **_FINE),
        # the largest batch: every expert is read
        _decode("decode_batch_wide", 128, renormalize=False, **_WIDE),
        # one request with its adapter, one new token
        _adapter("adapter_one", "adapter_forward", 1, 4096, 4096, 8, 16, 1),
        # a decode batch of requests with an adapter each, some with none
        _adapter("adapter_batch", "adapter_forward", 57, 2048, 2880, 32, 16, 57),
        # the prompts of a dozen requests in one call
        _adapter("adapter_prompts", "adapter_forward", 4096, 4096, 4096, 16, 16, 12),
        # tuning several adapters at once: a small step, ragged sequences, a large step
        _adapter("adapter_tune_small", "adapter_backward", 300, 2048, 768, 4, 8, 5),
        _adapter("adapter_tune_ragged", "adapter_backward", 2049, 2880, 2880, 48, 24, 29),
        _adapter("adapter_tune_large", "adapter_backward", 8192, 4096, 4096, 8, 64, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _by64(rng, lo, hi):
    return 64 * _log(rng, lo // 64, hi // 64)


def draw(rng):
    op = rng.choice(["decode", "decode", "adapter_forward", "adapter_backward"])
    if op == "decode":
        d, n = _by64(rng, 128, 4096), _by64(rng, 64, 14336)
        E = max(2, min(_log(rng, 2, 128), int(2.8e9 / (6 * d * n))))
        return dict(op=op, T=_log(rng, 1, 128), d=d, E=E, K=rng.randint(1, min(8, E)), n=n,
                    capacity=rng.choice([0.0, 0.0, 0.0, 1.25]), bias=rng.random() < 0.3,
                    renormalize=rng.random() < 0.75)
    T = _log(rng, 1, 4096) if op == "adapter_forward" else _log(rng, 16, 8192)
    requests = T if T <= 128 else _log(rng, 1, 64)
    return dict(op=op, T=T, d_in=_by64(rng, 64, 4096), d_out=_by64(rng, 64, 4096),
                adapters=_log(rng, 1, 64), rank=8 * _log(rng, 1, 8), requests=requests)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        out = torch.empty(*shape, dtype=dtype, device="cuda")
        return out.normal_(0.0, std, generator=g)

    s = dict(case=case)
    T = case["T"]
    if case["op"] == "decode":
        d, E, n = case["d"], case["E"], case["n"]
        s.update(x=normal(T, d), w_r=normal(d, E, std=0.02), w_gate=normal(E, d, n, std=0.02),
                 w_up=normal(E, d, n, std=0.02), w_down=normal(E, n, d, std=0.02), bias=None)
        if case["bias"]:  # a few experts draw most tokens
            rank = torch.arange(1, E + 1, dtype=torch.float64, device="cuda")
            s["bias"] = (1.75 * rank.pow(-1.2)).float()
        return s
    d_in, d_out, L, r = case["d_in"], case["d_out"], case["adapters"], case["rank"]
    # requests of uneven lengths, each with an adapter or (one in eight) with none
    R = min(case["requests"], T)
    cuts = torch.randperm(T - 1, generator=g, device="cuda")[:R - 1].sort().values + 1
    of_row = torch.zeros(T, dtype=torch.int64, device="cuda")
    of_row[cuts] = 1
    of_request = torch.randint(0, L, (R,), generator=g, device="cuda")
    none = torch.rand(R, generator=g, device="cuda") < 0.125
    of_request = torch.where(none, torch.full_like(of_request, -1), of_request)
    s.update(x=normal(T, d_in), w=normal(d_in, d_out, std=0.02),
             a=normal(L, d_in, r, std=d_in ** -0.5), b=normal(L, r, d_out, std=0.02),
             ids=of_request[of_row.cumsum(0)].int(),
             scale=0.5 + 1.5 * torch.rand(L, generator=g, device="cuda"))
    if case["op"] == "adapter_backward":
        s.update(d_y=normal(T, d_out, std=0.05), low=_low(s["x"].float(), s["a"].float(), s))
    return s


# ------------------------------------------------------------------ plain forms
def _layer(s):
    c, x = s["case"], s["x"].float()
    T, E, K = c["T"], c["E"], c["K"]
    logits = x @ s["w_r"].float()
    if s["bias"] is not None:
        logits = logits + s["bias"]
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :K]
    w = torch.softmax(logits, dim=1).gather(1, ids)
    if c["renormalize"]:
        w = torch.softmax(logits.gather(1, ids), dim=1)
    if c["capacity"] > 0:  # the first C rows of each expert, in order, are kept
        C = math.ceil(c["capacity"] * T * K / E)
        hot = torch.nn.functional.one_hot(ids.reshape(-1), E)
        place = ((hot.cumsum(0) - 1) * hot).sum(1).reshape(T, K)
        w = torch.where(place < C, w, torch.zeros_like(w))
    if T * K < E:  # only the experts that are taken
        e = ids.reshape(-1)
        rows = x.repeat_interleave(K, 0).unsqueeze(1)
        g = torch.bmm(rows, s["w_gate"][e].float())
        u = torch.bmm(rows, s["w_up"][e].float())
        y = torch.bmm(g * torch.sigmoid(g) * u, s["w_down"][e].float()).view(T, K, -1)
        return (w.unsqueeze(2) * y).sum(1).to(s["x"].dtype)
    g = torch.matmul(x, s["w_gate"].float())
    h = g * torch.sigmoid(g) * torch.matmul(x, s["w_up"].float())
    y = torch.bmm(h, s["w_down"].float())  # every expert for every row
    y = y[ids, torch.arange(T, device=x.device).unsqueeze(1)]
    return (w.unsqueeze(2) * y).sum(1).to(s["x"].dtype)


def _pick(ids, n):
    """[T, n] of 0 and 1: the adapter of each row."""
    return (ids.unsqueeze(1) == torch.arange(n, device=ids.device)).float()


def _low(x, a, s):
    """scale_l x A_l of each row's adapter, 0 where it has none."""
    L, d_in, r = a.shape
    every = (x @ a.transpose(0, 1).reshape(d_in, L * r)).view(-1, L, r)
    return (every * (_pick(s["ids"], L) * s["scale"]).unsqueeze(2)).sum(1)


def _spread(low, s):
    """[T, L * r]: a row's low-rank values at its adapter's place."""
    return (_pick(s["ids"], s["scale"].numel()).unsqueeze(2) * low.unsqueeze(1)).flatten(1)


def _project(s):
    x, b = s["x"].float(), s["b"].float()
    low = _low(x, s["a"].float(), s)
    y = x @ s["w"].float() + _spread(low, s) @ b.flatten(0, 1)
    return y.to(s["x"].dtype), low


def _project_backward(s):
    x, d_y, a, b = (s[k].float() for k in ("x", "d_y", "a", "b"))
    L, d_in, r = a.shape
    d_low = _spread(_low(d_y, b.transpose(1, 2), s), s)
    d_x = d_y @ s["w"].float().t() + d_low @ a.transpose(1, 2).flatten(0, 1)
    d_a = (x.t() @ d_low).view(d_in, L, r).transpose(0, 1).contiguous()
    d_b = (_spread(s["low"], s).t() @ d_y).view(L, r, -1)
    return d_x.to(s["x"].dtype), d_a, d_b


# ------------------------------------------------------------------ the package's calls
def _shape(s):
    """The shape and the workspace that a program keeps for its calls of one size."""
    import token_dispatch_router_b200 as tdr
    c = s["case"]
    if "shape" not in s:
        if c["op"] == "decode":
            s["shape"] = tdr.make_shape(c["T"], c["d"], c["E"], c["K"], c["n"], c["capacity"],
                                        c["renormalize"], torch.bfloat16)
            size = tdr.decode_workspace_size(s["shape"])
        else:
            s["shape"] = tdr.make_adapter_shape(c["T"], c["d_in"], c["d_out"], c["adapters"],
                                                c["rank"])
            size = tdr.adapter_workspace_size(s["shape"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return tdr, s["shape"], s["workspace"]


def _run_own(s):
    tdr, shape, ws = _shape(s)
    op = s["case"]["op"]
    if op == "decode":
        out, _ = tdr.decode(shape, s["x"], s["w_r"], s["w_gate"], s["w_up"], s["w_down"],
                            bias=s["bias"], workspace=ws)
        return {"out": out}
    if op == "adapter_forward":
        y, low, _ = tdr.adapter_forward(shape, s["x"], s["w"], s["a"], s["b"], s["ids"],
                                        s["scale"], workspace=ws)
        return {"y": y, "low": low}
    d_x, d_a, d_b = tdr.adapter_backward(shape, s["d_y"], s["x"], s["w"], s["a"], s["b"],
                                         s["ids"], s["scale"], s["low"], workspace=ws)
    return {"d_x": d_x, "d_a": d_a, "d_b": d_b}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "decode":
        return {"out": _layer(state)}
    if op == "adapter_forward":
        y, low = _project(state)
        return {"y": y, "low": low}
    d_x, d_a, d_b = _project_backward(state)
    return {"d_x": d_x, "d_a": d_a, "d_b": d_b}


# ------------------------------------------------------------------ work
def _taken(n, share, times):
    """How many of n are met at least once when each comes with `share` in each of `times`."""
    return n * (1.0 - (1.0 - share) ** times)


def work(case):
    T = case["T"]
    if case["op"] == "decode":
        d, E, K, n = case["d"], case["E"], case["K"], case["n"]
        experts = _taken(E, K / E, T)
        return {"bytes": 2.0 * (3 * experts * d * n + d * E + 2 * T * d),
                "flops": 2.0 * T * (3 * K * d * n + d * E)}
    d_in, d_out, L, r = case["d_in"], case["d_out"], case["adapters"], case["rank"]
    used = _taken(L, 0.875 / L, min(case["requests"], T))
    rows, ab = T * (d_in + d_out), used * r * (d_in + d_out)
    if case["op"] == "adapter_forward":
        return {"bytes": 2.0 * (rows + d_in * d_out + ab) + 4.0 * T * (r + 1),
                "flops": 2.0 * T * (d_in * d_out + r * (d_in + d_out))}
    return {"bytes": 2.0 * (rows + T * d_in + d_in * d_out + ab) + 4.0 * T * (r + 1)
            + 4.0 * L * r * (d_in + d_out),
            "flops": 2.0 * T * (d_in * d_out + 2 * r * (d_in + d_out))}


# ------------------------------------------------------------------ 64 bits
def _exact_layer(s):
    c = s["case"]
    x, T, K = s["x"].double(), c["T"], c["K"]
    logits = x @ s["w_r"].double()
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    ids = torch.argsort(-logits, dim=1, stable=True)[:, :K]
    top = torch.exp(logits - logits.max(1, keepdim=True).values)
    w = torch.gather(top, 1, ids)
    w = w / (w if c["renormalize"] else top).sum(1, keepdim=True)
    out = torch.zeros_like(x)
    C = math.ceil(c["capacity"] * T * K / c["E"]) if c["capacity"] > 0 else T * K
    for e in range(c["E"]):
        t, k = (ids == e).nonzero(as_tuple=True)
        t, k = t[:C], k[:C]
        if t.numel():
            g, u = x[t] @ s["w_gate"][e].double(), x[t] @ s["w_up"][e].double()
            y = (g / (1.0 + torch.exp(-g)) * u) @ s["w_down"][e].double()
            out[t] += w[t, k].unsqueeze(1) * y
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return {"out": _exact_layer(s)}
    x, w, a, b = (s[k].double() for k in ("x", "w", "a", "b"))
    low = torch.zeros(case["T"], case["rank"], dtype=torch.float64, device=x.device)
    if case["op"] == "adapter_forward":
        y = x @ w
        for l in range(case["adapters"]):
            t = (s["ids"] == l).nonzero().squeeze(1)
            low[t] = s["scale"][l].double() * (x[t] @ a[l])
            y[t] += low[t] @ b[l]
        return {"y": y, "low": low}
    d_y = s["d_y"].double()
    d_x, d_a, d_b = d_y @ w.t(), torch.zeros_like(a), torch.zeros_like(b)
    for l in range(case["adapters"]):
        t = (s["ids"] == l).nonzero().squeeze(1)
        d_low = s["scale"][l].double() * (d_y[t] @ b[l].t())
        d_x[t] += d_low @ a[l].t()
        d_a[l] = x[t].t() @ d_low
        d_b[l] = s["low"][t].double().t() @ d_y[t]
    return {"d_x": d_x, "d_a": d_a, "d_b": d_b}
