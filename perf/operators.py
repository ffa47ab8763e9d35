"""Cases of the int8 and expert-routing operators, in a plain form and through
the library.

Five operators, named by a case's "op":

  quantize   rows of activations to 8-bit integers with one scale a row
  int8       C = scaleA[i] * scaleB[j] * sum_p A[i][p] * B[p][j] + bias[j], A and B in int8
  experts    the same product with one B per expert, over rows sorted by expert
  dispatch   tokens sorted by expert and their rows moved there: "serve" quantizes
             them on the way, "train" also takes the gradient back
  combine    the experts' rows back in the tokens' order with the router's
             weights applied: "serve" forward only, "train" with both gradients

`run` computes them with elementary torch operations in 32 bits where `own` is
false, and through dense_fp32_matrix_09_gb300.sgemm where it is true.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_IDS = {"f32": 0, "bf16": 1, "f16": 2}      # the library's element type values
_DEV = "cuda"
_kept = {}                                   # the library's binding and one handle, as a program keeps them


def _library():
    if not _kept:
        from dense_fp32_matrix_09_gb300 import sgemm
        _kept["sgemm"], _kept["h"] = sgemm, sgemm.sgemm_create()
    return _kept["sgemm"], _kept["h"]


# ---------------------------------------------------------------- the cases
def _quantize(m, k, dtype, pad=0):
    return {"op": "quantize", "m": m, "k": k, "dtype": dtype, "pad": pad}


def _int8(m, n, k, dtype, trans_b=1, bias=False, pad=0):
    return {"op": "int8", "m": m, "n": n, "k": k, "dtype": dtype, "trans_b": trans_b, "bias": bias, "pad": pad}


def _experts(rows, n, k, experts, dtype, bias=False, skew=0.5):
    return {"op": "experts", "rows": rows, "n": n, "k": k, "experts": experts, "dtype": dtype, "bias": bias, "skew": skew}


def _dispatch(way, tokens, choices, experts, width, dtype, dropped=0.0):
    return {"op": "dispatch", "way": way, "tokens": tokens, "choices": choices, "experts": experts, "width": width, "dtype": dtype, "dropped": dropped}


def _combine(way, tokens, choices, experts, width, dtype, dropped=0.0):
    return {"op": "combine", "way": way, "tokens": tokens, "choices": choices, "experts": experts, "width": width, "dtype": dtype, "dropped": dropped}


def listed():
    cases = {
        # one decode step of a small batch: a launch's latency
        "quantize_decode": _quantize(16, 4096, "bf16"),
        # a long prompt's activations before the largest product: one pass over HBM
        "quantize_prompt": _quantize(8192, 8192, "bf16"),
        # one token against one layer's weights: reading B once is all there is
        "int8_token": _int8(1, 4096, 4096, "bf16"),
        # a decode batch against a large layer: B from HBM, and some arithmetic
        "int8_batch": _int8(64, 8192, 8192, "f16", bias=True),
        # the benchmark's ragged shape with padded rows and B stored K x N: odd sizes, no 16-byte alignment
        "int8_ragged": _int8(1000, 1500, 777, "f32", trans_b=0, pad=3),
        # the benchmark's largest shape: bound by the tensor cores
        "int8_prompt": _int8(8192, 8192, 8192, "bf16"),
        # decode through a mixture of experts: 128 rows over 32 experts, every expert's weights read
        "experts_decode": _experts(128, 4096, 4096, 32, "bf16"),
        # prefill through a mixture of experts: uneven groups of a thousand rows or so
        "experts_prompt": _experts(16384, 4096, 4096, 16, "bf16"),
        # routing of a decode step, quantized on the way to the experts: latency
        "dispatch_decode": _dispatch("serve", 32, 4, 32, 4096, "bf16"),
        # routing of a training step with its gradient, some choices dropped: HBM traffic
        "dispatch_train": _dispatch("train", 8192, 4, 64, 4096, "bf16", dropped=0.03),
        # the way back of a decode step: latency
        "combine_decode": _combine("serve", 32, 4, 32, 4096, "bf16"),
        # the way back of a training step, with the gradients of rows and weights
        "combine_train": _combine("train", 8192, 4, 64, 4096, "f16"),
    }
    return [dict(c, name=name) for name, c in cases.items()]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["quantize", "int8", "int8", "experts", "dispatch", "combine"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "quantize":
        return _quantize(_log(rng, 1, 8192), _log(rng, 16, 8192), dtype, pad=rng.choice([0, 0, 1, 8]))
    if op == "int8":
        m, n, k = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 8192)
        return _int8(m, n, k, dtype, trans_b=rng.choice([1, 1, 1, 0]), bias=rng.random() < 0.5, pad=rng.choice([0, 0, 3, 16]))
    if op == "experts":
        # rows from a decode step's to a long prompt's; the weights stay under a gigabyte
        e = rng.choice([4, 8, 16, 32, 64])
        k, n = 16 * _log(rng, 8, 256), _log(rng, 128, 4096)
        return _experts(_log(rng, 8, 16384), n, k, e, dtype, bias=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]))
    e = rng.choice([8, 16, 64, 128])
    make = _dispatch if op == "dispatch" else _combine
    return make(rng.choice(["serve", "train"]), _log(rng, 1, 8192), rng.choice([1, 2, 4]), e, _log(rng, 64, 4096), dtype, dropped=rng.choice([0.0, 0.0, 0.05]))


def work(case):
    """Each input read once, each output written once."""
    c, size = case, _TYPES[case["dtype"]].itemsize
    if c["op"] == "quantize":
        return {"bytes": c["m"] * (c["k"] * (size + 1) + 4), "flops": 3 * c["m"] * c["k"]}
    if c["op"] == "int8":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + (4 * n if c["bias"] else 0) + m * n * size, "flops": 2 * m * n * k}
    if c["op"] == "experts":
        r, n, k, e = c["rows"], c["n"], c["k"], min(c["experts"], c["rows"])
        return {"bytes": r * k + e * n * (k + 4 + (4 if c["bias"] else 0)) + 4 * r + r * n * size, "flops": 2 * r * n * k}
    t, w, slots = c["tokens"], c["width"], c["tokens"] * c["choices"]
    if c["op"] == "dispatch":
        sort = 4 * (3 * slots + c["experts"] + 1)
        if c["way"] == "serve":
            return {"bytes": sort + t * w * size + slots * (w + 4), "flops": 3 * t * w}
        return {"bytes": sort + 2 * (t + slots) * w * size, "flops": slots * w}
    forward = 8 * slots + (slots + t) * w * size
    if c["way"] == "serve":
        return {"bytes": forward, "flops": 2 * slots * w}
    return {"bytes": forward + 4 * slots + (2 * slots + t) * w * size, "flops": 5 * slots * w}


# ------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device=_DEV).manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=_DEV)


def _activations(g, rows, width, dtype):
    """Rows of unequal size with a few large channels, as a layer's input has them."""
    x = _normal(g, rows, width) * torch.exp(0.5 * _normal(g, rows, 1))
    x[:, ::97] *= 6
    return x.to(dtype)


def _padded(x, pad):
    """The same matrix in a buffer whose rows are `pad` elements longer."""
    if not pad:
        return x.contiguous()
    full = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=x.dtype, device=_DEV)
    full[:, :x.shape[1]] = x
    return full[:, :x.shape[1]]


def _integers(g, *shape):
    """What a symmetric 8-bit quantizer makes of a normal distribution."""
    return (_normal(g, *shape) * 32).round_().clamp_(-127, 127).to(torch.int8)


def _scales(g, *shape):
    return (0.5 + torch.rand(*shape, generator=g, device=_DEV)) / 1024


def _routes(g, tokens, choices, experts, dropped):
    """Distinct experts a token, some of them liked more than others; -1 where a choice is dropped."""
    liked = 0.7 * _normal(g, 1, experts)
    score = _normal(g, tokens, experts) + liked
    ids = score.topk(choices, dim=1).indices.to(torch.int32)
    if dropped:
        gone = torch.rand(tokens, choices, generator=g, device=_DEV) < dropped
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    weights = torch.softmax(_normal(g, tokens, choices), dim=1)
    return ids.contiguous(), weights.contiguous()


def prepare(case, seed):
    c, g, dtype = case, _generator(seed), _TYPES[case["dtype"]]
    empty = lambda *shape, kind=dtype: torch.zeros(*shape, dtype=kind, device=_DEV)  # noqa: E731
    s = {"case": c}
    if c["op"] == "quantize":
        s["x"] = _padded(_activations(g, c["m"], c["k"], dtype), c["pad"])
        s["q"], s["scale"] = empty(c["m"], c["k"], kind=torch.int8), empty(c["m"], kind=torch.float32)
    elif c["op"] == "int8":
        m, n, k = c["m"], c["n"], c["k"]
        s["a"] = _padded(_integers(g, m, k), c["pad"])
        s["b"] = _padded(_integers(g, *((n, k) if c["trans_b"] else (k, n))), c["pad"])
        s["scale_a"], s["scale_b"] = _scales(g, m), _scales(g, n)
        s["bias"] = _normal(g, n) if c["bias"] else None
        s["c"] = empty(m, n)
    elif c["op"] == "experts":
        r, n, k, e = c["rows"], c["n"], c["k"], c["experts"]
        share = torch.softmax(c["skew"] * _normal(g, e), dim=0)
        owner = torch.multinomial(share, r, replacement=True, generator=g)
        counts = (owner[None, :] == torch.arange(e, device=_DEV)[:, None]).sum(1)
        offsets = torch.zeros(e + 1, dtype=torch.int32, device=_DEV)
        offsets[1:] = counts.cumsum(0)
        s["offsets"], s["most"] = offsets, int(counts.max())
        s["a"], s["b"] = _integers(g, r, k), _integers(g, e, n, k)
        s["scale_a"], s["scale_b"] = _scales(g, r), _scales(g, e, n)
        s["bias"] = _normal(g, e, n) if c["bias"] else None
        s["c"] = empty(r, n)
    else:
        t, j, e, w = c["tokens"], c["choices"], c["experts"], c["width"]
        ids, weights = _routes(g, t, j, e, c["dropped"])
        if c["op"] == "dispatch":
            s["ids"], s["x"] = ids, _activations(g, t, w, dtype)
            s["offsets"] = empty(e + 1, kind=torch.int32)
            s["rows"], s["source"] = empty(t * j, kind=torch.int32), empty(t * j, kind=torch.int32)
            if c["way"] == "serve":
                s["q"], s["scale"] = empty(t * j, w, kind=torch.int8), empty(t * j, kind=torch.float32)
            else:
                s["y"], s["dx"] = empty(t * j, w), empty(t, w)
                s["dy"] = _normal(g, t * j, w).to(dtype)
        else:
            s["rows"], s["weights"] = _sorted(ids, e)[1], weights
            s["y"], s["out"] = _activations(g, t * j, w, dtype), empty(t, w)
            if c["way"] == "train":
                s["dout"] = _normal(g, t, w).to(dtype)
                s["dy"], s["dweights"] = empty(t * j, w), empty(t, j, kind=torch.float32)
    return s


# -------------------------------------------------------------- plain forms
def _sorted(ids, experts):
    """(offsets, row of each slot or -1, slot of each row or -1): a stable sort by expert, unknown experts left out."""
    key = ids.reshape(-1)
    key = torch.where((key >= 0) & (key < experts), key, torch.full_like(key, experts))
    in_order, order = torch.sort(key, stable=True)
    offsets = (in_order[None, :] < torch.arange(experts + 1, device=_DEV)[:, None]).sum(1).to(torch.int32)
    source = torch.where(in_order < experts, order, torch.full_like(order, -1)).to(torch.int32)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=_DEV)
    rows = torch.where(key < experts, place, torch.full_like(place, -1)).to(torch.int32)
    return offsets, rows, source


def _quantized(x):
    x = x.float()
    top = x.abs().amax(dim=1, keepdim=True)
    steps = torch.full_like(top, 127.0)
    q = torch.round(x * (steps / top)).clamp(-127, 127)
    return torch.where(top > 0, q, torch.zeros_like(q)).to(torch.int8), (top / steps).squeeze(1)


def _plain_int8(s):
    c, b = s["case"], s["b"].float()
    out = s["a"].float() @ (b.t() if c["trans_b"] else b)
    out = out * s["scale_a"][:, None] * s["scale_b"][None, :]
    if s["bias"] is not None:
        out = out + s["bias"]
    return {"c": out.to(_TYPES[c["dtype"]])}


def _plain_experts(s):
    # every expert's rows side by side, the shorter groups filled up, and one batched product
    c, offsets = s["case"], s["offsets"].long()
    at = offsets[:-1, None] + torch.arange(s["most"], device=_DEV)
    inside = at < offsets[1:, None]
    a = s["a"].float()[at.clamp(max=c["rows"] - 1)]
    out = torch.bmm(a, s["b"].float().transpose(1, 2)) * s["scale_b"][:, None, :]
    if s["bias"] is None:
        bias = 0
    else:
        bias = s["bias"][:, None, :]
    out = out * s["scale_a"][at.clamp(max=c["rows"] - 1)][:, :, None] + bias
    return {"c": out[inside].to(_TYPES[c["dtype"]])}


def _plain_dispatch(s):
    c = s["case"]
    offsets, rows, source = _sorted(s["ids"], c["experts"])
    there, token = source >= 0, source.clamp(min=0).long() // c["choices"]
    out = {"offsets": offsets, "rows": rows, "source": source}
    if c["way"] == "serve":
        q, scale = _quantized(s["x"])
        out["q"] = torch.where(there[:, None], q[token], torch.zeros_like(q[:1]))
        out["scale"] = torch.where(there, scale[token], torch.zeros_like(scale[:1]))
        return out
    x = s["x"].float()
    out["y"] = torch.where(there[:, None], x[token], torch.zeros_like(x[:1])).to(s["x"].dtype)
    kept = (rows >= 0)[:, None]
    back = torch.where(kept, s["dy"].float()[rows.clamp(min=0).long()], torch.zeros_like(x[:1]))
    out["dx"] = back.reshape(c["tokens"], c["choices"], c["width"]).sum(1).to(s["x"].dtype)
    return out


def _plain_combine(s):
    c, dtype = s["case"], s["y"].dtype
    shape = (c["tokens"], c["choices"], c["width"])
    rows = s["rows"]
    kept = (rows >= 0)[:, None]
    y = s["y"].float()
    mine = torch.where(kept, y[rows.clamp(min=0).long()], torch.zeros_like(y[:1])).reshape(shape)
    out = {"out": (mine * s["weights"][:, :, None]).sum(1).to(dtype)}
    if c["way"] == "train":
        dout = s["dout"].float()
        out["dweights"] = (mine * dout[:, None, :]).sum(2)
        grad = (s["weights"][:, :, None] * dout[:, None, :]).reshape(-1, c["width"]).to(dtype)
        # rows of dropped choices go to one row past the end
        to = torch.where(rows >= 0, rows, torch.full_like(rows, rows.numel())).long()
        dy = torch.zeros(rows.numel() + 1, c["width"], dtype=dtype, device=_DEV)
        dy[to] = grad
        out["dy"] = dy[:-1]
    return out


# ------------------------------------------------------- through the library
def _own(s):
    L, h = _library()
    c, op = s["case"], s["case"]["op"]
    kind = _IDS[c["dtype"]]
    if op == "quantize":
        L.sgemm_quantize_rows(h, kind, c["m"], c["k"], s["x"], c["k"] + c["pad"], s["q"], c["k"], s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    if op == "int8":
        m, n, k, pad = c["m"], c["n"], c["k"], c["pad"]
        L.sgemm_run_int8(h, c["trans_b"], kind, m, n, k, s["a"], k + pad, s["scale_a"], s["b"], (k if c["trans_b"] else n) + pad, s["scale_b"], s["bias"], s["c"], n)
        return {"c": s["c"]}
    if op == "experts":
        n, k = c["n"], c["k"]
        L.sgemm_run_int8_experts(h, 1, kind, c["experts"], c["rows"], n, k, s["offsets"], s["a"], k, s["scale_a"], s["b"], k, n * k, s["scale_b"], s["bias"], s["c"], n)
        return {"c": s["c"]}
    t, j, w = c["tokens"], c["choices"], c["width"]
    if op == "dispatch":
        L.sgemm_expert_sort(h, t, j, c["experts"], s["ids"], s["offsets"], s["rows"], s["source"])
        out = {"offsets": s["offsets"], "rows": s["rows"], "source": s["source"]}
        if c["way"] == "serve":
            L.sgemm_expert_dispatch_int8(h, kind, t, j, w, s["x"], w, s["rows"], s["q"], w, s["scale"])
            return dict(out, q=s["q"], scale=s["scale"])
        L.sgemm_expert_dispatch(h, kind, t, j, w, s["x"], w, s["rows"], s["y"], w)
        L.sgemm_expert_dispatch_grad(h, kind, t, j, w, s["dy"], w, s["rows"], s["dx"], w)
        return dict(out, y=s["y"], dx=s["dx"])
    L.sgemm_expert_combine(h, kind, t, j, w, s["y"], w, s["rows"], s["weights"], s["out"], w)
    if c["way"] == "serve":
        return {"out": s["out"]}
    L.sgemm_expert_combine_grad(h, kind, t, j, w, s["dout"], w, s["y"], w, s["rows"], s["weights"], s["dy"], w, s["dweights"])
    return {"out": s["out"], "dy": s["dy"], "dweights": s["dweights"]}


_PLAIN = {"int8": _plain_int8, "experts": _plain_experts, "dispatch": _plain_dispatch, "combine": _plain_combine}


def run(state):
    if own:
        return _own(state)
    if state["case"]["op"] == "quantize":
        q, scale = _quantized(state["x"])
        return {"q": q, "scale": scale}
    return _PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------- in 64 bits
def _slots(ids, experts):
    """Row of each slot by counting: slots of lower experts, and earlier slots of the same one."""
    seen, rows = [0] * experts, []
    flat = ids.reshape(-1).tolist()
    for i in flat:
        if 0 <= i < experts:
            seen[i] += 1
    start = [sum(seen[:i]) for i in range(experts)]
    for i in flat:
        if 0 <= i < experts:
            rows.append(start[i])
            start[i] += 1
        else:
            rows.append(-1)
    return rows


def exact(case, seed):
    """The outputs in 64 bits; None where they are whole numbers."""
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        return {"q": None, "scale": s["x"].double().abs().max(dim=1).values / 127}
    if c["op"] == "int8":
        b = s["b"].double()
        sums = torch.mm(s["a"].double(), b.T if c["trans_b"] else b)
        sums.mul_(s["scale_b"].double()).mul_(s["scale_a"].double().unsqueeze(1))
        return {"c": sums if s["bias"] is None else sums.add_(s["bias"].double())}
    if c["op"] == "experts":
        at, parts = s["offsets"].tolist(), []
        for e in range(c["experts"]):
            part = torch.mm(s["a"][at[e]:at[e + 1]].double(), s["b"][e].double().T)
            part.mul_(s["scale_b"][e].double()).mul_(s["scale_a"][at[e]:at[e + 1]].double().unsqueeze(1))
            parts.append(part if s["bias"] is None else part.add_(s["bias"][e].double()))
        return {"c": torch.cat(parts)}
    t, j, w = c["tokens"], c["choices"], c["width"]
    rows = _slots(s["ids"], c["experts"]) if c["op"] == "dispatch" else s["rows"].tolist()
    kept = [i for i, r in enumerate(rows) if r >= 0]
    slot = torch.tensor(kept, dtype=torch.long, device=_DEV)
    row = torch.tensor([rows[i] for i in kept], dtype=torch.long, device=_DEV)
    token = slot // j
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=_DEV)  # noqa: E731
    if c["op"] == "dispatch":
        out = {"offsets": None, "rows": None, "source": None}
        x = s["x"].double()
        if c["way"] == "serve":
            scale = zeros(t * j)
            scale[row] = (x.abs().max(dim=1).values / 127)[token]
            return dict(out, q=None, scale=scale)
        y = zeros(t * j, w)
        y[row] = x[token]
        return dict(out, y=y, dx=zeros(t, w).index_add_(0, token, s["dy"].double()[row]))
    y, weight = s["y"].double()[row], s["weights"].double().reshape(-1)[slot].unsqueeze(1)
    out = {"out": zeros(t, w).index_add_(0, token, y * weight)}
    if c["way"] == "train":
        dout = s["dout"].double()[token]
        dweights, dy = zeros(t * j), zeros(t * j, w)
        dweights[slot] = (dout * y).sum(1)
        dy[row] = dout * weight
        out.update(dy=dy, dweights=dweights.reshape(t, j))
    return out
