"""Cases of the RMS norm, the 4-bit floating-point products and the whole
mixture-of-experts layer, in a plain form and through the library.

Five operators, named by a case's "op":

  norm     h = x + residual, y = h * w / rms(h): "int8" gives y in 8 bits with a
           scale a row, "train" y itself and then the gradients of x and w
  rows     rows to microscaled 4-bit floating point and back to what it stands for
  linear   rows to 4 bits (with "norm" after the RMS norm) times weights in 4 bits
  product  the product of two matrices that are in 4 bits already
  layer    sum over a token's experts of weight * down(act(up(x))), a few tokens, int8 weights

`run` computes them with elementary torch operations in 32 bits where `own` is
false, and through dense_fp32_matrix_09_gb300.sgemm where it is true.

4-bit rows: two elements a byte, the even one in the low half; a scale for every 32
(format "mx": powers of two, E8M0) or 16 elements (format "nv": E4M3, and one FP32
a row).  The scales lie in tiles of 128 rows x 4 blocks: [row / 128][block / 4][row %
32][row / 32 % 4][block % 4].
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_IDS = {"f32": 0, "bf16": 1, "f16": 2}      # the library's element type values
_FORMATS = {"mx": 0, "nv": 1}               # and those of its 4-bit formats
_BLOCK = {"mx": 32, "nv": 16}
_EPS = 1e-5
_DEV = "cuda"
_kept = {}                                   # the library's binding and one handle, as a program keeps them


def _library():
    if not _kept:
        from dense_fp32_matrix_09_gb300 import sgemm
        _kept["sgemm"], _kept["h"] = sgemm, sgemm.sgemm_create()
    return _kept["sgemm"], _kept["h"]


# ---------------------------------------------------------------- the cases
def _norm(way, m, k, dtype, residual=True, pad=0):
    return {"op": "norm", "way": way, "m": m, "k": k, "dtype": dtype, "residual": residual, "pad": pad}


def _rows(m, k, dtype, form, pad=0):
    return {"op": "rows", "m": m, "k": k, "dtype": dtype, "form": form, "pad": pad}


def _linear(m, n, k, dtype, form, norm=False, bias=False):
    return {"op": "linear", "m": m, "n": n, "k": k, "dtype": dtype, "form": form, "norm": norm, "bias": bias}


def _product(m, n, k, dtype, form, bias=False, pad=0):
    return {"op": "product", "m": m, "n": n, "k": k, "dtype": dtype, "form": form, "bias": bias, "pad": pad}


def _layer(tokens, choices, experts, width, hidden, dtype, gated=True, dropped=0.0):
    return {"op": "layer", "tokens": tokens, "choices": choices, "experts": experts, "width": width, "hidden": hidden, "dtype": dtype, "gated": gated, "dropped": dropped}


def listed():
    cases = {
        # a decode step's rows before an int8 product: a launch's latency
        "norm_decode": _norm("int8", 32, 4096, "bf16"),
        # a long prompt's rows before an int8 product: one pass over HBM
        "norm_prompt": _norm("int8", 8192, 8192, "bf16"),
        # forward and backward of a training step, the gradient of w summed over the rows
        "norm_train": _norm("train", 8192, 4096, "bf16"),
        # a decode step's rows to 4 bits and back: latency
        "rows_decode": _rows(16, 4096, "bf16", "nv"),
        # a long prompt's: two passes over HBM
        "rows_prompt": _rows(8192, 8192, "f16", "mx"),
        # one token against one layer's weights: reading them is all there is
        "linear_token": _linear(1, 4096, 4096, "bf16", "nv"),
        # a decode batch, normed, against a large layer: weights from HBM, and some arithmetic
        "linear_batch": _linear(64, 8192, 8192, "f16", "mx", norm=True, bias=True),
        # the benchmark's ragged shape with rows that start on no 16-byte boundary
        "product_ragged": _product(1000, 1500, 777, "f32", "mx", pad=3),
        # the benchmark's largest shape: bound by the tensor cores
        "product_prompt": _product(8192, 8192, 8192, "bf16", "nv"),
        # one token through a mixture of experts: four experts' weights read
        "layer_token": _layer(1, 4, 32, 4096, 2048, "bf16"),
        # a small batch: two thirds of the experts
        "layer_few": _layer(8, 4, 32, 4096, 2048, "bf16"),
        # a decode batch, every expert with several tokens
        "layer_batch": _layer(48, 2, 16, 2048, 1408, "f16"),
    }
    return [dict(c, name=name) for name, c in cases.items()]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "rows", "linear", "linear", "product", "layer", "layer"])
    dtype, form = rng.choice(["f32", "bf16", "f16"]), rng.choice(["mx", "nv"])
    if op == "norm":
        return _norm(rng.choice(["int8", "train"]), _log(rng, 1, 8192), _log(rng, 16, 8192), dtype, residual=rng.random() < 0.7, pad=rng.choice([0, 0, 1, 8]))
    if op == "rows":
        return _rows(_log(rng, 1, 8192), _log(rng, 16, 8192), dtype, form, pad=rng.choice([0, 0, 1, 8]))
    if op == "linear":
        return _linear(_log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 8192), dtype, form, norm=rng.random() < 0.5, bias=rng.random() < 0.5)
    if op == "product":
        return _product(_log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 8192), dtype, form, bias=rng.random() < 0.5, pad=rng.choice([0, 0, 3, 16]))
    return _layer(_log(rng, 1, 64), rng.choice([1, 2, 4]), rng.choice([4, 8, 16, 32]), _log(rng, 64, 4096), _log(rng, 64, 2048), rng.choice(["bf16", "bf16", "f16", "f32"]), gated=rng.random() < 0.7, dropped=rng.choice([0.0, 0.0, 0.05]))


def _row_bytes(k, form):
    """A row in 4 bits: the elements, the blocks' scales and, where it has one, its own."""
    return (k + 1) // 2 + -(-k // _BLOCK[form]) + (4 if form == "nv" else 0)


def work(case):
    """Each input read once, each output written once."""
    c, size = case, _TYPES[case["dtype"]].itemsize
    if c["op"] == "norm":
        m, k = c["m"], c["k"]
        streams = (3 if c["residual"] else 1) * m * k * size + k * size    # x, the residual in and out, w
        if c["way"] == "int8":
            return {"bytes": streams + m * k + 4 * m, "flops": 8 * m * k}
        # y; then dy, h and the residual's gradient, dx, and dw
        return {"bytes": streams + m * k * size + 4 * m + (4 if c["residual"] else 3) * m * k * size + 4 * k, "flops": 16 * m * k}
    if c["op"] == "rows":
        m, k = c["m"], c["k"]
        return {"bytes": 2 * m * k * size + m * _row_bytes(k, c["form"]), "flops": 6 * m * k}
    if c["op"] == "layer":
        t, w, f = c["tokens"], c["width"], c["hidden"]
        up = 2 if c["gated"] else 1
        slots = t * c["choices"]
        # of `experts` equally liked ones, so many are asked by some token
        asked = c["experts"] * (1 - (1 - c["choices"] / c["experts"]) ** t)
        return {"bytes": int(asked * ((up + 1) * f * w + 4 * (up * f + w))) + 2 * t * w * size + 8 * slots, "flops": 2 * slots * (up + 1) * f * w}
    m, n, k = c["m"], c["n"], c["k"]
    rows = m * _row_bytes(k, c["form"])
    if c["op"] == "linear":
        # the rows as they come (normed: with the residual in and out, and w)
        rows = ((3 * m + 1) if c["norm"] else m) * k * size
    return {"bytes": rows + n * _row_bytes(k, c["form"]) + (4 * n if c["bias"] else 0) + m * n * size, "flops": 2 * m * n * k}


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


def _scale_bytes(rows, k, form):
    return -(-rows // 128) * -(-(-(-k // _BLOCK[form])) // 4) * 512


def _tiled(s):
    """Scales (rows x blocks, uint8) in tiles of 128 x 4, the rest of the last tiles zero."""
    rows, blocks = s.shape
    full = torch.zeros(-(-rows // 128) * 128, -(-blocks // 4) * 4, dtype=torch.uint8, device=_DEV)
    full[:rows, :blocks] = s
    return full.reshape(full.shape[0] // 128, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _untiled(s, rows, blocks):
    r, b = -(-rows // 128), -(-blocks // 4)
    return s.reshape(r, b, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r * 128, b * 4)[:rows, :blocks]


def _packed(codes):
    """Two 4-bit codes a byte, the even column's in the low half."""
    if codes.shape[1] % 2:
        codes = torch.nn.functional.pad(codes, (0, 1))
    return codes[:, ::2] | (codes[:, 1::2] << 4)


def _fp4_matrix(g, rows, k, form, pad):
    """A matrix in 4 bits: {codes, scales, row scales}, from a layer's weights or activations."""
    q, s, row = _to_fp4(_normal(g, rows, k) * torch.exp(0.3 * _normal(g, rows, 1)) / math.sqrt(k), form)
    wide = (k + 1) // 2
    # rows on 16-byte boundaries unless the case wants others
    ld = wide + pad if pad else -(-wide // 16) * 16
    full = torch.zeros(rows, ld, dtype=torch.uint8, device=_DEV)
    full[:, :wide] = _packed(_codes(q))
    return {"q": full, "ld": ld, "s": _tiled(s), "row": row}


def _routes(g, tokens, choices, experts, dropped):
    """Distinct experts a token; -1 where a choice is dropped."""
    ids = _normal(g, tokens, experts).topk(choices, dim=1).indices.to(torch.int32)
    if dropped:
        gone = torch.rand(tokens, choices, generator=g, device=_DEV) < dropped
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.contiguous(), torch.softmax(_normal(g, tokens, choices), dim=1).contiguous()


def _int8_weights(g, experts, n, k):
    w = torch.empty(experts, n, k, dtype=torch.int8, device=_DEV)
    for e in range(experts):
        w[e] = (_normal(g, n, k) * 32).round_().clamp_(-127, 127).to(torch.int8)
    return w, (0.5 + torch.rand(experts, n, generator=g, device=_DEV)) / (32 * math.sqrt(k))


def prepare(case, seed):
    c, g, dtype = case, _generator(seed), _TYPES[case["dtype"]]
    empty = lambda *shape, kind=dtype: torch.zeros(*shape, dtype=kind, device=_DEV)  # noqa: E731
    s = {"case": c}
    if c["op"] == "layer":
        t, e, w, f = c["tokens"], c["experts"], c["width"], c["hidden"]
        s["x"], s["out"] = _activations(g, t, w, dtype), empty(t, w)
        s["ids"], s["weights"] = _routes(g, t, c["choices"], e, c["dropped"])
        s["up"], s["up_scale"] = _int8_weights(g, e, (2 if c["gated"] else 1) * f, w)
        s["down"], s["down_scale"] = _int8_weights(g, e, w, f)
        s["most"] = int((s["ids"].reshape(1, -1) == torch.arange(e, device=_DEV)[:, None]).sum(1).max())
        return s
    m, k = c["m"], c["k"]
    if c["op"] == "norm" or c.get("norm"):
        residual = c.get("residual", True)
        pad = c.get("pad", 0)
        s["x"] = _padded(_activations(g, m, k, dtype), pad)
        s["residual"] = _padded(_activations(g, m, k, dtype), pad) if residual else None
        s["w"] = (1 + 0.2 * _normal(g, k)).to(dtype)
        s["h"] = empty(m, k) if residual else None
    if c["op"] == "norm":
        if c["way"] == "int8":
            s["q"], s["scale"] = empty(m, k, kind=torch.int8), empty(m, kind=torch.float32)
        else:
            s["dy"] = _normal(g, m, k).to(dtype)
            s["dh"] = _normal(g, m, k).to(dtype) if s["residual"] is not None else None
            s["y"], s["rstd"] = empty(m, k), empty(m, kind=torch.float32)
            s["dx"], s["dw"] = empty(m, k), empty(k, kind=torch.float32)
        return s
    form = c["form"]
    if c["op"] in ("rows", "linear"):
        if "x" not in s:
            s["x"] = _padded(_activations(g, m, k, dtype), c.get("pad", 0))
        wide = -(-k // 32) * 16
        s["a"] = {"q": empty(m, wide, kind=torch.uint8), "ld": wide, "s": empty(_scale_bytes(m, k, form), kind=torch.uint8), "row": empty(m, kind=torch.float32) if form == "nv" or c.get("norm") else None}
        if c["op"] == "rows":
            s["y"] = empty(m, k)
            return s
    else:
        s["a"] = _fp4_matrix(g, m, k, form, c["pad"])
    s["b"] = _fp4_matrix(g, c["n"], k, form, c.get("pad", 0))
    s["bias"] = _normal(g, c["n"]) if c["bias"] else None
    s["c"] = empty(m, c["n"])
    return s


# -------------------------------------------------------------- plain forms
def _by_block(x, block):
    """rows x blocks x block, zeros behind the last element."""
    rest = -x.shape[1] % block
    return torch.nn.functional.pad(x, (0, rest)).reshape(x.shape[0], -1, block)


def _e2m1(x):
    """The nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 with x's sign, ties to the even code."""
    a = x.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.clamp(torch.round(a / step) * step, max=6.0), x)


def _codes(q):
    """The 4-bit codes of values of that kind: sign, two bits of exponent, one of fraction."""
    a = q.abs()
    low = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    return low | (torch.signbit(q).to(torch.uint8) << 3)


_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _to_fp4(x, form):
    """(values, scale bytes, row scales) of FP32 rows."""
    k, blocks = x.shape[1], _by_block(x, _BLOCK[form])
    top = blocks.abs().amax(dim=2)
    if form == "mx":
        byte = ((top.view(torch.int32) >> 23) - 2).clamp(min=0)
        q = _e2m1(torch.ldexp(blocks, (127 - byte)[:, :, None].to(torch.float32)))
        return q.reshape(x.shape[0], -1)[:, :k], byte.to(torch.uint8), None
    m = top.amax(dim=1, keepdim=True)
    some = m >= 2688 * 2.0 ** -126
    steps = torch.full_like(m, 2688.0)
    up = torch.where(some, steps / m, torch.zeros_like(m))
    near = torch.where(some, torch.full_like(m, 448.0) / m, torch.zeros_like(m))
    scale = (top * near).to(torch.float8_e4m3fn)
    wide = scale.float()
    q = _e2m1(blocks * torch.where(wide > 0, up / wide, torch.zeros_like(wide))[:, :, None])
    return q.reshape(x.shape[0], -1)[:, :k], scale.view(torch.uint8), torch.where(some, m / steps, torch.zeros_like(m)).squeeze(1)


def _scale_values(s, form):
    return torch.ldexp(torch.ones_like(s, dtype=torch.float32), s.float() - 127) if form == "mx" else s.view(torch.float8_e4m3fn).float()


def _from_fp4(q, s, row, form):
    k, block = q.shape[1], _BLOCK[form]
    x = (_by_block(q, block) * _scale_values(s, form)[:, :, None]).reshape(q.shape[0], -1)[:, :k]
    return x if row is None else x * row[:, None]


def _unpacked(mat, rows, k, form):
    """The values of a matrix in 4 bits as prepare() has it, in FP32."""
    b = mat["q"][:, :(k + 1) // 2]
    values = torch.tensor(_VALUES, device=_DEV)
    q = values[torch.stack((b & 15, b >> 4), dim=2).reshape(rows, -1)[:, :k].int()]
    return _from_fp4(q, _untiled(mat["s"], rows, -(-k // _BLOCK[form])), mat["row"], form)


def _added(s):
    """h in the rows' type."""
    if s["residual"] is None:
        return s["x"]
    return (s["x"].float() + s["residual"].float()).to(s["x"].dtype)


def _rstd(h):
    return torch.rsqrt(h.square().sum(1) / h.shape[1] + _EPS)


def _plain_norm(s):
    c = s["case"]
    kept = _added(s)
    h, w, r = kept.float(), s["w"].float(), _rstd(kept.float())
    out = {} if s["residual"] is None else {"h": kept}
    if c["way"] == "int8":
        v = h * w
        top = v.abs().amax(dim=1)
        steps = torch.full_like(top, 127.0)
        q = torch.round(v * torch.where(top > 0, steps / top, torch.zeros_like(top))[:, None]).clamp(-127, 127).to(torch.int8)
        return dict(out, q=q, scale=top * r / steps)
    r = r[:, None]
    y = (h * r * w).to(kept.dtype)
    dy = s["dy"].float()
    g = dy * w
    dx = r * (g - h * r * r * ((g * h).sum(1, keepdim=True) / h.shape[1]))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dict(out, y=y, dx=dx.to(kept.dtype), dw=(dy * h * r).sum(0))


def _plain_multiplied(s, a):
    c = s["case"]
    out = a @ _unpacked(s["b"], c["n"], c["k"], c["form"]).t()
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(_TYPES[c["dtype"]])


def _plain_linear(s):
    c, out = s["case"], {}
    if c["norm"]:
        kept = _added(s)
        out["h"] = kept
        q, scale, row = _to_fp4(kept.float() * s["w"].float(), c["form"])
        r = _rstd(kept.float())
        row = r if row is None else row * r
    else:
        q, scale, row = _to_fp4(s["x"].float(), c["form"])
    return dict(out, c=_plain_multiplied(s, _from_fp4(q, scale, row, c["form"])))


def _plain_layer(s):
    # every expert's tokens side by side, the shorter groups filled up, and batched products
    c = s["case"]
    e, j, t, f = c["experts"], c["choices"], c["tokens"], c["hidden"]
    key = s["ids"].reshape(-1)
    key = torch.where((key >= 0) & (key < e), key, torch.full_like(key, e))
    in_order, order = torch.sort(key, stable=True)
    offsets = (in_order[None, :] < torch.arange(e + 1, device=_DEV)[:, None]).sum(1)
    at = offsets[:-1, None] + torch.arange(s["most"], device=_DEV)
    inside = at < offsets[1:, None]
    slot = order[at.clamp(max=t * j - 1)]
    x = s["x"].float()[slot // j]
    h = torch.bmm(x, s["up"].float().transpose(1, 2)) * s["up_scale"][:, None, :]
    h = torch.nn.functional.silu(h[:, :, :f]) * (h[:, :, f:] if c["gated"] else 1)
    y = torch.bmm(h, s["down"].float().transpose(1, 2)) * s["down_scale"][:, None, :]
    y = y * s["weights"].reshape(-1)[slot][:, :, None]
    # what fills the groups up goes to one row past the end
    back = torch.zeros(t * j + 1, c["width"], device=_DEV)
    back[torch.where(inside, slot, torch.full_like(slot, t * j)).reshape(-1)] = y.reshape(-1, c["width"])
    return {"out": back[:-1].reshape(t, j, -1).sum(1).to(s["x"].dtype)}


def run(state):
    if own:
        return _own(state)
    c, op = state["case"], state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "rows":
        return {"y": _from_fp4(*_to_fp4(state["x"].float(), c["form"]), c["form"]).to(state["x"].dtype)}
    if op == "linear":
        return _plain_linear(state)
    if op == "product":
        return {"c": _plain_multiplied(state, _unpacked(state["a"], c["m"], c["k"], c["form"]))}
    return _plain_layer(state)


# ------------------------------------------------------- through the library
def _own(s):
    L, h = _library()
    c, op = s["case"], s["case"]["op"]
    kind = _IDS[c["dtype"]]
    if op == "layer":
        L.sgemm_expert_layer_int8(h, kind, int(c["gated"]), c["tokens"], c["choices"], c["experts"], c["width"], c["hidden"], s["x"], c["width"], s["ids"], s["weights"], s["up"], s["up_scale"], s["down"], s["down_scale"], s["out"], c["width"])
        return {"out": s["out"]}
    m, k = c["m"], c["k"]
    ld = k + c.get("pad", 0)
    if op == "norm":
        out = {} if s["residual"] is None else {"h": s["h"]}
        if c["way"] == "int8":
            L.sgemm_rms_norm_int8(h, kind, m, k, s["x"], ld, s["residual"], ld, s["w"], _EPS, s["h"], k, s["q"], k, s["scale"])
            return dict(out, q=s["q"], scale=s["scale"])
        L.sgemm_rms_norm(h, kind, m, k, s["x"], ld, s["residual"], ld, s["w"], _EPS, s["h"], k, s["y"], k, s["rstd"])
        kept, kept_ld = (s["x"], ld) if s["residual"] is None else (s["h"], k)
        L.sgemm_rms_norm_grad(h, kind, m, k, s["dy"], k, s["dh"], k, kept, kept_ld, s["w"], s["rstd"], s["dx"], k, s["dw"])
        return dict(out, y=s["y"], dx=s["dx"], dw=s["dw"])
    form, a, out = _FORMATS[c["form"]], s["a"], {}
    if op == "linear" and c["norm"]:
        L.sgemm_rms_norm_fp4(h, kind, form, m, k, s["x"], ld, s["residual"], ld, s["w"], _EPS, s["h"], k, a["q"], a["ld"], a["s"], a["row"])
        out = {"h": s["h"]}
    elif op != "product":
        L.sgemm_quantize_fp4(h, kind, form, m, k, s["x"], ld, a["q"], a["ld"], a["s"], a["row"])
    if op == "rows":
        L.sgemm_dequantize_fp4(h, kind, form, m, k, a["q"], a["ld"], a["s"], a["row"], s["y"], k)
        return {"y": s["y"]}
    b = s["b"]
    L.sgemm_run_fp4(h, form, kind, m, c["n"], k, a["q"], a["ld"], a["s"], a["row"], b["q"], b["ld"], b["s"], b["row"], s["bias"], s["c"], c["n"])
    return dict(out, c=s["c"])


# ----------------------------------------------------------- in 64 bits
def _nearest_fp4(x):
    """Magnitudes to the nearest 4-bit value by the borders between them; a tie goes to the even code."""
    grid = torch.tensor(_VALUES[:8], dtype=torch.float64, device=_DEV)
    borders = (grid[1:] + grid[:-1]) / 2
    a = x.abs()
    below, above = torch.bucketize(a, borders, right=False), torch.bucketize(a, borders, right=True)
    index = torch.where(below % 2 == 0, below, above)
    return torch.where(x < 0, -grid[index], grid[index])


def _stands_for(x, form):
    """What FP32 rows stand for after the way through 4 bits, without the norm's factor, in 64 bits.
    (Format "nv" is defined with the quotients and products that choose a code rounded to FP32.)"""
    rows, k = x.shape
    n = _BLOCK[form]
    full = torch.zeros(rows, -(-k // n) * n, dtype=torch.float32, device=_DEV)
    full[:, :k] = x
    full = full.view(rows, -1, n)
    largest = full.abs().max(dim=2, keepdim=True).values
    if form == "mx":
        _, e = torch.frexp(largest)                    # largest = f * 2^e with f in [0.5, 1)
        size = torch.where(largest > 0, torch.exp2((e - 3).double().clamp(min=-127)), 1.0)
        q = _nearest_fp4(full.double() / size)
    else:
        row = largest.max(dim=1, keepdim=True).values
        inverse = lambda top: torch.where(row > 0, torch.tensor(top, dtype=torch.float32, device=_DEV) / row, 0.0)  # noqa: E731
        code = (largest * inverse(448.0)).to(torch.float8_e4m3fn).float()
        q = _nearest_fp4(full * torch.where(code > 0, inverse(2688.0) / code, 0.0))
        size = code.double() * (row.double() / 2688)
    return (q * size).view(rows, -1)[:, :k]


def _opened(mat, rows, k, form):
    """A matrix in 4 bits as prepare() has it, byte by byte, in 64 bits."""
    n, b = _BLOCK[form], mat["q"].long()
    p, i = torch.arange(k, device=_DEV), torch.arange(rows, device=_DEV)[:, None]
    code = (b[:, p // 2] >> (4 * (p % 2))) & 15
    exponent, fraction = (code >> 1) & 3, (code & 1).double()
    value = torch.where(exponent == 0, fraction / 2, (1 + fraction / 2) * torch.exp2(exponent.double() - 1))
    value = torch.where(code >= 8, -value, value)
    words = -(-(-(-k // n)) // 4)
    block = torch.arange(-(-k // n), device=_DEV)
    byte = mat["s"][((i // 128 * words + block // 4) * 32 + i % 32) * 16 + i // 32 % 4 * 4 + block % 4].long()
    if form == "mx":
        size = torch.exp2(byte.double() - 127)
    else:
        e, f = byte >> 3 & 15, (byte & 7).double() / 8
        size = torch.where(e == 0, f * 2.0 ** -6, (1 + f) * torch.exp2(e.double() - 7))
    value *= size[:, p // n]
    return value if mat["row"] is None else value * mat["row"].double()[:, None]


def exact(case, seed):
    """The outputs in 64 bits; None where they are whole numbers."""
    c, s = case, prepare(case, seed)
    if c["op"] == "layer":
        e, j, f, x = c["experts"], c["choices"], c["hidden"], s["x"].double()
        out = torch.zeros(c["tokens"], c["width"], dtype=torch.float64, device=_DEV)
        for i in range(e):
            token, choice = (s["ids"] == i).nonzero(as_tuple=True)
            if token.numel():
                h = (x[token] @ s["up"][i].double().T) * s["up_scale"][i].double()
                act = h[:, :f] / (1 + torch.exp(-h[:, :f]))
                y = ((act * h[:, f:] if c["gated"] else act) @ s["down"][i].double().T) * s["down_scale"][i].double()
                out.index_add_(0, token, y * s["weights"].double()[token, choice][:, None])
        return {"out": out}
    out = {}
    if c["op"] == "norm" or c.get("norm"):
        # the residual's sum is part of the result in the rows' own type
        kept = s["x"] if s["residual"] is None else (s["x"].double() + s["residual"].double()).to(s["x"].dtype)
        h, w = kept.double(), s["w"].double()
        if s["residual"] is not None:
            out["h"] = s["x"].double() + s["residual"].double()
        r = 1 / ((h * h).mean(dim=1, keepdim=True) + _EPS).sqrt()
        if c["op"] == "norm" and c["way"] == "int8":
            return dict(out, q=None, scale=((h * w).abs().max(dim=1, keepdim=True).values * r / 127).squeeze(1))
        if c["op"] == "norm":
            n, dy = h * r, s["dy"].double()
            g = dy * w
            dx = (g - n * (g * n).mean(dim=1, keepdim=True)) * r
            return dict(out, y=n * w, dx=dx if s["dh"] is None else dx + s["dh"].double(), dw=(dy * n).sum(dim=0))
        a = _stands_for(kept.float() * s["w"].float(), c["form"]) * r
    elif c["op"] == "product":
        a = _opened(s["a"], c["m"], c["k"], c["form"])
    else:
        a = _stands_for(s["x"].float(), c["form"])
        if c["op"] == "rows":
            return {"y": a}
    full = a @ _opened(s["b"], c["n"], c["k"], c["form"]).T
    return dict(out, c=full if s["bias"] is None else full + s["bias"].double())
