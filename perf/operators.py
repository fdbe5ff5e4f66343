"""The 8-bit operators in their plain form, and the calls a user makes of them.

Four operators on 8-bit floating point with one scale per block of 128:

  quantize    X -> codes (e4m3 or e5m2) and fp32 scales, one per row and 128 columns
              ("rows": activations, gradients) or one per 128 x 128 tile ("tiles": weights);
              with restore, codes and scales -> X in bf16
  matmul      C = A B^T or C = A B of two such matrices (A by rows, B by tiles)
  checkpoint  the backward pass of the NF4 linear layer whose input was kept in 8 bits
  linear      the linear layer over an 8-bit base weight with a LoRA branch: forward (which keeps
              its input in 8 bits) and backward

The definitions, shared by the plain form, the kernels and exact():

  scale  s = max(fp32(absmax / F), 2^-126), F = 448 (e4m3) or 57344 (e5m2); with pow2 the smallest
         power of two p >= 2^-126 with absmax <= F p
  code   c = round_to_8_bits(fp32(x * fp32(1 / s))), to nearest, ties to even
  value  c * s;  restored activations are bf16(c * s)
  NF4    the compute weight is bf16(fp32(level * block scale))
"""

import math

import torch

own = False

DEV = "cuda"
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
FTYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TINY = 2.0 ** -126


def listed():
    return [
        # the 8 bits that a decoding step of 16 sequences feeds its first linear
        dict(name="quantize_decode", op="quantize", rows=16, cols=4096, by="rows", fmt="e4m3",
             pow2=False, dtype="bf16"),
        # the input of the 7B down projection, 8 sequences of 1024 tokens, kept for the backward
        dict(name="quantize_activations", op="quantize", rows=8192, cols=11008, by="rows",
             fmt="e4m3", pow2=False, dtype="bf16"),
        # a merged 7B gate projection going into 8 bits for serving
        dict(name="quantize_weight", op="quantize", rows=11008, cols=4096, by="tiles", fmt="e4m3",
             pow2=True, dtype="bf16"),
        # a kept activation restored for a consumer that wants bf16
        dict(name="restore_activations", op="restore", rows=8192, cols=4096, by="rows", fmt="e4m3",
             pow2=False),
        # one decoding token through the 7B gate projection
        dict(name="matmul_decode", op="matmul", m=1, n=11008, k=4096, trans=True, fa="e4m3",
             fb="e4m3", pow2=False, out="bf16"),
        # 4096 tokens through a 7B attention projection
        dict(name="matmul_attn", op="matmul", m=4096, n=4096, k=4096, trans=True, fa="e4m3",
             fb="e4m3", pow2=False, out="bf16"),
        # the input gradient of the 65B gate projection, 2048 tokens, gradients in e5m2
        dict(name="matmul_dx_65b", op="matmul", m=2048, n=8192, k=22016, trans=False, fa="e5m2",
             fb="e4m3", pow2=False, out="bf16"),
        # a ragged batch through a small odd layer, fp32 out
        dict(name="matmul_ragged", op="matmul", m=333, n=1001, k=1111, trans=True, fa="e4m3",
             fb="e4m3", pow2=False, out="f32"),
        # backward of the 7B attention projection, rank 16, input kept in 8 bits
        dict(name="checkpoint_attn", op="checkpoint", m=4096, n=4096, k=4096, r=16, fmt="e4m3",
             pow2=False),
        # the same for a short batch through the 7B down projection, rank 64
        dict(name="checkpoint_short", op="checkpoint", m=16, n=4096, k=11008, r=64, fmt="e4m3",
             pow2=True),
        # one training step of a 65B attention projection over an 8-bit base, rank 64
        dict(name="linear_step_65b", op="linear", m=2048, n=8192, k=8192, r=64, train=True,
             fmt="e4m3", grad="e5m2", pow2=False),
        # 8 decoding sequences through a 7B projection over an 8-bit base
        dict(name="linear_decode", op="linear", m=8, n=4096, k=4096, r=16, train=False,
             fmt="e4m3", grad="e4m3", pow2=False),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return min(hi // step * step, max(step, int(round(v / step)) * step))

    fmt, pow2 = rng.choice(["e4m3", "e4m3", "e5m2"]), rng.random() < 0.4
    op = rng.choice(["quantize", "restore", "matmul", "matmul", "checkpoint", "linear"])
    if op in ("quantize", "restore"):
        case = dict(op=op, rows=size(1, 11008), cols=size(1, 11008), fmt=fmt, pow2=pow2,
                    by=rng.choice(["rows", "rows", "tiles"]))
        if op == "quantize":
            case["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        return case
    if op == "matmul":
        return dict(op=op, m=size(1, 4096), n=size(16, 11008), k=size(16, 11008),
                    trans=rng.random() < 0.6, fa=fmt, fb="e4m3", pow2=pow2,
                    out=rng.choice(["bf16", "bf16", "f32"]))
    r = rng.choice([8, 16, 32, 64])
    if op == "checkpoint":
        return dict(op=op, m=size(1, 4096), n=size(64, 8192, 8), k=size(64, 8192, 64), r=r,
                    fmt=fmt, pow2=pow2)
    return dict(op=op, m=size(1, 4096), n=size(64, 8192, 8), k=size(64, 8192, 8), r=r,
                train=rng.random() < 0.6, fmt="e4m3", grad=fmt, pow2=pow2)


# ------------------------------------------------------------------ plain forms

def _up(a, b):
    return -(-a // b)


def _blocks(x, by):
    """x (2-D) padded with zeros to whole blocks, as rows x kb x 128 or rb x 128 x kb x 128."""
    rows, cols = x.shape
    kb = _up(cols, 128)
    if by == "rows":
        y = x.new_zeros(rows, kb * 128)
        y[:, :cols] = x
        return y.view(rows, kb, 128)
    rb = _up(rows, 128)
    y = x.new_zeros(rb * 128, kb * 128)
    y[:rows, :cols] = x
    return y.view(rb, 128, kb, 128)


def _quantize(x, by, fmt, pow2):
    """codes (fp8, rows x cols) and scales (rows: kb x rows, tiles: rb x kb) of x."""
    rows, cols = x.shape
    b = _blocks(x.float(), by)
    amax = b.abs().amax(dim=2 if by == "rows" else (1, 3))
    if pow2:
        m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); F = 0.875 2^9 or 0.875 2^16
        e = e - (9 if fmt == "e4m3" else 16) + (m > 0.875).to(e.dtype)
        e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp_min(-126)
        s = torch.ldexp(torch.ones_like(amax), e)
    else:
        # divided by a tensor: a division by a Python number is a product with its reciprocal
        s = (amax / torch.full_like(amax, FMAX[fmt])).clamp_min(TINY)
    inv = torch.ones_like(s) / s
    inv = inv[:, :, None] if by == "rows" else inv[:, None, :, None]
    c = (b * inv).clamp(-FMAX[fmt], FMAX[fmt]).to(FTYPE[fmt])
    c = c.view(-1, _up(cols, 128) * 128)[:rows, :cols].contiguous()
    return c, (s.t().contiguous() if by == "rows" else s)


def _restore(codes, scales, by, dtype=torch.float32):
    """codes * scales, in dtype (fp32 or fp64)."""
    rows, cols = codes.shape
    if by == "rows":
        s = scales.t().to(dtype).repeat_interleave(128, dim=1)[:, :cols]
    else:
        s = scales.to(dtype).repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return codes.to(dtype) * s


def _nf4_levels():
    """7 levels below zero, an exact 0, 8 above: medians of equal parts of each half of N(0, 1)."""
    p = torch.tensor([0.5 + (j - 0.5) / 16 for j in range(1, 9)], dtype=torch.float64)
    n = torch.tensor([0.5 - (j - 0.5) / 14 for j in range(7, 0, -1)], dtype=torch.float64)
    p, n = torch.special.ndtri(p), torch.special.ndtri(n)
    z = torch.zeros(1, dtype=torch.float64)
    return torch.cat([n / -n[0], z, p / p[-1]]).float().to(DEV)


def _nf4_store(w):
    """A stored NF4 weight (blocks of 64, scales in int8 by groups of 256) as a dict of arrays."""
    n, k = w.shape
    b = w.float().view(-1, 64)
    s = b.abs().amax(1)
    lv = _nf4_levels()
    idx = torch.bucketize(b / s.clamp_min(TINY)[:, None], (lv[1:] + lv[:-1]) / 2).to(torch.uint8)
    idx = idx.view(-1, 2)
    mean = s.double().mean().float().view(1)
    g = torch.zeros(_up(s.numel(), 256) * 256, device=DEV)
    g[:s.numel()] = s - mean
    g = g.view(-1, 256)
    f = g.abs().amax(1) / 127
    sc = torch.round(g / f.clamp_min(TINY)[:, None]).clamp(-127, 127).to(torch.int8).view(-1)
    return dict(rows=n, cols=k, codes=(idx[:, 0] | (idx[:, 1] << 4)).contiguous(),
                scale_codes=sc[:s.numel()].contiguous(), factors=f.contiguous(), mean=mean)


def _nf4_weight(q):
    """The bf16 compute weight of a stored NF4 weight, as fp32."""
    idx = torch.stack([q["codes"] & 15, q["codes"] >> 4], 1).view(-1, 64).long()
    f = q["factors"].repeat_interleave(256)[:q["scale_codes"].numel()]
    s = q["scale_codes"].float() * f + q["mean"]
    w = _nf4_levels()[idx] * s[:, None]
    return w.view(q["rows"], q["cols"]).bfloat16().float()


def _lora_grads(dy, u, v, x, s):
    return s * (v.t() @ x), s * (dy.t() @ u)


def _plain(st):
    c = st["case"]
    if c["op"] == "quantize":
        codes, scales = _quantize(st["x"], c["by"], c["fmt"], c["pow2"])
        return {"codes": codes, "scales": scales}
    if c["op"] == "restore":
        return {"x": _restore(st["codes"], st["scales"], c["by"]).bfloat16()}
    if c["op"] == "matmul":
        a, b = _restore(st["ac"], st["as"], "rows"), _restore(st["bc"], st["bs"], "tiles")
        y = a @ (b.t() if c["trans"] else b)
        return {"c": y if c["out"] == "f32" else y.bfloat16()}
    s = st["alpha"] / c["r"]
    a, b = st["a"].float(), st["b"].float()
    if c["op"] == "checkpoint":
        dy = st["dy"].float()
        x = _restore(st["xc"], st["xs"], "rows").bfloat16().float()
        v = dy @ b
        da, db = _lora_grads(dy, st["u"], v, x, s)
        return {"dx": (dy @ _nf4_weight(st["w"]) + s * (v @ a)).bfloat16(), "da": da, "db": db}
    x = st["x"].float()
    xc, xs = _quantize(x, "rows", c["fmt"], c["pow2"])
    w = _restore(st["wc"], st["ws"], "tiles")
    u = x @ a.t()
    xq = _restore(xc, xs, "rows")
    out = {"y": (xq @ w.t() + s * (u @ b.t())).bfloat16(), "u": u}
    if not c["train"]:
        return out
    dy = st["dy"].float()
    dq = _restore(*_quantize(dy, "rows", c["grad"], c["pow2"]), "rows")
    v = dy @ b
    out["da"], out["db"] = _lora_grads(dy, u, v, xq.bfloat16().float(), s)
    out["dx"] = (dq @ w + s * (v @ a)).bfloat16()
    return out


# ------------------------------------------------------------------ inputs

def _heavy(shape, g, std, dtype=torch.float32):
    """Normal values, a few of them far out, as activations and weights have."""
    x = torch.randn(shape, generator=g, device=DEV) * std
    far = torch.rand(shape, generator=g, device=DEV) < 1e-3
    return torch.where(far, x * 8, x).to(dtype)


def _padded(codes):
    """The bytes of codes in rows padded to a multiple of 16, as the library keeps them."""
    rows, cols = codes.shape
    ld = _up(cols, 16) * 16
    p = torch.zeros(rows, ld, dtype=torch.uint8, device=DEV)
    p[:, :cols] = codes.view(torch.uint8)
    return p


def _kept(x, by, fmt, pow2):
    """What a program has of a matrix that is held in 8 bits: codes and scales, and the handle."""
    codes, scales = _quantize(x, by, fmt, pow2)
    p = _padded(codes)
    view = p.view(FTYPE[fmt])[:, :codes.shape[1]]
    if own:
        return view, scales, _matrix(codes.shape, p, scales, by, fmt, pow2)
    return view, scales, None


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    st = dict(case=case)
    op = case["op"]
    if op in ("quantize", "restore"):
        # rows of very different sizes: activations of a residual stream
        x = _heavy((case["rows"], case["cols"]), g, 0.02 if case["by"] == "tiles" else 1.0)
        if case["by"] == "rows":
            x *= torch.exp2(torch.randint(-6, 7, (case["rows"], 1), generator=g, device=DEV).float())
        if op == "quantize":
            st["x"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        else:
            st["codes"], st["scales"], st["h"] = _kept(x, case["by"], case["fmt"], case["pow2"])
        return st
    m, n, k = case["m"], case["n"], case["k"]
    if op == "matmul":
        a = _heavy((m, k), g, 1.0)
        b = _heavy((n, k) if case["trans"] else (k, n), g, 0.02)
        st["ac"], st["as"], st["ah"] = _kept(a, "rows", case["fa"], case["pow2"])
        st["bc"], st["bs"], st["bh"] = _kept(b, "tiles", case["fb"], case["pow2"])
        return st
    r = case["r"]
    bf = torch.bfloat16
    st["alpha"] = 2.0 * r if r <= 16 else 16.0
    st["a"] = (torch.randn(r, k, generator=g, device=DEV) / math.sqrt(r)).to(bf)
    st["b"] = (torch.randn(n, r, generator=g, device=DEV) * 0.01).to(bf)
    w = _heavy((n, k), g, 0.02)
    x = _heavy((m, k), g, 1.0, bf)
    if op == "checkpoint":
        st["w"] = _nf4_store(w)
        st["u"] = x.float() @ st["a"].float().t()
        st["xc"], st["xs"], st["xh"] = _kept(x, "rows", case["fmt"], case["pow2"])
        st["dy"] = torch.randn(m, n, generator=g, device=DEV).to(bf)
    else:
        st["wc"], st["ws"], st["wh"] = _kept(w, "tiles", "e4m3", case["pow2"])
        st["x"] = x
        if case["train"]:
            st["dy"] = torch.randn(m, n, generator=g, device=DEV).to(bf)
    if own:
        _keep_workspaces(st)
    return st


# ------------------------------------------------------------------ the framework's calls

def _matrix(shape, codes, scales, by, fmt, pow2):
    from bit_nf4_quantized_17_b200 import qlora as Q
    return Q.F8Matrix(shape[0], shape[1], Q.QLORA_F8_ROWS if by == "rows" else Q.QLORA_F8_TILES,
                      Q.QLORA_E4M3 if fmt == "e4m3" else Q.QLORA_E5M2, pow2, codes, scales)


def _keep_workspaces(st):
    """The workspaces and the NF4 handle that a training or serving program keeps."""
    from bit_nf4_quantized_17_b200 import qlora as Q
    c = st["case"]
    m, n, k, r = c["m"], c["n"], c["k"], c["r"]
    if c["op"] == "checkpoint":
        w = st["w"]
        st["q"] = Q.QuantizedWeight(n, k, 64, 256, Q.QLORA_TABLE_NF4, w["codes"],
                                    w["scale_codes"], w["factors"], w["mean"])
        sizes = (0, Q.qlora_linear_bwd_f8_workspace(m, n, k, r))
    else:
        sizes = Q.qlora_f8_linear_workspace(m, n, k, r)
    st["ws_f"], st["ws_b"] = (torch.zeros(max(b, 256), dtype=torch.uint8, device=DEV)
                              for b in sizes)


def _own(st):
    from bit_nf4_quantized_17_b200 import qlora as Q
    c = st["case"]
    fmt = {"e4m3": Q.QLORA_E4M3, "e5m2": Q.QLORA_E5M2}
    if c["op"] == "quantize":
        q = Q.qlora_f8_quantize(st["x"], Q.QLORA_F8_ROWS if c["by"] == "rows" else Q.QLORA_F8_TILES,
                                fmt[c["fmt"]], c["pow2"])
        return {"codes": q.values, "scales": q.scales}
    if c["op"] == "restore":
        return {"x": Q.qlora_f8_dequantize(st["h"], torch.bfloat16)}
    if c["op"] == "matmul":
        return {"c": Q.qlora_f8_matmul(st["ah"], st["bh"], c["trans"],
                                       torch.float32 if c["out"] == "f32" else torch.bfloat16)}
    if c["op"] == "checkpoint":
        dx, da, db = Q.qlora_linear_bwd_f8(st["q"], st["a"], st["b"], c["r"], st["alpha"], st["xh"],
                                           st["u"], st["dy"], workspace=st["ws_b"])
        return {"dx": dx, "da": da, "db": db}
    u = torch.empty(c["m"], c["r"], dtype=torch.float32, device=DEV)
    x8 = Q.F8Matrix.empty(c["m"], c["k"], Q.QLORA_F8_ROWS, fmt[c["fmt"]], c["pow2"], DEV)
    y = Q.qlora_f8_linear_fwd(st["wh"], st["a"], st["b"], st["alpha"], st["x"], x8, U_save=u,
                              workspace=st["ws_f"])
    if not c["train"]:
        return {"y": y, "u": u}
    dx, da, db = Q.qlora_f8_linear_bwd(st["wh"], st["a"], st["b"], st["alpha"], x8, u, st["dy"],
                                       fmt[c["grad"]], workspace=st["ws_b"])
    return {"y": y, "u": u, "dx": dx, "da": da, "db": db}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    scales = lambda r, c, by: 4 * (r if by == "rows" else _up(r, 128)) * _up(c, 128)  # noqa: E731
    if op in ("quantize", "restore"):
        n = case["rows"] * case["cols"]
        wide = 4 if case.get("dtype") == "f32" else 2
        return {"bytes": n * (wide + 1) + scales(case["rows"], case["cols"], case["by"]),
                "flops": 2 * n}
    m, n, k = case["m"], case["n"], case["k"]
    a8 = m * k + scales(m, k, "rows")
    if op == "matmul":
        return {"bytes": a8 + n * k + scales(n, k, "tiles")
                + m * n * (4 if case["out"] == "f32" else 2), "flops": 2 * m * n * k}
    r = case["r"]
    lora = 2 * r * (n + k)
    if op == "checkpoint":
        w = n * k // 2 + n * k // 64 + 4 * _up(n * k, 64 * 256)
        return {"bytes": w + a8 + lora + 4 * m * r + 2 * m * n + 2 * m * k + 4 * r * (n + k),
                "flops": 2 * m * n * k + 2 * m * r * (2 * n + 2 * k)}
    w = n * k + scales(n, k, "tiles")
    b = w + lora + 2 * m * k + a8 + 2 * m * n + 4 * m * r
    f = 2 * m * n * k + 2 * m * r * (n + k)
    if case["train"]:
        b += w + lora + a8 + 4 * m * r + 2 * m * n + 2 * m * k + 4 * r * (n + k)
        f += 2 * m * n * k + 2 * m * r * (2 * n + 2 * k)
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ the definitions in 64 bits

def _f32(x):
    return x.float().double()


def _exact_codes(x, by, fmt, pow2):
    """Codes as fp64 values and scales in fp64, block by block from the definition."""
    rows, cols = x.shape
    x = x.double()
    kb = _up(cols, 128)
    pad = torch.nn.functional.pad(x.abs(), (0, kb * 128 - cols, 0, (-rows) % 128))
    amax = pad.view(pad.shape[0], kb, 128).amax(2)
    if by == "tiles":
        amax = amax.view(-1, 128, kb).amax(1)
    else:
        amax = amax[:rows]
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2((amax / FMAX[fmt]).clamp_min(TINY))))
        s = torch.where(amax > s * FMAX[fmt], s * 2, s)
        s = torch.where((s > TINY) & (amax <= s / 2 * FMAX[fmt]), s / 2, s)
    else:
        s = _f32(amax / FMAX[fmt]).clamp_min(TINY)
    full = s.repeat_interleave(128, 1)[:, :cols]
    if by == "tiles":
        full = full.repeat_interleave(128, 0)[:rows]
    q = _f32(x * _f32(1.0 / full))
    # round to the format: steps of 2^(e - mantissa bits), e not below the smallest normal's
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    e = (torch.frexp(q)[1] - 1).clamp_min(low).double()
    step = torch.exp2(e - bits)
    c = (torch.round(q / step) * step).clamp(-FMAX[fmt], FMAX[fmt])
    return c, s, c * full


def _exact_restore(codes, scales, by):
    rows, cols = codes.shape
    c = codes.float().double()
    j = torch.arange(cols, device=DEV) // 128
    if by == "rows":
        return c * scales.double()[j].t()
    return c * scales.double()[torch.arange(rows, device=DEV) // 128][:, j]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        c, s, _ = _exact_codes(st["x"], case["by"], case["fmt"], case["pow2"])
        return {"codes": c, "scales": s.t().contiguous() if case["by"] == "rows" else s}
    if op == "restore":
        return {"x": _exact_restore(st["codes"], st["scales"], case["by"])}
    if op == "matmul":
        a = _exact_restore(st["ac"], st["as"], "rows")
        b = _exact_restore(st["bc"], st["bs"], "tiles")
        return {"c": torch.matmul(a, b.t() if case["trans"] else b)}
    s = st["alpha"] / case["r"]
    a, b = st["a"].double(), st["b"].double()
    if op == "checkpoint":
        dy, u = st["dy"].double(), st["u"].double()
        x = _exact_restore(st["xc"], st["xs"], "rows").bfloat16().double()
        q = st["w"]
        pos = torch.arange(q["rows"] * q["cols"], device=DEV)
        idx = (q["codes"][pos // 2] >> (4 * (pos % 2)).to(torch.uint8)) & 15
        blk = torch.arange(q["scale_codes"].numel(), device=DEV)
        sc = _f32(_f32(q["scale_codes"].double() * q["factors"].double()[blk // 256])
                  + q["mean"].double())
        w = _f32(_nf4_levels().double()[idx.long()] * sc[pos // 64]).bfloat16().double()
        w = w.view(q["rows"], q["cols"])
        v = dy @ b
        return {"dx": dy @ w + s * (v @ a), "da": s * (v.t() @ x), "db": s * (dy.t() @ u)}
    x = st["x"].double()
    w = _exact_restore(st["wc"], st["ws"], "tiles")
    xq = _exact_codes(st["x"], "rows", case["fmt"], case["pow2"])[2]
    u = x @ a.t()
    out = {"y": xq @ w.t() + s * (u @ b.t()), "u": u}
    if case["train"]:
        dy = st["dy"].double()
        dq = _exact_codes(st["dy"], "rows", case["grad"], case["pow2"])[2]
        v = dy @ b
        out["dx"] = dq @ w + s * (v @ a)
        out["da"] = s * (v.t() @ xq.bfloat16().double())
        out["db"] = s * (dy.t() @ u)
    return out
