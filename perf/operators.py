"""Measured cases of the 8-bit block operators and of the residual-binary layer's gradients.

Five operators share one storage format, e4m3 codes with one fp32 scale for
each block of 128 columns of a row (activations) or of 128 x 128 (weights):

  pack8    x -> codes, scales             (activation checkpoints, weights)
  unpack8  codes, scales -> x
  gemm8    y = W x from packed W and x    (decode and prefill)
  wgrad    dW = add + dY^T x, x packed    (backward pass from a checkpoint)
  dgrad    dX = dY W^, W^ = sum_k alpha_k B_k from the sign planes

``run`` computes them in elementary torch operations in fp32, or, where
``own`` is true, through the framework's entry points.
"""
import math

import torch

own = False

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
DTYPES = {"f16": F16, "bf16": BF16, "f32": F32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn
# the exponent at which a scale of 2^n lets 256 * 2^n overflow the input type
TOP = {"f16": 8, "bf16": 120, "f32": 120}


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one token's hidden state before an 8-bit projection: latency
        {"name": "pack8_token", "op": "pack8", "rows": 1, "K": 4096, "block_rows": 1, "dtype": "f16"},
        # the checkpoint of a prefill-sized block's wide activations
        {"name": "pack8_block", "op": "pack8", "rows": 2048, "K": 14336, "block_rows": 1, "dtype": "bf16"},
        # packing an 8-bit layer's weight once per optimizer step
        {"name": "pack8_weight", "op": "pack8", "rows": 11008, "K": 4096, "block_rows": 128, "dtype": "f32"},
        # a ragged micro-batch's checkpoint restored for a recomputation
        {"name": "unpack8_ragged", "op": "unpack8", "rows": 333, "K": 4096, "block_rows": 1, "dtype": "f16"},
        # the wide activations of a training block restored
        {"name": "unpack8_block", "op": "unpack8", "rows": 8192, "K": 11008, "block_rows": 1, "dtype": "bf16"},
        # decode, one token through a 7B attention projection kept in 8 bits
        {"name": "gemm8_token", "op": "gemm8", "T": 1, "M": 4096, "K": 4096, "dtype": "f16"},
        # decode, a small batch through a 70B up projection
        {"name": "gemm8_batch16", "op": "gemm8", "T": 16, "M": 28672, "K": 8192, "dtype": "bf16"},
        # prefill, 2048 tokens through an 8B up projection
        {"name": "gemm8_prefill", "op": "gemm8", "T": 2048, "M": 14336, "K": 4096, "dtype": "bf16"},
        # the small square layer's weight gradient over a ragged batch
        {"name": "wgrad_layer256", "op": "wgrad", "T": 777, "M": 256, "K": 256, "dtype": "f16", "out": "f32", "add": False},
        # a training step's up projection, added to the fp32 gradient of earlier micro-batches
        {"name": "wgrad_train", "op": "wgrad", "T": 2048, "M": 14336, "K": 4096, "dtype": "bf16", "out": "f32", "add": True},
        # a few tokens back through a 70B attention projection
        {"name": "dgrad_batch16", "op": "dgrad", "T": 16, "M": 8192, "K": 8192, "n_paths": 2, "group": 0,
         "order": "sliced", "alpha": "f32", "dtype": "f16", "out": "f16"},
        # a training step's up projection, two paths with one scale per row
        {"name": "dgrad_train", "op": "dgrad", "T": 2048, "M": 14336, "K": 4096, "n_paths": 2, "group": 0,
         "order": "sliced", "alpha": "f32", "dtype": "bf16", "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log_k(rng, lo, hi):
    return 128 * _log_int(rng, lo // 128, hi // 128)


def draw(rng):
    # no drawn case does more work than the largest listed one of its operator
    op = rng.choice(["pack8", "unpack8", "gemm8", "wgrad", "dgrad"])
    dtype = rng.choice(["f16", "bf16"])
    if op in ("pack8", "unpack8"):
        most = 90_000_000 if op == "unpack8" else 45_000_000
        K = _log_k(rng, 128, 28672)
        rows = _log_int(rng, 1, min(65536, max(2, most // K)))
        if rng.random() < 0.25:
            dtype = "f32"
        return {"op": op, "rows": rows, "K": K, "block_rows": rng.choice([1, 1, 128]), "dtype": dtype}
    most = 2048 * 14336 * 4096
    M, K = _log_int(rng, 64, 28672), _log_k(rng, 128, 16384)
    T = _log_int(rng, 1, min(16384, max(2, most // (M * K))))
    if op == "gemm8":
        return {"op": op, "T": T, "M": M, "K": K, "dtype": rng.choice(["f16", "bf16", "f32"])}
    out = rng.choice(["f32", dtype])
    if op == "wgrad":
        return {"op": op, "T": T, "M": M, "K": K, "dtype": dtype, "out": out, "add": rng.random() < 0.5}
    n_paths, group = rng.choice([1, 2, 2, 3, 4]), rng.choice([0, 0, 128])
    return {"op": op, "T": T, "M": M, "K": K, "n_paths": n_paths, "group": group, "order": rng.choice(["rows", "sliced"]),
            "alpha": "f16" if group else rng.choice(["f32", "f16"]), "dtype": dtype, "out": dtype}


# ------------------------------------------------------- elementary operations
def _blocks(x, block_rows):
    """[rows, K] -> [row blocks, block_rows, K / 128, 128], the last row block filled with zeros."""
    rows, K = x.shape
    pad = -rows % block_rows
    if pad:
        x = torch.cat([x, x.new_zeros((pad, K))])
    return x.view(-1, block_rows, K // 128, 128)


def _pack8(x, block_rows, dtype):
    rows, K = x.shape
    b = _blocks(x.float(), block_rows)
    finite = torch.isfinite(b)
    top = torch.where(finite, b.abs(), torch.zeros_like(b)).amax(dim=(1, 3))
    m, e = torch.frexp(top)                       # top = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    n = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    n = torch.where(top == 0, torch.zeros_like(n), n)
    scale = ((n + 127).to(torch.int32) << 23).view(F32)
    cap = torch.where(n >= TOP[dtype], 240.0, 448.0)[:, None, :, None]
    c = torch.minimum(torch.maximum(b / scale[:, None, :, None], -cap), cap)
    c = torch.where(finite, c, torch.full_like(c, math.nan))
    return c.view(-1, K)[:rows].to(E4M3), scale


def _unpack8(codes, scales, block_rows):
    rows, K = codes.shape
    b = _blocks(codes.float(), block_rows)
    return (b * scales[:, None, :, None]).view(-1, K)[:rows]


def _planes_rows(planes, K):
    """Row-major words [N, M, K/32] of planes in either order."""
    if planes.dim() == 4:
        N, S, M, w = planes.shape
        planes = planes.permute(0, 2, 1, 3).reshape(N, M, S * w)[:, :, :K // 32]
    return planes


def _weight(planes, alpha, K, dt):
    """W^ = sum_k alpha_k (.) B_k of type dt."""
    words = _planes_rows(planes, K)
    N, M, W = words.shape
    bits = (words[..., None] >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1
    G = alpha.shape[2]
    signs = (2 * bits - 1).view(N, M, G, K // G).to(dt)
    return (signs * alpha.to(dt)[..., None]).sum(0).view(M, K)


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, T, K, dt):
    """N(0, 1) with 0.5 % of the channels 20 times larger, as the linears of a transformer see them."""
    x = torch.randn((T, K), generator=g, device="cuda")
    n = max(1, K // 200)
    ch = torch.randperm(K, generator=g, device="cuda")[:n]
    x[:, ch] *= 20
    return x.to(dt)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op in ("pack8", "unpack8"):
        rows, K, dt = case["rows"], case["K"], DTYPES[case["dtype"]]
        if case["block_rows"] == 1:
            x = _activations(g, rows, K, dt)
        else:
            x = (torch.randn((rows, K), generator=g, device="cuda") * 0.02).to(dt)
        if op == "pack8":
            s["x"] = x
        else:
            s["codes"], s["scales"] = _pack8(x, case["block_rows"], case["dtype"])
        return s
    T, M, K = case["T"], case["M"], case["K"]
    if op == "gemm8":
        s["w"], s["ws"] = _pack8(torch.randn((M, K), generator=g, device="cuda") * 0.02, 128, "f32")
        s["x"], s["xs"] = _pack8(_activations(g, T, K, BF16), 1, "bf16")
        return s
    # output gradients: row pitch a multiple of 8 values, as the layer's own buffers have
    pitch = -(-M // 8) * 8
    dy = torch.randn((T, pitch), generator=g, device="cuda") * 0.01
    s["dy"] = dy.to(DTYPES[case["dtype"]])[:, :M]
    if op == "wgrad":
        s["x"], s["xs"] = _pack8(_activations(g, T, K, DTYPES[case["dtype"]]), 1, case["dtype"])
        s["add"] = (torch.randn((M, K), generator=g, device="cuda") * 0.1).to(DTYPES[case["out"]]) if case["add"] else None
        return s
    N, G = case["n_paths"], K // 128 if case["group"] else 1
    shape = (N, M, K // 32) if case["order"] == "rows" else (N, -(-K // 512), M, 16)
    s["planes"] = torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    # mean |R_k| of Gaussian rows of std 0.02, about 0.6 times smaller with each path
    base = 0.016 * 0.6 ** torch.arange(N, device="cuda", dtype=F32).view(N, 1, 1)
    s["alpha"] = (base * (0.75 + 0.5 * torch.rand((N, M, G), generator=g, device="cuda"))).to(DTYPES[case["alpha"]])
    return s


# -------------------------------------------------------------------- one pass
def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        import residual_binary_weight_b200 as rb
        if op == "pack8":
            return rb.pack8(state["x"], block_rows=case["block_rows"])
        if op == "unpack8":
            return rb.unpack8(state["codes"], state["scales"], block_rows=case["block_rows"], dtype=DTYPES[case["dtype"]])
        if op == "gemm8":
            return rb.gemm8(state["w"], state["ws"], state["x"], state["xs"], y_dtype=DTYPES[case["dtype"]])
        if op == "wgrad":
            return rb.gemm_wgrad(state["dy"], state["x"], state["xs"], add=state["add"], dw_dtype=DTYPES[case["out"]])
        return rb.gemm_dgrad(state["planes"], state["alpha"], state["dy"], case["K"], group=case["group"],
                             dx_dtype=DTYPES[case["out"]])
    if op == "pack8":
        return _pack8(state["x"], case["block_rows"], case["dtype"])
    if op == "unpack8":
        return _unpack8(state["codes"], state["scales"], case["block_rows"]).to(DTYPES[case["dtype"]])
    if op == "gemm8":
        w, x = _unpack8(state["w"], state["ws"], 128), _unpack8(state["x"], state["xs"], 1)
        return (x @ w.t()).to(DTYPES[case["dtype"]])
    if op == "wgrad":
        dw = state["dy"].float().t() @ _unpack8(state["x"], state["xs"], 1)
        if state["add"] is not None:
            dw = dw + state["add"].float()
        return dw.to(DTYPES[case["out"]])
    return (state["dy"].float() @ _weight(state["planes"], state["alpha"], case["K"], F32)).to(DTYPES[case["out"]])


def work(case):
    op = case["op"]
    if op in ("pack8", "unpack8"):
        rows, K = case["rows"], case["K"]
        blocks = -(-rows // case["block_rows"]) * (K // 128)
        n = rows * K
        # a maximum, a product and a rounding for each value (unpack8: a product)
        return {"bytes": n * (SIZE[case["dtype"]] + 1) + 4 * blocks, "flops": n * (3 if op == "pack8" else 1)}
    T, M, K = case["T"], case["M"], case["K"]
    flops = 2 * T * M * K
    if op == "gemm8":
        scales = 4 * (K // 128) * (T + -(-M // 128))
        return {"bytes": M * K + T * K + scales + T * M * SIZE[case["dtype"]], "flops": flops}
    if op == "wgrad":
        b = 2 * T * M + T * K + 4 * T * (K // 128) + M * K * SIZE[case["out"]] * (2 if case["add"] else 1)
        return {"bytes": b, "flops": flops}
    N, G = case["n_paths"], K // 128 if case["group"] else 1
    b = 2 * T * M + N * M * K // 8 + N * M * G * SIZE[case["alpha"]] + T * K * SIZE[case["out"]]
    return {"bytes": b, "flops": flops}


# ------------------------------------------------------ the definition, 64 bits
def _round_e4m3(v):
    """Nearest e4m3 value, ties to the even mantissa (|v| at most 448)."""
    mag = v.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(mag)) - 3)
    return torch.round(v / step) * step


def _expand(scales, rows, K, block_rows):
    s = scales.double().repeat_interleave(128, dim=1)
    return s.repeat_interleave(block_rows, dim=0)[:rows, :K]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "pack8":
        x, r = s["x"].double(), case["block_rows"]
        rows, K = x.shape
        full = torch.zeros((-(-rows // r) * r, K), dtype=torch.float64, device=x.device)
        full[:rows] = x.abs()
        top = full.reshape(-1, r, K // 128, 128).permute(0, 2, 1, 3).flatten(2).max(dim=2).values
        n = torch.floor(torch.log2(top.clamp(min=2.0 ** -1000))) - 8      # top in [2^(n+8), 2^(n+9))
        n = torch.where(top > 448 * torch.exp2(n), n + 1, n).clamp(min=-126)
        n = torch.where(top > 0, n, torch.zeros_like(n))
        scale = torch.exp2(n)
        each = _expand(scale, rows, K, r)
        most = torch.where(each >= 2.0 ** TOP[case["dtype"]], 240.0, 448.0)
        return torch.clamp(_round_e4m3(x / each), -most, most), scale
    if op == "unpack8":
        rows, K = s["codes"].shape
        return s["codes"].double() * _expand(s["scales"], rows, K, case["block_rows"])
    T, M, K = case["T"], case["M"], case["K"]
    if op == "gemm8":
        w = s["w"].double() * _expand(s["ws"], M, K, 128)
        return (s["x"].double() * _expand(s["xs"], T, K, 1)).matmul(w.t())
    dy = s["dy"].double()
    if op == "wgrad":
        dw = torch.einsum("tm,tk->mk", dy, s["x"].double() * _expand(s["xs"], T, K, 1))
        return dw if s["add"] is None else dw + s["add"].double()
    words = s["planes"].to(torch.int64) & 0xFFFFFFFF
    if case["order"] == "sliced":
        words = torch.cat(list(words.unbind(1)), dim=2)[:, :, :K // 32]
    w = torch.zeros((M, K), dtype=torch.float64, device=dy.device)
    for k in range(case["n_paths"]):
        a = s["alpha"][k].double().repeat_interleave(K // s["alpha"].shape[2], dim=1)
        for j in range(32):
            plus = (words[k] >> j) & 1
            w[:, j::32] += torch.where(plus == 1, a[:, j::32], -a[:, j::32])
    return dy.matmul(w)
