"""Cases for the block-scaled FP8 operators: the RMS norm that produces the
activations' codes, the quantizers, the product, and the product grouped by
expert.

Codes are E4M3; every block of 128 (of a row of activations, or 128 x 128 of
a weight) has a power-of-two scale in one E8M0 byte, and a row of scales is
padded to a multiple of 4 bytes with 127 (2^0).  The plain forms here state
the operators in elementary torch operations; `exact` states them in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128
_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the norm before a layer of one decoded token: all latency
        dict(name="norm_decode", op="norm", T=1, K=4096, dtype="fp16", residual=True, y=False),
        # the norm before an expert layer of a 4096-token prompt, whose router reads y
        dict(name="norm_prompt", op="norm", T=4096, K=4096, dtype="bf16", residual=True, y=True),
        # the ReLU'd inputs of the second feed-forward layer, a small batch of decoded tokens
        dict(name="qact_decode", op="qact", T=16, K=16384, dtype="fp16"),
        # the same of a 2048-token prompt, a row length that ends in half a block
        dict(name="qact_prompt", op="qact", T=2048, K=8256, dtype="bf16"),
        # a 1.3B model's up-projection, when it is loaded
        dict(name="qweight_layer", op="qweight", E=1, N=8192, K=2048, dtype="fp16"),
        # eight experts' weights, with half blocks at both ends
        dict(name="qweight_experts", op="qweight", E=8, N=4160, K=4160, dtype="bf16"),
        # a 6.7B model's up-projection of one decoded token: the weight is streamed
        dict(name="matmul_decode", op="matmul", T=1, K=4096, N=16384, dtype="fp16", bias=True, relu=False),
        # a short ragged prompt through a 1.3B model's up-projection
        dict(name="matmul_ragged", op="matmul", T=300, K=2048, N=8192, dtype="bf16", bias=True, relu=True),
        # a 4096-token prompt through a 6.7B model's up-projection: all matrix cores
        dict(name="matmul_prompt", op="matmul", T=4096, K=4096, N=16384, dtype="fp16", bias=False, relu=False),
        # 16 decoded tokens, 4 of 64 experts each: a row or two per expert
        dict(name="experts_decode", op="grouped", T=16, top=4, E=64, K=2048, N=1024, dtype="bf16",
             gather=True, bias=False, relu=False),
        # an odd prompt, 2 of 8 experts each, the loads uneven
        dict(name="experts_ragged", op="grouped", T=1111, top=2, E=8, K=4096, N=4096, dtype="fp16",
             gather=True, bias=True, relu=True),
        # a 4096-token prompt, 8 of 64 experts each, rows already in expert order
        dict(name="experts_prompt", op="grouped", T=4096, top=8, E=64, K=2048, N=2048, dtype="bf16",
             gather=False, bias=False, relu=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _by64(rng, lo, hi):
    return 64 * max(1, _log(rng, lo / 64, hi / 64))


def draw(rng):
    op = rng.choice(["norm", "qact", "qweight", "matmul", "matmul", "grouped", "grouped"])
    c = dict(op=op, dtype=rng.choice(["fp16", "bf16"]))
    if op in ("norm", "qact"):
        c["K"] = _by64(rng, 256, 16384)
        c["T"] = _log(rng, 1, max(1, min(8192, (1 << 25) // c["K"])))
        if op == "norm":
            c.update(residual=rng.random() < 0.75, y=rng.random() < 0.5)
    elif op == "qweight":
        c["E"] = rng.choice([1, 1, 4, 16])
        c["K"] = _by64(rng, 256, 16384)
        c["N"] = _by64(rng, 64, min(16384, (1 << 27) // (c["K"] * c["E"])))
    else:
        c.update(bias=rng.random() < 0.5, relu=rng.random() < 0.5)
        if op == "matmul":
            c["K"] = _by64(rng, 256, 16384)
            c["N"] = _by64(rng, 256, 16384)
            c["T"] = _log(rng, 1, max(1, min(4096, (1 << 38) // (c["K"] * c["N"]))))
        else:
            c["E"] = rng.choice([4, 8, 16, 64, 128])
            c["top"] = rng.choice([1, 2, 4])
            c["K"] = _by64(rng, 256, 8192)
            c["N"] = _by64(rng, 256, max(256, min(8192, (1 << 30) // (c["K"] * c["E"]))))
            c["T"] = _log(rng, 1, 4096)
            c["gather"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, T, K, dtype):
    """N(0, 1) with a few feature columns of large magnitude, as hidden states have."""
    x = torch.randn((T, K), generator=g, device="cuda")
    cols = torch.randperm(K, generator=g, device="cuda")[:6]
    x[:, cols] *= 20.0 + 40.0 * torch.rand((6,), generator=g, device="cuda")
    return x.to(dtype)


def _offsets(g, rows, E):
    """Rows per expert of an uneven router, as int32 [E+1] bounds on the GPU."""
    p = torch.softmax(torch.randn((E,), generator=g, device="cuda"), 0)
    pick = torch.multinomial(p, rows, replacement=True, generator=g)
    count = torch.bincount(pick, minlength=E)
    return torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    g, dt, op = _gen(seed), _DT[case["dtype"]], case["op"]
    st = dict(case, dt=dt)
    if op in ("norm", "qact"):
        st["X"] = _activations(g, case["T"], case["K"], dt)
    if op == "norm":
        st["gamma"] = (1.0 + 0.1 * torch.randn((case["K"],), generator=g, device="cuda")).to(dt)
        if case["residual"]:
            st["R"] = (2.0 * torch.randn((case["T"], case["K"]), generator=g, device="cuda")).to(dt)
    if op == "qweight":
        st["W"] = (0.02 * torch.randn((case["E"], case["N"], case["K"]), generator=g,
                                      device="cuda")).to(dt)
    if op in ("matmul", "grouped"):
        T, K, N, E = case["T"], case["K"], case["N"], case.get("E", 1)
        M = T * case.get("top", 1)
        A = T if case.get("gather", True) else M
        st["Xq"], st["SX"] = _quantize_rows(_activations(g, A, K, dt).float())
        W = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        S = []
        for e in range(E):
            w = (0.02 * torch.randn((N, K), generator=g, device="cuda")).to(dt)
            W[e], s = _quantize_blocks(w.float())
            S.append(s)
        st["CB"], st["SB"] = W.view(torch.uint8), torch.stack(S)
        shape = (E, N) if op == "grouped" else (N,)
        st["bias"] = torch.randn(shape, generator=g, device="cuda").to(dt) if case["bias"] else None
        if op == "grouped":
            st["offsets"] = _offsets(g, M, E)
            # how many rows the fullest expert has: the plain form's padding
            st["most"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())
            st["row_idx"] = (torch.randint(0, T, (M,), generator=g, device="cuda").to(torch.int32)
                             if case["gather"] else None)
        else:
            st["CB"], st["SB"] = st["CB"][0], st["SB"][0]
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _exponent(a):
    """e: the largest integer with a * 2^e <= 448, at most 126; 0 for a = 0 (a in fp32)."""
    m, ex = torch.frexp(a)                      # a = m * 2^ex, m in [0.5, 1)
    e = torch.where(m <= 0.875, 9 - ex, 8 - ex).clamp(max=126)
    return torch.where(a > 0, e, torch.zeros_like(e))


def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _pad_scales(s):
    """[..., blocks] E8M0 bytes -> rows padded to a multiple of 4 with 127."""
    return torch.nn.functional.pad(s, (0, -s.shape[-1] % 4), value=127).to(torch.uint8)


def _quantize_rows(y):
    """fp32 [T,K] -> E4M3 codes (uint8) [T,K] and the scales of its 1 x 128 blocks."""
    T, K = y.shape
    p = torch.nn.functional.pad(y, (0, -K % BLOCK)).view(T, -1, BLOCK)
    e = _exponent(p.abs().amax(-1))
    q = (p * _pow2(e)[..., None]).to(torch.float8_e4m3fn).view(T, -1)[:, :K]
    return q.view(torch.uint8).contiguous(), _pad_scales(127 - e)


def _quantize_blocks(w):
    """fp32 [..., N,K] -> E4M3 codes [..., N,K] and the scales of its 128 x 128 blocks."""
    N, K = w.shape[-2:]
    p = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK))
    p = p.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))      # [..., nb, 128, kb, 128]
    e = _exponent(p.abs().amax((-3, -1)))
    q = (p * _pow2(e)[..., :, None, :, None]).to(torch.float8_e4m3fn)
    q = q.flatten(-2).flatten(-3, -2)[..., :N, :K].contiguous()
    return q, _pad_scales(127 - e)


def _values_rows(q, s):
    """Codes [T,K] with row scales -> fp32 values."""
    K = q.shape[-1]
    sc = _pow2(s.to(torch.int32) - 127).repeat_interleave(BLOCK, -1)[..., :K]
    return q.view(torch.float8_e4m3fn).float() * sc


def _values_blocks(q, s):
    """Codes [..., N,K] with block scales -> fp32 values."""
    return _values_rows(q, s.repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :])


def _plain(st):
    op = st["op"]
    if op == "norm":
        h = st["X"].float()
        if st["residual"]:
            h = (h + st["R"].float()).to(st["dt"]).float()
        y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * st["gamma"].float()
        q, s = _quantize_rows(y)
        return (q, s, h.to(st["dt"]) if st["residual"] else None, y.to(st["dt"]) if st["y"] else None)
    if op == "qact":
        return _quantize_rows(st["X"].float())
    if op == "qweight":
        q, s = _quantize_blocks(st["W"].float())
        return q.view(torch.uint8), s
    x, w = _values_rows(st["Xq"], st["SX"]), _values_blocks(st["CB"], st["SB"])
    if op == "matmul":
        v = x @ w.t()
        if st["bias"] is not None:
            v = v + st["bias"].float()
    else:
        # every expert's rows, padded to the fullest expert's, in one batched product
        off = st["offsets"].long()
        M = st["T"] * st["top"]
        at = off[:-1, None] + torch.arange(st["most"], device="cuda")[None]
        used = at < off[1:, None]
        src = at.clamp(max=M - 1)
        src = st["row_idx"].long()[src] if st["gather"] else src
        p = torch.bmm(x[src], w.transpose(1, 2))
        if st["bias"] is not None:
            p = p + st["bias"].float()[:, None]
        v = torch.empty((M, st["N"]), device="cuda")
        v[at[used]] = p[used]
    return (torch.relu(v) if st["relu"] else v).to(st["dt"])


def _codes(q, s):
    """The 8-bit outputs as the values that their bits hold: E4M3 codes and powers of two."""
    return q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)


def run(st):
    op = st["op"]
    if own:
        import int8_quantized_matmul_02_amd as L
        if op == "norm":
            y = torch.empty_like(st["X"]) if st["y"] else None
            q, s, h = L.llmint8_rmsnorm_b128(st["X"], st["gamma"], 1e-6, residual=st.get("R"), Y=y)
            return (*_codes(q, s), h, y)
        if op == "qact":
            return _codes(*L.llmint8_quantize_act_b128(st["X"]))
        if op == "qweight":
            return _codes(*L.llmint8_quantize_weight_b128(st["W"]))
        act = L.ACT_RELU if st["relu"] else L.ACT_NONE
        if op == "matmul":
            return L.llmint8_matmul_b128(st["Xq"], st["SX"], st["CB"], st["SB"], bias=st["bias"],
                                         activation=act, out_dtype=st["dt"])
        return L.llmint8_matmul_grouped_b128(st["Xq"], st["SX"], st["CB"], st["SB"], st["offsets"],
                                             row_idx=st["row_idx"], bias=st["bias"],
                                             activation=act, out_dtype=st["dt"])
    r = _plain(st)
    return r if op in ("matmul", "grouped") else (*_codes(r[0], r[1]), *r[2:])


# ---------------------------------------------------------------------------
# what a pass has to move and compute
# ---------------------------------------------------------------------------
def work(case):
    op, K = case["op"], case["K"]
    kb = -(-K // BLOCK)
    if op == "norm":
        n = case["T"] * K
        return {"bytes": n * (2 + 1 + (4 if case["residual"] else 0) + (2 if case["y"] else 0))
                + case["T"] * kb + 2 * K, "flops": 8 * n}
    if op == "qact":
        return {"bytes": case["T"] * (3 * K + kb), "flops": 3 * case["T"] * K}
    if op == "qweight":
        return {"bytes": case["E"] * (3 * case["N"] * K + -(-case["N"] // BLOCK) * kb),
                "flops": 3 * case["E"] * case["N"] * K}
    T, N = case["T"], case["N"]
    M = T * case.get("top", 1)
    A = T if case.get("gather", True) else M
    # experts that an even router would leave without rows are not read
    E = case.get("E", 1)
    used = E * (1 - (1 - 1 / E) ** M) if E > 1 else 1
    return {"bytes": A * (K + kb) + used * (N * K + -(-N // BLOCK) * kb) + 2 * M * N,
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# the operators in 64 bits
# ---------------------------------------------------------------------------
def _f64(codes, s, rows_per_scale):
    """float64 values of codes under their scales, block by block."""
    N, K = codes.shape
    v = codes.view(torch.float8_e4m3fn).to(torch.float64)
    for kb in range(-(-K // BLOCK)):
        col = torch.exp2(s[:, kb].to(torch.float64) - 127)
        col = col.repeat_interleave(rows_per_scale)[:N]
        v[:, kb * BLOCK:(kb + 1) * BLOCK] *= col[:, None]
    return v


def _scaled64(v, rows):
    """v (float64) times the power of two of its blocks of `rows` x 128, unrounded."""
    v = v.clone()
    N, K = v.shape
    for kb in range(-(-K // BLOCK)):
        c = v[:, kb * BLOCK:(kb + 1) * BLOCK]
        a = c.abs().amax(1)
        a = torch.nn.functional.pad(a, (0, -N % rows)).view(-1, rows).amax(1)
        e = torch.floor(torch.log2(torch.where(a > 0, 448.0 / a, 1.0)))
        e = torch.where(a * torch.exp2(e + 1) <= 448.0, e + 1, e)      # log2 next to a whole number
        e = torch.where(a * torch.exp2(e) > 448.0, e - 1, e)
        e = torch.where(a > 0, e.clamp(max=126), 0.0)
        c *= torch.exp2(e).repeat_interleave(rows)[:N, None]
    return v


def exact(case, seed):
    """What run() returns in 64 bits.  Codes are given unrounded (the scaled
    values); a scale is a choice, not a computed number, and has no such value."""
    st, op = prepare(case, seed), case["op"]
    if op == "norm":
        h = st["X"].double()
        if st["residual"]:
            h = (h + st["R"].double()).to(st["dt"]).double()
        y = h / torch.sqrt(h.square().sum(-1, keepdim=True) / case["K"] + 1e-6) * st["gamma"].double()
        return (_scaled64(y, 1), None, h if st["residual"] else None, y if st["y"] else None)
    if op == "qact":
        return (_scaled64(st["X"].double(), 1), None)
    if op == "qweight":
        return (torch.stack([_scaled64(w.double(), BLOCK) for w in st["W"]]), None)
    x = _f64(st["Xq"], st["SX"], 1)
    if op == "matmul":
        v = torch.matmul(x, _f64(st["CB"], st["SB"], BLOCK).t().contiguous())
        if st["bias"] is not None:
            v += st["bias"].double()
    else:
        bounds = st["offsets"].tolist()
        v = torch.zeros((case["T"] * case["top"], case["N"]), dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
            if a < b:
                rows = x[st["row_idx"][a:b].long()] if case["gather"] else x[a:b]
                v[a:b] = rows @ _f64(st["CB"][e], st["SB"][e], BLOCK).t().contiguous()
                if st["bias"] is not None:
                    v[a:b] += st["bias"][e].double()
    return v.clamp(min=0) if case["relu"] else v
