"""The expert products between dispatch and combine: what is timed, on which shapes, and what the
results are.

Three operators over expert-major rows (rank d holds its rows at [d][0..B), expert d*L + l owning
rows expert_off[d][l] .. expert_off[d][l+1]):

  gemm   y = x . w[e]^T, bf16 operands, or e4m3 ones with an fp32 scale for each row and 128 values
         of x and for each 128 x 128 block of w
  gated  h = silu(x . w_gate[e]^T) * (x . w_up[e]^T), on its own for bf16 operands
  mlp    gated, then gemm with the down projection: one expert's whole MLP; with e4m3 operands h is
         quantised again between the two, one scale for each row and 128 values

`own` false: elementary torch operations in fp32.  `own` true: the library's calls.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    DEVICE = "cuda"
else:
    DEVICE = "cpu"

E4M3 = torch.float8_e4m3fn


def _case(name, op, fp8, N, T, E, R, K, C, skew):
    return {"name": name, "op": op, "fp8": fp8, "N": N, "T": T, "E": E, "R": R, "K": K, "C": C,
            "skew": skew}


def listed():
    """N ranks, T tokens a rank, E experts, R of them per token; K the width of the rows that come
    in, C of those that go out (the intermediate size for gated and mlp); skew: how the tokens
    choose ("even": alike; "zipf": popularity falls as 1 / rank of the expert)."""
    return [
        # one token being decoded: eight experts of one row each, bound by their weights
        _case("gemm bf16 one token", "gemm", False, 1, 1, 128, 8, 4096, 2048, "even"),
        # a small model's layer with odd sizes, two ranks, and experts that no token chose
        _case("gemm bf16 odd", "gemm", False, 2, 37, 10, 3, 1000, 1288, "zipf"),
        # a prefill batch over four ranks, 256 rows an expert
        _case("gemm bf16 prefill", "gemm", False, 4, 1024, 128, 8, 4096, 4096, "even"),
        # one rank's experts in a decode step of many ranks: 128 rows an expert
        _case("gemm fp8 decode", "gemm", True, 1, 512, 8, 2, 7168, 4096, "even"),
        # a shared expert: every token through one matrix, an odd number of them
        _case("gemm fp8 shared", "gemm", True, 1, 1001, 1, 1, 7168, 2048, "even"),
        # a long prompt through few experts, 2048 rows each: bound by arithmetic
        _case("gemm fp8 long", "gemm", True, 1, 8192, 8, 2, 4096, 8192, "even"),
        # a small decode batch on eight ranks of one expert each
        _case("gated bf16 decode", "gated", False, 8, 4, 8, 2, 4096, 2048, "even"),
        # a prompt through narrow experts
        _case("gated bf16 prompt", "gated", False, 1, 4096, 16, 2, 2048, 1408, "zipf"),
        # one token through its experts' whole MLPs
        _case("mlp fp8 one token", "mlp", True, 1, 1, 64, 8, 7168, 2048, "even"),
        # a decode batch whose tokens crowd onto some experts
        _case("mlp fp8 decode", "mlp", True, 1, 256, 64, 8, 7168, 2048, "zipf"),
        # a small decode batch over four ranks
        _case("mlp bf16 decode", "mlp", False, 4, 32, 32, 4, 4096, 1024, "zipf"),
        # a whole layer: 4096 tokens over all 256 experts
        _case("mlp fp8 layer", "mlp", True, 1, 4096, 256, 8, 7168, 2048, "even"),
    ]


def _cost(c):
    matrices = {"gemm": 1, "gated": 2, "mlp": 3}[c["op"]]
    rows = c["N"] * c["T"] * c["R"]
    weights = matrices * c["E"] * c["K"] * c["C"] * (1 if c["fp8"] else 2)
    # the plain form pads every expert's rows to the longest's: skewed choices cost it more
    return weights, 2 * matrices * rows * c["K"] * c["C"], c["E"] * rows * c["K"]


def draw(rng):
    """One more case of the same ranges: each size spread over its logarithm."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["gemm", "gated", "mlp"])
        fp8 = op != "gated" and rng.random() < 0.5
        L, N = log(1, 64), rng.choice([1, 1, 2, 4, 8])
        E = L * N
        R = rng.randint(1, min(E, 8))
        T = log(1, 8192)
        if fp8:
            K = 512 * rng.randint(1, 14)
            C = 8 * log(8, 1024) if op == "gemm" else 128 * rng.randint(1, 16)
        else:
            K, C = 8 * log(16, 896), 8 * log(8, 512)
        c = _case("", op, fp8, N, T, E, R, K, C, rng.choice(["even", "zipf"]))
        del c["name"]
        weights, flops, padded = _cost(c)
        if weights <= 4 << 30 and flops <= 1 << 40 and padded <= 2 << 30:
            return c


def _shape(c):
    """(rows a rank's arrays hold, experts of a rank, rows of the weight matrix that x meets)."""
    L = c["E"] // c["N"]
    return c["N"] * c["T"] * min(c["R"], L), L, c["C"] if c["op"] == "gemm" else 2 * c["C"]


def _quantise(v):
    """(e4m3 codes, fp32 scales) of fp32 values, a scale for each 128 of the last dimension."""
    b = v.unflatten(-1, (-1, 128))
    amax = b.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    return (b / scale.unsqueeze(-1)).clamp(-448, 448).to(E4M3).flatten(-2), scale


def _weights(g, E, C, K, fp8):
    """E matrices of C x K, made one by one; e4m3 ones have a scale for each 128 x 128 block."""
    if not fp8:
        w = torch.empty((E, C, K), dtype=torch.bfloat16, device=DEVICE)
        for e in range(E):
            w[e] = torch.randn((C, K), generator=g, device=DEVICE) * K ** -0.5
        return w, None
    Cb, Kb = -(-C // 128), K // 128
    w = torch.empty((E, C, K), dtype=torch.uint8, device=DEVICE)
    s = torch.empty((E, Cb, Kb), dtype=torch.float32, device=DEVICE)
    for e in range(E):
        v = torch.randn((Cb, 128, Kb, 128), generator=g, device=DEVICE) * K ** -0.5
        # blocks of different magnitude, as trained matrices have
        v *= torch.rand((Cb, 1, Kb, 1), generator=g, device=DEVICE) + 0.5
        s[e] = v.abs().amax((1, 3)) / 448
        w[e] = (v / s[e][:, None, :, None]).to(E4M3).view(torch.uint8).view(Cb * 128, K)[:C]
    return w, s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    N, E, R, K, C, fp8 = c["N"], c["E"], c["R"], c["K"], c["C"], c["fp8"]
    B, L, C1 = _shape(c)
    # which experts the tokens choose, and the expert-major rows that this gives each rank
    score = torch.randn((N * c["T"], E), generator=g, device=DEVICE)
    if c["skew"] == "zipf":
        score -= torch.log(1.0 + torch.randperm(E, generator=g, device=DEVICE))
    cnt = torch.bincount(score.topk(R, dim=1).indices.flatten(), minlength=E).view(N, L)
    off = torch.zeros((N, L + 1), dtype=torch.int32, device=DEVICE)
    off[:, 1:] = cnt.cumsum(1)
    st = {"case": c, "off": off}
    # where each row lies, for the plain form: its place in the arrays, its expert, its place there
    flat = cnt.flatten()
    expert = torch.repeat_interleave(torch.arange(E, device=DEVICE), flat)
    within = torch.arange(expert.numel(), device=DEVICE) - (flat.cumsum(0) - flat)[expert]
    st["rows"] = (expert // L) * B + off[:, :-1].flatten()[expert].long() + within
    st["used"], st["slot"] = torch.unique(expert, return_inverse=True)
    st["within"], st["most"] = within, int(flat.max())
    x = torch.zeros((N * B, K), dtype=torch.float32 if fp8 else torch.bfloat16, device=DEVICE)
    x[st["rows"]] = torch.randn((expert.numel(), K), generator=g, device=DEVICE).to(x.dtype)
    if fp8:
        codes, scale = _quantise(x)
        st["x"], st["x_scale"] = codes.view(torch.uint8).view(N, B, K), scale.view(N, B, K // 128)
    else:
        st["x"], st["x_scale"] = x.view(N, B, K), None
    st["w1"], st["w1_scale"] = _weights(g, E, C1, K, fp8)
    st["w2"], st["w2_scale"] = _weights(g, E, K, C, fp8) if c["op"] == "mlp" else (None, None)
    # what the calls write: zero where no row lies, and left so
    if c["op"] != "gemm":
        st["h"] = torch.zeros((N, B, C), dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEVICE)
        st["h_scale"] = torch.zeros((N, B, C // 128), dtype=torch.float32, device=DEVICE) if fp8 else None
    if c["op"] != "gated":
        st["y"] = torch.zeros((N, B, C if c["op"] == "gemm" else K), dtype=torch.bfloat16, device=DEVICE)
    return st


def _rows32(v, scale, st):
    """The rows that experts own, in fp32."""
    v = v.flatten(0, 1)[st["rows"]]
    if scale is None:
        return v.float()
    s = scale.flatten(0, 1)[st["rows"]]
    return (v.view(E4M3).float().unflatten(-1, (-1, 128)) * s.unsqueeze(-1)).flatten(-2)


def _product(x, w, scale, st):
    """Each row times its expert's matrix: rows padded to the longest expert's, one batched product."""
    w = w[st["used"]]
    if scale is None:
        w = w.float()
    else:
        s = scale[st["used"]].repeat_interleave(128, 1)[:, : w.shape[1]]
        w = (w.view(E4M3).float().unflatten(-1, (-1, 128)) * s.unsqueeze(-1)).flatten(-2)
    padded = torch.zeros((w.shape[0], st["most"], x.shape[1]), dtype=torch.float32, device=x.device)
    padded[st["slot"], st["within"]] = x
    return torch.bmm(padded, w.transpose(1, 2))[st["slot"], st["within"]]


def _plain(st):
    c = st["case"]
    v = _product(_rows32(st["x"], st["x_scale"], st), st["w1"], st["w1_scale"], st)
    if c["op"] == "gemm":
        st["y"].flatten(0, 1)[st["rows"]] = v.bfloat16()
        return
    gate, up = v[:, : c["C"]], v[:, c["C"] :]
    v = gate / (1 + torch.exp(-gate)) * up
    if c["fp8"]:
        codes, scale = _quantise(v)
        st["h"].flatten(0, 1)[st["rows"]] = codes.view(torch.uint8)
        st["h_scale"].flatten(0, 1)[st["rows"]] = scale
    else:
        st["h"].flatten(0, 1)[st["rows"]] = v.bfloat16()
    if c["op"] == "mlp":
        v = _product(_rows32(st["h"], st["h_scale"], st), st["w2"], st["w2_scale"], st)
        st["y"].flatten(0, 1)[st["rows"]] = v.bfloat16()


def _library(st):
    import combine_moe_route_top_amd as moe

    c = st["case"]
    # H is the width of the dispatched rows; a lone product takes its own widths
    H = c["K"] if c["op"] != "gemm" else 512
    shape = moe.make_shape(c["N"], c["T"], H, c["E"], c["R"], c["fp8"], st["x"].shape[1])
    if c["op"] == "gemm":
        moe.moe_expert_gemm(shape, c["K"], c["C"], st["x"], st["x_scale"], st["w1"], st["w1_scale"],
                            st["off"], st["y"])
    elif c["op"] == "gated":
        moe.moe_expert_gated(shape, c["K"], c["C"], st["x"], st["x_scale"], st["w1"], st["w1_scale"],
                             st["off"], st["h"], st["h_scale"])
    else:
        moe.moe_expert_mlp(shape, c["C"], st["x"], st["x_scale"], st["w1"], st["w1_scale"], st["w2"],
                           st["w2_scale"], st["off"], st["h"], st["h_scale"], st["y"])


def run(st):
    if own:
        _library(st)
    else:
        _plain(st)
    return {"h": st["h"]} if st["case"]["op"] == "gated" else {"y": st["y"]}


def work(case):
    """Each chosen expert's matrices once, each row in and out once; the number of chosen experts is
    its expectation (for zipf, as if the slots were drawn one by one)."""
    c = case
    E, rows, K, C = c["E"], c["N"] * c["T"] * c["R"], c["K"], c["C"]
    if c["skew"] == "even":
        used = E * (1 - (1 - c["R"] / E) ** (c["N"] * c["T"]))
    else:
        total = sum(1 / (e + 1) for e in range(E))
        used = sum(1 - (1 - 1 / (e + 1) / total) ** rows for e in range(E))
    matrices = {"gemm": 1, "gated": 2, "mlp": 3}[c["op"]]
    if c["fp8"]:
        weights, inp, mid = K * C * (1 + 4 / 128 / 128), K * (1 + 4 / 128), C * (1 + 4 / 128)
    else:
        weights, inp, mid = 2 * K * C, 2 * K, 2 * C
    out = {"gemm": 2 * C, "gated": mid, "mlp": 2 * K}[c["op"]]
    return {"bytes": used * matrices * weights + rows * (inp + out), "flops": 2.0 * matrices * rows * K * C}


def _e4m3_nearest(v):
    """The e4m3 value nearest to each double, ties to even: steps of 2^(exponent - 3), no finer than
    2^-9, and at most 448."""
    _, exponent = torch.frexp(v)  # v = m * 2^exponent with m in [0.5, 1)
    step = torch.ldexp(torch.ones_like(v), (exponent - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    N, E, K, C, fp8 = c["N"], c["E"], c["K"], c["C"], c["fp8"]
    L = E // N
    off = st["off"].tolist()
    out = torch.zeros_like(st["h"] if c["op"] == "gated" else st["y"], dtype=torch.float64)

    def matrix(w, scale, e):
        if scale is None:
            return w[e].double()
        m = w[e].view(E4M3).double()
        for i in range(scale.shape[1]):
            m[128 * i : 128 * (i + 1)] *= scale[e, i].double().repeat_interleave(128)
        return m

    for e in range(E):
        d, lo, hi = e // L, off[e // L][e % L], off[e // L][e % L + 1]
        if lo == hi:
            continue
        x = st["x"][d, lo:hi]
        x = x.view(E4M3).double() * st["x_scale"][d, lo:hi].double().repeat_interleave(128, 1) if fp8 else x.double()
        v = x @ matrix(st["w1"], st["w1_scale"], e).T
        if c["op"] != "gemm":
            v = v[:, :C] * torch.sigmoid(v[:, :C]) * v[:, C:]
        if c["op"] == "mlp":
            if fp8:
                amax = v.view(hi - lo, -1, 128).abs().amax(2)
                scale = torch.where(amax > 0, amax / 448.0, 1.0).float().double().repeat_interleave(128, 1)
                v = _e4m3_nearest(v / scale) * scale
            else:
                v = v.bfloat16().double()
            v = v @ matrix(st["w2"], st["w2_scale"], e).T
        out[d, lo:hi] = v
    return {"h" if c["op"] == "gated" else "y": out}
