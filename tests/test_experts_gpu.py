"""The experts' products on the GPU against the plain fp64 implementation of expert_ref, with its
derived bounds: ragged row counts around the tiles' edges, odd widths, both operand types, rank
ranges, rows that must stay as they were, non-finite rows, streams, graphs, far offsets, and the
whole layer from the router to the combined output."""
import numpy as np
import pytest
import torch

import expert_ref as ref
import moe_synth as ms

pytestmark = pytest.mark.gpu

POISON = 0xA5


class Setup:
    """Operands on the GPU for given row counts [N][L], and their host copies."""

    def __init__(self, counts, K, C, fp8, op, seed=0, capacity=0, rank_begin=0, rank_count=0, starts=None):
        import combine_moe_route_top_amd as moe
        self.moe, self.K, self.C, self.fp8, self.op = moe, K, C, fp8, op
        self.counts = counts
        N, L = len(counts), len(counts[0])
        E = N * L
        total = max(1, max(sum(c) for c in counts))
        B = max(capacity, N * total + 32)  # room for poisoned rows behind the last
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        H = K if op == "mlp" else 512
        self.shape = moe.make_shape(N, total, H, E, 1, fp8, B, status=self.status, rank_begin=rank_begin,
                                    rank_count=rank_count)
        off = torch.zeros((N, L + 1), dtype=torch.int32)
        off[:, 1:] = torch.tensor(counts, dtype=torch.int32).cumsum(1)
        if starts is not None:  # rows need not begin at 0
            off += torch.tensor(starts, dtype=torch.int32).view(N, 1)
        self.off_host, self.off = off, off.cuda()
        g = torch.Generator().manual_seed(seed)
        self.x_host, self.xs_host = [], []
        n_max = int(off.max()) + 8  # a few rows past the last, poisoned
        dt = torch.uint8 if fp8 else torch.int16
        self.a = torch.empty((N, B, K), dtype=dt, device="cuda")
        self.a_scale = torch.empty((N, B, K // 128), device="cuda") if fp8 else None
        for d in range(N):
            x, xs = ref.make_rows(g, (int(off[d, -1]), K), fp8)
            self.x_host.append(x)
            self.xs_host.append(xs)
            self.a[d, :n_max].view(torch.uint8).fill_(0xFF)       # NaN in either type behind the rows
            self.a[d, : x.shape[0]] = x.cuda()
            if fp8:
                self.a_scale[d, :n_max].fill_(float("nan"))
                self.a_scale[d, : x.shape[0]] = xs.cuda()
        rows1 = C if op == "gemm" else 2 * C
        self.w1h, self.w1sh = ref.make_weights(g, E, rows1, K, fp8)
        self.w1 = self.w1h.cuda()
        self.w1s = self.w1sh.cuda() if fp8 else None
        if op == "mlp":
            self.w2h, self.w2sh = ref.make_weights(g, E, K, C, fp8)
            self.w2 = self.w2h.cuda()
            self.w2s = self.w2sh.cuda() if fp8 else None
        self.n_max = n_max
        if op != "gemm":
            self.h = torch.empty((N, B, C), dtype=dt, device="cuda")
            self.hs = torch.empty((N, B, C // 128), device="cuda") if fp8 else None
        if op != "gated":
            self.y = torch.empty((N, B, C if op == "gemm" else K), dtype=torch.int16, device="cuda")
        self.poison()

    def outputs(self):
        o = []
        if self.op != "gemm":
            o += [self.h] + ([self.hs] if self.fp8 else [])
        if self.op != "gated":
            o.append(self.y)
        return o

    def poison(self):
        for t in self.outputs():
            t[:, : self.n_max].view(torch.uint8).fill_(POISON)

    def run(self, stream=None):
        m = self.moe
        if self.op == "gemm":
            m.moe_expert_gemm(self.shape, self.K, self.C, self.a, self.a_scale, self.w1, self.w1s, self.off,
                              self.y, stream)
        elif self.op == "gated":
            m.moe_expert_gated(self.shape, self.K, self.C, self.a, self.a_scale, self.w1, self.w1s, self.off,
                               self.h, self.hs, stream)
        else:
            m.moe_expert_mlp(self.shape, self.C, self.a, self.a_scale, self.w1, self.w1s, self.w2, self.w2s,
                             self.off, self.h, self.hs, self.y, stream)

    def check(self, ranks=None, skip=(), status=0):
        """Every owned row of the ranks against fp64, every other row still poisoned."""
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        N, L = len(self.counts), len(self.counts[0])
        got = [t[:, : self.n_max].cpu() for t in self.outputs()]
        owned = torch.zeros((N, self.n_max), dtype=torch.bool)
        for d in range(N) if ranks is None else ranks:
            for l in range(L):
                lo, hi = int(self.off_host[d, l]), int(self.off_host[d, l + 1])
                if hi <= lo or (d, l) in skip:
                    continue
                owned[d, lo:hi] = True
                e, name = d * L + l, f"{self.op} fp8={self.fp8} K={self.K} C={self.C} rank {d} expert {l} rows {hi - lo}"
                X = ref.decode(self.x_host[d][lo:hi], self.xs_host[d][lo:hi] if self.fp8 else None, self.fp8)
                W = ref.decode_weight(self.w1h[e], self.w1sh[e] if self.fp8 else None, self.fp8)
                if self.op == "gemm":
                    ref.check_bf16(name, got[0][d, lo:hi], *ref.product(X, W, self.fp8))
                    continue
                h, bound = ref.gated(X, W, self.fp8)
                mine = got[0][d, lo:hi]
                if self.fp8:
                    ref.check_e4m3(name, mine, got[1][d, lo:hi], h, bound)
                else:
                    ref.check_bf16(name, mine, h, bound)
                if self.op == "mlp":  # from the kernel's own h: each product is held to its own bound
                    X = ref.decode(mine, got[1][d, lo:hi] if self.fp8 else None, self.fp8)
                    W = ref.decode_weight(self.w2h[e], self.w2sh[e] if self.fp8 else None, self.fp8)
                    ref.check_bf16(name + " down", got[-1][d, lo:hi], *ref.product(X, W, self.fp8))
        for t in got:
            rest = t.contiguous().view(torch.uint8).view(N, self.n_max, -1)[~owned]
            assert bool((rest == POISON).all()), "a row that no expert owns was written"


def spread(total, L, seed):
    """Counts of L experts adding up to `total`, some of them zero."""
    r = np.random.default_rng(seed)
    p = r.dirichlet(np.full(L, 0.5))
    return r.multinomial(total, p).tolist()


EDGES = [0, 1, 2, 7, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 191, 192, 193, 255, 256, 257, 300]


@pytest.mark.parametrize("op", ["gemm", "gated", "mlp"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_row_counts_around_the_tiles(op, fp8):
    print(f"\ncase edges {op} {fp8}", flush=True)
    s = Setup([EDGES], 512, 256, fp8, op)
    s.run()
    s.check()


@pytest.mark.parametrize("n", [1, 2, 5, 16, 24, 40, 70, 130, 260, 700])
@pytest.mark.parametrize("op", ["gemm", "gated"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_one_expert_of_n_rows(op, fp8, n):
    print(f"\ncase one expert {op} {fp8} {n}", flush=True)
    s = Setup([[n]], 640, 384, fp8, op, seed=n)
    s.run()
    s.check()


@pytest.mark.parametrize("K,C", [(8, 8), (56, 24), (64, 136), (72, 264), (136, 120), (200, 8), (520, 520), (1000, 1288),
                                 (2056, 40)])
@pytest.mark.parametrize("op", ["gemm", "gated"])
@pytest.mark.parametrize("rows", [3, 40, 150, 330])
def test_odd_widths_bf16(op, K, C, rows):
    print(f"\ncase widths bf16 {op} {K} {C} {rows}", flush=True)
    s = Setup([[rows, 0, rows // 2]], K, C, False, op, seed=K + C)
    s.run()
    s.check()


@pytest.mark.parametrize("K,C", [(128, 8), (128, 128), (256, 136), (384, 1032), (640, 248), (1152, 520), (2176, 128)])
@pytest.mark.parametrize("rows", [3, 40, 150, 330])
def test_odd_widths_e4m3(K, C, rows):
    print(f"\ncase widths e4m3 {K} {C} {rows}", flush=True)
    s = Setup([[rows, 0, rows // 2]], K, C, True, "gemm", seed=K + C)
    s.run()
    s.check()
    if C % 128 == 0:
        s = Setup([[rows, 0, rows // 2]], K, C, True, "gated", seed=K + C + 1)
        s.run()
        s.check()


@pytest.mark.parametrize("op,K,C", [("mlp", 512, 384), ("mlp", 1024, 128), ("gemm", 512, 640)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("seed", [0, 1])
def test_ranks_and_ranges(op, K, C, fp8, seed):
    """Several ranks with empty experts and an empty rank; then the same in calls of rank ranges."""
    print(f"\ncase ranks {op} {fp8} {seed}", flush=True)
    counts = [spread(90, 6, seed), [0] * 6, spread(333, 6, seed + 10), spread(5, 6, seed + 20)]
    s = Setup(counts, K, C, fp8, op, seed=seed)
    s.run()
    s.check()
    for b, n in [(0, 1), (1, 1), (2, 2)]:
        s.poison()
        s.shape = s.moe.for_ranks(s.shape, b, n)
        s.run()
        s.check(ranks=range(b, b + n))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_no_rows_at_all(fp8):
    s = Setup([[0, 0], [0, 0]], 512, 128, fp8, "mlp")
    s.run()
    s.check()


@pytest.mark.parametrize("E", [256, 1024])
def test_many_experts(E):
    print(f"\ncase experts {E}", flush=True)
    s = Setup([spread(700, E // 4, i) for i in range(4)], 512, 128, True, "mlp")
    s.run()
    s.check()


@pytest.mark.parametrize("counts", [[[2000, 0, 0, 1]], [[1, 1, 900, 1]], [[17] * 40], [[130] * 12]])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("op", ["gemm", "gated"])
def test_skewed_counts(counts, fp8, op):
    print(f"\ncase skew {counts[0][:4]} {fp8} {op}", flush=True)
    s = Setup(counts, 384, 640, fp8, op)
    s.run()
    s.check()


def test_rows_that_begin_later():
    """Offsets of a rank need not begin at row 0."""
    s = Setup([[5, 40], [70, 0]], 512, 128, True, "mlp", starts=[3, 11])
    s.run()
    s.check()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_bad_offsets_flag_and_own_no_rows(fp8):
    """The kernel checks every entry: an expert with a bad one is left out and flagged, the others
    keep their results."""
    import combine_moe_route_top_amd as moe
    s = Setup([[20, 30, 9, 9]], 256, 128, fp8, "gemm")
    off = s.off_host.clone()
    off[0, 2] = -5                       # expert 1 would end before it begins, expert 2 begin before row 0
    s.off.copy_(off.cuda())
    s.off_host = off
    s.run()
    s.check(skip={(0, 2)}, status=moe.MOE_EINVAL)
    s.status.zero_()
    s.poison()
    off[0] = torch.tensor([-4, 2, 20, 50, 1 << 30], dtype=torch.int32)
    s.off.copy_(off.cuda())
    s.run()
    s.check(skip={(0, 0), (0, 3)}, status=moe.MOE_EINVAL)


@pytest.mark.parametrize("rows", [3, 40, 300])
@pytest.mark.parametrize("op", ["gemm", "gated"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_non_finite_values_stay_in_their_row(fp8, op, rows):
    """A NaN (or infinity) in a row makes that row's outputs NaN or infinite and no other's."""
    s = Setup([[rows, rows]], 256, 256, fp8, op)
    s.run()
    torch.cuda.synchronize()
    clean = [t.clone() for t in s.outputs()]
    bad = [1, rows - 1, rows]            # rows of the rank; the last is the second expert's first
    if fp8:
        s.a[0, bad[0], 7] = 0x7F
        s.a_scale[0, bad[1], 1] = float("inf")
        s.a_scale[0, bad[2], 0] = float("nan")
    else:
        s.a[0, bad[0], 7] = 0x7FC0
        s.a[0, bad[1], 130] = 0x7F80
        s.a[0, bad[2], 255] = -0x80      # -infinity
    s.poison()
    s.run()
    torch.cuda.synchronize()
    keep = torch.ones(s.n_max, dtype=torch.bool)
    keep[bad] = False
    for now, was in zip(s.outputs(), clean):
        assert torch.equal(now[0, : s.n_max].cpu()[keep], was[0, : s.n_max].cpu()[keep])
    out = s.outputs()[0][0, : s.n_max].cpu()
    for r in bad:
        if op == "gated" and fp8:
            v = ref.decode(out[r : r + 1], s.hs[0, r : r + 1].cpu(), True)
        else:
            v = out[r].view(torch.bfloat16).double()
        if r == bad[0]:
            assert torch.isnan(v).all()
        else:
            assert not torch.isfinite(v).any() if op == "gemm" else not torch.isfinite(v).all()


def test_the_same_call_gives_the_same_bits():
    for fp8 in (False, True):
        s = Setup([spread(600, 9, 4)], 1024, 640, fp8, "mlp")
        s.run()
        torch.cuda.synchronize()
        first = [t[:, : s.n_max].clone() for t in s.outputs()]
        for _ in range(3):
            s.poison()
            s.run()
            torch.cuda.synchronize()
            for now, was in zip(s.outputs(), first):
                assert torch.equal(now[:, : s.n_max].view(torch.uint8), was.view(torch.uint8))


def test_two_streams_at_once():
    """Two independent calls in flight on two streams (nothing in the library is shared)."""
    a = Setup([spread(500, 8, 1)], 1024, 512, True, "mlp", seed=1)
    b = Setup([spread(300, 8, 2)], 1024, 512, False, "mlp", seed=2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        a.run()
        b.run(side)
    a.check()
    b.check()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_graph_replays_follow_the_counts(fp8):
    """Captured once, replayed with other rows and other counts in the same buffers; every replay is
    checked, with eager calls and synchronisations between them."""
    counts = [spread(200, 8, 3)]
    s = Setup(counts, 512, 256, fp8, "mlp", seed=3, capacity=400)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for i in range(4):
        other = Setup([spread(200 if i % 2 else 150, 8, 30 + i)], 512, 256, fp8, "mlp", seed=40 + i, capacity=400)
        n = other.n_max
        s.a[:, :n].copy_(other.a[:, :n])
        if fp8:
            s.a_scale[:, :n].copy_(other.a_scale[:, :n])
        s.off.copy_(other.off)
        s.off_host, s.counts, s.x_host, s.xs_host = other.off_host, other.counts, other.x_host, other.xs_host
        s.poison()
        graph.replay()
        s.check()
        s.poison()
        s.run()
        s.check()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_offsets_past_32_bits(fp8):
    """Rank 1's rows lie more than 2^32 bytes into every row array."""
    capacity = (5 << 30) // (1024 if fp8 else 2048)
    s = Setup([[2, 3], [40, 70]], 1024, 1024, fp8, "mlp", capacity=capacity)
    assert s.a[1].data_ptr() - s.a.data_ptr() > 1 << 32
    s.run()
    s.check()


def test_weights_past_32_bits():
    """The last expert's matrices lie more than 2^32 bytes into the weights."""
    import combine_moe_route_top_amd as moe
    E, K, C, n = 160, 4096, 4096, 20
    g = torch.Generator().manual_seed(0)
    w = torch.empty((E, C, K), dtype=torch.int16, device="cuda")
    last, _ = ref.make_weights(g, 1, C, K, False)
    w[E - 1] = last[0].cuda()
    x, _ = ref.make_rows(g, (n, K), False)
    off = torch.zeros((1, E + 1), dtype=torch.int32, device="cuda")
    off[0, E] = n
    y = torch.empty((1, n, C), dtype=torch.int16, device="cuda")
    moe.moe_expert_gemm(moe.make_shape(1, n, K, E, 1, capacity=n), K, C, x.cuda(), None, w, None, off, y)
    torch.cuda.synchronize()
    W = last[0].view(torch.bfloat16).double()
    ref.check_bf16("far weights", y[0].cpu(), *ref.product(x.view(torch.bfloat16).double(), W, False))


def test_scales_at_any_4_byte_address():
    """Scale arrays need only their own alignment: the same bits from arrays shifted by one float."""
    s = Setup([[5, 70, 200]], 512, 256, True, "mlp", seed=8)
    s.run()
    torch.cuda.synchronize()
    want = [t[:, : s.n_max].clone() for t in s.outputs()]

    def shifted(t):
        flat = torch.empty(t.numel() + 1, device="cuda")
        flat[1:] = t.flatten()
        return flat[1:].view(t.shape)

    s.a_scale, s.w1s, s.w2s, s.hs = (shifted(t) for t in (s.a_scale, s.w1s, s.w2s, s.hs))
    s.poison()
    s.run()
    s.check()
    for now, was in zip(s.outputs(), want):
        assert torch.equal(now[:, : s.n_max].contiguous().view(torch.uint8), was.view(torch.uint8))


@pytest.mark.parametrize("rows", [3, 150])
@pytest.mark.parametrize("e,scale,code", [(-8, 1.0, 0.0), (-7, 2.0 ** -149, 256.0)])
def test_gated_rows_next_to_zero(rows, e, scale, code):
    """Gated e4m3 rows of which one half is zero and the other about the least fp32 values: 128 products
    of ones, scaled, make gate and up 2^(-63 + e), so h is 2^(-127 + 2e), all exact.  For e = -8 its
    448th, 2^-143 / 448, rounds to zero; for e = -7 it is 0.57 of the least fp32 value and rounds to it."""
    s = Setup([[rows]], 128, 128, True, "gated")
    s.a[:, :rows] = s.w1[:] = 0x38  # 1.0
    s.w1[:, 128 + 64:] = 0          # up rows of the last 64 columns
    s.a_scale[:, :rows] = 2.0 ** -70
    s.w1s[:] = 2.0 ** e
    s.run()
    torch.cuda.synchronize()
    assert bool((s.hs[0, :rows] == scale).all())
    got = s.h[0, :rows].contiguous().view(torch.float8_e4m3fn).float()
    assert bool((got[:, :64] == code).all()) and bool((got[:, 64:] == 0).all())


def test_shared_expert_is_one_group():
    """N = E = R = 1: the plain product of every token with one matrix."""
    for fp8, n in ((False, 77), (True, 333)):
        s = Setup([[n]], 512, 1024, fp8, "mlp", seed=n)
        s.run()
        s.check()


@pytest.mark.parametrize("layout", ["decode", "prefill"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "quant"])
def test_whole_layer(layout, kind):
    """Router, dispatch, experts, combine: expert_y against fp64 on the dispatched rows, the layer's
    output against the fp64 weighted sum of expert_y at each token's rows."""
    import combine_moe_route_top_amd as moe
    import parity
    if layout == "prefill" and kind == "quant":
        return  # the prefill layout takes no quantising dispatch
    print(f"\ncase layer {layout} {kind}", flush=True)
    N, T, H, E, R, I = 4, 40, 512, 16, 4, 256
    fp8 = kind != "bf16"
    if layout == "prefill":
        inp = parity.prefill_inputs(T, H, E, R, fp8, "none", 5)
        b = moe.alloc_prefill_buffers(N, T, H, E, R, fp8)
    else:
        inp = ms.make_inputs(N, T, H, E, R, kind == "e4m3", "zipf", 5)
        b = moe.alloc_buffers(N, T, H, E, R, fp8, quant=kind == "quant")
    parity.upload_inputs(b, inp)
    x = moe.alloc_experts(b, I)
    g = torch.Generator().manual_seed(9)
    w1, w1s = ref.make_weights(g, E, 2 * I, H, fp8)
    w2, w2s = ref.make_weights(g, E, H, I, fp8)
    x.w1.copy_(w1), x.w2.copy_(w2)
    if fp8:
        x.w1_scale.copy_(w1s), x.w2_scale.copy_(w2s)
    use_bias = inp["bias"] is not None
    if layout == "prefill":
        moe.run_prefill_dispatch(b, use_bias)
        moe.run_experts(b, x)
        moe.moe_prefill_combine(b.shape, b.expert_y, b.topk_idx, b.slot_pos, b.topk_w, b.partial, b.out)
    else:
        moe.run_dispatch(b, use_bias)
        moe.run_experts(b, x)
        moe.run_combine(b)
    torch.cuda.synchronize()
    assert int(b.status.item()) == 0
    sets = 1 if layout == "prefill" else N
    off, src = b.expert_off.cpu(), b.expert_src.cpu()
    sums = torch.zeros((sets * T, H), dtype=torch.float64)
    size = torch.zeros_like(sums)
    w = b.topk_w.cpu().double().flatten()
    seen = 0
    for d in range(N):
        for l in range(E // N):
            lo, hi, e = int(off[d, l]), int(off[d, l + 1]), d * (E // N) + l
            X = ref.decode(b.expert_x[d, lo:hi].cpu(), b.expert_scale[d, lo:hi].cpu() if fp8 else None, fp8)
            W1 = ref.decode_weight(w1[e], w1s[e] if fp8 else None, fp8)
            W2 = ref.decode_weight(w2[e], w2s[e] if fp8 else None, fp8)
            h, bound = ref.gated(X, W1, fp8)
            mine, hs = x.h[d, lo:hi].cpu(), x.h_scale[d, lo:hi].cpu() if fp8 else None
            ref.check_e4m3("h", mine, hs, h, bound) if fp8 else ref.check_bf16("h", mine, h, bound)
            y = b.expert_y[d, lo:hi].cpu()
            ref.check_bf16("y", y, *ref.product(ref.decode(mine, hs, fp8), W2, fp8))
            rows = src[d, lo:hi].long()
            v = y.view(torch.bfloat16).double() * w[rows].unsqueeze(1)
            sums.index_add_(0, rows // R, v)
            size.index_add_(0, rows // R, v.abs())
            seen += hi - lo
    assert seen == sets * T * R
    # R fused adds in fp32, then one rounding to bf16
    ref.check_bf16("out", b.out.cpu().view(sets * T, H), sums, 2 * R * ref.STEP * size)
    if layout == "decode":
        # one more rounding to bf16 for each owner rank's partial sum
        moe.run_combine_acc(b)
        torch.cuda.synchronize()
        assert int(b.status.item()) == 0
        ref.check_bf16("acc", b.out.cpu().view(sets * T, H), sums, (2 * R * ref.STEP + 2.0 ** -8) * size)
