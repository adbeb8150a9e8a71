"""The experts' products without a GPU: sizes and host-side refusals."""
import pytest
import torch

import combine_moe_route_top_amd as moe
import expert_ref as ref

GOOD = 1 << 20  # an aligned address that no call below gets as far as using


def shape(fp8=False, **kw):
    return moe.make_shape(2, 16, 512, 8, 2, fp8, **kw)


def gemm(sh, K=512, C=256, a=GOOD, a_scale=None, w=GOOD, w_scale=None, off=GOOD, y=GOOD):
    moe.moe_expert_gemm(sh, K, C, a, a_scale, w, w_scale, off, y, stream=0)


def gated(sh, K=512, I=256, a=GOOD, a_scale=None, w=GOOD, w_scale=None, off=GOOD, h=GOOD, h_scale=None):
    moe.moe_expert_gated(sh, K, I, a, a_scale, w, w_scale, off, h, h_scale, stream=0)


def mlp(sh, I=256, x=GOOD, xs=None, w1=GOOD, w1s=None, w2=GOOD, w2s=None, off=GOOD, h=GOOD, hs=None, y=GOOD):
    moe.moe_expert_mlp(sh, I, x, xs, w1, w1s, w2, w2s, off, h, hs, y, stream=0)


SCALED = dict(a_scale=GOOD, w_scale=GOOD)
MLP_SCALED = dict(xs=GOOD, w1s=GOOD, w2s=GOOD, hs=GOOD)


def refused(code, call, *args, **kw):
    with pytest.raises(moe.MoeError) as ex:
        call(*args, **kw)
    assert ex.value.code == code


@pytest.mark.parametrize("K,C,code", [
    (0, 256, moe.MOE_EINVAL), (512, 0, moe.MOE_EINVAL), (-8, 256, moe.MOE_EINVAL),
    (12, 256, moe.MOE_EUNSUPPORTED), (512, 12, moe.MOE_EUNSUPPORTED),
    ((1 << 20) + 8, 256, moe.MOE_EUNSUPPORTED), (512, (1 << 20) + 8, moe.MOE_EUNSUPPORTED)])
@pytest.mark.parametrize("call", [gemm, gated])
def test_widths_bf16(call, K, C, code):
    refused(code, call, shape(), K, C)


def test_widths_e4m3():
    refused(moe.MOE_EUNSUPPORTED, gemm, shape(True), 192, 256, **SCALED)    # K: whole blocks of 128
    refused(moe.MOE_EUNSUPPORTED, gemm, shape(True), 512, 12, **SCALED)
    refused(moe.MOE_EUNSUPPORTED, gated, shape(True), 512, 192, h_scale=GOOD, **SCALED)
    refused(moe.MOE_EUNSUPPORTED, mlp, shape(True), 64, **MLP_SCALED)
    refused(moe.MOE_EUNSUPPORTED, mlp, shape(), 12)
    refused(moe.MOE_EINVAL, mlp, shape(), 0)


@pytest.mark.parametrize("name", ["a", "w", "off", "y"])
@pytest.mark.parametrize("bad", [None, GOOD + 2])
def test_gemm_pointers(name, bad):
    refused(moe.MOE_EINVAL, gemm, shape(), **{name: bad})


@pytest.mark.parametrize("name", ["a", "w", "off", "h"])
@pytest.mark.parametrize("bad", [None, GOOD + 2])
def test_gated_pointers(name, bad):
    refused(moe.MOE_EINVAL, gated, shape(), **{name: bad})


@pytest.mark.parametrize("name", ["x", "w1", "w2", "off", "h", "y"])
@pytest.mark.parametrize("bad", [None, GOOD + 2])
def test_mlp_pointers(name, bad):
    refused(moe.MOE_EINVAL, mlp, shape(), **{name: bad})


def test_payloads_are_16_byte_aligned():
    for name in ("a", "w", "y"):
        refused(moe.MOE_EINVAL, gemm, shape(), **{name: GOOD + 8})


@pytest.mark.parametrize("name", ["a_scale", "w_scale"])
def test_scales_belong_to_e4m3(name):
    refused(moe.MOE_EINVAL, gemm, shape(), **{name: GOOD})                       # bf16 has none
    refused(moe.MOE_EINVAL, gemm, shape(True), **{**SCALED, name: None})         # e4m3 needs both
    refused(moe.MOE_EINVAL, gemm, shape(True), **{**SCALED, name: GOOD + 2})


def test_gated_and_mlp_scales():
    refused(moe.MOE_EINVAL, gated, shape(), h_scale=GOOD)
    refused(moe.MOE_EINVAL, gated, shape(True), **SCALED)
    for name in MLP_SCALED:
        refused(moe.MOE_EINVAL, mlp, shape(), **{name: GOOD})
        refused(moe.MOE_EINVAL, mlp, shape(True), **{**MLP_SCALED, name: None})
    quant = moe.make_shape(2, 16, 512, 8, 2, quant=True)  # its dispatched rows are e4m3 too
    refused(moe.MOE_EINVAL, gemm, quant)


def test_bad_shape_is_refused_first():
    bad = moe.make_shape(3, 16, 512, 8, 2)
    refused(moe.MOE_EINVAL, gemm, bad)
    refused(moe.MOE_EINVAL, gated, bad)
    refused(moe.MOE_EINVAL, mlp, bad)
    refused(moe.MOE_EINVAL, moe.moe_expert_sizes, bad, 256)


def test_host_tensors_and_views_are_refused():
    t = torch.zeros((8, 8), dtype=torch.int16)
    with pytest.raises(ValueError):
        gemm(shape(), a=t)


def test_sizes():
    sz = moe.moe_expert_sizes(moe.make_shape(32, 128, 7168, 256, 8, True), 2048)
    assert sz["w1"] == 256 * 4096 * 7168 and sz["w2"] == 256 * 7168 * 2048
    assert sz["w1_scale"] == 256 * 32 * 56 * 4 and sz["w2_scale"] == 256 * 56 * 16 * 4
    assert sz["h"] == 32 * 32768 * 2048 and sz["h_scale"] == 32 * 32768 * 16 * 4
    sz = moe.moe_expert_sizes(moe.make_shape(4, 64, 4096, 32, 4, prefill=True), 1408)
    assert sz["w1"] == 32 * 2816 * 4096 * 2 and sz["w2"] == 32 * 4096 * 1408 * 2
    assert sz["h"] == 4 * 64 * 8 * 1408 * 2  # T * max(R, E/N) rows a rank
    assert sz["w1_scale"] == sz["w2_scale"] == sz["h_scale"] == 0


def test_alloc_experts_on_the_host():
    for fp8 in (False, True):
        b = moe.alloc_buffers(2, 16, 512, 8, 2, fp8, device="cpu")
        x = moe.alloc_experts(b, 256)
        sz = moe.moe_expert_sizes(b.shape, 256)
        for k, n in sz.items():
            t = getattr(x, k)
            assert (0 if t is None else t.numel() * t.element_size()) == n, k


def test_the_reference_finds_a_mistake():
    """A misplaced scale, a swapped half and a lost block are over the bounds (the checks see what
    they are for)."""
    g = torch.Generator().manual_seed(3)
    w, s = ref.make_weights(g, 1, 256, 512, True)
    x, xs = ref.make_rows(g, (5, 512), True)
    X, W = ref.decode(x, xs, True), ref.decode_weight(w[0], s[0], True)
    want, bound = ref.product(X, W, True)
    ref.check_bf16("right", want.bfloat16(), want, bound)
    with pytest.raises(AssertionError):
        ref.check_bf16("scale", (X @ ref.decode_weight(w[0], s[0].roll(1, 1), True).T).bfloat16(), want, bound)
    lost = X.clone()
    lost[:, 128:256] = 0
    with pytest.raises(AssertionError):
        ref.check_bf16("block", (lost @ W.T).bfloat16(), want, bound)
    h, hb = ref.gated(X, W, True)
    codes, sc = ref.quantise(h)
    ref.check_e4m3("right", codes, sc, h, hb)
    swapped, _ = ref.gated(X, W.roll(128, 0), True)
    codes, sc = ref.quantise(swapped)
    with pytest.raises(AssertionError):
        ref.check_e4m3("halves", codes, sc, h, hb)
