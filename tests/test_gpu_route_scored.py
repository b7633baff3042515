"""moe_route_scored against 64 bits: the same experts always, the weights
within fp32."""
import pytest

torch = pytest.importorskip("torch")
import attn_common as ac  # noqa: E402
import rows_common as rc  # noqa: E402
from gpu_common import torch_cuda  # noqa: E402

pytestmark = pytest.mark.gpu

F32 = torch.float32


def _call(logits, k, sigmoid, bias=None, groups=1, top_groups=1, group_top=1, renorm=1, scale=1.0, stream=None):
    import bit_vq_routed_gb300 as bv
    T = logits.shape[0]
    ids = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    weights = torch.full((T, k), -5.0, device="cuda")
    bv.moe_route_scored(logits, k, ids, weights, scoring=int(sigmoid), bias=bias, groups=groups, top_groups=top_groups,
                        group_top=group_top, renormalize=renorm, scale=scale, stream=stream)
    return ids, weights


def _check(logits, k, sigmoid, bias=None, groups=1, top_groups=1, group_top=1, renorm=1, scale=1.0):
    ids, weights = _call(logits, k, sigmoid, bias, groups, top_groups, group_top, renorm, scale)
    want, w64 = rc.scored64(logits, k, sigmoid, bias, groups, top_groups, group_top, renorm, scale)
    assert torch.equal(ids.cpu(), want)
    # a softmax score: the exponent's difference rounds by 2^-24 of up to 104
    # (below, scores are under the smallest fp32), expf by 2 units, the sum of up
    # to 32 + 5 terms and two divisions and a product: below 160 units; and
    # scores below the normal range
    ac.within(weights.cpu(), w64, w64.abs() * 160 * 2.0 ** -23 + abs(scale) * 2.0 ** -120, "weights")


CASES = [(1, 1, 1, 1, 1), (2, 2, 1, 1, 1), (8, 2, 1, 1, 1), (8, 3, 4, 2, 2), (32, 32, 1, 1, 1), (32, 4, 32, 5, 1),
         (40, 7, 5, 3, 2), (60, 6, 3, 1, 2), (64, 32, 2, 1, 1), (72, 8, 9, 4, 2), (128, 8, 16, 4, 1), (160, 6, 8, 3, 1),
         (256, 8, 8, 4, 2), (256, 8, 8, 8, 2), (257, 5, 1, 1, 1), (384, 6, 12, 2, 2), (512, 10, 1, 1, 1), (1000, 31, 20, 7, 2),
         (1024, 32, 2, 2, 2), (1024, 16, 32, 8, 2), (1024, 1, 1, 1, 1), (97, 9, 1, 1, 1)]


@pytest.mark.parametrize("E,k,groups,top_groups,group_top", CASES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_choices(E, k, groups, top_groups, group_top, sigmoid, biased):
    torch_cuda()
    g = ac.gen(E + k)
    for T, std, renorm, scale in ((1, 1.5, 1, 1.0), (67, 1.5, 0, 2.5), (30, 6.0, 1, -0.5)):
        logits = ac.normal(g, T, E, dtype=F32, std=std)
        bias = ac.normal(g, E, dtype=F32, std=0.1) if biased else None
        _check(logits, k, sigmoid, bias, groups, top_groups, group_top, renorm, scale)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k,groups,top_groups,group_top", [(64, 8, 1, 1, 1), (256, 8, 8, 4, 2), (160, 6, 8, 3, 1),
                                                             (1024, 32, 16, 3, 2)])
def test_equal_values_go_to_the_lower_number(E, k, groups, top_groups, group_top, sigmoid):
    torch_cuda()
    g = ac.gen(E)
    for biased in (False, True):
        # few different values: equal choices in every row, equal groups in many
        logits = torch.randint(-2, 3, (50, E), generator=g, device="cuda").float() / 2
        bias = torch.randint(0, 2, (E,), generator=g, device="cuda").float() / 4 if biased else None
        logits[0] = 0.25
        logits[1, :] = -3.0
        _check(logits, k, sigmoid, bias, groups, top_groups, group_top)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k,groups,top_groups,group_top", [(64, 8, 1, 1, 1), (256, 8, 8, 4, 2), (240, 9, 12, 5, 1)])
def test_choices_that_fp32_cannot_tell_apart(E, k, groups, top_groups, group_top, sigmoid):
    """A bias that brings every choice of a row to 0.75 up to its own rounding:
    the choices differ by less than 2^-24, and in 64 bits by far more than that
    rounds."""
    torch_cuda()
    g = ac.gen(E + 1)
    for std in (0.5, 3.0):
        logits = ac.normal(g, 1, E, dtype=F32, std=std)
        score = torch.sigmoid(logits.double()) if sigmoid else torch.softmax(logits.double(), -1)
        bias = (0.75 - score[0]).float()
        _check(logits.repeat(3, 1), k, sigmoid, bias, groups, top_groups, group_top)


@pytest.mark.parametrize("E,k,groups,top_groups,group_top", [(256, 16, 1, 1, 1), (256, 8, 16, 5, 2), (384, 8, 32, 9, 2)])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -26, 2.0 ** -30, 2.0 ** -34])
def test_close_choices_over_the_sigmoids_range(E, k, groups, top_groups, group_top, scale):
    """Choices that meet at 0.75 from scores of all sizes, and differ by the bias'
    own rounding or by multiples of `scale`, which no fp32 bias can take away: a
    pair of experts with the same logit differs by the bias alone."""
    torch_cuda()
    g = ac.gen(E + k + int(scale > 0))
    for row in range(4):
        logits = 60 * torch.rand(1, E, generator=g, device="cuda") - 30
        logits[0, 1::2] = logits[0, ::2]  # (pairs)
        bias = (0.75 - torch.sigmoid(logits.double())[0]).float()
        if scale:
            step = torch.randint(-3, 4, (E,), generator=g, device="cuda").float() * scale
            bias = torch.where(bias.abs() < 2.0 ** -8, bias + step, bias)
        _check(logits, k, True, bias, groups, top_groups, group_top)


def test_logits_whose_scores_saturate():
    """Sigmoids of 20 to 90 are 1 in fp32 and most in 64 bits; without a bias the
    logits' order decides, with one the exact sums do."""
    torch_cuda()
    g = ac.gen(5)
    logits = 20 + 70 * torch.rand(20, 128, generator=g, device="cuda")
    _check(logits, 8, True)
    _check(-logits, 8, True, renorm=0)
    _check(logits, 8, False)
    _check(20 + 10 * torch.rand(20, 128, generator=g, device="cuda"), 8, True, bias=ac.normal(g, 128, dtype=F32, std=1e-9))


def test_infinities():
    torch_cuda()
    inf = float("inf")
    g = ac.gen(6)
    logits = ac.normal(g, 10, 64, dtype=F32)
    logits[:, 3] = -inf
    logits[4, :] = -inf
    logits[4, 10:20] = 1.0
    _check(logits, 4, False)
    _check(logits, 4, True, groups=4, top_groups=2, group_top=2)
    bias = ac.normal(g, 64, dtype=F32, std=0.1)
    bias[5:40] = -inf
    for sigmoid in (False, True):
        _check(logits, 8, sigmoid, bias)
    bias[5:40] = inf  # (35 equal choices)
    _check(logits, 8, True, bias)
    # sigmoids of -infinity: all scores 0, in their experts' order
    ids, w = _call(torch.full((2, 16), -inf, device="cuda"), 3, True)
    assert ids.tolist() == [[0, 1, 2]] * 2 and bool((w == 0).all())


@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (8, 4, 2), (8, 2, 1)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_nan_logits_give_distinct_experts(groups, top_groups, group_top, sigmoid, biased):
    torch_cuda()
    g = ac.gen(7)
    nan = float("nan")
    logits = ac.normal(g, 6, 64, dtype=F32)
    logits[0] = nan
    logits[1, ::2] = nan
    logits[2, 1:] = nan
    logits[3, 10] = nan
    logits[4, 5], logits[4, 6] = float("inf"), float("inf")
    bias = ac.normal(g, 64, dtype=F32) if biased else None
    ids, w = _call(logits, 8, sigmoid, bias, groups, top_groups, group_top)
    for row in ids.tolist():
        assert len(set(row)) == 8 and min(row) >= 0 and max(row) < 64
    assert bool(torch.isnan(w[0]).all()) and bool(torch.isfinite(w[5]).all())
    want = rc.scored64(logits[5:], 8, sigmoid, bias, groups, top_groups, group_top, 1, 1.0)
    assert torch.equal(ids[5:].cpu(), want[0])


def test_many_tokens_stream_and_graph():
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    g = ac.gen(8)
    logits, bias = ac.normal(g, 3001, 256, dtype=F32, std=1.5), ac.normal(g, 256, dtype=F32, std=0.05)
    _check(logits, 8, True, bias, 8, 4, 2, 1, 2.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = _call(logits, 8, True, bias, 8, 4, 2, stream=side)
    side.synchronize()
    ids, w = torch.zeros_like(a[0]), torch.zeros_like(a[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bv.moe_route_scored(logits, 8, ids, w, scoring=1, bias=bias, groups=8, top_groups=4, group_top=2)
    graph.replay()
    assert torch.equal(ids, a[0]) and torch.equal(w, a[1])


def test_it_is_the_softmax_top_k():
    """Without groups and bias: what moe_route_topk gives."""
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    g = ac.gen(9)
    for T, E, k in ((1, 8, 2), (40, 256, 8), (5, 1000, 32)):
        logits = ac.normal(g, T, E, dtype=F32, std=2.0)
        for renorm in (0, 1):
            ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
            bv.moe_route_topk(logits, k, renorm, ids, w)
            got = _call(logits, k, False, renorm=renorm)
            assert torch.equal(ids, got[0])
            assert float((w - got[1]).abs().max()) <= 64 * 2.0 ** -23


def test_no_tokens():
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    n = bv.moe_launch_count()
    _call(torch.zeros(0, 16, device="cuda"), 2, True)
    assert bv.moe_launch_count() == n
