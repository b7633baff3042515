"""DecoderLayer refuses norms that its experts cannot read, and more tokens than a norm
holds, before the attention side writes the cache (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")
import bit_vq_routed_gb300 as bv  # noqa: E402

BF, F16 = torch.bfloat16, torch.float16


class Attention:
    H, T_max = 8, 6

    def __init__(self, dtype=BF):
        self.dtype, self.calls = dtype, 0

    def forward(self, x, batch, residual=None, out=None, stream=None):
        self.calls += 1
        return x


class Experts:
    H, T_max = 8, 6

    def forward(self, x, out=None, stream=None, fresh=False):
        return x.float()


def _norm(T_max=6, H=8, dtype=BF, eight=False):
    return bv.RMSNorm(torch.ones(H, dtype=dtype), 1e-6, T_max, eight)


@pytest.mark.parametrize("norm,dtype", [(dict(eight=True), BF), (dict(H=16), BF), (dict(dtype=F16), BF), (dict(dtype=F16), F16),
                                        (dict(), F16)])
def test_a_norm_that_the_experts_cannot_read(norm, dtype):
    with pytest.raises(ValueError, match="norm"):
        bv.DecoderLayer(Attention(dtype), Experts(), norm=_norm(**norm))


def test_more_tokens_than_a_norm_holds():
    x = torch.ones(5, 8, dtype=BF)
    attention = Attention()
    block = bv.DecoderLayer(attention, Experts(), norm=_norm(4), norm_in=_norm())
    for call in (lambda: block.forward(x, None, x), lambda: block.step(x, None, None), lambda: block.step(x, x.float(), None)):
        with pytest.raises(ValueError, match="norm's T_max=4"):
            call()
    block = bv.DecoderLayer(attention, Experts(), norm=_norm(), norm_in=_norm(4))
    for y in (None, x.float()):
        with pytest.raises(ValueError, match="norm_in's T_max=4"):
            block.step(x, y, None)
    attention.T_max = 4
    with pytest.raises(ValueError, match="attention side's T_max=4"):
        bv.DecoderLayer(attention, Experts(), norm=_norm(), norm_in=_norm()).step(x, None, None)
    assert attention.calls == 0
