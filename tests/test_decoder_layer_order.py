"""DecoderLayer's calls and what it tells the routing about them (no GPU)."""
import pytest
import torch

import bit_vq_routed_gb300 as bv


class Attention:
    H, dtype = 8, torch.bfloat16

    def __init__(self):
        self.calls = 0

    def forward(self, x, batch, residual=None, out=None, stream=None):
        self.calls += 1
        return x + residual


class Experts:
    H, T_max = 8, 4

    def forward(self, x, out=None, stream=None, fresh=False):
        self.x, self.fresh = x, fresh
        return 2 * x


def test_routing_is_told_that_its_tokens_were_written_just_before():
    # the output projection is the launch ahead of the routing, and one-kernel routings
    # read their tokens before the wait for it unless they are told
    moe = Experts()
    x = torch.ones(3, 8, dtype=torch.bfloat16)
    h, y = bv.DecoderLayer(Attention(), moe).forward(x, None, x)
    assert moe.fresh is True
    assert torch.equal(moe.x, h) and torch.equal(h, 2 * x) and torch.equal(y, 4 * x)


def test_refuses_what_the_experts_would_misread():
    # (fp16 bits read as bf16 would give results that are wrong and finite)
    attention = Attention()
    attention.dtype = torch.float16
    with pytest.raises(ValueError, match="bfloat16"):
        bv.DecoderLayer(attention, Experts())


def test_refuses_too_many_tokens_before_the_cache_is_written():
    attention = Attention()
    x = torch.ones(5, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="T_max"):
        bv.DecoderLayer(attention, Experts()).forward(x, None, x)
    assert attention.calls == 0


def test_norm_between_attention_and_experts():
    # pre-norm: the experts read norm(h), the residual stream stays h
    moe = Experts()
    x = torch.ones(3, 8, dtype=torch.bfloat16)
    h, y = bv.DecoderLayer(Attention(), moe, norm=lambda h: h * 4).forward(x, None, x)
    assert torch.equal(h, 2 * x) and torch.equal(moe.x, 8 * x) and torch.equal(y, 16 * x)
    attention = Attention()
    attention.dtype = torch.float16  # (a norm may bring the experts' type)
    bv.DecoderLayer(attention, moe, norm=lambda h: h.to(torch.bfloat16)).forward(x, None, x)
    for wrong in (lambda h: h.float(), lambda h: h[:, :4]):
        with pytest.raises(ValueError, match="norm"):
            bv.DecoderLayer(Attention(), moe, norm=wrong).forward(x, None, x)
