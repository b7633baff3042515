"""DecoderLayer's calls and what it tells the routing about them (no GPU)."""
import torch

import bit_vq_routed_gb300 as bv


class Attention:
    H = 8

    def forward(self, x, batch, residual=None, out=None, stream=None):
        return x + residual


class Experts:
    H = 8

    def forward(self, x, out=None, stream=None, fresh=False):
        self.x, self.fresh = x, fresh
        return 2 * x


def test_routing_is_told_that_its_tokens_were_written_just_before():
    # the output projection is the launch ahead of the routing, and one-kernel routings
    # read their tokens before the wait for it unless they are told
    moe = Experts()
    x = torch.ones(3, 8)
    h, y = bv.DecoderLayer(Attention(), moe).forward(x, None, x)
    assert moe.fresh is True
    assert torch.equal(moe.x, h) and torch.equal(h, 2 * x) and torch.equal(y, 4 * x)
