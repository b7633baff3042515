"""moe_route_tokens_scored refuses tensors that its kernels would read or write past
(no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")
import bit_vq_routed_gb300 as bv  # noqa: E402

T, H, E, k = 3, 256, 16, 2
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _z(*s, dtype=F32):
    return torch.zeros(*s, dtype=dtype)


def _call(**kw):
    a = dict(x=_z(T, H, dtype=BF), w_router=_z(E, H, dtype=BF), router_bias=_z(E), k=k, logits=_z(T, E), ids=_z(T, k, dtype=I32),
             weights=_z(T, k), expert_offsets=_z(E + 1, dtype=I32), sorted_pair=_z(T * k, dtype=I32),
             pair_to_sorted=_z(T * k, dtype=I32), bias=_z(E))
    assert set(kw) <= set(a)
    bv.moe_route_tokens_scored(**dict(a, **kw))


@pytest.mark.parametrize("name,value", [
    ("x", _z(T, H)), ("w_router", _z(E, H)), ("w_router", _z(E, H - 8, dtype=BF)), ("router_bias", _z(E - 1)),
    ("router_bias", _z(E, dtype=BF)), ("logits", _z(T, E - 1)), ("logits", _z(T - 1, E)), ("logits", _z(T, E, dtype=BF)),
    ("ids", _z(T, k - 1, dtype=I32)), ("ids", _z(T, k, dtype=torch.int64)), ("weights", _z(T, k + 1)), ("weights", _z(T, k, dtype=BF)),
    ("expert_offsets", _z(E, dtype=I32)), ("expert_offsets", _z(E + 1, dtype=torch.int64)), ("sorted_pair", _z(T * k - 1, dtype=I32)),
    ("pair_to_sorted", _z(T * k - 1, dtype=I32)), ("pair_to_sorted", _z(T * k)), ("bias", _z(E + 1)), ("bias", _z(E, dtype=BF))])
def test_refuses(name, value):
    n = bv.moe_launch_count()
    with pytest.raises(ValueError, match=name):
        _call(**{name: value})
    assert bv.moe_launch_count() == n


def test_of_these_only_the_device_is_wrong():
    for kw in ({}, dict(expert_offsets=_z(2 * E + 1, dtype=I32)), dict(bias=None), dict(router_bias=None)):
        with pytest.raises(ValueError, match="CUDA"):
            _call(**kw)
