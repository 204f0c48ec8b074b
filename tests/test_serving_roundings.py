"""What the roundings inside the decode over 8-bit caches do to results, emulated on the host: the GPU
tests of small weights and small query components tell a kernel that lifts its fp16 operands from one that
does not.  No GPU."""
import pytest
import torch

import serving_plain as sp


def _with_fp16_weights(below, lift):
    """The case of twelve peaks and 1011 keys of weight 2^-below, even column: weights times 2^lift in fp16."""
    p = torch.cat([torch.ones(12, dtype=torch.float64), torch.full((1011,), 2.0 ** -below, dtype=torch.float64)])
    v = torch.cat([torch.zeros(12, dtype=torch.float64), torch.full((1011,), 64.0, dtype=torch.float64)])
    held = (p * 2.0 ** lift).half().double() * 2.0 ** -lift
    return (held * v).sum() / p.sum(), (p * v).sum() / p.sum()


@pytest.mark.parametrize("below", [20.5, 25.5, 26.0, 31.0])
def test_lifted_weights_stay_within_the_bound_and_unlifted_ones_do_not(below):
    zero = torch.zeros(1)
    got, o = _with_fp16_weights(below, 7)
    assert float((got - o).abs()) <= float(sp.bound(o.reshape(1, 1), zero, 1024, True))
    if below > 25:
        got, o = _with_fp16_weights(below, 0)
        assert float((got - o).abs()) > 10 * float(sp.bound(o.reshape(1, 1), zero, 1024, True))


def test_lifted_query_components_keep_the_logits_and_unlifted_ones_do_not():
    # the largest component 1 brought to 2^14, the small ones 2^-30 of it
    g = torch.Generator().manual_seed(0)
    q = (torch.randn((1, 128), generator=g) * 2.0 ** -30).bfloat16().double()
    q[:, 0] = 1.0
    k, v = (torch.randn((1, 300, 128), generator=g).double() for _ in range(2))
    k[..., 0], k[..., 1:] = 0.0, k[..., 1:] * 2.0 ** 30
    seen = torch.ones((1, 300), dtype=torch.bool)
    o, A, e = sp.attention64(q, k[0], v[0], seen)
    for lift, good in ((14, True), (0, False)):
        held = (q * 2.0 ** lift).half().double() * 2.0 ** -lift
        got, _, _ = sp.attention64(held, k[0], v[0], seen)
        assert bool(((got - o).abs() <= sp.bound(A, e, 300, True)).all()) == good
