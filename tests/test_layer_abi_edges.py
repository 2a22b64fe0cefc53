"""Refusals of the layer entry points at the ends of what they take, on the CPU."""
from test_layer_abi import P, norm


def test_out_and_sum_out_are_two_matrices():
    # either may be x or residual; both in one place would leave one of the results
    Q = P + (1 << 16)
    for kw in (dict(x=P, res=Q, out=P, sum=P), dict(x=P, res=Q, out=Q, sum=Q),
               dict(x=P, res=Q, out=P + 4096, sum=P + 4096)):
        assert norm(ldr=64, lds=64, **kw) == -3, kw
    assert norm(x=P, res=Q, ldr=64, out=P, sum=P, lds=64, rows=0) == 0
