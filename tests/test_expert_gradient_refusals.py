"""What the gradient of combine takes where it only clears, on the host."""
import pytest

from tests.test_expert_ops_host import INV, OK, REACHED, UNS, call, no_gpu

WIDE = dict(T=0, d=0, y=0, slots=0, w=0, dw=0, ds=1 << 20, ys=1 << 20, dys=1 << 20)


@no_gpu
@pytest.mark.parametrize("over,status", [
    (dict(WIDE, H=1 << 20), None), (dict(WIDE, H=(1 << 20) + 1, ds=1 << 21, ys=1 << 21, dys=1 << 21), UNS),
    (dict(WIDE, H=40000, used=0), OK), (dict(WIDE, H=40000, dy=0), INV), (dict(WIDE, H=40000, R=0), OK)])
def test_clearing_alone_takes_wide_rows(over, status):
    st = call("grad", **over)
    assert st in REACHED if status is None else st == status
