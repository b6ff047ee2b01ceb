"""The input of the adapters' product and gradient is required wherever a kernel
reads it, also where there is no adapter to multiply it with (the rows are loaded
before their adapter is known).  Host-side refusals; no GPU."""
import pytest

from test_boundary_lora import FAKE, NULL, OK, P, _lora, _msg, lib  # noqa: F401


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("rows,n", [(1, 1), (8, 3), (1000, 3)])
def test_input_without_adapters(lib, grad, rows, n):  # noqa: F811
    no = dict(ad=0, a=None, b=None, scale=None, x=None, rows=rows, n=n, wsb=1 << 30, c_in=4096, c_out=4096)
    assert _lora(lib, grad, **no) == NULL and "input" in _msg(lib)
    assert _lora(lib, grad, **dict(no, s=P(FAKE), base=None)) == NULL
    assert _lora(lib, grad, **dict(no, rows=0)) == OK and _lora(lib, grad, **dict(no, n=0)) == OK
