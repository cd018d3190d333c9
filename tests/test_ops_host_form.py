"""Refusals of the query for a product's kernel form."""
import pytest


@pytest.mark.parametrize("args,status", [
    ((0, 5, 64, 2), "ARG"), ((5, 0, 64, 2), "ARG"), ((5, 5, 0, 2), "ARG"), ((-1, 5, 64, 2), "ARG"), ((5, 5, 48, 2), "ALIGN"),
    ((5, 5, 64, 0), "DTYPE"), ((5, 5, 64, 3), "DTYPE"), ((2 ** 31, 5, 64, 2), "GEOMETRY"), ((5, 5, 2 ** 31, 2), "GEOMETRY"),
])
def test_refusals(hm, args, status):
    with pytest.raises(hm.HmError) as e:
        hm.mxfp8_gemm_form(*args)
    assert e.value.status == getattr(hm, "HM_ERR_" + status)
    assert hm.lib().mxfp8_gemm_form(5, 5, 64, 2, None, None, None) == hm.HM_ERR_ARG
