"""The smallest eps of AdamW: a normal fp32 number.  Host code only."""
import pytest


@pytest.fixture(scope="module")
def head():
    from dense_convolution_gb300 import build, head_capi
    build.build()
    return head_capi


def test_eps_is_a_normal_number(head):
    from dense_convolution_gb300 import capi
    d = head.adamw_desc_create([4])
    for eps in (2.0 ** -126, 1e-30, 1.0):
        head.adamw_desc_set_rates(d, 0.9, 0.95, eps)
    for eps in (2.0 ** -127, 2.0 ** -149, 1e-40):
        with pytest.raises(capi.Conv2dError) as e:
            head.adamw_desc_set_rates(d, 0.9, 0.95, eps)
        assert e.value.status == capi.ERR_BAD_PARAM
    head.adamw_desc_destroy(d)
