"""CPU checks of the paged attention's scale: what the kernels would compute
with is checked, before anything is launched."""
import pytest

from tests.test_paged_cpu import attn_args, pe  # noqa: F401


# not representable as a normal fp32 number: it would round to 0 or lose bits,
# and a masked score of -inf times 0 is NaN
@pytest.mark.parametrize("scale", [1e-50, 1e-45, 1e-39, 1.1754942e-38, 3e38, 1e39])
@pytest.mark.parametrize("dtype", [0, 1])
def test_attention_refuses_a_scale_outside_fp32(pe, scale, dtype):  # noqa: F811
    before = pe.peagle_kernel_launches()
    with pytest.raises(pe.PeagleError) as e:
        pe.peagle_paged_attention(*attn_args(pe, dtype=dtype, scale=scale), stream=0)
    assert e.value.status == pe.PEAGLE_ERR_INVALID_ARG
    assert "scale" in pe.peagle_last_error()
    assert pe.peagle_kernel_launches() == before
