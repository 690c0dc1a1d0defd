"""Argument handling of the expert-block operators' binding that needs no GPU."""
import pytest
import torch

from mixture_experts_feed_amd import binding as B

BF16 = torch.bfloat16
WRAPS = 2 ** 32 + 64      # 64 in the low 32 bits


@pytest.mark.parametrize("make", [
    lambda v: B.make_grouped_dims(1, 1, 4, v, 64, BF16),
    lambda v: B.make_grouped_dims(1, 1, 4, 64, v, BF16),
    lambda v: B.make_grouped_dims(1, 1, v, 64, 64, BF16),
    lambda v: B.make_swiglu_dims(1, v, BF16),
    lambda v: B.make_norm_dims(1, v, "rms", BF16, 1e-6),
    lambda v: B.make_dims(1, v, 4, 2, 0, 64, BF16),
    lambda v: B.make_dims(1, 64, 4, 2, 0, v, BF16),
    lambda v: B.make_dense_dims(1, v, 64, BF16),
    lambda v: B.make_dense_dims(1, 64, v, BF16),
    # the cached forms that the entry points call
    lambda v: B._grouped_plan(1, 1, 4, v, 64, BF16, BF16),
    lambda v: B._grouped_weight_grad_plan(1, 1, 4, 64, v, BF16, BF16),
    lambda v: B._swiglu_plan(1, v, BF16),
    lambda v: B._norm_plan(1, v, "layer", BF16, 1e-6),
])
@pytest.mark.parametrize("value", [WRAPS, 2 ** 31, -2 ** 32 + 64])
def test_a_width_past_32_bits_is_refused(make, value):
    """Its low 32 bits alone would be a size that the library takes, and a part of the row the result."""
    with pytest.raises(ValueError):
        make(value)


def test_the_library_refuses_what_32_bits_hold():
    with pytest.raises(B.InklingError) as e:
        B._norm_plan(1, 2 ** 31 - 1, "layer", BF16, 1e-6)
    assert e.value.code == B.INKLING_ERR_UNSUPPORTED


@pytest.mark.parametrize("shape", [(), (64,), (64, 64), (1, 2, 64, 64)])
def test_a_weight_of_other_dimensions_is_a_value_error(shape):
    rows, w, off = torch.zeros((3, 64), dtype=BF16), torch.zeros(shape, dtype=BF16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="n_groups, out_features, in_features"):
        B.grouped_linear(rows, w, off)
    with pytest.raises(ValueError, match="n_groups, out_features, in_features"):
        B.grouped_input_grad(rows, w, off)
