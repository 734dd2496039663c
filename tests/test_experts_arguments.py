"""Argument checks of the Python binding of 4-bit weights and expert layers (no GPU)."""
import pytest

torch = pytest.importorskip("torch")
tg = pytest.importorskip("tile_shape_autotuning_amd")

from tile_shape_autotuning_amd import experts    # noqa: E402

# what 32 bits would make of it is a legal value
LONG = 2 ** 32


@pytest.mark.parametrize("group", [LONG + 128, LONG + 32, 2 ** 31, -LONG + 128])
def test_a_group_beyond_32_bits_is_refused(group):
    with pytest.raises(ValueError, match="group"):
        tg.w4_quantize(torch.zeros((64, 16)), group)
    w = tg.W4(torch.zeros((1, 2, 64, 4), dtype=torch.int32), torch.zeros((1, 1, 16)), None, 256, 16, group)
    with pytest.raises(ValueError, match="group"):
        experts._w4(w, (), 256, 16, torch.device("cpu"), "B")


def test_a_group_of_any_length_below_that_is_taken():
    w = tg.W4(torch.zeros((1, 2, 64, 4), dtype=torch.int32), torch.zeros((1, 1, 16)), None, 256, 16, 2 ** 31 - 128)
    assert experts._w4(w, (), 256, 16, torch.device("cpu"), "B").group == 2 ** 31 - 128


@pytest.mark.parametrize("k", [LONG + 2, 2 ** 31, -LONG + 2])
def test_a_number_of_choices_beyond_32_bits_is_refused(k):
    with pytest.raises(ValueError, match="k ="):
        tg.moe_route(torch.zeros((1, 4)), k)
    with pytest.raises(ValueError, match="k ="):
        tg.moe_layer(torch.zeros((1, 64), dtype=torch.bfloat16), torch.zeros((1, 4)), None, None, k)


@pytest.mark.parametrize("w", [None, torch.zeros((64, 16)), torch.zeros(6), (1, 2, 3)])
def test_what_is_no_w4_is_said_to_be_none(w):
    with pytest.raises(TypeError, match="B must be a W4"):
        experts._w4(w, (), 64, None, torch.device("cpu"), "B")
