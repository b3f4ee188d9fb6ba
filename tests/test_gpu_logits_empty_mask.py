"""A mask without rows, whose address is NULL: the call is refused, and not taken for one without a mask."""
import pytest

import medusa_head_speculative_heads_gb300 as mg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    mg.build()


def words(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("mask", [lambda: words(0, 2), lambda: words(3, 2)[:0]])
def test_masks_without_a_row(mask):
    z = torch.zeros((2, 3, 40), device="cuda")
    for row in (0, -1):
        with pytest.raises(ValueError, match="mask"):
            mg.medusa_logits_process(z, mask=mask(), mask_row=words(2, 3).fill_(row))
    with pytest.raises(ValueError, match="mask"):
        mg.medusa_logits_process(z, mask=mask())
