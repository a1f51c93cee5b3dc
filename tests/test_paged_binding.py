"""The paged cache's binding: argument checks that need no GPU."""
import pytest

import hybrid_softmax_gated_b200 as arl2


def test_the_device_must_be_a_gpu():
    with pytest.raises(ValueError, match="device"):
        arl2.PagedCache(2, 2, 128, 4, 16, device="cpu")
