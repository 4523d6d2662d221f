"""The smoke check of the head runs, and says nothing but its result."""
import warnings

import pytest

pytestmark = pytest.mark.gpu


def test_smoke_of_the_head_without_warnings():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        __graft_entry__.smoke_head()
