"""What a dropout module does beside one plain call: where its seed comes from,
calls that are run again in the backward, capture, copies, and the longest rows.
On the CPU the kernel is replaced by the definition of its mask."""
import pytest
import torch

import unstructured_sparse_nn_amd as snk

gpu = pytest.mark.gpu


@pytest.mark.parametrize("make", [lambda: snk.Dropout(0.1).seed,
                                  lambda: snk.dropout.random_seed()])
def test_seeds_come_from_the_cpus_generator_whatever_the_default_device(make):
    torch.manual_seed(11)
    want = make()
    torch.manual_seed(11)
    with torch.device("meta"):
        assert make() == want
