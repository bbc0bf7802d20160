"""The exploration driver's checks, without a GPU."""

import numpy as np
import pytest
import torch

from experiment_network_simulation_amd import dse, inputs as I


@pytest.mark.parametrize("place", [np.zeros(7, int), np.zeros(9, int), np.zeros((8, 1), int), [], 3])
def test_every_expert_has_a_place(place):
    """An expert without a place would send its tokens nowhere, without a word."""
    good = dse.RouteDesign(top_k=2, place=np.zeros(8, int))
    never = lambda probes: pytest.fail("scored")
    for designs in ([dse.RouteDesign(top_k=2, place=place)], [good, dse.RouteDesign(top_k=2, place=place)]):
        with pytest.raises(ValueError, match="place"):
            dse.route_designs(torch.zeros(4, 8), [0, 4], [0], designs, I.fat_tree(4), never)
