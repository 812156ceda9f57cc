"""Refusals of the routed block where it is made, on the CPU."""
import pytest
import torch

from gemm_reduce_fusion_gb300.block import RoutedMLPBlock


def test_only_bfloat16_weights():
    shapes = dict(router=(8, 4), w1=(4, 8, 16), w2=(4, 16, 8))
    good = {k: torch.zeros(s, dtype=torch.bfloat16) for k, s in shapes.items()}
    RoutedMLPBlock(**good, p=2, k=2)
    for name in shapes:
        with pytest.raises(TypeError, match=name):
            RoutedMLPBlock(**{**good, name: good[name].float()}, p=2, k=2)
