"""The torch layers as modules, on the GPU: inputs off a 16-byte boundary, submodules that a user
changed, gradients of gradients, and the block's gradient along its own direction."""
import numpy as np
import pytest
import torch

from group_circulant_linear_p4_amd.layer import EQLayerNorm, EQLinear, EQLinearP4M, EQMLPBlock
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16 = torch.float16
