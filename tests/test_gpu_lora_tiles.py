"""The adapters' product where tiles of 256 x 256 fill more than three quarters of their rounds over 256
compute units, and where they do not and 128 x 128 are taken."""
import pytest
import torch

from test_gpu_layer_rules import lora_case

pytestmark = pytest.mark.gpu


# (columns of 512 rows: 256, 258, 384, 388 and 514 tiles)
@pytest.mark.parametrize("each", [False, True])
@pytest.mark.parametrize("N", [32768, 32769, 49152, 49409, 65537])
def test_rounds_of_the_largest_tiles(N, each):
    lora_case(512, N, 72, 24, 5, torch.bfloat16, torch.float32, N, each)
    lora_case(512, N, 72, 24, 5, torch.float16, torch.float16, N, each)
