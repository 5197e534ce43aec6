"""sketch_unpack looks at what it is given before the library sees its pointers. CPU only."""
import pytest
import torch


@pytest.mark.parametrize("packed,msg", [
    (dict(codes=torch.zeros(3, 4, 64, dtype=torch.uint8), scales=torch.ones(3, 4), format=0), "bytes a code"),
    (dict(codes=torch.zeros(3, 4, 64, dtype=torch.bfloat16), scales=torch.ones(3, 4), format=1), "bytes a code"),
    (dict(codes=torch.zeros(3, 4, 64, dtype=torch.uint8), scales=None, format=1), "scales is required"),
    (dict(codes=torch.zeros(3, 4, 64, dtype=torch.uint8), scales=torch.ones(3, 3), format=1), "scales has shape"),
    (dict(codes=torch.zeros(3, 4, 64, dtype=torch.uint8), scales=torch.ones(3, 4).double(), format=1), "scales has dtype"),
    (dict(codes=torch.zeros(3, 4, 64, dtype=torch.uint8), scales=torch.ones(3, 4, device="meta"), format=1), "scales is on"),
    (dict(codes=torch.zeros(3, 4, 128, dtype=torch.bfloat16)[:, :, ::2], format=0), "contiguous"),
    (dict(codes=torch.zeros(64, dtype=torch.bfloat16), format=0), "codes must be"),
    (dict(codes=None, format=0), "codes must be"),
    (dict(codes=torch.zeros(3, 4, 64, dtype=torch.bfloat16), format=7), "unknown format"),
    (dict(codes=torch.zeros(3, 4, 64, dtype=torch.bfloat16), scales=None, format=0), "CUDA devices only"),
])
def test_refuses(packed, msg):
    from prototype_sketch_attention_b200 import build
    build.build()
    from prototype_sketch_attention_b200 import binding as b
    with pytest.raises(b.SketchAttentionError, match=msg):
        b.sketch_unpack(packed)
