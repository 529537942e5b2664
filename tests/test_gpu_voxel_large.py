"""GPU gather of voxel features for more points than one launch has threads for."""

import pytest
import torch

import sparse_convolution_hash_amd as spc

pytestmark = pytest.mark.gpu


def test_gather_beyond_one_launch():
    # a thread takes 8 channels: 2^32 threads and some
    C, n, nv = 4096, (1 << 23) + 3, 1000
    print(f"gather n={n} C={C}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(9)
    seg = torch.randn((nv, C), generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(-1, nv, (n,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.full((n, C), 7.0, dtype=torch.bfloat16, device="cuda")
    assert spc.gather_by_voxel_id(seg, ids, out=out) is out
    table = torch.cat([seg, torch.zeros((1, C), dtype=seg.dtype, device="cuda")])     # id -1: zeros
    for a in range(0, n, 1 << 18):
        assert torch.equal(out[a:a + (1 << 18)], table[ids[a:a + (1 << 18)].long()]), f"points from {a}"
