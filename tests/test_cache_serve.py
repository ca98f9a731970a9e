"""The verification round over a paged cache (profile_cases serve): its paths, and the
whole round on the device for every cache type."""
import pytest
import torch

from conditional_draft_tree_gb300 import profile_cases


def test_deepest_paths():
    parents = torch.tensor([[-1, 0, 1, 0, 3, 4], [-1, 0, 0, -1, -1, -1], [-1] * 6], dtype=torch.int32)
    depths = torch.tensor([[0, 1, 2, 1, 2, 3], [0, 1, 1, -1, -1, -1], [0] + [-1] * 5], dtype=torch.int32)
    path, lengths = profile_cases.deepest_paths(parents, depths, 4)
    assert lengths.tolist() == [4, 2, 1]
    assert path.tolist() == [[0, 3, 4, 5], [0, 1, -1, -1], [0, -1, -1, -1]]


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
def test_serve_round(cache, capsys):
    out, paged, length = profile_cases.case_serve(0, 1, torch.device("cuda", 0), cache, H=8, Hkv=2, dh=64,
                                                  page=16, most=70, least=33)
    paged.check()
    assert bool(torch.isfinite(out).all()) and bool((out.float().abs().amax((1, 3))[:, 0] > 0).all())
    assert bool((length > 33).all())
    assert "layer_us" in capsys.readouterr().out
